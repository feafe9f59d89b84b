"""GPU: appends with the rotary embedding on the way (INT2 and BF16 caches)
against rotations in 64 bits; INT2 codes, scales, mins and channel 0 are
bit-exact, since the rotated key has one well-defined fp32 value."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import harness as H  # noqa: E402
import rows_ref as R  # noqa: E402
from bit_kv_cache_dqk_b200 import dualqk as Q  # noqa: E402
from oracle import oracle as O  # noqa: E402

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, cache, new, before, hq=8, hkv=2, d=128, rotary=None, inter=0, dtype="bf16", gs=32, v_ch0=0,
                 base=None, fused=True, with_q=True, seed=0, pool_pages=None, in_place=False, pad=0):
        self.__dict__.update(locals())
        self.rotary = rotary = rotary or d
        rng = np.random.default_rng([seed, 5])
        self.dev = torch.device("cuda:0")
        self.rows = n = sum(new)
        w = hq + 2 * hkv
        x = R.as_dtype(rng.standard_normal((n + 2, w + pad, d)), dtype)
        self.x = x.float().numpy()[:n, :w]
        xd = x.to(self.dev)
        parts = xd[:, :hq], xd[:, hq:hq + hkv], xd[:, hq + hkv:w]
        self.q, self.k, self.v = parts if fused else (p.contiguous() for p in parts)
        ends = [a + b for a, b in zip(new, before)]
        counts = [R.pages(e) for e in ends]
        total = max(1, sum(counts))
        self.num_pages = pool_pages or total
        perm = rng.permutation(total) + self.num_pages - total
        self.table = np.full((len(new), max(1, max(counts))), -1, np.int32)
        at = 0
        for i, c in enumerate(counts):
            self.table[i, :c] = perm[at:at + c]
            at += c
        self.t_k = np.eye(d, dtype=np.float32)[None] + 0.1 * rng.standard_normal((hkv, d, d)).astype(np.float32)
        tk = self.tk_dev = torch.from_numpy(self.t_k).to(self.dev)
        probe = Q.layer_desc(d, hq, hkv, 0, 0, 0, 1, v_ch0_protect=v_ch0, group_size=gs)
        self.bb = Q.dqk_block_bytes(probe) if cache == "int2" else Q.dqk_bf16_block_bytes(probe)
        self.pool = torch.full((self.num_pages * hkv * self.bb,), 0xA5, dtype=torch.uint8, device=self.dev)
        self.desc = Q.layer_desc(d, hq, hkv, tk, None, self.pool, self.num_pages, v_ch0_protect=v_ch0, group_size=gs)
        self.seq = np.repeat(np.arange(len(new)), new)
        self.slot = np.concatenate([np.arange(b, b + m) for m, b in zip(new, before)]).astype(np.int64)
        self.pos = self.slot + (0 if base is None else base)
        self.cs = R.rope_table(int(self.pos.max()) + 1 if n else 1, rotary)
        self.cs_dev = torch.from_numpy(self.cs).to(self.dev)
        self.q_out = self.q if in_place else torch.full((n + 2, hq, d), 7.0, dtype=self.q.dtype, device=self.dev)
        self.positions = None if base is None else torch.from_numpy(self.pos.astype(np.int32)).to(self.dev)

    def run(self, **over):
        a = dict(positions=self.positions, table=torch.from_numpy(self.table).to(self.dev),
                 new=torch.tensor(self.new, dtype=torch.int32, device=self.dev), max_new=max(self.new),
                 before=torch.tensor(self.before, dtype=torch.int32, device=self.dev), positions_n=self.cs.shape[0], stream=None)
        a.update(over)
        fn = Q.dqk_rope_append if self.cache == "int2" else Q.dqk_bf16_rope_append
        rope = Q.rope_desc(self.rotary, self.cs_dev, a["positions_n"], self.inter)
        q = self.q if self.with_q else None
        fn(self.desc, rope, self.k, self.k.stride(0), self.v, self.v.stride(0), q, self.q.stride(0),
           self.q_out if self.with_q else None, self.q_out.stride(0), R.lib_dtype(self.dtype), len(self.new), a["new"], a["before"],
           a["max_new"], a["positions"], a["table"], a["table"].shape[1], stream=a["stream"])
        self.keep_alive = (a, rope)
        torch.cuda.synchronize()

    def turned(self, lo, hi):
        return R.rotate(self.x[:, lo:hi], self.cs[self.pos], self.rotary, self.inter)

    def check(self, only=None):
        """Queries, cache rows and every byte of the cache that no row owns; only: mask of the rows that were taken."""
        only = np.ones(self.rows, bool) if only is None else only
        hq, hkv, d = self.hq, self.hkv, self.d
        if self.with_q:
            got = self.q_out[:self.rows].float().cpu().numpy()[only]
            ref = self.turned(0, hq)[only]
            pair = np.sqrt(2.0) * np.abs(self.x[only, :hq]).max()   # |a c| + |b s| at most
            tol = R.U[self.dtype] * np.abs(ref) + 3 * R.U["f32"] * pair
            assert (np.abs(got - ref) <= tol).all(), f"queries off by {np.abs(got - ref).max():.2e}"
        pool = self.pool.cpu().numpy().reshape(self.num_pages, hkv, self.bb)
        if self.cache == "bf16":
            owned = np.zeros((self.num_pages, 16), bool)
            k, v = self.turned(hq, hq + hkv), self.x[:, hq + hkv:].astype(np.float64)
            cells = pool.view(np.uint16).reshape(self.num_pages, hkv, 2, 16, d // 8, 8)
            for r in np.nonzero(only)[0]:
                page, t = self.table[self.seq[r], self.slot[r] // 16], self.slot[r] % 16
                owned[page, t] = True
                row = cells[page, :, :, t][:, :, np.arange(d // 8) ^ (t % 8)].reshape(hkv, 2, d)
                got = (row.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
                tol = R.U["bf16"] * np.abs(k[r]) + 3 * R.U["f32"] * np.sqrt(2.0) * np.abs(self.x[r]).max()
                assert (np.abs(got[:, 0] - k[r]) <= tol).all(), f"key row {r}"
                assert np.array_equal(got[:, 1], R.bf16(v[r]).astype(np.float64)), f"value row {r}"
            left = cells.transpose(0, 3, 1, 2, 4, 5)[~owned]
            assert (left == 0xA5A5).all(), "memory of no row was written"
            return
        k = self.turned(hq, hq + hkv).astype(np.float32)
        want = O.append(self.t_k, k, np.ascontiguousarray(self.x[:, hq + hkv:]), v_ch0=bool(self.v_ch0), gs=self.gs)
        stale = np.full_like(pool, 0xA5)
        for b in range(len(self.new)):
            end = self.before[b] + self.new[b]
            if not end:
                continue
            got = H.decode_pool(pool, self.table[b], end, d, self.v_ch0, self.gs)
            old = H.decode_pool(stale, self.table[b], end, d, self.v_ch0, self.gs)
            mine = only & (self.seq == b)
            for key in got:
                if key == "vch0" and not self.v_ch0:
                    continue
                old[key][self.slot[mine]] = want[key][mine]
                assert np.array_equal(got[key], old[key]), f"sequence {b}: {key}"


BOTH = pytest.mark.parametrize("cache", ["int2", "bf16"])
SHAPES = {
    "step": dict(new=[1, 1, 1], before=[0, 15, 40]),
    "ragged": dict(new=[3, 0, 17, 1, 64], before=[5, 9, 0, 31, 100], base=1000),
    "f32-interleaved": dict(new=[2, 33], before=[14, 3], dtype="f32", inter=1, base=50000),
    "partial-d64-g1": dict(new=[5, 20], before=[0, 70], hq=3, hkv=3, d=64, rotary=32, gs=64),
    "partial-interleaved": dict(new=[9, 1], before=[2, 16], rotary=48, inter=1, fused=False, v_ch0=1),
    "no-queries": dict(new=[4, 4], before=[0, 1], with_q=False, gs=128, v_ch0=1),
    "in-place": dict(new=[7, 2], before=[0, 30], in_place=True, hq=16),
    "g8-padded-rows": dict(new=[1, 6], before=[20, 12], hq=16, pad=3, dtype="f32"),
    "long": dict(new=[200, 71, 130], before=[0, 9, 3], hkv=1, hq=4),
    "long-d64": dict(new=[150, 65], before=[1, 16], hkv=2, hq=2, d=64, inter=1, v_ch0=1, gs=64, dtype="f32"),
}


@BOTH
@pytest.mark.parametrize("shape", list(SHAPES))
def test_rope_append_matches_64_bits(cache, shape):
    kw = dict(SHAPES[shape])
    c = Case(cache, kw.pop("new"), kw.pop("before"), **kw)
    before = c.q.clone()
    c.run()
    assert Q.dqk_last_device_error() == Q.DQK_OK
    c.check()
    if c.with_q:
        if not c.in_place:
            assert (c.q_out[c.rows:] == 7.0).all()           # rows behind the last sequence, left as they were
        else:
            assert torch.equal(c.q[c.rows:], before[c.rows:])


@BOTH
def test_rows_out_of_range_are_skipped_and_reported(cache):
    c = Case(cache, [3, 2, 4], [15, 0, 40])
    table = c.table.copy()
    table[0, 1] = c.num_pages + 7           # second and third row of sequence 0
    pos = c.pos.astype(np.int32).copy()
    pos[4], pos[7] = -1, c.cs.shape[0]      # second row of sequence 1, third of sequence 2
    only = np.array([True, False, False, True, False, True, True, False, True])
    c.run(table=torch.from_numpy(table).to(c.dev), positions=torch.from_numpy(pos).to(c.dev))
    assert Q.dqk_last_device_error() == Q.DQK_ERR_DEVICE_BOUNDS
    c.check(only)
    assert (c.q_out[:c.rows][torch.from_numpy(~only)] == 7.0).all()
    # more rows than max_new: the first max_new of each sequence are taken
    c = Case(cache, [3, 1], [0, 2])
    c.run(max_new=2)
    assert Q.dqk_last_device_error() == Q.DQK_ERR_DEVICE_BOUNDS
    c.check(np.array([True, True, False, True]))
    # negative lengths: nothing is appended there
    c = Case(cache, [2, 2], [4, 4])
    c.run(before=torch.tensor([-1, 4], dtype=torch.int32, device=c.dev),
          positions=torch.from_numpy(c.pos.astype(np.int32)).to(c.dev))
    assert Q.dqk_last_device_error() == Q.DQK_ERR_DEVICE_BOUNDS
    c.check(np.array([False, False, True, True]))


@BOTH
def test_row_by_row_equals_at_once(cache):
    """Appending one row at a time, and all at once, gives the same bytes."""
    a = Case(cache, [37, 70], [3, 0], seed=3)
    a.run()
    pool, q = a.pool.clone(), a.q_out.clone()
    b = Case(cache, [37, 70], [3, 0], seed=3)
    first = np.concatenate([[0], np.cumsum(b.new)])
    for t in range(max(b.new)):
        for i in range(2):
            if t < b.new[i]:
                r = first[i] + t
                new, before = [0, 0], [0, 0]
                new[i], before[i] = 1, b.before[i] + t
                k, v, qq, out = b.k, b.v, b.q, b.q_out
                b.k, b.v, b.q, b.q_out = k[r:], v[r:], qq[r:], out[r:]
                b.run(new=torch.tensor(new, dtype=torch.int32, device=b.dev), max_new=1,
                      before=torch.tensor(before, dtype=torch.int32, device=b.dev))
                b.k, b.v, b.q, b.q_out = k, v, qq, out
    assert torch.equal(pool, b.pool) and torch.equal(q, b.q_out)


@BOTH
def test_graph_replay_on_another_stream(cache):
    c = Case(cache, [2, 1], [7, 31], base=100)
    c.run()
    want_pool, want_q = c.pool.clone(), c.q_out.clone()
    t = [torch.from_numpy(c.table).to(c.dev), torch.tensor(c.new, dtype=torch.int32, device=c.dev),
         torch.tensor(c.before, dtype=torch.int32, device=c.dev)]
    rope = Q.rope_desc(c.rotary, c.cs_dev, c.cs.shape[0], c.inter)
    fn = Q.dqk_rope_append if cache == "int2" else Q.dqk_bf16_rope_append
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        fn(c.desc, rope, c.k, c.k.stride(0), c.v, c.v.stride(0), c.q, c.q.stride(0), c.q_out, c.q_out.stride(0), Q.DQK_BF16, 2, t[1],
           t[2], 2, c.positions, t[0], t[0].shape[1])
    for _ in range(2):
        c.pool.fill_(0xA5)
        c.q_out.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.pool, want_pool) and torch.equal(c.q_out, want_q)


@BOTH
def test_offsets_past_32_bits(cache):
    block = 1568 if cache == "int2" else 8192
    c = Case(cache, [3, 20], [10, 0], hq=8, hkv=8, pool_pages=(5 << 30) // (8 * block))
    c.run()
    assert Q.dqk_last_device_error() == Q.DQK_OK
    tail = torch.from_numpy(np.unique(c.table[c.table >= 0]).astype(np.int64)).to(c.dev)
    c.pool = c.pool.view(c.num_pages, -1)[tail].reshape(-1).contiguous()   # the pages in use, renumbered
    back = {int(p): i for i, p in enumerate(tail.cpu().tolist())}
    c.table = np.vectorize(lambda p: back.get(int(p), -1), otypes=[np.int32])(c.table)
    c.num_pages = len(back)
    c.check()


@BOTH
def test_serving_steps_behind_a_shared_prefix(cache):
    """The operators together, as a serving loop uses them: the prefix enters the
    cache rotated, then three steps each rotate and append one row per sequence
    at positions behind the prefix and decode over prefix and own tokens."""
    d, hq, hkv, P, steps, batch = 128, 8, 2, 100, 3, 4
    pre = Case(cache, [P], [0], hq=hq, hkv=hkv, seed=21, pool_pages=R.pages(P) + batch)   # behind the own pages
    own = np.arange(batch, dtype=np.int32)[:, None]
    pre.run()
    assert Q.dqk_last_device_error() == Q.DQK_OK
    L = R.Lists.__new__(R.Lists)
    L.cache, L.hq, L.hkv, L.d, L.gs, L.v_ch0, L.dev = cache, hq, hkv, d, 32, 0, pre.dev
    L.t_k = pre.t_k
    L.t_q = np.ascontiguousarray(np.linalg.inv(pre.t_k.astype(np.float64)).transpose(0, 2, 1)).astype(np.float32)
    L.tq_dev = torch.from_numpy(L.t_q).to(L.dev)
    L.desc = Q.layer_desc(d, hq, hkv, pre.tk_dev, L.tq_dev, pre.pool, pre.num_pages)
    L.tables, L.lens_list = [pre.table, own], [[P], [0] * batch]

    L.rows = [[L._stored(pre.turned(hq, hq + hkv).astype(np.float32), pre.x[:, hq + hkv:])], [None] * batch]
    ks, vs = [[] for _ in range(batch)], [[] for _ in range(batch)]
    for t in range(steps):
        c = Case(cache, [1] * batch, [t] * batch, hq=hq, hkv=hkv, seed=30 + t, base=P)
        c.pool, c.table, c.num_pages, c.t_k = pre.pool, own, pre.num_pages, pre.t_k
        c.desc = L.desc
        c.run()
        q = c.q_out[:batch].float().cpu().numpy()
        k = c.turned(hq, hq + hkv).astype(np.float32)
        for b in range(batch):
            ks[b].append(k[b])
            vs[b].append(c.x[b, hq + hkv:])
            L.rows[1][b] = L._stored(np.stack(ks[b]), np.stack(vs[b]))
        L.lens_list[1] = [t + 1] * batch
        out, sel = L.prefix_decode(q, "bf16", [0, batch])
        torch.cuda.synchronize()
        assert Q.dqk_last_device_error() == Q.DQK_OK
        for b in range(batch):
            qe, want = L.query(q[b], "bf16", 40)
            ref, bound = L.attend(qe, [L.rows[0][0], L.rows[1][b]], "bf16", "f32")
            if cache == "bf16":   # a key one BF16 step away at a rounding tie moves a score by at most that step
                bound = bound * 3
            R.check(out[b], ref, bound, f"step {t}, sequence {b}")
            if want is not None:
                assert np.array_equal(sel[b].cpu().numpy(), want)
