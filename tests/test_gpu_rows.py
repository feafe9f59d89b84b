"""GPU: the shared-prefix decode (INT2 and BF16 caches) and the cross attention
against attention in 64 bits over the cached values, with derived bounds."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import rows_ref as R  # noqa: E402
from bit_kv_cache_dqk_b200 import dualqk as Q  # noqa: E402

pytestmark = pytest.mark.gpu


def queries(L, rows, seed=5, scale=1.0):
    return (np.random.default_rng([seed, 3]).standard_normal((rows, L.hq, L.d)) * scale).astype(np.float32)


def check_prefix(L, q, dtype, start, pct=40, out_dtype="f32", own=True, out=None, sel=None):
    if out is None:
        out, sel = L.prefix_decode(q, dtype, start, pct, out_dtype, own)
        torch.cuda.synchronize()
        assert Q.dqk_last_device_error() == Q.DQK_OK
    for b in range(q.shape[0]):
        qe, want = L.query(q[b], dtype, pct)
        parts = [L.rows[0][g] for g in range(len(start) - 1) if start[g] <= b < start[g + 1]]
        if own:
            parts = parts + [L.rows[1][b]]
        if want is not None:
            assert np.array_equal(sel[b].cpu().numpy(), want), f"kept channels of sequence {b}"
        if not parts:
            parts = [(np.zeros((0, L.hkv, L.d)),) * 2]
        ref, bound = L.attend(qe, parts, dtype, out_dtype)
        R.check(out[b], ref, bound, f"sequence {b}")
    return out, sel


# cache, hq, hkv, d, gs, v_ch0, dtype, pct, out_dtype, group starts, prefix lengths, own lengths
CASES = {
    "int2-one-token": ("int2", 8, 2, 128, 32, 0, "bf16", 40, "f32", [0, 1], [1], [0]),
    "int2-empty": ("int2", 8, 2, 128, 32, 0, "bf16", 40, "f32", [0, 2, 3], [0, 5], [0, 3, 0]),
    "int2-page-ends": ("int2", 4, 1, 128, 32, 0, "f32", 20, "f32", [0, 1, 2, 3, 4], [15, 16, 17, 129], [16, 1, 128, 0]),
    "int2-g1-d64": ("int2", 3, 3, 64, 32, 0, "f32", 40, "f32", [0, 5], [200], [0, 1, 40, 127, 128]),
    "int2-g2-d64-one-group": ("int2", 8, 4, 64, 64, 1, "bf16", 60, "bf16", [0, 4], [333], [10, 0, 7, 31]),
    "int2-g8-one-group": ("int2", 16, 2, 128, 128, 1, "bf16", 0, "f32", [0, 3, 7], [140, 257], [3, 0, 20, 1, 0, 0, 64]),
    "int2-tiles": ("int2", 8, 2, 128, 32, 1, "bf16", 40, "f32", [0, 40, 41], [300, 20], [n % 7 for n in range(41)]),
    "bf16-one-token": ("bf16", 8, 2, 128, 32, 0, "bf16", 0, "f32", [0, 1], [1], [0]),
    "bf16-empty": ("bf16", 8, 2, 128, 32, 0, "f32", 0, "f32", [0, 2, 3], [0, 5], [0, 3, 0]),
    "bf16-page-ends": ("bf16", 4, 1, 128, 32, 0, "f32", 0, "f32", [0, 1, 2, 3, 4], [15, 16, 17, 129], [16, 1, 128, 0]),
    "bf16-g1-d64": ("bf16", 3, 3, 64, 32, 0, "bf16", 0, "bf16", [0, 17], [200], [i * 3 for i in range(17)]),
    "bf16-g8-gaps": ("bf16", 40, 5, 64, 32, 0, "bf16", 0, "f32", [1, 3, 3, 5], [140, 99, 257], [3, 0, 20, 1, 0, 0, 64]),
    "bf16-tiles": ("bf16", 8, 2, 128, 32, 0, "f32", 0, "bf16", [0, 70, 103], [300, 1000], [n % 5 for n in range(103)]),
    "bf16-long": ("bf16", 8, 2, 128, 32, 0, "bf16", 0, "f32", [0, 6], [5000], [700, 0, 3, 1500, 33, 1]),
    "int2-long": ("int2", 8, 2, 128, 32, 0, "bf16", 40, "f32", [0, 6], [5000], [700, 0, 3, 1500, 33, 1]),
}


def build(case, seed=1):
    cache, hq, hkv, d, gs, v0, dtype, pct, out_dtype, start, prefix, own = CASES[case]
    return R.Lists(cache, [prefix, own], hq, hkv, d, dtype=dtype, gs=gs, v_ch0=v0, seed=seed)


@pytest.mark.parametrize("case", list(CASES))
def test_prefix_decode_matches_64_bits(case):
    dtype, pct, out_dtype, start = CASES[case][6:10]
    L = build(case)
    check_prefix(L, queries(L, len(L.lens_list[1])), dtype, start, pct, out_dtype)


@pytest.mark.parametrize("cache", ["int2", "bf16"])
def test_prefix_alone_and_large_scores(cache):
    """No own lists at all; queries that make the weights uneven (one token
    carries nearly everything)."""
    L = R.Lists(cache, [[400, 131], [1]], 8, 2, 128, seed=4, k_scale=1.5)
    check_prefix(L, queries(L, 9, scale=3.0), "bf16", [0, 5, 9], own=False)


# hq, hkv, d, dtype, out_dtype, query counts, state counts
CROSS = {
    "step": (8, 2, 128, "bf16", "f32", [1, 1, 1], [100, 1, 257]),
    "rows": (8, 2, 128, "bf16", "bf16", [3, 0, 50, 1], [40, 77, 300, 0]),
    "f32-d64-g8": (16, 2, 64, "f32", "f32", [13, 33], [500, 129]),
    "g1": (5, 5, 64, "bf16", "f32", [130, 5], [64, 1000]),
    "tiles": (4, 1, 128, "f32", "bf16", [200, 31, 65], [128, 127, 129]),
    "wide": (8, 1, 128, "bf16", "f32", [100, 64], [700, 16]),
}


@pytest.mark.parametrize("case", list(CROSS))
def test_cross_attention_matches_64_bits(case):
    hq, hkv, d, dtype, out_dtype, nq, nkv = CROSS[case]
    L = R.Lists("bf16", [nkv], hq, hkv, d, dtype=dtype, seed=6)
    start = np.concatenate([[0], np.cumsum(nq)])
    q = queries(L, int(start[-1]) + 3)     # three rows behind the last sequence
    out = L.cross(q, dtype, start.tolist(), out_dtype)
    assert Q.dqk_last_device_error() == Q.DQK_OK
    assert torch.isnan(out[start[-1]:]).all()      # left as they were
    for b in range(len(nq)):
        for r in range(start[b], start[b + 1]):
            ref, bound = L.attend(L.query(q[r], dtype, 0)[0], [L.rows[0][b]], dtype, out_dtype)
            R.check(out[r], ref, bound, f"row {r}")


@pytest.mark.parametrize("cache", ["int2", "bf16"])
def test_same_as_the_plain_decode_over_repeated_pages(cache):
    """Whole-page prefixes: the decode whose page table repeats the prefix's
    pages for every sequence reads the same tokens."""
    L = R.Lists(cache, [[512, 96], [33, 0, 100, 16, 1]], 8, 2, 128, seed=9)
    start, group = [0, 3, 5], [0, 0, 0, 1, 1]
    q = queries(L, 5)
    out, sel = check_prefix(L, q, "bf16", start)
    lens = [L.lens_list[0][g] + n for g, n in zip(group, L.lens_list[1])]
    table = np.full((5, max(R.pages(n) for n in lens)), -1, np.int32)
    for b, g in enumerate(group):
        np_, no = R.pages(L.lens_list[0][g]), R.pages(L.lens_list[1][b])
        table[b, :np_], table[b, np_:np_ + no] = L.tables[0][g, :np_], L.tables[1][b, :no]
    td, ld = torch.from_numpy(table).to(L.dev), torch.tensor(lens, dtype=torch.int32, device=L.dev)
    qd = R.as_dtype(q, "bf16").to(L.dev)
    ref, ref_sel = torch.empty_like(out), torch.empty_like(sel)
    if cache == "int2":
        ws = torch.empty(Q.dqk_decode_workspace_size(L.desc, 5, table.shape[1]), dtype=torch.uint8, device=L.dev)
        Q.dqk_decode(L.desc, qd, Q.DQK_BF16, 5, ld, td, table.shape[1], 40, ref, ref_sel, ws, ws.numel())
        assert torch.equal(sel, ref_sel)
        tol = 2e-3      # the plain decode's own tolerance
    else:
        ws = torch.empty(Q.dqk_bf16_decode_workspace_size(L.desc, 5, table.shape[1]), dtype=torch.uint8, device=L.dev)
        Q.dqk_bf16_decode(L.desc, qd, Q.DQK_BF16, 5, ld, td, table.shape[1], ref, ws, ws.numel())
        tol = 0.0
    torch.cuda.synchronize()
    for b, g in enumerate(group):
        exact, bound = L.attend(L.query(q[b], "bf16", 40)[0], [L.rows[0][g], L.rows[1][b]], "bf16", "f32")
        off = np.abs(out[b].cpu().numpy() - ref[b].cpu().numpy())
        # each side is within its own bound of the exact value; the plain BF16 decode within this one's
        assert (off <= bound + (tol if tol else bound)).all()


@pytest.mark.parametrize("cache", ["int2", "bf16"])
def test_bad_pages_and_lengths_are_reported_and_skipped(cache):
    L = R.Lists(cache, [[300], [20, 5]], 8, 2, 128, seed=11)
    q = queries(L, 2)
    bad = L.table_dev(0).clone()
    bad[0, 3], bad[0, 7] = L.num_pages + 3, -5
    out, _ = L.prefix_decode(q, "bf16", [0, 2], table=bad)
    assert Q.dqk_last_device_error() == Q.DQK_ERR_DEVICE_BOUNDS
    keep = np.ones(300, bool)
    keep[48:64] = keep[112:128] = False
    parts = [tuple(x[keep] for x in L.rows[0][0])]
    for b in range(2):
        ref, bound = L.attend(L.query(q[b], "bf16", 40)[0], parts + [L.rows[1][b]], "bf16", "f32")
        R.check(out[b], ref, bound, f"sequence {b}")
    # a length past the page table's reach is cut to it: 304 slots, the last 4 of them unwritten (NaN)
    cut = torch.tensor([1 << 30], dtype=torch.int32, device=L.dev)
    L.prefix_decode(q, "bf16", [0, 2], lens=cut)
    assert Q.dqk_last_device_error() == Q.DQK_ERR_DEVICE_BOUNDS
    # groups that overlap or run backwards write nothing outside the workspace and are reported
    L.prefix_decode(q, "bf16", [-3, 99])
    assert Q.dqk_last_device_error() == Q.DQK_OK          # cut to [0, 2)
    check_prefix(L, q, "bf16", [0, 2])                     # the next call is unaffected


def test_infinite_and_nan_values_stay_in_their_rows():
    """A NaN or infinity among one sequence's own values reaches that sequence's
    outputs of that kv head only."""
    L = R.Lists("bf16", [[200], [40, 40, 40]], 8, 2, 128, seed=12)
    q = queries(L, 3)
    clean, _ = L.prefix_decode(q, "bf16", [0, 3])
    blk = L.pool.view(torch.bfloat16).view(L.num_pages, 2, 2, 16, 128)
    blk[int(L.tables[1][1, 0]), 0, 1, 3, 5] = float("nan")
    blk[int(L.tables[1][2, 0]), 1, 1, 3, 9] = float("inf")
    out, _ = L.prefix_decode(q, "bf16", [0, 3])
    torch.cuda.synchronize()
    assert torch.equal(out[0], clean[0]) and torch.equal(out[1, 4:], clean[1, 4:]) and torch.equal(out[2, :4], clean[2, :4])
    assert torch.isnan(out[1, :4, :]).any(-1).all() and not torch.isfinite(out[2, 4:]).all(-1).any()


@pytest.mark.parametrize("cache", ["int2", "bf16"])
def test_other_stream_graph_replay_and_shared_workspace(cache):
    """Two captured calls that share a workspace, replayed in turn with new
    queries in the captured buffers, on a stream of their own."""
    L = R.Lists(cache, [[260, 90], [30, 0, 17, 64]], 8, 2, 128, seed=13)
    start = [0, 3, 4]
    q1, q2 = queries(L, 4, seed=1), queries(L, 4, seed=2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    size_of = Q.dqk_prefix_decode_workspace_size if cache == "int2" else Q.dqk_bf16_prefix_decode_workspace_size
    ws = torch.empty(size_of(L.desc, 4, 2, L.tables[0].shape[1], L.tables[1].shape[1]), dtype=torch.uint8, device=L.dev)
    with torch.cuda.stream(s):
        L.prefix_decode(q1, "bf16", start, ws=ws)        # warm-up: function attributes are set
        s.synchronize()
        graphs = []
        for _ in range(2):
            qd = torch.zeros((4, 8, 128), dtype=torch.bfloat16, device=L.dev)
            t = [L.table_dev(0), L.table_dev(1), L.lens_dev(0), L.lens_dev(1), torch.tensor(start, dtype=torch.int32, device=L.dev)]
            out = torch.zeros((4, 8, 128), device=L.dev)
            sel = torch.zeros((4, 8, 77), dtype=torch.int16, device=L.dev)
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                head = (L.desc, qd, Q.DQK_BF16, 4, 2, t[4], t[2], t[0], t[0].shape[1], t[3], t[1], t[1].shape[1])
                if cache == "int2":
                    Q.dqk_prefix_decode(*head, 40, out, Q.DQK_F32, sel, ws, ws.numel())
                else:
                    Q.dqk_bf16_prefix_decode(*head, out, Q.DQK_F32, ws, ws.numel())
            graphs.append((g, qd, out, sel, t))
        for q in (q1, q2):
            graphs[0][1].copy_(R.as_dtype(q, "bf16"))
            graphs[1][1].copy_(R.as_dtype(-q, "bf16"))
            graphs[0][0].replay()
            graphs[1][0].replay()
            s.synchronize()
            check_prefix(L, q, "bf16", start, out=graphs[0][2], sel=graphs[0][3])
            check_prefix(L, -q, "bf16", start, out=graphs[1][2], sel=graphs[1][3])
    assert Q.dqk_last_device_error() == Q.DQK_OK


def test_calls_are_reproducible():
    """The same call gives the same bytes (no order of arrival decides a sum)."""
    for cache in ("int2", "bf16"):
        L = R.Lists(cache, [[3000], [200, 900]], 8, 2, 128, seed=14)
        q = queries(L, 2)
        a, _ = L.prefix_decode(q, "bf16", [0, 2])
        for _ in range(3):
            b, _ = L.prefix_decode(q, "bf16", [0, 2])
            assert torch.equal(a, b)


def test_offsets_past_32_bits():
    """Pages far into a pool of more than 4 GB, and a cross attention over them."""
    for cache in ("int2", "bf16"):
        hkv, d = 8, 128
        block = 1568 if cache == "int2" else 8192
        L = R.Lists(cache, [[70], [20, 3]], 16, hkv, d, seed=15, pool_pages=(5 << 30) // (hkv * block))
        check_prefix(L, queries(L, 2), "bf16", [0, 2])
        del L
        torch.cuda.empty_cache()


@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (128, "f32"), (64, "bf16")])
def test_many_short_lists_per_block(d, dtype):
    """Dozens of whole lists and a few split ones on every block: items that end
    inside a block hand records between its warpgroups, the others go through
    the merge."""
    rng = np.random.default_rng(8)
    nkv = rng.integers(0, 700, 150).tolist()
    nq = rng.integers(0, 4, 150).tolist()
    nq[7], nkv[7], nq[20], nkv[20] = 90, 650, 150, 300
    L = R.Lists("bf16", [nkv], 8, 4, d, dtype=dtype, seed=16)
    start = np.concatenate([[0], np.cumsum(nq)])
    q = queries(L, int(start[-1]))
    out = L.cross(q, dtype, start.tolist(), "bf16")
    assert Q.dqk_last_device_error() == Q.DQK_OK
    for b in range(len(nq)):
        for r in range(start[b], start[b + 1], 1 if nq[b] < 10 else 17):
            ref, bound = L.attend(L.query(q[r], dtype, 0)[0], [L.rows[0][b]], dtype, "bf16")
            R.check(out[r], ref, bound, f"row {r}")


@pytest.mark.parametrize("cache", ["int2", "bf16"])
def test_references_that_move(cache):
    """Scores that grow along the list: the running reference of nearly every
    row moves many times, by more than its slack."""
    L = R.Lists(cache, [[900, 260], [150, 300, 0, 64, 5]], 8, 2, 128, seed=17)
    q = queries(L, 5, scale=0.1)
    if cache == "bf16":
        # keys along one direction, growing with the token
        blk = L.pool.view(torch.bfloat16).view(L.num_pages, 2, 2, 16, 128)
        for i, (table, lens) in enumerate(zip(L.tables, L.lens_list)):
            for g, n in enumerate(lens):
                for t in range(n):
                    for j in range(2):
                        x = torch.full((128,), 0.02 * (t + 300 * i), dtype=torch.bfloat16, device=L.dev)
                        blk[int(table[g, t // 16]), j, 0, t % 16] = x      # equal channels: chunk order does not matter
                        L.rows[i][g][0][t, j] = float(x[0])
        q = np.abs(q) + 0.05
    else:
        q = q * 60.0
    check_prefix(L, q, "f32", [0, 3, 5])
