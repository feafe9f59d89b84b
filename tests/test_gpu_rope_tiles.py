"""GPU: rotated appends of many rows (tiles of rows per CTA), and the codes of
values that lie on, or a step beside, the borders between two codes."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import rows_ref as R  # noqa: E402
from bit_kv_cache_dqk_b200 import dualqk as Q  # noqa: E402
from test_gpu_rope import Case  # noqa: E402

pytestmark = pytest.mark.gpu


def ragged(seed, sequences, most):
    rng = np.random.default_rng(seed)
    new = [int(n) for n in rng.integers(0, most + 1, sequences)]
    new[1], new[2] = most, 1
    return dict(new=new, before=[int(n) for n in rng.integers(0, 50, sequences)])


# sequences and rows that reach tiles of 16 rows (few) and of 64 (many)
FEW, MANY = ragged(1, 5, 100), ragged(2, 33, 81)
SHAPES = {
    "few": dict(FEW, base=700),
    "few-d64-g1": dict(FEW, hq=2, hkv=2, d=64, rotary=32, gs=64, v_ch0=1, dtype="f32"),
    "few-one-group": dict(FEW, gs=128, inter=1, in_place=True),
    "many": dict(MANY, base=7),
    "many-d64": dict(MANY, d=64, hq=8, hkv=2, inter=1, rotary=48, dtype="f32"),
    "many-one-group": dict(MANY, gs=128, v_ch0=1, rotary=16, with_q=False),
    "many-d64-one-group": dict(MANY, d=64, gs=64, hq=4, hkv=4, in_place=True),
    "one-long": dict(new=[2500], before=[9], hkv=4, hq=4, fused=False),
}


@pytest.mark.parametrize("shape", list(SHAPES))
def test_tiles_match_64_bits(shape):
    kw = dict(SHAPES[shape])
    c = Case("int2", kw.pop("new"), kw.pop("before"), **kw)
    c.run()
    assert Q.dqk_last_device_error() == Q.DQK_OK
    c.check()
    if c.with_q and not c.in_place:
        assert (c.q_out[c.rows:] == 7.0).all()


@pytest.mark.parametrize("shape", [FEW, MANY], ids=["few", "many"])
def test_rows_out_of_range_inside_a_tile(shape):
    c = Case("int2", shape["new"], shape["before"])
    first = np.concatenate([[0], np.cumsum(c.new)])
    only = np.ones(c.rows, bool)
    pos, table = c.pos.astype(np.int32).copy(), c.table.copy()
    for r in (first[1] + 3, first[1] + 63, first[3] - 1, c.rows - 1):
        pos[r] = [-1, c.cs.shape[0]][r % 2]
        only[r] = False
    page = (c.before[1] + 20) // 16          # a page of sequence 1 that is not there
    table[1, page] = -5
    only &= ~((c.seq == 1) & (c.slot // 16 == page))
    c.run(table=torch.from_numpy(table).to(c.dev), positions=torch.from_numpy(pos).to(c.dev))
    assert Q.dqk_last_device_error() == Q.DQK_ERR_DEVICE_BOUNDS
    c.check(only)
    assert (c.q_out[:c.rows][torch.from_numpy(~only)] == 7.0).all()


def borders(rng, rows, hkv, d, group, special):
    """Rows whose groups hold min, min + 3 s and values within two fp32 steps of min + {1, 3, 5} s / 2."""
    x = np.zeros((rows, hkv, d), np.float32)
    for r in range(rows):
        for j in range(hkv):
            for g0 in range(0, d, group):
                s = np.float32(np.float16(2.0 ** rng.uniform(-12, 6)))
                lo = np.float32(np.float16(rng.choice([0.0, -0.5, -1.5, -2.5, rng.uniform(-40, 40), rng.uniform(-3, 0)]) * s))
                v = (lo + s * rng.choice([0.5, 1.5, 2.5], group).astype(np.float32)).astype(np.float32)
                for _ in range(2):
                    step = rng.integers(-1, 2, group)
                    v = np.where(step > 0, np.nextafter(v, np.float32(np.inf)), np.where(step < 0, np.nextafter(v, np.float32(-np.inf)), v))
                v = np.clip(v, lo, np.float32(lo + np.float32(3) * s))
                v[1], v[2] = lo, np.float32(lo + np.float32(3) * s)
                v[3] = np.clip(np.float32(rng.choice([1e-40, -1e-40, 1e-30, -1e-30])), v[1], v[2])
                kind = rng.integers(0, 12) if special else 99
                if kind == 0:
                    v[5] = np.nan
                elif kind == 1:
                    v[5] = np.inf
                elif kind == 2:
                    v[5], v[6] = -np.inf, np.inf
                elif kind == 3:
                    v[:] = np.nan
                elif kind == 4:
                    v[:] = lo
                elif kind == 5:
                    v[7] = np.float32(3e38)
                elif kind == 6:
                    v *= np.float32(1e-38)
                x[r, j, g0:g0 + group] = v
    return x


@pytest.mark.parametrize("d,gs,v_ch0", [(128, 32, 0), (128, 128, 1), (64, 32, 1), (64, 64, 0)])
@pytest.mark.parametrize("shape", [FEW, MANY], ids=["few", "many"])
def test_codes_at_the_borders_are_those_of_the_plain_append(shape, d, gs, v_ch0):
    """Angles of zero and T_K = 1: every byte is dqk_append's, whose codes come from divisions in 64 bits."""
    hkv = 2
    c = Case("int2", shape["new"], shape["before"], d=d, gs=gs, v_ch0=v_ch0, dtype="f32", hkv=hkv, hq=2, with_q=False, fused=False)
    rng = np.random.default_rng([d, gs, c.rows])
    c.k = torch.from_numpy(borders(rng, c.rows, hkv, d, gs, False)).to(c.dev)
    c.v = torch.from_numpy(borders(rng, c.rows, hkv, d, gs, True)).to(c.dev)
    c.tk_dev.copy_(torch.eye(d).expand(hkv, d, d))
    c.cs_dev[:, :d // 2] = 1.0
    c.cs_dev[:, d // 2:] = 0.0
    c.run()
    got = c.pool.clone()
    c.pool.fill_(0xA5)
    i32 = dict(dtype=torch.int32, device=c.dev)
    table = torch.from_numpy(c.table).to(c.dev)
    new, before = torch.tensor(c.new, **i32), torch.tensor(c.before, **i32)
    Q.dqk_append(c.desc, c.k, c.v, Q.DQK_F32, len(c.new), new, before, max(c.new), table, table.shape[1])
    torch.cuda.synchronize()
    assert Q.dqk_last_device_error() == Q.DQK_OK
    pool = got.reshape(-1, c.bb), c.pool.reshape(-1, c.bb)
    differ = (pool[0] != pool[1]).any(1).nonzero().flatten().tolist()
    assert not differ, f"{len(differ)} blocks differ, first {differ[:5]}"


def test_tiles_in_a_graph_on_another_stream():
    c = Case("int2", MANY["new"], MANY["before"], base=3)
    c.run()
    want_pool, want_q = c.pool.clone(), c.q_out.clone()
    i32 = dict(dtype=torch.int32, device=c.dev)
    t = [torch.from_numpy(c.table).to(c.dev), torch.tensor(c.new, **i32), torch.tensor(c.before, **i32)]
    rope = Q.rope_desc(c.rotary, c.cs_dev, c.cs.shape[0], c.inter)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        Q.dqk_rope_append(c.desc, rope, c.k, c.k.stride(0), c.v, c.v.stride(0), c.q, c.q.stride(0), c.q_out, c.q_out.stride(0),
                          R.lib_dtype(c.dtype), len(c.new), t[1], t[2], max(c.new), c.positions, t[0], t[0].shape[1])
    for _ in range(2):
        c.pool.fill_(0xA5)
        c.q_out.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(c.pool, want_pool) and torch.equal(c.q_out, want_q)
