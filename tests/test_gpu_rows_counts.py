"""GPU: every token of every list counts once, wherever the split over the CTAs
falls.

Queries of zeros give every token the weight 1, exact in every format, and
values are marks: channel c is 1 at the tokens whose mark -- their number, page
or unit of 128, counted over all lists -- is c modulo d, else 0.  So
out_c = (tokens marked c) / (tokens), and the only errors are: the rounding of a
stored mark (INT2: 3 fp16(1/3), taken into the reference by the oracle, and once
more to fp16, 2^-11), fp32 sums (n terms of one sign, each addition off by at most
2^-23 of the sum) and the output's rounding.  A token, page or unit that is missed
or counted twice is off by a whole mark in tokens / d of them."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import rows_ref as R  # noqa: E402
from bit_kv_cache_dqk_b200 import dualqk as Q  # noqa: E402

pytestmark = pytest.mark.gpu

STEP = {"token": 1, "page": 16, "unit": 128}


class Marked(R.Lists):
    def __init__(self, cache, lens_list, hq, hkv, d, mark, **kw):
        self.step, self.at = STEP[mark], 0
        super().__init__(cache, lens_list, hq, hkv, d, **kw)

    def _append(self, table, lens, ks, vs, dtype):
        for i, v in enumerate(vs):
            n, hkv, d = v.shape
            mark = (np.arange(n) // self.step + self.at) % d
            x = np.zeros((n, hkv, d), np.float32)
            x[np.arange(n), :, mark] = 1.0
            vs[i] = R.as_dtype(x, dtype)
            self.at += 7 * i + 5
        super()._append(table, lens, ks, vs, dtype)


def check(L, got, parts, what):
    v = np.concatenate([p[1] for p in parts])
    if not len(v):
        assert not got.float().abs().max().item(), what
        return
    n = len(v)
    ref = v.sum(0) / n                                      # [hkv][d]
    u = (2.0 ** -11 if L.cache == "int2" else 0.0) + (2 * n + 64) * 2.0 ** -23 + 2.0 ** -23
    bound = np.repeat(u * np.abs(v).sum(0) / n, L.hq // L.hkv, 0)
    assert bound.max() * n < 0.5 * L.step, "the bound would not see one mark"
    R.check(got, np.repeat(ref, L.hq // L.hkv, 0), bound, what)


def run_prefix(L, start, batch):
    q = np.zeros((batch, L.hq, L.d), np.float32)
    for own in (True, False):
        out, _ = L.prefix_decode(q, "bf16", start, own=own)
        torch.cuda.synchronize()
        assert Q.dqk_last_device_error() == Q.DQK_OK
        for b in range(batch):
            parts = [L.rows[0][g] for g in range(len(start) - 1) if start[g] <= b < start[g + 1]]
            parts += [L.rows[1][b]] if own else []
            check(L, out[b], parts or [(np.zeros((0, L.hkv, L.d)),) * 2], f"sequence {b}, own {own}")


@pytest.mark.parametrize("mark", list(STEP))
@pytest.mark.parametrize("cache", ["int2", "bf16"])
def test_long_prefix(cache, mark):
    """One list over all CTAs, tiles of 24 and of 300 row heads."""
    for rows in (6, 75):
        own = [[700, 0, 3, 1500, 33, 1][i % 6] if rows == 6 else i % 5 for i in range(rows)]
        run_prefix(Marked(cache, [[5000], own], 8, 2, 128, mark, seed=51), [0, rows], rows)


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("cache", ["int2", "bf16"])
def test_random_lists(cache, seed):
    rng = np.random.default_rng([seed, 91])
    d = int(rng.choice([64, 128]))
    g, hkv = int(rng.choice([1, 2, 4, 8])), int(rng.integers(1, 4))
    groups = int(rng.integers(1, 7))
    start = np.concatenate([[0], np.cumsum(rng.choice([0, 1, 2, 3, 17, 40], groups))]) + int(rng.integers(0, 2))
    batch = int(start[-1]) + int(rng.integers(1, 3))
    length = lambda most: int(rng.choice([0, 1, 127, 128, 129, int(rng.integers(1, most))]))  # noqa: E731
    L = Marked(cache, [[length(3000) for _ in range(groups)], [length(600) for _ in range(batch)]], g * hkv, hkv, d,
               ["token", "page", "unit"][seed % 3], seed=seed)
    run_prefix(L, [int(x) for x in start], batch)


@pytest.mark.parametrize("cache", ["int2", "bf16"])
def test_many_prefixes_with_own_lists(cache):
    """More lists than a warp has lanes, of both kinds."""
    rng = np.random.default_rng(92)
    start = np.concatenate([[0], np.cumsum(rng.integers(0, 4, 70))]).tolist()
    batch = start[-1] + 2
    L = Marked(cache, [rng.integers(0, 500, 70).tolist(), rng.integers(0, 260, batch).tolist()], 8, 2, 128, "token", seed=53)
    run_prefix(L, start, batch)


@pytest.mark.parametrize("hq,hkv,d", [(8, 4, 128), (8, 1, 64)])
def test_cross_attention_lists(hq, hkv, d):
    """Dozens of whole lists on a CTA, and long ones that cross their borders."""
    rng = np.random.default_rng(93)
    nkv, nq = rng.integers(0, 700, 120).tolist(), rng.integers(0, 4, 120).tolist()
    nq[7], nkv[7], nq[20], nkv[20], nq[50], nkv[50] = 90, 4000, 150, 300, 1, 6000
    L = Marked("bf16", [nkv], hq, hkv, d, "token", seed=54)
    start = np.concatenate([[0], np.cumsum(nq)]).tolist()
    out = L.cross(np.zeros((start[-1], hq, d), np.float32), "bf16", start)
    assert Q.dqk_last_device_error() == Q.DQK_OK
    for b in range(len(nq)):
        for r in range(start[b], start[b + 1]):
            check(L, out[r], [L.rows[0][b]], f"row {r}")


@pytest.mark.parametrize("d", [64, 128])
def test_many_items_without_own_lists(d):
    """More items than CTAs: records by CTA alone."""
    rng = np.random.default_rng(94)
    nkv, nq = rng.integers(1, 900, 60).tolist(), rng.integers(1, 80, 60).tolist()
    L = Marked("bf16", [nkv], 32, 8, d, "token", seed=55)
    start = np.concatenate([[0], np.cumsum(nq)]).tolist()
    out = L.cross(np.zeros((start[-1], 32, d), np.float32), "bf16", start)
    for b in range(len(nq)):
        for r in (start[b], start[b + 1] - 1, (start[b] + start[b + 1]) // 2):
            check(L, out[r], [L.rows[0][b]], f"row {r}")
