"""GPU: the shared-prefix decode and the cross attention where the split over
the CTAs falls anywhere: lists of random lengths, and calls at the same time."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import rows_ref as R  # noqa: E402
from bit_kv_cache_dqk_b200 import dualqk as Q  # noqa: E402
from test_gpu_rows import check_prefix, queries  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seed", range(8))
@pytest.mark.parametrize("cache", ["int2", "bf16"])
def test_random_lists(cache, seed):
    rng = np.random.default_rng([seed, 77])
    d = int(rng.choice([64, 128]))
    g, hkv = int(rng.choice([1, 2, 4, 8])), int(rng.integers(1, 4))
    groups = int(rng.integers(1, 6))
    sizes = rng.choice([0, 1, 2, 3, 17, 40], groups)
    start = np.concatenate([[0], np.cumsum(sizes)]) + int(rng.integers(0, 2))
    batch = int(start[-1]) + int(rng.integers(1, 3))
    length = lambda most: int(rng.choice([0, 1, 127, 128, 129, int(rng.integers(1, most))]))  # noqa: E731
    prefix, own = [length(3000) for _ in range(groups)], [length(600) for _ in range(batch)]
    dtype = str(rng.choice(["bf16", "f32"]))
    L = R.Lists(cache, [prefix, own], g * hkv, hkv, d, dtype=dtype, seed=seed)
    check_prefix(L, queries(L, batch, seed), dtype, [int(x) for x in start])
    check_prefix(L, queries(L, batch, seed + 50), dtype, [int(x) for x in start], own=False)


@pytest.mark.parametrize("cache", ["int2", "bf16"])
def test_two_calls_at_once(cache):
    """Two streams, a workspace each, over one pool."""
    L = R.Lists(cache, [[2000, 300], [200, 0, 1500, 9, 64]], 8, 2, 128, seed=5)
    start = [0, 3, 5]
    q = [queries(L, 5, seed=s) for s in (1, 2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s, x in zip(streams, q):
            with torch.cuda.stream(s):
                outs.append((x, *L.prefix_decode(x, "bf16", start)))
    torch.cuda.synchronize()
    assert Q.dqk_last_device_error() == Q.DQK_OK
    for x, out, sel in outs:
        check_prefix(L, x, "bf16", start, out=out, sel=sel)


def test_workspace_of_the_largest_call_serves_smaller_ones():
    """A workspace sized with own lists is enough without them."""
    for size in (Q.dqk_prefix_decode_workspace_size, Q.dqk_bf16_prefix_decode_workspace_size):
        for hkv, rows in ((1, 4), (8, 64), (8, 900)):
            probe = Q.layer_desc(128, 4 * hkv, hkv, 256, 256, 256, 4096)
            sizes = [size(probe, rows, 1, 64, own) for own in (0, 1, 9, 64)]
            assert sizes == sorted(sizes) and sizes[0] > 0


def test_groups_that_overlap_are_reported():
    """More row tiles than ascending starts could have: an error, no access past the workspace."""
    rows, times = 650, 20
    L = R.Lists("bf16", [[300] * (2 * times - 1)], 8, 1, 128, seed=9)
    q = queries(L, rows)
    q_start = [0, rows] * times
    ws_size = Q.dqk_bf16_cross_attention_workspace_size(L.desc, 2 * times - 1, rows, L.tables[0].shape[1])
    guard = 1 << 20
    ws = torch.full((ws_size + guard,), 0x5A, dtype=torch.uint8, device=L.dev)
    qd = R.as_dtype(q, "bf16").to(L.dev)
    out = torch.zeros((rows, 8, 128), device=L.dev)
    starts, lens, table = torch.tensor(q_start, dtype=torch.int32, device=L.dev), L.lens_dev(0), L.table_dev(0)
    Q.dqk_bf16_cross_attention(L.desc, qd, Q.DQK_BF16, 2 * times - 1, rows, starts, lens, table, table.shape[1], out, Q.DQK_F32,
                               ws, ws_size)
    torch.cuda.synchronize()
    assert Q.dqk_last_device_error() == Q.DQK_ERR_DEVICE_BOUNDS
    assert (ws[ws_size:] == 0x5A).all()
    one = R.Lists("bf16", [[300]], 8, 1, 128, seed=9)       # the next call is not affected
    got, = [one.cross(q[:40], "bf16", [0, 40])]
    torch.cuda.synchronize()
    assert Q.dqk_last_device_error() == Q.DQK_OK
    got = got[0] if isinstance(got, tuple) else got
    assert torch.isfinite(got.float()).all()
