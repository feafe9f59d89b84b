"""GPU: row starts that run backwards are reported, whatever the workspace
holds, and leave nothing behind."""
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import rows_ref as R  # noqa: E402
from bit_kv_cache_dqk_b200 import dualqk as Q  # noqa: E402
from test_gpu_rows import check_prefix, queries  # noqa: E402

pytestmark = pytest.mark.gpu

BACKWARDS = {"overlap": [0, 4, 2, 6], "descending": [6, 4, 2, 0], "one-step": [0, 3, 2, 6], "below": [0, 2, -1, 6]}


@pytest.mark.parametrize("own", [True, False])
@pytest.mark.parametrize("cache", ["int2", "bf16"])
@pytest.mark.parametrize("starts", list(BACKWARDS))
def test_prefix_starts_that_run_backwards(cache, own, starts):
    L = R.Lists(cache, [[60, 30, 200], [5, 0, 1, 9, 17, 3]], 8, 2, 128, seed=41)
    q = queries(L, 6)
    L.prefix_decode(q, "bf16", BACKWARDS[starts], own=own)
    torch.cuda.synchronize()
    assert Q.dqk_last_device_error() == Q.DQK_ERR_DEVICE_BOUNDS
    check_prefix(L, q, "bf16", [0, 2, 2, 6], own=own)   # the next call is right, and reports nothing


@pytest.mark.parametrize("starts", list(BACKWARDS))
def test_cross_starts_that_run_backwards(starts):
    L = R.Lists("bf16", [[60, 30, 200]], 8, 2, 128, seed=42)
    q = queries(L, 6)
    L.cross(q, "bf16", BACKWARDS[starts])
    assert Q.dqk_last_device_error() == Q.DQK_ERR_DEVICE_BOUNDS
    out = L.cross(q, "bf16", [0, 1, 1, 6])
    assert Q.dqk_last_device_error() == Q.DQK_OK
    for r in range(6):
        ref, bound = L.attend(L.query(q[r], "bf16", 0)[0], [L.rows[0][0 if r < 1 else 2]], "bf16", "f32")
        R.check(out[r], ref, bound, f"row {r}")


def test_starts_outside_the_rows_are_cut():
    L = R.Lists("bf16", [[60, 30]], 8, 2, 128, seed=43)
    q = queries(L, 4)
    out = L.cross(q, "bf16", [-7, 1, 1 << 30])
    assert Q.dqk_last_device_error() == Q.DQK_OK
    for r in range(4):
        ref, bound = L.attend(L.query(q[r], "bf16", 0)[0], [L.rows[0][min(r, 1)]], "bf16", "f32")
        R.check(out[r], ref, bound, f"row {r}")
