"""Failure detection of the row attention on the GPU, without faulting or
hanging it: dqk_test_prefix_stall leaves one stage unfilled and bounds every
wait by 1 ms.  All roles of that CTA end, the launch completes, the device
error word reads DQK_ERR_TIMEOUT, and the next ordinary call on the same
workspace gives the same bytes as before."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import rows_ref as R  # noqa: E402
from bit_kv_cache_dqk_b200 import dualqk as Q  # noqa: E402
from test_gpu_rows import queries  # noqa: E402

pytestmark = pytest.mark.gpu


# units of both warpgroups (more than 128 row heads), and of one and the other
@pytest.mark.parametrize("out_dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [3, 50], ids=["in-turn", "both"])
@pytest.mark.parametrize("cache", ["int2", "bf16"])
def test_unfilled_stage_reports_timeout_and_the_next_call_is_exact(cache, rows, out_dtype):
    # some 8 units of 128 tokens on every CTA
    L = R.Lists(cache, [[20000], [i % 40 for i in range(rows)]], 32, 8, 128, seed=61)
    q, start = queries(L, rows), [0, rows]
    t0, t1 = L.table_dev(0), L.table_dev(1)
    size_of = Q.dqk_prefix_decode_workspace_size if cache == "int2" else Q.dqk_bf16_prefix_decode_workspace_size
    ws = torch.zeros(size_of(L.desc, rows, 1, t0.shape[1], t1.shape[1]), dtype=torch.uint8, device=L.dev)
    ref, ref_sel = L.prefix_decode(q, "bf16", start, out_dtype=out_dtype, ws=ws)
    torch.cuda.synchronize()
    assert Q.dqk_last_device_error() == Q.DQK_OK
    qd, out, sel = R.as_dtype(q, "bf16").to(L.dev), torch.empty_like(ref), torch.empty_like(ref_sel)
    starts, lens, own = torch.tensor(start, dtype=torch.int32, device=L.dev), L.lens_dev(0), L.lens_dev(1)
    st = Q.dqk_test_prefix_stall(L.desc, int(cache == "bf16"), qd, Q.DQK_BF16, rows, 1, starts, lens, t0, t0.shape[1], own,
                                 t1, t1.shape[1], 40, out, R.lib_dtype(out_dtype), sel, ws, ws.numel())
    assert st == Q.DQK_OK                                   # the launches themselves are fine
    assert Q.dqk_last_device_error() == Q.DQK_ERR_TIMEOUT   # a bounded wait ran out
    assert Q.dqk_last_device_error() == Q.DQK_OK            # and the word was cleared
    for _ in range(2):
        got, got_sel = L.prefix_decode(q, "bf16", start, out_dtype=out_dtype, ws=ws)
        torch.cuda.synchronize()
        assert Q.dqk_last_device_error() == Q.DQK_OK
        assert torch.equal(got, ref) and torch.equal(got_sel, ref_sel)
    assert np.isfinite(ref.float().cpu().numpy()).all()
