"""GPU: the shared-prefix decode over the INT2 cache with key and value
channels 0 far outside fp16's range: they are kept in BF16, which has fp32's
exponents, and count as what they are (like key channel 0 in dqk_decode).

T_K and T_Q = T_K^-T scale channel 0 by f and 1 / f, so scores stay what they
were; value channel 0 (protected) is scaled by f too.  The bounds are those of
rows_ref: relative to the terms, whatever their magnitude."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import rows_ref as R  # noqa: E402
from test_gpu_rows import check_prefix, queries  # noqa: E402

pytestmark = pytest.mark.gpu


class Scaled(R.Lists):
    def __init__(self, factor, *a, **kw):
        self.factor, self.transforms_scaled = np.float32(factor), False
        super().__init__("int2", *a, **kw)

    def _append(self, table, lens, ks, vs, dtype):
        if not self.transforms_scaled:      # the second set of lists is appended with the same ones
            self.t_k[:, 0, :] *= self.factor
            self.t_q[:, 0, :] /= self.factor
            self.tk_dev.copy_(torch.from_numpy(self.t_k))
            self.tq_dev.copy_(torch.from_numpy(self.t_q))
            self.transforms_scaled = True
        if self.v_ch0:
            for i, v in enumerate(vs):
                vs[i] = v.clone()
                vs[i][..., 0] *= float(self.factor)
        super()._append(table, lens, ks, vs, dtype)


@pytest.mark.parametrize("factor", [2.0 ** -20, 2.0 ** -60, 2.0 ** 20, 2.0 ** 60], ids=["2^-20", "2^-60", "2^20", "2^60"])
@pytest.mark.parametrize("d,gs,v_ch0", [(128, 32, 0), (128, 128, 1), (64, 32, 1), (64, 64, 0)])
def test_channel_0_of_any_magnitude(d, gs, v_ch0, factor):
    L = Scaled(factor, [[300, 18], [5, 0, 130, 16, 33]], 8, 2, d, gs=gs, v_ch0=v_ch0, seed=31)
    q = queries(L, 5, scale=2.0)
    check_prefix(L, q, "bf16", [0, 3, 5])
    check_prefix(L, q, "f32", [0, 3, 5], own=False)


@pytest.mark.parametrize("v_ch0", [0, 1])
def test_many_row_heads(v_ch0):
    """Tiles of more than 128 row heads, items that several CTAs share."""
    L = Scaled(2.0 ** -20, [[3000], [n % 9 for n in range(40)]], 16, 2, 128, v_ch0=v_ch0, seed=32)
    check_prefix(L, queries(L, 40, scale=2.0), "bf16", [0, 40])


def test_stale_channel_0_behind_the_lists():
    """Infinities and NaN in the channel 0 slots behind a list's end, and an absent page, reach nothing."""
    L = Scaled(1.0, [[37], [3, 0]], 8, 2, 128, v_ch0=1, seed=33)
    bb = L.bb
    blk = L.pool.view(L.num_pages, 2, bb)
    for table, lens in zip(L.tables, L.lens_list):
        for g, n in enumerate(lens):
            for t in range(n, R.pages(n) * 16):
                page = int(table[g, t // 16])
                k0 = 4 * 128 + 64 * 4 + 2 * (2 * (t % 8) + (t % 16) // 8)
                v0 = bb - 32 + 2 * (t % 16)
                for at, bits in ((k0, (0x80, 0x7F) if t % 2 else (0xC0, 0x7F)), (v0, (0x80, 0xFF) if t % 3 else (0xC0, 0x7F))):
                    blk[page, :, at], blk[page, :, at + 1] = bits
    check_prefix(L, queries(L, 2), "bf16", [0, 2])
