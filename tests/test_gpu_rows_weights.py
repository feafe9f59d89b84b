"""GPU: fp32 outputs of the shared-prefix decode and the cross attention over
the BF16 cache keep the bits of dqk_bf16_decode: softmax weights as BF16 high
+ low parts.

Bound, by the formats: a weight is hi + lo with |p - hi - lo| <= 2^-8 2^-8 p;
scores are exact products of BF16 values (fp32 queries: hi + lo, 2^-16) summed
in fp32; an fp32 addition of the matrix unit may truncate, so a sum of n terms
is off by at most n 2^-23 of the sum of magnitudes, and there are two products
per term of a pair hi, lo.  With m = sum_c |q_c k_c| / sqrt(d), a = sum_t w_t |v_t|:
    e   = (u_q + (2 d + 16) 2^-23) m + 2^-20
    off = (exp(2 e) - 1) (a + |o|) + (2^-16 + (2 n + 64) 2^-23) a + 2^-24 |o|
The queries are small (m well below 1) and the lists short, so that this is
far below what weights of 8 bits would leave, 2^-8 a / sqrt(n).
"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA device", allow_module_level=True)

import rows_ref as R  # noqa: E402
from bit_kv_cache_dqk_b200 import dualqk as Q  # noqa: E402
from test_gpu_rows import queries  # noqa: E402

pytestmark = pytest.mark.gpu


def attend(L, q, parts, dtype):
    k = np.concatenate([p[0] for p in parts])
    v = np.concatenate([p[1] for p in parts])
    x = R.as_dtype(q, dtype).float().numpy().astype(np.float64)
    out, off = np.zeros((L.hq, L.d)), np.zeros((L.hq, L.d))
    for h in range(L.hq):
        j = h // (L.hq // L.hkv)
        s = k[:, j] @ x[h] / np.sqrt(L.d)
        m = (np.abs(k[:, j]) @ np.abs(x[h]) / np.sqrt(L.d)).max()
        w = np.exp(s - s.max())
        w /= w.sum()
        o, a = w @ v[:, j], w @ np.abs(v[:, j])
        e = ((2.0 ** -16 if dtype == "f32" else 0.0) + (2 * L.d + 16) * 2.0 ** -23) * m + 2.0 ** -20
        out[h] = o
        off[h] = np.expm1(2 * e) * (a + np.abs(o)) + (2.0 ** -16 + (2 * len(k) + 64) * 2.0 ** -23) * a + 2.0 ** -24 * np.abs(o)
    return out, off


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (16, 2, 64), (3, 3, 128)])
def test_prefix_decode_keeps_the_bits_of_fp32_outputs(hq, hkv, d, dtype):
    start, prefix, own = [0, 2, 2, 5], [17, 3, 40], [0, 9, 1, 16, 5]
    L = R.Lists("bf16", [prefix, own], hq, hkv, d, dtype=dtype, seed=21)
    q = queries(L, len(own), scale=0.05)
    out, _ = L.prefix_decode(q, dtype, start)
    alone, _ = L.prefix_decode(q, dtype, start, own=False)
    assert Q.dqk_last_device_error() == Q.DQK_OK
    for b, g in enumerate([0, 0, 2, 2, 2]):
        R.check(out[b], *attend(L, q[b], [L.rows[0][g], L.rows[1][b]], dtype), f"sequence {b}")
        R.check(alone[b], *attend(L, q[b], [L.rows[0][g]], dtype), f"sequence {b}, prefix alone")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (8, 1, 64)])
def test_cross_attention_keeps_the_bits_of_fp32_outputs(hq, hkv, d, dtype):
    nq, nkv = [1, 50, 3], [12, 30, 7]
    L = R.Lists("bf16", [nkv], hq, hkv, d, dtype=dtype, seed=22)
    start = np.concatenate([[0], np.cumsum(nq)]).tolist()
    q = queries(L, start[-1], scale=0.05)
    out = L.cross(q, dtype, start)
    assert Q.dqk_last_device_error() == Q.DQK_OK
    for b in range(3):
        for r in range(start[b], start[b + 1]):
            R.check(out[r], *attend(L, q[r], [L.rows[0][b]], dtype), f"row {r}")


def test_moved_references_keep_the_bits():
    """The reference of a row moves inside the list: both parts of the weights follow it."""
    L = R.Lists("bf16", [[200]], 8, 2, 128, seed=23)
    q = queries(L, 2, scale=0.02) * np.linspace(1, 2, 8)[None, :, None].astype(np.float32)
    blk = L.pool.view(torch.bfloat16).view(L.num_pages, 2, 2, 16, 128)
    for t in range(200):
        x = torch.full((128,), 4.0 * (t // 40), dtype=torch.bfloat16, device=L.dev)   # equal channels: chunk order does not matter
        blk[int(L.tables[0][0, t // 16]), :, 0, t % 16] = x
        L.rows[0][0][0][t] = float(x[0])
    q = np.abs(q) + 0.02
    out = L.cross(q, "bf16", [0, 2])
    for r in range(2):
        R.check(out[r], *attend(L, q[r], [L.rows[0][0]], "bf16"), f"row {r}")
