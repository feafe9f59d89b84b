"""Reference for the rotated appends, the shared-prefix decode and the cross
attention, in numpy float64, with the error bounds the kernels' formats allow.

Rounding to a type is off by at most half a step: 2^-8 of the value for BF16,
2^-11 for fp16, 2^-24 for fp32 (U below).  With softmax weights w_t, values
v_t and scores off by at most e, an output is off by at most
    (exp(2e) - 1) (sum_t w_t |v_t| + |o|)        scores
  + (u_p + u_v) sum_t w_t |v_t|                  rounded weights, values
  + u_out |o|                                    rounded output
and scores are off by at most
    e = (u_q + u_k + (d + 8) 2^-24) sum_c |q_c k_c| / sqrt(d) + 2^-20
(the operands' rounding; d fp32 additions and a few fp32 operations after
them; 2^-22 relative error of the hardware's 2^x).  fp32 sums of the weights
and of the weighted values and the merge of records add less than
(tokens + 64) 2^-24 of the sums, which is added to u_p.
"""
from __future__ import annotations

import numpy as np
import torch

from bit_kv_cache_dqk_b200 import dualqk as Q
from oracle import oracle as O

PAGE = 16
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}


def pages(n):
    return -(-n // PAGE)


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).float().numpy()


def as_dtype(x, dtype):
    """fp32 values as the library's input of that type: a tensor of it."""
    t = torch.from_numpy(np.ascontiguousarray(x, np.float32))
    return t.to(torch.bfloat16) if dtype == "bf16" else t


def lib_dtype(dtype):
    return Q.DQK_BF16 if dtype == "bf16" else Q.DQK_F32


def dequant(c, v_ch0):
    """(k^, v^) [n][hkv][d] of an oracle cache."""
    out = []
    for pre, prot in (("k", True), ("v", v_ch0)):
        codes = c[pre + "codes"].astype(np.float64)
        gs = codes.shape[-1] // c[pre + "scale"].shape[-1]
        s, m = (np.repeat(c[pre + f].view(np.float16).astype(np.float64), gs, -1) for f in ("scale", "min"))
        x = m + codes * s
        if prot:
            x[..., 0] = (c[pre + "ch0"].astype(np.uint32) << 16).view(np.float32)
        out.append(x)
    return out


class Lists:
    """Token lists (prefixes, own contexts or encoder states) of one layer in one
    pool, appended through the library, every page at a random place and all
    other memory filled with 0xFF (NaN)."""

    def __init__(self, cache, lens_list, hq, hkv, d, dtype="bf16", gs=32, v_ch0=0, seed=0, spare=2, pool_pages=None,
                 k_scale=1.0):
        self.cache, self.hq, self.hkv, self.d, self.gs, self.v_ch0 = cache, hq, hkv, d, gs, v_ch0
        self.rng = rng = np.random.default_rng([seed, 77])
        self.dev = torch.device("cuda:0")
        counts = [[pages(n) for n in lens] for lens in lens_list]
        total = sum(sum(c) for c in counts) + spare
        self.num_pages = pool_pages or total
        perm = rng.permutation(total) + (self.num_pages - total)
        self.t_k = np.eye(d, dtype=np.float32)[None] + 0.1 * rng.standard_normal((hkv, d, d)).astype(np.float32)
        self.t_q = np.ascontiguousarray(np.linalg.inv(self.t_k.astype(np.float64)).transpose(0, 2, 1)).astype(np.float32)
        self.tk_dev, self.tq_dev = (torch.from_numpy(x).to(self.dev) for x in (self.t_k, self.t_q))
        probe = Q.layer_desc(d, hq, hkv, 0, 0, 0, 1, v_ch0_protect=v_ch0, group_size=gs)
        self.bb = Q.dqk_block_bytes(probe) if cache == "int2" else Q.dqk_bf16_block_bytes(probe)
        self.pool = torch.full((self.num_pages * hkv * self.bb,), 0xFF, dtype=torch.uint8, device=self.dev)
        self.desc = Q.layer_desc(d, hq, hkv, self.tk_dev, self.tq_dev, self.pool, self.num_pages, v_ch0_protect=v_ch0,
                                 group_size=gs)
        self.lens_list, self.tables, self.rows = lens_list, [], []
        at = 0
        for lens, cnt in zip(lens_list, counts):
            table = np.full((max(1, len(lens)), max(1, max(cnt, default=1))), -1, np.int32)
            for i, n in enumerate(cnt):
                table[i, :n] = perm[at:at + n]
                at += n
            self.tables.append(table)
            ks = [as_dtype(rng.standard_normal((n, hkv, d)) * k_scale, dtype) for n in lens]
            vs = [as_dtype(rng.standard_normal((n, hkv, d)), dtype) for n in lens]
            self._append(table, lens, ks, vs, dtype)
            self.rows.append([self._stored(k.float().numpy(), v.float().numpy()) for k, v in zip(ks, vs)])

    def _append(self, table, lens, ks, vs, dtype):
        if not sum(lens):
            return
        k, v = torch.cat(ks).to(self.dev), torch.cat(vs).to(self.dev)
        new = torch.tensor(lens, dtype=torch.int32, device=self.dev)
        fn = Q.dqk_append if self.cache == "int2" else Q.dqk_bf16_append
        fn(self.desc, k, v, lib_dtype(dtype), len(lens), new, torch.zeros_like(new), max(lens),
           torch.from_numpy(table).to(self.dev), table.shape[1])
        torch.cuda.synchronize()

    def _stored(self, k, v):
        if self.cache == "bf16":
            return bf16(k).astype(np.float64), bf16(v).astype(np.float64)
        return dequant(O.append(self.t_k, k, v, v_ch0=bool(self.v_ch0), gs=self.gs), bool(self.v_ch0))

    def table_dev(self, i):
        return torch.from_numpy(self.tables[i]).to(self.dev)

    def lens_dev(self, i):
        return torch.tensor(self.lens_list[i], dtype=torch.int32, device=self.dev)

    def prefix_decode(self, q, dtype, start, pct=40, out_dtype="f32", own=True, ws=None, out=None, stream=None, **over):
        """One call over lists 0 (prefixes) and 1 (own); returns (out, sel) on the device."""
        b = q.shape[0]
        qd = as_dtype(q, dtype).to(self.dev)
        t0, t1 = over.get("table", self.table_dev(0)), self.table_dev(1)
        own_pages = t1.shape[1] if own else 0
        size_of = Q.dqk_prefix_decode_workspace_size if self.cache == "int2" else Q.dqk_bf16_prefix_decode_workspace_size
        size = size_of(self.desc, b, t0.shape[0], t0.shape[1], own_pages)
        assert size > 0
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=self.dev) if ws is None else ws
        out = torch.full((b, self.hq, self.d), float("nan"), device=self.dev,
                         dtype=torch.bfloat16 if out_dtype == "bf16" else torch.float32) if out is None else out
        keep = O.n_keep(self.d, pct)
        sel = torch.full((b, self.hq, keep), -1, dtype=torch.int16, device=self.dev)
        common = (self.desc, qd, lib_dtype(dtype), b, t0.shape[0], torch.tensor(start, dtype=torch.int32, device=self.dev),
                  over.get("lens", self.lens_dev(0)), t0, t0.shape[1], self.lens_dev(1) if own else None,
                  t1 if own else None, own_pages)
        if self.cache == "int2":
            Q.dqk_prefix_decode(*common, pct, out, lib_dtype(out_dtype), sel, ws, size, stream=stream)
        else:
            Q.dqk_bf16_prefix_decode(*common, out, lib_dtype(out_dtype), ws, size, stream=stream)
        self.keep_alive = (qd, t0, t1, ws) + common
        return out, sel

    def cross(self, q, dtype, q_start, out_dtype="f32", out=None, **over):
        rows = q.shape[0]
        qd = as_dtype(q, dtype).to(self.dev)
        t0 = over.get("table", self.table_dev(0))
        size = Q.dqk_bf16_cross_attention_workspace_size(self.desc, len(q_start) - 1, rows, t0.shape[1])
        assert size > 0
        ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=self.dev)
        out = torch.full((rows, self.hq, self.d), float("nan"), device=self.dev,
                         dtype=torch.bfloat16 if out_dtype == "bf16" else torch.float32) if out is None else out
        Q.dqk_bf16_cross_attention(self.desc, qd, lib_dtype(dtype), len(q_start) - 1, rows,
                                   torch.tensor(q_start, dtype=torch.int32, device=self.dev),
                                   over.get("lens", self.lens_dev(0)), t0, t0.shape[1], out, lib_dtype(out_dtype), ws, size)
        torch.cuda.synchronize()
        return out

    def query(self, q, dtype, pct):
        """Effective query rows [hq][d] (transformed and cut, INT2) and kept channels."""
        x = as_dtype(q, dtype).float().numpy()
        if self.cache == "bf16":
            return x.astype(np.float64), None
        g = self.hq // self.hkv
        out, sels = np.zeros((self.hq, self.d)), []
        for h in range(self.hq):
            qp, sel = O.qprep(self.t_q[h // g], x[h], pct)
            out[h, sel.astype(np.int64)] = qp[sel.astype(np.int64)]
            sels.append(sel)
        return out, np.stack(sels)

    def attend(self, qe, parts, dtype, out_dtype):
        """(out, bound) [hq][d] of effective queries over the concatenated parts."""
        k = np.concatenate([p[0] for p in parts])
        v = np.concatenate([p[1] for p in parts])
        out, bound = np.zeros((self.hq, self.d)), np.zeros((self.hq, self.d))
        if not len(k):
            return out, bound
        g, d = self.hq // self.hkv, self.d
        f = "f16" if self.cache == "int2" else "bf16"
        u_q = U["f16"] if self.cache == "int2" else (0.0 if dtype == "bf16" else U["bf16"] ** 2)
        u_kv = U["f16"] if self.cache == "int2" else 0.0
        for h in range(self.hq):
            kj, vj = k[:, h // g], v[:, h // g]
            s = kj @ qe[h] / np.sqrt(d)
            mass = np.abs(kj) @ np.abs(qe[h]) / np.sqrt(d)
            w = np.exp(s - s.max())
            w /= w.sum()
            o = w @ vj
            e = ((u_q + u_kv + (d + 8) * U["f32"]) * mass + 2.0 ** -20).max()
            a = w @ np.abs(vj)
            out[h] = o
            bound[h] = (np.expm1(2 * e) * (a + np.abs(o)) + (U[f] + u_kv + (len(k) + 64) * U["f32"]) * a
                        + U[out_dtype] * np.abs(o))
        return out, bound


def check(got, ref, bound, what=""):
    got = got.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all(), f"{what}: not finite"
    off = np.abs(got - ref)
    worst = (off / np.maximum(bound, 1e-30)).max() if (bound > 0).any() else 0.0
    assert (off <= bound).all(), f"{what}: {worst:.2f} times the bound, max abs {off.max():.2e}"
    return worst


def rope_table(positions, rotary, theta=5e5):
    inv = theta ** (-np.arange(rotary // 2) * 2.0 / rotary)
    ang = np.arange(positions, dtype=np.float64)[:, None] * inv
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)


def rotate(x, cs, rotary, interleaved):
    """x [rows][heads][d] (fp32 values) turned by cs [rows][rotary], in float64."""
    y = x.astype(np.float64).copy()
    h = rotary // 2
    a = np.arange(h) * 2 if interleaved else np.arange(h)
    b = a + (1 if interleaved else h)
    c, s = cs[:, None, :h].astype(np.float64), cs[:, None, h:].astype(np.float64)
    xa, xb = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    return y
