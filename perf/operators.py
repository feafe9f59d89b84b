"""Cases of the rotated appends, the shared-prefix decode and the cross
attention of the paged KV caches: inputs, plain forms, the library's calls, and
the definitions in 64 bits.

The two caches hold pages of 16 tokens, one block per (page, kv head):

* BF16 block: K [16][d] then V [16][d], the 16-byte chunk x of token t at chunk
  x ^ (t % 8);
* INT2 block: K codes, K scale and min (fp16), K channel 0 (BF16), V codes, V
  scale and min, in the order include/dualqk.h documents.

Lengths are a function of the case alone (a golden-ratio sequence), values of
the seed.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
DEV = "cuda"


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _rope(op, batch, new_lo, new_hi, ctx, **kw):
    c = dict(op=op, batch=batch, new_lo=new_lo, new_hi=new_hi, ctx=ctx, base=0, rotary=128, interleaved=False,
             fused=True, hq=32, hkv=8, d=128, dtype="bf16")
    if op == "rope_int2":
        c.update(group_size=32, v_ch0=0)
    c.update(kw)
    return c


def _prefix(op, batch, prefixes, prefix, own_len, **kw):
    c = dict(op=op, batch=batch, prefixes=prefixes, prefix=prefix, own=own_len, hq=32, hkv=8, d=128, dtype="bf16")
    if op == "prefix_int2":
        c.update(pct=40, group_size=32, v_ch0=0)
    c.update(kw)
    return c


def _cross(batch, q, kv, **kw):
    c = dict(op="cross", batch=batch, q=q, kv=kv, hq=32, hkv=8, d=128, dtype="bf16")
    c.update(kw)
    return c


def listed():
    return [
        # one decode step of a small batch: each sequence's new token enters the BF16 cache, latency alone
        dict(_rope("rope_bf16", 8, 1, 1, 1000), name="rope_bf16_step"),
        # prompts of several sequences at once, q, k and v slices of one projection's rows
        dict(_rope("rope_bf16", 4, 4096, 8192, 0), name="rope_bf16_prompt"),
        # one decode step behind a shared prefix (positions differ from the cache slots), INT2 cache
        dict(_rope("rope_int2", 16, 1, 1, 1000, base=32768), name="rope_int2_step"),
        # 64 rows for each of 16 sequences: the appends of the ragged workload, chunked prompts
        dict(_rope("rope_int2", 16, 64, 64, 4001), name="rope_int2_rows"),
        # the tiny layer: four queries over one context of 1024 tokens, one head, fp32
        dict(_prefix("prefix_int2", 4, 1, 1024, 40, hq=1, hkv=1, d=64, dtype="f32"), name="prefix_int2_tiny"),
        # a chat batch behind one system prompt
        dict(_prefix("prefix_int2", 16, 1, 8192, 1000), name="prefix_int2_chat"),
        # many samples of one 128K document
        dict(_prefix("prefix_int2", 64, 1, 131072, 700), name="prefix_int2_document"),
        # a few sequences behind a few hundred shared tokens, BF16 cache
        dict(_prefix("prefix_bf16", 3, 1, 300, 37, hq=8, hkv=4), name="prefix_bf16_short"),
        # two documents of 32K tokens, a dozen and a half samples each
        dict(_prefix("prefix_bf16", 32, 2, 32768, 1500), name="prefix_bf16_documents"),
        # decoder steps over encoder states: one query token each
        dict(_cross(16, 1, 1500), name="cross_step"),
        # whole decoder sequences over long encoder states: compute-bound
        dict(_cross(4, 1024, 4096), name="cross_sequences"),
        # odd lengths, 64-channel heads, fp32 queries
        dict(_cross(7, 77, 1213, hq=16, hkv=2, d=64, dtype="f32"), name="cross_ragged"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope_bf16", "rope_int2", "prefix_int2", "prefix_int2", "prefix_bf16", "cross", "cross"])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 5, 8])
    heads = dict(hkv=hkv, hq=hkv * rng.choice([1, 2, 4, 8]), d=d, dtype=rng.choice(["bf16", "bf16", "f32"]))
    if heads["hq"] > 32:
        heads["hq"] = 4 * hkv
    if op.startswith("rope"):
        batch = _log(rng, 1, 64)
        most = 8192 if op == "rope_bf16" else 2048
        hi = _log(rng, 1, max(1, most // batch))
        kw = dict(heads, base=rng.choice([0, _log(rng, 1, 131072)]), rotary=rng.choice([d, d, d // 2]),
                  interleaved=rng.random() < 0.4, fused=rng.random() < 0.7)
        if op == "rope_int2":
            kw.update(group_size=rng.choice([32, d]), v_ch0=rng.choice([0, 0, 1]))
        return _rope(op, batch, rng.choice([0, 1, hi]), hi, rng.randint(0, 1500), **kw)
    if op.startswith("prefix"):
        batch = _log(rng, 1, 64)
        prefix = _log(rng, 1, max(64, min(65536, (1 << 22) // batch)))
        own_len = rng.choice([0, _log(rng, 1, max(16, min(3000, 65536 // batch)))])
        kw = dict(heads)
        if op == "prefix_int2":
            kw.update(pct=rng.choice([0, 20, 40, 60]), group_size=rng.choice([32, d]), v_ch0=rng.choice([0, 0, 1]))
        return _prefix(op, batch, rng.choice([1, 1, 2, 3]), prefix, own_len, **kw)
    batch = _log(rng, 1, 32)
    q = _log(rng, 1, max(1, 2048 // batch))
    return _cross(batch, q, _log(rng, 1, max(64, min(16384, (1 << 22) // (batch * q)))), **heads)


def _spread(lo, hi, n, phase):
    """n lengths in [lo, hi], the first one hi."""
    return [hi if i == 0 else lo + int((hi - lo + 1) * ((phase + i * 0.6180339887498949) % 1.0)) for i in range(n)]


def _lens(c):
    """The case's lengths: new and cached tokens of an append, the groups and
    lengths of a prefix decode, or the query and state counts."""
    if c["op"].startswith("rope"):
        return dict(new=_spread(c["new_lo"], c["new_hi"], c["batch"], 0.3),
                    before=_spread(c["ctx"] // 2, c["ctx"], c["batch"], 0.7))
    if c["op"].startswith("prefix"):
        n = min(c["prefixes"], c["batch"])
        start = [0]
        for g in range(n):   # uneven groups, at least one sequence each
            left = c["batch"] - start[-1] - (n - 1 - g)
            start.append(start[-1] + (left if g == n - 1 else max(1, int(left * 0.45))))
        return dict(start=start, prefix=_spread(c["prefix"] // 2 + 1, c["prefix"], n, 0.1),
                    own=_spread(0, c["own"], c["batch"], 0.4))
    return dict(q=_spread(c["q"] // 2 + 1 if c["q"] > 1 else 1, c["q"], c["batch"], 0.2),
                kv=_spread(c["kv"] // 2, c["kv"], c["batch"], 0.8))


# ---------------------------------------------------------------------------
# work: every input read once, every output written once
# ---------------------------------------------------------------------------
def _token_bytes(c):
    """Cache bytes of one token of one kv head."""
    if c["op"].endswith("int2"):
        return c["d"] // 2 + 8 * (c["d"] // c["group_size"]) + 2 + 2 * c["v_ch0"]
    return 4 * c["d"]


def work(case):
    c, n = case, _lens(case)
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"].startswith("rope"):
        rows = sum(n["new"])
        byte = rows * (e * c["d"] * (2 * c["hkv"] + 2 * c["hq"]) + 4 * c["rotary"] + c["hkv"] * _token_bytes(c))
        flop = rows * 3 * c["rotary"] * (c["hkv"] + c["hq"])
        if c["op"] == "rope_int2":
            byte += 4 * c["hkv"] * c["d"] ** 2
            flop += rows * c["hkv"] * 2 * c["d"] ** 2
        return {"bytes": byte, "flops": flop}
    if c["op"].startswith("prefix"):
        seqs = [b - a for a, b in zip(n["start"], n["start"][1:])]
        tokens = sum(n["prefix"]) + sum(n["own"])
        pairs = (sum(p * s for p, s in zip(n["prefix"], seqs)) + sum(n["own"])) * c["hq"]
        rows = c["batch"] * c["hq"]
        keep = c["d"] - (c["pct"] * c["d"]) // 100 if "pct" in c else c["d"]
        byte = tokens * c["hkv"] * _token_bytes(c) + rows * c["d"] * (e + 2)
        flop = pairs * 2 * (keep + c["d"])
        if c["op"] == "prefix_int2":
            byte += 4 * c["hkv"] * c["d"] ** 2 + 2 * rows * keep
            flop += rows * 2 * c["d"] ** 2
        return {"bytes": byte, "flops": flop}
    rows, pairs = sum(n["q"]) * c["hq"], sum(a * b for a, b in zip(n["q"], n["kv"])) * c["hq"]
    return {"bytes": sum(n["kv"]) * c["hkv"] * _token_bytes(c) + rows * c["d"] * (e + 2), "flops": pairs * 4 * c["d"]}


# ---------------------------------------------------------------------------
# layout of the INT2 blocks
# ---------------------------------------------------------------------------
def _int2_layout(c):
    d, ns = c["d"], c["d"] // c["group_size"]
    ks = 4 * d
    km = ks + 32 * ns
    k0 = km + 32 * ns
    vc = k0 + 32
    vs = vc + 4 * d
    vm = vs + 32 * ns
    v0 = vm + 32 * ns
    return dict(ks=ks, km=km, k0=k0, vc=vc, vs=vs, vm=vm, v0=v0, bytes=v0 + (32 if c["v_ch0"] else 0), ns=ns)


_TABLES = {}


def _code_places(d):
    """Place (in 2-bit fields from the section's start) of the K and of the V
    code of (token, channel), as device index tensors [16][d]."""
    if d not in _TABLES:
        ng = d // 32
        t, ch = np.meshgrid(np.arange(16), np.arange(d), indexing="ij")
        g, cc = ch // 32, ch % 32
        r = 2 * (cc // 16) + t // 8
        lane = 4 * (t % 8) + (cc % 16) // 4
        kp = 16 * (lane * ng + r % ng) + 4 * (cc % 4) + g + ng * (r // ng)
        m, cr = ch // 16, (ch % 16) // 8
        lane = 4 * (ch % 8) + (t % 8) // 2
        if ng == 4:
            w, i = cr + 2 * (t // 8), m
        else:
            n = (2 * m + cr) * 2 + t // 8
            w, i = n // 8, n % 8
        vp = 16 * (lane * ng + w) + 8 * (t % 2) + i
        tt = np.arange(16)
        gg = np.arange(d)[None, :]
        _TABLES[d] = tuple(torch.from_numpy(x).to(DEV) for x in (kp, vp, 2 * (tt % 8) + tt // 8)) + (gg,)
    return _TABLES[d][:3]


def _v_scale_places(ns):
    t, g = np.meshgrid(np.arange(16), np.arange(ns), indexing="ij")
    return torch.from_numpy(2 * (ns * (t // 2) + g) + t % 2).to(DEV)


def _pack_codes(codes, place):
    """[..., 16, d] codes 0..3 -> [..., 4d] bytes."""
    flat = torch.empty(codes.shape[:-2] + (16 * codes.shape[-1],), dtype=torch.uint8, device=codes.device)
    flat[..., place.reshape(-1)] = codes.reshape(flat.shape)
    f = flat.view(flat.shape[:-1] + (-1, 4))
    return f[..., 0] | (f[..., 1] << 2) | (f[..., 2] << 4) | (f[..., 3] << 6)


def _unpack_codes(byte, place):
    sh = torch.tensor([0, 2, 4, 6], dtype=torch.uint8, device=byte.device)
    f = ((byte[..., None] >> sh) & 3).reshape(byte.shape[:-1] + (-1,))
    return f[..., place.reshape(-1)].reshape(byte.shape[:-1] + tuple(place.shape))


def _bytes_of(x):
    return x.contiguous().view(torch.uint8)


def _pack_int2(c, f):
    """Fields of whole pages ([n][hkv][16][...]) -> blocks [n][hkv][bytes]."""
    lay, (kp, vp, k0p) = _int2_layout(c), _code_places(c["d"])
    ns, vsp = lay["ns"], _v_scale_places(lay["ns"])
    n, h = f["kcodes"].shape[:2]
    out = torch.zeros((n, h, lay["bytes"]), dtype=torch.uint8, device=DEV)
    out[..., :lay["ks"]] = _pack_codes(f["kcodes"], kp)
    out[..., lay["ks"]:lay["km"]] = _bytes_of(f["kscale"].reshape(n, h, 16 * ns))
    out[..., lay["km"]:lay["k0"]] = _bytes_of(f["kmin"].reshape(n, h, 16 * ns))
    k0 = torch.empty_like(f["kch0"])
    k0[..., k0p] = f["kch0"]
    out[..., lay["k0"]:lay["vc"]] = _bytes_of(k0)
    out[..., lay["vc"]:lay["vs"]] = _pack_codes(f["vcodes"], vp)
    for key, at in (("vscale", lay["vs"]), ("vmin", lay["vm"])):
        x = torch.empty((n, h, 16 * ns), dtype=torch.float16, device=DEV)
        x[..., vsp.reshape(-1)] = f[key].reshape(n, h, 16 * ns)
        out[..., at:at + 32 * ns] = _bytes_of(x)
    if c["v_ch0"]:
        out[..., lay["v0"]:] = _bytes_of(f["vch0"])
    return out


def _unpack_int2(c, blocks):
    """Blocks [..., hkv, bytes] -> fields [..., hkv, 16, ...]."""
    lay, (kp, vp, k0p) = _int2_layout(c), _code_places(c["d"])
    ns, vsp = lay["ns"], _v_scale_places(lay["ns"])
    lead = blocks.shape[:-1]

    def half(a, b, dt=torch.float16):
        return blocks[..., a:b].contiguous().view(dt)

    f = dict(kcodes=_unpack_codes(blocks[..., :lay["ks"]], kp), vcodes=_unpack_codes(blocks[..., lay["vc"]:lay["vs"]], vp),
             kscale=half(lay["ks"], lay["km"]).reshape(lead + (16, ns)), kmin=half(lay["km"], lay["k0"]).reshape(lead + (16, ns)),
             kch0=half(lay["k0"], lay["vc"], torch.bfloat16)[..., k0p],
             vscale=half(lay["vs"], lay["vm"])[..., vsp.reshape(-1)].reshape(lead + (16, ns)),
             vmin=half(lay["vm"], lay["v0"])[..., vsp.reshape(-1)].reshape(lead + (16, ns)))
    if c["v_ch0"]:
        f["vch0"] = half(lay["v0"], lay["bytes"], torch.bfloat16)
    return f


def _half_nearest(x):
    """float64 -> float16, one rounding to nearest even, saturating at the
    largest finite value (a cast rounds to float32 on the way)."""
    _, e = torch.frexp(x)
    step = torch.ldexp(torch.ones_like(x), torch.clamp(e - 11, min=-24))
    return torch.clamp(torch.round(x / step) * step, -65504.0, 65504.0).to(torch.float16)


def _quantize(x, group_size, protect):
    """fp32 rows [..., d] -> codes, scale, min, channel 0 (the cache's INT2 format)."""
    d = x.shape[-1]
    ch0 = x[..., 0].to(torch.bfloat16)
    g = (x + 0.0).double().reshape(x.shape[:-1] + (d // group_size, group_size))
    lo_in, hi_in = g, g
    if protect:
        first = torch.zeros((d // group_size, group_size), dtype=torch.bool, device=x.device)
        first[0, 0] = True
        lo_in, hi_in = g.masked_fill(first, math.inf), g.masked_fill(first, -math.inf)
    lo, hi = lo_in.amin(-1), hi_in.amax(-1)
    scale, mn = _half_nearest((hi - lo) / 3.0), _half_nearest(lo)
    s = scale.double()[..., None]
    code = torch.clamp(torch.round((g - mn.double()[..., None]) / torch.where(s == 0, torch.ones_like(s), s)), 0, 3)
    code = torch.where(s == 0, torch.zeros_like(code), code).to(torch.uint8).reshape(x.shape)
    if protect:
        code[..., 0] = 0
    return code, scale, mn, ch0


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 17)


def _randn(shape, g):
    return torch.randn(shape, generator=g, device=DEV)


def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _outliers(c, g):
    """Gains of the raw keys: four channels of each kv head stand out."""
    gain = torch.ones((c["hkv"], c["d"]), device=DEV)
    at = torch.rand((c["hkv"], c["d"]), generator=g, device=DEV).argsort(-1)[:, :4]
    return gain.scatter_(1, at, 15.0)


def _kv_rows(c, n, g, gain):
    """n tokens of keys and values in the form the cache stands for: BF16 values,
    or the fields of the INT2 format.  Keys of the INT2 cache are already in the
    transformed basis, where the outliers are flattened."""
    k = _randn((n, c["hkv"], c["d"]), g)
    v = _randn((n, c["hkv"], c["d"]), g)
    if not c["op"].endswith("int2"):
        return dict(k=(k * (1.0 + (gain - 1.0) * 0.1)).to(torch.bfloat16), v=v.to(torch.bfloat16))
    f = {}
    f["kcodes"], f["kscale"], f["kmin"], f["kch0"] = _quantize(k * gain.sqrt(), c["group_size"], True)
    f["vcodes"], f["vscale"], f["vmin"], ch0 = _quantize(v, c["group_size"], bool(c["v_ch0"]))
    if c["v_ch0"]:
        f["vch0"] = ch0
    return f


def _pages(lens):
    return [-(-n // PAGE) for n in lens]


def _tables(lens_list, g):
    """Page tables of several lists of lengths over one pool in random order."""
    counts = [_pages(lens) for lens in lens_list]
    total = max(1, sum(sum(x) for x in counts))
    perm = torch.rand(total, generator=g, device=DEV).argsort().to(torch.int32).cpu().numpy()
    out, at = [], 0
    for x in counts:
        table = np.full((len(x), max(1, max(x))), -1, np.int32)
        for i, n in enumerate(x):
            table[i, :n] = perm[at:at + n]
            at += n
        out.append(table)
    return out, total


def _as_pages(c, x, lens):
    """Rows of sequences one after the other ([tokens][...]) -> the pages of
    all sequences in order, the tokens behind a sequence's end filled with
    bytes of ones (stale memory)."""
    pages = _pages(lens)
    dst = np.concatenate([np.arange(n) + PAGE * sum(pages[:i]) for i, n in enumerate(lens)]) if sum(lens) else np.zeros(0, np.int64)
    byte = x.contiguous().view(torch.uint8).flatten(1)
    out = torch.full((max(1, sum(pages)) * PAGE, byte.shape[1]), 3 if x.dtype == torch.uint8 else 255, dtype=torch.uint8, device=DEV)
    out[torch.from_numpy(dst).to(DEV)] = byte
    return out.view(x.dtype).reshape((-1, PAGE) + tuple(x.shape[1:])).transpose(1, 2)   # [pages][hkv][16]...


def _bf16_chunks(x):
    """[n][16][d] rows <-> the same rows with chunk x of token t at x ^ (t % 8) (its own inverse)."""
    d = x.shape[-1]
    t, ch = np.meshgrid(np.arange(16), np.arange(d), indexing="ij")
    src = ((ch // 8) ^ (t % 8)) * 8 + ch % 8
    return torch.gather(x, -1, torch.from_numpy(src).to(x.device).expand(x.shape))


def _fill_pool(c, total, tables, parts):
    """The pool's blocks holding `parts` (fields of the tables' sequences)."""
    int2 = c["op"].endswith("int2")
    size = _int2_layout(c)["bytes"] if int2 else 64 * c["d"]
    pool = torch.full((total, c["hkv"], size), 0xFF, dtype=torch.uint8, device=DEV)
    for table, (f, lens) in zip(tables, parts):
        if not sum(lens):
            continue
        where = torch.from_numpy(np.concatenate([table[i, :n] for i, n in enumerate(_pages(lens))]).astype(np.int64)).to(DEV)
        p = {key: _as_pages(c, x, lens) for key, x in f.items()}
        if int2:
            pool[where] = _pack_int2(c, p)
        else:
            kv = torch.stack([_bf16_chunks(p["k"]), _bf16_chunks(p["v"])], 2)
            pool[where] = kv.contiguous().view(torch.uint8).reshape(len(where), c["hkv"], size)
    return pool


def _transform(c, g):
    """fp32 [hkv][d][d], a well-conditioned mix of all channels."""
    eye = torch.eye(c["d"], device=DEV)
    return (eye + 0.1 * _randn((c["hkv"], c["d"], c["d"]), g)).contiguous()


def _rope_table(c, positions):
    """cos and sin of every position, from 64-bit angles (theta 5e5)."""
    r = c["rotary"]
    inv = 5e5 ** (-torch.arange(r // 2, dtype=torch.float64, device=DEV) * 2.0 / r)
    ang = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * inv
    return torch.cat([torch.cos(ang), torch.sin(ang)], 1).float()


def _make_rope(c, seed):
    g, n = _gen(seed), _lens(c)
    rows, dt = sum(n["new"]), _dtype(c)
    d, hq, hkv = c["d"], c["hq"], c["hkv"]
    x = _randn((max(1, rows), hq + 2 * hkv, d), g)
    x[:, hq:hq + hkv] *= _outliers(c, g)
    x = x.to(dt)
    s = dict(q=x[:rows, :hq], k=x[:rows, hq:hq + hkv], v=x[:rows, hq + hkv:])
    if not c["fused"]:
        s = {key: t.contiguous() for key, t in s.items()}
    ends = [a + b for a, b in zip(n["new"], n["before"])]
    (table,), total = _tables([ends], g)
    pos = np.concatenate([np.arange(b, b + m) for m, b in zip(n["new"], n["before"])]).astype(np.int64)
    seq = np.repeat(np.arange(c["batch"]), n["new"])
    s.update(case=c, rows=rows, new=_i32(n["new"]), before=_i32(n["before"]), max_new=max(n["new"]), table=torch.from_numpy(table).to(DEV),
             total=total, positions=torch.from_numpy((pos + c["base"]).astype(np.int32)).to(DEV),
             cos_sin=_rope_table(c, c["base"] + max(ends)), page=torch.from_numpy(table[seq, pos // PAGE].astype(np.int64)).to(DEV),
             slot=torch.from_numpy(pos % PAGE).to(DEV))
    if c["op"] == "rope_int2":
        s["t_k"] = _transform(c, g)
        # whole pages of an earlier context lie under the new rows
        s["pool"] = torch.randint(0, 256, (total, hkv, _int2_layout(c)["bytes"]), generator=g, device=DEV, dtype=torch.uint8)
        lay = _int2_layout(c)
        for a, b in ((lay["ks"], lay["vc"]), (lay["vs"], lay["bytes"])):   # finite scales, mins and channels 0
            s["pool"][..., a:b] &= 0x3F
    else:
        s["pool"] = torch.zeros((total, hkv, 2, PAGE, d), dtype=torch.bfloat16, device=DEV)
    return s


def _make_attention(c, seed):
    g, n = _gen(seed), _lens(c)
    gain = _outliers(c, g)
    if c["op"] == "cross":
        lists, rows = [n["kv"]], sum(n["q"])
    else:
        lists, rows = [n["prefix"], n["own"]], c["batch"]
    parts = [(_kv_rows(c, sum(x), g, gain), x) for x in lists]
    tables, total = _tables(lists, g)
    s = dict(case=c, lens=n, rows=rows, q=_randn((rows, c["hq"], c["d"]), g).to(_dtype(c)), parts=parts, tables=tables, total=total)
    if c["op"] == "prefix_int2":
        s["t_q"] = _transform(c, g)
    return s


def _library():
    from bit_kv_cache_dqk_b200 import dualqk
    return dualqk


def prepare(case, seed):
    c = case
    if c["op"].startswith("rope"):
        s = _make_rope(c, seed)
        s["q_out"] = torch.zeros((max(1, s["rows"]), c["hq"], c["d"]), dtype=_dtype(c), device=DEV)
    else:
        s = _make_attention(c, seed)
        parts, n = s.pop("parts"), s["lens"]
        s["pool"] = _fill_pool(c, s["total"], s["tables"], parts)
        s["tables"] = [torch.from_numpy(t).to(DEV) for t in s["tables"]]
        s["out"] = torch.zeros((s["rows"], c["hq"], c["d"]), dtype=torch.bfloat16, device=DEV)
        if c["op"] == "cross":
            s.update(q_start=_i32(np.concatenate([[0], np.cumsum(n["q"])]).tolist()), kv_lens=_i32(n["kv"]))
        else:
            s.update(start=_i32(n["start"]), prefix_lens=_i32(n["prefix"]), own_lens=_i32(n["own"]))
            if c["op"] == "prefix_int2":
                s["sel"] = torch.zeros((c["batch"], c["hq"], c["d"] - (c["pct"] * c["d"]) // 100), dtype=torch.int16, device=DEV)
    if own:
        # the layer and rope handles and the workspace, which a serving loop sets up once
        Q = _library()
        s["layer"] = Q.layer_desc(c["d"], c["hq"], c["hkv"], s.get("t_k"), s.get("t_q"), s["pool"], s["total"],
                                  v_ch0_protect=c.get("v_ch0", 0), group_size=c.get("group_size", 32))
        if c["op"].startswith("rope"):
            s["rope"] = Q.rope_desc(c["rotary"], s["cos_sin"], s["cos_sin"].shape[0], int(c["interleaved"]))
        else:
            t = s["tables"]
            if c["op"] == "cross":
                size = Q.dqk_bf16_cross_attention_workspace_size(s["layer"], c["batch"], s["rows"], t[0].shape[1])
            elif c["op"] == "prefix_int2":
                size = Q.dqk_prefix_decode_workspace_size(s["layer"], c["batch"], t[0].shape[0], t[0].shape[1], t[1].shape[1])
            else:
                size = Q.dqk_bf16_prefix_decode_workspace_size(s["layer"], c["batch"], t[0].shape[0], t[0].shape[1], t[1].shape[1])
            s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _rotated(c, x, cs):
    """x [rows][heads][d] turned by the angles of cs [rows][rotary], in cs's type."""
    r, h = c["rotary"], c["rotary"] // 2
    x = x.to(cs.dtype)
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if c["interleaved"] else (x[..., :h], x[..., h:r])
    co, si = cs[:, None, :h], cs[:, None, h:]
    y = torch.stack([a * co - b * si, b * co + a * si], -1 if c["interleaved"] else -2)
    return torch.cat([y.reshape(x.shape[:-1] + (r,)), x[..., r:]], -1)


def _plain_rope(s):
    c, rows = s["case"], s["rows"]
    cs = s["cos_sin"][s["positions"].long()]
    s["q_out"][:rows] = _rotated(c, s["q"], cs).to(s["q_out"].dtype)
    if c["op"] == "rope_bf16":
        kv = torch.stack([_rotated(c, s["k"], cs).to(torch.bfloat16), s["v"].to(torch.bfloat16)], 2)   # [rows][hkv][2][d]
        t = s["slot"]
        ch = torch.arange(c["d"], device=DEV)
        at = (((ch // 8)[None] ^ (t % 8)[:, None]) * 8 + ch % 8)[:, None, None].expand(kv.shape)
        s["pool"][s["page"], :, :, t] = torch.gather(kv, -1, at)
        return {"pool": s["pool"], "q": s["q_out"]}
    # keys: 64-bit products and sums throughout, since codes are decided by them
    k = _rotated(c, s["k"], cs.double()).float().double()
    k = torch.einsum("jci,rji->rjc", s["t_k"].double(), k).float()
    f = {}
    f["kcodes"], f["kscale"], f["kmin"], f["kch0"] = _quantize(k, c["group_size"], True)
    f["vcodes"], f["vscale"], f["vmin"], f["vch0"] = _quantize(s["v"].float(), c["group_size"], bool(c["v_ch0"]))
    pages, which = torch.unique(s["page"], return_inverse=True)
    whole = _unpack_int2(c, s["pool"][pages])
    for key in whole:
        whole[key][which, :, s["slot"]] = f[key]
    s["pool"][pages] = _pack_int2(c, whole)
    return {"pool": s["pool"], "q": s["q_out"]}


def _plain_kv(c, pool, table):
    """fp32 keys and values [lists][tokens][hkv][d] of the pages of a table."""
    blocks = pool[table.clamp(min=0).long()]                      # [n][pages][hkv][bytes]
    n, pages, d = blocks.shape[0], blocks.shape[1], c["d"]
    if c["op"].endswith("int2"):
        f = _unpack_int2(c, blocks)
        gs = c["group_size"]
        k = f["kmin"].float().repeat_interleave(gs, -1) + f["kcodes"].float() * f["kscale"].float().repeat_interleave(gs, -1)
        v = f["vmin"].float().repeat_interleave(gs, -1) + f["vcodes"].float() * f["vscale"].float().repeat_interleave(gs, -1)
        k[..., 0] = f["kch0"].float()
        if c["v_ch0"]:
            v[..., 0] = f["vch0"].float()
    else:
        kv = _bf16_chunks(blocks.view(torch.bfloat16).reshape(n, pages, c["hkv"], 2, PAGE, d))
        k, v = kv[:, :, :, 0].float(), kv[:, :, :, 1].float()
    return (x.transpose(2, 3).reshape(n, pages * PAGE, c["hkv"], d) for x in (k, v))


def _cut(x, valid):
    """Zeros (not stale memory) at the tokens behind each list's end."""
    return torch.where(valid[:, :, None, None], x, torch.zeros_like(x))


def _plain_q(s):
    """Query rows [rows][hkv][G][d], scaled; for the INT2 cache transformed and
    cut to the kept channels, and those channels."""
    c = s["case"]
    q = s["q"].reshape(s["rows"], c["hkv"], -1, c["d"])
    if c["op"] != "prefix_int2":
        return q.float() / math.sqrt(c["d"]), None
    # 64-bit sums: the kept channels are decided by them
    t = torch.einsum("jci,rjgi->rjgc", s["t_q"].double(), q.double()).float()
    keep = c["d"] - (c["pct"] * c["d"]) // 100
    order = torch.argsort(t[..., 1:].abs(), dim=-1, descending=True, stable=True)[..., :keep - 1] + 1
    sel = torch.cat([torch.zeros_like(t[..., :1], dtype=torch.int64), order], -1).sort(-1).values
    mask = torch.zeros_like(t).scatter_(-1, sel, 1.0)
    return t * mask / math.sqrt(c["d"]), sel.reshape(s["rows"], c["hq"], keep).to(torch.int16)


def _plain_prefix(s):
    c, n = s["case"], s["lens"]
    q, sel = _plain_q(s)
    pk, pv = _plain_kv(c, s["pool"], s["tables"][0])
    ok, ov = _plain_kv(c, s["pool"], s["tables"][1])
    pvalid = torch.arange(pk.shape[1], device=DEV)[None] < s["prefix_lens"][:, None]
    ovalid = torch.arange(ok.shape[1], device=DEV)[None] < s["own_lens"][:, None]
    pk, pv, ok, ov = _cut(pk, pvalid), _cut(pv, pvalid), _cut(ok, ovalid), _cut(ov, ovalid)
    # queries by group: sequence b is row b - start of its group
    b = torch.arange(c["batch"], device=DEV)
    group = torch.searchsorted(s["start"][1:].long(), b, right=True)
    row = b - s["start"].long()[group]
    most = max(y - x for x, y in zip(n["start"], n["start"][1:]))
    qg = torch.zeros((pk.shape[0], most) + tuple(q.shape[1:]), device=DEV)
    qg[group, row] = q
    sp = torch.einsum("prjgd,ptjd->prjgt", qg, pk)[group, row].masked_fill(~pvalid[group][:, None, None], -math.inf)
    so = torch.einsum("bjgd,btjd->bjgt", q, ok).masked_fill(~ovalid[:, None, None], -math.inf)
    m = torch.maximum(sp.amax(-1), so.amax(-1))
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)[..., None]
    wp, wo = torch.exp(sp - m), torch.exp(so - m)
    total = wp.sum(-1) + wo.sum(-1)
    wg = torch.zeros((pk.shape[0], most) + tuple(wp.shape[1:]), device=DEV)
    wg[group, row] = wp
    o = torch.einsum("prjgt,ptjd->prjgd", wg, pv)[group, row] + torch.einsum("bjgt,btjd->bjgd", wo, ov)
    o = torch.where(total[..., None] > 0, o / total[..., None], torch.zeros_like(o))
    out = {"out": o.reshape(c["batch"], c["hq"], c["d"]).to(torch.bfloat16)}
    if sel is not None:
        out["sel"] = sel
    return out


def _plain_cross(s):
    c = s["case"]
    q, _ = _plain_q(s)
    k, v = _plain_kv(c, s["pool"], s["tables"][0])
    valid = torch.arange(k.shape[1], device=DEV)[None] < s["kv_lens"][:, None]
    k, v = _cut(k, valid), _cut(v, valid)
    r = torch.arange(s["rows"], device=DEV)
    seq = torch.searchsorted(s["q_start"][1:].long(), r, right=True)
    row = r - s["q_start"].long()[seq]
    qs = torch.zeros((c["batch"], c["q"]) + tuple(q.shape[1:]), device=DEV)
    qs[seq, row] = q
    sc = torch.einsum("brjgd,btjd->brjgt", qs, k).masked_fill(~valid[:, None, None, None], -math.inf)
    m = sc.amax(-1, keepdim=True)
    w = torch.exp(sc - torch.where(m == -math.inf, torch.zeros_like(m), m))
    total = w.sum(-1)[..., None]
    o = torch.einsum("brjgt,btjd->brjgd", w, v)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))[seq, row]
    return {"out": o.reshape(s["rows"], c["hq"], c["d"]).to(torch.bfloat16)}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _own(s):
    Q, c = _library(), s["case"]
    dt = Q.DQK_BF16 if c["dtype"] == "bf16" else Q.DQK_F32
    if c["op"].startswith("rope"):
        call = Q.dqk_bf16_rope_append if c["op"] == "rope_bf16" else Q.dqk_rope_append
        call(s["layer"], s["rope"], s["k"], s["k"].stride(0), s["v"], s["v"].stride(0), s["q"], s["q"].stride(0), s["q_out"],
             s["q_out"].stride(0), dt, c["batch"], s["new"], s["before"], s["max_new"], s["positions"], s["table"], s["table"].shape[1])
        return {"pool": s["pool"], "q": s["q_out"]}
    t, ws = s["tables"], s["ws"]
    if c["op"] == "cross":
        Q.dqk_bf16_cross_attention(s["layer"], s["q"], dt, c["batch"], s["rows"], s["q_start"], s["kv_lens"], t[0], t[0].shape[1],
                                   s["out"], Q.DQK_BF16, ws, ws.numel())
        return {"out": s["out"]}
    if c["op"] == "prefix_bf16":
        Q.dqk_bf16_prefix_decode(s["layer"], s["q"], dt, c["batch"], t[0].shape[0], s["start"], s["prefix_lens"], t[0], t[0].shape[1],
                                 s["own_lens"], t[1], t[1].shape[1], s["out"], Q.DQK_BF16, ws, ws.numel())
        return {"out": s["out"]}
    Q.dqk_prefix_decode(s["layer"], s["q"], dt, c["batch"], t[0].shape[0], s["start"], s["prefix_lens"], t[0], t[0].shape[1],
                        s["own_lens"], t[1], t[1].shape[1], c["pct"], s["out"], Q.DQK_BF16, s["sel"], ws, ws.numel())
    return {"out": s["out"], "sel": s["sel"]}


def run(state):
    if own:
        return _own(state)
    op = state["case"]["op"]
    return _plain_rope(state) if op.startswith("rope") else _plain_cross(state) if op == "cross" else _plain_prefix(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_turn(c, x, ang_cos, ang_sin):
    """Rows as complex numbers times cos + i sin."""
    h = c["rotary"] // 2
    x = x.double()
    first = (torch.arange(h, device=DEV) * 2) if c["interleaved"] else torch.arange(h, device=DEV)
    second = first + (1 if c["interleaved"] else h)
    z = torch.complex(x[..., first], x[..., second]) * torch.complex(ang_cos, ang_sin)[:, None]
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_rows(c, part, lens):
    """Keys and values of each list, in 64 bits, straight from what was drawn."""
    f, at = part, 0
    for n in lens:
        w = {key: x[at:at + n] for key, x in f.items()}
        at += n
        if "k" in w:
            yield w["k"].double(), w["v"].double()
            continue
        both = []
        for a in "kv":
            shape = w[a + "codes"].shape
            x = w[a + "codes"].double().reshape(shape[:2] + (c["d"] // c["group_size"], c["group_size"]))
            x = (x * w[a + "scale"].double()[..., None] + w[a + "min"].double()[..., None]).reshape(shape)
            if a + "ch0" in w:
                x[..., 0] = w[a + "ch0"].double()
            both.append(x)
        yield both[0], both[1]


def _exact_softmax(q, k, v):
    """q [rows][hq][d], k and v [tokens][hkv][d] -> [rows][hq][d]."""
    g = q.shape[1] // k.shape[1]
    out = torch.zeros_like(q)
    if k.shape[0]:
        for j in range(k.shape[1]):
            p = torch.softmax(q[:, j * g:(j + 1) * g] @ k[:, j].T / math.sqrt(q.shape[-1]), -1)
            out[:, j * g:(j + 1) * g] = p @ v[:, j]
    return out


def exact(case, seed):
    c = case
    if c["op"].startswith("rope"):
        s = _make_rope(c, seed)
        h = c["rotary"] // 2
        cs = s["cos_sin"].double()[s["positions"].long()]
        q = torch.zeros((max(1, s["rows"]), c["hq"], c["d"]), dtype=torch.float64, device=DEV)
        q[:s["rows"]] = _exact_turn(c, s["q"], cs[:, :h], cs[:, h:])
        if c["op"] == "rope_int2":
            return {"pool": None, "q": q}   # bytes: compared for equality
        k, v = _exact_turn(c, s["k"], cs[:, :h], cs[:, h:]), s["v"].double()
        chunks = c["d"] // 8
        pool = torch.zeros((s["total"], c["hkv"], 2, PAGE, chunks, 8), dtype=torch.float64, device=DEV)
        for x in range(chunks):
            to = x ^ (s["slot"] % 8)
            pool[s["page"], :, 0, s["slot"], to] = k[..., 8 * x:8 * x + 8]
            pool[s["page"], :, 1, s["slot"], to] = v[..., 8 * x:8 * x + 8]
        return {"pool": pool.reshape(s["pool"].shape), "q": q}
    s = _make_attention(c, seed)
    n, q = s["lens"], s["q"].double()
    if c["op"] == "cross":
        out, at = torch.zeros_like(q), 0
        for rows, (k, v) in zip(n["q"], _exact_rows(c, *s["parts"][0])):
            out[at:at + rows] = _exact_softmax(q[at:at + rows], k, v)
            at += rows
        return {"out": out}
    sel = None
    if c["op"] == "prefix_int2":
        g = c["hq"] // c["hkv"]
        t = s["t_q"].double()
        q = torch.stack([q[:, h] @ t[h // g].T for h in range(c["hq"])], 1).float().double()
        keep = c["d"] - (c["pct"] * c["d"]) // 100
        mag = q[..., 1:].abs()
        edge = mag.sort(-1).values[..., c["d"] - keep:c["d"] - keep + 1]   # the smallest magnitude that is kept
        above = mag > edge
        left = keep - 1 - above.sum(-1, keepdim=True)
        tie = (mag == edge)
        kept = (above | (tie & (tie.cumsum(-1) <= left))) if keep > 1 else torch.zeros_like(above)
        kept = torch.cat([torch.ones_like(kept[..., :1]), kept], -1)
        q = torch.where(kept, q, torch.zeros_like(q))
        sel = kept.nonzero()[:, 2].reshape(c["batch"], c["hq"], keep).to(torch.int16)
    out = torch.zeros_like(q)
    own_rows = list(_exact_rows(c, *s["parts"][1]))
    for p, (k, v) in enumerate(_exact_rows(c, *s["parts"][0])):
        a, b = n["start"][p], n["start"][p + 1]
        g = c["hq"] // c["hkv"]
        for j in range(c["hkv"]):
            rows = q[a:b, j * g:(j + 1) * g] / math.sqrt(c["d"])
            shared = rows @ k[:, j].T
            for i in range(a, b):
                ok, ov = own_rows[i]
                w = torch.softmax(torch.cat([shared[i - a], rows[i - a] @ ok[:, j].T], -1), -1)
                out[i, j * g:(j + 1) * g] = w[:, :k.shape[0]] @ v[:, j] + w[:, k.shape[0]:] @ ov[:, j]
    return {"out": out} if sel is None else {"out": out, "sel": sel}
