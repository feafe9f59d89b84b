// rope.cuh -- rotary position embedding on the way into the cache: the new
// rows' keys are rotated and appended (to the INT2 cache through T_K and the
// quantizer, or to the BF16 cache), their values appended, and their queries
// rotated, in one launch.
//
// Pair (a, b) of a row at position p, with (c, s) = cos/sin of the pair's angle:
//   a' = a c - b s,   b' = b c + a s;
// pairs are (i, i + r/2) or (interleaved) (2i, 2i + 1), i < r/2, r = rotary_dim;
// channels r..d-1 pass unchanged.
#pragma once

#include "append.cuh"
#include "common.cuh"
#include "ptx.cuh"

namespace dqk {

struct RopeParams {
    const void *k, *v, *q;       // q may be null
    void *q_out;                 // may be q itself
    long long k_stride, v_stride, q_stride, q_out_stride;   // elements between rows
    int dtype, batch, hq, hkv;
    const int *new_lens, *seq_before, *positions;           // positions may be null
    int max_new;
    const float *cos_sin;        // [max_position][rotary]
    long long max_position;
    int rotary, interleaved;
    const int *page_table;
    int max_pages;
    uint8_t *pool;
    long long num_pages;
    const float *t_k;            // INT2 cache only
    int v_ch0;
    int tiles;                   // CTAs per sequence along the rows
};

// Rows of the sequences before b (negative counts read as 0), by each warp for itself.
__device__ __forceinline__ long long rows_before(const int *new_lens, int b) {
    long long n = 0;
    for (int i = threadIdx.x & 31; i < b; i += 32) n += max(new_lens[i], 0);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    return n;
}

// Physical page of token `pos` of sequence b, or -1 (flagged by the caller).
__device__ __forceinline__ int rope_page(const RopeParams &p, int b, long long pos) {
    if (pos < 0 || pos / kPage >= p.max_pages) return -1;
    const int phys = p.page_table[(size_t)b * p.max_pages + pos / kPage];
    return phys >= 0 && phys < p.num_pages ? phys : -1;
}

// Position of new row t of sequence b (input row `row`), or -1 outside the table.
__device__ __forceinline__ long long rope_position(const RopeParams &p, int b, int t, long long row) {
    const long long pos = p.positions ? (long long)p.positions[row] : (long long)p.seq_before[b] + t;
    return pos >= 0 && pos < p.max_position ? pos : -1;
}

// Eight consecutive elements as fp32.
__device__ __forceinline__ void load8(const void *base, int dtype, size_t idx, float (&x)[8]) {
    if (dtype == DQK_BF16) {
        const uint4 w = *reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(base) + idx);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(u[i] << 16);
            x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    } else {
        const float4 *f = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(base) + idx);
        const float4 a = f[0], b = f[1];
        x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
        x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
    }
}
__device__ __forceinline__ uint4 pack8_bf16(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                      pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store8(void *base, int dtype, size_t idx, const float (&x)[8]) {
    if (dtype == DQK_BF16) {
        *reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(base) + idx) = pack8_bf16(x);
    } else {
        float4 *f = reinterpret_cast<float4 *>(reinterpret_cast<float *>(base) + idx);
        f[0] = make_float4(x[0], x[1], x[2], x[3]);
        f[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
}

// A thread's share of one head row: two 16-byte chunks (8 channels each) that
// hold whole pairs.  Share u < r/16 is rotated -- chunks u and u + r/16, or
// (interleaved) 2u and 2u + 1 -- and the others, behind the rotated channels,
// pass.  r is a multiple of 16, so a chunk is never cut.
struct RopeShare {
    int c0, c1;      // chunk indices
    bool rotated;
};
__device__ __forceinline__ RopeShare rope_share(int u, int rotary, int interleaved) {
    const int n = rotary >> 4;
    if (u >= n) return {2 * u, 2 * u + 1, false};
    return interleaved ? RopeShare{2 * u, 2 * u + 1, true} : RopeShare{u, u + n, true};
}

// Rotate in fp32: the product b s rounded, then one fused multiply-add.  cs: the position's row.
__device__ __forceinline__ void rope_rotate(const float *__restrict__ cs, int rotary, int interleaved,
                                            const RopeShare &sh, float (&x0)[8], float (&x1)[8]) {
    const int half = rotary >> 1;
    if (!interleaved) {
        float c[8], s[8];
        load8(cs, DQK_F32, 8 * sh.c0, c);
        load8(cs, DQK_F32, half + 8 * sh.c0, s);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float a = x0[i], b = x1[i];
            x0[i] = fmaf(a, c[i], -(b * s[i]));
            x1[i] = fmaf(b, c[i], a * s[i]);
        }
    } else {
        // pairs 8u .. 8u+7: chunk 2u holds the first four, chunk 2u+1 the rest
        float c[8], s[8];
        load8(cs, DQK_F32, 4 * sh.c0, c);
        load8(cs, DQK_F32, half + 4 * sh.c0, s);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = x0[2 * i], b = x0[2 * i + 1], e = x1[2 * i], f = x1[2 * i + 1];
            x0[2 * i] = fmaf(a, c[i], -(b * s[i]));
            x0[2 * i + 1] = fmaf(b, c[i], a * s[i]);
            x1[2 * i] = fmaf(e, c[4 + i], -(f * s[4 + i]));
            x1[2 * i + 1] = fmaf(f, c[4 + i], e * s[4 + i]);
        }
    }
}

// ---------------------------------------------------------------------------
// BF16 cache: CTA = (sequence, kRopeTile consecutive new rows), all heads of q,
// k and v; a thread moves two 16-byte chunks of one head row at a time.  It is
// bound by memory: every row is read and written once.  4 prompts of 4096 to 8192
// rows (32 / 8 heads, head_dim 128, BF16; 679 MB): 138 us, 4.9 TB/s.  One row per CTA
// takes 20 us for 256 sequences of 8 rows where four take 15, and as long for single rows.
// ---------------------------------------------------------------------------
constexpr int kRopeThreads = 256, kRopeTile = 4;

template <int D>
__global__ void __launch_bounds__(kRopeThreads) k_rope_append_b16(const __grid_constant__ RopeParams p) {
    constexpr int U = D / 16;   // shares of a head row
    const int b = blockIdx.x / p.tiles, t0 = (blockIdx.x - b * p.tiles) * kRopeTile;
    __shared__ int sh_phys[kRopeTile];
    __shared__ long long sh_pos[kRopeTile];
    const int n = min(p.new_lens[b], p.max_new);
    if (p.new_lens[b] > p.max_new && threadIdx.x == 0) dqk_flag_error(kErrBounds);
    if (t0 >= n) return;
    const int nr = min(kRopeTile, n - t0);
    const long long row0 = rows_before(p.new_lens, b) + t0;
    const int L0 = p.seq_before[b];
    if ((int)threadIdx.x < nr) {
        const int t = t0 + threadIdx.x;
        const int phys = L0 < 0 ? -1 : rope_page(p, b, (long long)L0 + t);
        const long long pos = rope_position(p, b, t, row0 + threadIdx.x);
        if (phys < 0 || pos < 0) dqk_flag_error(kErrBounds);   // the row is skipped as a whole
        sh_phys[threadIdx.x] = pos < 0 ? -1 : phys;
        sh_pos[threadIdx.x] = pos;
    }
    __syncthreads();
    const int heads = 2 * p.hkv + (p.q ? p.hq : 0);
    const int items = nr * heads * U;
#pragma unroll 2
    for (int it = threadIdx.x; it < items; it += kRopeThreads) {
        const int u = it % U, hr = it / U, head = hr % heads, r = hr / heads;
        const int phys = sh_phys[r];
        if (phys < 0) continue;
        const long long row = row0 + r;
        const float *cs = p.cos_sin + sh_pos[r] * p.rotary;
        const int slot = (L0 + t0 + r) % kPage;
        const RopeShare sh = rope_share(u, p.rotary, p.interleaved);
        float x0[8], x1[8];
        if (head < 2 * p.hkv) {
            const int is_v = head >= p.hkv, j = is_v ? head - p.hkv : head;
            const void *in = is_v ? p.v : p.k;
            const size_t src = (size_t)row * (is_v ? p.v_stride : p.k_stride) + (size_t)j * D;
            load8(in, p.dtype, src + 8 * sh.c0, x0);
            load8(in, p.dtype, src + 8 * sh.c1, x1);
            if (!is_v && sh.rotated) rope_rotate(cs, p.rotary, p.interleaved, sh, x0, x1);
            // block layout of the BF16 cache: K [16][D] then V [16][D], chunk x of token t at x ^ (t & 7)
            uint8_t *dst = p.pool + ((size_t)phys * p.hkv + j) * (2 * kPage * D * 2) + is_v * kPage * 2 * D + slot * 2 * D;
            *reinterpret_cast<uint4 *>(dst + ((sh.c0 ^ (slot & 7)) << 4)) = pack8_bf16(x0);
            *reinterpret_cast<uint4 *>(dst + ((sh.c1 ^ (slot & 7)) << 4)) = pack8_bf16(x1);
        } else {
            const int h = head - 2 * p.hkv;
            const size_t src = (size_t)row * p.q_stride + (size_t)h * D, dst = (size_t)row * p.q_out_stride + (size_t)h * D;
            load8(p.q, p.dtype, src + 8 * sh.c0, x0);
            load8(p.q, p.dtype, src + 8 * sh.c1, x1);
            if (sh.rotated) rope_rotate(cs, p.rotary, p.interleaved, sh, x0, x1);
            store8(p.q_out, p.dtype, dst + 8 * sh.c0, x0);
            store8(p.q_out, p.dtype, dst + 8 * sh.c1, x1);
        }
    }
}

// ---------------------------------------------------------------------------
// INT2 cache.  The keys' codes have one well-defined value: the rotated key is
// fp32(a c - b s) with exact fp64 products and one rounding to fp64 and to
// fp32, then dqk_append's transform and quantizer take it from there.
// ---------------------------------------------------------------------------
__device__ __forceinline__ float rope_key(const RopeParams &p, const float *cs, size_t row_base, int c) {
    const float x = load_elem(p.k, p.dtype, row_base + c);
    if (c >= p.rotary) return x;
    const int half = p.rotary >> 1;
    int i, partner;
    bool second;
    if (p.interleaved) {
        i = c >> 1;
        partner = c ^ 1;
        second = c & 1;
    } else {
        second = c >= half;
        i = second ? c - half : c;
        partner = second ? i : c + half;
    }
    const double y = (double)load_elem(p.k, p.dtype, row_base + partner);
    const double co = (double)cs[i], si = (double)cs[half + i];
    const double ys = y * si;   // exact: 24 x 24 bits
    return __double2float_rn(second ? fma((double)x, co, ys) : fma((double)x, co, -ys));
}

// The queries of new row t of sequence b, by the CTA's threads.
template <int D>
__device__ __forceinline__ void rope_queries(const RopeParams &p, int b, int t, long long row) {
    constexpr int U = D / 16;
    const int L0 = p.seq_before[b];
    const long long pos = rope_position(p, b, t, row);
    if (pos < 0 || L0 < 0 || rope_page(p, b, (long long)L0 + t) < 0) return;   // flagged by the key's CTA
    for (int it = threadIdx.x; it < p.hq * U; it += blockDim.x) {
        const int u = it % U, h = it / U;
        const RopeShare sh = rope_share(u, p.rotary, p.interleaved);
        const size_t src = (size_t)row * p.q_stride + (size_t)h * D, dst = (size_t)row * p.q_out_stride + (size_t)h * D;
        float x0[8], x1[8];
        load8(p.q, p.dtype, src + 8 * sh.c0, x0);
        load8(p.q, p.dtype, src + 8 * sh.c1, x1);
        if (sh.rotated) rope_rotate(p.cos_sin + pos * p.rotary, p.rotary, p.interleaved, sh, x0, x1);
        store8(p.q_out, p.dtype, dst + 8 * sh.c0, x0);
        store8(p.q_out, p.dtype, dst + 8 * sh.c1, x1);
    }
}

// A few rows: a CTA of D threads per (new row, kv head), the structure of k_append_rows; CTAs at
// blockIdx.y = hkv rotate the rows' queries.  Bound by latency: T_K[j] in, a chain of D multiply-adds,
// the quantizer.  16 sequences of one row, 8 kv heads: 8 us (12 us a call with its launch).
template <int D, int NS>
__global__ void __launch_bounds__(D) k_rope_append_rows(const __grid_constant__ RopeParams p) {
    constexpr int kPad = D * 4 + 16;
    extern __shared__ __align__(16) unsigned char rope_rows_mem[];
    unsigned char *sT = rope_rows_mem;
    double *xs = reinterpret_cast<double *>(rope_rows_mem + (size_t)D * kPad);
    RowStoreScratch<D, NS, 1> &S = *reinterpret_cast<RowStoreScratch<D, NS, 1> *>(xs + D);
    const int j = blockIdx.y, c = threadIdx.x;
    const int b = blockIdx.x / p.tiles, t = blockIdx.x - b * p.tiles;
    const int n = min(p.new_lens[b], p.max_new);
    if (p.new_lens[b] > p.max_new && c == 0) dqk_flag_error(kErrBounds);
    if (t >= n) return;
    const long long row = rows_before(p.new_lens, b) + t;
    if (j == p.hkv) {
        rope_queries<D>(p, b, t, row);
        return;
    }
    {
        const float *tj = p.t_k + (size_t)j * D * D;
        const uint32_t base = smem_addr(sT);
#pragma unroll 4
        for (int q = c; q < D * D / 4; q += D)
            cp_async16(base + (uint32_t)((q / (D / 4)) * kPad + (q % (D / 4)) * 16), tj + 4 * q);
    }
    const int L0 = p.seq_before[b];
    const long long pos = rope_position(p, b, t, row);
    xs[c] = (double)rope_key(p, p.cos_sin + (pos < 0 ? 0 : pos) * p.rotary, (size_t)row * p.k_stride + (size_t)j * D, c);
    const float xv[1] = {load_elem(p.v, p.dtype, (size_t)row * p.v_stride + (size_t)j * D + c)};
    const int phys[1] = {pos < 0 || L0 < 0 ? -1 : rope_page(p, b, (long long)L0 + t)};   // -1: flagged and skipped below
    cp_async_wait_all();
    __syncthreads();
    double acc = 0.0;
    const unsigned char *tc = sT + (size_t)c * kPad;
#pragma unroll 8
    for (int i = 0; i < D; i += 4) {
        const float4 w = *reinterpret_cast<const float4 *>(tc + i * 4);
        acc = fma((double)w.x, xs[i], acc);
        acc = fma((double)w.y, xs[i + 1], acc);
        acc = fma((double)w.z, xs[i + 2], acc);
        acc = fma((double)w.w, xs[i + 3], acc);
    }
    const float kp[1] = {__double2float_rn(acc)};
    quantize_store_rows<D, NS, 1>(kp, xv, phys, 1, L0 + t, c, p.pool, p.num_pages, p.hkv, j, p.v_ch0, S,
                                  [] { __syncthreads(); });
}

// ---------------------------------------------------------------------------
// The same for many rows: a CTA takes 8 RW consecutive new rows of a sequence
// and one kv head.  What bounds it is the fp64 product K' = X T^T, D^2 fused
// multiply-adds a row at 64 per clock and SM, and what feeds it: shared memory
// returns 128 bytes a clock, broadcast or not.  So T (transposed) lies there as
// fp64 and the rotated rows as fp32 (which they are), a warp forms RW rows, a
// lane the channels lane + 32m, and the rows stay with the warp that quantizes and
// stores them.  Eight more warps rotate the group's queries meanwhile.
//
// 16 sequences of 64 rows, 8 kv heads, head_dim 128 (128 CTAs, 134 M multiply-adds, 7.2 us at the fp64 pipe's rate):
// 29.5 us, one row per CTA 118.  A CTA's clocks: T and the rows' places 6000, rotated keys 4000, product 32000 (1.05 fp64
// instructions a clock where independent ones reach 1.8), ranges, codes and stores 10500.
//
// The sums run over ascending i as in k_rope_append_rows, and the quantizer's
// codes are the same.  With y = fl(x - min) and a scale s > 0 of fp16's 11 bits,
//   clamp(rne(fl(y / s)), 0, 3) = (y > s/2) + (y >= 3s/2) + (y > 5s/2),
// since the fp64 neighbours of s/2, 3s/2 and 5s/2 lie far enough from them that
// their quotients don't round to 1/2, 3/2 or 5/2; and y > h (y >= h) for such an
// h, whose last fp64 bit is 0, means x > min + h + u (x >= min + h - u) with u half an
// fp64 step at h.  The fp32 x is compared with that, rounded down (up) to fp32.
// ---------------------------------------------------------------------------
constexpr int kRopeTileThreads = 512, kRopeTileWarps = 8;   // threads; warps that form the product

template <int D, int NS, int RW>
struct RopeTileSmem {
    static constexpr int R = kRopeTileWarps * RW;
    double t[D][D + 2];             // t[i][c] = T_K[j][c][i]
    float x[D][R + 4];              // x[i][row]
    float4 level[R][2 * NS];        // of each group of a row (keys, then values): what x is compared with
    long long pos[R];
    int phys[R];
};

template <int RW>
struct RopeRows {
    using T = float4;
    static __device__ __forceinline__ void widen(T w, double (&x)[4]) {
        x[0] = (double)w.x; x[1] = (double)w.y; x[2] = (double)w.z; x[3] = (double)w.w;
    }
};
template <>
struct RopeRows<2> {
    using T = float2;
    static __device__ __forceinline__ void widen(T w, double (&x)[2]) {
        x[0] = (double)w.x; x[1] = (double)w.y;
    }
};

// What the fp32 x is compared with (see above): y > h, or y >= h, for y = fl(x - lo).
__device__ __forceinline__ float rope_level(double lo, double h, bool equal) {
    const double u = __longlong_as_double((__double_as_longlong(h) & 0x7ff0000000000000LL) - (53LL << 52));
    return equal ? __double2float_ru(lo + h - u) : __double2float_rd(lo + h + u);
}

__device__ __forceinline__ float warp_lowest(float x) {
    float r;
    asm volatile("redux.sync.min.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float warp_highest(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// The ranges of a row's groups (channels lane + 32m of the key and of the value), group e of the keys (e < NS)
// or of the values by lane e.  -0 reads as +0, and a channel 0 that is kept apart takes no part.
template <int D, int NS>
__device__ __forceinline__ float2 rope_ranges(const float (&kx)[D / 32], const float (&vx)[D / 32], int lane, int v_ch0) {
    constexpr int NG = D / 32;
    const float inf = __int_as_float(0x7f800000);
    float2 mine = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        float lo = inf, hi = -inf;
#pragma unroll
        for (int m = 0; m < NG; ++m) {
            const float x = (kv ? vx[m] : kx[m]) + 0.0f;
            const bool out = m == 0 && lane == 0 && (kv == 0 || v_ch0 != 0);
            const float l = out ? inf : x, h = out ? -inf : x;
            lo = NS == 1 ? fminf(lo, l) : l;
            hi = NS == 1 ? fmaxf(hi, h) : h;
            if (NS != 1 || m == NG - 1) {
                lo = warp_lowest(lo);
                hi = warp_highest(hi);
                if (lane == kv * NS + (NS == 1 ? 0 : m)) mine = make_float2(lo, hi);
            }
        }
    }
    return mine;
}

// One row's codes and channel 0, by the warp.
template <int D, int NS>
__device__ __forceinline__ void rope_store_codes(const float (&kx)[D / 32], const float (&vx)[D / 32], int lane, int slot,
                                                 uint8_t *blk, const Layout &L, int v_ch0, const float4 *level) {
    constexpr int NG = D / 32;
    uint16_t *h16 = reinterpret_cast<uint16_t *>(blk);
    if (lane == 0) {
        h16[(L.k0 >> 1) + k0_idx(slot)] = f32_to_bf16_rne(kx[0]);
        if (v_ch0) h16[(L.v0 >> 1) + slot] = f32_to_bf16_rne(vx[0]);
    }
    uint32_t code[2 * NG];
#pragma unroll
    for (int e = 0; e < 2 * NG; ++e) {
        const int g = NS == 1 ? e / NG : e;
        const float4 at = level[g];
        const float x = e < NG ? kx[e] : vx[e - NG];
        const bool out = lane == 0 && (e == 0 || (e == NG && v_ch0 != 0));
        code[e] = out ? 0u : (x > at.x ? 1u : 0u) + (x >= at.y ? 1u : 0u) + (x > at.z ? 1u : 0u);
    }
    // a byte of key codes holds one token's (see kcode_pos)
    const int hi16 = lane >> 4;
    uint32_t kb = 0;
#pragma unroll
    for (int g = 0; g < NG; ++g) kb |= code[g] << (2 * (NG == 4 ? g : g + 2 * hi16));
    const int kl = 4 * (slot & 7) + ((lane & 15) >> 2), kj = lane & 3;
    if constexpr (NG == 4) {
        blk[L.kc + (kl * 4 + 2 * hi16 + (slot >> 3)) * 4 + kj] = (uint8_t)kb;
    } else {
        kb |= __shfl_xor_sync(0xffffffffu, kb, 16);
        if (lane < 16) blk[L.kc + (kl * 2 + (slot >> 3)) * 4 + kj] = (uint8_t)kb;
    }
    // value codes (see vcode_pos): with four groups a 16-bit half of a word holds one token's, with two
    // tokens t and t + 8 share it
    const int r = lane & 15, vl = (r & 7) * 4 + ((slot & 7) >> 1), tb = slot >> 3;
    if constexpr (NG == 4) {
        uint32_t vb = 0;
#pragma unroll
        for (int m = 0; m < NG; ++m) vb |= code[NG + m] << (2 * (2 * m + hi16));
        vb |= __shfl_xor_sync(0xffffffffu, vb, 16);
        if (lane < 16) h16[(L.vc >> 1) + (vl * 4 + (r >> 3) + 2 * tb) * 2 + (slot & 1)] = (uint16_t)vb;
    } else {
        uint32_t *vw = reinterpret_cast<uint32_t *>(blk + L.vc) + vl * 2;
        const int bit = 16 * (slot & 1) + 2 * tb;
#pragma unroll
        for (int m = 0; m < NG; ++m) {
            uint32_t vb = code[NG + m] << (bit + 2 * (4 * hi16 + 2 * (r >> 3)));
            vb |= __shfl_xor_sync(0xffffffffu, vb, 16);
            vb |= __shfl_xor_sync(0xffffffffu, vb, 8);
            if (lane < 8) {
                atomicAnd(vw + m, ~(0x3333u << bit));   // the token's fields 4 hi + 2 cr + tb
                atomicOr(vw + m, vb);
            }
        }
    }
}

template <int D, int NS, int RW>
__global__ void __launch_bounds__(kRopeTileThreads) k_rope_append_tile(const __grid_constant__ RopeParams p) {
    constexpr int R = kRopeTileWarps * RW, NG = D / 32, U = D / 16, kPosWarps = (R + 31) / 32;
    extern __shared__ __align__(16) unsigned char rope_tile_mem[];
    RopeTileSmem<D, NS, RW> &S = *reinterpret_cast<RopeTileSmem<D, NS, RW> *>(rope_tile_mem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, j = blockIdx.y;
    const int b = blockIdx.x / p.tiles, t0 = (blockIdx.x - b * p.tiles) * R;
    const int n = min(p.new_lens[b], p.max_new);
    if (p.new_lens[b] > p.max_new && tid == 0) dqk_flag_error(kErrBounds);
    if (t0 >= n) return;
    const int nr = min(R, n - t0);
    const long long row0 = rows_before(p.new_lens, b) + t0;
    const int L0 = p.seq_before[b];
    const int size = p.dtype == DQK_BF16 ? 2 : 4;
    if (warp < kPosWarps) {   // the rows' places; what is read later is brought nearer
        if (tid < R) {
            int phys = -1;
            long long pos = -1;
            if (tid < nr) {
                const char *k = reinterpret_cast<const char *>(p.k) + ((size_t)(row0 + tid) * p.k_stride + (size_t)j * D) * size;
                const char *v = reinterpret_cast<const char *>(p.v) + ((size_t)(row0 + tid) * p.v_stride + (size_t)j * D) * size;
                for (int o = 0; o < D * size; o += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(k + o));
                for (int o = 0; o < D * size; o += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(v + o));
                phys = L0 < 0 ? -1 : rope_page(p, b, (long long)L0 + t0 + tid);
                pos = rope_position(p, b, t0 + tid, row0 + tid);
                if (phys < 0 || pos < 0) {   // the row is skipped as a whole
                    dqk_flag_error(kErrBounds);
                    phys = -1;
                }
            }
            S.phys[tid] = phys;
            S.pos[tid] = max(pos, 0LL);
        }
    } else {
        // T: 8 columns of 4 rows a warp, so that the transposed stores meet no bank twice
        const float *tj = p.t_k + (size_t)j * D * D;
#pragma unroll 18
        for (int q = warp - kPosWarps; q < D * D / 32; q += kRopeTileThreads / 32 - kPosWarps) {
            const int i = 8 * (q % (D / 8)) + (lane & 7), c = 4 * (q / (D / 8)) + (lane >> 3);
            S.t[i][c] = (double)tj[(size_t)c * D + i];
        }
    }
    __syncthreads();
    // rotated keys, a pair (or two channels that pass) at a time
    {
        const int half = p.rotary >> 1;
        constexpr int kPairs = R * (D / 2) / kRopeTileThreads, kAtOnce = kPairs < 8 ? kPairs : 8;
        static_assert(kPairs % kAtOnce == 0, "pairs of a thread");
#pragma unroll 1
        for (int i0 = 0; i0 < kPairs; i0 += kAtOnce) {
            float xa[kAtOnce], xb[kAtOnce], co[kAtOnce], si[kAtOnce];
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e) {
                const int it = tid + (i0 + e) * kRopeTileThreads, r = it / (D / 2), u = it % (D / 2);
                const bool turned = u < half;
                const int ca = turned && !p.interleaved ? u : 2 * u, cb = turned && !p.interleaved ? u + half : 2 * u + 1;
                const size_t at = (size_t)(row0 + min(r, nr - 1)) * p.k_stride + (size_t)j * D;
                const float *cs = p.cos_sin + S.pos[r] * p.rotary + (turned ? u : 0);
                xa[e] = load_elem(p.k, p.dtype, at + ca);
                xb[e] = load_elem(p.k, p.dtype, at + cb);
                co[e] = cs[0];
                si[e] = cs[half];
            }
#pragma unroll
            for (int e = 0; e < kAtOnce; ++e) {
                const int it = tid + (i0 + e) * kRopeTileThreads, r = it / (D / 2), u = it % (D / 2);
                const bool turned = u < half;
                const int ca = turned && !p.interleaved ? u : 2 * u, cb = turned && !p.interleaved ? u + half : 2 * u + 1;
                if (turned) {   // as rope_key: exact products, one rounding to fp64, one to fp32
                    const double x = (double)xa[e], f = (double)xb[e], c = (double)co[e], s = (double)si[e];
                    xa[e] = __double2float_rn(fma(x, c, -(f * s)));
                    xb[e] = __double2float_rn(fma(f, c, x * s));
                }
                S.x[ca][r] = xa[e];
                S.x[cb][r] = xb[e];
            }
        }
    }
    __syncthreads();
    if (warp >= kRopeTileWarps) {
        // the queries of the rows and of the kv head's group, a few shares in flight
        if (!p.q) return;
        constexpr int kAtOnce = 4, kStep = kRopeTileThreads - 32 * kRopeTileWarps;
        const int G = p.hq / p.hkv, items = nr * G * U;
        for (int it0 = tid - 32 * kRopeTileWarps; it0 < items; it0 += kAtOnce * kStep) {
            float x[kAtOnce][2][8];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int it = it0 + k * kStep, u = it % U, hr = it / U, h = j * G + hr % G, r = hr / G;
                if (it >= items || S.phys[r] < 0) continue;
                const RopeShare sh = rope_share(u, p.rotary, p.interleaved);
                const size_t src = (size_t)(row0 + r) * p.q_stride + (size_t)h * D;
                load8(p.q, p.dtype, src + 8 * sh.c0, x[k][0]);
                load8(p.q, p.dtype, src + 8 * sh.c1, x[k][1]);
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int it = it0 + k * kStep, u = it % U, hr = it / U, h = j * G + hr % G, r = hr / G;
                if (it >= items || S.phys[r] < 0) continue;
                const RopeShare sh = rope_share(u, p.rotary, p.interleaved);
                const size_t dst = (size_t)(row0 + r) * p.q_out_stride + (size_t)h * D;
                if (sh.rotated) rope_rotate(p.cos_sin + S.pos[r] * p.rotary, p.rotary, p.interleaved, sh, x[k][0], x[k][1]);
                store8(p.q_out, p.dtype, dst + 8 * sh.c0, x[k][0]);
                store8(p.q_out, p.dtype, dst + 8 * sh.c1, x[k][1]);
            }
        }
        return;
    }
    // k' = x T^T: rows RW warp .., channels lane + 32m
    const int r0 = RW * warp;
    if (r0 >= nr) return;
    double acc[RW][NG];
#pragma unroll
    for (int a = 0; a < RW; ++a)
#pragma unroll
        for (int m = 0; m < NG; ++m) acc[a][m] = 0.0;
    using Pair = typename RopeRows<RW>::T;   // 2 or 4 rows of x
    constexpr int kPer = sizeof(Pair) / 4;
#pragma unroll 4
    for (int i = 0; i < D; ++i) {
        double t[NG];
#pragma unroll
        for (int m = 0; m < NG; ++m) t[m] = S.t[i][lane + 32 * m];
#pragma unroll
        for (int a = 0; a < RW; a += kPer) {
            const Pair w = *reinterpret_cast<const Pair *>(&S.x[i][r0 + a]);
            double x[kPer];
            RopeRows<RW>::widen(w, x);
#pragma unroll
            for (int e = 0; e < kPer; ++e)
#pragma unroll
                for (int m = 0; m < NG; ++m) acc[a + e][m] = fma(t[m], x[e], acc[a + e][m]);
        }
    }
    float kx[RW][NG], vx[RW][NG];
#pragma unroll
    for (int a = 0; a < RW; ++a)
#pragma unroll
        for (int m = 0; m < NG; ++m) {
            kx[a][m] = __double2float_rn(acc[a][m]);
            vx[a][m] = load_elem(p.v, p.dtype, (size_t)(row0 + min(r0 + a, nr - 1)) * p.v_stride + (size_t)j * D + lane + 32 * m);
        }
    // the groups' ranges, then their scales -- a (row, group) per lane --, then the codes
#pragma unroll
    for (int a = 0; a < RW; ++a) {
        const float2 range = rope_ranges<D, NS>(kx[a], vx[a], lane, p.v_ch0);
        if (lane < 2 * NS) *reinterpret_cast<float2 *>(&S.level[r0 + a][lane]) = range;
    }
    __syncwarp();
    const Layout L = make_layout(D, p.v_ch0, NS);
#pragma unroll
    for (int i0 = 0; i0 < RW * 2 * NS; i0 += 32) {
        const int i = i0 + lane, r = r0 + i / (2 * NS), e = i % (2 * NS);
        if (i < RW * 2 * NS && S.phys[r] >= 0) {
            const float2 range = *reinterpret_cast<const float2 *>(&S.level[r][e]);
            const uint16_t sh = f64_to_f16_rne(((double)range.y - (double)range.x) / 3.0), mh = f64_to_f16_rne((double)range.x);
            const double s = f16_to_f64(sh), lo = f16_to_f64(mh);
            const float none = __int_as_float(0x7fc00000);   // scale 0: every code is 0
            S.level[r][e] = s != 0.0 ? make_float4(rope_level(lo, 0.5 * s, false), rope_level(lo, 1.5 * s, true),
                                                   rope_level(lo, 2.5 * s, false), 0.0f)
                                     : make_float4(none, none, none, 0.0f);
            const int slot = (L0 + t0 + r) % kPage, g = e % NS;
            const int at = e < NS ? kscale_idx(NS, slot, g) : vscale_idx(NS, slot, g);
            uint16_t *h16 = reinterpret_cast<uint16_t *>(p.pool + ((size_t)S.phys[r] * p.hkv + j) * L.bytes);
            h16[((e < NS ? L.ks : L.vs) >> 1) + at] = sh;
            h16[((e < NS ? L.km : L.vm) >> 1) + at] = mh;
        }
    }
    __syncwarp();
#pragma unroll
    for (int a = 0; a < RW; ++a) {
        const int r = r0 + a, phys = S.phys[r];
        if (phys < 0) continue;   // uniform; rows behind the sequence's last too
        rope_store_codes<D, NS>(kx[a], vx[a], lane, (L0 + t0 + r) % kPage, p.pool + ((size_t)phys * p.hkv + j) * L.bytes, L,
                                p.v_ch0, S.level[r]);
    }
}

}  // namespace dqk
