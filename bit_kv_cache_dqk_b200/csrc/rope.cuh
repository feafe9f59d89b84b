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
// k and v; a thread moves two 16-byte chunks of one head row at a time.
// ---------------------------------------------------------------------------
constexpr int kRopeThreads = 256;

template <int D, int TT>
__global__ void __launch_bounds__(kRopeThreads) k_rope_append_b16(const __grid_constant__ RopeParams p) {
    constexpr int U = D / 16;   // shares of a head row
    const int b = blockIdx.x / p.tiles, t0 = (blockIdx.x - b * p.tiles) * TT;
    __shared__ int sh_phys[TT];
    __shared__ long long sh_pos[TT];
    const int n = min(p.new_lens[b], p.max_new);
    if (p.new_lens[b] > p.max_new && threadIdx.x == 0) dqk_flag_error(kErrBounds);
    if (t0 >= n) return;
    const int nr = min(TT, n - t0);
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

// The queries of rows t0 .. t0+nr-1, by the CTA's threads.
template <int D>
__device__ __forceinline__ void rope_queries(const RopeParams &p, int b, int t0, int nr, long long row0) {
    constexpr int U = D / 16;
    const int L0 = p.seq_before[b];
    for (int it = threadIdx.x; it < nr * p.hq * U; it += blockDim.x) {
        const int u = it % U, hr = it / U, h = hr % p.hq, r = hr / p.hq;
        const long long row = row0 + r, pos = rope_position(p, b, t0 + r, row);
        if (pos < 0 || L0 < 0 || rope_page(p, b, (long long)L0 + t0 + r) < 0) continue;   // flagged by the key's CTA
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

// CTA of D threads per (RW consecutive new rows of a sequence, kv head), the
// structure of k_append_rows; CTAs at blockIdx.y = hkv rotate the rows' queries.
template <int D, int NS, int RW>
__global__ void __launch_bounds__(D) k_rope_append_rows(const __grid_constant__ RopeParams p) {
    constexpr int kPad = D * 4 + 16;
    extern __shared__ __align__(16) unsigned char rope_rows_mem[];
    unsigned char *sT = rope_rows_mem;
    double *xs = reinterpret_cast<double *>(rope_rows_mem + (size_t)D * kPad);   // [D][RW], i-major
    RowStoreScratch<D, NS, RW> &S = *reinterpret_cast<RowStoreScratch<D, NS, RW> *>(xs + (size_t)RW * D);
    const int j = blockIdx.y, c = threadIdx.x;
    const int b = blockIdx.x / p.tiles, t0 = (blockIdx.x - b * p.tiles) * RW;
    const int n = min(p.new_lens[b], p.max_new);
    if (p.new_lens[b] > p.max_new && c == 0) dqk_flag_error(kErrBounds);
    if (t0 >= n) return;
    const int nr = min(RW, n - t0);
    const long long row0 = rows_before(p.new_lens, b) + t0;
    if (j == p.hkv) {
        rope_queries<D>(p, b, t0, nr, row0);
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
    float xv[RW];
    int phys[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) {
        const int t = t0 + (i < nr ? i : 0);
        const long long row = row0 + (i < nr ? i : 0);
        const long long pos = rope_position(p, b, t, row);
        xs[c * RW + i] = (double)rope_key(p, p.cos_sin + (pos < 0 ? 0 : pos) * p.rotary,
                                          (size_t)row * p.k_stride + (size_t)j * D, c);
        xv[i] = load_elem(p.v, p.dtype, (size_t)row * p.v_stride + (size_t)j * D + c);
        phys[i] = pos < 0 || L0 < 0 ? -1 : rope_page(p, b, (long long)L0 + t);   // -1: flagged and skipped below
    }
    cp_async_wait_all();
    __syncthreads();
    double acc[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) acc[i] = 0.0;
    const unsigned char *row = sT + (size_t)c * kPad;
#pragma unroll 1
    for (int k = 0; k < D / 32; ++k) {
#pragma unroll
        for (int u = 0; u < 8; ++u) {
            const float4 tv = *reinterpret_cast<const float4 *>(row + (32 * k + 4 * u) * 4);
            const double t4[4] = {(double)tv.x, (double)tv.y, (double)tv.z, (double)tv.w};
            const double *xi = xs + (32 * k + 4 * u) * RW;
#pragma unroll
            for (int e = 0; e < 4; ++e)
#pragma unroll
                for (int i = 0; i < RW; ++i) acc[i] = fma(t4[e], xi[e * RW + i], acc[i]);
        }
    }
    float kp[RW];
#pragma unroll
    for (int i = 0; i < RW; ++i) kp[i] = __double2float_rn(acc[i]);
    quantize_store_rows<D, NS, RW>(kp, xv, phys, nr, L0 + t0, c, p.pool, p.num_pages, p.hkv, j, p.v_ch0, S,
                                   [] { __syncthreads(); });
}

}  // namespace dqk
