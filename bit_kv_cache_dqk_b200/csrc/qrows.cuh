// qrows.cuh -- the query rows of the shared-prefix decode over the INT2 cache:
// q' = T_Q q and the channel selection of every query head (the arithmetic, hence
// the kept channels, of dqk_decode), written as fp16 rows for the matrix
// instructions of the row kernels.
#pragma once

#include "common.cuh"
#include "ptx.cuh"
#include "qprep.cuh"
#include "rows.cuh"

namespace dqk {

constexpr int kQueryThreads = 256;

// Shared memory: T_Q[j] in padded rows, the query rows [D][RB G] fp64 (i-major), q' [RB G][D] fp32.
template <int D, int G, int RB>
__host__ __device__ constexpr size_t query_rows_smem() {
    return (size_t)D * pad_row_bytes<D>() + (size_t)RB * G * D * 12;
}

// CTA per (RB query rows, kv head): T_Q[j] is staged once for the RB G heads.  Row head (row, h) becomes
//   qr [row][hq][D] fp16 = rne(2^k q'_c) on the kept channels c >= 1, 0 elsewhere, in
//   the channel order of the key operand tiles (rows_channel_pos), with
//   k such that the largest of their |q'_c| lies in [2^14, 2^15): fp16's 11 bits then
//   cover channels down to 2^-28 of it;
//   head [row][hq] = (2^-k, q'_0) log2(e)/sqrt(d): what those scores are multiplied by, and the factor of
//   the keys' channel 0, which has its own term in fp32 (it is BF16 in the cache, with exponents fp16 lacks).
// Channels of zeros (or subnormals) become a row of zeros: channel 0 alone gives the scores.
// Bound by latency (T_Q[j] in, the fp64 sums, the selection's rounds): 8 us for 16 rows of 8 kv heads, 17 us for 64.
template <int D, int G, int RB>
__global__ void __launch_bounds__(kQueryThreads) k_query_rows(
    const float *__restrict__ t_q, const void *__restrict__ q, int dtype, int rows, int hq, int pct, float qscale,
    uint16_t *__restrict__ qr, float2 *__restrict__ head, int16_t *__restrict__ sel_out) {
    constexpr int NG = D / 32, NH = RB * G, kParts = kQueryThreads / D, kPer = (NH + kParts - 1) / kParts;
    extern __shared__ __align__(16) unsigned char query_rows_mem[];
    unsigned char *sT = query_rows_mem;
    double *qin = reinterpret_cast<double *>(query_rows_mem + (size_t)D * pad_row_bytes<D>());
    float *qpv = reinterpret_cast<float *>(qin + (size_t)NH * D);
    const int row0 = blockIdx.x * RB, j = blockIdx.y, t = threadIdx.x, warp = t >> 5, lane = t & 31;
    grid_dependency_wait();
    {
        const float *tj = t_q + (size_t)j * D * D;
        const uint32_t base = smem_addr(sT);
#pragma unroll 8
        for (int i = t; i < D * D / 4; i += kQueryThreads)
            cp_async16(base + (uint32_t)((i / (D / 4)) * pad_row_bytes<D>() + (i % (D / 4)) * 16), tj + 4 * i);
    }
    for (int i = t; i < NH * D; i += kQueryThreads) {   // (row, head), channel
        const int n = i / D, c = i % D, row = row0 + n / G;
        qin[c * NH + n] = row < rows ? (double)load_elem_vol(q, dtype, ((size_t)row * hq + (size_t)j * G + n % G) * D + c) : 0.0;
    }
    cp_async_wait_all();
    __syncthreads();
    {
        // thread = channel c of kPer of the heads
        const int c = t % D, n0 = t / D * kPer;
        static_assert(NH % kPer == 0, "a thread's row heads");
        if (n0 < NH) {
            double acc[kPer];
            dot_rows_pad<D, kPer>(sT, c, qin + n0, NH, acc);
#pragma unroll
            for (int n = 0; n < kPer; ++n) qpv[(n0 + n) * D + c] = __double2float_rn(acc[n]);
        }
    }
    __syncthreads();
    grid_dependents_launch();
    const int nk = keep_count(D, pct);
    for (int n = warp; n < NH; n += kQueryThreads / 32) {
        const int row = row0 + n / G;
        if (row >= rows) break;
        const float *qp = qpv + n * D;
        uint32_t kmask[NG];
        select_kept<NG>(qp, nk, lane, kmask);
        float v[NG], hm = 0.0f;
        int before = 0;
        const size_t at = (size_t)row * hq + (size_t)j * G + n % G;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            const bool kept = (kmask[g] >> lane) & 1u;
            v[g] = kept && (g > 0 || lane > 0) ? qp[lane + 32 * g] : 0.0f;
            hm = fmaxf(hm, fabsf(v[g]));
            if (sel_out && kept)
                sel_out[at * nk + before + __popc(kmask[g] & ((1u << lane) - 1u))] = (int16_t)(lane + 32 * g);
            before += __popc(kmask[g]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) hm = fmaxf(hm, __shfl_xor_sync(0xffffffffu, hm, o));
        const int e = (int)(__float_as_uint(hm) >> 23);   // biased exponent: 0 zero or subnormal, 255 not finite
        const int k = e == 0 || e == 255 ? 0 : 14 - (e - 127);
#pragma unroll
        for (int g = 0; g < NG; ++g)
            qr[at * D + rows_channel_pos(lane + 32 * g)] = __half_as_ushort(__float2half_rn(ldexpf(v[g], k)));
        if (lane == 0) head[at] = make_float2(ldexpf(qscale, -k), qp[0] * qscale);
    }
}

}  // namespace dqk
