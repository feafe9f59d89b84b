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

// Shared memory: T_Q[j] in padded rows, the query rows [D][G] fp64 (i-major), q' [G][D] fp32.
template <int D, int G>
__host__ __device__ constexpr size_t query_rows_smem() {
    return (size_t)D * pad_row_bytes<D>() + (size_t)G * D * 12;
}
template <int D, int G>
__host__ __device__ constexpr int query_rows_threads() { return 32 * (D / 32 > G ? D / 32 : G); }

// CTA per (query row, kv head).  Row head (row, h) becomes
//   qr [row][hq][D] fp16 = rne(2^k q'_c) on the kept channels, 0 elsewhere, in the
//   channel order of the key operand tiles (rows_channel_pos), with
//   k such that the largest kept |q'_c| lies in [2^14, 2^15): fp16's 11 bits then
//   cover channels down to 2^-28 of it;
//   scale [row][hq] = 2^-k log2(e)/sqrt(d), which the scores are multiplied by.
// A query of zeros (or subnormals) becomes a row of zeros: every score 0.
template <int D, int G>
__global__ void __launch_bounds__(query_rows_threads<D, G>()) k_query_rows(
    const float *__restrict__ t_q, const void *__restrict__ q, int dtype, int hq, int pct, float qscale,
    uint16_t *__restrict__ qr, float *__restrict__ scale, int16_t *__restrict__ sel_out) {
    constexpr int NG = D / 32;
    extern __shared__ __align__(16) unsigned char query_rows_mem[];
    unsigned char *sT = query_rows_mem;
    double *qin = reinterpret_cast<double *>(query_rows_mem + (size_t)D * pad_row_bytes<D>());
    float *qpv = reinterpret_cast<float *>(qin + (size_t)G * D);
    const int row = blockIdx.x, j = blockIdx.y, t = threadIdx.x, warp = t >> 5, lane = t & 31;
    grid_dependency_wait();
    {
        const float *tj = t_q + (size_t)j * D * D;
        const uint32_t base = smem_addr(sT);
#pragma unroll 4
        for (int i = t; i < D * D / 4; i += blockDim.x)
            cp_async16(base + (uint32_t)((i / (D / 4)) * pad_row_bytes<D>() + (i % (D / 4)) * 16), tj + 4 * i);
    }
    const size_t qbase = ((size_t)row * hq + (size_t)j * G) * D;
    for (int i = t; i < G * D; i += blockDim.x) qin[(i % D) * G + i / D] = (double)load_elem_vol(q, dtype, qbase + i);
    cp_async_wait_all();
    __syncthreads();
    if (t < D) {
        double acc[G];
        dot_rows_pad<D, G>(sT, t, qin, G, acc);
#pragma unroll
        for (int n = 0; n < G; ++n) qpv[n * D + t] = __double2float_rn(acc[n]);
    }
    __syncthreads();
    grid_dependents_launch();
    if (warp >= G) return;
    const int nk = keep_count(D, pct);
    const float *qp = qpv + warp * D;
    uint32_t kmask[NG];
    select_kept<NG>(qp, nk, lane, kmask);
    float v[NG], hm = 0.0f;
    int before = 0;
    const size_t at = (size_t)row * hq + (size_t)j * G + warp;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
        const bool kept = (kmask[g] >> lane) & 1u;
        v[g] = kept ? qp[lane + 32 * g] : 0.0f;
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
    if (lane == 0) scale[at] = ldexpf(qscale, -k);
}

}  // namespace dqk
