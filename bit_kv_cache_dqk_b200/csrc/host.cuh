// host.cuh -- host-side pieces of the C ABI that its translation units share:
// argument checks, device queries, kernel preparation and launches.
#pragma once

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "attend.cuh"
#include "common.cuh"

namespace {

using namespace dqk;

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

constexpr int kMaxDevices = 64;

dqk_status check_layer(const dqk_layer_desc *L) {
    if (!L) return DQK_ERR_INVALID_ARG;
    if (L->head_dim != 64 && L->head_dim != 128) return DQK_ERR_UNSUPPORTED;
    if (L->num_kv_heads <= 0 || L->num_q_heads <= 0 || L->num_q_heads % L->num_kv_heads)
        return DQK_ERR_INVALID_ARG;
    const int G = L->num_q_heads / L->num_kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 8) return DQK_ERR_UNSUPPORTED;
    if (L->page_size != kPage) return DQK_ERR_UNSUPPORTED;
    // scale groups of 32 channels, or one group over the whole head
    if (L->group_size != kGroup && L->group_size != L->head_dim) return DQK_ERR_UNSUPPORTED;
    if (L->v_ch0_protect != 0 && L->v_ch0_protect != 1) return DQK_ERR_INVALID_ARG;
    if (!L->pool || !aligned(L->pool, 16) || L->num_pages <= 0) return DQK_ERR_INVALID_ARG;
    return DQK_OK;
}

int current_device() {
    int dev = -1;
    return cudaGetDevice(&dev) == cudaSuccess ? dev : -1;
}

int device_sms(int dev) {
    int sms = 0;
    if (dev < 0 || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return sms;
}

dqk_status check_layer_b16(const dqk_layer_desc *L) {
    if (!L) return DQK_ERR_INVALID_ARG;
    if (L->head_dim != 64 && L->head_dim != 128) return DQK_ERR_UNSUPPORTED;
    if (L->num_kv_heads <= 0 || L->num_q_heads <= 0 || L->num_q_heads % L->num_kv_heads)
        return DQK_ERR_INVALID_ARG;
    const int G = L->num_q_heads / L->num_kv_heads;
    if (G != 1 && G != 2 && G != 4 && G != 8) return DQK_ERR_UNSUPPORTED;
    if (L->page_size != kPage) return DQK_ERR_UNSUPPORTED;
    if (!L->pool || !aligned(L->pool, 16) || L->num_pages <= 0) return DQK_ERR_INVALID_ARG;
    return DQK_OK;
}

dqk_status launch_status() {
    return cudaGetLastError() == cudaSuccess ? DQK_OK : DQK_ERR_CUDA;
}

// Once per (kernel instance, device): the dynamic shared-memory bound, the
// largest carveout (consecutive kernels then do not make the SMs switch their
// L1 / shared split), and a check that one CTA fits on an SM (a cooperative
// launch needs every CTA resident).  Thread-safe; later calls cost a lookup.
template <auto Kernel>
dqk_status prepare_kernel(int dev, size_t smem, int threads) {
    static std::mutex mu;
    static size_t set_smem[kMaxDevices] = {};
    if (dev < 0 || dev >= kMaxDevices) return DQK_ERR_UNSUPPORTED;
    std::lock_guard<std::mutex> lock(mu);
    if (set_smem[dev] != 0 && set_smem[dev] >= smem) return DQK_OK;
    if (cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return DQK_ERR_CUDA;
    (void)cudaFuncSetAttribute(Kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                               (int)cudaSharedmemCarveoutMaxShared);
    int per_sm = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, Kernel, threads, smem) != cudaSuccess)
        return DQK_ERR_CUDA;
    if (per_sm < 1) return DQK_ERR_UNSUPPORTED;
    set_smem[dev] = smem;
    return DQK_OK;
}

constexpr unsigned long long kRingWaitNs = kWaitLimitNs;   // 1 s
constexpr unsigned long long kStallWaitNs = 1000000ull;    // 1 ms: the test-only stalls

// Launch with programmatic stream serialization: the kernel may start while the
// previous one finishes, and waits for it (griddepcontrol.wait) before reading anything.
template <typename... KArgs, typename... Args>
dqk_status launch_overlapped(void (*kernel)(KArgs...), dim3 grid, unsigned block, size_t smem, cudaStream_t stream,
                             Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...) == cudaSuccess ? DQK_OK : DQK_ERR_CUDA;
}

// This translation unit's device error word, read and cleared.
inline unsigned int take_error_word(bool &failed) {
    unsigned int word = 0, zero = 0;
    if (cudaMemcpyFromSymbol(&word, g_dqk_device_error, sizeof(word)) != cudaSuccess ||
        (word && cudaMemcpyToSymbol(g_dqk_device_error, &zero, sizeof(zero)) != cudaSuccess))
        failed = true;
    return word;
}

}  // namespace

// The same of rows.cu.
unsigned int dqk_rows_take_error(bool &failed);
