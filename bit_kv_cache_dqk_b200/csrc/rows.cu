// rows.cu -- libdualqk: the rotated appends, the shared-prefix decode and the
// cross attention of the C ABI (host side and kernels; see include/dualqk.h).
#include <cuda.h>

#include "host.cuh"

#include "append.cuh"
#include "bf16.cuh"
#include "qrows.cuh"
#include "rope.cuh"
#include "rows.cuh"

unsigned int dqk_rows_take_error(bool &failed) { return take_error_word(failed); }

// ---------------------------------------------------------------------------
// Rotated appends: rotary embedding, cache append and query rotation in one launch.
// ---------------------------------------------------------------------------
namespace {

struct RopeCall {
    const dqk_layer_desc *layer;
    const dqk_rope_desc *rope;
    const void *k;
    long long k_stride;
    const void *v;
    long long v_stride;
    const void *q;
    long long q_stride;
    void *q_out;
    long long q_out_stride;
    dqk_dtype dtype;
    int batch;
    const int *new_lens, *seq_before;
    int max_new;
    const int *positions, *page_table;
    int max_pages;
    cudaStream_t stream;
};

dqk_status check_rope(const RopeCall &a, RopeParams &p) {
    const dqk_layer_desc *L = a.layer;
    const dqk_rope_desc *r = a.rope;
    if (!r || !a.k || !a.v || !a.new_lens || !a.seq_before || !a.page_table) return DQK_ERR_INVALID_ARG;
    if (!r->cos_sin || !aligned(r->cos_sin, 16) || r->max_position <= 0) return DQK_ERR_INVALID_ARG;
    if (r->interleaved != 0 && r->interleaved != 1) return DQK_ERR_INVALID_ARG;
    if (r->rotary_dim <= 0 || r->rotary_dim > L->head_dim || r->rotary_dim % 16) return DQK_ERR_UNSUPPORTED;
    if (a.dtype != DQK_F32 && a.dtype != DQK_BF16) return DQK_ERR_INVALID_ARG;
    if (a.batch <= 0 || a.max_pages <= 0 || a.max_new < 0) return DQK_ERR_INVALID_ARG;
    if (!a.q != !a.q_out) return DQK_ERR_INVALID_ARG;
    // rows are read and written in 16-byte pieces
    const long long piece = a.dtype == DQK_BF16 ? 8 : 4, kv = (long long)L->num_kv_heads * L->head_dim,
                    qw = (long long)L->num_q_heads * L->head_dim;
    if (!aligned(a.k, 16) || !aligned(a.v, 16) || a.k_stride < kv || a.v_stride < kv || a.k_stride % piece ||
        a.v_stride % piece)
        return DQK_ERR_INVALID_ARG;
    if (a.q && (!aligned(a.q, 16) || !aligned(a.q_out, 16) || a.q_stride < qw || a.q_out_stride < qw ||
                a.q_stride % piece || a.q_out_stride % piece))
        return DQK_ERR_INVALID_ARG;
    if (a.q && a.q == a.q_out && a.q_stride != a.q_out_stride) return DQK_ERR_INVALID_ARG;
    p = RopeParams{};
    p.k = a.k;
    p.v = a.v;
    p.q = a.q;
    p.q_out = a.q_out;
    p.k_stride = a.k_stride;
    p.v_stride = a.v_stride;
    p.q_stride = a.q_stride;
    p.q_out_stride = a.q_out_stride;
    p.dtype = (int)a.dtype;
    p.batch = a.batch;
    p.hq = L->num_q_heads;
    p.hkv = L->num_kv_heads;
    p.new_lens = a.new_lens;
    p.seq_before = a.seq_before;
    p.positions = a.positions;
    p.max_new = a.max_new;
    p.cos_sin = r->cos_sin;
    p.max_position = r->max_position;
    p.rotary = r->rotary_dim;
    p.interleaved = r->interleaved;
    p.page_table = a.page_table;
    p.max_pages = a.max_pages;
    p.pool = static_cast<uint8_t *>(L->pool);
    p.num_pages = L->num_pages;
    p.t_k = L->t_k;
    p.v_ch0 = L->v_ch0_protect;
    return DQK_OK;
}

// CTAs of a launch with `rows` new rows of a sequence per CTA.
dqk_status rope_grid(RopeParams &p, int rows, unsigned &gx) {
    p.tiles = (int)(((long long)p.max_new + rows - 1) / rows);
    const long long n = (long long)p.batch * p.tiles;
    if (n > 0x7fffffffLL) return DQK_ERR_UNSUPPORTED;
    gx = (unsigned)n;
    return DQK_OK;
}

template <int D>
dqk_status run_rope_b16(RopeParams &p, cudaStream_t s) {
    unsigned gx = 0;
    const dqk_status st = rope_grid(p, kRopeTile, gx);
    if (st != DQK_OK) return st;
    k_rope_append_b16<D><<<gx, kRopeThreads, 0, s>>>(p);
    return launch_status();
}

template <int D, int NS>
dqk_status run_rope_rows(RopeParams &p, cudaStream_t s) {
    unsigned gx = 0;
    dqk_status st = rope_grid(p, 1, gx);
    if (st != DQK_OK) return st;
    const size_t smem = append_rows_smem<D, NS, 1>();
    st = prepare_kernel<k_rope_append_rows<D, NS>>(current_device(), smem, D);
    if (st != DQK_OK) return st;
    k_rope_append_rows<D, NS><<<dim3(gx, p.hkv + (p.q ? 1 : 0)), D, smem, s>>>(p);
    return launch_status();
}

template <int D, int NS, int RW>
dqk_status run_rope_tile(RopeParams &p, cudaStream_t s) {
    unsigned gx = 0;
    dqk_status st = rope_grid(p, kRopeTileWarps * RW, gx);
    if (st != DQK_OK) return st;
    constexpr size_t smem = sizeof(RopeTileSmem<D, NS, RW>);
    st = prepare_kernel<k_rope_append_tile<D, NS, RW>>(current_device(), smem, kRopeTileThreads);
    if (st != DQK_OK) return st;
    k_rope_append_tile<D, NS, RW><<<dim3(gx, p.hkv), kRopeTileThreads, smem, s>>>(p);
    return launch_status();
}

// One row per CTA, or tiles of 16 or 64 rows: whichever takes least by what they measured (us at head_dim 128,
// 148 SMs): a row per CTA 10 and 13 more per 7 CTAs of an SM, a wave of tiles of 16 rows 13 and 4 before the first, of
// 64 rows 17 and 13.  E.g. 16 sequences, 8 kv heads: 1 row each 12, 15, 19; 8 rows 23, 15, 23; 64 rows 118, 57, 30;
// 1 sequence of 256 rows 35, 17, 29; of 8192 rows 908, 393, 193.  The same rule serves head_dim 64, where all three
// are 2 to 3 times faster: over 38 sizes its choice was the fastest, but for 64 sequences of 8 rows (28 us in tiles of 16
// where a row per CTA takes 26); 1 sequence of 8192 rows 439, 205, 113, 16 of 64 rows 42, 31, 19, 64 of 1 row 13, 27, 41.
// The lengths are on the device, so the rule goes by max_new.
template <int D, int NS>
dqk_status run_rope_int2(RopeParams &p, cudaStream_t s) {
    const int sms = device_sms(current_device());
    if (sms <= 0) return DQK_ERR_CUDA;
    const double lists = (double)p.batch * p.hkv;
    auto waves = [&](int rows) { return std::ceil(lists * (((long long)p.max_new + rows - 1) / rows) / sms); };
    const double row = 10 + 13 * lists * p.max_new / (7.0 * sms), tile16 = 4 + 13 * waves(16), tile64 = 13 + 17 * waves(64);
    if (row <= std::min(tile16, tile64)) return run_rope_rows<D, NS>(p, s);
    if (tile16 < tile64) return run_rope_tile<D, NS, 2>(p, s);
    return run_rope_tile<D, NS, 8>(p, s);
}

}  // namespace

extern "C" {

#define DQK_ROPE_ARGS                                                                                      \
    const dqk_layer_desc *layer, const dqk_rope_desc *rope, const void *k, long long k_stride, const void *v, \
        long long v_stride, const void *q, long long q_stride, void *q_out, long long q_out_stride,        \
        dqk_dtype dtype, int batch, const int *new_lens, const int *seq_lens_before, int max_new,          \
        const int *positions, const int *page_table, int max_pages, dqk_stream_t stream
#define DQK_ROPE_PACK                                                                                      \
    const RopeCall a{layer, rope, k, k_stride, v, v_stride, q, q_stride, q_out, q_out_stride, dtype, batch, \
                     new_lens, seq_lens_before, max_new, positions, page_table, max_pages,                 \
                     static_cast<cudaStream_t>(stream)}

dqk_status dqk_rope_append(DQK_ROPE_ARGS) {
    DQK_ROPE_PACK;
    dqk_status st = check_layer(layer);
    if (st != DQK_OK) return st;
    if (!layer->t_k || !aligned(layer->t_k, 16)) return DQK_ERR_INVALID_ARG;
    RopeParams p;
    st = check_rope(a, p);
    if (st != DQK_OK || max_new == 0) return st;
    const bool one = layer->group_size == layer->head_dim;
    if (layer->head_dim == 128) return one ? run_rope_int2<128, 1>(p, a.stream) : run_rope_int2<128, 4>(p, a.stream);
    return one ? run_rope_int2<64, 1>(p, a.stream) : run_rope_int2<64, 2>(p, a.stream);
}

dqk_status dqk_bf16_rope_append(DQK_ROPE_ARGS) {
    DQK_ROPE_PACK;
    dqk_status st = check_layer_b16(layer);
    if (st != DQK_OK) return st;
    RopeParams p;
    st = check_rope(a, p);
    if (st != DQK_OK || max_new == 0) return st;
    return layer->head_dim == 128 ? run_rope_b16<128>(p, a.stream) : run_rope_b16<64>(p, a.stream);
}

}  // extern "C"

// ---------------------------------------------------------------------------
// Query rows over shared lists: the decode of a batch behind shared prefixes
// (INT2 and BF16 caches) and cross attention (BF16 cache).
// ---------------------------------------------------------------------------
namespace {

// Workspace: [query rows fp16 | their scales and factors of channel 0 | plan | group records | own records],
// sections 256-byte aligned.
struct RowsPlanHost {
    int d, G, bb;
    bool rec_pairs;
    long long rec_step;
    size_t off_head, off_plan, off_rec, off_own, bytes;
    long long max_units;
};

bool plan_rows(const dqk_layer_desc *L, bool int2, int total_rows, int n_groups, int max_pages, int n_own, int own_pages,
               RowsPlanHost &P) {
    P.d = L->head_dim;
    P.G = L->num_q_heads / L->num_kv_heads;
    const long long hkv = L->num_kv_heads;
    if ((long long)total_rows * L->num_q_heads >= (1LL << 31) / 2) return false;
    if (((long long)max_pages + own_pages) * kPage >= (1LL << 31)) return false;
    if (L->num_pages * hkv >= (1LL << 31)) return false;   // block numbers are tensor-copy coordinates
    const long long tiles = n_groups + (long long)total_rows * P.G / kRowsTile;   // >= the groups' row tiles
    if (tiles * hkv >= (1LL << 31) / 2 || (long long)n_own * hkv >= (1LL << 31) / 2) return false;
    P.max_units = hkv * (2 * tiles * ((max_pages + kRowsPages - 1) / kRowsPages) +
                         (long long)n_own * ((own_pages + kRowsPages - 1) / kRowsPages));
    // records (rows_record): both forms grow with every size, hence so does the smaller one
    const long long ctas = std::min<long long>(kRowsMaxCtas, P.max_units);
    P.rec_step = 2 * std::min<long long>(kRowsHalf, (long long)total_rows * P.G);
    const long long by_item = ctas * P.rec_step + 2 * (long long)total_rows * L->num_q_heads, by_cta = 2 * ctas * P.rec_step;
    P.rec_pairs = !n_own && by_cta < by_item;
    P.bb = int2 ? make_layout(P.d, L->v_ch0_protect, P.d / L->group_size).bytes : b16_block_bytes(P.d);
    const size_t heads = (size_t)total_rows * L->num_q_heads;
    P.off_head = int2 ? round_up(heads * P.d * 2, 256) : 0;
    P.off_plan = P.off_head + (int2 ? round_up(heads * sizeof(float2), 256) : 0);
    P.off_rec = P.off_plan + round_up(rows_plan_bytes((size_t)n_groups + n_own), 256);
    const size_t row = rec_stride(P.d) * sizeof(float);
    P.off_own = P.off_rec + round_up((size_t)(P.rec_pairs ? by_cta : by_item) * row, 256);
    P.bytes = P.off_own + round_up((size_t)(n_own ? ctas + n_own * hkv : 0) * 2 * P.G * row, 256);
    return true;
}

// The BF16 pool as a tensor of 16-bit elements [block][column block of 64][32 token rows, K then V][64]:
// one box is one page's 16 keys or values.
typedef CUresult (*EncodeTiled)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

dqk_status pool_map(const dqk_layer_desc *L, CUtensorMap &map) {
    static std::atomic<EncodeTiled> fn{nullptr};
    EncodeTiled encode = fn.load(std::memory_order_acquire);
    if (!encode) {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
            found != cudaDriverEntryPointSuccess || !f)
            return DQK_ERR_CUDA;
        encode = reinterpret_cast<EncodeTiled>(f);
        fn.store(encode, std::memory_order_release);
    }
    const cuuint64_t d = (cuuint64_t)L->head_dim;
    const cuuint64_t dims[4] = {64, 2 * kPage, d / 64, (cuuint64_t)(L->num_pages * L->num_kv_heads)};
    const cuuint64_t strides[3] = {2 * d, 128, (cuuint64_t)b16_block_bytes(L->head_dim)};
    const cuuint32_t box[4] = {64, kPage, (cuuint32_t)(d / 64), 1}, one[4] = {1, 1, 1, 1};
    return encode(&map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, L->pool, dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
                   CUDA_SUCCESS
               ? DQK_OK
               : DQK_ERR_CUDA;
}

struct RowsCall {
    const dqk_layer_desc *layer;
    bool int2;
    const void *q;
    dqk_dtype q_dtype;
    int total_rows, n_groups;
    const int *row_start, *kv_lens, *table;
    int max_pages;
    int n_own;                            // rows with an own list (0: none)
    const int *own_lens, *own_table;
    int own_pages;
    int pct;
    void *out;
    dqk_dtype out_dtype;
    int16_t *sel_out;
    void *ws;
    size_t ws_bytes;
    cudaStream_t stream;
    bool zero_rest;                       // rows of no group: zeros, or left as they were
    bool stall = false;                   // test only
};

template <int D, int kFmt, int kW, int NS, bool VCH0>
dqk_status run_rows_kernels(const RowsCall &a, RowsParams &p, const RowsPlanHost &P, int dev) {
    using T = RowsShape<D, kFmt>;
    // shared memory: 1024 bytes of alignment, the query tiles, the rings
    constexpr size_t kRoom = 227 * 1024 - 1024 - sizeof(RowsBars) - 2 * T::kParts * T::kTile;
    // a key tile is free again as soon as its scores are formed, a value tile only after its unit's weights: with an
    // odd number the values have one more
    const int tiles = T::kInt2 ? 4 : (int)std::min<size_t>(kRowsMaxTiles, kRoom / T::kTile);
    p.ktiles = tiles / 2;
    p.vtiles = tiles - p.ktiles;
    // page flags: at most kRowsFlags units between their copies and the softmax
    constexpr size_t kCh0 = T::kInt2 ? kRowsCh0 * rows_ch0_bytes(VCH0) : 0;
    p.raw_stages = T::kInt2 ? (int)std::min<size_t>(kRowsMaxRaw, (kRoom - 4 * T::kTile - kCh0) / (kRowsPages * P.bb)) : 0;
    const size_t smem = 1024 + 2 * T::kParts * T::kTile + (size_t)tiles * T::kTile + (size_t)p.raw_stages * kRowsPages * P.bb + kCh0;
    dqk_status st = prepare_kernel<k_rows<D, kFmt, kW, NS, VCH0>>(dev, smem, T::kThreads);
    if (st != DQK_OK) return st;
    CUtensorMap map = {};
    if (!T::kInt2) {
        st = pool_map(a.layer, map);
        if (st != DQK_OK) return st;
    }
    st = launch_overlapped(k_rows<D, kFmt, kW, NS, VCH0>, dim3(p.num_ctas), T::kThreads, smem, a.stream, p, map);
    if (st != DQK_OK) return st;
    if (p.n_own > 0) {
        return launch_overlapped(k_rows_merge<D>, dim3((unsigned)p.total_rows, (p.hq + kRowsMergeWarps - 1) / kRowsMergeWarps),
                                 32 * kRowsMergeWarps, 0, a.stream, p);
    }
    const int rows = (int)std::min<long long>(kRowsTile, (long long)p.total_rows * p.G);
    return launch_overlapped(k_rows_merge_items<D>,
                             dim3((unsigned)(p.num_ctas - 1 + std::min(p.n_groups, 32)),
                                  (rows + kRowsMergeWarps * kRowsMergeHeads - 1) / (kRowsMergeWarps * kRowsMergeHeads)),
                             32 * kRowsMergeWarps, 0, a.stream, p);
}

// the INT2 cache: transformed and pruned fp16 query rows first
template <int D, int G, int RB>
dqk_status launch_query_rows(const RowsCall &a, const RowsParams &p, int dev, uint16_t *rows, float2 *head) {
    const size_t smem = query_rows_smem<D, G, RB>();
    const dqk_status st = prepare_kernel<k_query_rows<D, G, RB>>(dev, smem, kQueryThreads);
    if (st != DQK_OK) return st;
    return launch_overlapped(k_query_rows<D, G, RB>, dim3((p.total_rows + RB - 1) / RB, p.hkv), kQueryThreads, smem, a.stream,
                             a.layer->t_q, a.q, (int)a.q_dtype, p.total_rows, p.hq, a.pct, p.qs, rows, head, a.sel_out);
}

template <int D, int G>
dqk_status run_query_rows(const RowsCall &a, const RowsParams &p, int dev, uint16_t *rows, float2 *head) {
    // four rows per staged transform once one row each makes more than three CTAs per SM: the whole decode with 1 and
    // 4 (us; 148 SMs, 8 kv heads, 1024 shared tokens) 38 and 42 at 32 rows, 49 and 51 at 48, 63 and 59 at 64, 97 and 93 at 128
    return (long long)p.total_rows * p.hkv > 3LL * device_sms(dev) ? launch_query_rows<D, G, 4>(a, p, dev, rows, head)
                                                     : launch_query_rows<D, G, 1>(a, p, dev, rows, head);
}

template <int D>
dqk_status run_rows_d(const RowsCall &a, const RowsPlanHost &P, RowsParams &p, int dev) {
    if (!a.int2) {
        if (a.out_dtype == DQK_BF16)
            return a.q_dtype == DQK_BF16 ? run_rows_kernels<D, 0, 1, 1, false>(a, p, P, dev)
                                         : run_rows_kernels<D, 1, 1, 1, false>(a, p, P, dev);
        return a.q_dtype == DQK_BF16 ? run_rows_kernels<D, 0, 2, 1, false>(a, p, P, dev)
                                     : run_rows_kernels<D, 1, 2, 1, false>(a, p, P, dev);
    }
    char *ws = static_cast<char *>(a.ws);
    uint16_t *rows = reinterpret_cast<uint16_t *>(ws);
    float2 *head = reinterpret_cast<float2 *>(ws + P.off_head);
    const dqk_status st = P.G == 1   ? run_query_rows<D, 1>(a, p, dev, rows, head)
                          : P.G == 2 ? run_query_rows<D, 2>(a, p, dev, rows, head)
                          : P.G == 4 ? run_query_rows<D, 4>(a, p, dev, rows, head)
                                     : run_query_rows<D, 8>(a, p, dev, rows, head);
    if (st != DQK_OK) return st;
    p.q = rows;
    p.q_head = head;
    const bool one = a.layer->group_size == D, v0 = a.layer->v_ch0_protect != 0;
    if (one) return v0 ? run_rows_kernels<D, 2, 1, 1, true>(a, p, P, dev)
                       : run_rows_kernels<D, 2, 1, 1, false>(a, p, P, dev);
    return v0 ? run_rows_kernels<D, 2, 1, D / kGroup, true>(a, p, P, dev)
              : run_rows_kernels<D, 2, 1, D / kGroup, false>(a, p, P, dev);
}

dqk_status run_rows(const RowsCall &a) {
    const dqk_layer_desc *L = a.layer;
    if (!a.q || !a.row_start || !a.kv_lens || !a.table || !a.out || !a.ws) return DQK_ERR_INVALID_ARG;
    if (a.q_dtype != DQK_F32 && a.q_dtype != DQK_BF16) return DQK_ERR_INVALID_ARG;
    if (a.out_dtype != DQK_F32 && a.out_dtype != DQK_BF16) return DQK_ERR_INVALID_ARG;
    if (!aligned(a.q, 16) || !aligned(a.out, 16) || !aligned(a.ws, 256)) return DQK_ERR_INVALID_ARG;
    RowsPlanHost P;
    if (!plan_rows(L, a.int2, a.total_rows, a.n_groups, a.max_pages, a.n_own, a.own_pages, P)) return DQK_ERR_UNSUPPORTED;
    if (a.ws_bytes < P.bytes) return DQK_ERR_WORKSPACE_TOO_SMALL;
    const int dev = current_device();
    if (dev < 0 || dev >= kMaxDevices) return DQK_ERR_CUDA;
    const int sms = device_sms(dev);
    if (sms <= 0) return DQK_ERR_CUDA;
    RowsParams p = {};
    p.pool = static_cast<const uint8_t *>(L->pool);
    p.num_pages = L->num_pages;
    p.n_groups = a.n_groups;
    p.total_rows = a.total_rows;
    p.row_start = a.row_start;
    p.kv_lens = a.kv_lens;
    p.table = a.table;
    p.max_pages = a.max_pages;
    p.n_own = a.n_own;
    p.own_lens = a.own_lens;
    p.own_table = a.own_table;
    p.own_max_pages = a.own_pages;
    p.q = a.q;
    p.qs = (float)(1.4426950408889634 / std::sqrt((double)P.d));
    char *ws = static_cast<char *>(a.ws);
    p.plan = reinterpret_cast<RowsPlan *>(ws + P.off_plan);
    p.rec = reinterpret_cast<float *>(ws + P.off_rec);
    p.own_rec = reinterpret_cast<float *>(ws + P.off_own);
    p.rec_pairs = P.rec_pairs;
    p.rec_step = (uint32_t)P.rec_step;
    p.zero_rest = a.zero_rest;
    p.out = a.out;
    p.out_dtype = (int)a.out_dtype;
    p.hq = L->num_q_heads;
    p.hkv = L->num_kv_heads;
    p.G = P.G;
    p.head = a.int2 ? kRowsHeadInt2 : kRowsHeadBf16;
    p.bb = P.bb;
    p.num_ctas = (int)std::max<long long>(1, std::min<long long>(std::min(sms, kRowsMaxCtas), P.max_units));
    p.wait_ns = a.stall ? kStallWaitNs : kRingWaitNs;
    p.stall = a.stall;
    return P.d == 128 ? run_rows_d<128>(a, P, p, dev) : run_rows_d<64>(a, P, p, dev);
}

// Sizes and own lists of a shared-prefix decode.
dqk_status check_prefix(int batch, int n_prefixes, int max_prefix_pages, const int *seq_lens, const int *page_table,
                        int max_pages) {
    if (batch <= 0 || n_prefixes <= 0 || max_prefix_pages <= 0 || max_pages < 0) return DQK_ERR_INVALID_ARG;
    if (max_pages > 0 && (!seq_lens || !page_table)) return DQK_ERR_INVALID_ARG;
    return DQK_OK;
}

}  // namespace

extern "C" {

size_t dqk_prefix_decode_workspace_size(const dqk_layer_desc *layer, int batch, int n_prefixes, int max_prefix_pages,
                                        int max_pages) {
    if (check_layer(layer) != DQK_OK || batch <= 0 || n_prefixes <= 0 || max_prefix_pages <= 0 || max_pages < 0) return 0;
    RowsPlanHost P;
    return plan_rows(layer, true, batch, n_prefixes, max_prefix_pages, max_pages ? batch : 0, max_pages, P) ? P.bytes : 0;
}

size_t dqk_bf16_prefix_decode_workspace_size(const dqk_layer_desc *layer, int batch, int n_prefixes, int max_prefix_pages,
                                             int max_pages) {
    if (check_layer_b16(layer) != DQK_OK || batch <= 0 || n_prefixes <= 0 || max_prefix_pages <= 0 || max_pages < 0) return 0;
    RowsPlanHost P;
    return plan_rows(layer, false, batch, n_prefixes, max_prefix_pages, max_pages ? batch : 0, max_pages, P) ? P.bytes : 0;
}

size_t dqk_bf16_cross_attention_workspace_size(const dqk_layer_desc *layer, int batch, int total_q, int max_pages) {
    if (check_layer_b16(layer) != DQK_OK || batch <= 0 || total_q <= 0 || max_pages <= 0) return 0;
    RowsPlanHost P;
    return plan_rows(layer, false, total_q, batch, max_pages, 0, 0, P) ? P.bytes : 0;
}

dqk_status dqk_prefix_decode(const dqk_layer_desc *layer, const void *q, dqk_dtype q_dtype, int batch, int n_prefixes,
                             const int *prefix_start, const int *prefix_lens, const int *prefix_table, int max_prefix_pages,
                             const int *seq_lens, const int *page_table, int max_pages, int sparsity_pct, void *out,
                             dqk_dtype out_dtype, int16_t *sel_out, void *workspace, size_t workspace_bytes,
                             dqk_stream_t stream) {
    dqk_status st = check_layer(layer);
    if (st != DQK_OK) return st;
    if (!layer->t_q || !aligned(layer->t_q, 16) || sparsity_pct < 0 || sparsity_pct > 99) return DQK_ERR_INVALID_ARG;
    st = check_prefix(batch, n_prefixes, max_prefix_pages, seq_lens, page_table, max_pages);
    if (st != DQK_OK) return st;
    return run_rows(RowsCall{layer, true, q, q_dtype, batch, n_prefixes, prefix_start, prefix_lens, prefix_table,
                             max_prefix_pages, max_pages ? batch : 0, seq_lens, page_table, max_pages, sparsity_pct, out,
                             out_dtype, sel_out, workspace, workspace_bytes, static_cast<cudaStream_t>(stream), true});
}

dqk_status dqk_bf16_prefix_decode(const dqk_layer_desc *layer, const void *q, dqk_dtype q_dtype, int batch, int n_prefixes,
                                  const int *prefix_start, const int *prefix_lens, const int *prefix_table,
                                  int max_prefix_pages, const int *seq_lens, const int *page_table, int max_pages, void *out,
                                  dqk_dtype out_dtype, void *workspace, size_t workspace_bytes, dqk_stream_t stream) {
    dqk_status st = check_layer_b16(layer);
    if (st != DQK_OK) return st;
    st = check_prefix(batch, n_prefixes, max_prefix_pages, seq_lens, page_table, max_pages);
    if (st != DQK_OK) return st;
    return run_rows(RowsCall{layer, false, q, q_dtype, batch, n_prefixes, prefix_start, prefix_lens, prefix_table,
                             max_prefix_pages, max_pages ? batch : 0, seq_lens, page_table, max_pages, 0, out, out_dtype,
                             nullptr, workspace, workspace_bytes, static_cast<cudaStream_t>(stream), true});
}

dqk_status dqk_test_prefix_stall(const dqk_layer_desc *layer, int bf16, const void *q, dqk_dtype q_dtype, int batch,
                                 int n_prefixes, const int *prefix_start, const int *prefix_lens, const int *prefix_table,
                                 int max_prefix_pages, const int *seq_lens, const int *page_table, int max_pages,
                                 int sparsity_pct, void *out, dqk_dtype out_dtype, int16_t *sel_out, void *workspace,
                                 size_t workspace_bytes, dqk_stream_t stream) {
    dqk_status st = bf16 ? check_layer_b16(layer) : check_layer(layer);
    if (st != DQK_OK) return st;
    if (!bf16 && (!layer->t_q || !aligned(layer->t_q, 16) || sparsity_pct < 0 || sparsity_pct > 99)) return DQK_ERR_INVALID_ARG;
    st = check_prefix(batch, n_prefixes, max_prefix_pages, seq_lens, page_table, max_pages);
    if (st != DQK_OK) return st;
    return run_rows(RowsCall{layer, !bf16, q, q_dtype, batch, n_prefixes, prefix_start, prefix_lens, prefix_table,
                             max_prefix_pages, max_pages ? batch : 0, seq_lens, page_table, max_pages, bf16 ? 0 : sparsity_pct,
                             out, out_dtype, bf16 ? nullptr : sel_out, workspace, workspace_bytes,
                             static_cast<cudaStream_t>(stream), true, true});
}

dqk_status dqk_bf16_cross_attention(const dqk_layer_desc *layer, const void *q, dqk_dtype q_dtype, int batch, int total_q,
                                    const int *q_start, const int *kv_lens, const int *page_table, int max_pages, void *out,
                                    dqk_dtype out_dtype, void *workspace, size_t workspace_bytes, dqk_stream_t stream) {
    dqk_status st = check_layer_b16(layer);
    if (st != DQK_OK) return st;
    if (batch <= 0 || total_q <= 0 || max_pages <= 0) return DQK_ERR_INVALID_ARG;
    return run_rows(RowsCall{layer, false, q, q_dtype, total_q, batch, q_start, kv_lens, page_table, max_pages, 0, nullptr,
                             nullptr, 0, 0, out, out_dtype, nullptr, workspace, workspace_bytes,
                             static_cast<cudaStream_t>(stream), false});
}

}  // extern "C"
