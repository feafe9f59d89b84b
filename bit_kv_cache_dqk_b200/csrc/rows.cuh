// rows.cuh -- attention of many query rows over shared paged lists: the batch
// behind a shared prefix (every sequence's queries against one page list, read
// once), the sequences' own pages after it, and cross attention (a sequence's
// query tokens against its encoder states).
//
// A group is a run of query rows [row_start[g], row_start[g+1]) that attends
// one list of pages; own list b belongs to query row b alone.  For kv head j a
// row counts G times (its G query heads), so a group of n rows is a matrix of
// n G "row heads" against the list's tokens:
//   S = Q K^T,  P = 2^(S qs - m),  O = P V,   qs = log2(e)/sqrt(d)
// with a reference m and the sum l of P per row head (online softmax).
//
// Work split: item = (group, tile of 256 row heads, kv head), then (own list,
// kv head); unit = 128 tokens of an item.  Units and items have costs (below); CTA
// c takes the units that begin in [cq, (c+1)q) of the cost U of them all, q =
// ceil(U / C), so every CTA does about the same work whatever the lengths.
//
// One CTA per SM, warp-specialized around the tensor core (tcgen05, operands in
// shared memory and TMEM, fp32 accumulators in TMEM):
//   producer warp   brings the pages in (BF16: tensor copies that leave each
//                   128-byte half row in the 128-byte-swizzled operand layout
//                   the block format already is; INT2: 1-D bulk copies of the
//                   packed blocks),
//   unpack warps    (INT2) turn packed blocks into fp16 operand tiles,
//   two softmax warpgroups, one row head per thread,
//   two matrix threads, one per warpgroup, which issue S = Q K^T and O += P V.
// The jobs of a CTA -- (unit, 128 row heads) -- go to the two warpgroups in
// turn: a tile of more than 128 row heads gives each unit to both, its halves;
// a smaller tile gives the units to one and the other, each with its own
// reference, sum and accumulator.  A job goes through in two halves of 64 tokens --
// half h: tokens 8h .. 8h + 7 of every page, in page order -- each with its own 64
// columns of TMEM for S and then P: while a warpgroup turns one
// half's scores into weights, the tensor core takes the other half's weights and
// forms the next job's scores.
//
// What bounds it.  Many row heads: the hand-over between the softmax warpgroups and the tensor core.  A unit of 256
// row heads takes 4300 clocks (BF16, head_dim 128), of which the products are 2050 and the 32768 powers of two 2050 of
// their units (both are busy 41 % of the time on the cross attention below); a half of 64 tokens is 1100 clocks of
// arithmetic and 900 of waiting, reading and writing TMEM.  INT2 takes about 5500: the four warps that unpack keep pace
// with neither, and CTAs of equal work differ by up to 40 %.  Few row
// heads: the chain key tile - scores - weights - values of a unit, 2630 clocks with two units in flight, and DRAM.
// Cross attention of 4 sequences of 540 to 1024 queries over 2121 to 4096 states (169 GFLOP): 218 us, 0.77 PFLOP/s; 64
// sequences behind 128K tokens, INT2 (110 GFLOP): 300 us; 32 sequences behind two documents of up to 32K tokens, BF16
// (354 MB): 86 us, 4.1 TB/s; one query token each for 16 sequences of 750 to 1500 states (74 MB): 30 us, of which about 6
// are the start.  The BF16 instances with weights of one part and the INT2 ones with a protected value channel 0 spill a
// few registers (42 to 46 and 74 to 82 bytes of stores).
#pragma once

#include <cuda.h>

#include "attend.cuh"
#include "common.cuh"
#include "ptx.cuh"

namespace dqk {

constexpr int kRowsTile = 256;                    // row heads of an item
constexpr int kRowsHalf = 128;                    // row heads of a job
constexpr int kRowsKv = 128;                      // tokens of a unit
constexpr int kRowsPages = kRowsKv / kPage;       // pages of a unit
constexpr int kRowsMaxCtas = 160;
constexpr int kRowsUnpackWarps = 4;
constexpr int kRowsFlags = 8;                     // units in flight at most (page flags)
// fp16 weights (INT2) are carried times 2^6, and so is their sum (the factor leaves with it): a
// weight is at most 2^8 (see kRowsSlack), so 2^14 at most, and keeps 11 bits down to 2^-20.
constexpr float kRowsLift = 6.0f;
// The reference m moves only when a score passes it by more than this (log2 units): weights
// are then at most 2^8 and the accumulator is rescaled a few times per item at most.
constexpr float kRowsSlack = 8.0f;

struct RowsParams {
    const uint8_t *pool;
    long long num_pages;
    // groups of query rows and their page lists
    int n_groups, total_rows;
    const int *row_start, *kv_lens, *table;
    int max_pages;
    // own lists of the query rows (n_own = 0: none)
    int n_own;
    const int *own_lens, *own_table;
    int own_max_pages;
    // queries: BF16 cache, the caller's rows [total_rows][hq][D]; INT2 cache,
    // prepared fp16 rows, their scales and their factors of channel 0 (k_query_rows)
    const void *q;
    const float2 *q_head;
    float qs;
    struct RowsPlan *plan;      // what the merge needs of the split (written by the row kernel)
    float *rec, *own_rec;       // split records of the groups' and of the own items
    bool rec_pairs;             // see rows_record
    uint32_t rec_step;
    bool zero_rest;             // rows of no group become zeros
    void *out;
    int out_dtype;
    int head;                   // cost of an item besides its units
    int hq, hkv, G, bb, ktiles, vtiles, raw_stages, num_ctas;
    unsigned long long wait_ns;
    bool stall;                 // test only: CTA 0's producer never fills the stage of its second unit
};

// Tokens of a list, cut to what its page table can hold.
__device__ __forceinline__ int rows_len(const int *lens, int i, int max_pages) {
    const long long cap = (long long)max_pages * kPage;
    const int n = max(lens[i], 0);
    return n > cap ? (int)cap : n;
}
__device__ __forceinline__ int rows_units(int len) { return (int)(((long long)len + kRowsKv - 1) / kRowsKv); }

// First row of group g, inside [0, total_rows].
__device__ __forceinline__ int rows_first(const RowsParams &p, int g) {
    return min(max(p.row_start[g], 0), p.total_rows);
}

// The work is split by cost: of a unit that both warpgroups take, of one that goes to one of them, and of
// an item besides (p.head: its queries, its outputs, the pipeline's end and start).  A CTA's clocks, head_dim
// 128: BF16 4300, 2630 and 4600; INT2 5500, 3500 and 2800; but units of one list beside others' are
// slower, and the ratios are those that measured best when they were chosen (us; the three largest cases above: cross
// attention, two documents, INT2 document): 2 : 1 : 0 312, 96, 359; 3 : 2 : 3 or 2 247, 83, 282;
// 5 : 4 : 6 or 4 218, 82, 285; 5 : 4 : 9 or 6 218, 82, 286 and less for short lists; 9 : 8 : 12 or 8 217, 83, 288.
constexpr int kRowsBothCost = 5, kRowsOneCost = 4, kRowsHeadBf16 = 9, kRowsHeadInt2 = 6;

// A list's shape: row tiles (the cost of a unit of the last one), units of a tile, their cost in all.
struct RowsList {
    int tiles, last, per;
    long long units;
};
// Cost of an item of `per` units.
__device__ __forceinline__ long long rows_cost(const RowsParams &p, int per, int w) { return p.head + (long long)per * w; }
__device__ __forceinline__ RowsList rows_list(const RowsParams &p, int i) {
    RowsList r;
    if (i < p.n_groups) {
        const int n = max(rows_first(p, i + 1) - rows_first(p, i), 0) * p.G;
        r.tiles = (n + kRowsTile - 1) / kRowsTile;
        r.last = n - (r.tiles - 1) * kRowsTile > kRowsHalf ? kRowsBothCost : kRowsOneCost;
        r.per = rows_units(rows_len(p.kv_lens, i, p.max_pages));
    } else {
        r.tiles = 1;
        r.last = kRowsOneCost;
        r.per = rows_units(rows_len(p.own_lens, i - p.n_groups, p.own_max_pages));
    }
    r.units = r.tiles && r.per ? (long long)p.hkv * ((r.tiles - 1) * rows_cost(p, r.per, kRowsBothCost) + rows_cost(p, r.per, r.last))
                               : 0;
    return r;
}

// Inclusive prefix sum over a warp.
__device__ __forceinline__ long long warp_scan(long long x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long t = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += t;
    }
    return x;
}

// Cost of the lists before list n; warp-collective.
__device__ __forceinline__ long long rows_sum(const RowsParams &p, int n, int lane) {
    long long u = 0;
    for (int i = lane; i < n; i += 32) u += rows_list(p, i).units;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
    return u;
}

// The start of a CTA's walk: its range of cost [u0, u1) -- a unit is its own if it begins there --, the item
// that holds u0 (whose first unit begins at `start`).
struct RowsCursor {
    long long u0, u1, start;
    int list, mt, j;
};

// Cost per CTA (and the general quotient: 32-bit division where it fits).
__device__ __forceinline__ long long rows_div(long long a, long long b) {
    return ((a | b) >> 32) == 0 ? (long long)((unsigned)a / (unsigned)b) : a / b;
}
__device__ __forceinline__ long long rows_share(long long U, int ctas) { return max(rows_div(U + ctas - 1, ctas), (long long)kRowsOneCost); }

// The CTA's cursor at its first list; warp-collective.
__device__ __forceinline__ RowsCursor rows_cursor(const RowsParams &p, int cta, int lane) {
    const int n = p.n_groups + p.n_own;
    // one pass when every list has a lane, else the sum first
    long long U = n > 32 ? rows_sum(p, n, lane) : 0, base = 0;
    RowsCursor c{0, 0, 0, n, 0, 0};
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        RowsList r{0, 1, 0, 0};
        if (i < n) r = rows_list(p, i);
        const long long ui = warp_scan(r.units, lane);
        if (n <= 32) U = __shfl_sync(0xffffffffu, ui, 31);
        if (i0 == 0) {
            const long long q = rows_share(U, p.num_ctas);
            c.u0 = min(cta * q, U);
            c.u1 = min((cta + 1) * q, U);
            if (c.u0 >= c.u1) return c;
        }
        const bool hit = r.units > 0 && base + ui - r.units <= c.u0 && c.u0 < base + ui;
        const unsigned m = __ballot_sync(0xffffffffu, hit);
        if (m) {
            int mt = 0, j = 0;   // the (tile, kv head) that holds u0
            long long start = 0;
            if (hit) {
                const long long first = base + ui - r.units, local = c.u0 - first, both = rows_cost(p, r.per, kRowsBothCost),
                                full = (long long)(r.tiles - 1) * p.hkv * both;
                const long long cost = local < full ? both : rows_cost(p, r.per, r.last);
                const int k = (int)rows_div(local < full ? local : local - full, cost);
                mt = local < full ? k / p.hkv : r.tiles - 1;
                j = local < full ? k - mt * p.hkv : k;
                start = first + (long long)mt * p.hkv * both + (long long)j * cost + p.head;
            }
            const int src = __ffs(m) - 1;
            c.list = i0 + src;
            c.start = __shfl_sync(0xffffffffu, start, src);
            c.mt = __shfl_sync(0xffffffffu, mt, src);
            c.j = __shfl_sync(0xffffffffu, j, src);
            break;
        }
        base += __shfl_sync(0xffffffffu, ui, 31);
    }
    return c;
}

// Units of cost w, one after another, that begin before x.
__device__ __forceinline__ int rows_begun(long long x, int w, int per) {
    const unsigned all = (unsigned)(per * w), y = x <= 0 ? 0u : x >= all ? all : (unsigned)x;
    return (int)(w == kRowsOneCost ? (y + kRowsOneCost - 1) / kRowsOneCost : (y + kRowsBothCost - 1) / kRowsBothCost);
}

// Walks the segments -- stretches [v0, v1) of one item's units -- of a CTA in order.
struct RowsWalk {
    long long start, u1;            // where the item's first unit begins, the CTA's end
    int list, tiles, last, per, len, row0, heads;   // the list: shape, tokens, first query row, row heads
    int mt, j, w;                   // the item: row tile, kv head, cost of a unit
    int v0, v1;
    bool live;
    __device__ __forceinline__ void load(const RowsParams &p) {
        const RowsList r = rows_list(p, list);
        tiles = r.tiles;
        last = r.last;
        per = r.per;
        if (list < p.n_groups) {
            row0 = rows_first(p, list);
            heads = (rows_first(p, list + 1) - row0) * p.G;
            len = rows_len(p.kv_lens, list, p.max_pages);
        } else {
            row0 = list - p.n_groups;
            heads = p.G;
            len = rows_len(p.own_lens, row0, p.own_max_pages);
        }
    }
    __device__ __forceinline__ void begin(const RowsParams &p, const RowsCursor &c) {
        list = c.list;
        live = c.u0 < c.u1 && list < p.n_groups + p.n_own;
        if (!live) return;
        load(p);
        start = c.start;
        u1 = c.u1;
        mt = c.mt;
        j = c.j;
        w = mt < tiles - 1 ? kRowsBothCost : last;
        v0 = rows_begun(c.u0 - start, w, per);
        v1 = rows_begun(u1 - start, w, per);
        if (v0 >= v1) next(p);   // none of its units begins in the CTA's range
    }
    __device__ __forceinline__ void next(const RowsParams &p) {
        start += rows_cost(p, per, w);
        if (++j == p.hkv) {
            j = 0;
            if (++mt == tiles) {
                do {
                    if (++list >= p.n_groups + p.n_own) {
                        live = false;
                        return;
                    }
                    load(p);
                } while (tiles == 0 || per == 0);
                mt = 0;
            }
            w = mt < tiles - 1 ? kRowsBothCost : last;
        }
        v0 = 0;
        v1 = rows_begun(u1 - start, w, per);
        live = v1 > 0;
    }
    __device__ __forceinline__ bool own(const RowsParams &p) const { return list >= p.n_groups; }
    __device__ __forceinline__ bool both() const { return w == kRowsBothCost; }   // both warpgroups take every unit
    __device__ __forceinline__ int units() const { return v1 - v0; }
    __device__ __forceinline__ int jobs() const { return both() ? 2 * units() : units(); }
    __device__ __forceinline__ int rows() const { return min(kRowsTile, heads - mt * kRowsTile); }
};

// What the row kernel leaves for the merge: cost per CTA, where each CTA's walk starts (without own
// lists), or where each list's cost begins (with).
struct RowsPlan {
    long long q;
    RowsCursor cursor[kRowsMaxCtas];
    long long first[1];   // n_groups + n_own of them
};
__host__ __device__ constexpr size_t rows_plan_bytes(size_t lists) { return sizeof(RowsPlan) + sizeof(long long) * lists; }

// By one warp of the grid's first CTA, which also reports starts that run backwards (their groups are taken as
// empty, and others may overlap).
__device__ __forceinline__ void rows_write_plan(const RowsParams &p, int lane) {
    const int n = p.n_groups + p.n_own;
    long long base = 0;
    for (int i0 = 0; i0 < n; i0 += 32) {
        const int i = i0 + lane;
        RowsList r{0, 1, 0, 0};
        if (i < n) r = rows_list(p, i);
        if (i < p.n_groups && p.row_start[i + 1] < p.row_start[i]) dqk_flag_error(kErrBounds);
        const long long ui = warp_scan(r.units, lane);
        if (i < n) p.plan->first[i] = base + ui - r.units;
        base += __shfl_sync(0xffffffffu, ui, 31);
    }
    if (lane == 0) p.plan->q = rows_share(base, p.num_ctas);
}

// Records of the groups' segments.  An item of n row heads has n records a segment (both warpgroups take its
// units) or, with n <= 128, two of each row head (the units go to one and the other); a segment never has more than
// step = 2 min(128, all row heads of a kv head).  With own lists every segment is joined with another: a CTA's segments
// are of consecutive items, so those of an item begin at CTA step + 2 (row heads of the items before), and reach no
// further than the next one's -- of the same CTA and the next item, or of the next CTA and the same item.
// Without, only items that cross a CTA's border are joined: the same, or, where it takes less room (rec_pairs), two
// places of `step` records a CTA, for the part of an item that began in an earlier CTA and for one that begins here.
// Starts that run backwards leave all of this inside the workspace, since row heads stay below those of the call.
// (There are less than 2^30 row heads, so record numbers fit in 32 bits.)
__device__ __forceinline__ uint32_t rows_record(const RowsParams &p, int cta, uint32_t before, bool begins) {
    return p.rec_pairs ? (uint32_t)(2 * cta + (begins ? 1 : 0)) * p.rec_step : (uint32_t)cta * p.rec_step + 2 * before;
}
// Row heads before those of an item: of its tile of `rows` row heads from `first` of its list, kv head j.
__device__ __forceinline__ uint32_t rows_heads_before(const RowsParams &p, int row0, int first, int rows, int j) {
    return (uint32_t)(row0 * p.G + first) * p.hkv + (uint32_t)(j * rows);
}
// A record's place in its segment of n row heads: row head x of a tile that both warpgroups take, or warpgroup g's of row
// head x (one warpgroup's behind the other's: 53.4 -> 51.7 us on a chat batch against the two of a row head side by side).
__device__ __forceinline__ uint32_t rows_place(bool both, int x, int g, int n) { return (uint32_t)(both ? x : g * n + x); }
// Own lists: CTA + item, two records of each of the G row heads.
__device__ __forceinline__ uint32_t rows_own_record(const RowsParams &p, int cta, int row, int j, int x, int g) {
    return (uint32_t)(cta + row * p.hkv + j) * 2 * p.G + rows_place(false, x, g, p.G);
}
__device__ __forceinline__ float *rows_at(float *rec, uint32_t record, int D) { return rec + (size_t)record * rec_stride(D); }

// ---------------------------------------------------------------------------
// tcgen05, TMEM and tensor copies
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tm_alloc(uint32_t *dst, int cols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(dst)), "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tm_dealloc(uint32_t base, int cols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols) : "memory");
}
__device__ __forceinline__ void tm_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Arrive on `bar` when every matrix instruction issued before has completed.
__device__ __forceinline__ void mma_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}
// One thread of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
    return e != 0;
}

// Shared-memory operand descriptor, 128-byte swizzle: groups of 8 rows of 128
// bytes are `group` bytes apart (high half); `lbo` is the distance of the 64-element
// blocks along N of an operand whose contiguous dimension is N (low half, with the
// address: a k-step further is one 32-bit addition).
__host__ __device__ constexpr uint32_t desc_high(uint32_t group) { return (group >> 4) | (1u << 14) | (2u << 29); }
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lbo) {
    return ((addr & 0x3ffffu) >> 4) | ((lbo >> 4) << 16);
}
// d (TMEM, 128 x N fp32) (+)= A B with A in shared memory, or in TMEM
template <uint32_t kGroupA, uint32_t kGroupB>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %6};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc),
                 "r"(desc_high(kGroupA)), "r"(desc_high(kGroupB))
                 : "memory");
}
template <uint32_t kGroupB>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t acc) {
    asm volatile("{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.u32 p, %4, 0;\n\t"
                 "mov.b64 db, {%2, %5};\n\t"
                 "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(acc),
                 "r"(desc_high(kGroupB))
                 : "memory");
}

// Instruction descriptor: fp32 accumulator, fp16 or BF16 operands, M = 128, N;
// b_n: B's contiguous dimension is N (else K).
__host__ __device__ constexpr uint32_t mma_idesc(bool bf16, int n, bool b_n) {
    return (1u << 4) | ((bf16 ? 1u : 0u) << 7) | ((bf16 ? 1u : 0u) << 10) | ((b_n ? 1u : 0u) << 16) |
           ((uint32_t)(n >> 3) << 17) | ((128u >> 4) << 24);
}

// 16 columns of the warp's 32 TMEM lanes: thread = lane, register = column.  The load is
// asynchronous; tm_ready16 waits for it and carries the registers, so that no use moves ahead.
#define DQK_R16(X) \
    X(0), X(1), X(2), X(3), X(4), X(5), X(6), X(7), X(8), X(9), X(10), X(11), X(12), X(13), X(14), X(15)
__device__ __forceinline__ void tm_ld16(uint32_t addr, uint32_t (&r)[16]) {
#define DQK_OUT(i) "=r"(r[i])
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
                 : DQK_R16(DQK_OUT)
                 : "r"(addr));
#undef DQK_OUT
}
__device__ __forceinline__ void tm_ready16(uint32_t (&r)[16]) {
#define DQK_INOUT(i) "+r"(r[i])
    asm volatile("tcgen05.wait::ld.sync.aligned;" : DQK_R16(DQK_INOUT)::"memory");
#undef DQK_INOUT
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ void tm_st8(uint32_t addr, const uint32_t *r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
                 "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void tm_st16(uint32_t addr, const uint32_t *r) {
#define DQK_IN(i) "r"(r[i])
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::DQK_R16(
                     DQK_IN),
                 "r"(addr)
                 : "memory");
#undef DQK_IN
}

// One box of the pool's tensor map: the 16 token rows from `row` of block `blk`, all columns.
__device__ __forceinline__ void tensor_copy(void *dst, const CUtensorMap *map, int row, int blk, uint64_t *bar) {
    asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
                 "[%6];" ::"r"(smem_addr(dst)),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(0), "r"(blk), "r"(smem_addr(bar))
                 : "memory");
}

__device__ __forceinline__ void stmatrix_x4(uint32_t addr, const uint32_t (&r)[4]) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                 "r"(r[3])
                 : "memory");
}

// ---------------------------------------------------------------------------
// INT2 blocks as fp16 operands
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
// One packed block in a warp's registers, in the operand order of the stored
// codes.  keys(s): key channels 16s..16s+15 of the page's 16 tokens, as four
// 8 x 8 matrices {b0, b1 of tokens 0-7, b0, b1 of tokens 8-15}; a lane holds
// channels 16s + 4tig + {0, 1} (b0) and + {2, 3} (b1) of token gid, so a row's
// channels come in the order rows_channel_pos gives, and the query rows use it too.
// values(m): value channels 16m..16m+15 (rows) by tokens, as matrices
// {channels 0-7: tokens 0-7, 8-15; channels 8-15: tokens 0-7, 8-15}.
// A protected channel 0's slot holds code 0, hence the group's finite min: the queries have a zero there, and
// the accumulator's column is not used (rows_half has the channel).
template <int D, int NS>
struct PageInt2 {
    static constexpr int NG = D / 32;
    uint32_t kw[NG], ks[2][NS], km[2][NS];
    uint32_t vw[NG], vh[NG], vs[2][NS], vm[2][NS];
    int gid, tig;
    template <int N>
    static __device__ __forceinline__ void words(uint32_t (&r)[N], uint32_t a) {
        if constexpr (N == 4) {
            const uint4 v = ld_s128(a);
            r[0] = v.x; r[1] = v.y; r[2] = v.z; r[3] = v.w;
        } else if constexpr (N == 2) {
            const uint2 v = ld_s64(a);
            r[0] = v.x; r[1] = v.y;
        } else {
            r[0] = ld_s32(a);
        }
    }
    // the NS fp16 entries at a, each repeated in both halves
    static __device__ __forceinline__ void pairs(uint32_t (&r)[NS], uint32_t a) {
        if constexpr (NS == 1) {
            const uint32_t h = ld_s16(a);
            r[0] = h | (h << 16);
        } else {
            uint32_t w[NS / 2];
            words<NS / 2>(w, a);
#pragma unroll
            for (int i = 0; i < NS / 2; ++i) {
                r[2 * i] = prmt(w[i], w[i], 0x1010u);
                r[2 * i + 1] = prmt(w[i], w[i], 0x3232u);
            }
        }
    }
    static constexpr Layout kL = make_layout(D, 0, NS);   // section offsets do not depend on v_ch0 (V0 is last)
    __device__ __forceinline__ void load_keys(uint32_t blk, int lane) {
        gid = lane >> 2;
        tig = lane & 3;
        words<NG>(kw, blk + kL.kc + lane * 4 * NG);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            pairs(ks[h], blk + kL.ks + (gid + 8 * h) * 2 * NS);
            pairs(km[h], blk + kL.km + (gid + 8 * h) * 2 * NS);
        }
    }
    __device__ __forceinline__ void load_values(uint32_t blk, int lane) {
        gid = lane >> 2;
        tig = lane & 3;
        words<NG>(vw, blk + kL.vc + lane * 4 * NG);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            words<NS>(vs[h], blk + kL.vs + (tig + 4 * h) * 4 * NS);
            words<NS>(vm[h], blk + kL.vm + (tig + 4 * h) * 4 * NS);
        }
#pragma unroll
        for (int k = 0; k < NG; ++k) vh[k] = vw[k] >> 10;
    }
    template <int F>
    __device__ __forceinline__ uint32_t key_pair(uint32_t w, int half, uint32_t s, uint32_t m) const {
        return hfma2(codes_to_f16x2<F>(prmt(w, 0u, half ? 0x4342u : 0x4140u)), s, m);
    }
    // k-step s = 2g + hi: k^ = code * scale + min in fp16 (one rounding)
    __device__ __forceinline__ void keys(int s, uint32_t (&r)[4]) const {
        const int g = s >> 1, hi = s & 1;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t w = NG == 4 ? kw[h + 2 * hi] : kw[h];
            const int f = NG == 4 ? g : g + 2 * hi, gs = NS == 1 ? 0 : g;
            switch (f) {
                case 0: r[2 * h] = key_pair<0>(w, 0, ks[h][gs], km[h][gs]); r[2 * h + 1] = key_pair<0>(w, 1, ks[h][gs], km[h][gs]); break;
                case 1: r[2 * h] = key_pair<1>(w, 0, ks[h][gs], km[h][gs]); r[2 * h + 1] = key_pair<1>(w, 1, ks[h][gs], km[h][gs]); break;
                case 2: r[2 * h] = key_pair<2>(w, 0, ks[h][gs], km[h][gs]); r[2 * h + 1] = key_pair<2>(w, 1, ks[h][gs], km[h][gs]); break;
                default: r[2 * h] = key_pair<3>(w, 0, ks[h][gs], km[h][gs]); r[2 * h + 1] = key_pair<3>(w, 1, ks[h][gs], km[h][gs]); break;
            }
        }
    }
    template <int I>
    __device__ __forceinline__ uint32_t value_pair(int W, int h, int gs) const {
        return hfma2(code_field<I>(vw[W], vh[W]), vs[h][gs], vm[h][gs]);
    }
    __device__ __forceinline__ uint32_t value(int m, int cr, int h) const {
        const int gs = NS == 1 ? 0 : m >> 1;
        const int W = NG == 4 ? cr + 2 * h : (4 * m + 2 * cr + h) >> 3, f = NG == 4 ? m : (4 * m + 2 * cr + h) & 7;
        switch (f) {
            case 0: return value_pair<0>(W, h, gs);
            case 1: return value_pair<1>(W, h, gs);
            case 2: return value_pair<2>(W, h, gs);
            case 3: return value_pair<3>(W, h, gs);
            case 4: return value_pair<4>(W, h, gs);
            case 5: return value_pair<5>(W, h, gs);
            case 6: return value_pair<6>(W, h, gs);
            default: return value_pair<7>(W, h, gs);
        }
    }
    __device__ __forceinline__ void values(int m, uint32_t (&r)[4]) const {
#pragma unroll
        for (int cr = 0; cr < 2; ++cr)
#pragma unroll
            for (int h = 0; h < 2; ++h) r[2 * cr + h] = value(m, cr, h);
    }
};


// Place of channel c in a key row of the operand tile (and in a prepared query row).
__host__ __device__ __forceinline__ int rows_channel_pos(int c) {
    return (c & ~15) + 8 * ((c >> 1) & 1) + 2 * ((c & 15) >> 2) + (c & 1);
}

// ---------------------------------------------------------------------------
// shared memory: operand tiles (K or V of a unit, 128 x D 16-bit values in
// 128-byte-swizzled rows of 64 columns), query tiles of the two warpgroups (and
// their low parts, fp32 queries), packed blocks (INT2), barriers.
//
// BF16 tile: page after page as one tensor copy lays it, [column block][16 token
// rows]; the 8-row groups of a half are then a page's size apart.  INT2 tile, keys:
// [column block][half][page][8 token rows]; values: [half][D channel rows], tokens
// along the row.  Behind the packed blocks: channel 0 of a unit's keys and (protected) of its values in fp32,
// [unit modulo kRowsCh0][keys, values][half][page][8 tokens], 0 where no token is.
// ---------------------------------------------------------------------------
constexpr int kRowsMaxTiles = 8, kRowsMaxRaw = 3;
// Units whose channel 0 is held.  A unit's is written once the key tile of two units before (INT2 has two) is free:
// both warpgroups have then formed scores of the two units before it, so they are through with all units before those.
constexpr int kRowsCh0 = 4;
__host__ __device__ constexpr uint32_t rows_ch0_bytes(bool v_ch0) { return kRowsKv * 4 * (v_ch0 ? 2 : 1); }   // of a unit
struct RowsBars {
    uint64_t full[kRowsMaxTiles], empty[kRowsMaxTiles];        // operand tiles: the ring of keys, then that of values
    uint64_t raw_full[kRowsMaxRaw], raw_empty[kRowsMaxRaw];    // packed blocks
    uint64_t q_full[2], o_step[2], o_full[2], done[2];         // per warpgroup: queries in; a half's product is in the
                                                               // accumulator, the segment's last one; nothing is in flight
    uint64_t s_full[2][2], p_full[2][2];                       // per warpgroup and half
    uint64_t join, read;                                       // the second warpgroup's record is written, has been read
    uint64_t v_full[kRowsFlags];                               // BF16, by unit: value tile in, stale rows zeroed
    uint32_t flags[kRowsFlags];                                // pages present, per unit
    uint32_t tmem;
    int abort;
    RowsCursor cursor;
};

template <int D, int kFmt>
struct RowsShape {
    static constexpr bool kInt2 = kFmt == 2;
    static constexpr int kParts = kFmt == 1 ? 2 : 1;                   // query parts
    static constexpr int kThreads = kInt2 ? 512 : 384;
    static constexpr int kTile = kRowsKv * D * 2;
    static constexpr int kPageBytes = kPage * D * 2;                   // of a tile
    // 8-row groups of the keys' half, of the values' (rows of tokens: a page apart; of channels: 1024)
    static constexpr uint32_t kGroupKv = kInt2 ? 1024 : kPageBytes;
    static constexpr uint32_t kS0 = 0, kO0 = 256;                      // TMEM columns: S of warpgroup w at 128 w, O at 256 + D w
    static constexpr uint32_t kIdescS = mma_idesc(!kInt2, kRowsKv / 2, false);
    static constexpr uint32_t kIdescO = mma_idesc(!kInt2, D, !kInt2);  // BF16 values: channels contiguous
    static constexpr int kFullCount = kInt2 ? kRowsUnpackWarps : 1;
    static constexpr float kLift = kInt2 ? kRowsLift : 0.0f;
};

// A place in a ring of n stages and the parity of its round.
struct RowsRing {
    int st = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int n) {
        if (++st == n) {
            st = 0;
            phase ^= 1u;
        }
    }
};

// Pages of a unit that are multiplied, in pairs (a k-step of 16 tokens of a half): those before the list's end.
__device__ __forceinline__ int rows_pairs(int nv) { return min((nv + 2 * kPage - 1) / (2 * kPage), kRowsPages / 2); }

// The units of a CTA in order, for the matrix threads.
struct RowsUnits {
    RowsWalk s;
    RowsRing k, t;     // places of the unit's key tile and of its value tile
    int v, n, unit;    // unit of the item, jobs and units before it
    __device__ __forceinline__ void start(const RowsParams &p, const RowsCursor &c) {
        n = unit = 0;
        s.begin(p, c);
        v = s.live ? s.v0 : 0;
    }
    __device__ __forceinline__ bool live() const { return s.live; }
    __device__ __forceinline__ bool mine(int w) const { return s.both() || ((n ^ w) & 1) == 0; }
    // the first, the last of a warpgroup's units in the segment
    __device__ __forceinline__ bool first() const { return s.both() ? v == s.v0 : v < s.v0 + 2; }
    __device__ __forceinline__ bool last() const { return s.both() ? v == s.v1 - 1 : v >= s.v1 - 2; }
    __device__ __forceinline__ void next(const RowsParams &p) {
        n += s.both() ? 2 : 1;
        ++unit;
        k.next(p.ktiles);
        t.next(p.vtiles);
        if (++v == s.v1) {
            s.next(p);
            v = s.v0;
        }
    }
};

// A bounded wait that, when it runs out, reports and raises the abort flag, on which every role ends.
__device__ __noinline__ bool rows_wait_long(uint64_t *bar, uint32_t phase, RowsBars &B, unsigned long long ns) {
    const uint64_t t0 = global_timer_ns();
    for (uint32_t it = 1;; ++it) {
        if (mbar_try_wait(bar, phase)) return true;
        if ((it & 63u) == 0u) {
            if (*(volatile int *)&B.abort) return false;
            if (global_timer_ns() - t0 > ns) {
                *(volatile int *)&B.abort = 1;
                dqk_flag_error(kErrTimeout);
                return false;
            }
        }
    }
}
__device__ __forceinline__ bool rows_wait(uint64_t *bar, uint32_t phase, RowsBars &B, unsigned long long ns) {
    for (int i = 0; i < 16; ++i)
        if (mbar_try_wait(bar, phase)) return true;
    return rows_wait_long(bar, phase, B, ns);
}

template <int D, int kFmt>
__device__ __forceinline__ void rows_producer(const RowsParams &p, const CUtensorMap *map, RowsBars &B, unsigned char *tiles,
                                              unsigned char *raw, int lane) {
    using T = RowsShape<D, kFmt>;
    RowsWalk s;
    RowsRing ring[2];   // raw blocks, or key and value tiles
    int unit = 0;
    bool ok = true;
    const int pg = lane & (kRowsPages - 1), h = lane >> 3;   // lanes 0 .. 7 copy a page each
    for (s.begin(p, B.cursor); ok && s.live; s.next(p)) {
        const int *tab = s.own(p) ? p.own_table + (size_t)s.row0 * p.own_max_pages : p.table + (size_t)s.list * p.max_pages;
        const int npages = (s.len + kPage - 1) / kPage;
        if (lane == 0 && (s.own(p) ? p.own_lens[s.row0] : p.kv_lens[s.list]) > s.len) dqk_flag_error(kErrBounds);
        int page = s.v0 * kRowsPages + pg;
        int phys = page < npages ? tab[page] : -1;
        for (int v = s.v0; ok && v < s.v1; ++v, ++unit) {
            const bool in = page < npages;
            const bool have = in && phys >= 0 && phys < p.num_pages;
            const int blk = have ? phys * p.hkv + s.j : 0;
            if (in && !have && h == 0) dqk_flag_error(kErrBounds);
            const bool fill = !(p.stall && blockIdx.x == 0 && unit == 1);
            page += kRowsPages;
            phys = page < npages ? tab[page] : -1;   // the next unit's, on its way while this one waits
            const uint32_t m = __ballot_sync(0xffffffffu, have) & ((1u << kRowsPages) - 1u);
            const int nb = __popc(m);
            if constexpr (T::kInt2) {
                ok = __all_sync(0xffffffffu, rows_wait(&B.raw_empty[ring[0].st], ring[0].phase ^ 1u, B, p.wait_ns));
                if (!ok) break;
                if (lane == 0) {
                    B.flags[unit & (kRowsFlags - 1)] = m;
                    if (fill) mbar_arrive_expect_tx(&B.raw_full[ring[0].st], nb * (uint32_t)p.bb);
                }
                __syncwarp();
                if (h == 0 && have && fill)
                    bulk_copy_g2s(raw + ((size_t)ring[0].st * kRowsPages + pg) * p.bb, p.pool + (size_t)blk * p.bb, (uint32_t)p.bb,
                                  &B.raw_full[ring[0].st]);
                ring[0].next(p.raw_stages);
            } else {
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    const int st = ring[kv].st + (kv ? p.ktiles : 0);
                    ok = ok && __all_sync(0xffffffffu, rows_wait(&B.empty[st], ring[kv].phase ^ 1u, B, p.wait_ns));
                    if (!ok) break;
                    if (lane == 0) {
                        if (kv == 0) B.flags[unit & (kRowsFlags - 1)] = m;
                        if (fill) mbar_arrive_expect_tx(&B.full[st], nb * (uint32_t)T::kPageBytes);
                    }
                    __syncwarp();
                    if (h == 0 && have && fill)
                        tensor_copy(tiles + (size_t)st * T::kTile + pg * T::kPageBytes, map, kv * kPage, blk, &B.full[st]);
                    ring[kv].next(kv ? p.vtiles : p.ktiles);
                }
            }
        }
    }
    // never leave with copies in flight, nor before the last arrivals on `empty`: every stage that was filled has
    // landed and (unless aborted) been released -- a stage's last round is the one before the ring's place, or the
    // present one if the place has passed it
    for (int kv = 0; kv < (T::kInt2 ? 1 : 2); ++kv) {
        const int n = T::kInt2 ? p.raw_stages : kv ? p.vtiles : p.ktiles, first = kv ? p.ktiles : 0;
        uint64_t *full = T::kInt2 ? B.raw_full : B.full, *empty = T::kInt2 ? B.raw_empty : B.empty;
        for (int st = 0; st < n; ++st) {
            if (st >= ring[kv].st && unit < n) continue;   // never filled
            const uint32_t phase = ring[kv].phase ^ (st >= ring[kv].st ? 1u : 0u);
            (void)mbar_wait_bounded(&full[first + st], phase, p.wait_ns);
            (void)rows_wait(&empty[first + st], phase, B, p.wait_ns);
        }
    }
}

// INT2: packed blocks -> fp16 operand tiles, and channel 0 in fp32.  Keys as rows of tokens; values as
// rows of channels (the order their codes are stored in), 64 tokens per 128-byte row.
// A unit's keys come first, and on their own: their tile is free as soon as the scores of
// two units before are formed, the values' only after that unit's weights.
template <int D, int NS, bool VCH0>
__device__ __forceinline__ void rows_unpack(const RowsParams &p, RowsBars &B, unsigned char *tiles, unsigned char *raw,
                                            uint32_t ch0, int warp, int lane) {
    constexpr int kTile = kRowsKv * D * 2;
    constexpr Layout kL = make_layout(D, VCH0 ? 1 : 0, NS);
    RowsWalk s;
    RowsRing rr, rk, rv;
    int unit = 0;
    bool ok = true;
    const int mi = lane >> 3, r8 = lane & 7, tig = lane & 3;
    // rows of the matrix this lane addresses: keys, token 8 (mi >> 1) + r8 of the page, column chunk
    // 2s + (mi & 1); values, channel 16m + 8 (mi >> 1) + r8, the page's tokens of half mi & 1
    const uint32_t tile0 = smem_addr(tiles), ka = (uint32_t)(64 * (mi >> 1) + r8) * 128,
                   va = (uint32_t)(mi & 1) * (D * 128) + (uint32_t)(8 * (mi >> 1) + r8) * 128;
    for (s.begin(p, B.cursor); ok && s.live; s.next(p)) {
        for (int v = s.v0; ok && v < s.v1; ++v, ++unit) {
            const int rs = rr.st, sk = rk.st, sv = p.ktiles + rv.st, nv = s.len - v * kRowsKv, pages = 2 * rows_pairs(nv);
            ok = rows_wait(&B.raw_full[rs], rr.phase, B, p.wait_ns) && rows_wait(&B.empty[sk], rk.phase ^ 1u, B, p.wait_ns);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint32_t have = B.flags[unit & (kRowsFlags - 1)];
            const uint32_t blk = smem_addr(raw) + (uint32_t)(rs * kRowsPages * p.bb);
            {   // channel 0 of the warp's two pages
                const int pg = warp + kRowsUnpackWarps * (lane / kPage), t = lane % kPage;
                const uint32_t at = ch0 + (uint32_t)(unit & (kRowsCh0 - 1)) * rows_ch0_bytes(VCH0) +
                                    (uint32_t)((t >> 3) * (kRowsKv * 2) + pg * 32 + (t & 7) * 4);
                const bool token = ((have >> pg) & 1u) && kPage * pg + t < nv;
                st_s32(at, token ? ld_s16(blk + (uint32_t)(pg * p.bb + kL.k0 + 2 * k0_idx(t))) << 16 : 0u);
                if constexpr (VCH0)
                    st_s32(at + kRowsKv * 4, token ? ld_s16(blk + (uint32_t)(pg * p.bb + kL.v0 + 2 * t)) << 16 : 0u);
            }
#pragma unroll 1
            for (int pg = warp; pg < pages; pg += kRowsUnpackWarps) {
                if (!((have >> pg) & 1u)) continue;   // its scores are masked
                PageInt2<D, NS> b;
                b.load_keys(blk + (uint32_t)(pg * p.bb), lane);
                const uint32_t row = tile0 + (uint32_t)sk * kTile + ka + (uint32_t)pg * 1024;
#pragma unroll
                for (int st = 0; st < D / 16; ++st) {
                    uint32_t k4[4];
                    b.keys(st, k4);
                    const int c = 2 * st + (mi & 1);
                    stmatrix_x4(row + (uint32_t)(c >> 3) * (kRowsKv * 128) + (uint32_t)(((c & 7) ^ r8) << 4), k4);
                }
            }
            fence_proxy_async_shared();   // the tiles are read by the tensor core
            __syncwarp();
            if (lane == 0) mbar_arrive(&B.full[sk]);
            ok = __all_sync(0xffffffffu, rows_wait(&B.empty[sv], rv.phase ^ 1u, B, p.wait_ns));
            if (!ok) break;
#pragma unroll 1
            for (int pg = warp; pg < pages; pg += kRowsUnpackWarps) {
                const uint32_t row = tile0 + (uint32_t)sv * kTile + va + (uint32_t)((pg ^ r8) << 4);
                if ((have >> pg) & 1u) {
                    PageInt2<D, NS> b;
                    b.load_values(blk + (uint32_t)(pg * p.bb), lane);
                    // tokens past the list's end hold stale bytes: zeros, so that they add nothing
                    const int n = nv - kPage * pg;
                    const uint32_t lo = (2 * tig < n ? 0x0000ffffu : 0u) | (2 * tig + 1 < n ? 0xffff0000u : 0u);
                    const uint32_t hi = (2 * tig + 8 < n ? 0x0000ffffu : 0u) | (2 * tig + 9 < n ? 0xffff0000u : 0u);
#pragma unroll
                    for (int m = 0; m < D / 16; ++m) {
                        uint32_t v4[4];
                        b.values(m, v4);
                        v4[0] &= lo;
                        v4[1] &= hi;
                        v4[2] &= lo;
                        v4[3] &= hi;
                        stmatrix_x4(row + (uint32_t)(m * 16 * 128), v4);
                    }
                } else {
                    const uint32_t z[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                    for (int m = 0; m < D / 16; ++m) stmatrix_x4(row + (uint32_t)(m * 16 * 128), z);
                }
            }
            fence_proxy_async_shared();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&B.full[sv]);
                mbar_arrive(&B.raw_empty[rs]);
            }
            rr.next(p.raw_stages);
            rk.next(p.ktiles);
            rv.next(p.vtiles);
        }
    }
    // the last arrivals on `empty` come before the block leaves
    for (int kv = 0; kv < 2; ++kv) {
        const RowsRing r = kv ? rv : rk;
        const int n = kv ? p.vtiles : p.ktiles;
        for (int st = 0; st < n; ++st)
            if (st < r.st || unit >= n)
                (void)rows_wait(&B.empty[(kv ? p.ktiles : 0) + st], r.phase ^ (st >= r.st ? 1u : 0u), B, p.wait_ns);
    }
}

// BF16: zeros the value rows of tokens that are not the list's (the tensor copies
// brought stale memory, or nothing, there) before the tile's first use.
template <int D>
__device__ __forceinline__ void rows_tails(const RowsParams &p, RowsBars &B, unsigned char *tiles, int lane) {
    constexpr int kChunks = D / 8, kTile = kRowsKv * D * 2, kRowStep = 32 / kChunks;   // rows a warp zeros at once
    RowsWalk s;
    RowsRing ring;
    int unit = 0;
    bool ok = true;
    for (s.begin(p, B.cursor); ok && s.live; s.next(p)) {
        for (int v = s.v0; ok && v < s.v1; ++v, ++unit) {
            ok = __all_sync(0xffffffffu, rows_wait(&B.full[p.ktiles + ring.st], ring.phase, B, p.wait_ns));
            if (!ok) break;
            const int nv = s.len - v * kRowsKv;
            const uint32_t have = B.flags[unit & (kRowsFlags - 1)];
            if (nv < kRowsKv || have != (1u << kRowsPages) - 1u) {
                const int c = lane % kChunks, r0 = lane / kChunks;
                const uint32_t at = smem_addr(tiles) + (uint32_t)(p.ktiles + ring.st) * kTile +
                                    (uint32_t)((c >> 3) * (kPage * 128) + (c & 7) * 16);
#pragma unroll 1
                for (int pg = 0; pg < 2 * rows_pairs(nv); ++pg) {
                    const int n = (have >> pg) & 1u ? nv - kPage * pg : 0;   // rows of the page that stay
                    if (n >= kPage) continue;
#pragma unroll
                    for (int r = 0; r < kPage; r += kRowStep)
                        if (r + r0 >= n) st_s128(at + (uint32_t)(pg * (kPage * D * 2) + (r + r0) * 128), make_uint4(0u, 0u, 0u, 0u));
                }
                fence_proxy_async_shared();
                __syncwarp();
            }
            if (lane == 0) mbar_arrive(&B.v_full[unit & (kRowsFlags - 1)]);
            ring.next(p.vtiles);
        }
    }
}

// The matrix thread of warpgroup w.  Half h of the next job's scores follows half h of this
// job's outputs, whose weights lie in the same columns.  Tiles of units that are the other
// warpgroup's alone are released here too (two arrivals free a tile).
template <int D, int kFmt, int kW>
__device__ __forceinline__ void rows_matrix(const RowsParams &p, RowsBars &B, unsigned char *tiles, unsigned char *qmem,
                                            uint32_t tmem, int w) {
    using T = RowsShape<D, kFmt>;
    const uint32_t tile0 = smem_addr(tiles), q0 = smem_addr(qmem) + (uint32_t)(w * T::kParts * T::kTile);
    const uint32_t tS = tmem + T::kS0 + 128 * w, tO = tmem + T::kO0 + D * w;
    uint32_t qn = 0, pn = 0;    // parities of the next waits on q_full, p_full
    bool ok = true;
    RowsUnits nx;               // the next unit that is this warpgroup's
    nx.start(p, B.cursor);
    bool key_seen = false;      // of a unit to be passed over: its key tile is released
    // Moves nx on; false: not there yet (a tile to be passed over has not landed), or abort.
    auto seek = [&](bool block) {
        while (nx.live() && !nx.mine(w)) {
            const int kt = nx.k.st, vt = p.ktiles + nx.t.st;
            if (!key_seen) {
                if (!(block ? rows_wait(&B.full[kt], nx.k.phase, B, p.wait_ns) : mbar_test_wait(&B.full[kt], nx.k.phase))) return false;
                mbar_arrive(&B.empty[kt]);
                key_seen = true;
            }
            if (!(block ? rows_wait(&B.full[vt], nx.t.phase, B, p.wait_ns) : mbar_test_wait(&B.full[vt], nx.t.phase))) return false;
            mbar_arrive(&B.empty[vt]);
            key_seen = false;
            nx.next(p);
        }
        return true;
    };
    auto scores = [&](int h) {
        const uint32_t b = desc_low(tile0 + (uint32_t)nx.k.st * T::kTile + (uint32_t)h * (T::kInt2 ? kRowsKv / 2 * 128 : 1024), 16);
#pragma unroll
        for (int part = 0; part < T::kParts; ++part) {
            const uint32_t a = desc_low(q0 + (uint32_t)(part * T::kTile), 16);
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                const uint32_t qo = (uint32_t)((s >> 2) * (kRowsKv * 128) + (s & 3) * 32) >> 4;
                const uint32_t ko = (uint32_t)((s >> 2) * (T::kInt2 ? kRowsKv * 128 : kPage * 128) + (s & 3) * 32) >> 4;
                mma_ss<1024, T::kGroupKv>(tS + 64 * h, a + qo, b + ko, T::kIdescS, s > 0 || part > 0 ? 1u : 0u);
            }
        }
        mma_commit(&B.s_full[w][h]);
    };
    // Waits for what the next job's scores read.
    auto operands = [&]() {
        if (nx.first()) {
            if (!rows_wait(&B.q_full[w], qn, B, p.wait_ns)) return false;
            qn ^= 1u;
        }
        return rows_wait(&B.full[nx.k.st], nx.k.phase, B, p.wait_ns);
    };
    ok = seek(true);
    if (ok && nx.live()) {
        ok = operands();
        if (ok) {
            tm_fence_after();
            scores(0);
            scores(1);
            mma_commit(&B.empty[nx.k.st]);
        }
    }
    while (ok && nx.live()) {
        // this job (nx moves on to the one after)
        const int vt = p.ktiles + nx.t.st, unit = nx.unit;
        const uint32_t vphase = nx.t.phase;
        const uint32_t acc = nx.first() ? 0u : 1u;
        const bool last = nx.last();
        const int pairs = rows_pairs(nx.s.len - nx.v * kRowsKv);
        // BF16: rows of tokens, contiguous channels; INT2: rows of channels, contiguous tokens
        const uint32_t b = desc_low(tile0 + (uint32_t)vt * T::kTile, T::kInt2 ? 16 : kPage * 128);
        nx.next(p);
        ok = T::kInt2 ? rows_wait(&B.full[vt], vphase, B, p.wait_ns)
                      : rows_wait(&B.v_full[unit & (kRowsFlags - 1)], (unit / kRowsFlags) & 1, B, p.wait_ns);
        bool ahead = false;   // the next job's first half is on its way
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // the next job's operands, if they are there (an item's queries are loaded after the item before is finished)
            const bool early = h == 0 && ok && seek(false) && nx.live() && !nx.first() && mbar_test_wait(&B.full[nx.k.st], nx.k.phase);
            ok = ok && rows_wait(&B.p_full[w][h], pn, B, p.wait_ns);
            if (!ok) break;
            tm_fence_after();
#pragma unroll
            for (int s = 0; s < kRowsKv / 32; ++s) {
                if (s >= pairs) break;
                const uint32_t off = (uint32_t)(T::kInt2 ? h * (D * 128) + s * 32 : 2 * s * T::kPageBytes + h * 1024) >> 4;
                mma_ts<T::kGroupKv>(tO, tS + 64 * h + 8 * s, b + off, T::kIdescO, h > 0 || s > 0 ? 1u : acc);
                if constexpr (kW == 2) mma_ts<T::kGroupKv>(tO, tS + 64 * h + 32 + 8 * s, b + off, T::kIdescO, 1u);
            }
            mma_commit(&B.o_step[w]);
            if (h == 0) {
                if (early) scores(0);
                ahead = early;
            }
        }
        if (!ok) break;
        pn ^= 1u;
        if (last) mma_commit(&B.o_full[w]);
        if (ahead) {
            scores(1);
            mma_commit(&B.empty[nx.k.st]);
        }
        mma_commit(&B.empty[vt]);
        if (!ahead) {
            ok = seek(true);
            if (ok && nx.live()) {
                ok = operands();
                if (!ok) break;
                tm_fence_after();
                scores(0);
                scores(1);
                mma_commit(&B.empty[nx.k.st]);
            }
        }
    }
    // nothing in flight when the block leaves (after an abort too)
    mma_commit(&B.done[w]);
    (void)mbar_wait_bounded(&B.done[w], 0u, p.wait_ns);
}

// Scores of half h of a unit whose tokens are not all the list's (its last unit, or an absent page): token t
// is one if t < nv and its page is present; the others' scores become -inf, in place.
__device__ __forceinline__ void rows_mask(uint32_t tS, int nv, uint32_t have, int h) {
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {   // 16 columns: half the tokens of pages 2c and 2c + 1
        uint32_t u[16];
        tm_ld16(tS + 16 * c, u);
        tm_ready16(u);
#pragma unroll
        for (int g = 0; g < 2; ++g) {
            const int pg = 2 * c + g, n = (have >> pg) & 1u ? nv - kPage * pg - 8 * h : 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i >= n) u[8 * g + i] = 0xff800000u;
        }
        tm_st16(tS + 16 * c, u);
    }
    tm_wait_st();
}

// Two weights as a pair of operands: high parts, and (kW == 2) what those leave, 2^-8 of it off.
template <bool F16, int kW>
__device__ __forceinline__ void rows_pack(float2 y, uint32_t &hi, uint32_t &lo) {
    hi = F16 ? pack_f16x2(y.x, y.y) : pack_bf16x2(y.x, y.y);
    if constexpr (kW == 2) lo = pack_bf16x2(y.x - __uint_as_float(hi << 16), y.y - __uint_as_float(hi & 0xffff0000u));
}

// INT2: channel 0 of half a unit's keys (and values) in shared memory, and the row's factor of it.
struct RowsKey0 {
    uint32_t k0;
    float q0;
    __device__ __forceinline__ RowsKey0 at(int c) const { return {k0 + 64u * c, q0}; }   // 16 tokens on
    __device__ __forceinline__ uint32_t v0() const { return k0 + kRowsKv * 4; }
};

// What the running sums of a half hold: weights, their products with value channel 0, largest score.
struct RowsSums {
    float2 s0, s1, z0, z1;
    float m0, m1;
    __device__ __forceinline__ void clear() { s0 = s1 = z0 = z1 = make_float2(0.0f, 0.0f); }
    __device__ __forceinline__ float largest() const { return fmaxf(m0, m1); }
};

// 16 scores of a thread's row -> weights 2^(x qs - base), packed in pairs (kW == 2: low parts 32 words on), their
// sums, and their largest: of x, or (INT2) of x qs + k_0 q_0 - base.
template <bool F16, int kW, bool VCH0>
__device__ __forceinline__ void rows_weights(const uint32_t (&u)[16], float2 q2, float2 b2, const RowsKey0 &ch, uint32_t *pk,
                                             RowsSums &a) {
    float2 e[8], y[8];
    if constexpr (F16) {
        const float2 c2 = make_float2(ch.q0, ch.q0);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            const uint4 k = ld_s128(ch.k0 + 8 * i);
            e[i] = fma2(make_float2(__uint_as_float(k.x), __uint_as_float(k.y)), c2, b2);
            e[i + 1] = fma2(make_float2(__uint_as_float(k.z), __uint_as_float(k.w)), c2, b2);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        e[i] = fma2(make_float2(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1])), q2, F16 ? e[i] : b2);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = make_float2(fast_exp2(e[i].x), fast_exp2(e[i].y));
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        a.m0 = F16 ? max3(a.m0, e[i].x, e[i].y) : max3(a.m0, __uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
        a.m1 = F16 ? max3(a.m1, e[i + 1].x, e[i + 1].y)
                   : max3(a.m1, __uint_as_float(u[2 * i + 2]), __uint_as_float(u[2 * i + 3]));
        if constexpr (VCH0) {
            const uint4 v = ld_s128(ch.v0() + 8 * i);
            a.z0 = fma2(y[i], make_float2(__uint_as_float(v.x), __uint_as_float(v.y)), a.z0);
            a.z1 = fma2(y[i + 1], make_float2(__uint_as_float(v.z), __uint_as_float(v.w)), a.z1);
        }
        a.s0 = add2(a.s0, y[i]);
        a.s1 = add2(a.s1, y[i + 1]);
        rows_pack<F16, kW>(y[i], pk[i], pk[i + (kW - 1) * 32]);
        rows_pack<F16, kW>(y[i + 1], pk[i + 1], pk[i + 1 + (kW - 1) * 32]);
    }
}

// The accumulator's row times f.
template <int D>
__device__ __forceinline__ void rows_rescale(uint32_t tO, float f) {
#pragma unroll 1
    for (int c = 0; c < D / 16; ++c) {
        uint32_t o[16];
        tm_ld16(tO + 16 * c, o);
        tm_ready16(o);
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
        tm_st16(tO + 16 * c, o);
    }
}

// The largest score of a first half.
template <bool F16>
__device__ __forceinline__ float rows_largest(uint32_t tS, float qs, const RowsKey0 &ch) {
    float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 4; ++c) {
        uint32_t u[16];
        tm_ld16(tS + 16 * c, u);
        tm_ready16(u);
        if constexpr (F16) {
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
                const uint4 k = ld_s128(ch.at(c).k0 + 4 * i);
                u[i] = __float_as_uint(fmaf(__uint_as_float(u[i]), qs, ch.q0 * __uint_as_float(k.x)));
                u[i + 1] = __float_as_uint(fmaf(__uint_as_float(u[i + 1]), qs, ch.q0 * __uint_as_float(k.y)));
                u[i + 2] = __float_as_uint(fmaf(__uint_as_float(u[i + 2]), qs, ch.q0 * __uint_as_float(k.z)));
                u[i + 3] = __float_as_uint(fmaf(__uint_as_float(u[i + 3]), qs, ch.q0 * __uint_as_float(k.w)));
            }
        }
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            m0 = max3(m0, __uint_as_float(u[i]), __uint_as_float(u[i + 1]));
            m1 = max3(m1, __uint_as_float(u[i + 2]), __uint_as_float(u[i + 3]));
        }
    }
    return F16 ? fmaxf(m0, m1) : fmaxf(m0, m1) * qs;
}

// The weights of a thread's row for half a unit: S (64 columns at tS) becomes P~
// (packed pairs: its first 32 columns, low parts in the others), and the reference m and the sum l of the row follow.  A half
// whose scores pass the reference by more than the slack (rare) is taken again after the reference
// has moved and what was summed -- l, z, and the accumulator, once `settled` has waited for it -- has been rescaled.
// Channel 0 of the INT2 cache does not go through fp16, which would round it below 2^-14 and cut it off at 65504: the
// keys' is added to the scores, the products with the values' (z, protected) are summed, both in fp32.  That costs 1 to 5 %
// (64 sequences behind 128K tokens 286 and 300 us, a chat batch 49.9 and 50.3).
template <int D, bool F16, int kW, bool VCH0, typename Settled>
__device__ __forceinline__ bool rows_half(uint32_t tS, uint32_t tO, bool valid, float qs, const RowsKey0 &ch, float lift, float &m,
                                          float &l, float &z, Settled settled) {
    uint32_t pk[32 * kW];
    const float2 q2 = make_float2(qs, qs);
    float base = (m == -INFINITY ? 0.0f : m) - lift;
    float2 b2 = make_float2(-base, -base);
    RowsSums a;
    a.clear();
    a.m0 = a.m1 = -INFINITY;
    // 16-column loads in registers together (INT2 has 128 registers a thread, and low parts take theirs)
    constexpr int kAtOnce = F16 || kW == 2 ? 2 : 4;
#pragma unroll
    for (int c0 = 0; c0 < 4; c0 += kAtOnce) {
        uint32_t x[kAtOnce][16];
#pragma unroll
        for (int c = 0; c < kAtOnce; ++c) tm_ld16(tS + 16 * (c0 + c), x[c]);
#pragma unroll
        for (int c = 0; c < kAtOnce; ++c) tm_ready16(x[c]);
#pragma unroll
        for (int c = 0; c < kAtOnce; ++c) rows_weights<F16, kW, VCH0>(x[c], q2, b2, ch.at(c0 + c), pk + 8 * (c0 + c), a);
    }
    const float mx = F16 ? a.largest() + base : a.largest() * qs;
    const bool move = valid && mx > m + kRowsSlack;   // (lanes without a row hold anything)
    bool stored = false;
    if (__any_sync(0xffffffffu, move)) {
        // the references are whole numbers: moving one scales by a power of two
        const float to = move ? ceilf(mx) : m, f = !move || m == -INFINITY ? 1.0f : fast_exp2(m - to);
        m = to;
        l *= f;
        z *= f;
        int acc = settled();   // 1: the accumulator holds earlier halves, 0: nothing yet, -1: abort
        if (acc < 0) return false;
        if (acc) rows_rescale<D>(tO, f);
        base = (m == -INFINITY ? 0.0f : m) - lift;
        b2 = make_float2(-base, -base);
        a.clear();
        if constexpr (F16) {   // (a loop, for little code and no spills: weights go to columns whose scores have been taken)
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t y[16], w[8];
                tm_ld16(tS + 16 * c, y);
                tm_ready16(y);
                rows_weights<F16, kW, VCH0>(y, q2, b2, ch.at(c), w, a);
                tm_st8(tS + 8 * c, w);
            }
        } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t y[16];
                tm_ld16(tS + 16 * c, y);
                tm_ready16(y);
                rows_weights<F16, kW, VCH0>(y, q2, b2, ch.at(c), pk + 8 * c, a);
            }
        }
        stored = F16;
    }
    l += (a.s0.x + a.s0.y) + (a.s1.x + a.s1.y);
    if constexpr (VCH0) z += (a.z0.x + a.z0.y) + (a.z1.x + a.z1.y);
    if (!stored) {
#pragma unroll
        for (int i = 0; i < 2 * kW; ++i) tm_st16(tS + 16 * i, pk + 16 * i);
    }
    tm_wait_st();
    return true;
}

// A softmax thread's part in a segment: thread = row head.
struct RowsPart {
    size_t at;               // its row of q and out
    int vf;                  // the warpgroup's units: vf, vf + step, ...
    bool mine, valid, any;   // it has one; the thread has a row; its warp has
};
__device__ __forceinline__ RowsPart rows_part(const RowsParams &p, const RowsWalk &s, int n, int w, int r) {
    RowsPart t;
    const int rows = s.rows() - (s.both() ? kRowsHalf * w : 0), rr = s.mt * kRowsTile + (s.both() ? kRowsHalf * w : 0) + r;
    t.vf = s.both() ? s.v0 : s.v0 + ((n ^ w) & 1);
    t.mine = s.live && t.vf < s.v1;
    t.valid = s.live && r < rows;
    t.any = s.live && (r & ~31) < rows;
    const int g = p.G == 8 ? 3 : p.G >> 1;   // log2 G
    t.at = t.valid ? (size_t)(s.row0 + (rr >> g)) * p.hq + (size_t)s.j * p.G + (rr & (p.G - 1)) : 0;
    return t;
}

// The thread's query row into its warpgroup's operand tile (asynchronously, unless it has to be split in parts).
template <int D, int kFmt>
__device__ __forceinline__ void rows_query(const RowsParams &p, const RowsPart &t, uint32_t tile, int r) {
    using T = RowsShape<D, kFmt>;
    if (!t.mine || !t.valid) return;
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
        const uint32_t dst = tile + (uint32_t)(r * 128 + (c >> 3) * (kRowsKv * 128) + (((c & 7) ^ (r & 7)) << 4));
        if constexpr (kFmt != 1) {
            cp_async16(dst, reinterpret_cast<const uint16_t *>(p.q) + t.at * D + 8 * c);
        } else {
            const float4 *f = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(p.q) + t.at * D + 8 * c);
            const float4 a = f[0], b = f[1];
            const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                hi[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
                lo[i] = pack_bf16x2(x[2 * i] - __uint_as_float(hi[i] << 16), x[2 * i + 1] - __uint_as_float(hi[i] & 0xffff0000u));
            }
            st_s128(dst, make_uint4(hi[0], hi[1], hi[2], hi[3]));
            st_s128(dst + T::kTile, make_uint4(lo[0], lo[1], lo[2], lo[3]));
        }
    }
}

// Softmax warpgroup w.
template <int D, int kFmt, int kW, bool VCH0>
__device__ __forceinline__ void rows_softmax(const RowsParams &p, RowsBars &B, unsigned char *qmem, uint32_t ch0, uint32_t tmem, int w,
                                             int cta) {
    using T = RowsShape<D, kFmt>;
    const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, r = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(32 * quad) << 16, qtile = smem_addr(qmem) + (uint32_t)(w * T::kParts * T::kTile);
    const uint32_t tS = tmem + lanes + T::kS0 + 128 * w, tO = tmem + lanes + T::kO0 + D * w;
    int n = 0, unit0 = 0;                     // jobs and units before the segment
    uint32_t jobs = 0, pn = 0, on = 0, jn = 0, rn = 0;   // jobs and halves done; waits done on o_full, join, read
    bool ok = true, pending = false;          // pending (second warpgroup): a record the first has yet to read
    RowsWalk s;
    s.begin(p, B.cursor);
    RowsPart t = rows_part(p, s, n, w, r);
    auto queries_in = [&](const RowsPart &x) {
        if (!x.mine) return;
        if constexpr (kFmt != 1) cp_async_wait_all();
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.q_full[w]);
    };
    rows_query<D, kFmt>(p, t, qtile, r);
    queries_in(t);
    while (s.live) {
        float m = -INFINITY, l = 0.0f, z = 0.0f, qs = p.qs, q0 = 0.0f;
        if constexpr (kFmt == 2) {
            if (t.valid) {
                const float2 x = p.q_head[t.at];
                qs = x.x;
                q0 = x.y;
            }
        }
        const int step = s.both() ? 1 : 2;
        RowsWalk sn;          // the next segment
        RowsPart tn;
        if (!t.mine) {
            sn = s;
            sn.next(p);
            tn = rows_part(p, sn, n + s.jobs(), w, r);
            rows_query<D, kFmt>(p, tn, qtile, r);
        }
        for (int v = t.vf; v < s.v1; v += step) {
            const int nv = s.len - v * kRowsKv;
#pragma unroll 1
            for (int h = 0; h < 2; ++h, ++pn) {
                ok = __all_sync(0xffffffffu, rows_wait(&B.s_full[w][h], jobs & 1u, B, p.wait_ns));
                if (!ok) return;
                tm_fence_after();
                if (h && v + step >= s.v1) {
                    // the last scores of the segment: its queries are not needed any more, the next segment's come
                    // in while these scores become weights
                    sn = s;
                    sn.next(p);
                    tn = rows_part(p, sn, n + s.jobs(), w, r);
                    rows_query<D, kFmt>(p, tn, qtile, r);
                }
                if (t.any) {   // warps whose 32 rows are all past the tile leave the weights as they are: rows do not mix
                    const int unit = unit0 + v - s.v0;
                    const uint32_t have = B.flags[unit & (kRowsFlags - 1)];
                    const RowsKey0 ch{kFmt == 2 ? ch0 + (uint32_t)(unit & (kRowsCh0 - 1)) * rows_ch0_bytes(VCH0) + h * (kRowsKv * 2) : 0u,
                                     q0};
                    if (nv < kRowsKv || have != (1u << kRowsPages) - 1u) rows_mask(tS + 64 * h, nv, have, h);
                    const bool none = v == t.vf && h == 0;
                    if (none) m = ceilf(rows_largest<kFmt == 2>(tS, qs, ch));   // no reference yet
                    // the half before this one may still be on its way into the accumulator (the one before that is not:
                    // these scores lie where its weights were)
                    ok = rows_half<D, kFmt == 2, kW, VCH0>(tS + 64 * h, tO, t.valid, qs, ch, T::kLift, m, l, z, [&]() {
                        if (none) return 0;
                        if (!__all_sync(0xffffffffu, rows_wait(&B.o_step[w], (pn - 1) & 1u, B, p.wait_ns))) return -1;
                        tm_fence_after();
                        return 1;
                    });
                    if (!ok) return;
                }
                tm_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&B.p_full[w][h]);
            }
            ++jobs;
        }
        // the next segment's scores are formed while this one's accumulator is read
        queries_in(tn);
        if (t.mine) {
            ok = __all_sync(0xffffffffu, rows_wait(&B.o_full[w], on & 1u, B, p.wait_ns));
            ++on;
            if (!ok) return;
            tm_fence_after();
        }
        // a list that is whole in this segment (and has nothing to be joined with) becomes outputs here; where
        // its units went to both warpgroups in turn, the second hands its record to the first
        const bool whole = p.n_own == 0 && s.v0 == 0 && s.v1 == s.per;
        const bool split = !s.both() && s.per > 1, joint = whole && split;
        auto record = [&](uint32_t place) {   // of a group's segment
            const uint32_t before = rows_heads_before(p, s.row0, s.mt * kRowsTile, s.rows(), s.j);
            return rows_at(p.rec, rows_record(p, cta, before, s.v0 == 0) + place, D);
        };
        if (w == 1 && pending && (joint || !whole)) {   // the first warpgroup has read the record before it is written again
            ok = __all_sync(0xffffffffu, rows_wait(&B.read, rn & 1, B, p.wait_ns));
            ++rn;
            if (!ok) return;
            pending = false;
        }
        if (whole && (!split || w == 0)) {
            float f = 1.0f, f1 = 0.0f;
            const float *other = nullptr;
            if (joint) {
                other = record(rows_place(false, r, 1, s.rows()));
                ok = __all_sync(0xffffffffu, rows_wait(&B.join, jn & 1, B, p.wait_ns));
                ++jn;
                if (!ok) return;
                if (t.valid) {
                    const float m1 = __ldcg(other), l1 = __ldcg(other + 1), to = fmaxf(m, m1), base = to == -INFINITY ? 0.0f : to;
                    f = exp2f(m - base);
                    f1 = exp2f(m1 - base);
                    l = l * f + l1 * f1;
                }
            }
            if (t.any && t.mine) {
                const float inv = l != 0.0f ? 1.0f / l : 0.0f;
                f *= inv;
                f1 *= inv;
#pragma unroll 2
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t o[16];
                    tm_ld16(tO + 16 * c, o);
                    tm_ready16(o);
                    if (VCH0 && c == 0) o[0] = __float_as_uint(z);
                    if (t.valid) {
                        float y[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) y[i] = __uint_as_float(o[i]) * f;
                        if (joint) {
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const float4 x = __ldcg(reinterpret_cast<const float4 *>(other + kRecHead + 16 * c) + i);
                                y[4 * i] = fmaf(x.x, f1, y[4 * i]);
                                y[4 * i + 1] = fmaf(x.y, f1, y[4 * i + 1]);
                                y[4 * i + 2] = fmaf(x.z, f1, y[4 * i + 2]);
                                y[4 * i + 3] = fmaf(x.w, f1, y[4 * i + 3]);
                            }
                        }
                        if (p.out_dtype == DQK_BF16) {
                            uint4 *dst = reinterpret_cast<uint4 *>(reinterpret_cast<uint16_t *>(p.out) + t.at * D + 16 * c);
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                dst[i] = make_uint4(pack_bf16x2(y[8 * i], y[8 * i + 1]), pack_bf16x2(y[8 * i + 2], y[8 * i + 3]),
                                                    pack_bf16x2(y[8 * i + 4], y[8 * i + 5]), pack_bf16x2(y[8 * i + 6], y[8 * i + 7]));
                        } else {
                            float4 *dst = reinterpret_cast<float4 *>(reinterpret_cast<float *>(p.out) + t.at * D + 16 * c);
#pragma unroll
                            for (int i = 0; i < 4; ++i) dst[i] = make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
                        }
                    }
                    __syncwarp();
                }
            }
            __syncwarp();
            if (joint && lane == 0) mbar_arrive(&B.read);
        } else {
            float *rec = s.own(p) ? rows_at(p.own_rec, rows_own_record(p, cta, s.row0, s.j, r, w), D)
                                  : record(rows_place(s.both(), s.both() ? kRowsHalf * w + r : r, w, s.rows()));
            if (t.valid) *reinterpret_cast<float2 *>(rec) = make_float2(m, l);   // no unit of this segment: (-inf, 0) alone
            if (t.any && t.mine) {
#pragma unroll 2
                for (int c = 0; c < D / 16; ++c) {
                    uint32_t o[16];
                    tm_ld16(tO + 16 * c, o);
                    tm_ready16(o);
                    if (VCH0 && c == 0) o[0] = __float_as_uint(z);
                    if (t.valid) {
                        float4 *dst = reinterpret_cast<float4 *>(rec + kRecHead + 16 * c);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            dst[i] = make_float4(__uint_as_float(o[4 * i]), __uint_as_float(o[4 * i + 1]),
                                                 __uint_as_float(o[4 * i + 2]), __uint_as_float(o[4 * i + 3]));
                    }
                    __syncwarp();
                }
            }
            if (joint) {   // w == 1
                __syncwarp();
                if (lane == 0) mbar_arrive(&B.join);
                pending = true;
            }
        }
        __syncwarp();
        tm_fence_before();   // the accumulator has been read before the next segment's first product
        unit0 += s.units();
        n += s.jobs();
        s = sn;
        t = tn;
    }
}

// kFmt: BF16 cache with BF16 (0) or fp32 queries (1), INT2 cache (2); kW: parts of a softmax weight.
// A BF16 output is rounded by half a step, 2^-8, itself, and so may the weights be, each for itself (against
// 64 bits 0.0023 where the output's rounding alone leaves 0.0017); an fp32 output gets weights of two parts, 2^-16, as in
// dqk_bf16_decode (3e-6 where one part leaves 0.0017).  The second product costs 12 to 16 % where many row heads bound
// (up to 1024 queries over up to 4096 states, fp32 out: 225 and 253 to 262 us), 4 to 6 % on long documents (81 and 84
// to 86) and up to 3 us of the smallest calls.
template <int D, int kFmt, int kW, int NS, bool VCH0>
__global__ void __launch_bounds__(RowsShape<D, kFmt>::kThreads, 1)
    k_rows(const __grid_constant__ RowsParams p, const __grid_constant__ CUtensorMap map) {
    using T = RowsShape<D, kFmt>;
    extern __shared__ __align__(1024) unsigned char rows_smem[];
    unsigned char *tiles = rows_smem + ((1024u - (smem_addr(rows_smem) & 1023u)) & 1023u);
    unsigned char *qmem = tiles + (size_t)(p.ktiles + p.vtiles) * T::kTile;
    unsigned char *raw = qmem + 2 * T::kParts * T::kTile;
    const uint32_t ch0 = T::kInt2 ? smem_addr(raw) + (uint32_t)(p.raw_stages * kRowsPages * p.bb) : 0u;
    __shared__ RowsBars B;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    if (threadIdx.x == 0) {
        for (int i = 0; i < kRowsMaxTiles; ++i) {
            mbar_init(&B.full[i], T::kFullCount);
            mbar_init(&B.empty[i], 2);
        }
        for (int i = 0; i < kRowsFlags; ++i) mbar_init(&B.v_full[i], 1);
        for (int i = 0; i < kRowsMaxRaw; ++i) {
            mbar_init(&B.raw_full[i], 1);
            mbar_init(&B.raw_empty[i], kRowsUnpackWarps);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&B.q_full[i], 4);
            mbar_init(&B.o_step[i], 1);
            mbar_init(&B.o_full[i], 1);
            mbar_init(&B.done[i], 1);
            for (int h = 0; h < 2; ++h) {
                mbar_init(&B.s_full[i][h], 1);
                mbar_init(&B.p_full[i][h], 4);
            }
        }
        mbar_init(&B.join, 4);
        mbar_init(&B.read, 4);
        B.abort = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        const RowsCursor c = rows_cursor(p, blockIdx.x, lane);
        if (lane == 0) {
            B.cursor = c;
            if (p.n_own == 0) p.plan->cursor[blockIdx.x] = c;
        }
    }
    if (warp == 10 && blockIdx.x == 0) rows_write_plan(p, lane);
    if (warp == 9) tm_alloc(&B.tmem, 512);
    tm_fence_before();
    __syncthreads();
    tm_fence_after();
    const uint32_t tmem = B.tmem;
    if (warp < 8) {
        rows_softmax<D, kFmt, kW, VCH0>(p, B, qmem, ch0, tmem, warp >> 2, blockIdx.x);
        cp_async_wait_all();   // after an abort, queries may be on their way still
    } else {
        if (warp == 8) rows_producer<D, kFmt>(p, &map, B, tiles, raw, lane);
        else if (warp < 11) {
            if (elect_one()) rows_matrix<D, kFmt, kW>(p, B, tiles, qmem, tmem, warp - 9);
            __syncwarp();
        } else if constexpr (!T::kInt2) {
            rows_tails<D>(p, B, tiles, lane);
        } else {
            if (warp >= 12) rows_unpack<D, NS, VCH0>(p, B, tiles, raw, ch0, warp - 12, lane);
        }
    }
    grid_dependents_launch();
    tm_fence_before();
    __syncthreads();
    tm_fence_after();
    if (warp == 9) tm_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// merge: out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i over the records of
// the row head's group item and own item, in order; 0 without any token.
// ---------------------------------------------------------------------------
template <int D>
struct RowsMerge {
    static constexpr int V = D / 32, kBatch = 8;
    float M = -INFINITY, L = 0.0f, O[V] = {};
    static __device__ __forceinline__ void load(const float *rec, int lane, float &m, float &l, float (&o)[V]) {
        m = __ldcg(rec);
        l = __ldcg(rec + 1);
        if constexpr (V == 4) {
            const float4 x = __ldcg(reinterpret_cast<const float4 *>(rec + kRecHead) + lane);
            o[0] = x.x; o[1] = x.y; o[2] = x.z; o[3] = x.w;
        } else {
            const float2 x = __ldcg(reinterpret_cast<const float2 *>(rec + kRecHead) + lane);
            o[0] = x.x; o[1] = x.y;
        }
    }
    // The reference moves to `to` where that is larger.
    __device__ __forceinline__ void scale(float to) {
        to = fmaxf(M, to);
        const float sc = exp2f(M - base(to));   // 0 while M is -inf
        M = to;
        L *= sc;
#pragma unroll
        for (int e = 0; e < V; ++e) O[e] *= sc;
    }
    static __device__ __forceinline__ float base(float m) { return m == -INFINITY ? 0.0f : m; }
    __device__ __forceinline__ void add(float m, float l, const float (&o)[V]) {
        const float f = exp2f(m - base(M));
        const bool none = m == -INFINITY && l == 0.0f;   // an empty record: its o was not written
        L = fmaf(f, l, L);
#pragma unroll
        for (int e = 0; e < V; ++e) O[e] = none ? O[e] : fmaf(f, o[e], O[e]);
    }
    // The records of a row head of an item whose first unit begins at `start`: CTAs cf .. cl, both warpgroups' where
    // the units went to one and the other.  A CTA's lie at rec + CTA step, the second warpgroup's `second` behind.
    __device__ __forceinline__ void take(const float *rec, int step, int second, long long start, int per, bool both, long long q, int lane) {
        if (per <= 0) return;
        const int w = both ? kRowsBothCost : kRowsOneCost, shares = both ? 1 : 2;
        const int cf = (int)rows_div(start, q), cl = (int)rows_div(start + (long long)(per - 1) * w, q), n = (cl - cf + 1) * shares;
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += kBatch) {
            float m[kBatch], l[kBatch], o[kBatch][V], to = -INFINITY;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int i = i0 + k;
                const int c = cf + (both ? i : i >> 1);
                m[k] = -INFINITY;
                l[k] = 0.0f;
#pragma unroll
                for (int e = 0; e < V; ++e) o[k][e] = 0.0f;
                // (no unit need begin in a short range)
                const bool has = rows_begun(c * q - start, w, per) < rows_begun((c + 1) * q - start, w, per);
                if (i < n && has) load(rec + (size_t)(c * step + (both ? 0 : (i & 1) * second)) * rec_stride(D), lane, m[k], l[k], o[k]);
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) to = fmaxf(to, m[k]);
            scale(to);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) add(m[k], l[k], o[k]);
        }
    }
    __device__ __forceinline__ void store(const RowsParams &p, size_t head, int lane) const {
        const float inv = L != 0.0f ? 1.0f / L : 0.0f;
        const size_t at = head * D + V * lane;
        if (p.out_dtype == DQK_BF16) {
            uint16_t *out = reinterpret_cast<uint16_t *>(p.out) + at;
            if constexpr (V == 4)
                *reinterpret_cast<uint2 *>(out) =
                    make_uint2(pack_bf16x2(O[0] * inv, O[1] * inv), pack_bf16x2(O[2] * inv, O[3] * inv));
            else
                *reinterpret_cast<uint32_t *>(out) = pack_bf16x2(O[0] * inv, O[1] * inv);
        } else {
            float *out = reinterpret_cast<float *>(p.out) + at;
#pragma unroll
            for (int e = 0; e < V; ++e) out[e] = O[e] * inv;
        }
    }
};

constexpr int kRowsMergeWarps = 8;

// With own lists (decode): a warp per row head, over the records of its group's item and its own.
template <int D>
__global__ void __launch_bounds__(32 * kRowsMergeWarps) k_rows_merge(const __grid_constant__ RowsParams p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = blockIdx.x, h = blockIdx.y * kRowsMergeWarps + warp;
    if (h >= p.hq) return;
    const int j = h / p.G, hh = h - j * p.G;
    grid_dependency_wait();
    const long long q = p.plan->q, own_first = p.plan->first[p.n_groups + row];
    const int per = rows_list(p, p.n_groups + row).per;
    int g = -1;   // the group of the row
    for (int i0 = 0; i0 < p.n_groups && g < 0; i0 += 32) {
        const int i = i0 + lane;
        const unsigned hit =
            __ballot_sync(0xffffffffu, i < p.n_groups && rows_first(p, i) <= row && row < rows_first(p, i + 1));
        if (hit) g = i0 + __ffs(hit) - 1;
    }
    RowsMerge<D> acc;
    if (g >= 0) {
        const RowsList r = rows_list(p, g);
        const long long first = p.plan->first[g];
        const int row0 = rows_first(p, g), heads = (rows_first(p, g + 1) - row0) * p.G;
        const int rr = (row - row0) * p.G + hh, mt = rr / kRowsTile, w = mt < r.tiles - 1 ? kRowsBothCost : r.last;
        const bool both = w == kRowsBothCost;
        const uint32_t before = rows_heads_before(p, row0, mt * kRowsTile, min(kRowsTile, heads - mt * kRowsTile), j);
        acc.take(rows_at(p.rec, rows_record(p, 0, before, false) + rows_place(both, rr - mt * kRowsTile, 0, 0), D), (int)p.rec_step, min(kRowsTile, heads - mt * kRowsTile),
                 first + (long long)mt * p.hkv * rows_cost(p, r.per, kRowsBothCost) + j * rows_cost(p, r.per, w) + p.head, r.per, both,
                 q, lane);
    }
    acc.take(rows_at(p.own_rec, rows_own_record(p, 0, row, j, hh, 0), D), 2 * p.G, p.G, own_first + j * rows_cost(p, per, kRowsOneCost) + p.head,
             per, false, q, lane);
    acc.store(p, (size_t)row * p.hq + h, lane);
}

// Without own lists, CTA (b, y): row heads 8 y .., a warp each, and those 8 gridDim.y further on, of the item that
// begins in CTA b of the row kernel and goes on in the next one (every other item's outputs are written already); the
// CTAs behind those zero the rows of groups without any token (and, zero_rest, of no group).
// What bounds it is the arithmetic of the items and records, which the warp's row heads share (cross attention of up to
// 1024 queries over up to 4096 states, all kernels, with 1, 2 and 4 of them: 220, 218, 218 us).
constexpr int kRowsMergeHeads = 2;
template <int D>
__global__ void __launch_bounds__(32 * kRowsMergeWarps) k_rows_merge_items(const __grid_constant__ RowsParams p) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, b = blockIdx.x, x0 = blockIdx.y * kRowsMergeWarps + warp;
    const int step = (int)gridDim.y * kRowsMergeWarps;
    grid_dependency_wait();
    if (b >= p.num_ctas - 1) {
        const int n_runs = p.n_groups + (p.zero_rest ? 2 : 0);   // and the rows before the first group, behind the last
        for (int g = b - (p.num_ctas - 1); g < n_runs; g += (int)gridDim.x - (p.num_ctas - 1)) {
            if (g < p.n_groups && rows_list(p, g).per > 0) continue;
            const int r0 = g <= p.n_groups ? rows_first(p, g) : 0;
            const int r1 = g < p.n_groups ? rows_first(p, g + 1) : g == p.n_groups ? p.total_rows : rows_first(p, 0);
            const size_t at = (size_t)r0 * p.hq, n = (size_t)max(r1 - r0, 0) * p.hq;
            const RowsMerge<D> zero;
            for (size_t i = x0; i < n; i += step) zero.store(p, at + i, lane);
        }
        return;
    }
    const RowsCursor c = p.plan->cursor[b + 1];
    const long long q = p.plan->q;
    if (c.u0 >= c.u1 || c.start >= c.u0) return;
    const RowsList r = rows_list(p, c.list);
    const int first = rows_first(p, c.list), w = c.mt < r.tiles - 1 ? kRowsBothCost : r.last;
    if (c.start < b * q || c.start + (long long)(r.per - 1) * w < c.u0) return;
    const int heads = min((rows_first(p, c.list + 1) - first) * p.G - c.mt * kRowsTile, kRowsTile);
    if (x0 >= heads) return;
    RowsMerge<D> acc[kRowsMergeHeads];
    const bool both = w == kRowsBothCost;
    // records in CTA b, in the next one and, from there, in CTA after CTA; the row heads' places in each
    const uint32_t before = rows_heads_before(p, first, c.mt * kRowsTile, heads, c.j);
    const uint32_t here = rows_record(p, b, before, true), next = rows_record(p, b + 1, before, false);
    const uint32_t step_cta = p.rec_pairs ? 2 * p.rec_step : p.rec_step;
    uint32_t place[kRowsMergeHeads];
#pragma unroll
    for (int k = 0; k < kRowsMergeHeads; ++k) place[k] = rows_place(both, min(x0 + k * step, heads - 1), 0, 0);
    const int cl = (int)rows_div(c.start + (long long)(r.per - 1) * w, q);
    const int shares = both ? 1 : 2, n = (cl - b + 1) * shares;
    for (int i0 = 0; i0 < n; i0 += 2) {   // two records of every row head at a time
        float m[2][kRowsMergeHeads], l[2][kRowsMergeHeads], o[2][kRowsMergeHeads][RowsMerge<D>::V];
        bool has[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int a = min(b + (i0 + e) / shares, cl), g = (i0 + e) % shares;
            has[e] = i0 + e < n && rows_begun(a * q - c.start, w, r.per) < rows_begun((a + 1) * q - c.start, w, r.per);
#pragma unroll
            for (int k = 0; k < kRowsMergeHeads; ++k)   // (a record that was not written is inside the workspace too)
                RowsMerge<D>::load(rows_at(p.rec, (a == b ? here : next + (uint32_t)(a - b - 1) * step_cta) + place[k] + g * heads, D), lane, m[e][k],
                                   l[e][k], o[e][k]);
        }
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            if (!has[e]) continue;
#pragma unroll
            for (int k = 0; k < kRowsMergeHeads; ++k) {
                acc[k].scale(m[e][k]);
                acc[k].add(m[e][k], l[e][k], o[e][k]);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kRowsMergeHeads; ++k) {
        const int x = x0 + k * step, rr = c.mt * kRowsTile + x;
        if (x < heads) acc[k].store(p, (size_t)(first + rr / p.G) * p.hq + (size_t)c.j * p.G + rr % p.G, lane);
    }
}

}  // namespace dqk
