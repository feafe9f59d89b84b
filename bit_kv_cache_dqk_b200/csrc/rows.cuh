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
// with the running maximum m and sum l per row head (online softmax), split
// over the tokens into records (m, l, o) that k_rows_merge joins.
//
// Work split: item = (group, tile of 128 row heads, kv head), then (own list,
// kv head); unit = kRowsKv tokens of an item.  CTA c of C takes units
// [floor(cU/C), floor((c+1)U/C)), so the CTAs stream the same number of tokens
// whatever the lengths.
#pragma once

#include "attend.cuh"
#include "common.cuh"
#include "ptx.cuh"

namespace dqk {

constexpr int kRowsTile = 128;                    // row heads of an item
constexpr int kRowsKv = 128;                      // tokens of a unit
constexpr int kRowsPages = kRowsKv / kPage;       // pages of a unit
constexpr int kRowsWarps = 8;                     // consumer warps
constexpr int kRowsThreads = 32 * (kRowsWarps + 1);
constexpr float kRowsPScale = 16384.0f;           // softmax weights in fp16 are carried times 2^14

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
    // queries: BF16 cache, the caller's rows [total_rows][hq][D] (q_dtype);
    // INT2 cache, prepared fp16 rows and their scales (k_query_rows)
    const void *q;
    int q_dtype;
    const float *q_scale;
    float qs;
    float *rec, *own_rec;       // split records of the groups' and of the own items
    long long rec_slots;        // slots `rec` holds (row_start out of order could ask for more)
    void *out;
    int out_dtype;
    int hq, hkv, G, bb, stages, num_ctas;
    unsigned long long wait_ns;
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
__device__ __forceinline__ int rows_tiles(const RowsParams &p, int g) {
    const int n = rows_first(p, g + 1) - rows_first(p, g);
    return n > 0 ? (int)(((long long)n * p.G + kRowsTile - 1) / kRowsTile) : 0;
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

// Units and row tiles of the groups before g (g = n_groups: all); warp-collective.
__device__ __forceinline__ void rows_before_group(const RowsParams &p, int g, int lane, long long &units,
                                                  long long &tiles) {
    long long u = 0, t = 0;
    for (int i = lane; i < g; i += 32) {
        const int nt = rows_tiles(p, i);
        t += nt;
        u += (long long)nt * p.hkv * rows_units(rows_len(p.kv_lens, i, p.max_pages));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        u += __shfl_xor_sync(0xffffffffu, u, o);
        t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    units = u;
    tiles = t;
}
// Units of the own lists before b.
__device__ __forceinline__ long long rows_before_own(const RowsParams &p, int b, int lane) {
    long long u = 0;
    for (int i = lane; i < b; i += 32) u += (long long)p.hkv * rows_units(rows_len(p.own_lens, i, p.own_max_pages));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) u += __shfl_xor_sync(0xffffffffu, u, o);
    return u;
}

// The CTA's units [u0, u1) of U (U_g of them the groups'), and the list that holds u0.
struct RowsPlan {
    long long U, Ug, u0, u1;
    long long first_unit;   // first unit of that list
    long long first_tile;   // row tiles of the groups before it
    int list;               // group index, or n_groups + own index
};

__device__ __forceinline__ RowsPlan rows_plan(const RowsParams &p, int cta, int num_ctas, int lane) {
    RowsPlan r;
    long long nt;
    rows_before_group(p, p.n_groups, lane, r.Ug, nt);
    r.U = r.Ug + rows_before_own(p, p.n_own, lane);
    r.u0 = (long long)cta * r.U / num_ctas;
    r.u1 = ((long long)cta + 1) * r.U / num_ctas;
    r.list = p.n_groups + p.n_own;
    r.first_unit = r.U;
    r.first_tile = nt;
    long long base = 0, tbase = 0;
    for (int i0 = 0; i0 < p.n_groups + p.n_own; i0 += 32) {
        const int i = i0 + lane;
        long long u = 0, t = 0;
        if (i < p.n_groups) {
            t = rows_tiles(p, i);
            u = t * p.hkv * rows_units(rows_len(p.kv_lens, i, p.max_pages));
        } else if (i < p.n_groups + p.n_own) {
            u = (long long)p.hkv * rows_units(rows_len(p.own_lens, i - p.n_groups, p.own_max_pages));
        }
        const long long ui = warp_scan(u, lane), ti = warp_scan(t, lane);
        const bool hit = u > 0 && base + ui - u <= r.u0 && r.u0 < base + ui;
        const unsigned m = __ballot_sync(0xffffffffu, hit);
        if (m) {
            const int src = __ffs(m) - 1;
            r.list = i0 + src;
            r.first_unit = base + __shfl_sync(0xffffffffu, ui - u, src);
            r.first_tile = tbase + __shfl_sync(0xffffffffu, ti - t, src);
            break;
        }
        base += __shfl_sync(0xffffffffu, ui, 31);
        tbase += __shfl_sync(0xffffffffu, ti, 31);
    }
    return r;
}

// One item's stretch of units inside the CTA.
struct RowsSeg {
    int own, list;          // own list, or group
    int j;                  // kv head
    int row0, rbase, nr;    // first query row of the list, first row head of the tile, row heads in it
    int len, v0, v1;        // tokens of the list, units [v0, v1) of it
    long long item;         // record slot: CTA + item
};

// Walks the segments of a CTA in order.
struct RowsCursor {
    long long u, u1, first_unit, first_tile;
    int list;
};
__device__ __forceinline__ RowsCursor rows_cursor(const RowsPlan &r) {
    return RowsCursor{r.u0, r.u1, r.first_unit, r.first_tile, r.list};
}
__device__ __forceinline__ bool rows_next(const RowsParams &p, RowsCursor &c, RowsSeg &s) {
    while (c.u < c.u1 && c.list < p.n_groups + p.n_own) {
        const bool own = c.list >= p.n_groups;
        const int i = own ? c.list - p.n_groups : c.list;
        const int nt = own ? 1 : rows_tiles(p, i);
        const int len = own ? rows_len(p.own_lens, i, p.own_max_pages) : rows_len(p.kv_lens, i, p.max_pages);
        const int per = rows_units(len);
        const long long total = (long long)nt * p.hkv * per;
        if (c.u >= c.first_unit + total) {
            c.first_unit += total;
            c.first_tile += own ? 0 : nt;
            ++c.list;
            continue;
        }
        const long long local = c.u - c.first_unit;
        const int k = (int)(local / per);            // (tile, kv head) of the list
        const int mt = k / p.hkv;
        s.own = own;
        s.list = i;
        s.j = k - mt * p.hkv;
        s.row0 = own ? i : rows_first(p, i);
        s.rbase = mt * kRowsTile;
        s.nr = own ? p.G : min(kRowsTile, (rows_first(p, i + 1) - s.row0) * p.G - s.rbase);
        s.len = len;
        s.v0 = (int)(local - (long long)k * per);
        s.v1 = (int)min((long long)per, s.v0 + (c.u1 - c.u));
        s.item = own ? (long long)i * p.hkv + s.j : (c.first_tile + mt) * p.hkv + s.j;
        c.u += s.v1 - s.v0;
        return true;
    }
    return false;
}

// Records: a group item's slot holds kRowsTile rows, row (warp w, i) at 16 w + i
// (warp w = share * wm + row block); an own item's slot 8 shares of G rows.
__device__ __forceinline__ size_t rows_rec(long long slot, int share, int wm, int row) {
    return ((size_t)slot * kRowsWarps + (size_t)share * wm + (row >> 4)) * 16 + (row & 15);
}
__device__ __forceinline__ size_t rows_own_rec(long long slot, int share, int G, int row) {
    return ((size_t)slot * kRowsWarps + share) * G + row;
}
// Blocks of 16 rows a tile of nr row heads is worked on in, rounded up to a power of two.
__device__ __forceinline__ int rows_blocks(int nr) { return nr <= 16 ? 1 : nr <= 32 ? 2 : nr <= 64 ? 4 : 8; }

// ---------------------------------------------------------------------------
// operand fetch: what differs between the two caches
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
// BF16 bits -> fp16, saturating at the largest finite value (channel 0 of the
// INT2 cache; fp16 holds every BF16 mantissa exactly from 2^-14 up).
__device__ __forceinline__ uint16_t bf16_to_f16_sat(uint32_t b) {
    const float x = __uint_as_float(b << 16);
    return __half_as_ushort(__float2half_rn(x > 65504.0f ? 65504.0f : x < -65504.0f ? -65504.0f : x));
}

// The score operand of one page: B registers of k-step s, token halves 0 and 1.
// BF16: k-step s = channels 16s..16s+15 in order.  INT2: a lane holds channels
// 32g + 16hi + 4tig + {0..3} of its tokens, taken as the k columns 2tig, 2tig+1,
// 2tig+8, 2tig+9 of step 2g + hi; the query operand uses the same order.
template <int D>
struct PageB16 {
    static constexpr int kSteps = D / 16;
    uint32_t blk;
    int lane;
    __device__ __forceinline__ void load(uint32_t b, int ln) {
        blk = b;
        lane = ln;
    }
    __device__ __forceinline__ void keys(int s, uint32_t (&r)[4]) const {   // {b0, b1} tokens 0-7, {b0, b1} tokens 8-15
        const int mi = lane >> 3, t = (lane & 7) + 8 * (mi >> 1);
        ldmatrix_x4(r, blk + t * 2 * D + (((2 * s + (mi & 1)) ^ (t & 7)) << 4));
    }
    // value operand of channels 16m..16m+15: {b0, b1} of the first 8, {b0, b1} of the next 8
    __device__ __forceinline__ void values(int m, uint32_t (&r)[4]) const {
        const int mi = lane >> 3, t = (lane & 7) + 8 * (mi & 1);
        ldmatrix_x4_trans(r, blk + kPage * 2 * D + t * 2 * D + (((2 * m + (mi >> 1)) ^ (t & 7)) << 4));
    }
};

template <int D, int NS, bool VCH0>
struct PageInt2 {
    static constexpr int kSteps = D / 16, NG = D / 32;
    uint32_t kw[NG], ks[2][NS], km[2][NS], k0[2];   // k0: fp16 bits of channel 0, token halves
    uint32_t vw[NG], vh[NG], vs[2][NS], vm[2][NS], v0[2];
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
    __device__ __forceinline__ void load(uint32_t blk, int lane) {
        constexpr Layout L = make_layout(D, VCH0 ? 1 : 0, NS);
        gid = lane >> 2;
        tig = lane & 3;
        words<NG>(kw, blk + L.kc + lane * 4 * NG);
        words<NG>(vw, blk + L.vc + lane * 4 * NG);
        const uint32_t k0w = ld_s32(blk + L.k0 + gid * 4);
        k0[0] = bf16_to_f16_sat(k0w & 0xffffu);
        k0[1] = bf16_to_f16_sat(k0w >> 16);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            pairs(ks[h], blk + L.ks + (gid + 8 * h) * 2 * NS);
            pairs(km[h], blk + L.km + (gid + 8 * h) * 2 * NS);
            words<NS>(vs[h], blk + L.vs + (tig + 4 * h) * 4 * NS);
            words<NS>(vm[h], blk + L.vm + (tig + 4 * h) * 4 * NS);
            if constexpr (VCH0) {
                const uint32_t w = ld_s32(blk + L.v0 + (tig + 4 * h) * 4);
                v0[h] = (uint32_t)bf16_to_f16_sat(w & 0xffffu) | ((uint32_t)bf16_to_f16_sat(w >> 16) << 16);
            }
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
            if (s == 0 && tig == 0) r[2 * h] = (r[2 * h] & 0xffff0000u) | k0[h];
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
            for (int h = 0; h < 2; ++h) {
                r[2 * cr + h] = value(m, cr, h);
                if constexpr (VCH0) {
                    if (m == 0 && cr == 0 && gid == 0) r[2 * cr + h] = v0[h];
                }
            }
    }
};

// ---------------------------------------------------------------------------
// the row kernel on warp-wide matrix instructions (m16n8k16): a warp owns 16
// row heads; the tile's blocks of 16 rows take wm warps, and the 8 / wm warps
// of a block share the pages of a unit.  kFmt 0: BF16 cache, queries in BF16;
// 1: BF16 cache, fp32 queries as BF16 high + low parts; 2: INT2 cache.
// ---------------------------------------------------------------------------
template <int D, int kFmt>
struct RowsState {
    static constexpr int kSteps = D / 16, kParts = kFmt == 1 ? 2 : 1;
    uint32_t qa[kParts][kSteps][4];
    float o[D / 8][4];
    float m0, m1, l0, l1;    // rows gid, gid + 8 (scores in log2 units)
    float qs0, qs1;
};

template <bool F16>
__device__ __forceinline__ void rows_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16) mma_f16(d, a[0], a[1], a[2], a[3], b0, b1);
    else mma_bf16(d, a[0], a[1], a[2], a[3], b0, b1);
}

// One page: the first nv of its 16 tokens are the list's (the rest is stale memory).
template <int D, int kFmt, typename Page>
__device__ __forceinline__ void rows_page(Page &pg, uint32_t blk, int nv, RowsState<D, kFmt> &st, int lane) {
    constexpr bool F16 = kFmt == 2;
    const int tig = lane & 3;
    pg.load(blk, lane);
    float c[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) c[h][e] = 0.0f;
#pragma unroll
    for (int s = 0; s < D / 16; ++s) {
        uint32_t kb[4];
        pg.keys(s, kb);
#pragma unroll
        for (int part = 0; part < RowsState<D, kFmt>::kParts; ++part) {
            rows_mma<F16>(c[0], st.qa[part][s], kb[0], kb[1]);
            rows_mma<F16>(c[1], st.qa[part][s], kb[2], kb[3]);
        }
    }
    float s0[4], s1[4];   // rows gid and gid + 8: tokens 2tig, 2tig+1, 2tig+8, 2tig+9
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const bool in = 8 * h + 2 * tig + e < nv;
            s0[2 * h + e] = in ? c[h][e] * st.qs0 : -INFINITY;
            s1[2 * h + e] = in ? c[h][2 + e] * st.qs1 : -INFINITY;
        }
    float x0 = fmaxf(fmaxf(s0[0], s0[1]), fmaxf(s0[2], s0[3]));
    float x1 = fmaxf(fmaxf(s1[0], s1[1]), fmaxf(s1[2], s1[3]));
    if (__any_sync(0xffffffffu, x0 > st.m0 || x1 > st.m1)) {
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
            x0 = fmaxf(x0, __shfl_xor_sync(0xffffffffu, x0, o));
            x1 = fmaxf(x1, __shfl_xor_sync(0xffffffffu, x1, o));
        }
        const float n0 = fmaxf(st.m0, x0), n1 = fmaxf(st.m1, x1);
        // a row with no finite score yet keeps m = -inf and scales by 1
        const float a0 = n0 == -INFINITY ? 1.0f : fast_exp2(st.m0 - n0), a1 = n1 == -INFINITY ? 1.0f : fast_exp2(st.m1 - n1);
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
            st.o[n][0] *= a0;
            st.o[n][1] *= a0;
            st.o[n][2] *= a1;
            st.o[n][3] *= a1;
        }
        st.l0 *= a0;
        st.l1 *= a1;
        st.m0 = n0;
        st.m1 = n1;
    }
    const float b0 = st.m0 == -INFINITY ? 0.0f : st.m0, b1 = st.m1 == -INFINITY ? 0.0f : st.m1;
    float p0[4], p1[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        p0[e] = fast_exp2(s0[e] - b0);
        p1[e] = fast_exp2(s1[e] - b1);
        st.l0 += p0[e];
        st.l1 += p1[e];
    }
    // P~ as the A operand: weights up to 1.  fp16 (INT2) carries them times 2^14, so
    // that a weight keeps full precision down to 2^-28 (the accumulator is scaled back
    // in the record).
    uint32_t pa[4];
    if constexpr (F16) {
        pa[0] = pack_f16x2(p0[0] * kRowsPScale, p0[1] * kRowsPScale);
        pa[1] = pack_f16x2(p1[0] * kRowsPScale, p1[1] * kRowsPScale);
        pa[2] = pack_f16x2(p0[2] * kRowsPScale, p0[3] * kRowsPScale);
        pa[3] = pack_f16x2(p1[2] * kRowsPScale, p1[3] * kRowsPScale);
    } else {
        pa[0] = pack_bf16x2(p0[0], p0[1]);
        pa[1] = pack_bf16x2(p1[0], p1[1]);
        pa[2] = pack_bf16x2(p0[2], p0[3]);
        pa[3] = pack_bf16x2(p1[2], p1[3]);
    }
    const uint32_t vlo = (2 * tig < nv ? 0x0000ffffu : 0u) | (2 * tig + 1 < nv ? 0xffff0000u : 0u);
    const uint32_t vhi = (2 * tig + 8 < nv ? 0x0000ffffu : 0u) | (2 * tig + 9 < nv ? 0xffff0000u : 0u);
#pragma unroll
    for (int m = 0; m < D / 16; ++m) {
        uint32_t vb[4];
        pg.values(m, vb);
        rows_mma<F16>(st.o[2 * m], pa, vb[0] & vlo, vb[1] & vhi);
        rows_mma<F16>(st.o[2 * m + 1], pa, vb[2] & vlo, vb[3] & vhi);
    }
}

// The query operand of rows r, r + 8 of the tile (row heads rb + 0..15).
template <int D, int kFmt>
__device__ __forceinline__ void rows_queries(const RowsParams &p, const RowsSeg &s, int rb, RowsState<D, kFmt> &st,
                                             int lane) {
    const int gid = lane >> 2, tig = lane & 3;
    size_t at[2];
    bool in[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = rb + gid + 8 * h;
        in[h] = r < s.nr;
        const int rr = s.rbase + (in[h] ? r : 0), row = s.row0 + rr / p.G, hh = rr % p.G;
        at[h] = (size_t)row * p.hq + (size_t)s.j * p.G + hh;
    }
    if constexpr (kFmt == 2) {
        st.qs0 = in[0] ? p.q_scale[at[0]] : 0.0f;
        st.qs1 = in[1] ? p.q_scale[at[1]] : 0.0f;
    } else {
        st.qs0 = st.qs1 = p.qs;
    }
#pragma unroll
    for (int k = 0; k < D / 16; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t lo = 0u, hi = 0u, lo2 = 0u, hi2 = 0u;   // k columns 2tig, 2tig+1 and 2tig+8, 2tig+9
            if (in[h]) {
                if constexpr (kFmt == 2) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(reinterpret_cast<const uint16_t *>(p.q) + at[h] * D +
                                                                     16 * k + 4 * tig);
                    lo = w.x;
                    hi = w.y;
                } else if constexpr (kFmt == 0) {
                    const uint16_t *q = reinterpret_cast<const uint16_t *>(p.q) + at[h] * D + 16 * k + 2 * tig;
                    lo = *reinterpret_cast<const uint32_t *>(q);
                    hi = *reinterpret_cast<const uint32_t *>(q + 8);
                } else {
                    const float *q = reinterpret_cast<const float *>(p.q) + at[h] * D + 16 * k + 2 * tig;
                    const float2 a = *reinterpret_cast<const float2 *>(q), b = *reinterpret_cast<const float2 *>(q + 8);
                    lo = pack_bf16x2(a.x, a.y);
                    hi = pack_bf16x2(b.x, b.y);
                    lo2 = pack_bf16x2(a.x - __uint_as_float(lo << 16), a.y - __uint_as_float(lo & 0xffff0000u));
                    hi2 = pack_bf16x2(b.x - __uint_as_float(hi << 16), b.y - __uint_as_float(hi & 0xffff0000u));
                }
            }
            st.qa[0][k][h] = lo;
            st.qa[0][k][2 + h] = hi;
            if constexpr (kFmt == 1) {
                st.qa[1][k][h] = lo2;
                st.qa[1][k][2 + h] = hi2;
            }
        }
    st.m0 = st.m1 = -INFINITY;
    st.l0 = st.l1 = 0.0f;
#pragma unroll
    for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.o[n][e] = 0.0f;
}

template <int D, int kFmt>
__device__ __forceinline__ void rows_record(const RowsParams &p, const RowsSeg &s, int cta, int share, int wm, int rb,
                                            RowsState<D, kFmt> &st, int lane) {
    const int gid = lane >> 2, tig = lane & 3;
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
        st.l0 += __shfl_xor_sync(0xffffffffu, st.l0, o);
        st.l1 += __shfl_xor_sync(0xffffffffu, st.l1, o);
    }
    constexpr float kBack = kFmt == 2 ? 1.0f / kRowsPScale : 1.0f;
    if (!s.own && cta + s.item >= p.rec_slots) {   // groups that overlap
        if (lane == 0) dqk_flag_error(kErrBounds);
        return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = rb + gid + 8 * h;
        if (r >= s.nr) continue;
        float *rec = (s.own ? p.own_rec + rows_own_rec(cta + s.item, share, p.G, r) * rec_stride(D)
                            : p.rec + rows_rec(cta + s.item, share, wm, r) * rec_stride(D));
        if (tig == 0) {
            rec[0] = h ? st.m1 : st.m0;
            rec[1] = h ? st.l1 : st.l0;
        }
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
            *reinterpret_cast<float2 *>(rec + kRecHead + 8 * n + 2 * tig) =
                make_float2(st.o[n][2 * h] * kBack, st.o[n][2 * h + 1] * kBack);
    }
}

// Brings the CTA's units into the ring, one stage each: lane l < 8 copies page l
// of the unit (one block of the item's kv head).  Pages past the list's end and
// bad page ids are marked absent.
__device__ __forceinline__ void rows_producer(const RowsParams &p, const RowsPlan &plan, unsigned char *stage_mem,
                                              uint64_t *full, uint64_t *empty, unsigned char *valid,
                                              volatile int *abort_flag, int lane) {
    const int S = p.stages;
    const uint32_t stage_bytes = (uint32_t)(kRowsPages * p.bb);
    RowsCursor cur = rows_cursor(plan);
    RowsSeg s;
    int stage = 0, filled = 0;
    uint32_t phase = 0;
    bool ok = true;
    while (ok && rows_next(p, cur, s)) {
        const int *tab = s.own ? p.own_table + (size_t)s.list * p.own_max_pages : p.table + (size_t)s.list * p.max_pages;
        const int npages = (s.len + kPage - 1) / kPage;
        if (lane == 0 && (s.own ? p.own_lens[s.list] : p.kv_lens[s.list]) > s.len) dqk_flag_error(kErrBounds);
        for (int v = s.v0; v < s.v1; ++v) {
            const int page = v * kRowsPages + lane;
            const bool in = lane < kRowsPages && page < npages;
            const int phys = in ? tab[page] : -1;
            const bool have = in && phys >= 0 && phys < p.num_pages;
            if (in && !have) dqk_flag_error(kErrBounds);
            int good = 1;
            if (lane == 0) good = mbar_wait_bounded(&empty[stage], phase ^ 1u, p.wait_ns, 2000u) && !*abort_flag;
            if (!__shfl_sync(0xffffffffu, good, 0)) {
                if (lane == 0) {
                    *abort_flag = 1;
                    dqk_flag_error(kErrTimeout);
                }
                ok = false;
                break;
            }
            const unsigned m = __ballot_sync(0xffffffffu, have);
            if (lane < kRowsPages) valid[stage * kRowsPages + lane] = have;
            __syncwarp();
            if (lane == 0) mbar_arrive_expect_tx(&full[stage], __popc(m) * (uint32_t)p.bb);
            __syncwarp();
            if (have)
                bulk_copy_g2s(stage_mem + (size_t)stage * stage_bytes + (size_t)lane * p.bb,
                              p.pool + ((size_t)phys * p.hkv + s.j) * p.bb, (uint32_t)p.bb, &full[stage]);
            ++filled;
            if (++stage == S) {
                stage = 0;
                phase ^= 1u;
            }
        }
    }
    // never leave with copies in flight
    if (lane == 0)
        for (int k = filled - 1; k >= 0 && k >= filled - S; --k)
            (void)mbar_wait_bounded(&full[k % S], (uint32_t)(k / S) & 1u, p.wait_ns);
}

// Shared memory besides the ring: full, empty, valid flags, abort flag.
constexpr size_t kRowsFixedSmem = 2 * kMaxStages * 8 + kMaxStages * kRowsPages + 16;

template <int D, int kFmt, int NS, bool VCH0>
__global__ void __launch_bounds__(kRowsThreads, 1) k_rows(const __grid_constant__ RowsParams p) {
    extern __shared__ __align__(128) unsigned char rows_smem[];
    const int S = p.stages;
    const uint32_t stage_bytes = (uint32_t)(kRowsPages * p.bb);
    unsigned char *stage_mem = rows_smem;
    uint64_t *full = reinterpret_cast<uint64_t *>(rows_smem + (size_t)S * stage_bytes);
    uint64_t *empty = full + kMaxStages;
    unsigned char *valid = reinterpret_cast<unsigned char *>(empty + kMaxStages);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(valid + kMaxStages * kRowsPages);
    __shared__ RowsPlan sh_plan;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], kRowsWarps);
        }
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 0) {
        const RowsPlan r = rows_plan(p, blockIdx.x, p.num_ctas, lane);
        if (lane == 0) sh_plan = r;
    }
    __syncthreads();
    const RowsPlan plan = sh_plan;
    if (warp == kRowsWarps) {
        rows_producer(p, plan, stage_mem, full, empty, valid, abort_flag, lane);
        return;
    }
    RowsCursor cur = rows_cursor(plan);
    RowsSeg s;
    RowsState<D, kFmt> st;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    while (ok && rows_next(p, cur, s)) {
        const int wm = rows_blocks(s.nr), share = warp / wm, shares = kRowsWarps / wm, rb = 16 * (warp % wm);
        rows_queries<D, kFmt>(p, s, rb, st, lane);
        for (int v = s.v0; v < s.v1; ++v) {
            if (!mbar_wait_bounded(&full[stage], phase, p.wait_ns)) {
                if (lane == 0) {
                    *abort_flag = 1;
                    dqk_flag_error(kErrTimeout);
                }
                ok = false;
                break;
            }
            const uint32_t base = smem_addr(stage_mem) + (uint32_t)stage * stage_bytes;
            if (rb < s.nr) {
                for (int k = share; k < kRowsPages; k += shares) {
                    if (!valid[stage * kRowsPages + k]) continue;
                    const int nv = s.len - (v * kRowsPages + k) * kPage;
                    if constexpr (kFmt == 2) {
                        PageInt2<D, NS, VCH0> pg;
                        rows_page<D, kFmt>(pg, base + (uint32_t)(k * p.bb), nv, st, lane);
                    } else {
                        PageB16<D> pg;
                        rows_page<D, kFmt>(pg, base + (uint32_t)(k * p.bb), nv, st, lane);
                    }
                }
            }
            __syncwarp();
            mbar_arrive_if(&empty[stage], lane == 0);
            if (++stage == S) {
                stage = 0;
                phase ^= 1u;
            }
        }
        if (ok) rows_record<D, kFmt>(p, s, (int)blockIdx.x, share, wm, rb, st, lane);
    }
    grid_dependents_launch();
}

// ---------------------------------------------------------------------------
// merge: out = sum_i 2^(m_i - M) o_i / sum_i 2^(m_i - M) l_i over the records of
// the row head's group item and own item, in unit order; 0 without any token.
// A warp per row head.
// ---------------------------------------------------------------------------
constexpr int kRowsMergeWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kRowsMergeWarps) k_rows_merge(const __grid_constant__ RowsParams p) {
    constexpr int V = D / 32, kBatch = 8;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long head = (long long)blockIdx.x * kRowsMergeWarps + warp;   // row * hq + h
    grid_dependency_wait();
    const int row = (int)(head / p.hq), h = (int)(head - (long long)row * p.hq), j = h / p.G, hh = h - j * p.G;
    if (row >= p.total_rows) return;
    // the group of the row: the last one that starts at or before it
    int g = -1;
    for (int i0 = 0; i0 < p.n_groups; i0 += 32) {
        const int i = i0 + lane;
        const bool in = i < p.n_groups && rows_first(p, i) <= row && row < rows_first(p, i + 1);
        const unsigned m = __ballot_sync(0xffffffffu, in);
        if (m) {
            g = i0 + __ffs(m) - 1;
            break;
        }
    }
    if (g < 0 && p.n_own == 0) return;   // behind the last sequence: left as it was
    long long Ug, tiles_all;
    rows_before_group(p, p.n_groups, lane, Ug, tiles_all);
    const long long U = Ug + rows_before_own(p, p.n_own, lane);
    const int C = p.num_ctas;
    float M = -INFINITY, Ls = 0.0f, O[V];
#pragma unroll
    for (int e = 0; e < V; ++e) O[e] = 0.0f;
    // record i of a part: CTA cf + i / shares, share i % shares
    auto take = [&](bool own, long long ua, int per, long long item, int wm, int r) {
        if (per <= 0) return;
        const int cf = (int)cta_of_unit(ua, U, C), cl = (int)cta_of_unit(ua + per - 1, U, C);
        const int shares = kRowsWarps / wm, n = (cl - cf + 1) * shares;
#pragma unroll 1
        for (int i0 = 0; i0 < n; i0 += kBatch) {
            float m[kBatch], l[kBatch], o[kBatch][V];
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const int i = i0 + q, c = cf + i / shares;
                m[q] = -INFINITY;
                l[q] = 0.0f;
#pragma unroll
                for (int e = 0; e < V; ++e) o[q][e] = 0.0f;
                if (i < n && (long long)c * U / C < ((long long)c + 1) * U / C && (own || c + item < p.rec_slots)) {
                    const float *rec = own ? p.own_rec + rows_own_rec(c + item, i % shares, p.G, r) * rec_stride(D)
                                           : p.rec + rows_rec(c + item, i % shares, wm, r) * rec_stride(D);
                    m[q] = __ldcg(rec);
                    l[q] = __ldcg(rec + 1);
                    if constexpr (V == 4) {
                        const float4 x = __ldcg(reinterpret_cast<const float4 *>(rec + kRecHead) + lane);
                        o[q][0] = x.x; o[q][1] = x.y; o[q][2] = x.z; o[q][3] = x.w;
                    } else {
                        const float2 x = __ldcg(reinterpret_cast<const float2 *>(rec + kRecHead) + lane);
                        o[q][0] = x.x; o[q][1] = x.y;
                    }
                }
            }
            float Mn = M;
#pragma unroll
            for (int q = 0; q < kBatch; ++q) Mn = fmaxf(Mn, m[q]);
            const float base = Mn == -INFINITY ? 0.0f : Mn;
            const float sc = exp2f(M - base);   // 0 while M is -inf
            Ls *= sc;
#pragma unroll
            for (int e = 0; e < V; ++e) O[e] *= sc;
            M = Mn;
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                const float w = exp2f(m[q] - base);   // 0 for an empty record, whose o holds zeros
                Ls = fmaf(w, l[q], Ls);
#pragma unroll
                for (int e = 0; e < V; ++e) O[e] = fmaf(w, o[q][e], O[e]);
            }
        }
    };
    if (g >= 0) {
        long long before, tiles;
        rows_before_group(p, g, lane, before, tiles);
        const int first = rows_first(p, g), per = rows_units(rows_len(p.kv_lens, g, p.max_pages));
        const int rr = (row - first) * p.G + hh, mt = rr / kRowsTile, r = rr - mt * kRowsTile;
        const int nr = min(kRowsTile, (rows_first(p, g + 1) - first) * p.G - mt * kRowsTile);
        const int k = mt * p.hkv + j;
        take(false, before + (long long)k * per, per, tiles * p.hkv + k, rows_blocks(nr), r);
    }
    if (p.n_own > 0) {
        const int per = rows_units(rows_len(p.own_lens, row, p.own_max_pages));
        const long long ua = Ug + rows_before_own(p, row, lane) + (long long)j * per;
        take(true, ua, per, (long long)row * p.hkv + j, 1, hh);
    }
    const float inv = Ls != 0.0f ? 1.0f / Ls : 0.0f;
    const size_t at = (size_t)head * D + V * lane;
    if (p.out_dtype == DQK_BF16) {
        uint16_t *out = reinterpret_cast<uint16_t *>(p.out) + at;
        if constexpr (V == 4)
            *reinterpret_cast<uint2 *>(out) = make_uint2(pack_bf16x2(O[0] * inv, O[1] * inv), pack_bf16x2(O[2] * inv, O[3] * inv));
        else
            *reinterpret_cast<uint32_t *>(out) = pack_bf16x2(O[0] * inv, O[1] * inv);
    } else {
        float *out = reinterpret_cast<float *>(p.out) + at;
#pragma unroll
        for (int e = 0; e < V; ++e) out[e] = O[e] * inv;
    }
}

}  // namespace dqk
