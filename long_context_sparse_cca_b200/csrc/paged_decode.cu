// cca_attn_decode_paged, cca_paged_step: attention of every row's newest
// token over a paged cache (core rows of the groups before its window, raw
// rows of the window; one softmax, sections 局部保留模块 and
// 全局-局部模块可微融合 of the CCA write-up), and with it the append of that
// token.
//
// Bound by HBM: every attended key and value row is read once, for all r
// query heads of its key/value head.  Keys are taken in tiles of 16 rows,
// which lie in one page one behind the other.  The tiles of all (row,
// key/value head) pairs form one list; every CTA, and in it every warp, gets
// an equal stretch of it, whatever the rows' lengths, found on the device
// from lens.  A warp keeps one tile of keys and one of values in registers
// and asks for the next ones as soon as the present ones are used.
//
// A tile's arithmetic runs on mma.m16n8k16 (the queries of a pair are at
// most 16 rows; tcgen05 wants 64 or 128 of them): S = Q K^T, then O += P V.
// Both contractions may take their index in any order, so the operands are
// read from the cache as 16-byte pieces of rows straight into fragments:
//   S: thread (i = lane / 4, j = lane % 4) holds dims 32 c + 8 j .. + 7 of
//      keys i and i + 8 (c = 0 .. D/32 - 1), and the same dims of query i;
//   O: dims 64 h + 8 i .. + 7 of keys 2j, 2j + 1, 2j + 8, 2j + 9; two keys'
//      rows interleave into the pairs of keys that a fragment holds.
// Raw rows are bf16 and core rows fp16, and both operands of a product have
// one type: for core tiles the query row is rounded to fp16 after a power of
// two brought its largest entry to 2^13 .. 2^14 (exact but for entries 2^-27
// below that one).  P is split into two numbers of the tile's type, P =
// P_hi + P_lo up to 2^-17, so that P V is as good as with fp32 weights; for
// up to 8 query heads P_lo takes the fragment rows that are free, and costs
// nothing.  Scores, running maximum and sum, and outputs are fp32.
//
// Stretches that share a pair are joined in shared memory within a CTA, and
// across CTAs by the last one that arrives at the pair (a ticket), always in
// the order of the list: results do not depend on the order of arrival.
#include <type_traits>

#include "paged.cuh"
#include "paged.h"
#include "pool_warp.cuh"

namespace cca {

__device__ unsigned int g_paged_decode_status;  // kStatusCapacity, kStatusPage, kStatusRange

namespace {

constexpr int kTile = 16;
constexpr int kCtas = 148;  // one per SM

// Floats of a warp's shared memory: two partial results of r query heads
// (m, l, O), or the scratch of a pooling.
__host__ __device__ constexpr int warp_floats(int D, int r, int g)
{
    const int part = 2 * r * (D + 2), pool = (r + 1) * g;
    return part > pool ? part : pool;
}

__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1, bool f16)
{
    if (f16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, "
                     "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
                     "{%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// (x0, x1) as a pair of the tile's type and the pair of what that leaves.
template <bool F16>
__device__ __forceinline__ void split2(float x0, float x1, uint32_t &hi, uint32_t &lo)
{
    if constexpr (F16) {
        hi = pack_f16x2(x0, x1);
        lo = pack_f16x2(x0 - f16_lo(hi), x1 - f16_hi(hi));
    } else {
        hi = pack_bf16x2(x0, x1);
        lo = pack_bf16x2(x0 - bf16_lo(hi), x1 - bf16_hi(hi));
    }
}

// Tiles of a row: core tiles, then raw ones (aligned to 16 tokens).
struct RowTiles {
    int64_t len, ws, n_core;
    int core, all;
};

__device__ __forceinline__ RowTiles row_tiles(const PagedView &c, int b, bool &over)
{
    RowTiles r;
    const int64_t len = c.lens[b];
    over = len > c.longest;  // a row longer than its table is taken as free
    r.len = over || len < 0 ? 0 : len;
    const PagedRow p = paged_row(r.len, c.g, c.w);
    r.ws = p.ws;
    r.n_core = p.n_core;
    r.core = static_cast<int>((p.n_core + kTile - 1) / kTile);
    r.all = r.len == 0 ? 0 : r.core + static_cast<int>(((r.len + kTile - 1) / kTile) - p.ws / kTile);
    return r;
}

// Where a warp stands in the list of tiles.
struct Place {
    int b, h, i;    // row, head, tile within the pair
    RowTiles row;
};

// One tile: rows [lo, hi) of it count; their page (or none).
struct Tile {
    bool core;
    int lo, hi;       // of 16
    int page, slot;   // slot of the tile's first row
    bool newest;      // row hi - 1 is the token that this launch appends
};

template <int D, int WARPS, bool WIDE, bool STEP>
__global__ void __launch_bounds__(WARPS * 32, 1)
    paged_decode_kernel(PagedView c, const uint16_t *__restrict__ q_t,
                        const uint16_t *__restrict__ k_t, const uint16_t *__restrict__ v_t,
                        void *__restrict__ o_t, int o_f32, float scale_log2,
                        float *__restrict__ part, unsigned int *__restrict__ tickets)
{
    constexpr int THREADS = WARPS * 32;
    constexpr int KC = D / 32, VH = D / 64;
    const int r = c.Hq / c.Hkv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, qi = lane >> 2, qj = lane & 3;
    const int PS = r * (D + 2);             // floats of a partial result
    const int WF = warp_floats(D, r, c.g);  // of a warp's shared memory
    extern __shared__ float smem[];
    float *mine = smem + warp * WF;
    // tiles of the rows before b, [B + 1]
    int64_t *before = reinterpret_cast<int64_t *>(smem + (WARPS * WF + 1) / 2 * 2);
    __shared__ int64_t sums[WARPS];
    __shared__ int ids[2 * WARPS];          // pairs of the warps' partial results, -1: none
    __shared__ int last_s[2];

    if (tid < 2 * WARPS) ids[tid] = -1;
    {  // the list: each thread sums its rows, then a scan over the block
        const int per = (c.B + THREADS - 1) / THREADS;
        const int b0 = min(tid * per, c.B), b1 = min(b0 + per, c.B);
        int64_t n = 0;
        for (int b = b0; b < b1; ++b) {
            bool over;
            n += row_tiles(c, b, over).all;
            if (over && blockIdx.x == 0) atomicOr(&g_paged_decode_status, kStatusCapacity);
        }
        int64_t x = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) sums[warp] = x;
        __syncthreads();
        int64_t at = x - n;
        for (int w = 0; w < warp; ++w) at += sums[w];
        for (int b = b0; b < b1; ++b) {
            bool over;
            before[b] = at;
            at += row_tiles(c, b, over).all;
        }
        if (b0 < c.B && b1 == c.B) before[c.B] = at;
        __syncthreads();
    }

    // Rows without tokens have a zero output; the newest token of the others
    // is appended.  No tile reads what is written here: its key and value
    // come from the inputs, and the core row of the group it completes is not
    // yet among those that it sees.  The last warps begin, which have no
    // tiles when there are few.
    for (int64_t pair = static_cast<int64_t>(gridDim.x) * WARPS - 1 - (blockIdx.x * WARPS + warp);
         pair < static_cast<int64_t>(c.B) * c.Hkv;
         pair += static_cast<int64_t>(gridDim.x) * WARPS) {
        const int b = static_cast<int>(pair / c.Hkv), h = static_cast<int>(pair - static_cast<int64_t>(b) * c.Hkv);
        const int64_t orow = static_cast<int64_t>(b) * c.Hq + h * r;
        if (before[b + 1] == before[b]) {
            for (int x = lane; x < r * D; x += 32) {
                if (o_f32)
                    static_cast<float *>(o_t)[orow * D + x] = 0.f;
                else
                    static_cast<uint16_t *>(o_t)[orow * D + x] = 0;
            }
            continue;
        }
        if (!STEP) continue;
        using VT = typename RowVec<D>::T;
        const int64_t t = c.lens[b] - 1;
        const int mask = (1 << c.shift) - 1;
        const int page =
            own_page_at(c.raw_table, c.raw_ref, b, c.raw_cols, t >> c.shift, c.raw_pages);
        if (page < 0) {
            if (lane == 0) atomicOr(&g_paged_decode_status, kStatusPage);
            continue;
        }
        const int64_t at = page_row<D>(page, h, c.Hkv, c.shift, static_cast<int>(t) & mask);
        reinterpret_cast<VT *>(c.k_raw + at)[lane] =
            reinterpret_cast<const VT *>(k_t + pair * D)[lane];
        reinterpret_cast<VT *>(c.v_raw + at)[lane] =
            reinterpret_cast<const VT *>(v_t + pair * D)[lane];
        if (c.core_cols == 0 || (t + 1) % c.g != 0) continue;
        const int64_t first = t - c.g + 1, j = t / c.g;
        int out = own_page_at(c.core_table, c.core_ref, b, c.core_cols, j >> c.shift, c.core_pages);
        for (int i = lane; i < c.g; i += 32)
            if (page_at(c.raw_table, b, c.raw_cols, (first + i) >> c.shift, c.raw_pages) < 0)
                out = -1;
        if (__any_sync(0xffffffffu, out < 0)) {
            if (lane == 0) atomicOr(&g_paged_decode_status, kStatusPage);
            continue;
        }
        auto old = [&](const uint16_t *pool, const uint16_t *in, int i) {
            if (i == c.g - 1) return in + pair * D;
            const int64_t pos = first + i;
            const int pg = page_at(c.raw_table, b, c.raw_cols, pos >> c.shift, c.raw_pages);
            return pool + page_row<D>(pg, h, c.Hkv, c.shift, static_cast<int>(pos) & mask);
        };
        const int64_t to = page_row<D>(out, h, c.Hkv, c.shift, static_cast<int>(j) & mask);
        const bool over = pool_group_warp<D>(
            [&](int i) { return old(c.k_raw, k_t, i); }, [&](int i) { return old(c.v_raw, v_t, i); },
            [&](int k) { return q_t + (orow + k) * D; }, r, c.g, scale_log2, mine, c.k_core + to,
            c.v_core + to);
        if (over && lane == 0) atomicOr(&g_paged_decode_status, kStatusRange);
        __syncwarp();
    }

    // This CTA's stretch of the list (at least a tile for each warp, as long
    // as there are enough), and this warp's part of it.
    auto first_of = [&](int b) { return before[b] * c.Hkv; };
    const int64_t total = first_of(c.B);
    if (total == 0) return;
    const int64_t n_ctas = min(static_cast<int64_t>(gridDim.x), (total + WARPS - 1) / WARPS);
    if (blockIdx.x >= n_ctas) return;
    const int64_t cta_lo = total * blockIdx.x / n_ctas, cta_hi = total * (blockIdx.x + 1) / n_ctas;
    const int64_t lo = cta_lo + (cta_hi - cta_lo) * warp / WARPS;
    const int64_t hi = cta_lo + (cta_hi - cta_lo) * (warp + 1) / WARPS;

    // The last row whose tiles begin at or before x.
    auto row_at = [&](int64_t x) {
        int a = 0, z = c.B - 1;
        while (a < z) {
            const int mid = (a + z + 1) >> 1;
            if (first_of(mid) <= x)
                a = mid;
            else
                z = mid - 1;
        }
        return a;
    };
    Place at = {};
    int ids_from = 0, ids_mine = 0;  // pages of tiles ids_from + lane of the pair
    auto load_ids = [&]() {
        ids_from = at.i;
        const int i = at.i + lane;
        ids_mine = -1;
        if (i < at.row.core)
            ids_mine = page_at(c.core_table, at.b, c.core_cols,
                               (static_cast<int64_t>(i) * kTile) >> c.shift, c.core_pages);
        else if (i < at.row.all)
            ids_mine = page_at(c.raw_table, at.b, c.raw_cols,
                               ((at.row.ws / kTile + (i - at.row.core)) * kTile) >> c.shift,
                               c.raw_pages);
    };
    auto tile_at = [&]() {
        Tile t;
        t.core = at.i < at.row.core;
        if (at.i - ids_from >= 32) load_ids();
        t.page = __shfl_sync(0xffffffffu, ids_mine, at.i - ids_from);
        if (t.core) {
            const int64_t p = static_cast<int64_t>(at.i) * kTile;
            t.slot = static_cast<int>(p) & ((1 << c.shift) - 1);
            t.lo = 0;
            t.hi = static_cast<int>(min(static_cast<int64_t>(kTile), at.row.n_core - p));
            t.newest = false;
        } else {
            const int64_t p = (at.row.ws / kTile + (at.i - at.row.core)) * kTile;
            t.slot = static_cast<int>(p) & ((1 << c.shift) - 1);
            t.lo = static_cast<int>(max(static_cast<int64_t>(0), at.row.ws - p));
            t.hi = static_cast<int>(min(static_cast<int64_t>(kTile), at.row.len - p));
            t.newest = STEP && p + t.hi == at.row.len;
        }
        return t;
    };
    auto next_place = [&]() {
        if (++at.i < at.row.all) return;
        at.i = 0;
        if (++at.h == c.Hkv) {
            at.h = 0;
            bool over;
            do {
                ++at.b;
                at.row = row_tiles(c, at.b, over);
            } while (at.row.all == 0);
        }
        load_ids();
    };

    uint4 kf[2][KC], vf[4][VH];
    auto load_k = [&](const Tile &t) {
        const uint16_t *base = (t.core ? c.k_core : c.k_raw) +
                               page_row<D>(max(t.page, 0), at.h, c.Hkv, c.shift, t.slot) + qj * 8;
        const uint16_t *in = k_t + (static_cast<int64_t>(at.b) * c.Hkv + at.h) * D + qj * 8;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const int row = n * 8 + qi;
            const uint16_t *src = base + row * D;
            bool ok = row >= t.lo && row < t.hi && t.page >= 0;
            if (STEP && t.newest && row == t.hi - 1) {
                src = in;
                ok = true;
            }
#pragma unroll
            for (int x = 0; x < KC; ++x)
                kf[n][x] = ok ? ldg_stream(src + x * 32) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    auto load_v = [&](const Tile &t, int b, int h) {
        const uint16_t *base = (t.core ? c.v_core : c.v_raw) +
                               page_row<D>(max(t.page, 0), h, c.Hkv, c.shift, t.slot) + qi * 8;
        const uint16_t *in = v_t + (static_cast<int64_t>(b) * c.Hkv + h) * D + qi * 8;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int row = (n >> 1) * 8 + qj * 2 + (n & 1);
            const uint16_t *src = base + row * D;
            bool ok = row >= t.lo && row < t.hi && t.page >= 0;
            if (STEP && t.newest && row == t.hi - 1) {
                src = in;
                ok = true;
            }
#pragma unroll
            for (int x = 0; x < VH; ++x)
                vf[n][x] = ok ? ldg_stream(src + x * 64) : make_uint4(0u, 0u, 0u, 0u);
        }
    };

    // Queries of the pair as fragments: rows qi and (WIDE) qi + 8.
    constexpr int QR = WIDE ? 2 : 1;
    uint4 qf[QR][KC];
    float q_scale[QR];
    auto load_q = [&](int b, int h, bool core) {
#pragma unroll
        for (int x = 0; x < QR; ++x) {
            const int row = x * 8 + qi;
            q_scale[x] = scale_log2;
#pragma unroll
            for (int e = 0; e < KC; ++e)
                qf[x][e] = row < r ? __ldg(reinterpret_cast<const uint4 *>(
                                         q_t + (static_cast<int64_t>(b) * c.Hq + h * r + row) * D +
                                         e * 32 + qj * 8))
                                   : make_uint4(0u, 0u, 0u, 0u);
            if (!core) continue;
            uint32_t top = 0;  // the row's largest magnitude, as bf16 bits
#pragma unroll
            for (int e = 0; e < KC; ++e)
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint32_t v = (&qf[x][e].x)[u] & 0x7fff7fffu;
                    top = max(top, max(v & 0xffffu, v >> 16));
                }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // entries times 2^(13 - e), e: exponent of the largest one (zero
            // rows and exponents that leave the type's range: the nearest)
            const int e2 = top == 0 ? 13 : static_cast<int>(top >> 7) - 127;
            const int up = max(-100, min(100, 13 - e2));
            const float f = __int_as_float((127 + up) << 23);
            q_scale[x] = scale_log2 * __int_as_float((127 - up) << 23);
#pragma unroll
            for (int e = 0; e < KC; ++e)
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint32_t &v = (&qf[x][e].x)[u];
                    v = pack_f16x2(bf16_lo(v) * f, bf16_hi(v) * f);
                }
        }
    };

    float o[D / 8][4], m[QR], l[QR];
    auto reset = [&]() {
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
#pragma unroll
        for (int x = 0; x < QR; ++x) {
            m[x] = -INFINITY;
            l[x] = 0.f;
        }
    };
    // S, softmax and P V of the tile in registers.
    auto scores = [&](bool f16, float (&s)[2][4]) {
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
            for (int x = 0; x < KC; ++x) {
                const uint4 k = kf[n][x], a = qf[0][x];
                const uint4 z = WIDE ? qf[QR - 1][x] : make_uint4(0u, 0u, 0u, 0u);
                mma16816(s[n], a.x, z.x, a.y, z.y, k.x, k.y, f16);
                mma16816(s[n], a.z, z.z, a.w, z.w, k.z, k.w, f16);
            }
        }
    };
    auto add_tile = [&](const Tile &t, float (&s)[2][4], auto f16_c) {
        constexpr bool F16 = decltype(f16_c)::value;
        uint32_t ph[QR][2], pl[QR][2];
#pragma unroll
        for (int x = 0; x < QR; ++x) {
            float top = -INFINITY;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int row = n * 8 + qj * 2 + e;
                    float &y = s[n][2 * x + e];
                    // a missing page leaves the newest row alone
                    const bool ok = t.page >= 0 ? row >= t.lo && row < t.hi
                                                : t.newest && row == t.hi - 1;
                    y = ok ? y * q_scale[x] : -INFINITY;
                    top = fmaxf(top, y);
                }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float to = fmaxf(m[x], top);
            const float use = to == -INFINITY ? 0.f : to;
            if (__any_sync(0xffffffffu, to > m[x])) {
                const float f = fast_exp2(m[x] - use);
                l[x] *= f;
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                    o[n][2 * x] *= f;
                    o[n][2 * x + 1] *= f;
                    if (!WIDE) {
                        o[n][2] *= f;
                        o[n][3] *= f;
                    }
                }
                m[x] = to;
            }
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                const float p0 = fast_exp2(s[n][2 * x] - use), p1 = fast_exp2(s[n][2 * x + 1] - use);
                l[x] += p0 + p1;
                split2<F16>(p0, p1, ph[x][n], pl[x][n]);
            }
        }
#pragma unroll
        for (int h = 0; h < VH; ++h)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint32_t v0 = (&vf[0][h].x)[u], v1 = (&vf[1][h].x)[u];
                const uint32_t v2 = (&vf[2][h].x)[u], v3 = (&vf[3][h].x)[u];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const uint32_t sel = e ? 0x7632 : 0x5410;
                    const uint32_t b0 = __byte_perm(v0, v1, sel), b1 = __byte_perm(v2, v3, sel);
                    float(&acc)[4] = o[h * 8 + u * 2 + e];
                    if constexpr (WIDE) {
                        mma16816(acc, ph[0][0], ph[1][0], ph[0][1], ph[1][1], b0, b1, F16);
                        mma16816(acc, pl[0][0], pl[1][0], pl[0][1], pl[1][1], b0, b1, F16);
                    } else {
                        mma16816(acc, ph[0][0], pl[0][0], ph[0][1], pl[0][1], b0, b1, F16);
                    }
                }
            }
    };
    auto put = [&](int64_t at, float y) {
        if (o_f32)
            static_cast<float *>(o_t)[at] = y;
        else
            static_cast<uint16_t *>(o_t)[at] = bf16_bits(y);
    };
    // The result of the tiles so far: the pair's output if they are all of
    // it, else a partial result in shared memory.
    auto finish = [&](int b, int h, bool whole, int entry) {
        float *to = mine + entry * PS;
#pragma unroll
        for (int x = 0; x < QR; ++x) {
            float sum = l[x];
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            const int row = x * 8 + qi;
            if (row >= r) continue;
            const float inv = whole ? (sum > 0.f ? 1.0f / sum : 0.f) : 1.f;
            const int64_t orow = (static_cast<int64_t>(b) * c.Hq + h * r + row) * D;
#pragma unroll
            for (int hh = 0; hh < VH; ++hh)
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int n = 0; n < 8; ++n) {
                        const float(&a)[4] = o[hh * 8 + n];
                        const float y = (WIDE ? a[2 * x + e] : a[e] + a[2 + e]) * inv;
                        const int dim = hh * 64 + (2 * qj + e) * 8 + n;
                        if (whole)
                            put(orow + dim, y);
                        else
                            to[row * D + dim] = y;
                    }
            if (!whole && qj == 0) {
                to[r * D + row] = m[x];
                to[r * D + r + row] = sum;
            }
        }
        if (!whole && lane == 0) ids[warp * 2 + entry] = b * c.Hkv + h;
    };

    if (lo < hi) {
        bool over, bad = false;
        at.b = row_at(lo);
        at.row = row_tiles(c, at.b, over);
        const int64_t in_row = lo - first_of(at.b);
        at.h = static_cast<int>(in_row / at.row.all);
        at.i = static_cast<int>(in_row - static_cast<int64_t>(at.h) * at.row.all);
        load_ids();
        reset();
        bool from_start = at.i == 0, loaded = false, q_core = false;
        int entry = 0;
        Tile t = tile_at();
        load_k(t);
        load_v(t, at.b, at.h);
        for (int64_t x = lo; x < hi; ++x) {
            const int b = at.b, h = at.h;
            const bool ends = at.i + 1 == at.row.all;
            const Tile cur = t;
            bad |= cur.page < 0;
            if (!loaded || q_core != cur.core) {
                load_q(b, h, cur.core);
                loaded = true;
                q_core = cur.core;
            }
            float s[2][4];
            scores(cur.core, s);
            const bool more = x + 1 < hi;
            if (more) {
                next_place();
                t = tile_at();
                load_k(t);
            }
            if (cur.core)
                add_tile(cur, s, std::true_type{});
            else
                add_tile(cur, s, std::false_type{});
            if (more) load_v(t, at.b, at.h);
            if (ends || !more) {
                const bool whole = ends && from_start;
                finish(b, h, whole, entry);
                entry += !whole;
                if (more) {
                    reset();
                    from_start = true;
                    loaded = false;
                }
            }
        }
        if (bad && lane == 0) atomicOr(&g_paged_decode_status, kStatusPage);
    }
    __syncthreads();

    // Join the warps' partial results, pair by pair.
    int n_slots = 0;
    int slot_pair[2];
    for (int e = 0; e < 2 * WARPS;) {
        const int pair = ids[e];
        if (pair < 0) {
            ++e;
            continue;
        }
        int z = e + 1;  // entries e .. z - 1 belong to it (those without a pair aside)
        while (z < 2 * WARPS && (ids[z] < 0 || ids[z] == pair)) ++z;
        const int b = pair / c.Hkv, h = pair - b * c.Hkv;
        const int64_t n = before[b + 1] - before[b], begin = first_of(b) + h * n;
        const bool whole = begin >= cta_lo && begin + n <= cta_hi;
        float *to = whole ? nullptr : part + (static_cast<int64_t>(blockIdx.x) * 2 + n_slots) * PS;
        for (int i = tid; i < r * D; i += THREADS) {
            const int row = i / D;
            float mx = -INFINITY, sum = 0.f, acc = 0.f;
            for (int y = e; y < z; ++y)
                if (ids[y] >= 0) mx = fmaxf(mx, smem[(y >> 1) * WF + (y & 1) * PS + r * D + row]);
            const float use = mx == -INFINITY ? 0.f : mx;
            for (int y = e; y < z; ++y) {
                if (ids[y] < 0) continue;
                const float *p = smem + (y >> 1) * WF + (y & 1) * PS;
                const float f = fast_exp2(p[r * D + row] - use);
                sum = fmaf(f, p[r * D + r + row], sum);
                acc = fmaf(f, p[i], acc);
            }
            if (whole) {
                put((static_cast<int64_t>(b) * c.Hq + h * r) * D + i, sum > 0.f ? acc / sum : 0.f);
            } else {
                to[i] = acc;
                if (i - row * D == 0) {
                    to[r * D + row] = mx;
                    to[r * D + r + row] = sum;
                }
            }
        }
        if (!whole) slot_pair[n_slots++] = pair;
        e = z;
    }
    if (n_slots == 0) return;

    // Pairs shared with other CTAs: the last one to arrive joins them.
    auto cta_of = [&](int64_t x) { return ((x + 1) * n_ctas - 1) / total; };
    __threadfence();
    __syncthreads();
    if (tid < n_slots) {
        const int pair = slot_pair[tid == 0 ? 0 : 1], b = pair / c.Hkv, h = pair - b * c.Hkv;
        const int64_t n = before[b + 1] - before[b], begin = first_of(b) + h * n;
        const unsigned int others =
            static_cast<unsigned int>(cta_of(begin + n - 1) - cta_of(begin));
        const bool last = atomicAdd(tickets + pair, 1u) == others;
        last_s[tid] = last;
        if (last) tickets[pair] = 0;  // ready for the next call
    }
    __syncthreads();
    for (int k = 0; k < n_slots; ++k) {
        if (!last_s[k]) continue;
        __threadfence();
        const int pair = slot_pair[k], b = pair / c.Hkv, h = pair - b * c.Hkv;
        const int64_t n = before[b + 1] - before[b], begin = first_of(b) + h * n;
        const int c0 = static_cast<int>(cta_of(begin)), c1 = static_cast<int>(cta_of(begin + n - 1));
        // CTA c0 holds the pair in its last slot: the second one if its
        // first is taken by a pair that began before it
        auto slot = [&](int cta) {
            if (cta > c0) return static_cast<int64_t>(cta) * 2;
            const int64_t clo = total * c0 / n_ctas;
            const int rb = row_at(clo);
            const int64_t rn = before[rb + 1] - before[rb], off = clo - first_of(rb);
            const int64_t pb = first_of(rb) + off / rn * rn;  // the pair at its first tile
            const bool open = pb < clo;                       // begins before it
            return static_cast<int64_t>(cta) * 2 + (open && pb != begin ? 1 : 0);
        };
        const int64_t slot0 = slot(c0);
        for (int i = tid; i < r * D; i += THREADS) {
            const int row = i / D;
            float mx = -INFINITY, sum = 0.f, acc = 0.f;
            for (int y = c0; y <= c1; ++y) {
                const float *p = part + (y == c0 ? slot0 : static_cast<int64_t>(y) * 2) * PS;
                mx = fmaxf(mx, __ldcg(p + r * D + row));
            }
            const float use = mx == -INFINITY ? 0.f : mx;
#pragma unroll 4
            for (int y = c0; y <= c1; ++y) {
                const float *p = part + (y == c0 ? slot0 : static_cast<int64_t>(y) * 2) * PS;
                const float f = fast_exp2(__ldcg(p + r * D + row) - use);
                sum = fmaf(f, __ldcg(p + r * D + r + row), sum);
                acc = fmaf(f, __ldcg(p + i), acc);
            }
            put((static_cast<int64_t>(b) * c.Hq + h * r) * D + i, sum > 0.f ? acc / sum : 0.f);
        }
    }
}

}  // namespace

size_t paged_decode_part_bytes(const cca_paged_cache &c)
{
    return sizeof(float) * 2 * kCtas * (c.Hq / c.Hkv) * (c.d + 2);
}

cudaError_t launch_paged_decode(const cca_paged_cache &c, int layer, const void *q_t,
                                const void *k_t, const void *v_t, void *o_t, bool o_f32,
                                void *workspace, cudaStream_t s)
{
    const PagedWorkspace w = paged_workspace(c);
    char *base = static_cast<char *>(workspace);
    const int r = c.Hq / c.Hkv;
    const PagedView v = paged_view(c, layer);
    const float scale_log2 = kLog2e / sqrtf(static_cast<float>(c.d));
    auto smem_of = [&](int warps) {
        return sizeof(float) * ((warps * warp_floats(c.d, r, c.g) + 1) / 2 * 2) +
               sizeof(int64_t) * (c.B + 1);
    };
    auto go = [&](auto kern, int warps) {
        const cudaError_t e = cudaFuncSetAttribute(
            kern, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem_of(warps)));
        if (e != cudaSuccess) return e;
        kern<<<kCtas, warps * 32, smem_of(warps), s>>>(
            v, static_cast<const uint16_t *>(q_t), static_cast<const uint16_t *>(k_t),
            static_cast<const uint16_t *>(v_t), o_t, o_f32 ? 1 : 0, scale_log2,
            reinterpret_cast<float *>(base + w.part),
            reinterpret_cast<unsigned int *>(base + w.tickets));
        return cudaGetLastError();
    };
    auto pick = [&](auto d, auto warps) {
        constexpr int D = decltype(d)::value, W = decltype(warps)::value;
        if (k_t != nullptr)
            return r > 8 ? go(paged_decode_kernel<D, W, true, true>, W)
                         : go(paged_decode_kernel<D, W, false, true>, W);
        return r > 8 ? go(paged_decode_kernel<D, W, true, false>, W)
                     : go(paged_decode_kernel<D, W, false, false>, W);
    };
    using std::integral_constant;
    if (c.d == 128) return pick(integral_constant<int, 128>{}, integral_constant<int, 8>{});
    if (smem_of(16) <= 220u * 1024u)
        return pick(integral_constant<int, 64>{}, integral_constant<int, 16>{});
    return pick(integral_constant<int, 64>{}, integral_constant<int, 8>{});
}

cudaError_t paged_decode_status_read_clear(unsigned int *v)
{
    unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(v, g_paged_decode_status, sizeof(*v));
    if (e == cudaSuccess && *v) e = cudaMemcpyToSymbol(g_paged_decode_status, &zero, sizeof(zero));
    return e;
}

}  // namespace cca
