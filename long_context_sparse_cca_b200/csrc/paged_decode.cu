// cca_attn_decode_paged, cca_paged_step: attention of every row's newest
// token over a paged cache (core rows of the groups before its window, raw
// rows of the window; one softmax, sections 局部保留模块 and
// 全局-局部模块可微融合 of the CCA write-up), and with it the append of that
// token.
//
// Bound by HBM: every attended key and value row is read once, for all r
// query heads of its key/value head (8 rows of 65K tokens, 32 heads, d = 128:
// 665 MB in 124 us, 5.4 TB/s; while all warps stream, 6.4).  Keys are taken
// in tiles of 8 KB of keys and values (16 rows, or 32 of d = 64), whose rows
// lie 16 by 16 in one page, one behind the other.  The tiles of all (row,
// key/value head) pairs form one list; every CTA, and in it every warp, gets
// an equal stretch of it, whatever the rows' lengths, found on the device
// from lens.  Each warp copies its tiles into a ring of its own in shared
// memory, two or three deep (cp.async: some 100 KB in flight for an SM
// without registers, and no barrier between warps; 16-byte loads into
// registers reached 80% of that).
//
// A tile's arithmetic runs on mma.m16n8k16 (the queries of a pair are at
// most 16 rows; tcgen05 wants 64 or 128 of them): S = Q K^T, then O += P V.
// Both contractions may take their index in any order, so the operands are
// read from the ring as 16-byte pieces of rows straight into fragments:
//   S: thread (i = lane / 4, j = lane % 4) holds dims 64 h + 16 j .. + 15 of
//      keys i and i + 8, and the same dims of query i;
//   O: dims 64 h + 8 i .. + 7 of keys 2j, 2j + 1, 2j + 8, 2j + 9; two keys'
//      rows interleave into the pairs of keys that a fragment holds.
// Raw rows are bf16 and core rows fp16, and both operands of a product have
// one type: for core tiles the query row is rounded to fp16 after a power of
// two brought its largest entry to 2^13 .. 2^14 (exact but for entries below
// 2^-27 of that one).  P is split into two numbers of the tile's type, P =
// P_hi + P_lo up to 2^-17 (raw rows of more than 8 query heads: 2^-16, see
// split2); for up to 8 query heads P_lo takes the fragment rows that are free,
// and costs nothing.  An infinite value gives an infinite output, as with one
// number, and not NaN.  fp16 has no numbers below 2^-24, so core tiles hold
// weights relative to 2^-15 of the largest one (up to 2^15 then): one of 2^-n
// of the largest is off by 2^-17 of itself down to n = 23, and by 2^-40 of the
// largest below.  Scores, running maximum and sum, and outputs are fp32.
//
// Stretches that share a pair are joined in shared memory within a CTA, and
// across CTAs by the last one that arrives at the pair (a ticket), always in
// the order of the list: results do not depend on the order of arrival.
// What is left beside the streaming is latency: of 32 us for 16 rows of up
// to 32K tokens (101 MB), 2 are for the list, 5 until the first tile, 2 for
// each join.  (Smaller stretches handed out as CTAs get done: 190 us instead
// of 130 for the 8 rows; a stretch's begin and end take 8 us.)
#include <type_traits>

#include "paged.cuh"
#include "paged.h"
#include "pool_warp.cuh"

namespace cca {

__device__ unsigned int g_paged_decode_status;  // kStatusCapacity, kStatusPage, kStatusRange

namespace {

constexpr int kPart = 16;  // rows of a part of a tile, which lie in one page
constexpr int kCtas = 148;  // one per SM
constexpr size_t kOwnSmem = 1100;  // at least the kernel's static shared memory

template <int D>
struct Pd {
    static constexpr int PARTS = 128 / D;        // of a tile: 16 or 32 rows, 8 KB
    static constexpr int KEYS = kPart * PARTS;
    static constexpr int ROWS = kPart * D * 2;   // bytes of a part's keys (or values)
    static constexpr int STAGE = 2 * PARTS * ROWS;
};

// Floats of a partial result of r query heads: O [r][D], m [r], l [r].
__host__ __device__ constexpr int part_floats(int D, int r) { return (r * (D + 2) + 3) / 4 * 4; }

// Shared memory: for every warp its ring and one partial result (the ring
// holds the other one at the end, and both together are a pooling's
// scratch), then the list of tiles, [B + 1].
__host__ __device__ constexpr int warp_bytes(int D, int r, int stages)
{
    return stages * 8192 + 4 * part_floats(D, r);
}
size_t decode_smem(int D, int r, int warps, int stages, int B)
{
    return static_cast<size_t>(warps) * warp_bytes(D, r, stages) + sizeof(int64_t) * (B + 1);
}

template <bool F16>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1)
{
    if constexpr (F16)
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
// ABOVE (bf16, x >= 0): what is left is above zero wherever x is, for sums
// that both numbers go into: with a value of infinity, zero would make them
// NaN, and less than zero too.  So the first number is cut off and not
// rounded (both together: off by 2^-16), and 2^-20 of x is added to the other.
template <bool F16, bool ABOVE>
__device__ __forceinline__ void split2(float x0, float x1, uint32_t &hi, uint32_t &lo)
{
    if constexpr (F16) {
        hi = pack_f16x2(x0, x1);
        lo = pack_f16x2(x0 - f16_lo(hi), x1 - f16_hi(hi));
    } else if constexpr (ABOVE) {
        hi = __byte_perm(__float_as_uint(x0), __float_as_uint(x1), 0x7632);
        lo = pack_bf16x2(fmaf(x0, 0x1p-20f, x0 - bf16_lo(hi)), fmaf(x1, 0x1p-20f, x1 - bf16_hi(hi)));
    } else {
        hi = pack_bf16x2(x0, x1);
        lo = pack_bf16x2(x0 - bf16_lo(hi), x1 - bf16_hi(hi));
    }
}

// 16 bytes from global to shared memory.
__device__ __forceinline__ void copy16(uint32_t to, const void *from)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// The same, or zeros.
__device__ __forceinline__ void copy16_or_0(uint32_t to, const void *from, bool ok)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from),
                 "r"(ok ? 16 : 0)
                 : "memory");
}

// Tiles of a row: core tiles, then raw ones (aligned to whole tiles of
// tokens).
struct RowTiles {
    int64_t len, ws, n_core;
    int core, all;
};

template <int KEYS, bool STEP>
__device__ __forceinline__ RowTiles row_tiles(const PagedView &c, int b, bool &over)
{
    RowTiles r;
    const int64_t len = __ldg(c.lens + b);
    // a step takes a row that was refused room for its token as free: it would
    // write the token over the row's last one
    const bool held = STEP && __ldg(c.held + b) == len;
    over = len > c.longest;  // a row longer than its table is taken as free
    r.len = over || held || len < 0 ? 0 : len;
    // groups before the window of token t: max(t - w, 0) / g, in 32 bits where
    // they do (a 64-bit division takes a hundred instructions)
    const int64_t past = r.len - 1 - c.w;
    if (past < c.g)
        r.n_core = 0;
    else if (past >> 32 == 0)
        r.n_core = static_cast<uint32_t>(past) / static_cast<uint32_t>(c.g);
    else
        r.n_core = past / c.g;
    r.ws = r.n_core * c.g;
    r.core = static_cast<int>((r.n_core + KEYS - 1) / KEYS);
    r.all = r.len == 0 ? 0 : r.core + static_cast<int>(((r.len + KEYS - 1) / KEYS) - r.ws / KEYS);
    return r;
}

__device__ __forceinline__ void put4(void *o_t, int o_f32, int64_t at, float4 y)
{
    if (o_f32)
        *reinterpret_cast<float4 *>(static_cast<float *>(o_t) + at) = y;
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(o_t) + at) =
            make_uint2(pack_bf16x2(y.x, y.y), pack_bf16x2(y.z, y.w));
}

__device__ __forceinline__ void put8(void *o_t, int o_f32, int64_t at, const float (&y)[8])
{
    if (o_f32) {
        float4 *to = reinterpret_cast<float4 *>(static_cast<float *>(o_t) + at);
        to[0] = make_float4(y[0], y[1], y[2], y[3]);
        to[1] = make_float4(y[4], y[5], y[6], y[7]);
    } else {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(o_t) + at) =
            make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                       pack_bf16x2(y[6], y[7]));
    }
}

// A tile in its stage: bits 0-5: first row that counts, 6-11: one behind the
// last, kPage << i: part i has a page.
constexpr int kCore = 1 << 12, kNewest = 1 << 13, kFirst = 1 << 14, kEnds = 1 << 15,
              kPage = 1 << 16;

// Weights of core tiles are 2^(score - maximum + kCoreUp).
constexpr float kCoreUp = 15.f;

// What a pair costs a warp beside its tiles (queries, output, page numbers),
// and what a pooling does, in tiles: by the timeline of one batch, 64 rows of
// 1 to 16K tokens, where CTAs with many short rows took twice as long as the
// others without (an earlier form of the kernel took 72 us instead of 58).
constexpr int kPairTiles = 3, kPoolTiles = 4;

// WIDE: 9 to 16 query heads for a key/value head; STEP: cca_paged_step.
template <int D, int WARPS, int STAGES, bool WIDE, bool STEP>
__global__ void __launch_bounds__(WARPS * 32, 1)
    paged_decode_kernel(PagedView c, const uint16_t *__restrict__ q_t,
                        const uint16_t *__restrict__ k_t, const uint16_t *__restrict__ v_t,
                        void *__restrict__ o_t, int o_f32, float scale_log2,
                        float *__restrict__ part, unsigned int *__restrict__ tickets)
{
    using P = Pd<D>;
    constexpr int kWarps = WARPS, kThreads = WARPS * 32;
    constexpr int CH = D / 8;        // 16-byte chunks of a row
    constexpr int VH = D / 64;       // 128-byte pieces of a row
    constexpr int QR = WIDE ? 2 : 1; // query rows of a thread
    const int r = c.Hq / c.Hkv;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, qi = lane >> 2, qj = lane & 3;
    const int PS = part_floats(D, r);
    extern __shared__ __align__(16) char smem[];
    const int WB = warp_bytes(D, r, STAGES);
    char *ring = smem + warp * WB;
    // a warp's two partial results: one begun before its stretch, and the last one
    auto entry_at = [&](int e) {
        return reinterpret_cast<float *>(smem + (e >> 1) * WB + (e & 1 ? 0 : STAGES * P::STAGE));
    };
    // of the rows before b: 2^13 times their tiles and the number of those
    // that have any
    int64_t *before = reinterpret_cast<int64_t *>(smem + kWarps * WB);
    auto tiles_before = [&](int b) { return before[b] >> 13; };
    __shared__ int64_t sums[kWarps];
    __shared__ int4 meta[kWarps][STAGES];  // row, head and flags of the tiles in the ring
    __shared__ int ids[2 * kWarps];        // pairs of the partial results, -1: none
    __shared__ int pools_s[kWarps];
    __shared__ unsigned int arrived_s[2];  // CTAs at a shared pair before this one
    __shared__ int3 join_s[2];             // its parts, CTA of the first, its slot

    chain_begin();
    if (tid < 2 * kWarps) ids[tid] = -1;
    {  // the list: each thread sums its rows, then a scan over the block
        const int per = (c.B + kThreads - 1) / kThreads;
        const int b0 = min(tid * per, c.B), b1 = min(b0 + per, c.B);
        int64_t n = 0;
        for (int b = b0; b < b1; ++b) {
            bool over;
            before[b] = n;
            const int all = row_tiles<P::KEYS, STEP>(c, b, over).all;
            n += (static_cast<int64_t>(all) << 13) + (all > 0);
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
        int64_t add = x - n;
        for (int w = 0; w < warp; ++w) add += sums[w];
        for (int b = b0; b < b1; ++b) before[b] += add;
        if (b0 < c.B && b1 == c.B) before[c.B] = add + n;
        __syncthreads();
    }

    const uint32_t ring_s = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
    const int cc = lane % CH;  // this lane's chunk of the rows it copies
    // 16 rows of keys or values to shared memory at `to`; those outside
    // [tlo, thi) become zeros, row `fresh` comes from `in`.  Row x's chunk y
    // lies at chunk y ^ (x % 8) of its 128 bytes, so that the fragments'
    // reads below, 8 lanes at a time, meet no bank twice.
    constexpr int RPC = 32 / CH;     // rows that the warp copies at once
    constexpr int NU = 8 / RPC;      // copies until x % 8 comes again
    uint32_t to_off[NU];
#pragma unroll
    for (int u = 0; u < NU; ++u) {
        const int x = u * RPC + lane / CH;
        to_off[u] = (cc >> 3) * (kPart * 128) + x * 128 + (((cc & 7) ^ x) << 4);
    }
    const int from_off = lane / CH * D + cc * 8;
    auto copy_rows = [&](uint32_t to, const uint16_t *from, const uint16_t *in, int tlo, int thi,
                         int fresh) {
        const uint16_t *src = from + from_off;
        if (tlo == 0 && thi == kPart && fresh < 0) {  // as nearly always
#pragma unroll
            for (int u = 0; u < kPart / RPC; ++u)
                copy16(to + to_off[u % NU] + u / NU * 1024, src + u * RPC * D);
            return;
        }
#pragma unroll 1
        for (int u = 0; u < kPart / RPC; ++u) {
            const int x = u * RPC + lane / CH;
            const bool is_new = STEP && x == fresh;
            copy16_or_0(to + (cc >> 3) * (kPart * 128) + x * 128 + (((cc ^ x) & 7) << 4),
                        is_new ? in + cc * 8 : src + u * RPC * D,
                        is_new || (x >= tlo && x < thi));
        }
    };
    auto commit = [&]() { asm volatile("cp.async.commit_group;" ::: "memory"); };
    auto chunk = [&](const char *tile, int x, int y) {
        return *reinterpret_cast<const uint4 *>(tile + (y >> 3) * (kPart * 128) + x * 128 +
                                                (((y & 7) ^ (x & 7)) << 4));
    };
    // Queries of the pair as fragments: rows qi and (WIDE) qi + 8, the
    // dims 64 h + 16 qj .. + 15.
    uint4 qf[QR][2 * VH];
    float q_scale[QR];
    auto load_q = [&](int b, int h, bool core) {
#pragma unroll
        for (int x = 0; x < QR; ++x) {
            const int qrow = x * 8 + qi;
            q_scale[x] = scale_log2;
#pragma unroll
            for (int e = 0; e < 2 * VH; ++e)
                qf[x][e] = qrow < r
                               ? __ldg(reinterpret_cast<const uint4 *>(
                                     q_t +
                                     (static_cast<int64_t>(b) * c.Hq + h * r + qrow) * D +
                                     (e >> 1) * 64 + qj * 16 + (e & 1) * 8))
                               : make_uint4(0u, 0u, 0u, 0u);
            if (!core) continue;
            uint32_t top = 0;  // the row's largest magnitude, as bf16 bits
#pragma unroll
            for (int e = 0; e < 2 * VH; ++e)
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint32_t v = (&qf[x][e].x)[u] & 0x7fff7fffu;
                    top = max(top, max(v & 0xffffu, v >> 16));
                }
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // entries times 2^(13 - e), e: exponent of the largest one
            // (zero rows and exponents that leave the range: the nearest)
            const int e2 = top == 0 ? 13 : static_cast<int>(top >> 7) - 127;
            const int up = max(-100, min(100, 13 - e2));
            const float f = __int_as_float((127 + up) << 23);
            q_scale[x] = scale_log2 * __int_as_float((127 - up) << 23);
#pragma unroll
            for (int e = 0; e < 2 * VH; ++e)
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    uint32_t &v = (&qf[x][e].x)[u];
                    v = pack_f16x2(bf16_lo(v) * f, bf16_hi(v) * f);
                }
        }
    };

    // S of a tile: rows qi and qi + 8, keys 8 n + 2 qj + e.
    auto scores = [&](const char *tile, float (&s)[2][4], auto f16_c) {
        constexpr bool F16 = decltype(f16_c)::value;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll
            for (int x = 0; x < 2 * VH; ++x) {
                const uint4 k = chunk(tile, n * 8 + qi, (x >> 1) * 8 + qj * 2 + (x & 1));
                const uint4 a = qf[0][x];
                const uint4 z = WIDE ? qf[QR - 1][x] : make_uint4(0u, 0u, 0u, 0u);
                mma16816<F16>(s[n], a.x, z.x, a.y, z.y, k.x, k.y);
                mma16816<F16>(s[n], a.z, z.z, a.w, z.w, k.z, k.w);
            }
        }
    };

    // The append of token t of row b for one head: its rows to its page, and
    // the pooling of the group it completes (section 全局感知池化): the scores
    // of the group's keys against this token's queries, a softmax for each
    // query head, and the sums of keys and values weighted by their mean.
    auto append = [&](int b, int h, int64_t t) {
        using VT = typename RowVec<D>::T;
        const int mask = (1 << c.shift) - 1, g = c.g;
        const uint16_t *kin = k_t + (static_cast<int64_t>(b) * c.Hkv + h) * D;
        const uint16_t *vin = v_t + (static_cast<int64_t>(b) * c.Hkv + h) * D;
        // the group's tiles of 16 tokens (g <= 256: at most 17), token t in
        // the last one, and their pages; the tables are read at once, and
        // the counts with the keys and values, whose copies need no counts
        const bool ends = c.core_cols > 0 && (t + 1) % g == 0;
        const int64_t first = ends ? t - g + 1 : t, j = t / g, tile0 = first / kPart;
        const int n_tiles = static_cast<int>(t / kPart - tile0) + 1;
        const int skip = static_cast<int>(first - tile0 * kPart);
        const VT kx = reinterpret_cast<const VT *>(kin)[lane];
        const VT vx = reinterpret_cast<const VT *>(vin)[lane];
        const int id = lane < n_tiles ? page_at(c.raw_table, b, c.raw_cols,
                                                ((tile0 + lane) * kPart) >> c.shift, c.raw_pages)
                                      : 0;
        const int out =
            ends ? page_at(c.core_table, b, c.core_cols, j >> c.shift, c.core_pages) : 0;
        const int page = __shfl_sync(0xffffffffu, id, n_tiles - 1);
        // (count 1: the page is the row's own)
        const bool mine = page >= 0 && __ldg(c.raw_ref + page) == 1;
        const bool out_mine = !ends || (out >= 0 && __ldg(c.core_ref + out) == 1);
        auto put_row = [&]() {
            const int64_t at = page_row<D>(page, h, c.Hkv, c.shift, static_cast<int>(t) & mask);
            reinterpret_cast<VT *>(c.k_raw + at)[lane] = kx;
            reinterpret_cast<VT *>(c.v_raw + at)[lane] = vx;
        };
        if (!ends || __any_sync(0xffffffffu, id < 0 || out < 0)) {
            if (mine) put_row();
            if (lane == 0 && (ends || !mine)) atomicOr(&g_paged_decode_status, kStatusPage);
            return;
        }
        // scratch: scores [r][g], weights [g], a factor for each head, and
        // before them room for tiles of keys or values (one at least)
        const int n_scratch = (r + 1) * g + r;
        float *logit = reinterpret_cast<float *>(ring + WB) - n_scratch;
        float *weight = logit + r * g, *factor = weight + g;
        const int slots = (WB - 4 * n_scratch) / P::ROWS;
        const bool at_once = 2 * n_tiles <= slots;  // keys and values fit
        auto load = [&](int i0, int n, bool v, int slot) {
            for (int i = 0; i < n; ++i) {
                const int64_t p = (tile0 + i0 + i) * kPart;
                const int pg = __shfl_sync(0xffffffffu, id, i0 + i);
                const int thi = static_cast<int>(min(static_cast<int64_t>(kPart), t + 1 - p));
                copy_rows(ring_s + (slot + i) * P::ROWS,
                          (v ? c.v_raw : c.k_raw) +
                              page_row<D>(pg, h, c.Hkv, c.shift, static_cast<int>(p) & mask),
                          v ? vin : kin, i0 + i == 0 ? skip : 0, thi,
                          p + thi == t + 1 ? thi - 1 : -1);
            }
            commit();
        };
        auto wait = [&]() {
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncwarp();
        };
        const int step = at_once ? n_tiles : slots;
        for (int i0 = 0; i0 < n_tiles; i0 += step) {
            load(i0, min(step, n_tiles - i0), false, 0);
            if (at_once) load(0, n_tiles, true, n_tiles);
            if (i0 == 0) load_q(b, h, false);
            wait();
            for (int i = 0; i < min(step, n_tiles - i0); ++i) {
                float s[2][4];
                scores(ring + i * P::ROWS, s, std::false_type{});
#pragma unroll
                for (int x = 0; x < QR; ++x)
#pragma unroll
                    for (int n = 0; n < 2; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int pos = (i0 + i) * kPart + n * 8 + qj * 2 + e - skip;
                            if (pos >= 0 && pos < g && x * 8 + qi < r)
                                logit[(x * 8 + qi) * g + pos] = s[n][2 * x + e] * scale_log2;
                        }
            }
            __syncwarp();
        }
        // softmax over the scores of each head: four heads at once, 8 lanes each
        for (int k0 = 0; k0 < r; k0 += 4) {
            const int k = k0 + (lane >> 3);
            float *y = logit + k * g;
            float mx = -INFINITY, sum = 0.f;
            if (k < r)
                for (int i = lane & 7; i < g; i += 8) mx = fmaxf(mx, y[i]);
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            if (k < r)
                for (int i = lane & 7; i < g; i += 8) sum += y[i] = fast_exp2(y[i] - mx);
#pragma unroll
            for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (k < r && (lane & 7) == 0) factor[k] = 1.0f / (sum * static_cast<float>(r));
        }
        __syncwarp();
        for (int i = lane; i < g; i += 32) {
            float a = 0.f;
            for (int k = 0; k < r; ++k) a = fmaf(logit[k * g + i], factor[k], a);
            weight[i] = a;
        }
        __syncwarp();
        if (mine) put_row();
        if (!mine || !out_mine) {
            if (lane == 0) atomicOr(&g_paged_decode_status, kStatusPage);
            return;
        }
        const int64_t to = page_row<D>(out, h, c.Hkv, c.shift, static_cast<int>(j) & mask);
        bool over = false;
        for (int v = 0; v < 2; ++v) {
            float acc[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = 0.f;
            for (int i0 = 0; i0 < n_tiles; i0 += step) {
                const int n = min(step, n_tiles - i0);
                if (!at_once) {
                    load(i0, n, v, 0);
                    wait();
                }
                for (int i = 0; i < n; ++i) {
                    const char *tile = ring + ((at_once && v ? n_tiles : 0) + i) * P::ROWS;
#pragma unroll
                    for (int x = lane / CH; x < kPart; x += 32 / CH) {
                        const int pos = (i0 + i) * kPart + x - skip;
                        const float a = pos >= 0 && pos < g ? weight[pos] : 0.f;
                        const uint4 y = chunk(tile, x, cc);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            acc[2 * e] = fmaf(a, bf16_lo((&y.x)[e]), acc[2 * e]);
                            acc[2 * e + 1] = fmaf(a, bf16_hi((&y.x)[e]), acc[2 * e + 1]);
                        }
                    }
                }
                __syncwarp();
            }
#pragma unroll
            for (int o = CH; o < 32; o <<= 1)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[e] += __shfl_xor_sync(0xffffffffu, acc[e], o);
            if (lane < CH) {
                uint4 y;
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    (&y.x)[e] = pack_f16x2(clamp_f16(acc[2 * e], over), clamp_f16(acc[2 * e + 1], over));
                *reinterpret_cast<uint4 *>((v ? c.v_core : c.k_core) + to + cc * 8) = y;
            }
        }
        if (over) atomicOr(&g_paged_decode_status, kStatusRange);
    };

    auto pooled = [&](int b) {
        return before[b + 1] > before[b] && c.core_cols > 0 && __ldg(c.lens + b) % c.g == 0;
    };
    // Rows without tokens have a zero output; the newest token of the others
    // is appended.  No tile reads what is written here: its key and value
    // come from the inputs, and the core row of the group it completes is not
    // yet among those that it sees.  The pairs go round the CTAs, the last
    // ones first, which have no tiles when there are few.
    const int64_t pairs = static_cast<int64_t>(c.B) * c.Hkv;
    const int64_t pair0 =
        kCtas - 1 - static_cast<int>(blockIdx.x) + kCtas * static_cast<int64_t>(warp);
    if (STEP) {  // groups that this warp is going to pool
        int pools = 0;
        for (int64_t pair = pair0; pair < pairs; pair += kCtas * kWarps)
            pools += pooled(static_cast<int>(pair / c.Hkv));
        if (lane == 0) pools_s[warp] = pools;
        __syncthreads();
    }
    for (int64_t pair = pair0; pair < pairs; pair += kCtas * kWarps) {
        const int b = static_cast<int>(pair / c.Hkv);
        const int h = static_cast<int>(pair - static_cast<int64_t>(b) * c.Hkv);
        if (before[b + 1] == before[b]) {
            const int64_t orow = static_cast<int64_t>(b) * c.Hq + h * r;
            for (int x = lane * 4; x < r * D; x += 128)
                put4(o_t, o_f32, orow * D + x, make_float4(0.f, 0.f, 0.f, 0.f));
        } else if (STEP) {
            append(b, h, __ldg(c.lens + b) - 1);
        }
    }

    // The list of the tiles, row by row and head by head, each pair preceded
    // by what it costs beside them, is cut into equal stretches: one for each
    // CTA (enough for each warp, as long as there is), and in it for each warp.
    auto first_of = [&](int b) { return tiles_before(b) * c.Hkv; };
    auto cost_of = [&](int b) {
        return (tiles_before(b) + kPairTiles * (before[b] & 8191)) * c.Hkv;
    };
    const int64_t total = cost_of(c.B);
    const int n_ctas =
        static_cast<int>(min(static_cast<int64_t>(gridDim.x), (total + kWarps - 1) / kWarps));
    if (blockIdx.x >= n_ctas) return;
    // the first tile at or behind place x of the list
    struct Place {
        int64_t tile;
        int b, h, i;
    };
    auto place_from = [&](int64_t x) {
        if (x >= total) return Place{first_of(c.B), c.B, 0, 0};
        int a = 0, z = c.B - 1;
        while (a < z) {
            const int mid = (a + z + 1) >> 1;
            if (cost_of(mid) <= x)
                a = mid;
            else
                z = mid - 1;
        }
        const int n = static_cast<int>(tiles_before(a + 1) - tiles_before(a));
        const int64_t in_row = x - cost_of(a);
        const int h = static_cast<int>(in_row >> 32 == 0
                                           ? static_cast<uint32_t>(in_row) / (n + kPairTiles)
                                           : in_row / (n + kPairTiles));
        const int i = static_cast<int>(
            max(static_cast<int64_t>(0),
                in_row - static_cast<int64_t>(h) * (n + kPairTiles) - kPairTiles));
        return Place{first_of(a) + static_cast<int64_t>(h) * n + i, a, h, i};
    };
    // the CTA that has tile i of a head's n in row b
    auto cta_of = [&](int b, int h, int64_t n, int64_t i) {
        const int64_t x = cost_of(b) + h * (n + kPairTiles) + kPairTiles + i;
        return static_cast<int>(((x + 1) * n_ctas - 1) / total);
    };
    const int64_t my_lo = total * blockIdx.x / n_ctas, my_hi = total * (blockIdx.x + 1) / n_ctas;
    int64_t cta_lo, cta_hi;
    int n_tiles, at_b, at_h, at_i;  // this warp's tiles; the first one's row, head and place
    {
        // lane w: where warp w's part ends
        const int mine = STEP && lane < kWarps ? pools_s[lane] : 0;
        int upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        const int all = __shfl_sync(0xffffffffu, upto, 31);
        const int64_t n = my_hi - my_lo;
        int64_t end = (n + kPoolTiles * all) * (lane + 1) / kWarps - kPoolTiles * upto;
        end = lane + 1 >= kWarps ? n : max(static_cast<int64_t>(0), min(n, end));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, end, o);
            if (lane >= o) end = max(end, y);
        }
        const int64_t lo = __shfl_sync(0xffffffffu, end, max(warp - 1, 0));
        const int64_t hi = __shfl_sync(0xffffffffu, end, warp);
        // lanes 0 and 1: this warp's part, 2 and 3: the CTA's stretch
        const Place at = place_from(lane == 0   ? my_lo + (warp > 0 ? lo : 0)
                                    : lane == 1 ? my_lo + hi
                                    : lane == 2 ? my_lo
                                                : my_hi);
        cta_lo = __shfl_sync(0xffffffffu, at.tile, 2);
        cta_hi = __shfl_sync(0xffffffffu, at.tile, 3);
        n_tiles = static_cast<int>(__shfl_sync(0xffffffffu, at.tile, 1) -
                                   __shfl_sync(0xffffffffu, at.tile, 0));
        at_b = __shfl_sync(0xffffffffu, at.b, 0);
        at_h = __shfl_sync(0xffffffffu, at.h, 0);
        at_i = __shfl_sync(0xffffffffu, at.i, 0);
    }

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

    if (n_tiles > 0) {
        bool over, bad = false;
        // (rows that have tiles are not held)
        RowTiles row = row_tiles<P::KEYS, false>(c, at_b, over);
        int from = 0, id = 0;  // pages of the parts PARTS * from + lane of the pair
        auto load_ids = [&]() {
            from = at_i;
            const int i = at_i + lane / P::PARTS, x = lane % P::PARTS * kPart;
            id = -1;
            if (i < row.core)
                id = page_at(c.core_table, at_b, c.core_cols,
                             (static_cast<int64_t>(i) * P::KEYS + x) >> c.shift, c.core_pages);
            else if (i < row.all)
                id = page_at(c.raw_table, at_b, c.raw_cols,
                             ((row.ws / P::KEYS + (i - row.core)) * P::KEYS + x) >> c.shift,
                             c.raw_pages);
        };
        load_ids();

        // Ask for the next tile.
        int asked = 0;
        auto ask = [&](int stage) {
            if (at_i - from >= 32 / P::PARTS) load_ids();
            const bool core = at_i < row.core;
            const int64_t p = (core ? at_i : row.ws / P::KEYS + (at_i - row.core)) *
                              static_cast<int64_t>(P::KEYS);
            const int tlo = core ? 0 : static_cast<int>(max(static_cast<int64_t>(0), row.ws - p));
            const int thi = static_cast<int>(min(static_cast<int64_t>(P::KEYS),
                                                 (core ? row.n_core : row.len) - p));
            const bool newest = STEP && !core && p + thi == row.len;
            const int64_t in = (static_cast<int64_t>(at_b) * c.Hkv + at_h) * D;
            int flags = tlo | thi << 6 | (core ? kCore : 0) | (newest ? kNewest : 0) |
                        (at_i == 0 ? kFirst : 0);
#pragma unroll
            for (int y = 0; y < P::PARTS; ++y) {
                const int page = __shfl_sync(0xffffffffu, id, (at_i - from) * P::PARTS + y);
                const int plo = max(0, tlo - y * kPart), phi = min(kPart, thi - y * kPart);
                const int64_t off =
                    page_row<D>(max(page, 0), at_h, c.Hkv, c.shift,
                                static_cast<int>(p + y * kPart) & ((1 << c.shift) - 1));
                const int valid = page >= 0 ? phi : 0;
                const int fresh = newest ? thi - 1 - y * kPart : -1;
                const uint32_t to = ring_s + stage * P::STAGE + y * P::ROWS;
                copy_rows(to, (core ? c.k_core : c.k_raw) + off, k_t + in, plo, valid, fresh);
                copy_rows(to + P::PARTS * P::ROWS, (core ? c.v_core : c.v_raw) + off, v_t + in, plo,
                          valid, fresh);
                if (page >= 0) flags |= kPage << y;
                bad |= page < 0 && plo < phi;
            }
            if (at_i == 0 || asked == 0) {  // the pair's queries, to L1
                const char *q = reinterpret_cast<const char *>(
                    q_t + (static_cast<int64_t>(at_b) * c.Hq + at_h * r) * D);
                if (lane * 128 < r * D * 2)
                    asm volatile("prefetch.global.L1 [%0];" ::"l"(q + lane * 128));
            }
            const bool ends = at_i + 1 == row.all;
            if (lane == 0)
                meta[warp][stage] = make_int4(at_b, at_h, flags | (ends ? kEnds : 0), 0);
            if (!ends) {
                ++at_i;
                return;
            }
            at_i = 0;
            if (++at_h == c.Hkv) {
                at_h = 0;
                do {
                    if (++at_b >= c.B) return;  // the end of the list
                } while (before[at_b + 1] == before[at_b]);
                row = row_tiles<P::KEYS, false>(c, at_b, over);
            }
            load_ids();
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
        // S, softmax and P V of a tile.
        auto add_tile = [&](const char *tile, int flags, auto f16_c) {
            constexpr bool F16 = decltype(f16_c)::value;
            constexpr int NK = 2 * P::PARTS;  // keys 8 n + 2 qj + e
            float s[NK][4];
#pragma unroll
            for (int y = 0; y < P::PARTS; ++y)
                scores(tile + y * P::ROWS, *reinterpret_cast<float(*)[2][4]>(s + 2 * y), f16_c);
            const int tlo = flags & 63, thi = flags >> 6 & 63;
            constexpr int kAll = kPage * ((1 << P::PARTS) - 1);
            const bool all = tlo == 0 && thi == P::KEYS && (flags & kAll) == kAll;
            uint32_t ph[QR][NK], pl[QR][NK];
#pragma unroll
            for (int x = 0; x < QR; ++x) {
                float top = -INFINITY;
                if (!all) {
#pragma unroll
                    for (int n = 0; n < NK; ++n)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            // a missing page leaves the newest row alone
                            const int key = n * 8 + qj * 2 + e;
                            const bool ok = flags & (kPage << (n / 2))
                                                ? key >= tlo && key < thi
                                                : (flags & kNewest) && key == thi - 1;
                            if (!ok) s[n][2 * x + e] = -INFINITY;
                        }
                }
#pragma unroll
                for (int n = 0; n < NK; ++n)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        s[n][2 * x + e] *= q_scale[x];
                        top = fmaxf(top, s[n][2 * x + e]);
                    }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                const float to = fmaxf(m[x], F16 ? top - kCoreUp : top);
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
                for (int n = 0; n < NK; ++n) {
                    const float p0 = fast_exp2(s[n][2 * x] - use);
                    const float p1 = fast_exp2(s[n][2 * x + 1] - use);
                    l[x] += p0 + p1;
                    split2<F16, WIDE>(p0, p1, ph[x][n], pl[x][n]);
                }
            }
#pragma unroll
            for (int y = 0; y < P::PARTS; ++y)
#pragma unroll
                for (int h = 0; h < VH; ++h) {
                    uint4 v[4];
#pragma unroll
                    for (int n = 0; n < 4; ++n)
                        v[n] = chunk(tile + (P::PARTS + y) * P::ROWS,
                                     (n >> 1) * 8 + qj * 2 + (n & 1), h * 8 + qi);
#pragma unroll
                    for (int u = 0; u < 4; ++u)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t sel = e ? 0x7632 : 0x5410;
                            const uint32_t b0 = __byte_perm((&v[0].x)[u], (&v[1].x)[u], sel);
                            const uint32_t b1 = __byte_perm((&v[2].x)[u], (&v[3].x)[u], sel);
                            float(&acc)[4] = o[h * 8 + u * 2 + e];
                            const uint32_t(&h0)[NK] = ph[0], (&l0)[NK] = pl[0];
                            if constexpr (WIDE) {
                                const uint32_t(&h1)[NK] = ph[QR - 1], (&l1)[NK] = pl[QR - 1];
                                mma16816<F16>(acc, h0[2 * y], h1[2 * y], h0[2 * y + 1],
                                              h1[2 * y + 1], b0, b1);
                                mma16816<F16>(acc, l0[2 * y], l1[2 * y], l0[2 * y + 1],
                                              l1[2 * y + 1], b0, b1);
                            } else {
                                mma16816<F16>(acc, h0[2 * y], l0[2 * y], h0[2 * y + 1],
                                              l0[2 * y + 1], b0, b1);
                            }
                        }
                }
        };

#pragma unroll 1
        for (; asked < STAGES - 1; ++asked) {
            if (asked < n_tiles) ask(asked);
            commit();
        }
        reset();
        bool from_start = false, q_core = false, loaded = false;
        int stage = 0, next = STAGES - 1;
#pragma unroll 1
        for (int x = 0; x < n_tiles; ++x) {
            // tile x has arrived for every lane, and every lane is done with
            // tile x - 1, whose stage the next copies take
            asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
            __syncwarp();
            if (asked < n_tiles) {
                ask(next);
                ++asked;
            }
            commit();
            const int4 mt = meta[warp][stage];
            const int flags = mt.z;
            const bool core = flags & kCore;
            if (flags & kFirst) from_start = true;
            if (loaded && q_core != core) {
                // from the pair's core rows to its raw ones, whose weights are
                // relative to the maximum itself
                const float f = fast_exp2(-kCoreUp);
#pragma unroll
                for (int y = 0; y < QR; ++y) {
                    m[y] += kCoreUp;
                    l[y] *= f;
                }
#pragma unroll
                for (int n = 0; n < D / 8; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) o[n][e] *= f;
            }
            if (!loaded || q_core != core) {
                load_q(mt.x, mt.y, core);
                loaded = true;
                q_core = core;
            }
            char *tile = ring + stage * P::STAGE;
            if (core)
                add_tile(tile, flags, std::true_type{});
            else
                add_tile(tile, flags, std::false_type{});
            const bool done = x + 1 == n_tiles;
            if ((flags & kEnds) || done) {
                // the pair's output if this warp has seen all of it, else a
                // partial result
                const bool whole = from_start && (flags & kEnds);
                if (done) __syncwarp();  // (its place is the ring, which all have read)
                float *to = entry_at(warp * 2 + done);
#pragma unroll
                for (int y = 0; y < QR; ++y) {
                    float sum = l[y];
                    sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                    sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                    const int qrow = y * 8 + qi;
                    if (qrow >= r) continue;
                    const float inv = whole ? (sum > 0.f ? 1.0f / sum : 0.f) : 1.f;
                    const int64_t orow = (static_cast<int64_t>(mt.x) * c.Hq + mt.y * r + qrow) * D;
#pragma unroll
                    for (int h = 0; h < VH; ++h)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float y8[8];
#pragma unroll
                            for (int n = 0; n < 8; ++n) {
                                const float(&a)[4] = o[h * 8 + n];
                                // (an infinite value times P_lo is infinite
                                // with any sign, or NaN)
                                const float hi = WIDE ? a[2 * y + e] : a[e];
                                const bool both = !WIDE && fabsf(hi) < INFINITY;
                                y8[n] = (both ? hi + a[2 + e] : hi) * inv;
                            }
                            const int dim = h * 64 + (2 * qj + e) * 8;
                            if (whole)
                                put8(o_t, o_f32, orow + dim, y8);
                            else
                                put8(to, 1, qrow * D + dim, y8);
                        }
                    if (!whole && qj == 0) {
                        to[r * D + qrow] = m[y];
                        to[r * D + r + qrow] = sum;
                    }
                }
                if (!whole && lane == 0) ids[warp * 2 + done] = mt.x * c.Hkv + mt.y;
                reset();
                loaded = false;
            }
            stage = stage + 1 == STAGES ? 0 : stage + 1;
            next = next + 1 == STAGES ? 0 : next + 1;
        }
        if (bad && lane == 0) atomicOr(&g_paged_decode_status, kStatusPage);
    }
    __syncthreads();

    // Join the warps' partial results, pair by pair: an output if this CTA
    // has all of the pair, else its partial result for the other CTAs.
    const int my_id = lane < 2 * kWarps ? ids[lane] : -1;
    unsigned int left = __ballot_sync(0xffffffffu, my_id >= 0);
    int n_slots = 0, slot0_pair = -1, slot1_pair = -1, turn = 0;
    while (left) {
        const int pair = ids[__ffs(left) - 1];
        const unsigned int group = __ballot_sync(0xffffffffu, my_id == pair);
        left &= ~group;
        const int b = pair / c.Hkv, h = pair - b * c.Hkv;
        const int64_t n = tiles_before(b + 1) - tiles_before(b), begin = first_of(b) + h * n;
        const bool whole = begin >= cta_lo && begin + n <= cta_hi;
        float *to = part + (static_cast<int64_t>(blockIdx.x) * 2 + n_slots) * PS;
        // a warp for a query head of a pair: the entries' weights lane by
        // lane, then the head's dims over the lanes
        for (int q = 0; q < r; ++q, turn = turn + 1 == kWarps ? 0 : turn + 1) {
            if (turn != warp) continue;
            const bool in = group >> lane & 1;
            const float m_e = in ? entry_at(lane)[r * D + q] : -INFINITY;
            const float l_e = in ? entry_at(lane)[r * D + r + q] : 0.f;
            const float mx = warp_max(m_e), use = mx == -INFINITY ? 0.f : mx;
            float f = fast_exp2(m_e - use);
            const float sum = warp_sum(f * l_e);
            if (whole) f *= sum > 0.f ? 1.0f / sum : 0.f;
            const int dim = lane * 4 % D;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (unsigned int x = group; x; x &= x - 1) {
                const int e = __ffs(x) - 1;
                const float f_e = __shfl_sync(0xffffffffu, f, e);
                const float4 y = *reinterpret_cast<const float4 *>(entry_at(e) + q * D + dim);
                acc.x = fmaf(f_e, y.x, acc.x);
                acc.y = fmaf(f_e, y.y, acc.y);
                acc.z = fmaf(f_e, y.z, acc.z);
                acc.w = fmaf(f_e, y.w, acc.w);
            }
            if (lane * 4 < D) {
                if (whole)
                    put4(o_t, o_f32, (static_cast<int64_t>(b) * c.Hq + h * r + q) * D + dim, acc);
                else
                    *reinterpret_cast<float4 *>(to + q * D + dim) = acc;
            }
            if (!whole && lane == 0) {
                to[r * D + q] = mx;
                to[r * D + r + q] = sum;
            }
        }
        if (!whole) (n_slots++ == 0 ? slot0_pair : slot1_pair) = pair;
    }
    if (n_slots == 0) return;

    // Pairs shared with other CTAs: the last one to arrive joins them.
    __syncthreads();
    if (lane < n_slots && warp < 2) {
        const int pair = lane == 0 ? slot0_pair : slot1_pair;
        if (warp == 0) {
            __threadfence();  // (for the whole CTA, which has met at the barrier)
            arrived_s[lane] = atomicAdd(tickets + pair, 1u);
            __threadfence();
        } else {
            const int b = pair / c.Hkv, h = pair - b * c.Hkv;
            const int64_t n = tiles_before(b + 1) - tiles_before(b), begin = first_of(b) + h * n;
            const int c0 = cta_of(b, h, n, 0), n_parts = cta_of(b, h, n, n - 1) - c0 + 1;
            // CTA c0 holds the pair in its last slot: the second one if a
            // pair that begins before the CTA takes the first
            bool second = false;
            const int64_t clo = place_from(total * c0 / n_ctas).tile;
            if (clo < begin) {
                const int rb = row_at(clo);
                second = (clo - first_of(rb)) % (tiles_before(rb + 1) - tiles_before(rb)) != 0;
            }
            join_s[lane] = make_int3(n_parts, c0, second);
        }
    }
    __syncthreads();
    for (int k = 0; k < n_slots; ++k) {
        const int n_parts = join_s[k].x;
        if (arrived_s[k] != static_cast<unsigned int>(n_parts - 1)) continue;
        const int pair = k == 0 ? slot0_pair : slot1_pair;
        if (tid == 0) tickets[pair] = 0;  // ready for the next call
        const int b = pair / c.Hkv, h = pair - b * c.Hkv;
        const float *p0 = part + static_cast<int64_t>(join_s[k].y) * 2 * PS;
        const int skip0 = join_s[k].z ? PS : 0;
        auto part_at = [&](int y) { return p0 + (y == 0 ? skip0 : y * 2 * PS); };
        // A thread for 4 dims of a head, and as many threads for those as
        // there are, each with parts of its own, 8 asked for at once.
        const int cols = r * D / 4, groups = max(1, kThreads / cols);
        const int grp = tid / min(cols, kThreads);
        float4 *red = reinterpret_cast<float4 *>(smem);               // [kThreads]
        float2 *red_ml = reinterpret_cast<float2 *>(red + kThreads);  // [kThreads]
        for (int i = tid - grp * cols; i < cols; i += kThreads) {
            const int q = i / (D / 4);
            float mx = -INFINITY, sum = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            auto add = [&](float m2, float l2, float4 v) {
                const float to = fmaxf(mx, m2), use = to == -INFINITY ? 0.f : to;
                const float f = fast_exp2(mx - use), f2 = fast_exp2(m2 - use);
                mx = to;
                sum = fmaf(sum, f, l2 * f2);
                acc.x = fmaf(acc.x, f, v.x * f2);
                acc.y = fmaf(acc.y, f, v.y * f2);
                acc.z = fmaf(acc.z, f, v.z * f2);
                acc.w = fmaf(acc.w, f, v.w * f2);
            };
            for (int y0 = grp; grp < groups && y0 < n_parts; y0 += 8 * groups) {
                float m8[8], l8[8];
                float4 v8[8];
#pragma unroll
                for (int u = 0; u < 8; ++u) {
                    const int y = y0 + u * groups;
                    m8[u] = -INFINITY;
                    l8[u] = 0.f;
                    v8[u] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (y < n_parts) {
                        const float *p = part_at(y);
                        m8[u] = __ldcg(p + r * D + q);
                        l8[u] = __ldcg(p + r * D + r + q);
                        v8[u] = __ldcg(reinterpret_cast<const float4 *>(p) + i);
                    }
                }
#pragma unroll
                for (int u = 0; u < 8; ++u) add(m8[u], l8[u], v8[u]);
            }
            if (groups > 1) {  // (one round: cols < kThreads)
                red[tid] = acc;
                red_ml[tid] = make_float2(mx, sum);
                __syncthreads();
                for (int y = 1; grp == 0 && y < groups; ++y)
                    add(red_ml[y * cols + i].x, red_ml[y * cols + i].y, red[y * cols + i]);
            }
            if (grp == 0) {
                const float inv = sum > 0.f ? 1.0f / sum : 0.f;
                put4(o_t, o_f32, (static_cast<int64_t>(b) * c.Hq + h * r) * D + i * 4,
                     make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv));
            }
        }
        __syncthreads();  // shared memory is used again
    }
}

}  // namespace

size_t paged_decode_part_bytes(const cca_paged_cache &c)
{
    return sizeof(float) * 2 * kCtas * part_floats(c.d, c.Hq / c.Hkv);
}

cudaError_t launch_paged_decode(const cca_paged_cache &c, int layer, const void *q_t,
                                const void *k_t, const void *v_t, void *o_t, bool o_f32,
                                void *workspace, cudaStream_t s)
{
    const PagedWorkspace w = paged_workspace(c);
    char *base = static_cast<char *>(workspace);
    const int r = c.Hq / c.Hkv;
    PagedView v = paged_view(c, layer);
    v.held = reinterpret_cast<const long long *>(base + w.held);
    const float scale_log2 = kLog2e / sqrtf(static_cast<float>(c.d));
    auto go = [&](auto kern, int warps, int stages) {
        const size_t smem = decode_smem(c.d, r, warps, stages, c.B);
        const cudaError_t e = allow_smem(kern, smem, kOwnSmem);
        if (e != cudaSuccess) return e;
        return launch_chained(kern, kCtas, warps * 32, smem, s, v, static_cast<const uint16_t *>(q_t),
                              static_cast<const uint16_t *>(k_t),
                              static_cast<const uint16_t *>(v_t), o_t, o_f32 ? 1 : 0, scale_log2,
                              reinterpret_cast<float *>(base + w.part),
                              reinterpret_cast<unsigned int *>(base + w.tickets));
    };
    auto run = [&](auto d, auto warps, auto stages, auto wide) {
        constexpr int D = decltype(d)::value, W = decltype(warps)::value,
                      S = decltype(stages)::value;
        constexpr bool WIDE = decltype(wide)::value;
        return k_t != nullptr ? go(paged_decode_kernel<D, W, S, WIDE, true>, W, S)
                              : go(paged_decode_kernel<D, W, S, WIDE, false>, W, S);
    };
    auto fits = [&](int warps, int stages) {
        return decode_smem(c.d, r, warps, stages, c.B) <= kSmemMost - kOwnSmem;
    };
    using std::integral_constant;
    const integral_constant<int, 128> d128{};
    const integral_constant<int, 64> d64{};
    const integral_constant<int, 12> n12{};
    const integral_constant<int, 8> n8{};
    const integral_constant<int, 3> n3{};
    const integral_constant<int, 2> n2{};
    const std::true_type wide{};
    const std::false_type narrow{};
    // 12 warps, as many as 168 registers allow, or 8 where more than 8 heads
    // or the room ask for it.  (8 with a ring of 3, everywhere: the 8 rows
    // above in 122 to 125 us instead of 124, 64 rows of 1 to 16K tokens with
    // 8 key/value heads in 43 instead of 50.)
    if (c.d == 128) {
        if (r > 8) return run(d128, n8, n2, wide);
        if (fits(12, 2)) return run(d128, n12, n2, narrow);
        if (fits(8, 3)) return run(d128, n8, n3, narrow);
        return run(d128, n8, n2, narrow);
    }
    if (r > 8) return run(d64, n8, n2, wide);
    if (fits(12, 2)) return run(d64, n12, n2, narrow);
    return run(d64, n8, n2, narrow);
}

cudaError_t paged_decode_status_read_clear(unsigned int *v)
{
    unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(v, g_paged_decode_status, sizeof(*v));
    if (e == cudaSuccess && *v) e = cudaMemcpyToSymbol(g_paged_decode_status, &zero, sizeof(zero));
    return e;
}

}  // namespace cca
