// The paged cache's pages: room for tokens (cca_paged_reserve), filling from
// packed prompts (cca_paged_fill), rows that take over other rows
// (cca_paged_fork) and compaction (cca_paged_compact).
//
// Everything about pages is decided on the device, from lens, tables and
// counts, by rules without an order that could vary: counts change by
// integer atomics (any order gives the same sum), and the k-th page that is
// wanted gets the k-th free page, by a scan over the pool.
#include <cooperative_groups.h>

#include "packed.cuh"
#include "paged.cuh"
#include "paged.h"

namespace cca {

__device__ unsigned int g_paged_tables_status;  // kStatusCapacity, kStatusPage, kStatusSeqlens

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;         // of the kernels that plan
constexpr int kChunk = 4 * kThreads;  // pages that a block looks at at once

struct Pool {  // one of the two pools' tables
    int *table, *ref;
    int cols, pages;
};

struct TablesView {
    Pool pool[2];  // core, raw
    long long *lens;
    int B, g, w, shift;
};

__device__ __forceinline__ void report(unsigned int bits)
{
    atomicOr(&g_paged_tables_status, bits);
}

// Exclusive sums over the block (kThreads threads) of each thread's x;
// total: the sums of all.  One barrier; `room` is used again only after
// another one.
template <int N, class T>
__device__ __forceinline__ void block_scan(T (&x)[N], T (&total)[N], T (&room)[kThreads / 32][N])
{
    constexpr int W = kThreads / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T in[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        in[i] = x[i];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T y = __shfl_up_sync(0xffffffffu, x[i], o);
            if (lane >= o) x[i] += y;
        }
        if (lane == 31) room[warp][i] = x[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        T y = lane < W ? room[lane][i] : T(0);
#pragma unroll
        for (int o = 1; o < W; o <<= 1) {
            const T z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
        }
        total[i] = __shfl_sync(0xffffffffu, y, W - 1);
        const T before = __shfl_sync(0xffffffffu, y, warp > 0 ? warp - 1 : 0);
        x[i] += (warp > 0 ? before : T(0)) - in[i];
    }
}

// Free pages among this thread's four of a chunk, a bit for each.
__device__ __forceinline__ int free_bits(const int *ref, int pages, int chunk)
{
    int bits = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        const int p = chunk + threadIdx.x * 4 + u;
        if (p < pages && __ldcg(ref + p) == 0) bits |= 1 << u;
    }
    return bits;
}

// use(k, page) for this thread's free pages, the first of them the k-th, as
// long as k < want.
template <class F>
__device__ __forceinline__ void use_free(int bits, int chunk, int k, int want, F use)
{
    for (int u = 0; u < 4; ++u)
        if (bits >> u & 1) {
            if (k < want) use(k, chunk + threadIdx.x * 4 + u);
            ++k;
        }
}

// cca_paged_reserve: a cluster of two blocks, one for each pool; both plan
// all rows, then each takes its own pool's pages.  Bound by the chain of
// loads and barriers (a scan of everything at once, one exchange between the
// blocks): 5 us for a few rows.
struct Grow {
    int64_t len, n;       // the row's length, the tokens it is given
    bool refused;         // asked for what its table cannot take
    int core, n_core;     // first column and number of its new pages
    int raw, n_raw;
    int gone, gone_end;   // raw columns that go
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads)
    reserve_kernel(TablesView v, const long long *__restrict__ n_new, long long n_all,
                   long long *__restrict__ held)
{
    // of each row: wanted pages of my pool before it, [B], and the column of
    // its first one (-1: nothing granted), [B]
    extern __shared__ int plan[];
    __shared__ int64_t rows_room[kThreads / 32][2];
    __shared__ int free_room[kThreads / 32][2], chunk_room[2][kThreads / 32][1];
    __shared__ int free_pages;
    chain_begin();
    cg::cluster_group cluster = cg::this_cluster();
    const int me = cluster.block_rank();
    int *before = plan, *column = plan + v.B;
    const Pool &pool = v.pool[me];
    const bool core = v.pool[0].cols > 0;
    const int64_t longest = paged_max_len(v.pool[1].cols, v.pool[0].cols, v.g, v.shift);
    auto grow = [&](int b) {
        Grow r = {};
        r.len = v.lens[b];
        const int64_t n = n_new != nullptr ? n_new[b] : (r.len > 0 ? n_all : 0);
        r.n = n > 0 && r.len >= 0 && n <= longest - r.len ? n : 0;
        r.refused = r.n != n;
        if (r.n == 0) return r;
        const PagedCols a = paged_cols(r.len, v.g, v.w, v.shift, core);
        const PagedCols z = paged_cols(r.len + r.n, v.g, v.w, v.shift, core);
        r.core = a.core_hi;
        r.n_core = z.core_hi - a.core_hi;
        r.raw = max(a.raw_hi, z.raw_lo);
        r.n_raw = z.raw_hi - r.raw;
        r.gone = a.raw_lo;
        r.gone_end = min(a.raw_hi, z.raw_lo);
        return r;
    };
    const int per = (v.B + kThreads - 1) / kThreads;
    const int b0 = min(static_cast<int>(threadIdx.x) * per, v.B), b1 = min(b0 + per, v.B);
    const int bits = free_bits(pool.ref, pool.pages, 0);
    Grow first = {};
    if (b0 < b1) first = grow(b0);
    auto row_of = [&](int b) { return b == b0 ? first : grow(b); };
    int64_t at[2] = {0, 0}, want[2];
    for (int b = b0; b < b1; ++b) {
        const Grow r = row_of(b);
        at[0] += r.n_core;
        at[1] += r.n_raw;
    }
    int free_at[2] = {__popc(bits), 0}, free_all[2];  // in the first chunk, behind it
    for (int chunk = kChunk; chunk < pool.pages; chunk += kChunk)
        free_at[1] += __popc(free_bits(pool.ref, pool.pages, chunk));
    block_scan(at, want, rows_room);
    block_scan(free_at, free_all, free_room);
    if (threadIdx.x == 0) free_pages = free_all[0] + free_all[1];
    cluster.sync();
    const int other = *cluster.map_shared_rank(&free_pages, me ^ 1);
    const int mine = free_all[0] + free_all[1];
    const int have[2] = {me == 0 ? mine : other, me == 0 ? other : mine};
    for (int b = b0; b < b1; ++b) {
        const Grow r = row_of(b);
        const bool ok = (r.n_core == 0 || at[0] + r.n_core <= have[0]) &&
                        (r.n_raw == 0 || at[1] + r.n_raw <= have[1]);
        // (no page is taken for what lies beyond the last free one)
        before[b] = static_cast<int>(min(at[me], static_cast<int64_t>(INT32_MAX)));
        column[b] = ok && r.n > 0 ? (me == 0 ? r.core : r.raw) : -1;
        if (me == 0 && (!ok || r.refused)) {
            report(kStatusCapacity);
            if (held != nullptr) held[b] = r.len;
        }
        at[0] += r.n_core;
        at[1] += r.n_raw;
    }
    __syncthreads();
    auto use = [&](int k, int page) {
        int lo = 0, hi = v.B - 1;  // the row of the k-th wanted page
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (before[mid] <= k)
                lo = mid;
            else
                hi = mid - 1;
        }
        if (column[lo] < 0) return;
        pool.table[static_cast<int64_t>(lo) * pool.cols + column[lo] + (k - before[lo])] = page;
        pool.ref[page] = 1;
    };
    const int wanted = static_cast<int>(min(want[me], static_cast<int64_t>(mine)));
    use_free(bits, 0, free_at[0], wanted, use);
    int base = free_all[0];
    for (int chunk = kChunk; chunk < pool.pages && base < wanted; chunk += kChunk) {
        const int more = free_bits(pool.ref, pool.pages, chunk);
        int x[1] = {__popc(more)}, n[1];
        block_scan(x, n, chunk_room[chunk / kChunk & 1]);
        use_free(more, chunk, base + x[0], wanted, use);
        base += n[0];
    }
    __syncthreads();
    // raw pages before the new window go
    if (me == 1)
        for (int b = b0; b < b1; ++b) {
            if (column[b] < 0) continue;
            const Grow r = row_of(b);
            for (int col = r.gone; col < r.gone_end; ++col) {
                int *e = pool.table + static_cast<int64_t>(b) * pool.cols + col;
                if (*e >= 0 && *e < pool.pages)
                    atomicSub(pool.ref + *e, 1);
                else
                    report(kStatusPage);
                *e = -1;
            }
        }
    cluster.sync();  // lens is read by both until here
    if (me == 0)
        for (int b = b0; b < b1; ++b)
            if (column[b] >= 0) {
                const Grow r = row_of(b);
                v.lens[b] = r.len + r.n;
                if (held != nullptr) held[b] = 0;
            }
}

// cca_paged_fill: a warp takes 32 packed rows (or core rows) of one head:
// first each lane finds the place of its row, then all copy the rows' keys
// and values, 8 rows asked for at once (D = 64: 16).
template <int D>
__global__ void __launch_bounds__(256)
    fill_kernel(PagedView c, PackedRows K, PackedRows V, const uint16_t *__restrict__ Kc,
                const uint16_t *__restrict__ Vc, const int *__restrict__ cu,
                const int *__restrict__ rows, int S, int64_t total, int64_t m)
{
    extern __shared__ int scu[];  // [S + 1] offsets, [B] the last sequence that names a row
    chain_begin();
    int *last = scu + S + 1;
    if (!load_offsets(cu, S, total, scu)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) report(kStatusSeqlens);
        return;
    }
    for (int b = threadIdx.x; b < c.B; b += blockDim.x) last[b] = -1;
    __syncthreads();
    for (int s = threadIdx.x; s < S; s += blockDim.x) {
        const int b = __ldg(rows + s);
        if (b >= 0 && b < c.B) atomicMax(last + b, s);
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int s = threadIdx.x; s < S; s += blockDim.x) {
            const int b = __ldg(rows + s);
            if (b < 0 || b >= c.B || last[b] != s || c.lens[b] != scu[s + 1] - scu[s])
                report(kStatusPage);
        }
    const int lane = threadIdx.x & 31;
    const int mask = (1 << c.shift) - 1;
    constexpr int CH = D / 8;        // 16-byte chunks of a row
    constexpr int AT = 32 / (2 * CH);  // rows (keys and values) that the warp copies at once
    const int e = lane % CH * 8, is_v = lane / CH % 2, sub = lane / (2 * CH);
    const int64_t raw_units = (total + 31) / 32, core_units = Kc != nullptr ? (m + 31) / 32 : 0;
    for (int64_t x = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
         x < (raw_units + core_units) * c.Hkv;
         x += (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5) {
        const int64_t unit = x / c.Hkv;
        const int h = static_cast<int>(x - unit * c.Hkv);
        const bool core = unit >= raw_units;
        const int64_t row0 = (core ? unit - raw_units : unit) * 32, row = row0 + lane;
        // this lane's row: its place in the pool, -1 if it has none
        int64_t to = -1;
        if (row < (core ? m : total)) {
            const int s = core ? core_row_sequence(scu, S, c.g, static_cast<int>(row))
                               : row_sequence(scu, S, row);
            const int len = scu[s + 1] - scu[s];
            const int64_t pos = row - (core ? scu[s] / c.g : scu[s]);
            const int b = __ldg(rows + s);
            if (pos >= (core ? 0 : window_start(len - 1, c.g, c.w)) && pos >= 0 &&
                pos < (core ? len / c.g : len) && b >= 0 && b < c.B && last[b] == s &&
                __ldg(c.lens + b) == len) {
                const int page = core ? own_page_at(c.core_table, c.core_ref, b, c.core_cols,
                                                    pos >> c.shift, c.core_pages)
                                      : own_page_at(c.raw_table, c.raw_ref, b, c.raw_cols,
                                                    pos >> c.shift, c.raw_pages);
                if (page >= 0)
                    to = page_row<D>(page, h, c.Hkv, c.shift, static_cast<int>(pos) & mask);
                else
                    report(kStatusPage);
            }
        }
        const uint16_t *from;
        int64_t stride;
        if (core) {
            from = (is_v ? Vc : Kc) + (static_cast<int64_t>(h) * m + row0) * D + e;
            stride = D;
        } else {
            const PackedRows &src = is_v ? V : K;
            from = static_cast<const uint16_t *>(src.data) + h * src.head + row0 * src.row + e;
            stride = src.row;
        }
        uint16_t *pool = (core ? (is_v ? c.v_core : c.k_core) : (is_v ? c.v_raw : c.k_raw)) + e;
        if (__ballot_sync(0xffffffffu, to >= 0) == 0) continue;
#pragma unroll 1
        for (int r0 = 0; r0 < 32; r0 += 8 * AT) {
            uint4 y[8];
            int64_t at[8];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const int i = r0 + u * AT + sub;
                at[u] = __shfl_sync(0xffffffffu, to, i);
                if (at[u] >= 0) y[u] = ldg_stream(from + i * stride);
            }
#pragma unroll
            for (int u = 0; u < 8; ++u)
                if (at[u] >= 0) *reinterpret_cast<uint4 *>(pool + at[u]) = y[u];
        }
    }
}

// Fork, step 1, a group of threads per row b: the row's old pages lose a count, the
// parent's shared ones gain one, and the row's new table goes to `tmp`.  A
// partly filled last page changes hands or is copied (flags, per pool).
constexpr int kFlagRow = 4;  // the row changes

struct ForkView {
    TablesView v;
    const int *parent;
    int *tmp[2];          // new tables
    long long *held;      // [B] of the workspace: goes with the row
    long long *old_lens, *old_held;  // [B]
    int *flags;           // [B]: bit p: a copy in pool p; kFlagRow
    int2 *list[2];        // copies (from, to); to = -1: none
    int *counts;          // [2] copies, [2] live
};

__device__ __forceinline__ int parent_of(const ForkView &f, int b)
{
    const int p = f.parent[b];
    return p >= -1 && p < f.v.B ? p : b;
}

// Used columns [lo, hi) of pool i of a row of len tokens, and whether the
// last one is partly filled.
__device__ __forceinline__ void used_cols(const TablesView &v, int i, int64_t len, int &lo, int &hi,
                                          bool &open)
{
    const PagedCols c = paged_cols(len, v.g, v.w, v.shift, v.pool[0].cols > 0);
    const int64_t mask = (int64_t(1) << v.shift) - 1;
    lo = i == 0 ? 0 : c.raw_lo;
    hi = min(i == 0 ? c.core_hi : c.raw_hi, v.pool[i].cols);
    lo = min(lo, hi);
    open = hi > lo && ((i == 0 ? len / v.g : len) & mask) != 0;
}

// me: this thread's number of n in the group; any(x): whether x holds for one
// of them.
template <class Any>
__device__ __forceinline__ void fork_row(const ForkView &f, int b, int me, int n_threads, Any any)
{
    const TablesView &v = f.v;
    const int p = parent_of(f, b);
    if (me == 0) {
        f.old_lens[b] = v.lens[b];
        if (p != f.parent[b]) report(kStatusPage);
    }
    if (p == b) {
        if (me == 0) f.flags[b] = 0;
        return;
    }
    // does this row get its parent's open pages themselves?
    bool earlier = false;
    if (p >= 0) {
        earlier = parent_of(f, p) == p;
        for (int x = me; x < b && !earlier; x += n_threads) earlier = parent_of(f, x) == p;
    }
    const bool copy = any(earlier);
    int flags = kFlagRow;
    for (int i = 0; i < 2; ++i) {
        const Pool &pool = v.pool[i];
        int lo, hi;
        bool open;
        used_cols(v, i, v.lens[b], lo, hi, open);
        const int *old = pool.table + static_cast<int64_t>(b) * pool.cols;
        for (int c = lo + me; c < hi; c += n_threads) {
            const int e = old[c];
            if (e >= 0 && e < pool.pages)
                atomicSub(pool.ref + e, 1);
            else
                report(kStatusPage);
        }
        if (p < 0) continue;
        used_cols(v, i, v.lens[p], lo, hi, open);
        if (open && copy) flags |= 1 << i;
        const int *from = pool.table + static_cast<int64_t>(p) * pool.cols;
        int *to = f.tmp[i] + static_cast<int64_t>(b) * pool.cols;
        for (int c = lo + me; c < hi; c += n_threads) {
            int e = from[c];
            if (e < 0 || e >= pool.pages) {
                report(kStatusPage);
                e = -1;
            } else if (!(open && copy && c == hi - 1)) {
                atomicAdd(pool.ref + e, 1);
            }
            to[c] = e;
        }
    }
    if (me == 0) f.flags[b] = flags;
}

// Fork, step 2, a block per pool: free pages for the copies.
// order: [copies] rows that want a page, in order.
__device__ __forceinline__ void fork_pages(const ForkView &f, int i, int *order)
{
    __shared__ int room[kThreads / 32][2], chunk_room[2][kThreads / 32][1];
    const TablesView &v = f.v;
    const Pool &pool = v.pool[i];
    const int per = (v.B + kThreads - 1) / kThreads;
    const int b0 = min(static_cast<int>(threadIdx.x) * per, v.B), b1 = min(b0 + per, v.B);
    const int bits = free_bits(pool.ref, pool.pages, 0);
    int at[2] = {0, __popc(bits)}, all[2];  // wanted, free in the first chunk
    for (int b = b0; b < b1; ++b) at[0] += f.flags[b] >> i & 1;
    block_scan(at, all, room);
    for (int b = b0, k = at[0]; b < b1; ++b)
        if (f.flags[b] >> i & 1) order[k++] = b;
    const int want = all[0];
    if (threadIdx.x == 0) f.counts[i] = want;
    __syncthreads();
    // the entry of a row's open page
    auto entry = [&](int b) {
        int lo, hi;
        bool open;
        used_cols(v, i, v.lens[parent_of(f, b)], lo, hi, open);
        return f.tmp[i] + static_cast<int64_t>(b) * pool.cols + hi - 1;
    };
    auto use = [&](int k, int page) {
        int *e = entry(order[k]);
        f.list[i][k] = make_int2(*e, *e >= 0 ? page : -1);
        *e = page;
        pool.ref[page] = 1;
    };
    use_free(bits, 0, at[1], want, use);
    int base = all[1];
    for (int chunk = kChunk; chunk < pool.pages && base < want; chunk += kChunk) {
        const int more = free_bits(pool.ref, pool.pages, chunk);
        int x[1] = {__popc(more)}, n[1];
        block_scan(x, n, chunk_room[chunk / kChunk & 1]);
        use_free(more, chunk, base + x[0], want, use);
        base += n[0];
    }
    // rows that got none
    for (int k = base + threadIdx.x; k < want; k += kThreads) {
        const int b = order[k];
        f.list[i][k] = make_int2(-1, -1);
        *entry(b) = -1;
        atomicOr(f.flags + b, 8);
        report(kStatusCapacity);
    }
}

// Beside step 2: the notes of rows that were refused room, as they were.
__device__ __forceinline__ void fork_held(const ForkView &f)
{
    for (int b = threadIdx.x; b < f.v.B; b += blockDim.x) f.old_held[b] = f.held[b];
}

__global__ void __launch_bounds__(256) fork_rows_kernel(ForkView f)
{
    chain_begin();
    fork_row(f, blockIdx.x, threadIdx.x, 256, [](bool x) { return __syncthreads_or(x) != 0; });
}

__global__ void __launch_bounds__(kThreads) fork_pages_kernel(ForkView f)
{
    extern __shared__ int order[];
    chain_begin();
    if (blockIdx.x < 2)
        fork_pages(f, blockIdx.x, order);
    else
        fork_held(f);
}

// Both steps for a small batch, in one cluster: a warp for each row, then a
// block for each pool.  One launch less is 2 us of host time (6.9 instead of
// 9.0 for a fork); on the GPU it gains nothing (8 rows with the copies and a
// reserve: 18.6 us in a graph, 18.7 with blocks of their own; 256 rows: 18.8
// and 15.7), and beyond two rows a warp it loses more (512 rows: 27.7 and 21.1).
constexpr int kForkBlocks = 8, kForkRows = 2 * kForkBlocks * kThreads / 32;

__global__ void __cluster_dims__(kForkBlocks, 1, 1) __launch_bounds__(kThreads)
    fork_plan_kernel(ForkView f)
{
    extern __shared__ int order[];
    chain_begin();
    cg::cluster_group cluster = cg::this_cluster();
    const int lane = threadIdx.x & 31;
    for (int b = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); b < f.v.B;
         b += kForkBlocks * kThreads / 32)
        fork_row(f, b, lane, 32, [](bool x) { return __any_sync(0xffffffffu, x) != 0; });
    cluster.sync();
    if (blockIdx.x < 2)
        fork_pages(f, blockIdx.x, order);
    else if (blockIdx.x == 2)
        fork_held(f);
}

// Copy whole pages of one pool, all layers: list of (from, to).
struct PoolData {
    uint4 *k, *v;
    int64_t page16, layer16;  // 16-byte units of a page and of a layer
};

__device__ __forceinline__ void copy_pages(const int2 *list, int n, int layers, const PoolData &d)
{
    constexpr int PIECE = 1024;  // 16-byte units a block copies at once
    const int64_t pieces = (d.page16 + PIECE - 1) / PIECE;
    const int64_t work = static_cast<int64_t>(n) * layers * 2 * pieces;
    for (int64_t x = blockIdx.x; x < work; x += gridDim.x) {
        const int64_t piece = x % pieces, y = x / pieces;
        const int kv = static_cast<int>(y & 1);
        const int64_t z = y >> 1;
        const int2 ft = list[z / layers];
        if (ft.y < 0) continue;
        uint4 *base = (kv ? d.v : d.k) + (z % layers) * d.layer16;
        const uint4 *from = base + ft.x * d.page16 + piece * PIECE;
        uint4 *to = base + ft.y * d.page16 + piece * PIECE;
        const int len = static_cast<int>(min(static_cast<int64_t>(PIECE), d.page16 - piece * PIECE));
        uint4 buf[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (threadIdx.x + u * 256 < len) buf[u] = from[threadIdx.x + u * 256];
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (threadIdx.x + u * 256 < len) to[threadIdx.x + u * 256] = buf[u];
    }
}

// Fork, step 3: the new tables and lengths, and the copies.
__global__ void __launch_bounds__(256)
    fork_apply_kernel(ForkView f, PoolData core, PoolData raw, int layers)
{
    chain_begin();
    const TablesView &v = f.v;
    for (int b = blockIdx.x; b < v.B; b += gridDim.x) {
        const int flags = f.flags[b];
        if (!(flags & kFlagRow)) continue;
        const int p = parent_of(f, b);
        const bool none = p < 0 || (flags & 8);
        const int64_t len = none ? 0 : f.old_lens[p];
        for (int i = 0; i < 2; ++i) {
            const Pool &pool = v.pool[i];
            int lo, hi, nlo = 0, nhi = 0, tlo = 0, thi = 0;
            bool open;
            used_cols(v, i, f.old_lens[b], lo, hi, open);
            if (p >= 0) used_cols(v, i, f.old_lens[p], tlo, thi, open);
            if (!none) {
                nlo = tlo;
                nhi = thi;
            }
            int *table = pool.table + static_cast<int64_t>(b) * pool.cols;
            const int *tmp = f.tmp[i] + static_cast<int64_t>(b) * pool.cols;
            for (int c = lo + threadIdx.x; c < hi; c += blockDim.x)
                if (c < nlo || c >= nhi) table[c] = -1;
            for (int c = nlo + threadIdx.x; c < nhi; c += blockDim.x) table[c] = tmp[c];
            if (none)  // a row without room gives back what it was given
                for (int c = tlo + threadIdx.x; c < thi; c += blockDim.x)
                    if (tmp[c] >= 0) atomicSub(pool.ref + tmp[c], 1);
        }
        if (threadIdx.x == 0) v.lens[b] = len;
    }
    copy_pages(f.list[0], f.counts[0], layers, core);
    copy_pages(f.list[1], f.counts[1], layers, raw);
    // the notes, by the blocks that have no row and the fewest pages (by the
    // rows' own: 0.5 us for 8 rows)
    if (threadIdx.x == 0)
        for (int b = gridDim.x - 1 - blockIdx.x; b < v.B; b += gridDim.x) {
            const int flags = f.flags[b], p = parent_of(f, b);
            if (flags & kFlagRow) f.held[b] = p < 0 || (flags & 8) ? 0 : f.old_held[p];
        }
}

// Compact, step 1, a block per pool: the k-th page in use at or above the
// number of pages in use moves to the k-th free page below it.  (Before page
// p lie p - f pages in use, f the free ones before it.)
__global__ void __launch_bounds__(kThreads)
    compact_plan_kernel(TablesView v, int2 *list0, int2 *list1, int *remap0, int *remap1,
                        int *counts, long long *live_out)
{
    __shared__ int room[kThreads / 32][2], chunk_room[2][kThreads / 32][1], moved_s;
    chain_begin();
    const int i = blockIdx.x;
    const Pool &pool = v.pool[i];
    int2 *list = i == 0 ? list0 : list1;
    int *remap = i == 0 ? remap0 : remap1;
    int bits = free_bits(pool.ref, pool.pages, 0);
    int at[2] = {__popc(bits), 0}, all[2];  // free in the first chunk, behind it
    for (int chunk = kChunk; chunk < pool.pages; chunk += kChunk)
        at[1] += __popc(free_bits(pool.ref, pool.pages, chunk));
    if (threadIdx.x == 0) moved_s = 0;  // free pages before `live`: pages that move
    block_scan(at, all, room);
    const int live = pool.pages - all[0] - all[1];
    int k = at[0], base = all[0];
    for (int chunk = 0; chunk < pool.pages; chunk += kChunk) {
        if (chunk > 0) {
            bits = free_bits(pool.ref, pool.pages, chunk);
            int x[1] = {__popc(bits)}, n[1];
            block_scan(x, n, chunk_room[chunk / kChunk & 1]);
            k = base + x[0];
            base += n[0];
        }
        const int p0 = chunk + threadIdx.x * 4;
        if (live < pool.pages && live >= p0 && live < p0 + 4)
            moved_s = k + __popc(bits & ((1 << (live - p0)) - 1));
        __syncthreads();
        for (int u = 0; u < 4 && p0 + u < pool.pages; ++u) {
            const int p = p0 + u;
            if (bits >> u & 1) {
                if (p < live) list[k].y = p;
                ++k;
            } else if (p >= live) {
                list[p - k - (live - moved_s)].x = p;
            }
        }
    }
    __syncthreads();
    const int moved = moved_s;
    for (int j = threadIdx.x; j < moved; j += kThreads) {
        const int2 ft = list[j];
        remap[ft.x] = ft.y;
        pool.ref[ft.y] = pool.ref[ft.x];
        pool.ref[ft.x] = 0;
    }
    if (threadIdx.x == 0) {
        counts[i] = moved;
        counts[2 + i] = live;
        live_out[i] = live;
    }
}

// Compact, step 2: the tables and the pages.
__global__ void __launch_bounds__(256)
    compact_apply_kernel(TablesView v, const int2 *list0, const int2 *list1, const int *remap0,
                         const int *remap1, const int *counts, PoolData core, PoolData raw,
                         int layers)
{
    chain_begin();
    for (int b = blockIdx.x; b < v.B; b += gridDim.x)
        for (int i = 0; i < 2; ++i) {
            const Pool &pool = v.pool[i];
            const int live = counts[2 + i];
            const int *remap = i == 0 ? remap0 : remap1;
            int lo, hi;
            bool open;
            used_cols(v, i, v.lens[b], lo, hi, open);
            int *table = pool.table + static_cast<int64_t>(b) * pool.cols;
            for (int c = lo + threadIdx.x; c < hi; c += blockDim.x) {
                const int e = table[c];
                if (e < 0 || e >= pool.pages)
                    report(kStatusPage);
                else if (e >= live)
                    table[c] = remap[e];
            }
        }
    copy_pages(list0, counts[0], layers, core);
    copy_pages(list1, counts[1], layers, raw);
}

TablesView tables_view(const cca_paged_cache &c)
{
    TablesView v;
    v.pool[0] = {c.core_table, c.core_ref, c.core_cols, c.core_pages};
    v.pool[1] = {c.raw_table, c.raw_ref, c.raw_cols, c.raw_pages};
    v.lens = c.lens;
    v.B = c.B;
    v.g = c.g;
    v.w = c.w;
    v.shift = __builtin_ctz(c.page);
    return v;
}

PoolData pool_data(const cca_paged_cache &c, bool core)
{
    PoolData d;
    d.k = static_cast<uint4 *>(core ? c.k_core : c.k_raw);
    d.v = static_cast<uint4 *>(core ? c.v_core : c.v_raw);
    d.page16 = static_cast<int64_t>(c.Hkv) * c.page * c.d / 8;
    d.layer16 = d.page16 * (core ? c.core_pages : c.raw_pages);
    return d;
}

int copy_grid()
{
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms * 8;
}

}  // namespace

PagedWorkspace paged_workspace(const cca_paged_cache &c)
{
    PagedWorkspace w;
    size_t at = 0;
    auto part = [&](size_t bytes) {
        const size_t here = at;
        at += (bytes + 255) / 256 * 256;
        return here;
    };
    w.tickets = part(sizeof(unsigned int) * c.B * c.Hkv);
    w.part = part(paged_decode_part_bytes(c));
    w.held = part(sizeof(long long) * c.B);
    w.lens = part(sizeof(long long) * c.B);
    w.old_held = part(sizeof(long long) * c.B);
    w.flags = part(sizeof(int) * c.B);
    w.core_tmp = part(sizeof(int) * static_cast<size_t>(c.B) * c.core_cols);
    w.raw_tmp = part(sizeof(int) * static_cast<size_t>(c.B) * c.raw_cols);
    // page moves: (from, to) of each pool, then the new number of each page
    w.lists = part((sizeof(int2) + sizeof(int)) * (static_cast<size_t>(c.core_pages) + c.raw_pages) +
                   2 * sizeof(int2) * c.B);
    w.counts = part(4 * sizeof(int));
    w.total = at;
    return w;
}

cudaError_t launch_paged_reserve(const cca_paged_cache &c, const long long *n_new, long long n,
                                 void *workspace, cudaStream_t s)
{
    long long *held = nullptr;
    if (workspace != nullptr)
        held = reinterpret_cast<long long *>(static_cast<char *>(workspace) +
                                             paged_workspace(c).held);
    return launch_chained(reserve_kernel, 2, kThreads, sizeof(int) * 2 * c.B, s, tables_view(c),
                          n_new, n, held);
}

cudaError_t launch_paged_fill(const cca_paged_cache &c, int layer, const PackedRows &K,
                              const PackedRows &V, const void *Kc, const void *Vc, const int *cu,
                              const int *rows, int S, int64_t total, cudaStream_t s)
{
    const PagedView v = paged_view(c, layer);
    if (c.core_cols == 0) Kc = Vc = nullptr;
    const int64_t m = total / c.g;
    const int64_t warps = ((total + 31) / 32 + (Kc != nullptr ? (m + 31) / 32 : 0)) * c.Hkv;
    const int64_t want = (warps + 7) / 8;
    const int most = copy_grid();
    const int grid = static_cast<int>(want < most ? want : most);
    const size_t smem = sizeof(int) * (S + 1 + c.B);
    cudaError_t e = cudaSuccess;
    auto go = [&](auto kern) {
        if ((e = allow_smem(kern, smem)) != cudaSuccess) return;
        e = launch_chained(kern, grid, 256, smem, s, v, K, V, static_cast<const uint16_t *>(Kc),
                           static_cast<const uint16_t *>(Vc), cu, rows, S, total, m);
    };
    if (c.d == 128)
        go(fill_kernel<128>);
    else
        go(fill_kernel<64>);
    return e;
}

cudaError_t launch_paged_fork(const cca_paged_cache &c, const int *parent, void *workspace,
                              cudaStream_t s)
{
    const PagedWorkspace w = paged_workspace(c);
    char *base = static_cast<char *>(workspace);
    ForkView f;
    f.v = tables_view(c);
    f.parent = parent;
    f.tmp[0] = reinterpret_cast<int *>(base + w.core_tmp);
    f.tmp[1] = reinterpret_cast<int *>(base + w.raw_tmp);
    f.held = reinterpret_cast<long long *>(base + w.held);
    f.old_lens = reinterpret_cast<long long *>(base + w.lens);
    f.old_held = reinterpret_cast<long long *>(base + w.old_held);
    f.flags = reinterpret_cast<int *>(base + w.flags);
    f.list[0] = reinterpret_cast<int2 *>(base + w.lists);
    f.list[1] = f.list[0] + c.B;
    f.counts = reinterpret_cast<int *>(base + w.counts);
    cudaError_t e;
    if (c.B <= kForkRows) {
        e = launch_chained(fork_plan_kernel, kForkBlocks, kThreads, sizeof(int) * c.B, s, f);
    } else {
        e = launch_chained(fork_rows_kernel, c.B, 256, 0, s, f);
        if (e == cudaSuccess)
            e = launch_chained(fork_pages_kernel, 3, kThreads, sizeof(int) * c.B, s, f);
    }
    if (e == cudaSuccess)
        e = launch_chained(fork_apply_kernel, copy_grid(), 256, 0, s, f, pool_data(c, true),
                           pool_data(c, false), c.layers);
    return e;
}

cudaError_t launch_paged_compact(const cca_paged_cache &c, long long *live, void *workspace,
                                 cudaStream_t s)
{
    const PagedWorkspace w = paged_workspace(c);
    char *base = static_cast<char *>(workspace);
    const TablesView v = tables_view(c);
    int2 *list0 = reinterpret_cast<int2 *>(base + w.lists), *list1 = list0 + c.core_pages;
    int *remap0 = reinterpret_cast<int *>(list1 + c.raw_pages), *remap1 = remap0 + c.core_pages;
    int *counts = reinterpret_cast<int *>(base + w.counts);
    const cudaError_t e = launch_chained(compact_plan_kernel, 2, kThreads, 0, s, v, list0, list1,
                                         remap0, remap1, counts, live);
    if (e != cudaSuccess) return e;
    return launch_chained(compact_apply_kernel, copy_grid(), 256, 0, s, v, list0, list1, remap0,
                          remap1, counts, pool_data(c, true), pool_data(c, false), c.layers);
}

cudaError_t paged_tables_status_read_clear(unsigned int *v)
{
    unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(v, g_paged_tables_status, sizeof(*v));
    if (e == cudaSuccess && *v) e = cudaMemcpyToSymbol(g_paged_tables_status, &zero, sizeof(zero));
    return e;
}

}  // namespace cca
