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

constexpr int kScanThreads = 1024;

struct Pool {  // one of the two pools' tables
    int *table, *ref;
    int cols, pages;
};

struct TablesView {
    Pool pool[2];  // core, raw
    long long *lens;
    int B, g, w, shift;
};

__device__ __forceinline__ void report(unsigned int bits) { atomicOr(&g_paged_tables_status, bits); }

// Exclusive sum over the block of each thread's x (kScanThreads threads);
// `total`: the sum of all.  Called by every thread, any number of times.
__device__ __forceinline__ int block_scan(int x, int &total)
{
    __shared__ int warp_sums[kScanThreads / 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int y = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y += z;
    }
    if (lane == 31) warp_sums[warp] = y;
    __syncthreads();
    if (warp == 0) {
        int v = warp_sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int z = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v += z;
        }
        warp_sums[lane] = v;
    }
    __syncthreads();
    const int before = warp > 0 ? warp_sums[warp - 1] : 0;
    total = warp_sums[kScanThreads / 32 - 1];
    __syncthreads();
    return before + y - x;
}

// Free pages of a pool, by the whole block.
__device__ __forceinline__ int count_free(const int *ref, int pages)
{
    int n = 0;
    for (int p = threadIdx.x; p < pages; p += kScanThreads) n += __ldcg(ref + p) == 0;
    int total;
    block_scan(n, total);
    return total;
}

// use(k, page) for the k-th free page, k < want, by the whole block.
template <class F>
__device__ __forceinline__ void take_free(const int *ref, int pages, int want, F use)
{
    for (int p0 = 0, base = 0; p0 < pages && base < want; p0 += kScanThreads) {
        const int p = p0 + threadIdx.x;
        const bool free = p < pages && __ldcg(ref + p) == 0;
        int total;
        const int k = base + block_scan(free ? 1 : 0, total);
        if (free && k < want) use(k, p);
        base += total;
    }
}

// cca_paged_reserve: a cluster of two blocks, one for each pool; both plan
// all rows, then each takes its own pool's pages.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kScanThreads)
    reserve_kernel(TablesView v, const long long *__restrict__ n_new, long long n_all)
{
    extern __shared__ int plan[];  // [B + 1] my pool's pages wanted before row b, [B] granted
    __shared__ int free_pages;
    cg::cluster_group cluster = cg::this_cluster();
    const int me = cluster.block_rank();
    int *before = plan, *granted = plan + v.B + 1;
    const bool core = v.pool[0].cols > 0;
    const int64_t longest = paged_max_len(v.pool[1].cols, v.pool[0].cols, v.g, v.shift);
    auto grow = [&](int b, int64_t &len) -> int64_t {
        len = v.lens[b];
        const int64_t n = n_new != nullptr ? n_new[b] : (len > 0 ? n_all : 0);
        return n > 0 && len >= 0 && n <= longest - len ? n : 0;
    };
    // pages that rows want: my pool's kept, the other's only for the decision
    int want[2] = {0, 0};
    const int per = (v.B + kScanThreads - 1) / kScanThreads;
    const int b0 = threadIdx.x * per, b1 = min(b0 + per, v.B);
    auto need = [&](int b, int (&x)[2]) {
        int64_t len;
        const int64_t n = grow(b, len);
        x[0] = x[1] = 0;
        if (n == 0) return;
        const PagedCols a = paged_cols(len, v.g, v.w, v.shift, core);
        const PagedCols z = paged_cols(len + n, v.g, v.w, v.shift, core);
        x[0] = z.core_hi - a.core_hi;
        x[1] = z.raw_hi - max(a.raw_hi, z.raw_lo);
    };
    for (int b = b0; b < b1; ++b) {
        int x[2];
        need(b, x);
        want[0] += x[0];
        want[1] += x[1];
    }
    int total[2], at[2];
    at[0] = block_scan(want[0], total[0]);
    at[1] = block_scan(want[1], total[1]);
    const int n_free = total[me] > 0 ? count_free(v.pool[me].ref, v.pool[me].pages) : 0;
    if (threadIdx.x == 0) free_pages = n_free;
    cluster.sync();
    const int other = *cluster.map_shared_rank(&free_pages, me ^ 1);
    const int have[2] = {me == 0 ? n_free : other, me == 0 ? other : n_free};
    for (int b = b0; b < b1; ++b) {
        int x[2];
        need(b, x);
        before[b] = at[me];
        const bool ok = (x[0] == 0 || at[0] + x[0] <= have[0]) && (x[1] == 0 || at[1] + x[1] <= have[1]);
        int64_t len;
        const int64_t n = grow(b, len);
        granted[b] = ok && n > 0;
        const int64_t asked = n_new != nullptr ? n_new[b] : (len > 0 ? n_all : 0);
        if (me == 0 && (!ok || (n == 0 && asked != 0))) report(kStatusCapacity);
        at[0] += x[0];
        at[1] += x[1];
    }
    if (threadIdx.x == 0) before[v.B] = total[me];
    cluster.sync();  // both have read lens and each other's count
    const Pool &pool = v.pool[me];
    take_free(pool.ref, pool.pages, total[me], [&](int k, int page) {
        int lo = 0, hi = v.B - 1;  // the row of the k-th wanted page
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (before[mid] <= k)
                lo = mid;
            else
                hi = mid - 1;
        }
        if (!granted[lo]) return;
        int64_t len;
        const int64_t n = grow(lo, len);
        const PagedCols a = paged_cols(len, v.g, v.w, v.shift, core);
        const PagedCols z = paged_cols(len + n, v.g, v.w, v.shift, core);
        const int col = (me == 0 ? a.core_hi : max(a.raw_hi, z.raw_lo)) + (k - before[lo]);
        pool.table[static_cast<int64_t>(lo) * pool.cols + col] = page;
        pool.ref[page] = 1;
    });
    __syncthreads();
    // raw pages before the new window go
    if (me == 1)
        for (int b = b0; b < b1; ++b) {
            if (!granted[b]) continue;
            int64_t len;
            const int64_t n = grow(b, len);
            const PagedCols a = paged_cols(len, v.g, v.w, v.shift, core);
            const PagedCols z = paged_cols(len + n, v.g, v.w, v.shift, core);
            for (int col = a.raw_lo; col < min(a.raw_hi, z.raw_lo); ++col) {
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
            if (granted[b]) {
                int64_t len;
                const int64_t n = grow(b, len);
                v.lens[b] = len + n;
            }
}

// cca_paged_fill: one warp per packed row (raw) or core row, all heads.
template <int D>
__global__ void __launch_bounds__(256)
    fill_kernel(PagedView c, PackedRows K, PackedRows V, const uint16_t *__restrict__ Kc,
                const uint16_t *__restrict__ Vc, const int *__restrict__ cu,
                const int *__restrict__ rows, int S, int64_t total, int64_t m)
{
    extern __shared__ int scu[];  // [S + 1] offsets, [B] the last sequence that names a row
    int *last = scu + S + 1;
    if (!load_offsets(cu, S, total, scu)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) report(kStatusSeqlens);
        return;
    }
    for (int b = threadIdx.x; b < c.B; b += blockDim.x) last[b] = -1;
    __syncthreads();
    for (int s = threadIdx.x; s < S; s += blockDim.x) {
        const int b = rows[s];
        if (b >= 0 && b < c.B) atomicMax(last + b, s);
    }
    __syncthreads();
    if (blockIdx.x == 0)
        for (int s = threadIdx.x; s < S; s += blockDim.x) {
            const int b = rows[s];
            if (b < 0 || b >= c.B || last[b] != s || c.lens[b] != scu[s + 1] - scu[s])
                report(kStatusPage);
        }
    const int lane = threadIdx.x & 31;
    const int mask = (1 << c.shift) - 1;
    constexpr int C = D / 8;  // 16-byte chunks of a row
    const int64_t n = total + (Kc != nullptr ? m : 0);
    for (int64_t i = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5; i < n;
         i += (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 5) {
        const bool core = i >= total;
        const int64_t row = core ? i - total : i;
        const int s = core ? core_row_sequence(scu, S, c.g, static_cast<int>(row))
                           : row_sequence(scu, S, row);
        const int len = scu[s + 1] - scu[s];
        const int64_t pos = row - (core ? scu[s] / c.g : scu[s]);
        if (pos < 0 || pos >= (core ? len / c.g : len)) continue;
        if (!core && pos < window_start(len - 1, c.g, c.w)) continue;
        const int b = rows[s];
        if (b < 0 || b >= c.B || last[b] != s || c.lens[b] != len) continue;
        const int page = core ? own_page_at(c.core_table, c.core_ref, b, c.core_cols,
                                            pos >> c.shift, c.core_pages)
                              : own_page_at(c.raw_table, c.raw_ref, b, c.raw_cols, pos >> c.shift,
                                            c.raw_pages);
        if (page < 0) {
            if (lane == 0) report(kStatusPage);
            continue;
        }
        const int slot = static_cast<int>(pos) & mask;
        for (int x = lane; x < c.Hkv * C; x += 32) {
            const int h = x / C, e = (x - h * C) * 8;
            const int64_t to = page_row<D>(page, h, c.Hkv, c.shift, slot) + e;
            const uint16_t *k, *v;
            if (core) {
                k = Kc + (h * m + row) * D + e;
                v = Vc + (h * m + row) * D + e;
            } else {
                k = static_cast<const uint16_t *>(K.data) + h * K.head + row * K.row + e;
                v = static_cast<const uint16_t *>(V.data) + h * V.head + row * V.row + e;
            }
            *reinterpret_cast<uint4 *>((core ? c.k_core : c.k_raw) + to) =
                *reinterpret_cast<const uint4 *>(k);
            *reinterpret_cast<uint4 *>((core ? c.v_core : c.v_raw) + to) =
                *reinterpret_cast<const uint4 *>(v);
        }
    }
}

// Fork, step 1, a block per row b: the row's old pages lose a count, the
// parent's shared ones gain one, and the row's new table goes to `tmp`.  A
// partly filled last page changes hands or is copied (flags, per pool).
constexpr int kFlagRow = 4;  // the row changes

struct ForkView {
    TablesView v;
    const int *parent;
    int *tmp[2];          // new tables
    long long *old_lens;  // [B]
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

__global__ void __launch_bounds__(256) fork_rows_kernel(ForkView f)
{
    const TablesView &v = f.v;
    const int b = blockIdx.x;
    const int p = parent_of(f, b);
    if (threadIdx.x == 0) {
        f.old_lens[b] = v.lens[b];
        if (p != f.parent[b]) report(kStatusPage);
    }
    if (p == b) {
        if (threadIdx.x == 0) f.flags[b] = 0;
        return;
    }
    // does this row get its parent's open pages themselves?
    bool earlier = false;
    if (p >= 0) {
        earlier = parent_of(f, p) == p;
        for (int x = threadIdx.x; x < b && !earlier; x += blockDim.x) earlier = parent_of(f, x) == p;
    }
    const bool copy = __syncthreads_or(earlier);
    int flags = kFlagRow;
    for (int i = 0; i < 2; ++i) {
        const Pool &pool = v.pool[i];
        int lo, hi;
        bool open;
        used_cols(v, i, v.lens[b], lo, hi, open);
        const int *old = pool.table + static_cast<int64_t>(b) * pool.cols;
        for (int c = lo + threadIdx.x; c < hi; c += blockDim.x) {
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
        for (int c = lo + threadIdx.x; c < hi; c += blockDim.x) {
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
    if (threadIdx.x == 0) f.flags[b] = flags;
}

// Fork, step 2, a block per pool: free pages for the copies.
__global__ void __launch_bounds__(kScanThreads) fork_pages_kernel(ForkView f)
{
    extern __shared__ int order[];  // [copies] rows that want a page, in order
    const TablesView &v = f.v;
    const int i = blockIdx.x;
    const Pool &pool = v.pool[i];
    int want = 0;
    for (int b0 = 0; b0 < v.B; b0 += kScanThreads) {
        const int b = b0 + threadIdx.x;
        const bool mine = b < v.B && (f.flags[b] >> i & 1);
        int total;
        const int k = want + block_scan(mine ? 1 : 0, total);
        if (mine) order[k] = b;
        want += total;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < want; k += kScanThreads) f.list[i][k] = make_int2(-1, -1);
    if (threadIdx.x == 0) f.counts[i] = want;
    __syncthreads();
    take_free(pool.ref, pool.pages, want, [&](int k, int page) {
        const int b = order[k];
        int lo, hi;
        bool open;
        used_cols(v, i, f.v.lens[parent_of(f, b)], lo, hi, open);
        int *e = f.tmp[i] + static_cast<int64_t>(b) * pool.cols + hi - 1;
        if (*e >= 0) f.list[i][k] = make_int2(*e, page);
        *e = page;
        pool.ref[page] = 1;
    });
    // rows that got none
    __syncthreads();
    for (int k = threadIdx.x; k < want; k += kScanThreads)
        if (f.list[i][k].y < 0) {
            const int b = order[k];
            int lo, hi;
            bool open;
            used_cols(v, i, f.v.lens[parent_of(f, b)], lo, hi, open);
            f.tmp[i][static_cast<int64_t>(b) * pool.cols + hi - 1] = -1;
            atomicOr(f.flags + b, 8);
            report(kStatusCapacity);
        }
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
}

// Compact, step 1, a block per pool: the k-th page in use at or above the
// number of pages in use moves to the k-th free page below it.
__global__ void __launch_bounds__(kScanThreads)
    compact_plan_kernel(TablesView v, int2 *list0, int2 *list1, int *remap0, int *remap1,
                        int *counts, long long *live_out)
{
    const int i = blockIdx.x;
    const Pool &pool = v.pool[i];
    int2 *list = i == 0 ? list0 : list1;
    int *remap = i == 0 ? remap0 : remap1;
    const int live = pool.pages - count_free(pool.ref, pool.pages);
    int moved = 0;
    for (int p0 = live; p0 < pool.pages; p0 += kScanThreads) {
        const int p = p0 + threadIdx.x;
        const bool mine = p < pool.pages && pool.ref[p] != 0;
        int total;
        const int k = moved + block_scan(mine ? 1 : 0, total);
        if (mine) list[k].x = p;
        moved += total;
    }
    __syncthreads();
    take_free(pool.ref, live, moved, [&](int k, int page) { list[k].y = page; });
    __syncthreads();
    for (int k = threadIdx.x; k < moved; k += kScanThreads) {
        const int2 ft = list[k];
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
    w.lens = part(sizeof(long long) * c.B);
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
                                 cudaStream_t s)
{
    const size_t smem = sizeof(int) * (2 * c.B + 1);
    reserve_kernel<<<2, kScanThreads, smem, s>>>(tables_view(c), n_new, n);
    return cudaGetLastError();
}

cudaError_t launch_paged_fill(const cca_paged_cache &c, int layer, const PackedRows &K,
                              const PackedRows &V, const void *Kc, const void *Vc, const int *cu,
                              const int *rows, int S, int64_t total, cudaStream_t s)
{
    const PagedView v = paged_view(c, layer);
    if (c.core_cols == 0) Kc = Vc = nullptr;
    const int64_t m = total / c.g, warps = total + m;
    const int64_t want = (warps + 7) / 8;
    const int most = copy_grid();
    const int grid = static_cast<int>(want < most ? want : most);
    const size_t smem = sizeof(int) * (S + 1 + c.B);
    cudaError_t e = cudaSuccess;
    auto go = [&](auto kern) {
        if (smem > 48 * 1024)
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(smem));
        if (e != cudaSuccess) return;
        kern<<<grid, 256, smem, s>>>(v, K, V, static_cast<const uint16_t *>(Kc),
                                     static_cast<const uint16_t *>(Vc), cu, rows, S, total, m);
        e = cudaGetLastError();
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
    f.old_lens = reinterpret_cast<long long *>(base + w.lens);
    f.flags = reinterpret_cast<int *>(base + w.flags);
    f.list[0] = reinterpret_cast<int2 *>(base + w.lists);
    f.list[1] = f.list[0] + c.B;
    f.counts = reinterpret_cast<int *>(base + w.counts);
    fork_rows_kernel<<<c.B, 256, 0, s>>>(f);
    fork_pages_kernel<<<2, kScanThreads, sizeof(int) * c.B, s>>>(f);
    fork_apply_kernel<<<copy_grid(), 256, 0, s>>>(f, pool_data(c, true), pool_data(c, false),
                                                  c.layers);
    return cudaGetLastError();
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
    compact_plan_kernel<<<2, kScanThreads, 0, s>>>(v, list0, list1, remap0, remap1, counts, live);
    compact_apply_kernel<<<copy_grid(), 256, 0, s>>>(v, list0, list1, remap0, remap1, counts,
                                                     pool_data(c, true), pool_data(c, false),
                                                     c.layers);
    return cudaGetLastError();
}

cudaError_t paged_tables_status_read_clear(unsigned int *v)
{
    unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(v, g_paged_tables_status, sizeof(*v));
    if (e == cudaSuccess && *v) e = cudaMemcpyToSymbol(g_paged_tables_status, &zero, sizeof(zero));
    return e;
}

}  // namespace cca
