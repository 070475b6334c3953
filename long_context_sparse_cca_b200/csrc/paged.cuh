// The paged decode cache (cca_paged_cache of the C ABI) on the device.
#pragma once

#include <cca.h>

#include "common.cuh"

namespace cca {

// One layer of a paged cache, as the kernels read it.
struct PagedView {
    uint16_t *k_core, *v_core, *k_raw, *v_raw;  // the layer's pools
    const int *core_table, *raw_table, *core_ref, *raw_ref;
    const long long *lens;
    const long long *held;  // [B] (cca_paged_step): a row of this many tokens is held
    int B, Hq, Hkv, g, w;
    int shift;  // log2(page)
    int core_cols, raw_cols, core_pages, raw_pages;
    int64_t longest;  // longest row the tables take
};

// Page-table columns of a row of L tokens: raw [raw_lo, raw_hi), core
// [0, core_hi).
struct PagedCols {
    int raw_lo, raw_hi, core_hi;
};

__host__ __device__ __forceinline__ PagedCols paged_cols(int64_t len, int g, int w, int shift,
                                                         bool core)
{
    PagedCols c;
    const int64_t up = (int64_t(1) << shift) - 1;
    // (no table has 2^30 columns of 16 rows and more; a length that says so
    // is cut, so that column numbers stay within 32 bits)
    len = len < 0 ? 0 : (len > (int64_t(1) << 33) ? int64_t(1) << 33 : len);
    c.raw_lo = len > 0 ? static_cast<int>(window_start(len - 1, g, w) >> shift) : 0;
    c.raw_hi = static_cast<int>((len + up) >> shift);
    c.core_hi = core ? static_cast<int>((len / g + up) >> shift) : 0;
    return c;
}

// Longest row the tables take.
__host__ __device__ __forceinline__ int64_t paged_max_len(int raw_cols, int core_cols, int g,
                                                          int shift)
{
    const int64_t raw = static_cast<int64_t>(raw_cols) << shift;
    if (core_cols == 0) return raw;
    const int64_t core = (static_cast<int64_t>(core_cols) << shift) * g + g - 1;
    return raw < core ? raw : core;
}

__device__ __forceinline__ int page_at(const int *table, int64_t b, int cols, int64_t col,
                                       int pages)
{
    if (col < 0 || col >= cols) return -1;
    const int p = __ldg(table + b * cols + col);
    return p >= 0 && p < pages ? p : -1;
}

// The page of a column that a row may write: its own alone (count 1).
__device__ __forceinline__ int own_page_at(const int *table, const int *ref, int64_t b, int cols,
                                           int64_t col, int pages)
{
    const int p = page_at(table, b, cols, col, pages);
    return p >= 0 && __ldg(ref + p) == 1 ? p : -1;
}

// Element offset of row `slot` of head h in a page.
template <int D>
__device__ __forceinline__ int64_t page_row(int page, int h, int Hkv, int shift, int slot)
{
    return ((((static_cast<int64_t>(page) * Hkv + h) << shift) + slot)) * D;
}

inline PagedView paged_view(const cca_paged_cache &c, int layer)
{
    const int64_t page = static_cast<int64_t>(c.Hkv) * c.page * c.d;
    const int64_t core = layer * page * c.core_pages, raw = layer * page * c.raw_pages;
    return {static_cast<uint16_t *>(c.k_core) + core, static_cast<uint16_t *>(c.v_core) + core,
            static_cast<uint16_t *>(c.k_raw) + raw, static_cast<uint16_t *>(c.v_raw) + raw,
            c.core_table, c.raw_table, c.core_ref, c.raw_ref, c.lens, nullptr, c.B, c.Hq, c.Hkv, c.g, c.w,
            __builtin_ctz(c.page), c.core_cols, c.raw_cols, c.core_pages, c.raw_pages,
            paged_max_len(c.raw_cols, c.core_cols, c.g, __builtin_ctz(c.page))};
}

}  // namespace cca
