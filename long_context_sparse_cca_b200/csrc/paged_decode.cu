// cca_attn_decode_paged, cca_paged_step: attention of every row's newest
// token over a paged cache (core rows of the groups before its window, raw
// rows of the window; one softmax, sections 局部保留模块 and
// 全局-局部模块可微融合 of the CCA write-up), and with it the append of that
// token.
#include "paged.cuh"
#include "paged.h"
#include "pool_warp.cuh"

namespace cca {

__device__ unsigned int g_paged_decode_status;  // kStatusCapacity, kStatusPage, kStatusRange

namespace {

constexpr int kWarps = 4;

// One block per (key/value head, row); its warps share the keys out, each
// with a softmax of its own, and join at the end.
template <int D, int R, bool STEP>
__global__ void __launch_bounds__(kWarps * 32)
    paged_decode_kernel(PagedView c, const uint16_t *__restrict__ q_t,
                        const uint16_t *__restrict__ k_t, const uint16_t *__restrict__ v_t,
                        void *__restrict__ o_t, int o_f32, float scale_log2)
{
    constexpr int DPL = D / 32;
    using V = RowVec<D>;
    using VT = typename V::T;
    extern __shared__ float smem[];  // [kWarps][R][D + 2]; then the pooling's scratch
    const int h = blockIdx.x, b = blockIdx.y, r = c.Hq / c.Hkv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t len = c.lens[b];
    // (a row longer than its table is taken as free, and reported)
    const PagedRow row = paged_row(len <= c.longest ? len : 0, c.g, c.w);
    if (len > c.longest && threadIdx.x == 0) atomicOr(&g_paged_decode_status, kStatusCapacity);
    const int64_t bh = static_cast<int64_t>(b) * c.Hkv + h;
    float q[R][DPL], o[R][DPL], m[R], l[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
        m[k] = -INFINITY;
        l[k] = 0.f;
#pragma unroll
        for (int e = 0; e < DPL; ++e) o[k][e] = q[k][e] = 0.f;
        if (k < r) V::to_f32(reinterpret_cast<const VT *>(
                                 q_t + (static_cast<int64_t>(b) * c.Hq + h * r + k) * D)[lane], q[k]);
    }
    bool bad = false;
    const int64_t n = row.t < 0 ? 0 : row.n_core + (row.t - row.ws + 1);
    const int mask = (1 << c.shift) - 1;
    for (int64_t i = warp; i < n; i += kWarps) {
        const bool core = i < row.n_core;
        const int64_t pos = core ? i : row.ws + (i - row.n_core);
        const uint16_t *kr, *vr;
        if (STEP && !core && pos == row.t) {
            kr = k_t + bh * D;
            vr = v_t + bh * D;
        } else {
            const int page = core ? page_at(c.core_table, b, c.core_cols, pos >> c.shift, c.core_pages)
                                  : page_at(c.raw_table, b, c.raw_cols, pos >> c.shift, c.raw_pages);
            if (page < 0) {
                bad = true;
                continue;
            }
            const int64_t at = page_row<D>(page, h, c.Hkv, c.shift, static_cast<int>(pos) & mask);
            kr = (core ? c.k_core : c.k_raw) + at;
            vr = (core ? c.v_core : c.v_raw) + at;
        }
        float kf[DPL], vf[DPL];
#pragma unroll
        for (int e = 0; e < DPL; ++e) {
            const uint16_t kb = kr[lane * DPL + e], vb = vr[lane * DPL + e];
            kf[e] = core ? f16_lo(kb) : bf16_lo(kb);
            vf[e] = core ? f16_lo(vb) : bf16_lo(vb);
        }
#pragma unroll
        for (int k = 0; k < R; ++k) {
            if (k >= r) continue;
            float x = 0.f;
#pragma unroll
            for (int e = 0; e < DPL; ++e) x = fmaf(q[k][e], kf[e], x);
            x = warp_sum(x) * scale_log2;
            const float mn = fmaxf(m[k], x);
            const float a = exp2f(m[k] - mn), p = exp2f(x - mn);
            m[k] = mn;
            l[k] = fmaf(l[k], a, p);
#pragma unroll
            for (int e = 0; e < DPL; ++e) o[k][e] = fmaf(o[k][e], a, p * vf[e]);
        }
    }
    if (bad && lane == 0) atomicOr(&g_paged_decode_status, kStatusPage);
#pragma unroll
    for (int k = 0; k < R; ++k) {
        float *s = smem + (warp * R + k) * (D + 2);
        if (lane == 0) {
            s[D] = m[k];
            s[D + 1] = l[k];
        }
#pragma unroll
        for (int e = 0; e < DPL; ++e) s[lane * DPL + e] = o[k][e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < r * D; i += kWarps * 32) {
        const int k = i / D, e = i - k * D;
        float mx = -INFINITY, sum = 0.f, acc = 0.f;
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, smem[(w * R + k) * (D + 2) + D]);
        for (int w = 0; w < kWarps; ++w) {
            const float *s = smem + (w * R + k) * (D + 2);
            const float f = s[D] == -INFINITY ? 0.f : exp2f(s[D] - mx);
            sum = fmaf(f, s[D + 1], sum);
            acc = fmaf(f, s[e], acc);
        }
        const float y = sum > 0.f ? acc / sum : 0.f;
        const int64_t at = (static_cast<int64_t>(b) * c.Hq + h * r) * D + i;
        if (o_f32)
            static_cast<float *>(o_t)[at] = y;
        else
            static_cast<uint16_t *>(o_t)[at] = bf16_bits(y);
    }
    if (!STEP || row.t < 0 || warp != 0) return;
    // the append: token t's rows to its page, and the group it completes
    const int page =
        own_page_at(c.raw_table, c.raw_ref, b, c.raw_cols, row.t >> c.shift, c.raw_pages);
    if (page < 0) {
        if (lane == 0) atomicOr(&g_paged_decode_status, kStatusPage);
        return;
    }
    const int64_t at = page_row<D>(page, h, c.Hkv, c.shift, static_cast<int>(row.t) & mask);
    reinterpret_cast<VT *>(c.k_raw + at)[lane] = reinterpret_cast<const VT *>(k_t + bh * D)[lane];
    reinterpret_cast<VT *>(c.v_raw + at)[lane] = reinterpret_cast<const VT *>(v_t + bh * D)[lane];
    if (c.core_cols == 0 || (row.t + 1) % c.g != 0) return;
    const int64_t first = row.t - c.g + 1, j = row.t / c.g;
    int out = own_page_at(c.core_table, c.core_ref, b, c.core_cols, j >> c.shift, c.core_pages);
    for (int i = lane; i < c.g; i += 32)
        if (page_at(c.raw_table, b, c.raw_cols, (first + i) >> c.shift, c.raw_pages) < 0) out = -1;
    if (__any_sync(0xffffffffu, out < 0)) {
        if (lane == 0) atomicOr(&g_paged_decode_status, kStatusPage);
        return;
    }
    auto old = [&](const uint16_t *pool, const uint16_t *in, int i) {
        if (i == c.g - 1) return in + bh * D;
        const int64_t pos = first + i;
        const int pg = page_at(c.raw_table, b, c.raw_cols, pos >> c.shift, c.raw_pages);
        return pool + page_row<D>(pg, h, c.Hkv, c.shift, static_cast<int>(pos) & mask);
    };
    const int64_t to = page_row<D>(out, h, c.Hkv, c.shift, static_cast<int>(j) & mask);
    const bool over = pool_group_warp<D>(
        [&](int i) { return old(c.k_raw, k_t, i); }, [&](int i) { return old(c.v_raw, v_t, i); },
        [&](int k) { return q_t + (static_cast<int64_t>(b) * c.Hq + h * r + k) * D; }, r, c.g,
        scale_log2, smem + kWarps * R * (D + 2), c.k_core + to, c.v_core + to);
    if (over && lane == 0) atomicOr(&g_paged_decode_status, kStatusRange);
}

}  // namespace

cudaError_t launch_paged_decode(const cca_paged_cache &c, int layer, const void *q_t,
                                const void *k_t, const void *v_t, void *o_t, bool o_f32,
                                void *workspace, cudaStream_t s)
{
    (void)workspace;
    const int r = c.Hq / c.Hkv;
    const PagedView v = paged_view(c, layer);
    const float scale_log2 = kLog2e / sqrtf(static_cast<float>(c.d));
    cudaError_t e = cudaSuccess;
    auto go = [&](auto kern, int R) {
        const size_t smem = sizeof(float) * (kWarps * R * (c.d + 2) + (r + 1) * c.g);
        if (smem > 48 * 1024)
            e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     static_cast<int>(smem));
        if (e != cudaSuccess) return;
        kern<<<dim3(c.Hkv, c.B), kWarps * 32, smem, s>>>(
            v, static_cast<const uint16_t *>(q_t), static_cast<const uint16_t *>(k_t),
            static_cast<const uint16_t *>(v_t), o_t, o_f32 ? 1 : 0, scale_log2);
        e = cudaGetLastError();
    };
#define CCA_PAGED(DD, RR)                                    \
    if (k_t != nullptr) go(paged_decode_kernel<DD, RR, true>, RR); \
    else go(paged_decode_kernel<DD, RR, false>, RR)
    if (c.d == 128) {
        if (r == 1) { CCA_PAGED(128, 1); }
        else if (r <= 4) { CCA_PAGED(128, 4); }
        else { CCA_PAGED(128, 16); }
    } else {
        if (r == 1) { CCA_PAGED(64, 1); }
        else if (r <= 4) { CCA_PAGED(64, 4); }
        else { CCA_PAGED(64, 16); }
    }
#undef CCA_PAGED
    return e;
}

cudaError_t paged_decode_status_read_clear(unsigned int *v)
{
    unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(v, g_paged_decode_status, sizeof(*v));
    if (e == cudaSuccess && *v) e = cudaMemcpyToSymbol(g_paged_decode_status, &zero, sizeof(zero));
    return e;
}

}  // namespace cca
