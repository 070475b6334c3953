// The C ABI of libcca (include/cca.h): argument checks on the host, then
// the kernel launches.  A call that fails a check returns its status before
// touching the GPU.
#include "../../include/cca.h"
#include "common.cuh"
#include "internal.h"
#include "paged.h"

#include <cstdint>

namespace {

constexpr int64_t kMaxT = (int64_t(1) << 31) - 256;  // 32-bit row indices

bool aligned16(const void *p)
{
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0;
}

bool ptr_ok(const void *p, bool needed)
{
    return !needed || (p != nullptr && aligned16(p));
}

bool overlap(const void *a, size_t na, const void *b, size_t nb)
{
    if (!a || !b || na == 0 || nb == 0) return false;
    const auto x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

cca_status shape_status(int B, int Hq, int Hkv, int64_t T, int d, int g, int w)
{
    if (B < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0 || T < 0 || g < 1 || w < 0)
        return CCA_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return CCA_ERR_UNSUPPORTED;
    if (g > CCA_MAX_G || T > kMaxT || w > (1 << 30)) return CCA_ERR_UNSUPPORTED;
    // pooling scratch: 8 warps x (r*g + g) floats of shared memory
    const int64_t r = Hq / Hkv;
    if ((r + 1) * g > 7000) return CCA_ERR_UNSUPPORTED;
    return CCA_OK;
}

// A packed tensor of `heads` x `total` rows of d elements: strides of the
// extents above 1 as the header asks for (`unit`: elements per aligned
// chunk; align: of the data), the others set to what a contiguous tensor
// would have.  distinct: no two rows overlap.
bool rows_ok(const cca_rows *x, int heads, int64_t total, int d, int unit, uintptr_t align,
             bool distinct, cca::PackedRows &out)
{
    if (!x || !x->data || (reinterpret_cast<uintptr_t>(x->data) & (align - 1)) != 0) return false;
    out.data = x->data;
    out.row = total > 1 ? x->row : d;
    out.head = heads > 1 ? x->head : out.row * total;
    constexpr int64_t most = int64_t(1) << 39;  // strides of a tensor map: below 2^40 bytes
    if (out.row < d || out.row % unit != 0 || out.row >= most) return false;
    if (out.head < d || out.head % unit != 0 || (heads > 1 && out.head >= most)) return false;
    if (!distinct || heads == 1 || total == 1) return true;
    return out.head >= (total - 1) * out.row + d || out.row >= (heads - 1) * out.head + d;
}

size_t rows_bytes(const cca::PackedRows &x, int heads, int64_t total, int d, size_t esz)
{
    return ((heads - 1) * static_cast<size_t>(heads > 1 ? x.head : 0) +
            (total - 1) * static_cast<size_t>(x.row) + d) * esz;
}

cca_status packed_status(int S, int Hq, int Hkv, int64_t total, int d, int g, int w,
                         const int32_t *cu)
{
    const cca_status s = shape_status(1, Hq, Hkv, total, d, g, w);
    if (s != CCA_OK) return s;
    if (S < 1 || cu == nullptr || (reinterpret_cast<uintptr_t>(cu) & 3u) != 0)
        return CCA_ERR_INVALID_ARG;
    return S > CCA_MAX_SEQS ? CCA_ERR_UNSUPPORTED : CCA_OK;
}

bool aligned_to(const void *p, uintptr_t n)
{
    return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0;
}

cca_status paged_status(const cca_paged_cache *c)
{
    if (!c) return CCA_ERR_INVALID_ARG;
    const cca_status s = shape_status(c->B, c->Hq, c->Hkv, 0, c->d, c->g, c->w);
    if (s != CCA_OK) return s;
    if (c->layers < 1 || c->raw_cols < 1 || c->raw_pages < 1 || c->core_cols < 0 ||
        c->core_pages < 0 || (c->core_cols == 0) != (c->core_pages == 0) || c->page < 1 ||
        (c->page & (c->page - 1)) != 0)
        return CCA_ERR_INVALID_ARG;
    if (c->page < 16 || c->page > 1024 || c->B > 4096 || c->Hq / c->Hkv > 16)
        return CCA_ERR_UNSUPPORTED;
    if (static_cast<int64_t>(c->raw_cols) * c->page > kMaxT) return CCA_ERR_UNSUPPORTED;
    const bool core = c->core_cols > 0;
    if (!core && c->w < static_cast<int64_t>(c->raw_cols) * c->page) return CCA_ERR_INVALID_ARG;
    if (!ptr_ok(c->k_raw, true) || !ptr_ok(c->v_raw, true) || !ptr_ok(c->k_core, core) ||
        !ptr_ok(c->v_core, core) || !aligned_to(c->lens, 8) || !aligned_to(c->raw_table, 4) ||
        !aligned_to(c->raw_ref, 4) ||
        (core && (!aligned_to(c->core_table, 4) || !aligned_to(c->core_ref, 4))))
        return CCA_ERR_INVALID_ARG;
    return CCA_OK;
}

bool paged_workspace_ok(const cca_paged_cache &c, const void *workspace, size_t bytes)
{
    return aligned_to(workspace, 256) && bytes >= cca::paged_workspace(c).total;
}

thread_local cudaError_t g_last_cuda_error = cudaSuccess;

cca_status from_cuda(cudaError_t e)
{
    if (e == cudaSuccess) return CCA_OK;
    g_last_cuda_error = e;
    return CCA_ERR_CUDA;
}

cca_status cache_status(const cca_cache *c)
{
    if (!c) return CCA_ERR_INVALID_ARG;
    const cca_status s = shape_status(c->B, c->Hq, c->Hkv, 0, c->d, c->g, c->w);
    if (s != CCA_OK) return s;
    if (c->core_cap < 0 || c->tail_cap < static_cast<int64_t>(c->w) + c->g ||
        c->len < 0)
        return CCA_ERR_INVALID_ARG;
    if (c->Hq / c->Hkv > 16) return CCA_ERR_UNSUPPORTED;
    if (!ptr_ok(c->k_tail, true) || !ptr_ok(c->v_tail, true) ||
        !ptr_ok(c->k_core, c->core_cap > 0) || !ptr_ok(c->v_core, c->core_cap > 0))
        return CCA_ERR_INVALID_ARG;
    return CCA_OK;
}

}  // namespace

extern "C" {

cca_status cca_pool(const void *Q, const void *K, const void *V, void *Kc, void *Vc,
                    int B, int Hq, int Hkv, int64_t T, int d, int g, cudaStream_t stream)
{
    const cca_status s = shape_status(B, Hq, Hkv, T, d, g, 0);
    if (s != CCA_OK) return s;
    const int64_t m = T / g;
    const bool any = m > 0;
    if (!ptr_ok(Q, any) || !ptr_ok(K, any) || !ptr_ok(V, any) || !ptr_ok(Kc, any) ||
        !ptr_ok(Vc, any))
        return CCA_ERR_INVALID_ARG;
    if (!any) return CCA_OK;
    const size_t in_q = size_t(B) * Hq * T * d * 2, in_kv = size_t(B) * Hkv * T * d * 2;
    const size_t out = size_t(B) * Hkv * m * d * 2;
    if (overlap(Kc, out, Q, in_q) || overlap(Kc, out, K, in_kv) ||
        overlap(Kc, out, V, in_kv) || overlap(Vc, out, Q, in_q) ||
        overlap(Vc, out, K, in_kv) || overlap(Vc, out, V, in_kv) ||
        overlap(Kc, out, Vc, out))
        return CCA_ERR_INVALID_ARG;
    return from_cuda(cca::launch_pool(Q, K, V, Kc, Vc, B, Hq, Hkv, T, d, g, m, stream));
}

cca_status cca_attn_prefill(const void *Q, const void *K, const void *V, const void *Kc,
                            const void *Vc, void *O, cca_dtype o_dtype, int B, int Hq,
                            int Hkv, int64_t T, int d, int g, int w, cudaStream_t stream)
{
    const cca_status s = shape_status(B, Hq, Hkv, T, d, g, w);
    if (s != CCA_OK) return s;
    if (o_dtype != CCA_BF16 && o_dtype != CCA_F32) return CCA_ERR_INVALID_ARG;
    const bool any = T > 0;
    const int64_t m = T / g;
    if (!ptr_ok(Q, any) || !ptr_ok(K, any) || !ptr_ok(V, any) || !ptr_ok(O, any) ||
        !ptr_ok(Kc, m > 0) || !ptr_ok(Vc, m > 0))
        return CCA_ERR_INVALID_ARG;
    if (any && (reinterpret_cast<uintptr_t>(O) & 31u) != 0)
        return CCA_ERR_INVALID_ARG;  // output rows are written with 32-byte stores
    if (!any) return CCA_OK;
    const int64_t n_items = ((T + 255) / 256) * int64_t(B) * Hq;
    if (n_items > INT32_MAX) return CCA_ERR_UNSUPPORTED;
    const size_t esz = o_dtype == CCA_F32 ? 4 : 2;
    const size_t out = size_t(B) * Hq * T * d * esz;
    const size_t in_q = size_t(B) * Hq * T * d * 2, in_kv = size_t(B) * Hkv * T * d * 2;
    const size_t in_c = size_t(B) * Hkv * m * d * 2;
    if (overlap(O, out, Q, in_q) || overlap(O, out, K, in_kv) || overlap(O, out, V, in_kv) ||
        overlap(O, out, Kc, in_c) || overlap(O, out, Vc, in_c))
        return CCA_ERR_INVALID_ARG;
    return from_cuda(cca::launch_prefill(Q, K, V, Kc, Vc, O, o_dtype == CCA_F32, B, Hq,
                                         Hkv, T, d, g, w, stream));
}

cca_status cca_attn_prefill_lse(const void *Q, const void *K, const void *V, const void *Kc,
                                const void *Vc, void *O, cca_dtype o_dtype, float *lse, int B,
                                int Hq, int Hkv, int64_t T, int d, int g, int w,
                                cudaStream_t stream)
{
    const cca_status s = shape_status(B, Hq, Hkv, T, d, g, w);
    if (s != CCA_OK) return s;
    if (o_dtype != CCA_BF16 && o_dtype != CCA_F32) return CCA_ERR_INVALID_ARG;
    const bool any = T > 0;
    const int64_t m = T / g;
    if (!ptr_ok(Q, any) || !ptr_ok(K, any) || !ptr_ok(V, any) || !ptr_ok(O, any) ||
        !ptr_ok(lse, any) || !ptr_ok(Kc, m > 0) || !ptr_ok(Vc, m > 0))
        return CCA_ERR_INVALID_ARG;
    if (any && (reinterpret_cast<uintptr_t>(O) & 31u) != 0)
        return CCA_ERR_INVALID_ARG;  // output rows are written with 32-byte stores
    if (!any) return CCA_OK;
    const int64_t n_items = ((T + 255) / 256) * int64_t(B) * Hq;
    if (n_items > INT32_MAX) return CCA_ERR_UNSUPPORTED;
    const size_t esz = o_dtype == CCA_F32 ? 4 : 2;
    const size_t out = size_t(B) * Hq * T * d * esz, lse_b = size_t(B) * Hq * T * 4;
    const size_t in_q = size_t(B) * Hq * T * d * 2, in_kv = size_t(B) * Hkv * T * d * 2;
    const size_t in_c = size_t(B) * Hkv * m * d * 2;
    if (overlap(O, out, Q, in_q) || overlap(O, out, K, in_kv) || overlap(O, out, V, in_kv) ||
        overlap(O, out, Kc, in_c) || overlap(O, out, Vc, in_c) || overlap(lse, lse_b, O, out) ||
        overlap(lse, lse_b, Q, in_q) || overlap(lse, lse_b, K, in_kv) ||
        overlap(lse, lse_b, V, in_kv) || overlap(lse, lse_b, Kc, in_c) ||
        overlap(lse, lse_b, Vc, in_c))
        return CCA_ERR_INVALID_ARG;
    return from_cuda(cca::launch_prefill(Q, K, V, Kc, Vc, O, o_dtype == CCA_F32, B, Hq, Hkv, T,
                                         d, g, w, stream, lse));
}

size_t cca_attn_backward_workspace_bytes(int B, int Hq, int Hkv, int64_t T, int d, int g)
{
    if (shape_status(B, Hq, Hkv, T, d, g, 0) != CCA_OK) return 0;
    return cca::bw_layout(B, Hq, Hkv, T, d, g).total;
}

cca_status cca_attn_backward(const void *Q, const void *K, const void *V, const void *Kc,
                             const void *Vc, const void *O, cca_dtype o_dtype,
                             const float *lse, const void *dO, float *dQ, float *dK,
                             float *dV, int B, int Hq, int Hkv, int64_t T, int d, int g,
                             int w, void *workspace, size_t workspace_bytes,
                             cudaStream_t stream)
{
    const cca_status s = shape_status(B, Hq, Hkv, T, d, g, w);
    if (s != CCA_OK) return s;
    if (o_dtype != CCA_BF16 && o_dtype != CCA_F32) return CCA_ERR_INVALID_ARG;
    if (Hq / Hkv > 32) return CCA_ERR_UNSUPPORTED;
    const bool any = T > 0;
    const int64_t m = T / g;
    if (!ptr_ok(Q, any) || !ptr_ok(K, any) || !ptr_ok(V, any) || !ptr_ok(O, any) ||
        !ptr_ok(lse, any) || !ptr_ok(dO, any) || !ptr_ok(dQ, any) || !ptr_ok(dK, any) ||
        !ptr_ok(dV, any) || !ptr_ok(Kc, m > 0) || !ptr_ok(Vc, m > 0))
        return CCA_ERR_INVALID_ARG;
    // the gradient rows are written with 32-byte stores
    if (any && ((reinterpret_cast<uintptr_t>(dQ) | reinterpret_cast<uintptr_t>(dK) |
                 reinterpret_cast<uintptr_t>(dV)) & 31u) != 0)
        return CCA_ERR_INVALID_ARG;
    if (!any) return CCA_OK;
    if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 ||
        workspace_bytes < cca::bw_layout(B, Hq, Hkv, T, d, g).total)
        return CCA_ERR_INVALID_ARG;
    if (((T + 127) / 128) * int64_t(B) * Hq > INT32_MAX) return CCA_ERR_UNSUPPORTED;
    // the outputs alias nothing the call reads, nor each other, nor the workspace
    const size_t nq = size_t(B) * Hq * T * d, nk = size_t(B) * Hkv * T * d;
    const size_t nc = size_t(B) * Hkv * m * d;
    const void *ins[9] = {Q, K, V, Kc, Vc, O, lse, dO, workspace};
    const size_t in_n[9] = {nq * 2, nk * 2, nk * 2, nc * 2, nc * 2,
                            nq * (o_dtype == CCA_F32 ? 4 : 2), size_t(B) * Hq * T * 4, nq * 2,
                            workspace_bytes};
    void *outs[3] = {dQ, dK, dV};
    const size_t out_n[3] = {nq * 4, nk * 4, nk * 4};
    for (int i = 0; i < 3; ++i) {
        for (int j = 0; j < 9; ++j)
            if (overlap(outs[i], out_n[i], ins[j], in_n[j])) return CCA_ERR_INVALID_ARG;
        for (int j = i + 1; j < 3; ++j)
            if (overlap(outs[i], out_n[i], outs[j], out_n[j])) return CCA_ERR_INVALID_ARG;
    }
    return from_cuda(cca::launch_backward(Q, K, V, Kc, Vc, O, o_dtype == CCA_F32, lse, dO, dQ, dK,
                                          dV, B, Hq, Hkv, T, d, g, w, workspace, stream));
}

cca_status cca_cache_prefill(cca_cache *c, const void *Q, const void *K, const void *V,
                             int64_t T, cudaStream_t stream)
{
    cca_status s = cache_status(c);
    if (s != CCA_OK) return s;
    if (T < 0 || T > kMaxT) return CCA_ERR_INVALID_ARG;
    const bool any = T > 0;
    if (!ptr_ok(Q, any) || !ptr_ok(K, any) || !ptr_ok(V, any))
        return CCA_ERR_INVALID_ARG;
    if (any && (T - 1) / c->g >= c->core_cap) return CCA_ERR_CAPACITY;
    if (any) {
        cudaError_t e = cca::launch_pool(Q, K, V, c->k_core, c->v_core, c->B, c->Hq,
                                         c->Hkv, T, c->d, c->g, c->core_cap, stream);
        if (e != cudaSuccess) return from_cuda(e);
        const int64_t p0 = T > c->tail_cap ? T - c->tail_cap : 0;
        e = cca::launch_tail_fill(K, V, c->k_tail, c->v_tail, c->B, c->Hkv, T, c->d, p0,
                                  c->tail_cap, stream);
        if (e != cudaSuccess) return from_cuda(e);
    }
    c->len = T;
    return CCA_OK;
}

cca_status cca_cache_append(cca_cache *c, const void *q_t, const void *k_t,
                            const void *v_t, cudaStream_t stream)
{
    const cca_status s = cache_status(c);
    if (s != CCA_OK) return s;
    if (!ptr_ok(q_t, true) || !ptr_ok(k_t, true) || !ptr_ok(v_t, true))
        return CCA_ERR_INVALID_ARG;
    const int64_t t = c->len;
    if (t >= kMaxT || t / c->g >= c->core_cap) return CCA_ERR_CAPACITY;
    const cudaError_t e = cca::launch_append(q_t, k_t, v_t, c->k_core, c->v_core,
                                             c->k_tail, c->v_tail, c->B, c->Hq, c->Hkv,
                                             c->d, c->g, c->core_cap, c->tail_cap, t,
                                             stream);
    if (e != cudaSuccess) return from_cuda(e);
    c->len = t + 1;
    return CCA_OK;
}

// ---- the LCA variant -------------------------------------------------------

cca_status cca_lca_pool(const void *Q, const void *K, const void *V, void *Kc, void *Vc, int B,
                        int Hq, int Hkv, int64_t T, int d, int g, int d_rope,
                        cudaStream_t stream)
{
    const cca_status s = shape_status(B, Hq, Hkv, T, d, g, 0);
    if (s != CCA_OK) return s;
    if (d_rope < 0 || d_rope > d || d_rope % 8 != 0) return CCA_ERR_INVALID_ARG;
    const int64_t m = T / g;
    const bool any = m > 0;
    if (!ptr_ok(Q, any) || !ptr_ok(K, any) || !ptr_ok(V, any) || !ptr_ok(Kc, any) ||
        !ptr_ok(Vc, any))
        return CCA_ERR_INVALID_ARG;
    if (!any) return CCA_OK;
    const size_t in_q = size_t(B) * Hq * T * d * 2, in_kv = size_t(B) * Hkv * T * d * 2;
    const size_t out = size_t(B) * Hkv * m * d * 2;
    if (overlap(Kc, out, Q, in_q) || overlap(Kc, out, K, in_kv) ||
        overlap(Kc, out, V, in_kv) || overlap(Vc, out, Q, in_q) ||
        overlap(Vc, out, K, in_kv) || overlap(Vc, out, V, in_kv) ||
        overlap(Kc, out, Vc, out))
        return CCA_ERR_INVALID_ARG;
    return from_cuda(
        cca::launch_lca_pool(Q, K, V, Kc, Vc, B, Hq, Hkv, T, d, g, d_rope, m, stream));
}

cca_status cca_lca_cache_prefill(cca_cache *c, float *q_sum, const void *Q, const void *K,
                                 const void *V, int64_t T, int d_rope, cudaStream_t stream)
{
    cca_status s = cache_status(c);
    if (s != CCA_OK) return s;
    if (T < 0 || T > kMaxT) return CCA_ERR_INVALID_ARG;
    if (d_rope < 0 || d_rope > c->d || d_rope % 8 != 0) return CCA_ERR_INVALID_ARG;
    const bool any = T > 0;
    if (!ptr_ok(Q, any) || !ptr_ok(K, any) || !ptr_ok(V, any) || !ptr_ok(q_sum, true))
        return CCA_ERR_INVALID_ARG;
    if (any && (T - 1) / c->g >= c->core_cap) return CCA_ERR_CAPACITY;
    const int64_t m = T / c->g;
    cudaError_t e = cudaSuccess;
    if (m > 0)
        e = cca::launch_lca_pool(Q, K, V, c->k_core, c->v_core, c->B, c->Hq, c->Hkv, T, c->d,
                                 c->g, d_rope, c->core_cap, stream);
    if (e == cudaSuccess && any) {
        const int64_t p0 = T > c->tail_cap ? T - c->tail_cap : 0;
        e = cca::launch_tail_fill(K, V, c->k_tail, c->v_tail, c->B, c->Hkv, T, c->d, p0,
                                  c->tail_cap, stream);
    }
    if (e == cudaSuccess)
        e = cca::launch_lca_qsum_fill(Q, q_sum, c->B, c->Hq, c->d, T, m * c->g, stream);
    if (e != cudaSuccess) return from_cuda(e);
    c->len = T;
    return CCA_OK;
}

cca_status cca_lca_cache_append(cca_cache *c, float *q_sum, const void *q_t, const void *k_t,
                                const void *v_t, int d_rope, cudaStream_t stream)
{
    const cca_status s = cache_status(c);
    if (s != CCA_OK) return s;
    if (d_rope < 0 || d_rope > c->d || d_rope % 8 != 0) return CCA_ERR_INVALID_ARG;
    if (!ptr_ok(q_t, true) || !ptr_ok(k_t, true) || !ptr_ok(v_t, true) ||
        !ptr_ok(q_sum, true))
        return CCA_ERR_INVALID_ARG;
    const int64_t t = c->len;
    if (t >= kMaxT || t / c->g >= c->core_cap) return CCA_ERR_CAPACITY;
    const cudaError_t e = cca::launch_lca_append(q_t, k_t, v_t, q_sum, c->k_core, c->v_core,
                                                 c->k_tail, c->v_tail, c->B, c->Hq, c->Hkv,
                                                 c->d, c->g, d_rope, c->core_cap, c->tail_cap,
                                                 t, stream);
    if (e != cudaSuccess) return from_cuda(e);
    c->len = t + 1;
    return CCA_OK;
}

size_t cca_decode_workspace_bytes(const cca_cache *c)
{
    if (cache_status(c) != CCA_OK) return 0;
    return cca::decode_workspace_bytes(c->B, c->Hq, c->Hkv, c->d, c->core_cap, c->tail_cap);
}

cca_status cca_attn_decode(const cca_cache *c, const void *q_t, void *o_t,
                           cca_dtype o_dtype, void *workspace, size_t workspace_bytes,
                           cudaStream_t stream)
{
    const cca_status s = cache_status(c);
    if (s != CCA_OK) return s;
    if (o_dtype != CCA_BF16 && o_dtype != CCA_F32) return CCA_ERR_INVALID_ARG;
    if (c->len < 1) return CCA_ERR_INVALID_ARG;
    if (!ptr_ok(q_t, true) || !ptr_ok(o_t, true) || workspace == nullptr ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return CCA_ERR_INVALID_ARG;
    if (workspace_bytes < cca::decode_workspace_bytes(c->B, c->Hq, c->Hkv, c->d, c->core_cap,
                                                      c->tail_cap))
        return CCA_ERR_INVALID_ARG;
    const int64_t t = c->len - 1;
    const int64_t ws = cca::window_start(t, c->g, c->w);
    if (ws / c->g > c->core_cap) return CCA_ERR_CAPACITY;
    return from_cuda(cca::launch_decode(c->k_core, c->v_core, c->k_tail, c->v_tail, q_t,
                                        o_t, o_dtype == CCA_F32, workspace, c->B, c->Hq,
                                        c->Hkv, c->d, c->g, c->w, c->core_cap,
                                        c->tail_cap, t, stream));
}

cca_status cca_decode_step(cca_cache *c, const void *q_t, const void *k_t, const void *v_t,
                           void *o_t, cca_dtype o_dtype, void *workspace,
                           size_t workspace_bytes, cudaStream_t stream)
{
    const cca_status s = cache_status(c);
    if (s != CCA_OK) return s;
    if (o_dtype != CCA_BF16 && o_dtype != CCA_F32) return CCA_ERR_INVALID_ARG;
    if (!ptr_ok(q_t, true) || !ptr_ok(k_t, true) || !ptr_ok(v_t, true) || !ptr_ok(o_t, true) ||
        workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
        return CCA_ERR_INVALID_ARG;
    if (workspace_bytes < cca::decode_workspace_bytes(c->B, c->Hq, c->Hkv, c->d, c->core_cap,
                                                      c->tail_cap))
        return CCA_ERR_INVALID_ARG;
    const int64_t t = c->len;
    if (t >= kMaxT || t / c->g >= c->core_cap) return CCA_ERR_CAPACITY;
    const size_t out = size_t(c->B) * c->Hq * c->d * (o_dtype == CCA_F32 ? 4 : 2);
    const size_t in_q = size_t(c->B) * c->Hq * c->d * 2, in_kv = size_t(c->B) * c->Hkv * c->d * 2;
    if (overlap(o_t, out, q_t, in_q) || overlap(o_t, out, k_t, in_kv) ||
        overlap(o_t, out, v_t, in_kv) || overlap(o_t, out, workspace, workspace_bytes))
        return CCA_ERR_INVALID_ARG;
    const cudaError_t e = cca::launch_decode_step(
        c->k_core, c->v_core, c->k_tail, c->v_tail, q_t, k_t, v_t, o_t, o_dtype == CCA_F32,
        workspace, c->B, c->Hq, c->Hkv, c->d, c->g, c->w, c->core_cap, c->tail_cap, t, stream);
    if (e != cudaSuccess) return from_cuda(e);
    c->len = t + 1;
    return CCA_OK;
}

cca_status cca_cache_append_rows(const cca_cache *c, long long *lens, const void *q_t,
                                 const void *k_t, const void *v_t, cudaStream_t stream)
{
    const cca_status s = cache_status(c);
    if (s != CCA_OK) return s;
    if (!ptr_ok(q_t, true) || !ptr_ok(k_t, true) || !ptr_ok(v_t, true) ||
        lens == nullptr || (reinterpret_cast<uintptr_t>(lens) & 7u) != 0)
        return CCA_ERR_INVALID_ARG;
    // one CTA per row, one warp per key/value head
    if (c->Hkv > 32 || cca::append_rows_smem_bytes(c->Hq, c->Hkv, c->g) > 200u * 1024u)
        return CCA_ERR_UNSUPPORTED;
    return from_cuda(cca::launch_append_rows(q_t, k_t, v_t, c->k_core, c->v_core, c->k_tail,
                                             c->v_tail, lens, c->B, c->Hq, c->Hkv, c->d,
                                             c->g, c->core_cap, c->tail_cap, stream));
}

cca_status cca_attn_decode_rows(const cca_cache *c, const long long *lens, const void *q_t,
                                void *o_t, cca_dtype o_dtype, void *workspace,
                                size_t workspace_bytes, cudaStream_t stream)
{
    const cca_status s = cache_status(c);
    if (s != CCA_OK) return s;
    if (o_dtype != CCA_BF16 && o_dtype != CCA_F32) return CCA_ERR_INVALID_ARG;
    if (!ptr_ok(q_t, true) || !ptr_ok(o_t, true) || workspace == nullptr ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0 || lens == nullptr ||
        (reinterpret_cast<uintptr_t>(lens) & 7u) != 0)
        return CCA_ERR_INVALID_ARG;
    if (workspace_bytes < cca::decode_workspace_bytes(c->B, c->Hq, c->Hkv, c->d, c->core_cap,
                                                      c->tail_cap))
        return CCA_ERR_INVALID_ARG;
    return from_cuda(cca::launch_decode_rows(c->k_core, c->v_core, c->k_tail, c->v_tail, q_t,
                                             o_t, o_dtype == CCA_F32, workspace, lens, c->B,
                                             c->Hq, c->Hkv, c->d, c->g, c->w, c->core_cap,
                                             c->tail_cap, stream));
}

// ---- packed prompts ---------------------------------------------------------

cca_status cca_pool_packed(const cca_rows *Q, const cca_rows *K, const cca_rows *V,
                           const int32_t *cu, void *Kc, void *Vc, int S, int Hq, int Hkv,
                           int64_t total, int d, int g, cudaStream_t stream)
{
    const cca_status s = packed_status(S, Hq, Hkv, total, d, g, 0, cu);
    if (s != CCA_OK) return s;
    if (cca::pool_packed_smem(S, Hq / Hkv, g) > cca::kSmemMost) return CCA_ERR_UNSUPPORTED;
    const int64_t m = total / g;
    if (m == 0) return CCA_OK;
    cca::PackedRows q, k, v;
    if (!rows_ok(Q, Hq, total, d, 8, 16, false, q) || !rows_ok(K, Hkv, total, d, 8, 16, false, k) ||
        !rows_ok(V, Hkv, total, d, 8, 16, false, v) || !ptr_ok(Kc, true) || !ptr_ok(Vc, true))
        return CCA_ERR_INVALID_ARG;
    const size_t out = size_t(Hkv) * m * d * 2;
    const size_t nq = rows_bytes(q, Hq, total, d, 2), nk = rows_bytes(k, Hkv, total, d, 2),
                 nv = rows_bytes(v, Hkv, total, d, 2);
    for (void *o : {Kc, Vc})
        if (overlap(o, out, q.data, nq) || overlap(o, out, k.data, nk) ||
            overlap(o, out, v.data, nv) || overlap(o, out, cu, sizeof(int) * (S + 1)))
            return CCA_ERR_INVALID_ARG;
    if (overlap(Kc, out, Vc, out)) return CCA_ERR_INVALID_ARG;
    return from_cuda(cca::launch_pool_packed(q, k, v, cu, Kc, Vc, S, Hq, Hkv, total, d, g, stream));
}

size_t cca_packed_workspace_bytes(int S, int64_t total)
{
    if (S < 1 || S > CCA_MAX_SEQS || total < 0 || total > kMaxT) return 0;
    if (cca::packed_inline(S, total)) return 0;
    return 256 + 16 * static_cast<size_t>(cca::packed_max_blocks(S, total));
}

cca_status cca_attn_prefill_packed(const cca_rows *Q, const cca_rows *K, const cca_rows *V,
                                   const void *Kc, const void *Vc, const int32_t *cu,
                                   const cca_rows *O, cca_dtype o_dtype, int S, int Hq, int Hkv,
                                   int64_t total, int d, int g, int w, void *workspace,
                                   size_t workspace_bytes, cudaStream_t stream)
{
    const cca_status s = packed_status(S, Hq, Hkv, total, d, g, w, cu);
    if (s != CCA_OK) return s;
    if (o_dtype != CCA_BF16 && o_dtype != CCA_F32) return CCA_ERR_INVALID_ARG;
    if (total == 0) return CCA_OK;
    const int64_t m = total / g;
    const bool core = m > 0 && w < total;
    cca::PackedRows q, k, v, o;
    if (!rows_ok(Q, Hq, total, d, 8, 16, false, q) || !rows_ok(K, Hkv, total, d, 8, 16, false, k) ||
        !rows_ok(V, Hkv, total, d, 8, 16, false, v) || !rows_ok(O, Hq, total, d, 16, 32, true, o) ||
        !ptr_ok(Kc, core) || !ptr_ok(Vc, core))
        return CCA_ERR_INVALID_ARG;
    const size_t need = cca_packed_workspace_bytes(S, total);
    if (need > 0 && (!aligned_to(workspace, 256) || workspace_bytes < need))
        return CCA_ERR_INVALID_ARG;
    workspace_bytes = need;
    if (cca::packed_max_blocks(S, total) * Hq > INT32_MAX) return CCA_ERR_UNSUPPORTED;
    const size_t out = rows_bytes(o, Hq, total, d, o_dtype == CCA_F32 ? 4 : 2);
    const size_t nc = core ? size_t(Hkv) * m * d * 2 : 0, ncu = sizeof(int) * (S + 1);
    if (overlap(o.data, out, q.data, rows_bytes(q, Hq, total, d, 2)) ||
        overlap(o.data, out, k.data, rows_bytes(k, Hkv, total, d, 2)) ||
        overlap(o.data, out, v.data, rows_bytes(v, Hkv, total, d, 2)) ||
        overlap(o.data, out, Kc, nc) || overlap(o.data, out, Vc, nc) ||
        overlap(o.data, out, cu, ncu) || overlap(o.data, out, workspace, workspace_bytes) ||
        overlap(workspace, workspace_bytes, cu, ncu))
        return CCA_ERR_INVALID_ARG;
    return from_cuda(cca::launch_prefill_packed(q, k, v, core ? Kc : nullptr, core ? Vc : nullptr,
                                                o, o_dtype == CCA_F32, cu, S, Hq, Hkv, total, d, g,
                                                w, workspace, stream));
}

// ---- the paged cache ----------------------------------------------------------

size_t cca_paged_workspace_bytes(const cca_paged_cache *c)
{
    if (paged_status(c) != CCA_OK) return 0;
    return cca::paged_workspace(*c).total;
}

cca_status cca_paged_reserve(const cca_paged_cache *c, const long long *n_new, long long n,
                             cudaStream_t stream)
{
    const cca_status s = paged_status(c);
    if (s != CCA_OK) return s;
    if (n_new != nullptr ? !aligned_to(n_new, 8) : n < 0) return CCA_ERR_INVALID_ARG;
    return from_cuda(cca::launch_paged_reserve(*c, n_new, n, nullptr, stream));
}

cca_status cca_paged_reserve_held(const cca_paged_cache *c, const long long *n_new, long long n,
                                  void *workspace, size_t workspace_bytes, cudaStream_t stream)
{
    const cca_status s = paged_status(c);
    if (s != CCA_OK) return s;
    if ((n_new != nullptr ? !aligned_to(n_new, 8) : n < 0) ||
        !paged_workspace_ok(*c, workspace, workspace_bytes))
        return CCA_ERR_INVALID_ARG;
    return from_cuda(cca::launch_paged_reserve(*c, n_new, n, workspace, stream));
}

cca_status cca_paged_fill(const cca_paged_cache *c, int layer, const cca_rows *K,
                          const cca_rows *V, const void *Kc, const void *Vc, const int32_t *cu,
                          const int32_t *rows, int S, int64_t total, cudaStream_t stream)
{
    cca_status s = paged_status(c);
    if (s != CCA_OK) return s;
    if ((s = packed_status(S, c->Hq, c->Hkv, total, c->d, c->g, c->w, cu)) != CCA_OK) return s;
    if (layer < 0 || layer >= c->layers || !aligned_to(rows, 4)) return CCA_ERR_INVALID_ARG;
    if (total == 0) return CCA_OK;
    const bool core = c->core_cols > 0 && total / c->g > 0;
    cca::PackedRows k, v;
    if (!rows_ok(K, c->Hkv, total, c->d, 8, 16, false, k) ||
        !rows_ok(V, c->Hkv, total, c->d, 8, 16, false, v) || !ptr_ok(Kc, core) ||
        !ptr_ok(Vc, core))
        return CCA_ERR_INVALID_ARG;
    const size_t page = size_t(c->layers) * c->Hkv * c->page * c->d * 2;
    const void *ins[4] = {k.data, v.data, core ? Kc : nullptr, core ? Vc : nullptr};
    const size_t n_core = size_t(c->Hkv) * (total / c->g) * c->d * 2;
    const size_t n_in[4] = {rows_bytes(k, c->Hkv, total, c->d, 2),
                            rows_bytes(v, c->Hkv, total, c->d, 2), n_core, n_core};
    for (int i = 0; i < 4; ++i)
        if (overlap(c->k_raw, page * c->raw_pages, ins[i], n_in[i]) ||
            overlap(c->v_raw, page * c->raw_pages, ins[i], n_in[i]) ||
            overlap(c->k_core, page * c->core_pages, ins[i], n_in[i]) ||
            overlap(c->v_core, page * c->core_pages, ins[i], n_in[i]))
            return CCA_ERR_INVALID_ARG;
    return from_cuda(cca::launch_paged_fill(*c, layer, k, v, core ? Kc : nullptr,
                                            core ? Vc : nullptr, cu, rows, S, total, stream));
}

static cca_status paged_decode(const cca_paged_cache *c, int layer, const void *q_t,
                               const void *k_t, const void *v_t, bool step, void *o_t,
                               cca_dtype o_dtype, void *workspace, size_t workspace_bytes,
                               cudaStream_t stream)
{
    const cca_status s = paged_status(c);
    if (s != CCA_OK) return s;
    if (o_dtype != CCA_BF16 && o_dtype != CCA_F32) return CCA_ERR_INVALID_ARG;
    if (layer < 0 || layer >= c->layers || !ptr_ok(q_t, true) || !ptr_ok(k_t, step) ||
        !ptr_ok(v_t, step) || !ptr_ok(o_t, true) ||
        !paged_workspace_ok(*c, workspace, workspace_bytes))
        return CCA_ERR_INVALID_ARG;
    const size_t in_q = size_t(c->B) * c->Hq * c->d * 2, in_kv = size_t(c->B) * c->Hkv * c->d * 2;
    const size_t out = size_t(c->B) * c->Hq * c->d * (o_dtype == CCA_F32 ? 4 : 2);
    if (overlap(o_t, out, q_t, in_q) || overlap(o_t, out, k_t, step ? in_kv : 0) ||
        overlap(o_t, out, v_t, step ? in_kv : 0) || overlap(o_t, out, workspace, workspace_bytes))
        return CCA_ERR_INVALID_ARG;
    return from_cuda(cca::launch_paged_decode(*c, layer, q_t, step ? k_t : nullptr,
                                              step ? v_t : nullptr, o_t, o_dtype == CCA_F32,
                                              workspace, stream));
}

cca_status cca_attn_decode_paged(const cca_paged_cache *c, int layer, const void *q_t, void *o_t,
                                 cca_dtype o_dtype, void *workspace, size_t workspace_bytes,
                                 cudaStream_t stream)
{
    return paged_decode(c, layer, q_t, nullptr, nullptr, false, o_t, o_dtype, workspace,
                        workspace_bytes, stream);
}

cca_status cca_paged_step(const cca_paged_cache *c, int layer, const void *q_t, const void *k_t,
                          const void *v_t, void *o_t, cca_dtype o_dtype, void *workspace,
                          size_t workspace_bytes, cudaStream_t stream)
{
    return paged_decode(c, layer, q_t, k_t, v_t, true, o_t, o_dtype, workspace, workspace_bytes,
                        stream);
}

cca_status cca_paged_fork(const cca_paged_cache *c, const int32_t *parent, void *workspace,
                          size_t workspace_bytes, cudaStream_t stream)
{
    const cca_status s = paged_status(c);
    if (s != CCA_OK) return s;
    if (!aligned_to(parent, 4) || !paged_workspace_ok(*c, workspace, workspace_bytes))
        return CCA_ERR_INVALID_ARG;
    return from_cuda(cca::launch_paged_fork(*c, parent, workspace, stream));
}

cca_status cca_paged_compact(const cca_paged_cache *c, long long *live, void *workspace,
                             size_t workspace_bytes, cudaStream_t stream)
{
    const cca_status s = paged_status(c);
    if (s != CCA_OK) return s;
    if (!aligned_to(live, 8) || !paged_workspace_ok(*c, workspace, workspace_bytes))
        return CCA_ERR_INVALID_ARG;
    return from_cuda(cca::launch_paged_compact(*c, live, workspace, stream));
}

cca_status cca_device_status(cudaStream_t stream)
{
    cudaError_t e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return from_cuda(e);
    unsigned int a = 0, b = 0, c = 0, d = 0, f = 0, h = 0, l = 0, p = 0, t = 0, u = 0;
    if ((e = cca::prefill_status_read_clear(&a)) != cudaSuccess ||
        (e = cca::pool_status_read_clear(&b)) != cudaSuccess ||
        (e = cca::append_status_read_clear(&c)) != cudaSuccess ||
        (e = cca::selftest_status_read_clear(&d)) != cudaSuccess ||
        (e = cca::decode_status_read_clear(&f)) != cudaSuccess ||
        (e = cca::backward_status_read_clear(&h)) != cudaSuccess ||
        (e = cca::lca_status_read_clear(&l)) != cudaSuccess ||
        (e = cca::packed_status_read_clear(&p)) != cudaSuccess ||
        (e = cca::paged_decode_status_read_clear(&t)) != cudaSuccess ||
        (e = cca::paged_tables_status_read_clear(&u)) != cudaSuccess)
        return from_cuda(e);
    const unsigned int st = a | b | c | d | f | h | l | p | t | u;
    if (st & cca::kStatusTimeout) return CCA_ERR_TIMEOUT;
    if (st & cca::kStatusCapacity) return CCA_ERR_CAPACITY;
    if (st & cca::kStatusSeqlens) return CCA_ERR_SEQLENS;
    if (st & cca::kStatusPage) return CCA_ERR_PAGE;
    if (st & cca::kStatusRange) return CCA_ERR_RANGE;
    return CCA_OK;
}

const char *cca_status_string(cca_status s)
{
    switch (s) {
    case CCA_OK: return "CCA_OK";
    case CCA_ERR_INVALID_ARG: return "CCA_ERR_INVALID_ARG";
    case CCA_ERR_UNSUPPORTED: return "CCA_ERR_UNSUPPORTED";
    case CCA_ERR_CAPACITY: return "CCA_ERR_CAPACITY";
    case CCA_ERR_CUDA: return "CCA_ERR_CUDA";
    case CCA_ERR_TIMEOUT: return "CCA_ERR_TIMEOUT";
    case CCA_ERR_RANGE: return "CCA_ERR_RANGE";
    case CCA_ERR_SCRATCH: return "CCA_ERR_SCRATCH";
    case CCA_ERR_SEQLENS: return "CCA_ERR_SEQLENS";
    case CCA_ERR_PAGE: return "CCA_ERR_PAGE";
    }
    return "CCA_ERR_UNKNOWN";
}

const char *cca_version(void) { return "0.1.0"; }

const char *cca_last_error(void)
{
    return g_last_cuda_error == cudaSuccess ? "no error" : cudaGetErrorString(g_last_cuda_error);
}

}  // extern "C"
