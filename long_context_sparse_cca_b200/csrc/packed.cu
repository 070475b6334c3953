// Packed prompts: sequences of different lengths one behind the other.
// Here: the checked offsets, the order of the query blocks for the attention
// kernel (prefill.cu), and the pooling of every sequence's groups (section
// 全局感知池化 of the CCA write-up).
#include "internal.h"
#include "packed.cuh"
#include "pool_warp.cuh"

namespace cca {

__device__ unsigned int g_packed_status;  // kStatusSeqlens, kStatusRange

namespace {

constexpr int kPlanThreads = 256;
constexpr int kPoolWarps = 8;

// The list of the attention kernel's query blocks (packed.cuh).
__global__ void __launch_bounds__(kPlanThreads)
    packed_plan_kernel(const int *__restrict__ cu, int S, int64_t total, int g,
                       int4 *__restrict__ blocks, int *__restrict__ count)
{
    extern __shared__ int scu[];  // [S + 1] offsets
    chain_begin();
    if (!load_offsets(cu, S, total, scu)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) {
            *count = 0;
            atomicOr(&g_packed_status, kStatusSeqlens);
        }
        return;
    }
    if (blockIdx.x == 0) {
        __shared__ int warp_sum_s[kPlanThreads / 32];
        int n = 0;
        for (int s = threadIdx.x; s < S; s += kPlanThreads) n += packed_blocks(scu, s);
        n = __reduce_add_sync(0xffffffffu, n);
        if ((threadIdx.x & 31) == 0) warp_sum_s[threadIdx.x >> 5] = n;
        __syncthreads();
        if (threadIdx.x == 0) {
            int sum = 0;
            for (int i = 0; i < kPlanThreads / 32; ++i) sum += warp_sum_s[i];
            *count = sum;
        }
    }
    const int64_t i = static_cast<int64_t>(blockIdx.x) * kPlanThreads + threadIdx.x;
    if (i >= total / 256 + S) return;
    const PackedPair pair = packed_pair(scu, S, i);
    if (pair.blk < 0) return;
    const int first = scu[pair.s];
    blocks[packed_place(scu, S, pair)] =
        make_int4(first, scu[pair.s + 1] - first, pair.blk, first / g);
}

// As pool_kernel (pool.cu), one warp per (head, core row): the core row's
// sequence is the last one whose first core row cu[s] / g is not behind it.
// Rows that hold no group become zero.
// Three blocks fit an SM where the group's keys take up to 32 registers of
// a thread and its values are loaded only after them: 32K tokens of 32 heads
// take 125 us instead of 137 with two (D = 128, G = 32 would spill).
template <int D, int G>
__global__ void __launch_bounds__(kPoolWarps * 32, G > 0 && D * G <= 2048 ? 3 : 2)
    pool_packed_kernel(PackedRows Q, PackedRows K, PackedRows V, const int *__restrict__ cu,
                       uint16_t *__restrict__ Kc, uint16_t *__restrict__ Vc, int S, int Hkv, int r,
                       int64_t total, int g, int64_t m, float scale_log2)
{
    extern __shared__ int scu[];  // [S + 1] offsets, then the warps' scratch
    chain_begin();
    if (!load_offsets(cu, S, total, scu)) {
        if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(&g_packed_status, kStatusSeqlens);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float *scratch = reinterpret_cast<float *>(scu + S + 1) + warp * (r * g + g);
    const auto *q = static_cast<const uint16_t *>(Q.data);
    const auto *k = static_cast<const uint16_t *>(K.data);
    const auto *v = static_cast<const uint16_t *>(V.data);
    const int64_t n = static_cast<int64_t>(Hkv) * m;
    const int64_t step = static_cast<int64_t>(gridDim.x) * kPoolWarps;
    // first token of group gid = h m + c (-1: none) and its head
    auto place = [&](int64_t gid, int &h) {
        h = static_cast<int>(gid / m);
        const int c = static_cast<int>(gid - h * m);
        const int s = core_row_sequence(scu, S, g, c);
        const int j = c - scu[s] / g;
        return j < 0 || j >= (scu[s + 1] - scu[s]) / g ? -1 : scu[s] + j * g;
    };
    int64_t gid = static_cast<int64_t>(blockIdx.x) * kPoolWarps + warp;
    int h_next = 0, next = gid < n ? place(gid, h_next) : -1;
    for (; gid < n; gid += step) {
        const int64_t first = next;
        const int h = h_next;
        if (gid + step < n) {
            // the next group's rows on their way to L2 while this one is pooled
            next = place(gid + step, h_next);
            constexpr int LINES = D / 64;  // 128-byte lines of a row
            if (next >= 0)
                for (int i = lane; i < g * LINES; i += 32) {
                    const int64_t row = next + i / LINES;
                    const uint16_t *kl = k + h_next * K.head + row * K.row + i % LINES * 64;
                    const uint16_t *vl = v + h_next * V.head + row * V.row + i % LINES * 64;
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(kl));
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(vl));
                }
        }
        uint16_t *kc = Kc + gid * D, *vc = Vc + gid * D;
        if (first < 0) {
            if (lane < D / 8) {
                reinterpret_cast<uint4 *>(kc)[lane] = make_uint4(0u, 0u, 0u, 0u);
                reinterpret_cast<uint4 *>(vc)[lane] = make_uint4(0u, 0u, 0u, 0u);
            }
            continue;
        }
        const uint16_t *Kg = k + h * K.head + first * K.row;
        const uint16_t *Vg = v + h * V.head + first * V.row;
        const uint16_t *Qb = q + static_cast<int64_t>(h) * r * Q.head + (first + g - 1) * Q.row;
        auto krow = [&](int i) { return Kg + i * K.row; };
        auto vrow = [&](int i) { return Vg + i * V.row; };
        auto qrow = [&](int i) { return Qb + i * Q.head; };
        bool over;
        if constexpr (G > 0)
            over = pool_group_warp_fast<D, G, false>(krow, vrow, qrow, r, scale_log2, scratch, kc,
                                                     vc);
        else
            over = pool_group_warp<D>(krow, vrow, qrow, r, g, scale_log2, scratch, kc, vc);
        if (over && lane == 0) atomicOr(&g_packed_status, kStatusRange);
        __syncwarp();  // the scratch is read before the next group's scores
    }
}

}  // namespace

cudaError_t launch_packed_plan(const int *cu, int S, int64_t total, int g, int4 *blocks,
                               int *count, cudaStream_t s)
{
    const int64_t n = packed_max_blocks(S, total);
    const int grid = static_cast<int>((n + kPlanThreads - 1) / kPlanThreads);
    return launch_chained(packed_plan_kernel, grid, kPlanThreads, sizeof(int) * (S + 1), s, cu, S,
                          total, g, blocks, count);
}

size_t pool_packed_smem(int S, int r, int g)
{
    return sizeof(float) * kPoolWarps * (r * g + g) + sizeof(int) * (S + 1);
}

cudaError_t launch_pool_packed(const PackedRows &Q, const PackedRows &K, const PackedRows &V,
                               const int *cu, void *Kc, void *Vc, int S, int Hq, int Hkv,
                               int64_t total, int d, int g, cudaStream_t s)
{
    const int64_t m = total / g, n = m * Hkv;
    const int r = Hq / Hkv;
    const size_t smem = pool_packed_smem(S, r, g);
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t want = (n + kPoolWarps - 1) / kPoolWarps;
    // few enough that a block's offsets are loaded for many groups
    const int blocks = static_cast<int>(want < 8LL * sms ? want : 8LL * sms);
    const float scale_log2 = kLog2e / sqrtf(static_cast<float>(d));
    cudaError_t e = cudaSuccess;
    auto go = [&](auto kern) {
        if ((e = allow_smem(kern, smem)) != cudaSuccess) return;
        e = launch_chained(kern, blocks, kPoolWarps * 32, smem, s, Q, K, V, cu,
                           static_cast<uint16_t *>(Kc), static_cast<uint16_t *>(Vc), S, Hkv, r,
                           total, g, m, scale_log2);
    };
    if (d == 128) {
        if (g == 16)
            go(pool_packed_kernel<128, 16>);
        else if (g == 32)
            go(pool_packed_kernel<128, 32>);
        else
            go(pool_packed_kernel<128, 0>);
    } else {
        if (g == 16)
            go(pool_packed_kernel<64, 16>);
        else if (g == 32)
            go(pool_packed_kernel<64, 32>);
        else
            go(pool_packed_kernel<64, 0>);
    }
    return e;
}

cudaError_t packed_status_read_clear(unsigned int *v)
{
    unsigned int zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(v, g_packed_status, sizeof(*v));
    if (e == cudaSuccess && *v) e = cudaMemcpyToSymbol(g_packed_status, &zero, sizeof(zero));
    return e;
}

}  // namespace cca
