// Test helper (compiled by tests/test_gpu_ring_give_up.py): the paged attention kernels with one warp of one CTA whose n-th wait
// for a copy reports that it ran out, although the copy lands as ever. Nothing waits longer for it, and nothing else is changed.
// Beside that the helper keeps, for the warp, how often each stage's barrier was waited on, so that the parities
// that the ring asks for can be compared with it.
#include "token_cache.cuh"

namespace skv {
__device__ int g_block, g_warp, g_at;      // who gives up, and at which of its waits (-1: no one)
__device__ int g_waits, g_gave_up;         // the warp's waits so far; 1 once it gave up
__device__ int g_drained, g_wrong;         // stages waited for afterwards, parities that were not the expected ones
__device__ int g_count[8];                 // completed waits of each of the warp's stages

__device__ __forceinline__ bool watched() { return blockIdx.x == g_block && threadIdx.x >> 5 == g_warp; }

__device__ __forceinline__ void seen(uint64_t *bar, uint32_t parity) {
    int &n = g_count[smem_u32(bar) >> 3 & 7];
    if ((n & 1) != static_cast<int>(parity & 1)) ++g_wrong;
    ++n;
}

// the ring's first look at a stage: one per wait. The volatile reads are the same in all lanes: lane 0 alone writes, behind
// a warp barrier.
__device__ __noinline__ bool watched_try_wait(uint64_t *bar, uint32_t parity) {
    if (!watched()) return mbar_try_wait(bar, parity);
    const int n = *const_cast<volatile int *>(&g_waits), at = g_at;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) *const_cast<volatile int *>(&g_waits) = n + 1;
    __syncwarp();
    if (n == at) return false;
    const bool ok = __all_sync(0xffffffffu, mbar_try_wait(bar, parity));
    if (ok && (threadIdx.x & 31) == 0) seen(bar, parity);
    __syncwarp();
    return ok;
}

__device__ __noinline__ bool watched_wait(uint64_t *bar, uint32_t parity) {
    if (!watched()) return mbar_wait(bar, parity);
    const bool now = *const_cast<volatile int *>(&g_waits) == g_at + 1, before = *const_cast<volatile int *>(&g_gave_up);
    __syncwarp();
    if (now && !before) {
        if ((threadIdx.x & 31) == 0) *const_cast<volatile int *>(&g_gave_up) = 1;
        __syncwarp();
        return false;
    }
    const bool ok = __all_sync(0xffffffffu, mbar_wait(bar, parity));
    if ((threadIdx.x & 31) == 0) {
        if (ok) seen(bar, parity);
        if (before) ++g_drained;
    }
    __syncwarp();
    return ok;
}
}  // namespace skv

#define mbar_try_wait watched_try_wait
#define mbar_wait watched_wait
// the library's own choice of a kernel is not needed (nor compiled): a template that no one instantiates
#define launch_paged_attn(...) not_defined(); template <int> cudaError_t not_used(__VA_ARGS__)
#include "paged_attn.cu"
#undef launch_paged_attn

using namespace skv;

// kind 0: bf16 queries over e4m3 pages at d = 128; 1: over raw ones at d = 64; 2: fp32 queries over raw pages at d = 64.
// result: {waits, gave up, drained, wrong}
extern "C" int run_give_up(int kind, const void *q, const void *pages, int64_t num_pages, const int32_t *table, int max_pages,
                           const int32_t *lens, void *out, float *lse, void *flags, int32_t *counters, float *part_o,
                           float *part_l, int B, int Hq, int Hkv, int block, int warp, int at, int *result) {
    const int zero[8] = {};
    cudaMemcpyToSymbol(g_block, &block, 4);
    cudaMemcpyToSymbol(g_warp, &warp, 4);
    cudaMemcpyToSymbol(g_at, &at, 4);
    cudaMemcpyToSymbol(g_waits, zero, 4);
    cudaMemcpyToSymbol(g_gave_up, zero, 4);
    cudaMemcpyToSymbol(g_drained, zero, 4);
    cudaMemcpyToSymbol(g_wrong, zero, 4);
    cudaMemcpyToSymbol(g_count, zero, 32);
    const int d = kind == 0 ? 128 : 64;
    PagedArgs a{};
    a.q = q;
    a.q_h = d;
    a.q_r = a.q_b = static_cast<int64_t>(Hq) * d;
    a.pages = static_cast<const uint8_t *>(pages);
    a.num_pages = num_pages;
    a.page_table = table;
    a.max_pages = max_pages;
    a.lens = lens;
    a.scale = d == 128 ? 0.08838834764831845f : 0.125f;
    a.out = out;
    a.lse = lse;
    a.B = B;
    a.R = 1;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.G = a.rows = Hq / Hkv;   // 8 at most: one pass
    a.inv_G = 1.0f / a.G;
    a.d = d;
    a.dtype = kind == 2 ? SKV_F32 : SKV_BF16;
    a.format = kind == 0 ? SKV_CACHE_E4M3 : SKV_CACHE_RAW;
    a.pass_rows = 8;
    a.passes = 1;
    a.part_o = part_o;
    a.part_l = part_l;
    a.counters = counters;
    a.flags = static_cast<uint32_t *>(flags);
    const cudaError_t e = kind == 0 ? launch_mma<true, 128, 1, 8, 2, 2, 1>(a, nullptr)
                          : kind == 1 ? launch_mma<false, 64, 1, 8, 2, 1, 2>(a, nullptr) : launch_f32<false, 64, 8, 2>(a, nullptr);
    if (e != cudaSuccess || cudaDeviceSynchronize() != cudaSuccess) return 1;
    cudaMemcpyFromSymbol(result, g_waits, 4);
    cudaMemcpyFromSymbol(result + 1, g_gave_up, 4);
    cudaMemcpyFromSymbol(result + 2, g_drained, 4);
    cudaMemcpyFromSymbol(result + 3, g_wrong, 4);
    return 0;
}
