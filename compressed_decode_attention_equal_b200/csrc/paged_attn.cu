// skv_paged_attn: attention of the new token's query rows over the exact-token cache.
//
// k_paged_f32 (fp32 caches and queries): CUDA cores, exact fp32 products. A warp takes 32 tokens:
// for the logits each lane owns one token and walks its key chunk by chunk against up to 8 query rows
// broadcast from shared memory (32 FMAs per 16-byte key load and 8 broadcast loads); for the values
// the lanes own dimensions, so that a value row is one coalesced load, with the 8 weights of the
// token broadcast. Each warp keeps its own running maximum, sum and outputs; the CTA's eight join
// at the end of a piece.
#include <mutex>

#include "token_cache.cuh"

namespace skv {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;

// cap tanh(x / cap) with t = x / cap given: tanh t = 1 - 2 / (e^(2t) + 1), whose absolute error is a few
// 2^-24 over the whole range (the hardware tanh's 2^-11 would show in the logits)
__device__ __forceinline__ float capped(float t, float cap) {
    const float e = exp2f(t * (2.0f * kLog2e));
    return cap * (1.0f - 2.0f / (e + 1.0f));
}

constexpr int kSimpleWarps = 8, kSimpleThreads = 32 * kSimpleWarps, kSimplePass = 8;
constexpr int kSimpleRound = 2 * kSimpleWarps;   // token groups of a round: 32 tokens per warp

template <int D>
struct SimpleSmem {
    PagedSched sched;
    alignas(16) float q[kSimplePass][D];
    float p[kSimpleWarps][32][kSimplePass];
    float o[kSimpleWarps][kSimplePass][D];
    float m[kSimpleWarps][kSimplePass], l[kSimpleWarps][kSimplePass];
};

template <typename T, bool E4M3, int D>
__global__ void __launch_bounds__(kSimpleThreads) k_paged_f32(const PagedArgs a) {
    using G = CacheGeom<T, E4M3, D>;
    using CV = ChunkValues<T, E4M3>;
    constexpr int NR = kSimplePass, PER = D / 32;   // PER output dimensions per lane
    extern __shared__ __align__(16) uint8_t smem_raw[];
    SimpleSmem<D> &sm = *reinterpret_cast<SimpleSmem<D> *>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    paged_schedule<kSimpleThreads, kSimpleRound>(a, sm.sched);
    PagedWalk walk;
    walk.begin(a, sm.sched);
    PagedPiece pc;
    const int64_t page_bytes = static_cast<int64_t>(a.Hkv) * kPageGroups * G::kGroup;
    const T *q = static_cast<const T *>(a.q);
    while (walk.next(a, sm.sched, &pc)) {
        const int row0 = pc.pass * NR, rows = min(NR, a.rows - row0);
        for (int i = tid; i < NR * D; i += kSimpleThreads) {
            const int r = i / D, d = i % D;
            float x = 0.f;
            if (r < rows) {
                const int rr = (row0 + r) / a.G, g = (row0 + r) % a.G;
                x = static_cast<float>(q[pc.b * a.q_b + rr * a.q_r + (static_cast<int64_t>(pc.h) * a.G + g) * a.q_h + d]);
            }
            sm.q[r][d] = x;
        }
        float slope[NR];
#pragma unroll
        for (int r = 0; r < NR; ++r)
            slope[r] = a.slopes && r < rows ? a.slopes[pc.h * a.G + (row0 + r) % a.G] : 0.f;
        __syncthreads();
        const int lo = sm.sched.lo[pc.b], hi = sm.sched.hi[pc.b];
        const int g0 = lo / kGroupTokens;
        const int t_end = min(hi, (g0 + pc.r1 * kSimpleRound) * kGroupTokens);
        float m[NR], l[NR], o[NR][PER];
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            m[r] = -INFINITY;
            l[r] = 0.f;
#pragma unroll
            for (int i = 0; i < PER; ++i) o[r][i] = 0.f;
        }
        for (int t0 = (g0 + pc.r0 * kSimpleRound) * kGroupTokens + 32 * warp; t0 < t_end; t0 += 32 * kSimpleWarps) {
            // logits: lane = token
            const int t = t0 + lane;
            bool valid = t >= lo && t < t_end;
            const uint8_t *grp = nullptr;
            if (valid) {
                const int page = a.page_table[static_cast<int64_t>(pc.b) * a.max_pages + t / SKV_CACHE_PAGE_TOKENS];
                if (page < 0 || page >= a.num_pages) {
                    raise_flag(a.flags, FLAG_BAD_PAGE);
                    valid = false;
                } else {
                    grp = a.pages + page * page_bytes +
                          (static_cast<int64_t>(pc.h) * kPageGroups + t % SKV_CACHE_PAGE_TOKENS / kGroupTokens) * G::kGroup;
                }
            }
            const int n = t % kGroupTokens;
            float s[NR];
#pragma unroll
            for (int r = 0; r < NR; ++r) s[r] = 0.f;
            float vs = 1.f;
            if (valid) {
                const uint8_t *key = grp + n * G::kVec;
#pragma unroll 2
                for (int c = 0; c < G::kChunks; ++c) {
                    float x[CV::N];
                    CV::get(*reinterpret_cast<const uint4 *>(key + 16 * cache_chunk(c, n, G::kChunks)), x);
#pragma unroll
                    for (int r = 0; r < NR; ++r)
#pragma unroll
                        for (int i = 0; i < CV::N; i += 4) {
                            const float4 y = *reinterpret_cast<const float4 *>(&sm.q[r][c * CV::N + i]);
                            s[r] = fmaf(x[i], y.x, s[r]);
                            s[r] = fmaf(x[i + 1], y.y, s[r]);
                            s[r] = fmaf(x[i + 2], y.z, s[r]);
                            s[r] = fmaf(x[i + 3], y.w, s[r]);
                        }
                }
                float ks = a.scale;
                if constexpr (E4M3) {
                    ks *= scale_of(grp[2 * G::kBlock + n]);
                    vs = scale_of(grp[2 * G::kBlock + kGroupTokens + n]);
                }
                const float gap = static_cast<float>(hi - 1 - t);
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    s[r] *= ks;
                    if (a.softcap > 0.f) s[r] = capped(s[r] / a.softcap, a.softcap);
                    s[r] = (s[r] - slope[r] * gap) * kLog2e;
                }
            } else {
#pragma unroll
                for (int r = 0; r < NR; ++r) s[r] = -INFINITY;
            }
            // running maximum and sum (each lane keeps the sum of its own tokens)
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                float top = s[r];
#pragma unroll
                for (int x = 16; x; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                top = fmaxf(top, m[r]);
                const float f = top > -INFINITY ? exp2f(m[r] - top) : 1.f;
                const float p = top > -INFINITY || s[r] != s[r] ? exp2f(s[r] - top) : 0.f;
                m[r] = top;
                l[r] = l[r] * f + p;
#pragma unroll
                for (int i = 0; i < PER; ++i) o[r][i] *= f;
                sm.p[warp][lane][r] = p * vs;
            }
            __syncwarp();
            // values: lane = dimensions
            const uint32_t mask = __ballot_sync(0xffffffffu, valid);
            const uint64_t base = reinterpret_cast<uint64_t>(grp);
#pragma unroll 4
            for (int j = 0; j < 32; ++j) {
                if (!(mask >> j & 1)) continue;   // masked rows are not read: they may hold anything
                const uint8_t *g = reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, base, j));
                const int nj = (t0 + j) % kGroupTokens;
                const int byte = lane * PER * G::kElem;
                const uint8_t *vp = g + G::kBlock + nj * G::kVec + 16 * cache_chunk(byte / 16, nj, G::kChunks) + byte % 16;
                float x[PER];
                if constexpr (E4M3) {
                    const uint16_t w0 = *reinterpret_cast<const unsigned short *>(vp);
                    const float2 f0 = f16x2_to_f32(e4m3x2_to_f16x2(w0));
                    x[0] = f0.x, x[1] = f0.y;
                    if constexpr (PER == 4) {
                        const float2 f1 = f16x2_to_f32(
                            e4m3x2_to_f16x2(*reinterpret_cast<const unsigned short *>(vp + 2)));
                        x[2] = f1.x, x[3] = f1.y;
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < PER; ++i) x[i] = static_cast<float>(reinterpret_cast<const T *>(vp)[i]);
                }
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const float p = sm.p[warp][j][r];
#pragma unroll
                    for (int i = 0; i < PER; ++i) o[r][i] = fmaf(p, x[i], o[r][i]);
                }
            }
            __syncwarp();
        }
        // join the warps
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            float sum = l[r];
#pragma unroll
            for (int x = 16; x; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
            if (lane == 0) sm.m[warp][r] = m[r], sm.l[warp][r] = sum;
#pragma unroll
            for (int i = 0; i < PER; ++i) sm.o[warp][r][lane * PER + i] = o[r][i];
        }
        __syncthreads();
        for (int i = tid; i < rows * (D / 4); i += kSimpleThreads) {
            const int r = i / (D / 4), d0 = (i % (D / 4)) * 4;
            float top = -INFINITY;
            for (int w = 0; w < kSimpleWarps; ++w) top = fmaxf(top, sm.m[w][r]);
            top = top > -INFINITY ? top : 0.f;
            float sum = 0.f;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = 0; w < kSimpleWarps; ++w) {
                const float f = exp2f(sm.m[w][r] - top);
                sum += f * sm.l[w][r];
                const float4 y = load4(&sm.o[w][r][d0]);
                x.x = fmaf(f, y.x, x.x);
                x.y = fmaf(f, y.y, x.y);
                x.z = fmaf(f, y.z, x.z);
                x.w = fmaf(f, y.w, x.w);
            }
            const float inv = sum == 0.f ? 0.f : 1.0f / sum;
            x = make_float4(x.x * inv, x.y * inv, x.z * inv, x.w * inv);
            const float l2 = sum == 0.f ? -INFINITY : top + log2f(sum);
            if (pc.whole) {
                paged_write<T, D>(a, pc.b, pc.h, row0 + r, d0, x, l2);
            } else {
                const int64_t slot = (2 * static_cast<int64_t>(blockIdx.x) +
                                      (walk.start_of(blockIdx.x) == pc.unit0 + pc.r0 ? 0 : 1)) * NR + r;
                store4(a.part_o + slot * D + d0, x);
                if (d0 == 0) a.part_l[slot] = l2;
            }
        }
        if (pc.whole) __syncthreads();
        else paged_finish_piece<T, D, NR, kSimpleThreads>(a, walk, pc, sm.sched);
    }
}

// CTAs of a kernel that fit the current device at once (kept per kernel and device in a fixed table:
// nothing here allocates or throws).
struct GridEntry {
    const void *fn;
    int dev, ctas;
};
std::mutex g_grid_mu;
GridEntry g_grids[256];
int g_grid_count = 0;

cudaError_t resident_ctas(const void *fn, int threads, size_t smem, int *ctas) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(g_grid_mu);
    for (int i = 0; i < g_grid_count; ++i)
        if (g_grids[i].fn == fn && g_grids[i].dev == dev) {
            *ctas = g_grids[i].ctas;
            return cudaSuccess;
        }
    if ((e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem))) != cudaSuccess)
        return e;
    int sms = 0, occ = 0;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, fn, threads, smem)) != cudaSuccess) return e;
    *ctas = sms * occ;
    if (*ctas < 1) return cudaErrorInvalidConfiguration;
    if (*ctas > kMaxPagedCtas) *ctas = kMaxPagedCtas;
    if (g_grid_count < 256) g_grids[g_grid_count++] = {fn, dev, *ctas};
    return cudaSuccess;
}

template <typename K>
cudaError_t launch(K kernel, const PagedArgs &a0, int threads, size_t smem, cudaStream_t s) {
    PagedArgs a = a0;
    cudaError_t e = resident_ctas(reinterpret_cast<const void *>(kernel), threads, smem, &a.ncta);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.ncta);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename T, bool E4M3>
cudaError_t launch_simple(const PagedArgs &a, cudaStream_t s) {
    if (a.d == 128) return launch(k_paged_f32<T, E4M3, 128>, a, kSimpleThreads, sizeof(SimpleSmem<128>), s);
    return launch(k_paged_f32<T, E4M3, 64>, a, kSimpleThreads, sizeof(SimpleSmem<64>), s);
}

}  // namespace

int paged_pass_rows(int dtype, int rows) { return kSimplePass; }

cudaError_t launch_paged_attn(const PagedArgs &a, cudaStream_t s) {
    if (a.dtype == SKV_F32)
        return a.format == SKV_CACHE_E4M3 ? launch_simple<float, true>(a, s) : launch_simple<float, false>(a, s);
    return a.format == SKV_CACHE_E4M3 ? launch_simple<__nv_bfloat16, true>(a, s)
                                      : launch_simple<__nv_bfloat16, false>(a, s);
}

}  // namespace skv
