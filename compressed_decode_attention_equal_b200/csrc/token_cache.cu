// skv_cache_append and skv_cache_read: the exact-token cache written (quantising it on the way)
// and read back.
//
// An e4m3 vector is held as codes c_i = e4m3(x_i 2^-e), with the smallest e for which the largest
// finite |x_i| <= 448 2^e. A power-of-two scale keeps x_i 2^-e exact, so that a code is one rounding
// (to nearest even, at most 2^-4 relative), and c_i 2^e has 4 significant bits, so that reading it
// back into bf16 or fp32 adds none. Both kernels move every byte once: HBM bounds them, and a call
// of few tokens its launch.
#include "token_cache.cuh"

namespace skv {

namespace {

// ---------------------------------------------------------------------------
// append: a warp takes kHeads heads of one token, half of it the key and half the value, d / 16
// elements per lane
// ---------------------------------------------------------------------------
constexpr int kAppendWarps = 4;
constexpr int kHeads = 4;   // independent loads in flight per lane, and one page lookup for all of them

// two fp32 to two e4m3 codes (round to nearest even, saturating; lo in the low byte)
__device__ __forceinline__ uint32_t pack_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Smallest e with a <= 448 2^e (448 = 1.75 2^8), within the stored range; 0 for a = 0. a >= 0, finite.
__device__ __forceinline__ int scale_exponent(float a) {
    const uint32_t u = __float_as_uint(a);
    const int p = static_cast<int>(u >> 23) - 127;   // a subnormal a gives -127: below the range like its true exponent
    const int e = (u & 0x7fffffu) > 0x600000u ? p - 7 : p - 8;
    return a > 0.f ? min(max(e, kScaleExpMin), kScaleExpMax) : 0;
}

template <typename T, int N>
__device__ __forceinline__ void load_row(const T *p, uint32_t (&w)[N * sizeof(T) / 4]) {
    constexpr int W = N * sizeof(T) / 4;   // 2, 4 or 8 words, 8- or 16-byte aligned
    if constexpr (W == 2) {
        const uint2 u = *(reinterpret_cast<const uint2 *>(p));
        w[0] = u.x, w[1] = u.y;
    } else {
#pragma unroll
        for (int i = 0; i < W; i += 4) {
            const uint4 u = *(reinterpret_cast<const uint4 *>(p) + i / 4);
            w[i] = u.x, w[i + 1] = u.y, w[i + 2] = u.z, w[i + 3] = u.w;
        }
    }
}

// Tokens of sequence b, from its offsets (null: the same number for each); false if they do not
// run upwards within the n_tokens rows.
__device__ __forceinline__ bool append_count(const AppendArgs &a, int b, int *count) {
    if (!a.cu) {
        *count = a.per_seq;
        return true;
    }
    const int c0 = a.cu[b], c1 = a.cu[b + 1];
    const bool ok = c0 >= 0 && c1 >= c0 && c1 <= a.n_tokens;
    *count = ok ? c1 - c0 : 0;
    return ok;
}

template <typename T, bool E4M3, int D>
__global__ void __launch_bounds__(32 * kAppendWarps) k_cache_append(const AppendArgs a) {
    using G = CacheGeom<T, E4M3, D>;
    constexpr int N = D / 16;                     // elements per lane
    constexpr int W = N * static_cast<int>(sizeof(T)) / 4;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, half = lane >> 4, l = lane & 15;
    const int chunks = (a.Hkv + kHeads - 1) / kHeads;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
    const int64_t tok = item / chunks;
    const int h0 = static_cast<int>(item - tok * chunks) * kHeads;
    if (tok < a.n_tokens) {
        const int i = static_cast<int>(tok);
        const T *src = half ? static_cast<const T *>(a.v) + tok * a.v_token : static_cast<const T *>(a.k) + tok * a.k_token;
        const int64_t head = half ? a.v_head : a.k_head;
        uint32_t w[kHeads][W];
#pragma unroll
        for (int j = 0; j < kHeads; ++j)
            if (h0 + j < a.Hkv) load_row<T, N>(src + (h0 + j) * head + l * N, w[j]);
        // the token's sequence and position
        int b, off;
        bool ok = true;
        if (a.cu) {
            int lo = -1, hi = a.B;   // cu[lo] <= i < cu[hi] (cu[-1] = -inf, cu[B] only read below)
            while (hi - lo > 1) {
                const int m = (lo + hi) >> 1;
                if (a.cu[m] <= i) lo = m;
                else hi = m;
            }
            b = lo;
            int count = 0;
            ok = b >= 0 && append_count(a, b, &count);
            off = ok ? i - a.cu[b] : 0;
            ok = ok && off >= 0 && off < count;   // rows behind the last sequence are no one's
        } else {
            b = i / a.per_seq;
            off = i - b * a.per_seq;
        }
        if (ok) {
            const int len = a.lens[b];
            const int64_t pos = static_cast<int64_t>(len) + off;
            if (len >= 0 && pos < static_cast<int64_t>(a.max_pages) * SKV_CACHE_PAGE_TOKENS) {   // else flagged below
                const int page = a.page_table[static_cast<int64_t>(b) * a.max_pages + pos / SKV_CACHE_PAGE_TOKENS];
                if (page < 0 || page >= a.num_pages) {
                    if (lane == 0) raise_flag(a.flags, FLAG_BAD_PAGE);
                } else {
                    const int slot = static_cast<int>(pos % SKV_CACHE_PAGE_TOKENS), n = slot % kGroupTokens;
                    uint8_t *grp = a.pages + (static_cast<int64_t>(page) * a.Hkv * kPageGroups + slot / kGroupTokens) * G::kGroup;
#pragma unroll
                    for (int j = 0; j < kHeads; ++j) {
                        if (h0 + j >= a.Hkv) break;
                        uint8_t *g = grp + static_cast<int64_t>(h0 + j) * kPageGroups * G::kGroup;
                        uint8_t *row = g + half * G::kBlock + n * G::kVec;
                        if constexpr (E4M3) {
                            float x[N], top = 0.f;
#pragma unroll
                            for (int e = 0; e < N; ++e) {
                                if constexpr (sizeof(T) == 2) x[e] = e & 1 ? bf16hi(w[j][e / 2]) : bf16lo(w[j][e / 2]);
                                else x[e] = __uint_as_float(w[j][e]);
                                const float ax = fabsf(x[e]);
                                top = ax < INFINITY ? fmaxf(top, ax) : top;   // finite ones only
                            }
#pragma unroll
                            for (int s = 8; s; s >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, s));
                            const int e = scale_exponent(top);
                            const float inv = scale_of(127 - e);   // 2^-e, exact
                            uint32_t c[N / 4];
#pragma unroll
                            for (int q = 0; q < N / 4; ++q)
                                c[q] = pack_e4m3x2(x[4 * q] * inv, x[4 * q + 1] * inv) |
                                       pack_e4m3x2(x[4 * q + 2] * inv, x[4 * q + 3] * inv) << 16;
                            uint8_t *to = row + 16 * cache_chunk(l * N / 16, n, G::kChunks) + l * N % 16;
                            if constexpr (N == 8) *reinterpret_cast<uint2 *>(to) = make_uint2(c[0], c[1]);
                            else *reinterpret_cast<uint32_t *>(to) = c[0];
                            if (l == 0) g[2 * G::kBlock + half * kGroupTokens + n] = static_cast<uint8_t>(e + 127);
                        } else {
                            const int byte = l * W * 4;
                            if constexpr (W == 2) {
                                *reinterpret_cast<uint2 *>(row + 16 * cache_chunk(byte / 16, n, G::kChunks) + byte % 16) =
                                    make_uint2(w[j][0], w[j][1]);
                            } else {
#pragma unroll
                                for (int q = 0; q < W; q += 4)
                                    *reinterpret_cast<uint4 *>(row + 16 * cache_chunk(byte / 16 + q / 4, n, G::kChunks)) =
                                        make_uint4(w[j][q], w[j][q + 1], w[j][q + 2], w[j][q + 3]);
                            }
                        }
                    }
                }
            }
        }
    }
    // The CTA that finishes last writes the new lengths: new_lens may be lens itself, which every CTA
    // has read by then.
    __shared__ int s_last;
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        s_last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
        const int len = a.lens[b];
        int count;
        bool ok = append_count(a, b, &count);
        const int64_t cap = static_cast<int64_t>(a.max_pages) * SKV_CACHE_PAGE_TOKENS;
        int64_t n = static_cast<int64_t>(len) + count;
        if (len < 0 || len > cap) {
            ok = false;
            n = len;   // left as it is
        } else if (n > cap) {
            ok = false;
            n = cap;   // the tokens that fit were written
        }
        if (!ok) raise_flag(a.flags, FLAG_BAD_LENS);
        a.new_lens[b] = static_cast<int32_t>(n);
    }
    if (threadIdx.x == 0) *a.ticket = 0;   // ready for the next call
}

// ---------------------------------------------------------------------------
// read: a warp takes one group (16 tokens of one head); each lane makes 16 output bytes at a time,
// so that both sides are read and written in full lines
// ---------------------------------------------------------------------------
constexpr int kReadWarps = 8;

template <typename T, bool E4M3, int D>
__global__ void __launch_bounds__(32 * kReadWarps) k_cache_read(const ReadArgs a, const __grid_constant__ ReadTable t) {
    using G = CacheGeom<T, E4M3, D>;
    constexpr int N = 16 / static_cast<int>(sizeof(T));   // elements per lane and step
    constexpr int LPR = D / N;                            // lanes per row: 8, 16 or 32
    constexpr int RPS = 32 / LPR;                         // rows per step
    constexpr int IN = N * G::kElem;                      // cached bytes per lane and step: 4, 8 or 16
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31;
    const int64_t item64 = static_cast<int64_t>(blockIdx.x) * kReadWarps + (threadIdx.x >> 5);
    if (item64 >= a.items) return;
    const int item = static_cast<int>(item64);
    int lo = 0, hi = a.B;
    while (hi - lo > 1) {
        const int m = (lo + hi) >> 1;
        if (t.rows[m].item0 <= item) lo = m;
        else hi = m;
    }
    const int b = lo, first = t.rows[b].first, T_b = t.rows[b].T;
    const int g0 = first / kGroupTokens, groups = (first + T_b + kGroupTokens - 1) / kGroupTokens - g0;
    const int rel = item - t.rows[b].item0, h = rel / groups, gi = g0 + rel - h * groups;
    const int page = a.page_table[static_cast<int64_t>(b) * a.max_pages + gi / kPageGroups];
    const bool bad = page < 0 || page >= a.num_pages;
    if (bad && lane == 0) raise_flag(a.flags, FLAG_BAD_PAGE);
    const uint8_t *grp = a.pages + ((static_cast<int64_t>(bad ? 0 : page) * a.Hkv + h) * kPageGroups + gi % kPageGroups) * G::kGroup;
    const int64_t out0 = t.rows[b].row_off + static_cast<int64_t>(h) * T_b - first;   // + position = output row
    const int col = lane % LPR, sub = lane / LPR;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
        T *out = static_cast<T *>(kv ? a.v : a.k);
#pragma unroll
        for (int s = 0; s < kGroupTokens / RPS; ++s) {
            const int n = s * RPS + sub, pos = gi * kGroupTokens + n;
            if (pos < first || pos >= first + T_b) continue;
            const int byte = col * IN;
            const uint8_t *src = grp + kv * G::kBlock + n * G::kVec + 16 * cache_chunk(byte / 16, n, G::kChunks) + byte % 16;
            uint4 r = make_uint4(0, 0, 0, 0);
            if (!bad) {
                if constexpr (!E4M3) {
                    r = *reinterpret_cast<const uint4 *>(src);
                } else {
                    const float sc = scale_of(grp[2 * G::kBlock + kv * kGroupTokens + n]);
                    if constexpr (IN == 8) {
                        const uint2 u = *reinterpret_cast<const uint2 *>(src);
                        uint32_t o[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t wd = i < 2 ? u.x : u.y;
                            const float2 f = f16x2_to_f32(e4m3x2_to_f16x2(static_cast<uint16_t>(i & 1 ? wd >> 16 : wd)));
                            o[i] = pack_bf16x2(f.x * sc, f.y * sc);   // 4 significant bits: exact
                        }
                        r = make_uint4(o[0], o[1], o[2], o[3]);
                    } else {
                        const uint32_t wd = *reinterpret_cast<const uint32_t *>(src);
                        const float2 f0 = f16x2_to_f32(e4m3x2_to_f16x2(static_cast<uint16_t>(wd)));
                        const float2 f1 = f16x2_to_f32(e4m3x2_to_f16x2(static_cast<uint16_t>(wd >> 16)));
                        r = make_uint4(__float_as_uint(f0.x * sc), __float_as_uint(f0.y * sc),
                                       __float_as_uint(f1.x * sc), __float_as_uint(f1.y * sc));
                    }
                }
            }
            *reinterpret_cast<uint4 *>(out + (out0 + pos) * D + col * N) = r;
        }
    }
}

template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), int64_t grid, int threads, cudaStream_t s, const A &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(threads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, bool E4M3>
cudaError_t append_t(const AppendArgs &a, cudaStream_t s) {
    const int64_t items = static_cast<int64_t>(a.n_tokens) * ((a.Hkv + kHeads - 1) / kHeads);
    const int64_t grid = items > 0 ? (items + kAppendWarps - 1) / kAppendWarps : 1;   // the lengths are written at least
    return a.d == 128 ? launch(k_cache_append<T, E4M3, 128>, grid, 32 * kAppendWarps, s, a)
                      : launch(k_cache_append<T, E4M3, 64>, grid, 32 * kAppendWarps, s, a);
}

template <typename T, bool E4M3>
cudaError_t read_t(const ReadArgs &a, const ReadTable &t, cudaStream_t s) {
    const int64_t grid = (a.items + kReadWarps - 1) / kReadWarps;
    return a.d == 128 ? launch(k_cache_read<T, E4M3, 128>, grid, 32 * kReadWarps, s, a, t)
                      : launch(k_cache_read<T, E4M3, 64>, grid, 32 * kReadWarps, s, a, t);
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs &a, cudaStream_t s) {
    if (a.dtype == SKV_BF16)
        return a.format == SKV_CACHE_E4M3 ? append_t<__nv_bfloat16, true>(a, s) : append_t<__nv_bfloat16, false>(a, s);
    return a.format == SKV_CACHE_E4M3 ? append_t<float, true>(a, s) : append_t<float, false>(a, s);
}

cudaError_t launch_cache_read(const ReadArgs &a, const ReadTable &t, cudaStream_t s) {
    if (a.items == 0) return cudaSuccess;
    if (a.dtype == SKV_BF16)
        return a.format == SKV_CACHE_E4M3 ? read_t<__nv_bfloat16, true>(a, t, s) : read_t<__nv_bfloat16, false>(a, t, s);
    return a.format == SKV_CACHE_E4M3 ? read_t<float, true>(a, t, s) : read_t<float, false>(a, t, s);
}

}  // namespace skv
