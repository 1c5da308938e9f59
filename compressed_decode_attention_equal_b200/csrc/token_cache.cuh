// The exact-token cache's page geometry and the scheduling, joining and output code that its
// attention kernels share.
//
// A page holds 64 tokens of one sequence for all its KV heads, [Hkv][4][group]; a group holds 16
// tokens of one head, K[16][d] | V[16][d] in the inputs' type (SKV_CACHE_RAW) or as e4m3 codes
// followed by one exponent byte per key and per value (SKV_CACHE_E4M3). A group is one contiguous
// block, so that a kernel fetches it with one bulk copy.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "skv.h"
#include "skv_common.cuh"
#include "skv_internal.h"

namespace skv {

constexpr int kGroupTokens = 16;
constexpr int kPageGroups = SKV_CACHE_PAGE_TOKENS / kGroupTokens;
constexpr int kScaleExpMin = -100, kScaleExpMax = 119;   // scale exponents of an e4m3 row

// Where the 16-byte chunk c of slot n's vector is stored (`chunks` 16-byte chunks per vector, a
// power of two >= 4). The attention kernel's key loads take four neighbouring chunks of two
// neighbouring slots at once and its value loads two chunks of four slots two apart; this
// permutation sends both sets to different banks.
__host__ __device__ __forceinline__ int cache_chunk(int c, int n, int chunks) {
    return c ^ (((n & 6) ^ ((n & 1) << 2)) & (chunks - 1));
}

// Element type, vector and group sizes of one cache format.
template <typename T, bool E4M3, int D>
struct CacheGeom {
    static constexpr int kElem = E4M3 ? 1 : static_cast<int>(sizeof(T));
    static constexpr int kVec = D * kElem;                 // bytes of one key or value
    static constexpr int kChunks = kVec / 16;
    static constexpr int kBlock = kGroupTokens * kVec;     // keys (or values) of a group
    static constexpr int kGroup = 2 * kBlock + (E4M3 ? 2 * kGroupTokens : 0);
};

// 2^(byte - 127), the scale that an exponent byte stands for (stored bytes are 27 .. 246)
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// 4 e4m3 codes of one 32-bit word to fp32
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t w) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(w));
    return r;
}

__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// 16 bytes of a cached vector to fp32: 4 (fp32), 8 (bf16) or 16 (e4m3) values
template <typename T, bool E4M3>
struct ChunkValues {
    static constexpr int N = E4M3 ? 16 : 16 / static_cast<int>(sizeof(T));
    __device__ static __forceinline__ void get(const uint4 &u, float (&x)[N]) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (E4M3) {
                const float2 a = f16x2_to_f32(e4m3x2_to_f16x2(static_cast<uint16_t>(w[i])));
                const float2 b = f16x2_to_f32(e4m3x2_to_f16x2(static_cast<uint16_t>(w[i] >> 16)));
                x[4 * i] = a.x, x[4 * i + 1] = a.y, x[4 * i + 2] = b.x, x[4 * i + 3] = b.y;
            } else if constexpr (sizeof(T) == 2) {
                x[2 * i] = bf16lo(w[i]), x[2 * i + 1] = bf16hi(w[i]);
            } else {
                x[i] = __uint_as_float(w[i]);
            }
        }
    }
};

// ---------------------------------------------------------------------------
// attention: which CTA reads which tokens
//
// A unit is one (sequence, KV head, pass over at most PASS query rows). Its keys [lo, hi) are cut
// into rounds of RG token groups (one CTA-wide step); a unit without keys keeps one empty round, so
// that it is scheduled and writes its outputs like the others. All rounds of all units, in order,
// are dealt to the CTAs in equal contiguous ranges; a unit that a range end cuts is joined by the CTA
// that finishes its last piece, in the order of the pieces, so that the result does not depend on
// which CTA that is.
// ---------------------------------------------------------------------------
struct PagedSched {
    int lo[SKV_MAX_SEQS], hi[SKV_MAX_SEQS];
    int rounds[SKV_MAX_SEQS];            // rounds of one unit of the sequence
    long long cum[SKV_MAX_SEQS + 1];     // rounds before the sequence (all its units)
    long long warp_sum[32];
    int last;                            // this CTA completed the unit
};

__device__ __forceinline__ void paged_range(const PagedArgs &a, int b, bool report, int *lo, int *hi) {
    int n = a.lens[b];
    const int cap = a.max_pages * SKV_CACHE_PAGE_TOKENS;
    if (n < 0 || n > cap) {
        if (report) raise_flag(a.flags, FLAG_BAD_LENS);
        n = n < 0 ? 0 : cap;
    }
    int f = a.first ? a.first[b] : 0;
    f = f < 0 ? 0 : f;
    if (a.window > 0 && n - a.window > f) f = n - a.window;
    *lo = f < n ? f : n;
    *hi = n;
}

// Fill the schedule (all threads of the CTA; ends with a barrier).
template <int THREADS, int RG>
__device__ __forceinline__ void paged_schedule(const PagedArgs &a, PagedSched &s) {
    constexpr int PER = (SKV_MAX_SEQS + THREADS - 1) / THREADS;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int mult = a.Hkv * a.passes;
    long long mine[PER], sum = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = tid * PER + i;
        mine[i] = 0;
        if (b < a.B) {
            int lo, hi;
            paged_range(a, b, blockIdx.x == 0, &lo, &hi);
            const int g0 = lo / kGroupTokens, g1 = (hi + kGroupTokens - 1) / kGroupTokens;
            const int r = hi > lo ? (g1 - g0 + RG - 1) / RG : 1;
            s.lo[b] = lo;
            s.hi[b] = hi;
            s.rounds[b] = r;
            mine[i] = static_cast<long long>(r) * mult;
        }
        sum += mine[i];
    }
    long long inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
    }
    if (lane == 31) s.warp_sum[warp] = inc;
    __syncthreads();
    long long base = inc - sum;
    for (int w = 0; w < warp; ++w) base += s.warp_sum[w];
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = tid * PER + i;
        if (b < a.B) s.cum[b] = base;
        base += mine[i];
        if (b == a.B - 1) s.cum[a.B] = base;
    }
    __syncthreads();
}

// One piece of a unit: rounds [r0, r1) of unit (b, h, pass).
struct PagedPiece {
    int b, h, pass;
    int r0, r1, rounds;
    long long unit0;   // first round of the unit, counted over all units
    bool whole;        // the piece is the whole unit
};

// A CTA's walk over its range of rounds.
struct PagedWalk {
    long long x, end, total;
    int ctas;   // CTAs that get a range
    int b;

    __device__ __forceinline__ long long start_of(int c) const { return total * c / ctas; }
    __device__ __forceinline__ int cta_of(long long round) const {
        return static_cast<int>(((round + 1) * ctas - 1) / total);
    }
    __device__ __forceinline__ void begin(const PagedArgs &a, const PagedSched &s) {
        total = s.cum[a.B];
        ctas = total < a.ncta ? static_cast<int>(total) : a.ncta;
        const int c = blockIdx.x;
        x = c < ctas ? start_of(c) : 0;
        end = c < ctas ? start_of(c + 1) : 0;
        int l = 0, r = a.B;   // the sequence whose rounds hold x
        while (r - l > 1) {
            const int m = (l + r) >> 1;
            if (s.cum[m] <= x) l = m;
            else r = m;
        }
        b = l;
    }
    __device__ __forceinline__ bool next(const PagedArgs &a, const PagedSched &s, PagedPiece *p) {
        if (x >= end) return false;
        while (s.cum[b + 1] <= x) ++b;
        const int r = s.rounds[b];
        const int rem = static_cast<int>(x - s.cum[b]);   // < rounds x heads x passes of one sequence: checked on the host
        const int m = rem / r;
        p->b = b;
        p->h = m / a.passes;
        p->pass = m - p->h * a.passes;
        p->rounds = r;
        p->r0 = rem - m * r;
        p->unit0 = x - p->r0;
        p->r1 = end - x < r - p->r0 ? p->r0 + static_cast<int>(end - x) : r;
        p->whole = p->r0 == 0 && p->r1 == r;
        x += p->r1 - p->r0;
        return true;
    }
};

// ---------------------------------------------------------------------------
// attention: outputs and the join of a unit's pieces
// ---------------------------------------------------------------------------
__device__ __forceinline__ void store4(float *p, const float4 &v) { *reinterpret_cast<float4 *>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float4 &v) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}
__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 u = *reinterpret_cast<const uint2 *>(p);
    return make_float4(bf16lo(u.x), bf16hi(u.x), bf16lo(u.y), bf16hi(u.y));
}

// Write four outputs of one query row (o normalised, l2 its log2 partition; no key seen: l2 = -inf
// and o = 0), joined with the prior attention's if there is one: both weights are 2^(l - joint),
// at most 1, so that neither partition can overflow.
template <typename T, int D>
__device__ __forceinline__ void paged_write(const PagedArgs &a, int b, int h, int row, int d0, float4 o, float l2) {
    const int rr = row / a.G, g = row - rr * a.G;
    const int64_t r = (static_cast<int64_t>(b) * a.R + rr) * a.Hq + static_cast<int64_t>(h) * a.G + g;
    T *out = static_cast<T *>(a.out) + r * D + d0;
    if (a.prior_lse) {
        const float p2 = a.prior_lse[r] * 1.44269504088896340736f;
        if (p2 != -INFINITY) {   // a prior without weight is not read
            const float top = fmaxf(l2, p2);
            const float w = exp2f(l2 - top), u = exp2f(p2 - top);
            const float inv = 1.0f / (w + u);
            const float4 p = load4(static_cast<const T *>(a.prior_out) + r * D + d0);
            o.x = (w * o.x + u * p.x) * inv;
            o.y = (w * o.y + u * p.y) * inv;
            o.z = (w * o.z + u * p.z) * inv;
            o.w = (w * o.w + u * p.w) * inv;
            l2 = top + log2f(w + u);
        }
    }
    store4(out, o);
    if (d0 == 0) a.lse[r] = l2 * 0.69314718055994530942f;
}

// Join the pieces of one unit (in their order) and write its outputs. All threads of the CTA.
template <typename T, int D, int PASS, int THREADS>
__device__ __forceinline__ void paged_join(const PagedArgs &a, const PagedWalk &w, const PagedPiece &p) {
    const int c0 = w.cta_of(p.unit0), c1 = w.cta_of(p.unit0 + p.rounds - 1);
    const int slot0 = 2 * c0 + (w.start_of(c0) == p.unit0 ? 0 : 1);   // the others start their CTA's range
    const int rows = min(PASS, a.rows - p.pass * PASS);
    for (int i = threadIdx.x; i < rows * (D / 4); i += THREADS) {
        const int row = i / (D / 4), d0 = (i % (D / 4)) * 4;
        float top = -INFINITY;
        for (int c = c0; c <= c1; ++c)
            top = fmaxf(top, __ldcg(a.part_l + static_cast<int64_t>(c == c0 ? slot0 : 2 * c) * PASS + row));
        top = top > -INFINITY ? top : 0.f;   // no piece with a key: every weight is 2^-inf = 0
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        float sum = 0.f;
#pragma unroll 4
        for (int c = c0; c <= c1; ++c) {
            const int64_t slot = static_cast<int64_t>(c == c0 ? slot0 : 2 * c) * PASS + row;
            const float f = exp2f(__ldcg(a.part_l + slot) - top);
            const float4 v = __ldcg(reinterpret_cast<const float4 *>(a.part_o + slot * D + d0));
            sum += f;
            o.x = fmaf(f, v.x, o.x);
            o.y = fmaf(f, v.y, o.y);
            o.z = fmaf(f, v.z, o.z);
            o.w = fmaf(f, v.w, o.w);
        }
        const float inv = sum == 0.f ? 0.f : 1.0f / sum;
        o = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
        paged_write<T, D>(a, p.b, p.h, p.pass * PASS + row, d0, o, sum == 0.f ? -INFINITY : top + log2f(sum));
    }
}

// Count this CTA's piece of the unit; the CTA that counts the last one joins them. All threads
// of the CTA, after its partial is written.
template <typename T, int D, int PASS, int THREADS>
__device__ __forceinline__ void paged_finish_piece(const PagedArgs &a, const PagedWalk &w, const PagedPiece &p,
                                                   PagedSched &s) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        const int pieces = w.cta_of(p.unit0 + p.rounds - 1) - w.cta_of(p.unit0) + 1;
        int *counter = a.counters + (static_cast<int64_t>(p.b) * a.Hkv + p.h) * a.passes + p.pass;
        const bool last = atomicAdd(counter, 1) == pieces - 1;
        if (last) *counter = 0;   // ready for the next call
        s.last = last;
        __threadfence();
    }
    __syncthreads();
    if (s.last) paged_join<T, D, PASS, THREADS>(a, w, p);
    __syncthreads();
}

}  // namespace skv
