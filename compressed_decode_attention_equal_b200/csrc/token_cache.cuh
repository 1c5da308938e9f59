// The exact-token cache's launch arguments, page geometry and the scheduling, joining and output code that its
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

// ---------------------------------------------------------------------------
// arguments of the launches (token_cache.cu, paged_attn.cu)
// ---------------------------------------------------------------------------
struct AppendArgs {
    const void *k, *v;                   // [n_tokens][Hkv][d], strides in elements
    int64_t k_token, k_head, v_token, v_head;
    int B, Hkv, d, dtype, format;
    int n_tokens;
    int per_seq;                         // tokens per sequence when cu is null
    int per_warp;                        // steps that one warp takes
    const int32_t *cu;                   // [B + 1] offsets of the sequences' new tokens, or null
    uint8_t *pages;
    int64_t num_pages;
    const int32_t *page_table;
    int max_pages;
    const int32_t *lens;
    int32_t *new_lens;
    uint32_t *flags;
    uint32_t *ticket;                    // CTAs done (zero between calls)
};

// What cache_read takes of each sequence, passed by value.
struct ReadRow {
    int64_t row_off;                     // first output row of the sequence
    int32_t first, T;                    // positions [first, first + T)
    int32_t item0;                       // 16-token groups (x heads) of the sequences before it
    int32_t pad;
};
struct ReadTable {
    ReadRow rows[SKV_MAX_SEQS];
};
struct ReadArgs {
    int B, Hkv, d, dtype, format;
    int items;                           // groups x heads of all sequences
    const uint8_t *pages;
    int64_t num_pages;
    const int32_t *page_table;
    int max_pages;
    void *k, *v;
    uint32_t *flags;
};

constexpr int kMaxPagedCtas = 512;       // split partials are sized for this grid
constexpr int kMaxPagedUnits = 1 << 16;  // (sequence, KV head, pass) units of one call

struct PagedArgs {
    const void *q;
    int64_t q_b, q_r, q_h;               // strides in elements
    const uint8_t *pages;
    int64_t num_pages;
    const int32_t *page_table;
    int max_pages;
    const int32_t *lens, *first;         // first may be null
    int window;                          // 0: no window
    float scale;                         // logit scale (natural units)
    float softcap;                       // 0: none
    const float *slopes;                 // [Hq] or null
    const void *prior_out;
    const float *prior_lse;              // null: no prior
    void *out;
    float *lse;
    int B, R, Hq, Hkv, G, d, dtype, format;
    float inv_G;                         // 1 / G
    int rows;                            // R * G query rows per KV head
    int pass_rows, passes;               // rows one pass over the keys serves, ceil(rows / pass_rows)
    int ncta;
    float *part_o;                       // [ncta][2][pass_rows][d] split partial outputs (normalised)
    float *part_l;                       // [ncta][2][pass_rows] their log2 partitions
    int32_t *counters;                   // pieces done: [kMaxPagedUnits], then by group of pieces [2 kMaxPagedCtas] (zero between calls)
    uint32_t *flags;
};

// Rows a pass over the keys serves for this call (paged_attn.cu chooses the kernel by it).
int paged_pass_rows(int dtype, int rows);
cudaError_t launch_cache_append(const AppendArgs &a, cudaStream_t s);
cudaError_t launch_cache_read(const ReadArgs &a, const ReadTable &t, cudaStream_t s);
cudaError_t launch_paged_attn(const PagedArgs &a, cudaStream_t s);

// ---------------------------------------------------------------------------
// page geometry
// ---------------------------------------------------------------------------
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
// into rounds of W tiles of TT tokens, one per warp; a unit without keys keeps one empty round, so
// that it is scheduled and writes its outputs like the others. A unit weighs its rounds and COST more
// (its query rows' load and its outputs take about as long as that many rounds). The weights of all
// units, in order, are dealt to the CTAs in equal contiguous ranges; a unit that a range end cuts is
// joined by the CTA that finishes its last piece, in the order of the pieces, so that the result
// does not depend on which CTA that is.
// ---------------------------------------------------------------------------
constexpr int kPieceTable = 32;   // pieces of a CTA's range that are laid out at once

// Place of a partial: a unit's pieces but the first start their CTA's range, its first ends it.
__device__ __forceinline__ int64_t paged_slot(int c0, int k) { return 2 * static_cast<int64_t>(c0 + k) + (k == 0 ? 1 : 0); }

struct PagedPiece {
    int b, h, pass;
    int r0, r1, rounds;   // rounds [r0, r1) of the unit's; r1 = r0: the range cuts only the unit's fixed weight
    int lo, hi;           // the sequence's keys
    int c0, np;           // CTA of the unit's first piece, pieces (1: this one is the whole unit)
    __device__ __forceinline__ int64_t slot(int cta) const { return paged_slot(c0, cta - c0); }
};

struct PagedSched {
    int lo[SKV_MAX_SEQS], hi[SKV_MAX_SEQS];
    long long cum[SKV_MAX_SEQS + 1];     // weight before the sequence (all its units)
    long long warp_sum[32];
    PagedPiece piece[kPieceTable];
    int unit0, n;                        // first unit of the range, pieces in the table
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

template <int W, int TT>
__device__ __forceinline__ int paged_rounds(int lo, int hi) {
    const int tiles = (hi + TT - 1) / TT - lo / TT;
    return hi > lo ? (tiles + W - 1) / W : 1;
}

// Weight before every sequence (all threads of the CTA; ends with a barrier).
template <int THREADS, int W, int TT, int COST>
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
            s.lo[b] = lo;
            s.hi[b] = hi;
            mine[i] = static_cast<long long>(paged_rounds<W, TT>(lo, hi) + COST) * mult;
        }
        sum += mine[i];
    }
    long long inc = sum;
#pragma unroll 1
    for (int o = 1; o < 32; o <<= 1) {
        const long long up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
    }
    if (lane == 31) s.warp_sum[warp] = inc;
    __syncthreads();
    long long base = inc - sum;
#pragma unroll 1
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

// Lay out pieces `from` .. `from` + 31 of this CTA's range (all threads; ends with a barrier; the caller
// puts one in front where the table is still in use). One lane per unit. With too little work fewer CTAs
// get a range. A kernel runs this code once or
// twice, so that it is kept short: instruction fetches, not arithmetic, are its time.
template <int W, int TT, int COST>
__device__ __forceinline__ void paged_pieces(const PagedArgs &a, PagedSched &s, int from) {
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x, mult = a.Hkv * a.passes;
        const long long total = s.cum[a.B];
        // as many ranges as there is weight for: with a least weight of 2 one sequence of 10,500 tokens and 2 heads (82
        // pieces a unit, or 41) takes 13.8 us, not 13.3
        const int ctas = static_cast<int>(min(static_cast<long long>(a.ncta), max(1ll, total)));
        // lanes 0 and 1: this CTA's range
        const int c = blockIdx.x + (lane & 1);
        const long long edge = c <= ctas ? total * c / ctas : total;
        const long long x0 = __shfl_sync(0xffffffffu, edge, 0), x1 = __shfl_sync(0xffffffffu, edge, 1);
        if (from == 0) {
            int l = 0, r = a.B;   // the sequence whose weight holds x0
            while (r - l > 1) {
                const int m = (l + r) >> 1;
                if (s.cum[m] <= x0) l = m;
                else r = m;
            }
            const int wt = paged_rounds<W, TT>(s.lo[l], s.hi[l]) + COST;
            if (lane == 0) s.unit0 = l * mult + static_cast<int>(x0 - s.cum[l]) / wt;   // one sequence's weight: host-checked
        }
        __syncwarp();
        const int u = s.unit0 + from + lane, b = u / mult;
        bool in = false;
        if (b < a.B && x0 < x1) {
            const int m = u - b * mult, lo = s.lo[b], hi = s.hi[b];
            const int rounds = paged_rounds<W, TT>(lo, hi), wt = rounds + COST;
            const long long at = s.cum[b] + static_cast<long long>(m) * wt;   // where the unit's weight starts
            in = at < x1;
            if (in) {
                PagedPiece p;
                p.b = b;
                p.h = m / a.passes;
                p.pass = m - p.h * a.passes;
                p.rounds = rounds;
                p.lo = lo;
                p.hi = hi;
                p.r0 = max(static_cast<int>(max(x0 - at, 0ll)) - COST, 0);
                p.r1 = max(static_cast<int>(min(x1 - at, static_cast<long long>(wt))) - COST, 0);
                p.c0 = blockIdx.x;
                p.np = 1;
                if (p.r0 > 0 || p.r1 < rounds) {
                    // CTA of weight w: the largest c with total c / ctas (rounded down) <= w
                    const long long w0 = at + COST, w1 = at + wt - 1;
                    p.c0 = static_cast<int>(((w0 + 1) * ctas - 1) / total);
                    p.np = static_cast<int>(((w1 + 1) * ctas - 1) / total) - p.c0 + 1;
                }
                s.piece[lane] = p;
            }
        }
        const uint32_t have = __ballot_sync(0xffffffffu, in);
        if (lane == 0) s.n = __popc(have);
    }
    __syncthreads();
}

// The next piece of the table at or after i that has rounds (s.n: none).
__device__ __forceinline__ int paged_next(const PagedSched &s, int i) {
    while (i < s.n && s.piece[i].r1 <= s.piece[i].r0) ++i;
    return i;
}

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
    const int rr = static_cast<int>((row + 0.5f) * a.inv_G), g = row - rr * a.G;   // row / G: exact below 2^22
    const int64_t r = (static_cast<int64_t>(b) * a.R + rr) * a.Hq + static_cast<int64_t>(h) * a.G + g;
    T *out = static_cast<T *>(a.out) + r * D + d0;
    if (a.prior_lse) {
        const float p2 = a.prior_lse[r] * 1.44269504088896340736f;
        if (p2 != -INFINITY) {   // a prior without weight is not read
            const float top = fmaxf(l2, p2);
            const float w = ex2(l2 - top), u = ex2(p2 - top), sum = w + u;   // 1 <= sum <= 2
            const float inv = __frcp_rn(sum), wi = w * inv, ui = u * inv;
            const float4 p = load4(static_cast<const T *>(a.prior_out) + r * D + d0);
            o = make_float4(wi * o.x + ui * p.x, wi * o.y + ui * p.y, wi * o.z + ui * p.z, wi * o.w + ui * p.w);
            l2 = top + __log2f(sum);
        }
    }
    store4(out, o);
    if (d0 == 0) a.lse[r] = l2 * 0.69314718055994530942f;
}

constexpr int kJoinAhead = 8;    // partial outputs that a joining thread has in flight
constexpr int kJoinWhole = 24;   // a unit's pieces that one CTA joins
constexpr int kJoinGroup = 8;    // more are joined in groups of 8, or larger ones from 256 pieces on
static_assert(kMaxPagedCtas <= 32 * 32 && kJoinWhole <= 32, "at most 32 pieces or groups are joined at once");

// Join the np <= 32 pieces k0, k0 + step, ... of one unit, into its outputs (`whole`) or into the first one's
// partial. All threads of the CTA. First the pieces' weights, 2^(l - largest l) over their sum, into `scratch` (33
// words per row; a warp per row, a lane per piece); then each thread sums four outputs of a row over the
// pieces, kJoinAhead loads in flight. The order of the sum is that of the pieces.
template <typename T, int D, int PASS, int THREADS>
__device__ __forceinline__ void paged_join(const PagedArgs &a, const PagedPiece &p, float *scratch, int k0, int step, int np, bool whole) {
    constexpr int AHEAD = kJoinAhead, WARPS = THREADS / 32, RPW = (PASS + WARPS - 1) / WARPS;   // rows per warp, together
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c0 = p.c0, row0 = p.pass * PASS;
    const int rows = min(PASS, a.rows - row0);
    const auto slot = [&](int k, int row) { return paged_slot(c0, k0 + k * step) * PASS + row; };
    float l[RPW];
#pragma unroll
    for (int i = 0; i < RPW; ++i)
        l[i] = warp + i * WARPS < rows && lane < np ? __ldcg(a.part_l + slot(lane, warp + i * WARPS)) : -INFINITY;
    const auto across = [](float x, auto op) {
#pragma unroll
        for (int o = 16; o; o >>= 1) x = op(x, __shfl_xor_sync(0xffffffffu, x, o));
        return x;
    };
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
        float top = across(l[i], [](float x, float y) { return fmaxf(x, y); });
        top = top > -INFINITY ? top : 0.f;   // no piece with a key: every weight is 2^-inf = 0
        const float w = ex2(l[i] - top), sum = across(w, [](float x, float y) { return x + y; });
        if (warp + i * WARPS < rows) {
            scratch[33 * (warp + i * WARPS) + lane] = sum == 0.f ? 0.f : w * __frcp_rn(sum);
            if (lane == 0) scratch[33 * (warp + i * WARPS) + 32] = sum == 0.f ? -INFINITY : top + __log2f(sum);   // the row's log2 partition
        }
    }
    __syncthreads();
#pragma unroll 1
    for (int i = threadIdx.x; i < rows * (D / 4); i += THREADS) {
        const int row = i / (D / 4), d0 = (i % (D / 4)) * 4;
        const float *wt = scratch + 33 * row;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int k = 0; k < np; k += AHEAD) {
            float4 v[AHEAD];
#pragma unroll
            for (int e = 0; e < AHEAD; ++e)
                v[e] = __ldcg(reinterpret_cast<const float4 *>(a.part_o + slot(min(k + e, np - 1), row) * D + d0));
#pragma unroll
            for (int e = 0; e < AHEAD; ++e) {
                const float f = wt[k + e];   // 0 behind the last piece
                o = make_float4(fmaf(f, v[e].x, o.x), fmaf(f, v[e].y, o.y), fmaf(f, v[e].z, o.z), fmaf(f, v[e].w, o.w));
            }
        }
        if (whole) {
            paged_write<T, D>(a, p.b, p.h, row0 + row, d0, o, wt[32]);
        } else {   // read before by this thread alone, the partitions before the barrier
            store4(a.part_o + slot(0, row) * D + d0, o);
            if (d0 == 0) a.part_l[slot(0, row)] = wt[32];
        }
    }
}

// Count this CTA's piece of the unit; the CTA that counts the last one joins them, whichever it is in the same
// order. More than kJoinWhole pieces are joined in two steps, each group of neighbours by the CTA that counts its
// last, so that no CTA walks along many pieces: 37 pieces of 28 rows (one sequence of 32,768 tokens, 4 heads) 37.5
// -> 33.5 us; the second step costs about 2 us, so that 20 pieces take 21.0 us in one and 22.9 in two. All threads
// of the CTA, after its partial is written.
template <typename T, int D, int PASS, int THREADS>
__device__ __forceinline__ void paged_finish_piece(const PagedArgs &a, const PagedPiece &p, PagedSched &s, float *scratch) {
    int *unit = a.counters + (static_cast<int64_t>(p.b) * a.Hkv + p.h) * a.passes + p.pass;
    const int group = max(kJoinGroup, (p.np + 31) / 32);
    bool whole = p.np <= kJoinWhole;
    int k0 = whole ? 0 : (static_cast<int>(blockIdx.x) - p.c0) / group * group, step = 1;
    int n = whole ? p.np : min(group, p.np - k0);
#pragma unroll 1
    while (true) {
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) {
            int *counter = whole ? unit : a.counters + kMaxPagedUnits + paged_slot(p.c0, k0);
            const bool last = atomicAdd(counter, 1) == n - 1;
            if (last) *counter = 0;   // ready for the next call
            s.last = last;
            __threadfence();
        }
        __syncthreads();
        if (!s.last) return;
        paged_join<T, D, PASS, THREADS>(a, p, scratch, k0, step, n, whole);
        __syncthreads();
        if (whole) return;
        whole = true;
        k0 = 0, step = group;
        n = (p.np + group - 1) / group;
    }
}

}  // namespace skv
