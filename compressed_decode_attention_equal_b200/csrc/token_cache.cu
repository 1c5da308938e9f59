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
// append: a vector is 8 elements per lane, so that a warp takes the key and value of one row (d = 128) or two
// (d = 64) at once, kHeads times that per step; the next step's loads are in flight while one is quantised, and
// the lanes look the tokens' pages up side by side. The instruction rate bounds it for long prompts (74,211 tokens
// x 4 heads of bf16 to e4m3: 40.5 us, 87% of the copy rate; without the limit of 64 registers 48): one round of
// page lookups per warp, bf16 maxima of two vectors in one word and packed products keep it there.
// ---------------------------------------------------------------------------
constexpr int kAppendWarps = 4;
constexpr int kHeads = 4;          // independent loads in flight per lane
constexpr int kLaneElems = 8;
// most steps of a warp: 2, 4, 8, 16 measured 51.5, 43.7, 45.8, 53.3 us (74,211 tokens x 4 heads). A lane looks up one
// place, so that a warp's tokens (its rows, in the flat form, 8 to a step at d = 64) are 32 at most.
constexpr int kAppendTokens = 4;

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

template <typename T, int W>
__device__ __forceinline__ void load_row(const T *p, uint32_t (&w)[W]) {   // 4 or 8 words, 16-byte aligned
#pragma unroll
    for (int i = 0; i < W; i += 4) {
        const uint4 u = *(reinterpret_cast<const uint4 *>(p) + i / 4);
        w[i] = u.x, w[i + 1] = u.y, w[i + 2] = u.z, w[i + 3] = u.w;
    }
}

// Offsets that do not all run upwards within the n_tokens rows are walked from the first one on: a sequence gets its
// rows if they run upwards and begin at or behind the end of those that the sequences before it got, so that no row
// is two sequences' and a length counts what was written. For i >= 0 the sequence that row i went to and i's place
// there, else `seq` and how many rows it got; b = -1: none.
struct Walked {
    int b, n;
};
__device__ __noinline__ Walked walk_offsets(const int32_t *cu, int B, int n_tokens, int i, int seq) {
    int end = 0;
    for (int b = 0; b < B; ++b) {
        const int c0 = cu[b], c1 = cu[b + 1];
        const bool ok = c0 >= end && c1 >= c0 && c1 <= n_tokens;
        if (i >= 0 ? ok && i >= c0 && i < c1 : b == seq) return {ok ? b : -1, ok ? (i >= 0 ? i : c1) - c0 : 0};
        if (ok) end = c1;
    }
    return {-1, 0};
}

// the larger of each bf16 pair; of a number and NaN the number
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t x, uint32_t y) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
    return r;
}

// The largest magnitude of a lane's share: a pair of bf16 (both halves to be compared yet), or the bits of an
// fp32 (which order like the magnitudes). `finite`: infinities and NaN count as zero.
template <typename T, int W>
__device__ __forceinline__ uint32_t magnitude(const uint32_t (&w)[W], bool finite) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < W; ++i) {
        if constexpr (sizeof(T) == 2) {
            uint32_t m = w[i] & 0x7fff7fffu;
            if (finite) m = ((m & 0xffffu) < 0x7f80u ? m & 0xffffu : 0u) | ((m >> 16) < 0x7f80u ? m & 0xffff0000u : 0u);
            top = max_bf16x2(top, m);
        } else {
            const uint32_t m = w[i] & 0x7fffffffu;
            top = max(top, finite && m >= 0x7f800000u ? 0u : m);
        }
    }
    return top;
}

// Scale exponents of kHeads vectors, each spread over LANES lanes that agree on it; the whole warp takes part.
// bf16 magnitudes are reduced two vectors to a word. FINITE false: one over all elements, false if some vector
// holds an infinity (a bf16 NaN is passed over, an fp32 one counts as an infinity).
template <typename T, int W, int LANES, bool FINITE>
__device__ __forceinline__ bool scale_exponents(const uint32_t (&w)[kHeads][W], int (&e)[kHeads]) {
    constexpr bool PAIRS = sizeof(T) == 2;
    constexpr int REGS = PAIRS ? kHeads / 2 : kHeads;
    uint32_t r[REGS];
#pragma unroll
    for (int i = 0; i < REGS; ++i) {
        if constexpr (PAIRS) {
            const uint32_t x = magnitude<T, W>(w[2 * i], FINITE), y = magnitude<T, W>(w[2 * i + 1], FINITE);
            r[i] = max_bf16x2(__byte_perm(x, y, 0x5410), __byte_perm(x, y, 0x7632));
        } else {
            r[i] = magnitude<T, W>(w[i], FINITE);
        }
    }
#pragma unroll
    for (int s = LANES / 2; s; s >>= 1)
#pragma unroll
        for (int i = 0; i < REGS; ++i) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, r[i], s);
            r[i] = PAIRS ? max_bf16x2(r[i], other) : max(r[i], other);
        }
    bool inf = false;
#pragma unroll
    for (int j = 0; j < kHeads; ++j) {
        const uint32_t bits = !PAIRS ? r[j % REGS] : j & 1 ? r[j / 2] & 0xffff0000u : r[j / 2] << 16;
        inf |= bits >= 0x7f800000u;
        e[j] = scale_exponent(__uint_as_float(bits));
    }
    return FINITE || !__any_sync(0xffffffffu, inf);
}

// One vector's share of a lane times 2^-e (exact) to e4m3 codes.
template <typename T, int N, int W>
__device__ __forceinline__ void quantise(const uint32_t (&w)[W], int e, uint32_t (&c)[N / 4]) {
    const float inv = scale_of(127 - e);
    const uint64_t inv2 = f2pack(inv, inv);
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
        float x[4];
        if constexpr (sizeof(T) == 2) {
            x[0] = bf16lo(w[2 * q]), x[1] = bf16hi(w[2 * q]), x[2] = bf16lo(w[2 * q + 1]), x[3] = bf16hi(w[2 * q + 1]);
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(w[4 * q + i]);
        }
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
            uint64_t y;
            asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(f2pack(x[i], x[i + 1])), "l"(inv2));
            f2unpack(y, x[i], x[i + 1]);
        }
        c[q] = pack_e4m3x2(x[0], x[1]) | pack_e4m3x2(x[2], x[3]) << 16;
    }
}

// FLAT false: a step is that many heads of one token. FLAT true: as many consecutive (token, head) rows, whatever
// their tokens; for head counts that do not fill steps (74,211 tokens x 1 head 26.4 us instead of 56.8; 4 heads
// would take 44.6 instead of 40.1 with a lookup per row).
template <typename T, bool E4M3, int D, bool FLAT>
__global__ void __launch_bounds__(32 * kAppendWarps, sizeof(T) == 2 ? 8 : 4) k_cache_append(const AppendArgs a) {
    using G = CacheGeom<T, E4M3, D>;
    constexpr int N = kLaneElems, W = N * static_cast<int>(sizeof(T)) / 4;
    constexpr int LANES = D / N, SUBS = 32 / (2 * LANES);   // lanes of a vector, rows side by side
    constexpr int ROWS = kHeads * SUBS;                     // rows of a step
    static_assert(kAppendTokens * (FLAT ? ROWS : 1) <= 32, "a lane per place");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, sub = lane / (2 * LANES), half = lane / LANES & 1, l = lane % LANES;
    const unsigned item = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    // this warp: tokens i0 .. i0 + count - 1, heads h0 .. h0 + ROWS - 1; or (FLAT) rows i0 .. i0 + count - 1.
    // n_tokens * Hkv fits 32 bits (checked on the host); items may reach a little beyond, so 64 here.
    int64_t i0;
    int h0 = 0, count;
    if constexpr (FLAT) {
        i0 = static_cast<int64_t>(item) * (a.per_warp * ROWS);
        count = static_cast<int>(max(min(static_cast<int64_t>(a.per_warp * ROWS), static_cast<int64_t>(a.n_tokens) * a.Hkv - i0), int64_t{0}));
    } else {
        const unsigned chunks = a.Hkv / ROWS, part = item / chunks;
        h0 = static_cast<int>(item - part * chunks) * ROWS;
        i0 = static_cast<int64_t>(part) * a.per_warp;
        count = static_cast<int>(max(min(static_cast<int64_t>(a.per_warp), a.n_tokens - i0), int64_t{0}));
    }
    const int steps = FLAT ? (count + ROWS - 1) / ROWS : count;
    const int64_t token_stride = half ? a.v_token : a.k_token, head_stride = half ? a.v_head : a.k_head;
    // where this lane loads next; FLAT walks over the rows i0 + sub, i0 + sub + SUBS, ...
    const T *src = (half ? static_cast<const T *>(a.v) : static_cast<const T *>(a.k)) + l * N;
    int hd = h0 + sub;
    if constexpr (FLAT) {
        const int64_t tk = (i0 + sub) / a.Hkv;
        hd = static_cast<int>(i0 + sub - tk * a.Hkv);
        src += tk * token_stride + hd * head_stride;
    } else {
        src += i0 * token_stride + hd * head_stride;
    }
    const auto load_step = [&](int t, uint32_t (&w)[kHeads][W]) {
        if (t >= steps) return;
#pragma unroll
        for (int j = 0; j < kHeads; ++j) {
            if constexpr (FLAT) {
                if (t * ROWS + j * SUBS + sub < count) load_row<T, W>(src, w[j]);
                src += SUBS * head_stride;
                for (hd += SUBS; hd >= a.Hkv; hd -= a.Hkv) src += token_stride - a.Hkv * head_stride;
            } else {
                load_row<T, W>(src + j * SUBS * head_stride, w[j]);
            }
        }
        if constexpr (!FLAT) src += token_stride;
    };
    uint32_t next[kHeads][W] = {};
    load_step(0, next);
    bool down = false;   // offsets that do not run upwards within the rows
    if (a.cu)
        for (int b = threadIdx.x; b <= a.B; b += 32 * kAppendWarps)
            down |= a.cu[b] < (b > 0 ? a.cu[b - 1] : 0) || a.cu[b] > a.n_tokens;
    // lane t: the group that token (row) t goes to (-1: none; the first head's) and its slot there
    int where = -1, slot16 = 0, i = 0, head = h0;
    bool bad_page = false;
    const auto place = [&](int b, int off) {
        const int len = a.lens[b];
        const int64_t pos = static_cast<int64_t>(len) + off;
        if (len < 0 || pos >= static_cast<int64_t>(a.max_pages) * SKV_CACHE_PAGE_TOKENS) return;   // flagged below
        const int page = a.page_table[static_cast<int64_t>(b) * a.max_pages + pos / SKV_CACHE_PAGE_TOKENS];
        const int slot = static_cast<int>(pos) % SKV_CACHE_PAGE_TOKENS;
        slot16 = slot % kGroupTokens;
        bad_page = page < 0 || page >= a.num_pages;
        if (!bad_page) where = (page * a.Hkv + head) * kPageGroups + slot / kGroupTokens;   // fits: checked on the host
    };
    if (lane < count) {
        i = static_cast<int>(FLAT ? (i0 + lane) / a.Hkv : i0 + lane);
        if constexpr (FLAT) head = static_cast<int>(i0 + lane - static_cast<int64_t>(i) * a.Hkv);
        if (a.cu) {
            int lo = -1, hi = a.B;   // cu[lo] <= i < cu[hi] (cu[-1] = -inf)
            while (hi - lo > 1) {
                const int m = (lo + hi) >> 1;
                if (a.cu[m] <= i) lo = m;
                else hi = m;
            }
            if (lo >= 0 && i < a.cu[lo + 1]) place(lo, i - a.cu[lo]);   // rows behind the last sequence are no one's
        } else {
            const int b = i / a.per_seq;
            place(b, i - b * a.per_seq);
        }
    }
    const bool walk = __syncthreads_or(down);
    if (walk) {
        where = -1;
        bad_page = false;
        if (lane < count) {
            const Walked at = walk_offsets(a.cu, a.B, a.n_tokens, i, 0);
            if (at.b >= 0) place(at.b, at.n);
        }
        __syncthreads();
    }
    if (bad_page) raise_flag(a.flags, FLAG_BAD_PAGE);
    // The CTA that comes last to this point writes the new lengths: new_lens may be lens itself, which every
    // CTA has read by then (here and not at the end, so that no warp waits for the others' tokens).
    __shared__ int s_last;
    if (threadIdx.x == 0) {
        __threadfence();
        s_last = atomicAdd(a.ticket, 1u) == gridDim.x - 1;
        if (s_last) *a.ticket = 0;   // ready for the next call
    }
    __syncthreads();
    if (s_last) {
        for (int b = threadIdx.x; b < a.B; b += blockDim.x) {
            const int len = a.lens[b];
            int n = a.per_seq;
            bool ok = true;
            if (walk) {
                const Walked got = walk_offsets(a.cu, a.B, a.n_tokens, -1, b);
                ok = got.b >= 0;
                n = got.n;
            } else if (a.cu) {
                n = a.cu[b + 1] - a.cu[b];
            }
            const int64_t cap = static_cast<int64_t>(a.max_pages) * SKV_CACHE_PAGE_TOKENS;
            int64_t to = static_cast<int64_t>(len) + n;
            if (len < 0 || len > cap) {
                ok = false;
                to = len;   // left as it is
            } else if (to > cap) {
                ok = false;
                to = cap;   // the tokens that fit are written
            }
            if (!ok) raise_flag(a.flags, FLAG_BAD_LENS);
            a.new_lens[b] = static_cast<int32_t>(to);
        }
    }
#pragma unroll 1
    for (int t = 0; t < steps; ++t) {
        uint32_t w[kHeads][W];
#pragma unroll
        for (int j = 0; j < kHeads; ++j)
#pragma unroll
            for (int q = 0; q < W; ++q) w[j][q] = next[j][q];
        load_step(t + 1, next);
        int group = 0, n = 0;
        if constexpr (!FLAT) {
            group = __shfl_sync(0xffffffffu, where, t);
            if (group < 0) continue;
            n = __shfl_sync(0xffffffffu, slot16, t);
        }
        int e[kHeads];
        if constexpr (E4M3)
            if (!scale_exponents<T, W, LANES, false>(w, e)) scale_exponents<T, W, LANES, true>(w, e);
        uint8_t *grp = a.pages + (static_cast<int64_t>(group) + sub * kPageGroups) * G::kGroup;
#pragma unroll
        for (int j = 0; j < kHeads; ++j) {
            if constexpr (FLAT) {
                const int r = (t * ROWS + j * SUBS + sub) & 31;
                group = __shfl_sync(0xffffffffu, where, r);
                n = __shfl_sync(0xffffffffu, slot16, r);
                if (group < 0) continue;   // rows behind the last one among them
                grp = a.pages + static_cast<int64_t>(group) * G::kGroup;
            }
            uint8_t *row = grp + half * G::kBlock + n * G::kVec;
            uint8_t *exps = grp + 2 * G::kBlock + half * kGroupTokens + n;
            if constexpr (!FLAT) grp += SUBS * kPageGroups * G::kGroup;   // the next heads
            if constexpr (E4M3) {
                uint32_t c[N / 4];
                quantise<T, N, W>(w[j], e[j], c);
                *reinterpret_cast<uint2 *>(row + 16 * cache_chunk(l * N / 16, n, G::kChunks) + l * N % 16) = make_uint2(c[0], c[1]);
                if (l == 0) *exps = static_cast<uint8_t>(e[j] + 127);
            } else {
#pragma unroll
                for (int q = 0; q < W; q += 4)
                    *reinterpret_cast<uint4 *>(row + 16 * cache_chunk((l * W + q) / 4, n, G::kChunks)) =
                        make_uint4(w[j][q], w[j][q + 1], w[j][q + 2], w[j][q + 3]);
            }
        }
    }
}

// ---------------------------------------------------------------------------
// read: a warp takes one group (16 tokens of one head); each lane makes 16 output bytes at a time, so that
// both sides are read and written in full lines. All of a group's loads are issued before the first
// conversion: 148,706 tokens x 4 heads of e4m3 to bf16 take 73.3 us (97% of the copy rate), 106 us when
// each step waited for its own.
// ---------------------------------------------------------------------------
constexpr int kReadWarps = 8;

template <typename T, bool E4M3, int D>
__global__ void __launch_bounds__(32 * kReadWarps) k_cache_read(const ReadArgs a, const __grid_constant__ ReadTable t) {
    using G = CacheGeom<T, E4M3, D>;
    constexpr int N = 16 / static_cast<int>(sizeof(T));   // elements per lane and step
    constexpr int LPR = D / N;                            // lanes per row: 8, 16 or 32
    constexpr int RPS = 32 / LPR;                         // rows per step
    constexpr int IN = N * G::kElem / 4;                  // cached words per lane and step: 1, 2 or 4
    constexpr int STEPS = kGroupTokens / RPS;             // 4, 8 or 16
    constexpr int BATCH = IN * STEPS <= 16 ? STEPS : 16 / IN;   // steps whose loads are in flight, keys and values each
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
    const uint8_t *grp = a.pages + ((static_cast<int64_t>(page) * a.Hkv + h) * kPageGroups + gi % kPageGroups) * G::kGroup;
    const int64_t row0 = t.rows[b].row_off + static_cast<int64_t>(h) * T_b - first + gi * kGroupTokens;   // of the group's first token
    const int col = lane % LPR, sub = lane / LPR, byte = col * IN * 4;
    // lane: exponent byte of key `lane`, or of value `lane` - 16
    uint32_t scales = 0;
    if constexpr (E4M3) scales = bad ? 0u : grp[2 * G::kBlock + lane];
#pragma unroll
    for (int s0 = 0; s0 < STEPS; s0 += BATCH) {
        uint32_t w[2][BATCH][IN];
#pragma unroll
        for (int kv = 0; kv < 2; ++kv)
#pragma unroll
            for (int s = 0; s < BATCH; ++s) {
                const int n = (s0 + s) * RPS + sub;
                const uint8_t *src = grp + kv * G::kBlock + n * G::kVec + 16 * cache_chunk(byte / 16, n, G::kChunks) + byte % 16;
#pragma unroll
                for (int i = 0; i < IN; ++i) w[kv][s][i] = 0;
                if (!bad) {
                    if constexpr (IN == 4) {
                        const uint4 u = *reinterpret_cast<const uint4 *>(src);
                        w[kv][s][0] = u.x, w[kv][s][1] = u.y, w[kv][s][2] = u.z, w[kv][s][3] = u.w;
                    } else if constexpr (IN == 2) {
                        const uint2 u = *reinterpret_cast<const uint2 *>(src);
                        w[kv][s][0] = u.x, w[kv][s][1] = u.y;
                    } else {
                        w[kv][s][0] = *reinterpret_cast<const uint32_t *>(src);
                    }
                }
            }
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
            T *out = static_cast<T *>(kv ? a.v : a.k) + row0 * D + col * N;
#pragma unroll
            for (int s = 0; s < BATCH; ++s) {
                const int n = (s0 + s) * RPS + sub, pos = gi * kGroupTokens + n;
                uint32_t r[4];
                if constexpr (!E4M3) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) r[i] = w[kv][s][i % IN];
                } else {
                    const float sc = scale_of(__shfl_sync(0xffffffffu, scales, kv * kGroupTokens + n));
#pragma unroll
                    for (int i = 0; i < IN; ++i) {
                        const float2 f0 = f16x2_to_f32(e4m3x2_to_f16x2(static_cast<uint16_t>(w[kv][s][i])));
                        const float2 f1 = f16x2_to_f32(e4m3x2_to_f16x2(static_cast<uint16_t>(w[kv][s][i] >> 16)));
                        if constexpr (sizeof(T) == 2) {   // 4 significant bits: exact
                            r[2 * i] = pack_bf16x2(f0.x * sc, f0.y * sc);
                            r[2 * i + 1] = pack_bf16x2(f1.x * sc, f1.y * sc);
                        } else {
                            r[0] = __float_as_uint(f0.x * sc), r[1] = __float_as_uint(f0.y * sc);
                            r[2] = __float_as_uint(f1.x * sc), r[3] = __float_as_uint(f1.y * sc);
                        }
                    }
                }
                if (pos >= first && pos < first + T_b)
                    *reinterpret_cast<uint4 *>(out + static_cast<int64_t>(n) * D) = make_uint4(r[0], r[1], r[2], r[3]);
            }
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

template <typename T, bool E4M3, int D>
cudaError_t append_d(const AppendArgs &a0, cudaStream_t s) {
    AppendArgs a = a0;
    constexpr int ROWS = kHeads * (128 / D);   // rows of a step
    const bool flat = a.Hkv % ROWS != 0;
    const int64_t rows = static_cast<int64_t>(a.n_tokens) * a.Hkv, all = (rows + ROWS - 1) / ROWS;   // steps
    // steps of a warp: one while there are not enough warps for the GPU (148 SMs, 32 warps each)
    const int64_t per = all / (148 * 32);
    a.per_warp = static_cast<int>(per < 1 ? 1 : per > kAppendTokens ? kAppendTokens : per);
    const int64_t items = flat ? (all + a.per_warp - 1) / a.per_warp
                               : (a.n_tokens + a.per_warp - 1) / a.per_warp * static_cast<int64_t>(a.Hkv / ROWS);
    const int64_t grid = items > 0 ? (items + kAppendWarps - 1) / kAppendWarps : 1;   // the lengths are written at least
    return flat ? launch(k_cache_append<T, E4M3, D, true>, grid, 32 * kAppendWarps, s, a)
                : launch(k_cache_append<T, E4M3, D, false>, grid, 32 * kAppendWarps, s, a);
}

template <typename T, bool E4M3>
cudaError_t append_t(const AppendArgs &a, cudaStream_t s) {
    return a.d == 128 ? append_d<T, E4M3, 128>(a, s) : append_d<T, E4M3, 64>(a, s);
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
