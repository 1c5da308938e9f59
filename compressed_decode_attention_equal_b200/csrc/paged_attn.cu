// skv_paged_attn: attention of the new token's query rows over the exact-token cache.
//
// One launch: every CTA takes an equal share of the token groups of all (sequence, KV head) units, its warps
// stream the groups through private rings of bulk copies and keep their own running maximum, sum and outputs;
// they join at the end of a unit's piece, and the CTA that ends a unit's last piece joins the pieces. Two
// kernels on that frame: k_paged_mma (bf16 queries, tensor cores) and k_paged_f32 (fp32 queries, exact fp32 FMAs).
#include <mutex>

#include "token_cache.cuh"

namespace skv {

namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kSlack = 8.f;                  // 2^8 times a value's scale, 2^119 at most, stays within fp32
constexpr float kRaise = 7.f;                  // a weight is at most 2^(kSlack + kRaise), half of what fp16 holds
constexpr float kSpan = 126.f;                 // 2^126 stays finite, and 2^-126 is the smallest normal output
constexpr float kNoLogit = -3.402823466e38f;   // no maximum yet: finite, so that a masked logit (-inf) less it is not NaN

// log2(e) c tanh(x / c), relative to itself 2^-20 or better for every c: up to |x / c| = 1/4 x times the series of
// tanh(u) / u (the next term is 2^-26), so that no difference of numbers near 1 enters a small logit whatever the cap;
// above it tanh u = 1 - 2 / (e^(2u) + 1), whose absolute error is a few ulps of 1. (The hardware's tanh is 2^-11 off.)
struct SoftCap {
    float inv, cap;   // 1 / c and log2(e) c
    __device__ __forceinline__ explicit SoftCap(float c) : inv(fminf(1.0f / c, 3.402823466e38f)), cap(c * kLog2e) {}
    __device__ __forceinline__ float near(float x, float u) const {
        const float w = u * u;
        const float t = fmaf(w, fmaf(w, fmaf(w, fmaf(w, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f), 1.0f);
        return x * kLog2e * t;
    }
    __device__ __forceinline__ float far(float u) const {
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(ex2(u * (2.0f * kLog2e)) + 1.0f));
        return fmaf(-2.0f * cap, r, cap);
    }
};

// ---------------------------------------------------------------------------
// bf16 queries: tensor cores
// ---------------------------------------------------------------------------
// Shared memory of k_paged_mma<E4M3, D, NT, W, S, CTAS, TP>: per warp a ring of S token groups, each one bulk
// copy; the pass's query rows; the warps' outputs at the end of a piece.
template <bool E4M3, int D, int NT, int W, int S, int CTAS, int TP>
struct MmaSmem {
    using G = CacheGeom<__nv_bfloat16, E4M3, D>;
    static constexpr int kStage = (TP * G::kGroup + 127) / 128 * 128;
    static constexpr int kRows = 8 * NT;
    // rounds that a unit's query load and outputs take as long as: 1, 2, 3 measured 90.3, 72.4, 73.3 us with one row
    // (64 ragged sequences x 16 heads), and 1, 2, 3, 4 with 28 rows 58.4, 48.8, 49.8, 47.7 us (48 x 4 heads)
    static constexpr int kCost = NT == 1 ? 2 : 4;
    static constexpr int kQRow = 2 * D + 8;      // bytes of a query row: 8 more than 2 D against bank conflicts
    static constexpr int kMerge = 33;            // words per accumulator element of a warp's 32 lanes
    static constexpr int kMaxCtas = CTAS * 160;
    static constexpr int kTurn = NT < 2 ? NT : 2;   // tiles of 8 rows that the warps join at once
    static constexpr int kOut = kTurn * W * 4 * (D / 16) * kMerge;
    static constexpr int kJoin = kRows * 33;     // the join of a unit's pieces keeps their weights in o
    alignas(128) uint8_t ring[W][S][kStage];
    float o[kOut > kJoin ? kOut : kJoin];        // kTurn tiles of all warps: [kTurn][W][4 D / 16][kMerge]
    alignas(16) uint8_t q[kRows][kQRow];
    float qfac[kRows], slope[kRows];
    float m[W][kRows], mw[E4M3 ? W : 1][kRows], l[W][kRows], part[kRows];
    alignas(8) uint64_t full[W][S];
    PagedSched sched;
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

template <bool E4M3>
__device__ __forceinline__ void mma_tile(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    if constexpr (E4M3) mma_f16(c, a0, a1, a2, a3, b0, b1);
    else mma_bf16(c, a0, a1, a2, a3, b0, b1);
}

__device__ __forceinline__ uint32_t cvt_lo(uint32_t w) { return e4m3x2_to_f16x2(static_cast<uint16_t>(w)); }
__device__ __forceinline__ uint32_t cvt_hi(uint32_t w) { return e4m3x2_to_f16x2(static_cast<uint16_t>(w >> 16)); }
__device__ __forceinline__ uint32_t word(const uint4 &u, int i) { return i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w; }

// Transposed load of two matrices of 16 rows x 16 bytes (lanes 0-15 and 16-31 give their rows' addresses): r[0] is column
// lane / 4, r[1] column lane / 4 + 8 of the first, rows 4 (lane % 4) .. + 3; r[2], r[3] of the second.
__device__ __forceinline__ void ldsm_t8(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x2.trans.shared.b8 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// One warp's ring of S stages, a tile of TP token groups each (neighbours of one page): copies are issued S
// tiles ahead of the computation, one bulk copy per tile, and across piece ends. The warp takes every W-th tile
// of the table's pieces, in order, 32 tiles of a piece at a time: lane j looks up the page of the j-th and
// issues its copy. A tile on a bad page is reported and skipped. When a wait gives up the warp issues and waits
// for nothing more (bar the copies in flight, at the end).
template <int W, int S, int TP, int GROUP, int STAGE>
struct GroupRing {
    static constexpr int BYTES = TP * GROUP, TT = TP * kGroupTokens;
    uint8_t *buf;           // [S][STAGE]
    uint64_t *full;         // [S]
    int i, g, g_end;        // piece of the table, first of the 32 tiles, the piece's end
    int group;              // this lane's tile: its first group in the pool
    int at, count;          // tiles issued of how many (0: there are no more)
    uint32_t bad;           // lanes whose tile's page id is bad
    uint32_t skip;          // stages whose tile's page id is bad: nothing was copied
    uint32_t phase;
    int stage, ahead;       // ahead: stages from this one on that have been issued
    bool dead;

    __device__ __forceinline__ void init(uint8_t *ring, uint64_t *bars) {
        buf = ring;
        full = bars;
        skip = phase = 0;
        stage = ahead = 0;
        dead = false;
        if ((threadIdx.x & 31) == 0) {
            for (int s = 0; s < S; ++s) mbar_init(&full[s], 1);
            fence_mbar_init();
        }
        __syncwarp();
    }
    __device__ __forceinline__ void look_up(const PagedArgs &a, const PagedSched &sched) {
        const PagedPiece &p = sched.piece[i];
        const int tile = g + W * static_cast<int>(threadIdx.x & 31);
        int page = 0;
        if (tile < g_end) page = ld_global_s32(a.page_table + static_cast<int64_t>(p.b) * a.max_pages + tile / (kPageGroups / TP));
        count = min((g_end - g + W - 1) / W, 32);
        bad = __ballot_sync(0xffffffffu, tile < g_end && (page < 0 || page >= a.num_pages));
        group = (page * a.Hkv + p.h) * kPageGroups + tile % (kPageGroups / TP) * TP;   // a pool's groups stay below 2^31
        at = 0;
    }
    // to the first tile of piece i or, where this warp has none there, of the pieces after it
    __device__ __forceinline__ void settle(const PagedArgs &a, const PagedSched &sched) {
        for (; i < sched.n; ++i) {
            const PagedPiece &p = sched.piece[i];
            const int g0 = p.lo / TT;
            g = g0 + p.r0 * W + static_cast<int>(threadIdx.x >> 5);
            g_end = p.hi > p.lo ? min((p.hi + TT - 1) / TT, g0 + p.r1 * W) : 0;
            if (g < g_end) return look_up(a, sched);
        }
        at = count = 0;
    }
    __device__ __forceinline__ void issue(const PagedArgs &a, const PagedSched &sched, int s) {
        if (at >= count) return;
        const bool mine = (threadIdx.x & 31) == at;
        if (bad | skip) {
            const bool none = bad >> at & 1;
            skip = none ? skip | 1u << s : skip & ~(1u << s);
            if (mine && none) {
                raise_flag(a.flags, FLAG_BAD_PAGE);
                mbar_arrive(&full[s]);
            }
        }
        if (mine && !(bad >> at & 1)) {
            mbar_arrive_expect_tx(&full[s], BYTES);
            bulk_g2s(buf + s * STAGE, a.pages + static_cast<int64_t>(group) * GROUP, BYTES, &full[s]);
        }
        ++ahead;
        if (++at == count) {
            g += 32 * W;
            if (g < g_end) {
                look_up(a, sched);
            } else {
                ++i;
                settle(a, sched);
            }
        }
    }
    // a new piece table: nothing is in flight
    __device__ __forceinline__ void begin(const PagedArgs &a, const PagedSched &sched) {
        i = 0;
        settle(a, sched);
        if (dead) count = 0;
#pragma unroll 1
        for (int s = 0; s < S; ++s) issue(a, sched, stage + s < S ? stage + s : stage + s - S);
    }
    // false: nothing to compute (a wait gave up; the stage stays)
    __device__ __forceinline__ bool wait(const PagedArgs &a) {
        if (dead) return false;
        if (!__all_sync(0xffffffffu, mbar_try_wait(&full[stage], phase))) {
            dead = !__all_sync(0xffffffffu, mbar_wait(&full[stage], phase));
            if (dead) {
                if ((threadIdx.x & 31) == 0) raise_flag(a.flags, FLAG_TIMEOUT);
                count = 0;
                return false;
            }
        }
        --ahead;
        return true;
    }
    __device__ __forceinline__ bool skipped() const { return skip >> stage & 1; }
    __device__ __forceinline__ const uint8_t *data() const { return buf + stage * STAGE; }
    // every lane is done with the stage: copy the next tile there, go on to the next stage
    __device__ __forceinline__ void release(const PagedArgs &a, const PagedSched &sched) {
        __syncwarp();
        issue(a, sched, stage);
        if (++stage == S) stage = 0, phase ^= 1;
    }
    // a warp that gave up leaves only when the copies that it issued have landed (bounded again)
    __device__ __forceinline__ void drain() {
        if (dead)
            for (int j = 0; j < ahead; ++j) {
                const int s = stage + j < S ? stage + j : stage + j - S;
                mbar_wait(&full[s], s < stage ? phase ^ 1 : phase);
            }
    }
};

// k_paged_mma (bf16 queries): mma.sync m16n8k16 with the tokens as M and 8 NT query rows as N, so that
// a group of up to 8 query heads reads every key once and the logits' accumulators, after one 8x8
// transpose per tile, are the second product's operand. HBM bounds it: a key and value are 258
// (e4m3) or 512 (raw) bytes at d = 128 and 4 d flops per query row, ~10 flops per byte at 7 rows,
// a tenth of what even this older matrix path does in that time; tcgen05 would need the
// converted keys stored to shared or tensor memory again (its fp16 operand cannot be an e4m3 tile) and a
// round trip of the scores through tensor memory per tile. So each warp works alone: it takes every W-th
// token group of a piece, one bulk copy per group into a private ring, S groups ahead across piece ends,
// and meets the other warps only at the end of a piece.
//   Keys: the contraction order over d is free as long as keys and queries agree; a lane's 16
//   bytes of a key row serve several steps, so that a group's keys are 4 (e4m3) or 8 (raw) 16-byte loads.
//   Values: transposed by byte permutes of neighbouring tokens' words or, up to 8 rows of e4m3, by the load.
//   e4m3: codes go to fp16 (exact); a query row is scaled by a power of two into fp16's range, exactly; the key's
//   scale multiplies the logit, and the value's the weight: the fp16 weight is 2^(s + ve - mw), with mw the
//   running maximum of base-2 logit + value exponent less 7, beside m, the logits' own, for the partition sum 2^(s - m).
//   So neither a value's scale nor a value of zeros can take precision from the partition or the other values.
//   Weights are 16-bit operands of the second product, the partition keeps them in fp32. e4m3 caches: one fp16 number
//   (2^-11 relative), far below what the codes themselves hold; the 7 put the largest near fp16's top, so that its
//   smallest steps, 2^-24, are 2^-31 of it: 2^19 keys, a warp's share of a full memory, lose 2^-13 by them. Raw caches
//   hold values whole, so that a weight of one bf16 number (2^-8) would be their largest error: it is two, its upper
//   half and the rest (2^-16), for twice the second product's instructions (up to 16 rows in the shadow of the copies:
//   79.9 and 51.9 us with one or two; 28 rows over 8 x 4 x 16,384 keys 63.1 -> 69.5 us). Sums and maxima are fp32. A
//   reference maximum moves only when it is exceeded by 8 (2^8), so that the rescale of O runs rarely.
// Measured: 32 sequences x 4 heads x 32,768 e4m3 keys at 7 rows take 174 us, 96% of the copy rate (raw, ragged:
// 80 us, 93%). An mma.sync, a conversion and an FMA add up on one scheduler here instead of overlapping, so
// that many rows are bound by the instruction rate: 28 rows over 8 x 4 x 16,384 e4m3 keys take 60.8 us, 34%.
template <bool E4M3, int D, int NT, int W, int S, int CTAS, int TP>
__global__ void __launch_bounds__(32 * W, CTAS) k_paged_mma(const PagedArgs a) {
    using Sm = MmaSmem<E4M3, D, NT, W, S, CTAS, TP>;
    using G = typename Sm::G;
    constexpr int KS = D / 16, MT = D / 16, ROWS = 8 * NT, THREADS = 32 * W, TT = TP * kGroupTokens;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Sm &sm = *reinterpret_cast<Sm *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tq = lane & 3;
    // Values transposed by the load instead of byte permutes: up to 8 rows 73.3 -> 72.2 us (64 x 16 heads) and 58.9 ->
    // 54.9 (d = 64), where many warps hide its bank conflicts; 28 rows 62.4 -> 63.4. Then rows g, g + 8 of the
    // logits' matrix are tokens tg, tg + 2, in the order that the load deals them out.
    constexpr bool LDSM = E4M3 && NT == 1;
    constexpr int TD = LDSM ? 2 : 8;
    const int tg = LDSM ? 4 * (g >> 1) + (g & 1) : g;
    GroupRing<W, S, TP, G::kGroup, Sm::kStage> ring;
    ring.init(sm.ring[warp][0], sm.full[warp]);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    paged_schedule<THREADS, W, TT, Sm::kCost>(a, sm.sched);
    paged_pieces<W, TT, Sm::kCost>(a, sm.sched, 0);

    constexpr int PER = D / 32, RPW = (ROWS + W - 1) / W;   // query elements per lane and row, rows per warp
    uint32_t qx[RPW][PER / 2];
    float qslope[RPW];
    const auto load_queries = [&](const PagedPiece &p) {
        const int row0 = p.pass * ROWS, rows = min(ROWS, a.rows - row0);
        const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + p.b * a.q_b + static_cast<int64_t>(p.h) * a.G * a.q_h + lane * PER;
#pragma unroll
        for (int i = 0; i < RPW; ++i) {
            const int r = warp + W * i;
            qslope[i] = 0.f;
#pragma unroll
            for (int e = 0; e < PER / 2; ++e) qx[i][e] = 0;
            if (r < rows) {
                const int rr = static_cast<int>((row0 + r + 0.5f) * a.inv_G), gq = row0 + r - rr * a.G;
                const __nv_bfloat16 *src = q + rr * a.q_r + gq * a.q_h;
                if constexpr (PER == 4) {
                    const uint2 u = *reinterpret_cast<const uint2 *>(src);
                    qx[i][0] = u.x, qx[i][1] = u.y;
                } else {
                    qx[i][0] = *reinterpret_cast<const uint32_t *>(src);
                }
                if (a.slopes) qslope[i] = a.slopes[p.h * a.G + gq];
            }
        }
    };
    const SoftCap softcap(a.softcap);
    int from = 0, at = paged_next(sm.sched, 0);
    bool fresh = true;   // a new table: nothing is ahead
#pragma unroll 1
    while (true) {
        if (at == sm.sched.n) {
            if (at < kPieceTable) break;
            __syncthreads();
            from += kPieceTable;
            paged_pieces<W, TT, Sm::kCost>(a, sm.sched, from);
            at = paged_next(sm.sched, 0);
            fresh = true;
            continue;
        }
        const PagedPiece &pc = sm.sched.piece[at];
        if (fresh) {   // the queries' loads before anything waits, then the ring
            load_queries(pc);
            ring.begin(a, sm.sched);
            fresh = false;
        }
        const int row0 = pc.pass * ROWS, rows = min(ROWS, a.rows - row0);
        // the pass's query rows, one warp per row: e4m3 caches take them as fp16, scaled by a power of two
        // that puts the largest finite element into [2^14, 2^15): exact down to 2^-29 of it
#pragma unroll
        for (int i = 0; i < RPW; ++i) {
            const int r = warp + W * i;
            if (r >= ROWS) break;
            float x[PER], fac = a.scale;
#pragma unroll
            for (int e = 0; e < PER; e += 2) x[e] = bf16lo(qx[i][e / 2]), x[e + 1] = bf16hi(qx[i][e / 2]);
            if constexpr (E4M3) {
                float top = 0.f;
#pragma unroll
                for (int e = 0; e < PER; ++e) top = fabsf(x[e]) < INFINITY ? fmaxf(top, fabsf(x[e])) : top;
#pragma unroll
                for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                const int up = min(14 + 127 - static_cast<int>(__float_as_uint(top) >> 23), 126);   // >= -113
                const float mul = top > 0.f ? scale_of(127 + up) : 1.f;
                fac = top > 0.f ? fac * scale_of(127 - up) : fac;
#pragma unroll
                for (int e = 0; e < PER; ++e) x[e] *= mul;
            }
            uint32_t *dst = reinterpret_cast<uint32_t *>(sm.q[r] + lane * PER * 2);
#pragma unroll
            for (int e = 0; e < PER; e += 2) dst[e / 2] = E4M3 ? pack_f16x2(x[e], x[e + 1]) : pack_bf16x2(x[e], x[e + 1]);
            if (lane == 0) {
                sm.qfac[r] = a.softcap > 0.f ? fac : fac * kLog2e;
                sm.slope[r] = qslope[i] * kLog2e;
            }
        }
        __syncthreads();
        const int lo = pc.lo, hi = pc.hi, g0 = lo / TT;
        const int g_end = hi > lo ? min((hi + TT - 1) / TT, g0 + pc.r1 * W) : 0;
        // element pairs d0, d0 + 1 and d0 + 2, d0 + 3 of row g of tile nt for step ks
        const auto qfrag = [&](int nt, int ks) {
            const int d0 = E4M3 ? 64 * (ks / 4) + 16 * tq + 4 * (ks % 4) : 32 * (ks / 2) + 8 * tq + 4 * (ks % 2);
            return *reinterpret_cast<const uint2 *>(sm.q[8 * nt + g] + 2 * d0);
        };
        // The queries stay in registers (16 rows: 43.1 -> 41.1 us). Four tiles of rows have none left for them: at d = 128
        // they spill 64 bytes (e4m3) and 108 (raw) without; with, 61 -> 71 us.
        constexpr bool QREG = NT <= 2;
        uint2 qf[QREG ? NT : 1][QREG ? KS : 1];
        if constexpr (QREG) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) qf[nt][ks] = qfrag(nt, ks);
        }
        float fac[NT][2], slope[NT][2], mref[NT][2], mw[NT][2], l[NT][2], o[NT][MT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                fac[nt][c] = sm.qfac[8 * nt + 2 * tq + c];
                slope[nt][c] = sm.slope[8 * nt + 2 * tq + c];
                mref[nt][c] = mw[nt][c] = kNoLogit;
                l[nt][c] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[nt][j][c] = 0.f;
        }
#pragma unroll 1
        for (int gi = g0 + pc.r0 * W + warp; gi < g_end; gi += W) {
            if (!ring.wait(a)) continue;
            {
#pragma unroll 1
                for (int half = 0; half < TP; ++half) {
                    const int t0 = gi * TT + half * kGroupTokens;
                    if (ring.skipped() || (TP > 1 && (t0 >= hi || t0 + kGroupTokens <= lo))) continue;
                    const uint8_t *buf = ring.data() + half * G::kGroup;
                    const uint32_t base = smem_u32(buf);
                    // ---- logits: tokens tg, tg + TD x rows 2 tq, 2 tq + 1 of every tile
                    float s[NT][4], s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) s[nt][c] = 0.f;
                    const uint32_t krow = base + tg * G::kVec;
                    constexpr int STEPS = E4M3 ? 4 : 2;   // steps that one 16-byte chunk serves
#pragma unroll
                    for (int i = 0; i < KS / STEPS; ++i) {
                        const uint4 ka = lds128(krow + 16 * cache_chunk(4 * i + tq, tg, G::kChunks));
                        const uint4 kb = lds128(krow + TD * G::kVec + 16 * cache_chunk(4 * i + tq, tg + TD, G::kChunks));
#pragma unroll
                        for (int w = 0; w < STEPS; ++w) {
                            uint32_t a0, a1, a2, a3;
                            if constexpr (E4M3) {
                                a0 = cvt_lo(word(ka, w)), a2 = cvt_hi(word(ka, w));
                                a1 = cvt_lo(word(kb, w)), a3 = cvt_hi(word(kb, w));
                            } else {
                                a0 = word(ka, 2 * w), a2 = word(ka, 2 * w + 1);
                                a1 = word(kb, 2 * w), a3 = word(kb, 2 * w + 1);
                            }
                            const int ks = STEPS * i + w;
                            if constexpr (NT == 1) {   // two chains
                                if (w & 1) mma_tile<E4M3>(s2, a0, a1, a2, a3, qf[0][ks].x, qf[0][ks].y);
                                else mma_tile<E4M3>(s[0], a0, a1, a2, a3, qf[0][ks].x, qf[0][ks].y);
                            } else {
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt) {
                                    const uint2 b = QREG ? qf[QREG ? nt : 0][QREG ? ks : 0] : qfrag(nt, ks);
                                    mma_tile<E4M3>(s[nt], a0, a1, a2, a3, b.x, b.y);
                                }
                            }
                        }
                    }
                    if constexpr (NT == 1) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) s[0][c] += s2[c];
                    }
                    float ve[2] = {0.f, 0.f}, vs[2] = {1.f, 1.f};   // a value's exponent and scale
                    float ksc[2] = {1.f, 1.f};
                    if constexpr (E4M3) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const uint32_t kb = buf[2 * G::kBlock + tg + TD * c];
                            const uint32_t vb = buf[2 * G::kBlock + kGroupTokens + tg + TD * c];
                            ksc[c] = scale_of(kb);
                            ve[c] = __uint_as_float(0x4b000000u | vb) - (8388608.f + 127.f);   // vb - 127
                            vs[c] = scale_of(vb);
                        }
                    }
                    const float gap0 = static_cast<float>(hi - 1 - t0 - tg);
                    const bool partial = t0 < lo || t0 + kGroupTokens > hi;
                    const bool in0 = t0 + tg >= lo && t0 + tg < hi, in1 = t0 + tg + TD >= lo && t0 + tg + TD < hi;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            float x = s[nt][c] * fac[nt][c & 1];
                            if constexpr (E4M3) x *= ksc[c >> 1];
                            s[nt][c] = x;
                        }
                    if (a.softcap > 0.f) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            float u[4];
                            bool far = false;
#pragma unroll
                            for (int c = 0; c < 4; ++c) {
                                u[c] = s[nt][c] * softcap.inv;
                                s[nt][c] = softcap.near(s[nt][c], u[c]);
                                far |= !(fabsf(u[c]) < 0.25f);
                            }
                            if (__any_sync(0xffffffffu, far)) {
#pragma unroll
                                for (int c = 0; c < 4; ++c)
                                    if (!(fabsf(u[c]) < 0.25f)) s[nt][c] = softcap.far(u[c]);
                            }
                        }
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) s[nt][c] = fmaf(-slope[nt][c & 1], gap0 - static_cast<float>(TD) * (c >> 1), s[nt][c]);
                    if (partial) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            if (!in0) s[nt][0] = s[nt][1] = -INFINITY;
                            if (!in1) s[nt][2] = s[nt][3] = -INFINITY;
                        }
                        if (!in0) vs[0] = 0.f;   // an exponent byte behind the end may be anything
                        if (!in1) vs[1] = 0.f;
                    }
                    // The reference maxima: of the logits for the partition and, e4m3, of logit + value exponent for the
                    // weights of the outputs. Both move only when one is exceeded by kSlack (or may be: the larger
                    // of a lane's two exponents stands for both).
                    const float vtop = fmaxf(ve[0], ve[1]) - kRaise;
                    float over = -INFINITY;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float m = E4M3 ? fminf(mref[nt][c], mw[nt][c] - vtop) : mref[nt][c];
                            over = fmaxf(over, fmaxf(s[nt][c], s[nt][c + 2]) - m);
                        }
                    if (__any_sync(0xffffffffu, over > kSlack)) {
                        if (E4M3 && __any_sync(0xffffffffu, ve[0] == 0.f || ve[1] == 0.f)) {
                            // a value of zeros is held with exponent 0, which must not set the scale that the other
                            // values' weights are rounded at
                            const uint32_t at = base + G::kBlock + (lane >> 1) * G::kVec + (lane & 1) * (G::kVec / 2);
                            uint32_t any = 0;
#pragma unroll
                            for (int i = 0; i < G::kVec / 32; ++i) {
                                const uint4 u = lds128(at + 16 * i);
                                any |= u.x | u.y | u.z | u.w;
                            }
                            const uint32_t empty = __ballot_sync(0xffffffffu, (any & 0x7f7f7f7fu) == 0);   // half vectors
                            const uint32_t zero = empty & empty >> 1 & 0x55555555u;
                            if (zero >> 2 * tg & 1) ve[0] = -INFINITY, vs[0] = 0.f;
                            if (zero >> 2 * (tg + TD) & 1) ve[1] = -INFINITY, vs[1] = 0.f;
                        }
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int c = 0; c < 2; ++c) {
                                float top = fmaxf(s[nt][c], s[nt][c + 2]);
                                float topw = fmaxf(s[nt][c] + ve[0], s[nt][c + 2] + ve[1]);
#pragma unroll
                                for (int x = 4; x < 32; x <<= 1) {
                                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                                    if constexpr (E4M3) topw = fmaxf(topw, __shfl_xor_sync(0xffffffffu, topw, x));
                                }
                                top = fmaxf(top, mref[nt][c]);
                                float f = ex2(mref[nt][c] - top);
                                l[nt][c] *= f;
                                mref[nt][c] = top;
                                if constexpr (E4M3) {
                                    topw = fmaxf(fmaxf(topw - kRaise, mw[nt][c]), top - kSpan);   // zeros only so far: finite
                                    f = ex2(mw[nt][c] - topw);
                                    mw[nt][c] = topw;
                                }
#pragma unroll
                                for (int j = 0; j < MT; ++j) o[nt][j][c] *= f, o[nt][j][c + 2] *= f;
                            }
                    }
                    uint32_t pb[NT][2], pr[E4M3 ? 1 : NT][2];   // raw: a weight is pb + pr
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float p[4];
                        float rw[2] = {1.f, 1.f};   // from the partition's reference to the outputs'
                        if constexpr (E4M3) rw[0] = ex2(mref[nt][0] - mw[nt][0]), rw[1] = ex2(mref[nt][1] - mw[nt][1]);
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            p[c] = ex2(s[nt][c] - mref[nt][c & 1]);
                            l[nt][c & 1] += p[c];
                            if constexpr (E4M3) p[c] = p[c] * vs[c >> 1] * rw[c & 1];   // in this order within fp32's range
                        }
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            const float x = p[2 * c], y = p[2 * c + 1];
                            if constexpr (E4M3) {
                                pb[nt][c] = movmatrix_t(pack_f16x2(x, y));
                            } else {   // upper halves, and what they leave: 2^-24 at least, not 0, which would make an infinite value NaN
                                const uint32_t u = __float_as_uint(x), w = __float_as_uint(y);
                                pb[nt][c] = movmatrix_t(__byte_perm(u, w, 0x7632));
                                pr[nt][c] = movmatrix_t(pack_bf16x2(fmaxf(x - __uint_as_float(u & 0xffff0000u), x * 0x1p-24f),
                                                                    fmaxf(y - __uint_as_float(w & 0xffff0000u), y * 0x1p-24f)));
                            }
                        }
                    }
                    // ---- outputs: weight 0 times what a masked token holds may be NaN
                    if constexpr (LDSM) {   // tokens 4 tq .. 4 tq + 3 x d = 16 j + g, + 8
                        uint32_t keep = 0xffffffffu;
                        if (partial) {
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (t0 + 4 * tq + e < lo || t0 + 4 * tq + e >= hi) keep &= ~(0xffu << 8 * e);
                        }
                        const int n = lane & 15;
#pragma unroll
                        for (int j = 0; j < MT; j += 2) {
                            uint32_t v[4];
                            ldsm_t8(v, base + G::kBlock + n * G::kVec + 16 * cache_chunk(j + (lane >> 4), n, G::kChunks));
                            if (partial) {
#pragma unroll
                                for (int e = 0; e < 4; ++e) v[e] &= keep;
                            }
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                mma_f16(o[0][j + h], cvt_lo(v[2 * h]), cvt_lo(v[2 * h + 1]), cvt_hi(v[2 * h]), cvt_hi(v[2 * h + 1]), pb[0][0], pb[0][1]);
                        }
                    } else {   // tokens 2 tq, 2 tq + 1, 2 tq + 8, 2 tq + 9 x this lane's d
                        const uint32_t vrow = base + G::kBlock + 2 * tq * G::kVec;
                        constexpr int HALVES = D * G::kElem / 128 > 0 ? D * G::kElem / 128 : 1;   // 16-byte chunks per lane and row
                        constexpr int WORDS = D * G::kElem / 32 / HALVES;                          // words of one: 4, or 2 (e4m3, d = 64)
#pragma unroll
                        for (int hf = 0; hf < HALVES; ++hf) {
                            uint32_t v[4][WORDS];
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const int n = 2 * tq + (r & 1) + 8 * (r >> 1);
                                const int dn = (r & 1) + 8 * (r >> 1);
                                if constexpr (WORDS == 4) {
                                    const uint4 u = lds128(vrow + dn * G::kVec + 16 * cache_chunk(g + 8 * hf, n, G::kChunks));
                                    v[r][0] = u.x, v[r][1] = u.y, v[r][2] = u.z, v[r][3] = u.w;
                                } else {
                                    const uint2 u = *reinterpret_cast<const uint2 *>(
                                        buf + G::kBlock + n * G::kVec + 16 * cache_chunk(g / 2, n, G::kChunks) + 8 * (g & 1));
                                    v[r][0] = u.x, v[r][1] = u.y;
                                }
                                if (partial && (t0 + n < lo || t0 + n >= hi)) {
#pragma unroll
                                    for (int w = 0; w < WORDS; ++w) v[r][w] = 0;
                                }
                            }
                            if constexpr (E4M3) {
#pragma unroll
                                for (int w = 0; w < WORDS; ++w) {
                                    const uint32_t lo01 = __byte_perm(v[0][w], v[1][w], 0x5140);
                                    const uint32_t lo23 = __byte_perm(v[2][w], v[3][w], 0x5140);
                                    const uint32_t hi01 = __byte_perm(v[0][w], v[1][w], 0x7362);
                                    const uint32_t hi23 = __byte_perm(v[2][w], v[3][w], 0x7362);
                                    const uint32_t a0 = cvt_lo(lo01), a1 = cvt_hi(lo01), a2 = cvt_lo(lo23), a3 = cvt_hi(lo23);
                                    const uint32_t b0 = cvt_lo(hi01), b1 = cvt_hi(hi01), b2 = cvt_lo(hi23), b3 = cvt_hi(hi23);
#pragma unroll
                                    for (int nt = 0; nt < NT; ++nt) {
                                        mma_f16(o[nt][2 * w], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                                        mma_f16(o[nt][2 * w + 1], b0, b1, b2, b3, pb[nt][0], pb[nt][1]);
                                    }
                                }
                            } else {
                                uint32_t x[WORDS][4];
#pragma unroll
                                for (int w = 0; w < WORDS; ++w) {
                                    x[w][0] = __byte_perm(v[0][w], v[1][w], 0x5410), x[w][1] = __byte_perm(v[0][w], v[1][w], 0x7632);
                                    x[w][2] = __byte_perm(v[2][w], v[3][w], 0x5410), x[w][3] = __byte_perm(v[2][w], v[3][w], 0x7632);
                                }
#pragma unroll
                                for (int rest = 1; rest >= 0; --rest)   // the small parts first; the two of one sum apart
#pragma unroll
                                    for (int w = 0; w < WORDS; ++w)
#pragma unroll
                                        for (int nt = 0; nt < NT; ++nt) {
                                            const auto &b = rest ? pr[nt] : pb[nt];
                                            mma_bf16(o[nt][WORDS * hf + w], x[w][0], x[w][1], x[w][2], x[w][3], b[0], b[1]);
                                        }
                            }
                        }
                    }
                }
                ring.release(a, sm.sched);
            }
        }
        const int after = paged_next(sm.sched, at + 1);
        if (after < sm.sched.n) load_queries(sm.sched.piece[after]);   // they arrive while the warps join
        // ---- join the warps, one tile of 8 rows at a time; those that had no group have nothing to add
        const int act = max(1, min(W, g_end - (g0 + pc.r0 * W)));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float sum = l[nt][c];
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                if (g == 0) {
                    sm.m[warp][8 * nt + 2 * tq + c] = mref[nt][c];
                    if constexpr (E4M3) sm.mw[warp][8 * nt + 2 * tq + c] = mw[nt][c];
                    sm.l[warp][8 * nt + 2 * tq + c] = sum;
                }
            }
        __syncthreads();
        static_assert(ROWS * W <= THREADS && (W & (W - 1)) == 0, "one lane per row and warp");
        if (tid < ROWS * W) {   // the warps' weights, 2^(mw - largest m) over the joint sum, and the row's partition
            const int r = tid / W, w = tid % W;
            const float mine = sm.m[w][r];
            float top = mine;
#pragma unroll
            for (int x = 1; x < W; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            const float f = ex2(mine - top);
            float sum = f * sm.l[w][r];
#pragma unroll
            for (int x = 1; x < W; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
            // 2^7 apart, since ex2 flushes what is below 2^-126; the product may be subnormal
            const float part = E4M3 ? ex2(sm.mw[E4M3 ? w : 0][r] + kRaise - top) * 0x1p-7f : f;
            static_assert(kRaise == 7.f, "one factor");
            sm.m[w][r] = sum == 0.f ? 0.f : part * __frcp_rn(sum);
            if (w == 0) sm.part[r] = sum == 0.f ? -INFINITY : top + __log2f(sum);
        }
        // one copy of this code for all tiles: each turn writes the first kTurn and moves the others down
        constexpr int TURN = Sm::kTurn, TILE = W * 4 * MT * Sm::kMerge;
#pragma unroll 1
        for (int nt = 0; 8 * nt < rows; nt += TURN) {
            if (warp < act) {
#pragma unroll
                for (int j = 0; j < MT; ++j)
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
#pragma unroll
                        for (int n = 0; n < TURN; ++n) sm.o[n * TILE + ((warp * 4 + c) * MT + j) * Sm::kMerge + lane] = o[n][j][c];
#pragma unroll
                        for (int n = 0; n + TURN < NT; ++n) o[n][j][c] = o[n + TURN][j][c];
                    }
            }
            __syncthreads();
#pragma unroll 1
            for (int i = tid; i < 8 * TURN * (D / 4); i += THREADS) {
                const int rt = i / (D / 4), r8 = rt % 8, r = 8 * nt + rt, d0 = (i % (D / 4)) * 4;
                if (r >= rows) break;
                // where d0 .. d0 + 3 lie: lane group gd, tile j, element c, and how far apart in tiles, elements or groups
                int gd, j, c = r8 & 1;
                if constexpr (LDSM) gd = d0 % 8, j = d0 / 16, c += d0 % 16 / 8 * 2;
                else if constexpr (!E4M3 && D == 128) gd = d0 % 64 / 8, j = 4 * (d0 / 64) + d0 % 8 / 2;
                else gd = d0 / (D / 8), j = d0 % (D / 8) / 2;
                constexpr int D1 = LDSM ? 4 : 2 * MT * Sm::kMerge, D2 = LDSM ? 8 : Sm::kMerge;
                const float *src = sm.o + rt / 8 * TILE + (c * MT + j) * Sm::kMerge + 4 * gd + r8 / 2;
                float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int w = 0; w < act; ++w, src += 4 * MT * Sm::kMerge) {
                    const float f = sm.m[w][r];
                    x.x = fmaf(f, src[0], x.x);
                    x.y = fmaf(f, src[D1], x.y);
                    x.z = fmaf(f, src[D2], x.z);
                    x.w = fmaf(f, src[D1 + D2], x.w);
                }
                if (pc.np == 1) {
                    paged_write<__nv_bfloat16, D>(a, pc.b, pc.h, row0 + r, d0, x, sm.part[r]);
                } else {
                    const int64_t to = pc.slot(blockIdx.x) * ROWS + r;
                    store4(a.part_o + to * D + d0, x);
                    if (d0 == 0) a.part_l[to] = sm.part[r];
                }
            }
            if (8 * (nt + TURN) < rows) __syncthreads();   // the last turn: the next piece's query rows bring a barrier
        }
        if (pc.np > 1) paged_finish_piece<__nv_bfloat16, D, ROWS, THREADS>(a, pc, sm.sched, sm.o);
        at = after;
    }
    ring.drain();
}

// ---------------------------------------------------------------------------
// fp32 queries: CUDA cores
// ---------------------------------------------------------------------------
// k_paged_f32: exact fp32 products on packed FMAs, out of the same rings. For the logits a lane takes four tokens x
// four rows over a quarter of d (64 FMAs to eight 16-byte loads), and four lanes add their quarters up, each
// keeping one token; for the outputs it takes d / 32 dimensions of all 8 rows (one load of its values per
// token and the 8 weights broadcast). Raw caches at d = 128 are 16 KB per group, 712 clocks of one SM at the copy
// rate; its ~350 shared-memory wavefronts and ~1,700 issue slots of one scheduler lie below that, but
// 8 warps do not hide a group's latency: 8 sequences x 4 heads x 8,192 keys take 63.5 us, 65% of the copy rate
// (88 us with two tokens x two rows per lane).
constexpr int kF32Rows = 8;

template <bool E4M3, int D, int W, int S>
struct F32Smem {
    using G = CacheGeom<float, E4M3, D>;
    static constexpr int kStage = (G::kGroup + 127) / 128 * 128;
    static constexpr int kMaxCtas = 160;
    static constexpr int kCost = 2;
    static constexpr int kOut = W * kF32Rows * D, kJoin = kF32Rows * 33;   // kJoin: the weights of a unit's pieces
    alignas(128) uint8_t ring[W][S][kStage];
    alignas(16) float o[kOut > kJoin ? kOut : kJoin];   // [W][rows][D]
    alignas(16) float q[kF32Rows][D + 4];
    alignas(16) float p[W][kGroupTokens][kF32Rows];     // a group's weights (times the values' scales)
    alignas(16) float f[W][kF32Rows];                   // what the outputs are rescaled by
    float slope[kF32Rows];
    float m[W][kF32Rows], l[W][kF32Rows], part[kF32Rows];
    alignas(8) uint64_t full[W][S];
    PagedSched sched;
};

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

template <bool E4M3, int D, int W, int S>
__global__ void __launch_bounds__(32 * W, 1) k_paged_f32(const PagedArgs a) {
    using Sm = F32Smem<E4M3, D, W, S>;
    using G = typename Sm::G;
    using CV = ChunkValues<float, E4M3>;
    constexpr int NR = kF32Rows, PER = D / 32, THREADS = 32 * W;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    Sm &sm = *reinterpret_cast<Sm *>((reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int part = lane & 3, tg = lane >> 2 & 3, rg = lane >> 4;   // quarter of d, tokens tg + 4 k, rows 4 rg + r
    const int mine = tg + 4 * part;                                   // the token whose logits this lane ends up with
    GroupRing<W, S, 1, G::kGroup, Sm::kStage> ring;
    ring.init(sm.ring[warp][0], sm.full[warp]);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    paged_schedule<THREADS, W, kGroupTokens, Sm::kCost>(a, sm.sched);
    paged_pieces<W, kGroupTokens, Sm::kCost>(a, sm.sched, 0);
    int from = 0, at = paged_next(sm.sched, 0);
    bool fresh = true;   // a new table: nothing is ahead
#pragma unroll 1
    while (true) {
        if (at == sm.sched.n) {
            if (at < kPieceTable) break;
            __syncthreads();
            from += kPieceTable;
            paged_pieces<W, kGroupTokens, Sm::kCost>(a, sm.sched, from);
            at = paged_next(sm.sched, 0);
            fresh = true;
            continue;
        }
        const PagedPiece &pc = sm.sched.piece[at];
        if (fresh) {
            ring.begin(a, sm.sched);
            fresh = false;
        }
        const int row0 = pc.pass * NR, rows = min(NR, a.rows - row0);
        for (int i = tid; i < NR * (D / 4); i += THREADS) {
            const int r = i / (D / 4), d0 = (i % (D / 4)) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
            float slope = 0.f;
            if (r < rows) {
                const int rr = static_cast<int>((row0 + r + 0.5f) * a.inv_G), hq = pc.h * a.G + row0 + r - rr * a.G;
                x = load4(static_cast<const float *>(a.q) + pc.b * a.q_b + rr * a.q_r + hq * a.q_h + d0);
                if (a.slopes && d0 == 0) slope = a.slopes[hq];
            }
            store4(&sm.q[r][d0], x);
            if (d0 == 0) sm.slope[r] = slope;
        }
        __syncthreads();
        const int lo = pc.lo, hi = pc.hi, g0 = lo / kGroupTokens;
        const int g_end = hi > lo ? min((hi + kGroupTokens - 1) / kGroupTokens, g0 + pc.r1 * W) : 0;
        float m[4], l[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) m[r] = -INFINITY, l[r] = 0.f;
        uint64_t o[PER][NR / 2];   // row pairs
#pragma unroll
        for (int i = 0; i < PER; ++i)
#pragma unroll
            for (int r = 0; r < NR / 2; ++r) o[i][r] = 0;
#pragma unroll 1
        for (int gi = g0 + pc.r0 * W + warp; gi < g_end; gi += W) {
            if (!ring.wait(a)) continue;
            if (!ring.skipped()) {
                const uint8_t *buf = ring.data();
                const int t0 = gi * kGroupTokens;
                // ---- logits: this quarter's share, then the sum of the quarters
                uint64_t acc[4][4] = {};
#pragma unroll 2
                for (int i = 0; i < G::kChunks / 4; ++i) {
                    const int c = 4 * i + part;
                    float x[4][CV::N];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int n = tg + 4 * k;
                        CV::get(*reinterpret_cast<const uint4 *>(buf + n * G::kVec + 16 * cache_chunk(c, n, G::kChunks)), x[k]);
                    }
#pragma unroll
                    for (int e = 0; e < CV::N; e += 4)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float4 y = load4(&sm.q[4 * rg + r][c * CV::N + e]);
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                acc[k][r] = ffma2(f2pack(x[k][e], x[k][e + 1]), f2pack(y.x, y.y), acc[k][r]);
                                acc[k][r] = ffma2(f2pack(x[k][e + 2], x[k][e + 3]), f2pack(y.z, y.w), acc[k][r]);
                            }
                        }
                }
                float s[4], vs = 1.f, ks = a.scale;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float z[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        float x, y;
                        f2unpack(acc[k][r], x, y);
                        z[k] = x + y;
                    }
                    // lane pairs swap tokens: the odd quarter keeps k = 1, 3, then the upper ones k = 2, 3
                    const bool odd = part & 1, upper = part & 2;
                    const float g0 = __shfl_xor_sync(0xffffffffu, odd ? z[0] : z[1], 1);
                    const float g1 = __shfl_xor_sync(0xffffffffu, odd ? z[2] : z[3], 1);
                    const float h0 = (odd ? z[1] : z[0]) + g0, h1 = (odd ? z[3] : z[2]) + g1;
                    s[r] = (upper ? h1 : h0) + __shfl_xor_sync(0xffffffffu, upper ? h0 : h1, 2);
                }
                if constexpr (E4M3) {
                    ks *= scale_of(buf[2 * G::kBlock + mine]);
                    vs = scale_of(buf[2 * G::kBlock + kGroupTokens + mine]);
                }
                const bool in = t0 + mine >= lo && t0 + mine < hi;
                const float gap = static_cast<float>(hi - 1 - t0 - mine);
                // ---- running maximum and sum (each lane keeps the sum of its own tokens)
                bool moved = false;
                float p[4], f[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float z = s[r] * ks;
                    if (a.softcap > 0.f) {   // c tanh(z / c); below 2^-12 that is z to the last bit, and z / c may be subnormal
                        const float t = z / a.softcap;
                        if (!(fabsf(t) < 0x1p-12f)) z = a.softcap * tanhf(t);
                    }
                    z = in ? z - sm.slope[4 * rg + r] * gap : -INFINITY;
                    float top = z;
#pragma unroll
                    for (int x = 1; x < 16; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                    top = fmaxf(top, m[r]);
                    const float ref = top > -INFINITY ? top : 0.f;   // no key yet: weights 2^-inf = 0
                    f[r] = ex2((m[r] - ref) * kLog2e);   // differences first: a base-2 logit would be rounded at its full size
                    moved |= f[r] != 1.f;
                    m[r] = top;
                    const float w = ex2((z - ref) * kLog2e);
                    l[r] = fmaf(l[r], f[r], w);
                    p[r] = w * vs;
                }
                // a masked token's scale may be anything: its weight is never read
                store4(&sm.p[warp][mine][4 * rg], make_float4(p[0], p[1], p[2], p[3]));
                if ((lane & 15) == 0) store4(&sm.f[warp][4 * rg], make_float4(f[0], f[1], f[2], f[3]));
                moved = __any_sync(0xffffffffu, moved);
                __syncwarp();
                if (moved) {
                    const uint64_t *by = reinterpret_cast<const uint64_t *>(sm.f[warp]);
#pragma unroll
                    for (int r = 0; r < NR / 2; ++r)
#pragma unroll
                        for (int i = 0; i < PER; ++i) o[i][r] = mul2(o[i][r], by[r]);
                }
                // ---- outputs: dimensions lane PER .. of the tokens that are seen (others may hold anything)
                const int n0 = max(lo - t0, 0), n1 = min(hi - t0, kGroupTokens);
                constexpr int bytes = PER * G::kElem;
#pragma unroll 8
                for (int n = n0; n < n1; ++n) {
                    const uint8_t *vp = buf + G::kBlock + n * G::kVec + 16 * cache_chunk(lane * bytes / 16, n, G::kChunks) + lane * bytes % 16;
                    float x[PER];
                    if constexpr (E4M3) {
                        if constexpr (PER == 4) {
                            const uint32_t u = *reinterpret_cast<const uint32_t *>(vp);
                            const float2 f0 = f16x2_to_f32(cvt_lo(u)), f1 = f16x2_to_f32(cvt_hi(u));
                            x[0] = f0.x, x[1] = f0.y, x[2] = f1.x, x[3] = f1.y;
                        } else {
                            const float2 f0 = f16x2_to_f32(e4m3x2_to_f16x2(*reinterpret_cast<const unsigned short *>(vp)));
                            x[0] = f0.x, x[1] = f0.y;
                        }
                    } else if constexpr (PER == 4) {
                        const float4 u = *reinterpret_cast<const float4 *>(vp);
                        x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
                    } else {
                        const float2 u = *reinterpret_cast<const float2 *>(vp);
                        x[0] = u.x, x[1] = u.y;
                    }
                    const ulonglong2 p01 = *reinterpret_cast<const ulonglong2 *>(&sm.p[warp][n][0]);
                    const ulonglong2 p23 = *reinterpret_cast<const ulonglong2 *>(&sm.p[warp][n][4]);
#pragma unroll
                    for (int i = 0; i < PER; ++i) {
                        const uint64_t v = f2pack(x[i], x[i]);
                        o[i][0] = ffma2(p01.x, v, o[i][0]);
                        o[i][1] = ffma2(p01.y, v, o[i][1]);
                        o[i][2] = ffma2(p23.x, v, o[i][2]);
                        o[i][3] = ffma2(p23.y, v, o[i][3]);
                    }
                }
            }
            ring.release(a, sm.sched);
        }
        // ---- join the warps; those that had no group have nothing to add
        const int act = max(1, min(W, g_end - (g0 + pc.r0 * W)));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            float sum = l[r];
#pragma unroll
            for (int x = 1; x < 16; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
            if ((lane & 15) == 0) sm.m[warp][4 * rg + r] = m[r], sm.l[warp][4 * rg + r] = sum;
        }
#pragma unroll
        for (int r = 0; r < NR / 2; ++r)
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                float x, y;
                f2unpack(o[i][r], x, y);
                sm.o[(warp * NR + 2 * r) * D + lane * PER + i] = x;
                sm.o[(warp * NR + 2 * r + 1) * D + lane * PER + i] = y;
            }
        __syncthreads();
        static_assert((W & (W - 1)) == 0, "one lane per row and warp");
        if (tid < NR * W) {   // the warps' weights, 2^(m - largest m) over the joint sum, and the row's partition
            const int r = tid / W, w = tid % W;
            const float mine = sm.m[w][r];
            float top = mine;
#pragma unroll
            for (int x = 1; x < W; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
            top = top > -INFINITY ? top : 0.f;
            const float f = ex2((mine - top) * kLog2e);
            float sum = f * sm.l[w][r];
#pragma unroll
            for (int x = 1; x < W; x <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
            sm.m[w][r] = sum == 0.f ? 0.f : f * __frcp_rn(sum);
            if (w == 0) sm.part[r] = sum == 0.f ? -INFINITY : fmaf(top, kLog2e, __log2f(sum));
        }
        __syncthreads();
        for (int i = tid; i < rows * (D / 4); i += THREADS) {
            const int r = i / (D / 4), d0 = (i % (D / 4)) * 4;
            float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int w = 0; w < act; ++w) {
                const float f = sm.m[w][r];
                const float4 y = load4(&sm.o[(w * NR + r) * D + d0]);
                x = make_float4(fmaf(f, y.x, x.x), fmaf(f, y.y, x.y), fmaf(f, y.z, x.z), fmaf(f, y.w, x.w));
            }
            if (pc.np == 1) {
                paged_write<float, D>(a, pc.b, pc.h, row0 + r, d0, x, sm.part[r]);
            } else {
                const int64_t to = pc.slot(blockIdx.x) * NR + r;
                store4(a.part_o + to * D + d0, x);
                if (d0 == 0) a.part_l[to] = sm.part[r];
            }
        }
        // no barrier: what follows writes none of this before the next one (the next piece's query rows')
        if (pc.np > 1) paged_finish_piece<float, D, NR, THREADS>(a, pc, sm.sched, sm.o);
        at = paged_next(sm.sched, at + 1);
    }
    ring.drain();
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
cudaError_t launch(K kernel, const PagedArgs &a0, int threads, size_t smem, int max_ctas, cudaStream_t s) {
    PagedArgs a = a0;
    cudaError_t e = resident_ctas(reinterpret_cast<const void *>(kernel), threads, smem, &a.ncta);
    if (e != cudaSuccess) return e;
    if (a.ncta > max_ctas) a.ncta = max_ctas;
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

template <bool E4M3, int D, int W, int S>
cudaError_t launch_f32(const PagedArgs &a, cudaStream_t s) {
    return launch(k_paged_f32<E4M3, D, W, S>, a, 32 * W, sizeof(F32Smem<E4M3, D, W, S>) + 128, F32Smem<E4M3, D, W, S>::kMaxCtas, s);
}

template <bool E4M3, int D, int NT, int W, int S, int CTAS, int TP>
cudaError_t launch_mma(const PagedArgs &a, cudaStream_t s) {
    return launch(k_paged_mma<E4M3, D, NT, W, S, CTAS, TP>, a, 32 * W, sizeof(MmaSmem<E4M3, D, NT, W, S, CTAS, TP>) + 128,
                  MmaSmem<E4M3, D, NT, W, S, CTAS, TP>::kMaxCtas, s);
}

template <bool E4M3, int D>
cudaError_t launch_rows(const PagedArgs &a, cudaStream_t s) {
    // at d = 64 two groups make a tile, which halves what a tile costs beside its products: 32 x 8 heads x 8,192 keys
    // 58.9 -> 55.0 us (e4m3), 89.6 -> 86.4 us (raw)
    constexpr int TP = D == 64 ? 2 : 1;
    // Warps and CTAs per SM. e4m3, 8 rows: two CTAs of 8 warps at 128 registers (7B batch 174 us; one CTA of 8 warps
    // 188 us: too few to hide a tile's latency). Raw tiles are twice the bytes for the same work: one CTA of 8
    // warps (80 us; two of 4 84.2). More rows need the registers: 16 and 28 rows 41.6 and 60.8 us; with three
    // and two CTAs of 4 warps 55.8 and 75.2.
    if constexpr (E4M3) {
        if (a.pass_rows == 8) return launch_mma<E4M3, D, 1, 8, 2, 2, TP>(a, s);
        if (a.pass_rows == 16) return launch_mma<E4M3, D, 2, 8, 3, 1, TP>(a, s);
        return launch_mma<E4M3, D, 4, 8, 3, 1, TP>(a, s);
    } else {
        if (a.pass_rows == 8) return launch_mma<E4M3, D, 1, 8, 2, 1, TP>(a, s);
        if (a.pass_rows == 16) return launch_mma<E4M3, D, 2, 8, 2, 1, TP>(a, s);
        return launch_mma<E4M3, D, 4, 8, 2, 1, TP>(a, s);
    }
}

}  // namespace

int paged_pass_rows(int dtype, int rows) {
    if (dtype == SKV_F32) return kF32Rows;
    return rows <= 8 ? 8 : rows <= 16 ? 16 : 32;
}

cudaError_t launch_paged_attn(const PagedArgs &a, cudaStream_t s) {
    if (a.dtype == SKV_F32) {
        if (a.format == SKV_CACHE_E4M3) return a.d == 128 ? launch_f32<true, 128, 8, 4>(a, s) : launch_f32<true, 64, 8, 4>(a, s);
        return a.d == 128 ? launch_f32<false, 128, 8, 1>(a, s) : launch_f32<false, 64, 8, 2>(a, s);
    }
    if (a.format == SKV_CACHE_E4M3) return a.d == 128 ? launch_rows<true, 128>(a, s) : launch_rows<true, 64>(a, s);
    return a.d == 128 ? launch_rows<false, 128>(a, s) : launch_rows<false, 64>(a, s);
}

}  // namespace skv
