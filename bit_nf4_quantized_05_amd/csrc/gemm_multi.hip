// BF16 MFMA contraction of the calls with many adapters on gfx950:
//     C[order[p], :] = bf16( P[order[p], K] Q[N, K]^T + T[p, r] R_a[N, r]^T )
// for the positions p of a batch sorted by adapter, a the adapter of position p:
//     forward : P = X,  Q = W_hat,    T = s_a A_a x,    R_a = B_a
//     dX      : P = dY, Q = W_hat^T,  T = s_a B_a^T dy, R_a = A_a^T
// (A_a itself is read, rank-major: its rows go to LDS as they are and transposing reads hand
// out the fragments). T comes as two bf16 terms, 16 bits: with one term its 2^-9 would show in
// the output, whose own rounding is no coarser.
//
// The main K-steps are those of the single-adapter GEMM (256 x 256 tiles, 8 waves of
// 128 x 64, K-steps of 64 double-buffered in LDS by direct loads, swizzled rows; the
// reasons are told there); only the token rows of P are gathered and those of C scattered
// through the plan's order, each lane loading the tokens of its 4 rows once. Sorting keeps
// the adapters per tile few: over all tile rows there are at most (tile rows + adapters in
// use) pairs, however the requests came in.
//
// Rank steps. After the last main step a tile walks the adapters with tokens in it, 16 ranks
// of 4 adapters or 32 of 2 a step (as many loads as of one term and 64 ranks of one), double-buffered in the same stages (the first
// one's loads go out under the last main step). A 32-row MFMA tile skips an adapter that has
// none of its rows, adds straight to its accumulators when all 32 rows are the adapter's, and
// otherwise forms the product apart and adds it where the lane's row is the adapter's. So a row
// only ever meets its own adapter: zeros in place of the other rows would let an infinity or NaN in
// one adapter's weights reach its neighbours' tokens, and this costs fewer MFMAs besides.
//
// The last round of tiles, at most 128 past a multiple of the 256 CUs, as whole tiles would
// leave half the CUs idle (last_tiles has the rule):
//   half tiles of 128 x 256: a half tile's step takes 0.6 of a whole one's (4 LDS reads for 4
//   MFMAs, not 6 for 8), more than half, so whole tiles stay the rule (4096 x 4096 at 4096
//   tokens: 119 us whole, 133 us in halves);
//   K split in up to 16, gemm_multi_reduce adding the partials, and so are the adapters (256
//   tokens of 256 users, 16 tiles: 64 rank steps of 2.6 us would stand in one split's way).
//   Each XCD takes a run of neighbouring tiles of one slice: dealt out in turn, 800 x 11008 x
//   4096 took 166 us in place of 112.
// Alone they run on three stages of 48 KB, whose loads have two steps to arrive (1531 x 4096
// x 4096, 96 tiles: 59 us; two stages 73; whole, split in two 77 and 13 for the sums); after whole
// tiles, in the same launch, on the two stages of those (11008 columns of 2048 tokens, 256 +
// 88 tiles: 174 us; in two launches 124 + 58; split 170 + 12).
// Dealing the last tiles' steps out evenly over all CUs, parts joined by the last workgroup
// to finish, was slower than the split: 112 us for the 96 tiles (127 us with device-scope
// fences in place of write-through stores), for 88 MB of partials.
#include <hip/hip_runtime.h>

#include "gemm_common.h"
#include "internal.h"
#include "mfma_device.h"
#include "multi.h"
#include "nf4_device.h"

#include <algorithm>

namespace qn {
namespace {

__shared__ uint4 g_st0[2 * kChunks];
__shared__ uint4 g_st1[2 * kChunks];
// half tiles: three stages of [P 128 rows | Q 256 rows], distinct objects as above
constexpr int kHalfStage = kChunks / 2 + kChunks;
__shared__ uint4 g_h0[kHalfStage];
__shared__ uint4 g_h1[kHalfStage];
__shared__ uint4 g_h2[kHalfStage];
// the adapters with tokens in the tile: which, and their positions [lo, hi)
__shared__ int g_ad[BM];
__shared__ int g_lo[BM];
__shared__ int g_hi[BM];

constexpr int kWM = 2, kWN = 4;                 // waves
constexpr int kNT = 64 * kWM * kWN;             // threads
constexpr int kMaxSplits = 16;                  // of a tile's K-steps

struct MultiGemm {
    GemmArgs g;                                 // P, Q, C, sizes, splits
    MultiPlan plan;
    const uint16_t* T;                          // [2][M, r]: two bf16 terms
    const uint16_t* R;                          // [adapters, N, r], or [adapters, r, N]
    int r;
};

// LDS reads and MFMAs of a k16 sub-step in turn: one read, then PER MFMAs, N times
#define QN_INTERLEAVE(N, PER)                                     \
    _Pragma("unroll") for (int _i = 0; _i < (N); ++_i) {          \
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);        \
        __builtin_amdgcn_sched_group_barrier(0x008, PER, 0);      \
    }

// BMT rows per tile: 256, or 128. Half tiles are the two halves of each of the last g.rem tiles
// or, alone on three LDS stages (kThree), g.rem tiles of their own raster (g.tiles_m rows of 128)
template <int BMT, bool kSplit, bool kThree, bool kRankMajor>
__device__ __forceinline__ void gemm_multi_body(const MultiGemm& mg, int bid) {
    const GemmArgs& g = mg.g;
    constexpr bool kHalf = BMT < BM;
    static_assert(!(kHalf && kSplit) || kThree, "half tiles split in K are alone");
    static_assert(kHalf || !kThree, "three stages hold half tiles only");
    constexpr int TM = BMT / kWM / 32;          // 4 (2) m sub-tiles per wave
    constexpr int TN = BN / kWN / 32;           // 2 n sub-tiles
    constexpr int SEGP = BMT / (kWM * kWN) / 8; // 4 (2) 8-row load segments of P per wave
    constexpr int SEG = BN / (kWM * kWN) / 8;   // 4 of Q
    constexpr int kPer = kHalf ? 1 : 2;         // MFMAs per LDS read
    constexpr int kQ = kThree ? kChunks / 2 : kChunks;   // Q's place in a stage
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave / kWN, wn = wave % kWN;
    const int M = g.M, N = g.N;

    const bool split_wg = kSplit && bid >= g.full;
    const int T = kHalf && !kThree ? 2 * g.rem : split_wg || kThree ? g.rem : g.full;   // tiles of this kind
    // Workgroups go to the 8 XCDs in turn: each takes a run of neighbouring tiles (of one
    // K-slice after the other), whose rows of P and Q its L2 then holds for all of them
    // (g.full is a multiple of 256 here; past the last slice: nothing)
    const int w = split_wg ? bid - g.full : bid;
    const int units = split_wg ? T * g.splits : T;
    const int run = split_wg ? (units + 7) >> 3 : units >> 3;
    const int u = split_wg || T % 8 == 0 ? (w & 7) * run + (w >> 3) : w;
    if (split_wg && u >= units) return;
    const int sk = split_wg ? u / T : 0;
    const int place = split_wg ? u % T : u;
    const int logical = kHalf && !kThree ? g.full + place / 2 : split_wg ? g.full + place : place;
    int tm, tn;
    tile_coords(g, logical, tm, tn);
    const int m0 = kThree ? tm * BMT : tm * BM + (kHalf ? (place & 1) * BMT : 0), n0 = tn * BN;
    if (kHalf && !kThree && m0 >= M) return;

    // this tile's adapters, one a thread (at most one per row); sorted out below, under the
    // first loads
    const int2 kr = mg.plan.tile[m0 / BM];
    const int mine = mg.plan.used[min(kr.x + tid, max(kr.y, 1) - 1)];

    const uint32_t kcE = static_cast<uint32_t>((lane & 7) ^ (lane >> 4)) * 16u;
    const uint32_t kcO = static_cast<uint32_t>((lane & 7) ^ (4 | (lane >> 4))) * 16u;
    uint32_t voP[SEGP], voQ[SEG];
#pragma unroll
    for (int j = 0; j < SEGP; ++j) {
        const int rr = 8 * SEGP * wave + 8 * j + (lane >> 3);
        const uint32_t rp = static_cast<uint32_t>(mg.plan.order[min(m0 + rr, M - 1)]);
        voP[j] = rp * static_cast<uint32_t>(g.ldp * 2) + (((SEGP * wave + j) & 1) ? kcO : kcE);
    }
#pragma unroll
    for (int j = 0; j < SEG; ++j) {
        const int rr = 8 * SEG * wave + 8 * j + (lane >> 3);
        const uint32_t rq = static_cast<uint32_t>(min(n0 + rr, N - 1));
        voQ[j] = rq * static_cast<uint32_t>(g.ldq * 2) + (((SEG * wave + j) & 1) ? kcO : kcE);
    }
    const __amdgpu_buffer_rsrc_t rsP = make_rsrc(g.P, g.bytesP);
    const __amdgpu_buffer_rsrc_t rsQ = make_rsrc(g.Q, g.bytesQ);
    const int kb = split_wg ? sk * g.kper : 0;
    const int ke = split_wg ? min(kb + g.kper, g.kt1) : g.kt1;
    const int KT = ke - kb;

#define QN_ISSUE(KTV, ST)                                                                         \
    {                                                                                             \
        uint4* sp_ = (ST) + wave * (64 * SEGP);                                                   \
        uint4* sq_ = (ST) + kQ + wave * (64 * SEG);                                          \
        const int so_ = ((KTV) + kb) * (BK * 2);                                                  \
        _Pragma("unroll") for (int j = 0; j < SEG; ++j) {                                         \
            if (j < SEGP)                                                                         \
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsP, (lds_ptr_t)(sp_ + 64 * j), 16, voP[j < SEGP ? j : 0], so_, 0, 0); \
            __builtin_amdgcn_raw_ptr_buffer_load_lds(rsQ, (lds_ptr_t)(sq_ + 64 * j), 16, voQ[j], so_, 0, 0); \
        }                                                                                         \
    }

    if constexpr (kThree) {
        QN_ISSUE(0, g_h0)
        if (KT > 1) QN_ISSUE(1, g_h1)
    } else {
        QN_ISSUE(0, g_st0)
    }
    // the list g_ad, g_lo, g_hi of the adapters with `steps` rank steps in all (seen by all after
    // the first barrier)
    int first = 0, used = kr.y - kr.x;
    int lo_mine = 0, hi_mine = 0;
    const bool in = tid < used;
    if (in) {
        lo_mine = mg.plan.start[mine];
        hi_mine = mg.plan.start[mine + 1];
    }
    if constexpr (kHalf) {                      // those of this half alone
        first = __syncthreads_count(in && hi_mine <= m0);
        used -= first + __syncthreads_count(in && lo_mine >= m0 + BMT);
    }
    if (split_wg) {                             // this split's share of them
        const int all = used;
        first += all * sk / g.splits;
        used = all * (sk + 1) / g.splits - all * sk / g.splits;
    }
    if (tid >= first && tid < first + used) {
        g_ad[tid - first] = mine;
        g_lo[tid - first] = lo_mine;
        g_hi[tid - first] = hi_mine;
    }
    // a rank step holds 64 rows of R: 16 ranks of 4 adapters or 32 of 2 (8 << sh ranks each), jsteps
    // steps per adapter of more than 32; and beside them both terms of T at those ranks
    const int sh = mg.r == 16 ? 1 : 2;
    const int per = 8 >> sh;
    const int jsteps = (mg.r + (8 << sh) - 1) / (8 << sh);
    const int steps = (used + per - 1) / per * jsteps;

    // Rank step S into stage ST: ranks j0 .. of T's rows (8 << sh of the first term, then the
    // second's, over and over) and of the rows of R of its adapters. Pieces past r re-read the last
    // one, adapters past the last re-read it (no MFMA reads either); the addresses are formed
    // from an opaque copy of the lane index, so they hold no registers through the main steps.
    auto issue_rank = [&](int s, uint4* st) {
        const int j0 = (s % jsteps) * (8 << sh), k0 = s / jsteps * per;
        int ln = lane;
        asm volatile("" : "+v"(ln));
        uint4* sp = st + wave * (64 * SEGP);
        uint4* sq = st + kQ + wave * (64 * SEG);
        const int last = mg.r / 8 - 1 - j0 / 8;
#pragma unroll
        for (int j = 0; j < SEGP; ++j) {
            const int rr = 8 * SEGP * wave + 8 * j + (ln >> 3);
            const int c = (ln & 7) ^ ((rr >> 1) & 7);
            const int64_t row = min(m0 + rr, M - 1) + ((c >> sh) & 1 ? static_cast<int64_t>(M) : 0);
            load_lds16(mg.T + row * mg.r + j0 + 8 * min(c & ((1 << sh) - 1), last), sp + 64 * j);
        }
#pragma unroll
        for (int j = 0; j < SEG; ++j) {
            if constexpr (kRankMajor) {
                // 2 rank rows of 256 columns a segment, 16-byte piece c of rank k at c ^ 2 (k % 4)
                const int k = 2 * (SEG * wave + j) + (ln >> 5);
                const int n = min(n0 + 8 * ((ln & 31) ^ (2 * (k & 3))), N - 8);
                const int64_t a = g_ad[min(k0 + (k >> (sh + 3)), used - 1)];
                load_lds16(mg.R + (a * mg.r + min(j0 + (k & ((8 << sh) - 1)), mg.r - 1)) * N + n, sq + 64 * j);
            } else {
                const int rr = 8 * SEG * wave + 8 * j + (ln >> 3);
                const int c = (ln & 7) ^ ((rr >> 1) & 7);
                const int64_t a = g_ad[min(k0 + (c >> sh), used - 1)];
                load_lds16(mg.R + (a * N + min(n0 + rr, N - 1)) * mg.r + j0 + 8 * min(c & ((1 << sh) - 1), last),
                           sq + 64 * j);
            }
        }
    };

    const uint32_t frow = lane & 31;
    const uint32_t fsw = (frow >> 1) & 7;
    const uint32_t prow = (wm * (TM * 32) + frow) * 8;
    const uint32_t qrow = kQ + (wn * (TN * 32) + frow) * 8;
    uint32_t chs[4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) chs[kk] = (2 * kk + (lane >> 5)) ^ fsw;
#define QN_FRAGS(ST, CH, F)                                             \
    {                                                                   \
        F[0] = (ST)[qrow + (CH)];                                       \
        _Pragma("unroll") for (int i = 0; i < TM; ++i) F[TN + i] = (ST)[prow + i * 256 + (CH)]; \
        _Pragma("unroll") for (int i = 1; i < TN; ++i) F[i] = (ST)[qrow + i * 256 + (CH)];      \
    }

    f32x16 acc[TN][TM];
#pragma unroll
    for (int a = 0; a < TN; ++a)
#pragma unroll
        for (int b = 0; b < TM; ++b) acc[a][b] = f32x16{};
#define QN_MFMAS(F)                                                            \
    _Pragma("unroll") for (int a = 0; a < TN; ++a)                             \
        _Pragma("unroll") for (int b = 0; b < TM; ++b)                         \
            acc[a][b] = mfma32(F[a], F[TN + b], acc[a][b]);

    uint4 fa[TM + TN], fb[TM + TN];
#define QN_STEP(ISSUE, CUR, NXT, NEXT_FRAGS)                                   \
    {                                                                          \
        ISSUE;                                                                 \
        QN_FRAGS(CUR, chs[1], fb)                                              \
        __builtin_amdgcn_s_setprio(1);                                         \
        QN_MFMAS(fa)                                                           \
        QN_INTERLEAVE(TM + TN, kPer);                                         \
        QN_FRAGS(CUR, chs[2], fa)                                              \
        QN_MFMAS(fb)                                                           \
        QN_INTERLEAVE(TM + TN, kPer);                                         \
        QN_FRAGS(CUR, chs[3], fb)                                              \
        QN_MFMAS(fa)                                                           \
        QN_INTERLEAVE(TM + TN, kPer);                                         \
        __builtin_amdgcn_s_setprio(0);                                         \
        __builtin_amdgcn_s_waitcnt(0);                                         \
        QN_BARRIER();                                                          \
        NEXT_FRAGS                                                             \
        QN_MFMAS(fb)                                                           \
        QN_INTERLEAVE(TM + TN, kPer);                                         \
    }
#define QN_MAIN(K, CUR, NXT) QN_STEP(QN_ISSUE((K) + 1, NXT), CUR, NXT, QN_FRAGS(NXT, chs[0], fa))
#define QN_LAST(CUR, NXT) QN_STEP(if (steps > 0) issue_rank(0, NXT), CUR, NXT, )

    int stage = 0;                              // the stage of rank step 0, of two
    auto third = [&](int v) { return v % 3 == 0 ? g_h0 : v % 3 == 1 ? g_h1 : g_h2; };   // of step v, of three
    if constexpr (kThree) {
        // Three stages, main and rank steps in one sequence: a step waits for its own stage only
        // (the 6 loads of the next may be in flight), passes the barrier that certifies it for all
        // waves and the stage of the step before as read, and sends the loads of the step after
        // next into that one.
#define QN_HALF(K, CUR, FREE, MORE)                                            \
    {                                                                          \
        if (MORE || (K) + 1 < KT + steps) QN_WAIT_VM(SEGP + SEG); else QN_WAIT_VM(0); \
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");        \
        if (MORE || (K) + 2 < KT) QN_ISSUE((K) + 2, FREE)                      \
        else if ((K) + 2 < KT + steps) issue_rank((K) + 2 - KT, FREE);         \
        QN_FRAGS(CUR, chs[0], fa)                                              \
        QN_FRAGS(CUR, chs[1], fb)                                              \
        __builtin_amdgcn_s_setprio(1);                                         \
        QN_MFMAS(fa)                                                           \
        QN_FRAGS(CUR, chs[2], fa)                                              \
        QN_INTERLEAVE(TM + TN, kPer)                                           \
        QN_MFMAS(fb)                                                           \
        QN_FRAGS(CUR, chs[3], fb)                                              \
        QN_INTERLEAVE(TM + TN, kPer)                                           \
        QN_MFMAS(fa)                                                           \
        QN_MFMAS(fb)                                                           \
        __builtin_amdgcn_s_setprio(0);                                         \
    }
        if (KT == 1 && steps > 0) {             // step 1 is a rank step
            __syncthreads();                    // (the list)
            issue_rank(0, g_h1);
        }
        int k = 0;
        // (no condition inside the loop: with one the compiler, not knowing how many loads are
        // in flight, waited for nearly all of them; it still does once per turn, hence six
        // steps to a turn)
        for (; k + 8 <= KT; k += 6) {
            QN_HALF(k, g_h0, g_h2, true)
            QN_HALF(k + 1, g_h1, g_h0, true)
            QN_HALF(k + 2, g_h2, g_h1, true)
            QN_HALF(k + 3, g_h0, g_h2, true)
            QN_HALF(k + 4, g_h1, g_h0, true)
            QN_HALF(k + 5, g_h2, g_h1, true)
        }
        for (; k < KT; k += 3) {
            QN_HALF(k, g_h0, g_h2, false)
            if (k + 1 < KT) QN_HALF(k + 1, g_h1, g_h0, false)
            if (k + 2 < KT) QN_HALF(k + 2, g_h2, g_h1, false)
        }
#undef QN_HALF
    } else {
        stage = KT & 1;
        __builtin_amdgcn_s_waitcnt(0);          // (the adapter list's LDS writes too)
        QN_BARRIER();
        QN_FRAGS(g_st0, chs[0], fa)
        // the last main step stands outside the loop, which then has no branch in it
        int kt = 0;
        for (; kt + 2 < KT; kt += 2) {
            QN_MAIN(kt, g_st0, g_st1)
            QN_MAIN(kt + 1, g_st1, g_st0)
        }
        if (kt + 1 < KT) QN_MAIN(kt, g_st0, g_st1)
        const uint4* cur = (KT & 1) ? g_st0 : g_st1;
        uint4* nxt = (KT & 1) ? g_st1 : g_st0;
        QN_LAST(cur, nxt)
    }
#undef QN_LAST
#undef QN_MAIN
#undef QN_STEP
#undef QN_MFMAS
#undef QN_FRAGS
#undef QN_ISSUE

    // ---- rank steps. Of three stages they go on as the main steps. Of two, step 0 is in the
    // stage the last main step did not read, and complete (that step's wait and barrier); each
    // step: the next one's loads, this one's products, then every wave's loads and LDS reads
    // are waited for before the barrier.
    for (int s = 0; s < steps; ++s) {
        const uint4* cur;
        if constexpr (kThree) {
            if (s + 1 < steps) QN_WAIT_VM(SEGP + SEG); else QN_WAIT_VM(0);
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            if (s + 2 < steps) issue_rank(s + 2, third(KT + s + 2));
            cur = third(KT + s);
        } else {
            cur = ((stage + s) & 1) ? g_st1 : g_st0;
            if (s + 1 < steps) issue_rank(s + 1, ((stage + s) & 1) ? g_st0 : g_st1);
        }
        const int k0 = s / jsteps * per;
        const int subs = min(8 << sh, mg.r - (s % jsteps) * (8 << sh)) / 16;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
            // sub-step kk: 16 ranks of adapter k0 + (kk >> (sh - 1)), both terms of T at them
            const int k = k0 + (kk >> (sh - 1));
            if (k >= used || (sh == 2 && (kk & 1) >= subs)) continue;
            const uint32_t term0 = sh == 1 ? chs[0] : chs[kk & 1], term1 = sh == 1 ? chs[1] : chs[2 + (kk & 1)];
            const int lo = __builtin_amdgcn_readfirstlane(g_lo[k]), hi = __builtin_amdgcn_readfirstlane(g_hi[k]);
            const int w0 = m0 + wm * (TM * 32);
            if (w0 >= hi || w0 + TM * 32 <= lo) continue;                // none of the wave's positions
            uint4 q[TN];
            if constexpr (kRankMajor) {
                const int kr0 = 16 * kk + 8 * (lane >> 5) + ((lane >> 2) & 3);
                uint32_t qa[TN];
#pragma unroll
                for (int a = 0; a < TN; ++a) {
                    const int n = wn * (TN * 32) + a * 32 + 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
                    qa[a] = lds_addr(cur + kQ) + kr0 * 512 + ((((n >> 3) ^ (2 * (kr0 & 3))) << 4) | ((n & 7) << 1));
                }
                static_assert(TN == 2, "two column tiles");
                unsigned long long v[4];
                asm volatile("ds_read_b64_tr_b16 %0, %4\n\tds_read_b64_tr_b16 %1, %4 offset:2048\n\t"
                             "ds_read_b64_tr_b16 %2, %5\n\tds_read_b64_tr_b16 %3, %5 offset:2048\n\t"
                             "s_waitcnt lgkmcnt(0)"
                             : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]) : "v"(qa[0]), "v"(qa[1]) : "memory");
#pragma unroll
                for (int a = 0; a < TN; ++a)
                    q[a] = uint4{static_cast<uint32_t>(v[2 * a]), static_cast<uint32_t>(v[2 * a] >> 32),
                                 static_cast<uint32_t>(v[2 * a + 1]), static_cast<uint32_t>(v[2 * a + 1] >> 32)};
            } else {
#pragma unroll
                for (int a = 0; a < TN; ++a) q[a] = cur[qrow + a * 256 + chs[kk]];
            }
#pragma unroll
            for (int b = 0; b < TM; ++b) {
                const int p0 = w0 + b * 32;                              // the sub-tile's positions p0 .. p0 + 31
                if (p0 >= hi || p0 + 32 <= lo) continue;                 // wave-uniform
                const uint4 p = cur[prow + b * 256 + term0], e = cur[prow + b * 256 + term1];
                if (p0 >= lo && p0 + 32 <= hi) {
#pragma unroll
                    for (int a = 0; a < TN; ++a) acc[a][b] = mfma32(q[a], p, mfma32(q[a], e, acc[a][b]));
                } else {
                    const bool mine = p0 + static_cast<int>(frow) >= lo && p0 + static_cast<int>(frow) < hi;
#pragma unroll
                    for (int a = 0; a < TN; ++a) {
                        const f32x16 t = mfma32(q[a], p, mfma32(q[a], e, f32x16{}));
#pragma unroll
                        for (int i = 0; i < 16; ++i) acc[a][b][i] = mine ? acc[a][b][i] + t[i] : acc[a][b][i];
                    }
                }
            }
        }
        if constexpr (!kThree) {
            __builtin_amdgcn_s_waitcnt(0);
            QN_BARRIER();
        }
    }
    // (the last step's LDS reads, before the epilogue writes there)
    if constexpr (kThree) asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");

    if (split_wg) {
        float* pt = g.part + (static_cast<int64_t>(sk) * T + place) * (BMT * BN);
#pragma unroll
        for (int b = 0; b < TM; ++b) {
            const int ml = wm * (TM * 32) + b * 32 + static_cast<int>(frow);
            if (m0 + ml >= M) continue;
#pragma unroll
            for (int a = 0; a < TN; ++a) {
#pragma unroll
                for (int gq = 0; gq < 4; ++gq) {
                    const int nl = wn * (TN * 32) + a * 32 + 8 * gq + 4 * (lane >> 5);
                    *reinterpret_cast<float4*>(pt + ml * BN + nl) =
                        float4{acc[a][b][4 * gq], acc[a][b][4 * gq + 1], acc[a][b][4 * gq + 2], acc[a][b][4 * gq + 3]};
                }
            }
        }
        return;
    }
    // ---- epilogue: the bf16 tile through LDS (conflict-free, as the single-adapter GEMM),
    // then each row as 512 contiguous bytes to its token's row of C
    constexpr int kRowsIn = (kThree ? 64 : 128) - 1;     // rows of the tile in one stage, less 1
#pragma unroll
    for (int b = 0; b < TM; ++b) {
        const int rl = wm * (TM * 32) + b * 32 + static_cast<int>(frow);
        uint4* arr = kThree ? ((rl >> 6) ? g_h1 : g_h0) : (rl >> 7) ? g_st1 : g_st0;
        char* rowp = reinterpret_cast<char*>(arr) + (rl & kRowsIn) * 512;
#pragma unroll
        for (int a = 0; a < TN; ++a) {
#pragma unroll
            for (int gq = 0; gq < 4; ++gq) {
                const int nl = wn * (TN * 32) + a * 32 + 8 * gq + 4 * (lane >> 5);
                uint2 o;
                o.x = pack_bf16x2(acc[a][b][4 * gq + 0], acc[a][b][4 * gq + 1]);
                o.y = pack_bf16x2(acc[a][b][4 * gq + 2], acc[a][b][4 * gq + 3]);
                *reinterpret_cast<uint2*>(rowp + (((nl >> 3) ^ (rl & 31)) << 4) + ((nl & 7) << 1)) = o;
            }
        }
    }
    __syncthreads();
    const int cj = tid & 31;
    constexpr int kRowsPerPass = kNT / 32;
#pragma unroll 4
    for (int i = 0; i < BMT / kRowsPerPass; ++i) {
        const int r = i * kRowsPerPass + (tid >> 5);
        const uint4* arr = kThree ? ((r >> 6) ? g_h1 : g_h0) : (r >> 7) ? g_st1 : g_st0;
        const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(arr) + (r & kRowsIn) * 512 +
                                                        ((cj ^ (r & 31)) << 4));
        const int m = m0 + r;
        const int n = n0 + cj * 8;
        if (m < M && n < N)
            *reinterpret_cast<uint4*>(g.C + static_cast<int64_t>(mg.plan.order[m]) * g.ldc + n) = v;
    }
}

// The kernels, for R as rows (forward) and rank-major (input gradient):
//   kernel  whole tiles
//   split   whole tiles, then the last ones split in K
//   mixed   whole tiles, then the last ones as half tiles on the same two stages
//   half    half tiles alone, on three stages
//   half_split  these split in K
#define QN_MULTI_KERNELS(SUFFIX, RANK_MAJOR)                                                          \
    __global__ __launch_bounds__(kNT, 1) void gemm_multi_kernel##SUFFIX(MultiGemm mg) {                \
        gemm_multi_body<BM, false, false, RANK_MAJOR>(mg, static_cast<int>(blockIdx.x));               \
    }                                                                                                 \
    __global__ __launch_bounds__(kNT, 1) void gemm_multi_split##SUFFIX(MultiGemm mg) {                 \
        gemm_multi_body<BM, true, false, RANK_MAJOR>(mg, static_cast<int>(blockIdx.x));                \
    }                                                                                                 \
    __global__ __launch_bounds__(kNT, 1) void gemm_multi_mixed##SUFFIX(MultiGemm mg) {                 \
        const int bid = static_cast<int>(blockIdx.x);                                                 \
        if (bid < mg.g.full) gemm_multi_body<BM, false, false, RANK_MAJOR>(mg, bid);                   \
        else gemm_multi_body<BM / 2, false, false, RANK_MAJOR>(mg, bid - mg.g.full);                   \
    }                                                                                                 \
    __global__ __launch_bounds__(kNT, 1) void gemm_multi_half##SUFFIX(MultiGemm mg) {                  \
        gemm_multi_body<BM / 2, false, true, RANK_MAJOR>(mg, static_cast<int>(blockIdx.x));            \
    }                                                                                                 \
    __global__ __launch_bounds__(kNT, 1) void gemm_multi_half_split##SUFFIX(MultiGemm mg) {            \
        gemm_multi_body<BM / 2, true, true, RANK_MAJOR>(mg, static_cast<int>(blockIdx.x));             \
    }
QN_MULTI_KERNELS(, false)
QN_MULTI_KERNELS(_dx, true)
#undef QN_MULTI_KERNELS

// Split tiles of `rows` rows (g.tiles_m counts those): C[order[m], n..n+3] = bf16(sum of the
// tile's partials in split order), 4 rows per workgroup
__global__ __launch_bounds__(256)
void gemm_multi_reduce(MultiGemm mg, int rows) {
    const GemmArgs& g = mg.g;
    const int per = rows / 4;
    const int j = static_cast<int>(blockIdx.x) / per;
    const int ml = (static_cast<int>(blockIdx.x) % per) * 4 + (threadIdx.x >> 6);
    const int nl = (threadIdx.x & 63) * 4;
    int tm, tn;
    tile_coords(g, g.full + j, tm, tn);
    const int m = tm * rows + ml, n = tn * BN + nl;
    if (m >= g.M || n >= g.N) return;
    const int64_t row = mg.plan.order[m];
    const float4 t = ordered_sum4<8>(g.part + (static_cast<int64_t>(j) * rows + ml) * BN + nl,
                                     static_cast<int64_t>(g.rem) * rows * BN, g.splits);
    *reinterpret_cast<uint2*>(g.C + row * g.ldc + n) = uint2{pack_bf16x2(t.x, t.y), pack_bf16x2(t.z, t.w)};
}

// What becomes of the tiles past a multiple of 256 (if at most 128; more run whole): rem tiles
// of `rows` rows, 256 or 128, with K split in `splits`; half tiles beside whole ones (full > 0)
// stay pairs, and rem counts the pairs.
struct LastTiles { int full, rem, rows, splits, kper; };

// Counted in K-steps of a whole tile (1.5 us): a half tile's takes 0.6; the launch that adds the
// partials takes 8 (its start included) and one for every 14 partials of 256 KB. Half tiles are
// split only where no whole tiles run beside them. (Calls at 4096 x 4096: 100 tokens 33.9 us in
// split halves, 36.4 split whole, 47.0 whole in four; 256 tokens 39.1, 43.4 and 48.4; 1000 tokens
// 60.5 either way, 70.3 whole in four. 1000 tokens on 1024 x 1024 25.5 in halves, 35.3 whole in two.)
LastTiles last_tiles(int64_t M, int64_t N, int64_t K) {
    const int64_t tm = (M + BM - 1) / BM, tn = (N + BN - 1) / BN, tiles = tm * tn;
    const int64_t rem = tiles % 256, kt = K / BK;
    LastTiles best{static_cast<int>(tiles), 0, BM, 1, static_cast<int>(kt)};
    if (rem == 0 || rem > 128) return best;
    double cost = 1e30;
    for (const int rows : {BM / 2, BM}) {
        const bool alone = tiles == rem;
        const int64_t count = rows == BM || !alone ? rem : (M + rows - 1) / rows * tn;
        const int64_t most = rows == BM || alone ? std::min<int64_t>({kMaxSplits, 256 / count, kt / 4}) : 1;
        for (int64_t s = 1; s <= std::max<int64_t>(1, most); ++s) {
            const int64_t kper = (kt + s - 1) / s;
            if ((kt + kper - 1) / kper != s) continue;                  // a split would be empty
            double c = (rows == BM ? 1.0 : 0.6) * static_cast<double>(kper);
            if (s > 1) c += 8.0 + static_cast<double>(count * s * rows) / (14.0 * BM);
            if (c < cost) {
                cost = c;
                best = LastTiles{static_cast<int>(tiles - rem), static_cast<int>(count), rows, static_cast<int>(s),
                                 static_cast<int>(kper)};
            }
        }
    }
    if (best.rows == BM && best.splits == 1) best = LastTiles{static_cast<int>(tiles), 0, BM, 1, static_cast<int>(kt)};
    return best;
}

}  // namespace

int64_t gemm_multi_part_floats(int64_t M, int64_t N, int64_t K) {
    const LastTiles lt = last_tiles(M, N, K);
    return lt.splits > 1 ? static_cast<int64_t>(lt.splits) * lt.rem * lt.rows * BN : 0;
}

hipError_t launch_gemm_multi(const uint16_t* P, int64_t ldp, const uint16_t* Q, int64_t K, const uint16_t* T,
                             const uint16_t* R, bool rank_major, int r, const MultiPlan& plan, uint16_t* C,
                             int64_t ldc, int64_t M, int64_t N, float* part, hipStream_t st) {
    MultiGemm mg{};
    GemmArgs& g = mg.g;
    g.tiles_m = static_cast<int>((M + BM - 1) / BM);
    g.tiles_n = static_cast<int>((N + BN - 1) / BN);
    g.P = P; g.ldp = ldp; g.Q = Q; g.ldq = K; g.kt1 = static_cast<int>(K / BK);
    g.C = C; g.ldc = ldc; g.M = static_cast<int>(M); g.N = static_cast<int>(N);
    g.bytesP = static_cast<uint32_t>(2 * ldp * M);
    g.bytesQ = static_cast<uint32_t>(2 * K * N);
    mg.plan = plan; mg.T = T; mg.R = R; mg.r = r;
    const int tiles = g.tiles_m * g.tiles_n;
    g.part = part;
#define QN_GEMM(KERNEL, GRID)                                                                          \
    do {                                                                                               \
        if (rank_major) QN_LAUNCH(#KERNEL "_dx", st, KERNEL##_dx, dim3(GRID), dim3(kNT), 0, st, mg);     \
        else QN_LAUNCH(#KERNEL, st, KERNEL, dim3(GRID), dim3(kNT), 0, st, mg);                          \
    } while (0)
    const LastTiles lt = last_tiles(M, N, K);
    g.full = lt.full; g.rem = lt.rem; g.splits = lt.splits; g.kper = lt.kper;
    if (lt.rem == 0) QN_GEMM(gemm_multi_kernel, tiles);
    else if (lt.rows == BM) QN_GEMM(gemm_multi_split, g.full + (g.rem * g.splits + 7) / 8 * 8);
    else if (g.full > 0) QN_GEMM(gemm_multi_mixed, g.full + 2 * g.rem);
    else {
        g.tiles_m = static_cast<int>((M + lt.rows - 1) / lt.rows);
        if (lt.splits > 1) QN_GEMM(gemm_multi_half_split, (g.rem * g.splits + 7) / 8 * 8);
        else QN_GEMM(gemm_multi_half, g.rem);
    }
#undef QN_GEMM
    if (g.splits > 1)
        QN_LAUNCH("gemm_multi_reduce", st, gemm_multi_reduce, dim3(static_cast<unsigned>(g.rem * (lt.rows / 4))),
                  dim3(256), 0, st, mg, lt.rows);
    return hipGetLastError();
}

}  // namespace qn
