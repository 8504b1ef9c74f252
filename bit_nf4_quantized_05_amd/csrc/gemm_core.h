// The K loop of the BF16 MFMA contractions whose operands come from memory (gemm_nt.hip,
// gated.hip, head_loss.hip): a 256 x 256 tile of P Q^T (+ P2 Q2^T) in the accumulators of a
// workgroup's waves. The tile's place, its rows and what becomes of the sums are the caller's.
#pragma once
#include <hip/hip_runtime.h>

#include "gemm_common.h"
#include "mfma_device.h"

namespace qn {
namespace {

// Two LDS stages as distinct objects, so the compiler can tell that reads of one
// stage do not depend on in-flight direct-to-LDS loads into the other. Each holds
// [P tile | Q tile] = 2 x 2048 chunks = 64 KB.
__shared__ uint4 g_st0[2 * kChunks];
__shared__ uint4 g_st1[2 * kChunks];

// How WM x WN waves share a tile: each owns a (256 / WM) x (256 / WN) sub-tile of 32 x 32
// MFMA tiles and fills SEG 8-row segments of each operand per K-step.
template <int WM, int WN>
struct GemmWaves {
    static constexpr int NW = WM * WN;
    static constexpr int NT = 64 * NW;                 // threads
    static constexpr int TM = BM / WM / 32;            // m sub-tiles per wave
    static constexpr int TN = BN / WN / 32;            // n sub-tiles per wave
    static constexpr int SEG = BM / NW / 8;
};

// acc = the K-steps [kb, ke) of P Q^T, then (lora) the g.kt2 steps of P2 Q2^T; at least one
// step in all. rowP(r), rowQ(r): the row of P and P2 (Q and Q2) that tile row r takes (uint32,
// inside the operand). acc[a][b], lane l: C[m][n .. n + 3] of the four v / 4, at m = l % 32 +
// 32 b + 32 TM wm and n = 8 (v / 4) + 4 (l / 32) + 32 a + 32 TN wn. On return every wave is past
// the last barrier, so the LDS stages are free and no load is in flight.
template <int WM, int WN, bool kRank, class RowP, class RowQ>
__device__ __forceinline__ void gemm_core(const GemmArgs& g, const RowP& rowP, const RowQ& rowQ, int kb, int ke, bool lora,
                                          f32x16 (&acc)[GemmWaves<WM, WN>::TN][GemmWaves<WM, WN>::TM]) {
    using W = GemmWaves<WM, WN>;
    constexpr int TM = W::TM, TN = W::TN, SEG = W::SEG;
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int wm = wave / WN, wn = wave % WN;

    // ---- global -> LDS with buffer_load ... lds (16 B per lane). A tile row is 64
    // bf16 = 128 B = 8 chunks; chunk c of tile row r is stored at c ^ ((r >> 1) & 7).
    // The LDS has 64 banks of 4 B, so two consecutive rows cover all banks once, and
    // 16 lanes reading one logical chunk of 16 consecutive rows hit 16 distinct 4-bank
    // groups. One load fills a 1 KB segment = 8 rows: lane i lands at row i/8,
    // position i%8, so it fetches chunk (i%8) ^ ((r >> 1) & 7). Wave w fills rows
    // 8*SEG*w .. of both operand tiles; the per-lane byte offsets are fixed for the
    // whole K loop, the K position goes in the scalar offset.
    // 128-B rows, chunk c of row r at c ^ ((r >> 1) & 7); segment j = 8 rows starting
    // at 8 (SEG w + j): (r >> 1) & 7 = 4 ((SEG w + j) & 1) + i/16 for lane i.
    const uint32_t kcE = static_cast<uint32_t>((lane & 7) ^ (lane >> 4)) * 16u;
    const uint32_t kcO = static_cast<uint32_t>((lane & 7) ^ (4 | (lane >> 4))) * 16u;
    uint32_t voP[SEG], voQ[SEG], voP2[SEG], voQ2[SEG];
#pragma unroll
    for (int j = 0; j < SEG; ++j) {
        const int rr = 8 * SEG * wave + 8 * j + (lane >> 3);
        const uint32_t kc16 = (((SEG * wave + j) & 1) ? kcO : kcE);
        const uint32_t rp = rowP(rr);
        const uint32_t rq = rowQ(rr);
        voP[j] = rp * static_cast<uint32_t>(g.ldp * 2) + kc16;
        voQ[j] = rq * static_cast<uint32_t>(g.ldq * 2) + kc16;
        voP2[j] = kRank ? rp * static_cast<uint32_t>(g.ldp2 * 2) + kc16 : 0u;
        voQ2[j] = kRank ? rq * static_cast<uint32_t>(g.ldq2 * 2) + kc16 : 0u;
    }
    const __amdgpu_buffer_rsrc_t rsP = make_rsrc(g.P, g.bytesP);
    const __amdgpu_buffer_rsrc_t rsQ = make_rsrc(g.Q, g.bytesQ);
    const __amdgpu_buffer_rsrc_t rsP2 = make_rsrc(kRank ? g.P2 : g.P, kRank ? g.bytesP2 : g.bytesP);
    const __amdgpu_buffer_rsrc_t rsQ2 = make_rsrc(kRank ? g.Q2 : g.Q, kRank ? g.bytesQ2 : g.bytesQ);
    // step k of the loop is main step kb + k while k < ke - kb, then rank step k - (ke - kb)
    const int KT = (ke - kb) + (kRank && lora ? g.kt2 : 0);
    const int kshift = kb;
    const int kmain = ke - kb;

#define QN_ISSUE(KTV, ST)                                                                         \
    {                                                                                             \
        const int kl_ = (KTV);                                                                    \
        uint4* sp_ = (ST) + wave * (64 * SEG);                                                    \
        uint4* sq_ = sp_ + kChunks;                                                               \
        if (!kRank || kl_ < kmain) {                                                              \
            const int so_ = (kl_ + kshift) * (BK * 2);                                            \
            _Pragma("unroll") for (int j = 0; j < SEG; ++j) {                                     \
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsP, (lds_ptr_t)(sp_ + 64 * j), 16, voP[j], so_, 0, 0); \
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsQ, (lds_ptr_t)(sq_ + 64 * j), 16, voQ[j], so_, 0, 0); \
            }                                                                                     \
        } else {                                                                                  \
            const int so_ = (kl_ - kmain) * (BK * 2);                                             \
            _Pragma("unroll") for (int j = 0; j < SEG; ++j) {                                     \
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsP2, (lds_ptr_t)(sp_ + 64 * j), 16, voP2[j], so_, 0, 0); \
                __builtin_amdgcn_raw_ptr_buffer_load_lds(rsQ2, (lds_ptr_t)(sq_ + 64 * j), 16, voQ2[j], so_, 0, 0); \
            }                                                                                     \
        }                                                                                         \
    }

    // ---- fragments: 32-row x 16-K reads per k16 sub-step kk (0..3)
    const uint32_t frow = lane & 31;
    const uint32_t fsw = (frow >> 1) & 7;
    const uint32_t prow = (wm * (TM * 32) + frow) * 8;
    const uint32_t qrow = kChunks + (wn * (TN * 32) + frow) * 8;
    uint32_t chs[4];
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) chs[kk] = (2 * kk + (lane >> 5)) ^ fsw;
#define QN_FRAGS(ST, CH, F)                                             \
    {                                                                   \
        F[0] = (ST)[qrow + (CH)];                                       \
        _Pragma("unroll") for (int i = 0; i < TM; ++i) F[TN + i] = (ST)[prow + i * 256 + (CH)]; \
        _Pragma("unroll") for (int i = 1; i < TN; ++i) F[i] = (ST)[qrow + i * 256 + (CH)];      \
    }

#pragma unroll
    for (int a = 0; a < TN; ++a)
#pragma unroll
        for (int b = 0; b < TM; ++b) acc[a][b] = f32x16{};
#define QN_MFMAS(F)                                                            \
    _Pragma("unroll") for (int a = 0; a < TN; ++a)                             \
        _Pragma("unroll") for (int b = 0; b < TM; ++b)                         \
            acc[a][b] = mfma32(F[a], F[TN + b], acc[a][b]);

    uint4 fa[TM + TN], fb[TM + TN];
    // One K-step on stage CUR (its kk = 0 fragments already in fa) while NXT receives
    // step k+1; NXT last held step k-1, whose reads all finished before the previous
    // step's barrier. Before the last sub-step every wave waits for its own loads and
    // the barrier certifies NXT complete, so NXT's first fragments are read under the
    // last MFMAs; CUR's reads are all done by then, so the next step may refill it.
    // A wave runs its first three sub-steps at raised issue priority and drops it for
    // the barrier, the next step's loads and the sub-step after the barrier, so the
    // waves of a SIMD that are still in their MFMA run go first (2-4 % faster on the
    // 4096^2 layer than equal priority; the results do not change).
#define QN_STEP(KTV, CUR, NXT)                                                 \
    {                                                                          \
        const int k_ = (KTV);                                                  \
        if (k_ + 1 < KT) QN_ISSUE(k_ + 1, NXT)                                 \
        QN_FRAGS(CUR, chs[1], fb)                                              \
        __builtin_amdgcn_s_setprio(1);                                         \
        QN_MFMAS(fa)                                                           \
        QN_INTERLEAVE_DS_MFMA((TM + TN));                                      \
        QN_FRAGS(CUR, chs[2], fa)                                              \
        QN_MFMAS(fb)                                                           \
        QN_INTERLEAVE_DS_MFMA((TM + TN));                                      \
        QN_FRAGS(CUR, chs[3], fb)                                              \
        QN_MFMAS(fa)                                                           \
        QN_INTERLEAVE_DS_MFMA((TM + TN));                                      \
        __builtin_amdgcn_s_setprio(0);                                         \
        __builtin_amdgcn_s_waitcnt(0);                                         \
        QN_BARRIER();                                                          \
        if (k_ + 1 < KT) QN_FRAGS(NXT, chs[0], fa)                             \
        QN_MFMAS(fb)                                                           \
        QN_INTERLEAVE_DS_MFMA((TM + TN));                                      \
    }

    QN_ISSUE(0, g_st0)
    QN_WAIT_VM(0);
    QN_BARRIER();
    QN_FRAGS(g_st0, chs[0], fa)
    int kt = 0;
    for (; kt + 2 <= KT; kt += 2) {
        QN_STEP(kt, g_st0, g_st1)
        QN_STEP(kt + 1, g_st1, g_st0)
    }
    if (kt < KT) QN_STEP(kt, g_st0, g_st1)
#undef QN_STEP
#undef QN_MFMAS
#undef QN_FRAGS
#undef QN_ISSUE
}

}  // namespace
}  // namespace qn
