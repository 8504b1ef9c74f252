// The K loop of small BF16 MFMA contractions (head_loss.hip, gated.hip): a 64 x 64 tile of
// P Q^T (+ P2 Q2^T), operands as in gemm_turns.h, by a workgroup of 4 waves (32 x 32 each).
//
// For products with too few 256 x 256 tiles to fill the chip, and those whose time is the stream of Q
// past few rows of P. What such a tile costs is latency, so it keeps loads in flight: K-steps of 64 in a
// ring of 4 stages (16 KB each), three of them on their way while one is multiplied, one barrier a
// step; two workgroups fit a CU, 96 KB in flight. Each value read from LDS feeds 2 MFMAs, so the LDS
// holds it to about half of what the large tile's waves reach.
#pragma once
#include "gemm_turns.h"

namespace qn {

constexpr int kFewTile = 64, kFewThreads = 256, kFewStages = 4;

namespace {

__shared__ uint4 g_few[kFewStages * 1024];           // stage: 64 rows of P, then Q; 8 KB each

// The sums of a wave: acc[0][0][i][j], lane l, is C[m][n .. n + 3] with m = 32 wm + 16 i + l % 16 and
// n = 32 wn + 16 j + 4 (l / 16), wm = wave / 2, wn = wave % 2.
typedef f32x4t FewSums[1][1][2][2];

// As gemm_turns, of a tile of 64 rows of P and of Q.
template <bool kRank, bool kQCols, class RowP, class RowQ>
__device__ __forceinline__ void gemm_few(const TurnArgs& g, const RowP& rowP, const RowQ& rowQ, int kb, int ke, bool rank,
                                         FewSums& acc) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 1, wn = wave & 1;
    const uint32_t lds = lds_addr(g_few);

    // rows of 128 B, chunk c of row r at c ^ ((r >> 1) & 7); an instruction fills 8 rows, wave w rows 16 w .. + 15.
    // K-major Q: 64 k-rows of 4 units of 32 B, unit u of row k at u ^ swz(k): the 8 rows that 32 lanes of a
    // transposing read take (4 of each of two 8-row groups) lie in 8 distinct 32-byte parts of the 64 banks.
    const auto swz = [](int k) { return ((k >> 1) & 1) | ((k >> 2) & 2); };
    uint32_t voP[2], voQ[2];
    auto places = [&](int64_t ldp, int64_t ldq) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int r = 16 * wave + 8 * j + (lane >> 3);
            const uint32_t chunk = static_cast<uint32_t>((lane & 7) ^ (4 * j + (lane >> 4))) * 16u;
            voP[j] = rowP(r) * static_cast<uint32_t>(ldp * 2) + chunk;
            if constexpr (!kQCols) voQ[j] = rowQ(r) * static_cast<uint32_t>(ldq * 2) + chunk;
        }
    };
    auto columns = [&](int64_t ldq, int last) __attribute__((always_inline)) {      // last: Q's last row, from the first of the step
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int k = 16 * wave + 8 * j + (lane >> 3), at = lane & 7;
            const int n = 16 * ((at >> 1) ^ swz(k)) + 8 * (at & 1);
            voQ[j] = static_cast<uint32_t>(min(k, last)) * static_cast<uint32_t>(ldq * 2) + rowQ(n) * 2u;
        }
    };
    places(g.ldp, g.ldq);
    if constexpr (kQCols) columns(g.ldq, g.rowsQ - 1);
    // values, not members: the choice between two of them was made of their addresses, in scratch
    const uint32_t bytesP = g.bytesP, bytesQ = g.bytesQ, bytesP2 = g.bytesP2, bytesQ2 = g.bytesQ2;
    const int kmain = ke - kb;
    const int KT = kmain + (kRank && rank ? g.kt2 : 0);
    int next = 0;                                    // the step whose loads are issued
    int so = kb * (kTurnK * 2);
    uint32_t qstep = static_cast<uint32_t>(g.ldq) * (kTurnK * 2);
    int sq = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<uint32_t>(kb) * qstep));
    auto issue = [&]() __attribute__((always_inline)) {                             // a step past the last: descriptors of no extent
        if (kRank && next == kmain) {
            places(g.ldp2, g.ldq2);
            if constexpr (kQCols) columns(g.ldq2, kTurnK - 1);
            qstep = static_cast<uint32_t>(g.ldq2) * (kTurnK * 2);
            so = sq = 0;
        }
        if (kQCols && (!kRank || next < kmain) && kb + next == g.kt1 - 1)     // rows past the last: the last again
            columns(g.ldq, g.rowsQ - 1 - kTurnK * (g.kt1 - 1));
        const bool first = !kRank || next < kmain, none = next >= KT;
        const i32x4t rsP = turn_rsrc(first ? g.P : g.P2, none ? 0u : first ? bytesP : bytesP2);
        const i32x4t rsQ = turn_rsrc(first ? g.Q : g.Q2, none ? 0u : first ? bytesQ : bytesQ2);
        const uint32_t to = lds + 16384u * (next & (kFewStages - 1)) + 2048u * wave;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            turn_load(rsP, to + 1024u * j, voP[j], so);
            turn_load(rsQ, to + 8192u + 1024u * j, voQ[j], kQCols ? sq : so);
        }
        ++next;
        so += kTurnK * 2;
        sq = __builtin_amdgcn_readfirstlane(static_cast<int>(sq + qstep));
    };

    const int fr = lane & 15;
    const uint32_t c0 = static_cast<uint32_t>((lane >> 4) ^ ((fr >> 1) & 7));
    const uint32_t prow = static_cast<uint32_t>(32 * wm + fr) * 8, qrow = static_cast<uint32_t>(32 * wn + fr) * 8;
    uint32_t qcol[2];                                // K-major, by k / 4 of the 8
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int k = 8 * (lane >> 4) + 4 * q + (fr >> 2);
        qcol[q] = static_cast<uint32_t>(128 * k + 32 * ((2 * wn) ^ swz(k)) + 8 * (fr & 3));
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[0][0][i][j] = f32x4t{0.0f, 0.0f, 0.0f, 0.0f};

#pragma unroll
    for (int s = 0; s < kFewStages - 1; ++s) issue();
    for (int t = 0; t < KT; ++t) {
        // the step's own loads are all but the newest 2 stages' 4 each; past the barrier every wave's
        // are there, and the step before has been read
        QN_WAIT_VM(4 * (kFewStages - 2));
        QN_TURN()
        issue();
        const uint4* P = g_few + 1024 * (t & (kFewStages - 1));
        const uint4* Q = P + 512;
        uint4 a[2][2], b[2][2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                a[i][k] = P[prow + 128 * i + (c0 ^ (4 * k))];
                if constexpr (kQCols) {
                    const turn_bytes_t at = (turn_bytes_t)Q + 4096 * k;
                    const u32x2t lo = turn_read_cols(at + (qcol[0] ^ (32u * i))), hi = turn_read_cols(at + (qcol[1] ^ (32u * i)));
                    b[i][k] = uint4{lo.x, lo.y, hi.x, hi.y};
                } else {
                    b[i][k] = Q[qrow + 128 * i + (c0 ^ (4 * k))];
                }
            }
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    acc[0][0][i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8, b[j][k]), __builtin_bit_cast(bf16x8, a[i][k]), acc[0][0][i][j], 0, 0, 0);
    }
    QN_WAIT_VM(0);
    QN_TURN()
}

}  // namespace

// The split of the tiles' K-steps (turn_split): two workgroups fit a CU, and a share has 16 steps or
// more, since the launch that adds the shares costs as much as 10.
inline TurnSplit few_split(int64_t M, int64_t tiles_n, int64_t kt) { return turn_split_of(6, M, tiles_n, kt, 512, 16); }

namespace {

// The tile's sums to a 64 x 64 float32 piece
__device__ __forceinline__ void few_put_sums(float* piece, const FewSums& acc, bool add) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float* at = piece + (32 * (wave >> 1) + (lane & 15)) * kFewTile + 32 * (wave & 1) + 4 * (lane >> 4);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            f32x4t* p = reinterpret_cast<f32x4t*>(at + 16 * i * kFewTile + 16 * j);
            *p = add ? *p + acc[0][0][i][j] : acc[0][0][i][j];
        }
}

}  // namespace
}  // namespace qn
