// The K loop of the gated block's and the head's BF16 MFMA contractions (gated.hip,
// head_loss.hip): a 256 x 256 tile of P Q^T (+ P2 Q2^T), P row-major with K contiguous, Q so or
// with its rows along K (a weight as it lies, in the product for its input's gradient), in the
// accumulators of a workgroup of 8 waves. The tile's place, its rows and what becomes of the sums
// are the caller's.
//
// Two groups of 4 waves (one wave of each on every SIMD) take turns: between two barriers one
// group runs 32 MFMAs of 16 x 16 x 32 while the other reads its next fragments from LDS and issues
// loads, so the matrix pipe of a SIMD has one wave's run after the other's and no MFMA waits for
// an LDS read. A K-step of 64 has two such phases, one per half of the tile's rows (a wave has 64 of
// each half's 128 rows, and 32 of each half's 128 columns):
//   phase   reads from LDS                        issues loads of         multiplies
//   0       P half 0, Q halves 0, 1 (16 x 16 B)   P half 1 of t + 1       P0 Q0, P0 Q1
//   1       P half 1 (8)                          the others of t + 2     P1 Q1, P1 Q0
// The reads are waited for before a phase's barrier, so a half (128 rows x 64 k, 16 KB) is refilled one
// phase after it was read, the first point where both groups' reads are known to be done; a load has
// three phases to land: the waits are for all but the 8 newest of a wave's loads and never empty the
// queue before the tile's last steps. Eight halves, 128 KB of LDS.
// In 4096 x 4096 x 16128, one round of tiles, the matrix pipes are busy 76 to 79 % of the kernel's cycles
// (MfmaUtil; MFMA cycles over GRBM_GUI_ACTIVE) at the 1.8 GHz that this load leaves (the chip is
// power-limited); with more rounds, each with its start and epilogue, 60 to 70 %. It takes 350 us (1.54
// PFLOP/s), the library's product 342 on the same board. Four phases of 16 MFMAs took the same; 32 x 32 x
// 16 MFMAs on the same schedule 394. With Q's rows along K (8-byte LDS reads that transpose, twice as many)
// it takes 353: the transposed copy that the other form needs cost 88 more.
#pragma once
#include <hip/hip_runtime.h>

#include "internal.h"
#include "mfma_device.h"
#include "nf4_device.h"

namespace qn {

constexpr int kTurnTile = 256, kTurnK = 64, kTurnThreads = 512;

struct TurnArgs {
    const uint16_t* P; int64_t ldp;
    const uint16_t* Q; int64_t ldq;
    const uint16_t* P2; int64_t ldp2;
    const uint16_t* Q2; int64_t ldq2;
    uint32_t bytesP, bytesQ, bytesP2, bytesQ2;      // extents for the load descriptors
    int kt1, kt2;                                   // K-steps of P Q^T, and of P2 Q2^T
    int rowsQ;                                      // rows of Q
};

// rowsP, rowsQ: rows of the operands (their extents: every operand is below 4 GiB)
inline TurnArgs turn_args(const uint16_t* P, int64_t ldp, int64_t rowsP, const uint16_t* Q, int64_t ldq, int64_t rowsQ,
                          int64_t K) {
    TurnArgs g{};
    g.P = P; g.ldp = ldp; g.Q = Q; g.ldq = ldq;
    g.bytesP = static_cast<uint32_t>(2 * ldp * rowsP);
    g.bytesQ = static_cast<uint32_t>(2 * ldq * rowsQ);
    g.kt1 = static_cast<int>(K / kTurnK);
    g.rowsQ = static_cast<int>(rowsQ);
    return g;
}

namespace {

typedef float f32x4t __attribute__((ext_vector_type(4)));

typedef uint32_t u32x2t __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4t __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) char* turn_bytes_t;

__device__ __forceinline__ u32x2t turn_read_cols(turn_bytes_t at) {
    typedef short s16x4 __attribute__((ext_vector_type(4)));
    return __builtin_bit_cast(u32x2t, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)at));
}

// halves: stage, operand, rows 0..127 or 128..255 of the tile
__shared__ uint4 g_p00[1024], g_p01[1024], g_q00[1024], g_q01[1024];
__shared__ uint4 g_p10[1024], g_p11[1024], g_q10[1024], g_q11[1024];

// The sums of a wave: acc[h][g][i][j], lane l, is C[m][n .. n + 3] with m = 128 h + 64 wm + 16 i +
// l % 16 and n = 128 g + 32 wn + 16 j + 4 (l / 16), wm = wave / 4, wn = wave % 4.
typedef f32x4t TurnSums[2][2][4][2];

typedef int32_t i32x4t __attribute__((ext_vector_type(4)));

// (base, no stride, extent in bytes, raw): offsets at or past the extent read as zero
__device__ __forceinline__ i32x4t turn_rsrc(const void* base, uint32_t bytes) {
    const uint64_t at = reinterpret_cast<uint64_t>(base);
    return i32x4t{static_cast<int>(at), static_cast<int>(at >> 32) & 0xFFFF, static_cast<int>(bytes), 0x00020000};
}

// 16 bytes per lane from a buffer at `offset` + `base` to LDS address `to` + 16 lane. The instruction
// itself, since the compiler's own form made it wait for loads into other halves before some LDS
// reads (after 2 of the phases a load has); the waits are this file's. It writes no register.
__device__ __forceinline__ void turn_load(const i32x4t& rsrc, uint32_t to, uint32_t offset, int base) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds"
                 :
                 : "s"(to), "v"(offset), "s"(rsrc), "s"(base)
                 : "memory", "m0");
}

// A barrier that keeps memory accesses (clobber) and MFMAs (sched_barrier) on their side and
// waits for no load; LDS reads in flight are waited for where their values are used.
#define QN_TURN()                                  \
    {                                              \
        __builtin_amdgcn_sched_barrier(0);         \
        asm volatile("s_barrier" ::: "memory");    \
        __builtin_amdgcn_sched_barrier(0);         \
    }

#define QN_WAIT_LDS() __builtin_amdgcn_s_waitcnt(0xC07F)      // lgkmcnt(0), no other counter

// acc = the K-steps [kb, ke) of P Q^T, then (kRank and rank) the g.kt2 steps of P2 Q2^T; at least
// one step in all. rowP(r), rowQ(r): the row of P and P2 (Q and Q2) that tile row r takes (uint32,
// inside the operand). With kQCols, Q and Q2 are K-major instead, their rows along K: rowQ(r) is
// then the column of tile row r, for r a multiple of 8 and the 7 after it. Rows of Q from g.rowsQ on
// are taken as the last one (P must be zero there); Q2 has whole steps of them. On return every wave
// has finished its reads of LDS and no load is in flight.
template <bool kRank, bool kQCols, class RowP, class RowQ>
__device__ __forceinline__ void gemm_turns(const TurnArgs& g, const RowP& rowP, const RowQ& rowQ, int kb, int ke, bool rank,
                                           TurnSums& acc) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wm = wave >> 2, wn = wave & 3;

    // A half's row is 64 bf16 = 128 B = 8 chunks of 16 B; chunk c of row r is stored at c ^ ((r >> 1) & 7):
    // two rows cover the 64 banks once, and 16 lanes reading one chunk of 16 rows hit 16 distinct 4-bank
    // groups. A load instruction fills 8 rows; wave w fills rows 16 w .. 16 w + 15 of every half, lane i
    // the chunk that belongs at position i % 8 of row i / 8.
    uint32_t voP[2][2], voQ[2][2];                  // half, instruction
    i32x4t rsP, rsQ;
    auto places = [&](int64_t ldp, int64_t ldq) __attribute__((always_inline)) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int r = 128 * h + 16 * wave + 8 * j + (lane >> 3);
                const uint32_t chunk = static_cast<uint32_t>((lane & 7) ^ (4 * j + (lane >> 4))) * 16u;
                voP[h][j] = rowP(r) * static_cast<uint32_t>(ldp * 2) + chunk;
                if constexpr (!kQCols) voQ[h][j] = rowQ(r) * static_cast<uint32_t>(ldq * 2) + chunk;
            }
    };
    // K-major Q: a half is 64 k-rows of 128 columns = 256 B = 8 units of 32 B; unit u of row k is stored
    // at u ^ swz(k), which puts the 8 rows that 32 lanes of a transposing read take (4 of each of two
    // 8-row groups) into 8 distinct units. A load instruction fills 4 rows; wave w fills 8 w .. 8 w + 7.
    const auto swz = [](int k) { return (k & 3) | ((k >> 1) & 4); };
    auto columns = [&](int64_t ldq, int last) __attribute__((always_inline)) {     // last: the operand's last row, from the first of the step
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int k = 8 * wave + 4 * j + (lane >> 4), at = lane & 15;
                const int n = 128 * h + 16 * ((at >> 1) ^ swz(k)) + 8 * (at & 1);
                voQ[h][j] = static_cast<uint32_t>(min(k, last)) * static_cast<uint32_t>(ldq * 2) + rowQ(n) * 2u;
            }
    };
    places(g.ldp, g.ldq);
    if constexpr (kQCols) columns(g.ldq, g.rowsQ - 1);
    // values, not members: the choice between two of them was made of their addresses, in scratch
    const uint32_t bytesP = g.bytesP, bytesQ = g.bytesQ, bytesP2 = g.bytesP2, bytesQ2 = g.bytesQ2;
    const int kmain = ke - kb;
    const int KT = kmain + (kRank && rank ? g.kt2 : 0);
    // Loads are issued for two steps past the last as well, so that the loop has no branch around a
    // load (with one the compiler emptied the load queue before the LDS reads); their descriptors have
    // no extent, so nothing is fetched.
    int next = 0;                                   // the step whose loads are issued
    int so = kb * (kTurnK * 2);                     // its byte offset in a row
    uint32_t qstep = static_cast<uint32_t>(g.ldq) * (kTurnK * 2);      // K-major: bytes of 64 rows
    int sq = __builtin_amdgcn_readfirstlane(static_cast<int>(static_cast<uint32_t>(kb) * qstep));
    auto enter = [&]() __attribute__((always_inline)) {                            // before the first load of step `next`
        if (kRank && next == kmain) {
            places(g.ldp2, g.ldq2);
            if constexpr (kQCols) columns(g.ldq2, kTurnK - 1);
            qstep = static_cast<uint32_t>(g.ldq2) * (kTurnK * 2);
            so = sq = 0;
        }
        if (kQCols && (!kRank || next < kmain) && kb + next == g.kt1 - 1)     // rows past the last: the last again
            columns(g.ldq, g.rowsQ - 1 - kTurnK * (g.kt1 - 1));
        const bool first = !kRank || next < kmain, none = next >= KT;
        rsP = turn_rsrc(first ? g.P : g.P2, none ? 0u : first ? bytesP : bytesP2);
        rsQ = turn_rsrc(first ? g.Q : g.Q2, none ? 0u : first ? bytesQ : bytesQ2);
    };
    auto leave = [&]() { ++next; so += kTurnK * 2; sq = __builtin_amdgcn_readfirstlane(static_cast<int>(sq + qstep)); };
#define QN_LOAD(OBJ, RS, VO, SO)                                    \
    {                                                               \
        const uint32_t to_ = lds_addr(OBJ) + 2048 * wave;           \
        turn_load(RS, to_, (VO)[0], SO);                            \
        turn_load(RS, to_ + 1024, (VO)[1], SO);                     \
    }
#define QN_LOAD_P(OBJ, H) QN_LOAD(OBJ, rsP, voP[H], so)
#define QN_LOAD_Q(OBJ, H) QN_LOAD(OBJ, rsQ, voQ[H], kQCols ? sq : so)

    // fragments: lane l has row l % 16, k 8 (l / 16) .. + 7 of each 32
    const int fr = lane & 15;
    const uint32_t c0 = static_cast<uint32_t>((lane >> 4) ^ ((fr >> 1) & 7)), c1 = c0 ^ 4u;    // chunks of k 0..31 and 32..63
    const uint32_t prow = static_cast<uint32_t>(64 * wm + fr) * 8, qrow = static_cast<uint32_t>(32 * wn + fr) * 8;
    uint4 a[4][2], b0[2][2], b1[2][2];
#define QN_READ_P(OBJ)                                                                  \
    _Pragma("unroll") for (int k = 0; k < 2; ++k)                                       \
        _Pragma("unroll") for (int i = 0; i < 4; ++i) a[i][k] = (OBJ)[prow + 128 * i + (k ? c1 : c0)];
    // K-major: a transposing read hands lane p of 16 column p of a 4 x 16 block whose row p / 4 the
    // address of lanes 4 (p / 4) .. + 3 gives, 8 bytes a lane; two make the 8 k of a fragment
    uint32_t qcol[2];                               // by k / 4 of the 8
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int k = 8 * (lane >> 4) + 4 * q + (fr >> 2);
        qcol[q] = static_cast<uint32_t>(256 * k + 32 * ((2 * wn) ^ swz(k)) + 8 * (fr & 3));
    }
#define QN_READ_Q(OBJ, B)                                                               \
    _Pragma("unroll") for (int k = 0; k < 2; ++k)                                       \
        _Pragma("unroll") for (int j = 0; j < 2; ++j) {                                 \
            if constexpr (kQCols) {                                                     \
                const turn_bytes_t at_ = (turn_bytes_t)(OBJ) + 8192 * k;                \
                const u32x2t lo_ = turn_read_cols(at_ + (qcol[0] ^ (32u * j))), hi_ = turn_read_cols(at_ + (qcol[1] ^ (32u * j))); \
                B[j][k] = uint4{lo_.x, lo_.y, hi_.x, hi_.y};                            \
            } else {                                                                    \
                B[j][k] = (OBJ)[qrow + 128 * j + (k ? c1 : c0)];                        \
            }                                                                           \
        }
#define QN_MULTIPLY(H, G, B)                                                            \
    {                                                                                   \
        __builtin_amdgcn_s_setprio(1);                                                  \
        _Pragma("unroll") for (int k = 0; k < 2; ++k)                                   \
            _Pragma("unroll") for (int i = 0; i < 4; ++i)                               \
                _Pragma("unroll") for (int j = 0; j < 2; ++j)                           \
                    acc[H][G][i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(          \
                        __builtin_bit_cast(bf16x8, B[j][k]), __builtin_bit_cast(bf16x8, a[i][k]), acc[H][G][i][j], 0, 0, 0); \
        __builtin_amdgcn_s_setprio(0);                                                  \
    }
    // One K-step on stage (P0, P1, Q0, Q1), NP1 a half of the other stage. A phase's LDS reads are
    // waited for before its barrier, so a half may be refilled one phase after it was read.
#define QN_STEP(P0, P1, Q0, Q1, NP1)                                                    \
    {                                                                                   \
        QN_READ_P(P0)                                                                   \
        QN_READ_Q(Q0, b0)                                                               \
        QN_READ_Q(Q1, b1)                                                               \
        QN_LOAD_P(NP1, 1)                                                               \
        leave();                                                                        \
        QN_WAIT_VM(8);                                                                  \
        QN_WAIT_LDS();                                                                  \
        QN_TURN()                                                                       \
        QN_MULTIPLY(0, 0, b0)                                                           \
        QN_MULTIPLY(0, 1, b1)                                                           \
        QN_TURN()                                                                       \
        QN_READ_P(P1)                                                                   \
        enter();                                                                        \
        QN_LOAD_P(P0, 0)                                                                \
        QN_LOAD_Q(Q0, 0)                                                                \
        QN_LOAD_Q(Q1, 1)                                                                \
        QN_WAIT_VM(8);                                                                  \
        QN_WAIT_LDS();                                                                  \
        QN_TURN()                                                                       \
        QN_MULTIPLY(1, 1, b1)                                                           \
        QN_MULTIPLY(1, 0, b0)                                                           \
        QN_TURN()                                                                       \
    }

#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[h][q][i][j] = f32x4t{0.0f, 0.0f, 0.0f, 0.0f};

    enter();
    QN_LOAD_P(g_p00, 0)
    QN_LOAD_Q(g_q00, 0)
    QN_LOAD_Q(g_q01, 1)
    QN_LOAD_P(g_p01, 1)
    leave();
    enter();
    QN_LOAD_P(g_p10, 0)
    QN_LOAD_Q(g_q10, 0)
    QN_LOAD_Q(g_q11, 1)
    QN_WAIT_VM(8);
    QN_TURN()
    if (wm == 1) QN_TURN()                          // the second group starts one turn later
    for (int left = KT;;) {
        QN_STEP(g_p00, g_p01, g_q00, g_q01, g_p11)
        if (--left == 0) break;
        QN_STEP(g_p10, g_p11, g_q10, g_q11, g_p01)
        if (--left == 0) break;
    }
    if (wm == 0) QN_TURN()
    QN_WAIT_VM(0);                                  // the loads past the last step
    QN_TURN()
#undef QN_STEP
#undef QN_MULTIPLY
#undef QN_READ_Q
#undef QN_READ_P
#undef QN_LOAD_Q
#undef QN_LOAD_P
#undef QN_LOAD
}

// ---- epilogue: a bf16 tile through LDS, so that it leaves in whole rows ----

// object `index` (0..7; a constant after unrolling, or uniform)
__device__ __forceinline__ turn_bytes_t turn_object(int index) {
    const turn_bytes_t lo = index & 2 ? (index & 1 ? (turn_bytes_t)g_q01 : (turn_bytes_t)g_q00)
                                      : (index & 1 ? (turn_bytes_t)g_p01 : (turn_bytes_t)g_p00);
    const turn_bytes_t hi = index & 2 ? (index & 1 ? (turn_bytes_t)g_q11 : (turn_bytes_t)g_q10)
                                      : (index & 1 ? (turn_bytes_t)g_p11 : (turn_bytes_t)g_p10);
    return index & 4 ? hi : lo;
}

// 4 neighbouring columns of a row: of a 256-column tile (32 rows of 512 B per object, 16-byte chunk j
// of row r at j ^ (r & 31)) or of a 128-column one (64 rows of 256 B, j ^ (r & 15)). The rows are
// 16 per wave instruction, so 16 distinct 4-bank groups.
template <int kCols>
__device__ __forceinline__ void turn_put(int row, int col, float a, float b, float c, float d) {
    constexpr int kRows = 8192 / kCols;
    const int uniform = __builtin_amdgcn_readfirstlane(row / kRows);
    *(__attribute__((address_space(3))) u32x2t*)(turn_object(uniform) + (row % kRows) * (2 * kCols) +
                                                (((col >> 3) ^ (row & (kCols / 8 - 1))) << 4) + ((col & 7) << 1)) =
        u32x2t{bf16_pair(a, b), bf16_pair(c, d)};
}

// chunk (8 columns) c of row `row`; the rows of a wave lie in one object
template <int kCols>
__device__ __forceinline__ uint4 turn_get(int row, int c) {
    constexpr int kRows = 8192 / kCols;
    const int uniform = __builtin_amdgcn_readfirstlane(row / kRows);
    const u32x4t v = *(__attribute__((address_space(3))) u32x4t*)(turn_object(uniform) + (row % kRows) * (2 * kCols) +
                                                                 ((c ^ (row & (kCols / 8 - 1))) << 4));
    return uint4{v.x, v.y, v.z, v.w};
}

// ---- places of the tiles ----
// Workgroup -> one of n items, contiguous ranges per XCD (workgroups go to the 8 XCDs in turn), so
// that each XCD's L2 sees neighbouring tiles; -1: none. The grid is at least 8 ceil(n / 8).
__device__ __forceinline__ int turn_item(int bid, int n) {
    const int x = bid & 7, i = bid >> 3;
    const int q = n >> 3, rest = n & 7;
    return i < q + (x < rest ? 1 : 0) ? x * q + min(x, rest) + i : -1;
}

// item -> (tile row, tile column): groups of 4 tile rows, column by column
__device__ __forceinline__ void turn_tile(int item, int tiles_m, int tiles_n, int& tm, int& tn) {
    const int size = 4 * tiles_n;
    const int first = item / size * 4;
    const int rows = min(tiles_m - first, 4);
    tm = first + item % size % rows;
    tn = item % size / rows;
}

}  // namespace

// The K-steps of the last round of tiles split over several workgroups each where it would leave
// most CUs idle: of T tiles the first full run whole, the K-steps of the rem others in `splits`
// shares of kper whose float32 sums (256 x 256 a piece, share s of tile j at s rem + j) a second
// kernel adds. Up to 16 shares, of 4 K-steps or more (1531 tokens of the 11008 x 4096 block leave 4 tiles:
// 243 us with up to 4 shares of 8 steps).
struct TurnSplit { int lt, tiles_m, tiles_n, splits, full, rem, kper; };       // tiles of 1 << lt
inline TurnSplit turn_split_of(int lt, int64_t M, int64_t tiles_n, int64_t kt, int slots, int64_t steps) {
    TurnSplit s{};
    s.lt = lt;
    s.tiles_m = static_cast<int>((M + (1 << lt) - 1) >> lt);
    s.tiles_n = static_cast<int>(tiles_n);
    const int T = s.tiles_m * s.tiles_n, rem = T % slots;
    int want = rem == 0 || rem > slots / 2 ? 1 : slots / rem;
    if (want > 16) want = 16;
    if (want > kt / steps) want = static_cast<int>(kt / steps);
    s.splits = want < 2 ? 1 : want;
    s.full = s.splits > 1 ? T - rem : T;
    s.rem = s.splits > 1 ? rem : 0;
    s.kper = static_cast<int>((kt + s.splits - 1) / s.splits);
    if (s.splits > 1) s.splits = static_cast<int>((kt + s.kper - 1) / s.kper);
    return s;
}
inline TurnSplit turn_split(int64_t M, int64_t tiles_n, int64_t kt) { return turn_split_of(8, M, tiles_n, kt, 256, 4); }
inline int64_t turn_split_floats(const TurnSplit& s) {
    return s.splits > 1 ? (static_cast<int64_t>(s.splits) * s.rem) << (2 * s.lt) : 0;
}
inline unsigned turn_split_grid(const TurnSplit& s) {
    return static_cast<unsigned>((s.full + 7) / 8 * 8 + s.rem * s.splits);
}

namespace {

// A workgroup's tile and share (share -1: the whole tile; tile -1: none)
struct TurnPlace { int tm, tn, tile, share, kb, ke; };
__device__ __forceinline__ TurnPlace turn_place(const TurnSplit& s, int bid, int kt) {
    TurnPlace p;
    const int whole = (s.full + 7) / 8 * 8;
    int item;
    if (bid < whole) {
        item = turn_item(bid, s.full);
        p.tile = item;
        p.share = -1;
        p.kb = 0;
        p.ke = kt;
    } else {
        p.tile = (bid - whole) % s.rem;
        item = s.full + p.tile;
        p.share = (bid - whole) / s.rem;
        p.kb = p.share * s.kper;
        p.ke = min(p.kb + s.kper, kt);
    }
    if (item >= 0) turn_tile(item, s.tiles_m, s.tiles_n, p.tm, p.tn);
    return p;
}

// A share's sums to its 256 x 256 float32 piece
__device__ __forceinline__ void turn_put_sums(float* piece, const TurnSums& acc, bool add) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float* at = piece + (64 * (wave >> 2) + (lane & 15)) * kTurnTile + 32 * (wave & 3) + 4 * (lane >> 4);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int q = 0; q < 2; ++q)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    f32x4t* p = reinterpret_cast<f32x4t*>(at + (128 * h + 16 * i) * kTurnTile + 128 * q + 16 * j);
                    *p = add ? *p + acc[h][q][i][j] : acc[h][q][i][j];
                }
}

}  // namespace
}  // namespace qn
