// BF16 MFMA contractions of the QLoRA linear layer on gfx950.
//
// Forward (whoami-wesleyyou.top "LoRA": Y = W0 X + s B (A X)) and input gradient
// (learn.ifs.name deck card 1: gradients flow through the dequantised BF16 weights)
// are both written as an "NT" product of two K-contiguous operands,
//     C[M, N] = P[M, K] Q[N, K]^T  (+ P2[M, K2] Q2[N, K2]^T),
// with M = tokens. The rank-r LoRA branch is the second term, folded in as extra
// K-steps of the same accumulators:
//     forward : P = X,  Q = W_hat,    P2 = s (X A^T),   Q2 = B
//     dX      : P = dY, Q = W_hat^T,  P2 = s (dY B),    Q2 = A^T
// so it costs r extra K (1.6 % of the flops at r = 64, K = 4096).
//
// gemm_nt: 256x256 output tile per workgroup, 8 waves (two per SIMD, so one wave's
// MFMAs cover the other's waits) in a 2x4 grid, each wave a 128x64 sub-tile of 4x2
// v_mfma_f32_32x32x16_bf16 accumulators (fp32). K-steps of 64 are double-buffered
// in LDS (2 x 64 KB) and filled by buffer_load ... lds (direct to LDS, no staging
// registers): a tile row is then 128 B, one whole cache line per row and load, which
// halves the L2 requests per byte compared with 64-byte rows. Rows are stored with
// their 16-byte chunks XOR-swizzled by ((row >> 1) & 7), which makes the 32-row
// fragment reads (ds_read_b128) free of bank conflicts on the 64-bank LDS. The stage
// barrier sits before the last k16 sub-step, so the next stage's first fragments are
// read under the last MFMAs. Tiles are handed to the 8 XCDs in contiguous ranges so
// each XCD's L2 sees a compact block of P and Q panels.
//
// gemm_nt_split: the same body when the last round of tiles would leave most CUs idle
// (T tiles, T mod 256 <= 128): the first 256 floor(T / 256) tiles run whole, and the
// K-steps of each of the R = T mod 256 others are split over S = min(4, 256 / R)
// workgroups (the LoRA K-steps go to the last split), each writing its fp32 partial
// tile; gemm_split_reduce adds a tile's S partials in split order and rounds to bf16.
#include <hip/hip_runtime.h>

#include "gemm_core.h"
#include "internal.h"
#include "mfma_device.h"
#include "nf4_device.h"

#include <algorithm>

namespace qn {
namespace {

// ---------------------------------------------------------------------------
// Main NT GEMM
// ---------------------------------------------------------------------------
template <int WM, int WN, bool kSplit>
__device__ __forceinline__ void gemm_nt_body(const GemmArgs& g) {
    using W = GemmWaves<WM, WN>;
    constexpr int NT = W::NT, TM = W::TM, TN = W::TN;
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = tid >> 6;
    const int wm = wave / WN, wn = wave % WN;
    const uint32_t frow = lane & 31;
    const int M = g.M, N = g.N;

    // ---- tile assignment: contiguous logical ranges per XCD, grouped raster. On the
    // split path, workgroups [0, full) take whole tiles, the rest (tile full + j % rem,
    // split j / rem) the split ones.
    const int bid = static_cast<int>(blockIdx.x);
    const bool split_wg = kSplit && bid >= g.full;
    const int T = kSplit ? g.full : g.tiles_m * g.tiles_n;
    const int w = split_wg ? 0 : bid;
    const int sj = split_wg ? bid - g.full : 0;
    const int sk = split_wg ? sj / g.rem : 0;                          // split of this workgroup
    const int logical = split_wg ? g.full + sj % g.rem : ((T % 8 == 0) ? (w & 7) * (T >> 3) + (w >> 3) : w);
    int tm, tn;
    tile_coords(g, logical, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;

    // K-steps of this workgroup: main steps [kb, ke) of P Q^T, then (last split, or no split)
    // the kt2 LoRA steps
    const int kb = split_wg ? sk * g.kper : 0;
    const int ke = split_wg ? min(kb + g.kper, g.kt1) : g.kt1;
    const bool lora = !split_wg || sk == g.splits - 1;
    f32x16 acc[TN][TM];
    gemm_core<WM, WN, true>(
        g, [&](int r) { return static_cast<uint32_t>(min(m0 + r, M - 1)); },
        [&](int r) { return static_cast<uint32_t>(min(n0 + r, N - 1)); }, kb, ke, lora, acc);

    if (split_wg) {
        // fp32 partial tile of this split, compact 256 x 256: the lane's 4 consecutive n
        // of tile row ml as 16 bytes
        float* pt = g.part + (static_cast<int64_t>(sk) * g.rem + sj % g.rem) * (BM * BN);
#pragma unroll
        for (int b = 0; b < TM; ++b) {
            const int ml = wm * (TM * 32) + b * 32 + static_cast<int>(frow);
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
    // ---- epilogue. Every wave is past the last barrier, so the LDS stages are free
    // and no load is in flight. The bf16 C tile (256 rows x 512 B) goes to LDS: rows
    // 128q .. 128q+127 in stage q (q = 0, 1), 16-byte chunk j of row r at position
    // j ^ (r & 31) (two-pass, conflict-free 8-byte writes, conflict-free 16-byte
    // reads); then each row leaves as 512 contiguous bytes, 16 B per lane.
    // The lane holds C[m][n..n+3] for m = tile row frow + 32 b + 32 TM wm and
    // n = 8 gq + 4 (lane >> 5) + 32 a + 32 TN wn.
#pragma unroll
    for (int b = 0; b < TM; ++b) {
        const int rl = wm * (TM * 32) + b * 32 + static_cast<int>(frow);
        uint4* arr = (rl >> 7) ? g_st1 : g_st0;
        char* rowp = reinterpret_cast<char*>(arr) + (rl & 127) * 512;
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
    const int cj = tid & 31;                     // 16-byte chunk of the row
    constexpr int kRowsPerPass = NT / 32;
#pragma unroll
    for (int i = 0; i < BM / kRowsPerPass; ++i) {
        const int r = i * kRowsPerPass + (tid >> 5);
        const uint4* arr = (r >> 7) ? g_st1 : g_st0;
        const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(arr) + (r & 127) * 512 +
                                                        ((cj ^ (r & 31)) << 4));
        const int m = m0 + r;
        const int n = n0 + cj * 8;
        if (m < M && n < N) *reinterpret_cast<uint4*>(g.C + static_cast<int64_t>(m) * g.ldc + n) = v;
    }
}

#ifndef QN_GEMM_WAVES_N
#define QN_GEMM_WAVES_N 4
#endif
constexpr int kGemmWM = 2, kGemmWN = QN_GEMM_WAVES_N;

__global__ __launch_bounds__(64 * kGemmWM * kGemmWN, 1)
void gemm_nt_kernel(GemmArgs g) {
    gemm_nt_body<kGemmWM, kGemmWN, false>(g);
}

__global__ __launch_bounds__(64 * kGemmWM * kGemmWN, 1)
void gemm_nt_split(GemmArgs g) {
    gemm_nt_body<kGemmWM, kGemmWN, true>(g);
}

// Split tiles: C[m, n..n+3] = bf16(sum of the tile's partials in split order), 4 outputs
// per thread; 64 workgroups per tile (4 rows each). SP = the split count (2..4): that
// many partial loads per thread.
template <int SP>
__global__ __launch_bounds__(256)
void gemm_split_reduce(GemmArgs g) {
    const int j = static_cast<int>(blockIdx.x) / 64;                  // split tile
    const int ml = (static_cast<int>(blockIdx.x) % 64) * 4 + (threadIdx.x >> 6);
    const int nl = (threadIdx.x & 63) * 4;
    int tm, tn;
    tile_coords(g, g.full + j, tm, tn);
    const int m = tm * BM + ml, n = tn * BN + nl;
    if (m >= g.M || n >= g.N) return;
    const float* p = g.part + static_cast<int64_t>(j) * (BM * BN) + ml * BN + nl;
    const int64_t stride = static_cast<int64_t>(g.rem) * (BM * BN);
    float4 v[SP];
#pragma unroll
    for (int s = 0; s < SP; ++s) v[s] = *reinterpret_cast<const float4*>(p + s * stride);
    float4 t = v[0];
#pragma unroll
    for (int s = 1; s < SP; ++s) { t.x += v[s].x; t.y += v[s].y; t.z += v[s].z; t.w += v[s].w; }
    *reinterpret_cast<uint2*>(g.C + static_cast<int64_t>(m) * g.ldc + n) =
        uint2{pack_bf16x2(t.x, t.y), pack_bf16x2(t.z, t.w)};
}

}  // namespace

GemmSplit gemm_split(int64_t M, int64_t N, int64_t K1) {
    const int64_t T = ((M + BM - 1) / BM) * ((N + BN - 1) / BN);
    const int64_t rem = T % 256;
    GemmSplit gs{1, static_cast<int>(T), 0};
    if (rem == 0 || rem > 128) return gs;
    const int64_t s = std::min<int64_t>({4, 256 / rem, K1 / BK / 8});    // at least 8 K-steps per split
    if (s < 2) return gs;
    gs.splits = static_cast<int>(s);
    gs.full = static_cast<int>(T - rem);
    gs.rem = static_cast<int>(rem);
    return gs;
}

int64_t gemm_split_part_floats(int64_t M, int64_t N, int64_t K1) {
    const GemmSplit gs = gemm_split(M, N, K1);
    return gs.splits > 1 ? static_cast<int64_t>(gs.splits) * gs.rem * BM * BN : 0;
}

GemmArgs gemm_args(const uint16_t* P, int64_t ldp, const uint16_t* Q, int64_t ldq, int64_t K1, const uint16_t* P2,
                   int64_t ldp2, const uint16_t* Q2, int64_t ldq2, int64_t K2, uint16_t* C, int64_t ldc, int64_t M,
                   int64_t N, float* part) {
    GemmArgs g{};
    g.tiles_m = static_cast<int>((M + BM - 1) / BM);
    g.tiles_n = static_cast<int>((N + BN - 1) / BN);
    if (P2 == nullptr) { P2 = P; Q2 = Q; ldp2 = ldp; ldq2 = ldq; K2 = 0; }
    g.P = P; g.ldp = ldp; g.Q = Q; g.ldq = ldq; g.kt1 = static_cast<int>(K1 / BK);
    g.P2 = P2; g.ldp2 = ldp2; g.Q2 = Q2; g.ldq2 = ldq2; g.kt2 = static_cast<int>(K2 / BK);
    g.C = C; g.ldc = ldc; g.M = static_cast<int>(M); g.N = static_cast<int>(N);
    // every operand is < 4 GiB (checked by the caller): the extents fit 32 bits
    g.bytesP = static_cast<uint32_t>(2 * ldp * M);
    g.bytesQ = static_cast<uint32_t>(2 * ldq * N);
    g.bytesP2 = static_cast<uint32_t>(2 * ldp2 * M);
    g.bytesQ2 = static_cast<uint32_t>(2 * ldq2 * N);
    const GemmSplit gs = gemm_split(M, N, K1);
    g.splits = part == nullptr ? 1 : gs.splits;
    g.full = gs.full;
    g.rem = gs.rem;
    g.kper = (g.kt1 + g.splits - 1) / g.splits;
    g.part = part;
    return g;
}

hipError_t launch_gemm_nt(const uint16_t* P, int64_t ldp, const uint16_t* Q, int64_t ldq, int64_t K1,
                          const uint16_t* P2, int64_t ldp2, const uint16_t* Q2, int64_t ldq2,
                          int64_t K2, uint16_t* C, int64_t ldc, int64_t M, int64_t N, float* part,
                          hipStream_t st, const uint8_t* codes, const BlockConsts* bc) {
    const bool deq = codes != nullptr;              // Q = W_hat formed from the codes in the kernel
    if (deq) { Q = P; ldq = ldp; }                  // no bf16 weight operand
    GemmArgs g = gemm_args(P, ldp, Q, ldq, K1, P2, ldp2, Q2, ldq2, K2, C, ldc, M, N, part);
    g.codes = codes;
    g.bc = deq ? *bc : BlockConsts{nullptr, nullptr, nullptr, 0, 0};
    {
        const NF4Tables& tab = tables();
        for (int i = 0; i < 16; ++i) g.code[i] = tab.code[i];
    }
    const int64_t nblk = deq ? N * (K1 / BK) : 0;   // NF4 blocks of the weight (K1 % 64 == 0)
    g.bytesC = static_cast<uint32_t>(nblk * 32);
    g.bytesBq = static_cast<uint32_t>(nblk);
    g.bytesBs = static_cast<uint32_t>(deq ? 4 * (((nblk - 1) >> g.bc.gshift) + 1) : 0);
    if (g.splits <= 1) {
        if (deq) return launch_gemm_nf4_body(g, false, st);
        QN_LAUNCH("gemm_nt_kernel", st, gemm_nt_kernel, dim3(g.tiles_m * g.tiles_n), dim3(64 * kGemmWM * kGemmWN), 0,
                  st, g);
        return hipGetLastError();
    }
    if (deq) {
        const hipError_t e = launch_gemm_nf4_body(g, true, st);
        if (e != hipSuccess) return e;
    } else {
        QN_LAUNCH("gemm_nt_split", st, gemm_nt_split, dim3(g.full + g.rem * g.splits), dim3(64 * kGemmWM * kGemmWN),
                  0, st, g);
    }
    const dim3 rgrid(static_cast<unsigned>(g.rem * 64));
    if (g.splits == 2) QN_LAUNCH("gemm_split_reduce", st, gemm_split_reduce<2>, rgrid, dim3(256), 0, st, g);
    else if (g.splits == 3) QN_LAUNCH("gemm_split_reduce", st, gemm_split_reduce<3>, rgrid, dim3(256), 0, st, g);
    else QN_LAUNCH("gemm_split_reduce", st, gemm_split_reduce<4>, rgrid, dim3(256), 0, st, g);
    return hipGetLastError();
}

}  // namespace qn
