// The gated feed-forward block's product on gfx950:
//   H = act(G) * U,  G = X W_g^T + T_g B_g^T,  U = X W_u^T + T_u B_u^T,  T = s X A^T
// (the gate and up projections of the MLP pair, each a QLoRA linear layer: whoami-wesleyyou.top
// "LoRA", learn.ifs.name deck card 1).
//
// One MFMA contraction makes both: the weights are dequantised into one [2 d_ff, d_in] operand
// in which runs of 32 gate rows and the 32 up rows of the same outputs alternate, so that the
// 64-wide sub-tile of a wave (two 32 x 32 accumulators) has G in the first and U in the second,
// for the same lane and register. The activation and the product are then register arithmetic
// in the epilogue, G and U reach memory only where the gradient needs them, and X is read once.
// The K loop is the linear layer's (gemm_core.h), with the same split of the last round's tiles.
#include <hip/hip_runtime.h>

#include "gated.h"
#include "gemm_core.h"

#include <algorithm>

namespace qn {
namespace {

constexpr int kWM = 2, kWN = 4;
using Waves = GemmWaves<kWM, kWN>;
static_assert(Waves::TN == 2, "a wave's two column tiles are the gate's and the up projection's");

struct GatedOut {
    uint16_t* H; int64_t ldh;
    uint16_t* GU; int64_t ldgu;       // or null
    int d_ff, act;
};

template <bool kSplit>
__global__ __launch_bounds__(Waves::NT, 1)
void gated_gemm_kernel(GemmArgs g, GatedOut o) {
    constexpr int TM = Waves::TM, TN = Waves::TN;
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = tid >> 6;
    const int wm = wave / kWN, wn = wave % kWN;
    const int frow = lane & 31;
    // tiles as in gemm_nt: contiguous ranges per XCD; on the split path [0, full) whole, then
    // tile full + j % rem, split j / rem
    const int bid = static_cast<int>(blockIdx.x);
    const bool split_wg = kSplit && bid >= g.full;
    const int T = kSplit ? g.full : g.tiles_m * g.tiles_n;
    const int sj = split_wg ? bid - g.full : 0;
    const int sk = split_wg ? sj / g.rem : 0;
    const int logical = split_wg ? g.full + sj % g.rem : ((T % 8 == 0) ? (bid & 7) * (T >> 3) + (bid >> 3) : bid);
    int tm, tn;
    tile_coords(g, logical, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const int kb = split_wg ? sk * g.kper : 0;
    const int ke = split_wg ? min(kb + g.kper, g.kt1) : g.kt1;
    f32x16 acc[TN][TM];
    gemm_core<kWM, kWN, true>(
        g, [&](int r) { return static_cast<uint32_t>(min(m0 + r, g.M - 1)); },
        [&](int r) { return static_cast<uint32_t>(min(n0 + r, g.N - 1)); }, kb, ke, !split_wg || sk == g.splits - 1, acc);
    if (split_wg) {
        float* pt = g.part + (static_cast<int64_t>(sk) * g.rem + sj % g.rem) * (BM * BN);
#pragma unroll
        for (int b = 0; b < TM; ++b) {
            const int ml = wm * (TM * 32) + b * 32 + frow;
#pragma unroll
            for (int a = 0; a < TN; ++a)
#pragma unroll
                for (int gq = 0; gq < 4; ++gq) {
                    const int nl = wn * 64 + a * 32 + 8 * gq + 4 * (lane >> 5);
                    *reinterpret_cast<float4*>(pt + ml * BN + nl) =
                        float4{acc[a][b][4 * gq], acc[a][b][4 * gq + 1], acc[a][b][4 * gq + 2], acc[a][b][4 * gq + 3]};
                }
        }
        return;
    }
    const int h0 = tn * (BN / 2);                    // the tile's first output column
    if (o.GU != nullptr) {
        // G and U as a 256 x 512 B tile in LDS, rows 0..127 in the first stage, 16-byte chunk j of
        // row r at j ^ (r & 31); out as 256-byte runs of G and of U
#pragma unroll
        for (int b = 0; b < TM; ++b) {
            const int rl = wm * (TM * 32) + b * 32 + frow;
            char* rowp = reinterpret_cast<char*>((rl >> 7) ? g_st1 : g_st0) + (rl & 127) * 512;
#pragma unroll
            for (int a = 0; a < TN; ++a)
#pragma unroll
                for (int gq = 0; gq < 4; ++gq) {
                    const int nl = a * 128 + wn * 32 + 8 * gq + 4 * (lane >> 5);      // G first, then U
                    *reinterpret_cast<uint2*>(rowp + (((nl >> 3) ^ (rl & 31)) << 4) + ((nl & 7) << 1)) =
                        uint2{pack_bf16x2(acc[a][b][4 * gq], acc[a][b][4 * gq + 1]),
                              pack_bf16x2(acc[a][b][4 * gq + 2], acc[a][b][4 * gq + 3])};
                }
        }
        __syncthreads();
        const int cj = tid & 31;
        const int col = h0 + (cj & 15) * 8;
#pragma unroll
        for (int i = 0; i < BM / (Waves::NT / 32); ++i) {
            const int r = i * (Waves::NT / 32) + (tid >> 5);
            const char* arr = reinterpret_cast<const char*>((r >> 7) ? g_st1 : g_st0);
            const uint4 v = *reinterpret_cast<const uint4*>(arr + (r & 127) * 512 + ((cj ^ (r & 31)) << 4));
            if (m0 + r < g.M && col < o.d_ff)
                *reinterpret_cast<uint4*>(o.GU + static_cast<int64_t>(m0 + r) * o.ldgu + (cj >> 4) * o.d_ff + col) = v;
        }
        __syncthreads();
    }
    // H as a 256 x 256 B tile in the first stage, chunk j of row r at j ^ (r & 15)
#pragma unroll
    for (int b = 0; b < TM; ++b) {
        const int rl = wm * (TM * 32) + b * 32 + frow;
        char* rowp = reinterpret_cast<char*>(g_st0) + rl * 256;
#pragma unroll
        for (int gq = 0; gq < 4; ++gq) {
            const int nl = wn * 32 + 8 * gq + 4 * (lane >> 5);
            float h[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) h[e] = gated_act(o.act, acc[0][b][4 * gq + e]) * acc[1][b][4 * gq + e];
            *reinterpret_cast<uint2*>(rowp + (((nl >> 3) ^ (rl & 15)) << 4) + ((nl & 7) << 1)) =
                uint2{pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3])};
        }
    }
    __syncthreads();
    const int cj = tid & 15;
    const int col = h0 + cj * 8;
#pragma unroll
    for (int i = 0; i < BM / (Waves::NT / 16); ++i) {
        const int r = i * (Waves::NT / 16) + (tid >> 4);
        const uint4 v = *reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(g_st0) + r * 256 + ((cj ^ (r & 15)) << 4));
        if (m0 + r < g.M && col < o.d_ff) *reinterpret_cast<uint4*>(o.H + static_cast<int64_t>(m0 + r) * o.ldh + col) = v;
    }
}

// Split tiles: G and U summed over the splits in order, then the activation and the product;
// 4 outputs per thread, 32 workgroups per tile (8 rows each).
template <int SP>
__global__ __launch_bounds__(256)
void gated_split_reduce(GemmArgs g, GatedOut o) {
    const int j = static_cast<int>(blockIdx.x) / 32;
    const int ml = (static_cast<int>(blockIdx.x) % 32) * 8 + (threadIdx.x >> 5);
    const int q = (threadIdx.x & 31) * 4;                             // output column of the tile
    int tm, tn;
    tile_coords(g, g.full + j, tm, tn);
    const int m = tm * BM + ml, n = tn * (BN / 2) + q;
    if (m >= g.M || n >= o.d_ff) return;
    const float* p = g.part + static_cast<int64_t>(j) * (BM * BN) + ml * BN + (q >> 5) * 64 + (q & 31);
    const int64_t stride = static_cast<int64_t>(g.rem) * (BM * BN);
    float4 v[2][SP];
#pragma unroll
    for (int s = 0; s < SP; ++s)
#pragma unroll
        for (int w = 0; w < 2; ++w) v[w][s] = *reinterpret_cast<const float4*>(p + s * stride + 32 * w);
    float4 t[2] = {v[0][0], v[1][0]};
#pragma unroll
    for (int s = 1; s < SP; ++s)
#pragma unroll
        for (int w = 0; w < 2; ++w) { t[w].x += v[w][s].x; t[w].y += v[w][s].y; t[w].z += v[w][s].z; t[w].w += v[w][s].w; }
    if (o.GU != nullptr) {
#pragma unroll
        for (int w = 0; w < 2; ++w)
            *reinterpret_cast<uint2*>(o.GU + static_cast<int64_t>(m) * o.ldgu + w * o.d_ff + n) =
                uint2{pack_bf16x2(t[w].x, t[w].y), pack_bf16x2(t[w].z, t[w].w)};
    }
    *reinterpret_cast<uint2*>(o.H + static_cast<int64_t>(m) * o.ldh + n) =
        uint2{pack_bf16x2(gated_act(o.act, t[0].x) * t[1].x, gated_act(o.act, t[0].y) * t[1].y),
              pack_bf16x2(gated_act(o.act, t[0].z) * t[1].z, gated_act(o.act, t[0].w) * t[1].w)};
}

}  // namespace

int64_t gated_part_floats(int64_t M, int64_t d_ff, int64_t d_in) { return gemm_split_part_floats(M, 2 * d_ff, d_in); }

hipError_t launch_gated_gemm(const GatedCall& c, const uint16_t* X, int64_t ldx, const uint16_t* what, const uint16_t* t,
                             const uint16_t* adapt, uint16_t* H, int64_t ldh, uint16_t* GU, int64_t ldgu, float* part,
                             hipStream_t st) {
    const int64_t N = 2 * c.d_ff;
    GemmArgs g = gemm_args(X, ldx, what, c.d_in, c.d_in, c.r > 0 ? t : nullptr, gated_k2(c.r), adapt, gated_k2(c.r),
                           gated_k2(c.r), nullptr, 0, c.M, N, part);
    const GatedOut o{H, ldh, GU, ldgu, static_cast<int>(c.d_ff), c.act};
    if (g.splits <= 1) {
        QN_LAUNCH("gated_gemm_kernel", st, gated_gemm_kernel<false>, dim3(g.tiles_m * g.tiles_n), dim3(Waves::NT), 0, st, g, o);
        return hipGetLastError();
    }
    QN_LAUNCH("gated_gemm_split", st, gated_gemm_kernel<true>, dim3(g.full + g.rem * g.splits), dim3(Waves::NT), 0, st, g, o);
    const dim3 rgrid(static_cast<unsigned>(g.rem * 32));
    if (g.splits == 2) QN_LAUNCH("gated_split_reduce", st, gated_split_reduce<2>, rgrid, dim3(256), 0, st, g, o);
    else if (g.splits == 3) QN_LAUNCH("gated_split_reduce", st, gated_split_reduce<3>, rgrid, dim3(256), 0, st, g, o);
    else QN_LAUNCH("gated_split_reduce", st, gated_split_reduce<4>, rgrid, dim3(256), 0, st, g, o);
    return hipGetLastError();
}

}  // namespace qn
