// The gated feed-forward block's product on gfx950:
//   H = act(G) * U,  G = X W_g^T + T_g B_g^T,  U = X W_u^T + T_u B_u^T,  T = s X A^T
// (the gate and up projections of the MLP pair, each a QLoRA linear layer: whoami-wesleyyou.top
// "LoRA", learn.ifs.name deck card 1).
//
// One MFMA contraction makes both: the weights are dequantised into one [2 d_ff, d_in] operand, gate
// above up, and a 256 x 256 tile takes 128 gate rows and the 128 up rows of the same outputs, so that
// G and U of an output are sums of the same lane (gemm_turns.h: the two column halves of a tile).
// The activation and the product are then register arithmetic in the epilogue, G and U reach memory
// only where the gradient needs them, and X is read once.
// Bound by the matrix pipes at the clock that they leave, and by whole rounds of tiles: 2048 tokens of
// 11008 x 4096 (688 tiles on 256 CUs) take 291 us with G and U kept (1.30 PFLOP/s), dX there 252 (1.49).
#include <hip/hip_runtime.h>

#include "gated.h"
#include "gemm_few.h"
#include "gemm_turns.h"

#include <algorithm>
#include <type_traits>

namespace qn {
namespace {

struct GatedOut {
    uint16_t* H; int64_t ldh;
    uint16_t* GU; int64_t ldgu;       // or null
    int M, d_ff, act;
    float* part;
};

// A tile's 256 x 256 bf16 values from LDS to rows of C: columns col(c) .. + 7 for chunk c (0..31)
template <class Col>
__device__ __forceinline__ void store_rows(uint16_t* C, int64_t ldc, int m0, int M, int limit, const Col& col) {
    const int c = threadIdx.x & 31;
    const int n = col(c);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int row = 16 * i + (threadIdx.x >> 5);
        const uint4 v = turn_get<256>(row, c);
        if (m0 + row < M && n < limit) *reinterpret_cast<uint4*>(C + static_cast<int64_t>(m0 + row) * ldc + n) = v;
    }
}

// 4 outputs n .. n + 3 of token m from their G and U
template <bool kKeep>
__device__ __forceinline__ void gated_store(const GatedOut& o, int m, int n, const f32x4t& g, const f32x4t& u) {
    if constexpr (kKeep) {
        uint16_t* at = o.GU + static_cast<int64_t>(m) * o.ldgu + n;
        *reinterpret_cast<uint2*>(at) = uint2{bf16_pair(g[0], g[1]), bf16_pair(g[2], g[3])};
        *reinterpret_cast<uint2*>(at + o.d_ff) = uint2{bf16_pair(u[0], u[1]), bf16_pair(u[2], u[3])};
    }
    *reinterpret_cast<uint2*>(o.H + static_cast<int64_t>(m) * o.ldh + n) =
        uint2{bf16_pair(gated_act(o.act, g[0]) * u[0], gated_act(o.act, g[1]) * u[1]),
              bf16_pair(gated_act(o.act, g[2]) * u[2], gated_act(o.act, g[3]) * u[3])};
}

template <bool kKeep>
__global__ __launch_bounds__(kTurnThreads, 1)
void gated_gemm_kernel(TurnArgs g, TurnSplit s, GatedOut o) {
    const TurnPlace p = turn_place(s, static_cast<int>(blockIdx.x), g.kt1);
    if (p.tile < 0) return;
    const int m0 = p.tm * kTurnTile, h0 = p.tn * (kTurnTile / 2);
    TurnSums acc;
    gemm_turns<true, false>(
        g, [&](int r) { return static_cast<uint32_t>(min(m0 + r, o.M - 1)); },
        [&](int r) { return static_cast<uint32_t>((r < 128 ? 0 : o.d_ff) + min(h0 + (r & 127), o.d_ff - 1)); }, p.kb, p.ke,
        p.share < 0 || p.share == s.splits - 1, acc);
    if (p.share >= 0) {
        turn_put_sums(o.part + (static_cast<int64_t>(p.share) * s.rem + p.tile) * (kTurnTile * kTurnTile), acc, false);
        return;
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int row0 = 64 * (wave >> 2) + (lane & 15), col0 = 32 * (wave & 3) + 4 * (lane >> 4);
    if constexpr (kKeep) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const f32x4t v = acc[h][q][i][j];
                        turn_put<256>(128 * h + 16 * i + row0, 128 * q + 16 * j + col0, v[0], v[1], v[2], v[3]);
                    }
        __syncthreads();
        // 256 bytes of G, then 256 of U, per row
        store_rows(o.GU, o.ldgu, m0, o.M, 2 * o.d_ff, [&](int c) {
            const int n = h0 + 8 * (c & 15);
            return n < o.d_ff ? n + (c >> 4) * o.d_ff : 2 * o.d_ff;
        });
        __syncthreads();
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = gated_act(o.act, acc[h][0][i][j][e]) * acc[h][1][i][j][e];
                turn_put<128>(128 * h + 16 * i + row0, 16 * j + col0, v[0], v[1], v[2], v[3]);
            }
    __syncthreads();
    const int c = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int row = 32 * i + (threadIdx.x >> 4);
        const uint4 v = turn_get<128>(row, c);
        if (m0 + row < o.M && h0 + 8 * c < o.d_ff)
            *reinterpret_cast<uint4*>(o.H + static_cast<int64_t>(m0 + row) * o.ldh + h0 + 8 * c) = v;
    }
}

// The same on tiles of 64 tokens x 32 outputs (gemm_few.h): of every 32 columns of the tile the first
// 16 are gate rows, the others the up rows of the same outputs, so that a lane has both.
template <bool kKeep>
__global__ __launch_bounds__(kFewThreads, 2)
void gated_few_gemm_kernel(TurnArgs g, TurnSplit s, GatedOut o) {
    const TurnPlace p = turn_place(s, static_cast<int>(blockIdx.x), g.kt1);
    if (p.tile < 0) return;
    const int m0 = p.tm * kFewTile, h0 = p.tn * (kFewTile / 2);
    FewSums acc;
    gemm_few<true, false>(
        g, [&](int r) { return static_cast<uint32_t>(min(m0 + r, o.M - 1)); },
        [&](int r) { return static_cast<uint32_t>((r & 16 ? o.d_ff : 0) + h0 + 16 * (r >> 5) + (r & 15)); }, p.kb, p.ke,
        p.share < 0 || p.share == s.splits - 1, acc);
    if (p.share >= 0) {
        few_put_sums(o.part + (static_cast<int64_t>(p.share) * s.rem + p.tile) * (kFewTile * kFewTile), acc, false);
        return;
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int n = h0 + 16 * (wave & 1) + 4 * (lane >> 4);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int m = m0 + 32 * (wave >> 1) + 16 * i + (lane & 15);
        if (m < o.M) gated_store<kKeep>(o, m, n, acc[0][0][i][0], acc[0][0][i][1]);
    }
}

// Split tiles: G and U summed over the shares in order, then the activation and the product;
// 4 outputs per thread, 2^(2 lt - 3) threads per tile.
__global__ __launch_bounds__(256)
void gated_split_reduce(TurnSplit s, GatedOut o) {
    const int at = static_cast<int>(blockIdx.x) * 256 + threadIdx.x;
    const int j = at >> (2 * s.lt - 3), in = at & ((1 << (2 * s.lt - 3)) - 1);
    const int ml = in >> (s.lt - 3), q = (in & ((1 << (s.lt - 3)) - 1)) * 4;      // row and output of the tile
    int tm, tn;
    turn_tile(s.full + j, s.tiles_m, s.tiles_n, tm, tn);
    const int m = (tm << s.lt) + ml, n = (tn << (s.lt - 1)) + q;
    if (m >= o.M || n >= o.d_ff) return;
    const bool few = s.lt == 6;
    const float* p = o.part + (static_cast<int64_t>(j) << (2 * s.lt)) + (ml << s.lt) + (few ? 32 * (q >> 4) + (q & 15) : q);
    const int64_t stride = static_cast<int64_t>(s.rem) << (2 * s.lt);
    const float4 g = ordered_sum4<4>(p, stride, s.splits), u = ordered_sum4<4>(p + (few ? 16 : 128), stride, s.splits);
    const f32x4t gv = {g.x, g.y, g.z, g.w}, uv = {u.x, u.y, u.z, u.w};
    if (o.GU != nullptr) gated_store<true>(o, m, n, gv, uv);
    else gated_store<false>(o, m, n, gv, uv);
}

// dX = dGU [W_g; W_u] + U' [A_g; A_u]: a plain product whose weights lie with their rows along K
// (read by transposing LDS reads), bf16 out
struct GatedDx {
    uint16_t* C; int64_t ldc;
    int M, N;
    float* part;
};

template <bool kFew>
__global__ __launch_bounds__(kFew ? kFewThreads : kTurnThreads, kFew ? 2 : 1)
void gated_dx_kernel(TurnArgs g, TurnSplit s, GatedDx o) {
    constexpr int kTile = kFew ? kFewTile : kTurnTile;
    const TurnPlace p = turn_place(s, static_cast<int>(blockIdx.x), g.kt1);
    if (p.tile < 0) return;
    const int m0 = p.tm * kTile, n0 = p.tn * kTile;
    const int last_p = o.M - 1, last_q = o.N - 8;
    const auto row_p = [=](int r) { return static_cast<uint32_t>(min(m0 + r, last_p)); };
    const auto col_q = [=](int r) { return static_cast<uint32_t>(min(n0 + r, last_q)); };
    const bool rank = p.share < 0 || p.share == s.splits - 1;
    float* const piece = o.part + (static_cast<int64_t>(p.share) * s.rem + p.tile) * (kTile * kTile);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    std::conditional_t<kFew, FewSums, TurnSums> acc;
    if constexpr (kFew) {
        gemm_few<true, true>(g, row_p, col_q, p.kb, p.ke, rank, acc);
        if (p.share >= 0) {
            few_put_sums(piece, acc, false);
            return;
        }
        const int n = n0 + 32 * (wave & 1) + 4 * (lane >> 4);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int m = m0 + 32 * (wave >> 1) + 16 * i + (lane & 15);
            if (m >= o.M) continue;
#pragma unroll
            for (int j = 0; j < 2; ++j) {             // N % 64 == 0: whole tiles
                const f32x4t v = acc[0][0][i][j];
                *reinterpret_cast<uint2*>(o.C + static_cast<int64_t>(m) * o.ldc + n + 16 * j) =
                    uint2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
            }
        }
    } else {
        gemm_turns<true, true>(g, row_p, col_q, p.kb, p.ke, rank, acc);
        if (p.share >= 0) {
            turn_put_sums(piece, acc, false);
            return;
        }
        const int row0 = 64 * (wave >> 2) + (lane & 15), col0 = 32 * (wave & 3) + 4 * (lane >> 4);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int q = 0; q < 2; ++q)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const f32x4t v = acc[h][q][i][j];
                        turn_put<256>(128 * h + 16 * i + row0, 128 * q + 16 * j + col0, v[0], v[1], v[2], v[3]);
                    }
        __syncthreads();
        store_rows(o.C, o.ldc, m0, o.M, o.N, [&](int c) { return n0 + 8 * c; });
    }
}

// Split tiles: the shares' sums in order; 4 outputs per thread, 2^(2 lt - 2) threads per tile
__global__ __launch_bounds__(256)
void gated_dx_reduce(TurnSplit s, GatedDx o) {
    const int at = static_cast<int>(blockIdx.x) * 256 + threadIdx.x;
    const int j = at >> (2 * s.lt - 2), in = at & ((1 << (2 * s.lt - 2)) - 1);
    const int ml = in >> (s.lt - 2), nl = (in & ((1 << (s.lt - 2)) - 1)) * 4;
    int tm, tn;
    turn_tile(s.full + j, s.tiles_m, s.tiles_n, tm, tn);
    const int m = (tm << s.lt) + ml, n = (tn << s.lt) + nl;
    if (m >= o.M || n >= o.N) return;
    const float* p = o.part + (static_cast<int64_t>(j) << (2 * s.lt)) + (ml << s.lt) + nl;
    const float4 t = ordered_sum4<4>(p, static_cast<int64_t>(s.rem) << (2 * s.lt), s.splits);
    *reinterpret_cast<uint2*>(o.C + static_cast<int64_t>(m) * o.ldc + n) = uint2{bf16_pair(t.x, t.y), bf16_pair(t.z, t.w)};
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Tiles of 64 or of 256, by their numbers. Forward, tiles of 64 where they are at most two rounds of the
// chip, 1024, and the 256-wide ones at most 96 (us with tiles of 64 and of 256: 203 tokens of the 512 x 256
// block 14 and 17; 512 of 2048 x 4096, 512 small tiles, 43 and 55; 512 of 4096 x 4096, 1024, 77 and 82 [75 and
// 74 with the weights' copy in the Infinity Cache]; 768 there, 1536, 101 and 96 [99 and 82]; 128 of 11008 x
// 4096, 688, 123 and 126; 256 there, 1376, 157 and 133 [117 and 106]; 70 of 28672 x 8192, 224 large tiles, 496
// and 436). The gradient's sums are long and its tiles few, and shares of
// them fill the chip: up to 64 tiles and 128 K-steps (128 tokens of 4096 x 4096 55 and 59; of 11008 x
// 4096, 344 steps, 116 and 110; 256 of 5504 x 2048, 172 steps, 60 and 56).
bool fwd_few(int64_t M, int64_t d_ff) {
    return ceil_div(M, kFewTile) * (2 * d_ff / kFewTile) <= 1024 && ceil_div(M, kTurnTile) * ceil_div(2 * d_ff, kTurnTile) <= 96;
}
bool dx_few(int64_t M, int64_t d_ff, int64_t d_in) {
    return ceil_div(M, kTurnTile) * ceil_div(d_in, kTurnTile) <= 64 && 2 * d_ff / kTurnK <= 128;
}

TurnSplit fwd_split(int64_t M, int64_t d_ff, int64_t d_in) {
    return fwd_few(M, d_ff) ? few_split(M, d_ff / (kFewTile / 2), d_in / kTurnK)
                            : turn_split(M, ceil_div(d_ff, kTurnTile / 2), d_in / kTurnK);
}
TurnSplit dx_split(int64_t M, int64_t d_ff, int64_t d_in) {
    return dx_few(M, d_ff, d_in) ? few_split(M, d_in / kFewTile, 2 * d_ff / kTurnK)
                                 : turn_split(M, ceil_div(d_in, kTurnTile), 2 * d_ff / kTurnK);
}

// P2 Q2^T of a call with adapters: adapt's rows are ldq2 long
void add_ranks(TurnArgs& g, const uint16_t* t, const uint16_t* adapt, int k2, int64_t ldq2, int64_t M, int64_t N) {
    if (k2 == 0) return;
    g.P2 = t; g.ldp2 = k2; g.Q2 = adapt; g.ldq2 = ldq2;
    g.bytesP2 = static_cast<uint32_t>(2 * static_cast<int64_t>(k2) * M);
    g.bytesQ2 = static_cast<uint32_t>(2 * static_cast<int64_t>(k2) * N);
    g.kt2 = k2 / kTurnK;
}

}  // namespace

int64_t gated_part_floats(int64_t M, int64_t d_ff, int64_t d_in) { return turn_split_floats(fwd_split(M, d_ff, d_in)); }
int64_t gated_dx_part_floats(int64_t M, int64_t d_ff, int64_t d_in) { return turn_split_floats(dx_split(M, d_ff, d_in)); }

hipError_t launch_gated_gemm(const GatedCall& c, const uint16_t* X, int64_t ldx, const uint16_t* what, const uint16_t* t,
                             const uint16_t* adapt, uint16_t* H, int64_t ldh, uint16_t* GU, int64_t ldgu, float* part,
                             hipStream_t st) {
    TurnArgs g = turn_args(X, ldx, c.M, what, c.d_in, 2 * c.d_ff, c.d_in);
    const int k2 = gated_k2(c.r, c.terms);
    add_ranks(g, t, adapt, k2, k2, c.M, 2 * c.d_ff);
    const TurnSplit s = fwd_split(c.M, c.d_ff, c.d_in);
    const GatedOut o{H, ldh, GU, ldgu, static_cast<int>(c.M), static_cast<int>(c.d_ff), c.act, part};
    const dim3 grid(turn_split_grid(s));
    const bool few = s.lt == 6;
    if (few && GU != nullptr) QN_LAUNCH("gated_few_gemm_kernel", st, gated_few_gemm_kernel<true>, grid, dim3(kFewThreads), 0, st, g, s, o);
    else if (few) QN_LAUNCH("gated_few_gemm_kernel", st, gated_few_gemm_kernel<false>, grid, dim3(kFewThreads), 0, st, g, s, o);
    else if (GU != nullptr) QN_LAUNCH("gated_gemm_kernel", st, gated_gemm_kernel<true>, grid, dim3(kTurnThreads), 0, st, g, s, o);
    else QN_LAUNCH("gated_gemm_kernel", st, gated_gemm_kernel<false>, grid, dim3(kTurnThreads), 0, st, g, s, o);
    const dim3 rgrid(static_cast<unsigned>((s.rem << (2 * s.lt - 3)) / 256));
    if (s.splits > 1) QN_LAUNCH("gated_split_reduce", st, gated_split_reduce, rgrid, dim3(256), 0, st, s, o);
    return hipGetLastError();
}

hipError_t launch_gated_dx(const GatedCall& c, const uint16_t* dGU, int64_t lddgu, const uint16_t* what, const uint16_t* t,
                           const uint16_t* adapt, uint16_t* dX, int64_t lddx, float* part, hipStream_t st) {
    TurnArgs g = turn_args(dGU, lddgu, c.M, what, c.d_in, 2 * c.d_ff, 2 * c.d_ff);
    add_ranks(g, t, adapt, gated_k2(c.r, c.terms), c.d_in, c.M, c.d_in);
    const TurnSplit s = dx_split(c.M, c.d_ff, c.d_in);
    const GatedDx o{dX, lddx, static_cast<int>(c.M), static_cast<int>(c.d_in), part};
    const dim3 grid(turn_split_grid(s));
    if (s.lt == 6) QN_LAUNCH("gated_dx_kernel", st, gated_dx_kernel<true>, grid, dim3(kFewThreads), 0, st, g, s, o);
    else QN_LAUNCH("gated_dx_kernel", st, gated_dx_kernel<false>, grid, dim3(kTurnThreads), 0, st, g, s, o);
    const dim3 rgrid(static_cast<unsigned>((s.rem << (2 * s.lt - 2)) / 256));
    if (s.splits > 1) QN_LAUNCH("gated_dx_reduce", st, gated_dx_reduce, rgrid, dim3(256), 0, st, s, o);
    return hipGetLastError();
}

}  // namespace qn
