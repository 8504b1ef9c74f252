// Forward of few tokens (1 .. 64) that belong to many adapters, on gfx950: a decode batch.
//
// Y[t] = W_hat x_t + s_a B_a (A_a x_t), in two launches:
//   skinny_nf4<., true> (skinny.hip) streams the weight's packed codes once for all tokens
//   into K-split partials of W_hat x, and beside them reads A of every adapter in use once
//   for the partials of s_a A_a x;
//   multi_reduce_small adds the partials and the rank term;
// or, for one token with r <= 16 and d_in <= 4096, in the streaming GEMV's one launch, which
// reads the token's adapter from the plan (4096 x 4096: 10.9 -> 6.9 us per graph-replayed call).
//
// multi_reduce_small: a workgroup takes 16 rows of W and all tokens. It forms T = the sum
// of the A x partials in slice order of every position in LDS, as two bf16 terms (16 bits: one
// term's 2^-9 would show in the output); its waves take the plan's
// items (the tokens of one adapter) in turn, v_mfma_f32_16x16x32_bf16 with the item's 16
// rows of B_a, straight from memory, as one operand and both terms of 16 of its tokens' T as the other;
// the products go to LDS by position, and each output is the ordered sum of its W_hat x
// partials plus its product, rounded once. Every byte of B is read by one wave, 64
// contiguous bytes per 4 lanes (one thread per row and token read its row in eight strided
// pieces before: 34 us for the 67 MB of 48 adapters of rank 64 on 11008 rows). A wave has
// the loads of several items in flight, the first ones from before T is formed. Bound by
// latency for few tokens and by the read of B beyond.
#include <hip/hip_runtime.h>

#include "internal.h"
#include "mfma_device.h"
#include "multi.h"
#include "nf4_device.h"

#include <algorithm>

namespace qn {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kRows = 16;               // rows of W per workgroup
constexpr int kWaves = 4;

struct SmallArgs {
    MultiPlan plan;
    const uint16_t* B;                  // [n, d_out, r]
    int d_out, M, r, splits, tsplits, max_items;
    const float* part;                  // [splits][M][d_out], by token
    const float* part_t;                // [tsplits][M][r], by position
    uint16_t* Y; int64_t ldy;
};

// RC: 32-rank chunks (r <= 32 RC); TT: 16-token tiles (M <= 16 TT); SPL >= splits
template <int RC, int TT, int SPL>
__global__ __launch_bounds__(64 * kWaves)
void multi_reduce_small(SmallArgs a) {
    constexpr int kPitch = 32 * RC + 8;                  // bf16 per row of T: 16-byte rows, banks 4 apart
    constexpr int kBatch = RC >= 4 ? 2 : 8 / RC;         // items whose B a wave has in flight
    constexpr bool kSkip = RC >= 2;
    __shared__ __align__(16) uint16_t s_t[2][16 * TT * kPitch];
    __shared__ float s_y[16 * TT][kRows + 1];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int o0 = static_cast<int>(blockIdx.x) * kRows;
    const int M = a.M, r = a.r;
    const int items = a.plan.head[1], live = a.plan.head[2];

    // rows o0 + i of B of items k0, k0 + 4, ..; ranks past r are zeros
    auto load_b = [&](int k0, uint4 (&w)[kBatch][RC]) {
        int ad[kBatch];
#pragma unroll
        for (int n = 0; n < kBatch; ++n)
            // (no wait for the count: the list is full of items of adapter -1 past its end)
            ad[n] = a.plan.items[min(k0 + kWaves * n, a.max_items - 1)].adapter;
#pragma unroll
        for (int n = 0; n < kBatch; ++n) {
            // larger ranks: nothing is read for no item (64 tokens of 11008 x 4096, r = 64: a call
            // 51.0 -> 49.7 us; at r = 16 the branch costs more, 64 of 4096 x 4096 20.6 -> 22.3)
            if (kSkip && __builtin_amdgcn_readfirstlane(ad[n]) < 0) continue;
            const uint16_t* row = a.B + (static_cast<int64_t>(max(ad[n], 0)) * a.d_out + o0 + i) * r;
#pragma unroll
            for (int c = 0; c < RC; ++c) {
                const uint4 v = *reinterpret_cast<const uint4*>(row + min(32 * c + 8 * g, r - 8));
                w[n][c] = 32 * c + 8 * g < r ? v : uint4{0, 0, 0, 0};
            }
        }
    };
    uint4 bw[kBatch][RC];
    load_b(wave, bw);
    float pv[TT][SPL];
    int64_t tok[TT];
#pragma unroll
    for (int q = 0; q < TT; ++q) {
        tok[q] = a.plan.order[min((tid >> 4) + 16 * q, M - 1)];
#pragma unroll
        for (int sp = 0; sp < SPL; ++sp)
            pv[q][sp] = a.part[(static_cast<int64_t>(min(sp, a.splits - 1)) * M + tok[q]) * a.d_out + o0 + (tid & 15)];
    }
    // T: 4 ranks per thread and pass; the ranks past r are zeros
    const int quads = 8 * RC;                            // per position
    for (int e = tid; e < live * quads; e += 64 * kWaves) {
        const int p = e / quads, j = e % quads * 4;
        float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (j < r) {
            const float* pt = a.part_t + static_cast<int64_t>(p) * r + j;
            const int64_t stride = static_cast<int64_t>(M) * r;
            // as many loads as there are slices (uniform)
            const float4 t = a.tsplits == 1 ? *reinterpret_cast<const float4*>(pt)
                             : a.tsplits <= 4 ? ordered_sum4<4>(pt, stride, a.tsplits)
                                              : ordered_sum4<8>(pt, stride, a.tsplits);
            v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) *reinterpret_cast<uint2*>(&s_t[h][p * kPitch + j]) = take_bf16x4(v);
    }
    __syncthreads();
    for (int k0 = wave; k0 < items; k0 += kWaves * kBatch) {
        if (k0 != wave) load_b(k0, bw);
#pragma unroll
        for (int n = 0; n < kBatch; ++n) {
            const int k = k0 + kWaves * n;
            if (k >= items) break;                       // wave-uniform
            const MultiItem it = a.plan.items[k];
            const int count = item_count(it);
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                if (16 * t >= count) break;
                const int row = 16 * t + i;
                f32x4 acc = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int c = 0; c < RC; ++c)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const uint4 tv = *reinterpret_cast<const uint4*>(
                            &s_t[h][(it.pos + min(row, count - 1)) * kPitch + 32 * c + 8 * g]);
                        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, bw[n][c]),
                                                                      __builtin_bit_cast(bf16x8, tv), acc, 0, 0, 0);
                    }
                // D of a 16 x 16 tile: lane l holds rows 4 (l / 16) .. + 3 of token l % 16
                if (row < count) {
#pragma unroll
                    for (int v = 0; v < 4; ++v) s_y[it.pos + row][4 * g + v] = acc[v];
                }
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < TT; ++q) {
        const int p = (tid >> 4) + 16 * q;
        if (p >= M) continue;
        float d = 0.0f;
#pragma unroll
        for (int sp = 0; sp < SPL; ++sp) d += sp < a.splits ? pv[q][sp] : 0.0f;
        a.Y[tok[q] * a.ldy + o0 + (tid & 15)] = bf16_bits(p < live ? d + s_y[p][tid & 15] : d);
    }
}

template <int RC>
hipError_t launch_reduce(const SmallArgs& a, hipStream_t st) {
    const dim3 grid(static_cast<unsigned>(a.d_out / kRows));
#define QN_RED(TT, SPL) \
    QN_LAUNCH("multi_reduce_small", st, (multi_reduce_small<RC, TT, SPL>), grid, dim3(64 * kWaves), 0, st, a)
    // as many partial loads per output as the split count allows
    switch ((a.M + 15) / 16) {
        case 1: if (a.splits <= 4) QN_RED(1, 4); else QN_RED(1, 8); break;
        case 2: if (a.splits <= 4) QN_RED(2, 4); else QN_RED(2, 8); break;
        default: if (a.splits <= 4) QN_RED(4, 4); else QN_RED(4, 8); break;
    }
#undef QN_RED
    return hipGetLastError();
}

}  // namespace

hipError_t launch_multi_small(const uint8_t* codes, const BlockConsts& bc, int64_t d_out, int64_t d_in,
                              const MultiPool& pool, const uint16_t* X, int64_t ldx, int64_t M,
                              const MultiPlan& plan, float* part, float* part_t, uint16_t* Y, int64_t ldy,
                              hipStream_t st) {
    // one token: the first item's adapter is its own (none: -1)
    if (M == 1 && gemv_selects(d_in, pool.r))
        return launch_gemv_nf4_select(codes, bc, d_out, d_in, pool.A, pool.B, pool.s, pool.r, &plan.items[0].adapter, X,
                                      Y, st);
    const hipError_t e = launch_skinny_multi(codes, bc, d_out, d_in, pool, plan, X, ldx, M, part, part_t, st);
    if (e != hipSuccess) return e;
    SmallArgs a{};
    a.plan = plan; a.B = pool.B;
    a.d_out = static_cast<int>(d_out); a.M = static_cast<int>(M); a.r = pool.r;
    a.splits = multi_splits(d_out, d_in, M);
    a.tsplits = multi_small_splits(d_in, M, pool.n, pool.r);
    a.max_items = static_cast<int>(multi_max_items(M, pool.n));
    a.part = part; a.part_t = part_t; a.Y = Y; a.ldy = ldy;
    if (pool.r <= 32) return launch_reduce<1>(a, st);
    if (pool.r <= 64) return launch_reduce<2>(a, st);
    if (pool.r <= 128) return launch_reduce<4>(a, st);
    return launch_reduce<8>(a, st);
}

}  // namespace qn
