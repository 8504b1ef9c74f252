// Forward of few tokens (1 .. 64) that belong to many adapters, on gfx950: a decode batch.
//
// Y[t] = W_hat x_t + s_a B_a (A_a x_t). The weight's packed codes are streamed once for all
// tokens (skinny_nf4, its K-split partials); beside them every adapter in use is read once:
//
// multi_ax_small: the partials of s_a A_a x. A workgroup takes one item of the plan (the
// tokens of one adapter, at most 64 here), 16 ranks and a slice of K; its 4 waves take the
// slice's 64-wide blocks in turn. v_mfma_f32_16x16x32_bf16 with the adapter's 16 rank rows
// as one operand and 16 gathered tokens as the other, both straight from memory into
// registers (a lane takes 32 contiguous bytes of its row, the k order permuted alike on both
// sides; each byte of A is used by one wave only, so LDS would add a trip and save none).
// The waves' sums are added through LDS in wave order.
// multi_reduce_small: per 16 rows of W, adds the split partials of W_hat x in order, forms
// T = bf16(sum of the A x partials) in LDS and adds T B_a^T, B_a's rows read straight from
// memory by the threads of its tokens (16 rows of r values are contiguous); rounds once.
// Bound by latency for few tokens and by the reads of the codes and adapters beyond.
#include <hip/hip_runtime.h>

#include "internal.h"
#include "mfma_device.h"
#include "multi.h"
#include "nf4_device.h"

#include <algorithm>

namespace qn {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kAxBlocks = 16;           // 64-wide K-blocks per slice at least
constexpr int kAxSplits = 8;            // slices at most

__device__ __forceinline__ f32x4 mfma16(const uint4& a, const uint4& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c,
                                                   0, 0, 0);
}

struct SmallArgs {
    MultiPlan plan;
    MultiPool pool;
    const uint16_t* X; int64_t ldx;
    int d_out, d_in, M, splits, bper, tsplits;   // K-splits of W_hat x; K-blocks per slice and slices of A x
    const float* part;                  // [splits][M][d_out], by token
    float* part_t;                      // [tsplits][M][r], by position
    uint16_t* Y; int64_t ldy;
};

__global__ __launch_bounds__(256)
void multi_ax_small(SmallArgs a, int max_items) {
    __shared__ f32x4 red[3 * 4 * 64];
    int b = blockIdx.x;
    const int item = b % max_items;
    b /= max_items;
    const int sp = b % a.tsplits;
    const int j0 = b / a.tsplits * 16;
    if (item >= a.plan.head[1]) return;
    const MultiItem it = a.plan.items[item];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int nb = a.d_in / 64;
    const int b0 = sp * a.bper, b1 = min(b0 + a.bper, nb);
    const int tiles = (it.count + 15) / 16;             // 16-token tiles, <= 4
    const uint16_t* arow = a.pool.A + (static_cast<int64_t>(it.adapter) * a.pool.r + j0 + i) * a.d_in + 16 * g;
    const uint16_t* xrow[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int64_t tok = a.plan.order[it.pos + min(16 * t + i, it.count - 1)];
        xrow[t] = a.X + tok * a.ldx + 16 * g;
    }
    f32x4 acc[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int k = b0 + wave; k < b1; k += 4) {
        const uint4* ap = reinterpret_cast<const uint4*>(arow + static_cast<int64_t>(k) * 64);
        const uint4 a0 = ap[0], a1 = ap[1];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            if (t < tiles) {
                const uint4* xp = reinterpret_cast<const uint4*>(xrow[t] + static_cast<int64_t>(k) * 64);
                acc[t] = mfma16(a0, xp[0], acc[t]);
                acc[t] = mfma16(a1, xp[1], acc[t]);
            }
        }
    }
    if (wave > 0) {
#pragma unroll
        for (int t = 0; t < 4; ++t) red[((wave - 1) * 4 + t) * 64 + lane] = acc[t];
    }
    __syncthreads();
    if (wave > 0) return;
    const float s = a.pool.s[it.adapter];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
        const int row = 16 * t + i;
        if (row >= it.count) continue;
        f32x4 v = acc[t];
#pragma unroll
        for (int q = 0; q < 3; ++q) v = v + red[(q * 4 + t) * 64 + lane];
        // D of a 16 x 16 tile: lane l holds ranks 4 (l / 16) .. + 3 of token l % 16
        float* out = a.part_t + (static_cast<int64_t>(sp) * a.M + it.pos + row) * a.pool.r + j0 + 4 * g;
        *reinterpret_cast<float4*>(out) = float4{s * v[0], s * v[1], s * v[2], s * v[3]};
    }
}

constexpr int kRows = 16;               // rows of W per workgroup
constexpr int kJ = 64;                  // ranks per chunk

template <int SPL>                      // >= splits loads per output issued at once (clamped)
__global__ __launch_bounds__(256)
void multi_reduce_small(SmallArgs a) {
    __shared__ float s_t[kSkinnyMaxTokens * kJ];
    __shared__ int s_adapter[kSkinnyMaxTokens];
    const int tid = threadIdx.x;
    const int o = static_cast<int>(blockIdx.x) * kRows + (tid & 15);
    const int M = a.M, r = a.pool.r;
    const int live = a.plan.head[2];                     // positions with an adapter
    if (tid < a.plan.head[1]) {                          // one item per adapter in use (at most 64 tokens)
        const MultiItem it = a.plan.items[tid];
        for (int k = 0; k < it.count; ++k) s_adapter[it.pos + k] = it.adapter;
    }
    float pv[4][SPL];
    int64_t tok[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        tok[q] = a.plan.order[min((tid >> 4) + 16 * q, M - 1)];
#pragma unroll
        for (int sp = 0; sp < SPL; ++sp)
            pv[q][sp] = a.part[(static_cast<int64_t>(min(sp, a.splits - 1)) * M + tok[q]) * a.d_out + o];
    }
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int j0 = 0; j0 < r; j0 += kJ) {
        const int nj = min(kJ, r - j0);
        __syncthreads();                                 // s_adapter is there; the last chunk's reads are done
        for (int e = tid; e < live * nj; e += 256) {
            const int p = e / nj, j = e % nj;
            const float v = ordered_sum<8>(a.part_t + static_cast<int64_t>(p) * r + j0 + j,
                                           static_cast<int64_t>(M) * r, a.tsplits);
            s_t[p * kJ + j] = bf16_to_f32(bf16_bits(v));
        }
        __syncthreads();
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int p = (tid >> 4) + 16 * q;
            if (p >= live) continue;
            const uint4* bp = reinterpret_cast<const uint4*>(
                a.pool.B + (static_cast<int64_t>(s_adapter[p]) * a.d_out + o) * r + j0);
            for (int c = 0; c < nj / 8; ++c) {
                const uint4 w = bp[c];
                const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    acc[q] += s_t[p * kJ + 8 * c + 2 * e] * __uint_as_float(ws[e] << 16);
                    acc[q] += s_t[p * kJ + 8 * c + 2 * e + 1] * __uint_as_float(ws[e] & 0xFFFF0000u);
                }
            }
        }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int p = (tid >> 4) + 16 * q;
        if (p >= M) continue;
        float d = 0.0f;
#pragma unroll
        for (int sp = 0; sp < SPL; ++sp) d += sp < a.splits ? pv[q][sp] : 0.0f;
        a.Y[tok[q] * a.ldy + o] = bf16_bits(d + acc[q]);
    }
}

}  // namespace

int multi_small_splits(int64_t d_in) {
    const int64_t nb = d_in / 64;
    const int64_t per = std::max<int64_t>(kAxBlocks, (nb + kAxSplits - 1) / kAxSplits);
    return static_cast<int>((nb + per - 1) / per);
}

hipError_t launch_multi_small(const uint8_t* codes, const BlockConsts& bc, int64_t d_out, int64_t d_in,
                              const MultiPool& pool, const uint16_t* X, int64_t ldx, int64_t M,
                              const MultiPlan& plan, float* part, float* part_t, uint16_t* Y, int64_t ldy,
                              hipStream_t st) {
    SmallArgs a{};
    a.plan = plan; a.pool = pool; a.X = X; a.ldx = ldx;
    a.d_out = static_cast<int>(d_out); a.d_in = static_cast<int>(d_in); a.M = static_cast<int>(M);
    a.splits = skinny_splits(d_in, M);
    const int64_t nb = d_in / 64;
    a.bper = static_cast<int>(std::max<int64_t>(kAxBlocks, (nb + kAxSplits - 1) / kAxSplits));
    a.tsplits = multi_small_splits(d_in);
    a.part = part; a.part_t = part_t; a.Y = Y; a.ldy = ldy;
    hipError_t e = launch_skinny_stream(codes, bc, d_out, d_in, X, ldx, M, part, st);
    if (e != hipSuccess) return e;
    const int items = static_cast<int>(multi_max_items(M, pool.n));
    QN_LAUNCH("multi_ax_small", st, multi_ax_small, dim3(static_cast<unsigned>(items * a.tsplits * (pool.r / 16))),
              dim3(256), 0, st, a, items);
    const dim3 grid(static_cast<unsigned>(d_out / kRows));
    if (a.splits <= 4) QN_LAUNCH("multi_reduce_small", st, multi_reduce_small<4>, grid, dim3(256), 0, st, a);
    else QN_LAUNCH("multi_reduce_small", st, multi_reduce_small<8>, grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

}  // namespace qn
