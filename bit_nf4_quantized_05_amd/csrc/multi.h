// Internal declarations of the operators for many adapters on one layer (plan, forward,
// gradients) and of the AdamW step over their tensors.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "nf4_device.h"

namespace qn {

// ---- adamw.hip ----
constexpr int kAdamBlock = 256;             // elements per state block (one wave, 4 per lane)
constexpr int kAdamChunkBlocks = 4;         // blocks per workgroup
constexpr int kAdamChunk = kAdamBlock * kAdamChunkBlocks;
constexpr int64_t kAdamMaxChunks = (int64_t{1} << 24) - 1;        // a launch has under 2^32 threads

// One tensor of a step's table; the table is an array of these, then one AdamChunk per
// workgroup.
struct AdamTensor {
    void* p;                                // float32 or bf16 parameters [n]
    const void* g;                          // float32 or bf16 gradient [n]
    uint16_t* copy;                         // bf16 copy of p [n], or null
    int64_t n;
    int64_t first_block;                    // its first block in the state arrays
    int64_t vec;                            // 1: p, g, copy take 4 elements per access
};
struct AdamChunk {
    int32_t tensor;
    int32_t chunk;                          // chunk of the tensor
};

struct AdamArgs {
    const AdamTensor* tensors;
    const AdamChunk* chunks;
    void* m; void* v;                       // float32, or uint8 codes [blocks * 256]
    float* m_scale; float* v_scale;         // 8-bit states: largest magnitude per block
    const float* grad_scale;                // device scalar or null
    const float* lr_dev;                    // device learning rate or null (then lr)
    const int64_t* step_dev;                // device step number or null (then step)
    double lr, beta1, beta2, weight_decay;
    int64_t step;
    float eps;
    uint32_t seed;
};

hipError_t launch_adamw(const AdamArgs& a, int64_t n_chunks, bool states8, bool grad_bf16, bool param_bf16,
                        hipStream_t st);
// float32 values of the 8-bit states of `blocks` blocks
hipError_t launch_adamw_moments(const uint8_t* m, const float* m_scale, const uint8_t* v, const float* v_scale,
                                int64_t blocks, float* m_out, float* v_out, hipStream_t st);

// ---- multi_plan.hip ----
// The plan of a batch: its tokens sorted (stably) by adapter, as int32 words on the device.
// A position is an index into that order; tokens without an adapter come last.
constexpr int kMultiMaxAdapters = 1024;
constexpr int kMultiItem = 128;             // positions per work item at most
constexpr int kMultiTile = 256;             // positions per GEMM tile

// A run of at most 128 positions of one adapter: the first, how many are left from there to
// the adapter's last, and the item's number within its adapter. adapter -1: no item (the list
// is filled up with these, so that a kernel needs no count before it reads its item).
struct MultiItem { int32_t adapter, pos, left, index; };
__host__ __device__ inline int item_count(const MultiItem& it) { return it.left < kMultiItem ? it.left : kMultiItem; }
struct MultiPlan {
    const int32_t* head;                    // [0] adapters in use, [1] items, [2] positions with an adapter
    const int32_t* order;                   // [M] token at each position
    const int32_t* start;                   // [n + 1] first position of each adapter's tokens
    const int32_t* first_item;              // [n] each adapter's first item (adapters in use)
    const int32_t* used;                    // [min(n, M)] adapters in use, ascending
    const int2* tile;                       // [ceil(M / 256)] range of `used` with tokens in the tile
    const MultiItem* items;                 // [multi_max_items] runs of <= 128 positions of one adapter
};
inline int64_t multi_max_items(int64_t M, int64_t n) { return (M + kMultiItem - 1) / kMultiItem + (n < M ? n : M); }
// the plan's parts in a buffer of multi_plan_words(M, n) int32 words (16-byte aligned)
int64_t multi_plan_words(int64_t M, int64_t n);
MultiPlan multi_plan_at(const void* buf, int64_t M, int64_t n);
hipError_t launch_multi_plan(const int32_t* ids, int64_t M, int n, void* buf, hipStream_t st);

// ---- rank products as bf16 terms ----
// v rounded to bf16; v keeps what the rounding left (nothing of an infinity or NaN)
__device__ __forceinline__ uint16_t take_bf16(float& v) {
    const uint16_t h = bf16_bits(v);
    const float f = __uint_as_float(static_cast<uint32_t>(h) << 16);
    v = fabsf(f) < __builtin_inff() ? v - f : 0.0f;
    return h;
}

// 4 values as their next bf16 terms; the values keep the remainders
__device__ __forceinline__ uint2 take_bf16x4(float (&v)[4]) {
    const uint32_t a = take_bf16(v[0]), b = take_bf16(v[1]), c = take_bf16(v[2]), d = take_bf16(v[3]);
    return uint2{a | (b << 16), c | (d << 16)};
}

// ---- the adapters of a call ----
struct MultiPool {
    const uint16_t* A;                      // [n, r, d_in]
    const uint16_t* B;                      // [n, d_out, r]
    const float* s;                         // [n]
    int n, r;
};

// ---- prologue.hip ----
// Pre-passes of the multi-adapter calls and the double dequantisation of the weight to what
// (transposed or not; null: none) in one launch: T[piece][pos][r] = s_a P[order[pos], K]
// R_a[r, K]^T in `pieces` bf16 terms, each what the ones before left (2: 16 bits; 3: 24 bits),
// R [n, r, K] for the first product, [n, K, r] for the second (none if its R is null). K is
// cut in multi_pre_split(M, K).splits slices; with more than one, part holds their float32
// sums [slice][pos][r] and a second launch adds them in slice order.
struct MultiPre { const uint16_t* P; int64_t ldp; int64_t K; const uint16_t* R; float* part; uint16_t* T; };
// (A K of at most 512 is one slice: the second launch costs 4.8 us, a K-chunk of 64 about 0.4 us;
// backward of 203 tokens on 512 x 512 29.3 us against 29.9 in two slices. Slices of 4 chunks: 26 us
// in place of 22 with 256 adapters of one token on 4096 features, 14 as well with two; of 16:
// 21 and 18.)
PrepassSplit multi_pre_split(int64_t M, int64_t K);
hipError_t launch_multi_prologue(const uint8_t* codes, const BlockConsts& bc, int64_t d_out, int64_t d_in,
                                 bool transposed, uint16_t* what, const MultiPlan& plan, const float* s, int64_t M,
                                 int n, int r, int pieces, const MultiPre& p0, const MultiPre& p1, hipStream_t st);

// ---- gemm_multi.hip ----
// C[order[pos], :] = bf16( P[order[pos], K] Q[N, K]^T + (T[0] + T[1])[pos, r] R_a[N, r]^T ), T
// [2 or more][M, r] in bf16 terms, R [n, N, r] or, with rank_major, R_a^T given as [n, r, N]; a the adapter of the
// position (no second term without one). part holds gemm_multi_part_floats floats.
int64_t gemm_multi_part_floats(int64_t M, int64_t N, int64_t K);
hipError_t launch_gemm_multi(const uint16_t* P, int64_t ldp, const uint16_t* Q, int64_t K, const uint16_t* T,
                             const uint16_t* R, bool rank_major, int r, const MultiPlan& plan,
                             uint16_t* C, int64_t ldc, int64_t M, int64_t N, float* part, hipStream_t st);

// ---- gemv.hip ----
// One token with the adapter *adapter (none if negative) of a pool, in one launch: W_hat x +
// s_a B_a (A_a x), for r <= 16 and d_in <= 4096 (gemv_selects).
bool gemv_selects(int64_t d_in, int r);
hipError_t launch_gemv_nf4_select(const uint8_t* codes, const BlockConsts& bc, int64_t d_out, int64_t d_in,
                                  const uint16_t* A, const uint16_t* B, const float* s, int r, const int32_t* adapter,
                                  const uint16_t* x, uint16_t* y, hipStream_t st);

// ---- skinny.hip, multi_small.hip ----
// Forward of up to kSkinnyMaxTokens tokens from the packed codes: the W_hat x partials
// [multi_splits(d_out, d_in, M)][M][d_out] by token and the s_a A_a x partials
// [multi_small_splits][M][r] by position in one launch, then Y from both.
int multi_splits(int64_t d_out, int64_t d_in, int64_t M);
int multi_small_splits(int64_t d_in, int64_t M, int n, int r);
hipError_t launch_skinny_multi(const uint8_t* codes, const BlockConsts& bc, int64_t d_out, int64_t d_in,
                               const MultiPool& pool, const MultiPlan& plan, const uint16_t* X, int64_t ldx,
                               int64_t M, float* part, float* part_t, hipStream_t st);
hipError_t launch_multi_small(const uint8_t* codes, const BlockConsts& bc, int64_t d_out, int64_t d_in,
                              const MultiPool& pool, const uint16_t* X, int64_t ldx, int64_t M,
                              const MultiPlan& plan, float* part, float* part_t, uint16_t* Y, int64_t ldy,
                              hipStream_t st);

// ---- multi_grads.hip ----
// dB[a] [d_out, r] = sum over a's positions of dY^T T, dA[a] [r, d_in] of U^T X (zeros for an
// adapter without tokens); T, U [3][M][r]. part holds multi_grads_part_floats floats.
int64_t multi_grads_part_floats(int64_t d_out, int64_t d_in, int64_t M, int n, int r);
hipError_t launch_multi_grads(const MultiPlan& plan, const uint16_t* X, int64_t ldx, const uint16_t* dY, int64_t lddy,
                              const uint16_t* T, const uint16_t* U, int64_t d_out, int64_t d_in, int64_t M, int n,
                              int r, float* part, float* dA, float* dB, hipStream_t st);

}  // namespace qn
