// The gated feed-forward block's launches, shared by gated.hip, gated_small.hip, prologue.hip and api.hip.
//   H = act(G) * U,  G = W_g x + s_g B_g (A_g x),  U = W_u x + s_u B_u (A_u x)
// and its gradient. Index 0 is the gate projection, 1 the up projection.
#pragma once
#include <hip/hip_runtime.h>

#include "internal.h"
#include "mfma_device.h"
#include "nf4_device.h"

namespace qn {

constexpr int kActSilu = 0, kActGelu = 1;

struct GatedCall {
    const uint8_t* codes[2]; BlockConsts bc[2];
    int64_t d_ff, d_in;
    const uint16_t* A[2];             // [r, d_in]
    const uint16_t* B[2];             // [d_ff, r]
    float s[2];
    int r, act;                       // r 0: no adapters
    int64_t M;
    int terms;                        // bf16 terms of the rank products past kGatedSmall tokens (gated_terms)
};

// The rank products s A x and s B^T dY of one projection as `terms` bf16 terms, the second what the
// first leaves (16 bits; with one term its 2^-9 shows in every output beside the output's own
// rounding: 41 % of rank-dominated outputs were not the rounded result, 0.2 to 0.6 % with two): columns of one
// term, of the projection, and of both, which are whole K-steps of 64 (0 without adapters). Up to rank 16
// the second term takes room that the first leaves; at rank 64 it is two K-steps more (forward of 2048
// tokens of 11008 x 4096 336 -> 345 us, the gradient 366 -> 368).
inline int gated_term(int r, int terms) { return terms == 2 ? (r + 15) / 16 * 16 : (r + 31) / 32 * 32; }
inline int gated_pad(int r, int terms) { return terms * gated_term(r, terms); }
inline int gated_k2(int r, int terms) { return 2 * gated_pad(r, terms); }
// Two terms, or one where an operand of them would reach 4 GiB (at rank 256 from 2^21 tokens, d_in or rows of
// both weights on, at rank 64 from 2^23; up to rank 16 one term is as long)
inline int gated_terms(int64_t d_ff, int64_t d_in, int64_t M, int r) {
    const int64_t rows = M > d_in ? M : d_in;
    return r == 0 || (rows > 2 * d_ff ? rows : 2 * d_ff) <= ((int64_t{1} << 31) - 1) / gated_k2(r, 2) ? 2 : 1;
}

// act(g), and its derivative. sigma(x) = 1 / (1 + 2^(-x log2 e)) with the hardware's 2^x and
// 1/x (1 ulp each), 0 or 1 where 2^x leaves float32.
__device__ __forceinline__ float gated_sigmoid(float x) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504088896341f * x));
}
// silu: g sigma(g); gelu: g sigma(2 c (g + k g^3)), the tanh form g / 2 (1 + tanh(..)) without
// its cancellation for negative g
constexpr float kGeluC2 = 1.59576912160573071f, kGeluK = 0.044715f;      // 2 sqrt(2 / pi)
__device__ __forceinline__ float gated_act(int act, float g) {
    const float x = act == kActSilu ? g : kGeluC2 * (g + kGeluK * (g * g) * g);
    return g * gated_sigmoid(x);
}
__device__ __forceinline__ float gated_act_grad(int act, float g, float& value) {
    if (act == kActSilu) {
        const float s = gated_sigmoid(g);
        value = g * s;
        return s * (1.0f + g * (1.0f - s));
    }
    const float s = gated_sigmoid(kGeluC2 * (g + kGeluK * (g * g) * g));
    value = g * s;
    // past |g| = 16, s (1 - s) is 0 in float32; the bound keeps g^2 from overflowing beside it
    const float q = fminf(fmaxf(g, -16.0f), 16.0f);
    return s + q * (s * (1.0f - s)) * (kGeluC2 * (1.0f + 3.0f * kGeluK * (q * q)));
}

// dG = dH U act'(G), dU = dH act(G), elementwise over [M, d_ff]; G | U and dG | dU stand side by
// side in rows of GU and dGU. They are outputs in bf16, and dX is formed from these: of two bf16 terms it
// would take a second product (another 250 us at 2048 tokens of 11008 x 4096) for an error of 0.0017 in
// place of 0.0023, relative, beside the 0.0017 that dX's own rounding makes.
struct GatedGradArgs {
    const uint16_t* dH; int64_t lddh;
    const uint16_t* GU; int64_t ldgu;
    uint16_t* dGU; int64_t lddgu;
    int M, d_ff, act;
};
constexpr int kGradPer = 2;           // 8-wide pieces per thread, 256 apart (4: 88 registers, 2048 tokens of 11008 x 4096 6 us more)
inline int gated_grad_blocks(const GatedGradArgs& g) {
    const int64_t pieces = static_cast<int64_t>(g.M) * (g.d_ff / 8);
    return static_cast<int>((pieces + 256 * kGradPer - 1) / (256 * kGradPer));
}

__device__ __forceinline__ void gated_grad_job(const GatedGradArgs& a, int b) {
    const int cpr = a.d_ff / 8;
    const int64_t total = static_cast<int64_t>(a.M) * cpr;
    const int64_t first = static_cast<int64_t>(b) * (256 * kGradPer) + threadIdx.x;
    uint4 h[kGradPer], g[kGradPer], u[kGradPer];
    int64_t row[kGradPer];
    int col[kGradPer];
#pragma unroll
    for (int k = 0; k < kGradPer; ++k) {
        const int64_t at = min(first + 256 * k, total - 1);
        row[k] = at / cpr;
        col[k] = static_cast<int>(at - row[k] * cpr) * 8;
        h[k] = *reinterpret_cast<const uint4*>(a.dH + row[k] * a.lddh + col[k]);
        g[k] = *reinterpret_cast<const uint4*>(a.GU + row[k] * a.ldgu + col[k]);
        u[k] = *reinterpret_cast<const uint4*>(a.GU + row[k] * a.ldgu + a.d_ff + col[k]);
    }
#pragma unroll
    for (int k = 0; k < kGradPer; ++k) {
        if (first + 256 * k >= total) break;
        const uint32_t hw[4] = {h[k].x, h[k].y, h[k].z, h[k].w};
        const uint32_t gw[4] = {g[k].x, g[k].y, g[k].z, g[k].w};
        const uint32_t uw[4] = {u[k].x, u[k].y, u[k].z, u[k].w};
        uint32_t og[4], ou[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float dg[2], du[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float hv = __uint_as_float(e ? hw[q] & 0xFFFF0000u : hw[q] << 16);
                const float gv = __uint_as_float(e ? gw[q] & 0xFFFF0000u : gw[q] << 16);
                const float uv = __uint_as_float(e ? uw[q] & 0xFFFF0000u : uw[q] << 16);
                float act;
                const float slope = gated_act_grad(a.act, gv, act);
                dg[e] = hv * uv * slope;
                du[e] = hv * act;
            }
            og[q] = bf16_pair(dg[0], dg[1]);
            ou[q] = bf16_pair(du[0], du[1]);
        }
        uint16_t* out = a.dGU + row[k] * a.lddgu + col[k];
        *reinterpret_cast<uint4*>(out) = uint4{og[0], og[1], og[2], og[3]};
        *reinterpret_cast<uint4*>(out + a.d_ff) = uint4{ou[0], ou[1], ou[2], ou[3]};
    }
}

// ---- prologue.hip ----
// Both weights dequantised to what, gate above up, [2 d_ff, d_in], and both adapters to adapt
// (forward: B, [2 d_ff, k2]; gradient: A, [k2, d_in]); in the gradient the elementwise part grad and, where
// bt is not null, B^T [r, d_ff]. Then (r > 0) the rank products of in: t [M, k2] = s_w X A_w^T, or
// s_w (half w of dGU) B_w, in c.terms bf16 terms; part: gated_ranks_floats, K = d_in or d_ff.
struct GatedProlog {
    uint16_t* what; uint16_t* adapt;
    const uint16_t* in; int64_t ld_in; uint16_t* t; float* part;
    uint16_t* bt[2];                  // gradient: null where B itself can be read (gated_reads_b)
    GatedGradArgs grad;
};
inline bool gated_reads_b(int r) { return r % 8 == 0; }
int64_t gated_ranks_floats(int64_t M, int64_t K, int r, int terms);
hipError_t launch_gated_prologue(const GatedCall& c, bool backward, const GatedProlog& o, hipStream_t st);

// W_hat [d_out, d_in] bf16, row-major (d_in % 64 == 0)
hipError_t launch_dequant_weight(const uint8_t* codes, const BlockConsts& bc, int64_t d_out, int64_t d_in, uint16_t* what,
                                 hipStream_t st);

// ---- gated.hip ----
// H (and GU, if not null) from X, the weights what, the rank products t [M, k2] and the adapters
// adapt [2 d_ff, k2] (t, adapt unused without adapters); part holds gated_part_floats floats.
int64_t gated_part_floats(int64_t M, int64_t d_ff, int64_t d_in);
hipError_t launch_gated_gemm(const GatedCall& c, const uint16_t* X, int64_t ldx, const uint16_t* what, const uint16_t* t,
                             const uint16_t* adapt, uint16_t* H, int64_t ldh, uint16_t* GU, int64_t ldgu, float* part,
                             hipStream_t st);
// dX from dGU, what [2 d_ff, d_in], t [M, k2] and adapt [k2, d_in]; part: gated_dx_part_floats
int64_t gated_dx_part_floats(int64_t M, int64_t d_ff, int64_t d_in);
hipError_t launch_gated_dx(const GatedCall& c, const uint16_t* dGU, int64_t lddgu, const uint16_t* what, const uint16_t* t,
                           const uint16_t* adapt, uint16_t* dX, int64_t lddx, float* part, hipStream_t st);

// ---- gated_small.hip ----
// The forward on up to kGatedSmall tokens; part holds gated_small_part_floats floats.
constexpr int kGatedSmall = 64;
int64_t gated_small_part_floats(int64_t M, int64_t d_ff, int64_t d_in, int r);
hipError_t launch_gated_small(const GatedCall& c, const uint16_t* X, int64_t ldx, uint16_t* H, int64_t ldh, uint16_t* GU,
                              int64_t ldgu, float* part, hipStream_t st);

}  // namespace qn
