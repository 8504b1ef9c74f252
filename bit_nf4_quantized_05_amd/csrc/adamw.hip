// AdamW step over many tensors in one launch on gfx950, moments in 32 bits or in 8.
//
// Per element, with g the gradient times an optional device scalar (a clip factor):
//     m = b1 m + (1 - b1) g            v = b2 v + (1 - b2) g^2
//     p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// each product and sum one float32 operation in that order (the library is built without
// contraction), so the moments are the same bits as the same operations done one by one.
//
// 8-bit moments: blocks of 256 elements of a tensor with the block's largest magnitude
// `big` as float32. |x| / big in [0, 1] is kept as the upper bits of its float32 pattern,
// 3 mantissa bits: m as a sign and 127 levels (1 down to 1.25 2^-16), v as 255 levels (1
// down to 1.25 2^-32, so that sqrt(v) spans the range of m), level 0 is zero, and a v > 0
// never falls to zero (the update divides by its root). The bits cut off are rounded up
// with the probability of the part cut off: 16 random bits per moment from a 32-bit mix
// of the element's place and the step. Rounding to the nearest level would freeze v: b2 =
// 0.999 moves it by 0.1 % a step where half a level is 3 to 6 %; this way its mean follows
// the recurrence. The update itself uses the moments before they are rounded.
//
// adamw_kernel: a workgroup takes a chunk of 4 blocks of one tensor (a table built once
// names tensor and place), one wave per block, 4 elements per lane: every access is 16
// bytes a lane (4 for codes) and the block's largest magnitude is a wave reduction. Bound by
// HBM: p, g, m, v are read and p, m, v and the bf16 copy written once. 160 M float32
// parameters with float32 gradients and bf16 copies: 870 us, 5.5 TB/s (a 1 GiB device copy runs at
// 5.1); with 8-bit moments 553 to 569 us, 5.2 TB/s. Chunks of 8 blocks, two per wave: 908 and 540 us, but
// later to fill the chip with small sets (4 tensors of 8000 elements: 5.4 against 4.9 us a
// graph-replayed call); of 16: 895 and 545 us.
#include <hip/hip_runtime.h>

#include "internal.h"
#include "multi.h"
#include "nf4_device.h"

namespace qn {
namespace {

constexpr int kTopM = 127, kTopV = 255;          // code of 1.0
constexpr int kOneBits = 0x3F800000 >> 20;       // 1.0f's pattern with 3 mantissa bits
constexpr int kWaves = 4;

// 32-bit mixer: three xor-shifts around two odd multipliers (A. Appleby's constants)
__device__ __forceinline__ uint32_t mix32(uint32_t h) {
    h ^= h >> 16;
    h *= 0x85EBCA6Bu;
    h ^= h >> 13;
    h *= 0xC2B2AE35u;
    return h ^ (h >> 16);
}

__device__ __forceinline__ float level_value(int c, int top) {
    return c > 0 ? __uint_as_float(static_cast<uint32_t>(c + (kOneBits - top)) << 20) : 0.0f;
}

// x >= 0, inv = 1 / big (0 for a block of zeros)
__device__ __forceinline__ int level_code(float x, float inv, uint32_t bits16, int top) {
    const uint32_t b = __float_as_uint(fminf(x * inv, 1.0f)) + (bits16 << 4);
    return max(static_cast<int>(b >> 20) - (kOneBits - top), 0);
}

// largest magnitude of a block, a NaN above all (the patterns of magnitudes order as integers)
__device__ __forceinline__ float block_max(const float (&x)[4]) {
    uint32_t b = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) b = max(b, __float_as_uint(fabsf(x[e])));
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) b = max(b, static_cast<uint32_t>(__shfl_xor(static_cast<int>(b), o)));
    return __uint_as_float(b);
}

__device__ __forceinline__ float bf16_val(uint32_t u) { return __uint_as_float(u << 16); }

// 4 elements at p + i as float32 (0 past n)
template <bool kBf16>
__device__ __forceinline__ float4 load4(const void* p, int64_t i, int64_t n, bool whole) {
    float4 v = {0.0f, 0.0f, 0.0f, 0.0f};
    if constexpr (kBf16) {
        const uint16_t* q = static_cast<const uint16_t*>(p) + i;
        if (whole) {
            const uint2 w = *reinterpret_cast<const uint2*>(q);
            return float4{bf16_val(w.x & 0xFFFFu), bf16_val(w.x >> 16), bf16_val(w.y & 0xFFFFu), bf16_val(w.y >> 16)};
        }
        if (i < n) v.x = bf16_val(q[0]);
        if (i + 1 < n) v.y = bf16_val(q[1]);
        if (i + 2 < n) v.z = bf16_val(q[2]);
        if (i + 3 < n) v.w = bf16_val(q[3]);
    } else {
        const float* q = static_cast<const float*>(p) + i;
        if (whole) return *reinterpret_cast<const float4*>(q);
        if (i < n) v.x = q[0];
        if (i + 1 < n) v.y = q[1];
        if (i + 2 < n) v.z = q[2];
        if (i + 3 < n) v.w = q[3];
    }
    return v;
}

template <bool kBf16>
__device__ __forceinline__ void store4(void* p, int64_t i, int64_t n, bool whole, const float (&v)[4]) {
    if constexpr (kBf16) {
        uint16_t* q = static_cast<uint16_t*>(p) + i;
        if (whole) {
            *reinterpret_cast<uint2*>(q) = uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
            return;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i + e < n) q[e] = bf16_bits(v[e]);
    } else {
        float* q = static_cast<float*>(p) + i;
        if (whole) {
            *reinterpret_cast<float4*>(q) = float4{v[0], v[1], v[2], v[3]};
            return;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (i + e < n) q[e] = v[e];
    }
}

// b^t by squaring in float64 (t >= 1)
__device__ __forceinline__ double power(double b, int64_t t) {
    double r = 1.0;
    for (; t > 0; t >>= 1) {
        if (t & 1) r *= b;
        b *= b;
    }
    return r;
}

struct Coefs { float b1, c1, b2, c2, keep, step_size, inv_root; uint32_t key; };

__host__ __device__ inline Coefs coefs_of(double lr, double beta1, double beta2, double wd, double b1t, double b2t,
                                          double root2) {
    Coefs c{};
    c.b1 = static_cast<float>(beta1);
    c.c1 = static_cast<float>(1.0 - beta1);
    c.b2 = static_cast<float>(beta2);
    c.c2 = static_cast<float>(1.0 - beta2);
    c.keep = static_cast<float>(1.0 - lr * wd);
    c.step_size = static_cast<float>(lr / (1.0 - b1t));
    c.inv_root = static_cast<float>(1.0 / root2);
    return c;
}

template <bool k8, bool kGradBf16, bool kParamBf16>
__global__ __launch_bounds__(64 * kWaves)
void adamw_kernel(AdamArgs a, Coefs hc) {
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const AdamChunk ck = a.chunks[blockIdx.x];
    const AdamTensor t = a.tensors[ck.tensor];
    Coefs c = hc;
    uint32_t step = static_cast<uint32_t>(a.step);
    if (a.step_dev || a.lr_dev) {
        const int64_t n = a.step_dev ? a.step_dev[0] : a.step;
        if (n < 1) return;                              // 1 - beta^n would be 0 or less; nothing is written
        const double b2t = power(a.beta2, n);
        c = coefs_of(a.lr_dev ? static_cast<double>(a.lr_dev[0]) : a.lr, a.beta1, a.beta2, a.weight_decay,
                     power(a.beta1, n), b2t, sqrt(1.0 - b2t));
        step = static_cast<uint32_t>(n);
    }
    const uint32_t key = mix32(step ^ mix32(a.seed));
    const float gs = a.grad_scale ? a.grad_scale[0] : 1.0f;
    constexpr int kIt = kAdamChunkBlocks / kWaves;
    const int64_t blocks = (t.n + kAdamBlock - 1) / kAdamBlock;
    const int64_t b0 = static_cast<int64_t>(ck.chunk) * kAdamChunkBlocks;
    float4 p[kIt], g[kIt], m[kIt], v[kIt];
    uint32_t mc[kIt], vc[kIt];
    float ms[kIt], vs[kIt];
#pragma unroll
    for (int k = 0; k < kIt; ++k) {
        const int64_t b = min(b0 + wave + kWaves * k, blocks - 1);          // past the end: re-read, not stored
        const int64_t i = b * kAdamBlock + 4 * lane;
        const int64_t sb = t.first_block + b;
        const bool whole = t.vec && i + 4 <= t.n;
        p[k] = load4<kParamBf16>(t.p, i, t.n, whole);
        g[k] = load4<kGradBf16>(t.g, i, t.n, whole);
        if constexpr (k8) {
            mc[k] = static_cast<const uint32_t*>(a.m)[sb * 64 + lane];
            vc[k] = static_cast<const uint32_t*>(a.v)[sb * 64 + lane];
            ms[k] = a.m_scale[sb];
            vs[k] = a.v_scale[sb];
        } else {
            m[k] = static_cast<const float4*>(a.m)[sb * 64 + lane];
            v[k] = static_cast<const float4*>(a.v)[sb * 64 + lane];
        }
    }
#pragma unroll
    for (int k = 0; k < kIt; ++k) {
        const int64_t b = b0 + wave + kWaves * k;
        if (b >= blocks) break;                                             // wave-uniform
        const int64_t i = b * kAdamBlock + 4 * lane;
        const int64_t sb = t.first_block + b;
        const bool whole = t.vec && i + 4 <= t.n;
        const float pv[4] = {p[k].x, p[k].y, p[k].z, p[k].w};
        const float gv[4] = {g[k].x, g[k].y, g[k].z, g[k].w};
        float mo[4], vo[4], po[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            float m0, v0;
            if constexpr (k8) {
                const uint32_t cm = (mc[k] >> (8 * e)) & 0xFFu, cv = (vc[k] >> (8 * e)) & 0xFFu;
                m0 = level_value(static_cast<int>(cm & 0x7Fu), kTopM) * ms[k];
                m0 = (cm & 0x80u) ? -m0 : m0;
                v0 = level_value(static_cast<int>(cv), kTopV) * vs[k];
            } else {
                m0 = e == 0 ? m[k].x : e == 1 ? m[k].y : e == 2 ? m[k].z : m[k].w;
                v0 = e == 0 ? v[k].x : e == 1 ? v[k].y : e == 2 ? v[k].z : v[k].w;
            }
            const float ge = gv[e] * gs;
            const bool in = i + e < t.n;                       // past the end: zeros whatever the scales
            mo[e] = in ? m0 * c.b1 + ge * c.c1 : 0.0f;
            vo[e] = in ? v0 * c.b2 + (ge * ge) * c.c2 : 0.0f;
            const float den = sqrtf(vo[e]) * c.inv_root + a.eps;
            po[e] = pv[e] * c.keep - c.step_size * (mo[e] / den);
        }
        store4<kParamBf16>(t.p, i, t.n, whole, po);
        if (t.copy) store4<true>(t.copy, i, t.n, whole, po);
        if constexpr (k8) {
            const float bm = block_max(mo), bv = block_max(vo);
            // a block whose largest magnitude is below the normal numbers is kept as zeros; one
            // with an infinity or NaN keeps that as its scale, which no level makes finite
            const bool um = !(bm < 0x1p-126f), uv = !(bv < 0x1p-126f);
            const float im = bm >= 0x1p-126f ? 1.0f / bm : 0.0f, iv = bv >= 0x1p-126f ? 1.0f / bv : 0.0f;
            uint32_t wm = 0, wv = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t h = mix32((static_cast<uint32_t>(sb) * kAdamBlock + 4 * lane + e) ^ key);
                const int cm = level_code(fabsf(mo[e]), im, h & 0xFFFFu, kTopM);
                int cv = level_code(vo[e], iv, h >> 16, kTopV);
                if (vo[e] > 0.0f && uv) cv = max(cv, 1);
                wm |= static_cast<uint32_t>(cm | (mo[e] < 0.0f && cm > 0 ? 0x80 : 0)) << (8 * e);
                wv |= static_cast<uint32_t>(cv) << (8 * e);
            }
            static_cast<uint32_t*>(a.m)[sb * 64 + lane] = wm;
            static_cast<uint32_t*>(a.v)[sb * 64 + lane] = wv;
            if (lane == 0) {
                a.m_scale[sb] = um ? bm : 0.0f;
                a.v_scale[sb] = uv ? bv : 0.0f;
            }
        } else {
            static_cast<float4*>(a.m)[sb * 64 + lane] = float4{mo[0], mo[1], mo[2], mo[3]};
            static_cast<float4*>(a.v)[sb * 64 + lane] = float4{vo[0], vo[1], vo[2], vo[3]};
        }
    }
}

// The values of 8-bit moments: 4 codes of each per thread (one wave per block).
__global__ __launch_bounds__(256)
void adamw_moments_kernel(const uint32_t* __restrict__ m, const float* __restrict__ m_scale,
                          const uint32_t* __restrict__ v, const float* __restrict__ v_scale, int64_t words,
                          float4* __restrict__ m_out, float4* __restrict__ v_out) {
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= words) return;
    const uint32_t cm = m[i], cv = v[i];
    const float ms = m_scale[i >> 6], vs = v_scale[i >> 6];
    float a[4], b[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t x = (cm >> (8 * e)) & 0xFFu, y = (cv >> (8 * e)) & 0xFFu;
        const float t = level_value(static_cast<int>(x & 0x7Fu), kTopM) * ms;
        a[e] = (x & 0x80u) ? -t : t;
        b[e] = level_value(static_cast<int>(y), kTopV) * vs;
    }
    m_out[i] = float4{a[0], a[1], a[2], a[3]};
    v_out[i] = float4{b[0], b[1], b[2], b[3]};
}

}  // namespace

hipError_t launch_adamw(const AdamArgs& a, int64_t n_chunks, bool states8, bool grad_bf16, bool param_bf16,
                        hipStream_t st) {
    if (n_chunks == 0) return hipSuccess;
    Coefs c{};
    if (!a.step_dev && !a.lr_dev) {
        const double b2t = pow(a.beta2, static_cast<double>(a.step));
        c = coefs_of(a.lr, a.beta1, a.beta2, a.weight_decay, pow(a.beta1, static_cast<double>(a.step)), b2t,
                     sqrt(1.0 - b2t));
    }
    const dim3 grid(static_cast<unsigned>(n_chunks));
#define QN_ADAM(S8, GB, PB) \
    QN_LAUNCH(S8 ? "adamw_kernel_8" : "adamw_kernel_32", st, (adamw_kernel<S8, GB, PB>), grid, dim3(64 * kWaves), 0, \
              st, a, c)
    if (states8) {
        if (grad_bf16) { if (param_bf16) QN_ADAM(true, true, true); else QN_ADAM(true, true, false); }
        else { if (param_bf16) QN_ADAM(true, false, true); else QN_ADAM(true, false, false); }
    } else {
        if (grad_bf16) { if (param_bf16) QN_ADAM(false, true, true); else QN_ADAM(false, true, false); }
        else { if (param_bf16) QN_ADAM(false, false, true); else QN_ADAM(false, false, false); }
    }
#undef QN_ADAM
    return hipGetLastError();
}

hipError_t launch_adamw_moments(const uint8_t* m, const float* m_scale, const uint8_t* v, const float* v_scale,
                                int64_t blocks, float* m_out, float* v_out, hipStream_t st) {
    if (blocks == 0) return hipSuccess;
    const int64_t words = blocks * (kAdamBlock / 4);
    QN_LAUNCH("adamw_moments_kernel", st, adamw_moments_kernel, dim3(static_cast<unsigned>((words + 255) / 256)),
              dim3(256), 0, st, reinterpret_cast<const uint32_t*>(m), m_scale, reinterpret_cast<const uint32_t*>(v),
              v_scale, words, reinterpret_cast<float4*>(m_out), reinterpret_cast<float4*>(v_out));
    return hipGetLastError();
}

}  // namespace qn
