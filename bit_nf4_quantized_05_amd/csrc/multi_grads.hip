// Gradients of many adapters' factors in one batch on gfx950, and the transposed copies of
// the factors that the backward's products read.
//
// For the tokens t of adapter a (learn.ifs.name deck card 1: only the adapters are trained;
// the derivatives of Y = W_hat x + s_a B_a A_a x):
//     dB_a [d_out, r] = sum_t dY[t]^T T[t],   T[t] = s_a A_a x_t
//     dA_a [r, d_in]  = sum_t U[t]^T X[t],    U[t] = s_a B_a^T dy_t
// T and U come from the pre-passes as three bf16 terms each (24 bits together): the
// outputs are float32, and with one bf16 term they would carry its 2^-9 for the sake of a
// product that the reads of dY and X bound in any case.
//
// multi_grad_mfma: as the single-adapter kernel, a workgroup takes 128 columns of P = dY or
// X (32 per wave), 64 (or 32) ranks and a slice of one adapter's positions; per step of 32
// positions the gathered rows of P and the rows of the three terms go straight into LDS
// (two stages), and ds_read_b64_tr_b16 hands each lane 4 consecutive rows of a column, the
// MFMA's K order. A slice is `per` items (128 positions each) of the plan. An adapter whose
// tokens fit one slice is written to dA, dB at once; the others leave one partial per
// slice, added in slice order by multi_grad_reduce, which also writes the zeros of adapters
// without tokens. Deterministic; rows of other adapters are never read.
#include <hip/hip_runtime.h>

#include "internal.h"
#include "mfma_device.h"
#include "multi.h"
#include "nf4_device.h"

#include <algorithm>

namespace qn {
namespace {

constexpr int kGCols = 128;       // columns n per workgroup, 32 per wave
constexpr int kGJ = 64;           // ranks per workgroup (two 32-wide MFMA blocks)
constexpr int kGK = 32;           // positions per LDS stage
constexpr int kTerms = 3;
constexpr int kMaxPer = 8;        // items per slice at most

struct GradJob {
    const uint16_t* P; int64_t N, ldp;
    const uint16_t* T;               // [3][M][r]
    float* part;                     // [slots][N][r]
    float* out;                      // dB [n, N, r] or dA [n, r, N]
    int rows;                        // 1: out is [r, N]
    int tiles;                       // column tiles
};

struct GradArgs {
    GradJob job[2];                  // 0: dB (P = dY), 1: dA (P = X)
    MultiPlan plan;
    int M, r, jchunks, max_items, per;
};

__device__ __forceinline__ int swz(int m) { return 2 * (m & 3); }

struct GradTile {
    uint4 P[kGK * 16];               // 32 rows x 16 chunks of 8 columns
    uint4 T[kTerms][kGK * 8];        // 32 rows x 8 chunks of 8 ranks
};

#define QN_TR(d, a, off) "ds_read_b64_tr_b16 %" #d ", %" #a " offset:" #off "\n\t"

// 4 transposing reads of one operand (rows +0, +4, +16, +20 of the lane's block), waited for
template <int kRow>      // bytes per row
__device__ __forceinline__ void tr_read(uint32_t addr, unsigned long long (&v)[4]) {
    static_assert(kRow == 256 || kRow == 128, "row pitch");
    if constexpr (kRow == 256) {
        asm volatile(QN_TR(0, 4, 0) QN_TR(1, 4, 1024) QN_TR(2, 4, 4096) QN_TR(3, 4, 5120) "s_waitcnt lgkmcnt(0)"
                     : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]) : "v"(addr) : "memory");
    } else {
        asm volatile(QN_TR(0, 4, 0) QN_TR(1, 4, 512) QN_TR(2, 4, 2048) QN_TR(3, 4, 2560) "s_waitcnt lgkmcnt(0)"
                     : "=&v"(v[0]), "=&v"(v[1]), "=&v"(v[2]), "=&v"(v[3]) : "v"(addr) : "memory");
    }
}
#undef QN_TR

template <int JB>
__device__ __forceinline__ void grad_compute(const GradTile& t, int wave, int lane, int valid, f32x16 (&acc)[JB]) {
    const int g4 = lane >> 4, r = (lane >> 2) & 3, bq = lane & 3;
    const int m = 8 * (g4 >> 1) + r;
    const int n = 32 * wave + 16 * (g4 & 1) + 4 * bq;
    const uint32_t pa = lds_addr(t.P) + 2 * (m * 128 + ((((n >> 3) ^ swz(m)) << 3) | (n & 7)));
    unsigned long long a[4];
    tr_read<256>(pa, a);
    uint4 A[2];
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
        const int mb = 16 * sub + 8 * (g4 >> 1);                       // first position of this lane's 8
        uint32_t aw[4] = {static_cast<uint32_t>(a[2 * sub]), static_cast<uint32_t>(a[2 * sub] >> 32),
                          static_cast<uint32_t>(a[2 * sub + 1]), static_cast<uint32_t>(a[2 * sub + 1] >> 32)};
        if (valid < kGK) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t keep = (mb + 2 * i < valid ? 0xFFFFu : 0u) | (mb + 2 * i + 1 < valid ? 0xFFFF0000u : 0u);
                aw[i] &= keep;
            }
        }
        A[sub] = uint4{aw[0], aw[1], aw[2], aw[3]};
    }
#pragma unroll
    for (int p = 0; p < kTerms; ++p) {
#pragma unroll
        for (int jb = 0; jb < JB; ++jb) {
            const int j = 32 * jb + 16 * (g4 & 1) + 4 * bq;
            unsigned long long b[4];
            tr_read<128>(lds_addr(t.T[p]) + 2 * (m * 64 + ((((j >> 3) ^ swz(m)) << 3) | (j & 7))), b);
#pragma unroll
            for (int sub = 0; sub < 2; ++sub) {
                uint32_t bw[4] = {static_cast<uint32_t>(b[2 * sub]), static_cast<uint32_t>(b[2 * sub] >> 32),
                                  static_cast<uint32_t>(b[2 * sub + 1]), static_cast<uint32_t>(b[2 * sub + 1] >> 32)};
                if (valid < kGK) {          // rows past the slice belong to others: their terms must not count either
                    const int mb = 16 * sub + 8 * (g4 >> 1);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t keep = (mb + 2 * i < valid ? 0xFFFFu : 0u) |
                                              (mb + 2 * i + 1 < valid ? 0xFFFF0000u : 0u);
                        bw[i] &= keep;
                    }
                }
                acc[jb] = mfma32(A[sub], uint4{bw[0], bw[1], bw[2], bw[3]}, acc[jb]);
            }
        }
    }
}

template <int JB>   // 32-wide rank blocks per workgroup: 1 (r <= 32) or 2
__global__ __launch_bounds__(256)
void multi_grad_mfma(GradArgs g) {
    __shared__ GradTile s0, s1;
    __shared__ int s_order[kMaxPer * kMultiItem];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int b = static_cast<int>(blockIdx.x);
    const int nb0 = g.job[0].tiles * g.max_items * g.jchunks;
    const bool second = b >= nb0;
    const GradJob jb = second ? g.job[1] : g.job[0];
    b -= second ? nb0 : 0;
    const int tile = b % jb.tiles;
    b /= jb.tiles;
    const int item = b % g.max_items;
    const int j0 = (b / g.max_items) * kGJ;
    if (item >= g.plan.head[1]) return;
    const MultiItem it = g.plan.items[item];
    if (it.index % g.per != 0) return;
    const int end = g.plan.start[it.adapter + 1];
    const int m_lo = it.pos, m_hi = min(m_lo + g.per * kMultiItem, end);
    const bool alone = it.index == 0 && m_hi == end;                   // the adapter's only slice
    const int64_t n0 = static_cast<int64_t>(tile) * kGCols;
    const int steps = (m_hi - m_lo + kGK - 1) / kGK;
    const int64_t mr = static_cast<int64_t>(g.M) * g.r;

    f32x16 acc[JB];
#pragma unroll
    for (int k = 0; k < JB; ++k) acc[k] = f32x16{};

    // the slice's tokens, so that a step's loads wait for no index from memory
    for (int i = threadIdx.x; i < m_hi - m_lo; i += 256) s_order[i] = g.plan.order[m_lo + i];
    __syncthreads();
    // rows 4 (2 w + q) + lane / 16 of P, row 8 w + lane / 8 of each term
    auto issue = [&](GradTile& t, int m) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int row = 4 * (2 * wave + q) + (lane >> 4);
            const int64_t tok = s_order[min(m + row, m_hi - 1) - m_lo];
            const int64_t ng = min(n0 + 8 * ((lane & 15) ^ swz(row)), jb.N - 8);
            load_lds16(jb.P + tok * jb.ldp + ng, &t.P[(2 * wave + q) * 64]);
        }
        const int row = 8 * wave + (lane >> 3);
        const int64_t at = static_cast<int64_t>(min(m + row, m_hi - 1)) * g.r + min(j0 + 8 * ((lane & 7) ^ swz(row)), g.r - 8);
#pragma unroll
        for (int p = 0; p < kTerms; ++p) load_lds16(jb.T + p * mr + at, &t.T[p][wave * 64]);
    };
#define QN_GRAD_BARRIER() asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory")
    issue(s0, m_lo);
    for (int s = 0; s < steps; s += 2) {
        if (s + 1 < steps) { issue(s1, m_lo + (s + 1) * kGK); QN_WAIT_VM(2 + kTerms); }
        else QN_WAIT_VM(0);
        QN_GRAD_BARRIER();
        grad_compute<JB>(s0, wave, lane, min(kGK, m_hi - (m_lo + s * kGK)), acc);
        QN_GRAD_BARRIER();
        if (s + 1 >= steps) break;
        if (s + 2 < steps) { issue(s0, m_lo + (s + 2) * kGK); QN_WAIT_VM(2 + kTerms); }
        else QN_WAIT_VM(0);
        QN_GRAD_BARRIER();
        grad_compute<JB>(s1, wave, lane, min(kGK, m_hi - (m_lo + (s + 1) * kGK)), acc);
        QN_GRAD_BARRIER();
    }
#undef QN_GRAD_BARRIER
    // D of a 32 x 32 tile: lane l holds rows 8 (v / 4) + 4 (l / 32) + v % 4 of column l % 32
    const int64_t Nr = jb.N * g.r;
    float* dst = alone ? jb.out + it.adapter * Nr
                       : jb.part + (g.plan.first_item[it.adapter] / g.per + it.adapter + it.index / g.per) * Nr;
#pragma unroll
    for (int k = 0; k < JB; ++k) {
        const int j = j0 + 32 * k + (lane & 31);
        if (j >= g.r) continue;
#pragma unroll
        for (int v = 0; v < 16; v += 4) {
            const int64_t n = n0 + 32 * wave + 8 * (v >> 2) + 4 * (lane >> 5);
            if (n >= jb.N) continue;                                   // N % 64 == 0: 4 columns in or out together
            if (alone && jb.rows) {
                *reinterpret_cast<float4*>(dst + j * jb.N + n) = float4{acc[k][v], acc[k][v + 1], acc[k][v + 2], acc[k][v + 3]};
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e) dst[(n + e) * g.r + j] = acc[k][v + e];
            }
        }
    }
}

// Adapters of several slices: out = the sum of their partials in slice order; adapters
// without tokens: zeros; adapters of one slice are done. A workgroup takes 1024 elements of
// one adapter (blockIdx.y): 64 columns x 16 ranks, so that both layouts are written in
// runs of 16 or 64 elements.
__global__ __launch_bounds__(256)
void multi_grad_reduce(GradArgs g, int blocks0) {
    __shared__ float tile[64 * 17];
    const bool second = static_cast<int>(blockIdx.x) >= blocks0;
    const GradJob& jb = g.job[second ? 1 : 0];
    const int b = static_cast<int>(blockIdx.x) - (second ? blocks0 : 0);
    const int a = static_cast<int>(blockIdx.y);
    const int lo = g.plan.start[a], count = g.plan.start[a + 1] - lo;
    const int span = g.per * kMultiItem;
    const int slices = (count + span - 1) / span;
    if (slices == 1) return;
    const int jt = g.r / 16;
    const int64_t n0 = static_cast<int64_t>(b / jt) * 64;
    const int j0 = (b % jt) * 16;
    const int64_t Nr = jb.N * g.r;
    const int tid = threadIdx.x;
    const float* p = jb.part + (slices ? g.plan.first_item[a] / g.per + a : 0) * Nr;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int col = (tid >> 4) + 16 * q, j = tid & 15;
        const int64_t at = (n0 + col) * g.r + j0 + j;
        const float v = slices ? ordered_sum<4>(p + at, Nr, slices) : 0.0f;
        if (jb.rows) tile[col * 17 + j] = v;
        else jb.out[a * Nr + at] = v;
    }
    if (!jb.rows) return;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int col = tid & 63, j = (tid >> 6) + 4 * q;
        jb.out[a * Nr + (j0 + j) * jb.N + n0 + col] = tile[col * 17 + j];
    }
}

// dst[a] [cols, rows] = src[a] [rows, cols]^T in 64 x 64 tiles through LDS; adapter
// used[blockIdx.y]. rows and cols are multiples of 16.
struct TransposeJob { const uint16_t* src; uint16_t* dst; int rows, cols, tiles; };

__global__ __launch_bounds__(256)
void multi_transpose(TransposeJob j0, TransposeJob j1, const int32_t* __restrict__ head, const int32_t* __restrict__ used) {
    __shared__ uint16_t t[64 * 66];
    if (static_cast<int>(blockIdx.y) >= head[0]) return;
    const bool second = static_cast<int>(blockIdx.x) >= j0.tiles;
    const TransposeJob& j = second ? j1 : j0;
    const int b = static_cast<int>(blockIdx.x) - (second ? j0.tiles : 0);
    const int64_t base = static_cast<int64_t>(used[blockIdx.y]) * j.rows * j.cols;
    const int ct = (j.cols + 63) / 64;
    const int r0 = b / ct * 64, c0 = b % ct * 64;
    const int tid = threadIdx.x;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int row = (tid >> 3) + 32 * q, c = 8 * (tid & 7);
        if (r0 + row < j.rows && c0 + c < j.cols) {
            const uint4 v = *reinterpret_cast<const uint4*>(j.src + base + static_cast<int64_t>(r0 + row) * j.cols + c0 + c);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) *reinterpret_cast<uint32_t*>(&t[row * 66 + c + 2 * e]) = w[e];
        }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int col = (tid >> 3) + 32 * q, r = 8 * (tid & 7);
        if (c0 + col < j.cols && r0 + r < j.rows) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                w[e] = t[(r + 2 * e) * 66 + col] | (static_cast<uint32_t>(t[(r + 2 * e + 1) * 66 + col]) << 16);
            *reinterpret_cast<uint4*>(j.dst + base + static_cast<int64_t>(c0 + col) * j.rows + r0 + r) =
                uint4{w[0], w[1], w[2], w[3]};
        }
    }
}

int jchunks_of(int r) { return (r + kGJ - 1) / kGJ; }

// Items per slice: about 512 workgroups over both gradients if the tokens were evenly
// spread, at most 1024 positions a slice.
int per_of(int64_t d_out, int64_t d_in, int64_t M, int r) {
    const int64_t tiles = ((d_out + kGCols - 1) / kGCols + (d_in + kGCols - 1) / kGCols) * jchunks_of(r);
    const int64_t items = (M + kMultiItem - 1) / kMultiItem;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kMaxPer, items * tiles / 512)));
}

}  // namespace

hipError_t launch_multi_transpose(const MultiPlan& plan, int64_t max_used, const uint16_t* src0, int64_t rows0,
                                  int64_t cols0, uint16_t* dst0, const uint16_t* src1, int64_t rows1, int64_t cols1,
                                  uint16_t* dst1, hipStream_t st) {
    auto job = [](const uint16_t* s, int64_t rows, int64_t cols, uint16_t* d) {
        return TransposeJob{s, d, static_cast<int>(rows), static_cast<int>(cols),
                            static_cast<int>(((rows + 63) / 64) * ((cols + 63) / 64))};
    };
    const TransposeJob j0 = job(src0, rows0, cols0, dst0), j1 = job(src1, rows1, cols1, dst1);
    QN_LAUNCH("multi_transpose", st, multi_transpose,
              dim3(static_cast<unsigned>(j0.tiles + j1.tiles), static_cast<unsigned>(max_used)), dim3(256), 0, st, j0, j1,
              plan.head, plan.used);
    return hipGetLastError();
}

namespace {
int64_t slots_of(int64_t d_out, int64_t d_in, int64_t M, int n, int r) {
    return multi_max_items(M, n) / per_of(d_out, d_in, M, r) + n;
}
}  // namespace

int64_t multi_grads_part_floats(int64_t d_out, int64_t d_in, int64_t M, int n, int r) {
    return slots_of(d_out, d_in, M, n, r) * (d_out + d_in) * r;
}

hipError_t launch_multi_grads(const MultiPlan& plan, const uint16_t* X, int64_t ldx, const uint16_t* dY, int64_t lddy,
                              const uint16_t* T, const uint16_t* U, int64_t d_out, int64_t d_in, int64_t M, int n,
                              int r, float* part, float* dA, float* dB, hipStream_t st) {
    GradArgs g{};
    g.plan = plan;
    g.M = static_cast<int>(M); g.r = r; g.jchunks = jchunks_of(r);
    g.max_items = static_cast<int>(multi_max_items(M, n));
    g.per = per_of(d_out, d_in, M, r);
    auto tiles = [](int64_t N) { return static_cast<int>((N + kGCols - 1) / kGCols); };
    g.job[0] = GradJob{dY, d_out, lddy, T, part, dB, 0, tiles(d_out)};
    g.job[1] = GradJob{X, d_in, ldx, U, part + slots_of(d_out, d_in, M, n, r) * d_out * r, dA, 1, tiles(d_in)};
    const dim3 grid(static_cast<unsigned>((g.job[0].tiles + g.job[1].tiles) * g.max_items * g.jchunks));
    if (r <= 32) QN_LAUNCH("multi_grad_mfma", st, multi_grad_mfma<1>, grid, dim3(256), 0, st, g);
    else QN_LAUNCH("multi_grad_mfma", st, multi_grad_mfma<2>, grid, dim3(256), 0, st, g);
    const int b0 = static_cast<int>(d_out / 64 * (r / 16)), b1 = static_cast<int>(d_in / 64 * (r / 16));
    QN_LAUNCH("multi_grad_reduce", st, multi_grad_reduce, dim3(static_cast<unsigned>(b0 + b1), static_cast<unsigned>(n)),
              dim3(256), 0, st, g, b0);
    return hipGetLastError();
}

}  // namespace qn
