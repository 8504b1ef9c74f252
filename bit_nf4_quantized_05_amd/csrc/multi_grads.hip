// Gradients of many adapters' factors in one batch on gfx950.
//
// For the tokens t of adapter a (learn.ifs.name deck card 1: only the adapters are trained;
// the derivatives of Y = W_hat x + s_a B_a A_a x):
//     dB_a [d_out, r] = sum_t dY[t]^T T[t],   T[t] = s_a A_a x_t
//     dA_a [r, d_in]  = sum_t U[t]^T X[t],    U[t] = s_a B_a^T dy_t
// T and U come from the pre-passes as three bf16 terms each (24 bits together): the
// outputs are float32, and with one bf16 term they would carry its 2^-9 for the sake of a
// product that the reads of dY and X bound in any case.
//
// multi_grad_mfma: as for one adapter, a workgroup takes 128 columns of P = dY or X (32 per
// wave), 64 (or 32) ranks and a slice of one adapter's positions; per step of 32 positions the
// gathered rows of P and the rows of the three terms go straight into LDS (two stages), and
// transposing reads hand each lane 4 consecutive rows of a column, the MFMA's K order. A slice is
// `per` items (128 positions each) of the plan. An adapter whose tokens fit one slice is written
// to dA, dB at once; the others leave one partial per slice, added in slice order by
// multi_grad_reduce, which also writes the zeros of adapters without tokens. A batch of up to 512
// tokens is one slice per adapter, its last workgroups write the zeros, and there is no second
// launch. Deterministic; rows of other adapters count nowhere.
// Slots of partials: only an adapter of more than one slice's tokens ("span", 128 per) has any,
// c > span tokens ceil(c / span) of them, which is at most floor(2 c / span). So the first slot
// floor(2 start[a] / span) leaves room for all of a's before the next adapter's, and there are at
// most 2 M / span, whatever the pool holds. With few adapters first_item[a] / per + a is less and
// does as well (at most items / per + n); the smaller of two such numbers does too.
// Bound by the reads of dY and X and, with many slices, of the partials.
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
    int zero_at, zero_blocks;        // workgroups from zero_at on: zeros, zero_blocks per adapter
};

// 16-byte piece c of row m sits at c ^ swz(m), so that the 4 rows of a transposing read fall in
// different banks (rows of 64 bytes do without)
__device__ __forceinline__ int swz(int m) { return 2 * (m & 3); }

template <int JB>
struct GradTile {
    uint4 P[kGK * 16];               // 32 rows x 16 pieces of 8 columns
    uint4 T[kTerms][kGK * 4 * JB];   // 32 rows x 4 JB pieces of 8 ranks
};

// Transposing reads, each asm block ending with its own wait. (The builtin form would have
// the compiler wait for every load in flight, the next stage's too, before each read.) A
// lane's reads are its rows +0, +4, +16 and +20: two 16-row MFMA steps.
#define QN_TR(d, a, off) "ds_read_b64_tr_b16 %" #d ", %" #a " offset:%" #off "\n\t"
#define QN_TR4(d0, d1, d2, d3, a, o0, o1, o2, o3) QN_TR(d0, a, o0) QN_TR(d1, a, o1) QN_TR(d2, a, o2) QN_TR(d3, a, o3)
typedef unsigned long long u64;

__device__ __forceinline__ uint4 fragment(u64 a, u64 b) {
    return uint4{static_cast<uint32_t>(a), static_cast<uint32_t>(a >> 32), static_cast<uint32_t>(b),
                 static_cast<uint32_t>(b >> 32)};
}

// rows past `valid` as zeros (they belong to other adapters); first row of the lane's 8 is mb
__device__ __forceinline__ uint4 masked(const uint4& f, int mb, int valid) {
    uint32_t w[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] &= (mb + 2 * i < valid ? 0xFFFFu : 0u) | (mb + 2 * i + 1 < valid ? 0xFFFF0000u : 0u);
    return uint4{w[0], w[1], w[2], w[3]};
}

// the 4 reads of term kP at each of the JB rank blocks' addresses
template <int JB, int kP>
__device__ __forceinline__ void read_term(const uint32_t (&ta)[JB], u64 (&b)[JB][4]) {
    constexpr int kRow = 64 * JB, kOff = kP * kGK * kRow;
    if constexpr (JB == 1) {
        asm volatile(QN_TR4(0, 1, 2, 3, 4, 5, 6, 7, 8) "s_waitcnt lgkmcnt(0)"
                     : "=&v"(b[0][0]), "=&v"(b[0][1]), "=&v"(b[0][2]), "=&v"(b[0][3])
                     : "v"(ta[0]), "n"(kOff), "n"(kOff + 4 * kRow), "n"(kOff + 16 * kRow), "n"(kOff + 20 * kRow)
                     : "memory");
    } else {
        asm volatile(QN_TR4(0, 1, 2, 3, 8, 10, 11, 12, 13) QN_TR4(4, 5, 6, 7, 9, 10, 11, 12, 13) "s_waitcnt lgkmcnt(0)"
                     : "=&v"(b[0][0]), "=&v"(b[0][1]), "=&v"(b[0][2]), "=&v"(b[0][3]), "=&v"(b[1][0]), "=&v"(b[1][1]),
                       "=&v"(b[1][2]), "=&v"(b[1][3])
                     : "v"(ta[0]), "v"(ta[1]), "n"(kOff), "n"(kOff + 4 * kRow), "n"(kOff + 16 * kRow),
                       "n"(kOff + 20 * kRow)
                     : "memory");
    }
}

template <int JB>
__device__ __forceinline__ void grad_compute(const GradTile<JB>& t, int wave, int lane, int valid, f32x16 (&acc)[JB]) {
    const int g4 = lane >> 4;
    const int m = 8 * (g4 >> 1) + ((lane >> 2) & 3);
    const int col = 16 * (g4 & 1) + 4 * (lane & 3);                    // of a 32-wide block
    const int n = 32 * wave + col;
    const uint32_t pa = lds_addr(t.P) + m * 256 + ((((n >> 3) ^ swz(m)) << 4) | ((n & 7) << 1));
    uint32_t ta[JB];
#pragma unroll
    for (int jb = 0; jb < JB; ++jb) {
        const int j = 32 * jb + col;
        ta[jb] = lds_addr(t.T) + m * (64 * JB) + ((((j >> 3) ^ (JB == 2 ? swz(m) : 0)) << 4) | ((j & 7) << 1));
    }
    u64 a[4];
    asm volatile(QN_TR4(0, 1, 2, 3, 4, 5, 6, 7, 8) "s_waitcnt lgkmcnt(0)"
                 : "=&v"(a[0]), "=&v"(a[1]), "=&v"(a[2]), "=&v"(a[3])
                 : "v"(pa), "n"(0), "n"(4 * 256), "n"(16 * 256), "n"(20 * 256)
                 : "memory");
    const int mb = 8 * (lane >> 5);
    uint4 A[2] = {fragment(a[0], a[1]), fragment(a[2], a[3])};
    if (valid < kGK) {
        A[0] = masked(A[0], mb, valid);
        A[1] = masked(A[1], mb + 16, valid);
    }
    auto add = [&](const u64 (&b)[JB][4]) {
#pragma unroll
        for (int jb = 0; jb < JB; ++jb)
#pragma unroll
            for (int sub = 0; sub < 2; ++sub) {
                uint4 B = fragment(b[jb][2 * sub], b[jb][2 * sub + 1]);
                if (valid < kGK) B = masked(B, mb + 16 * sub, valid);
                acc[jb] = mfma32(A[sub], B, acc[jb]);
            }
    };
    u64 b[JB][4];
    read_term<JB, 0>(ta, b);
    add(b);
    read_term<JB, 1>(ta, b);
    add(b);
    read_term<JB, 2>(ta, b);
    add(b);
    static_assert(kTerms == 3, "three terms");
}
#undef QN_TR4
#undef QN_TR

// slot of the first slice of adapter a (of several), whose tokens begin at position `start`
__device__ __forceinline__ int first_slot(const GradArgs& g, int a, int start) {
    return min(2 * start / (g.per * kMultiItem), g.plan.first_item[a] / g.per + a);
}

constexpr int kZero = 4096;          // elements of dB_a, dA_a per workgroup that writes zeros

// zeros for an adapter without tokens: chunk c of its dB_a, then dA_a (sizes multiples of 1024)
__device__ __forceinline__ void zero_job(const GradArgs& g, int b) {
    const int a = b / g.zero_blocks;
    if (g.plan.start[a + 1] > g.plan.start[a]) return;
    const int64_t n0 = g.job[0].N * g.r, n1 = g.job[1].N * g.r;
    const int64_t at = static_cast<int64_t>(b % g.zero_blocks) * kZero + 4 * threadIdx.x;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int64_t i = at + 1024 * q;
        if (i >= n0 + n1) return;
        float* p = i < n0 ? g.job[0].out + a * n0 + i : g.job[1].out + a * n1 + (i - n0);
        *reinterpret_cast<float4*>(p) = float4{0.0f, 0.0f, 0.0f, 0.0f};
    }
}

template <int JB>   // 32-wide rank blocks per workgroup: 1 (r <= 32) or 2
__global__ __launch_bounds__(256)
void multi_grad_mfma(GradArgs g) {
    __shared__ GradTile<JB> s0, s1;
    __shared__ int s_order[kMaxPer * kMultiItem];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    int b = static_cast<int>(blockIdx.x);
    if (b >= g.zero_at) {
        zero_job(g, b - g.zero_at);
        return;
    }
    const int nb0 = g.job[0].tiles * g.max_items * g.jchunks;
    const bool second = b >= nb0;
    const GradJob jb = second ? g.job[1] : g.job[0];
    b -= second ? nb0 : 0;
    const int tile = b % jb.tiles;
    b /= jb.tiles;
    const int item = b % g.max_items;
    const int j0 = (b / g.max_items) * kGJ;
    const MultiItem it = g.plan.items[item];
    if (it.adapter < 0 || it.index % g.per != 0) return;
    const int m_lo = it.pos, m_hi = m_lo + min(g.per * kMultiItem, it.left);
    const bool alone = it.index == 0 && m_hi == m_lo + it.left;        // the adapter's only slice
    const int64_t n0 = static_cast<int64_t>(tile) * kGCols;
    const int steps = (m_hi - m_lo + kGK - 1) / kGK;
    const int64_t mr = static_cast<int64_t>(g.M) * g.r;

    f32x16 acc[JB];
#pragma unroll
    for (int k = 0; k < JB; ++k) acc[k] = f32x16{};

    // the slice's tokens, so that a step's loads wait for no index from memory
    for (int i = threadIdx.x; i < m_hi - m_lo; i += 256) s_order[i] = g.plan.order[m_lo + i];
    __syncthreads();
    // P: rows 4 (2 w + q) + lane / 16. T: JB = 2, row 8 w + lane / 8 of each term; JB = 1, the 6
    // half terms (16 rows each) dealt to the waves, the last two to two waves each (the same
    // bytes), so that every wave has as many loads in flight
    constexpr int kTLoads = JB == 2 ? kTerms : 2;
    auto issue = [&](GradTile<JB>& t, int m) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const int row = 4 * (2 * wave + q) + (lane >> 4);
            const int64_t tok = s_order[min(m + row, m_hi - 1) - m_lo];
            const int64_t ng = min(n0 + 8 * ((lane & 15) ^ swz(row)), jb.N - 8);
            load_lds16(jb.P + tok * jb.ldp + ng, &t.P[(2 * wave + q) * 64]);
        }
        if constexpr (JB == 2) {
            const int row = 8 * wave + (lane >> 3);
            const int64_t at = static_cast<int64_t>(min(m + row, m_hi - 1)) * g.r +
                               min(j0 + 8 * ((lane & 7) ^ swz(row)), g.r - 8);
#pragma unroll
            for (int p = 0; p < kTerms; ++p) load_lds16(jb.T + p * mr + at, &t.T[p][wave * 64]);
        } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int half = h == 0 ? wave : 4 + (wave & 1);       // half term
                const int p = half >> 1, row = 16 * (half & 1) + (lane >> 2);
                const int64_t at = static_cast<int64_t>(min(m + row, m_hi - 1)) * g.r + min(8 * (lane & 3), g.r - 8);
                load_lds16(jb.T + p * mr + at, &t.T[p][(half & 1) * 64]);
            }
        }
    };
#define QN_GRAD_BARRIER() asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory")
    constexpr int kLoads = 2 + kTLoads;
    auto compute = [&](const GradTile<JB>& t, int s) {
        grad_compute<JB>(t, wave, lane, min(kGK, m_hi - (m_lo + s * kGK)), acc);
    };
#define QN_GRAD(S, CUR, NXT)                                                                   \
    if ((S) + 1 < steps) { issue(NXT, m_lo + ((S) + 1) * kGK); QN_WAIT_VM(kLoads); }           \
    else QN_WAIT_VM(0);                                                                        \
    QN_GRAD_BARRIER();                                                                         \
    compute(CUR, S);                                                                           \
    QN_GRAD_BARRIER();
    issue(s0, m_lo);
    for (int s = 0; s < steps; s += 2) {
        QN_GRAD(s, s0, s1)
        if (s + 1 >= steps) break;
        QN_GRAD(s + 1, s1, s0)
    }
#undef QN_GRAD
#undef QN_GRAD_BARRIER
    // D of a 32 x 32 tile: lane l holds rows 8 (v / 4) + 4 (l / 32) + v % 4 of column l % 32
    const int64_t Nr = jb.N * g.r;
    float* dst = alone ? jb.out + it.adapter * Nr
                       : jb.part + (first_slot(g, it.adapter, it.pos - it.index * kMultiItem) + it.index / g.per) * Nr;
#pragma unroll
    for (int k = 0; k < JB; ++k) {
        const int j = j0 + 32 * k + (lane & 31);
        if (j >= g.r) continue;
#pragma unroll
        for (int v = 0; v < 16; v += 4) {
            const int64_t n = n0 + 32 * wave + 8 * (v >> 2) + 4 * (lane >> 5);
            if (n >= jb.N) continue;                                   // N % 64 == 0: 4 columns in or out together
            const float4 o = float4{acc[k][v], acc[k][v + 1], acc[k][v + 2], acc[k][v + 3]};
            if (alone && jb.rows) {
                *reinterpret_cast<float4*>(dst + j * jb.N + n) = o;
            } else {
                dst[n * g.r + j] = o.x;
                dst[(n + 1) * g.r + j] = o.y;
                dst[(n + 2) * g.r + j] = o.z;
                dst[(n + 3) * g.r + j] = o.w;
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
    const float* p = jb.part + (slices ? first_slot(g, a, lo) : 0) * Nr;
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

int jchunks_of(int r) { return (r + kGJ - 1) / kGJ; }

// Items per slice: about 512 workgroups over both gradients if the tokens were evenly spread,
// at most 1024 positions a slice. (256 of twice the length: 31 against 23 us on 4096 x 4096,
// 4096 tokens, r = 16, and 39 against 34 us on 11008 + 4096 columns, 2048 tokens, r = 64, whose
// partials then take 8 instead of 12 us; 1024 of half of it: 26 us for the partials there.)
// Up to 512 tokens one slice per adapter: a second launch costs 4.9 us, a step of 32 positions
// about 0.4 us (203 tokens of 3 adapters on 256 x 256 23.4 us against 24.7, 512 of 8 on 4096 x
// 4096 with r = 64 73.5 against 76.1; 512 of a single adapter on 1024 x 1024 45.5 against 41.1,
// but how the tokens are spread is not known on the host).
constexpr int64_t kOneSlice = 512;
int per_of(int64_t d_out, int64_t d_in, int64_t M, int r) {
    if (M <= kOneSlice) return static_cast<int>((M + kMultiItem - 1) / kMultiItem);
    const int64_t tiles = ((d_out + kGCols - 1) / kGCols + (d_in + kGCols - 1) / kGCols) * jchunks_of(r);
    const int64_t items = (M + kMultiItem - 1) / kMultiItem;
    return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kMaxPer, items * tiles / 512)));
}

}  // namespace

namespace {
int64_t slots_of(int64_t d_out, int64_t d_in, int64_t M, int n, int r) {
    const int64_t per = per_of(d_out, d_in, M, r);
    return std::min(2 * M / (per * kMultiItem), multi_max_items(M, n) / per + n);
}
}  // namespace

// (Up to 4 MB a slot is counted for every adapter of the pool, used or not: small pools keep the
// workspace they had when slots were numbered by adapter alone.)
int64_t multi_grads_part_floats(int64_t d_out, int64_t d_in, int64_t M, int n, int r) {
    if (M <= kOneSlice) return 0;
    const int64_t slot = (d_out + d_in) * r, kept = (int64_t{1} << 20) / slot;
    const int64_t of_pool = multi_max_items(M, n) / per_of(d_out, d_in, M, r) + n;
    return std::max(slots_of(d_out, d_in, M, n, r), std::min(of_pool, kept)) * slot;
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
    g.zero_at = (g.job[0].tiles + g.job[1].tiles) * g.max_items * g.jchunks;
    g.zero_blocks = static_cast<int>(((d_out + d_in) * r + kZero - 1) / kZero);
    const bool whole = M <= kOneSlice;
    const dim3 grid(static_cast<unsigned>(whole ? g.zero_at + n * g.zero_blocks : g.zero_at));
    if (r <= 32) QN_LAUNCH("multi_grad_mfma", st, multi_grad_mfma<1>, grid, dim3(256), 0, st, g);
    else QN_LAUNCH("multi_grad_mfma", st, multi_grad_mfma<2>, grid, dim3(256), 0, st, g);
    if (whole) return hipGetLastError();
    const int b0 = static_cast<int>(d_out / 64 * (r / 16)), b1 = static_cast<int>(d_in / 64 * (r / 16));
    QN_LAUNCH("multi_grad_reduce", st, multi_grad_reduce, dim3(static_cast<unsigned>(b0 + b1), static_cast<unsigned>(n)),
              dim3(256), 0, st, g, b0);
    return hipGetLastError();
}

}  // namespace qn
