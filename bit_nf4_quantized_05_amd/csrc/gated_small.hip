// The gated block on 1 to 64 tokens (decode batches) on gfx950: both weights' codes are streamed
// once and dequantised in registers straight into MFMA operands; no bf16 copy is made.
//
// gated_small_kernel: the rows of W_g, W_u, A_g and A_u one after the other as tiles of 16; a
// wave multiplies a tile with the tokens over its share of K (v_mfma_f32_16x16x32_bf16, the tile's
// rows against up to four 16-token tiles). Lane l (row l % 16, group l / 16) takes 16 code bytes =
// 32 weights of each 128, one 16-byte load, and forms bf16(code * a_hat) exactly as the dequantiser
// does. The tokens' slice of K stands in LDS, chunks XOR-swizzled by the token.
//   up to 16 tokens  the 8 waves of a workgroup share a tile, each an eighth of its K, and add
//                    their sums through LDS; workgroups walk over the tiles, the next tile's loads
//                    under the present one's work
//   17 to 64         a wave per tile, K in slices that fit the LDS (more tokens, shorter slices)
// gated_join_kernel: the slices' sums in order, the rank products, the activation and the product.
// Bound by the code stream and by the 2.9 VALU operations and one LDS lookup that a weight takes.
#include <hip/hip_runtime.h>

#include "gated.h"
#include "mfma_device.h"
#include "nf4_device.h"

#include <algorithm>

namespace qn {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kGroupPairs = 4;                  // 128-weight pieces of a row loaded at a time
constexpr int kXBytes = 64 * 1024;              // the tokens' slice in LDS (two workgroups per CU)

struct SmallArgs {
    const uint8_t* codes[2]; BlockConsts bc[2];
    const uint16_t* A[2];
    const uint16_t* X; int64_t ldx;
    int T, d_ff, d_in, r;
    int wtiles, tiles;                          // 16-row tiles of both weights, and of everything
    int splits, pairs;                          // slices of K, 128-wide pieces per slice
    float* part;                                // [splits][T][16 tiles]
};

__device__ __forceinline__ f32x4 mfma16(const uint4& a, const uint4& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// The loads of up to kGroupPairs pieces of a tile's rows: code words and block constants
struct Codes {
    uint4 w[kGroupPairs];
    int8_t q[kGroupPairs];
    float s[kGroupPairs];
};

// KW waves share a tile (8 or 1); TT 16-token tiles
template <int TT, int KW>
__global__ __launch_bounds__(kThreads, 4)
void gated_small_kernel(SmallArgs a, NF4Tables tab) {
    static_assert(KW == 1 || (KW == kWaves && TT == 1), "shared tiles have 16 tokens at most");
    __shared__ uint4 xs[kXBytes / 16];          // [token][chunk of 8]
    __shared__ float s_code[16 * 64];           // code book, a copy per lane
    __shared__ float s_q[256];                  // second-level steps
    __shared__ float red[KW == 1 ? 1 : 2][KW == 1 ? 1 : kWaves][256];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int kw = KW == 1 ? 0 : wave;
    const int nb = a.d_in / 64, npair = (nb + 1) / 2;
    const int split = static_cast<int>(blockIdx.y);
    const int p0 = split * a.pairs, np = min(a.pairs, npair - p0);     // the slice's pieces
    const int groups = (np + KW * kGroupPairs - 1) / (KW * kGroupPairs);
    const int chunks = a.pairs * 16;                                   // LDS chunks per token
    const int step = static_cast<int>(gridDim.x) * (kWaves / KW);
    int tile = static_cast<int>(blockIdx.x) * (kWaves / KW) + (KW == 1 ? wave : 0);

    auto load = [&](Codes& c, int tile, int group) {
        const int w = tile * 16 >= a.d_ff ? 1 : 0;
        const int64_t row = tile * 16 - w * a.d_ff + i;
        const uint4* codes = reinterpret_cast<const uint4*>(a.codes[w]) + row * (a.d_in / 32);
        const BlockConsts& bc = a.bc[w];
#pragma unroll
        for (int k = 0; k < kGroupPairs; ++k) {
            const int p = p0 + min((group * kGroupPairs + k) * KW + kw, np - 1);
            const int64_t blk = row * nb + min(2 * p + (g >> 1), nb - 1);
            c.w[k] = codes[min(4 * p + g, a.d_in / 32 - 1)];
            c.q[k] = bc.q[blk];
            c.s[k] = bc.scale[blk >> bc.gshift];
        }
    };

    // the tokens' slice first (the codes' loads would be ahead of it in the queue), then the first
    // tile's codes, then the tables
    {
        const int rows = a.T, per = np * 16;
        for (int e = tid; e < rows * per; e += kThreads) {
            const int t = e / per, c = e - t * per;
            const int col = (p0 * 16 + c) * 8;
            uint4 v = uint4{0, 0, 0, 0};
            if (col < a.d_in) v = *reinterpret_cast<const uint4*>(a.X + t * a.ldx + col);
            xs[t * chunks + (c ^ (t & 15))] = v;
        }
    }
    for (int e = tid; e < 16 * 64; e += kThreads) {
        float v = tab.code[0];
#pragma unroll
        for (int q = 1; q < 16; ++q) v = (e >> 6) == q ? tab.code[q] : v;
        s_code[e] = v;
    }
    if (tid < 256) s_q[tid] = dq_step(a.bc[0].fmt, static_cast<int8_t>(tid - 128));
    Codes cur, nxt;
    if (tile < a.wtiles) load(cur, tile, 0);
    __syncthreads();

    const float mu[2] = {a.bc[0].mean[0], a.bc[1].mean[0]};
    const char* code_lds = reinterpret_cast<const char*>(s_code);
    const uint32_t lane4 = static_cast<uint32_t>(lane) << 2;
    int xrow[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) xrow[t] = min(16 * t + i, a.T - 1);
    f32x4 acc[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    auto multiply = [&](const uint4& frag, int p, int st) {            // p: the slice's piece
#pragma unroll
        for (int t = 0; t < TT; ++t)
            acc[t] = mfma16(frag, xs[xrow[t] * chunks + ((16 * p + 4 * g + st) ^ (xrow[t] & 15))], acc[t]);
    };
    int parity = 0;
    auto finish = [&](int tile) {
        float* out = a.part + (static_cast<int64_t>(split) * a.T) * (16 * a.tiles) + 16 * tile;
        if constexpr (KW == 1) {
            // D of a 16 x 16 tile: lane l holds rows 4 (l / 16) .. + 3 of token l % 16
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                if (16 * t + i < a.T)
                    *reinterpret_cast<f32x4*>(out + static_cast<int64_t>(16 * t + i) * (16 * a.tiles) + 4 * g) = acc[t];
                acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            }
        } else {
            *reinterpret_cast<f32x4*>(&red[parity][wave][4 * lane]) = acc[0];
            acc[0] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            __syncthreads();
            if (tid < 256) {
                float v = 0.0f;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) v += red[parity][w][tid];
                const int t = (tid >> 2) & 15, row = 4 * (tid >> 6) + (tid & 3);
                if (t < a.T) out[static_cast<int64_t>(t) * (16 * a.tiles) + row] = v;
            }
            parity ^= 1;                         // the next tile's sums beside these: one barrier a tile
        }
    };

    for (; tile < a.tiles; tile += step) {
        if (tile < a.wtiles) {
            const int w = tile * 16 >= a.d_ff ? 1 : 0;
            for (int grp = 0; grp < groups; ++grp) {
                // the next group's loads, or the next tile's
                const bool more = grp + 1 < groups;
                const int nt = more ? tile : tile + step;
                if (nt < a.wtiles) load(nxt, nt, more ? grp + 1 : 0);
#pragma unroll
                for (int k = 0; k < kGroupPairs; ++k) {
                    const int p = (grp * kGroupPairs + k) * KW + kw;
                    if (p >= np) break;                                // uniform
                    const int bl = 2 * (p0 + p) + (g >> 1);
                    const float rel = s_q[static_cast<int>(cur.q[k]) + 128];
                    const float prod = cur.s[k] * rel;                 // a_hat = mu + b r, each step rounded
                    const float full = a.bc[0].fmt == kDqNone ? cur.s[k] : mu[w] + prod;
                    const float ah = bl < nb ? full : 0.0f;
                    const uint32_t words[4] = {cur.w[k].x, cur.w[k].y, cur.w[k].z, cur.w[k].w};
#pragma unroll
                    for (int st = 0; st < 4; ++st) {
                        // code c's value, the lane's copy, at byte c << 8 | lane << 2: one v_perm_b32
                        const uint32_t nib[2] = {words[st] & 0x0F0F0F0Fu, (words[st] >> 4) & 0x0F0F0F0Fu};
                        float v[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            v[e] = *reinterpret_cast<const float*>(
                                       code_lds + __builtin_amdgcn_perm(lane4, nib[e & 1], 0x0C0C0004u | ((e >> 1) << 8))) *
                                   ah;
                        multiply(uint4{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                       pack_bf16x2(v[6], v[7])},
                                 p, st);
                    }
                }
                cur = nxt;
            }
        } else {
            // 16 rows of A (past r: the last one again, not read)
            const int at = tile - a.wtiles, per = (a.r + 15) / 16;
            const int w = at >= per ? 1 : 0;
            const uint16_t* row = a.A[w] + static_cast<int64_t>(min((at - w * per) * 16 + i, a.r - 1)) * a.d_in;
            for (int p = kw; p < np; p += KW) {
                const int col = (p0 + p) * 128 + 32 * g;
                const bool ok = col < a.d_in;
                uint4 v[4];
#pragma unroll
                for (int st = 0; st < 4; ++st) v[st] = *reinterpret_cast<const uint4*>(row + min(col, a.d_in - 32) + 8 * st);
#pragma unroll
                for (int st = 0; st < 4; ++st) multiply(ok ? v[st] : uint4{0, 0, 0, 0}, p, st);
            }
        }
        finish(tile);
    }
}

// H (and GU) of 64 outputs for all tokens: the slices' sums in order, G += s_g sum_j T_g[j] B_g[., j]
// with T = the A tiles' sums, in float32, U likewise.
struct JoinArgs {
    const float* part; int splits, T, d_ff, r, wtiles, tiles;
    const uint16_t* B[2]; float s[2];
    int act;
    uint16_t* H; int64_t ldh;
    uint16_t* GU; int64_t ldgu;
};
constexpr int kJoinRows = 64, kJoinRanks = 32;

template <int PT>       // tokens per thread (a quarter of the tokens, rounded up)
__global__ __launch_bounds__(256)
void gated_join_kernel(JoinArgs a) {
    __shared__ float s_b[2][kJoinRows][kJoinRanks + 1];
    __shared__ float s_t[2][64][kJoinRanks];
    const int n0 = static_cast<int>(blockIdx.x) * kJoinRows;
    const int i = threadIdx.x & 63, q = threadIdx.x >> 6;
    const int64_t pitch = 16 * a.tiles, slice = pitch * a.T;
    const int rp = (a.r + 15) / 16 * 16;
    float v[2][PT];
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int k = 0; k < PT; ++k)
            v[w][k] = ordered_sum<4>(a.part + min(q + 4 * k, a.T - 1) * pitch + w * a.d_ff + n0 + i, slice, a.splits);
    for (int j0 = 0; j0 < a.r; j0 += kJoinRanks) {
        const int nj = min(kJoinRanks, a.r - j0);
        __syncthreads();
        for (int e = threadIdx.x; e < 2 * kJoinRows * nj; e += 256) {
            const int w = e / (kJoinRows * nj), row = e / nj % kJoinRows, j = e % nj;
            s_b[w][row][j] = __uint_as_float(static_cast<uint32_t>(a.B[w][static_cast<int64_t>(n0 + row) * a.r + j0 + j]) << 16);
        }
        for (int e = threadIdx.x; e < 2 * a.T * nj; e += 256) {
            const int w = e / (a.T * nj), t = e / nj % a.T, j = e % nj;
            s_t[w][t][j] = a.s[w] * ordered_sum<4>(a.part + t * pitch + 16 * a.wtiles + w * rp + j0 + j, slice, a.splits);
        }
        __syncthreads();
#pragma unroll
        for (int w = 0; w < 2; ++w)
            for (int j = 0; j < nj; ++j) {
                const float b = s_b[w][i][j];
#pragma unroll
                for (int k = 0; k < PT; ++k) v[w][k] += s_t[w][min(q + 4 * k, a.T - 1)][j] * b;
            }
    }
#pragma unroll
    for (int k = 0; k < PT; ++k) {
        const int64_t t = q + 4 * k;
        if (t >= a.T) break;
        a.H[t * a.ldh + n0 + i] = bf16_bits(gated_act(a.act, v[0][k]) * v[1][k]);
        if (a.GU != nullptr) {
            a.GU[t * a.ldgu + n0 + i] = bf16_bits(v[0][k]);
            a.GU[t * a.ldgu + a.d_ff + n0 + i] = bf16_bits(v[1][k]);
        }
    }
}

// Slices of K: as few as fit the LDS with T tokens
struct SmallPlan { int splits, pairs, wtiles, tiles; };
SmallPlan small_plan(int64_t M, int64_t d_ff, int64_t d_in, int r) {
    const int npair = static_cast<int>((d_in / 64 + 1) / 2);
    const int most = static_cast<int>(kXBytes / (256 * M));
    SmallPlan s;
    s.splits = (npair + most - 1) / most;
    s.pairs = (npair + s.splits - 1) / s.splits;
    s.splits = (npair + s.pairs - 1) / s.pairs;
    s.wtiles = static_cast<int>(2 * d_ff / 16);
    s.tiles = s.wtiles + 2 * ((r + 15) / 16);
    return s;
}

}  // namespace

int64_t gated_small_part_floats(int64_t M, int64_t d_ff, int64_t d_in, int r) {
    const SmallPlan s = small_plan(M, d_ff, d_in, r);
    return static_cast<int64_t>(s.splits) * M * 16 * s.tiles;
}

hipError_t launch_gated_small(const GatedCall& c, const uint16_t* X, int64_t ldx, uint16_t* H, int64_t ldh, uint16_t* GU,
                              int64_t ldgu, float* part, hipStream_t st) {
    const SmallPlan s = small_plan(c.M, c.d_ff, c.d_in, c.r);
    SmallArgs a{};
    JoinArgs j{};
    for (int w = 0; w < 2; ++w) {
        a.codes[w] = c.codes[w]; a.bc[w] = c.bc[w]; a.A[w] = c.A[w];
        j.B[w] = c.B[w]; j.s[w] = c.s[w];
    }
    a.X = X; a.ldx = ldx;
    a.T = static_cast<int>(c.M); a.d_ff = static_cast<int>(c.d_ff); a.d_in = static_cast<int>(c.d_in); a.r = c.r;
    a.wtiles = s.wtiles; a.tiles = s.tiles; a.splits = s.splits; a.pairs = s.pairs; a.part = part;
    const NF4Tables& tab = tables();
    if (c.M <= 16) {
        const dim3 grid(static_cast<unsigned>(std::max(1, std::min(s.tiles, 512 / s.splits))), static_cast<unsigned>(s.splits));
        QN_LAUNCH("gated_small_kernel", st, (gated_small_kernel<1, kWaves>), grid, dim3(kThreads), 0, st, a, tab);
    } else {
        const dim3 grid(static_cast<unsigned>((s.tiles + kWaves - 1) / kWaves), static_cast<unsigned>(s.splits));
        if (c.M <= 32) QN_LAUNCH("gated_small_kernel", st, (gated_small_kernel<2, 1>), grid, dim3(kThreads), 0, st, a, tab);
        else if (c.M <= 48) QN_LAUNCH("gated_small_kernel", st, (gated_small_kernel<3, 1>), grid, dim3(kThreads), 0, st, a, tab);
        else QN_LAUNCH("gated_small_kernel", st, (gated_small_kernel<4, 1>), grid, dim3(kThreads), 0, st, a, tab);
    }
    j.part = part; j.splits = s.splits; j.T = a.T; j.d_ff = a.d_ff; j.r = c.r; j.wtiles = s.wtiles; j.tiles = s.tiles;
    j.act = c.act; j.H = H; j.ldh = ldh; j.GU = GU; j.ldgu = ldgu;
    const dim3 jgrid(static_cast<unsigned>(c.d_ff / kJoinRows));
    if (c.M <= 4) QN_LAUNCH("gated_join_kernel", st, gated_join_kernel<1>, jgrid, dim3(256), 0, st, j);
    else if (c.M <= 16) QN_LAUNCH("gated_join_kernel", st, gated_join_kernel<4>, jgrid, dim3(256), 0, st, j);
    else QN_LAUNCH("gated_join_kernel", st, gated_join_kernel<16>, jgrid, dim3(256), 0, st, j);
    return hipGetLastError();
}

}  // namespace qn
