// The gated block on 1 to 64 tokens (decode batches) on gfx950: both weights' codes are streamed
// once and dequantised in registers straight into MFMA operands; no bf16 copy is made.
//
// gated_small_kernel: the rows of A_g, A_u, W_g and W_u one after the other as tiles of 16; a
// wave multiplies a tile with the tokens over its share of K (v_mfma_f32_16x16x32_bf16, the tile's
// rows against up to four 16-token tiles). Lane l (row l % 16, group l / 16) takes 16 code bytes =
// 32 weights of each 128, one 16-byte load, and forms bf16(code * a_hat) exactly as the dequantiser
// does, a byte of codes per lookup (2 VALU operations per weight; a nibble at a time 2.9). A
// workgroup per CU has a slice of K, the tokens' part of it in LDS (chunks XOR-swizzled by the
// token), and walks over tiles, the next tile's loads under the present one's work; its 16 waves
// share a tile (up to 16 tokens), take one in twos (up to 32) or one each.
// gated_join_kernel: the slices' sums in order, the rank products, the activation and the product.
// 24 tokens of 11008 x 4096: 24 us, bound by LDS (a lookup per code byte and the tokens' values), and 6.6.
// gated_few_kernel: up to 16 tokens on rows of up to 4096, without the join (below).
#include <hip/hip_runtime.h>

#include "gated.h"
#include "mfma_device.h"
#include "nf4_device.h"

#include <algorithm>

namespace qn {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 16, kThreads = 64 * kWaves;
constexpr int kGroupPairs = 4;                  // 128-weight pieces of a row loaded at a time

// A barrier for LDS writes that leaves loads in flight
#define QN_LDS_BARRIER() asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory")

struct SmallArgs {
    const uint8_t* codes[2]; BlockConsts bc[2];
    uint32_t code_bytes, q_bytes, s_bytes;      // extents
    const uint16_t* A[2];
    const uint16_t* X; int64_t ldx;
    int T, d_ff, d_in, r;
    int atiles, tiles;                          // 16-row tiles of both A (first), and of everything
    int splits, pairs;                          // slices of K, 128-wide pieces per slice
    float* part;                                // [splits][T][16 tiles]
};

__device__ __forceinline__ f32x4 mfma16(const uint4& a, const uint4& b, const f32x4& c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t small_rsrc(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), static_cast<short>(0), static_cast<int>(bytes), 0x00020000);
}

// 32 weights of a row: their codes, their block's 8-bit constant and its scale
struct Piece {
    uint4 w;
    int8_t q;
    float s;
};

// One weight's descriptors; without extent (nothing is fetched, the number of loads in flight stays
// the same) where there is nothing to load
struct PieceSource {
    __amdgpu_buffer_rsrc_t codes, q, s;
};
template <class Args>
__device__ __forceinline__ PieceSource piece_source(const Args& a, int w, bool live) {
    return PieceSource{small_rsrc(a.codes[w], live ? a.code_bytes : 0u), small_rsrc(a.bc[w].q, live ? a.q_bytes : 0u),
                       small_rsrc(a.bc[w].scale, live ? a.s_bytes : 0u)};
}
__device__ __forceinline__ void load_piece(Piece& c, const PieceSource& src, uint32_t row, int d_in, int gshift, int word,
                                           int block) {
    typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
    const uint32_t blk = row * (d_in / 64) + block;
    const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(src.codes, row * (d_in / 2) + 16 * word, 0, 0);
    c.w = uint4{v.x, v.y, v.z, v.w};
    c.q = static_cast<int8_t>(__builtin_amdgcn_raw_buffer_load_b8(src.q, blk, 0, 0));
    c.s = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(src.s, 4 * (blk >> gshift), 0, 0));
}

// byte -> the float32 values of its two codes, 32 copies (lanes l and l + 32 share one: 32 lanes of 8
// bytes fill all banks); and the second level's steps
struct CodeTables {
    uint4 pairs[256 * 16];
    float q[256];
};
__device__ __forceinline__ void build_tables(CodeTables& t, const NF4Tables& tab, int fmt) {
    // thread n: byte n / 4, copies 8 (n % 4) .. + 7
    const int n = threadIdx.x, byte = n >> 2;
    float lo = tab.code[0], hi = tab.code[0];
#pragma unroll
    for (int q = 1; q < 16; ++q) {
        lo = (byte & 15) == q ? tab.code[q] : lo;
        hi = (byte >> 4) == q ? tab.code[q] : hi;
    }
    const uint4 v = uint4{__float_as_uint(lo), __float_as_uint(hi), __float_as_uint(lo), __float_as_uint(hi)};
#pragma unroll
    for (int c = 0; c < 4; ++c) t.pairs[byte * 16 + (n & 3) * 4 + c] = v;
    // a_hat = mu + b r; without a second level the constant itself, 0 + b 1
    if (n < 256) t.q[n] = fmt == kDqNone ? 1.0f : dq_step(fmt, static_cast<int8_t>(n - 128));
}

// A piece's weights bf16(code * a_hat), 8 of them: MFMA operand `st` of its four. Byte e's pair, the
// lane's copy, stands at byte << 8 | (lane % 32) << 3: one v_perm_b32.
__device__ __forceinline__ float piece_constant(const Piece& c, const CodeTables& t, float mu, uint32_t keep) {
    const float prod = c.s * t.q[static_cast<int>(c.q) + 128];         // each step rounded
    return __uint_as_float(__float_as_uint(mu + prod) & keep);
}
__device__ __forceinline__ uint4 piece_weights(const Piece& c, int st, float a_hat, const CodeTables& t, uint32_t lane8) {
    const uint32_t words[4] = {c.w.x, c.w.y, c.w.z, c.w.w};
    uint32_t v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const float2 f = *reinterpret_cast<const float2*>(reinterpret_cast<const char*>(t.pairs) +
                                                          __builtin_amdgcn_perm(lane8, words[st], 0x0C0C0004u | (e << 8)));
        v[e] = bf16_pair(f.x * a_hat, f.y * a_hat);
    }
    return uint4{v[0], v[1], v[2], v[3]};
}

// KW of a workgroup's 16 waves share a tile (each a part of its K), TT 16-token tiles
template <int TT, int KW>
struct SmallLds {
    // bytes for the tokens' slice beside the tables and the sums that the waves of a tile hand on
    static constexpr int kX = (KW == 16 ? 78 : KW == 4 ? 70 : KW == 2 ? 60 : 92) * 1024;
    CodeTables tables;                          // first: their offsets fit an LDS read's 16 bits
    float red[KW == 1 || KW == 16 ? 1 : 2][KW == 1 ? 1 : KW == 16 ? 16 : kWaves - kWaves / KW][KW == 1 ? 1 : TT * 256];
    uint4 x[kX / 16];                           // [token][chunk of 8], chunks XORed with the token
};

template <int TT, int KW>
__global__ __launch_bounds__(kThreads, 4)
void gated_small_kernel(SmallArgs a, NF4Tables tab) {
    constexpr int kTiles = kWaves / KW;
    __shared__ SmallLds<TT, KW> lds;
    static_assert(sizeof(lds) <= 160 * 1024, "a CU's LDS");
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int kw = wave % KW, tl = wave / KW;
    const int nb = a.d_in / 64, npair = (nb + 1) / 2;
    const int split = static_cast<int>(blockIdx.y);
    const int p0 = split * a.pairs, np = min(a.pairs, npair - p0);     // the slice's pieces
    const int groups = (np + KW * kGroupPairs - 1) / (KW * kGroupPairs);
    const int chunks = a.pairs * 16;                                   // LDS chunks per token
    const int step = static_cast<int>(gridDim.x) * kTiles;
    // the k-th piece of the wave's group: neighbouring pieces in twos, which are a 128-byte line of codes
    auto piece_at = [&](int group, int k) { return ((group * (kGroupPairs / 2) + (k >> 1)) * KW + kw) * 2 + (k & 1); };
    auto load = [&](Piece (&c)[kGroupPairs], int tile, int group) {
        const bool live = tile >= a.atiles && tile < a.tiles;
        const int at = live ? (tile - a.atiles) * 16 : 0, w = at >= a.d_ff ? 1 : 0;
        const uint32_t row = static_cast<uint32_t>(at - w * a.d_ff) + i;
        const PieceSource src = piece_source(a, w, live);
#pragma unroll
        for (int k = 0; k < kGroupPairs; ++k) {
            const int p = p0 + min(piece_at(group, k), np - 1);
            load_piece(c[k], src, row, a.d_in, a.bc[0].gshift, min(4 * p + g, a.d_in / 32 - 1), min(2 * p + (g >> 1), nb - 1));
        }
    };

    // the tokens' slice (before the codes' loads, which it would queue behind)
    for (int e = tid, per = np * 16; e < a.T * per; e += kThreads) {
        const int t = e / per, c = e - t * per;
        const int col = (p0 * 16 + c) * 8;
        uint4 v = uint4{0, 0, 0, 0};
        if (col < a.d_in) v = *reinterpret_cast<const uint4*>(a.X + t * a.ldx + col);
        lds.x[t * chunks + (c ^ (t & 15))] = v;
    }
    // every workgroup's waves make the same number of rounds (they meet at barriers)
    int base = static_cast<int>(blockIdx.x) * kTiles;
    Piece cur[kGroupPairs], nxt[kGroupPairs];
    load(cur, base + tl, 0);
    build_tables(lds.tables, tab, a.bc[0].fmt);
    const bool plain = a.bc[0].fmt == kDqNone;
    const float mu[2] = {plain ? 0.0f : a.bc[0].mean[0], plain ? 0.0f : a.bc[1].mean[0]};
    QN_LDS_BARRIER();

    const uint32_t lane8 = static_cast<uint32_t>(lane & 31) << 3;
    int xrow[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) xrow[t] = min(16 * t + i, a.T - 1);
    f32x4 acc[TT];
    auto multiply = [&](const uint4& frag, int p, int st) {            // p: the slice's piece
#pragma unroll
        for (int t = 0; t < TT; ++t)
            acc[t] = mfma16(frag, lds.x[xrow[t] * chunks + ((16 * p + 4 * g + st) ^ (xrow[t] & 15))], acc[t]);
    };
    // D of a 16 x 16 tile: lane l holds rows 4 (l / 16) .. + 3 of token l % 16
    auto store = [&](int tile) {
        float* out = a.part + static_cast<int64_t>(split) * a.T * (16 * a.tiles) + 16 * tile;
#pragma unroll
        for (int t = 0; t < TT; ++t)
            if (16 * t + i < a.T) *reinterpret_cast<f32x4*>(out + static_cast<int64_t>(16 * t + i) * (16 * a.tiles) + 4 * g) = acc[t];
    };
    int parity = 0;
    for (; base < a.tiles; base += step) {
        const int tile = base + tl;
#pragma unroll
        for (int t = 0; t < TT; ++t) acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (tile < a.atiles) {
            // 16 rows of A (past r: the last one again, not read), two pieces' loads at a time
            const int per = a.atiles / 2, w = tile >= per ? 1 : 0;
            const uint16_t* row = a.A[w] + static_cast<int64_t>(min((tile - w * per) * 16 + i, a.r - 1)) * a.d_in;
            for (int p = kw; p < np; p += 2 * KW) {
                uint4 v[2][4];
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int st = 0; st < 4; ++st) {
                        const int col = (p0 + min(p + k * KW, np - 1)) * 128 + 32 * g;
                        v[k][st] = *reinterpret_cast<const uint4*>(row + min(col, a.d_in - 32) + 8 * st);
                    }
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int at = min(p + k * KW, np - 1);
                    const uint32_t keep = p + k * KW < np && (p0 + at) * 128 + 32 * g < a.d_in ? ~0u : 0u;
#pragma unroll
                    for (int st = 0; st < 4; ++st)
                        multiply(uint4{v[k][st].x & keep, v[k][st].y & keep, v[k][st].z & keep, v[k][st].w & keep}, at, st);
                }
            }
            load(cur, tile + step, 0);
        } else if (tile < a.tiles) {
            const float m = mu[(tile - a.atiles) * 16 >= a.d_ff ? 1 : 0];
            for (int grp = 0; grp < groups; ++grp) {
                // the next group's loads, or the next tile's
                const bool more = grp + 1 < groups;
                load(nxt, more ? tile : tile + step, more ? grp + 1 : 0);
#pragma unroll
                for (int k2 = 0; k2 < kGroupPairs; k2 += 2) {
                    if (piece_at(grp, k2) >= np) break;                // uniform
#pragma unroll
                    for (int k = k2; k < k2 + 2; ++k) {
                        // past the slice: the last piece again, times zero
                        const int at = piece_at(grp, k), p = min(at, np - 1);
                        const uint32_t keep = at < np && 2 * (p0 + p) + (g >> 1) < nb ? ~0u : 0u;
                        const float ah = piece_constant(cur[k], lds.tables, m, keep);
#pragma unroll
                        for (int st = 0; st < 4; ++st) multiply(piece_weights(cur[k], st, ah, lds.tables, lane8), p, st);
                    }
                }
#pragma unroll
                for (int k = 0; k < kGroupPairs; ++k) cur[k] = nxt[k];
            }
        }
        if constexpr (KW == 1) {
            if (tile < a.tiles) store(tile);
        } else if constexpr (KW < 16) {
            // the others' sums to the tile's first wave; the next tile's beside these: one barrier a tile
            auto slot = [&](int k, int t) { return reinterpret_cast<f32x4*>(&lds.red[parity][tl * (KW - 1) + k - 1][256 * t + 4 * lane]); };
            if (kw > 0) {
#pragma unroll
                for (int t = 0; t < TT; ++t) *slot(kw, t) = acc[t];
            }
            QN_LDS_BARRIER();
            if (kw == 0 && tile < a.tiles) {
#pragma unroll
                for (int k = 1; k < KW; ++k)
#pragma unroll
                    for (int t = 0; t < TT; ++t) acc[t] = acc[t] + *slot(k, t);
                store(tile);
            }
            parity ^= 1;
        } else {
            static_assert(TT == 1, "16 waves a tile: one token tile");
            *reinterpret_cast<f32x4*>(&lds.red[0][wave][4 * lane]) = acc[0];
            QN_LDS_BARRIER();
            if (tid < 256) {
                float v = 0.0f;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) v += lds.red[0][w][tid];
                const int t = (tid >> 2) & 15, row = 4 * (tid >> 6) + (tid & 3);
                if (t < a.T)
                    a.part[(static_cast<int64_t>(split) * a.T + t) * (16 * a.tiles) + 16 * tile + row] = v;
            }
            QN_LDS_BARRIER();
        }
    }
}

// ---------------------------------------------------------------------------
// Up to 16 tokens, rows of up to 4096: a workgroup per CU, 16 waves, walks over items of 16
// outputs; a wave has two of a row's 32 pieces of 128 weights, of the gate row and of the up row
// (four code loads per lane and item, the next item's under the present one's work), and the
// tokens' values of its pieces in registers for the whole walk. A code byte is looked up as a pair
// of float32 code values (64 KB of LDS, 32 copies), 2 VALU operations per weight in place of 2.9.
// s A x stands as two bf16 terms; of each item the waves in turn add B (s A x) by MFMAs with 16
// ranks, both terms, as K. The terms of up to 16 ranks and 4 tokens are formed by every workgroup at
// its start, a wave per rank of each projection (rows of A read whole, 1 KB an instruction: read as
// MFMA operands, 64 bytes of 16 rows, they took 10 us); otherwise by gated_ax_kernel before. The 16
// waves' sums meet in LDS, one barrier an item, four of the waves in turn finish it. One token of 11008 x
// 4096: 20 us, of which reading the 45 MB of codes at a copy's rate would take 9.
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 16, kFewTokens = 16, kFewIn = 4096, kFewOwn = 4;

// s A x: [projection][16 ranks][16 tokens][16 ranks' bf16 | what bf16 left of them, bf16]
typedef uint4 FewRanks[kFewTokens][4];

struct FewArgs {
    const uint8_t* codes[2]; BlockConsts bc[2];
    uint32_t code_bytes, q_bytes, s_bytes;      // extents
    const uint16_t* A[2]; const uint16_t* B[2]; float s[2];
    const uint16_t* X; int64_t ldx;
    int T, d_ff, d_in, r, act;
    FewRanks* t;
    uint16_t* H; int64_t ldh;
    uint16_t* GU; int64_t ldgu;
};

// Of the wave's two pieces of a row: which, and where its lane's 32 values and their block are. Past
// the row: the last piece again, times zero.
struct FewPlace {
    int piece[2], block[2];
    uint32_t in[2];                             // all bits, or none past the row
};
__device__ __forceinline__ FewPlace few_place(int d_in, int wave, int g) {
    FewPlace p;
    const int nb = d_in / 64, last = (nb + 1) / 2 - 1;
#pragma unroll
    for (int k = 0; k < 2; ++k) {               // pieces 2 wave, 2 wave + 1: a 128-byte line of codes
        p.piece[k] = min(2 * wave + k, last);
        p.block[k] = min(2 * p.piece[k] + (g >> 1), nb - 1);
        p.in[k] = 2 * wave + k <= last && 2 * p.piece[k] + (g >> 1) < nb ? ~0u : 0u;
    }
    return p;
}

// The lane's 64 values of a row of X (or A)
__device__ __forceinline__ void few_row(const uint16_t* row, const FewPlace& p, int d_in, int g, uint4 (&x)[2][4]) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int st = 0; st < 4; ++st)
            x[k][st] = *reinterpret_cast<const uint4*>(row + min(128 * p.piece[k] + 32 * g + 8 * st, d_in - 8));
}

// v at a rank of a token's terms (an infinity or NaN: in the first alone)
__device__ __forceinline__ void put_terms(uint4 (&t)[4], int rank, float v) {
    uint16_t* out = reinterpret_cast<uint16_t*>(t);
    const float head = bf16_to_f32(bf16_bits(v));
    out[rank] = bf16_bits(v);
    out[16 + rank] = fabsf(head) < __builtin_inff() ? bf16_bits(v - head) : uint16_t{0};
}

// 16 ranks of one projection per workgroup
__global__ __launch_bounds__(64 * kFewWaves)
void gated_ax_kernel(FewArgs a) {
    __shared__ float red[kFewWaves][256];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int chunks = (a.r + 15) / 16;
    const int w = static_cast<int>(blockIdx.x) >= chunks ? 1 : 0, j0 = (static_cast<int>(blockIdx.x) - w * chunks) * 16;
    const FewPlace p = few_place(a.d_in, wave, g);
    uint4 x[2][4], v[2][4];
    few_row(a.A[w] + static_cast<int64_t>(min(j0 + i, a.r - 1)) * a.d_in, p, a.d_in, g, v);
    few_row(a.X + min(i, a.T - 1) * a.ldx, p, a.d_in, g, x);
    f32x4 t = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int st = 0; st < 4; ++st)
            t = mfma16(uint4{v[k][st].x & p.in[k], v[k][st].y & p.in[k], v[k][st].z & p.in[k], v[k][st].w & p.in[k]}, x[k][st], t);
    *reinterpret_cast<f32x4*>(&red[wave][4 * lane]) = t;
    __syncthreads();
    if (tid >= 256) return;
    float sum = 0.0f;
#pragma unroll
    for (int k = 0; k < kFewWaves; ++k) sum += red[k][tid];
    const int token = (tid >> 2) & 15, rank = 4 * (tid >> 6) + (tid & 3);
    put_terms(a.t[blockIdx.x][token], rank, j0 + rank < a.r ? a.s[w] * sum : 0.0f);
}

struct FewLds {
    CodeTables tables;
    FewRanks t[2];                              // own terms
    float red[2][kFewWaves][2][256];
};

// kOwn: the terms of s A x formed here (r <= 16, up to kFewOwn tokens)
template <bool kOwn>
__global__ __launch_bounds__(64 * kFewWaves, 4)
void gated_few_kernel(FewArgs a, NF4Tables tab) {
    __shared__ FewLds lds;
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int i = lane & 15, g = lane >> 4;
    const int items = a.d_ff / 16;
    const FewPlace p = few_place(a.d_in, wave, g);
    // of an item: gate pieces 0, 1, up pieces 0, 1
    auto load = [&](Piece (&c)[4], int item) {
        const bool live = item < items;
        const uint32_t row = static_cast<uint32_t>(live ? item : 0) * 16 + i;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const PieceSource src = piece_source(a, w, live);
#pragma unroll
            for (int k = 0; k < 2; ++k)
                load_piece(c[2 * w + k], src, row, a.d_in, a.bc[0].gshift, min(4 * p.piece[k] + g, a.d_in / 32 - 1), p.block[k]);
        }
    };
    int item = static_cast<int>(blockIdx.x);
    Piece cur[4], nxt[4];
    if constexpr (kOwn) {
        // row `wave` of A_g and of A_u times every token, lane l the 16-byte chunks l + 64 e (before the
        // codes: behind them one token took 26.7 us in place of 26.1, four 37.8 in place of 28.7)
        const int nch = a.d_in / 8;
        uint4 av[2][8];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const uint4* row = reinterpret_cast<const uint4*>(a.A[w] + static_cast<int64_t>(min(wave, a.r - 1)) * a.d_in);
#pragma unroll
            for (int e = 0; e < 8; ++e) av[w][e] = row[min(lane + 64 * e, nch - 1)];
        }
        for (int k = 0; k < a.T; ++k) {
            const uint4* row = reinterpret_cast<const uint4*>(a.X + k * a.ldx);
            float t[2] = {0.0f, 0.0f};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const uint4 v = row[min(lane + 64 * e, nch - 1)];
                const uint32_t keep = lane + 64 * e < nch ? ~0u : 0u;
                const uint32_t xw[4] = {v.x & keep, v.y & keep, v.z & keep, v.w & keep};
#pragma unroll
                for (int w = 0; w < 2; ++w) {
                    const uint32_t aw[4] = {av[w][e].x & keep, av[w][e].y & keep, av[w][e].z & keep, av[w][e].w & keep};
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        t[w] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, aw[q]),
                                                               __builtin_bit_cast(bf16x2, xw[q]), t[w], false);
                }
            }
#pragma unroll
            for (int o = 32; o > 0; o >>= 1)
#pragma unroll
                for (int w = 0; w < 2; ++w) t[w] += __shfl_xor(t[w], o);
            if (lane < 2) put_terms(lds.t[lane][k], wave, wave < a.r ? a.s[lane] * (lane == 0 ? t[0] : t[1]) : 0.0f);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    // the tokens' values of the wave's pieces (a token past the last: the last one's, not stored)
    uint4 x[2][4];
    few_row(a.X + min(i, a.T - 1) * a.ldx, p, a.d_in, g, x);
    // the rank products of the walk, 16 ranks at a time: the n-th item's chunk c is number
    // n chunks + c and falls to wave number % 16, which has 16 rows of B (ranks 8 (g % 2) .. + 7 for
    // both terms) and the terms loaded ahead
    const int chunks = (a.r + 15) / 16;
    int number = wave;
    uint4 b[2], t[2];
    auto load_ranks = [&]() {
        if (chunks == 0) return;
        const int n = number / chunks, j0 = (number - n * chunks) * 16 + 8 * (g & 1);
        const int64_t at = static_cast<int64_t>(blockIdx.x) + static_cast<int64_t>(n) * gridDim.x;
        if (at >= items) return;
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            const uint16_t* row = a.B[w] + (at * 16 + i) * a.r;
            if ((a.r & 7) == 0) {
                const uint4 v = *reinterpret_cast<const uint4*>(row + min(j0, a.r - 8));
                b[w] = j0 < a.r ? v : uint4{0, 0, 0, 0};
            } else {
                uint32_t v[4] = {0u, 0u, 0u, 0u};
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (j0 + e < a.r) v[e >> 1] |= static_cast<uint32_t>(row[j0 + e]) << (16 * (e & 1));
                b[w] = uint4{v[0], v[1], v[2], v[3]};
            }
            if constexpr (!kOwn) t[w] = a.t[w * chunks + number - n * chunks][i][g];
        }
    };
    load_ranks();
    __builtin_amdgcn_sched_barrier(0);
    load(cur, item);
    build_tables(lds.tables, tab, a.bc[0].fmt);
    const bool plain = a.bc[0].fmt == kDqNone;
    const float mu[2] = {plain ? 0.0f : a.bc[0].mean[0], plain ? 0.0f : a.bc[1].mean[0]};
    QN_LDS_BARRIER();
    const uint32_t lane8 = static_cast<uint32_t>(lane & 31) << 3;
    for (int n = 0; item < items; ++n, item += static_cast<int>(gridDim.x)) {
        load(nxt, item + static_cast<int>(gridDim.x));
        f32x4 acc[2];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
            acc[w] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float ah = piece_constant(cur[2 * w + k], lds.tables, mu[w], p.in[k]);
#pragma unroll
                for (int st = 0; st < 4; ++st)
                    acc[w] = mfma16(piece_weights(cur[2 * w + k], st, ah, lds.tables, lane8), x[k][st], acc[w]);
            }
        }
        while (number < (n + 1) * chunks) {
#pragma unroll
            for (int w = 0; w < 2; ++w) acc[w] = mfma16(b[w], kOwn ? lds.t[w][min(i, kFewOwn - 1)][g] : t[w], acc[w]);
            number += kFewWaves;
            load_ranks();
        }
        const int parity = n & 1;
#pragma unroll
        for (int w = 0; w < 2; ++w) *reinterpret_cast<f32x4*>(&lds.red[parity][wave][w][4 * lane]) = acc[w];
        QN_LDS_BARRIER();
        // four waves in turn finish the item: output row e % 16 of token e / 16 (the sums that the
        // next item writes stand beside these)
        const int e = (wave - 4 * (n & 3)) * 64 + lane;
        if (e >= 0 && e < 16 * a.T) {
            const int row = e & 15, token = e >> 4;
            const int at = 4 * (16 * (row >> 2) + token) + (row & 3);
            float v[2] = {0.0f, 0.0f};
#pragma unroll
            for (int k = 0; k < kFewWaves; ++k)
#pragma unroll
                for (int w = 0; w < 2; ++w) v[w] += lds.red[parity][k][w][at];
            const int64_t out = static_cast<int64_t>(item) * 16 + row;
            a.H[token * a.ldh + out] = bf16_bits(gated_act(a.act, v[0]) * v[1]);
            if (a.GU != nullptr) {
                a.GU[token * a.ldgu + out] = bf16_bits(v[0]);
                a.GU[token * a.ldgu + a.d_ff + out] = bf16_bits(v[1]);
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) cur[k] = nxt[k];
    }
}

// H (and GU) of 64 outputs of 16 tokens: the slices' sums in order, G += s_g sum_j T_g[j] B_g[., j]
// with T = the A tiles' sums, in float32, U likewise. A thread has 4 outputs of a token; what it costs
// is trips to memory, so the first slices' loads are on their way while the ranks come to LDS (24
// tokens of 11008 outputs: 10 us with a thread per output and its loads one after the other).
struct JoinArgs {
    const float* part; int splits, T, d_ff, r, atiles, tiles;
    const uint16_t* B[2]; float s[2];
    int act;
    uint16_t* H; int64_t ldh;
    uint16_t* GU; int64_t ldgu;
};
constexpr int kJoinRows = 64, kJoinTokens = 16, kJoinRanks = 32, kJoinFirst = 4;

__global__ __launch_bounds__(256)
void gated_join_kernel(JoinArgs a) {
    __shared__ float s_b[2][kJoinRanks][kJoinRows + 4];
    __shared__ float s_t[2][kJoinTokens][kJoinRanks];
    const int n0 = static_cast<int>(blockIdx.x) * kJoinRows, t0 = static_cast<int>(blockIdx.y) * kJoinTokens;
    const int nt = min(kJoinTokens, a.T - t0);
    const int tid = threadIdx.x, n = 4 * (tid & 15), q = tid >> 4;
    const int64_t pitch = 16 * a.tiles, slice = pitch * a.T;
    const int rp = (a.r + 15) / 16 * 16;
    const float* part = a.part + t0 * pitch;
    const float* own = part + min(q, nt - 1) * pitch + 16 * a.atiles + n0 + n;
    f32x4 first[2][kJoinFirst];
#pragma unroll
    for (int w = 0; w < 2; ++w)
#pragma unroll
        for (int k = 0; k < kJoinFirst; ++k)
            first[w][k] = *reinterpret_cast<const f32x4*>(own + w * a.d_ff + min(k, a.splits - 1) * slice);
    f32x4 v[2];
    for (int j0 = 0; j0 < a.r || j0 == 0; j0 += kJoinRanks) {
        const int nj = min(kJoinRanks, a.r - j0);
        if (j0 > 0) __syncthreads();
        if ((a.r & 7) == 0) {
            // 8 ranks of a row; neighbouring threads have neighbouring rows
            for (int e = tid; e < 2 * kJoinRows * (nj / 8); e += 256) {
                const int row = e % kJoinRows, w = e / kJoinRows & 1, j = e / (2 * kJoinRows) * 8;
                const uint4 b = *reinterpret_cast<const uint4*>(a.B[w] + static_cast<int64_t>(n0 + row) * a.r + j0 + j);
                const uint32_t words[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    s_b[w][j + 2 * k][row] = __uint_as_float(words[k] << 16);
                    s_b[w][j + 2 * k + 1][row] = __uint_as_float(words[k] & 0xFFFF0000u);
                }
            }
        } else {
            for (int e = tid; e < 2 * kJoinRows * nj; e += 256) {
                const int row = e % kJoinRows, w = e / kJoinRows & 1, j = e / (2 * kJoinRows);
                s_b[w][j][row] = bf16_to_f32(a.B[w][static_cast<int64_t>(n0 + row) * a.r + j0 + j]);
            }
        }
        for (int e = tid; e < 2 * kJoinTokens * nj; e += 256) {
            const int w = e & 1, t = e / 2 % kJoinTokens, j = e / (2 * kJoinTokens);
            s_t[w][t][j] = a.s[w] * ordered_sum<4>(part + min(t, nt - 1) * pitch + w * rp + j0 + j, slice, a.splits);
        }
        __syncthreads();
        if (j0 == 0) {
#pragma unroll
            for (int w = 0; w < 2; ++w) {
                v[w] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int k = 0; k < kJoinFirst; ++k)
                    if (k < a.splits) v[w] = v[w] + first[w][k];
                for (int k = kJoinFirst; k < a.splits; ++k)
                    v[w] = v[w] + *reinterpret_cast<const f32x4*>(own + w * a.d_ff + k * slice);
            }
        }
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll 4
            for (int j = 0; j < nj; ++j) v[w] = v[w] + s_t[w][q][j] * *reinterpret_cast<const f32x4*>(&s_b[w][j][n]);
    }
    if (q >= nt) return;
    const int64_t t = t0 + q;
    *reinterpret_cast<uint2*>(a.H + t * a.ldh + n0 + n) =
        uint2{bf16_pair(gated_act(a.act, v[0][0]) * v[1][0], gated_act(a.act, v[0][1]) * v[1][1]),
              bf16_pair(gated_act(a.act, v[0][2]) * v[1][2], gated_act(a.act, v[0][3]) * v[1][3])};
    if (a.GU != nullptr) {
#pragma unroll
        for (int w = 0; w < 2; ++w)
            *reinterpret_cast<uint2*>(a.GU + t * a.ldgu + w * a.d_ff + n0 + n) =
                uint2{bf16_pair(v[w][0], v[w][1]), bf16_pair(v[w][2], v[w][3])};
    }
}

// Slices of K: as few as fit the LDS with T tokens
// With up to 16 tokens: 16 waves a tile where that leaves each 2 pieces or more (one token on 28672 x
// 8192 81 us), else 4 (16 tokens there, whose slices have 16 pieces: 276 us with 16 waves a tile)
struct SmallPlan { int splits, pairs, atiles, tiles, kw; };
SmallPlan small_plan(int64_t M, int64_t d_ff, int64_t d_in, int r) {
    const int npair = static_cast<int>((d_in / 64 + 1) / 2);
    int most = static_cast<int>(SmallLds<1, 16>::kX / (256 * M));
    SmallPlan s;
    s.kw = M > 32 ? 1 : M > 16 ? 2 : std::min(npair, most) >= 32 ? 16 : 4;
    if (s.kw != 16) most = static_cast<int>((s.kw == 4 ? SmallLds<1, 4>::kX : s.kw == 2 ? SmallLds<2, 2>::kX : SmallLds<4, 1>::kX) / (256 * M));
    s.atiles = 2 * ((r + 15) / 16);
    s.tiles = s.atiles + static_cast<int>(2 * d_ff / 16);
    // Of up to 4 times as many slices as must be: the fewest pieces that a wave takes one after the other
    // (rounds of a workgroup over its tiles), about 0.9 us each, against the sums' way to memory and back.
    // (17 tokens on 11008 x 4096: 3 slices 46.7 us, 4 35. With 16 waves a tile the barriers count, not
    // the pieces: as few as must be.)
    const int least = (npair + most - 1) / most, per = kWaves / s.kw;
    double best = 0.0;
    for (int n = least; n <= (s.kw == 16 ? least : std::min(npair, 4 * least)); ++n) {
        const int pairs = (npair + n - 1) / n, slices = (npair + pairs - 1) / pairs;
        const int walkers = std::max(1, std::min((s.tiles + per - 1) / per, 256 / slices)) * per;
        const double us = 0.9 * ((s.tiles + walkers - 1) / walkers) * ((pairs + s.kw - 1) / s.kw) +
                          static_cast<double>(slices) * static_cast<double>(M) * s.tiles * 128 / 4.0e6;
        if (n == least || us < best) {
            best = us;
            s.splits = slices;
            s.pairs = pairs;
        }
    }
    return s;
}

// Whether the walk over items takes the call
bool few(int64_t M, int64_t d_in) { return M <= kFewTokens && d_in <= kFewIn; }

}  // namespace

int64_t gated_small_part_floats(int64_t M, int64_t d_ff, int64_t d_in, int r) {
    if (few(M, d_in)) return 2 * ((r + 15) / 16) * static_cast<int64_t>(sizeof(FewRanks) / 4);
    const SmallPlan s = small_plan(M, d_ff, d_in, r);
    return static_cast<int64_t>(s.splits) * M * 16 * s.tiles;
}

hipError_t launch_gated_small(const GatedCall& c, const uint16_t* X, int64_t ldx, uint16_t* H, int64_t ldh, uint16_t* GU,
                              int64_t ldgu, float* part, hipStream_t st) {
    const int64_t blocks = c.d_ff * c.d_in / kBlock;
    const uint32_t code_bytes = static_cast<uint32_t>(blocks * 32), q_bytes = static_cast<uint32_t>(blocks);
    const uint32_t s_bytes = static_cast<uint32_t>(4 * (((blocks - 1) >> c.bc[0].gshift) + 1));
    if (few(c.M, c.d_in)) {
        FewArgs f{};
        for (int w = 0; w < 2; ++w) {
            f.codes[w] = c.codes[w]; f.bc[w] = c.bc[w]; f.A[w] = c.A[w]; f.B[w] = c.B[w]; f.s[w] = c.s[w];
        }
        f.code_bytes = code_bytes; f.q_bytes = q_bytes; f.s_bytes = s_bytes;
        f.X = X; f.ldx = ldx; f.T = static_cast<int>(c.M); f.d_ff = static_cast<int>(c.d_ff);
        f.d_in = static_cast<int>(c.d_in); f.r = c.r; f.act = c.act; f.H = H; f.ldh = ldh; f.GU = GU; f.ldgu = ldgu;
        f.t = reinterpret_cast<FewRanks*>(part);
        const dim3 grid(static_cast<unsigned>(std::min<int64_t>(256, c.d_ff / 16)));
        if (c.r > 0 && c.r <= 16 && c.M <= kFewOwn) {
            QN_LAUNCH("gated_few_kernel", st, gated_few_kernel<true>, grid, dim3(64 * kFewWaves), 0, st, f, tables());
            return hipGetLastError();
        }
        if (c.r > 0)
            QN_LAUNCH("gated_ax_kernel", st, gated_ax_kernel, dim3(static_cast<unsigned>(2 * ((c.r + 15) / 16))),
                      dim3(64 * kFewWaves), 0, st, f);
        QN_LAUNCH("gated_few_kernel", st, gated_few_kernel<false>, grid, dim3(64 * kFewWaves), 0, st, f, tables());
        return hipGetLastError();
    }
    const SmallPlan s = small_plan(c.M, c.d_ff, c.d_in, c.r);
    SmallArgs a{};
    JoinArgs j{};
    for (int w = 0; w < 2; ++w) {
        a.codes[w] = c.codes[w]; a.bc[w] = c.bc[w]; a.A[w] = c.A[w];
        j.B[w] = c.B[w]; j.s[w] = c.s[w];
    }
    a.X = X; a.ldx = ldx;
    a.T = static_cast<int>(c.M); a.d_ff = static_cast<int>(c.d_ff); a.d_in = static_cast<int>(c.d_in); a.r = c.r;
    a.atiles = s.atiles; a.tiles = s.tiles; a.splits = s.splits; a.pairs = s.pairs; a.part = part;
    const NF4Tables& tab = tables();
    a.code_bytes = code_bytes; a.q_bytes = q_bytes; a.s_bytes = s_bytes;
    // a workgroup per CU: 256 / splits walk over the tiles of a slice
    const int per = kWaves / s.kw;
    const dim3 grid(static_cast<unsigned>(std::max(1, std::min((s.tiles + per - 1) / per, 256 / s.splits))),
                    static_cast<unsigned>(s.splits));
#define QN_SMALL(TT, KW) \
    QN_LAUNCH("gated_small_kernel", st, (gated_small_kernel<TT, KW>), grid, dim3(kThreads), 0, st, a, tab)
    if (s.kw == 16) QN_SMALL(1, 16);
    else if (s.kw == 4) QN_SMALL(1, 4);
    else if (s.kw == 2) QN_SMALL(2, 2);
    else if (c.M <= 48) QN_SMALL(3, 1);
    else QN_SMALL(4, 1);
#undef QN_SMALL
    j.part = part; j.splits = s.splits; j.T = a.T; j.d_ff = a.d_ff; j.r = c.r; j.atiles = s.atiles; j.tiles = s.tiles;
    j.act = c.act; j.H = H; j.ldh = ldh; j.GU = GU; j.ldgu = ldgu;
    const unsigned jx = static_cast<unsigned>(c.d_ff / kJoinRows);
    QN_LAUNCH("gated_join_kernel", st, gated_join_kernel,
              dim3(jx, static_cast<unsigned>((c.M + kJoinTokens - 1) / kJoinTokens)), dim3(256), 0, st, j);
    return hipGetLastError();
}

}  // namespace qn
