// Softmax cross entropy over a large vocabulary, in pieces of it, and its gradient to the
// hidden states, on gfx950. The logits are never kept.
//
//   loss_t = log sum_v exp(z_tv) - z_ty,   z = X W^T,  y the token's target
//   dX_t   = scale_t (sum_v p_tv W_v - W_y),   p = softmax(z_t)
//
// The exponentials are taken relative to the target's own logit, which is one short dot product
// per token known before the sweep: with l = sum over v != y of exp(z_v - z_y),
//   loss = log(1 + l),    dX = scale / (1 + l) (sum_{v != y} exp(z_v - z_y) W_v - l W_y).
// Nothing underflows that matters (the sum is at least 1), the loss of a sure token keeps its
// digits, the gradient has no difference of nearly equal terms, and the sweep needs no maximum
// first: each piece's exponentials (bf16, so that they can be an MFMA operand) are multiplied
// with W in the same pass and the sums divided at the end. Two products where forming the
// logits again for the gradient would take three. (The exponentials' rounding, 2^-9 at most of each of many
// terms, moves dX by 0.0002 to 0.0007, relative, beside the 0.0017 of its own; a second term would be a
// third product.) Where z_v - z_y is large (past kMaxLog2 in powers of two) a tile of a row is scaled down
// by a power of two, and head_join brings the row to one scale: exact in every case, and no work where it
// does not happen.
//
// Tokens without a target (prompts, padding) are left out before the products: head_plan_kernel
// numbers the others, the GEMM gathers their rows, and workgroups past the last one end at once.
//
// Per piece: an NF4 head's rows dequantised; head_logits (the product and its exponentials),
// head_join (after the last piece the loss), head_grad (their product with W, whose rows are along K
// there: read by transposing LDS reads, no transposed copy; added to float32 sums). Then head_final. All sums are in fixed order.
// Bound by both products at the power-limited clock: 4096 tokens on 128000 rows of 4096 5.9 to 6.2 ms by
// the card (1.39 to 1.46 PFLOP/s), and on few tokens by the head's stream: 17 on 32000 rows 46 to 48 us,
// as a plain read of its 262 MB (46 to 52).
#include <hip/hip_runtime.h>

#include "gated.h"
#include "gemm_few.h"
#include "gemm_turns.h"
#include "head_loss.h"
#include "nf4_device.h"

#include <algorithm>
#include <type_traits>

namespace qn {
namespace {

constexpr int BK = kTurnK;
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;
// a tile's sum past which its rows are looked at one by one, and the power of two that a row's
// exponentials may reach (2^80 times 2^31 rows stays in float32)
constexpr float kLargest = 0x1p80f, kMaxLog2 = 80.0f;

// K-steps that a split of the gradient's product has at least, by its tiles' size (1 << lt)
__host__ __device__ constexpr int head_steps(int lt) { return lt == 6 ? 4 : 8; }
// Tiles of 64 are taken on up to 64 tokens (17 on 32000 rows of 4096: loss 61 us against 85 with tiles of
// 256, with the gradient 120 / 170; 64: 66 / 85 and 130 / 174) and, where they are at most kFewSmall (two
// rounds of the chip) in a piece, on up to kFewTokens tokens (65 on 32000 rows: 82 / 84 and 161 / 171, 128: 95 / 90
// and 187 / 186; not 65 and 128 on 128000 rows, 2000 small tiles: loss 284 / 273 and 335 / 276) and for up to
// kFewMost tiles of 256 (256 tokens on 16128 rows, 63 of them: 85 / 91 and 165 / 157; 512 on 8192, 64: 61 / 77
// and 134 / 143; 1024 on 8192, 128: 108 / 80 and 244 / 167).
constexpr int64_t kFewTokens = 128, kFewSmall = 1024, kFewMost = 64;
// Past this many tokens one workgroup numbers them in a launch of its own (on 4096 rows of 64, a
// launch of its own and each workgroup counting for itself: 4096 tokens 22 us and 20, 16384 61 and 66,
// 65536 212 and 400).
constexpr int64_t kPlanFrom = 8192;

// The numbering of the counted tokens and what is known of each (arrays of T)
struct HeadRows {
    int32_t* count;                           // [0]
    int32_t* idx;                             // token of a counted position
    int32_t* pos;                             // position of a token, -1: not counted
    int32_t* tgt;                             // a position's target
    float* zt;                                // its target's logit
    float* shift;                             // powers of two taken off its exponentials
    float* l;                                 // sum of 2^((z - zt) log2 e - shift), v != target
};

__host__ __device__ inline int64_t head_int_count(int64_t T) { return 16 + 6 * ((T + 3) / 4 * 4); }
HeadRows head_rows(char* ws, int64_t T) {
    const int64_t n = (T + 3) / 4 * 4;
    int32_t* p = reinterpret_cast<int32_t*>(ws);
    float* f = reinterpret_cast<float*>(p + 16 + 3 * n);
    return HeadRows{p, p + 16, p + 16 + n, p + 16 + 2 * n, f, f + n, f + 2 * n};
}

// One workgroup: wave w takes a 16th of the tokens, 64 at a time; counts, then numbers them.
__global__ __launch_bounds__(1024)
void head_plan_kernel(const int64_t* __restrict__ target, int64_t T, int64_t V, float* __restrict__ loss, HeadRows r) {
    __shared__ int counts[16];
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    const int64_t per = ((T + 15) / 16 + 63) / 64 * 64;
    const int64_t t0 = wave * per, t1 = min(t0 + per, T);
    int n = 0;
    for (int64_t t = t0; t < t1; t += 64) {
        const int64_t y = t + lane < t1 ? target[t + lane] : -1;
        n += __popcll(__ballot(y >= 0 && y < V));
    }
    if (lane == 0) counts[wave] = n;
    __syncthreads();
    int at = 0, all = 0;
    for (int w = 0; w < 16; ++w) {
        at += w < wave ? counts[w] : 0;
        all += counts[w];
    }
    for (int64_t t = t0; t < t1; t += 64) {
        const int64_t y = t + lane < t1 ? target[t + lane] : -1;
        const bool ok = y >= 0 && y < V;
        const unsigned long long m = __ballot(ok);
        const int p = at + __popcll(m & ((1ull << lane) - 1));
        if (ok) {
            r.idx[p] = static_cast<int32_t>(t + lane);
            r.tgt[p] = static_cast<int32_t>(y);
        }
        if (t + lane < t1) {
            r.pos[t + lane] = ok ? p : -1;
            if (!ok) loss[t + lane] = 0.0f;
        }
        at += __popcll(m);
    }
    if (threadIdx.x == 0) r.count[0] = all;
}

// The target's logit of each counted token, a wave each; of an NF4 head also the target's row in
// bf16 (wt, if not null). Without head_plan_kernel before it (planned 0), workgroup b takes tokens
// 4 b .. 4 b + 3, counts the tokens before them itself and writes their numbering; else positions.
__global__ __launch_bounds__(256)
void head_target_kernel(HeadCall c, HeadRows r, uint16_t* wt, int planned, NF4Tables tab) {
    __shared__ float s_code[16];
    __shared__ int s_before[4];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int t0 = static_cast<int>(blockIdx.x) * 4;
    if (threadIdx.x < 16) s_code[threadIdx.x] = tab.code[threadIdx.x];
    int64_t t = 0, y = 0;
    int m = t0 + wave;
    if (!planned) {
        auto counted = [&](int64_t v) { return v >= 0 && v < c.V; };
        const int64_t own = lane < 4 && t0 + lane < c.T ? c.target[t0 + lane] : -1;
        int n = 0;
#pragma unroll 4
        for (int i = threadIdx.x; i < t0; i += 256) n += counted(c.target[i]) ? 1 : 0;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) n += __shfl_xor(n, o);
        if (lane == 0) s_before[wave] = n;
        __syncthreads();
        const unsigned long long here = __ballot(counted(own));
        const int before = (s_before[0] + s_before[1]) + (s_before[2] + s_before[3]);
        if (t0 + 4 >= c.T && threadIdx.x == 0) r.count[0] = before + __popcll(here);
        t = t0 + wave;
        y = __shfl(own, wave);
        m = before + __popcll(here & ((1ull << wave) - 1));
        if (t >= c.T) return;
        if (lane == 0) {
            r.pos[t] = counted(y) ? m : -1;
            if (!counted(y)) {
                c.loss[t] = 0.0f;
            } else {
                r.idx[m] = static_cast<int32_t>(t);
                r.tgt[m] = static_cast<int32_t>(y);
            }
        }
        if (!counted(y)) return;
    } else {
        __syncthreads();
        if (m >= r.count[0]) return;
        t = r.idx[m];
        y = r.tgt[m];
    }
    const uint16_t* x = c.X + t * c.ldx;
    float sum = 0.0f;
    for (int64_t k0 = 8 * lane; k0 < c.d; k0 += 2048) {
        uint4 xv[4], wv[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {                // all loads first; past the end the last again
            const int64_t k = min(k0 + 512 * p, c.d - 8);
            xv[p] = *reinterpret_cast<const uint4*>(x + k);
            if (c.codes == nullptr) {
                wv[p] = *reinterpret_cast<const uint4*>(c.W + y * c.ldw + k);
            } else {
                const int64_t e = y * c.d + k, blk = e >> 6;
                const uint32_t word = *reinterpret_cast<const uint32_t*>(c.codes + (e >> 1));
                const float a = block_constant(c.bc.fmt, c.bc.q[blk], c.bc.scale[blk >> c.bc.gshift], c.bc.mean[0]);
                float w[8];
#pragma unroll
                for (int q = 0; q < 8; ++q) w[q] = s_code[(word >> (4 * q)) & 0xFu] * a;
                wv[p] = uint4{bf16_pair(w[0], w[1]), bf16_pair(w[2], w[3]), bf16_pair(w[4], w[5]), bf16_pair(w[6], w[7])};
            }
        }
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const int64_t k = k0 + 512 * p;
            if (k >= c.d) break;
            if (wt != nullptr) *reinterpret_cast<uint4*>(wt + m * c.d + k) = wv[p];
            const uint32_t xw[4] = {xv[p].x, xv[p].y, xv[p].z, xv[p].w}, ww[4] = {wv[p].x, wv[p].y, wv[p].z, wv[p].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                sum += __uint_as_float(xw[q] << 16) * __uint_as_float(ww[q] << 16);
                sum += __uint_as_float(xw[q] & 0xFFFF0000u) * __uint_as_float(ww[q] & 0xFFFF0000u);
            }
        }
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    if (lane == 0) {
        r.zt[m] = sum;
        r.shift[m] = 0.0f;
        r.l[m] = 0.0f;
    }
}

struct HeadTile {
    int v0, cols, tiles_n;                    // the piece's first row of the head, its rows and tiles
    int64_t T;
    float2* part;                             // [tiles_n][T]: a tile's sum, and the power taken off
    uint16_t* E; int64_t lde;                 // exponentials [T, lde] (gradient)
};

// A tile of counted tokens x rows of the piece: z in the accumulators, then the exponentials.
// kFew: tiles of 64 x 64 (gemm_few.h), else of 256 x 256.
template <bool kGrad, bool kFew>
__global__ __launch_bounds__(kFew ? kFewThreads : kTurnThreads, kFew ? 2 : 1)
void head_logits_kernel(TurnArgs g, HeadTile h, HeadRows r) {
    constexpr int BM = kFew ? kFewTile : kTurnTile, BN = BM;
    constexpr int kH = kFew ? 1 : 2, kI = kFew ? 2 : 4, kWn = kFew ? 2 : 4;      // halves, 16-row blocks, waves side by side
    __shared__ float s_top[kWn][BM], s_sum[kWn][BM];
    const int count = r.count[0];
    const int tiles_m = (count + BM - 1) / BM;
    const int item = turn_item(static_cast<int>(blockIdx.x), tiles_m * h.tiles_n);
    if (item < 0) return;
    int tm, tn;
    turn_tile(item, tiles_m, h.tiles_n, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const auto row_p = [&](int i) { return static_cast<uint32_t>(r.idx[min(m0 + i, count - 1)]); };
    const auto row_q = [&](int i) { return static_cast<uint32_t>(min(n0 + i, h.cols - 1)); };
    std::conditional_t<kFew, FewSums, TurnSums> acc;
    if constexpr (kFew) gemm_few<false, false>(g, row_p, row_q, 0, g.kt1, false, acc);
    else gemm_turns<false, false>(g, row_p, row_q, 0, g.kt1, false, acc);
    // e = 2^((z - zt) log2 e - shift), 0 at the target and past the piece. The lane has rows 128 hh +
    // row0 + 16 i and of each 16 columns, base + 128 q + 16 j + e.
    const int tid = threadIdx.x;
    const int lane = tid & 63, wave = tid >> 6;
    const int wn = wave % kWn;
    const int row0 = 16 * kI * (wave / kWn) + (lane & 15), base = 32 * wn + 4 * (lane >> 4);
    const int columns = h.cols - n0 - base;          // of the lane's, those below are in the piece
    // the tile's columns that stay out of the lane's row: its target's (none: outside 0..255)
    auto put = [&](int row, int col, const f32x4t& v) {       // of the tile: four values of E
        if constexpr (!kFew) turn_put<256>(row, col, v[0], v[1], v[2], v[3]);
        else if (m0 + row < count)
            *reinterpret_cast<uint2*>(h.E + static_cast<int64_t>(m0 + row) * h.lde + n0 + col) =
                uint2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    };
    auto target = [&](int m) { return r.tgt[m] - h.v0 - n0 - base; };
    auto keep = [&](f32x4t v, int off, int skip, float out) {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (off + e == skip || off + e >= columns) v[e] = out;
        return v;
    };
#pragma unroll
    for (int hh = 0; hh < kH; ++hh)
#pragma unroll
        for (int i = 0; i < kI; ++i) {
            const int ml = 128 * hh + 16 * i + row0;
            const int m = min(m0 + ml, count - 1);
            const float c = -r.zt[m] * kLog2e - r.shift[m];
            const int skip = target(m);
            // few groups of 16 rows have a target in the tile, one tile of a piece has an edge
            const bool some = __any(skip >= 0 && skip < BN) || n0 + BN > h.cols;
            float sum = 0.0f;
#pragma unroll
            for (int q = 0; q < kH; ++q)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    f32x4t v = acc[hh][q][i][j];
#pragma unroll
                    for (int e = 0; e < 4; ++e) v[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(v[e], kLog2e, c));
                    if (some) v = keep(v, 128 * q + 16 * j, skip, 0.0f);
                    sum += (v[0] + v[1]) + (v[2] + v[3]);
                    if constexpr (kGrad) put(ml, base + 128 * q + 16 * j, v);
                }
            sum += __shfl_xor(sum, 16);
            sum += __shfl_xor(sum, 32);
            if (lane < 16) s_sum[wn][ml] = sum;
        }
    __syncthreads();
    auto total = [&](int row) {
        const float two = s_sum[0][row] + s_sum[1][row];
        return kFew ? two : two + (s_sum[kWn - 2][row] + s_sum[kWn - 1][row]);
    };
    float sum = 0.0f, power = 0.0f;
    bool large = false;
    if (tid < BM && m0 + tid < count) {
        sum = total(tid);
        large = !(sum <= kLargest);
    }
    if (__syncthreads_or(large)) {
        // a row far above its target (or not a number): the tile again, each row less its own power of
        // two; the other rows' bits are those of above
        auto relative = [&](f32x4t v, int off, int skip, int m) {
            const float c = -r.zt[m] * kLog2e - r.shift[m];
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(v[e], kLog2e, c);
            return keep(v, off, skip, -__builtin_inff());
        };
        for (int hh = 0; hh < kH; ++hh)
#pragma unroll
            for (int i = 0; i < kI; ++i) {
                const int ml = 128 * hh + 16 * i + row0, m = min(m0 + ml, count - 1);
                float t = -__builtin_inff();
#pragma unroll
                for (int q = 0; q < kH; ++q)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const f32x4t v = relative(hh == 0 ? acc[0][q][i][j] : acc[kH - 1][q][i][j], 128 * q + 16 * j, target(m), m);
                        t = fmaxf(fmaxf(fmaxf(t, v[0]), fmaxf(v[1], v[2])), v[3]);
                    }
                t = fmaxf(t, __shfl_xor(t, 16));
                t = fmaxf(t, __shfl_xor(t, 32));
                if (lane < 16) s_top[wn][ml] = t;
            }
        __syncthreads();
        auto off_of = [&](int row) {
            const float t = fmaxf(fmaxf(s_top[0][row], s_top[1][row]), fmaxf(s_top[kWn - 2][row], s_top[kWn - 1][row]));
            return t > kMaxLog2 ? ceilf(t) : 0.0f;
        };
        for (int hh = 0; hh < kH; ++hh)
#pragma unroll
            for (int i = 0; i < kI; ++i) {
                const int ml = 128 * hh + 16 * i + row0, m = min(m0 + ml, count - 1);
                const float off = off_of(ml);
                float s = 0.0f;
#pragma unroll
                for (int q = 0; q < kH; ++q)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        f32x4t v = relative(hh == 0 ? acc[0][q][i][j] : acc[kH - 1][q][i][j], 128 * q + 16 * j, target(m), m);
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = __builtin_amdgcn_exp2f(v[e] - off);
                        s += (v[0] + v[1]) + (v[2] + v[3]);
                        if constexpr (kGrad) put(ml, base + 128 * q + 16 * j, v);
                    }
                s += __shfl_xor(s, 16);
                s += __shfl_xor(s, 32);
                if (lane < 16) s_sum[wn][ml] = s;
            }
        __syncthreads();
        if (tid < BM) {
            sum = total(tid);
            power = off_of(tid);
        }
    }
    if (tid < BM && m0 + tid < count) h.part[tn * h.T + m0 + tid] = float2{sum, power};
    if constexpr (kGrad && !kFew) {
        const int c = tid & 31;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int row = 16 * i + (tid >> 5);
            const uint4 v = turn_get<256>(row, c);
            if (m0 + row < count) *reinterpret_cast<uint4*>(h.E + static_cast<int64_t>(m0 + row) * h.lde + n0 + c * 8) = v;
        }
    }
}

// The gradient's float32 sums: tiles of 1 << lt, tiles_n of them across d, room for slots
struct HeadAcc { float* acc; int lt, tiles_n, slots, kt_first; };

// its product's tiles, and the splits of their K-steps that fill the slots
struct HeadSplit { int tiles, splits, kper; };
__device__ __forceinline__ HeadSplit head_split(const HeadAcc& a, int count, int kt) {
    HeadSplit s;
    s.tiles = ((count + (1 << a.lt) - 1) >> a.lt) * a.tiles_n;
    // at least head_steps(lt) K-steps per split of the first (longest) piece, and no split of it without any
    const int want = max(1, min(a.slots / max(1, s.tiles), a.kt_first / head_steps(a.lt)));
    const int per = (a.kt_first + want - 1) / want;
    s.splits = (a.kt_first + per - 1) / per;
    s.kper = (kt + s.splits - 1) / s.splits;
    return s;
}
// the sums of position m's row, column n, of split 0; the next split's are tiles << 2 lt further
__device__ __forceinline__ float* head_sums(const HeadAcc& a, int m, int64_t n) {
    const int in = (1 << a.lt) - 1;
    const int64_t tile = static_cast<int64_t>(m >> a.lt) * a.tiles_n + (n >> a.lt);
    return a.acc + (tile << (2 * a.lt)) + (static_cast<int64_t>(m & in) << a.lt) + (n & in);
}

// A piece's sums joined to the row's: l, and, where a tile was scaled down, the row brought to one
// scale (its exponentials in E and the sums of earlier pieces in acc times exact powers of two); after
// the last piece the loss. 16 rows per workgroup, 16 threads a row (64 rows of 4 threads took 8 us of 17
// tokens on 32000 rows, in trips to memory one after another).
struct HeadJoin {
    const float2* part; int tiles_n, lt; int64_t T;   // tiles 1 << lt wide
    uint16_t* E; int64_t lde;                 // or null
    HeadAcc a;                                // acc null: no earlier piece
    int64_t d;
    float* loss;                              // null: more pieces follow
};

__global__ __launch_bounds__(256)
void head_join_kernel(HeadJoin j, HeadRows r) {
    __shared__ float s_sum[16][17], s_top[16][17], s_off[16];
    const int count = r.count[0];
    const int m0 = static_cast<int>(blockIdx.x) * 16;
    if (m0 >= count) return;
    const int i = threadIdx.x & 15, q = threadIdx.x >> 4;
    const int m = min(m0 + i, count - 1);
    float sum = 0.0f, top = 0.0f;
#pragma unroll 8
    for (int n = q; n < j.tiles_n; n += 16) {
        const float2 p = j.part[n * j.T + m];
        sum += p.x;
        top = fmaxf(top, p.y);
    }
    s_sum[q][i] = sum;
    s_top[q][i] = top;
    __syncthreads();
    if (q == 0) {
        sum = 0.0f;
#pragma unroll
        for (int k = 0; k < 16; ++k) {
            sum += s_sum[k][i];
            top = fmaxf(top, s_top[k][i]);
        }
        s_off[i] = top;
        if (m0 + i < count) {
            float l = r.l[m], shift = r.shift[m];
            if (top == 0.0f) {
                l += sum;
            } else {
                l *= __builtin_amdgcn_exp2f(-top);
                for (int n = 0; n < j.tiles_n; ++n) {
                    const float2 p = j.part[n * j.T + m];
                    l += p.x * __builtin_amdgcn_exp2f(p.y - top);
                }
                shift += top;
                r.shift[m] = shift;
            }
            r.l[m] = l;
            // log(1 + l), where 1 = exp(z_y - z_y) is 2^-shift on the row's scale
            if (j.loss != nullptr)
                j.loss[r.idx[m]] = shift == 0.0f ? log1pf(l) : shift * kLn2 + logf(__builtin_amdgcn_exp2f(-shift) + l);
        }
    }
    if (!__syncthreads_or(q == 0 && top != 0.0f) || j.E == nullptr) return;
    for (int k = 0; k < 16 && m0 + k < count; ++k) {
        const float off = s_off[k];
        if (off == 0.0f) continue;                   // uniform
        const int row = m0 + k;
        uint16_t* e = j.E + static_cast<int64_t>(row) * j.lde;
        for (int n = threadIdx.x; n < j.tiles_n << j.lt; n += 256) {
            const float f = __builtin_amdgcn_exp2f(j.part[(n >> j.lt) * j.T + row].y - off);
            e[n] = bf16_bits(__uint_as_float(static_cast<uint32_t>(e[n]) << 16) * f);
        }
        if (j.a.acc != nullptr) {
            const float f = __builtin_amdgcn_exp2f(-off);
            const HeadSplit s = head_split(j.a, count, j.a.kt_first);
            for (int sp = 0; sp < s.splits; ++sp)
                for (int64_t n = threadIdx.x; n < j.d; n += 256)
                    head_sums(j.a, row, n)[static_cast<int64_t>(sp) * s.tiles << (2 * j.a.lt)] *= f;
        }
    }
}

// acc += E W of a piece (the first piece: =), float32 tiles; tile (tm, tn) of split s is slot
// s tiles + tm tiles_n + tn.
template <bool kFew>
__global__ __launch_bounds__(kFew ? kFewThreads : kTurnThreads, kFew ? 2 : 1)
void head_grad_kernel(TurnArgs g, HeadAcc h, int first, int d, HeadRows r) {
    constexpr int BM = kFew ? kFewTile : kTurnTile, BN = BM;
    const int count = r.count[0];
    const HeadSplit s = head_split(h, count, g.kt1);
    const int item = turn_item(static_cast<int>(blockIdx.x), s.tiles * s.splits);
    if (item < 0) return;
    const int sp = item / s.tiles;
    const int kb = __builtin_amdgcn_readfirstlane(sp * s.kper), ke = min(kb + s.kper, g.kt1);
    if (kb >= ke) return;                            // a later, shorter piece adds nothing here
    int tm, tn;
    turn_tile(item % s.tiles, (count + BM - 1) / BM, h.tiles_n, tm, tn);
    const int m0 = tm * BM, n0 = tn * BN;
    const auto row_p = [&](int i) { return static_cast<uint32_t>(min(m0 + i, count - 1)); };
    const auto row_q = [&](int i) { return static_cast<uint32_t>(min(n0 + i, d - 8)); };
    float* const at = h.acc + (static_cast<int64_t>(sp) * s.tiles + tm * h.tiles_n + tn) * (BM * BN);
    std::conditional_t<kFew, FewSums, TurnSums> acc;
    if constexpr (kFew) {
        gemm_few<false, true>(g, row_p, row_q, kb, ke, false, acc);
        few_put_sums(at, acc, !first);
    } else {
        gemm_turns<false, true>(g, row_p, row_q, kb, ke, false, acc);
        turn_put_sums(at, acc, !first);
    }
}

// dX of a token from the sums (zeros for one that is not counted).
__global__ __launch_bounds__(256)
void head_final_kernel(HeadCall c, HeadAcc a, const uint16_t* wt, HeadRows r) {
    const int64_t t = blockIdx.x;
    const int m = r.pos[t];
    const int count = r.count[0];
    uint16_t* out = c.dX + t * c.lddx;
    if (m < 0) {
        for (int64_t n = 4 * threadIdx.x; n < c.d; n += 1024) *reinterpret_cast<uint2*>(out + n) = uint2{0u, 0u};
        return;
    }
    const HeadSplit s = head_split(a, count, a.kt_first);
    const float l = r.l[m];
    const float k = (c.scale != nullptr ? c.scale[t] : 1.0f) / (__builtin_amdgcn_exp2f(-r.shift[m]) + l);
    const uint16_t* w = wt != nullptr ? wt + m * c.d : c.W + r.tgt[m] * c.ldw;      // the target's row
    for (int64_t n = 4 * threadIdx.x; n < c.d; n += 1024) {
        const float4 v = ordered_sum4<4>(head_sums(a, m, n), static_cast<int64_t>(s.tiles) << (2 * a.lt), s.splits);
        const uint2 wv = *reinterpret_cast<const uint2*>(w + n);
        uint2 o;
        o.x = bf16_pair(k * (v.x - l * __uint_as_float(wv.x << 16)), k * (v.y - l * __uint_as_float(wv.x & 0xFFFF0000u)));
        o.y = bf16_pair(k * (v.z - l * __uint_as_float(wv.y << 16)), k * (v.w - l * __uint_as_float(wv.y & 0xFFFF0000u)));
        *reinterpret_cast<uint2*>(out + n) = o;
    }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace

bool head_plan(int64_t V, int64_t d, int64_t ldw, int64_t T, bool nf4, bool grad, HeadPlan* p) {
    constexpr int64_t kLimit = int64_t{1} << 31;     // elements of bf16 in 4 GiB
    // Pieces of up to 65536 rows (dequantised rows of 4096: 512 MB), of a gradient 32768 and
    // fewer where T rows of exponentials would pass 2^27 (256 MB), but 4096 rows of them up to 2 GiB.
    int64_t most = grad ? 32768 : 65536;
    if (grad) most = std::min(most, std::max((int64_t{1} << 27) / T, std::min<int64_t>(4096, kLimit / 2 / T)) / 256 * 256);
    // up to 2^22 tiles of a piece: a launch has less than 2^32 threads
    most = std::min(most, (int64_t{1} << 22) / ceil_div(T, kTurnTile) * kTurnTile);
    auto cut = [&](int64_t ld) {                     // in even pieces that stay below 4 GiB at this row stride
        most = std::max<int64_t>(256, std::min(most, (kLimit - 1) / ld / 256 * 256));
        p->pieces = static_cast<int>(ceil_div(V, most));
        p->piece = ceil_div(ceil_div(V, p->pieces), 256) * 256;
        p->pieces = static_cast<int>(ceil_div(V, p->piece));
    };
    cut(d);
    if (grad && p->piece >= kLimit / T) return false;
    if (std::min(V, p->piece) > (kLimit - 1) / d) return false;
    const int64_t large = ceil_div(T, kTurnTile) * ceil_div(p->piece, kTurnTile), rows = std::min(V, p->piece);
    const bool two_rounds = ceil_div(T, kFewTile) * ceil_div(rows, kFewTile) <= kFewSmall;
    p->lt = T <= kFewTile || (two_rounds && (T <= kFewTokens || large <= kFewMost)) ? 6 : 8;
    // Rows further apart may need smaller pieces. The tiles stay as they are, and with them every part
    // of the workspace is at most what it is for ldw = d.
    if (ldw > d) cut(ldw);
    const int64_t tile = int64_t{1} << p->lt;
    const int64_t tm = ceil_div(T, tile), tn = ceil_div(d, tile), kt = p->piece / BK;
    p->slots = !grad ? 0 : static_cast<int>(std::max(tm * tn, std::min<int64_t>(p->lt == 6 ? 512 : 256,
                                                                                tm * tn * std::max<int64_t>(1, kt / head_steps(p->lt)))));
    int64_t off = 0;
    auto take = [&off](int64_t bytes) {
        const int64_t at = off;
        off += ceil_div(bytes, 256) * 256;
        return at;
    };
    p->ints = take(4 * head_int_count(T));
    p->part = take(8 * (p->piece >> p->lt) * T);
    p->E = take(grad ? 2 * T * p->piece : 0);
    p->rows = take(nf4 ? 2 * d * p->piece : 0);
    p->wt = take(nf4 && grad ? 2 * T * d : 0);
    p->acc = take((static_cast<int64_t>(p->slots) << (2 * p->lt)) * 4);
    p->bytes = off;
    return true;
}

hipError_t launch_head_loss(const HeadCall& c, const HeadPlan& p, char* ws, hipStream_t st) {
    const bool grad = c.dX != nullptr, nf4 = c.codes != nullptr;
    const HeadRows r = head_rows(ws + p.ints, c.T);
    float2* part = reinterpret_cast<float2*>(ws + p.part);
    uint16_t* E = grad ? reinterpret_cast<uint16_t*>(ws + p.E) : nullptr;
    uint16_t* rows = nf4 ? reinterpret_cast<uint16_t*>(ws + p.rows) : nullptr;
    uint16_t* wt = nf4 && grad ? reinterpret_cast<uint16_t*>(ws + p.wt) : nullptr;
    float* acc = grad ? reinterpret_cast<float*>(ws + p.acc) : nullptr;
    const bool few = p.lt == 6;
    const int64_t tile = int64_t{1} << p.lt;
    const int tm = static_cast<int>(ceil_div(c.T, tile));
    const dim3 threads(few ? kFewThreads : kTurnThreads);
    const HeadAcc sums{acc, p.lt, static_cast<int>(ceil_div(c.d, tile)), p.slots,
                       static_cast<int>(ceil_div(std::min(p.piece, c.V), BK))};
    const bool planned = c.T > kPlanFrom;
    if (planned) QN_LAUNCH("head_plan_kernel", st, head_plan_kernel, dim3(1), dim3(1024), 0, st, c.target, c.T, c.V, c.loss, r);
    QN_LAUNCH("head_target_kernel", st, head_target_kernel, dim3(static_cast<unsigned>(ceil_div(c.T, 4))), dim3(256), 0, st,
              c, r, wt, planned ? 1 : 0, tables());
    hipError_t e = hipGetLastError();
    for (int i = 0; i < p.pieces && e == hipSuccess; ++i) {
        const int64_t v0 = i * p.piece, cols = std::min(p.piece, c.V - v0);
        const uint16_t* W = nf4 ? rows : c.W + v0 * c.ldw;
        const int64_t ldw = nf4 ? c.d : c.ldw;
        if (nf4) {
            // v0 d / 64 blocks is a multiple of 256 of them: whole groups of constants
            BlockConsts bc = c.bc;
            const int64_t blk = v0 * c.d / kBlock;
            bc.q += bc.fmt == kDqNone ? 0 : blk;
            bc.scale += blk >> bc.gshift;
            if ((e = launch_dequant_weight(c.codes + v0 * c.d / 2, bc, cols, c.d, rows, st)) != hipSuccess) return e;
        }
        const int tn = static_cast<int>(ceil_div(cols, tile));
        const TurnArgs g = turn_args(c.X, c.ldx, c.T, W, ldw, cols, c.d);
        const HeadTile h{static_cast<int>(v0), static_cast<int>(cols), tn, c.T, part, E, p.piece};
        const dim3 lgrid(static_cast<unsigned>(ceil_div(tm * tn, 8) * 8));
        if (grad && few) QN_LAUNCH("head_logits_kernel", st, (head_logits_kernel<true, true>), lgrid, threads, 0, st, g, h, r);
        else if (grad) QN_LAUNCH("head_logits_kernel", st, (head_logits_kernel<true, false>), lgrid, threads, 0, st, g, h, r);
        else if (few) QN_LAUNCH("head_logits_kernel", st, (head_logits_kernel<false, true>), lgrid, threads, 0, st, g, h, r);
        else QN_LAUNCH("head_logits_kernel", st, (head_logits_kernel<false, false>), lgrid, threads, 0, st, g, h, r);
        HeadJoin j{part, tn, p.lt, c.T, E, p.piece, sums, c.d, i == p.pieces - 1 ? c.loss : nullptr};
        if (i == 0) j.a.acc = nullptr;
        QN_LAUNCH("head_join_kernel", st, head_join_kernel, dim3(static_cast<unsigned>(ceil_div(c.T, 16))), dim3(256), 0, st,
                  j, r);
        if (grad) {
            const TurnArgs q = turn_args(E, p.piece, c.T, W, ldw, cols, ceil_div(cols, BK) * BK);
            const dim3 ggrid(static_cast<unsigned>(ceil_div(p.slots, 8) * 8));
            const int first = i == 0, d = static_cast<int>(c.d);
            if (few) QN_LAUNCH("head_grad_kernel", st, head_grad_kernel<true>, ggrid, threads, 0, st, q, sums, first, d, r);
            else QN_LAUNCH("head_grad_kernel", st, head_grad_kernel<false>, ggrid, threads, 0, st, q, sums, first, d, r);
        }
        e = hipGetLastError();
    }
    if (e != hipSuccess) return e;
    if (grad) QN_LAUNCH("head_final_kernel", st, head_final_kernel, dim3(static_cast<unsigned>(c.T)), dim3(256), 0, st, c, sums, wt, r);
    return hipGetLastError();
}

}  // namespace qn
