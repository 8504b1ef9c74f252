// extern "C" entry points of libqlora_nf4: argument checks, workspace layout and
// kernel sequencing. Every step of the layer runs in the kernels of quantize.hip,
// prologue.hip, gemm_nt.hip, gemv.hip, skinny.hip, lora_grads.hip, factors.hip,
// multi_plan.hip, multi_small.hip, gemm_multi.hip, multi_grads.hip, adamw.hip, gated.hip,
// gated_small.hip and head_loss.hip; this file does no arithmetic on the data.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>
#include <map>
#include <mutex>
#include <string>
#include <vector>

#include "../../include/qlora_nf4.h"
#include "gated.h"
#include "head_loss.h"
#include "internal.h"
#include "multi.h"

namespace {

thread_local std::string g_err;

int fail(int code, const char* msg) {
    g_err = msg;
    return code;
}

int hip_fail(hipError_t e, const char* where) {
    g_err = std::string(where) + ": " + hipGetErrorString(e);
    return -4;
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int64_t align_up(int64_t v, int64_t a) { return (v + a - 1) / a * a; }

constexpr int64_t kMaxBlocks = (int64_t{1} << 32) - 1;

// Whether `rows` >= 1 rows of bf16 at stride ld >= 1 reach 4 GiB: the kernels address an
// operand with 32-bit byte offsets. (A division, since the product can pass 64 bits.)
bool reaches_4gib(int64_t rows, int64_t ld) { return ld > ((int64_t{1} << 31) - 1) / rows; }

bool nf4_counts(int64_t d_out, int64_t d_in, int64_t* n, int64_t* n_b, int64_t* n_g) {
    if (d_out < 1 || d_in < 1) return false;
    if (d_out > (int64_t{1} << 40) / d_in) return false;
    *n = d_out * d_in;
    *n_b = (*n + qn::kBlock - 1) / qn::kBlock;
    *n_g = (*n_b + qn::kGroup - 1) / qn::kGroup;
    return *n_b <= kMaxBlocks;
}

// The block-constant arrays of a quantised weight in format dq. Checks pointers and
// alignment; for QN_DQ_NONE, qconst and qmean are not part of the format (may be
// null) and readable stand-ins replace them, since kernels load them unconditionally.
int make_consts(int dq, const uint8_t* codes, const int8_t* qconst, const float* qscale, const float* qmean,
                qn::BlockConsts* bc) {
    if (dq != QN_DQ_INT8 && dq != QN_DQ_FP8 && dq != QN_DQ_NONE) return fail(-1, "unknown second-level format");
    if (!codes || !qscale) return fail(-1, "null pointer argument");
    if (!aligned(qscale, 4)) return fail(-1, "misaligned pointer");
    if (dq == QN_DQ_NONE) {
        *bc = qn::BlockConsts{reinterpret_cast<const int8_t*>(codes), qscale, qscale, qn::kDqNone, 0};
        return 0;
    }
    if (!qconst || !qmean) return fail(-1, "null pointer argument");
    if (!aligned(qmean, 4)) return fail(-1, "misaligned pointer");
    *bc = qn::BlockConsts{qconst, qscale, qmean, dq == QN_DQ_FP8 ? qn::kDqFp8 : qn::kDqInt8, 8};
    return 0;
}

static_assert(QN_DQ_INT8 == qn::kDqInt8 && QN_DQ_FP8 == qn::kDqFp8 && QN_DQ_NONE == qn::kDqNone,
              "format codes");

struct QuantWs {
    int64_t absmax_off, limbs_off, bytes;
    int grid;
};

QuantWs quant_ws(int64_t n_b) {
    QuantWs w{};
    w.grid = qn::quant_grid(n_b);
    w.absmax_off = 0;
    w.limbs_off = align_up(n_b * 4, 256);
    w.bytes = w.limbs_off + align_up(static_cast<int64_t>(w.grid) * qn::kLimbs * 8, 256);
    return w;
}

struct LinWs {
    int64_t what, lora, adapt, adapt2, t, part, gpart, ppart, bytes;
    int r_pad;
};

// fp32 partials of a K-split LoRA pre-pass over M tokens and K columns (0 if unsplit)
int64_t prepass_part_bytes(int64_t M, int64_t K, int r) {
    const qn::PrepassSplit ps = qn::prepass_split(M, K);
    return ps.splits > 1 ? 4 * static_cast<int64_t>(ps.splits) * M * 32 * ((r + 31) / 32) : 0;
}

// Workspace layout of one linear call. The forward with d_seq <= kSkinnyMaxTokens streams
// the packed codes (GEMV or small batch) and needs only its partial sums; every other
// call dequantises W into the workspace and runs the GEMM. Regions a call does not use
// have size 0.
LinWs linear_ws(int64_t d_out, int64_t d_in, int64_t d_seq, int r, bool bwd) {
    LinWs w{};
    w.r_pad = static_cast<int>(align_up(r, 64));
    const bool streams = !bwd && d_seq <= qn::kSkinnyMaxTokens;
    const bool gemm = !streams;
    int64_t off = 0;
    w.what = off;   if (gemm) off += align_up(2 * d_out * d_in, 256);                        // W_hat or W_hat^T
    w.lora = off;   if (gemm) off += align_up(2 * d_seq * w.r_pad, 256);                     // s(XA^T) or s(dY B)
    w.adapt = off;  if (gemm) off += align_up(2 * (bwd ? d_in : d_out) * w.r_pad, 256);      // B padded or A^T padded
    w.adapt2 = off;                                                                          // B^T (unless the pre-pass reads B)
    if (bwd && !qn::prepass_takes_kmajor(r)) off += align_up(2 * static_cast<int64_t>(r) * d_out, 256);
    w.t = off;                                                                               // GEMV: partial A x
    if (streams && qn::gemv_takes_tokens(d_seq, d_out, d_in, r)) off += align_up(4 * qn::gemv_part_floats(d_seq, d_in, r), 256);
    w.part = off;                                                                            // small batch: K-split partials
    if (streams && !qn::gemv_takes_tokens(d_seq, d_out, d_in, r))
        off += align_up(4 * static_cast<int64_t>(qn::skinny_splits(d_in, d_seq)) * d_seq * (d_out + w.r_pad), 256);
    w.gpart = off;                                                                           // GEMM K-split partials (few tiles)
    if (gemm) off += align_up(4 * (bwd ? qn::gemm_split_part_floats(d_seq, d_in, d_out)
                                       : qn::gemm_split_part_floats(d_seq, d_out, d_in)), 256);
    w.ppart = off;                                                                           // pre-pass K-split partials
    if (gemm) off += align_up(bwd ? prepass_part_bytes(d_seq, d_out, r) : prepass_part_bytes(d_seq, d_in, r), 256);
    w.bytes = off;
    return w;
}

bool linear_sizes_ok(int64_t d_out, int64_t d_in, int64_t d_seq, int r) {
    return d_out >= 1 && d_in >= 1 && d_seq >= 1 && r >= 1 && r <= 256 && d_out <= (int64_t{1} << 40) / d_in &&
           d_seq <= INT32_MAX;
}

// Checks of a linear call; `in` [d_seq, in_cols] with row stride ldi, `out` [d_seq, out_cols]
// with row stride ldo (in elements).
int check_linear(const uint8_t* codes, const int8_t* qconst, const float* qscale, const float* qmean, int dq,
                 int64_t d_out, int64_t d_in, const uint16_t* A, const uint16_t* B, int r,
                 const uint16_t* in, int64_t ldi, int64_t d_seq, uint16_t* out, int64_t ldo, bool bwd, void* ws,
                 int64_t ws_bytes, LinWs* lw, qn::BlockConsts* bc) {
    if (int rc = make_consts(dq, codes, qconst, qscale, qmean, bc)) return rc;
    if (!A || !B || !in || !out || !ws) return fail(-1, "null pointer argument");
    if (d_out < 1 || d_in < 1 || d_seq < 1) return fail(-1, "sizes must be >= 1");
    if (r < 1 || r > 256) return fail(-1, "r must be in [1, 256]");
    const int64_t in_cols = bwd ? d_out : d_in, out_cols = bwd ? d_in : d_out;
    if (ldi < in_cols || ldo < out_cols) return fail(-1, "a leading dimension is smaller than its row");
    if (ldi % 8 != 0 || ldo % 8 != 0) return fail(-1, "leading dimensions must be multiples of 8 elements");
    if (!aligned(codes, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(in, 16) ||
        !aligned(out, 16) || !aligned(ws, 256))
        return fail(-1, "misaligned pointer (16 B for arrays, 256 B for the workspace)");
    if (d_in % 64 != 0 || d_out % 64 != 0) return fail(-2, "d_in and d_out must be multiples of 64");
    if (d_in > INT32_MAX || d_out > INT32_MAX || d_seq > INT32_MAX) return fail(-2, "dimension too large");
    int64_t n, n_b, n_g;
    if (!nf4_counts(d_out, d_in, &n, &n_b, &n_g)) return fail(-2, "weight too large");
    if (reaches_4gib(d_out, d_in) || reaches_4gib(d_seq, std::max(ldi, ldo)))
        return fail(-2, "an operand reaches 4 GiB");
    *lw = linear_ws(d_out, d_in, d_seq, r, bwd);
    if (ws_bytes < lw->bytes) return fail(-3, "workspace too small");
    return 0;
}

}  // namespace

// ---- optional kernel timing -------------------------------------------------
namespace qn {
namespace {
struct ProfRec {
    const char* name;
    hipEvent_t start, stop;
};
std::mutex g_prof_mu;
std::atomic<bool> g_prof_on{false};
std::vector<ProfRec> g_prof;
// Events are created once and reused: creating one per launch costs the host more than
// a short kernel runs, which left the device idle between launches while timing was on.
std::vector<hipEvent_t> g_pool;
constexpr size_t kPoolPrefill = 1024;

hipEvent_t take_event_locked() {
    if (!g_pool.empty()) {
        hipEvent_t e = g_pool.back();
        g_pool.pop_back();
        return e;
    }
    hipEvent_t e = nullptr;
    return hipEventCreate(&e) == hipSuccess ? e : nullptr;
}

void prof_clear_locked() {
    for (auto& r : g_prof) {
        g_pool.push_back(r.start);
        g_pool.push_back(r.stop);
    }
    g_prof.clear();
}
}  // namespace

void* prof_begin(hipStream_t st) {
    if (!g_prof_on.load(std::memory_order_relaxed)) return nullptr;
    std::lock_guard<std::mutex> lk(g_prof_mu);
    hipEvent_t e = take_event_locked();
    if (!e) return nullptr;
    if (hipEventRecord(e, st) != hipSuccess) {
        g_pool.push_back(e);
        return nullptr;
    }
    return e;
}

void prof_end(void* token, const char* name, hipStream_t st) {
    if (!token) return;
    std::lock_guard<std::mutex> lk(g_prof_mu);
    hipEvent_t e = take_event_locked();
    if (!e || hipEventRecord(e, st) != hipSuccess) {
        g_pool.push_back(static_cast<hipEvent_t>(token));
        if (e) g_pool.push_back(e);
        return;
    }
    g_prof.push_back({name, static_cast<hipEvent_t>(token), e});
}
}  // namespace qn

namespace {

// The forward once the arguments are checked: d_seq == 1 (and up to 3 tokens when r <= 16
// and d_in <= 4096) streams the codes (GEMV), d_seq <= 64 runs the small-batch kernel,
// otherwise dequantise + pre-pass + GEMM.
// forward GEMM form for d_seq > 64 (qlora_set_fwd_gemm)
std::atomic<int> g_fwd_gemm{QN_FWD_GEMM_AUTO};

// AUTO picks the in-GEMM dequantisation for a weight whose bf16 copy would not fit the
// 256 MB Infinity Cache (d_out d_in >= 2^27) at up to 1024 tokens (at most 4 tile rows of
// 256 tokens, each of which dequantises every weight again); otherwise W_hat is staged.
// Measured at 65..2048 tokens: fused / staged call time 0.55..0.95 for 28672 x 8192 up
// to 1024 tokens and 1.10 at 2048; 0.98..1.37 for the 11008 x 4096 and 4096 x 11008 MLP
// layers and 1.00..1.23 for 4096 x 4096, whose staged W_hat stays in the cache.
bool fwd_gemm_fused(int64_t d_seq, int64_t d_out, int64_t d_in) {
    const int form = g_fwd_gemm.load(std::memory_order_relaxed);
    if (form != QN_FWD_GEMM_AUTO) return form == QN_FWD_GEMM_FUSED;
    return d_out * d_in >= (int64_t{1} << 27) && d_seq <= 1024;
}

int linear_fwd_run(const uint8_t* codes, const qn::BlockConsts& bc, int64_t d_out, int64_t d_in,
                   const uint16_t* A, const uint16_t* B, int r, float s, const uint16_t* X, int64_t ldx,
                   int64_t d_seq, uint16_t* Y, int64_t ldy, char* ws, const LinWs& lw, hipStream_t st) {
    hipError_t e;
    if (qn::gemv_takes_tokens(d_seq, d_out, d_in, r)) {
        e = qn::launch_gemv_nf4(codes, bc, d_out, d_in, A, B, r, s, X, ldx, d_seq, Y, ldy,
                                reinterpret_cast<float*>(ws + lw.t), st);
        if (e != hipSuccess) return hip_fail(e, "qlora_linear_fwd (gemv)");
        return 0;
    }
    if (d_seq <= qn::kSkinnyMaxTokens) {
        // few tokens: the codes streamed once, A x in the same launch
        float* part = reinterpret_cast<float*>(ws + lw.part);
        float* part_a = part + static_cast<int64_t>(qn::skinny_splits(d_in, d_seq)) * d_seq * d_out;
        if ((e = qn::launch_skinny_nf4(codes, bc, d_out, d_in, X, ldx, d_seq, A, B, r, lw.r_pad, s,
                                       part, part_a, Y, ldy, st)) != hipSuccess)
            return hip_fail(e, "qlora_linear_fwd (small batch)");
        return 0;
    }
    const bool fused = fwd_gemm_fused(d_seq, d_out, d_in);
    uint16_t* what = fused ? nullptr : reinterpret_cast<uint16_t*>(ws + lw.what);
    uint16_t* t = reinterpret_cast<uint16_t*>(ws + lw.lora);
    uint16_t* bpad = reinterpret_cast<uint16_t*>(ws + lw.adapt);
    const bool pad = r != lw.r_pad;
    // T = s (X A^T) + B padded to r_pad columns (+ the dequantised W_hat when staged), in
    // one launch
    if ((e = qn::launch_prologue(codes, bc, d_out, d_in, false, what, X, ldx, d_seq, d_in,
                                 A, d_in, false, r, s, t, lw.r_pad, pad ? 1 : 0, B, bpad, d_out, r,
                                 reinterpret_cast<float*>(ws + lw.ppart), st)) != hipSuccess)
        return hip_fail(e, "qlora_linear_fwd (prologue)");
    if ((e = qn::launch_gemm_nt(X, ldx, what, d_in, d_in, t, lw.r_pad, pad ? bpad : B, lw.r_pad, lw.r_pad, Y,
                                ldy, d_seq, d_out, reinterpret_cast<float*>(ws + lw.gpart), st,
                                fused ? codes : nullptr, &bc)) != hipSuccess)
        return hip_fail(e, "qlora_linear_fwd (gemm)");
    return 0;
}

}  // namespace

// workspace of qlora_lora_grads
namespace {
struct GradWs {
    int64_t tp, up, bt, part, ppart, ppart1, bytes;
    int r_pad;
};

GradWs grad_ws(int64_t d_out, int64_t d_in, int64_t d_seq, int r) {
    GradWs w{};
    w.r_pad = static_cast<int>(align_up(r, 64));
    int64_t off = 0;
    w.tp = off;   off += align_up(2 * d_seq * w.r_pad, 256);                        // T' = bf16(s X A^T)
    w.up = off;   off += align_up(2 * d_seq * w.r_pad, 256);                        // U' = bf16(s dY B)
    w.bt = off;   off += align_up(2 * static_cast<int64_t>(r) * d_out, 256);        // B^T (unless the pre-pass reads B)
    w.part = off; off += align_up(4 * qn::lora_grads_partials(d_out, d_in, d_seq, r), 256);
    w.ppart = off; off += align_up(prepass_part_bytes(d_seq, d_in, r), 256);       // X A^T K-split partials
    w.ppart1 = off; off += align_up(prepass_part_bytes(d_seq, d_out, r), 256);     // dY B K-split partials
    w.bytes = off;
    return w;
}
}  // namespace

// workspaces of qlora_gated_fwd and qlora_gated_bwd
namespace {
struct GatedWs {
    int64_t what, t, adapt, rpart, bt[2], part, bytes;
};

GatedWs gated_ws(int64_t d_ff, int64_t d_in, int64_t d_seq, int r, bool bwd) {
    GatedWs w{};
    int64_t off = 0;
    auto take = [&off](int64_t bytes) {
        const int64_t at = off;
        off += align_up(bytes, 256);
        return at;
    };
    if (!bwd && d_seq <= qn::kGatedSmall) {                                          // the codes streamed: sums only
        w.part = take(std::max<int64_t>(1, 4 * qn::gated_small_part_floats(d_seq, d_ff, d_in, r)));   // 0: sizes refused
        w.bytes = off;
        return w;
    }
    const int terms = qn::gated_terms(d_ff, d_in, d_seq, r), k2 = qn::gated_k2(r, terms);
    w.what = take(4 * d_ff * d_in);                                                  // both weights
    w.t = take(2 * d_seq * k2);                                                      // both rank products
    w.adapt = take(2 * (bwd ? d_in : 2 * d_ff) * k2);                                // both adapters
    w.rpart = take(4 * qn::gated_ranks_floats(d_seq, bwd ? d_ff : d_in, r, terms));  // their partial sums
    for (int i = 0; i < 2; ++i) w.bt[i] = take(bwd && !qn::gated_reads_b(r) ? 2 * static_cast<int64_t>(r) * d_ff : 0);
    w.part = take(4 * (bwd ? qn::gated_dx_part_floats(d_seq, d_ff, d_in) : qn::gated_part_floats(d_seq, d_ff, d_in)));
    w.bytes = off;
    return w;
}

// Whether an operand that the call makes reaches 4 GiB (sizes >= 1): both weights, the rank
// products or the adapters' layouts (in one term; gated_terms)
bool gated_too_large(int64_t d_ff, int64_t d_in, int64_t d_seq, int r) {
    const int64_t k2 = std::max(1, qn::gated_k2(r, 1));
    return reaches_4gib(2 * d_ff, std::max(d_in, k2)) || reaches_4gib(std::max(d_seq, d_in), k2);
}

// The sizes that a call takes with its activations at their least row strides. The forward's GU counts where
// the call keeps it.
bool gated_sizes_ok(int64_t d_ff, int64_t d_in, int64_t d_seq, int r, bool bwd) {
    return d_ff >= 1 && d_in >= 1 && d_seq >= 1 && r >= 0 && r <= 256 && d_ff % 64 == 0 && d_in % 64 == 0 &&
           d_in <= INT32_MAX && d_ff <= INT32_MAX / 2 && d_seq <= INT32_MAX && !gated_too_large(d_ff, d_in, d_seq, r) &&
           !reaches_4gib(d_seq, std::max(bwd ? 2 * d_ff : d_ff, d_in));
}

// What both gated calls check; `rows` are the row strides of the call's activations, each at
// least its row length.
int check_gated(const uint8_t* const (&codes)[2], const int8_t* const (&qconst)[2], const float* const (&qscale)[2],
                const float* const (&qmean)[2], int64_t d_ff, int64_t d_in, int dq, const uint16_t* const (&A)[2],
                const uint16_t* const (&B)[2], const float (&s)[2], int r, int act, int64_t d_seq, qn::GatedCall* c) {
    for (int i = 0; i < 2; ++i) {
        if (int rc = make_consts(dq, codes[i], qconst[i], qscale[i], qmean[i], &c->bc[i])) return rc;
        if (r > 0 && (!A[i] || !B[i])) return fail(-1, "null pointer argument");
        if (!aligned(codes[i], 16) || !aligned(A[i], 16) || !aligned(B[i], 16))
            return fail(-1, "misaligned pointer (16 B for arrays, 256 B for the workspace)");
        c->codes[i] = codes[i]; c->A[i] = A[i]; c->B[i] = B[i]; c->s[i] = s[i];
    }
    if (d_ff < 1 || d_in < 1 || d_seq < 1) return fail(-1, "sizes must be >= 1");
    if (r < 0 || r > 256) return fail(-1, "r must be in [0, 256]");
    if (act != QN_ACT_SILU && act != QN_ACT_GELU) return fail(-1, "unknown activation");
    if (d_in % 64 != 0 || d_ff % 64 != 0) return fail(-2, "d_in and d_ff must be multiples of 64");
    if (d_in > INT32_MAX || d_ff > INT32_MAX / 2 || d_seq > INT32_MAX) return fail(-2, "dimension too large");
    if (gated_too_large(d_ff, d_in, d_seq, r)) return fail(-2, "an operand reaches 4 GiB");
    c->d_ff = d_ff; c->d_in = d_in; c->M = d_seq; c->r = r; c->act = act;
    c->terms = qn::gated_terms(d_ff, d_in, d_seq, r);
    return 0;
}

static_assert(QN_ACT_SILU == qn::kActSilu && QN_ACT_GELU == qn::kActGelu, "activation codes");

// one activation of a gated call: `cols` wide at row stride ld
int check_rows(const uint16_t* p, int64_t rows, int64_t cols, int64_t ld) {
    if (!p) return fail(-1, "null pointer argument");
    if (!aligned(p, 16)) return fail(-1, "misaligned pointer (16 B for arrays, 256 B for the workspace)");
    if (ld < cols) return fail(-1, "a leading dimension is smaller than its row");
    if (ld % 8 != 0) return fail(-1, "leading dimensions must be multiples of 8 elements");
    if (reaches_4gib(rows, ld)) return fail(-2, "an operand reaches 4 GiB");
    return 0;
}

// The sizes of a qlora_head_loss call, and its plan.
int head_sizes(int64_t vocab, int64_t d_in, int64_t ldw, int64_t d_seq, bool nf4, bool grad, qn::HeadPlan* p) {
    if (vocab < 1 || d_in < 1 || d_seq < 1) return fail(-1, "sizes must be >= 1");
    if (d_in % 64 != 0 || (nf4 && vocab % 64 != 0)) return fail(-2, "d_in (and an NF4 head's rows) must be multiples of 64");
    if (d_in > INT32_MAX / 2 || vocab > INT32_MAX / 2 || d_seq > INT32_MAX / 2) return fail(-2, "dimension too large");
    int64_t n, n_b, n_g;
    if (!nf4_counts(vocab, d_in, &n, &n_b, &n_g)) return fail(-2, "weight too large");
    if (reaches_4gib(d_seq, d_in) || !qn::head_plan(vocab, d_in, ldw, d_seq, nf4, grad, p))
        return fail(-2, "an operand reaches 4 GiB");
    return 0;
}

int check_workspace(const void* ws, int64_t given, int64_t need) {
    if (!ws) return fail(-1, "null pointer argument");
    if (!aligned(ws, 256)) return fail(-1, "misaligned pointer (16 B for arrays, 256 B for the workspace)");
    if (given < need) return fail(-3, "workspace too small");
    return 0;
}
}  // namespace

namespace qn {
// polls a persistent one-token GEMV workgroup makes for each published A x slice word
// before forming every slice itself (process-wide, gemv.hip); returns the previous value
int set_ax_polls(int polls);
}  // namespace qn

// ---- scratch of the allocation-free forward ---------------------------------
// One static device array (each device holds its own copy, from module load until the
// process ends). Host code never uses the array's name as an address: the address of
// each device's copy is taken once with hipGetSymbolAddress, with that device current,
// and kept per device.
namespace {
constexpr int64_t kNoAllocScratchBytes = QN_NOALLOC_SCRATCH_BYTES;
static_assert(kNoAllocScratchBytes % 256 == 0, "scratch size");

static __device__ __align__(256) char scratch[kNoAllocScratchBytes];

constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
char* g_scratch_ptr[kMaxDevices] = {};

// The current device's copy of `scratch` (nullptr and the error text set on failure).
char* scratch_of_current_device() {
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) {
        hip_fail(e, "hipGetDevice");
        return nullptr;
    }
    if (dev < 0 || dev >= kMaxDevices) {
        fail(-4, "device index out of range");
        return nullptr;
    }
    std::lock_guard<std::mutex> lk(g_scratch_mu);
    if (g_scratch_ptr[dev] == nullptr) {
        void* p = nullptr;
        e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (e != hipSuccess || p == nullptr) {
            hip_fail(e != hipSuccess ? e : hipErrorInvalidSymbol, "hipGetSymbolAddress(scratch)");
            return nullptr;
        }
        g_scratch_ptr[dev] = static_cast<char*>(p);
    }
    return g_scratch_ptr[dev];
}
}  // namespace

extern "C" {

int qn_profile_enable(int on) {
    std::lock_guard<std::mutex> lk(qn::g_prof_mu);
    qn::prof_clear_locked();
    while (on && qn::g_pool.size() < qn::kPoolPrefill) {
        hipEvent_t e = nullptr;
        const hipError_t err = hipEventCreate(&e);
        if (err != hipSuccess) return hip_fail(err, "qn_profile_enable");
        qn::g_pool.push_back(e);
    }
    qn::g_prof_on.store(on != 0);
    return 0;
}

int qn_profile_read(char* names, int name_len, int64_t* launches, double* total_ms, int cap) {
    if (!names || !launches || !total_ms || name_len < 2 || cap < 0) return fail(-1, "bad argument");
    std::lock_guard<std::mutex> lk(qn::g_prof_mu);
    std::map<std::string, std::pair<int64_t, double>> agg;
    for (auto& r : qn::g_prof) {
        hipError_t e = hipEventSynchronize(r.stop);
        if (e != hipSuccess) return hip_fail(e, "qn_profile_read");
        float ms = 0.0f;
        e = hipEventElapsedTime(&ms, r.start, r.stop);
        if (e != hipSuccess) return hip_fail(e, "qn_profile_read");
        auto& a = agg[r.name];
        a.first += 1;
        a.second += ms;
    }
    int i = 0;
    for (auto& kv : agg) {
        if (i >= cap) break;
        std::strncpy(names + static_cast<size_t>(i) * name_len, kv.first.c_str(), name_len - 1);
        names[static_cast<size_t>(i) * name_len + name_len - 1] = 0;
        launches[i] = kv.second.first;
        total_ms[i] = kv.second.second;
        ++i;
    }
    return static_cast<int>(agg.size());
}

int qn_profile_durations(const char* name, float* ms, int cap) {
    if (!name || (!ms && cap > 0) || cap < 0) return fail(-1, "bad argument");
    std::lock_guard<std::mutex> lk(qn::g_prof_mu);
    int n = 0;
    for (auto& r : qn::g_prof) {
        if (std::strcmp(r.name, name) != 0) continue;
        hipError_t e = hipEventSynchronize(r.stop);
        if (e != hipSuccess) return hip_fail(e, "qn_profile_durations");
        float t = 0.0f;
        e = hipEventElapsedTime(&t, r.start, r.stop);
        if (e != hipSuccess) return hip_fail(e, "qn_profile_durations");
        if (n < cap) ms[n] = t;
        ++n;
    }
    return n;
}

int qn_version(void) { return 100; }

const char* qn_last_error(void) { return g_err.c_str(); }

int qn_codebook(float* out16) {
    if (!out16) return fail(-1, "null pointer argument");
    std::memcpy(out16, qn::tables().code, sizeof(float) * 16);
    return 0;
}

int qn_nf4_sizes(int64_t d_out, int64_t d_in, int64_t* codes_bytes, int64_t* n_blocks, int64_t* n_groups) {
    int64_t n, n_b, n_g;
    if (!nf4_counts(d_out, d_in, &n, &n_b, &n_g)) return fail(-1, "bad weight shape");
    if (codes_bytes) *codes_bytes = n_b * (qn::kBlock / 2);
    if (n_blocks) *n_blocks = n_b;
    if (n_groups) *n_groups = n_g;
    return 0;
}

int qn_nf4_sizes_ex(int64_t d_out, int64_t d_in, int dq, int64_t* codes_bytes, int64_t* qconst_entries,
                    int64_t* qscale_entries) {
    if (dq != QN_DQ_INT8 && dq != QN_DQ_FP8 && dq != QN_DQ_NONE) return fail(-1, "unknown second-level format");
    int64_t n, n_b, n_g;
    if (!nf4_counts(d_out, d_in, &n, &n_b, &n_g)) return fail(-1, "bad weight shape");
    if (codes_bytes) *codes_bytes = n_b * (qn::kBlock / 2);
    if (qconst_entries) *qconst_entries = dq == QN_DQ_NONE ? 0 : n_b;
    if (qscale_entries) *qscale_entries = dq == QN_DQ_NONE ? n_b : n_g;
    return 0;
}

int64_t nf4_quantize_workspace_bytes(int64_t d_out, int64_t d_in) {
    int64_t n, n_b, n_g;
    if (!nf4_counts(d_out, d_in, &n, &n_b, &n_g)) return 0;
    return quant_ws(n_b).bytes;
}

int nf4_quantize_ex(const float* W, int64_t d_out, int64_t d_in, int dq, uint8_t* codes, int8_t* qconst,
                    float* qscale, float* qmean, void* workspace, int64_t workspace_bytes, void* stream) {
    if (!W || !workspace) return fail(-1, "null pointer argument");
    qn::BlockConsts bc;
    if (int rc = make_consts(dq, codes, qconst, qscale, qmean, &bc)) return rc;
    int64_t n, n_b, n_g;
    if (!nf4_counts(d_out, d_in, &n, &n_b, &n_g)) return fail(-1, "bad weight shape");
    if (!aligned(W, 16) || !aligned(codes, 16) || !aligned(workspace, 256)) return fail(-1, "misaligned pointer");
    const QuantWs w = quant_ws(n_b);
    if (workspace_bytes < w.bytes) return fail(-3, "workspace too small");
    char* ws = static_cast<char*>(workspace);
    hipError_t e = qn::launch_quantize(W, n, n_b, n_g, bc.fmt, codes, qconst, qscale, qmean,
                                       reinterpret_cast<float*>(ws + w.absmax_off),
                                       reinterpret_cast<unsigned long long*>(ws + w.limbs_off), w.grid,
                                       static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "nf4_quantize");
    return 0;
}

int nf4_quantize(const float* W, int64_t d_out, int64_t d_in, uint8_t* codes, int8_t* qconst,
                 float* qscale, float* qmean, void* workspace, int64_t workspace_bytes, void* stream) {
    return nf4_quantize_ex(W, d_out, d_in, QN_DQ_INT8, codes, qconst, qscale, qmean, workspace, workspace_bytes,
                           stream);
}

int nf4_double_dequant_ex(const uint8_t* codes, const int8_t* qconst, const float* qscale, const float* qmean,
                          int64_t d_out, int64_t d_in, int dq, uint16_t* W_bf16, void* stream) {
    qn::BlockConsts bc;
    if (int rc = make_consts(dq, codes, qconst, qscale, qmean, &bc)) return rc;
    if (!W_bf16) return fail(-1, "null pointer argument");
    int64_t n, n_b, n_g;
    if (!nf4_counts(d_out, d_in, &n, &n_b, &n_g)) return fail(-1, "bad weight shape");
    if (!aligned(codes, 16) || !aligned(W_bf16, 16)) return fail(-1, "misaligned pointer");
    hipError_t e = qn::launch_dequant_rows(codes, bc, n, W_bf16, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "nf4_double_dequant");
    return 0;
}

int nf4_double_dequant(const uint8_t* codes, const int8_t* qconst, const float* qscale, const float* qmean,
                       int64_t d_out, int64_t d_in, uint16_t* W_bf16, void* stream) {
    return nf4_double_dequant_ex(codes, qconst, qscale, qmean, d_out, d_in, QN_DQ_INT8, W_bf16, stream);
}

int64_t qlora_linear_workspace_bytes(int64_t d_out, int64_t d_in, int64_t d_seq, int r) {
    if (!linear_sizes_ok(d_out, d_in, d_seq, r)) return 0;
    return std::max(linear_ws(d_out, d_in, d_seq, r, false).bytes, linear_ws(d_out, d_in, d_seq, r, true).bytes);
}

int64_t qlora_linear_fwd_workspace_bytes(int64_t d_out, int64_t d_in, int64_t d_seq, int r) {
    if (!linear_sizes_ok(d_out, d_in, d_seq, r)) return 0;
    return linear_ws(d_out, d_in, d_seq, r, false).bytes;
}

int64_t qlora_linear_bwd_x_workspace_bytes(int64_t d_out, int64_t d_in, int64_t d_seq, int r) {
    if (!linear_sizes_ok(d_out, d_in, d_seq, r)) return 0;
    return linear_ws(d_out, d_in, d_seq, r, true).bytes;
}

int qlora_linear_fwd_ex(const uint8_t* codes, const int8_t* qconst, const float* qscale, const float* qmean,
                        int64_t d_out, int64_t d_in, int dq, const uint16_t* A, const uint16_t* B, int r, float s,
                        const uint16_t* X, int64_t ldx, int64_t d_seq, uint16_t* Y, int64_t ldy, void* workspace,
                        int64_t workspace_bytes, void* stream) {
    LinWs lw;
    qn::BlockConsts bc;
    int rc = check_linear(codes, qconst, qscale, qmean, dq, d_out, d_in, A, B, r, X, ldx, d_seq, Y, ldy, false,
                          workspace, workspace_bytes, &lw, &bc);
    if (rc) return rc;
    return linear_fwd_run(codes, bc, d_out, d_in, A, B, r, s, X, ldx, d_seq, Y, ldy, static_cast<char*>(workspace),
                          lw, static_cast<hipStream_t>(stream));
}

int qlora_set_ax_wait(int polls) {
    if (polls < 0) return -1;
    return qn::set_ax_polls(polls);
}

int qlora_set_fwd_gemm(int form) {
    if (form != QN_FWD_GEMM_AUTO && form != QN_FWD_GEMM_STAGED && form != QN_FWD_GEMM_FUSED) return -1;
    return g_fwd_gemm.exchange(form);
}

int qlora_linear_fwd(const uint8_t* codes, const int8_t* qconst, const float* qscale, const float* qmean,
                     int64_t d_out, int64_t d_in, const uint16_t* A, const uint16_t* B, int r, float s,
                     const uint16_t* X, int64_t ldx, int64_t d_seq, uint16_t* Y, int64_t ldy, void* workspace,
                     int64_t workspace_bytes, void* stream) {
    return qlora_linear_fwd_ex(codes, qconst, qscale, qmean, d_out, d_in, QN_DQ_INT8, A, B, r, s, X, ldx, d_seq, Y,
                               ldy, workspace, workspace_bytes, stream);
}

int qlora_linear_fwd_noalloc(const uint8_t* codes, const int8_t* qconst, const float* qscale, const float* qmean,
                             int64_t d_out, int64_t d_in, int dq, const uint16_t* A, const uint16_t* B, int r,
                             float s, const uint16_t* X, int64_t ldx, int64_t d_seq, uint16_t* Y, int64_t ldy,
                             void* stream) {
    if (d_seq < 1) return fail(-1, "sizes must be >= 1");
    if (d_seq > qn::kSkinnyMaxTokens)
        return fail(-2, "qlora_linear_fwd_noalloc takes at most 64 tokens (more would dequantise W into scratch)");
    char* ws = scratch_of_current_device();
    if (ws == nullptr) return -4;
    LinWs lw;
    qn::BlockConsts bc;
    int rc = check_linear(codes, qconst, qscale, qmean, dq, d_out, d_in, A, B, r, X, ldx, d_seq, Y, ldy, false, ws,
                          kNoAllocScratchBytes, &lw, &bc);
    if (rc == -3) return fail(-2, "qlora_linear_fwd_noalloc: these sizes need more than the static scratch holds");
    if (rc) return rc;
    return linear_fwd_run(codes, bc, d_out, d_in, A, B, r, s, X, ldx, d_seq, Y, ldy, ws, lw,
                          static_cast<hipStream_t>(stream));
}

int qlora_linear_bwd_x_ex(const uint8_t* codes, const int8_t* qconst, const float* qscale, const float* qmean,
                          int64_t d_out, int64_t d_in, int dq, const uint16_t* A, const uint16_t* B, int r,
                          float s, const uint16_t* dY, int64_t lddy, int64_t d_seq, uint16_t* dX, int64_t lddx,
                          void* workspace, int64_t workspace_bytes, void* stream) {
    LinWs lw;
    qn::BlockConsts bc;
    int rc = check_linear(codes, qconst, qscale, qmean, dq, d_out, d_in, A, B, r, dY, lddy, d_seq, dX, lddx, true,
                          workspace, workspace_bytes, &lw, &bc);
    if (rc) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    uint16_t* whatT = reinterpret_cast<uint16_t*>(ws + lw.what);
    uint16_t* u = reinterpret_cast<uint16_t*>(ws + lw.lora);
    uint16_t* atpad = reinterpret_cast<uint16_t*>(ws + lw.adapt);
    uint16_t* bt = reinterpret_cast<uint16_t*>(ws + lw.adapt2);
    hipError_t e;
    // the pre-pass reads B itself (k-major) where it can; else K-contiguous rows of B^T
    const bool km = qn::prepass_takes_kmajor(r);
    if (!km && (e = qn::launch_transpose_pad(B, d_out, r, bt, d_out, st)) != hipSuccess)
        return hip_fail(e, "qlora_linear_bwd_x (B^T)");
    // dequant W_hat^T + U = s (dY B) + A^T padded to r_pad columns, in one launch
    if ((e = qn::launch_prologue(codes, bc, d_out, d_in, true, whatT, dY, lddy, d_seq, d_out,
                                 km ? B : bt, d_out, km, r, s, u, lw.r_pad, 2, A, atpad, r, d_in,
                                 reinterpret_cast<float*>(ws + lw.ppart), st)) != hipSuccess)
        return hip_fail(e, "qlora_linear_bwd_x (prologue)");
    if ((e = qn::launch_gemm_nt(dY, lddy, whatT, d_out, d_out, u, lw.r_pad, atpad, lw.r_pad, lw.r_pad, dX,
                                lddx, d_seq, d_in, reinterpret_cast<float*>(ws + lw.gpart), st)) != hipSuccess)
        return hip_fail(e, "qlora_linear_bwd_x (gemm)");
    return 0;
}

int qlora_linear_bwd_x(const uint8_t* codes, const int8_t* qconst, const float* qscale, const float* qmean,
                       int64_t d_out, int64_t d_in, const uint16_t* A, const uint16_t* B, int r, float s,
                       const uint16_t* dY, int64_t lddy, int64_t d_seq, uint16_t* dX, int64_t lddx, void* workspace,
                       int64_t workspace_bytes, void* stream) {
    return qlora_linear_bwd_x_ex(codes, qconst, qscale, qmean, d_out, d_in, QN_DQ_INT8, A, B, r, s, dY, lddy, d_seq,
                                 dX, lddx, workspace, workspace_bytes, stream);
}

// ---- quantised low-rank factors (W ~ Q + L R) --------------------------------
int int8_quantize(const float* W, int64_t rows, int64_t cols, int8_t* q, float* absmax, void* stream) {
    if (!W || !q || !absmax) return fail(-1, "null pointer argument");
    int64_t n, n_b, n_g;
    if (!nf4_counts(rows, cols, &n, &n_b, &n_g)) return fail(-1, "bad shape");
    if (!aligned(W, 16) || !aligned(q, 16) || !aligned(absmax, 4)) return fail(-1, "misaligned pointer");
    hipError_t e = qn::launch_int8_quantize(W, n, q, absmax, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "int8_quantize");
    return 0;
}

int int8_dequant(const int8_t* q, const float* absmax, int64_t rows, int64_t cols, uint16_t* W_bf16, void* stream) {
    if (!q || !absmax || !W_bf16) return fail(-1, "null pointer argument");
    int64_t n, n_b, n_g;
    if (!nf4_counts(rows, cols, &n, &n_b, &n_g)) return fail(-1, "bad shape");
    if (!aligned(q, 16) || !aligned(absmax, 4) || !aligned(W_bf16, 16)) return fail(-1, "misaligned pointer");
    hipError_t e = qn::launch_int8_dequant(q, absmax, n, W_bf16, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "int8_dequant");
    return 0;
}

int64_t qlr_linear_workspace_bytes(int64_t d_out, int64_t d_in, int64_t d_seq, int r) {
    if (!linear_sizes_ok(d_out, d_in, d_seq, r)) return 0;
    return linear_ws(d_out, d_in, d_seq, r, false).bytes + align_up(2 * r * d_in, 256) + align_up(2 * d_out * r, 256);
}

int qlr_linear_fwd(const uint8_t* codes, const int8_t* qconst, const float* qscale, const float* qmean,
                   int64_t d_out, int64_t d_in, int dq, int a_bits, const void* a_codes, const float* a_scale,
                   int b_bits, const void* b_codes, const float* b_scale, int r, float s, const uint16_t* X,
                   int64_t ldx, int64_t d_seq, uint16_t* Y, int64_t ldy, void* workspace, int64_t workspace_bytes,
                   void* stream) {
    if ((a_bits != 4 && a_bits != 8) || (b_bits != 4 && b_bits != 8)) return fail(-1, "factor bits must be 4 or 8");
    if (!a_codes || !a_scale || !b_codes || !b_scale) return fail(-1, "null pointer argument");
    if (!aligned(a_codes, 16) || !aligned(b_codes, 16) || !aligned(a_scale, 4) || !aligned(b_scale, 4))
        return fail(-1, "misaligned pointer");
    if (!linear_sizes_ok(d_out, d_in, d_seq, r)) return fail(-1, "sizes must be >= 1, r <= 256");
    // the dequantised factors sit after the forward's workspace (A [r, d_in], then B [d_out, r])
    const LinWs lw0 = linear_ws(d_out, d_in, d_seq, r, false);
    if (workspace_bytes < qlr_linear_workspace_bytes(d_out, d_in, d_seq, r)) return fail(-3, "workspace too small");
    char* ws = static_cast<char*>(workspace);
    uint16_t* a_hat = reinterpret_cast<uint16_t*>(ws + lw0.bytes);
    uint16_t* b_hat = reinterpret_cast<uint16_t*>(ws + lw0.bytes + align_up(2 * r * d_in, 256));
    LinWs lw;
    qn::BlockConsts bc;
    int rc = check_linear(codes, qconst, qscale, qmean, dq, d_out, d_in, a_hat, b_hat, r, X, ldx, d_seq, Y, ldy,
                          false, workspace, workspace_bytes, &lw, &bc);
    if (rc) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    hipError_t e;
    struct { int bits; const void* codes; const float* scale; int64_t n; uint16_t* out; } f[2] = {
        {a_bits, a_codes, a_scale, static_cast<int64_t>(r) * d_in, a_hat},
        {b_bits, b_codes, b_scale, d_out * static_cast<int64_t>(r), b_hat}};
    for (auto& fa : f) {
        if (fa.bits == 4) {
            const uint8_t* c = static_cast<const uint8_t*>(fa.codes);
            e = qn::launch_dequant_rows(c, qn::BlockConsts{reinterpret_cast<const int8_t*>(c), fa.scale, fa.scale,
                                                           qn::kDqNone, 0},
                                        fa.n, fa.out, st);
        } else {
            e = qn::launch_int8_dequant(static_cast<const int8_t*>(fa.codes), fa.scale, fa.n, fa.out, st);
        }
        if (e != hipSuccess) return hip_fail(e, "qlr_linear_fwd (factors)");
    }
    return linear_fwd_run(codes, bc, d_out, d_in, a_hat, b_hat, r, s, X, ldx, d_seq, Y, ldy, ws, lw, st);
}

// ---- adapter gradients ----------------------------------------------------

int64_t qlora_lora_grads_workspace_bytes(int64_t d_out, int64_t d_in, int64_t d_seq, int r) {
    if (d_out < 1 || d_in < 1 || d_seq < 1 || r < 1 || r > 256) return 0;
    return grad_ws(d_out, d_in, d_seq, r).bytes;
}

int qlora_lora_grads(const uint16_t* A, const uint16_t* B, int r, float s, const uint16_t* X, int64_t ldx,
                     const uint16_t* dY, int64_t lddy, int64_t d_out, int64_t d_in, int64_t d_seq, float* dA,
                     float* dB, void* workspace, int64_t workspace_bytes, void* stream) {
    if (!A || !B || !X || !dY || !dA || !dB || !workspace) return fail(-1, "null pointer argument");
    if (d_out < 1 || d_in < 1 || d_seq < 1) return fail(-1, "sizes must be >= 1");
    if (r < 1 || r > 256) return fail(-1, "r must be in [1, 256]");
    if (ldx < d_in || lddy < d_out) return fail(-1, "a leading dimension is smaller than its row");
    if (ldx % 8 != 0 || lddy % 8 != 0) return fail(-1, "leading dimensions must be multiples of 8 elements");
    if (!aligned(A, 16) || !aligned(B, 16) || !aligned(X, 16) || !aligned(dY, 16) || !aligned(dA, 16) ||
        !aligned(dB, 16) || !aligned(workspace, 256))
        return fail(-1, "misaligned pointer (16 B for arrays, 256 B for the workspace)");
    if (d_in % 64 != 0 || d_out % 64 != 0) return fail(-2, "d_in and d_out must be multiples of 64");
    if (d_in > INT32_MAX || d_out > INT32_MAX || d_seq > INT32_MAX) return fail(-2, "dimension too large");
    if (reaches_4gib(d_seq, std::max(ldx, lddy))) return fail(-2, "an operand reaches 4 GiB");
    const GradWs gw = grad_ws(d_out, d_in, d_seq, r);
    if (workspace_bytes < gw.bytes) return fail(-3, "workspace too small");
    hipStream_t st = static_cast<hipStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    uint16_t* tp = reinterpret_cast<uint16_t*>(ws + gw.tp);
    uint16_t* up = reinterpret_cast<uint16_t*>(ws + gw.up);
    uint16_t* bt = reinterpret_cast<uint16_t*>(ws + gw.bt);
    float* part = reinterpret_cast<float*>(ws + gw.part);
    hipError_t e;
    // T' = bf16(s X A^T) and U' = bf16(s dY B): the forward's and the input gradient's
    // pre-passes (without the dequantisation) in one launch; U' on B itself where it can
    const bool km = qn::prepass_takes_kmajor(r);
    if (!km && (e = qn::launch_transpose_pad(B, d_out, r, bt, d_out, st)) != hipSuccess)
        return hip_fail(e, "qlora_lora_grads (B^T)");
    if ((e = qn::launch_prepass_pair(X, ldx, d_in, A, d_in, tp, reinterpret_cast<float*>(ws + gw.ppart),
                                     dY, lddy, d_out, km ? B : bt, d_out, km, up,
                                     reinterpret_cast<float*>(ws + gw.ppart1), d_seq, r, s, gw.r_pad, st)) !=
        hipSuccess)
        return hip_fail(e, "qlora_lora_grads (X A^T, dY B)");
    if ((e = qn::launch_lora_grads(X, ldx, dY, lddy, tp, up, d_out, d_in, d_seq, r, gw.r_pad, part, dA, dB, st)) !=
        hipSuccess)
        return hip_fail(e, "qlora_lora_grads (reduction)");
    return 0;
}

// ---- many adapters on one layer -------------------------------------------------
namespace {

struct MultiWs {
    int64_t what, pre0, pre1, t, u, gpart, grads, part, part_t, bytes;
};

// Workspace of a multi-adapter call; regions a call does not use have size 0.
MultiWs multi_ws(int64_t d_out, int64_t d_in, int64_t M, int r, int n, bool bwd) {
    MultiWs w{};
    int64_t off = 0;
    auto take = [&](int64_t bytes) { const int64_t at = off; off += align_up(bytes, 256); return at; };
    if (!bwd && M <= qn::kSkinnyMaxTokens) {
        w.part = take(4 * static_cast<int64_t>(qn::multi_splits(d_out, d_in, M)) * M * d_out);    // W_hat x, K-split
        w.part_t = take(4 * static_cast<int64_t>(qn::multi_small_splits(d_in, M, n, r)) * M * r);    // A x, K-split
        w.bytes = off;
        return w;
    }
    // float32 sums of a pre-pass of several K-slices
    auto pre = [&](int64_t K) {
        const int sp = qn::multi_pre_split(M, K).splits;
        return take(sp > 1 ? 4 * static_cast<int64_t>(sp) * M * r : 0);
    };
    w.what = take(2 * d_out * d_in);                                                // W_hat or W_hat^T
    w.pre0 = pre(d_in);                                                             // A x
    w.t = take(2 * (bwd ? 3 : 2) * M * r);                                          // T = s A x
    if (bwd) {
        w.pre1 = pre(d_out);                                                        // B^T dy
        w.u = take(2 * 3 * M * r);                                                  // U = s B^T dy
        w.grads = take(4 * qn::multi_grads_part_floats(d_out, d_in, M, n, r));      // dA, dB partials
    }
    w.gpart = take(4 * (bwd ? qn::gemm_multi_part_floats(M, d_in, d_out) : qn::gemm_multi_part_floats(M, d_out, d_in)));
    w.bytes = off;
    return w;
}

// Sizes that check_multi takes with rows as short as they can be.
bool multi_sizes_ok(int64_t d_out, int64_t d_in, int64_t d_seq, int r, int n) {
    if (!linear_sizes_ok(d_out, d_in, d_seq, r) || n < 1 || n > QN_MULTI_MAX_ADAPTERS) return false;
    if (d_in % 64 != 0 || d_out % 64 != 0 || r % 16 != 0) return false;
    const int64_t wide = std::max(d_in, d_out);
    return !reaches_4gib(d_out, d_in) && !reaches_4gib(d_seq, std::max<int64_t>(wide, r)) && !reaches_4gib(wide, r);
}

static_assert(QN_MULTI_MAX_ADAPTERS == qn::kMultiMaxAdapters, "adapter limit");

int check_multi(const uint8_t* codes, const int8_t* qconst, const float* qscale, const float* qmean, int dq,
                int64_t d_out, int64_t d_in, const uint16_t* A, const uint16_t* B, const float* s, int n, int r,
                const uint16_t* X, int64_t ldx, const uint16_t* dY, int64_t lddy, int64_t d_seq, const void* plan,
                uint16_t* out, int64_t ldo, bool bwd, void* ws, int64_t ws_bytes, MultiWs* mw, qn::BlockConsts* bc) {
    if (int rc = make_consts(dq, codes, qconst, qscale, qmean, bc)) return rc;
    if (!A || !B || !s || !X || (bwd && !dY) || !plan || !out || !ws) return fail(-1, "null pointer argument");
    if (d_out < 1 || d_in < 1 || d_seq < 1) return fail(-1, "sizes must be >= 1");
    if (n < 1) return fail(-1, "the pool must hold at least one adapter");
    if (r < 1 || r > 256) return fail(-1, "r must be in [1, 256]");
    const int64_t out_cols = bwd ? d_in : d_out;
    if (ldx < d_in || ldo < out_cols || (bwd && lddy < d_out))
        return fail(-1, "a leading dimension is smaller than its row");
    if (ldx % 8 != 0 || ldo % 8 != 0 || (bwd && lddy % 8 != 0))
        return fail(-1, "leading dimensions must be multiples of 8 elements");
    if (!aligned(codes, 16) || !aligned(A, 16) || !aligned(B, 16) || !aligned(s, 4) || !aligned(X, 16) ||
        !aligned(dY, 16) || !aligned(plan, 16) || !aligned(out, 16) || !aligned(ws, 256))
        return fail(-1, "misaligned pointer (16 B for arrays, 256 B for the workspace)");
    if (d_in % 64 != 0 || d_out % 64 != 0) return fail(-2, "d_in and d_out must be multiples of 64");
    if (r % 16 != 0) return fail(-2, "the pool's rank must be a multiple of 16");
    if (n > QN_MULTI_MAX_ADAPTERS) return fail(-2, "too many adapters in the pool");
    if (d_in > INT32_MAX || d_out > INT32_MAX || d_seq > INT32_MAX) return fail(-2, "dimension too large");
    int64_t cnt, n_b, n_g;
    if (!nf4_counts(d_out, d_in, &cnt, &n_b, &n_g)) return fail(-2, "weight too large");
    if (reaches_4gib(d_out, d_in) || reaches_4gib(d_seq, std::max<int64_t>({ldx, ldo, bwd ? lddy : 0, r})) ||
        reaches_4gib(std::max(d_in, d_out), r))
        return fail(-2, "an operand reaches 4 GiB");
    *mw = multi_ws(d_out, d_in, d_seq, r, n, bwd);
    if (ws_bytes < mw->bytes) return fail(-3, "workspace too small");
    return 0;
}

}  // namespace

int64_t qlora_multi_plan_bytes(int64_t d_seq, int n) {
    if (d_seq < 1 || d_seq > INT32_MAX || n < 1 || n > QN_MULTI_MAX_ADAPTERS) return 0;
    return 4 * qn::multi_plan_words(d_seq, n);
}

int qlora_multi_plan(const int32_t* ids, int64_t d_seq, int n, void* plan, int64_t plan_bytes, void* stream) {
    if (!ids || !plan) return fail(-1, "null pointer argument");
    if (d_seq < 1 || n < 1) return fail(-1, "sizes must be >= 1");
    if (!aligned(ids, 4) || !aligned(plan, 16)) return fail(-1, "misaligned pointer");
    if (n > QN_MULTI_MAX_ADAPTERS) return fail(-2, "too many adapters in the pool");
    if (d_seq > INT32_MAX - 4096) return fail(-2, "dimension too large");
    if (plan_bytes < 4 * qn::multi_plan_words(d_seq, n)) return fail(-3, "plan buffer too small");
    hipError_t e = qn::launch_multi_plan(ids, d_seq, n, plan, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "qlora_multi_plan");
    return 0;
}

int64_t qlora_multi_fwd_workspace_bytes(int64_t d_out, int64_t d_in, int64_t d_seq, int r, int n) {
    return multi_sizes_ok(d_out, d_in, d_seq, r, n) ? multi_ws(d_out, d_in, d_seq, r, n, false).bytes : 0;
}

int64_t qlora_multi_bwd_workspace_bytes(int64_t d_out, int64_t d_in, int64_t d_seq, int r, int n) {
    return multi_sizes_ok(d_out, d_in, d_seq, r, n) ? multi_ws(d_out, d_in, d_seq, r, n, true).bytes : 0;
}

int qlora_multi_fwd(const uint8_t* codes, const int8_t* qconst, const float* qscale, const float* qmean,
                    int64_t d_out, int64_t d_in, int dq, const uint16_t* A, const uint16_t* B, const float* s, int n,
                    int r, const uint16_t* X, int64_t ldx, int64_t d_seq, const void* plan, uint16_t* Y, int64_t ldy,
                    void* workspace, int64_t workspace_bytes, void* stream) {
    MultiWs mw;
    qn::BlockConsts bc;
    int rc = check_multi(codes, qconst, qscale, qmean, dq, d_out, d_in, A, B, s, n, r, X, ldx, nullptr, 0, d_seq, plan,
                         Y, ldy, false, workspace, workspace_bytes, &mw, &bc);
    if (rc) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    auto f32 = [&](int64_t off) { return reinterpret_cast<float*>(ws + off); };
    auto u16 = [&](int64_t off) { return reinterpret_cast<uint16_t*>(ws + off); };
    const qn::MultiPlan pl = qn::multi_plan_at(plan, d_seq, n);
    hipError_t e;
    if (d_seq <= qn::kSkinnyMaxTokens) {
        e = qn::launch_multi_small(codes, bc, d_out, d_in, qn::MultiPool{A, B, s, n, r}, X, ldx, d_seq, pl, f32(mw.part),
                                   f32(mw.part_t), Y, ldy, st);
        if (e != hipSuccess) return hip_fail(e, "qlora_multi_fwd (small batch)");
        return 0;
    }
    if ((e = qn::launch_multi_prologue(codes, bc, d_out, d_in, false, u16(mw.what), pl, s, d_seq, n, r, 2,
                                       qn::MultiPre{X, ldx, d_in, A, f32(mw.pre0), u16(mw.t)}, qn::MultiPre{}, st)) !=
        hipSuccess)
        return hip_fail(e, "qlora_multi_fwd (prologue)");
    if ((e = qn::launch_gemm_multi(X, ldx, u16(mw.what), d_in, u16(mw.t), B, false, r, pl, Y, ldy, d_seq, d_out,
                                   f32(mw.gpart), st)) != hipSuccess)
        return hip_fail(e, "qlora_multi_fwd (gemm)");
    return 0;
}

int qlora_multi_bwd(const uint8_t* codes, const int8_t* qconst, const float* qscale, const float* qmean,
                    int64_t d_out, int64_t d_in, int dq, const uint16_t* A, const uint16_t* B, const float* s, int n,
                    int r, const uint16_t* X, int64_t ldx, const uint16_t* dY, int64_t lddy, int64_t d_seq,
                    const void* plan, uint16_t* dX, int64_t lddx, float* dA, float* dB, void* workspace,
                    int64_t workspace_bytes, void* stream) {
    if (!dA || !dB) return fail(-1, "null pointer argument");
    if (!aligned(dA, 16) || !aligned(dB, 16)) return fail(-1, "misaligned pointer (16 B for arrays, 256 B for the workspace)");
    MultiWs mw;
    qn::BlockConsts bc;
    int rc = check_multi(codes, qconst, qscale, qmean, dq, d_out, d_in, A, B, s, n, r, X, ldx, dY, lddy, d_seq, plan, dX,
                         lddx, true, workspace, workspace_bytes, &mw, &bc);
    if (rc) return rc;
    hipStream_t st = static_cast<hipStream_t>(stream);
    char* ws = static_cast<char*>(workspace);
    auto f32 = [&](int64_t off) { return reinterpret_cast<float*>(ws + off); };
    auto u16 = [&](int64_t off) { return reinterpret_cast<uint16_t*>(ws + off); };
    const qn::MultiPlan pl = qn::multi_plan_at(plan, d_seq, n);
    hipError_t e;
    if ((e = qn::launch_multi_prologue(codes, bc, d_out, d_in, true, u16(mw.what), pl, s, d_seq, n, r, 3,
                                       qn::MultiPre{X, ldx, d_in, A, f32(mw.pre0), u16(mw.t)},
                                       qn::MultiPre{dY, lddy, d_out, B, f32(mw.pre1), u16(mw.u)}, st)) != hipSuccess)
        return hip_fail(e, "qlora_multi_bwd (prologue)");
    if ((e = qn::launch_gemm_multi(dY, lddy, u16(mw.what), d_out, u16(mw.u), A, true, r, pl, dX, lddx, d_seq, d_in,
                                   f32(mw.gpart), st)) != hipSuccess)
        return hip_fail(e, "qlora_multi_bwd (gemm)");
    if ((e = qn::launch_multi_grads(pl, X, ldx, dY, lddy, u16(mw.t), u16(mw.u), d_out, d_in, d_seq, n, r, f32(mw.grads),
                                    dA, dB, st)) != hipSuccess)
        return hip_fail(e, "qlora_multi_bwd (adapter gradients)");
    return 0;
}

// ---- AdamW over many tensors --------------------------------------------------

int64_t qlora_adamw_blocks(const int64_t* n, int count) {
    if (count < 0 || (!n && count > 0)) return fail(-1, "bad tensor list");
    int64_t b = 0;
    for (int i = 0; i < count; ++i) {
        if (n[i] < 0 || n[i] > (int64_t{1} << 40)) return fail(-1, "bad tensor size");
        b += (n[i] + qn::kAdamBlock - 1) / qn::kAdamBlock;
    }
    return b;
}

int64_t qlora_adamw_table_bytes(const int64_t* n, int count) {
    if (qlora_adamw_blocks(n, count) < 0) return -1;
    int64_t chunks = 0;
    for (int i = 0; i < count; ++i) chunks += (n[i] + qn::kAdamChunk - 1) / qn::kAdamChunk;
    return static_cast<int64_t>(sizeof(qn::AdamTensor)) * count + static_cast<int64_t>(sizeof(qn::AdamChunk)) * chunks;
}

int64_t qlora_adamw_table(void* const* p, const void* const* g, uint16_t* const* copy, const int64_t* n, int count,
                          int flags, void* table) {
    if (!table && count > 0) return fail(-1, "null pointer argument");
    if (count > 0 && (!p || !g)) return fail(-1, "null pointer argument");
    if (flags & ~7) return fail(-1, "unknown flags");
    if (qlora_adamw_blocks(n, count) < 0) return -1;
    int64_t need = 0;
    for (int i = 0; i < count; ++i) need += (n[i] + qn::kAdamChunk - 1) / qn::kAdamChunk;
    if (need > qn::kAdamMaxChunks) return fail(-1, "too many elements");
    const bool gb = flags & QN_ADAMW_GRAD_BF16, pb = flags & QN_ADAMW_PARAM_BF16;
    auto* t = static_cast<qn::AdamTensor*>(table);
    auto* c = reinterpret_cast<qn::AdamChunk*>(t + count);
    int64_t blocks = 0, chunks = 0;
    for (int i = 0; i < count; ++i) {
        uint16_t* cp = copy ? copy[i] : nullptr;
        if (n[i] > 0 && (!p[i] || !g[i])) return fail(-1, "null pointer argument");
        if (!aligned(p[i], pb ? 2 : 4) || !aligned(g[i], gb ? 2 : 4) || !aligned(cp, 2))
            return fail(-1, "misaligned pointer");
        const bool vec = aligned(p[i], pb ? 8 : 16) && aligned(g[i], gb ? 8 : 16) && aligned(cp, 8);
        t[i] = qn::AdamTensor{p[i], g[i], cp, n[i], blocks, vec ? 1 : 0};
        blocks += (n[i] + qn::kAdamBlock - 1) / qn::kAdamBlock;
        const int64_t nc = (n[i] + qn::kAdamChunk - 1) / qn::kAdamChunk;
        for (int64_t k = 0; k < nc; ++k) c[chunks + k] = qn::AdamChunk{i, static_cast<int32_t>(k)};
        chunks += nc;
    }
    return chunks;
}

int qlora_adamw_step(const void* table, int count, int64_t n_chunks, int flags, void* m, void* v, float* m_scale,
                     float* v_scale, int64_t step, const int64_t* step_dev, double lr, const float* lr_dev,
                     double beta1, double beta2, double eps, double weight_decay, const float* grad_scale,
                     uint32_t seed, void* stream) {
    if (count < 0 || n_chunks < 0 || n_chunks > qn::kAdamMaxChunks) return fail(-1, "bad tensor list");
    if (flags & ~7) return fail(-1, "unknown flags");
    const bool s8 = flags & QN_ADAMW_STATES_8;
    if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0)) return fail(-1, "betas must be in [0, 1)");
    if (!(static_cast<float>(eps) > 0.0f)) return fail(-1, "eps must be > 0 as a float32");
    if (!step_dev && step < 1) return fail(-1, "step must be >= 1");
    if (n_chunks == 0) return 0;
    if (!table || !m || !v || (s8 && (!m_scale || !v_scale))) return fail(-1, "null pointer argument");
    if (!aligned(table, 8) || !aligned(m, 16) || !aligned(v, 16) || !aligned(m_scale, 4) || !aligned(v_scale, 4) ||
        !aligned(step_dev, 8) || !aligned(lr_dev, 4) || !aligned(grad_scale, 4))
        return fail(-1, "misaligned pointer");
    qn::AdamArgs a{};
    a.tensors = static_cast<const qn::AdamTensor*>(table);
    a.chunks = reinterpret_cast<const qn::AdamChunk*>(a.tensors + count);
    a.m = m; a.v = v; a.m_scale = m_scale; a.v_scale = v_scale;
    a.grad_scale = grad_scale; a.lr_dev = lr_dev; a.step_dev = step_dev;
    a.lr = lr; a.beta1 = beta1; a.beta2 = beta2; a.weight_decay = weight_decay;
    a.step = step; a.eps = static_cast<float>(eps); a.seed = seed;
    hipError_t e = qn::launch_adamw(a, n_chunks, s8, flags & QN_ADAMW_GRAD_BF16, flags & QN_ADAMW_PARAM_BF16,
                                    static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "qlora_adamw_step");
    return 0;
}

int qlora_adamw_moments(const uint8_t* m, const float* m_scale, const uint8_t* v, const float* v_scale,
                        int64_t blocks, float* m_out, float* v_out, void* stream) {
    if (blocks < 0 || blocks > qn::kAdamMaxChunks * qn::kAdamChunkBlocks) return fail(-1, "bad block count");
    if (blocks == 0) return 0;
    if (!m || !m_scale || !v || !v_scale || !m_out || !v_out) return fail(-1, "null pointer argument");
    if (!aligned(m, 4) || !aligned(v, 4) || !aligned(m_scale, 4) || !aligned(v_scale, 4) || !aligned(m_out, 16) ||
        !aligned(v_out, 16))
        return fail(-1, "misaligned pointer");
    hipError_t e = qn::launch_adamw_moments(m, m_scale, v, v_scale, blocks, m_out, v_out,
                                            static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "qlora_adamw_moments");
    return 0;
}

int64_t qlora_gated_fwd_workspace_bytes(int64_t d_ff, int64_t d_in, int64_t d_seq, int r) {
    return gated_sizes_ok(d_ff, d_in, d_seq, r, false) ? gated_ws(d_ff, d_in, d_seq, r, false).bytes : 0;
}

int64_t qlora_gated_bwd_workspace_bytes(int64_t d_ff, int64_t d_in, int64_t d_seq, int r) {
    return gated_sizes_ok(d_ff, d_in, d_seq, r, true) ? gated_ws(d_ff, d_in, d_seq, r, true).bytes : 0;
}

int qlora_gated_fwd(const uint8_t* codes_g, const int8_t* qconst_g, const float* qscale_g, const float* qmean_g,
                    const uint8_t* codes_u, const int8_t* qconst_u, const float* qscale_u, const float* qmean_u,
                    int64_t d_ff, int64_t d_in, int dq, const uint16_t* A_g, const uint16_t* B_g, float s_g,
                    const uint16_t* A_u, const uint16_t* B_u, float s_u, int r, int act, const uint16_t* X, int64_t ldx,
                    int64_t d_seq, uint16_t* H, int64_t ldh, uint16_t* GU, int64_t ldgu, void* workspace,
                    int64_t workspace_bytes, void* stream) {
    qn::GatedCall c{};
    if (int rc = check_gated({codes_g, codes_u}, {qconst_g, qconst_u}, {qscale_g, qscale_u}, {qmean_g, qmean_u}, d_ff, d_in,
                             dq, {A_g, A_u}, {B_g, B_u}, {s_g, s_u}, r, act, d_seq, &c))
        return rc;
    if (int rc = check_rows(X, d_seq, d_in, ldx)) return rc;
    if (int rc = check_rows(H, d_seq, d_ff, ldh)) return rc;
    if (GU != nullptr)
        if (int rc = check_rows(GU, d_seq, 2 * d_ff, ldgu)) return rc;
    const GatedWs w = gated_ws(d_ff, d_in, d_seq, r, false);
    if (int rc = check_workspace(workspace, workspace_bytes, w.bytes)) return rc;
    char* ws = static_cast<char*>(workspace);
    hipStream_t st = static_cast<hipStream_t>(stream);
    if (d_seq <= qn::kGatedSmall) {
        const hipError_t es = qn::launch_gated_small(c, X, ldx, H, ldh, GU, ldgu, reinterpret_cast<float*>(ws + w.part), st);
        return es == hipSuccess ? 0 : hip_fail(es, "qlora_gated_fwd (small batch)");
    }
    qn::GatedProlog o{};
    o.what = reinterpret_cast<uint16_t*>(ws + w.what);
    o.adapt = reinterpret_cast<uint16_t*>(ws + w.adapt);
    o.in = X; o.ld_in = ldx;
    o.t = reinterpret_cast<uint16_t*>(ws + w.t);
    o.part = reinterpret_cast<float*>(ws + w.rpart);
    hipError_t e = qn::launch_gated_prologue(c, false, o, st);
    if (e != hipSuccess) return hip_fail(e, "qlora_gated_fwd (prologue)");
    e = qn::launch_gated_gemm(c, X, ldx, o.what, o.t, o.adapt, H, ldh, GU, ldgu, reinterpret_cast<float*>(ws + w.part),
                              st);
    if (e != hipSuccess) return hip_fail(e, "qlora_gated_fwd (gemm)");
    return 0;
}

int qlora_gated_bwd(const uint8_t* codes_g, const int8_t* qconst_g, const float* qscale_g, const float* qmean_g,
                    const uint8_t* codes_u, const int8_t* qconst_u, const float* qscale_u, const float* qmean_u,
                    int64_t d_ff, int64_t d_in, int dq, const uint16_t* A_g, const uint16_t* B_g, float s_g,
                    const uint16_t* A_u, const uint16_t* B_u, float s_u, int r, int act, const uint16_t* GU, int64_t ldgu,
                    const uint16_t* dH, int64_t lddh, int64_t d_seq, uint16_t* dGU, int64_t lddgu, uint16_t* dX,
                    int64_t lddx, void* workspace, int64_t workspace_bytes, void* stream) {
    qn::GatedCall c{};
    if (int rc = check_gated({codes_g, codes_u}, {qconst_g, qconst_u}, {qscale_g, qscale_u}, {qmean_g, qmean_u}, d_ff, d_in,
                             dq, {A_g, A_u}, {B_g, B_u}, {s_g, s_u}, r, act, d_seq, &c))
        return rc;
    if (int rc = check_rows(GU, d_seq, 2 * d_ff, ldgu)) return rc;
    if (int rc = check_rows(dH, d_seq, d_ff, lddh)) return rc;
    if (int rc = check_rows(dGU, d_seq, 2 * d_ff, lddgu)) return rc;
    if (int rc = check_rows(dX, d_seq, d_in, lddx)) return rc;
    if (dGU == GU && lddgu != ldgu && d_seq > 1) return fail(-1, "dGU in the place of GU needs GU's row stride");
    const GatedWs w = gated_ws(d_ff, d_in, d_seq, r, true);
    if (int rc = check_workspace(workspace, workspace_bytes, w.bytes)) return rc;
    char* ws = static_cast<char*>(workspace);
    hipStream_t st = static_cast<hipStream_t>(stream);
    // the elementwise part beside the layouts, the rank products of dG and dU, dX
    qn::GatedProlog o{};
    o.what = reinterpret_cast<uint16_t*>(ws + w.what);
    o.adapt = reinterpret_cast<uint16_t*>(ws + w.adapt);
    o.grad = qn::GatedGradArgs{dH, lddh, GU, ldgu, dGU, lddgu, static_cast<int>(d_seq), static_cast<int>(d_ff), act};
    o.in = dGU; o.ld_in = lddgu;
    o.t = reinterpret_cast<uint16_t*>(ws + w.t);
    o.part = reinterpret_cast<float*>(ws + w.rpart);
    if (!qn::gated_reads_b(r))
        for (int i = 0; i < 2; ++i) o.bt[i] = reinterpret_cast<uint16_t*>(ws + w.bt[i]);
    hipError_t e = qn::launch_gated_prologue(c, true, o, st);
    if (e != hipSuccess) return hip_fail(e, "qlora_gated_bwd (prologue)");
    e = qn::launch_gated_dx(c, dGU, lddgu, o.what, o.t, o.adapt, dX, lddx, reinterpret_cast<float*>(ws + w.part), st);
    if (e != hipSuccess) return hip_fail(e, "qlora_gated_bwd (gemm)");
    return 0;
}

int64_t qlora_head_loss_workspace_bytes(int64_t vocab, int64_t d_in, int64_t d_seq, int nf4, int grad) {
    qn::HeadPlan p;
    return head_sizes(vocab, d_in, d_in, d_seq, nf4 != 0, grad != 0, &p) == 0 ? p.bytes : 0;
}

int qlora_head_loss(const uint16_t* W, int64_t ldw, const uint8_t* codes, const int8_t* qconst, const float* qscale,
                    const float* qmean, int dq, int64_t vocab, int64_t d_in, const uint16_t* X, int64_t ldx, int64_t d_seq,
                    const int64_t* target, const float* scale, float* loss, uint16_t* dX, int64_t lddx, void* workspace,
                    int64_t workspace_bytes, void* stream) {
    qn::HeadCall c{};
    qn::HeadPlan p;
    if ((W == nullptr) == (codes == nullptr)) return fail(-1, "give the head as bf16 or as an NF4 weight");
    if (!target || !loss) return fail(-1, "null pointer argument");
    if (!aligned(target, 8) || !aligned(scale, 4) || !aligned(loss, 4)) return fail(-1, "misaligned pointer");
    if (codes != nullptr) {
        if (int rc = make_consts(dq, codes, qconst, qscale, qmean, &c.bc)) return rc;
        if (!aligned(codes, 16)) return fail(-1, "misaligned pointer (16 B for arrays, 256 B for the workspace)");
    }
    if (int rc = head_sizes(vocab, d_in, codes != nullptr ? d_in : ldw, d_seq, codes != nullptr, dX != nullptr, &p)) return rc;
    if (W != nullptr) {
        // a piece of the head is an operand; the head itself may be larger
        if (int rc = check_rows(W, std::min(vocab, p.piece), d_in, ldw)) return rc;
        if (ldw > (int64_t{1} << 46) / vocab) return fail(-2, "weight too large");
    }
    if (int rc = check_rows(X, d_seq, d_in, ldx)) return rc;
    if (dX != nullptr)
        if (int rc = check_rows(dX, d_seq, d_in, lddx)) return rc;
    if (int rc = check_workspace(workspace, workspace_bytes, p.bytes)) return rc;
    c.W = W; c.ldw = ldw; c.codes = codes; c.V = vocab; c.d = d_in;
    c.X = X; c.ldx = ldx; c.target = target; c.T = d_seq; c.scale = scale; c.loss = loss; c.dX = dX; c.lddx = lddx;
    const hipError_t e = qn::launch_head_loss(c, p, static_cast<char*>(workspace), static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return hip_fail(e, "qlora_head_loss");
    return 0;
}

}  // extern "C"
