"""The operators for many adapters over one shared NF4 projection, as measured cases.

Three operators, in the order a program that trains and serves several low-rank
adapters on one frozen 4-bit layer uses them:

  fwd    Y[t] = W_hat x[t] + s_a B_a (A_a x[t]),  a = ids[t]  (no adapter for a < 0)
  bwd    dX, and dA_a, dB_a of every adapter, for the loss gradient dY of that forward
  adamw  one AdamW step over all adapter tensors, moments in 32 bits or in 8

`own` chooses between the plain form (elementary torch operations in 32 bits) and the
package's calls on the same inputs.
"""
import math
import random

import numpy as np
import torch

own = False

# The NF4 code book (16 normal quantiles, both ends and an exact zero), float32 values.
CODE = [-1.0, -0.6962038278579712, -0.5250832438468933, -0.3949258327484131, -0.28444764018058777,
        -0.1847776174545288, -0.09105207771062851, 0.0, 0.07958215475082397, 0.16093382339241736,
        0.24611778557300568, 0.33792251348495483, 0.4407188892364502, 0.5626275539398193, 0.7229675054550171, 1.0]

BETA1, BETA2, EPS, DECAY, LR = 0.9, 0.999, 1e-8, 0.01, 2e-4
BLOCK = 256                    # elements per block of an 8-bit moment
M32 = 0xFFFFFFFF


def _dev():
    return torch.device("cuda", torch.cuda.current_device())


# ---- cases ---------------------------------------------------------------------------

def listed():
    def fwd(name, d_out, d_in, tokens, r, adapters, requests, base=0):
        return {"name": name, "op": "fwd", "d_out": d_out, "d_in": d_in, "tokens": tokens, "r": r,
                "adapters": adapters, "requests": requests, "base": base}

    def bwd(name, *a, **k):
        return dict(fwd(name, *a, **k), op="bwd")

    def adam(name, bits, layers, d, f, r, grad="float32", clip=True):
        return {"name": name, "op": "adamw", "bits": bits, "layers": layers, "d": d, "f": f, "r": r, "grad": grad,
                "clip": clip}

    return [
        # one user's next token on a 4096-wide projection: the smallest call, all latency
        fwd("fwd_one_token", 4096, 4096, 1, 16, 8, 1),
        # a decode batch, every token another user's, one of them without an adapter
        fwd("fwd_decode_24", 4096, 4096, 24, 16, 32, 24, base=1),
        # a full decode batch on the up projection with large ranks
        fwd("fwd_decode_64_r64", 11008, 4096, 64, 64, 48, 64, base=4),
        # packed prompts of uneven lengths, an odd number of tokens in all
        fwd("fwd_prompts_1531", 4096, 4096, 1531, 32, 24, 37, base=3),
        # long prompts of a few users
        fwd("fwd_prompts_4096", 4096, 4096, 4096, 16, 8, 8),
        # the check layer of the repository in training: small and ragged
        bwd("bwd_small", 256, 256, 203, 16, 3, 5, base=1),
        # a training batch of several adapters on the square layer
        bwd("bwd_4096", 4096, 4096, 4096, 16, 8, 11, base=1),
        # the down projection with large ranks
        bwd("bwd_mlp_r64", 4096, 11008, 2048, 64, 6, 9),
        # the adapter pair of the check layer: one launch's latency
        adam("adamw32_small", 32, 1, 256, 512, 16),
        # all adapters of a 32-layer model at rank 64, float32 moments
        adam("adamw32_large", 32, 32, 4096, 11008, 64),
        # adapters of 8 layers with odd rank (ragged blocks), bf16 gradients, 8-bit moments
        adam("adamw8_ragged", 8, 8, 4096, 11008, 9, grad="bfloat16"),
        # the large set with 8-bit moments
        adam("adamw8_large", 8, 32, 4096, 11008, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.34:
        return {"op": "adamw", "bits": rng.choice([8, 32]), "layers": _log(rng, 1, 16), "d": _log(rng, 200, 4096),
                "f": _log(rng, 500, 11008), "r": _log(rng, 4, 64), "grad": rng.choice(["float32", "bfloat16"]),
                "clip": rng.random() < 0.5}
    while True:
        d_out, d_in = 64 * _log(rng, 4, 172), 64 * _log(rng, 4, 172)
        tokens, r = _log(rng, 1, 4096), rng.choice([16, 32, 48, 64])
        adapters = _log(rng, 1, 64)
        if d_out * d_in * tokens <= 11008 * 4096 * 2048 and adapters * r <= 2048:
            break
    requests = tokens if tokens <= 64 and rng.random() < 0.7 else min(tokens, _log(rng, 1, 64))
    return {"op": rng.choice(["fwd", "fwd", "bwd"]), "d_out": d_out, "d_in": d_in, "tokens": tokens, "r": r,
            "adapters": adapters, "requests": requests, "base": rng.randrange(requests) // 4}


def _ids(case, seed):
    """The adapter of every token: requests of random lengths, one after the other; the
    adapters are dealt out in turn and shuffled, `base` requests have none."""
    rng = random.Random(seed)
    n, reqs, m = case["adapters"], case["requests"], case["tokens"]
    cuts = [0] + sorted(rng.sample(range(1, m), reqs - 1)) + [m]
    who = [i % n for i in range(reqs - case["base"])] + [-1] * case["base"]
    rng.shuffle(who)
    return np.repeat(np.array(who, np.int32), np.diff(cuts))


def _tensor_sizes(case):
    """Element counts of a model's adapters: A [r, in] and B [out, r] of 4 square, 2 up and
    1 down projections per layer."""
    d, f, r = case["d"], case["f"], case["r"]
    return ([r * d, d * r] * 4 + [r * d, f * r] * 2 + [r * f, d * r]) * case["layers"]


def work(case):
    if case["op"] == "adamw":
        n = sum(_tensor_sizes(case))
        moments = 16 if case["bits"] == 32 else 4 + 8     # read and written; 8 bits: their values read out too
        return {"bytes": n * (4 + 4 + 2 + (4 if case["grad"] == "float32" else 2) + moments), "flops": 14 * n}
    d_out, d_in, m, r = case["d_out"], case["d_in"], case["tokens"], case["r"]
    live = m * (case["requests"] - case["base"]) / case["requests"]      # tokens with an adapter
    used = min(case["adapters"], case["requests"] - case["base"])
    weight = d_out * d_in // 2 + d_out * d_in // 64 + d_out * d_in // 4096
    pool = 2 * used * r * (d_out + d_in)
    product, rank = 2 * m * d_out * d_in, 2 * live * r
    if case["op"] == "fwd":
        return {"bytes": weight + pool + 2 * m * (d_in + d_out), "flops": product + rank * (d_in + d_out)}
    return {"bytes": weight + pool + 2 * m * (2 * d_in + d_out) + 4 * case["adapters"] * r * (d_in + d_out),
            "flops": product + rank * (3 * d_in + 2 * d_out)}


# ---- inputs --------------------------------------------------------------------------

def _quantise(W):
    """NF4 codes with 8-bit block constants of a weight, in the packed layout that the
    projection keeps (two codes a byte, blocks of 64, constants in groups of 256)."""
    blocks = W.reshape(-1, 64)
    absmax = blocks.abs().amax(1)
    book = torch.tensor(CODE, device=W.device)
    codes = torch.bucketize(blocks / absmax[:, None], (book[1:] + book[:-1]) / 2).to(torch.uint8).reshape(-1, 2)
    mean = absmax.double().mean().float().reshape(1)
    group = torch.nn.functional.pad(absmax - mean, (0, -absmax.numel() % 256)).reshape(-1, 256)
    scale = group.abs().amax(1)
    q = torch.round(group / scale.clamp_min(1e-30)[:, None] * 127).to(torch.int8).reshape(-1)[:absmax.numel()]
    return (codes[:, 0] | (codes[:, 1] << 4)).contiguous(), q.contiguous(), scale, mean


def _prepare_linear(case, seed):
    dev = _dev()
    g = torch.Generator(device=dev).manual_seed(seed)
    d_out, d_in, m, r, n = (case[k] for k in ("d_out", "d_in", "tokens", "r", "adapters"))

    def normal(*shape, sigma=1.0):
        return torch.randn(*shape, generator=g, device=dev) * sigma

    s = {"case": case}
    s["codes"], s["qconst"], s["qscale"], s["qmean"] = _quantise(normal(d_out, d_in, sigma=0.02))
    # trained adapters: their part is a good share of the output
    s["A"] = normal(n, r, d_in, sigma=0.03).bfloat16()
    s["B"] = normal(n, d_out, r, sigma=0.03).bfloat16()
    s["s"] = torch.rand(n, generator=g, device=dev) * 1.5 + 0.5
    s["X"] = normal(m, d_in).bfloat16()
    if case["op"] == "bwd":
        s["dY"] = normal(m, d_out).bfloat16()
    s["ids"] = torch.from_numpy(_ids(case, seed)).to(dev)
    if own:
        import bit_nf4_quantized_05_amd as qn

        s["q"] = qn.NF4Weight(s["codes"], s["qconst"], s["qscale"], s["qmean"], d_out, d_in)
        s["pool"] = qn.AdapterPool(s["A"], s["B"], s["s"])
        # made once for a batch: every projection of every layer of the model then uses it
        s["plan"] = qn.multi_plan(s["ids"], n)
        bytes_of = qn.multi_linear_fwd_workspace_bytes if case["op"] == "fwd" else qn.multi_linear_bwd_workspace_bytes
        s["ws"] = torch.empty(max(1, bytes_of(d_out, d_in, m, r, n)), dtype=torch.uint8, device=dev)
    return s


def _padded(sizes):
    return [-(-n // BLOCK) * BLOCK for n in sizes]


def _prepare_adamw(case, seed):
    dev = _dev()
    g = torch.Generator(device=dev).manual_seed(seed)
    sizes = _tensor_sizes(case)
    pads = _padded(sizes)
    total = sum(pads)
    real = torch.zeros(total, dtype=torch.bool, device=dev)      # all tensors in one buffer, each from a block's start
    starts = np.concatenate([[0], np.cumsum(pads)[:-1]]).tolist()
    # gradients of one adapter to another differ by orders of magnitude, and some rows have none
    size_of = torch.exp(torch.randn(total // BLOCK, 1, generator=g, device=dev) * 1.5 - 7).expand(-1, BLOCK).reshape(-1)
    grad = torch.randn(total, generator=g, device=dev) * size_of
    grad *= torch.rand(total // BLOCK, 1, generator=g, device=dev).gt(0.05).expand(-1, BLOCK).reshape(-1)
    for a, n in zip(starts, sizes):
        real[a:a + n] = True
    grad = torch.where(real, grad, 0).to(getattr(torch, case["grad"]))
    p = torch.where(real, torch.randn(total, generator=g, device=dev) * 0.02, 0)
    m = torch.where(real, torch.randn(total, generator=g, device=dev) * size_of * 0.3, 0)
    v = torch.where(real, (torch.rand(total, generator=g, device=dev) + 0.5) * size_of * size_of, 0)
    s = {"case": case, "p": p, "grad": grad, "copy": p.bfloat16(), "step": 100,
         "scale": torch.rand(1, generator=g, device=dev) * 0.9 + 0.1 if case["clip"] else None}
    if case["bits"] == 32:
        s["m"], s["v"] = m, v
    else:
        s["m"], s["ms"], s["v"], s["vs"] = _encode(m, v, _mixed(total, 77, dev))
    if own:
        import bit_nf4_quantized_05_amd as qn

        def views(flat):
            return [flat[a:a + n] for a, n in zip(starts, sizes)]

        s["opt"] = qn.adamw_state(views(p), views(grad), copies=views(s["copy"]), bits=case["bits"])
        s["opt"].m.copy_(s["m"])
        s["opt"].v.copy_(s["v"])
        if case["bits"] == 8:
            s["opt"].m_scale.copy_(s["ms"])
            s["opt"].v_scale.copy_(s["vs"])
    return s


def prepare(case, seed):
    return _prepare_adamw(case, seed) if case["op"] == "adamw" else _prepare_linear(case, seed)


# ---- plain forms ---------------------------------------------------------------------

def _weight(s):
    """W_hat: block constants first, then code * constant, rounded to bf16 as the layer defines it."""
    c = s["case"]
    nb = s["qconst"].numel()
    scale = s["qscale"].repeat_interleave(256)[:nb]
    absmax = s["qmean"] + scale * (s["qconst"].float() / 127.0)
    code = torch.stack([s["codes"] & 15, s["codes"] >> 4], 1).reshape(-1, 64).int()
    return (torch.tensor(CODE, device=code.device)[code] * absmax[:, None]).bfloat16().float().reshape(c["d_out"], c["d_in"])


def _ranks(s):
    """All adapters side by side: A [n r, d_in], B [n r, d_out], and which of the n r columns
    a token has, with its adapter's scale."""
    n, r = s["A"].shape[:2]
    A = s["A"].float().reshape(n * r, -1)
    B = s["B"].float().transpose(1, 2).reshape(n * r, -1)
    mine = s["ids"][:, None] == torch.arange(n, device=A.device)
    pick = torch.where(mine, s["s"][None, :], 0).repeat_interleave(r, 1)
    return A, B, pick


def _plain_fwd(s):
    X = s["X"].float()
    A, B, pick = _ranks(s)
    return (X @ _weight(s).T + ((X @ A.T) * pick) @ B).bfloat16()


def _plain_bwd(s):
    n, r, d_in = s["A"].shape
    X, dY = s["X"].float(), s["dY"].float()
    A, B, pick = _ranks(s)
    T, U = (X @ A.T) * pick, (dY @ B.T) * pick
    dX = (dY @ _weight(s) + U @ A).bfloat16()
    dB = (T.T @ dY).reshape(n, r, -1).transpose(1, 2).contiguous()
    return {"dX": dX, "dA": (U.T @ X).reshape(n, r, d_in), "dB": dB}


def _mix(h):
    """A 32-bit integer mixer (two multiplications and three shifts, the finaliser of MurmurHash3)."""
    h = h ^ (h >> 16)
    h = (h * 0x85EBCA6B) & M32
    h = h ^ (h >> 13)
    h = (h * 0xC2B2AE35) & M32
    return h ^ (h >> 16)


def _mixed(total, step, dev):
    """One 32-bit word per element for its rounding, from the step and the element's place."""
    key = _mix(torch.tensor(step, dtype=torch.int64, device=dev))
    return _mix(torch.arange(total, dtype=torch.int64, device=dev) ^ key)


def _encode(m, v, h):
    """The moments in 8 bits: |x| / (its block's largest) as a float with 3 mantissa bits,
    rounded up with the probability of the part cut off (16 random bits each). m: sign and 127
    magnitudes, v: 255 magnitudes; 0 is the zero code."""
    m, v = m.reshape(-1, BLOCK), v.reshape(-1, BLOCK)
    h = h.reshape(-1, BLOCK)

    def level(x, bits16, top):
        big = x.amax(1, keepdim=True)
        usable = big >= 2.0 ** -126
        big = torch.where(usable, big, 0)
        inv = torch.where(usable, 1.0 / big, 0)
        at = (torch.clamp(x * inv, max=1.0).view(torch.int32) + (bits16 << 4).int()) >> 20
        return (at - (1016 - top)).clamp(0, top), big

    cm, big_m = level(m.abs(), h & 0xFFFF, 127)
    cv, big_v = level(v, h >> 16, 255)
    cv = torch.where((v > 0) & (big_v > 0), cv.clamp_min(1), cv)
    cm = torch.where((m < 0) & (cm > 0), cm + 128, cm)
    return cm.to(torch.uint8).reshape(-1), big_m.reshape(-1), cv.to(torch.uint8).reshape(-1), big_v.reshape(-1)


def _decode(code, big, signed):
    c = code.int().reshape(-1, BLOCK)
    mag = c & 127 if signed else c
    x = torch.where(mag > 0, ((mag + (889 if signed else 761)) << 20).view(torch.float32), 0) * big[:, None]
    return (torch.where(c > 127, -x, x) if signed else x).reshape(-1)


def _plain_adamw(s):
    s["step"] += 1
    t, eight = s["step"], s["case"]["bits"] == 8
    g = s["grad"].float()
    if s["scale"] is not None:
        g = g * s["scale"]
    m, v = (_decode(s["m"], s["ms"], True), _decode(s["v"], s["vs"], False)) if eight else (s["m"], s["v"])
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + (g * g) * (1 - BETA2)
    denom = torch.sqrt(v) * (1 / math.sqrt(1 - BETA2 ** t)) + EPS
    s["p"] = s["p"] * (1 - LR * DECAY) - (LR / (1 - BETA1 ** t)) * (m / denom)
    if eight:
        s["m"], s["ms"], s["v"], s["vs"] = _encode(m, v, _mixed(m.numel(), t, m.device))
        m, v = _decode(s["m"], s["ms"], True), _decode(s["v"], s["vs"], False)
    else:
        s["m"], s["v"] = m, v
    return {"p": s["p"], "copy": s["p"].bfloat16(), "m": m, "v": v}


# ---- the package's calls -------------------------------------------------------------

def _own(s):
    import bit_nf4_quantized_05_amd as qn

    op = s["case"]["op"]
    if op == "fwd":
        return qn.multi_linear_fwd(s["q"], s["pool"], s["plan"], s["X"], workspace=s["ws"])
    if op == "bwd":
        dX, dA, dB = qn.multi_linear_bwd(s["q"], s["pool"], s["plan"], s["X"], s["dY"], workspace=s["ws"])
        return {"dX": dX, "dA": dA, "dB": dB}
    s["step"] += 1
    opt = s["opt"]
    qn.adamw_step(opt, s["step"], LR, BETA1, BETA2, EPS, DECAY, grad_scale=s["scale"])
    # 8-bit moments are read out as the values that they stand for
    m, v = qn.adamw_moments(opt) if s["case"]["bits"] == 8 else (opt.m, opt.v)
    return {"p": s["p"], "copy": s["copy"], "m": m, "v": v}


def run(state):
    if own:
        return _own(state)
    return {"fwd": _plain_fwd, "bwd": _plain_bwd, "adamw": _plain_adamw}[state["case"]["op"]](state)


# ---- the definitions in 64 bits -------------------------------------------------------

def _exact_weight(s):
    c = s["case"]
    low, high = s["codes"].long() & 15, s["codes"].long() >> 4
    book = torch.tensor(CODE, dtype=torch.float64, device=low.device)
    flat = torch.empty(low.numel(), 2, dtype=torch.float64, device=low.device)
    flat[:, 0], flat[:, 1] = book[low], book[high]
    group = torch.arange(s["qconst"].numel(), device=low.device) // 256
    absmax = s["qmean"].double() + s["qscale"].double()[group] * s["qconst"].double() / 127
    # the layer's weight is a bf16 number by definition
    return (flat.reshape(-1, 64) * absmax[:, None]).bfloat16().double().reshape(c["d_out"], c["d_in"])


def _exact_linear(s):
    W, X, c = _exact_weight(s), s["X"].double(), s["case"]
    rows = [torch.nonzero(s["ids"] == a).reshape(-1) for a in range(c["adapters"])]
    A, B = s["A"].double(), s["B"].double()
    sc = s["s"].double().tolist()
    if c["op"] == "fwd":
        Y = X @ W.T
        for a, t in enumerate(rows):
            Y[t] += sc[a] * (X[t] @ A[a].T @ B[a].T)
        return Y
    dY = s["dY"].double()
    dX, dA, dB = dY @ W, torch.zeros_like(A), torch.zeros_like(B)
    for a, t in enumerate(rows):
        x, dy = X[t], dY[t]
        back = dy @ B[a]
        dX[t] += sc[a] * (back @ A[a])
        dA[a] = sc[a] * (back.T @ x)
        dB[a] = sc[a] * (dy.T @ (x @ A[a].T))
    return {"dX": dX, "dA": dA, "dB": dB}


def _exact_words(total, step):
    """The rounding words again, in numpy's wrapping 32-bit integers."""
    def mix(h):
        h ^= h >> np.uint32(16)
        h *= np.uint32(0x85EBCA6B)
        h ^= h >> np.uint32(13)
        h *= np.uint32(0xC2B2AE35)
        h ^= h >> np.uint32(16)
        return h

    return mix(np.arange(total, dtype=np.uint32) ^ mix(np.array([step], np.uint32)))


def _exact_grid(x, frac, low_exponent, low_eighth):
    """x in [0, 1] on the grid (1 + k / 8) 2^e, up with probability of the rest (frac in [0, 1));
    below the grid's smallest value, 0."""
    e = torch.floor(torch.log2(x.clamp_min(1e-300)))
    e = e + (x >= torch.exp2(e + 1)).double() - (x < torch.exp2(e)).double()
    step = torch.floor((x * torch.exp2(-e) - 1) * 8 + frac)
    y = (1 + step / 8) * torch.exp2(e)
    return torch.where(y >= (1 + low_eighth / 8) * 2.0 ** low_exponent, y, 0)


def _exact_adamw(s):
    dev, t = s["p"].device, s["step"] + 1
    eight = s["case"]["bits"] == 8

    def stored(code, big, signed):
        c = code.long().reshape(-1, BLOCK)
        k = (c & 127 if signed else c) + (889 if signed else 761)
        x = (1 + (k & 7).double() / 8) * torch.exp2((k >> 3).double() - 127) * big.double()[:, None]
        x = torch.where((c & 127 if signed else c) == 0, 0, x)
        return (torch.where(c >= 128, -x, x) if signed else x).reshape(-1)

    m = stored(s["m"], s["ms"], True) if eight else s["m"].double()
    v = stored(s["v"], s["vs"], False) if eight else s["v"].double()
    g = s["grad"].double() * (s["scale"].double() if s["scale"] is not None else 1.0)
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g.square()
    p = s["p"].double() * (1 - LR * DECAY) - LR * (m / (1 - BETA1 ** t)) / (torch.sqrt(v / (1 - BETA2 ** t)) + EPS)
    if eight:
        words = torch.from_numpy(_exact_words(p.numel(), t).view(np.int32)).to(dev).long() & M32
        big_m, big_v = (x.abs().reshape(-1, BLOCK).amax(1).repeat_interleave(BLOCK) for x in (m, v))
        m = torch.sign(m) * big_m * _exact_grid(m.abs() / big_m.clamp_min(1e-300), (words & 0xFFFF).double() / 65536, -16, 2)
        w = _exact_grid(v / big_v.clamp_min(1e-300), (words >> 16).double() / 65536, -32, 2)
        v = big_v * torch.where(v > 0, w.clamp_min(1.25 * 2.0 ** -32), 0)
    return {"p": p, "copy": p, "m": m, "v": v}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_adamw(s) if case["op"] == "adamw" else _exact_linear(s)
