"""Many adapters on one layer against the float64 oracle: the plan, the forward in both its
forms (up to 64 tokens, and the GEMM), and the gradients.

Tolerances. Y and dX: those of the single-adapter products (parity.py). dA, dB are float32
sums of up to ~1500 tokens of products with rank sums over up to 1536 features: with
u = 2^-24 per addition and independent roundings, sqrt(1500 + 1536) u = 3.3e-6 of the norm
(5e-6 allowed), and 5 deviations of that on the largest element (2e-5 of it)."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_05_amd as qn
import workloads as WL
from oracle import multi_oracle as MO
from oracle import nf4_oracle as O
from parity import bf16_f64, check_close, dev, to_gpu_f32

pytestmark = pytest.mark.gpu


def _say(*a):
    print(*a, flush=True)


def _pool(n, r, d_out, d_in, gen, sigma=0.05):
    return qn.AdapterPool((torch.randn(n, r, d_in, generator=gen, device=dev()) * sigma).bfloat16(),
                          (torch.randn(n, d_out, r, generator=gen, device=dev()) * sigma).bfloat16(),
                          torch.rand(n, generator=gen, device=dev()) + 0.5)


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _ids(kind, M, n, rng):
    if kind == "none":
        return np.full(M, -1, np.int32)
    if kind == "one":
        return np.full(M, n - 1, np.int32)
    if kind == "mixed":                                     # every token anybody's, some nobody's
        return rng.integers(-1, n, M).astype(np.int32)
    if kind == "outside":                                   # ids past the pool count as none
        return rng.choice(np.array([0, n, n + 5, -7, 2 ** 31 - 1], np.int64), M).astype(np.int32)
    # packed requests of uneven lengths
    reqs = min(M, max(1, n + 2))
    cuts = np.sort(rng.choice(np.arange(1, M), reqs - 1, replace=False)) if reqs > 1 else np.array([], int)
    who = rng.integers(-1, n, reqs)
    return np.repeat(who, np.diff(np.concatenate([[0], cuts, [M]]))).astype(np.int32)


class Layer:
    def __init__(self, d_out, d_in, M, r, n, kind, seed, dq="int8"):
        self.gen = torch.Generator(device=dev()).manual_seed(seed)
        rng = np.random.default_rng(seed)
        w = WL.make_weight(WL.custom("m", d_out, d_in, 1, 8, seed=seed))
        self.q = qn.quantize(to_gpu_f32(w), dq=dq)
        self.W = bf16_f64(qn.double_dequant(self.q))
        self.pool = _pool(n, r, d_out, d_in, self.gen)
        self.ids_np = _ids(kind, M, n, rng)
        self.ids = torch.from_numpy(self.ids_np).to(dev())
        self.plan = qn.multi_plan(self.ids, n)
        self.X = torch.randn(M, d_in, generator=self.gen, device=dev()).bfloat16()
        self.dY = torch.randn(M, d_out, generator=self.gen, device=dev()).bfloat16()
        self.A, self.B, self.s = _f64(self.pool.A), _f64(self.pool.B), _f64(self.pool.s)

    def forward(self):
        return MO.forward(self.W, self.A, self.B, self.s, self.ids_np, _f64(self.X))

    def backward(self):
        return MO.backward(self.W, self.A, self.B, self.s, self.ids_np, _f64(self.X), _f64(self.dY))


def _close32(got, ref, what):
    got = _f64(got)
    assert np.all(np.isfinite(got)), what
    norm = np.linalg.norm(ref)
    if norm == 0:
        assert np.all(got == 0), what
        return
    rel, big = np.linalg.norm(got - ref) / norm, np.max(np.abs(got - ref)) / np.max(np.abs(ref))
    assert rel <= 5e-6 and big <= 2e-5, f"{what}: {rel:.2e} {big:.2e}"


# ---- the plan -------------------------------------------------------------------------

def _plan_parts(plan):
    """(head, order, start, first_item, used, tile, items) of a plan's buffer."""
    w = plan.buf.cpu().numpy().view(np.int32)
    M, n = plan.d_seq, plan.n
    up = lambda v: (v + 3) // 4 * 4  # noqa: E731
    at, out = 4, [w[:4]]
    for size in (M, n + 1, n, min(n, M), 2 * ((M + 255) // 256)):
        out.append(w[at:at + size])
        at += up(size)
    items = w[at:at + 4 * ((M + 127) // 128 + min(n, M))].reshape(-1, 4)
    return out + [items]


@pytest.mark.parametrize("M,n,kind", [(1, 1, "one"), (1, 5, "none"), (63, 64, "mixed"), (64, 3, "packed"),
                                      (65, 1, "mixed"), (1000, 7, "packed"), (1024, 7, "outside"),
                                      (4097, 1024, "mixed"), (5000, 1000, "packed"), (20011, 33, "mixed")])
def test_plan(M, n, kind):
    _say(f"[multi] plan {M} tokens, {n} adapters, {kind}")
    ids = _ids(kind, M, n, np.random.default_rng(M + n))
    plan = qn.multi_plan(torch.from_numpy(ids).to(dev()), n)
    torch.cuda.synchronize()
    head, order, start, first, used, tile, items = _plan_parts(plan)
    key = np.where((ids >= 0) & (ids < n), ids, n)
    want = np.argsort(key, kind="stable")
    assert np.array_equal(order, want)
    counts = np.bincount(key, minlength=n + 1)
    assert np.array_equal(start, np.concatenate([[0], np.cumsum(counts[:n])]))
    act = np.flatnonzero(counts[:n])
    assert head[0] == len(act) and np.array_equal(used[:len(act)], act) and head[2] == counts[:n].sum()
    rows = []
    for a in act:
        assert first[a] == len(rows)
        rows += [(a, start[a] + k, counts[a] - k, k // 128) for k in range(0, counts[a], 128)]
    assert head[1] == len(rows) and np.array_equal(items[:len(rows)].reshape(-1, 4), np.array(rows, int).reshape(-1, 4))
    assert np.all(items[len(rows):] == [-1, 0, 0, 0])
    for t in range((M + 255) // 256):
        have = [a for k, a in enumerate(act) if start[a] < min(256 * t + 256, head[2]) and start[a + 1] > 256 * t]
        k0, k1 = tile[2 * t], tile[2 * t + 1]
        assert list(used[k0:k1]) == have, t
    again = qn.multi_plan(torch.from_numpy(ids[::-1].copy()).to(dev()), n, out=plan)
    assert again is plan and np.array_equal(_plan_parts(plan)[1], np.argsort(key[::-1], kind="stable"))


# ---- forward --------------------------------------------------------------------------

SMALL = [(64, 64, 1, 16, 1, "one"), (256, 320, 1, 16, 4, "none"), (512, 4096, 3, 32, 3, "mixed"),
         (1024, 1088, 16, 16, 40, "mixed"), (320, 192, 17, 48, 2, "mixed"), (512, 2048, 33, 64, 33, "packed"),
         (192, 11008, 64, 80, 64, "mixed"), (4096, 512, 64, 256, 5, "mixed"), (256, 256, 64, 16, 1, "one"),
         (128, 64, 40, 128, 300, "outside"),
         # one token on the streaming GEMV, up to 4096 rows and more, with an adapter and without
         (4096, 4096, 1, 16, 3, "one"), (4160, 256, 1, 16, 3, "one"), (4160, 256, 1, 16, 3, "none"),
         (128, 4160, 1, 16, 2, "one"), (128, 256, 1, 32, 2, "one")]
LARGE = [(256, 256, 65, 16, 3, "mixed"), (320, 192, 300, 32, 5, "packed"), (512, 4096, 200, 48, 40, "mixed"),
         (1024, 1536, 1531, 16, 7, "packed"), (256, 512, 1024, 64, 4, "packed"), (64, 64, 257, 256, 2, "mixed"),
         (192, 128, 513, 80, 64, "outside"), (256, 320, 700, 112, 1, "one"), (256, 256, 600, 16, 9, "none"),
         (128, 192, 2000, 16, 1000, "mixed"), (2048, 2048, 2100, 16, 3, "packed"),
         # 96 tiles (halves alone), 336 (whole ones and halves), 257 (whole ones and one split)
         (4096, 128, 1531, 32, 30, "packed"), (4096, 64, 5200, 16, 5, "packed"), (4096, 1024, 4097, 16, 6, "mixed"),
         # a few tiles of a short K (halves) and of a long one (split), after whole ones too
         (512, 512, 203, 16, 3, "mixed"), (256, 4096, 300, 32, 3, "mixed"), (4096, 2560, 4097, 16, 6, "mixed"),
         (448, 10112, 100, 64, 5, "mixed"), (448, 10112, 130, 64, 140, "mixed"), (1024, 8192, 900, 16, 30, "mixed"),
         # 64 whole tiles split in four
         (4096, 4864, 1000, 16, 6, "mixed")]


@pytest.mark.parametrize("d_out,d_in,M,r,n,kind", SMALL + LARGE)
def test_forward(d_out, d_in, M, r, n, kind):
    _say(f"[multi] forward {d_out}x{d_in}, {M} tokens, r={r}, {n} adapters, {kind}")
    L = Layer(d_out, d_in, M, r, n, kind, seed=M + r)
    Y = qn.multi_linear_fwd(L.q, L.pool, L.plan, L.X)
    torch.cuda.synchronize()
    check_close(_f64(Y), L.forward(), "forward")
    again = qn.multi_linear_fwd(L.q, L.pool, L.plan, L.X)
    assert torch.equal(Y.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("r", [16, 32, 48, 96, 112, 160, 208, 256])
@pytest.mark.parametrize("d_in", [448, 1216])
def test_adapters_of_few_and_many_tokens(r, d_in):
    """Adapters of 1, 15, 16, 17 and 70 tokens in one batch, in one and in several K-slices."""
    _say(f"[multi] few tokens per adapter, r={r}, {d_in} features")
    counts = [1, 15, 16, 17, 70, 1, 1, 3]
    L = Layer(128, d_in, sum(counts), r, len(counts) + 1, "one", seed=r + d_in)
    L.ids_np = np.random.default_rng(r).permutation(np.repeat(np.arange(len(counts)), counts)).astype(np.int32)
    L.plan = qn.multi_plan(torch.from_numpy(L.ids_np).to(dev()), len(counts) + 1)
    check_close(_f64(qn.multi_linear_fwd(L.q, L.pool, L.plan, L.X)), L.forward(), "forward")
    gX, gA, gB = qn.multi_linear_bwd(L.q, L.pool, L.plan, L.X, L.dY)
    wX, wA, wB = L.backward()
    check_close(_f64(gX), wX, "dX")
    _close32(gA, wA, "dA")
    _close32(gB, wB, "dB")


@pytest.mark.parametrize("d_out,d_in", [(4096, 4096), (4160, 1024), (256, 4160)])
@pytest.mark.parametrize("M", [1, 5, 64, 80])
def test_weights_are_the_dequantisers(d_out, d_in, M):
    """Whatever path a batch takes, its weights are the dequantised bf16 ones: what is left
    is the output's own rounding, 2^-8 / sqrt(3) = 0.0023 of a value at its binade's start
    and half of that at its end, 0.0017 over values spread evenly in log, and the rank
    sum's, the same share of a smaller part: 0.0021 holds both."""
    _say(f"[multi] weights, {d_out}x{d_in}, {M} tokens")
    L = Layer(d_out, d_in, M, 16, 3, "mixed", seed=M)
    Y, ref = _f64(qn.multi_linear_fwd(L.q, L.pool, L.plan, L.X)), L.forward()
    assert np.linalg.norm(Y - ref) <= 0.0021 * np.linalg.norm(ref)


@pytest.mark.parametrize("dq", ["fp8", "none"])
@pytest.mark.parametrize("M", [1, 20, 150])
def test_second_level_formats(dq, M):
    _say(f"[multi] second level {dq}, {M} tokens")
    L = Layer(256, 320, M, 16, 4, "mixed", seed=5, dq=dq)
    check_close(_f64(qn.multi_linear_fwd(L.q, L.pool, L.plan, L.X)), L.forward(), "forward")
    check_close(_f64(qn.multi_linear_bwd(L.q, L.pool, L.plan, L.X, L.dY)[0]), L.backward()[0], "dX")


@pytest.mark.parametrize("M", [1, 30, 64, 65, 400])
def test_rows_of_wider_arrays(M):
    """Strided inputs and outputs: the contiguous call's bits, and nothing else is written."""
    _say(f"[multi] windows, {M} tokens")
    d_out, d_in, r, n = 320, 256, 32, 5
    L = Layer(d_out, d_in, M, r, n, "mixed", seed=M)
    ref = qn.multi_linear_fwd(L.q, L.pool, L.plan, L.X)
    dX, dA, dB = qn.multi_linear_bwd(L.q, L.pool, L.plan, L.X, L.dY)
    wide = torch.full((M, d_in + 40), 7.0, device=dev()).bfloat16()
    wide[:, 16:16 + d_in] = L.X
    wdy = torch.full((M, d_out + 8), 7.0, device=dev()).bfloat16()
    wdy[:, :d_out] = L.dY
    out = torch.full((M + 2, d_out + 24), 3.0, device=dev()).bfloat16()
    gx = torch.full((M + 2, d_in + 24), 3.0, device=dev()).bfloat16()
    qn.multi_linear_fwd(L.q, L.pool, L.plan, wide[:, 16:16 + d_in], out=out[1:M + 1, 8:8 + d_out])
    _, wA, wB = qn.multi_linear_bwd(L.q, L.pool, L.plan, wide[:, 16:16 + d_in], wdy[:, :d_out], dX=gx[1:M + 1, 8:8 + d_in])
    torch.cuda.synchronize()
    for got, want, cols in ((out, ref, d_out), (gx, dX, d_in)):
        assert torch.equal(got[1:M + 1, 8:8 + cols].reshape(M, cols).view(torch.int16), want.view(torch.int16))
        got[1:M + 1, 8:8 + cols] = 3.0
        assert torch.all(got == 3.0)
    assert torch.equal(wA, dA) and torch.equal(wB, dB)


@pytest.mark.parametrize("M", [48, 64, 300, 700])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_adapters_do_not_reach_each_other(M, value):
    """An adapter of NaN or infinity leaves every other token's Y and dX, and every other
    adapter's gradients, at the bits they have with a finite one."""
    _say(f"[multi] isolation, {M} tokens, {value}")
    L = Layer(192, 256, M, 16, 6, "mixed", seed=M)
    ref = qn.multi_linear_fwd(L.q, L.pool, L.plan, L.X)
    rX, rA, rB = qn.multi_linear_bwd(L.q, L.pool, L.plan, L.X, L.dY)
    bad = 2
    L.pool.A[bad, 3, 5] = value
    L.pool.B[bad, 7, 2] = value
    Y = qn.multi_linear_fwd(L.q, L.pool, L.plan, L.X)
    dX, dA, dB = qn.multi_linear_bwd(L.q, L.pool, L.plan, L.X, L.dY)
    torch.cuda.synchronize()
    other = L.ids != bad
    assert torch.equal(Y[other].view(torch.int16), ref[other].view(torch.int16))
    assert torch.equal(dX[other].view(torch.int16), rX[other].view(torch.int16))
    assert not torch.isfinite(Y[~other].float()).all() and not torch.isfinite(dX[~other].float()).all()
    keep = [a for a in range(6) if a != bad]
    assert torch.equal(dA[keep], rA[keep]) and torch.equal(dB[keep], rB[keep])


@pytest.mark.parametrize("d_out", [256, 4160])
@pytest.mark.parametrize("who", [-1, 1])
def test_one_token_keeps_off_other_adapters(d_out, who):
    _say(f"[multi] one token beside adapters of NaN, {d_out} rows, adapter {who}")
    L = Layer(d_out, 256, 1, 16, 3, "one", seed=2)
    plan = qn.multi_plan(torch.tensor([who], dtype=torch.int32, device=dev()), 3)
    ref = qn.multi_linear_fwd(L.q, L.pool, plan, L.X)
    for a in (0, 2):
        L.pool.A[a] = float("nan")
        L.pool.B[a] = float("inf")
    L.pool.s[0] = float("nan")
    Y = qn.multi_linear_fwd(L.q, L.pool, plan, L.X)
    torch.cuda.synchronize()
    assert torch.isfinite(ref.float()).all() and torch.equal(Y.view(torch.int16), ref.view(torch.int16))


@pytest.mark.parametrize("M", [50, 400])
def test_tokens_of_nan_stay_apart(M):
    """A token of NaN changes only its own rows and its own adapter's gradients."""
    _say(f"[multi] NaN token, {M} tokens")
    L = Layer(128, 192, M, 32, 4, "mixed", seed=3 + M)
    ref = qn.multi_linear_fwd(L.q, L.pool, L.plan, L.X)
    rX, rA, rB = qn.multi_linear_bwd(L.q, L.pool, L.plan, L.X, L.dY)
    t = int(np.flatnonzero(L.ids_np == 1)[0])
    L.X[t] = float("nan")
    L.dY[t] = float("inf")
    Y = qn.multi_linear_fwd(L.q, L.pool, L.plan, L.X)
    dX, dA, dB = qn.multi_linear_bwd(L.q, L.pool, L.plan, L.X, L.dY)
    torch.cuda.synchronize()
    rows = [k for k in range(M) if k != t]
    assert torch.equal(Y[rows].view(torch.int16), ref[rows].view(torch.int16)) and torch.isnan(Y[t]).all()
    assert torch.equal(dX[rows].view(torch.int16), rX[rows].view(torch.int16))
    assert torch.equal(dA[[0, 2, 3]], rA[[0, 2, 3]]) and torch.equal(dB[[0, 2, 3]], rB[[0, 2, 3]])


def test_ranks_padded_by_the_pool():
    """Adapters of ranks 1, 5 and 20 in one pool give what each gives by its own rank."""
    _say("[multi] mixed ranks")
    L = Layer(256, 192, 90, 16, 3, "mixed", seed=9)
    pool = qn.alloc_pool(3, 20, 256, 192, dev())
    assert pool.r == 32
    A, B = [], []
    for i, k in enumerate((1, 5, 20)):
        A.append((torch.randn(k, 192, generator=L.gen, device=dev()) * 0.05).bfloat16())
        B.append((torch.randn(256, k, generator=L.gen, device=dev()) * 0.05).bfloat16())
        pool.set(i, A[i], B[i], 1.5 + i)
    Y = qn.multi_linear_fwd(L.q, pool, L.plan, L.X)
    _, dA, dB = qn.multi_linear_bwd(L.q, pool, L.plan, L.X, L.dY)
    X, dY = _f64(L.X), _f64(L.dY)
    ref = X @ L.W.T
    for i, k in enumerate((1, 5, 20)):
        t = np.flatnonzero(L.ids_np == i)
        T = X[t] @ _f64(A[i]).T
        ref[t] += (1.5 + i) * (T @ _f64(B[i]).T)
        _close32(dB[i, :, :k], (1.5 + i) * (dY[t].T @ T), f"dB rank {k}")
        assert torch.all(dB[i, :, k:] == 0) and torch.all(dA[i, k:] == 0)
    check_close(_f64(Y), ref, "mixed ranks")


# ---- gradients ------------------------------------------------------------------------

BWD = [(64, 64, 1, 16, 2, "one"), (256, 256, 203, 16, 3, "packed"), (320, 192, 40, 48, 6, "mixed"),
       (192, 320, 700, 32, 2, "packed"), (512, 1024, 1300, 16, 1, "one"), (128, 256, 900, 80, 5, "mixed"),
       (256, 192, 1500, 64, 3, "packed"), (64, 128, 300, 256, 4, "mixed"), (128, 128, 500, 16, 200, "mixed"),
       (256, 256, 130, 16, 4, "none"), (1536, 1088, 640, 128, 3, "packed"),
       (128, 4096, 1531, 48, 30, "packed"), (64, 4096, 5200, 16, 5, "packed"), (1024, 512, 2000, 240, 3, "mixed"),
       (512, 512, 512, 16, 3, "mixed"), (4096, 256, 300, 32, 3, "mixed"), (2560, 4096, 4097, 16, 6, "packed"),
       (576, 640, 513, 32, 600, "mixed"), (5056, 320, 54, 64, 5, "packed"), (4160, 640, 200, 16, 100, "mixed"),
       (4864, 4096, 1000, 16, 6, "mixed")]


@pytest.mark.parametrize("d_out,d_in,M,r,n,kind", BWD)
def test_gradients(d_out, d_in, M, r, n, kind):
    _say(f"[multi] gradients {d_out}x{d_in}, {M} tokens, r={r}, {n} adapters, {kind}")
    L = Layer(d_out, d_in, M, r, n, kind, seed=M + r + 1)
    junk = torch.full(L.pool.A.shape, float("nan"), device=dev()), torch.full(L.pool.B.shape, float("nan"), device=dev())
    dX, dA, dB = qn.multi_linear_bwd(L.q, L.pool, L.plan, L.X, L.dY, dA=junk[0], dB=junk[1])
    torch.cuda.synchronize()
    wX, wA, wB = L.backward()
    check_close(_f64(dX), wX, "dX")
    _close32(dA, wA, "dA")
    _close32(dB, wB, "dB")
    again = qn.multi_linear_bwd(L.q, L.pool, L.plan, L.X, L.dY)
    for x, y in zip((dX, dA, dB), again):
        assert torch.equal(x, y)


@pytest.mark.parametrize("M", [7, 64, 150])
def test_gradients_against_differences(M):
    """<dY, Y> is linear in each of X, A and B alone, so a whole step D of one of them moves it
    by the gradient's product with D. Y's two roundings leave noise of 2^-8 / sqrt(3) per
    element and call (test_weights_are_the_dequantisers), the rank sum's less: 5 deviations of
    0.0024 sqrt(2) |dY Y| per element; dX's own roundings 0.0024 |dX D| per element."""
    _say(f"[multi] gradients against differences, {M} tokens")
    L = Layer(320, 256, M, 16, 3, "mixed", seed=40 + M)
    dX, dA, dB = (_f64(g) for g in qn.multi_linear_bwd(L.q, L.pool, L.plan, L.X, L.dY))
    dY, Y0 = _f64(L.dY), _f64(qn.multi_linear_fwd(L.q, L.pool, L.plan, L.X))
    for what, t, grad in (("X", L.X, dX), ("A", L.pool.A, dA), ("B", L.pool.B, dB)):
        was = t.clone()
        t += (torch.randn(t.shape, generator=L.gen, device=dev()) * t.float().std()).bfloat16()
        D = _f64(t) - _f64(was)
        Y1 = _f64(qn.multi_linear_fwd(L.q, L.pool, L.plan, L.X))
        t.copy_(was)
        noise = 0.0024 * np.sqrt(np.sum((dY * Y0) ** 2) + np.sum((dY * Y1) ** 2) + np.sum((grad * D) ** 2))
        assert abs(np.sum(dY * (Y1 - Y0)) - np.sum(grad * D)) <= 5 * noise, what


def test_pool_of_more_than_2_32_elements():
    """Adapters on both sides of element 2^31 and 2^32 of the pool and of dA."""
    n, r, d_out, d_in = 1024, 64, 64, 65536 + 64
    _say(f"[multi] pool of {n} adapters, r={r}, {d_in} features")
    L = Layer(d_out, d_in, 80, r, 1, "one", seed=77)
    A = torch.full((n, r, d_in), float("nan"), dtype=torch.bfloat16, device=dev())
    B = torch.full((n, d_out, r), float("nan"), dtype=torch.bfloat16, device=dev())
    who = [0, 510, 513, 1023]
    for a in who:
        A[a] = (torch.randn(r, d_in, generator=L.gen, device=dev()) * 0.02).bfloat16()
        B[a] = (torch.randn(d_out, r, generator=L.gen, device=dev()) * 0.02).bfloat16()
    pool = qn.AdapterPool(A, B, torch.ones(n, device=dev()))
    ids = np.array(who, np.int32)[np.random.default_rng(7).integers(0, 4, 80)]
    small = np.searchsorted(who, ids)
    nA, nB, X, dY = _f64(A[who]), _f64(B[who]), _f64(L.X), _f64(L.dY)
    for M in (5, 80):
        plan = qn.multi_plan(torch.from_numpy(ids[:M].copy()).to(dev()), n)
        Y = qn.multi_linear_fwd(L.q, pool, plan, L.X[:M])
        check_close(_f64(Y), MO.forward(L.W, nA, nB, np.ones(4), small[:M], X[:M]), f"forward, {M} tokens")
    gX, gA, gB = qn.multi_linear_bwd(L.q, pool, plan, L.X, L.dY)
    wX, wA, wB = MO.backward(L.W, nA, nB, np.ones(4), small, X, dY)
    check_close(_f64(gX), wX, "dX")
    for k, a in enumerate(who):
        assert np.linalg.norm(_f64(gA[a]) - wA[k]) <= 5e-6 * np.linalg.norm(wA[k]), a
        # T sums 65600 products: sqrt(65600) 2^-24 = 1.5e-5
        assert np.linalg.norm(_f64(gB[a]) - wB[k]) <= 3e-5 * np.linalg.norm(wB[k]), a
        gA[a] = 0
        gB[a] = 0
    assert all(gA[i:i + 64].count_nonzero() == 0 for i in range(0, n, 64)) and gB.count_nonzero() == 0


def test_operands_near_4_gib():
    """131072 tokens of 16320 features: X and dX take 4.28 GB, the largest the calls accept.
    dA sums 65536 tokens: sqrt(65536) 2^-24 = 1.5e-5 of the norm, twice that allowed."""
    M, d_in, d_out, r, n = 131072, 16320, 64, 16, 2
    _say(f"[multi] {M} tokens of {d_in} features")
    L = Layer(d_out, d_in, 1, r, n, "one", seed=91)
    X = torch.empty(M, d_in, dtype=torch.bfloat16, device=dev())
    for i in range(0, M, 16384):
        X[i:i + 16384] = torch.randn(16384, d_in, generator=L.gen, device=dev()).bfloat16()
    dY = torch.randn(M, d_out, generator=L.gen, device=dev()).bfloat16()
    ids = (torch.arange(M, device=dev()) % 3 - 1).int()
    plan = qn.multi_plan(ids, n)
    Y = qn.multi_linear_fwd(L.q, L.pool, plan, X)
    dX, dA, dB = qn.multi_linear_bwd(L.q, L.pool, plan, X, dY)
    torch.cuda.synchronize()
    rows = np.unique(np.concatenate([np.arange(0, M, 4099), np.arange(M - 40, M), np.arange(65520, 65560)]))
    at = torch.from_numpy(rows).to(dev())
    who = ids[at].cpu().numpy()
    check_close(_f64(Y[at]), MO.forward(L.W, L.A, L.B, L.s, who, _f64(X[at])), "forward")
    check_close(_f64(dX[at]), MO.backward(L.W, L.A, L.B, L.s, who, _f64(X[at]), _f64(dY[at]))[0], "dX")
    A, B, s = L.pool.A.double(), L.pool.B.double(), L.s
    for a in range(n):
        wA, wB = torch.zeros_like(A[a]), torch.zeros_like(B[a])
        for i in range(0, M, 16384):
            t = i + torch.nonzero(ids[i:i + 16384] == a).reshape(-1)
            x, dy = X[t].double(), dY[t].double()
            wA += s[a] * torch.mm(torch.mm(dy, B[a]).t().contiguous(), x)
            wB += s[a] * torch.mm(dy.t().contiguous(), torch.mm(x, A[a].t().contiguous()))
        assert (dA[a].double() - wA).norm() <= 3e-5 * wA.norm() and (dB[a].double() - wB).norm() <= 3e-5 * wB.norm(), a


# ---- streams and graphs ---------------------------------------------------------------

@pytest.mark.parametrize("M", [24, 300])
def test_other_stream_and_graph(M):
    _say(f"[multi] side stream and graph replays, {M} tokens")
    L = Layer(512, 256, M, 16, 7, "mixed", seed=M)
    Y, dX = torch.empty_like(L.dY), torch.empty_like(L.X)
    dA, dB = (torch.empty(p.shape, dtype=torch.float32, device=dev()) for p in (L.pool.A, L.pool.B))
    ws = torch.empty(max(qn.multi_linear_fwd_workspace_bytes(512, 256, M, 16, 7),
                         qn.multi_linear_bwd_workspace_bytes(512, 256, M, 16, 7)), dtype=torch.uint8, device=dev())

    def calls():
        qn.multi_plan(L.ids, 7, out=L.plan)
        qn.multi_linear_fwd(L.q, L.pool, L.plan, L.X, out=Y, workspace=ws)
        qn.multi_linear_bwd(L.q, L.pool, L.plan, L.X, L.dY, dX=dX, dA=dA, dB=dB, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    rng = np.random.default_rng(M)
    for k in range(4):
        L.ids.copy_(torch.from_numpy(_ids("mixed" if k % 2 else "packed", M, 7, rng)))
        L.X.copy_(torch.randn(L.X.shape, generator=L.gen, device=dev()))
        L.dY.copy_(torch.randn(L.dY.shape, generator=L.gen, device=dev()))
        (torch.randn(256, 256, device=dev()) @ torch.randn(256, 256, device=dev())).sum().item()
        graph.replay()
        torch.cuda.synchronize()
        plan = qn.multi_plan(L.ids, 7)
        eY = qn.multi_linear_fwd(L.q, L.pool, plan, L.X)
        eX, eA, eB = qn.multi_linear_bwd(L.q, L.pool, plan, L.X, L.dY)
        torch.cuda.synchronize()
        for x, y in ((Y, eY), (dX, eX), (dA, eA), (dB, eB)):
            assert torch.equal(x, y), f"replay {k}"


def test_training_step_lowers_the_loss():
    """Plan, forward, gradients and AdamW together: two adapters learn two targets."""
    _say("[multi] training steps")
    L = Layer(256, 256, 240, 16, 2, "mixed", seed=21)
    L.pool.B.zero_()
    target = torch.randn(240, 256, generator=L.gen, device=dev()) * 0.3 + (L.X @ torch.from_numpy(L.W.T).to(dev()).bfloat16()).float()
    masters = [L.pool.A.float(), L.pool.B.float()]
    dA, dB = (torch.empty_like(m) for m in masters)
    opt = qn.adamw_state(masters, [dA, dB], copies=[L.pool.A, L.pool.B], bits=8)
    losses = []
    for step in range(1, 31):
        Y = qn.multi_linear_fwd(L.q, L.pool, L.plan, L.X)
        err = Y.float() - target
        live = (L.ids >= 0)[:, None]
        losses.append((err * live).square().sum().item())
        dY = (err * live * (2.0 / err.numel())).bfloat16()
        qn.multi_linear_bwd(L.q, L.pool, L.plan, L.X, dY, dA=dA, dB=dB)
        qn.adamw_step(opt, step, 3e-3)
    assert losses[-1] < 0.7 * losses[0], losses[::10]
