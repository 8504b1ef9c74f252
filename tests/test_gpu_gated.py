"""The gated feed-forward block on the GPU against float64 on the dequantised weights.

Tolerances, per element, from the arithmetic (f = 2^-24 and b = 2^-8, half a step of float32
and bfloat16; |.| sums over the products' terms):
  G, U   2 n f sum|x w| for the float32 sums of n terms, b sum|t b| for the rank products
         rounded to bf16 once
  H      b |H| for its one rounding, |act| dU + 1.2 |U| dG + 1.2 dG dU for those two (|act'| < 1.2),
         and 100 2^-22 of |act U| for the activation (2^x, 1/x of 1 ulp each, x up to 100)
  dG     b |dG|, and 100 2^-22 of |dH U| times the terms of act' (64 2^-24 where 1 - sigma cancels)
  dX     from dG, dU as the call rounded them: b |dX|, 2 n f sum|dY w|, b sum|u a|"""
import pytest
import torch

import bit_nf4_quantized_05_amd as qn
from oracle import gated_oracle as GO
from parity import dev

pytestmark = pytest.mark.gpu

F, B8, ACT = 2.0 ** -24, 2.0 ** -8, 100 * 2.0 ** -22
# d_ff, d_in, tokens, rank, activation, second level
CASES = [(64, 64, 1, 1, "silu", "int8"), (64, 128, 3, 0, "gelu", "int8"), (128, 320, 17, 9, "silu", "fp8"),
         (512, 256, 203, 8, "gelu", "int8"), (192, 1088, 65, 33, "silu", "none"), (64, 4096, 64, 16, "gelu", "int8"),
         (704, 1024, 300, 64, "silu", "int8"), (320, 4096, 130, 16, "gelu", "fp8"), (4160, 128, 1025, 100, "silu", "int8"),
         (2752, 512, 1, 16, "silu", "none"), (1088, 2112, 24, 256, "gelu", "int8"), (128, 64, 257, 24, "silu", "int8"),
         (1024, 4032, 7, 16, "silu", "int8"), (192, 3968, 16, 5, "gelu", "none"), (9152, 64, 2, 11, "silu", "fp8"),
         (64, 4160, 4, 16, "gelu", "int8"), (640, 640, 9, 17, "silu", "int8"), (128, 2048, 33, 16, "silu", "int8"),
         (66624, 64, 3, 16, "silu", "int8"), (2112, 1024, 1540, 40, "silu", "int8"), (64, 2816, 3000, 16, "gelu", "fp8")]
IDS = ["x".join(map(str, c)) for c in CASES]


def _say(*a):
    print(*a, flush=True)


def make(d_ff, d_in, r, act, dq="int8", seed=0):
    g = torch.Generator(device=dev()).manual_seed(seed)

    def normal(*shape, sigma=1.0):
        return torch.randn(*shape, generator=g, device=dev()) * sigma

    ws = [qn.quantize(normal(d_ff, d_in, sigma=1.3 * d_in ** -0.5), dq=dq) for _ in range(2)]
    ab = [(normal(r, d_in, sigma=0.5 * d_in ** -0.5).bfloat16(), normal(d_ff, r, sigma=0.5 * r ** -0.5).bfloat16())
          for _ in range(2)] if r else [(None, None)] * 2
    return qn.GatedLayer(ws[0], ws[1], *ab[0], 2.0, *ab[1], 0.75, act), normal


def halves(layer):
    """(W, A, B, s) of both projections in float64; no adapter: rank 0."""
    out = []
    for w, A, B, s in ((layer.gate, layer.A_gate, layer.B_gate, layer.s_gate), (layer.up, layer.A_up, layer.B_up, layer.s_up)):
        W = qn.double_dequant(w).double()
        out.append((W, W.new_zeros(0, layer.d_in) if A is None else A.double(),
                    W.new_zeros(layer.d_ff, 0) if B is None else B.double(), s))
    return out


def _numpy(*ts):
    return [t.cpu().numpy() for t in ts]


def act64(g, kind):
    return torch.from_numpy(GO.act(g.cpu().numpy(), kind)).to(g.device)


def sums(half, X):
    """A projection in float64, and what its float32 sums and rounded rank product may be off by."""
    W, A, B, s = half
    T = s * (X @ A.T)
    n = W.shape[1] + 2 * A.shape[0] + 8
    mass = X.abs() @ W.abs().T + (T.abs() @ B.abs().T)
    return X @ W.T + T @ B.T, 2 * n * F * mass + (B8 + n * F) * (T.abs() @ B.abs().T)


def within(got, ref, tol, what):
    assert torch.isfinite(got.double()).all(), what
    bad = (got.double() - ref).abs() - tol
    assert bad.max().item() <= 0, f"{what}: {bad.max().item():.3e} past the bound at {bad.argmax().item()}"


def check_forward(layer, X, H, GU):
    (g, eg), (u, eu) = (sums(h, X.double()) for h in halves(layer))
    a = act64(g, layer.act)
    # the upper bounds on H's terms take |act(g)| at g plus its own error
    tol = (B8 * (a * u).abs() + (a.abs() + 1.2 * eg) * eu + 1.2 * u.abs() * eg + ACT * (a * u).abs() +
           ACT * (g.abs() + eg) * eu) * 1.01 + 1e-30
    within(H, a * u, tol, "H")
    if GU is not None:
        within(GU[:, :layer.d_ff], g, B8 * (g.abs() + eg) + eg, "G")
        within(GU[:, layer.d_ff:], u, B8 * (u.abs() + eu) + eu, "U")


def check_gradient(layer, GU, dH, dGU, dX):
    G, U = GU[:, :layer.d_ff].double(), GU[:, layer.d_ff:].double()
    h = dH.double()
    dG, dU = (torch.from_numpy(x).to(dH.device) for x in GO.grads(*_numpy(G, U, h), layer.act))
    hu = (h * U).abs()
    # 2.2: the largest sum of the magnitudes of act' terms of either activation
    within(dGU[:, :layer.d_ff], dG, B8 * dG.abs() + hu * (2.2 * ACT + 64 * F) + 1e-37, "dG")
    within(dGU[:, layer.d_ff:], dU, B8 * dU.abs() + ACT * dU.abs() + 1e-37, "dU")
    ref, tol = 0, 0
    for (W, A, B, s), dY in zip(halves(layer), (dGU[:, :layer.d_ff].double(), dGU[:, layer.d_ff:].double())):
        V = s * (dY @ B)
        n = 2 * W.shape[0] + 4 * A.shape[0] + 16
        ref = ref + dY @ W + V @ A
        tol = tol + 2 * n * F * (dY.abs() @ W.abs() + abs(s) * (dY.abs() @ B.abs()) @ A.abs()) + B8 * (V.abs() @ A.abs())
    within(dX, ref, tol * 1.01 + B8 * (ref.abs() + tol) + 1e-37, "dX")


@pytest.mark.parametrize("d_ff,d_in,m,r,act,dq", CASES, ids=IDS)
def test_forward(d_ff, d_in, m, r, act, dq):
    _say("[gated]", d_ff, d_in, m, r, act, dq)
    layer, normal = make(d_ff, d_in, r, act, dq)
    X = normal(m, d_in).bfloat16()
    H, GU = qn.gated_fwd(layer, X, save=True)
    check_forward(layer, X, H, GU)
    # the same H without keeping G and U, and on a second call
    assert torch.equal(qn.gated_fwd(layer, X), H) and torch.equal(qn.gated_fwd(layer, X, save=True)[1], GU)


@pytest.mark.parametrize("d_ff,d_in,m,r,act,dq", CASES, ids=IDS)
def test_gradient(d_ff, d_in, m, r, act, dq):
    _say("[gated gradient]", d_ff, d_in, m, r, act, dq)
    layer, normal = make(d_ff, d_in, r, act, dq)
    GU, dH = normal(m, 2 * d_ff, sigma=2.0).bfloat16(), normal(m, d_ff, sigma=1e-3).bfloat16()
    keep = GU.clone()
    dX, dGU = qn.gated_bwd(layer, GU, dH)
    assert torch.equal(GU, keep)
    check_gradient(layer, GU, dH, dGU, dX)
    # dG and dU in the place of G and U
    dX2, place = qn.gated_bwd(layer, GU, dH, dGU=GU)
    assert place is GU and torch.equal(GU, dGU) and torch.equal(dX2, dX)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_activation_over_its_whole_range(act):
    """Every finite bf16 gate value, up to where g^2 and exp(-g) leave float32."""
    layer, _ = make(64, 64, 0, act)
    bits = torch.arange(-32768, 32768, device=dev(), dtype=torch.int32).to(torch.int16)
    g = bits.view(torch.bfloat16)
    g = g[torch.isfinite(g)]
    m = g.numel() // 64
    G = g[:64 * m].view(m, 64)
    GU = torch.cat([G, torch.ones_like(G)], 1)
    dX, dGU = qn.gated_bwd(layer, GU, torch.ones_like(G))
    x = G.double()
    if act == "silu":
        s = torch.sigmoid(x)
        da, a = s + x * s * torch.sigmoid(-x), x * s
    else:
        inner = 2 * (2 / torch.pi) ** 0.5 * (x + 0.044715 * x ** 3)
        s = torch.sigmoid(inner)
        q = x.clamp(-1e3, 1e3)
        da = s + q * s * torch.sigmoid(-inner) * 2 * (2 / torch.pi) ** 0.5 * (1 + 3 * 0.044715 * q * q)
        a = x * s
    # 1e-37: results below float32's normal range may be flushed. So may a sigma below 2^-126: act =
    # g sigma is then off by |g| sigma < |g| 2^-126 (sigma < 2^-126 needs |g| > 87 (silu), 5 (gelu))
    flushed = torch.where(s < 2.0 ** -126, x.abs() * s, 0)
    within(dGU[:, :64], da, B8 * da.abs() + 2.2 * ACT + 64 * F, "act'")
    within(dGU[:, 64:], a, (B8 + ACT) * a.abs() + flushed + 1e-37, "act")


def test_extreme_values_stay_with_their_token():
    layer, normal = make(192, 256, 16, "silu")
    X = normal(300, 256).bfloat16()
    clean = qn.gated_fwd(layer, X, save=True)
    bad = X.clone()
    bad[7, 3], bad[130, 100], bad[299, 255] = float("inf"), float("nan"), float("-inf")
    rows = torch.ones(300, dtype=torch.bool, device=dev())
    rows[[7, 130, 299]] = False
    for got, want in zip(qn.gated_fwd(layer, bad, save=True), clean):
        assert torch.equal(got[rows], want[rows])
        assert not torch.isfinite(got[~rows].float()).all(1).any()
    dH = normal(300, 192).bfloat16()
    GU = clean[1]
    want = qn.gated_bwd(layer, GU, dH)
    dH[7, 3], dH[130, 100], dH[299, 191] = float("inf"), float("nan"), float("-inf")
    for got, w in zip(qn.gated_bwd(layer, GU, dH), want):
        assert torch.equal(got[rows], w[rows])
        assert not torch.isfinite(got[~rows].float()).all(1).any()


@pytest.mark.parametrize("m", [5, 70, 300])
def test_windows_of_wider_arrays(m):
    layer, normal = make(320, 192, 16, "gelu")
    f, d = 320, 192

    def window(cols, offset):
        wide = torch.full((m, cols + 40), 7.0, dtype=torch.bfloat16, device=dev())
        return wide, wide[:, offset:offset + cols]

    (xw, X), (hw, H), (gw, GU) = window(d, 8), window(f, 16), window(2 * f, 24)
    X.copy_(normal(m, d))
    want = qn.gated_fwd(layer, X.contiguous(), save=True)
    qn.gated_fwd(layer, X, out=H, GU=GU)
    assert torch.equal(H, want[0]) and torch.equal(GU, want[1])
    (dw, dH), (ow, dGU), (ew, dX) = window(f, 8), window(2 * f, 16), window(d, 32)
    dH.copy_(normal(m, f))
    wx, wg = qn.gated_bwd(layer, want[1], dH.contiguous())
    qn.gated_bwd(layer, GU, dH, dX=dX, dGU=dGU)
    assert torch.equal(dX, wx) and torch.equal(dGU, wg)
    for wide, cols, at in ((hw, f, 16), (gw, 2 * f, 24), (ow, 2 * f, 16), (ew, d, 32)):
        assert (wide[:, :at] == 7).all() and (wide[:, at + cols:] == 7).all()


def test_gradient_against_differences():
    """dX and the adapters' gradients as slopes of <dH, H>: the float64 forward at points beside X
    and the adapters. Steps of 2^-10 of unit-size values; the bounds allow bf16's rounding of dG, dU
    and dX (b each) over the directions' mass."""
    layer, normal = make(128, 64, 16, "silu", seed=5)
    X, dH = normal(33, 64).bfloat16(), normal(33, 128).bfloat16()
    _, GU = qn.gated_fwd(layer, X, save=True)
    dX, dGU = qn.gated_bwd(layer, GU, dH)

    def value(hs, x):
        (g, _), (u, _) = (sums(h, x) for h in hs)
        return (dH.double() * act64(g, layer.act) * u).sum()

    hs, h = halves(layer), 2.0 ** -10
    for k in range(3):
        d = normal(33, 64).double()
        slope = (value(hs, X.double() + h * d) - value(hs, X.double() - h * d)) / (2 * h)
        # G, U rounded to bf16 move dG, dU by b of their own size, and so do the roundings of both and of dX
        mass = sum((dY.double().abs() @ w.abs()) + (dY.double().abs() @ B.abs()) @ A.abs() * abs(s)
                   for (w, A, B, s), dY in zip(hs, (dGU[:, :128], dGU[:, 128:])))
        scale = (mass * d.abs()).sum()
        assert abs(slope - (dX.double() * d).sum()) <= 8 * B8 * scale
    for i, (A, B, s, dY) in enumerate(((layer.A_gate, layer.B_gate, layer.s_gate, dGU[:, :128]),
                                       (layer.A_up, layer.B_up, layer.s_up, dGU[:, 128:]))):
        dA, dB = qn.lora_grads(A, B, s, X, dY)
        for which, grad in ((1, dA), (2, dB)):
            d = normal(*grad.shape).double()
            moved = []
            for sign in (1, -1):
                part = list(hs[i])
                part[which] = part[which] + sign * h * d
                moved.append(value([tuple(part), hs[1]] if i == 0 else [hs[0], tuple(part)], X.double()))
            slope = (moved[0] - moved[1]) / (2 * h)
            x, y = X.double().abs(), dY.double().abs()
            mass = ((y @ B.double().abs()).T @ x if which == 1 else y.T @ (x @ A.double().abs().T)) * abs(s)
            assert abs(slope - (grad.double() * d).sum()) <= 8 * B8 * (mass * d.abs()).sum()


@pytest.mark.parametrize("m", [1, 24, 300])
def test_replayed_from_a_graph(m):
    """A captured forward and gradient, replayed on new inputs with eager work in between."""
    layer, normal = make(704, 1024, 16, "silu")
    f, d = 704, 1024
    X, dH = normal(m, d).bfloat16(), normal(m, f).bfloat16()
    H, GU = torch.empty(m, f, dtype=torch.bfloat16, device=dev()), torch.empty(m, 2 * f, dtype=torch.bfloat16, device=dev())
    dX, dGU = torch.empty_like(X), torch.empty_like(GU)
    need = max(qn.gated_fwd_workspace_bytes(f, d, m, 16), qn.gated_bwd_workspace_bytes(f, d, m, 16))
    ws = torch.empty(need, dtype=torch.uint8, device=dev())

    def calls():
        qn.gated_fwd(layer, X, out=H, GU=GU, workspace=ws)
        qn.gated_bwd(layer, GU, dH, dX=dX, dGU=dGU, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for _ in range(4):
        X.copy_(normal(m, d))
        dH.copy_(normal(m, f))
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (H, GU, dX, dGU)]
        (a @ a).sum().item() if (a := torch.randn(256, 256, device=dev())) is not None else None
        wh, wg = qn.gated_fwd(layer, X, save=True)
        wx, wd = qn.gated_bwd(layer, wg, dH)
        for g, w in zip(got, (wh, wg, wx, wd)):
            assert torch.equal(g, w)


@pytest.mark.parametrize("m", [3, 40, 70])
def test_offsets_past_2_gib(m):
    """Both weights together 3.76 GB in bf16: the last outputs of the forward, the last columns and the sums
    over all rows of the gradient."""
    f, d = 65536, 14336
    layer, normal = make(f, d, 8, "silu")
    rows = torch.tensor([0, 1, f // 2, f - 2, f - 1], device=dev())
    cols = torch.tensor([0, 63, d - 64, d - 1], device=dev())
    X, dH = normal(m, d).bfloat16(), normal(m, f).bfloat16()
    H, GU = qn.gated_fwd(layer, X, save=True)
    dX, dGU = qn.gated_bwd(layer, GU, dH)
    x, want, mass = X.double(), 0.0, 0.0
    for k, (w, A, B, s) in enumerate(((layer.gate, layer.A_gate, layer.B_gate, layer.s_gate),
                                      (layer.up, layer.A_up, layer.B_up, layer.s_up))):
        W = qn.double_dequant(w)
        A, B = A.double(), B.double()
        y, a = x @ W[rows].double().T + s * (x @ A.T) @ B[rows].T, x.abs() @ W[rows].double().abs().T
        low = abs(s) * (x.abs() @ A.abs().T) @ B[rows].abs().T
        # d float32 products; the rank product's rounding; the output's
        within(GU[:, k * f:(k + 1) * f][:, rows], y, 2 * d * F * a + (2 * B8 + 2 * d * F) * low + B8 * y.abs(), "G or U")
        dY = dGU[:, k * f:(k + 1) * f].double()
        Wc = W[:, cols].double()
        want = want + dY @ Wc + s * (dY @ B) @ A[:, cols]
        mass = mass + 2 * f * F * (dY.abs() @ Wc.abs()) + (2 * B8 + 2 * f * F) * abs(s) * (dY.abs() @ B.abs()) @ A[:, cols].abs()
        del W
    within(dX[:, cols], want, 2 * mass + B8 * want.abs(), "dX")
