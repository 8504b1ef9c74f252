"""The loss over a large vocabulary on the GPU against float64.

Tolerances from the arithmetic (f = 2^-24, b = 2^-8: half a step of float32 and bfloat16). A logit is
a float32 sum of d products: off by e = 2 d f sum|x w| at most. Every exponential is then off by the
relative error rel = 2 e + |z_v - z_y| 2^-22 + 2^-20 (the reference's logit too; the exponent's
rounding, log2 e and 2^x), its sum by 128 + V / 256 half steps more, and
  loss   rel (1 - p_y) + 4 f loss      (loss = log1p(l): d loss = dl / (1 + l))
  dX     scale ((b + 2 rel + 2 V f) sum_{v != y} p_v |W_v| + 2 rel (1 - p_y) |W_y|) + b |dX|"""
import pytest
import torch

import bit_nf4_quantized_05_amd as qn
from parity import dev

pytestmark = pytest.mark.gpu

F, B8 = 2.0 ** -24, 2.0 ** -8
# vocabulary, width, tokens, share without a target, head
CASES = [(1, 64, 1, 0.0, "bf16"), (2, 64, 3, 0.0, "bf16"), (257, 64, 5, 0.0, "bf16"), (1001, 256, 203, 0.3, "bf16"),
         (64, 128, 70, 0.0, "int8"), (4160, 320, 300, 0.5, "fp8"), (20000, 128, 65, 0.0, "bf16"), (33000, 192, 513, 0.2, "bf16"),
         (16448, 128, 257, 0.1, "none"), (50001, 64, 17, 0.0, "bf16"), (40000, 1088, 1, 0.0, "bf16"), (512, 64, 1025, 0.97, "bf16"),
         (300, 64, 9001, 0.4, "bf16"), (33000, 64, 100, 0.2, "bf16"), (33024, 128, 128, 0.1, "int8"), (32000, 64, 300, 0.0, "int8")]
IDS = ["x".join(map(str, c)) for c in CASES]


def _say(*a):
    print(*a, flush=True)


def make(V, d, m, masked=0.0, head="bf16", gain=1.0, seed=0):
    """(head, its float64 values, X, targets, scale)."""
    g = torch.Generator(device=dev()).manual_seed(seed)
    W = torch.randn(V, d, generator=g, device=dev()) * (1.3 * d ** -0.5)
    if head == "bf16":
        own = W.bfloat16()
        full = own.double()
    else:
        own = qn.quantize(W, dq=head)
        full = qn.double_dequant(own).double()
    t = torch.randint(0, V, (m,), generator=g, device=dev())
    lift = torch.rand(m, 1, generator=g, device=dev()) * 16 / 1.69
    X = ((torch.randn(m, d, generator=g, device=dev()) + lift * W[t]) * gain).bfloat16()
    hidden = torch.rand(m, generator=g, device=dev()) < masked
    outside = torch.tensor([-100, -1, V, V + 5, 2 ** 40, -2 ** 62], device=dev())
    t = torch.where(hidden, outside[torch.arange(m, device=dev()) % 6], t)
    return own, full, X, t, torch.rand(m, generator=g, device=dev()) + 0.1


def check(full, X, t, scale, loss, dX):
    V, d = full.shape
    live = (t >= 0) & (t < V)
    assert (loss[~live] == 0).all()
    if dX is not None:
        assert (dX[~live] == 0).all()
    if not live.any():
        return
    x, y = X[live].double(), t[live][:, None]
    z = x @ full.T
    e = 2 * d * F * (x.abs() @ full.abs().T)
    ref = torch.logsumexp(z, 1) - z.gather(1, y)[:, 0]
    rel = (e.amax(1) * 2 + (z - z.gather(1, y)).abs().amax(1) * 2.0 ** -22 + 2.0 ** -20 + (128 + V / 256) * F)
    p = torch.softmax(z, 1)
    rest = p.scatter(1, y, 0.0)
    some = rest.sum(1)
    # where a logit error is not small the loss moves by the error itself, not by its share
    off = (loss[live].double() - ref).abs()
    tol = torch.where(rel < 0.01, 1.02 * rel * some, 2 * e.amax(1) + rel) + 4 * F * ref.abs()
    assert torch.isfinite(loss).all()
    assert (off <= tol).all(), f"loss: {(off - tol).max().item():.3e} past the bound"
    if dX is None:
        return
    s = scale[live].double()[:, None] if scale is not None else 1.0
    want = s * (rest @ full - some[:, None] * full[y[:, 0]])
    r = 1.02 * rel[:, None]
    tol = s * ((B8 + 2 * r + 2 * V * F) * (rest @ full.abs()) + 2 * r * some[:, None] * full[y[:, 0]].abs())
    tol = tol * 1.01 + B8 * want.abs() + 1e-37
    assert torch.isfinite(dX.float()).all()
    off = (dX[live].double() - want).abs()
    assert (off <= tol).all(), f"dX: {(off - tol).max().item():.3e} past the bound"


@pytest.mark.parametrize("V,d,m,masked,head", CASES, ids=IDS)
def test_loss_and_gradient(V, d, m, masked, head):
    _say("[head loss]", V, d, m, masked, head)
    own, full, X, t, scale = make(V, d, m, masked, head)
    loss, dX = qn.head_loss_grad(own, X, t, scale=scale)
    check(full, X, t, scale, loss, dX)
    alone = qn.head_loss(own, X, t)
    check(full, X, t, scale, alone, None)
    again = qn.head_loss_grad(own, X, t, scale=scale)
    assert torch.equal(again[0], loss) and torch.equal(again[1], dX) and torch.equal(qn.head_loss(own, X, t), alone)


@pytest.mark.parametrize("V,m", [(700, 40), (20000, 300)])
@pytest.mark.parametrize("gain", [8.0, 60.0])
def test_logits_far_above_the_target(V, m, gain):
    """Exponentials relative to the target's logit that would leave float32 (differences of hundreds)
    are scaled down per row: in one tile, and after earlier pieces of the vocabulary."""
    own, full, X, t, scale = make(V, 128, m, 0.1, "bf16", gain)
    x = X.double()
    z = x @ full.T
    # targets among the least likely rows, so that others are far above them
    t = torch.where((t >= 0) & (t < V), z.argsort(1)[torch.arange(m, device=dev()), torch.arange(m, device=dev()) % 5], t)
    over = ((z.amax(1) - z.gather(1, t.clamp(0, V - 1)[:, None])[:, 0]) > 60).sum().item()
    _say("[head loss] rows past the range:", over)
    loss, dX = qn.head_loss_grad(own, X, t, scale=scale)
    check(full, X, t, scale, loss, dX)
    check(full, X, t, scale, qn.head_loss(own, X, t), None)


@pytest.mark.parametrize("m", [101, 270])
def test_a_later_piece_far_above_the_earlier_ones(m):
    V, d = 33000, 64
    own, full, X, t, scale = make(V, d, m)
    own[20000:20003] = (X[:3].float() * 8).bfloat16()          # huge logits for some tokens, late in the vocabulary
    own[32999] = (X[100].float() * 16).bfloat16()
    loss, dX = qn.head_loss_grad(own, X, t, scale=scale)
    check(own.double(), X, t, scale, loss, dX)
    check(own.double(), X, t, scale, qn.head_loss(own, X, t), None)


def test_no_token_counted():
    own, _, X, t, scale = make(1000, 64, 300)
    t.fill_(-100)
    loss = torch.full((300,), 3.0, device=dev())
    dX = torch.full((300, 64), 3.0, dtype=torch.bfloat16, device=dev())
    qn.head_loss_grad(own, X, t, loss=loss, dX=dX)
    assert (loss == 0).all() and (dX == 0).all()
    assert (qn.head_loss(own, X, t) == 0).all()


@pytest.mark.parametrize("V,m", [(3001, 100), (20001, 300), (300, 9001)])
def test_rows_without_a_target_are_not_read(V, m):
    """A padded batch: whatever the rows of the tokens that are not counted hold, and their scales."""
    own, _, X, t, scale = make(V, 64, m, 0.5)
    live = (t >= 0) & (t < V)
    loss, dX = qn.head_loss_grad(own, X, t, scale=scale)
    bad, wild = X.clone(), scale.clone()
    bad[~live] = torch.tensor([float("nan"), float("inf")], device=dev()).repeat(32).bfloat16()
    wild[~live] = float("nan")
    l2, d2 = qn.head_loss_grad(own, bad, t, scale=wild)
    assert torch.equal(l2, loss) and torch.equal(d2, dX) and torch.equal(qn.head_loss(own, bad, t), qn.head_loss(own, X, t))


@pytest.mark.parametrize("V", [3001, 20001])
def test_infinities_stay_with_their_token(V):
    own, _, X, t, scale = make(V, 128, 300)
    loss, dX = qn.head_loss_grad(own, X, t, scale=scale)
    bad = X.clone()
    bad[5, 1], bad[128, 2], bad[299, 3] = float("inf"), float("nan"), float("-inf")
    rows = torch.ones(300, dtype=torch.bool, device=dev())
    rows[[5, 128, 299]] = False
    l2, d2 = qn.head_loss_grad(own, bad, t, scale=scale)
    assert torch.equal(l2[rows], loss[rows]) and torch.equal(d2[rows], dX[rows])
    assert not torch.isfinite(l2[~rows]).any() and not torch.isfinite(d2[~rows].float()).all(1).any()


@pytest.mark.parametrize("m", [5, 300])
def test_windows_of_wider_arrays(m):
    V, d = 3001, 192
    own, full, X, t, scale = make(V, d, m, 0.2)

    def window(rows, src=None):
        wide = torch.full((rows, d + 24), 7.0, dtype=torch.bfloat16, device=dev())
        view = wide[:, 8:8 + d]
        if src is not None:
            view.copy_(src)
        return wide, view

    (_, Wv), (_, Xv), (ow, Ov) = window(V, own), window(m, X), window(m)
    loss, dX = qn.head_loss_grad(own, X, t, scale=scale)
    got = qn.head_loss_grad(Wv, Xv, t, scale=scale, dX=Ov)
    assert torch.equal(got[0], loss) and torch.equal(Ov, dX) and torch.equal(qn.head_loss(Wv, Xv, t), qn.head_loss(own, X, t))
    assert (ow[:, :8] == 7).all() and (ow[:, 8 + d:] == 7).all()


def test_gradient_against_differences():
    own, full, X, t, scale = make(500, 64, 40, 0.2)
    _, dX = qn.head_loss_grad(own, X, t, scale=scale)
    live = (t >= 0) & (t < 500)

    def value(x):
        z = x[live] @ full.T
        return ((torch.logsumexp(z, 1) - z.gather(1, t[live][:, None])[:, 0]) * scale[live].double()).sum()

    g = torch.Generator(device=dev()).manual_seed(9)
    for _ in range(4):
        d = torch.randn(40, 64, generator=g, device=dev(), dtype=torch.float64)
        slope = (value(X.double() + 1e-5 * d) - value(X.double() - 1e-5 * d)) / 2e-5
        # b for dX's rounding and b for the exponentials', over the terms' magnitudes
        p = torch.softmax(X.double() @ full.T, 1)
        mass = ((p @ full.abs() + full.abs()[t.clamp(0, 499)]) * scale.double()[:, None] * d.abs())[live].sum()
        assert abs(slope - (dX.double() * d).sum()) <= 2 * B8 * mass


@pytest.mark.parametrize("V,m,head", [(1001, 7, "bf16"), (20000, 300, "bf16"), (4160, 70, "int8")])
def test_replayed_from_a_graph(V, m, head):
    """Captured once, replayed with other hidden states and other counts of targets."""
    own, full, X, t, scale = make(V, 128, m, 0.3, head)
    loss, dX = torch.empty(m, device=dev()), torch.empty_like(X)
    alone = torch.empty(m, device=dev())
    ws = torch.empty(qn.head_loss_workspace_bytes(own, m, grad=True), dtype=torch.uint8, device=dev())

    def calls():
        qn.head_loss_grad(own, X, t, scale=scale, loss=loss, dX=dX, workspace=ws)
        qn.head_loss(own, X, t, loss=alone, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for k, masked in enumerate((0.0, 0.9, 1.1, 0.4)):
        _, _, x2, t2, _ = make(V, 128, m, masked, head, seed=20 + k)
        X.copy_(x2)
        t.copy_(t2)
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        got = loss.clone(), dX.clone(), alone.clone()
        a = torch.randn(256, 256, device=dev())
        (a @ a).sum().item()
        want = qn.head_loss_grad(own, X, t, scale=scale)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(got[2], qn.head_loss(own, X, t))
        check(full, X, t, scale, got[0], got[1])


@pytest.mark.parametrize("m", [20, 200])
def test_offsets_past_2_gib(m):
    V, d = 30000, 49152
    own, _, X, t, scale = make(V, d, m, 0.1)
    loss, dX = qn.head_loss_grad(own, X, t, scale=scale)
    check(own.double(), X, t, scale, loss, dX)
