"""A step of fine-tuning made of the library's calls: the gated block, the down projection, the loss
over the head, the gradients back through all of them, and AdamW on the adapters. The gradients
against float64 (autograd on the dequantised weights); then the adapters' step."""
import pytest
import torch

import bit_nf4_quantized_05_amd as qn
from parity import dev

pytestmark = pytest.mark.gpu

D, F, V, R = 256, 704, 3001, 16


class Model:
    def __init__(self, m, seed=0):
        g = torch.Generator(device=dev()).manual_seed(seed)

        def normal(*shape, sigma=1.0):
            return torch.randn(*shape, generator=g, device=dev()) * sigma

        self.gate, self.up = (qn.quantize(normal(F, D, sigma=1.3 * D ** -0.5)) for _ in range(2))
        self.down = qn.quantize(normal(D, F, sigma=F ** -0.5))
        self.head = normal(V, D, sigma=1.3 * D ** -0.5).bfloat16()
        shapes = [(R, D), (F, R), (R, D), (F, R), (R, F), (D, R)]
        self.masters = [normal(*s, sigma=0.5 * s[1] ** -0.5) for s in shapes]
        self.adapters = [p.bfloat16() for p in self.masters]
        a = self.adapters
        self.layer = qn.GatedLayer(self.gate, self.up, a[0], a[1], 2.0, a[2], a[3], 2.0)
        self.X = normal(m, D).bfloat16()
        self.target = torch.randint(0, V, (m,), generator=g, device=dev())
        self.target[::3] = -100
        self.scale = torch.full((m,), 1.0 / (self.target >= 0).sum().item(), device=dev())
        self.grads = [torch.zeros_like(p) for p in self.masters]
        self.opt = qn.adamw_state(self.masters, self.grads, copies=self.adapters)

    def step(self, number):
        a, g = self.adapters, self.grads
        H, GU = qn.gated_fwd(self.layer, self.X, save=True)
        Y = qn.linear_fwd(self.down, a[4], a[5], 2.0, H)
        loss, dY = qn.head_loss_grad(self.head, Y, self.target, scale=self.scale)
        dH = qn.linear_bwd_x(self.down, a[4], a[5], 2.0, dY)
        qn.lora_grads(a[4], a[5], 2.0, H, dY, dA=g[4], dB=g[5])
        dX, dGU = qn.gated_bwd(self.layer, GU, dH)
        qn.lora_grads(a[0], a[1], 2.0, self.X, dGU[:, :F], dA=g[0], dB=g[1])
        qn.lora_grads(a[2], a[3], 2.0, self.X, dGU[:, F:], dA=g[2], dB=g[3])
        if number:
            qn.adamw_step(self.opt, number, 1e-3)
        return loss, dX

    def exact(self):
        a = [p.double().requires_grad_() for p in self.adapters]
        X = self.X.double().requires_grad_()
        W = [qn.double_dequant(w).double() for w in (self.gate, self.up, self.down)]
        G, U = (X @ w.T + 2.0 * (X @ A.T) @ B.T for w, A, B in ((W[0], a[0], a[1]), (W[1], a[2], a[3])))
        H = torch.nn.functional.silu(G) * U
        Z = (H @ W[2].T + 2.0 * (H @ a[4].T) @ a[5].T) @ self.head.double().T
        live = self.target >= 0
        loss = torch.where(live, torch.logsumexp(Z, 1) - Z.gather(1, self.target.clamp_min(0)[:, None])[:, 0], 0)
        grads = torch.autograd.grad((loss * self.scale.double()).sum(), [X, *a])
        return loss.detach(), grads[0], grads[1:]


def _far(x, ref):
    return ((x.double() - ref).norm() / ref.norm()).item()


@pytest.mark.parametrize("m", [40, 300])
def test_gradients_of_a_step(m):
    model = Model(m)
    loss, dX = model.step(0)
    ref_loss, ref_dx, ref = model.exact()
    # each of at most 8 roundings to bf16 on the way (H, Y, T, dY, dH, dG|dU, U', dX) is off by 2^-8 of
    # its value at most, and random-weight products carry a relative error on as it is
    tol = 8 * 2.0 ** -8
    assert _far(loss, ref_loss) <= tol and _far(dX, ref_dx) <= tol
    for got, want in zip(model.grads, ref):
        assert _far(got, want) <= tol


def test_steps_change_every_adapter():
    model = Model(300)
    before = [p.clone() for p in model.adapters]
    for k in (1, 2, 3):
        loss, _ = model.step(k)
        assert torch.isfinite(loss).all()
    for p, q, master in zip(model.adapters, before, model.masters):
        assert not torch.equal(p, q) and torch.equal(p, master.bfloat16())


def test_two_steps_at_once_on_two_streams():
    """The same step of two models on two streams, each with what it allocates there."""
    want = []
    for seed in (1, 2):
        loss, dX = Model(300, seed).step(0)
        want.append((loss, dX))
    models = [Model(300, seed) for seed in (1, 2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i] = models[i].step(0)
    torch.cuda.synchronize()
    for (loss, dX), (l, d) in zip(got, want):
        assert torch.equal(loss, l) and torch.equal(dX, d)
