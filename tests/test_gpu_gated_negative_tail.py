"""act' and dG where the gate is negative, relative to the derivative's own terms.

There nothing cancels in 1 - sigma (sigma <= 1/2), so that the kernel's two terms of act' = sigma + g sigma
(1 - sigma) x' (x' = 1 of silu, c2 (1 + 3 k g^2) of gelu) are each off by a relative error, counted in half
steps f = 2^-24 of float32:
  2^e and 1 / (1 + 2^e) of 1 ulp each, and the sum's rounding: 5 f
  the exponent e = x log2 e: |x| f for each of the product, the constant and x's own 7 steps: 9 |x| f
  the other products, sums and constants of both terms and of dG: 16 f
sigma is either right to that, or below float32's normal range and flushed (to 0, or any value up to 2^-126):
then the terms are off by their size. dG is the product with dH U, rounded to bf16 (2^-8)."""
import pytest
import torch

import bit_nf4_quantized_05_amd as qn
from parity import dev

pytestmark = pytest.mark.gpu

F, B8, TINY = 2.0 ** -24, 2.0 ** -8, 2.0 ** -126
C2, K = 2 * (2 / torch.pi) ** 0.5, 0.044715


def terms(g, act):
    """sigma, the two terms of act', and the exponent's size, in float64."""
    x = g if act == "silu" else C2 * (g + K * g ** 3)
    dx = torch.ones_like(g) if act == "silu" else C2 * (1 + 3 * K * g * g)
    s = torch.sigmoid(x)
    return s, s, g * s * torch.sigmoid(-x) * dx, x.abs()


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("d_ff", [128, 32640])
def test_every_negative_gate_value(act, d_ff):
    bits = torch.arange(-32768, 0, device=dev(), dtype=torch.int32).to(torch.int16)
    g = bits.view(torch.bfloat16)
    G = g[torch.isfinite(g)].view(-1, d_ff)
    W = torch.zeros(d_ff, 64, device=dev())
    W[:, 0] = 1.0
    w = qn.quantize(W)
    layer = qn.GatedLayer(w, w, act=act)
    # dH U = 2^3 exactly, so that dG is the rounded derivative, scaled
    U, dH = torch.full_like(G, 16.0), torch.full_like(G, 0.5)
    _, dGU = qn.gated_bwd(layer, torch.cat([G, U], 1), dH)
    got = dGU[:, :d_ff].double() / 8
    s, one, two, x = terms(G.double(), act)
    want = one + two
    rel = (21 + 9 * x) * F
    mass = one.abs() + two.abs()
    # a sigma below the normal range, or a term that falls below it
    lost = torch.where(s < 2 * TINY, mass, 0) + 4 * TINY
    bound = (rel * mass + lost) * 1.01 + B8 * (want.abs() + rel * mass) + 2.0 ** -133
    off = (got - want).abs() - bound
    assert torch.isfinite(got).all()
    assert off.max().item() <= 0, f"{off.max().item():.3e} past the bound at g = {G.flatten()[off.argmax()].item()}"
    # nothing else than the rounding is allowed in the tail where the derivative is an ordinary number
    tail = (G.double() < -14) & (s > 4 * TINY) if act == "silu" else (G.double() < -5) & (s > 4 * TINY)
    if tail.any():
        assert ((got - want).abs()[tail] <= 0.01 * want.abs()[tail]).all()
        assert (got[tail] < 0).all()
