"""The rank products of the gated block carry no rounding of their own to the outputs, whatever the
number of tokens.

With weights so small that the rank term makes up G, U and dX, they are compared with the correctly
rounded bf16 of the float64 result (dX with that of dG and dU as the call returned them). Rank products of
at least 16 bits are off by 2^-18 / sqrt(3) of each product at the root mean square, float32 sums by no
more (partial sums of n terms in steps of 32: sqrt(n / 32) 2^-25 / sqrt(3), under 2^-20 for the 8320 terms of
the longest sum here): an error of 2^-18 of the output's root mean square Y. The output's rounding falls on
the other side with probability error / ulp, and ulp >= |y| 2^-8; over a normal y the mean of Y / |y| from
the error on is 0.8 ln(2^18) = 10: 2^-18 2^8 10 = 1 %. Twice that is allowed. Products rounded to bf16
(2^-9) change 40 % of the elements."""
import pytest
import torch

import bit_nf4_quantized_05_amd as qn
from parity import dev
from test_gpu_gated import check_forward, check_gradient, halves, make

pytestmark = pytest.mark.gpu

SHARE = 0.02


def rank_layer(d_ff, d_in, r, act, seed):
    g = torch.Generator(device=dev()).manual_seed(seed)

    def normal(*shape, sigma=1.0):
        return torch.randn(*shape, generator=g, device=dev()) * sigma

    ws = [qn.quantize(normal(d_ff, d_in, sigma=1e-6)) for _ in range(2)]
    ab = [(normal(r, d_in, sigma=d_in ** -0.5).bfloat16(), normal(d_ff, r, sigma=r ** -0.5).bfloat16()) for _ in range(2)]
    return qn.GatedLayer(ws[0], ws[1], *ab[0], 2.0, *ab[1], 0.75, act), normal


def off(got, ref):
    """The share of elements that are not the rounded result."""
    return (got.view(torch.int16) != ref.float().bfloat16().view(torch.int16)).double().mean().item()


# tiles of 64 and of 256, K in one slice and in several, one workgroup's ranks and more, r % 8 != 0
@pytest.mark.parametrize("d_ff,d_in,m,r", [(256, 512, 3, 16), (256, 512, 40, 64), (64, 4160, 9, 16), (256, 512, 65, 16),
                                           (256, 512, 80, 9), (256, 512, 300, 64), (256, 512, 300, 33), (256, 512, 1025, 256),
                                           (6400, 512, 300, 64), (4160, 128, 300, 24), (320, 1088, 130, 17)])
def test_outputs_are_the_rounded_result(d_ff, d_in, m, r):
    print(f"[gated] rank products of {m} tokens, {d_ff} x {d_in}, r={r}", flush=True)
    layer, normal = rank_layer(d_ff, d_in, r, "silu", 3 * m + r)
    X, dH = normal(m, d_in).bfloat16(), normal(m, d_ff).bfloat16()
    _, GU = qn.gated_fwd(layer, X, save=True)
    dX, dGU = qn.gated_bwd(layer, GU, dH)
    x, want = X.double(), 0
    shares = []
    for k, (W, A, B, s) in enumerate(halves(layer)):
        cols = slice(k * d_ff, (k + 1) * d_ff)
        shares.append(off(GU[:, cols].contiguous(), x @ W.T + s * (x @ A.T) @ B.T))
        dY = dGU[:, cols].double()
        want = want + dY @ W + s * (dY @ B) @ A
    shares.append(off(dX, want))
    print("[gated] off the rounded result: G {:.4f}, U {:.4f}, dX {:.4f}".format(*shares), flush=True)
    assert max(shares) <= SHARE


def test_two_million_tokens_at_the_largest_rank():
    """Both terms of the rank products would reach 4 GiB: the call takes one, with the bounds of one
    rounding to bf16."""
    m = (1 << 21) + 3
    layer, normal = make(64, 64, 256, "silu")
    X, dH = normal(m, 64).bfloat16(), normal(m, 64, sigma=1e-3).bfloat16()
    H, GU = qn.gated_fwd(layer, X, save=True)
    dX, dGU = qn.gated_bwd(layer, GU, dH)
    rows = torch.tensor([0, 1, 63, 64, 255, 256, 1 << 20, (1 << 21) - 1, 1 << 21, m - 2, m - 1], device=dev())
    check_forward(layer, X[rows], H[rows], GU[rows])
    check_gradient(layer, GU[rows], dH[rows], dGU[rows], dX[rows])
