"""The rank products of the multi-adapter calls carry no rounding of their own to the outputs.

With adapters so large that the rank term makes up the output, Y and dX are compared with the
correctly rounded bf16 of the float64 result. Rank products of at least 16 bits are off by
2^-18 / sqrt(3) of each product at the root mean square, float32 sums of up to 512 terms by
no more: an error of 2^-18 of the output's root mean square Y. The output's rounding falls
on the other side with probability error / ulp, and ulp >= |y| 2^-8; over a normal y the
mean of Y / |y| from the error on is 0.8 ln(2^18) = 10: 2^-18 * 2^8 * 10 = 1 %. Twice that is
allowed. Products rounded to bf16 (2^-9) change 40 % of the elements."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_05_amd as qn
from oracle import nf4_oracle as O
from parity import bf16_bits, dev
from test_gpu_multi import Layer, _f64

pytestmark = pytest.mark.gpu

SHARE = 0.02


def _layer(M, r, n, kind, d_out=256, d_in=512):
    L = Layer(d_out, d_in, M, r, n, kind, seed=3 * M + r)
    L.pool.B.copy_((torch.randn(L.pool.B.shape, generator=L.gen, device=dev())).bfloat16())
    L.B = _f64(L.pool.B)
    return L


def _off(got, ref, ids, n):
    """The share of elements that are not the rounded result, over the tokens with an adapter."""
    rows = np.flatnonzero((ids >= 0) & (ids < n))
    want = O.f32_to_bf16_bits(ref[rows].astype(np.float32))
    return float(np.mean(bf16_bits(got)[rows] != want))


@pytest.mark.parametrize("M,r,n,kind", [(1, 16, 2, "one"), (1, 48, 2, "one"), (7, 16, 3, "mixed"), (30, 64, 30, "mixed"),
                                        (64, 256, 4, "mixed"), (64, 32, 1, "one"), (80, 16, 6, "mixed"),
                                        (300, 16, 1, "one"), (300, 32, 3, "packed"), (300, 48, 40, "mixed"),
                                        (700, 64, 3, "packed"), (700, 112, 2, "mixed"), (700, 256, 2, "one"),
                                        (1000, 16, 500, "mixed"), (1000, 240, 3, "packed")])
def test_outputs_are_the_rounded_result(M, r, n, kind):
    print(f"[multi] rank products of {M} tokens, r={r}, {n} adapters, {kind}", flush=True)
    L = _layer(M, r, n, kind)
    Y = qn.multi_linear_fwd(L.q, L.pool, L.plan, L.X)
    dX, _, _ = qn.multi_linear_bwd(L.q, L.pool, L.plan, L.X, L.dY)
    torch.cuda.synchronize()
    y, x = _off(Y, L.forward(), L.ids_np, n), _off(dX, L.backward()[0], L.ids_np, n)
    print(f"[multi] off the rounded result: Y {y:.4f}, dX {x:.4f}", flush=True)
    assert y <= SHARE and x <= SHARE


@pytest.mark.parametrize("value", [float("inf"), float("nan")])
@pytest.mark.parametrize("M", [40, 300])
def test_an_infinite_rank_product_stays(M, value):
    """A token of infinities keeps an infinity or NaN in its own outputs, and only there."""
    print(f"[multi] {value} in a token of {M}", flush=True)
    L = _layer(M, 32, 3, "mixed")
    t = int(np.flatnonzero(L.ids_np == 1)[0])
    ref = qn.multi_linear_fwd(L.q, L.pool, L.plan, L.X)
    L.X[t, 3] = value
    Y = qn.multi_linear_fwd(L.q, L.pool, L.plan, L.X)
    torch.cuda.synchronize()
    rows = [k for k in range(M) if k != t]
    assert torch.equal(Y[rows].view(torch.int16), ref[rows].view(torch.int16))
    assert not torch.isfinite(Y[t].float()).any()
