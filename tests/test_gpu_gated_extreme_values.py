"""Infinities and NaN in a token of a small batch stay with it, in every kernel of up to 64 tokens: those
that multiply pieces past a row by zeroed weights, and tokens past the last one, among them."""
import pytest
import torch

import bit_nf4_quantized_05_amd as qn
from parity import dev
from test_gpu_gated import make

pytestmark = pytest.mark.gpu

# d_ff, d_in, tokens, rank: ranks formed by every workgroup (1..4 tokens, r <= 16), by a launch of their own, none; odd
# numbers of blocks in a row; longer rows with 16 waves a tile, with 4; two, three and four token tiles
CASES = [(128, 320, 4, 16), (128, 320, 16, 16), (704, 1088, 3, 40), (320, 4096, 16, 0), (64, 4160, 5, 16), (64, 9280, 2, 9),
         (64, 4160, 16, 16), (128, 320, 17, 9), (192, 2112, 32, 16), (128, 320, 33, 0), (192, 1088, 48, 33), (128, 320, 64, 16)]


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("d_ff,d_in,m,r", CASES, ids=["x".join(map(str, c)) for c in CASES])
def test_extreme_values_stay_with_their_token(d_ff, d_in, m, r, value):
    print("[gated]", value, d_ff, d_in, m, r, flush=True)
    layer, normal = make(d_ff, d_in, r, "silu")
    X = normal(m, d_in).bfloat16()
    want = qn.gated_fwd(layer, X, save=True)
    # the last value of a row is in the piece that is read again past it; the last token's values are
    # read again for the tokens past it
    for t, k in {(0, 3), (m // 2, d_in - 1), (m - 1, d_in - 64)}:
        bad = X.clone()
        bad[t, k] = value
        rows = torch.ones(m, dtype=torch.bool, device=dev())
        rows[t] = False
        for got, w in zip(qn.gated_fwd(layer, bad, save=True), want):
            assert torch.equal(got[rows], w[rows])
            assert not torch.isfinite(got[t].float()).all()


@pytest.mark.parametrize("d_ff,d_in,m,r", CASES, ids=["x".join(map(str, c)) for c in CASES])
def test_extreme_gradients_stay_with_their_token(d_ff, d_in, m, r):
    layer, normal = make(d_ff, d_in, r, "gelu")
    GU, dH = normal(m, 2 * d_ff).bfloat16(), normal(m, d_ff).bfloat16()
    want = qn.gated_bwd(layer, GU, dH)
    for t, k, value in ((0, 1, float("inf")), (m - 1, d_ff - 1, float("nan"))):
        bad = dH.clone()
        bad[t, k] = value
        rows = torch.ones(m, dtype=torch.bool, device=dev())
        rows[t] = False
        for got, w in zip(qn.gated_bwd(layer, GU, bad), want):
            assert torch.equal(got[rows], w[rows])
            assert not torch.isfinite(got[t].float()).all()
