"""The gated feed-forward block without a GPU: sizes, refusals, the binding's checks, and the
oracle's gradients against differences."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_05_amd as qn
from bit_nf4_quantized_05_amd import _lib
from oracle import gated_oracle as GO

FAKE = 1 << 20


def _fwd(**kw):
    a = dict(codes_g=FAKE, codes_u=FAKE, qscale=FAKE, d_ff=64, d_in=128, dq=0, A=FAKE, B=FAKE, r=8, act=0, X=FAKE, ldx=128,
             M=100, H=FAKE, ldh=64, GU=FAKE, ldgu=128, ws=FAKE, bytes=1 << 40)
    a.update(kw)
    return _lib.lib().qlora_gated_fwd(a["codes_g"], FAKE, a["qscale"], FAKE, a["codes_u"], FAKE, FAKE, FAKE, a["d_ff"],
                                      a["d_in"], a["dq"], a["A"], FAKE, 1.0, FAKE, a["B"], 1.0, a["r"], a["act"], a["X"],
                                      a["ldx"], a["M"], a["H"], a["ldh"], a["GU"], a["ldgu"], a["ws"], a["bytes"], None)


def _bwd(**kw):
    a = dict(codes_u=FAKE, d_ff=64, d_in=128, r=8, act=0, GU=FAKE, ldgu=128, dH=FAKE, lddh=64, M=100, dGU=FAKE, lddgu=128,
             dX=FAKE, lddx=128, ws=FAKE, bytes=1 << 40)
    a.update(kw)
    return _lib.lib().qlora_gated_bwd(FAKE, FAKE, FAKE, FAKE, a["codes_u"], FAKE, FAKE, FAKE, a["d_ff"], a["d_in"], 0, FAKE,
                                      FAKE, 1.0, FAKE, FAKE, 1.0, a["r"], a["act"], a["GU"], a["ldgu"], a["dH"], a["lddh"],
                                      a["M"], a["dGU"], a["lddgu"], a["dX"], a["lddx"], a["ws"], a["bytes"], None)


COMMON = [(dict(codes_u=None), -1), (dict(M=0), -1), (dict(d_ff=0), -1), (dict(r=-1), -1), (dict(r=257), -1),
          (dict(act=2), -1), (dict(ldgu=120), -1), (dict(ldgu=132), -1), (dict(GU=FAKE + 2), -1), (dict(ws=None), -1),
          (dict(ws=FAKE + 16), -1), (dict(d_ff=96), -2), (dict(d_in=96), -2), (dict(ldgu=1 << 62), -2),
          (dict(M=1 << 24), -2), (dict(d_ff=1 << 24), -2), (dict(d_ff=1 << 30), -2), (dict(bytes=64), -3)]


@pytest.mark.parametrize("bad,code", COMMON + [(dict(codes_g=None), -1), (dict(qscale=None), -1), (dict(A=None), -1),
                                               (dict(B=None), -1), (dict(B=FAKE + 8), -1), (dict(dq=3), -1),
                                               (dict(X=None), -1), (dict(H=None), -1), (dict(ldx=120), -1),
                                               (dict(ldx=132), -1), (dict(ldh=56), -1), (dict(ldh=1 << 62), -2),
                                               (dict(GU=None, bytes=64), -3), (dict(r=0, A=None, B=None, bytes=64), -3)])
def test_forward_refusals(bad, code):
    assert _fwd(**bad) == code
    assert _lib.lib().qn_last_error()


@pytest.mark.parametrize("bad,code", COMMON + [(dict(GU=None), -1), (dict(dH=None), -1), (dict(dGU=None), -1),
                                               (dict(dX=None), -1), (dict(lddh=56), -1), (dict(lddgu=120), -1),
                                               (dict(lddx=120), -1), (dict(lddx=132), -1), (dict(lddx=1 << 62), -2)])
def test_gradient_refusals(bad, code):
    assert _bwd(**bad) == code
    assert _lib.lib().qn_last_error()


def test_sizes():
    for f in (qn.gated_fwd_workspace_bytes, qn.gated_bwd_workspace_bytes):
        assert f(64, 64, 0, 8) == 0 and f(0, 64, 8, 8) == 0 and f(64, 64, 8, 257) == 0 and f(96, 64, 8, 8) == 0
        assert f(1 << 24, 128, 8, 8) == 0 and f(64, 64, 1 << 24, 256) == 0
        assert f(64, 64, 8, 0) > 0
    assert qn.gated_bwd_workspace_bytes(11008, 4096, 2048, 64) > 2 * 2 * 11008 * 4096


def _weight(d_out, d_in, dq="int8"):
    return qn.alloc_weight(d_out, d_in, "cpu", dq)


def test_layer_checks():
    w, b = _weight(64, 128), torch.bfloat16
    A, B = torch.zeros(8, 128, dtype=b), torch.zeros(64, 8, dtype=b)
    layer = qn.GatedLayer(w, w, A, B, 1.0, A, B, 1.0, "gelu")
    assert (layer.r, layer.d_in, layer.d_ff) == (8, 128, 64)
    assert qn.GatedLayer(w, w).r == 0
    with pytest.raises(ValueError, match="one shape"):
        qn.GatedLayer(w, _weight(128, 128))
    with pytest.raises(ValueError, match="one shape"):
        qn.GatedLayer(w, _weight(64, 128, "fp8"))
    with pytest.raises(ValueError, match="both projections"):
        qn.GatedLayer(w, w, A, B)
    with pytest.raises(ValueError, match="act"):
        qn.GatedLayer(w, w, act="relu")
    with pytest.raises(ValueError, match="A_up"):
        qn.GatedLayer(w, w, A, B, 1.0, A[:4].contiguous(), B)
    with pytest.raises(TypeError, match="B_gate"):
        qn.GatedLayer(w, w, A, B.float(), 1.0, A, B)


def test_call_checks():
    w, b = _weight(64, 128), torch.bfloat16
    layer = qn.GatedLayer(w, w)
    X, GU, dH = (torch.zeros(3, n, dtype=b) for n in (128, 128, 64))
    with pytest.raises(ValueError, match="input"):
        qn.gated_fwd(layer, X[:, :64])
    with pytest.raises(TypeError, match="input"):
        qn.gated_fwd(layer, X.float())
    with pytest.raises(ValueError, match="out"):
        qn.gated_fwd(layer, X, out=torch.zeros(3, 128, dtype=b))
    with pytest.raises(ValueError, match="GU is an input"):
        qn.gated_fwd(layer, X, GU=X)
    with pytest.raises(ValueError, match="d_seq"):
        qn.gated_bwd(layer, GU, dH[:2])
    with pytest.raises(ValueError, match="dGU is an input"):
        qn.gated_bwd(layer, GU, dH, dGU=GU.view(3, 128))
    with pytest.raises(ValueError, match="dX is an input"):
        qn.gated_bwd(layer, GU, dH, dX=GU)
    with pytest.raises(ValueError, match="dX is an input"):
        qn.gated_bwd(layer, GU, dH, dGU=GU, dX=GU)


@pytest.mark.parametrize("kind", ["silu", "gelu"])
def test_oracle_gradients_against_differences(kind):
    rng = np.random.default_rng(3)
    gate, up = ((rng.normal(size=(6, 5)), rng.normal(size=(2, 5)), rng.normal(size=(6, 2)), s) for s in (1.5, 0.5))
    X, dH = rng.normal(size=(4, 5)), rng.normal(size=(4, 6))
    H, G, U = GO.forward(gate, up, X, kind)
    dG, dU = GO.grads(G, U, dH, kind)
    dX = GO.input_grad(gate, up, dG, dU)
    h = 1e-6
    for i in np.ndindex(*X.shape):
        e = np.zeros_like(X)
        e[i] = h
        num = np.sum(dH * (GO.forward(gate, up, X + e, kind)[0] - GO.forward(gate, up, X - e, kind)[0])) / (2 * h)
        # central differences: h^2 times the third derivative, and 2^-52 / h times the values
        assert abs(num - dX[i]) < 1e-7 * (1 + abs(num)) * 10
    for i in np.ndindex(*G.shape):
        e = np.zeros_like(G)
        e[i] = h
        num = np.sum(dH * (GO.act(G + e, kind) - GO.act(G - e, kind)) * U) / (2 * h)
        assert abs(num - dG[i]) < 1e-6 * (1 + abs(num))
