"""The loss over a large vocabulary without a GPU: sizes, refusals and the binding's checks."""
import pytest
import torch

import bit_nf4_quantized_05_amd as qn
from bit_nf4_quantized_05_amd import _lib

FAKE = 1 << 20


def _call(**kw):
    a = dict(W=FAKE, ldw=128, codes=None, qconst=None, qscale=None, qmean=None, dq=0, vocab=1001, d=128, X=FAKE, ldx=128,
             M=100, target=FAKE, scale=FAKE, loss=FAKE, dX=FAKE, lddx=128, ws=FAKE, bytes=1 << 50)
    a.update(kw)
    return _lib.lib().qlora_head_loss(a["W"], a["ldw"], a["codes"], a["qconst"], a["qscale"], a["qmean"], a["dq"],
                                      a["vocab"], a["d"], a["X"], a["ldx"], a["M"], a["target"], a["scale"], a["loss"],
                                      a["dX"], a["lddx"], a["ws"], a["bytes"], None)


NF4 = dict(W=None, ldw=0, codes=FAKE, qconst=FAKE, qscale=FAKE, qmean=FAKE, vocab=1024)


@pytest.mark.parametrize("bad,code", [
    (dict(W=None), -1), (dict(codes=FAKE), -1), (dict(NF4, qscale=None), -1), (dict(NF4, dq=3), -1),
    (dict(NF4, codes=FAKE + 8), -1), (dict(W=FAKE + 8), -1), (dict(ldw=120), -1), (dict(ldw=132), -1), (dict(X=None), -1),
    (dict(ldx=120), -1), (dict(target=None), -1), (dict(target=FAKE + 4), -1), (dict(loss=None), -1),
    (dict(scale=FAKE + 2), -1), (dict(lddx=120), -1), (dict(dX=FAKE + 8), -1), (dict(vocab=0), -1), (dict(M=0), -1),
    (dict(ws=None), -1), (dict(ws=FAKE + 16), -1), (dict(d=96), -2), (dict(NF4, vocab=1001), -2), (dict(ldx=1 << 62), -2),
    (dict(lddx=1 << 62), -2), (dict(ldw=1 << 62), -2), (dict(M=1 << 24), -2), (dict(M=1 << 30, d=64, ldx=64, lddx=64), -2),
    (dict(vocab=1 << 30, d=1 << 12, ldw=1 << 12, ldx=1 << 12, lddx=1 << 12), -2), (dict(bytes=64), -3),
    (dict(dX=None, scale=None, bytes=64), -3), (dict(NF4, bytes=64), -3)])
def test_refusals(bad, code):
    assert _call(**bad) == code
    assert _lib.lib().qn_last_error()


def test_sizes():
    f = _lib.lib().qlora_head_loss_workspace_bytes
    assert f(0, 64, 8, 0, 0) == 0 and f(100, 63, 8, 0, 0) == 0 and f(100, 64, 0, 0, 1) == 0 and f(100, 64, 8, 1, 0) == 0
    # the loss alone keeps two words per token and 256 rows; no logits
    assert f(128000, 4096, 4096, 0, 0) < 4 * 4096 * 128000 / 64
    # with the gradient, one piece of the vocabulary
    assert f(128000, 4096, 4096, 0, 1) < 2 * 4096 * 128000
    # twice the vocabulary past a piece needs no more
    assert f(256000, 4096, 4096, 0, 1) <= f(128000, 4096, 4096, 0, 1) * 1.1


def test_a_launch_has_less_than_2_32_threads():
    """Two words per token and tile of a piece are kept, and per token six more: that tells the tiles of
    256 x 256, of 512 threads each."""
    d_seq = 1 << 24
    got = _lib.lib().qlora_head_loss_workspace_bytes(65536, 64, d_seq, 0, 0)
    tiles = (got - 4 * 6 * d_seq) / (8 * d_seq) * (d_seq / 256)
    assert 0 < tiles * 512 < 2 ** 32 and got > 0


def test_tensors_off_the_current_device_are_refused(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError, match="not the current device"):
        _lib._own_stream(torch.device("cuda", 0))


def test_call_checks():
    b = torch.bfloat16
    W, X, t = torch.zeros(100, 64, dtype=b), torch.zeros(5, 64, dtype=b), torch.zeros(5, dtype=torch.int64)
    with pytest.raises(ValueError, match="head"):
        qn.head_loss(W[0], X, t)
    with pytest.raises(TypeError, match="head"):
        qn.head_loss(W.float(), X, t)
    with pytest.raises(ValueError, match="head"):
        qn.head_loss(W.t(), X, t)
    with pytest.raises(ValueError, match="input"):
        qn.head_loss(W, X[:, :32], t)
    with pytest.raises(TypeError, match="target"):
        qn.head_loss(W, X, t.int())
    with pytest.raises(ValueError, match="target"):
        qn.head_loss(W, X, t[:4])
    with pytest.raises(TypeError, match="scale"):
        qn.head_loss_grad(W, X, t, scale=torch.zeros(5, dtype=torch.float64))
    s = torch.zeros(5)
    with pytest.raises(ValueError, match="loss is an input"):
        qn.head_loss_grad(W, X, t, scale=s, loss=s)
    with pytest.raises(ValueError, match="dX is an input"):
        qn.head_loss_grad(W, X, t, dX=X)
