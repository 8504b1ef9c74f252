"""A gated layer whose tensors' storage moves after it was made: calls go by where the tensors are, and
by what they are, at the time of the call. Without a GPU; the library is a stand-in that keeps the
arguments."""
import pytest
import torch

import bit_nf4_quantized_05_amd as qn
from bit_nf4_quantized_05_amd import _lib

D_FF, D_IN, R = 64, 128, 8


class Recorder:
    def __init__(self):
        self.last = None

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("workspace_bytes"):
                return 256
            self.last = args
            return 0
        return call


@pytest.fixture
def recorder(monkeypatch):
    rec = Recorder()
    monkeypatch.setattr(_lib, "lib", lambda: rec)
    monkeypatch.setattr(_lib, "_own_stream", lambda dev: 0)
    return rec


def make():
    w = [qn.alloc_weight(D_FF, D_IN, "cpu") for _ in range(2)]
    ab = [(torch.zeros(R, D_IN, dtype=torch.bfloat16), torch.zeros(D_FF, R, dtype=torch.bfloat16)) for _ in range(2)]
    return w, ab, qn.GatedLayer(w[0], w[1], *ab[0], 1.0, *ab[1], 1.0)


# positions of the addresses among the arguments of both calls
CODES, ADAPTERS = {0: "codes", 1: "qconst", 2: "qscale", 3: "qmean"}, (11, 12, 14, 15)


def addresses(w, ab):
    want = {4 * i + k: getattr(w[i], name).data_ptr() for i in range(2) for k, name in CODES.items()}
    want.update(zip(ADAPTERS, (t.data_ptr() for pair in ab for t in pair)))
    return want


def run(layer):
    X, GU, dH = (torch.zeros(3, n, dtype=torch.bfloat16) for n in (D_IN, 2 * D_FF, D_FF))
    rec = _lib.lib()
    qn.gated_fwd(layer, X)
    fwd = rec.last
    qn.gated_bwd(layer, GU, dH)
    return fwd, rec.last


def test_calls_read_the_tensors_where_they_are(recorder):
    w, ab, layer = make()
    keep = []                                   # so that no freed address is handed out again
    for move in range(8):
        if move:
            i = move % 2
            for t in ab[i] if move % 3 else (w[i].codes, w[i].qconst, w[i].qscale, w[i].qmean):
                keep.append(t.data)
                t.data = t.data.clone()
        for args in run(layer):
            assert {k: args[k] for k in addresses(w, ab)} == addresses(w, ab)


def test_an_adapter_of_another_rank_set_in_place_is_taken_or_refused(recorder):
    w, ab, layer = make()
    ab[0][0].data = torch.zeros(16, D_IN, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="B_gate"):
        run(layer)
    ab[0][1].data = torch.zeros(D_FF, 16, dtype=torch.bfloat16)
    for A, B in (ab[1],):
        A.data, B.data = torch.zeros(16, D_IN, dtype=torch.bfloat16), torch.zeros(D_FF, 16, dtype=torch.bfloat16)
    for args in run(layer):
        assert args[17] == 16
    ab[1][0].data = torch.zeros(16, D_IN)
    with pytest.raises((TypeError, RuntimeError)):
        run(layer)


def test_weights_apart_are_refused():
    w, ab, _ = make()
    w[1].qscale = w[1].qscale.to("meta")
    with pytest.raises(ValueError, match="must all be on"):
        qn.GatedLayer(w[0], w[1])


def test_what_a_weight_does_not_have_may_be_anywhere():
    """Without a second level the constants and their mean are empty, on whatever device."""
    w = qn.alloc_weight(D_FF, D_IN, "cpu", "none")
    w.qconst, w.qmean = w.qconst.to("meta"), w.qmean.to("meta")
    assert qn.GatedLayer(w, w).d_ff == D_FF
