"""Tensors that share memory where a call would read what it has already written: refused by
the binding."""
import pytest
import torch

import bit_nf4_quantized_05_amd as qn
from bit_nf4_quantized_05_amd import _lib


def test_parameters_that_overlap():
    buf, g = torch.zeros(1000), torch.zeros(1000)
    p = buf[:300]
    with pytest.raises(ValueError, match="share"):
        qn.adamw_state([p, p], [g[:300], g[300:600]])
    with pytest.raises(ValueError, match="share"):
        qn.adamw_state([buf[200:500], buf[700:], buf[:201]], [g[:300], g[:300], g[:201]])
    with pytest.raises(ValueError, match="share"):
        qn.adamw_state([buf.view(10, 100), buf[:1]], [g.view(10, 100), g[:1]])


def test_copies_that_overlap():
    p, g, c = torch.zeros(2, 300), torch.zeros(300), torch.zeros(500, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="share"):
        qn.adamw_state([p[0], p[1]], [g, g], copies=[c[:300], c[200:]])
    b = torch.zeros(600, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="share"):
        qn.adamw_state([b[:300], b[300:]], [g, g], copies=[b[300:], None])


def test_tensors_side_by_side_are_taken():
    buf, g, c = torch.zeros(1000), torch.zeros(1000), torch.zeros(1000, dtype=torch.bfloat16)
    st = qn.adamw_state([buf[300:], buf[:300], buf[5:5]], [g[300:], g[300:600], g[:0]], copies=[c[:700], c[700:], None])
    assert st.blocks == 3 + 2
    assert qn.adamw_state([c[:300]], [g[:300]], copies=[c[:300]]).blocks == 2      # the parameters' own bfloat16


def _batch(d_out=64, d_in=64, M=5):
    q, pool = qn.alloc_weight(d_out, d_in, "cpu"), qn.alloc_pool(3, 16, d_out, d_in, "cpu")
    return q, pool, _lib.MultiPlan(torch.zeros(4096, dtype=torch.uint8), M, 3), torch.zeros(M, d_in).bfloat16()


def test_output_that_is_an_input():
    q, pool, plan, X = _batch()
    dY = torch.zeros_like(X)
    with pytest.raises(ValueError, match="out"):
        qn.multi_linear_fwd(q, pool, plan, X, out=X)
    with pytest.raises(ValueError, match="dX"):
        qn.multi_linear_bwd(q, pool, plan, X, dY, dX=X)
    with pytest.raises(ValueError, match="dX"):
        qn.multi_linear_bwd(q, pool, plan, X, dY, dX=dY)
