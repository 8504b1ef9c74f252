"""Many adapters on one layer without a GPU: sizes, refusals, the binding's checks, and the
oracle's gradients against differences."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_05_amd as qn
from bit_nf4_quantized_05_amd import _lib
from oracle import multi_oracle as MO
from oracle import nf4_oracle as O

FAKE = 1 << 20


def test_sizes():
    lib = _lib.lib()
    assert lib.qlora_multi_plan_bytes(0, 4) == 0 and lib.qlora_multi_plan_bytes(10, 0) == 0
    assert lib.qlora_multi_plan_bytes(10, 1025) == 0
    # head 4, order 12, start 4, first items 4, used 4, tiles 4, items 4 * (1 + 3) words
    assert lib.qlora_multi_plan_bytes(10, 3) == 4 * (4 + 12 + 4 + 4 + 4 + 4 + 16)
    assert qn.multi_linear_fwd_workspace_bytes(64, 64, 0, 16, 1) == 0
    assert qn.multi_linear_fwd_workspace_bytes(64, 64, 8, 16, 0) == 0
    # up to 64 tokens: partial sums only; above: W_hat as well
    assert qn.multi_linear_fwd_workspace_bytes(4096, 4096, 64, 16, 8) < 2 * 4096 * 4096
    assert qn.multi_linear_fwd_workspace_bytes(4096, 4096, 65, 16, 8) > 2 * 4096 * 4096
    # the backward keeps gradient partials that grow with the pool
    few, many = (qn.multi_linear_bwd_workspace_bytes(256, 256, 2000, 16, n) for n in (1, 101))
    assert many - few >= 100 * 2 * 16 * 512


def _fwd(**kw):
    a = dict(codes=FAKE, d_out=64, d_in=64, A=FAKE, B=FAKE, s=FAKE, n=2, r=16, X=FAKE, ldx=64, M=8, plan=FAKE, Y=FAKE,
             ldy=64, ws=FAKE, bytes=1 << 30, dq=0)
    a.update(kw)
    return _lib.lib().qlora_multi_fwd(a["codes"], FAKE, FAKE, FAKE, a["d_out"], a["d_in"], a["dq"], a["A"], a["B"],
                                      a["s"], a["n"], a["r"], a["X"], a["ldx"], a["M"], a["plan"], a["Y"], a["ldy"],
                                      a["ws"], a["bytes"], None)


def _bwd(**kw):
    a = dict(d_out=64, d_in=128, n=2, r=16, X=FAKE, ldx=128, dY=FAKE, lddy=64, M=100, plan=FAKE, dX=FAKE, lddx=128,
             dA=FAKE, dB=FAKE, ws=FAKE, bytes=1 << 30)
    a.update(kw)
    return _lib.lib().qlora_multi_bwd(FAKE, FAKE, FAKE, FAKE, a["d_out"], a["d_in"], 0, FAKE, FAKE, FAKE, a["n"], a["r"],
                                      a["X"], a["ldx"], a["dY"], a["lddy"], a["M"], a["plan"], a["dX"], a["lddx"],
                                      a["dA"], a["dB"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("bad,code", [(dict(A=None), -1), (dict(s=None), -1), (dict(plan=None), -1), (dict(Y=None), -1),
                                      (dict(codes=None), -1), (dict(M=0), -1), (dict(n=0), -1), (dict(r=0), -1),
                                      (dict(r=272), -1), (dict(ldx=56), -1), (dict(ldx=68), -1), (dict(ldy=32), -1),
                                      (dict(X=FAKE + 2), -1), (dict(plan=FAKE + 4), -1), (dict(ws=FAKE + 16), -1),
                                      (dict(dq=3), -1), (dict(r=8), -2), (dict(r=40), -2), (dict(n=1025), -2),
                                      (dict(d_in=96, ldx=96), -2), (dict(d_out=96, ldy=96), -2),
                                      (dict(M=1 << 25, ldx=64), -2),
                                      (dict(ldx=1 << 62), -2), (dict(M=(1 << 31) - 1, ldy=1 << 40), -2), (dict(bytes=64), -3)])
def test_forward_refusals(bad, code):
    assert _fwd(**bad) == code
    assert _lib.lib().qn_last_error()


@pytest.mark.parametrize("bad,code", [(dict(dA=None), -1), (dict(dB=None), -1), (dict(dY=None), -1), (dict(dX=None), -1),
                                      (dict(lddy=56), -1), (dict(lddx=120), -1), (dict(ldx=120), -1),
                                      (dict(dA=FAKE + 4), -1), (dict(r=24), -2), (dict(n=2000), -2),
                                      (dict(d_in=96, ldx=96, lddx=96), -2), (dict(bytes=1024), -3)])
def test_backward_refusals(bad, code):
    assert _bwd(**bad) == code


def test_plan_refusals():
    lib = _lib.lib()
    assert lib.qlora_multi_plan(None, 8, 2, FAKE, 1 << 20, None) == -1
    assert lib.qlora_multi_plan(FAKE, 8, 2, None, 1 << 20, None) == -1
    assert lib.qlora_multi_plan(FAKE, 0, 2, FAKE, 1 << 20, None) == -1
    assert lib.qlora_multi_plan(FAKE, 8, 0, FAKE, 1 << 20, None) == -1
    assert lib.qlora_multi_plan(FAKE, 8, 1025, FAKE, 1 << 20, None) == -2
    assert lib.qlora_multi_plan(FAKE, 8, 2, FAKE + 4, 1 << 20, None) == -1
    assert lib.qlora_multi_plan(FAKE, 8, 2, FAKE, 16, None) == -3


def test_binding_refusals():
    cpu = torch.device("cpu")
    q = qn.alloc_weight(64, 128, cpu)
    pool = qn.alloc_pool(3, 10, 64, 128, cpu)
    assert pool.r == 16 and pool.n == 3
    plan = _lib.MultiPlan(torch.zeros(64, dtype=torch.uint8), 5, 3)
    X = torch.zeros(5, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        qn.multi_linear_fwd(q, pool, plan, X[:4])                        # another batch's plan
    with pytest.raises(ValueError):
        qn.multi_linear_fwd(q, qn.alloc_pool(4, 10, 64, 128, cpu), plan, X)
    with pytest.raises(ValueError):
        qn.multi_linear_fwd(q, qn.alloc_pool(3, 10, 64, 64, cpu), plan, X)
    with pytest.raises(TypeError):
        qn.multi_linear_fwd(q, pool, plan, X.float())
    with pytest.raises(TypeError):
        qn.multi_linear_fwd(q, qn.AdapterPool(pool.A, pool.B, pool.s.double()), plan, X)
    with pytest.raises(ValueError):
        qn.multi_linear_bwd(q, pool, plan, X, torch.zeros(4, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        qn.multi_linear_fwd(q, pool, plan, X, workspace=torch.zeros(64, 64, dtype=torch.uint8)[:, :8])
    with pytest.raises(ValueError):
        pool.set(0, torch.zeros(17, 128), torch.zeros(64, 17), 1.0)
    with pytest.raises(TypeError):
        qn.multi_plan(torch.zeros(5, dtype=torch.int64), 3)
    with pytest.raises(ValueError):
        qn.alloc_pool(3, 257, 64, 128, cpu)
    pool.set(1, torch.ones(5, 128), torch.ones(64, 5), 2.0)
    assert pool.A[1, :5].eq(1).all() and pool.A[1, 5:].eq(0).all() and pool.B[1, :, 5:].eq(0).all() and pool.s[1] == 2


def test_oracle_single_adapter_is_the_layer_oracle():
    rng = np.random.default_rng(0)
    w, a, b = (O.f32_to_bf16_bits(rng.standard_normal(s).astype(np.float32)) for s in ((6, 8), (2, 8), (6, 2)))
    x, dy = (O.f32_to_bf16_bits(rng.standard_normal(s).astype(np.float32)) for s in ((5, 8), (5, 6)))
    f = lambda v: O.bf16_bits_to_f32(v).astype(np.float64)  # noqa: E731
    A, B, ids = f(a)[None], f(b)[None], np.zeros(5, int)
    assert np.allclose(MO.forward(f(w), A, B, [1.5], ids, f(x)), O.linear_fwd(w, a, b, 1.5, x), rtol=1e-12)
    assert np.allclose(MO.backward(f(w), A, B, [1.5], ids, f(x), f(dy))[0], O.linear_bwd_x(w, a, b, 1.5, dy), rtol=1e-12)


def test_oracle_gradients_against_differences():
    """<dY, Y> differentiated by central differences in every input."""
    rng = np.random.default_rng(2)
    n, r, d_in, d_out, M = 3, 2, 5, 4, 7
    W, A, B = rng.standard_normal((d_out, d_in)), rng.standard_normal((n, r, d_in)), rng.standard_normal((n, d_out, r))
    s, X, dY = rng.random(n) + 0.5, rng.standard_normal((M, d_in)), rng.standard_normal((M, d_out))
    ids = np.array([0, 2, -1, 2, 0, 5, 2])                             # adapter 1 has no tokens
    grads = MO.backward(W, A, B, s, ids, X, dY)
    for v, g in zip((X, A, B), grads):
        num = np.zeros_like(v)
        for k in np.ndindex(v.shape):
            old = v[k]
            v[k] = old + 1e-4
            up = np.sum(dY * MO.forward(W, A, B, s, ids, X))
            v[k] = old - 1e-4
            num[k] = (up - np.sum(dY * MO.forward(W, A, B, s, ids, X))) / 2e-4
            v[k] = old
        assert np.allclose(num, g, rtol=1e-7, atol=1e-7)
    assert np.all(grads[1][1] == 0) and np.all(grads[2][1] == 0)
