"""Adapter gradients whose partials are added from several slices of tokens: adapters just
below, at and above a slice, one after the other, in a pool most of which is not in use; in a
workspace of exactly the size the library asks for.

Tolerance: that of test_gpu_multi.py (float32 sums of up to 4000 tokens and 1024 features:
sqrt(5024) 2^-24 = 4.2e-6 of the norm, 5e-6 allowed)."""
import numpy as np
import pytest
import torch

import bit_nf4_quantized_05_amd as qn
from oracle import multi_oracle as MO
from parity import dev
from test_gpu_multi import Layer, _close32, _f64

pytestmark = pytest.mark.gpu


# slices of 128 tokens on the small layers; of 256, 512 and 1024 in the last three cases
CASES = [(320, 256, 16, 40, [129, 129, 129, 129]), (320, 256, 16, 1024, [256, 1, 257, 128, 130, 127, 500]),
         (320, 256, 64, 700, [1, 1, 1, 300, 1, 1, 2, 900]), (64, 64, 16, 3, [2000]), (64, 64, 256, 3, [1999, 129]),
         (1280, 1024, 64, 20, [700, 129, 1, 385, 256, 640]), (1280, 1024, 64, 1000, [4000]),
         (64, 64, 16, 100, [10] * 50 + [200]), (1280, 1024, 256, 20, [700, 257, 1, 513, 256, 640]),
         (1024, 1024, 256, 12, [513, 512, 1, 1500, 300, 511, 700]),
         (1024, 1024, 256, 16, [1025, 1024, 2049, 1023, 700, 1300, 1079])]


@pytest.mark.parametrize("d_out,d_in,r,n,counts", CASES)
@pytest.mark.parametrize("loose", [0, 70])                   # tokens without an adapter
def test_slices(d_out, d_in, r, n, counts, loose):
    M = sum(counts) + loose
    print(f"[multi] slices {d_out}x{d_in}, {M} tokens, r={r}, {n} adapters, {counts[:8]}", flush=True)
    who = [min(2 * i, n - 1) if n >= 2 * len(counts) else i for i in range(len(counts))]
    ids = np.concatenate([np.repeat(who, counts), np.full(loose, -1)]).astype(np.int32)
    ids = np.random.default_rng(M).permutation(ids)
    L = Layer(d_out, d_in, M, r, max(who) + 1, "one", seed=M)
    pool = qn.alloc_pool(n, r, d_out, d_in, dev())
    for a in who:
        pool.set(a, L.pool.A[a], L.pool.B[a], float(L.s[a]))
    plan = qn.multi_plan(torch.from_numpy(ids).to(dev()), n)
    need = qn.multi_linear_bwd_workspace_bytes(d_out, d_in, M, r, n)
    ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device=dev())
    junk = torch.full(pool.A.shape, float("nan"), device=dev()), torch.full(pool.B.shape, float("nan"), device=dev())
    _, dA, dB = qn.multi_linear_bwd(L.q, pool, plan, L.X, L.dY, dA=junk[0], dB=junk[1], workspace=ws[:need])
    torch.cuda.synchronize()
    assert torch.all(ws[need:] == 0x5A)
    _, wA, wB = MO.backward(L.W, L.A, L.B, L.s, ids, _f64(L.X), _f64(L.dY))
    for a in who:
        _close32(dA[a], wA[a], f"dA {a}")
        _close32(dB[a], wB[a], f"dB {a}")
    idle = [a for a in range(n) if a not in who]
    assert dA[idle].count_nonzero() == 0 and dB[idle].count_nonzero() == 0
    again = qn.multi_linear_bwd(L.q, pool, plan, L.X, L.dY)
    assert torch.equal(again[1], dA) and torch.equal(again[2], dB)
