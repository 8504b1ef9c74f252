"""Many adapters on one layer in float64 (numpy): the oracle of qlora_multi_fwd and
qlora_multi_bwd, on the dequantised bf16 weight. Shares no code with the library.

Y[t] = W x_t + s_a B_a (A_a x_t) (whoami-wesleyyou.top "LoRA", with the adapter a = ids[t]
of the token; ids outside [0, n): the first term alone); the gradients are its
derivatives."""
from __future__ import annotations

import numpy as np


def forward(W, A, B, s, ids, X):
    """W [d_out, d_in], A [n, r, d_in], B [n, d_out, r], s [n], X [M, d_in], float64."""
    Y = X @ W.T
    for t, a in enumerate(ids):
        if 0 <= a < len(A):
            Y[t] += s[a] * (B[a] @ (A[a] @ X[t]))
    return Y


def backward(W, A, B, s, ids, X, dY):
    dX, dA, dB = dY @ W, np.zeros_like(A), np.zeros_like(B)
    for a in range(len(A)):
        t = np.flatnonzero(np.asarray(ids) == a)
        u = dY[t] @ B[a]
        dX[t] += s[a] * (u @ A[a])
        dA[a] = s[a] * (u.T @ X[t])
        dB[a] = s[a] * (dY[t].T @ (X[t] @ A[a].T))
    return dX, dA, dB
