"""The gated feed-forward block in float64 (numpy): the oracle of qlora_gated_fwd and
qlora_gated_bwd, on the dequantised bf16 weights. Shares no code with the library.

G = W_g x + s_g B_g (A_g x), U likewise, H = act(G) U (whoami-wesleyyou.top "LoRA" for each
projection); the gradients are its derivatives."""
from __future__ import annotations

import numpy as np


def _inner(g, kind):
    """x of act(g) = g sigma(x): g itself, or for (1 + tanh(y)) / 2 = sigma(2 y) twice the tanh's
    argument (1 + tanh loses every digit far below zero, sigma none)."""
    return g if kind == "silu" else 2 * np.sqrt(2 / np.pi) * (g + 0.044715 * g ** 3)


def _sigma(x):
    with np.errstate(over="ignore"):
        return 1 / (1 + np.exp(-x))


def act(g, kind):
    return g * _sigma(_inner(g, kind))


def act_grad(g, kind):
    x = _inner(g, kind)
    dx = 1 if kind == "silu" else 2 * np.sqrt(2 / np.pi) * (1 + 3 * 0.044715 * g * g)
    return _sigma(x) + g * _sigma(x) * _sigma(-x) * dx


def project(W, A, B, s, X):
    """W [d_ff, d_in], A [r, d_in], B [d_ff, r] (r may be 0), X [M, d_in]."""
    return X @ W.T + s * ((X @ A.T) @ B.T)


def forward(gate, up, X, kind):
    """gate, up: (W, A, B, s). Returns H, G, U."""
    G, U = project(*gate, X), project(*up, X)
    return act(G, kind) * U, G, U


def grads(G, U, dH, kind):
    return dH * U * act_grad(G, kind), dH * act(G, kind)


def input_grad(gate, up, dG, dU):
    return sum(dY @ W + s * ((dY @ B) @ A) for (W, A, B, s), dY in ((gate, dG), (up, dU)))
