"""AdamW step in float64 (numpy), with the 8-bit moment format: the oracle of the library's
qlora_adamw_step. Shares no code with the library."""
from __future__ import annotations

import numpy as np

BLOCK = 256
TINY = 2.0 ** -126            # smallest normal float32


def mix32(h):
    """The format's 32-bit mixer (three xor-shifts, two odd multipliers) on uint32 arrays."""
    h = np.array(h, dtype=np.uint32)
    h ^= h >> np.uint32(16)
    h *= np.uint32(0x85EBCA6B)
    h ^= h >> np.uint32(13)
    h *= np.uint32(0xC2B2AE35)
    return h ^ (h >> np.uint32(16))


def words(n, step, seed=0):
    """The random 32-bit word of state elements 0 .. n - 1 at a step."""
    key = mix32(np.array([step & 0xFFFFFFFF], np.uint32) ^ mix32(np.array([seed], np.uint32)))
    return mix32(np.arange(n, dtype=np.uint32) ^ key)


def levels(signed):
    """Values of the level indices 0 .. 127 (m) or 0 .. 255 (v): float32 bit patterns."""
    k = np.arange(128 if signed else 256, dtype=np.int64)
    bits = ((k + (889 if signed else 761)) << 20).astype(np.uint32)
    return np.where(k == 0, 0.0, bits.view(np.float32).astype(np.float64))


def decode(codes, scale, signed):
    c = codes.reshape(-1, BLOCK).astype(np.int64)
    v = levels(signed)[c & 127 if signed else c] * scale.astype(np.float64)[:, None]
    return (np.where(c >= 128, -v, v) if signed else v).reshape(-1)


def encode(x, frac, signed):
    """(codes, scale, slack) of values x [256 blocks], frac in [0, 1) the random part per
    element; slack: how far, in levels, the cut is from turning out one level off."""
    b = np.abs(x).reshape(-1, BLOCK)
    scale = b.max(1)
    scale = np.where(scale < TINY, 0.0, scale)
    with np.errstate(divide="ignore", invalid="ignore"):
        r = np.where(scale[:, None] > 0, b / scale[:, None], 0.0).reshape(-1)
    mant, expo = np.frexp(r)                      # r = mant 2^expo, mant in [1/2, 1)
    # position on the grid of 8 levels per binade, 1.0 at the top level
    top = 127 if signed else 255
    with np.errstate(invalid="ignore"):
        pos = np.where(r > 0, (2 * mant - 1) * 8 + 8.0 * (expo - 1) + top, -1.0) + frac
    k = np.clip(np.floor(pos), 0, top).astype(np.int64)
    slack = np.abs(pos - np.round(pos))
    xs = x.reshape(-1)
    if signed:
        code = np.where((xs < 0) & (k > 0), k + 128, k)
    else:
        code = np.where((xs > 0) & np.repeat(scale > 0, BLOCK), np.maximum(k, 1), k)
    return code.astype(np.uint8), scale, slack


def step(p, g, m, v, t, lr, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01, grad_scale=1.0):
    """(p, m, v) after one step, float64 arrays."""
    g = g * grad_scale
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    den = np.sqrt(v / (1 - beta2 ** t)) + eps
    return p * (1 - lr * weight_decay) - lr * (m / (1 - beta1 ** t)) / den, m, v
