"""Plain NumPy oracle of the block operators: gated feed-forward block, layer norm, AdamW.

64-bit floats throughout, except adamw_step with 8-bit states: the stored bytes follow from fp32
arithmetic bit for bit (m and v in fp32, each operation rounded), so that part is fp32 here too.
"""
from __future__ import annotations

import numpy as np

BLOCK = 128


def _sigmoid(g):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-g))


def ffn_forward(x, W1, W3, W2):
    g, u = x @ W1.T, x @ W3.T
    return (g * _sigmoid(g) * u) @ W2.T


def ffn_backward(x, W1, W3, W2, dy):
    """dx, dW1, dW3, dW2."""
    g, u = x @ W1.T, x @ W3.T
    s = _sigmoid(g)
    h = g * s * u
    dh = dy @ W2
    dg = dh * u * s * (1 + g * (1 - s))
    du = dh * g * s
    return dg @ W1 + du @ W3, dg.T @ x, du.T @ x, dy.T @ h


def layernorm_forward(x, w, b, eps):
    """y, mean, rstd."""
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1 / np.sqrt((c * c).mean(1) + eps)
    return c * rstd[:, None] * w + b, mean, rstd


def layernorm_backward(dy, x, w, mean, rstd):
    """dx, dw, db, for the forward pass's mean and rstd."""
    xh = (x - mean[:, None]) * rstd[:, None]
    gy = dy * w
    dx = rstd[:, None] * (gy - gy.mean(1, keepdims=True) - xh * (gy * xh).mean(1, keepdims=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def adamw_step(p, g, m, v, lr, beta1, beta2, eps, weight_decay, step):
    """p, m, v in 64 bits."""
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    mh, vh = m / (1 - beta1 ** step), v / (1 - beta2 ** step)
    return p - lr * weight_decay * p - lr * mh / (np.sqrt(vh) + eps), m, v


# ---- states in 8 bits ---------------------------------------------------------------------------

def moments_f32(g, m, v, beta1, beta2):
    f = np.float32
    with np.errstate(over="ignore", invalid="ignore"):
        return (m * f(beta1) + g * f(1 - beta1)).astype(f), (v * f(beta2) + (g * g) * f(1 - beta2)).astype(f)


def mix32(x, k):
    M = 0xFFFFFFFF
    x = x ^ (x >> 16)
    x = x * 0x7FEB352D & M
    x = (x ^ (x >> 15)) + k & M
    x = x * 0x846CA68B & M
    return x ^ (x >> 16)


def noise(n, seed, step, base=0):
    """32 random bits for each of values base .. base + n - 1."""
    k0 = mix32((seed & 0xFFFFFFFF) ^ (step & 0xFFFFFFFF), seed >> 32 & 0xFFFFFFFF)
    k1 = mix32(k0 ^ 0x9E3779B9, step >> 32 & 0xFFFFFFFF)
    i = base + np.arange(n, dtype=np.int64)
    return mix32((i & 0xFFFFFFFF) ^ k0, k1 + (i >> 32) * 0x9E3779B9 & 0xFFFFFFFF)


def _formats(name):
    # exponent of a block's largest value, exponent bias, exponent bits, sign
    return {"m": (7, 7, 4, True), "v": (15, 15, 5, False)}[name]


def decode(codes, scales, name):
    """float64 values of codes [n] with one scale byte per block."""
    top, bias, ebits, signed = _formats(name)
    c = codes.astype(np.int64)
    e, f = (c >> 3) & ((1 << ebits) - 1), c & 7
    a = np.where(e > 0, (8 + f) * 2.0 ** (np.maximum(e, 1) - bias - 3), f * 2.0 ** (1 - bias - 3))
    if signed:
        a = np.where(c & 0x80, -a, a)
    s = np.repeat(scales.astype(np.int64), BLOCK)[:len(c)]
    return np.where(s == 255, np.nan, np.where(s == 0, 0.0, a * 2.0 ** (s - 127.0)))


def encode(x, r16, name):
    """Codes and scales of fp32 values x with 16 random bits each (stochastic rounding)."""
    top, bias, ebits, signed = _formats(name)
    n, blocks = len(x), -(-len(x) // BLOCK)
    b = np.zeros(blocks * BLOCK)
    b[:n] = x
    r = np.zeros(blocks * BLOCK)
    r[:n] = r16
    b, r = b.reshape(blocks, BLOCK), r.reshape(blocks, BLOCK)
    most = np.abs(b).max(1)
    fine = np.isfinite(most)
    k = np.frexp(np.where(fine & (most >= 2.0 ** -126), most, 2.0 ** -127))[1] - 1 - top  # floor(log2) - top
    k = np.maximum(k, -126)
    y = np.abs(np.where(fine[:, None], b, 0.0)) * 2.0 ** -k[:, None].astype(float)
    e = np.maximum(np.frexp(y)[1] - 1, 1 - bias)
    q = np.floor(y / 2.0 ** (e - 3.0) + (r + 0.5) / 65536).astype(np.int64)  # 0 .. 16 steps of 2^(e-3)
    code = np.where(q >= 8, ((e + bias) << 3) + (q - 8), q)
    if signed:
        code = np.where(np.signbit(b), code | 0x80, code)
    code = np.where(fine[:, None], code, 0).reshape(-1)[:n]
    return code.astype(np.uint8), np.where(fine, k + 127, 255).astype(np.uint8)
