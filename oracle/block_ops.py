"""Oracle of the feed-forward block's operators: numpy float64, plain and slow.

TEST INFRASTRUCTURE (see the package docstring).

* Linear layers with a bias, an activation and a residual: z = x w^T + bias, y = act(z) + residual; the input gradient
  through the activation, dz = (dy w) act'(z); the bias gradient sum_t dz.
* Activations in 8 bits: 32 columns of a row share a unit 2^(scale - 127); a code is a sign and a magnitude up to 127.
* The norms around a block: h = a x + b gate PostNorm(y), n = PreNorm(h), its input and its weight gradients.
"""
from __future__ import annotations

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])
_erfc = np.vectorize(math.erfc, otypes=[np.float64])

# ---------------------------------------------------------------- activations


def _logistic(x):
    e = np.exp(-np.abs(x))
    return np.where(x >= 0, 1.0 / (1.0 + e), e / (1.0 + e))


def act(z, kind):
    if kind == "relu":
        return np.maximum(z, 0.0)
    if kind == "relu2":
        return np.maximum(z, 0.0) ** 2
    if kind == "gelu":
        return 0.5 * z * _erfc(-z / math.sqrt(2.0))
    if kind == "gelu_tanh":
        return z * _logistic(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    if kind == "silu":
        return z * _logistic(z)
    return np.array(z, dtype=np.float64)


def act_slope(z, kind):
    if kind == "relu":
        return (z > 0.0).astype(np.float64)
    if kind == "relu2":
        return 2.0 * np.maximum(z, 0.0)
    if kind == "gelu":
        return 0.5 * _erfc(-z / math.sqrt(2.0)) + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        s = _logistic(c * (z + 0.044715 * z ** 3))
        return s + z * s * (1.0 - s) * c * (1.0 + 3.0 * 0.044715 * z * z)
    if kind == "silu":
        s = _logistic(z)
        return s + z * s * (1.0 - s)
    return np.ones_like(z)


# ---------------------------------------------------------------- activations in 8 bits


def pack(x):
    """(codes, scales) of a matrix of bf16 numbers, element by element from the definition."""
    rows, width = x.shape
    codes, scales = np.zeros((rows, width), dtype=np.uint8), np.zeros((rows, width // 32), dtype=np.uint8)
    for r in range(rows):
        for b in range(width // 32):
            v = x[r, 32 * b: 32 * b + 32]
            if not np.all(np.isfinite(v)):
                scales[r, b] = 255
                continue
            top = np.max(np.abs(v))
            scale = 1
            while scale < 248 and top >= 127.5 * 2.0 ** (scale - 127):
                scale += 1
            m = np.minimum(np.rint(np.abs(v) * 2.0 ** (127 - scale)), 127).astype(np.int64)  # rint: ties to even
            codes[r, 32 * b: 32 * b + 32] = m | np.where(np.signbit(v), 128, 0)
            scales[r, b] = scale
    return codes, scales


def unpack(codes, scales):
    unit = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127.0))
    unit = np.where(scales == 0, 0.0, unit)
    m = (codes & 127).astype(np.float64) * np.repeat(unit, 32, axis=1)
    return np.where(codes > 127, -m, m)


# ---------------------------------------------------------------- norms around a block


def norm_stats(x, kind, eps):
    """(mean, rstd) of rows; zeros without a norm."""
    if kind == "none":
        return np.zeros(x.shape[0]), np.zeros(x.shape[0])
    mean = x.mean(1) if kind == "layer" else np.zeros(x.shape[0])
    return mean, 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)


def norm(x, kind, gamma, beta, eps):
    if kind == "none":
        return np.array(x)
    mean, rstd = norm_stats(x, kind, eps)
    y = gamma * (x - mean[:, None]) * rstd[:, None]
    return y if beta is None else y + beta


def norm_backward(dy, x, kind, gamma, eps):
    """(dx, dgamma, dbeta) of y = norm(x)."""
    if kind == "none":
        return np.array(dy), None, None
    mean, rstd = norm_stats(x, kind, eps)
    hat = (x - mean[:, None]) * rstd[:, None]
    d = dy * gamma
    dx = d - hat * (d * hat).mean(1, keepdims=True)
    if kind == "layer":
        dx -= d.mean(1, keepdims=True)
    return dx * rstd[:, None], (dy * hat).sum(0), dy.sum(0)


class ResidualNorm:
    """h = a x + b gate PostNorm(y), n = PreNorm(h).  gate: None, [hidden] or [tokens, hidden]."""

    def __init__(self, post="none", pre="none", gate=None, post_gamma=None, post_beta=None, pre_gamma=None, pre_beta=None,
                 a=1.0, b=1.0, post_eps=1e-5, pre_eps=1e-5):
        self.__dict__.update(locals())

    def branch(self, y):
        u = norm(y, self.post, self.post_gamma, self.post_beta, self.post_eps)
        return u if self.gate is None else u * self.gate

    def h(self, x, y):
        return self.a * x + self.b * self.branch(y)

    def n(self, h):
        return norm(h, self.pre, self.pre_gamma, self.pre_beta, self.pre_eps)

    def backward(self, dn, dres, h, y, dh=None):
        """Every gradient; `dh` given: the weights' of a block whose dh is already known."""
        out = {}
        total = 0.0 if dres is None else dres
        if dn is not None:
            d, out["dpre_gamma"], out["dpre_beta"] = norm_backward(dn, h, self.pre, self.pre_gamma, self.pre_eps)
            total = total + d
        dh = total if dh is None else dh
        out["dh"], out["dx"] = dh, self.a * dh
        u = norm(y, self.post, self.post_gamma, self.post_beta, self.post_eps)
        out["dgate"] = self.b * dh * u
        du = self.b * dh if self.gate is None else self.b * dh * self.gate
        out["dy"], out["dpost_gamma"], out["dpost_beta"] = norm_backward(du, y, self.post, self.post_gamma, self.post_eps)
        return out
