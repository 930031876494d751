"""Oracle of the training operators beside a stage's own steps: numpy float64, plain and slow.

TEST INFRASTRUCTURE (see the package docstring).

* Rotary positions: pair (a, b) number i of a head at position p turns by p f_i.
* Attention inside packed documents: row i sees key j of the same document when j <= i or j is one of the
  document's first `prefix` rows; scores q.k / sqrt(d), then cap tanh(s / cap), then minus slope |i - j|.
* AdamW, and its 8-bit states: blocks of 256 elements with one scale, codes whose values are the integers
  (8 + f) 2^(e - 1) times the scale.  The codes depend on float32 arithmetic in a stated order (separately rounded
  products and sums), which numpy's float32 operations give.
"""
from __future__ import annotations

import numpy as np

# ---------------------------------------------------------------- rotary positions


def rotary_frequencies(rot, base=10000.0, scaling="none", factor=1.0, context=0.0, low=1.0, high=32.0):
    """(f_i, magnitude), straight from the definitions."""
    pairs = range(rot // 2)
    if scaling == "ntk":
        base = base * factor ** (rot / (rot - 2.0))
    f = np.array([base ** (-2.0 * i / rot) for i in pairs])
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "banded":
        out = []
        for x in f:
            wave = 2.0 * np.pi / x
            if wave < context / high:
                out.append(x)
            elif wave > context / low:
                out.append(x / factor)
            else:
                w = (context / wave - low) / (high - low)
                out.append((1.0 - w) * x / factor + w * x)
        return np.array(out), 1.0
    if scaling == "yarn":
        pair_of = lambda turns: rot * np.log(context / (2.0 * np.pi * turns)) / (2.0 * np.log(base))  # noqa: E731
        lo, hi = max(np.floor(pair_of(high)), 0.0), min(np.ceil(pair_of(low)), rot - 1.0)
        ramp = np.array([min(1.0, max(0.0, (i - lo) / (hi - lo))) if hi > lo else float(i >= hi) for i in pairs])
        return (f / factor) * ramp + f * (1.0 - ramp), 0.1 * np.log(factor) + 1.0
    return f, 1.0


def rotary(x, positions, f, magnitude, pairs, backward=False):
    """x [T, heads, d]; the first 2 len(f) elements of every head turn."""
    r = 2 * len(f)
    y = np.array(x, dtype=np.float64)
    a = np.arange(len(f)) if pairs == "half" else 2 * np.arange(len(f))
    b = a + len(f) if pairs == "half" else a + 1
    # whole turns off first: the angles reach 10^9 radians
    turns = np.asarray(positions, dtype=np.longdouble)[:, None] * (np.asarray(f, dtype=np.longdouble) / (2.0 * np.longdouble(np.pi)))
    angle = 2.0 * np.pi * (turns - np.floor(turns)).astype(np.float64)
    c, s = magnitude * np.cos(angle)[:, None, :], magnitude * np.sin(angle)[:, None, :]
    if backward:
        s = -s
    xa, xb = y[..., a].copy(), y[..., b].copy()
    y[..., a], y[..., b] = xa * c - xb * s, xb * c + xa * s
    assert r <= y.shape[-1]
    return y


# ---------------------------------------------------------------- attention inside packed documents


def document_visible(t, offsets, prefix=None):
    """[t, t] truth values: row i sees key j."""
    see = np.zeros((t, t), dtype=bool)
    for d in range(len(offsets) - 1):
        s, e = offsets[d], offsets[d + 1]
        see[s:e, s:e] = np.tril(np.ones((e - s, e - s), dtype=bool))
        if prefix is not None:
            see[s:e, s:min(e, s + max(0, prefix[d]))] = True
    return see


def _document_scores(q, k, see, cap, slope):
    """(scores with -inf where hidden, the cap's derivative)."""
    s = np.where(see, (q @ k.T) / np.sqrt(q.shape[1]), 0.0)
    deriv = np.ones_like(s)
    if cap:
        r = np.tanh(s / cap)
        deriv, s = 1.0 - r * r, cap * r
    i = np.arange(q.shape[0])
    return np.where(see, s - slope * np.abs(i[:, None] - i[None, :]), -np.inf), deriv


def document_attention(qkv, nh, nkv, d, see, cap=0.0, slopes=None):
    """(a [t, nh d], lse [nh, t] in base 2); rows that see nothing get zeros and -inf.  Values of hidden keys are never
    used: they may be NaN."""
    t = qkv.shape[0]
    x = qkv.reshape(t, nh + 2 * nkv, d)
    a, lse = np.zeros((t, nh, d)), np.full((nh, t), -np.inf)
    live = see.any(axis=1)
    for h in range(nh):
        j = nh + h // (nh // nkv)
        with np.errstate(invalid="ignore"):
            s, _ = _document_scores(x[:, h], x[:, j], see, cap, 0.0 if slopes is None else slopes[h])
        for i in np.nonzero(live)[0]:
            keys = np.nonzero(see[i])[0]
            z = s[i, keys]
            top = z.max()
            p = np.exp(z - top)
            lse[h, i] = (top + np.log(p.sum())) / np.log(2.0)
            a[i, h] = (p / p.sum()) @ x[keys, j + nkv]
    return a.reshape(t, nh * d), lse


def document_attention_grad(da, qkv, nh, nkv, d, see, cap=0.0, slopes=None):
    """Gradient of document_attention with respect to qkv (finite inputs)."""
    t = qkv.shape[0]
    x, dy = qkv.reshape(t, nh + 2 * nkv, d), da.reshape(t, nh, d)
    out = np.zeros_like(x)
    for h in range(nh):
        j = nh + h // (nh // nkv)
        s, deriv = _document_scores(x[:, h], x[:, j], see, cap, 0.0 if slopes is None else slopes[h])
        top = np.where(see.any(axis=1), s.max(axis=1, initial=-np.inf), 0.0)
        p = np.exp(s - top[:, None])
        total = p.sum(axis=1, keepdims=True)
        p = np.divide(p, total, out=np.zeros_like(p), where=total > 0)
        out[:, j + nkv] += p.T @ dy[:, h]
        dp = dy[:, h] @ x[:, j + nkv].T
        ds = p * (dp - np.sum(p * dp, axis=1, keepdims=True)) * deriv / np.sqrt(d)
        out[:, h] = ds @ x[:, j]
        out[:, j] += ds.T @ x[:, h]
    return out.reshape(t, -1)


# ---------------------------------------------------------------- AdamW

F32 = np.float32


def adamw(p, g, m, v, step, lr, beta1, beta2, eps, decay):
    """One step in float64: (p, m, v)."""
    m = beta1 * m + (1.0 - beta1) * g
    v = beta2 * v + (1.0 - beta2) * g * g
    p = p - lr * decay * p
    return p - lr * (m / (1.0 - beta1 ** step)) / (np.sqrt(v / (1.0 - beta2 ** step)) + eps), m, v


def moments_f32(g, m, v, beta1, beta2, scale=None):
    """The moments in float32, every product and sum rounded on its own."""
    g = g.astype(F32)
    if scale is not None:
        g = g * F32(scale)
    m = m * F32(beta1) + g * F32(1.0 - beta1)
    v = v * F32(beta2) + (g * g) * F32(1.0 - beta2)
    return m, v


M_TOP, V_TOP, BLOCK = F32(15 * 2 ** 14), F32(15 * 2 ** 30), 256


def mix32(x):
    """A 32-bit hash of xorshifts and multiplications, with the constants that C. Wellons published in 2018 as the result of
    a search for the least bias."""
    x = np.asarray(x, dtype=np.uint64) & np.uint64(0xFFFFFFFF)
    x = ((x ^ (x >> np.uint64(16))) * np.uint64(0x7FEB352D)) & np.uint64(0xFFFFFFFF)
    x = ((x ^ (x >> np.uint64(15))) * np.uint64(0x846CA68B)) & np.uint64(0xFFFFFFFF)
    return x ^ (x >> np.uint64(16))


def noise32(seed, step, tensor, count):
    key = int(mix32((seed ^ (step * 0x9E3779B1)) & 0xFFFFFFFF))
    key = int(mix32((key + tensor * 0x85EBCA77) & 0xFFFFFFFF))
    return mix32(np.arange(count, dtype=np.uint64) ^ np.uint64(key))


def code_values(signed):
    c = np.arange(128 if signed else 256)
    v = np.where(c < 8, c.astype(np.float64), (8.0 + c % 8) * 2.0 ** (c // 8 - 1.0))
    return np.concatenate([v, -v]) if signed else v


def unpack(codes, scales, signed):
    """float32 values of 8-bit codes."""
    return code_values(signed).astype(F32)[codes] * np.repeat(scales, BLOCK)[: codes.size].astype(F32)


def pack(x, signed, noise16):
    """(codes, scales) of float32 x; noise16: 16 random bits per element, or 0x8000 for the nearest code.

    The code is the largest one whose value is at most z, or the next, taken when the remainder's first 16
    bits plus the noise carry."""
    top = M_TOP if signed else V_TOP
    n = x.size
    blocks = -(-n // BLOCK)
    ax = np.abs(np.pad(x, (0, blocks * BLOCK - n))).reshape(blocks, BLOCK)
    most = np.minimum(np.fmax.reduce(ax, axis=1), np.finfo(F32).max)  # values that are not finite count as the largest
    scale = np.maximum(most * (F32(1.0) / top), np.finfo(F32).tiny).astype(F32)
    z = np.fmin(ax * (F32(1.0) / scale)[:, None], top).reshape(-1)[:n]
    grid = code_values(False)
    low = z < F32(8.0)
    zz = np.where(low, z + F32(8.0), z).astype(np.float64)  # the subnormal codes are spaced as those of [8, 16)
    e = np.floor(np.log2(zz))
    e = np.where(2.0 ** e > zz, e - 1, np.where(2.0 ** (e + 1) <= zz, e + 1, e))
    frac = np.floor((zz / 2.0 ** e - 1.0) * 8.0)
    base = np.where(low, frac, 8.0 * (e - 2.0) + frac).astype(np.int64)
    rest = np.floor(((zz / 2.0 ** e - 1.0) * 8.0 - frac) * 2.0 ** 20).astype(np.int64)  # the code's remainder, 20 bits
    code = base + ((rest + (np.asarray(noise16, dtype=np.int64) << 4)) >> 20)
    assert np.all(code < grid.size)
    if signed:
        code = code | np.where(np.signbit(x), 128, 0)
    else:
        code = np.maximum(code, z > 0)
    return code.astype(np.uint8), scale
