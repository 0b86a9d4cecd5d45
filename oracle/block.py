"""Plain forms of the operators of a transformer block beside attention: layer
norm and the linear layer with their gradients in binary64, and the AdamW step
in binary32, one rounding an operation, with its 8-bit states.

The formulas are the header's; no outside implementation is involved.  The
activations' integrals come from ``math`` and ``scipy``-free identities, pinned
by differences in the tests.
"""

from __future__ import annotations

import math

import numpy as np

from .philox import philox4x32_10

F32 = np.float32
KEY_TAG = 0x41444D57
BLOCK = 256
_MASK = 0xFFFFFFFF
_erfc = np.frompyfunc(math.erfc, 1, 1)


# ---------------------------------------------------------------- layer norm
def layer_norm(x, weight, bias, eps):
    """(y, mean, rstd) by rows."""
    x = np.asarray(x, np.float64)
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(1) + float(F32(eps)))
    return d * rstd[:, None] * weight + bias, mean, rstd


def layer_norm_grad(dy, x, mean, rstd, weight):
    """(dx, dweight, dbias) with the mean and rstd that are given."""
    h = (x - mean[:, None]) * rstd[:, None]
    u = dy * weight
    dx = rstd[:, None] * (u - u.mean(1, keepdims=True) - h * (u * h).mean(1, keepdims=True))
    return dx, (dy * h).sum(0), dy.sum(0)


# ---------------------------------------------------------------- linear layer
def _sigmoid(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def _phi(z):
    return 0.5 * _erfc(-z / math.sqrt(2.0)).astype(np.float64)


_RATE, _CUBIC = 2.0 * math.sqrt(2.0 / math.pi), 0.044715


def activate(z, act):
    return {"none": lambda: z, "relu": lambda: np.maximum(z, 0.0), "gelu": lambda: z * _phi(z),
            "gelu_tanh": lambda: z * _sigmoid(_RATE * (z + _CUBIC * z ** 3)),
            "silu": lambda: z * _sigmoid(z)}[act]()


def slope(z, act):
    if act == "none":
        return np.ones_like(z)
    if act == "relu":
        return (z > 0).astype(np.float64)
    if act == "gelu":
        return _phi(z) + z * np.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    s = _sigmoid(z if act == "silu" else _RATE * (z + _CUBIC * z ** 3))
    rate = 1.0 if act == "silu" else _RATE * (1 + 3 * _CUBIC * z * z)
    return s + z * s * (1 - s) * rate


def linear(x, w, bias, act, residual=None):
    """(y, z)."""
    z = x @ w.T + bias
    y = activate(z, act)
    return (y if residual is None else y + residual), z


def linear_grad(dy, x, w, act, pre):
    """(dx, dw, dbias, dz)."""
    dz = dy if act == "none" else dy * slope(pre, act)
    return dz @ w, dz.T @ x, dz.sum(0), dz


# ---------------------------------------------------------------- AdamW
def draws(n, tensor, step, seed, first=0):
    """The 16-bit draws of n elements of a tensor, from `first` (a multiple of 8) on."""
    groups = (n + 7) // 8
    ctr = np.zeros((groups, 4), dtype=np.uint32)
    ctr[:, 0] = np.arange(groups, dtype=np.uint32) + np.uint32(first // 8)
    ctr[:, 1] = tensor
    ctr[:, 3] = np.uint32(step & _MASK)
    key = np.array([seed & _MASK, ((seed >> 32) & _MASK) ^ KEY_TAG], dtype=np.uint32)
    w = philox4x32_10(ctr, key)
    return np.stack([w & np.uint32(0xFFFF), w >> np.uint32(16)], axis=-1).reshape(-1)[:n]


def decode(codes, digits):
    """Values of e4m3 (digits 3) or e5m2 (digits 2) codes."""
    bias = 7 if digits == 3 else 15
    c = codes.astype(np.int64)
    e, f = (c & 0x7F) >> digits, c & ((1 << digits) - 1)
    y = np.where(e == 0, np.ldexp(f.astype(np.float64), 1 - bias - digits),
                 np.ldexp((f + (1 << digits)).astype(np.float64), e - bias - digits))
    if digits == 3:
        y = np.where((c & 0x7F) == 0x7F, np.nan, y)
    else:
        y = np.where(e == 31, np.where(f == 0, np.inf, np.nan), y)
    return np.where(c & 0x80, -y, y).astype(F32)


def encode(x, u, digits, positive):
    """(codes, scales) of binary32 values with the draws u."""
    n = x.size
    top, least, nan = (7, -6, 0x7F) if digits == 3 else (14, -14, 0x7E)
    codes, scales = np.zeros(n, np.uint8), np.zeros((n + BLOCK - 1) // BLOCK, F32)
    for b in range(scales.size):
        s = slice(b * BLOCK, min(n, (b + 1) * BLOCK))
        v = x[s]
        ok = np.isfinite(v)
        most = float(np.abs(v[ok]).max(initial=0.0))
        e = max(math.frexp(most)[1] - 1 - top if most > 0 else -126, -126)
        scales[b] = F32(math.ldexp(1.0, e))
        y = np.ldexp(np.abs(np.where(ok, v, 0)).astype(np.float64), -e)
        step = np.ldexp(1.0, np.maximum(np.frexp(y)[1] - 1, least) - digits)
        r = np.floor(y / step + (u[s] + 0.5) / 65536.0) * step
        f, k = np.frexp(r)
        ex = np.where(r == 0, least, np.maximum(k - 1, least))
        whole = np.ldexp(r, digits - ex)  # mantissa with its leading one
        field = np.where(whole >= (1 << digits), ex - least + 1, 0)
        c = (field << digits) + (whole.astype(np.int64) & ((1 << digits) - 1))
        if positive:
            c = np.where((v > 0) & (c == 0), 1, c)
        c = np.where(ok, c, np.where(np.isinf(v) & positive, 0x7C, nan))
        codes[s] = c | (np.signbit(v).astype(np.int64) << 7 if not positive else 0)
    return codes, scales


def adamw(x, g, m, v, lr, beta1, beta2, eps, step, lr_scale=1.0, weight_decay=0.0, g_scale=None):
    """(x, m, v) after a step, binary32 throughout."""
    lr, b1, b2, eps = F32(lr), F32(beta1), F32(beta2), F32(eps)
    bc1 = F32(1.0 / (1.0 - float(b1) ** step))
    bc2 = F32(1.0 / math.sqrt(1.0 - float(b2) ** step))
    one, lr_t = F32(1.0), lr * F32(lr_scale)
    g = g.astype(F32)
    with np.errstate(all="ignore"):
        if g_scale is not None:
            g = g * F32(g_scale)
        m = b1 * m + (one - b1) * g
        v = b2 * v + (one - b2) * (g * g)
        x = x * (one - lr_t * F32(weight_decay)) - (lr_t * bc1) * (m / (np.sqrt(v) * bc2 + eps))
    return x, m, v
