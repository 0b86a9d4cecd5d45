"""Plain 64-bit forms of the training operators: dropout from a counter-based
mask, the relative position bias by buckets with its gradient, and attention
with both, forward and backward.

Everything is binary64 numpy from the definitions; the only whole-number work
is the generator (oracle/philox.py) and the buckets.  The library's results
are compared within tolerances derived from its roundings.
"""

from __future__ import annotations

import math

import numpy as np

from .philox import philox4x32_10

KEY_TAG = 0x44524F50
_MASK = 0xFFFFFFFF


def threshold(p: float) -> int:
    """Kept draws out of 65536."""
    return max(1, math.floor((1.0 - float(np.float32(p))) * 65536.0 + 0.5))


def draws(rows: int, cols: int, seed: int, step: int, row0: int = 0) -> np.ndarray:
    """The 16-bit draws of a [rows, cols] mask."""
    groups = (cols + 7) // 8
    R = np.arange(row0, row0 + rows, dtype=np.uint64)[:, None]
    ctr = np.zeros((rows, groups, 4), dtype=np.uint32)
    ctr[..., 0] = np.arange(groups, dtype=np.uint32)[None, :]
    ctr[..., 1] = (R & np.uint64(_MASK)).astype(np.uint32)
    ctr[..., 2] = (R >> np.uint64(32)).astype(np.uint32)
    ctr[..., 3] = np.uint32(step & _MASK)
    key = np.array([seed & _MASK, ((seed >> 32) & _MASK) ^ KEY_TAG], dtype=np.uint32)
    w = philox4x32_10(ctr, key)
    halves = np.stack([w & np.uint32(0xFFFF), w >> np.uint32(16)], axis=-1)
    return halves.reshape(rows, groups * 8)[:, :cols]


def keep_factor(rows, cols, p, seed, step, row0=0):
    """0 where dropped, 65536 / threshold where kept."""
    T = threshold(p)
    return np.where(draws(rows, cols, seed, step, row0) < T, 65536.0 / T, 0.0)


def dropout(x, p, seed, step, row0=0, residual=None):
    x = np.asarray(x, dtype=np.float64)
    f = keep_factor(x.shape[0], x.shape[1], p, seed, step, row0)
    with np.errstate(invalid="ignore"):
        y = np.where(f > 0, x * f, 0.0)
    return y if residual is None else np.asarray(residual, dtype=np.float64) + y


def bucket_map(n_buckets: int, max_distance: int, two_sided: bool) -> np.ndarray:
    """Bucket of each distance -max_distance ... max_distance: on a side with
    n buckets the distances below e = n // 2 have one each, and distance d
    from there on bucket e + floor((n - e) log(d / e) / log(max / e)), at most
    n - 1; decided by comparing whole powers."""
    out = []
    for d in range(-max_distance, max_distance + 1):
        n, base = n_buckets, 0
        if two_sided:
            n //= 2
            base, a = (n if d > 0 else 0), abs(d)
        else:
            a = max(-d, 0)
        e = n // 2
        if a < e or n == 1:
            out.append(base + min(a, n - 1))
            continue
        if e == 0:
            e = 1
        k = 0
        while (e + k + 1 < n
               and a ** (n - e) >= e ** (n - e - (k + 1)) * max_distance ** (k + 1)):
            k += 1
        out.append(base + e + k if a >= e else base + a)
    return np.array(out, dtype=np.int32)


def distances(Tq: int, Tk: int, q_pos: int, radius: int) -> np.ndarray:
    """Index into the map of every (query, key)."""
    d = np.arange(Tk)[None, :] - (np.arange(Tq)[:, None] + q_pos)
    return np.clip(d, -radius, radius) + radius


def rel_bias(table, bmap, Tq, Tk, q_pos=0):
    """[H, Tq, Tk]; a bucket outside the table counts as no bias."""
    table = np.asarray(table, dtype=np.float64)
    b = np.asarray(bmap)[distances(Tq, Tk, q_pos, len(bmap) // 2)]
    ok = (b >= 0) & (b < table.shape[0])
    out = table[np.where(ok, b, 0)] * ok[..., None]
    return np.ascontiguousarray(out.transpose(2, 0, 1))


def rel_bias_grad(ds, bmap, n_buckets, q_pos=0):
    """[n_buckets, H] from ds [B, H, Tq, Tk]."""
    ds = np.asarray(ds, dtype=np.float64)
    _, H, Tq, Tk = ds.shape
    b = np.asarray(bmap)[distances(Tq, Tk, q_pos, len(bmap) // 2)].ravel()
    s = ds.sum(0).reshape(H, Tq * Tk)
    out = np.zeros((n_buckets, H))
    for k in range(n_buckets):
        out[k] = s[:, b == k].sum(1)
    return out


def attention(q, k, v, scale, causal=False, q_pos=0, k_len=None, table=None, bmap=None, p=0.0,
              seed=0, step=0, do=None):
    """q [B, Tq, H, D], k and v [B, Tk, Hkv, D]; q_pos a number or one per
    sequence.  Returns o and lse, and with do the gradients.  A query that
    sees no key gives o = 0, lse = -inf and no gradient."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    B, Tq, H, D = q.shape
    Tk, Hkv = k.shape[1], k.shape[2]
    G = H // Hkv
    out = dict(o=np.zeros_like(q), lse=np.full((B, H, Tq), -np.inf))
    if do is not None:
        do = np.asarray(do, dtype=np.float64)
        out.update(dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v))
        if table is not None:
            out["dtable"] = np.zeros(np.asarray(table).shape)
    for b in range(B):
        pos = int(q_pos[b]) if np.ndim(q_pos) else int(q_pos)
        n = Tk if k_len is None else int(np.clip(k_len[b], 0, Tk))
        seen = np.broadcast_to(np.arange(Tk)[None, :] < n, (Tq, Tk)).copy()
        if causal:
            seen &= np.arange(Tk)[None, :] <= np.arange(Tq)[:, None] + pos
        bias = rel_bias(table, bmap, Tq, Tk, pos) if table is not None else None
        for h in range(H):
            kh, vh = k[b, :, h // G], v[b, :, h // G]
            z = (q[b, :, h] @ kh.T) * scale
            if bias is not None:
                z = z + bias[h]
            z = np.where(seen, z, -np.inf)
            m = z.max(1, initial=-np.inf, keepdims=True)
            some = np.isfinite(m)
            e = np.where(seen, np.exp(z - np.where(some, m, 0.0)), 0.0)
            total = e.sum(1, keepdims=True)
            prob = e / np.where(some, total, 1.0)
            with np.errstate(divide="ignore"):
                out["lse"][b, h] = np.where(some, m + np.log(total), -np.inf)[:, 0]
            f = keep_factor(Tq, Tk, p, seed, step, (b * H + h) * Tq) if p > 0 else 1.0
            out["o"][b, :, h] = (prob * f) @ vh
            if do is None:
                continue
            g = do[b, :, h]
            dp = (g @ vh.T) * f
            ds = prob * (dp - (prob * dp).sum(1, keepdims=True))
            out["dv"][b, :, h // G] += (prob * f).T @ g
            out["dq"][b, :, h] = ds @ kh * scale
            out["dk"][b, :, h // G] += ds.T @ q[b, :, h] * scale
            if table is not None:
                out["dtable"][:, h] += rel_bias_grad(ds[None, None], bmap, len(table), pos)[:, 0]
    return out
