"""Inputs, calls and error bounds of the attention tests.

Bounds.  With u half a step of the element type (bf16 2^-8, fp16 2^-11) and
e = 2^-24 (binary32), to first order and per element:

  score     off by  ds = (D + 8) e (scale |q|.|k| + |bias| + |s|): D products
            are summed in binary32, then one fused scale-and-bias and the
            base-2 exponential's argument round
  weight    relative  ep = 2 max ds + (Tk + 24) e + 4 e (|lse| + 1): its own
            score, the row sum's scores and additions, the normaliser
  o         u |o| (stored) + (u + ep) sum P keep |v| (weights rounded for the
            product)
  dP        D e keep |do|.|v|;  delta from the stored o: sum_d |do| (bound of o)
            + D e |do|.|o|, exact delta: sum P (ep |dP| + bound of dP) + Tk e
            sum P |dP|
  dS        P (ep (|dP| + |delta|) + bound of dP + bound of delta), and u |dS|
            where it is rounded for a product
  dq, dk    scale times the product of that bound with |k| or |q|, (n + 8) e
            of the sum's own terms, u of the result; dv as o
  short     up to 64 queries and keys the gradients' products take P and dS as a
            rounded part and a rounded rest (u^2), with the exact delta
  below     a weight or dS below the type's normal range is rounded by up to half
            its smallest step instead (`sub`); weights are at least as large
            against their row's sum as they are alone
  dtable    the unrounded dS's bounds summed, and the additions' e: fewer than
            8 roundings a tile of 32 and one a tile on the way
"""

from __future__ import annotations

import numpy as np
import torch

from momentum_compression_amd import onebit as ob
from oracle import training as ref

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
E = 2.0 ** -24
SEED = 0xFEED_0123_4567_89AB


def half_step(dtype):
    return torch.finfo(TYPES[dtype]).eps / 2


def below_normal(u):
    """Half the smallest step of the type with half step u."""
    return 2.0 ** -25 if u == 2.0 ** -11 else 2.0 ** -134


def expected(q, k, v, do, scale, causal, q_pos, k_len, table, bmap, p, seed, step, u):
    """(oracle results, bounds), both dicts of numpy arrays."""
    want = ref.attention(q, k, v, scale, causal, q_pos, k_len, table, bmap, p, seed, step, do=do)
    B, Tq, H, D = q.shape
    Tk, Hkv = k.shape[1], k.shape[2]
    G = H // Hkv
    sub = below_normal(u)
    short = max(Tq, Tk) <= 64
    u_p = u * u if short else u
    tol = {n: np.zeros_like(x) for n, x in want.items()}
    for b in range(B):
        pos = int(q_pos[b]) if np.ndim(q_pos) else int(q_pos)
        n = Tk if k_len is None else int(np.clip(k_len[b], 0, Tk))
        seen = np.broadcast_to(np.arange(Tk)[None, :] < n, (Tq, Tk)).copy()
        if causal:
            seen &= np.arange(Tk)[None, :] <= np.arange(Tq)[:, None] + pos
        bias = ref.rel_bias(table, bmap, Tq, Tk, pos) if table is not None else None
        for h in range(H):
            qh, kh, vh = q[b, :, h], k[b, :, h // G], v[b, :, h // G]
            lse = want["lse"][b, h][:, None]
            some = np.isfinite(lse)
            bh = bias[h] if bias is not None else np.zeros((Tq, Tk))
            s = qh @ kh.T * scale + bh
            prob = np.where(seen, np.exp(s - np.where(some, lse, 0.0)), 0.0)
            size = scale * (np.abs(qh) @ np.abs(kh).T) + np.abs(bh) + np.abs(s)
            ds_ = (D + 8) * E * np.where(seen, size, 0.0)
            worst = ds_.max(1, initial=0.0, keepdims=True)
            ln = np.where(some, np.abs(lse), 0.0) + 1
            ep = 2 * worst + (Tk + 24) * E + 4 * E * ln
            tol["lse"][b, h] = (worst + (Tk + 24) * E + 4 * E * ln)[:, 0]
            f = ref.keep_factor(Tq, Tk, p, seed, step, (b * H + h) * Tq) if p > 0 else 1.0
            o = want["o"][b, :, h]
            to = u * np.abs(o) + ((u + ep) * prob * f + sub * seen * f) @ np.abs(vh)
            tol["o"][b, :, h] = to
            if do is None:
                continue
            g = do[b, :, h]
            A = f * (np.abs(g) @ np.abs(vh).T)
            dp = (g @ vh.T) * f
            delta = (prob * dp).sum(1, keepdims=True)
            tdp = (D + 2) * E * A
            t_delta = (np.abs(g) * (to + D * E * np.abs(o))).sum(1, keepdims=True)
            t_exact = ((prob * (ep * np.abs(dp) + tdp)).sum(1, keepdims=True)
                       + Tk * E * (prob * np.abs(dp)).sum(1, keepdims=True))
            ds = prob * (dp - delta)
            t_ds = prob * (ep * (np.abs(dp) + np.abs(delta)) + tdp)
            t_round = (t_ds + prob * (t_exact if short else t_delta) + u_p * np.abs(ds)
                       + sub * seen * np.max(f))
            tol["dq"][b, :, h] = scale * ((t_round + (Tk + 8) * E * np.abs(ds)) @ np.abs(kh))
            tol["dk"][b, :, h // G] += scale * ((t_round + (G * Tq + 8) * E * np.abs(ds)).T
                                                @ np.abs(qh))
            tol["dv"][b, :, h // G] += ((u_p + ep + (G * Tq + 8) * E) * prob * f
                                        + sub * seen * f).T @ np.abs(g)
            if table is not None:
                adds = 8 * (Tq + Tk) / 32 + Tk / 8 + 64
                both = t_ds + prob * t_exact + adds * E * np.abs(ds)
                # sums past the radius are the difference of two sums
                both += adds * E * prob * (np.abs(dp) + np.abs(delta))
                tol["dtable"][:, h] += ref.rel_bias_grad(both[None, None], bmap, len(table),
                                                         pos)[:, 0]
    if do is not None:
        for name in ("dq", "dk", "dv"):
            tol[name] += u * np.abs(want[name])
        if table is not None:
            tol["dtable"] += 2 * E * np.abs(want["dtable"])
    return want, tol


def check(got, want, tol, names, tiny):
    """Every element within its bound (`tiny`: half the smallest step of the
    type, for results below its normal range)."""
    for name in names:
        g = got[name].double().cpu().numpy()
        w, t = want[name], tol[name]
        assert g.shape == w.shape, name
        same = (g == w) & ~np.isfinite(w)
        with np.errstate(invalid="ignore"):
            bad = ~(same | (np.abs(g - w) <= 1.02 * t + tiny))
        if bad.any():
            at = tuple(np.argwhere(bad)[0])
            raise AssertionError(f"{name}: {bad.sum()} of {bad.size} outside their bound, first at "
                                 f"{at}: {g[at]} for {w[at]} +- {t[at]}")


def make(dtype, B, H, Hkv, Tq, Tk, D, gen, dev, fused=False, scale=1.0):
    def rand(*shape):
        return (torch.randn(shape, generator=gen, device=dev) * scale).to(TYPES[dtype])

    if fused:
        qkv = rand(B, Tq, H + 2 * Hkv, D)
        return qkv[:, :, :H], qkv[:, :, H:H + Hkv], qkv[:, :, H + Hkv:]
    return rand(B, Tq, H, D), rand(B, Tk, Hkv, D), rand(B, Tk, Hkv, D)


def workspace(q, k, radius=0, backward=False):
    B, Tq, H, D = q.shape
    n = ob.rel_attention_workspace_bytes(B, H, k.shape[2], Tq, k.shape[1], D, radius, backward)
    assert n > 0
    return torch.full((n,), 0xFF, dtype=torch.uint8, device=q.device)  # NaN where it is read


def host64(x):
    return None if x is None else x.double().cpu().numpy()


def numbers(x):
    """q_pos or k_len as the oracle takes it."""
    return x.cpu().numpy() if torch.is_tensor(x) else x
