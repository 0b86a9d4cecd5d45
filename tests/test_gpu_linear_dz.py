"""The gradients of a linear layer with a smooth activation, whose products take
dy act'(pre) in two parts: within the roundings of the results alone, past float16's
range, with an infinite operand; and rounded once where the caller asks for it."""

import numpy as np
import pytest
import torch

from momentum_compression_amd import onebit as ob
from oracle import block as ref
from tests._gpu import device
from tests.test_gpu_linear import (E, TYPES, check_backward, close, h64, half, inputs, least, t_slope,
                                   workspace)

pytestmark = pytest.mark.gpu

# what the two parts leave of dz: a part of bfloat16 is cut off after 8 bits and the
# rest, at most 2^-7 of it, rounded to 8 (float16: 11 and 2^-10)
PARTS = {"bf16": (2.0 ** -15, 2.0 ** -133), "f16": (2.0 ** -21, 2.0 ** -25)}
SHAPES = [(1, 1, 1), (1, 16, 8), (3, 5, 7), (33, 31, 65), (70, 127, 200), (129, 130, 136),
          (200, 24, 2000), (257, 264, 1), (64, 12, 4), (640, 300, 512), (1030, 1000, 9),
          (2100, 65, 70)]


def run(x, w, dy, pre, act, dw_type=None, round_dz=False):
    (M, K), N = x.shape, w.shape[0]
    dx, db = torch.empty_like(x), torch.empty(N, device=x.device)
    dw = torch.empty(N, K, dtype=dw_type or x.dtype, device=x.device)
    ob.linear_backward(dy, x, w, dx=dx, dw=dw, dbias=db, activation=act, pre=pre,
                       ws=workspace(M, N, K, True, x.device), round_dz=round_dz)
    return dx, dw, db


def check(x, w, dy, pre, act, dtype, got, name, rel=None):
    G, X, W, Z = h64(dy), h64(x), h64(w), h64(pre)
    dx, dw, _ = got
    wdx, wdw, _, dz = ref.linear_grad(G, X, W, act, Z)
    M, N = G.shape
    rel, tiny = (rel or PARTS[dtype][0]), PARTS[dtype][1]
    t_dz = np.abs(G) * t_slope(Z, act) + (2 * E + rel) * np.abs(dz) + tiny
    # two products of each element are summed
    t = t_dz @ np.abs(W) + 2 * (2 * N + 4) * E * ((np.abs(dz) + t_dz) @ np.abs(W))
    close(dx, wdx, t + half(dx.dtype) * (np.abs(wdx) + t) + least(dx.dtype), f"{name} dx")
    t = t_dz.T @ np.abs(X) + 2 * (2 * M + 4) * E * ((np.abs(dz) + t_dz).T @ np.abs(X))
    close(dw, wdw, t + half(dw.dtype) * (np.abs(wdw) + t) + least(dw.dtype), f"{name} dw")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_results_are_rounded_once(dtype, M, N, K):
    dev = device()
    x, w, _, dy, pre = inputs(M, N, K, dtype, dev)
    for act in ("gelu", "gelu_tanh", "silu"):
        for dw_type in (None, torch.float32):
            print(f"[linear] dz {dtype} {M}x{N}x{K} {act}", flush=True)
            got = run(x, w, dy, pre, act, dw_type)
            check(x, w, dy, pre, act, dtype, got, f"{M}x{N}x{K} {act}")
            rounded = run(x, w, dy, pre, act, dw_type, round_dz=True)
            check_backward(dy, x, w, act, pre, *rounded, f"{M}x{N}x{K} {act} rounded")
            assert torch.equal(got[2], rounded[2])
    for act in ("none", "relu"):  # dz is a number of the type
        a, b = (run(x, w, dy, pre, act, torch.float32, round_dz=r) for r in (False, True))
        assert all(torch.equal(p, q) for p, q in zip(a, b)), act


@pytest.mark.parametrize("dtype", TYPES)
def test_large_products(dtype):
    """Sizes of the large tiles and of sums in parts, against float64 on the GPU; the
    same bits again, eagerly and from a graph."""
    dev = device()
    for M, N, K in ((2048, 4096, 1024), (4100, 2056, 520), (16384, 128, 256)):
        print(f"[linear] dz large {dtype} {M}x{N}x{K}", flush=True)
        x, w, _, dy, pre = inputs(M, N, K, dtype, dev)
        dx, dw, db = run(x, w, dy, pre, "silu", torch.float32)
        Z, G = pre.double(), dy.double()
        s = torch.sigmoid(Z)
        dz = G * (s + Z * s * torch.sigmoid(-Z))
        rel, tiny = PARTS[dtype]
        t_dz = G.abs() * (1e-7 + 40 * E * (1 + Z.abs())) + (2 * E + rel) * dz.abs() + tiny
        for name, got, a, ta, b, n in (("dx", dx, dz, t_dz, w.double(), N),
                                       ("dw", dw, dz.t().contiguous(), t_dz.t().contiguous(),
                                        x.double(), M)):
            want = a @ b
            t = ta @ b.abs() + 2 * (2 * n + 4) * E * ((a.abs() + ta) @ b.abs())
            t = t + half(got.dtype) * (want.abs() + t) + least(got.dtype)
            bad = ~((got.double() - want).abs() <= t)
            assert not bool(bad.any()), (name, int(bad.sum()))
        outs = dict(dx=torch.empty_like(dx), dw=torch.empty_like(dw), dbias=torch.empty_like(db))
        ws = workspace(M, N, K, True, dev)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ob.linear_backward(dy, x, w, **outs, activation="silu", pre=pre, ws=ws)
        for k in range(3):
            dy.mul_(0.5)
            graph.replay()
            want = run(x, w, dy, pre, "silu", torch.float32)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs.values(), want)), (M, N, K, k)


def test_past_the_range_of_float16():
    """A slope above 1 takes dz past the type's range where dx and dw are inside it."""
    dev, t = device(), torch.float16
    M, N, K = 40, 72, 24
    dy = torch.full((M, N), 60000.0, dtype=t, device=dev)
    dy[::2] *= -1
    pre = torch.full((M, N), 1.5, dtype=t, device=dev)
    x = torch.full((M, K), 2.0 ** -8, dtype=t, device=dev)
    w = torch.full((N, K), 2.0 ** -8, dtype=t, device=dev)
    got = run(x, w, dy, pre, "gelu", torch.float32)
    assert float(ref.slope(np.array([1.5]), "gelu")[0]) * 60000 > 65504 * 1.03
    # the first part is the type's largest number, the rest up to 2^-3 of dz
    check(x, w, dy, pre, "gelu", "f16", got, "range", rel=2.0 ** -14)
    assert bool(got[0].isfinite().all())


@pytest.mark.parametrize("dtype", TYPES)
def test_infinite_operands(dtype):
    """An infinite weight or input makes infinities of dz's sign, as one product does."""
    dev = device()
    M, N, K = 40, 24, 16
    x, w, _, dy, pre = inputs(M, N, K, dtype, dev)
    dy[3], pre[3] = 1.0, 40.0   # a slope of 1: dz is a number of the type
    inf = float("inf")
    w[5, 7], x[3, 2], x[6, 9] = inf, -inf, inf
    for act in ("gelu", "gelu_tanh", "silu"):
        dx, dw, _ = run(x, w, dy, pre, act)
        dz = h64(dy) * ref.slope(h64(pre), act)
        assert (np.abs(dz[:, 5]) > 1e-6).all() and (np.abs(dz[[3, 6]]) > 1e-6).all()
        assert np.array_equal(h64(dx)[:, 7], np.sign(dz[:, 5]) * inf), act
        assert np.array_equal(h64(dw)[:, 2], -np.sign(dz[3]) * inf), act
        assert np.array_equal(h64(dw)[:, 9], np.sign(dz[6]) * inf), act
        assert np.isfinite(np.delete(h64(dx), 7, 1)).all()
        assert np.isfinite(np.delete(h64(dw), [2, 9], 1)).all()
    # infinite and NaN gradients
    x, w, _, dy, pre = inputs(M, N, K, dtype, dev, seed=2)
    dy[4, 1], dy[9, 2] = -inf, float("nan")
    pre[4, 1] = 2.0
    dx, dw, _ = run(x, w, dy, pre, "silu")
    assert np.array_equal(h64(dx)[4], np.where(h64(w)[1] > 0, -inf, inf))
    assert np.array_equal(h64(dw)[1], np.where(h64(x)[4] > 0, -inf, inf))
    assert bool(dx[9].isnan().all()) and bool(dw[2].isnan().all())
    assert int((~dx.isfinite()).any(1).sum()) == 2 and int((~dw.isfinite()).any(1).sum()) == 2
