"""linear_forward and linear_backward against the 64-bit forms, within bounds
that count their roundings."""

import numpy as np
import pytest
import torch

from momentum_compression_amd import onebit as ob
from oracle import block as ref
from tests._gpu import device, gen

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
E = 2.0 ** -24
# rows of one token and of batches, tiles' edges, odd sizes, depths of less than a
# tile and of many
SHAPES = [(1, 1, 1), (1, 8, 8), (3, 5, 7), (1, 1000, 333), (2, 264, 64), (17, 96, 128),
          (32, 160, 72), (33, 31, 65), (70, 127, 200), (128, 128, 64), (129, 130, 136),
          (5, 2050, 1096), (200, 24, 2000), (300, 520, 40), (257, 264, 1), (513, 1, 96),
          (640, 300, 512)]


def h64(t):
    return None if t is None else t.double().cpu().numpy()


def half(t):
    return torch.finfo(t).eps / 2 * 1.001


def least(t):
    """Half the smallest step of the type."""
    return 2.0 ** -25 if t == torch.float16 else 2.0 ** -140


def close(got, want, tol, name):
    got = h64(got)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size}, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {want[bad][0]} +- {tol[bad][0]}")


def t_act(z, act):
    """What an activation's own arithmetic adds: the integral of the normal
    distribution to 7.5e-8, a few roundings of binary32 otherwise."""
    if act in ("none", "relu"):
        return 0.0 * z
    return np.abs(z) * (1e-7 + 16 * E)


def t_slope(z, act):
    if act in ("none", "relu"):
        return 0.0 * z
    return 1e-7 + 40 * E * (1 + np.abs(z))


def workspace(M, N, K, backward, dev):
    n = ob.linear_workspace_bytes(M, N, K, backward)
    assert n > 0
    return torch.full((n,), 0xFF, dtype=torch.uint8, device=dev)  # NaN where it is read


def check_forward(x, w, y, bias, act, residual, pre, name):
    X, W = h64(x), h64(w)
    Bv = 0.0 if bias is None else h64(bias)
    want, z = ref.linear(X, W, Bv, act, h64(residual))
    t = 2 * (X.shape[1] + 4) * E * (np.abs(X) @ np.abs(W).T) + 2 * E * np.abs(z)
    if pre is not None:
        close(pre, z, t + half(y.dtype) * (np.abs(z) + t) + least(y.dtype), f"{name} pre")
    t = 1.2 * t + t_act(z, act) + 2 * E * (np.abs(want) + np.abs(z))
    close(y, want, t + half(y.dtype) * (np.abs(want) + t) + least(y.dtype), f"{name} y")


def check_backward(dy, x, w, act, pre, dx, dw, db, name, before=0.0):
    G, X, W = h64(dy), h64(x), h64(w)
    Z = np.zeros_like(G) if pre is None else h64(pre)
    wdx, wdw, wdb, dz = ref.linear_grad(G, X, W, act, Z)
    M, N = G.shape
    t_unrounded = np.abs(G) * t_slope(Z, act) + 2 * E * np.abs(dz)
    t_dz = 0.0 * dz
    if act != "none":
        t_dz = t_unrounded + half(dy.dtype) * (np.abs(dz) + t_unrounded) + least(dy.dtype)
    if dx is not None:
        t = t_dz @ np.abs(W) + 2 * (N + 4) * E * ((np.abs(dz) + t_dz) @ np.abs(W))
        close(dx, wdx, t + half(dx.dtype) * (np.abs(wdx) + t) + least(dx.dtype), f"{name} dx")
    if dw is not None:
        wdw = wdw + before
        t = t_dz.T @ np.abs(X) + 2 * (M + 4) * E * ((np.abs(dz) + t_dz).T @ np.abs(X))
        t = t + 2 * E * np.abs(wdw)
        u = half(dw.dtype)
        close(dw, wdw, t + u * (np.abs(wdw) + t) + least(dw.dtype), f"{name} dw")
    if db is not None:
        wdb = wdb + before
        t = t_unrounded.sum(0) + (M + 8) * E * np.abs(dz).sum(0) + 2 * E * np.abs(wdb) + 1e-30
        close(db, wdb, t, f"{name} dbias")


def inputs(M, N, K, dtype, dev, seed=0):
    g = gen(seed + 7 * M + 3 * N + K, dev)
    t = TYPES[dtype]

    def rand(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(t)

    return rand(M, K), rand(N, K, scale=max(1, K) ** -0.5), rand(M, N), rand(M, N), rand(M, N)


def both(M, N, K, dtype, act, dev, residual=True, dw_type=None, wide_bias=True, seed=0):
    x, w, r, dy, pre_in = inputs(M, N, K, dtype, dev, seed)
    t = TYPES[dtype]
    b = torch.randn(N, generator=gen(1, dev), device=dev).to(torch.float32 if wide_bias else t)
    r = r if residual else None
    y, pre = torch.empty(M, N, dtype=t, device=dev), torch.empty(M, N, dtype=t, device=dev)
    name = f"{M}x{N}x{K} {act}"
    ob.linear_forward(x, w, y, bias=b, activation=act, residual=r, pre=pre,
                      ws=workspace(M, N, K, False, dev))
    check_forward(x, w, y, b, act, r, pre, name)
    dx, db = torch.empty_like(x), torch.empty(N, device=dev)
    dw = torch.empty(N, K, dtype=dw_type or t, device=dev)
    ob.linear_backward(dy, x, w, dx=dx, dw=dw, dbias=db, activation=act, pre=pre_in,
                       ws=workspace(M, N, K, True, dev))
    check_backward(dy, x, w, act, pre_in, dx, dw, db, name)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_shapes(dtype, M, N, K):
    dev = device()
    for k, act in enumerate(("none", ACTS[1 + (M + N) % 4])):
        print(f"[linear] {dtype} {M}x{N}x{K} {act}", flush=True)
        both(M, N, K, dtype, act, dev, residual=k == 0, wide_bias=k == 0,
             dw_type=torch.float32 if k == 0 else None)


@pytest.mark.parametrize("act", ACTS)
def test_activations(act):
    """Each activation over a wide range of sums, and its slope."""
    dev = device()
    for dtype in TYPES:
        both(40, 72, 24, dtype, act, dev, seed=5)
    # one feature times one weight: the sum is the input
    x = torch.linspace(-12, 12, 4096, device=dev).to(torch.float16).view(-1, 1)
    w = torch.ones(1, 1, device=dev, dtype=torch.float16)
    y = torch.empty_like(x)
    ws = workspace(4096, 1, 1, True, dev)
    ob.linear_forward(x, w, y, activation=act, ws=ws)
    check_forward(x, w, y, None, act, None, None, act)
    dx, dy = torch.empty_like(x), torch.ones_like(x)
    ob.linear_backward(dy, x, w, dx=dx, activation=act, pre=x, ws=ws)
    check_backward(dy, x, w, act, x, dx, None, None, act)


@pytest.mark.parametrize("act", ACTS)
def test_what_is_no_number(act):
    """Infinite and NaN sums give the limits, and no others do."""
    dev = device()
    bf = torch.bfloat16
    inf, nan = float("inf"), float("nan")
    x = torch.tensor([[inf], [-inf], [nan], [1.0], [-3e38], [3e38]], device=dev, dtype=bf)
    w = torch.ones(8, 1, device=dev, dtype=bf)
    y = torch.empty(6, 8, device=dev, dtype=bf)
    ws = workspace(6, 8, 1, True, dev)
    ob.linear_forward(x, w, y, activation=act, ws=ws)
    want = [inf, -inf if act == "none" else 0.0, nan]
    for row, v in enumerate(want):
        got = y[row].float()
        assert bool(got.isnan().all()) if v != v else bool((got == v).all()), (row, got)
    assert bool(y[3].isfinite().all())
    assert bool((y[4].float() == (float(x[4]) if act == "none" else 0.0)).all())
    assert bool((y[5] == x[5]).all())
    if act == "none":
        return
    dy = torch.ones(6, 8, device=dev, dtype=bf)
    pre = x.expand(6, 8).contiguous()
    db, dx = torch.empty(8, device=dev), torch.empty(6, 1, device=dev, dtype=bf)
    ob.linear_backward(dy, x, w, dx=dx, activation=act, pre=pre, ws=ws)
    for row, v in ((0, 8.0), (1, 0.0), (4, 0.0), (5, 8.0)):
        assert float(dx[row]) == v, (row, dx[row])
    assert bool(dx[2].isnan())
    # a NaN in one row reaches that row of dx and all of its columns of dw alone
    M, N, K = 40, 24, 40
    x, w, _, dy, _ = inputs(M, N, K, "bf16", dev)
    dy[7, 3] = nan
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ob.linear_backward(dy, x, w, dx=dx, dw=dw, ws=workspace(M, N, K, True, dev))
    assert bool(dx[7].isnan().all()) and int(dx.isnan().any(1).sum()) == 1
    assert bool(dw[3].isnan().all()) and int(dw.isnan().any(1).sum()) == 1


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad,shift", [(8, 0), (8, 8), (5, 0), (8, 3)])
def test_views_and_what_lies_between(dtype, pad, shift):
    """Operands and results inside wider matrices, on 16 bytes and not; what lies
    beside them is NaN and stays as it is."""
    dev, t = device(), TYPES[dtype]
    M, N, K = 75, 104, 88
    x, w, r, dy, pre_in = inputs(M, N, K, dtype, dev)

    def inside(a, fill=float("nan")):
        whole = torch.full((a.shape[0], a.shape[1] + pad + shift), fill, device=dev, dtype=a.dtype)
        part = whole[:, shift:shift + a.shape[1]]
        part.copy_(a)
        return whole, part

    (_, x), (_, w), (_, r), (_, dy) = inside(x), inside(w), inside(r), inside(dy)
    _, pre_in = inside(pre_in)
    yy, y = inside(r.new_empty(M, N).zero_(), 7.0)
    pp, pre = inside(r.new_empty(M, N).zero_(), 7.0)
    b = torch.randn(N, generator=gen(1, dev), device=dev)
    ob.linear_forward(x, w, y, bias=b, activation="gelu", residual=r, pre=pre,
                      ws=workspace(M, N, K, False, dev))
    check_forward(x, w, y, b, "gelu", r, pre, "views")
    xx, dx = inside(x.new_empty(M, K).zero_(), 7.0)
    ww, dw = inside(torch.full((N, K), 0.5, device=dev), 7.0)
    db = torch.full((N,), 0.5, device=dev)
    for act, z in (("none", None), ("silu", pre_in)):
        dw.fill_(0.5), db.fill_(0.5)
        ob.linear_backward(dy, x, w, dx=dx, dw=dw, dbias=db, activation=act, pre=z, accumulate=True,
                           ws=workspace(M, N, K, True, dev))
        check_backward(dy, x, w, act, z, dx, dw, db, f"views {act}", before=0.5)
    for whole, part in ((yy, y), (pp, pre), (xx, dx), (ww, dw)):
        n = part.shape[1]
        assert bool((whole[:, :shift] == 7).all()) and bool((whole[:, shift + n:] == 7).all())
    # the residual's own place
    z = r.clone()
    ob.linear_forward(x, w, z, bias=b, activation="gelu", residual=z,
                      ws=workspace(M, N, K, False, dev))
    assert torch.equal(z, y)


def test_parts_of_the_gradients():
    """dx, dw and dbias alone are what they are together."""
    dev = device()
    M, N, K = 90, 56, 130
    x, w, _, dy, pre = inputs(M, N, K, "bf16", dev)
    for act in ("none", "gelu"):
        whole = dict(dx=torch.empty_like(x), dw=torch.empty_like(w), dbias=torch.empty(N, device=dev))
        how = dict(activation=act, pre=pre, ws=workspace(M, N, K, True, dev))
        ob.linear_backward(dy, x, w, **whole, **how)
        for name, want in whole.items():
            got = torch.empty_like(want)
            ob.linear_backward(dy, x, w, **{name: got}, **how)
            assert torch.equal(got, want), (act, name)
        ob.linear_backward(dy, x, w, **how)


def test_empty_sizes():
    dev, bf = device(), torch.bfloat16

    def e(*shape, fill=5.0, dtype=bf):
        return torch.full(shape, fill, device=dev, dtype=dtype)

    # no features to sum over: the bias, the activation and the residual are left
    b = torch.linspace(-2, 2, 9, device=dev)
    y, r = e(4, 9), torch.randn(4, 9, device=dev).to(bf)
    ob.linear_forward(e(4, 0), e(9, 0), y, bias=b, activation="relu", residual=r,
                      ws=workspace(4, 9, 0, False, dev))
    check_forward(e(4, 0), e(9, 0), y, b, "relu", r, None, "no features")
    # no rows
    dw, db = e(9, 6), e(9, dtype=torch.float32)
    how = dict(dx=e(0, 6), dw=dw, dbias=db, ws=workspace(0, 9, 6, True, dev))
    ob.linear_forward(e(0, 6), e(9, 6), e(0, 9), ws=workspace(0, 9, 6, False, dev))
    ob.linear_backward(e(0, 9), e(0, 6), e(9, 6), accumulate=True, **how)
    assert bool((dw == 5).all()) and bool((db == 5).all())
    ob.linear_backward(e(0, 9), e(0, 6), e(9, 6), **how)
    assert bool((dw == 0).all()) and bool((db == 0).all())
    # no columns
    dx = e(4, 6)
    ob.linear_backward(e(4, 0), e(4, 6), e(0, 6), dx=dx, dw=e(0, 6),
                       dbias=e(0, dtype=torch.float32), ws=workspace(4, 0, 6, True, dev))
    assert bool((dx == 0).all())


def test_large_and_the_same_bits_again():
    """Sizes that fill the GPU, against float64 products on it; twice the same
    bits, also on another stream and in a graph."""
    dev, bf = device(), torch.bfloat16
    for M, N, K in ((2048, 4096, 1024), (4100, 2056, 520), (16, 8192, 2048), (1, 1024, 8192)):
        print(f"[linear] large {M}x{N}x{K}", flush=True)
        x, w, r, dy, _ = inputs(M, N, K, "bf16", dev)
        y, pre = torch.empty_like(r), torch.empty_like(r)
        ws, wsb = workspace(M, N, K, False, dev), workspace(M, N, K, True, dev)
        ob.linear_forward(x, w, y, residual=r, pre=pre, ws=ws)
        X, W, G = x.double(), w.double(), dy.double()
        outs = dict(dx=torch.empty_like(x), dw=torch.empty(N, K, device=dev))
        ob.linear_backward(dy, x, w, **outs, ws=wsb)
        z = X @ W.t().contiguous()
        cases = [("pre", pre, z, X.abs() @ W.t().contiguous().abs(), K),
                 ("y", y, z + r.double(), X.abs() @ W.t().contiguous().abs(), K),
                 ("dx", outs["dx"], G @ W, G.abs() @ W.abs(), N),
                 ("dw", outs["dw"], G.t().contiguous() @ X, G.t().contiguous().abs() @ X.abs(), M)]
        for name, got, want, size, n in cases:
            t = 2 * (n + 4) * E * size + 3 * E * want.abs()
            t = t + half(got.dtype) * (want.abs() + t)
            bad = ~((got.double() - want).abs() <= t)
            assert not bool(bad.any()), (name, int(bad.sum()))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        y2, again = torch.empty_like(y), {k: torch.empty_like(v) for k, v in outs.items()}
        with torch.cuda.stream(side):
            ob.linear_forward(x, w, y2, residual=r, ws=ws)
            ob.linear_backward(dy, x, w, **again, ws=wsb)
        side.synchronize()
        assert torch.equal(y, y2) and all(torch.equal(outs[k], again[k]) for k in outs)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ob.linear_forward(x, w, y2, residual=r, ws=ws)
            ob.linear_backward(dy, x, w, **again, ws=wsb)
        for k in range(3):
            x.mul_(0.5)
            graph.replay()
            ob.linear_forward(x, w, y, residual=r, ws=ws)
            ob.linear_backward(dy, x, w, **outs, ws=wsb)
            torch.cuda.synchronize()
            assert torch.equal(y, y2) and all(torch.equal(outs[k], again[k]) for k in outs), k


def test_gradient_against_differences():
    """dx, dw and dbias in a direction against differences of the form."""
    dev = device()
    M, N, K, step = 12, 20, 16, 1e-4
    for act in ACTS[2:]:
        x, w, r, dy, _ = inputs(M, N, K, "bf16", dev, seed=3)
        b = torch.randn(N, generator=gen(4, dev), device=dev)
        ux, uw, _, _, _ = inputs(M, N, K, "bf16", dev, seed=11)
        y, pre = torch.empty_like(dy), torch.empty_like(dy)
        ob.linear_forward(x, w, y, bias=b, activation=act, pre=pre, ws=workspace(M, N, K, False, dev))
        dx, dw, db = torch.empty_like(x), torch.empty(N, K, device=dev), torch.empty(N, device=dev)
        ob.linear_backward(dy, x, w, dx=dx, dw=dw, dbias=db, activation=act, pre=pre,
                           ws=workspace(M, N, K, True, dev))

        def value(t):
            out = ref.linear(h64(x) + t * h64(ux), h64(w) + t * h64(uw), h64(b) + t, act)[0]
            return (h64(dy) * out).sum()

        want = (value(step) - value(-step)) / (2 * step)
        parts = (h64(dx) * h64(ux), h64(dw) * h64(uw), h64(db))
        # roundings of pre, dz and dx, each off by at most 2^-8 of what it rounds
        size = sum(np.abs(p).sum() for p in parts)
        assert abs(sum(p.sum() for p in parts) - want) < 3 * 2.0 ** -8 * size, act
