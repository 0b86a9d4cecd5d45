"""layer_norm_forward and layer_norm_backward against the 64-bit forms, within
bounds that count their roundings."""

import numpy as np
import pytest
import torch

from momentum_compression_amd import onebit as ob
from oracle import block as ref
from tests._gpu import device, gen

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E = 2.0 ** -24
# every number of lanes a row has, its edges, rows that stay in registers and not
COLS = [1, 3, 8, 9, 31, 33, 127, 130, 512, 513, 1003, 1025, 2048, 2051, 4096, 4099, 8200, 16384,
        16385, 40007]


def h64(t):
    return None if t is None else t.double().cpu().numpy()


def adds(cols):
    """Additions that one column's value passes on its way into a row's sum."""
    return 96 + cols / 1024


def close(got, want, tol, name):
    got = h64(got)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (f"{name}: {bad.sum()} of {bad.size}, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]} for {want[bad][0]} +- {tol[bad][0]}")


def half(t):
    return torch.finfo(t).eps / 2 * 1.001


def least(t):
    return 2.0 ** -25 if t == torch.float16 else 2.0 ** -140


def check_forward(x, y, w, b, eps, mean, rstd, name):
    X, W = h64(x), np.ones(x.shape[1]) if w is None else h64(w)
    Bv = np.zeros(x.shape[1]) if b is None else h64(b)
    want, m, r = ref.layer_norm(X, W, Bv, eps)
    a = adds(x.shape[1])
    # deviations from a mean that is off by the roundings of its sum; what it is
    # off comes off again, to the roundings of a second sum
    D = np.abs(X - m[:, None]) + a * E * np.abs(X).mean(1, keepdims=True)
    t_mean = (a + 4) * E * D.mean(1, keepdims=True)
    t_var = (a + 8) * E * (D * D).mean(1, keepdims=True)
    rel = 0.5 * t_var * r[:, None] ** 2 + 4 * E
    t = np.abs(W) * r[:, None] * (D * (rel + 4 * E) + t_mean) + 2 * E * (np.abs(Bv) + np.abs(want))
    close(y, want, t + half(y.dtype) * (np.abs(want) + t) + least(y.dtype), f"{name} y")
    if mean is not None:
        close(mean, m, (t_mean + 3 * E * np.abs(m)[:, None])[:, 0], f"{name} mean")
    if rstd is not None:
        close(rstd, r, (rel * 1.01 * r[:, None])[:, 0], f"{name} rstd")


def check_backward(dy, x, mean, rstd, w, dx, dw, db, name, before=(0.0, 0.0)):
    G, X, M, R = h64(dy), h64(x), h64(mean), h64(rstd)
    rows, cols = X.shape
    W = np.ones(cols) if w is None else h64(w)
    want, wdw, wdb = ref.layer_norm_grad(G, X, M, R, W)
    h, u = (X - M[:, None]) * R[:, None], G * W
    a = adds(cols)
    mu, muh = np.abs(u).mean(1, keepdims=True), np.abs(u * h).mean(1, keepdims=True)
    if dx is not None:
        t = R[:, None] * (4 * E * np.abs(u) + (a + 6) * E * mu + (a + 10) * E * np.abs(h) * muh)
        t += 4 * E * np.abs(want)
        close(dx, want, t + half(dx.dtype) * (np.abs(want) + t) + least(dx.dtype), f"{name} dx")
    # a column's sum over rows: a lane's rows, the lanes' sums, then binary64
    n = min(rows, rows / 64 + 300) + 6
    if dw is not None:
        wdw = wdw + before[0]
        close(dw, wdw, n * E * np.abs(G * h).sum(0) + 2 * E * np.abs(wdw) + 1e-30, f"{name} dweight")
    if db is not None:
        wdb = wdb + before[1]
        close(db, wdb, n * E * np.abs(G).sum(0) + 2 * E * np.abs(wdb) + 1e-30, f"{name} dbias")


def workspace(rows, cols, dev):
    n = ob.layer_norm_workspace_bytes(rows, cols)
    assert n > 0
    return torch.full((n,), 0xFF, dtype=torch.uint8, device=dev)  # NaN where it is read


def both(x, dy, w, b, name, eps=1e-5):
    rows, cols = x.shape
    dev = x.device
    y, dx = torch.empty(rows, cols, dtype=x.dtype, device=dev), torch.empty_like(dy)
    mean, rstd = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
    ob.layer_norm_forward(x, y, rows, cols, eps, weight=w, bias=b, mean=mean, rstd=rstd)
    check_forward(x, y, w, b, eps, mean, rstd, name)
    dw, db = torch.empty(cols, device=dev), torch.empty(cols, device=dev)
    ob.layer_norm_backward(dy, x, mean, rstd, rows, cols, dx=dx, weight=w, dweight=dw, dbias=db,
                           ws=workspace(rows, cols, dev))
    check_backward(dy, x, mean, rstd, w, dx, dw, db, name)
    return y, mean, rstd, dx, dw, db


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", COLS)
def test_rows_of_every_length(dtype, cols):
    dev, t = device(), TYPES[dtype]
    g = gen(cols, dev)
    for rows, wide in ((1, True), (7, False), (70 if cols > 3000 else 1100, True)):
        print(f"[norm] {dtype} {rows}x{cols}", flush=True)
        x = (torch.randn((rows, cols), generator=g, device=dev) * 2 + 0.5).to(t)
        dy = torch.randn((rows, cols), generator=g, device=dev).to(t)
        wt = torch.float32 if wide else t
        w = (1 + 0.2 * torch.randn(cols, generator=g, device=dev)).to(wt)
        b = torch.randn(cols, generator=g, device=dev).to(wt)
        both(x, dy, w, b, f"{rows}x{cols}")


@pytest.mark.parametrize("dtype", TYPES)
def test_views_and_what_lies_between(dtype):
    """Rows further apart than they are long, at odd element offsets; what lies
    between them stays; parameters and outputs that are left out."""
    dev, t = device(), TYPES[dtype]
    rows, cols = 45, 77
    g = gen(3, dev)
    x = torch.randn((rows, cols + 9), generator=g, device=dev).to(t)[:, 3:3 + cols]
    dy = torch.randn((rows, cols + 2), generator=g, device=dev).to(t)[:, 1:1 + cols]
    yy = torch.full((rows, cols + 6), 7.0, device=dev, dtype=t)
    dd = torch.full((rows, cols + 5), 7.0, device=dev, dtype=t)
    y, dx = yy[:, 5:5 + cols], dd[:, 2:2 + cols]
    b = torch.randn(cols, generator=g, device=dev)
    mean, rstd = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
    ob.layer_norm_forward(x, y, rows, cols, 1e-3, bias=b, mean=mean, rstd=rstd)
    check_forward(x, y, None, b, 1e-3, mean, rstd, "view")
    dw = torch.full((cols,), 2.0, device=dev)
    ob.layer_norm_backward(dy, x, mean, rstd, rows, cols, dx=dx, dweight=dw, accumulate=True,
                           ws=workspace(rows, cols, dev))
    check_backward(dy, x, mean, rstd, None, dx, dw, None, "view", before=(2.0, 0.0))
    for whole, at in ((yy, 5), (dd, 2)):
        assert bool((whole[:, :at] == 7).all()) and bool((whole[:, at + cols:] == 7).all())
    # without weights' gradients no workspace, without dx no dx
    again = torch.empty(rows, cols, dtype=t, device=dev)
    ob.layer_norm_backward(dy, x, mean, rstd, rows, cols, dx=again)
    assert torch.equal(again, dx)
    db = torch.empty(cols, device=dev)
    ob.layer_norm_backward(dy, x, mean, rstd, rows, cols, dbias=db, ws=workspace(rows, cols, dev))
    check_backward(dy, x, mean, rstd, None, None, None, db, "dbias alone")


@pytest.mark.parametrize("cols", [1000, 20001])
def test_in_place(cols):
    """y over x, dx over x and dx over dy are what they are elsewhere."""
    dev, rows = device(), 33
    g = gen(5, dev)
    x = torch.randn((rows, cols), generator=g, device=dev)
    dy = torch.randn((rows, cols), generator=g, device=dev)
    w = torch.randn(cols, generator=g, device=dev)
    y, mean, rstd, dx, dw, _ = both(x, dy, w, None, "apart")
    z = x.clone()
    ob.layer_norm_forward(z, z, rows, cols, 1e-5, weight=w)
    assert torch.equal(z, y)
    for over in ("x", "dy"):
        a = {"x": x.clone(), "dy": dy.clone()}
        dw2 = torch.empty_like(dw)
        ob.layer_norm_backward(a["dy"], a["x"], mean, rstd, rows, cols, dx=a[over], weight=w,
                               dweight=dw2, ws=workspace(rows, cols, dev))
        assert torch.equal(a[over], dx) and torch.equal(dw2, dw), over


@pytest.mark.parametrize("cols", [5, 600, 30000])
def test_offsets_constants_and_what_is_no_number(cols):
    """A common offset of 10^4 leaves the deviations' precision; a constant row
    has y = bias; a row with a NaN or an infinity is NaN and its neighbours are
    not."""
    dev, rows = device(), 9
    g = gen(cols, dev)
    x = torch.randn((rows, cols), generator=g, device=dev) + 1e4
    x[2] = 3.25
    b = torch.randn(cols, generator=g, device=dev)
    y = torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
    ob.layer_norm_forward(x, y, rows, cols, 1e-5, bias=b, mean=mean, rstd=rstd)
    check_forward(x, y, None, b, 1e-5, mean, rstd, "offset")
    assert torch.equal(y[2], b)
    clean = y.clone()
    x[1, cols // 2] = float("nan")
    x[4, cols - 1] = float("inf")
    ob.layer_norm_forward(x, y, rows, cols, 1e-5, bias=b)
    assert bool(y[[1, 4]].isnan().all())
    keep = [0, 2, 3, 5, 6, 7, 8]
    assert torch.equal(y[keep], clean[keep])


def test_no_rows():
    dev = device()
    for cols in (40, 20000):
        x = torch.empty((0, cols), device=dev)
        s = torch.empty(0, device=dev)
        dw = torch.full((cols,), 3.0, device=dev)
        db = torch.full((cols,), 3.0, device=dev)
        how = dict(dweight=dw, dbias=db, ws=workspace(0, cols, dev))
        ob.layer_norm_forward(x, x, 0, cols, 1e-5)
        ob.layer_norm_backward(x, x, s, s, 0, cols, accumulate=True, **how)
        assert bool((dw == 3).all()) and bool((db == 3).all())
        ob.layer_norm_backward(x, x, s, s, 0, cols, **how)
        assert bool((dw == 0).all()) and bool((db == 0).all())


def test_many_rows_and_the_same_bits_again():
    """Sums over many rows, twice the same bits, also on another stream."""
    dev = device()
    for rows, cols, t in ((100_003, 9, torch.float32), (20_001, 260, torch.bfloat16)):
        g = gen(rows, dev)
        x = torch.randn((rows, cols), generator=g, device=dev).to(t)
        dy = (torch.randn((rows, cols), generator=g, device=dev) + 0.3).to(t)
        _, mean, rstd, dx, dw, db = both(x, dy, None, None, f"{rows}x{cols}")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        dx2, dw2, db2 = (torch.empty_like(a) for a in (dx, dw, db))
        with torch.cuda.stream(side):
            ws = workspace(rows, cols, dev)
            ob.layer_norm_backward(dy, x, mean, rstd, rows, cols, dx=dx2, dweight=dw2, dbias=db2,
                                   ws=ws)
        side.synchronize()
        for a, b in ((dx, dx2), (dw, dw2), (db, db2)):
            assert torch.equal(a, b)


def test_gradient_against_differences():
    """The backward call's dx and dweight against differences of the forward
    form, in a direction."""
    dev = device()
    rows, cols, step = 4, 50, 1e-4
    g = gen(2, dev)
    x, dy, ux = (torch.randn((rows, cols), generator=g, device=dev) for _ in range(3))
    w, uw = (torch.randn(cols, generator=g, device=dev) for _ in range(2))
    _, _, _, dx, dw, _ = both(x, dy, w, None, "differences")

    def value(t):
        y = ref.layer_norm(h64(x) + t * h64(ux), h64(w) + t * h64(uw), 0.0, 1e-5)[0]
        return (h64(dy) * y).sum()

    slope = (value(step) - value(-step)) / (2 * step)
    mine = (h64(dx) * h64(ux)).sum() + (h64(dw) * h64(uw)).sum()
    # the difference's own error is step^2 times a third derivative of order one
    size = np.abs(h64(dx) * h64(ux)).sum() + np.abs(h64(dw) * h64(uw)).sum()
    assert abs(slope - mine) < 2e-6 * size
