"""dropout_apply against the 64-bit form: the mask exactly, values within the
roundings of one scaled product, one sum and one store."""

import numpy as np
import pytest
import torch

from momentum_compression_amd import onebit as ob
from oracle import training as ref
from tests._gpu import device, gen

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SEED = 0x1234_5678_9ABC_DEF1


def _check(y, x, r, p, seed, step, row0, name):
    """k = x * (65536 / T): the scale and the product round once each; the sum
    once; the store once to its type.  Values here stay in the normal range."""
    y64, x64 = y.double().cpu().numpy(), x.double().cpu().numpy()
    want = ref.dropout(x64, p, seed, step, row0)
    k = np.abs(want)
    res = 0.0 if r is None else r.double().cpu().numpy()
    want = want + res
    half = torch.finfo(y.dtype).eps / 2
    tol = (2 * 2.0 ** -24) * k + (2.0 ** -24 + half) * 1.001 * np.abs(want) + 2.0 ** -25
    bad = ~(np.abs(y64 - want) <= tol)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size}, first at {np.argwhere(bad)[0]}"
    if r is None:
        kept = ref.keep_factor(*x64.shape, p, seed, step, row0) > 0
        assert np.array_equal(y64 != 0, kept & (x64 != 0)), f"{name}: mask"


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (1, 8), (3, 9), (5, 1000), (64, 64),
                                       (129, 513), (1000, 1), (2, 40001)])
def test_values_and_mask(dtype, rows, cols):
    dev = device()
    g = gen(rows * 1000 + cols, dev)
    for residual in (False, True):
        for p, row0 in ((0.1, 0), (0.0, 3), (0.5, 2 ** 33 + 5), (0.999, 0)):
            print(f"[dropout] {dtype} {rows}x{cols} residual={residual} p={p}", flush=True)
            x = (torch.randn((rows, cols), generator=g, device=dev).abs() + 0.5).to(TYPES[dtype])
            r = torch.randn((rows, cols), generator=g, device=dev).to(TYPES[dtype])
            r = r if residual else None
            y = torch.empty_like(x)
            ob.dropout_apply(x, y, rows, cols, p, SEED, 9, residual=r, row0=row0)
            _check(y, x, r, p, SEED, 9, row0, f"p={p} residual={residual}")


@pytest.mark.parametrize("dtype", TYPES)
def test_strided_rows_and_neighbours(dtype):
    """Views with rows further apart than they are long, at odd element
    offsets; what lies between the rows stays."""
    dev = device()
    rows, cols = 37, 53
    g = gen(4, dev)
    x = (torch.rand((rows, cols + 11), generator=g, device=dev) + 0.5).to(TYPES[dtype])
    r = torch.randn((rows, cols + 4), generator=g, device=dev).to(TYPES[dtype])
    y = torch.full((rows, cols + 7), 7.0, device=dev, dtype=TYPES[dtype])
    xs, rs, ys = x[:, 3:3 + cols], r[:, 1:1 + cols], y[:, 5:5 + cols]
    ob.dropout_apply(xs, ys, rows, cols, 0.3, SEED, 2, residual=rs)
    _check(ys, xs, rs, 0.3, SEED, 2, 0, "strided")
    assert bool((y[:, :5] == 7).all()) and bool((y[:, 5 + cols:] == 7).all())


def test_in_place_parts_and_backward():
    """In place equals out of place; rows in two parts with their row0 equal
    the whole; the gradient call draws the forward's mask."""
    dev = device()
    rows, cols = 130, 264
    x = torch.rand((rows, cols), generator=gen(1, dev), device=dev) + 0.5
    whole = torch.empty_like(x)
    ob.dropout_apply(x, whole, rows, cols, 0.25, SEED, 7)
    z = x.clone()
    ob.dropout_apply(z, z, rows, cols, 0.25, SEED, 7)
    assert torch.equal(z, whole)
    z = x.clone()
    ob.dropout_apply(x, z, rows, cols, 0.25, SEED, 7, residual=z)
    assert torch.equal(z, x + whole)
    parts = torch.empty_like(x)
    ob.dropout_apply(x[:77], parts[:77], 77, cols, 0.25, SEED, 7)
    ob.dropout_apply(x[77:], parts[77:], rows - 77, cols, 0.25, SEED, 7, row0=77)
    assert torch.equal(parts, whole)
    dy = torch.rand((rows, cols), generator=gen(2, dev), device=dev) + 0.5
    dx = torch.empty_like(dy)
    ob.dropout_apply(dy, dx, rows, cols, 0.25, SEED, 7)
    assert torch.equal(dx != 0, whole != 0)
    # the gradient by differences of the forward map, which is linear in x
    h = torch.empty_like(x)
    ob.dropout_apply(x + dy, h, rows, cols, 0.25, SEED, 7)
    assert torch.allclose(h - whole, dx, atol=2e-6)


def test_dropped_values_are_zero_whatever_they_held():
    dev = device()
    x = torch.full((64, 80), float("nan"), device=dev)
    x[::2] = float("inf")
    y = torch.empty_like(x)
    ob.dropout_apply(x, y, 64, 80, 0.4, 3, 1)
    kept = torch.from_numpy(ref.keep_factor(64, 80, 0.4, 3, 1) > 0).to(dev)
    assert bool((y[~kept] == 0).all())
    assert torch.equal(y.isnan(), x.isnan() & kept) and torch.equal(y.isinf(), x.isinf() & kept)


def test_share_kept_and_independence_of_neighbours():
    """4 million draws: the kept share and the products of neighbouring
    decisions within six standard deviations of independent draws."""
    dev = device()
    n, p = 1 << 22, 0.1
    x = torch.ones((1 << 11, 1 << 11), device=dev)
    y = torch.empty_like(x)
    ob.dropout_apply(x, y, 1 << 11, 1 << 11, p, 99, 1)
    k = (y != 0).double()
    q = ref.threshold(p) / 65536
    assert abs(float(k.mean()) - q) < 6 * (q * (1 - q) / n) ** 0.5
    for a, b in ((k[:, 1:], k[:, :-1]), (k[1:], k[:-1]), (k[:, 8:], k[:, :-8])):
        cov = float(((a - q) * (b - q)).mean())
        assert abs(cov) < 6 * q * (1 - q) / a.numel() ** 0.5


def test_replayed_graph_takes_the_device_step():
    """A captured call draws a new mask each replay from *step_dev, equal to
    the eager call of that step."""
    dev = device()
    rows, cols = 96, 200
    x = torch.rand((rows, cols), generator=gen(5, dev), device=dev) + 0.5
    y, step = torch.empty_like(x), torch.zeros(1, dtype=torch.int32, device=dev)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        ob.dropout_apply(x, y, rows, cols, 0.2, SEED, 40, step_dev=step)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ob.dropout_apply(x, y, rows, cols, 0.2, SEED, 40, step_dev=step)
    seen = []
    for t in range(4):
        step.fill_(t)
        graph.replay()
        torch.cuda.synchronize()
        want = torch.empty_like(x)
        ob.dropout_apply(x, want, rows, cols, 0.2, SEED, 40 + t)
        torch.cuda.synchronize()
        assert torch.equal(y, want), t
        seen.append(want)
    assert not torch.equal(seen[0], seen[1])


def test_more_elements_than_32_bits_count():
    """The last rows of a tensor of 2^31 elements and more, in place, are what
    a call on them alone gives."""
    dev = device()
    rows, cols, tail = 262_147, 8200, 5
    x = torch.full((rows, cols), 1.5, dtype=torch.bfloat16, device=dev)
    want = torch.empty((tail, cols), dtype=torch.bfloat16, device=dev)
    ob.dropout_apply(x[-tail:], want, tail, cols, 0.3, SEED, 4, row0=rows - tail)
    ob.dropout_apply(x, x, rows, cols, 0.3, SEED, 4)
    assert torch.equal(x[-tail:], want)
    assert bool((want == 0).any()) and bool((want != 0).any())
