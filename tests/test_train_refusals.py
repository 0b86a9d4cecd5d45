"""The training operators' checks that need no GPU: the C ABI refuses invalid
calls with the documented status before any HIP call (the fake addresses are
never dereferenced), the binding refuses what the C ABI cannot see, and the
bucket map is the oracle's."""

import numpy as np
import pytest
import torch

from momentum_compression_amd import onebit as ob
from momentum_compression_amd.attention import rel_bucket_map
from oracle import training as ref

P = 0x10000
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    return ob.load()


def test_dropout_refusals(lib):
    def call(x=P, r=None, y=P, dt=0, rows=4, cols=10, lx=10, lr=10, ly=10, p=0.1, sd=None, row0=0):
        return lib.dropout_apply(x, r, y, dt, rows, cols, lx, lr, ly, p, 1, 1, sd, row0, None)

    assert call(dt=3) == ob.ONEBIT_E_ARG
    assert call(p=1.0) == ob.ONEBIT_E_ARG
    assert call(p=-0.1) == ob.ONEBIT_E_ARG
    assert call(p=NAN) == ob.ONEBIT_E_ARG
    assert call(rows=-1) == ob.ONEBIT_E_SIZE
    assert call(row0=-1) == ob.ONEBIT_E_SIZE
    assert call(lx=9) == ob.ONEBIT_E_SIZE
    assert call(ly=9) == ob.ONEBIT_E_SIZE
    assert call(r=P, lr=9) == ob.ONEBIT_E_SIZE
    assert call(lx=(1 << 40) + 1) == ob.ONEBIT_E_SIZE
    assert call(x=None) == ob.ONEBIT_E_NULL
    assert call(y=None) == ob.ONEBIT_E_NULL
    assert call(x=P + 2) == ob.ONEBIT_E_ALIGN
    assert call(r=P + 2) == ob.ONEBIT_E_ALIGN
    assert call(dt=1, x=P + 1) == ob.ONEBIT_E_ALIGN
    assert call(sd=P + 2) == ob.ONEBIT_E_ALIGN
    # 2^31 groups of 8 columns
    assert call(rows=1 << 28, cols=64, lx=64, ly=64) == ob.ONEBIT_E_SIZE
    assert call(rows=1 << 62, cols=1 << 30, lx=1 << 30, ly=1 << 30) == ob.ONEBIT_E_SIZE
    # nothing to do: no launch, whatever the pointers
    assert call(x=None, y=None, rows=0) == ob.ONEBIT_OK
    assert call(cols=0) == ob.ONEBIT_OK


def test_rel_bias_refusals(lib):
    def call(t=P, m=P, o=P, dt=0, H=2, nb=8, R=16, Tq=4, Tk=4, pos=0):
        return lib.rel_bias_expand(t, m, o, dt, H, nb, R, Tq, Tk, pos, None)

    assert call(dt=-1) == ob.ONEBIT_E_ARG
    assert call(pos=(1 << 29) + 1) == ob.ONEBIT_E_ARG
    assert call(pos=-(1 << 29) - 1) == ob.ONEBIT_E_ARG
    for bad in (dict(H=0), dict(H=65536), dict(nb=0), dict(nb=1025), dict(R=0), dict(R=1025),
                dict(Tq=-1), dict(Tk=-1), dict(Tk=(1 << 29) + 1),
                dict(Tq=1 << 20, Tk=1 << 15)):
        assert call(**bad) == ob.ONEBIT_E_SIZE, bad
    assert call(t=None) == call(m=None) == call(o=None) == ob.ONEBIT_E_NULL
    assert call(t=P + 2) == call(m=P + 1) == call(o=P + 2) == ob.ONEBIT_E_ALIGN
    assert call(o=None, Tq=0) == ob.ONEBIT_OK


def test_rel_bias_grad_refusals(lib):
    def call(ds=P, dt=0, m=P, d=P, B=1, H=2, nb=8, R=16, Tq=4, Tk=4, pos=0, acc=0, ws=P,
             wsb=1 << 30):
        return lib.rel_bias_grad(ds, dt, m, d, B, H, nb, R, Tq, Tk, pos, acc, ws, wsb, None)

    assert call(dt=9) == ob.ONEBIT_E_ARG
    assert call(acc=2) == ob.ONEBIT_E_ARG
    assert call(pos=1 << 30) == ob.ONEBIT_E_ARG
    for bad in (dict(B=-1), dict(H=0), dict(nb=2000), dict(R=0), dict(Tq=-4)):
        assert call(**bad) == ob.ONEBIT_E_SIZE, bad
    assert call(ds=None) == call(m=None) == call(d=None) == ob.ONEBIT_E_NULL
    assert call(ds=P + 2) == call(m=P + 2) == call(d=P + 2) == ob.ONEBIT_E_ALIGN
    assert call(ws=P + 64) == ob.ONEBIT_E_ALIGN
    assert call(ws=None) == call(wsb=16) == ob.ONEBIT_E_WORKSPACE
    # an empty ds needs no pointer, but still a workspace
    assert call(ds=None, B=0, ws=None) == ob.ONEBIT_E_WORKSPACE


def test_rel_bias_workspace(lib):
    f = ob.rel_bias_workspace_bytes
    assert f(1, 1, 32, 64, 16) == (33 * 4 + 255) // 256 * 256    # one part of one head
    assert f(0, 1, 32, 64, 16) == 256
    assert f(1, 0, 32, 64, 16) == f(1, 1, -1, 64, 16) == f(1, 1, 32, 64, 0) == 0
    for B, H, Tq, Tk in ((16, 16, 512, 512), (1, 1, 8192, 8192), (64, 32, 1, 4096)):
        assert f(B, H, Tq, Tk, 128) % (257 * 4) < 256 and f(B, H, Tq, Tk, 128) > 0


def test_binding_refuses_shapes_and_types(monkeypatch):
    monkeypatch.setattr(ob, "_on_gpu", lambda t: True)
    x = torch.zeros(4, 16)
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        ob.dropout_apply(x.double(), x, 4, 16, 0.1, 1, 1)
    with pytest.raises(ValueError, match="needs"):
        ob.dropout_apply(x, x, 5, 16, 0.1, 1, 1)
    with pytest.raises(ValueError, match="must be float32"):
        ob.dropout_apply(x, x.half(), 4, 16, 0.1, 1, 1)
    with pytest.raises(ValueError, match="shape"):
        ob.dropout_apply(torch.zeros(4, 32)[:, :20], x, 4, 16, 0.1, 1, 1)
    with pytest.raises(ValueError, match="rows"):
        ob.dropout_apply(torch.zeros(16, 4).t(), x, 4, 16, 0.1, 1, 1)
    t, m = torch.zeros(8, 2), torch.zeros(9, dtype=torch.int32)
    with pytest.raises(ValueError, match="heads"):
        ob.rel_bias_expand(t, m, torch.zeros(3, 4, 4))
    with pytest.raises(ValueError, match="2 \\* radius"):
        ob.rel_bias_expand(t, m[:8], torch.zeros(2, 4, 4))
    with pytest.raises(ValueError, match="dimensions"):
        ob.rel_bias_expand(t, m, torch.zeros(2, 16))
    with pytest.raises(ValueError, match="int32"):
        ob.rel_bias_expand(t, m.long(), torch.zeros(2, 4, 4))
    with pytest.raises(ValueError, match="heads"):
        ob.rel_bias_grad(torch.zeros(1, 3, 4, 4), m, t)


@pytest.mark.parametrize("n,far,two", [(32, 128, True), (32, 128, False), (4, 40, True),
                                       (8, 300, True), (65, 128, False), (2, 16, True),
                                       (1, 9, False), (3, 17, False), (128, 1024, True)])
def test_bucket_map_is_the_oracles(n, far, two):
    got = rel_bucket_map(n, far, two)
    assert got.dtype == torch.int32
    assert np.array_equal(got.numpy(), ref.bucket_map(n, far, two))


def test_bucket_map_borders_are_whole():
    """e = 8, n = 16, max 128: bucket 8 + k begins at 8 * 2^(k / 2), whole for
    even k, where a rounded logarithm may fall short."""
    m = rel_bucket_map(32, 128, True).tolist()
    for k, d in ((2, 16), (4, 32), (6, 64)):
        assert m[128 + d] == 16 + 8 + k and m[128 + d - 1] == 16 + 8 + k - 1
    with pytest.raises(ValueError):
        rel_bucket_map(1, 10, True)
    with pytest.raises(ValueError):
        rel_bucket_map(32, 16, False)
