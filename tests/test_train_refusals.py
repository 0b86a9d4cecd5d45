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


def test_dropout_refuses_rows_over_rows(lib):
    """In place and between the rows is allowed (the address of the device step,
    which is checked next and not aligned here, stops those calls), crossing
    rows are not."""
    def call(y, ly, x=P, lx=32, r=None, lr=32, rows=4, cols=10, sd=P + 2):
        return lib.dropout_apply(x, r, y, 0, rows, cols, lx, lr, ly, 0.1, 1, 1, sd, 0, None)

    for y, ly in ((P, 40), (P + 4, 32), (P + 4 * 32, 32), (P + 4 * 95, 32), (P + 4 * 9, 32),
                  (P + 4 * 23, 32), (P - 4, 32), (P - 4 * 23, 32), (P - 4 * 96, 32)):
        assert call(y, ly) == ob.ONEBIT_E_ARG, (y - P, ly)
        assert call(y, ly, x=4 * P, r=P) == ob.ONEBIT_E_ARG, (y - P, ly)
    for y, ly in ((P, 32), (P + 4 * 10, 32), (P + 4 * 22, 32), (P - 4 * 10, 32), (P + 4 * 106, 32),
                  (P - 4 * 106, 32), (P + 4 * (96 + 23), 32), (P - 4 * 128, 32)):
        assert call(y, ly) == ob.ONEBIT_E_ALIGN, (y - P, ly)
    # strides and rows whose product passes 64 bits
    far = dict(lx=1 << 40, ly=1 << 40, rows=1 << 29)
    assert call(P + 4 * 9, **far) == call(P + 4 * ((1 << 40) - 9), **far) == ob.ONEBIT_E_ARG
    assert call(P + 4 * 10, **far) == call(P + 4 * ((1 << 40) - 10), **far) == ob.ONEBIT_E_ALIGN
    assert call(P, 40, rows=1) == ob.ONEBIT_E_ALIGN


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


@pytest.mark.parametrize("B", [(1 << 30) - 1, (1 << 30) + 1, (1 << 31) - 1])
def test_rel_bias_grad_of_the_most_sequences(lib, B):
    """Sequences past 2^30 (2^30 + 1 scores of one query and key are 2 GiB): the
    plan's numbers stay positive, its workspace takes less than the scores, and
    a call without that workspace is refused."""
    for Tq, Tk in ((1, 1), (3, 1), (70, 9)):
        n = ob.rel_bias_workspace_bytes(B, 1, Tq, Tk, 16)
        assert 33 * 4 <= n < 2 * B * Tq * Tk
        for dt in (0, 1, 2):
            assert lib.rel_bias_grad(P, dt, P, P, B, 1, 8, 16, Tq, Tk, 0, 0, P, n - 256,
                                     None) == ob.ONEBIT_E_WORKSPACE


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


def _args(**kw):
    a = ob.RelAttentionArgs(dtype=1, B=1, H=4, Hkv=2, Tq=8, Tk=8, D=64, scale=0.125, q=P, k=P, v=P,
                            o=P, lse=P, d_o=P, dq=P, dk=P, dv=P)
    for n, heads in (("q", 4), ("k", 2), ("v", 2), ("o", 4), ("do", 4), ("dq", 4), ("dk", 2),
                     ("dv", 2)):
        setattr(a, n + "_stride", (8 * heads * 64, heads * 64, 64))
    for n, x in kw.items():
        setattr(a, n, x)
    return a


def test_attention_refusals(lib):
    import ctypes

    def both(ws=P, wsb=1 << 30, **kw):
        a = _args(**kw)
        f = lib.rel_attention_forward(ctypes.byref(a), ws, wsb, None)
        b = lib.rel_attention_backward(ctypes.byref(a), ws, wsb, None)
        assert f == b, (kw, f, b)
        return f

    assert lib.rel_attention_forward(None, P, 1, None) == ob.ONEBIT_E_NULL
    assert lib.rel_attention_backward(None, P, 1, None) == ob.ONEBIT_E_NULL
    for bad in (dict(dtype=0), dict(dtype=3), dict(p=1.0), dict(p=-1.0), dict(p=NAN),
                dict(scale=NAN), dict(scale=float("inf")), dict(scale=0.0), dict(scale=-0.1),
                dict(scale=2.0 ** -65), dict(scale=2.0 ** 65), dict(causal=2), dict(q_pos=1 << 30),
                dict(q_pos=-(1 << 30))):
        assert both(**bad) == ob.ONEBIT_E_ARG, bad
    for bad in (dict(B=-1), dict(H=0), dict(H=5), dict(Hkv=0), dict(Hkv=3), dict(Tq=-1),
                dict(Tk=(1 << 29) + 1), dict(D=0), dict(D=12), dict(D=136), dict(radius=-1),
                dict(radius=1025, n_buckets=4, table=P, map=P),
                dict(radius=8, n_buckets=0, table=P, map=P), dict(B=1 << 30, H=8, Hkv=8),
                dict(q_stride=(2048, 252, 64)), dict(k_stride=(1024, -128, 64)),
                dict(v_stride=(1 << 41, 128, 64)), dict(k_stride=(1 << 30, (1 << 23) + 8, 64)),
                dict(o_stride=(2048, 0, 64)), dict(o_stride=(2048, 256, 32)),
                dict(o_stride=(2048, 64, 64)), dict(o_stride=(2048, 248, 64)),
                dict(B=2, o_stride=(1024, 256, 64)), dict(B=2, o_stride=(128, 256, 64)),
                dict(B=1 << 24, o_stride=(1 << 40, 256, 64))):
        assert both(**bad) == ob.ONEBIT_E_SIZE, bad
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(table=P),
                dict(map=P, table=None), dict(radius=8, n_buckets=4)):
        assert both(**bad) == ob.ONEBIT_E_NULL, bad
    for bad in (dict(q=P + 8), dict(k=P + 2), dict(v=P + 4), dict(o=P + 8), dict(lse=P + 2),
                dict(k_len=P + 1), dict(q_pos_of=P + 2), dict(step_dev=P + 1),
                dict(table=P + 1, map=P, radius=4, n_buckets=4)):
        assert both(**bad) == ob.ONEBIT_E_ALIGN, bad

    def bwd(ws=P, wsb=1 << 30, **kw):
        return lib.rel_attention_backward(ctypes.byref(_args(**kw)), ws, wsb, None)

    for n in ("d_o", "dq", "dk", "dv", "lse"):
        assert bwd(**{n: None}) == ob.ONEBIT_E_NULL, n
    for n in ("d_o", "dq", "dk", "dv"):
        assert bwd(**{n: P + 8}) == ob.ONEBIT_E_ALIGN, n
    assert bwd(dk_stride=(1024, 0, 64)) == ob.ONEBIT_E_SIZE
    assert bwd(dtable=P) == ob.ONEBIT_E_ARG
    assert bwd(accumulate=2) == ob.ONEBIT_E_ARG
    assert bwd(table=P, map=P, radius=4, n_buckets=4, dtable=P + 2) == ob.ONEBIT_E_ALIGN
    assert bwd(ws=None) == bwd(wsb=8) == ob.ONEBIT_E_WORKSPACE
    assert bwd(ws=P + 64) == ob.ONEBIT_E_ALIGN
    # outputs of other orders: heads outermost, sequences inmost, gaps
    for order in ((2048, 64, 512), (64, 512, 128), (4096, 512, 72)):
        assert bwd(B=2, o_stride=order, dq_stride=order, ws=None) == ob.ONEBIT_E_WORKSPACE, order
    # few rows over many keys: the forward call needs its workspace too
    a = _args(Tq=1, Tk=1 << 14)
    assert lib.rel_attention_forward(ctypes.byref(a), None, 0, None) == ob.ONEBIT_E_WORKSPACE
    assert lib.rel_attention_forward(ctypes.byref(_args(Tq=0, q=None, o=None)), None, 0,
                                     None) == ob.ONEBIT_OK


def test_attention_refuses_outputs_over_its_tensors(lib):
    import ctypes

    apart = dict(q=P, k=2 * P, v=3 * P, o=4 * P, d_o=5 * P, dq=6 * P, dk=7 * P, dv=8 * P)

    def fwd(**kw):
        a = _args(**{**apart, **kw})
        return lib.rel_attention_forward(ctypes.byref(a), 16 * P, 1 << 30, None)

    def bwd(**kw):
        a = _args(**{**apart, **kw})
        return lib.rel_attention_backward(ctypes.byref(a), 16 * P, 1 << 30, None)

    for n in "qkv":
        assert fwd(o=apart[n]) == ob.ONEBIT_E_ARG
    for out, n in (("dq", 5), ("dk", 6), ("dv", 7)):
        for other in list(apart)[:n]:
            assert bwd(**{out: apart[other]}) == ob.ONEBIT_E_ARG, (out, other)


def test_attention_workspace(lib):
    f = ob.rel_attention_workspace_bytes
    assert f(1, 4, 2, 8, 8, 64) == 256
    assert f(1, 4, 2, 8, 8, 64, backward=True) == 256
    assert f(1, 4, 2, 1, 1 << 14, 64) > 256
    assert f(1, 4, 2, 8, 8, 64, radius=16, backward=True) > f(1, 4, 2, 8, 8, 64, backward=True)
    assert f(1, 4, 3, 8, 8, 64) == f(1, 4, 2, 8, 8, 65) == f(-1, 4, 2, 8, 8, 64) == 0
    assert f(0, 4, 2, 0, 8, 64) == 256


def test_attention_struct_matches_header():
    """Offsets that the C declaration implies (LP64)."""
    import ctypes

    A = ob.RelAttentionArgs
    assert A.seed.offset == 56 and A.step_dev.offset == 64 and A.table.offset == 88
    assert A.q.offset == 104 and A.lse.offset == 136 and A.q_stride.offset == 144
    assert A.d_o.offset == 240 and A.do_stride.offset == 272 and A.dtable.offset == 368
    assert A.accumulate.offset == 376 and ctypes.sizeof(A) == 384


def test_attention_binding_refuses(monkeypatch):
    monkeypatch.setattr(ob, "_on_gpu", lambda t: True)
    q = torch.zeros((1, 4, 2, 16), dtype=torch.bfloat16)
    f = ob.rel_attention_forward
    with pytest.raises(ValueError, match="bfloat16 or float16"):
        f(q.float(), q.float(), q.float(), q.float())
    with pytest.raises(ValueError, match="shape"):
        f(q, q, q[:, :3], q)
    with pytest.raises(ValueError, match="must be bfloat16"):
        f(q, q.half(), q, q)
    with pytest.raises(ValueError, match="side by side"):
        f(q, q, q, torch.zeros((1, 4, 2, 32), dtype=torch.bfloat16)[..., ::2])
    with pytest.raises(ValueError, match="its bucket map"):
        f(q, q, q, q, table=torch.zeros(4, 2))
    with pytest.raises(ValueError, match="heads"):
        f(q, q, q, q, table=torch.zeros(4, 3), bucket_map=torch.zeros(9, dtype=torch.int32))
    with pytest.raises(ValueError, match="needs"):
        f(q, q, q, q, lse=torch.zeros(7))
    with pytest.raises(ValueError, match="int32"):
        f(q, q, q, q, k_len=torch.zeros(1, dtype=torch.int64))
    t, m = torch.zeros(4, 2), torch.zeros(9, dtype=torch.int32)
    with pytest.raises(ValueError, match="dtable has shape"):
        ob.rel_attention_backward(q, q, q, q, torch.zeros(1, 2, 4), q, q, q, q, table=t,
                                  bucket_map=m, dtable=torch.zeros(2, 4))


def test_binding_refuses_numbers_past_32_bits(monkeypatch):
    monkeypatch.setattr(ob, "_on_gpu", lambda t: True)
    q = torch.zeros((1, 4, 2, 16), dtype=torch.bfloat16)
    t, m = torch.zeros(4, 2), torch.zeros(9, dtype=torch.int32)
    for far in (1 << 31, 1 << 32, -(1 << 31) - 1):
        with pytest.raises(ValueError, match="32 bits"):
            ob.rel_attention_forward(q, q, q, q, q_pos=far)
        with pytest.raises(ValueError, match="32 bits"):
            ob.rel_bias_expand(t, m, torch.zeros(2, 3, 3), q_pos=far)
        with pytest.raises(ValueError, match="32 bits"):
            ob.rel_bias_grad(torch.zeros(1, 2, 3, 3), m, t, q_pos=far)
        with pytest.raises(ValueError, match="32 bits"):
            ob.rel_bias_workspace_bytes(1, 2, 3, far, 4)
        with pytest.raises(ValueError, match="32 bits"):
            ob.rel_attention_workspace_bytes(1, 2, 2, 3, far, 64)


def test_binding_refuses_tensors_of_another_device(monkeypatch):
    """Host tensors stand for another device's."""
    monkeypatch.setattr(ob, "_on_gpu", lambda t: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    q = torch.zeros((1, 4, 2, 16), dtype=torch.bfloat16)
    t, m = torch.zeros(4, 2), torch.zeros(9, dtype=torch.int32)
    ws = torch.zeros(256, dtype=torch.uint8)
    for call in (lambda: ob.dropout_apply(q, q, 4, 32, 0.1, 1, 2),
                 lambda: ob.rel_bias_expand(t, m, torch.zeros(2, 3, 3)),
                 lambda: ob.rel_bias_grad(torch.zeros(1, 2, 3, 3), m, t, ws=ws),
                 lambda: ob.rel_attention_forward(q, q, q, q),
                 lambda: ob.rel_attention_backward(q, q, q, q, torch.zeros(1, 2, 4), q, q, q, q)):
        with pytest.raises(ValueError, match="current device"):
            call()


def test_attention_packing_matches_the_struct():
    """The binding packs the struct's fields in one go; each lands where the
    declaration has it."""
    import ctypes

    n = 11 + 2 + 1 + 1 + 10 + 12 + 4 + 12 + 1 + 1
    packed = ob._ATTENTION.pack(*range(1, n + 1))
    assert len(packed) == ctypes.sizeof(ob.RelAttentionArgs)
    a = ob.RelAttentionArgs.from_buffer_copy(packed)
    got = []
    for name, kind in a._fields_:
        x = getattr(a, name)
        got += list(x) if kind is ctypes.c_int64 * 3 else [x]
    assert [float(x) for x in got] == [float(x) for x in range(1, n + 1)]
