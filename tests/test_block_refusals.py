"""The checks of layer norm, the linear layer and AdamW that need no GPU: the C ABI
refuses invalid calls with the documented status before any HIP call (the fake
addresses are never dereferenced), the binding refuses what the C ABI cannot see,
the argument structs are mirrored, and the plan is what the kernel reads."""

import ctypes
import os
import shutil
import struct
import subprocess

import pytest
import torch

from momentum_compression_amd import build as B
from momentum_compression_amd import onebit as ob
from momentum_compression_amd.state import AdamW

P = 0x100000
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    return ob.load()


# ---------------------------------------------------------------- layer norm
def _norm(lib, x=P, y=4 * P, dt=0, rows=4, cols=10, lx=10, ly=10, w=None, b=None, wdt=0, eps=1e-5,
          mean=None, rstd=None):
    return lib.layer_norm_forward(x, y, dt, rows, cols, lx, ly, w, b, wdt, eps, mean, rstd, None)


def test_layer_norm_refusals(lib):
    assert _norm(lib, dt=3) == _norm(lib, dt=1, wdt=2) == _norm(lib, wdt=-1) == ob.ONEBIT_E_ARG
    for eps in (-1e-9, NAN, INF):
        assert _norm(lib, eps=eps) == ob.ONEBIT_E_ARG
    for bad in (dict(rows=-1), dict(cols=-1), dict(lx=9), dict(ly=9), dict(lx=(1 << 40) + 1),
                dict(cols=(1 << 29) + 1, lx=1 << 30, ly=1 << 30)):
        assert _norm(lib, **bad) == ob.ONEBIT_E_SIZE, bad
    assert _norm(lib, x=None) == _norm(lib, y=None) == ob.ONEBIT_E_NULL
    for bad in (dict(x=P + 2), dict(y=P + 2), dict(w=P + 2), dict(b=P + 1), dict(mean=P + 2),
                dict(rstd=P + 2), dict(dt=1, x=P + 1)):
        assert _norm(lib, **bad) == ob.ONEBIT_E_ALIGN, bad
    # rows over rows, and outputs at one address
    for bad in (dict(y=P, ly=11), dict(y=P + 4), dict(y=P - 8, lx=32, ly=32), dict(w=4 * P),
                dict(mean=P), dict(mean=8 * P, rstd=8 * P), dict(rstd=4 * P)):
        assert _norm(lib, **bad) == ob.ONEBIT_E_ARG, bad
    assert _norm(lib, x=None, y=None, rows=0) == _norm(lib, x=None, cols=0) == ob.ONEBIT_OK


def _norm_grad(lib, dy=P, x=2 * P, mean=3 * P, rstd=4 * P, dx=5 * P, dt=0, rows=4, cols=10, lg=10,
               lx=10, ld=10, w=None, wdt=0, dw=6 * P, db=7 * P, acc=0, ws=8 * P, wsb=1 << 30):
    return lib.layer_norm_backward(dy, x, mean, rstd, dx, dt, rows, cols, lg, lx, ld, w, wdt, dw, db,
                                   acc, ws, wsb, None)


def test_layer_norm_backward_refusals(lib):
    assert _norm_grad(lib, dt=7) == _norm_grad(lib, acc=2) == ob.ONEBIT_E_ARG
    for bad in (dict(rows=-1), dict(lg=9), dict(lx=9), dict(ld=9)):
        assert _norm_grad(lib, **bad) == ob.ONEBIT_E_SIZE, bad
    for name in ("dy", "x", "mean", "rstd"):
        assert _norm_grad(lib, **{name: None}) == ob.ONEBIT_E_NULL, name
        assert _norm_grad(lib, **{name: P + 2}) == ob.ONEBIT_E_ALIGN, name
    for name in ("dx", "w", "dw", "db"):
        assert _norm_grad(lib, **{name: P + 2}) == ob.ONEBIT_E_ALIGN, name
    for bad in (dict(dx=2 * P, ld=12), dict(dx=P + 8), dict(dx=3 * P), dict(dw=P), dict(db=2 * P),
                dict(dw=7 * P), dict(dw=5 * P), dict(db=4 * P), dict(w=6 * P)):
        assert _norm_grad(lib, **bad) == ob.ONEBIT_E_ARG, bad
    assert _norm_grad(lib, ws=None) == _norm_grad(lib, wsb=64) == ob.ONEBIT_E_WORKSPACE
    assert _norm_grad(lib, ws=P + 64) == ob.ONEBIT_E_ALIGN
    # nothing to compute
    none = dict(dw=None, db=None, ws=None, wsb=0)
    assert _norm_grad(lib, dx=None, **none) == _norm_grad(lib, rows=0, **none) == ob.ONEBIT_OK
    assert _norm_grad(lib, cols=0) == ob.ONEBIT_OK


def test_layer_norm_partial_overlaps(lib):
    """Outputs that start inside another argument, or that another starts inside."""
    # x: 4 rows of 40 bytes from P on
    for bad in (dict(mean=P + 156), dict(mean=P - 12), dict(rstd=P + 40), dict(w=4 * P + 8),
                dict(b=4 * P + 156), dict(mean=8 * P, rstd=8 * P + 12),
                dict(mean=8 * P, w=8 * P - 36), dict(y=P + 156), dict(y=P - 156)):
        assert _norm(lib, **bad) == ob.ONEBIT_E_ARG, bad
    # dw, db: 40 bytes from 6 P and 7 P on
    for bad in (dict(db=6 * P + 36), dict(db=6 * P - 36), dict(dw=5 * P + 156), dict(dw=3 * P + 12),
                dict(dx=3 * P - 156), dict(w=7 * P + 20), dict(dx=P + 156)):
        assert _norm_grad(lib, **bad) == ob.ONEBIT_E_ARG, bad


def test_layer_norm_workspace():
    f = ob.layer_norm_workspace_bytes
    assert f(0, 100) == 256 and f(-1, 100) == f(10, -1) == 0
    assert f(1, 100) == 1024                        # one workgroup's two sums of 100 columns
    assert f(10 ** 6, 1024) == 512 * 2 * 1024 * 4   # the most workgroups that are joined
    assert f(10, 100000) == 10 * 2 * 100000 * 4


# ---------------------------------------------------------------- linear layer
def _linear_args(**kw):
    a = ob.LinearArgs(dtype=1, activation=0, M=100, N=16, K=24, x=P, w=2 * P, ld_x=24, ld_w=24,
                      y=3 * P, ld_y=16, dy=4 * P, ld_dy=16, dx=5 * P, ld_dx=24, dw=6 * P, ld_dw=24,
                      dw_dtype=0, dbias=7 * P)
    for k, v in kw.items():
        setattr(a, k, v)
    return ctypes.byref(a)


def test_linear_refusals(lib):
    def f(ws=9 * P, wsb=1 << 30, **kw):
        return lib.linear_forward(_linear_args(**kw), ws, wsb, None)

    assert lib.linear_forward(None, P, 1 << 30, None) == ob.ONEBIT_E_NULL
    for bad in (dict(dtype=0), dict(dtype=3), dict(activation=-1), dict(activation=5),
                dict(bias=8 * P, bias_dtype=2)):
        assert f(**bad) == ob.ONEBIT_E_ARG, bad
    for bad in (dict(M=-1), dict(N=-1), dict(K=-1), dict(M=1 << 31), dict(N=(1 << 22) + 1),
                dict(K=(1 << 22) + 1), dict(M=1 << 30, N=1 << 10), dict(ld_x=23), dict(ld_w=23),
                dict(ld_y=15), dict(pre=8 * P, ld_pre=15), dict(residual=8 * P, ld_residual=3),
                dict(ld_x=(1 << 40) + 1)):
        assert f(**bad) == ob.ONEBIT_E_SIZE, bad
    assert f(x=None) == f(w=None) == f(y=None) == ob.ONEBIT_E_NULL
    for bad in (dict(x=P + 1), dict(w=P + 1), dict(y=P + 1), dict(pre=P + 1, ld_pre=16),
                dict(residual=P + 1, ld_residual=16), dict(bias=P + 2, bias_dtype=0),
                dict(ws=P + 128)):
        assert f(**bad) == ob.ONEBIT_E_ALIGN, bad
    for bad in (dict(y=P), dict(y=2 * P + 64), dict(pre=3 * P, ld_pre=16), dict(pre=P, ld_pre=16),
                dict(residual=3 * P, ld_residual=18), dict(residual=3 * P + 16, ld_residual=16),
                dict(bias=3 * P + 8, bias_dtype=1),
                dict(residual=8 * P, ld_residual=16, pre=8 * P, ld_pre=16)):
        assert f(**bad) == ob.ONEBIT_E_ARG, bad
    assert f(ws=None) == f(wsb=64) == ob.ONEBIT_E_WORKSPACE
    assert f(M=0, x=None, y=None, ws=None) == f(N=0, w=None, y=None) == ob.ONEBIT_OK


def test_linear_backward_refusals(lib):
    def f(ws=9 * P, wsb=1 << 30, **kw):
        return lib.linear_backward(_linear_args(**kw), ws, wsb, None)

    for bad in (dict(accumulate=2), dict(dw_dtype=2), dict(dtype=0), dict(activation=9)):
        assert f(**bad) == ob.ONEBIT_E_ARG, bad
    for bad in (dict(ld_dy=15), dict(ld_dx=23), dict(ld_dw=23), dict(ld_x=20), dict(ld_w=20),
                dict(activation=2, pre=8 * P, ld_pre=15)):
        assert f(**bad) == ob.ONEBIT_E_SIZE, bad
    assert f(dy=None) == f(x=None) == f(w=None) == f(activation=2) == ob.ONEBIT_E_NULL
    for bad in (dict(dy=P + 1), dict(dx=P + 1), dict(dw=P + 2), dict(dbias=P + 2), dict(ws=P + 1)):
        assert f(**bad) == ob.ONEBIT_E_ALIGN, bad
    for bad in (dict(dx=P), dict(dx=4 * P), dict(dw=2 * P), dict(dw=5 * P + 96), dict(dbias=4 * P),
                dict(dbias=6 * P + 4), dict(dx=2 * P + 16),
                dict(activation=1, pre=5 * P, ld_pre=16)):
        assert f(**bad) == ob.ONEBIT_E_ARG, bad
    assert f(ws=None) == f(wsb=64) == ob.ONEBIT_E_WORKSPACE
    # x and w are not needed for gradients that are not asked for (the workspace,
    # which is checked last, stops these calls)
    assert f(dw=None, x=None, ws=None) == f(dx=None, w=None, ws=None) == ob.ONEBIT_E_WORKSPACE


def test_linear_outputs_between_rows(lib):
    """Rows between another matrix's rows are no overlap (the workspace, which is
    checked last, stops these calls); crossing ones are."""
    def f(y, x=P, ld=64, **kw):
        return lib.linear_forward(_linear_args(x=x, ld_x=ld, y=y, ld_y=ld, **kw), None, 0, None)

    for y in (P + 48, P + 96, P - 32, P + 48 + 128 * 7):
        assert f(y) == ob.ONEBIT_E_WORKSPACE, y - P
    for y in (P + 46, P + 98, P - 30, P + 128 * 99, P - 128 * 99, P + 46 + 128 * 7):
        assert f(y) == ob.ONEBIT_E_ARG, y - P


def test_linear_workspace():
    f = ob.linear_workspace_bytes
    assert f(-1, 8, 8) == f(8, 8, (1 << 22) + 1) == f(1 << 31, 8, 8, True) == 0
    assert f(1, 4096, 4096) == 256                  # few rows take none
    # operands laid out anew and no parts
    assert f(8192, 4096, 1024) == 2 * (8192 + 4096) * 1024
    assert f(8192, 4096, 1024, True) > 2 * (8192 * 1024 + 4096 * 1024 + 8192 * 4096)
    assert f(0, 0, 0, True) == 256


# ---------------------------------------------------------------- AdamW
def _tensors(*rows):
    table = (ob.AdamWTensor * max(1, len(rows)))()
    for e, kw in zip(table, rows):
        for k, v in dict(dict(x=P, g=2 * P, m=3 * P, v=4 * P, n=1000, lr_scale=1.0,
                              weight_decay=0.0), **kw).items():
            setattr(e, k, v)
    return table, len(rows)


def _plan(lib, rows, bits=32, g=0, c=0, short=0, plan=True):
    table, n = _tensors(*rows)
    size = lib.adamw_plan_bytes(table, n, None)
    room = (ctypes.c_uint64 * (max(size, 8) // 8 + 1))()
    st = lib.adamw_plan(table, n, bits, g, c, ctypes.addressof(room) if plan else None, size - short)
    return st, bytes(room), size


def test_adamw_plan(lib):
    tiles = ctypes.c_int64(-1)
    table, n = _tensors(dict(n=0, x=None), dict(n=2048), dict(x=8 * P, g=9 * P, m=10 * P, v=11 * P,
                                                               n=2049, lr_scale=2.0, weight_decay=.5))
    size = lib.adamw_plan_bytes(table, n, ctypes.byref(tiles))
    assert tiles.value == 3
    st, room, _ = _plan(lib, [dict(n=0, x=None), dict(n=2048),
                              dict(x=8 * P, g=9 * P, m=10 * P, v=11 * P, n=2049, lr_scale=2.0,
                                   weight_decay=.5)])
    assert st == ob.ONEBIT_OK
    entry = struct.Struct("<7Q2q2f")
    assert entry.unpack_from(room, entry.size) == (P, 2 * P, 0, 3 * P, 4 * P, 0, 0, 2048, 0, 1.0, 0.0)
    assert entry.unpack_from(room, 2 * entry.size)[7:] == (2049, 1, 2.0, 0.5)
    at = -(-3 * entry.size // 256) * 256
    assert struct.unpack_from("<3i", room, at) == (1, 2, 2) and size >= at + 12


def test_adamw_plan_refusals(lib):
    E = ob
    assert lib.adamw_plan_bytes(None, 1, None) == lib.adamw_plan_bytes(None, -1, None) == 0
    assert lib.adamw_plan_bytes(None, 0, None) == 256
    for bad in (dict(bits=16), dict(g=5), dict(c=-1)):
        assert _plan(lib, [{}], **bad)[0] == E.ONEBIT_E_ARG, bad
    assert _plan(lib, [{}], short=8)[0] == E.ONEBIT_E_WORKSPACE
    assert _plan(lib, [{}], plan=False)[0] == E.ONEBIT_E_NULL
    for bad in (dict(lr_scale=NAN), dict(weight_decay=INF)):
        assert _plan(lib, [bad])[0] == E.ONEBIT_E_ARG, bad
    for name in ("x", "g", "m", "v"):
        assert _plan(lib, [{name: None}])[0] == E.ONEBIT_E_NULL, name
        assert _plan(lib, [{name: P * 16 + 2}])[0] == E.ONEBIT_E_ALIGN, name
    assert _plan(lib, [{}], bits=8)[0] == _plan(lib, [{}], c=1)[0] == E.ONEBIT_E_NULL
    eight = dict(m_scale=5 * P, v_scale=6 * P, m=3 * P + 1, v=4 * P + 3)
    assert _plan(lib, [eight], bits=8)[0] == E.ONEBIT_OK
    assert _plan(lib, [dict(eight, v_scale=6 * P + 2)], bits=8)[0] == E.ONEBIT_E_ALIGN
    # what is written over anything else: the same tensor twice, states that share
    # bytes, a gradient inside a parameter; gradients may be one
    other = dict(x=8 * P, g=9 * P, m=10 * P, v=11 * P)
    assert _plan(lib, [{}, {}])[0] == E.ONEBIT_E_ARG
    for bad in (dict(x=P + 3996), dict(m=4 * P), dict(v=8 * P), dict(g=8 * P + 64), dict(g=3 * P)):
        assert _plan(lib, [{}, dict(other, **bad)])[0] == E.ONEBIT_E_ARG, bad
    assert _plan(lib, [{}, dict(other, g=2 * P)])[0] == E.ONEBIT_OK
    assert _plan(lib, [{}, dict(other, x=P + 4000)])[0] == E.ONEBIT_OK
    assert _plan(lib, [dict(eight, m_scale=3 * P + 999)], bits=8)[0] != E.ONEBIT_OK
    table, n = _tensors(dict(n=(1 << 34) + 1))
    assert lib.adamw_plan_bytes(table, n, None) == 0


def test_adamw_step_refusals(lib):
    def f(plan=P, n=2, tiles=4, bits=32, g=0, c=0, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, step=1,
          scale=None):
        return lib.adamw_step(plan, n, tiles, bits, g, c, lr, b1, b2, eps, step, 0, scale, None)

    for bad in (dict(bits=4), dict(g=3), dict(c=3), dict(step=0), dict(b1=1.0), dict(b1=-0.1),
                dict(b2=NAN), dict(b2=1.0), dict(eps=-1.0), dict(eps=INF), dict(lr=NAN)):
        assert f(**bad) == ob.ONEBIT_E_ARG, bad
    for bad in (dict(n=-1), dict(tiles=-1), dict(tiles=1 << 24), dict(n=0)):
        assert f(**bad) == ob.ONEBIT_E_SIZE, bad
    assert f(plan=None) == ob.ONEBIT_E_NULL
    assert f(plan=P + 64) == f(scale=P + 2) == ob.ONEBIT_E_ALIGN
    assert f(plan=None, n=0, tiles=0) == ob.ONEBIT_OK


# ---------------------------------------------------------------- the binding
def test_binding_refusals():
    x, y = torch.zeros(4, 8), torch.zeros(4, 8)
    with pytest.raises(ValueError, match="device tensor"):
        ob.layer_norm_forward(x, y, 4, 8, 1e-5)
    with pytest.raises(ValueError, match="float32, bfloat16 or float16"):
        ob.layer_norm_forward(x.double(), y, 4, 8, 1e-5)
    with pytest.raises(ValueError, match="takes bfloat16 or float16"):
        ob.linear_forward(x, y, torch.zeros(4, 4))
    with pytest.raises(ValueError, match="w has 7 columns"):
        ob.linear_forward(x.half(), torch.zeros(3, 7).half(), y)
    with pytest.raises(ValueError, match="device tensor"):
        ob.linear_forward(x.half(), y.half(), torch.zeros(4, 4).half())
    with pytest.raises(ValueError, match="2 dimensions"):
        ob.linear_forward(torch.zeros(2, 4, 8).half(), y.half(), y)
    with pytest.raises(ValueError, match="activation must be"):
        ob._activation("tanh")
    p, g = [torch.zeros(5)], [torch.zeros(5)]
    with pytest.raises(ValueError, match="device tensor"):
        ob.AdamWPlan(p, g, p, p)
    with pytest.raises(ValueError, match="both scales"):
        ob.AdamWPlan(p, g, p, p, m_scale=p)
    with pytest.raises(ValueError, match="g has 2 entries"):
        ob.AdamWPlan(p, g * 2, p, p)
    with pytest.raises(ValueError, match="8 or 32 bits"):
        AdamW.create(p, g, bits=16)


def _meta(*shape, dtype=torch.float16):
    """A tensor that the binding takes for one on the device, with no memory."""
    class OnDevice(torch.Tensor):
        is_cuda = True

        def get_device(self):
            return 0

        def data_ptr(self):
            return P
    return torch.empty(*shape, dtype=dtype).as_subclass(OnDevice)


def test_binding_checks_shapes_and_types():
    x, w, y = _meta(4, 8), _meta(6, 8), _meta(4, 6)
    for kw, said in ((dict(y=_meta(4, 5)), "y has shape"), (dict(y=_meta(6, 4).t()), "contiguous"),
                     (dict(residual=_meta(4, 7)), "residual has shape"),
                     (dict(pre=_meta(4, 6, dtype=torch.float32)), "pre must be float16"),
                     (dict(bias=_meta(5, dtype=torch.float32)), "bias holds 5"),
                     (dict(bias=_meta(6, dtype=torch.bfloat16)), "bias must be float32 or")):
        with pytest.raises(ValueError, match=said):
            ob.linear_forward(x, w, **dict(dict(y=y), **kw))
    for kw, said in ((dict(activation="gelu"), "needs pre"), (dict(dx=_meta(4, 9)), "dx has shape"),
                     (dict(dw=_meta(6, 8, dtype=torch.bfloat16)), "dw must be float32 or"),
                     (dict(dbias=_meta(6)), "dbias must be float32"),
                     (dict(dy=_meta(1, 6).expand(4, 6)), "contiguous, disjoint")):
        with pytest.raises(ValueError, match=said):
            ob.linear_backward(**dict(dict(dy=y, x=x, w=w), **kw))
    f = _meta(5, dtype=torch.float32)
    for kw, said in ((dict(m=[_meta(4, dtype=torch.float32)]), "m\\[0\\] has 4"),
                     (dict(g=[_meta(5, dtype=torch.float64)]), "g must be"),
                     (dict(v=[_meta(5)]), "v\\[0\\] must be float32"),
                     (dict(copies=[f]), "copies must be bfloat16"),
                     (dict(m_scale=[f], v_scale=[f]), "m\\[0\\] must be uint8")):
        with pytest.raises(ValueError, match=said):
            ob.AdamWPlan(**dict(dict(x=[f], g=[f], m=[f], v=[f]), **kw))


@pytest.mark.parametrize("name,mirror", [("linear_args", ob.LinearArgs),
                                         ("adamw_tensor", ob.AdamWTensor)])
def test_struct_mirrors(tmp_path, name, mirror):
    """Field offsets and sizes as gcc lays them out from the header, against the
    binding's mirrors and its packing."""
    if shutil.which("gcc") is None:
        pytest.skip("gcc not available")
    names = [f[0] for f in mirror._fields_]
    lines = "\n".join(f'printf("{n} %zu\\n", offsetof({name}, {n}));' for n in names)
    src, exe = tmp_path / "off.c", tmp_path / "off"
    src.write_text(f'#include <stddef.h>\n#include <stdio.h>\n#include "onebit.h"\n'
                   f'int main(void) {{\n{lines}\nprintf("sizeof %zu\\n", sizeof({name}));\n'
                   'return 0;\n}\n')
    res = subprocess.run(["gcc", "-std=c99", "-D__HIP_PLATFORM_AMD__",
                          f"-I{os.path.join(B._rocm(), 'include')}", f"-I{B.INCLUDE}", str(src),
                          "-o", str(exe)], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    said = subprocess.run([str(exe)], capture_output=True, text=True).stdout
    out = dict(line.split() for line in said.splitlines())
    for n in names:
        assert int(out[n]) == getattr(mirror, n).offset, n
    assert int(out["sizeof"]) == ctypes.sizeof(mirror)
    if mirror is ob.LinearArgs:
        values = list(range(1, len(names) + 1))
        packed = mirror.from_buffer_copy(ob._LINEAR.pack(*values))
        assert [getattr(packed, n) for n in names] == values
