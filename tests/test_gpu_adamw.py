"""AdamW over many tensors against the plain binary32 form, bit for bit: the
parameters, the 32-bit states, and the 8-bit codes with their scales."""

import numpy as np
import pytest
import torch

from momentum_compression_amd import checkpoint
from momentum_compression_amd import onebit as ob
from momentum_compression_amd.state import AdamW
from oracle import block as ref
from tests._gpu import device, gen, same_bits, same_f32

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HP = dict(lr=2e-3, beta1=0.9, beta2=0.999, eps=1e-8)
SEED = 0x0123_4567_89AB_CDEF
SIZES = [1, 7, 8, 9, 255, 256, 257, 300, 511, 2049, 4095, 4096, 4097, 8200, 20011, 3]


def make(sizes, dtype, dev, seed=1, spread=1.0):
    g = gen(seed, dev)
    params = [torch.randn(n, generator=g, device=dev) * 0.05 for n in sizes]
    grads = [(torch.randn(n, generator=g, device=dev)
              * torch.exp(spread * torch.randn(n, generator=g, device=dev)) * 1e-2).to(TYPES[dtype])
             for n in sizes]
    return params, grads


def np_of(t):
    return t.detach().float().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


class Plain:
    """The optimizer in numpy."""

    def __init__(self, params, bits, lr_scale, decay, seed):
        self.x = [np_of(p).copy() for p in params]
        self.bits, self.lr_scale, self.decay, self.seed, self.t = bits, lr_scale, decay, seed, 0
        self.m = [np.zeros_like(x) for x in self.x]
        self.v = [np.zeros_like(x) for x in self.x]
        self.codes = [None] * len(self.x)

    def step(self, grads, g_scale=None, **hp):
        self.t += 1
        for i, g in enumerate(grads):
            self.x[i], m, v = ref.adamw(self.x[i], np_of(g), self.m[i], self.v[i], step=self.t,
                                        lr_scale=self.lr_scale[i], weight_decay=self.decay[i],
                                        g_scale=g_scale, **hp)
            if self.bits == 32:
                self.m[i], self.v[i] = m, v
                continue
            u = ref.draws(m.size, i, self.t, self.seed)
            mc, ms = ref.encode(m, u, 3, False)
            vc, vs = ref.encode(v, u, 2, True)
            self.codes[i] = mc, ms, vc, vs
            n = m.size
            self.m[i] = ref.decode(mc, 3) * np.repeat(ms, ref.BLOCK)[:n]
            self.v[i] = ref.decode(vc, 2) * np.repeat(vs, ref.BLOCK)[:n]


def compare(opt, plain, name):
    torch.cuda.synchronize()
    for i in range(len(plain.x)):
        what = f"{name} tensor {i} of {plain.x[i].size}"
        same_f32(np_of(opt.params[i]), plain.x[i], f"{what} x")
        if plain.bits == 32:
            same_f32(np_of(opt.m[i]), plain.m[i], f"{what} m")
            same_f32(np_of(opt.v[i]), plain.v[i], f"{what} v")
        else:
            mc, ms, vc, vs = plain.codes[i]
            same_f32(np_of(opt.m_scale[i]), ms, f"{what} m_scale")
            same_f32(np_of(opt.v_scale[i]), vs, f"{what} v_scale")
            same_bits(np_of(opt.m[i]), mc, f"{what} m codes")
            same_bits(np_of(opt.v[i]), vc, f"{what} v codes")
            m, v = opt.state_values(i)
            same_f32(np_of(m), plain.m[i], f"{what} m values")
            same_f32(np_of(v), plain.v[i], f"{what} v values")
        if opt.copies is not None:
            assert torch.equal(opt.copies[i], opt.params[i].to(opt.copies[i].dtype)), what


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,copy", [("f32", None), ("bf16", "bf16"), ("f16", "f16"),
                                        ("f32", "f16")])
def test_steps(bits, dtype, copy):
    dev = device()
    params, grads = make(SIZES, dtype, dev)
    copies = None if copy is None else [torch.zeros_like(p, dtype=TYPES[copy]) for p in params]
    lr_scale = [1.0 + 0.25 * (i % 3) for i in range(len(SIZES))]
    decay = [0.1 * (i % 2) for i in range(len(SIZES))]
    plain = Plain(params, bits, lr_scale, decay, SEED)
    opt = AdamW.create(params, grads, copies, decay, lr_scale, bits, SEED)
    scale = torch.tensor([0.125], device=dev) if dtype == "f16" else None
    for t in range(1, 5):
        print(f"[adamw] bits={bits} {dtype} copy={copy} t={t}", flush=True)
        for k, g in enumerate(grads):
            g.mul_(-0.5 if (t + k) % 3 else 1.5)
        opt.step(grad_scale=scale, **HP)
        plain.step(grads, None if scale is None else 0.125, **HP)
        compare(opt, plain, f"t={t}")


@pytest.mark.parametrize("bits", [32, 8])
def test_views_at_odd_places(bits):
    """Tensors that start at any element of a larger buffer; what lies around
    them stays."""
    dev = device()
    sizes, pad = [1, 13, 300, 4097, 777], 3
    params, grads = make(sizes, "bf16", dev, seed=4)

    def inside(parts, dtype, fill):
        flat = torch.full((sum(p.numel() + pad for p in parts) + pad,), fill, dtype=dtype, device=dev)
        out, at = [], pad
        for p in parts:
            out.append(flat[at:at + p.numel()])
            out[-1].copy_(p)
            at += p.numel() + pad
        return flat, out

    xf, x = inside(params, torch.float32, 7.0)
    _, g = inside(grads, torch.bfloat16, 0.0)
    cf, c = inside(params, torch.bfloat16, 7.0)
    kind = torch.float32 if bits == 32 else torch.uint8
    zeros = [torch.zeros(n, device=dev, dtype=kind) for n in sizes]
    (mf, m), (vf, v) = inside(zeros, kind, 7), inside(zeros, kind, 7)
    state = {"m": m, "v": v}
    if bits == 8:
        blocks = [torch.ones(-(-n // 256), device=dev) for n in sizes]
        state.update(m_scale=blocks, v_scale=[b.clone() for b in blocks])
    plain = Plain(x, bits, [1.0] * 5, [0.05] * 5, 9)
    opt = AdamW.create(x, g, c, 0.05, 1.0, bits, 9, state=state)
    opt.step(**HP)
    plain.step(g, **HP)
    compare(opt, plain, "views")
    for flat in (xf, cf, mf, vf):
        at = 0
        for n in sizes:
            assert bool((flat[at:at + pad] == 7).all())
            at += n + pad
        assert bool((flat[at:] == 7).all())


@pytest.mark.parametrize("bits", [32, 8])
def test_values_of_every_size(bits):
    """Gradients over 60 binades, zeros, and such as are no numbers."""
    dev = device()
    n = 5000
    rng = np.random.default_rng(3)
    g = (rng.standard_normal(n) * 2.0 ** rng.integers(-50, 10, n)).astype(np.float32)
    g[256:512] = 0.0
    g[512:768] = 1e-30                     # squares below the normal numbers
    g[900:930] = np.float32(2.0) ** 3      # a block's largest at a power of two
    params = [torch.from_numpy(rng.standard_normal(n).astype(np.float32)).to(dev)]
    grads = [torch.from_numpy(g).to(dev)]
    plain = Plain(params, bits, [1.0], [0.0], 5)
    opt = AdamW.create(params, grads, bits=bits, seed=5)
    for t in range(3):
        opt.step(**HP)
        plain.step(grads, **HP)
        compare(opt, plain, f"t={t}")
    # a NaN and an infinity reach their own elements alone
    before = [np_of(p).copy() for p in opt.state_values(0)]
    grads[0].zero_()
    grads[0][3], grads[0][1000] = float("nan"), float("inf")
    opt.step(**HP)
    torch.cuda.synchronize()
    m, v = (np_of(a) for a in opt.state_values(0))
    x = np_of(opt.params[0])
    hit = np.zeros(n, bool)
    hit[[3, 1000]] = True
    assert not np.isfinite(m[hit]).any() and not np.isfinite(v[hit]).any()
    assert np.isnan(x[hit]).all() and np.isfinite(x[~hit]).all()
    assert np.isfinite(m[~hit]).all() and np.isfinite(v[~hit]).all()
    assert np.abs(m[~hit]).max() <= np.abs(before[0]).max()


def test_rounding_keeps_the_mean():
    """2^17 elements of one value, their coded m and v: with draws of 16 bits the
    means are the values to 2^-17 of a step and the scatter of as many draws (six
    deviations of at most half a step)."""
    dev = device()
    n = 1 << 17
    p, g = [torch.zeros(n, device=dev)], [torch.full((n,), 0.3, device=dev)]
    g[0][::256] = 1.0  # the scale's element
    opt = AdamW.create(p, g, bits=8, seed=77)
    opt.step(**HP)
    m, v = opt.state_values(0)
    rest = torch.ones(n, dtype=torch.bool, device=dev)
    rest[::256] = False
    b1, b2 = np.float32(0.9), np.float32(0.999)
    f = np.float32
    want = (float((f(1) - b1) * f(0.3)), float((f(1) - b2) * (f(0.3) * f(0.3))))
    for got, w, digits in ((m, want[0], 3), (v, want[1], 2)):
        step = 2.0 ** (np.floor(np.log2(w)) - digits)
        off = abs(float(got[rest].double().mean()) - w)
        assert off < step * (2.0 ** -17 + 6 * 0.5 / np.sqrt(n - n // 256)), (off / step, digits)
        assert len(torch.unique(got[rest])) == 2


def test_another_stream_and_a_graph():
    """The same bits on another stream; a captured step replays itself, with the
    program's own work between replays."""
    dev = device()
    sizes = [5000, 300, 1]
    for bits in (32, 8):
        params, grads = make(sizes, "bf16", dev, seed=8)
        a = AdamW.create([p.clone() for p in params], grads, bits=bits, seed=3)
        b = AdamW.create([p.clone() for p in params], grads, bits=bits, seed=3)
        a.step(**HP)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            b.step(**HP)
        side.synchronize()
        torch.cuda.synchronize()
        for x, y in zip(a.params + a.m + a.v, b.params + b.m + b.v):
            assert torch.equal(x, y)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            ob.adamw_step(b.plan, step=2, seed=3, **HP)
        for k in range(3):
            for g in grads:
                g.mul_(0.5)
            graph.replay()
            ob.adamw_step(a.plan, step=2, seed=3, **HP)
            torch.cuda.synchronize()
            for x, y in zip(a.params + a.m + a.v, b.params + b.m + b.v):
                assert torch.equal(x, y), (bits, k)


def test_checkpoint_and_other_gradients(tmp_path):
    """A run that is saved and resumed goes on as one that is not, and set_grads
    takes other gradient tensors."""
    dev = device()
    sizes = [700, 256, 33]
    for bits in (32, 8):
        params, grads = make(sizes, "f32", dev, seed=9)
        opt = AdamW.create(params, grads, weight_decay=0.01, bits=bits, seed=4)
        opt.step(**HP)
        path = str(tmp_path / f"ck{bits}")
        checkpoint.save(path, opt.state_dict(), meta={"steps": opt.steps, "seed": opt.seed})
        other = [g * 2 for g in grads]
        opt.set_grads(other)
        opt.step(**HP)
        tensors, meta = checkpoint.load(path, dev)
        back = AdamW.from_state(tensors, other, weight_decay=0.01, **meta)
        back.step(**HP)
        assert back.steps == 2
        for x, y in zip(opt.params + opt.m + opt.v, back.params + back.m + back.v):
            assert torch.equal(x, y), bits


def test_many_tensors_and_none():
    dev = device()
    sizes = [1 + (37 * i) % 900 for i in range(700)]
    params, grads = make(sizes, "f16", dev, seed=6)
    params.append(torch.empty(0, device=dev))
    grads.append(torch.empty(0, device=dev, dtype=torch.float16))
    plain = Plain(params, 32, [1.0] * 701, [0.01] * 701, 0)
    opt = AdamW.create(params, grads, weight_decay=0.01)
    opt.step(**HP)
    plain.step(grads, **HP)
    compare(opt, plain, "many")
    empty = AdamW.create([], [])
    empty.step(**HP)
    assert empty.steps == 1
