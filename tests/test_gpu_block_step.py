"""The block operators together, as a model uses them: a pre-norm feed-forward
block (layer norm, first product with GELU, second product, dropout with the
residual) over a padded batch, its gradients by hand through the backward calls,
and AdamW steps on all of its tensors, whose 16-bit copies are the next step's
weights; eager, and captured into a graph."""

import numpy as np
import pytest
import torch

from momentum_compression_amd import onebit as ob
from momentum_compression_amd.state import AdamW
from oracle import block as ref
from oracle import training
from tests._gpu import device, gen, same_f32

pytestmark = pytest.mark.gpu

B, T, W, F = 3, 50, 72, 200
SEED, P_DROP = 0x55AA_1234, 0.1
BF = torch.bfloat16
HP = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8)


class Block:
    """Buffers and calls of one block; the weights are the optimizer's copies."""

    def __init__(self, dev, bits, seed):
        g = gen(seed, dev)
        rows = B * T

        def rand(*shape, scale):
            return torch.randn(shape, generator=g, device=dev) * scale

        # norm's weight and bias stay float32, the products' weights are read as copies
        self.master = [1 + rand(W, scale=0.1), rand(W, scale=0.1), rand(F, W, scale=W ** -0.5),
                       rand(F, scale=0.1), rand(W, F, scale=F ** -0.5), rand(W, scale=0.1)]
        self.copies = [p.to(BF) for p in self.master]
        # gradients of one type: the products write theirs in it, the sums are
        # brought to it
        self.grads = [torch.zeros_like(p) for p in self.master]
        self.opt = AdamW.create(self.master, self.grads, self.copies, bits=bits, seed=SEED,
                                weight_decay=[0.0, 0.0, 0.1, 0.0, 0.1, 0.0])
        e = lambda *s, dtype=BF: torch.empty(s, dtype=dtype, device=dev)  # noqa: E731
        self.h, self.z, self.a = e(rows, W), e(rows, F), e(rows, F)
        self.o, self.out, self.do = e(rows, W), e(rows, W), e(rows, W)
        self.da, self.dh, self.dn = e(rows, F), e(rows, W), e(rows, W)
        self.mean, self.rstd = e(rows, dtype=torch.float32), e(rows, dtype=torch.float32)
        n = max(ob.linear_workspace_bytes(rows, F, W, k) + ob.linear_workspace_bytes(rows, W, F, k)
                + ob.layer_norm_workspace_bytes(rows, W) for k in (False, True))
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=dev)

    def step(self, x, target, real, t):
        rows = B * T
        nw, nb, _, b1, _, b2 = self.master
        _, _, w1, _, w2, _ = self.copies
        ob.layer_norm_forward(x, self.h, rows, W, 1e-5, weight=nw, bias=nb, mean=self.mean,
                              rstd=self.rstd)
        ob.linear_forward(self.h, w1, self.a, bias=b1, activation="gelu", pre=self.z, ws=self.ws)
        ob.linear_forward(self.a, w2, self.o, bias=b2, ws=self.ws)
        ob.dropout_apply(self.o, self.out, rows, W, P_DROP, SEED, t, residual=x)
        # the gradient of 0.5 |out - target|^2 over the real tokens
        dout = ((self.out.float() - target) * real).to(BF)
        ob.dropout_apply(dout, self.do, rows, W, P_DROP, SEED, t)
        gnw, gnb, gw1, gb1, gw2, gb2 = self.grads
        ob.linear_backward(self.do, self.a, w2, dx=self.da, dw=gw2, dbias=gb2, ws=self.ws)
        ob.linear_backward(self.da, self.h, w1, dx=self.dh, dw=gw1, dbias=gb1, activation="gelu",
                           pre=self.z, ws=self.ws)
        ob.layer_norm_backward(self.dh, x, self.mean, self.rstd, rows, W, dx=self.dn, weight=nw,
                               dweight=gnw, dbias=gnb, ws=self.ws)
        ob.adamw_step(self.opt.plan, step=t, seed=SEED, **HP)
        return dout


def _exact(x, target, real, params, t):
    """Output, gradients and the input's gradient in 64 bits."""
    nw, nb, w1, b1, w2, b2 = params
    rows = B * T
    h, mean, rstd = ref.layer_norm(x, nw, nb, 1e-5)
    a, z = ref.linear(h, w1, b1, "gelu")
    o, _ = ref.linear(a, w2, b2, "none")
    f = training.keep_factor(rows, W, P_DROP, SEED, t)
    out = x + f * o
    dout = (out - target) * real
    da, gw2, gb2, _ = ref.linear_grad(f * dout, a, w2, "none", None)
    dh, gw1, gb1, _ = ref.linear_grad(da, h, w1, "gelu", z)
    dx, gnw, gnb = ref.layer_norm_grad(dh, x, mean, rstd, nw)
    return out, [gnw, gnb, gw1, gb1, gw2, gb2], dx


def _inputs(dev):
    g = gen(11, dev)
    x = (torch.randn((B * T, W), generator=g, device=dev) + 0.2).to(BF)
    target = torch.randn((B * T, W), generator=g, device=dev)
    lens = torch.tensor([T, 31, 1], device=dev)
    real = (torch.arange(T, device=dev)[None] < lens[:, None]).view(B * T, 1).float()
    return x, target, real


@pytest.mark.parametrize("bits", [32, 8])
def test_block_and_its_optimizer(bits):
    dev = device()
    x, target, real = _inputs(dev)
    blk = Block(dev, bits, 3)
    h64 = lambda a: a.double().cpu().numpy()  # noqa: E731
    states = [(np.zeros(p.numel(), np.float32),) * 2 for p in blk.master]
    for t in range(1, 4):
        print(f"[block] bits={bits} t={t}", flush=True)
        start = [p.clone() for p in blk.master]
        seen = [h64(c) if i in (2, 4) else h64(p)
                for i, (p, c) in enumerate(zip(blk.master, blk.copies))]
        blk.step(x, target, real, t)
        out, grads, dx = _exact(h64(x), h64(target), h64(real), seen, t)
        # Ten bfloat16 roundings at most stand between the inputs and a result (h, z,
        # a, o, out, the gradients of out, o, a, z and h), each off by at most 2^-8 of
        # what it rounds; over sums of many terms of either sign their parts of the
        # norm stay below that.
        for name, a, b in (("out", blk.out, out), ("dx", blk.dn, dx),
                           *((f"grad {i}", a, b) for i, (a, b) in enumerate(zip(blk.grads, grads)))):
            rel = np.linalg.norm(h64(a) - b) / np.linalg.norm(b)
            assert rel < 10 * 2.0 ** -8, (t, name, rel)
        # the optimizer on those gradients, bit for bit
        for i, (p, g) in enumerate(zip(start, blk.grads)):
            m, v = states[i]
            want, m, v = ref.adamw(p.cpu().numpy().ravel(), g.cpu().numpy().ravel(), m, v, step=t,
                                   weight_decay=blk.opt.weight_decay[i], **HP)
            same_f32(blk.master[i].cpu().numpy().ravel(), want, f"t={t} tensor {i}")
            if bits == 8:
                u = ref.draws(m.size, i, t, SEED)
                (mc, ms), (vc, vs) = ref.encode(m, u, 3, False), ref.encode(v, u, 2, True)
                m = ref.decode(mc, 3) * np.repeat(ms, 256)[:m.size]
                v = ref.decode(vc, 2) * np.repeat(vs, 256)[:v.size]
            states[i] = m, v
            assert torch.equal(blk.copies[i], blk.master[i].to(BF))


def test_captured_step_replays():
    """A captured step, replayed with the program's own work between replays, leaves
    what the eager step leaves; two captured graphs share a workspace, one after the
    other."""
    dev = device()
    x, target, real = _inputs(dev)
    eager, graphed = Block(dev, 8, 5), Block(dev, 8, 5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # torch's own work of the step, once before
        ((graphed.out.float() - target) * real).to(BF)
    torch.cuda.current_stream().wait_stream(side)
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        graphed.step(x, target, real, 1)
    with torch.cuda.graph(second):
        graphed.step(x, target, real, 2)
    for k, (graph, t) in enumerate([(first, 1), (second, 2), (first, 1), (second, 2)]):
        x.mul_(1.25)
        graph.replay()
        eager.step(x, target, real, t)
        torch.cuda.synchronize()
        for a, b in zip(eager.master + eager.copies + eager.grads + eager.opt.m + [eager.dn],
                        graphed.master + graphed.copies + graphed.grads + graphed.opt.m
                        + [graphed.dn]):
            assert torch.equal(a, b), k


def test_past_32_bits():
    """Rows, products and tensors past 2^31 elements: the last ones are what they are
    in a call of their own."""
    dev = device()
    g = gen(2, dev)
    # layer norm
    rows, cols = (1 << 31) // 1000 + 7, 1000
    x = torch.zeros((rows, cols), device=dev, dtype=BF)
    x[-5:] = torch.randn((5, cols), generator=g, device=dev).to(BF)
    y = torch.empty_like(x)
    mean, rstd = torch.empty(rows, device=dev), torch.empty(rows, device=dev)
    ob.layer_norm_forward(x, y, rows, cols, 1e-5, mean=mean, rstd=rstd)
    small = torch.empty(5, cols, device=dev, dtype=BF)
    ob.layer_norm_forward(x[-5:], small, 5, cols, 1e-5)
    assert torch.equal(y[-5:], small) and bool((y[:-5] == 0).all())
    db = torch.empty(cols, device=dev)
    ob.layer_norm_backward(y, x, mean, rstd, rows, cols, dx=y, dbias=db,
                           ws=torch.empty(ob.layer_norm_workspace_bytes(rows, cols),
                                          dtype=torch.uint8, device=dev))
    want = small.double().sum(0)
    assert bool(((db.double() - want).abs() <= 8 * 2.0 ** -24 * small.double().abs().sum(0)).all())
    print("[past 32 bits] linear", flush=True)
    # the same rows through a product, and back
    w = torch.randn((24, cols), generator=g, device=dev).to(BF)
    out = torch.empty((rows, 24), device=dev, dtype=BF)
    ws = torch.empty(ob.linear_workspace_bytes(rows, 24, cols, True), dtype=torch.uint8, device=dev)
    ob.linear_forward(x, w, out, ws=ws)
    few = torch.empty(5, 24, device=dev, dtype=BF)
    ob.linear_forward(x[-5:], w, few)
    # both sum in binary32, in their own orders, and round once
    size = x[-5:].double().abs() @ w.double().abs().t().contiguous()
    off = (out[-5:].double() - few.double()).abs()
    assert bool((off <= 4 * cols * 2.0 ** -24 * size + 2.0 ** -8 * few.double().abs()).all())
    assert bool((out[:-5] == 0).all())
    dw = torch.empty(24, cols, device=dev)
    ob.linear_backward(out, x, w, dw=dw, ws=ws)
    want = out[-5:].double().t().contiguous() @ x[-5:].double()
    size = out[-5:].double().abs().t().contiguous() @ x[-5:].double().abs()
    assert bool(((dw.double() - want).abs() <= 64 * 2.0 ** -24 * size + 1e-30).all())
    del x, y, out, ws
    print("[past 32 bits] adamw", flush=True)
    n = (1 << 31) + 300
    p, gr = torch.zeros(n, device=dev), torch.zeros(n, device=dev, dtype=BF)
    p[-300:] = torch.randn(300, generator=g, device=dev)
    gr[-300:] = torch.randn(300, generator=g, device=dev).to(BF)
    opt = AdamW.create([p], [gr], bits=8, seed=9)
    start = p[-300:].cpu().numpy()
    opt.step(**HP)
    want, m, v = ref.adamw(start, gr[-300:].float().cpu().numpy(), np.zeros(300, np.float32),
                           np.zeros(300, np.float32), step=1, **HP)
    same_f32(p[-300:].cpu().numpy(), want, "x")
    u = ref.draws(300, 0, 1, 9, first=1 << 31)
    mc, ms = ref.encode(m, u, 3, False)
    assert np.array_equal(opt.m[0][-300:].cpu().numpy(), mc)
    assert np.array_equal(opt.m_scale[0][-2:].cpu().numpy(), ms)
    assert bool((p[:-300] == 0).all()) and bool((opt.m[0][:-300] == 0).all())
