"""The training operators together, as a model uses them, and their gradients
into the optimizer: one attention block (fused projection, attention with the
learned position bias and dropout on its map, output projection, dropout with
the residual), a padded batch, its gradients by hand through the backward
calls, gathered in one flat buffer with a layer table, and LAMB warm-up steps
and a compression on that buffer."""

import numpy as np
import pytest
import torch

from momentum_compression_amd import onebit as ob
from momentum_compression_amd.attention import rel_bucket_map
from momentum_compression_amd.state import LambWarmup, OneBitGroup
from oracle import onebit
from oracle import training as ref
from oracle import warmup
from tests._gpu import device, gen, host, same_bits, same_f32

pytestmark = pytest.mark.gpu

B, T, H, D, N_BUCKETS, FAR = 3, 70, 2, 32, 8, 20
W = H * D
P_MAP, P_OUT, SEED = 0.1, 0.2, 0xABCD_0123
F32 = np.float32
HP = dict(lr=1e-3, eps=1e-6, beta1=0.9, beta2=0.999)


def _block(x, lens, w_qkv, w_o, table, bmap, target, t, dev):
    """The block's output, and the gradients of 0.5 |out - target|^2 over the
    real tokens."""
    bf = torch.bfloat16
    qkv = (x @ w_qkv).to(bf).view(B, T, 3 * H, D)
    q, k, v = qkv[:, :, :H], qkv[:, :, H:2 * H], qkv[:, :, 2 * H:]
    o = torch.empty((B, T, H, D), dtype=bf, device=dev)
    lse = torch.empty((B, H, T), device=dev)
    ws = torch.empty(ob.rel_attention_workspace_bytes(B, H, H, T, T, D, FAR, True),
                     dtype=torch.uint8, device=dev)
    how = dict(k_len=lens, table=table, bucket_map=bmap, p=P_MAP, seed=SEED, step=t, ws=ws)
    ob.rel_attention_forward(q, k, v, o, lse=lse, **how)
    a = o.view(B * T, W).float() @ w_o
    out = torch.empty_like(a)
    xf = x.reshape(B * T, W)
    ob.dropout_apply(a, out, B * T, W, P_OUT, SEED + 1, t, residual=xf)
    real = (torch.arange(T, device=dev)[None] < lens[:, None]).view(B * T, 1)
    dout = (out - target) * real
    da = torch.empty_like(dout)
    ob.dropout_apply(dout, da, B * T, W, P_OUT, SEED + 1, t)
    dw_o = o.view(B * T, W).float().t() @ da
    do = (da @ w_o.t()).to(bf).view(B, T, H, D)
    dqkv = torch.empty_like(qkv)
    dq, dk, dv = dqkv[:, :, :H], dqkv[:, :, H:2 * H], dqkv[:, :, 2 * H:]
    dtable = torch.empty_like(table)
    ob.rel_attention_backward(q, k, v, o, lse, do, dq, dk, dv, dtable=dtable, **how)
    dw_qkv = xf.t() @ dqkv.view(B * T, 3 * W).float()
    return out, dw_qkv, dw_o, dtable


def _exact_block(x, lens, w_qkv, w_o, table, bmap, target, t):
    """The same block in 64 bits."""
    qkv = (x @ w_qkv).reshape(B, T, 3 * H, D)
    q, k, v = qkv[:, :, :H], qkv[:, :, H:2 * H], qkv[:, :, 2 * H:]
    kw = dict(scale=D ** -0.5, k_len=lens, table=table, bmap=bmap, p=P_MAP, seed=SEED, step=t)
    o = ref.attention(q, k, v, **kw)["o"].reshape(B * T, W)
    xf = x.reshape(B * T, W)
    f = ref.keep_factor(B * T, W, P_OUT, SEED + 1, t)
    out = xf + f * (o @ w_o)
    real = (np.arange(T)[None] < lens[:, None]).reshape(B * T, 1)
    da = f * ((out - target) * real)
    do = (da @ w_o.T).reshape(B, T, H, D)
    g = ref.attention(q, k, v, do=do, **kw)
    dqkv = np.concatenate([g["dq"], g["dk"], g["dv"]], 2).reshape(B * T, 3 * W)
    return out, xf.T @ dqkv, o.T @ da, g["dtable"]


def test_block_gradients_into_the_optimizer():
    dev = device()
    g = gen(7, dev)
    x = torch.randn((B, T, W), generator=g, device=dev)
    target = torch.randn((B * T, W), generator=g, device=dev)
    lens = torch.tensor([T, 41, 1], dtype=torch.int32, device=dev)
    bmap = rel_bucket_map(N_BUCKETS, FAR, True, dev)
    # one flat buffer of three layers: the two projections and the table
    n = 4
    shapes = [(W, 3 * W), (W, W), (N_BUCKETS, H)]
    off = np.concatenate([[0], np.cumsum([a * b for a, b in shapes])]).astype(np.int64)
    off[-1] = -(-off[-1] // (64 * n)) * (64 * n)
    N = int(off[-1])
    print(f"[train step] N={N} tokens={B * T}", flush=True)

    def parts(buf):
        return [buf[int(o):int(o) + a * b].reshape(a, b) for o, (a, b) in zip(off, shapes)]

    off_d = torch.from_numpy(off).to(dev)
    start = torch.randn(N, generator=g, device=dev) * W ** -0.5
    st = LambWarmup.create(start.clone(), off_d)
    grad = torch.zeros(N, device=dev)
    xh, mh, vh, cav = host(start), np.zeros(N, F32), np.zeros(N, F32), None
    for t in range(1, 4):
        got = _block(x, lens, *parts(st.x), bmap, target, t, dev)
        want = _exact_block(x.double().cpu().numpy(), lens.cpu().numpy(),
                            *parts(xh.astype(np.float64)), bmap.cpu().numpy(),
                            target.double().cpu().numpy(), t)
        # Five bfloat16 roundings stand between the inputs and a gradient (the
        # projection, o, its gradient, a probability or dS, dqkv), each off by
        # at most 2^-8 of what it rounds; over sums of many terms of either
        # sign their parts of the norm stay below 5 * 2^-8.
        for name, a, b in zip(("out", "dw_qkv", "dw_o", "dtable"), got, want):
            rel = np.linalg.norm(a.double().cpu().numpy() - b) / np.linalg.norm(b)
            print(f"t={t} {name} {rel:.2e}", flush=True)
            assert rel < 5 * 2.0 ** -8, (t, name, rel)
        for to, a in zip(parts(grad), got[1:]):
            to.copy_(a)
        # the optimizer takes the flat gradient as any other
        st.step(grad, beta_c=0.9, **HP)
        torch.cuda.synchronize()
        o = warmup.lamb_warmup_step(xh, mh, vh, host(grad), off, c_avg=cav, beta_c=0.9, **HP)
        same_f32(host(st.m), o["m"], f"t={t} m")
        same_f32(host(st.x), o["x"], f"t={t} x")
        xh, mh, vh, cav = host(st.x), host(st.m), host(st.v), host(st.c_avg)
    # and so does the compressed phase that follows
    k = st.momentum_scale()
    grp = OneBitGroup(N, n, dev, seg_off=off_d, seg_k=k)
    mloc = st.m.unsqueeze(0).repeat(n, 1)
    grp.compress(mloc, 1, first=True)
    grp.server(1, first=True)
    torch.cuda.synchronize()
    k_el = onebit.per_element_k(off, host(k))
    w = onebit.worker_compress(host(mloc), np.zeros((n, N), F32), reset=True, k=k_el)
    sv = onebit.server_reduce(w["bits"], w["s"], np.zeros(N, F32), reset=True)
    same_bits(host(grp.bits), w["bits"], "worker bits")
    same_bits(host(grp.sv_bits), sv["bits"], "server bits")
