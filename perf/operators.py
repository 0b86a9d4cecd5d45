"""Training operators beside the optimizer's kernels: dropout whose mask is
regenerated from a counter, a relative position bias learned per bucket and
head, and the attention that carries both, forward, backward and for single
tokens.  This file states what is measured: the cases, their inputs, the plain
torch form of every operator, the calls of the library and the definition in
64 bits."""

from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}

# key tweak that keeps the dropout draws apart from the INT8 rounding's draws
# under the same seed ("DROP")
KEY_TAG = 0x44524F50


# ---------------------------------------------------------------- cases
def listed():
    return [
        # dropout(x) + residual at a block's end: a handful of rows, where the
        # launch is what counts; the hidden states of a BERT-Large batch of
        # 16 x 512; the gradient over long sequences of odd width in float32
        dict(name="dropout_few_rows", op="dropout", rows=7, cols=1000, dtype="bf16", residual=True,
             p=0.1, row0=0, direction="forward"),
        dict(name="dropout_bert_hidden", op="dropout", rows=16 * 512, cols=1024, dtype="bf16",
             residual=True, p=0.1, row0=0, direction="forward"),
        dict(name="dropout_grad_odd_f32", op="dropout", rows=16411, cols=4099, dtype="f32",
             residual=False, p=0.25, row0=5, direction="backward"),
        # the bias written out for an attention that takes it as a tensor: one
        # new token against a long context, and a BERT-Large map
        dict(name="bias_one_token", op="bias", H=16, Tq=1, Tk=8191, buckets=32, max_distance=128,
             two_sided=False, dtype="f32", past=8190),
        dict(name="bias_bert_map", op="bias", H=16, Tq=512, Tk=512, buckets=32, max_distance=128,
             two_sided=True, dtype="bf16", past=0),
        # its gradient from the gradient of the score map: a BERT-Large batch,
        # and an odd rectangle in float32
        dict(name="bias_grad_bert", op="bias_grad", B=16, H=16, Tq=512, Tk=512, buckets=32,
             max_distance=128, two_sided=True, dtype="bf16", past=0),
        dict(name="bias_grad_odd_f32", op="bias_grad", B=3, H=7, Tq=1021, Tk=2053, buckets=64,
             max_distance=500, two_sided=True, dtype="f32", past=1032),
        # attention: a short batch of odd lengths; BERT-Large training with
        # padded sequences and dropout on the map; a 2048-wide decoder's
        # training; a prompt; single tokens over caches of many lengths
        dict(name="attn_train_short", op="attn_train", B=2, H=4, Hkv=4, Tq=37, Tk=37, D=64,
             causal=False, ragged=True, p=0.1, bias=True, buckets=32, max_distance=128,
             two_sided=True, dtype="bf16", past=0),
        dict(name="attn_train_bert", op="attn_train", B=16, H=16, Hkv=16, Tq=512, Tk=512, D=64,
             causal=False, ragged=True, p=0.1, bias=True, buckets=32, max_distance=128,
             two_sided=True, dtype="bf16", past=0),
        dict(name="attn_train_decoder", op="attn_train", B=2, H=16, Hkv=16, Tq=2048, Tk=2048, D=128,
             causal=True, ragged=False, p=0.0, bias=True, buckets=32, max_distance=128,
             two_sided=False, dtype="bf16", past=0),
        dict(name="attn_prompt", op="attn", B=1, H=16, Hkv=4, Tq=4093, Tk=4093, D=128, causal=True,
             ragged=False, bias=True, buckets=32, max_distance=128, two_sided=False, dtype="f16",
             past=0),
        dict(name="attn_one_token", op="attn", B=32, H=16, Hkv=4, Tq=1, Tk=8192, D=128, causal=True,
             ragged=True, bias=True, buckets=32, max_distance=128, two_sided=False, dtype="bf16",
             past="end"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dropout", "bias", "bias_grad", "attn_train", "attn_train", "attn", "attn"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "dropout":
        cols = _log(rng, 1, 16384)
        rows = _log(rng, 1, max(2, (16411 * 4099) // cols // (1 if dtype == "f32" else 2)))
        return dict(op=op, rows=rows, cols=cols, dtype=dtype, residual=rng.random() < 0.6,
                    p=round(rng.uniform(0.0, 0.6), 3), row0=rng.choice([0, 3, 1 << 33]),
                    direction=rng.choice(["forward", "backward"]))
    two_sided = rng.random() < 0.5
    common = dict(buckets=rng.choice([4, 8, 32, 64, 128]) if two_sided else rng.choice([4, 16, 32, 65]),
                  max_distance=rng.choice([40, 128, 300, 800]), two_sided=two_sided)
    if common["buckets"] >= 64:
        common["max_distance"] = max(128, common["max_distance"])
    if op == "bias":
        H, Tk = rng.randint(1, 32), _log(rng, 1, 8192)
        Tq = 1 if rng.random() < 0.3 else _log(rng, 1, max(1, min(4096, (1 << 26) // (H * Tk))))
        return dict(op=op, H=H, Tq=Tq, Tk=Tk, dtype=dtype, past=rng.choice([0, max(0, Tk - Tq)]),
                    **common)
    if op == "bias_grad":
        B, H, Tk = rng.randint(1, 8), rng.randint(1, 24), _log(rng, 1, 4096)
        Tq = _log(rng, 1, max(1, min(4096, (1 << 26) // (B * H * Tk))))
        return dict(op=op, B=B, H=H, Tq=Tq, Tk=Tk, dtype=dtype,
                    past=rng.choice([0, max(0, Tk - Tq)]), **common)
    dtype = rng.choice(["bf16", "f16"])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    H = Hkv * rng.choice([1, 1, 2, 3, 4])
    D = rng.choice([16, 40, 64, 64, 80, 96, 128, 128])
    causal, ragged, bias = rng.random() < 0.5, rng.random() < 0.4, rng.random() < 0.8
    base = dict(H=H, Hkv=Hkv, D=D, causal=causal, ragged=ragged, bias=bias, dtype=dtype, **common)
    if op == "attn_train":
        T = _log(rng, 1, 2100)
        if T == 1:  # one key: the weights are 1 and the bias has no gradient
            base["bias"] = False
        B = rng.randint(1, max(1, min(16, (1 << 26) // (H * T * T))))
        return dict(op=op, B=B, Tq=T, Tk=T, p=rng.choice([0.0, 0.1, 0.35]), past=0, **base)
    if rng.random() < 0.5:  # single tokens, or a few, over a cache
        Tq, Tk = rng.choice([1, 1, 1, 2, 5]), _log(rng, 1, 16384)
        B = rng.randint(1, max(1, min(64, (1 << 26) // (Hkv * Tk * D))))
        return dict(op=op, B=B, Tq=Tq, Tk=Tk, past="end", **base)
    Tk = _log(rng, 2, 4096)
    Tq = _log(rng, 1, Tk)
    B = rng.randint(1, max(1, min(8, (1 << 27) // (H * Tq * Tk))))
    return dict(op=op, B=B, Tq=Tq, Tk=Tk, past=Tk - Tq, **base)


# ---------------------------------------------------------------- inputs
def _bucket(case, d):
    """Bucket of the distance d = key position - query position, in whole
    numbers: distances below half the buckets of a side have one each, the
    others share them by the logarithm up to max_distance."""
    n, shift = case["buckets"], 0
    if case["two_sided"]:
        n //= 2
        shift = n if d > 0 else 0
        d = abs(d)
    else:
        d = max(-d, 0)
    e = max(1, n // 2)
    if d < e or n == 1:
        return shift + min(d, n - 1)
    k = 0
    while k + 1 < n - e and d ** (n - e) >= e ** (n - e - k - 1) * case["max_distance"] ** (k + 1):
        k += 1
    return shift + e + k


def _map(case):
    R = case["max_distance"]
    return [_bucket(case, d) for d in range(-R, R + 1)]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def prepare(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    dev = "cuda"

    def rand(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(dt)

    rng_seed = int(torch.randint(0, 1 << 62, (1,), generator=g, device=dev).item())
    st = dict(case=case, seed=rng_seed, step=seed % 1000 + 1)
    if case["op"] == "dropout":
        x = rand(case["rows"], case["cols"])
        st.update(x=x, y=torch.empty_like(x),
                  residual=rand(case["rows"], case["cols"]) if case["residual"] else None)
        return st
    st["map"] = torch.tensor(_map(case), dtype=torch.int32, device=dev)
    H = case["H"]
    st["table"] = torch.randn((case["buckets"], H), generator=g, device=dev)
    if case["op"] == "bias":
        st["out"] = torch.empty((H, case["Tq"], case["Tk"]), dtype=dt, device=dev)
        return st
    if case["op"] == "bias_grad":
        st["ds"] = rand(case["B"], H, case["Tq"], case["Tk"], scale=1e-2)
        st["dtable"] = torch.empty((case["buckets"], H), device=dev)
        return st
    B, Tq, Tk, Hkv, D = (case[k] for k in ("B", "Tq", "Tk", "Hkv", "D"))
    if not case["bias"]:
        st["table"] = st["map"] = None
    if case["op"] == "attn_train" and H == Hkv:
        # the fused projection's output, and its gradient's buffer
        qkv = rand(B, Tq, 3 * H, D)
        st["q"], st["k"], st["v"] = qkv[:, :, :H], qkv[:, :, H:2 * H], qkv[:, :, 2 * H:]
        dqkv = torch.empty_like(qkv)
        st["dq"], st["dk"], st["dv"] = dqkv[:, :, :H], dqkv[:, :, H:2 * H], dqkv[:, :, 2 * H:]
    else:
        st["q"], st["k"], st["v"] = rand(B, Tq, H, D), rand(B, Tk, Hkv, D), rand(B, Tk, Hkv, D)
        st["dq"], st["dk"], st["dv"] = (torch.empty_like(st[n]) for n in "qkv")
    st["o"] = torch.empty((B, Tq, H, D), dtype=dt, device=dev)
    st["k_len"] = None
    if case["ragged"]:
        low = max(1, Tk // 4)
        k_len = torch.randint(low, Tk + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        k_len[0] = Tk
        st["k_len"] = k_len
    st["past"] = 0 if case["past"] == "end" else case["past"]
    if case["past"] == "end":  # the new tokens are the last of each sequence
        st["past"] = (st["k_len"] - Tq if case["ragged"]
                      else torch.full((B,), Tk - Tq, dtype=torch.int32, device=dev))
    train = case["op"] == "attn_train"
    if train:
        st["do"] = rand(B, Tq, H, D)
        st["lse"] = torch.empty((B, H, Tq), device=dev)
        st["dtable"] = torch.empty((case["buckets"], H), device=dev) if case["bias"] else None
    return st


# ---------------------------------------------------------------- plain form
def _threshold(p):
    """Kept draws out of 65536 (p as the binary32 number that a call carries)."""
    return max(1, math.floor((1.0 - float(np.float32(p))) * 65536.0 + 0.5))


def _draws(row_ids, cols, seed, step):
    """16-bit draws [rows, cols]: Philox4x32-10 on the counter (column / 8,
    row low, row high, step), eight draws to a call, low half of a word first."""
    low = 0xFFFFFFFF
    c = [torch.arange((cols + 7) // 8, device=row_ids.device)[None, :], (row_ids & low)[:, None],
         (row_ids >> 32)[:, None], torch.full_like(row_ids, step)[:, None]]
    k0, k1 = seed & low, (seed >> 32) ^ KEY_TAG
    for _ in range(10):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((p1 >> 32) & low) ^ c[1] ^ k0, p1 & low, ((p0 >> 32) & low) ^ c[3] ^ k1, p0 & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack(torch.broadcast_tensors(*c), -1)
    halves = torch.stack((words & 0xFFFF, words >> 16), -1)
    return halves.flatten(1)[:, :cols]


def _keep(rows, cols, row0, case, st):
    ids = torch.arange(row0, row0 + rows, device="cuda")
    return _draws(ids, cols, st["seed"], st["step"]) < _threshold(case["p"])


def _distances(case, q_pos):
    """Key position minus query position, one map or one for each sequence."""
    i = torch.arange(case["Tq"], device="cuda")
    j = torch.arange(case["Tk"], device="cuda")
    if torch.is_tensor(q_pos):
        return j[None, None, :] - (q_pos.long()[:, None, None] + i[None, :, None])
    return (j[None, :] - (q_pos + i[:, None]))[None]


def _bias_of(case, table, bucket_map, d):
    R = case["max_distance"]
    return table[bucket_map.long()[d.clamp(-R, R) + R]].permute(0, 3, 1, 2)


def _by_bucket(case, ds, bucket_map, q_pos):
    """Sum of ds [..., H, Tq, Tk] over everything that reads a table entry:
    down the diagonals, then over the distances of a bucket, in 64 bits."""
    H, Tq, Tk = ds.shape[-3:]
    s = ds.reshape(-1, H, Tq, Tk).sum(0, dtype=torch.float64).flip(1)
    wide = torch.nn.functional.pad(s, (0, Tq)).reshape(H, Tq * (Tk + Tq))
    diag = wide[:, :Tq * (Tk + Tq - 1)].reshape(H, Tq, Tk + Tq - 1).sum(1)
    R = case["max_distance"]
    d = torch.arange(Tk + Tq - 1, device="cuda") - (Tq - 1) - q_pos
    hot = torch.nn.functional.one_hot(bucket_map.long()[d.clamp(-R, R) + R], case["buckets"])
    return (hot.double()[:, :, None] * diag.t()[:, None, :]).sum(0).float()


def _heads(x, G=1):
    """[B, T, H, D] in 32 bits with the heads first, shared heads repeated."""
    x = x.float().permute(0, 2, 1, 3)
    return x.repeat_interleave(G, 1) if G > 1 else x.contiguous()


def _plain_attention(st):
    case = st["case"]
    B, H, Hkv, Tq, Tk, D = (case[k] for k in ("B", "H", "Hkv", "Tq", "Tk", "D"))
    G, scale, dt = H // Hkv, D ** -0.5, DTYPES[case["dtype"]]
    q, k, v = _heads(st["q"]), _heads(st["k"], G), _heads(st["v"], G)
    d = _distances(case, st["past"])
    s = (q @ k.transpose(2, 3)) * scale
    if case["bias"]:
        s = s + _bias_of(case, st["table"], st["map"], d)
    if case["causal"]:
        s = s.masked_fill((d > 0)[:, None], -math.inf)
    if case["ragged"]:
        off = torch.arange(Tk, device="cuda")[None, :] >= st["k_len"][:, None]
        s = s.masked_fill(off[:, None, None, :], -math.inf)
    m = s.amax(3, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    e = (s - m).exp()
    total = e.sum(3, keepdim=True)
    prob = e / torch.where(total == 0, torch.ones_like(total), total)
    if case["op"] == "attn":
        return {"o": (prob @ v).permute(0, 2, 1, 3).to(dt)}
    if case["p"] > 0:
        keep = _keep(B * H * Tq, Tk, 0, case, st).view(B, H, Tq, Tk)
        factor = keep.float() * (65536.0 / _threshold(case["p"]))
        dropped = prob * factor
    else:
        factor, dropped = None, prob
    do = _heads(st["do"])
    o = dropped @ v
    dv = dropped.transpose(2, 3) @ do
    dp = do @ v.transpose(2, 3)
    if factor is not None:
        dp = dp * factor
    ds = prob * (dp - (prob * dp).sum(3, keepdim=True))
    dq, dk = (ds @ k) * scale, (ds.transpose(2, 3) @ q) * scale
    out = {"o": o, "dq": dq}
    for name, x in (("dk", dk), ("dv", dv)):
        out[name] = x.view(B, Hkv, G, Tk, D).sum(2)
    out = {name: x.permute(0, 2, 1, 3).to(dt) for name, x in out.items()}
    if case["bias"]:
        out["dtable"] = _by_bucket(case, ds, st["map"], st["past"])
    return out


def _plain(st):
    case = st["case"]
    if case["op"] == "dropout":
        keep = _keep(case["rows"], case["cols"], case["row0"], case, st)
        y = torch.where(keep, st["x"].float() * (65536.0 / _threshold(case["p"])), 0.0)
        if st["residual"] is not None:
            y = st["residual"].float() + y
        return y.to(DTYPES[case["dtype"]])
    if case["op"] == "bias":
        d = _distances(case, case["past"])
        return _bias_of(case, st["table"], st["map"], d)[0].to(DTYPES[case["dtype"]]).contiguous()
    if case["op"] == "bias_grad":
        return _by_bucket(case, st["ds"], st["map"], case["past"])
    return _plain_attention(st)


# ---------------------------------------------------------------- the library's calls
def _workspace(st, nbytes):
    """The caller's workspace, made once and kept with the buffers."""
    if "ws" not in st:
        st["ws"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    return st["ws"]


def _own(st):
    from momentum_compression_amd import onebit as ob

    case = st["case"]
    if case["op"] == "dropout":
        ob.dropout_apply(st["x"], st["y"], case["rows"], case["cols"], case["p"], st["seed"],
                         st["step"], residual=st["residual"], row0=case["row0"])
        return st["y"]
    if case["op"] == "bias":
        ob.rel_bias_expand(st["table"], st["map"], st["out"], q_pos=case["past"])
        return st["out"]
    if case["op"] == "bias_grad":
        ws = _workspace(st, ob.rel_bias_workspace_bytes(*st["ds"].shape, case["max_distance"]))
        ob.rel_bias_grad(st["ds"], st["map"], st["dtable"], q_pos=case["past"], ws=ws)
        return st["dtable"]
    ws = _workspace(st, ob.rel_attention_workspace_bytes(
        *(case[k] for k in ("B", "H", "Hkv", "Tq", "Tk", "D")),
        radius=case["max_distance"] if case["bias"] else 0, backward=case["op"] == "attn_train"))
    how = dict(scale=case["D"] ** -0.5, causal=case["causal"], q_pos=st["past"], k_len=st["k_len"],
               table=st["table"], bucket_map=st["map"], ws=ws)
    if case["op"] == "attn":
        ob.rel_attention_forward(st["q"], st["k"], st["v"], st["o"], **how)
        return {"o": st["o"]}
    how.update(p=case["p"], seed=st["seed"], step=st["step"])
    ob.rel_attention_forward(st["q"], st["k"], st["v"], st["o"], lse=st["lse"], **how)
    ob.rel_attention_backward(st["q"], st["k"], st["v"], st["o"], st["lse"], st["do"], st["dq"],
                              st["dk"], st["dv"], dtable=st["dtable"], **how)
    out = {name: st[name] for name in ("o", "dq", "dk", "dv")}
    if case["bias"]:
        out["dtable"] = st["dtable"]
    return out


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- work
def work(case):
    size = SIZE[case["dtype"]]
    if case["op"] == "dropout":
        n = case["rows"] * case["cols"]
        # flops: the scaling (and the sum); the generator's whole-number work
        # is not counted
        return {"bytes": n * size * (3 if case["residual"] else 2),
                "flops": n * (2 if case["residual"] else 1)}
    tables = 4 * (2 * case["max_distance"] + 1 + case["buckets"] * case["H"])
    if case["op"] == "bias":
        return {"bytes": case["H"] * case["Tq"] * case["Tk"] * size + tables, "flops": 0}
    if case["op"] == "bias_grad":
        n = case["B"] * case["H"] * case["Tq"] * case["Tk"]
        return {"bytes": n * size + tables, "flops": n}
    B, H, Hkv, Tq, Tk, D = (case[k] for k in ("B", "H", "Hkv", "Tq", "Tk", "D"))
    q, kv = B * Tq * H * D, 2 * B * Tk * Hkv * D
    pairs = Tq * Tk
    if case["ragged"]:  # lengths are drawn evenly from a quarter to the whole
        kv, pairs = kv * 5 // 8, pairs * 5 // 8
    if case["causal"] and case["op"] == "attn_train":
        pairs = pairs / 2 + Tq / 2
    elif case["causal"] and Tq > 1:
        pairs = pairs - Tq * (Tq - 1) / 2
    per = 2 * B * H * max(1, pairs) * D
    if case["op"] == "attn":
        return {"bytes": (2 * q + kv) * size, "flops": 2 * per}
    # forward: two products; backward: the scores again and four gradients
    return {"bytes": (4 * q + 2 * kv) * size, "flops": 7 * per}


# ---------------------------------------------------------------- the definition in 64 bits
def _mul32(a, m):
    """High and low half of the product of two 32-bit numbers, by 16-bit parts."""
    a0, a1, m0, m1 = a & 0xFFFF, a >> 16, m & 0xFFFF, m >> 16
    mid = a1 * m0 + ((a0 * m0) >> 16)
    mid2 = a0 * m1 + (mid & 0xFFFF)
    return a1 * m1 + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | ((a0 * m0) & 0xFFFF)


def _exact_factor(ids, cols, p, seed, step):
    """0 or 1 / (kept share) for the rows `ids`, in 64 bits."""
    n = (cols + 7) // 8
    x0 = torch.arange(n, device="cuda").repeat(ids.numel(), 1)
    x1 = (ids % (1 << 32)).view(-1, 1).expand_as(x0)
    x2 = (ids // (1 << 32)).view(-1, 1).expand_as(x0)
    x3 = torch.full_like(x0, step)
    for r in range(10):
        a = (seed % (1 << 32) + r * 0x9E3779B9) % (1 << 32)
        b = ((seed >> 32) ^ 0x44524F50) + r * 0xBB67AE85
        (h0, l0), (h1, l1) = _mul32(x0, 0xD2511F53), _mul32(x2, 0xCD9E8D57)
        x0, x1, x2, x3 = h1 ^ x1 ^ a, l1, h0 ^ x3 ^ (b % (1 << 32)), l0
    u = torch.empty((ids.numel(), n, 8), dtype=torch.int64, device="cuda")
    for w, x in enumerate((x0, x1, x2, x3)):
        u[:, :, 2 * w], u[:, :, 2 * w + 1] = x % 65536, x // 65536
    kept = max(1, int((1.0 - float(np.float32(p))) * 65536 + 0.5))
    return (u.view(ids.numel(), -1)[:, :cols] < kept).double() * (65536 / kept)


def _exact_buckets(case, q_pos):
    """Bucket of every (query, key) of one sequence, -1 nowhere."""
    m = torch.tensor(_map(case), device="cuda")
    R = case["max_distance"]
    j = torch.arange(case["Tk"], device="cuda").view(1, -1)
    i = torch.arange(case["Tq"], device="cuda").view(-1, 1)
    return m[torch.clamp(j - i - q_pos, min=-R, max=R) + R]


def _exact_attention(case, st):
    B, H, Hkv, Tq, Tk, D = (case[k] for k in ("B", "H", "Hkv", "Tq", "Tk", "D"))
    train, G = case["op"] == "attn_train", H // Hkv
    f64 = dict(dtype=torch.float64, device="cuda")
    out = {"o": torch.zeros((B, Tq, H, D), **f64)}
    if train:
        out.update(dq=torch.zeros((B, Tq, H, D), **f64), dk=torch.zeros((B, Tk, Hkv, D), **f64),
                   dv=torch.zeros((B, Tk, Hkv, D), **f64))
        if case["bias"]:
            out["dtable"] = torch.zeros((case["buckets"], H), **f64)
    j = torch.arange(Tk, device="cuda").view(1, -1)
    i = torch.arange(Tq, device="cuda").view(-1, 1)
    for b in range(B):
        past = int(st["past"][b]) if torch.is_tensor(st["past"]) else st["past"]
        seen = j < (int(st["k_len"][b]) if case["ragged"] else Tk)
        if case["causal"]:
            seen = seen & (j <= i + past)
        seen = seen.expand(Tq, Tk)
        buckets = _exact_buckets(case, past) if case["bias"] else None
        for h in range(H):
            q, k, v = (st[n][b, :, h if n == "q" else h // G].double() for n in "qkv")
            z = (q @ k.t()) / math.sqrt(D)
            if case["bias"]:
                z = z + st["table"][:, h].double()[buckets]
            z = torch.where(seen, z, -math.inf)
            prob = torch.nan_to_num(torch.softmax(z, 1))
            if not train:
                out["o"][b, :, h] = prob @ v
                continue
            f = 1.0
            if case["p"] > 0:
                first = (b * H + h) * Tq
                f = _exact_factor(torch.arange(first, first + Tq, device="cuda"), Tk, case["p"],
                                  st["seed"], st["step"])
            do = st["do"][b, :, h].double()
            out["o"][b, :, h] = (prob * f) @ v
            out["dv"][b, :, h // G] += (prob * f).t() @ do
            dp = (do @ v.t()) * f
            ds = prob * dp - prob * (prob * dp).sum(1, keepdim=True)
            out["dq"][b, :, h] = ds @ k / math.sqrt(D)
            out["dk"][b, :, h // G] += ds.t() @ q / math.sqrt(D)
            if case["bias"]:
                out["dtable"][:, h] += torch.bincount(buckets.flatten(), ds.flatten(),
                                                      case["buckets"])
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "dropout":
        rows, cols = case["rows"], case["cols"]
        y = torch.empty((rows, cols), dtype=torch.float64, device="cuda")
        part = max(1, (1 << 24) // cols)
        for r in range(0, rows, part):
            ids = torch.arange(r, min(rows, r + part), device="cuda") + case["row0"]
            f = _exact_factor(ids, cols, case["p"], st["seed"], st["step"])
            y[r:r + part] = st["x"][r:r + part].double() * f
        return y if st["residual"] is None else y + st["residual"].double()
    if case["op"] == "bias":
        return st["table"].double()[_exact_buckets(case, case["past"])].permute(2, 0, 1).contiguous()
    if case["op"] == "bias_grad":
        buckets = _exact_buckets(case, case["past"]).flatten()
        s = st["ds"].double().sum(0).flatten(1)
        return torch.stack([torch.bincount(buckets, s[h], case["buckets"])
                            for h in range(case["H"])], 1)
    return _exact_attention(case, st)
