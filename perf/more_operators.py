"""Operators of a transformer block's training step beside attention and
dropout: layer norm forward and backward, the matrix product with bias,
activation and residual in its epilogue (rows of one token to whole batches)
with its gradients, and the AdamW step over many tensors at once with states in
32 or 8 bits.  This file states what is measured: the cases, their inputs, the
plain torch form of every operator, the calls of the library and the definition
in 64 bits."""

from __future__ import annotations

import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2, "none": 0}

BLOCK = 256  # elements that share a scale of the 8-bit states

# key tweak that keeps the rounding draws of the states apart from the draws of
# other operators under the same seed ("ADMW")
KEY_TAG = 0x41444D57

HYPER = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8)


# ---------------------------------------------------------------- cases
def listed():
    return [
        # layer norm: the hidden states of four new tokens while serving, where
        # the launch is what counts; a BERT-Large batch of 16 x 512 in training
        # (mean and 1 / deviation kept for the backward pass); the backward
        # pass of a 2048-wide decoder with both parameter gradients; the same
        # in float32 over rows of odd width
        dict(name="ln_four_tokens", op="ln", rows=4, cols=2048, dtype="bf16", w_dtype="bf16",
             stats=False),
        dict(name="ln_bert_hidden", op="ln", rows=16 * 512, cols=1024, dtype="bf16",
             w_dtype="f32", stats=True),
        dict(name="ln_grad_decoder", op="ln_grad", rows=8 * 2048, cols=2048, dtype="bf16",
             w_dtype="f32"),
        dict(name="ln_grad_odd_f32", op="ln_grad", rows=16411, cols=1003, dtype="f32",
             w_dtype="f32"),
        # matrix products: one new token through the first feed-forward product
        # of a 2048-wide decoder; BERT-Large's first feed-forward product with
        # its activation, the sum before it kept for the backward pass; all
        # gradients of that product; an odd shape with the residual, as the
        # product behind an activation has it
        dict(name="linear_one_token", op="linear", M=1, N=8192, K=2048, dtype="bf16", bias="bf16",
             act="gelu", residual=False, pre=False, pad=0),
        dict(name="linear_bert_up", op="linear", M=16 * 512, N=4096, K=1024, dtype="bf16",
             bias="f32", act="gelu", residual=False, pre=True, pad=0),
        dict(name="linear_bert_up_grad", op="linear_grad", M=16 * 512, N=4096, K=1024,
             dtype="bf16", bias="f32", act="gelu", dw="bf16", pad=0),
        dict(name="linear_odd_residual", op="linear", M=1021, N=2051, K=1003, dtype="f16",
             bias="f32", act="none", residual=True, pre=False, pad=0),
        # AdamW: a block of a small model, where the launch is what counts; the
        # 302 tensors of BERT-Large with bfloat16 gradients and a bfloat16 copy
        # of the parameters, states in 32 and in 8 bits; many tensors of odd
        # sizes with scaled float16 gradients
        dict(name="adamw_small_block", op="adamw", tensors="block", hidden=64, count=0, low=0,
             high=0, sizes=0, bits=32, g_dtype="f32", copy="none", scaled=False),
        dict(name="adamw_bert_large", op="adamw", tensors="bert_large", hidden=1024, count=0,
             low=0, high=0, sizes=0, bits=32, g_dtype="bf16", copy="bf16", scaled=False),
        dict(name="adamw_bert_large_8bit", op="adamw", tensors="bert_large", hidden=1024, count=0,
             low=0, high=0, sizes=0, bits=8, g_dtype="bf16", copy="bf16", scaled=False),
        dict(name="adamw_odd_8bit", op="adamw", tensors="mixed", hidden=0, count=75, low=1,
             high=2000003, sizes=3, bits=8, g_dtype="f16", copy="f16", scaled=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln", "ln_grad", "linear", "linear", "linear_grad", "linear_grad", "adamw",
                     "adamw"])
    if op == "adamw":
        kind = rng.choice(["mixed", "mixed", "mixed", "block"])
        low = _log(rng, 1, 5000)
        high = _log(rng, low + 1, 4000000)
        return dict(op=op, tensors=kind, hidden=_log(rng, 16, 2048), count=_log(rng, 1, 100),
                    low=low, high=high, sizes=rng.randrange(1 << 20), bits=rng.choice([32, 8]),
                    g_dtype=rng.choice(["f32", "bf16", "f16"]),
                    copy=rng.choice(["none", "bf16", "f16"]), scaled=rng.random() < 0.5)
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op in ("ln", "ln_grad"):
        # two columns leave the gradient nothing but what rounding makes of it
        cols = _log(rng, 1 if op == "ln" else 3, 40000)
        rows = _log(rng, 1, max(2, (1 << 25) // cols // (2 if dtype == "f32" else 1)))
        case = dict(op=op, rows=rows, cols=cols, dtype=dtype,
                    w_dtype=rng.choice(["f32", dtype]))
        if op == "ln":
            case["stats"] = rng.random() < 0.5
        return case
    dtype = rng.choice(["bf16", "f16"])
    few = rng.random() < 0.4
    M = _log(rng, 1, 40 if few else 16384)
    N = _log(rng, 1, 16384)
    K = _log(rng, 1, max(1, min(16384, (1 << 35) // (M * N))))
    act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"])
    case = dict(op=op, M=M, N=N, K=K, dtype=dtype, bias=rng.choice(["none", "f32", dtype]),
                act=act, pad=rng.choice([0, 0, 8, 5]))
    if op == "linear":
        case.update(residual=rng.random() < 0.5, pre=rng.random() < 0.3)
    else:
        # 32-bit weight gradients where the gradient of the product is an input
        case.update(dw=rng.choice(["f32", dtype]) if act == "none" else dtype)
    return case


def _sizes(case):
    """Elements of each tensor of an AdamW case, and whether its weights decay
    (matrices do, biases and norms do not)."""
    if case["tensors"] == "mixed":
        r = random.Random(case["sizes"])
        sizes = [_log(r, case["low"], case["high"]) for _ in range(case["count"])]
        return sizes, [n % 3 != 0 for n in sizes]
    h = case["hidden"]
    f = 4 * h
    layer = [3 * h * h, 3 * h, h * h, h, h, h, f * h, f, h * f, h, h, h]
    if case["tensors"] == "block":
        return layer, [n >= h * h for n in layer]
    vocab = 30522
    sizes = [vocab * h, 512 * h, 2 * h, h, h] + 24 * layer
    sizes += [h * h, h, h * h, h, h, h, vocab, 2 * h, 2]
    return sizes, [n >= h * h for n in sizes]


# ---------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _rows_of(rand, rows, cols, pad):
    """[rows, cols], part of a wider matrix where `pad` is given."""
    return rand(rows, cols + pad)[:, :cols] if pad else rand(rows, cols)


def _power_of_two(e):
    return (e << 23).view(torch.float32)


def _prepare_adamw(case, g, seed):
    dev = "cuda"
    sizes, decays = _sizes(case)
    blocks = [-(-n // BLOCK) for n in sizes]
    count = torch.tensor(blocks, device=dev)
    tensor_of = torch.repeat_interleave(torch.arange(len(sizes), device=dev), count)
    first = torch.cumsum(count, 0) - count
    N = BLOCK * len(tensor_of)
    # elements that exist: the flat buffers hold each tensor from a whole block on
    left = torch.tensor(sizes, device=dev)[tensor_of] - BLOCK * (
        torch.arange(len(tensor_of), device=dev) - first[tensor_of])
    real = torch.arange(BLOCK, device=dev)[None] < left[:, None]

    def rand():
        return torch.randn(len(tensor_of), BLOCK, generator=g, device=dev)

    # gradients differ by tensor and by element; the states follow them
    scale = torch.exp(torch.randn(len(sizes), generator=g, device=dev)) * 1e-3
    sigma = torch.exp(0.7 * rand()) * scale[tensor_of][:, None] * real
    boost = 1024.0 if case["scaled"] else 1.0
    st = dict(case=case, sizes=sizes, t=seed % 1000 + 1,
              seed=int(torch.randint(0, 1 << 62, (1,), generator=g, device=dev).item()),
              decay=[0.01 if d else 0.0 for d in decays],
              lr_scale=[1.0 if d else 0.5 for d in decays],
              tensor_of=tensor_of, block_of=torch.arange(len(tensor_of), device=dev) - first[tensor_of],
              start=[BLOCK * int(f) for f in first.tolist()],
              g=(rand() * sigma * boost).to(DTYPES[case["g_dtype"]]).view(N),
              x=(rand() * 0.02 * real).view(N),
              g_scale=torch.full((1,), 1.0 / boost, device=dev) if case["scaled"] else None)
    m = rand() * sigma * 0.3
    v = sigma * sigma * (0.7 + 0.6 * torch.rand(sigma.shape, generator=g, device=dev))
    st["copy"] = (None if case["copy"] == "none"
                  else torch.zeros(N, dtype=DTYPES[case["copy"]], device=dev))
    if case["bits"] == 32:
        st.update(m=m.view(N), v=v.view(N))
        return st
    # the states as an earlier step left them: 8-bit values times a power of two
    # a block, whose largest value has 2^7 in m and 2^14 in v
    em = torch.clamp(m.abs().amax(1).view(torch.int32) >> 23, min=8) - 7
    ev = torch.clamp(v.amax(1).view(torch.int32) >> 23, min=15) - 14
    st.update(m=(m * _power_of_two(254 - em)[:, None]).to(torch.float8_e4m3fn).view(N),
              v=(v * _power_of_two(254 - ev)[:, None]).to(torch.float8_e5m2).view(N),
              m_scale=_power_of_two(em), v_scale=_power_of_two(ev))
    return st


def prepare(case, seed):
    g = _gen(seed)
    dev = "cuda"
    if case["op"] == "adamw":
        return _prepare_adamw(case, g, seed)
    dt = DTYPES[case["dtype"]]

    def rand(*shape, scale=1.0, kind=dt):
        return (torch.randn(shape, generator=g, device=dev) * scale).to(kind)

    st = dict(case=case)
    if case["op"] in ("ln", "ln_grad"):
        rows, cols = case["rows"], case["cols"]
        # rows of different spread about a common offset, a few wide channels
        spread = torch.exp(0.5 * torch.randn((rows, 1), generator=g, device=dev))
        wide = 1.0 + 9.0 * (torch.rand(cols, generator=g, device=dev) < 0.01)
        x = (torch.randn((rows, cols), generator=g, device=dev) * wide + 0.3) * spread
        wt = DTYPES[case["w_dtype"]]
        st.update(x=x.to(dt), weight=(1.0 + 0.1 * rand(cols, kind=torch.float32)).to(wt),
                  bias=rand(cols, scale=0.1, kind=wt), eps=1e-5)
        if case["op"] == "ln":
            st["y"] = torch.empty((rows, cols), dtype=dt, device=dev)
            st["mean"] = torch.empty(rows, device=dev) if case["stats"] else None
            st["rstd"] = torch.empty(rows, device=dev) if case["stats"] else None
            return st
        x = st["x"].double()
        mean = x.mean(1)
        var = (x - mean[:, None]).square().mean(1)
        st.update(mean=mean.float(), rstd=(var + st["eps"]).rsqrt().float(), dy=rand(rows, cols),
                  dx=torch.empty((rows, cols), dtype=dt, device=dev),
                  dweight=torch.empty(cols, device=dev), dbias=torch.empty(cols, device=dev))
        return st
    M, N, K = case["M"], case["N"], case["K"]
    st["x"] = _rows_of(rand, M, K, case["pad"])
    st["w"] = rand(N, K, scale=K ** -0.5)
    st["bias"] = None if case["bias"] == "none" else rand(N, scale=0.1, kind=DTYPES[case["bias"]])
    if case["op"] == "linear":
        st["y"] = torch.empty((M, N), dtype=dt, device=dev)
        st["pre"] = torch.empty((M, N), dtype=dt, device=dev) if case["pre"] else None
        st["residual"] = _rows_of(rand, M, N, case["pad"]) if case["residual"] else None
        return st
    st["dy"] = _rows_of(rand, M, N, case["pad"])
    st["pre"] = None if case["act"] == "none" else rand(M, N)
    st["dx"] = torch.empty((M, K), dtype=dt, device=dev)
    st["dw"] = torch.empty((N, K), dtype=DTYPES[case["dw"]], device=dev)
    st["dbias"] = None if case["bias"] == "none" else torch.empty(N, device=dev)
    return st


# ---------------------------------------------------------------- plain form
def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    if act == "gelu":
        return (0.5 * (1.0 + torch.erf(z * math.sqrt(0.5)))
                + z * torch.exp(-0.5 * z * z) * math.sqrt(0.5 / math.pi))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z * z * z))
    return 0.5 * (1.0 + t) + 0.5 * z * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * z * z)


def _plain_linear(st):
    case = st["case"]
    dt = DTYPES[case["dtype"]]
    if case["op"] == "linear":
        z = st["x"].float() @ st["w"].float().t()
        if st["bias"] is not None:
            z = z + st["bias"].float()
        y = _act(z, case["act"])
        if st["residual"] is not None:
            y = y + st["residual"].float()
        out = {"y": y.to(dt)}
        if case["pre"]:
            out["pre"] = z.to(dt)
        return out
    dz = st["dy"].float()
    if case["act"] != "none":
        dz = dz * _slope(st["pre"].float(), case["act"])
    out = {"dx": (dz @ st["w"].float()).to(dt),
           "dw": (dz.t() @ st["x"].float()).to(DTYPES[case["dw"]])}
    if st["bias"] is not None:
        out["dbias"] = dz.sum(0, dtype=torch.float64).float()
    return out


def _plain_ln(st):
    case = st["case"]
    dt = DTYPES[case["dtype"]]
    x = st["x"].float()
    if case["op"] == "ln":
        mean = x.mean(1, keepdim=True)
        d = x - mean
        rstd = torch.rsqrt((d * d).mean(1, keepdim=True) + st["eps"])
        out = {"y": (d * rstd * st["weight"].float() + st["bias"].float()).to(dt)}
        if case["stats"]:
            out.update(mean=mean.view(-1), rstd=rstd.view(-1))
        return out
    rstd = st["rstd"][:, None]
    h = (x - st["mean"][:, None]) * rstd
    dy = st["dy"].float()
    dh = dy * st["weight"].float()
    dx = rstd * (dh - dh.mean(1, keepdim=True) - h * (dh * h).mean(1, keepdim=True))
    return {"dx": dx.to(dt), "dweight": (dy * h).sum(0, dtype=torch.float64).float(),
            "dbias": dy.sum(0, dtype=torch.float64).float()}


def _draws(st):
    """16-bit draws [blocks, BLOCK]: Philox4x32-10 on the counter (element / 8,
    tensor, 0, step), eight draws to a call, low half of a word first."""
    low = 0xFFFFFFFF
    group = st["block_of"][:, None] * (BLOCK // 8) + torch.arange(BLOCK // 8, device="cuda")[None]
    c = [group, st["tensor_of"][:, None].expand_as(group), torch.zeros_like(group),
         torch.full_like(group, st["t"])]
    k0, k1 = st["seed"] & low, (st["seed"] >> 32) ^ KEY_TAG
    for _ in range(10):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [((p1 >> 32) & low) ^ c[1] ^ k0, p1 & low, ((p0 >> 32) & low) ^ c[3] ^ k1, p0 & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack(c, -1)
    return torch.stack((words & 0xFFFF, words >> 16), -1).flatten(1).to(torch.int32)


def _encode(y, draws, least, kept):
    """Codes of y >= 0 in the 8-bit format of `kept` mantissa bits whose normal
    values begin at 2^least: the draw is added below the kept bits and the rest
    cut off, so the mean over the draws is y."""
    drop = 23 - kept
    noise = (draws << (drop - 16)) + (1 << (drop - 17)) - ((126 + least) << 23)
    tiny = y < 2.0 ** least
    bits = torch.where(tiny, y + 2.0 ** least, y).view(torch.int32)
    return ((bits + noise) >> drop) - torch.where(tiny, 1 << kept, 0)


def _plain_adamw(st):
    case = st["case"]
    f32 = torch.float32
    rows = st["tensor_of"].numel()
    t, lr = st["t"], HYPER["lr"]
    b1, b2 = (torch.tensor(HYPER[k], device="cuda") for k in ("beta1", "beta2"))
    of = st["tensor_of"]
    lr_t = (torch.tensor(st["lr_scale"], device="cuda") * torch.tensor(lr, dtype=f32).item())
    decay = 1.0 - lr_t * torch.tensor(st["decay"], device="cuda")
    rate = lr_t * torch.tensor(1.0 / (1.0 - float(b1.double()) ** t), dtype=f32).item()
    root = torch.tensor(1.0 / math.sqrt(1.0 - float(b2.double()) ** t), dtype=f32).item()
    g = st["g"].view(rows, BLOCK).float()
    if st["g_scale"] is not None:
        g = g * st["g_scale"]
    m, v = st["m"].view(rows, BLOCK).float(), st["v"].view(rows, BLOCK).float()
    if case["bits"] == 8:
        m, v = m * st["m_scale"][:, None], v * st["v_scale"][:, None]
    m = b1 * m + (1.0 - b1) * g
    v = b2 * v + (1.0 - b2) * (g * g)
    x = st["x"].view(rows, BLOCK)
    x = x * decay[of][:, None] - rate[of][:, None] * (
        m / (torch.sqrt(v) * root + torch.tensor(HYPER["eps"], dtype=f32).item()))
    st["x"].copy_(x.view(-1))
    st["t"] = t + 1
    out = {"x": st["x"]}
    if st["copy"] is not None:
        out["copy"] = st["copy"].copy_(st["x"])
    if case["bits"] == 32:
        out["m"], out["v"] = st["m"].copy_(m.view(-1)), st["v"].copy_(v.view(-1))
        return out
    draws = _draws(dict(st, t=t))
    em = torch.clamp(m.abs().amax(1).view(torch.int32) >> 23, min=8) - 7
    ev = torch.clamp(v.amax(1).view(torch.int32) >> 23, min=15) - 14
    cm = _encode(m.abs() * _power_of_two(254 - em)[:, None], draws, -6, 3)
    cm = torch.where(m.view(torch.int32) < 0, cm + 128, cm)
    cv = _encode(v * _power_of_two(254 - ev)[:, None], draws, -14, 2)
    cv = torch.where(v > 0, cv.clamp(min=1), cv)
    st["m"].view(torch.uint8).copy_(cm.view(-1))
    st["v"].view(torch.uint8).copy_(cv.view(-1))
    st["m_scale"].copy_(_power_of_two(em))
    st["v_scale"].copy_(_power_of_two(ev))
    out.update({k: st[k] for k in ("m", "v", "m_scale", "v_scale")})
    return out


def _plain(st):
    op = st["case"]["op"]
    return (_plain_adamw if op == "adamw" else
            _plain_ln if op in ("ln", "ln_grad") else _plain_linear)(st)


# ---------------------------------------------------------------- the library's calls
def _workspace(st, nbytes):
    """The caller's workspace, made once and kept with the buffers."""
    if "ws" not in st:
        st["ws"] = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    return st["ws"]


def _optimizer(st):
    """The optimizer over the tensors, which a training program keeps."""
    if "opt" not in st:
        from momentum_compression_amd.state import AdamW

        case = st["case"]

        def parts(flat, per=1):
            return [flat[a // per:a // per + -(-n // per)] for a, n in zip(st["start"], st["sizes"])]

        state = {"m": parts(st["m"]), "v": parts(st["v"])}
        if case["bits"] == 8:
            state.update(m_scale=parts(st["m_scale"], BLOCK), v_scale=parts(st["v_scale"], BLOCK))
        st["opt"] = AdamW.create(
            parts(st["x"]), parts(st["g"]), copies=None if st["copy"] is None else parts(st["copy"]),
            weight_decay=st["decay"], lr_scale=st["lr_scale"], bits=case["bits"], seed=st["seed"],
            state=state, steps=st["t"] - 1)
    return st["opt"]


def _own(st):
    from momentum_compression_amd import onebit as ob

    case = st["case"]
    if case["op"] == "adamw":
        _optimizer(st).step(grad_scale=st["g_scale"], **HYPER)
        names = ("x", "copy", "m", "v", "m_scale", "v_scale")
        return {k: st[k] for k in names if st.get(k) is not None}
    if case["op"] == "ln":
        ob.layer_norm_forward(st["x"], st["y"], case["rows"], case["cols"], st["eps"],
                              weight=st["weight"], bias=st["bias"], mean=st["mean"],
                              rstd=st["rstd"])
        out = {"y": st["y"]}
        if case["stats"]:
            out.update(mean=st["mean"], rstd=st["rstd"])
        return out
    if case["op"] == "ln_grad":
        ws = _workspace(st, ob.layer_norm_workspace_bytes(case["rows"], case["cols"]))
        ob.layer_norm_backward(st["dy"], st["x"], st["mean"], st["rstd"], case["rows"],
                               case["cols"], dx=st["dx"], weight=st["weight"],
                               dweight=st["dweight"], dbias=st["dbias"], ws=ws)
        return {k: st[k] for k in ("dx", "dweight", "dbias")}
    ws = _workspace(st, ob.linear_workspace_bytes(case["M"], case["N"], case["K"],
                                                  backward=case["op"] == "linear_grad"))
    if case["op"] == "linear":
        ob.linear_forward(st["x"], st["w"], st["y"], bias=st["bias"], activation=case["act"],
                          residual=st["residual"], pre=st["pre"], ws=ws)
        return {k: st[k] for k in ("y", "pre") if st[k] is not None}
    ob.linear_backward(st["dy"], st["x"], st["w"], dx=st["dx"], dw=st["dw"], dbias=st["dbias"],
                       activation=case["act"], pre=st["pre"], ws=ws)
    return {k: st[k] for k in ("dx", "dw", "dbias") if st[k] is not None}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- work
def work(case):
    if case["op"] == "adamw":
        n = sum(_sizes(case)[0])
        state = 8 if case["bits"] == 32 else 2 + 8 / BLOCK
        # the parameter and both states are read and written; the generator's
        # whole-number work is not counted
        return {"bytes": n * (8 + 2 * state + SIZE[case["g_dtype"]] + SIZE[case["copy"]]),
                "flops": n * 14}
    size = SIZE[case["dtype"]]
    if case["op"] in ("ln", "ln_grad"):
        n, cols = case["rows"] * case["cols"], case["cols"]
        if case["op"] == "ln":
            return {"bytes": 2 * n * size + 2 * cols * SIZE[case["w_dtype"]]
                    + (8 * case["rows"] if case["stats"] else 0), "flops": 8 * n}
        return {"bytes": 3 * n * size + cols * (SIZE[case["w_dtype"]] + 8) + 8 * case["rows"],
                "flops": 13 * n}
    M, N, K = case["M"], case["N"], case["K"]
    if case["op"] == "linear":
        outs = 1 + (1 if case["residual"] else 0) + (1 if case["pre"] else 0)
        return {"bytes": (M * K + N * K + outs * M * N) * size + N * SIZE[case["bias"]],
                "flops": 2 * M * N * K}
    ins = 1 if case["act"] == "none" else 2
    return {"bytes": (2 * M * K + N * K + ins * M * N) * size + N * K * SIZE[case["dw"]]
            + (0 if case["bias"] == "none" else 4 * N), "flops": 4 * M * N * K}


# ---------------------------------------------------------------- the definition in 64 bits
def _normal_cdf(z):
    return 0.5 * torch.special.erfc(-z / math.sqrt(2.0))


def _exact_linear(case, st):
    act = case["act"]
    f64 = {k: st[k].double() for k in ("x", "w", "bias", "residual", "dy", "pre")
           if st.get(k) is not None and not (k == "pre" and case["op"] == "linear")}
    if case["op"] == "linear":
        z = torch.nn.functional.linear(f64["x"], f64["w"], f64.get("bias"))
        if act == "gelu":
            y = z * _normal_cdf(z)
        elif act == "gelu_tanh":
            y = z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
        else:
            y = {"none": lambda u: u, "relu": torch.relu, "silu": torch.nn.functional.silu}[act](z)
        if "residual" in f64:
            y = y + f64["residual"]
        return {"y": y, "pre": z} if case["pre"] else {"y": y}
    dz = f64["dy"]
    if act != "none":
        z = f64["pre"]
        s = torch.sigmoid(z)
        if act == "relu":
            dz = torch.where(z > 0, dz, torch.zeros_like(dz))
        elif act == "silu":
            dz = dz * (s + z * s * torch.sigmoid(-z))
        elif act == "gelu":
            dz = dz * (_normal_cdf(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi))
        else:
            k = 2.0 * math.sqrt(2.0 / math.pi)
            u = torch.sigmoid(k * (z + 0.044715 * z ** 3))
            dz = dz * (u + z * u * (1 - u) * k * (1 + 3 * 0.044715 * z ** 2))
    out = {"dx": dz @ f64["w"], "dw": dz.t().contiguous() @ f64["x"]}
    if st["bias"] is not None:
        out["dbias"] = dz.sum(0)
    return out


def _exact_ln(case, st):
    x, w, b = st["x"].double(), st["weight"].double(), st["bias"].double()
    if case["op"] == "ln":
        var, mean = torch.var_mean(x, 1, correction=0)
        sd = torch.sqrt(var + st["eps"])
        y = torch.addcmul(b, (x - mean[:, None]) / sd[:, None], w)
        return {"y": y, "mean": mean, "rstd": 1.0 / sd} if case["stats"] else {"y": y}
    h = (x - st["mean"].double()[:, None]) * st["rstd"].double()[:, None]
    dy = st["dy"].double()
    u = dy * w
    n = case["cols"]
    along = (u * h).sum(1, keepdim=True) / n
    dx = st["rstd"].double()[:, None] * (u - u.sum(1, keepdim=True) / n - along * h)
    return {"dx": dx, "dweight": (dy * h).sum(0), "dbias": dy.sum(0)}


def _mul32(a, m):
    """High and low half of the product of two 32-bit numbers, by 16-bit parts."""
    a0, a1, m0, m1 = a & 0xFFFF, a >> 16, m & 0xFFFF, m >> 16
    mid = a1 * m0 + ((a0 * m0) >> 16)
    mid2 = a0 * m1 + (mid & 0xFFFF)
    return a1 * m1 + (mid >> 16) + (mid2 >> 16), ((mid2 & 0xFFFF) << 16) | ((a0 * m0) & 0xFFFF)


def _exact_uniform(n, tensor, step, seed):
    """The n elements' draws as numbers in (0, 1)."""
    x0 = torch.arange((n + 7) // 8, device="cuda")
    x1, x2, x3 = torch.full_like(x0, tensor), torch.zeros_like(x0), torch.full_like(x0, step)
    for r in range(10):
        a = (seed % (1 << 32) + r * 0x9E3779B9) % (1 << 32)
        b = (((seed >> 32) ^ 0x41444D57) + r * 0xBB67AE85) % (1 << 32)
        (h0, l0), (h1, l1) = _mul32(x0, 0xD2511F53), _mul32(x2, 0xCD9E8D57)
        x0, x1, x2, x3 = h1 ^ x1 ^ a, l1, h0 ^ x3 ^ b, l0
    u = torch.empty((len(x0), 8), dtype=torch.int64, device="cuda")
    for w, x in enumerate((x0, x1, x2, x3)):
        u[:, 2 * w], u[:, 2 * w + 1] = x % 65536, x // 65536
    return (u.flatten()[:n].double() + 0.5) / 65536


def _single(x):
    """What a binary32 operation leaves of an exact result."""
    return x.float().double()


def _exact_codes(value, u, top, least, digits):
    """The block scales that put each block's largest value into [2^top,
    2^(top + 1)), and the values over them on the format's grid: the point below,
    or the one above with the probability of the distance to it."""
    n = value.numel()
    padded = torch.nn.functional.pad(value, (0, -n % BLOCK)).view(-1, BLOCK)
    most = padded.abs().amax(1)
    e = torch.floor(torch.log2(most)).clamp(min=top - 126)
    e = torch.where(most == 0, torch.full_like(e, top - 126), e) - top
    scale = torch.exp2(e)
    y = (padded / scale[:, None]).flatten()[:n]
    step = torch.exp2(torch.floor(torch.log2(y.abs())).clamp(min=least) - digits)
    return scale, torch.sign(y) * torch.floor(y.abs() / step + u) * step


def _exact_adamw(case, st):
    f64 = dict(dtype=torch.float64, device="cuda")
    t = st["t"]
    lr, b1, b2, eps = (float(torch.tensor(HYPER[k])) for k in ("lr", "beta1", "beta2", "eps"))
    out = {"x": torch.zeros(st["x"].numel(), **f64)}
    out.update({k: torch.zeros_like(out["x"]) for k in ("m", "v")})
    if case["bits"] == 8:
        out.update({k: st[k].double() for k in ("m_scale", "v_scale")})
    for i, (a, n) in enumerate(zip(st["start"], st["sizes"])):
        s, blocks = slice(a, a + n), slice(a // BLOCK, a // BLOCK + -(-n // BLOCK))
        g, x, m, v = (st[k][s].to(torch.float32).double() for k in "gxmv")
        if st["g_scale"] is not None:
            g = _single(g * st["g_scale"].double())
        if case["bits"] == 8:
            m = m * st["m_scale"][blocks].double().repeat_interleave(BLOCK)[:n]
            v = v * st["v_scale"][blocks].double().repeat_interleave(BLOCK)[:n]
        m0, v0 = m, v
        m, v = b1 * m + (1 - b1) * g, b2 * v + (1 - b2) * g * g
        rate = lr * st["lr_scale"][i]
        wd = float(torch.tensor(st["decay"][i]))
        out["x"][s] = x - rate * wd * x - rate * (m / (1 - b1 ** t)) / (
            torch.sqrt(v / (1 - b2 ** t)) + eps)
        if case["bits"] == 32:
            out["m"][s], out["v"][s] = m, v
            continue
        # the states that are rounded to 8 bits are binary32 numbers, of one
        # rounding an operation: a block's largest value decides its scale
        m, v = (_single(_single(b * old) + _single(float(torch.tensor(1 - b)) * new))
                for b, old, new in ((b1, m0, g), (b2, v0, _single(g * g))))
        u = _exact_uniform(n, i, t, st["seed"])
        out["m_scale"][blocks], out["m"][s] = _exact_codes(m, u, 7, -6, 3)
        out["v_scale"][blocks], q = _exact_codes(v, u, 14, -14, 2)
        out["v"][s] = torch.where(v > 0, q.clamp(min=2.0 ** -16), q)
    if st["copy"] is not None:
        out["copy"] = out["x"]
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(case, st)
    return (_exact_ln if case["op"] in ("ln", "ln_grad") else _exact_linear)(case, st)
