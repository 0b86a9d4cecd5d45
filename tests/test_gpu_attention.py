"""rel_attention_forward and rel_attention_backward against the 64-bit forms,
element by element within derived bounds (tests/_attention.py)."""

import numpy as np
import pytest
import torch

from momentum_compression_amd import onebit as ob
from momentum_compression_amd.attention import rel_bucket_map
from tests._attention import (SEED, TYPES, check, expected, half_step, host64, make, numbers,
                              workspace)
from tests._gpu import device, gen

pytestmark = pytest.mark.gpu

# name: B, H, Hkv, Tq, Tk, D, causal, q_pos, k_len, buckets, max_distance, two_sided, p
FORWARD = {
    "one": (1, 1, 1, 1, 1, 8, False, 0, None, 0, 0, False, 0.0),
    "tiny": (2, 3, 3, 5, 7, 16, True, 2, None, 4, 8, False, 0.0),
    "plain": (2, 2, 2, 64, 64, 64, False, 0, None, 0, 0, False, 0.0),
    "bias": (1, 2, 2, 70, 129, 64, False, 0, None, 32, 40, True, 0.0),
    "causal_grouped": (1, 6, 2, 150, 150, 128, True, 0, None, 32, 128, False, 0.0),
    "odd_width": (2, 2, 1, 33, 200, 40, True, 167, None, 8, 20, True, 0.0),
    "wide_odd": (1, 2, 2, 130, 97, 104, False, -5, None, 32, 64, True, 0.0),
    "padded": (4, 2, 2, 90, 90, 64, False, 0, (90, 33, 1, 64), 32, 128, True, 0.0),
    "empty_rows": (4, 2, 1, 40, 70, 80, True, (-8, 30, -100, 3), (70, 0, 20, 5), 8, 20, False, 0.0),
    "dropout": (2, 2, 2, 75, 139, 64, False, 0, (139, 100), 32, 40, True, 0.2),
    "dropout_causal": (1, 4, 2, 140, 140, 128, True, 0, None, 0, 0, False, 0.5),
    "far_radius": (1, 1, 1, 300, 900, 64, True, 600, None, 64, 1024, False, 0.0),
    "narrow_radius": (1, 2, 2, 260, 400, 32, False, 0, None, 4, 8, True, 0.0),
    "one_token": (3, 4, 2, 1, 1000, 128, True, (999, 500, 0), (1000, 501, 1), 32, 128, False, 0.0),
    "one_token_many_heads": (2, 16, 2, 1, 777, 64, True, 776, None, 32, 128, False, 0.0),
    "few_tokens": (2, 4, 4, 5, 1500, 96, True, 1495, None, 32, 128, False, 0.0),
    "few_tokens_dropout": (1, 2, 2, 3, 1100, 64, False, 0, (1050,), 8, 100, True, 0.3),
    "long_cache": (1, 1, 1, 2, 9000, 64, True, 8998, None, 32, 128, False, 0.0),
}


def _setup(name, dtype, cases, fused=False):
    B, H, Hkv, Tq, Tk, D, causal, q_pos, k_len, n, far, two, p = cases[name]
    dev = device()
    print(f"[attention] {name} {dtype} {cases[name]}", flush=True)
    g = gen(sum(map(ord, name)), dev)
    q, k, v = make(dtype, B, H, Hkv, Tq, Tk, D, g, dev, fused=fused)
    if isinstance(q_pos, tuple):
        q_pos = torch.tensor(q_pos, dtype=torch.int32, device=dev)
    if k_len is not None:
        k_len = torch.tensor(k_len, dtype=torch.int32, device=dev)
    table = torch.randn((n, H), generator=g, device=dev) if n else None
    bmap = rel_bucket_map(n, far, two, dev) if n else None
    how = dict(scale=D ** -0.5, causal=causal, q_pos=q_pos, k_len=k_len, table=table,
               bucket_map=bmap, p=p, seed=SEED, step=17)
    return q, k, v, how, g


def _oracle(q, k, v, do, how, dtype):
    kl = host64(how["k_len"])
    return expected(host64(q), host64(k), host64(v), host64(do), how["scale"], how["causal"],
                    numbers(how["q_pos"]), None if kl is None else kl.astype(int),
                    host64(how["table"]),
                    None if how["bucket_map"] is None else how["bucket_map"].cpu().numpy(),
                    how["p"], SEED, 17, half_step(dtype))


def _poison_past(k_len, *tensors):
    """NaN in every key and value that no query may read."""
    if k_len is not None:
        for x in tensors:
            for b, n in enumerate(k_len.tolist()):
                x[b, max(0, n):] = float("nan")


def _tiny(dtype):
    # the smallest step of the type, for results below its normal range
    return 2.0 ** -133 if dtype == "bf16" else 2.0 ** -24


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name", FORWARD)
def test_forward(name, dtype):
    q, k, v, how, _ = _setup(name, dtype, FORWARD)
    want, tol = _oracle(q, k, v, None, how, dtype)
    _poison_past(how["k_len"], k, v)
    o = torch.full_like(q, 9.0)
    lse = torch.full((q.shape[0], q.shape[2], q.shape[1]), 9.0, device=q.device)
    ws = workspace(q, k)
    ob.rel_attention_forward(q, k, v, o, lse=lse, ws=ws, **how)
    check(dict(o=o, lse=lse), want, tol, ("o", "lse"), _tiny(dtype))
    again = torch.empty_like(o)
    ob.rel_attention_forward(q, k, v, again, ws=ws, **how)
    assert torch.equal(again, o)


# Narrow heads over many splits: fewer lanes of the join have a column than
# have a split's weight.
NARROW = {
    f"narrow_{D}_{Tq}": (1, 2, 1, Tq, 9000, D, True, 9000 - Tq, None, 32, 128, False, p)
    for D, Tq, p in ((8, 1, 0.0), (16, 1, 0.2), (16, 40, 0.0), (40, 3, 0.0), (8, 130, 0.1))
}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name", NARROW)
def test_forward_of_narrow_heads_over_many_splits(name, dtype):
    q, k, v, how, _ = _setup(name, dtype, NARROW)
    want, tol = _oracle(q, k, v, None, how, dtype)
    o = torch.full_like(q, 9.0)
    lse = torch.full((q.shape[0], q.shape[2], q.shape[1]), 9.0, device=q.device)
    ob.rel_attention_forward(q, k, v, o, lse=lse, ws=workspace(q, k), **how)
    check(dict(o=o, lse=lse), want, tol, ("o", "lse"), _tiny(dtype))


BACKWARD = {
    "one": (1, 1, 1, 1, 1, 8, False, 0, None, 0, 0, False, 0.0),
    "tiny": (2, 3, 3, 5, 7, 16, True, 2, None, 4, 8, False, 0.0),
    "plain": (2, 2, 2, 64, 64, 64, False, 0, None, 0, 0, False, 0.0),
    "bias": (1, 2, 2, 70, 129, 64, False, 0, None, 32, 40, True, 0.0),
    "causal_grouped": (2, 6, 2, 150, 150, 128, True, 0, None, 32, 128, False, 0.0),
    "odd_width": (2, 2, 1, 33, 200, 40, True, 167, None, 8, 20, True, 0.1),
    "wide_odd": (1, 2, 2, 130, 97, 104, False, -5, None, 32, 64, True, 0.3),
    "padded_dropout": (4, 2, 2, 90, 90, 64, False, 0, (90, 33, 1, 64), 32, 128, True, 0.1),
    "empty_rows": (4, 2, 1, 40, 70, 80, True, (-8, 30, -100, 3), (70, 0, 20, 5), 8, 20, False, 0.0),
    "dropout_causal": (1, 4, 2, 140, 140, 128, True, 0, None, 0, 0, False, 0.5),
    "dropout_plain": (1, 2, 2, 100, 170, 64, False, 0, None, 0, 0, False, 0.25),
    "far_radius": (1, 1, 1, 300, 500, 64, True, 200, None, 64, 1024, False, 0.0),
    "narrow_radius": (1, 2, 2, 260, 400, 32, False, 0, None, 4, 8, True, 0.0),
    "ragged_tile": (1, 1, 1, 129, 385, 64, False, 100, None, 8, 24, True, 0.0),
    "one_token": (2, 4, 4, 1, 300, 128, True, 299, None, 32, 128, False, 0.2),
}


def _backward(q, k, v, how, do, dtable=None, ws=None, fused=False, accumulate=False):
    o = torch.full_like(do, 9.0)
    lse = torch.full((q.shape[0], q.shape[2], q.shape[1]), 9.0, device=q.device)
    radius = 0 if dtable is None else how["bucket_map"].numel() // 2
    if ws is None:
        ws = workspace(q, k, radius, True)
    if fused:
        H, Hkv = q.shape[2], k.shape[2]
        d = torch.full((*q.shape[:2], H + 2 * Hkv, q.shape[3]), 9.0, dtype=q.dtype,
                       device=q.device)
        dq, dk, dv = d[:, :, :H], d[:, :, H:H + Hkv], d[:, :, H + Hkv:]
    else:
        dq, dk, dv = (torch.full(x.shape, 9.0, dtype=x.dtype, device=x.device) for x in (q, k, v))
    ob.rel_attention_forward(q, k, v, o, lse=lse, ws=ws, **how)
    ob.rel_attention_backward(q, k, v, o, lse, do, dq, dk, dv, dtable=dtable,
                              accumulate=accumulate, ws=ws, **how)
    return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv, dtable=dtable)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name", BACKWARD)
def test_backward(name, dtype):
    fused = BACKWARD[name][3] == BACKWARD[name][4]
    q, k, v, how, g = _setup(name, dtype, BACKWARD, fused=fused)
    do = torch.randn(q.shape, generator=g, device=q.device).to(TYPES[dtype])
    want, tol = _oracle(q, k, v, do, how, dtype)
    if not fused:
        _poison_past(how["k_len"], k, v)
    dtable = None if how["table"] is None else torch.full_like(how["table"], 9.0)
    got = _backward(q, k, v, how, do, dtable, fused=fused)
    names = ["o", "lse", "dq", "dk", "dv"] + (["dtable"] if dtable is not None else [])
    check(got, want, tol, names, _tiny(dtype))
    if dtable is None:
        return
    # the same bits again, and the table's gradient added to itself; without it
    # another kernel computes dk and dv, within the same bounds
    twice = _backward(q, k, v, how, do, dtable.clone(), fused=fused)
    for n in names:
        assert torch.equal(twice[n], got[n]), n
    bare = _backward(q, k, v, how, do, None, fused=fused)
    check(bare, want, tol, ("dq", "dk", "dv"), _tiny(dtype))
    more = _backward(q, k, v, how, do, dtable.clone(), fused=fused, accumulate=True)
    assert torch.allclose(more["dtable"], 2 * dtable, rtol=2 ** -22, atol=0)


# Causal prompts behind a cache.  From positions of 1 to 32 modulo 64 on, the
# first waves of a tile of 97 queries or more are through with the keys while
# the last ones still have a tile to come, of which they brought their part.
BEHIND = {
    f"behind_{pos}_{Tq}": (2, 4, 2, Tq, pos + Tq, D, True, pos, None, n, 64, False, p)
    for pos, Tq, D, n, p in ((1, 97, 64, 0, 0.0), (20, 128, 64, 32, 0.0), (32, 129, 128, 0, 0.1),
                             (33, 128, 64, 0, 0.0), (64 + 16, 300, 128, 32, 0.0),
                             (256 + 1, 257, 64, 32, 0.1), (512 + 32, 99, 128, 32, 0.0))
}
BEHIND["behind_two"] = (2, 4, 4, 200, 700, 64, True, (500, 65), (700, 265), 32, 64, False, 0.0)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("name", BEHIND)
def test_prompts_behind_a_cache(name, dtype):
    q, k, v, how, g = _setup(name, dtype, BEHIND)
    do = torch.randn(q.shape, generator=g, device=q.device).to(TYPES[dtype])
    want, tol = _oracle(q, k, v, do, how, dtype)
    dtable = None if how["table"] is None else torch.full_like(how["table"], 9.0)
    names = ["o", "lse", "dq", "dk", "dv"] + (["dtable"] if dtable is not None else [])
    got = _backward(q, k, v, how, do, dtable)
    check(got, want, tol, names, _tiny(dtype))
    again = _backward(q, k, v, how, do, dtable.clone() if dtable is not None else None)
    for n in names:
        assert torch.equal(again[n], got[n]), n


def test_gradients_by_differences():
    """The gradients against differences of the oracle's forward map at the
    rounded inputs, along random directions."""
    from oracle import training as ref

    name = "padded_dropout"
    q, k, v, how, g = _setup(name, "bf16", BACKWARD)
    do = torch.randn(q.shape, generator=g, device=q.device).to(torch.bfloat16)
    dtable = torch.empty_like(how["table"])
    got = _backward(q, k, v, how, do, dtable)
    x = {n: host64(t) for n, t in (("q", q), ("k", k), ("v", v), ("table", how["table"]))}
    m = how["bucket_map"].cpu().numpy()
    kl = how["k_len"].cpu().numpy()

    def loss(y):
        o = ref.attention(y["q"], y["k"], y["v"], how["scale"], how["causal"], 0, kl, y["table"],
                          m, how["p"], SEED, 17)["o"]
        return (o * host64(do)).sum()

    rng = np.random.default_rng(1)
    for n, d in (("q", "dq"), ("k", "dk"), ("v", "dv"), ("table", "dtable")):
        e = rng.standard_normal(x[n].shape)
        h = 1e-5
        by = (loss({**x, n: x[n] + h * e}) - loss({**x, n: x[n] - h * e})) / (2 * h)
        grad = host64(got[d])
        # random signs: the roundings of the terms add like their squares
        spread = np.sqrt(((grad * e) ** 2).sum())
        assert abs((grad * e).sum() - by) < 6 * 2.0 ** -8 * spread + 1e-6, n


def test_dropout_mask_is_dropout_applys():
    """Equal scores and one-hot values show the weights: each is kept where
    dropout_apply keeps it on the score map's rows."""
    dev = device()
    B, H, Tq, Tk, p = 2, 2, 70, 64, 0.3
    q = torch.zeros((B, Tq, H, 64), dtype=torch.bfloat16, device=dev)
    k = torch.zeros((B, Tk, H, 64), dtype=torch.bfloat16, device=dev)
    v = torch.eye(64, dtype=torch.bfloat16, device=dev)[None, :, None].expand(B, Tk, H, 64)
    v = v.contiguous()
    o = torch.empty_like(q)
    ob.rel_attention_forward(q, k, v, o, p=p, seed=SEED, step=3)
    ones = torch.ones((B * H * Tq, Tk), device=dev)
    kept = torch.empty_like(ones)
    ob.dropout_apply(ones, kept, B * H * Tq, Tk, p, SEED, 3)
    assert torch.equal(o.permute(0, 2, 1, 3).reshape(B * H * Tq, Tk) != 0, kept != 0)


def test_caches_and_orders_of_other_strides():
    """[B, H, T, D] caches, one cache for all sequences (stride 0), and rows
    further apart than they are wide give what contiguous copies give."""
    dev = device()
    g = gen(3, dev)
    B, H, Hkv, Tq, Tk, D = 3, 4, 2, 60, 200, 64
    q = torch.randn((B, H, Tq, D), generator=g, device=dev).bfloat16().transpose(1, 2)
    kv = torch.randn((1, Hkv, Tk, 2 * D + 24), generator=g, device=dev).bfloat16()
    k = kv[..., 8:8 + D].transpose(1, 2).expand(B, Tk, Hkv, D)
    v = kv[..., D + 16:2 * D + 16].transpose(1, 2).expand(B, Tk, Hkv, D)
    o = torch.full((B, H, Tq, D + 8), 5.0, dtype=torch.bfloat16, device=dev)
    ov = o[..., :D].transpose(1, 2)
    plain = torch.empty((B, Tq, H, D), dtype=torch.bfloat16, device=dev)
    how = dict(causal=True, q_pos=140)
    ob.rel_attention_forward(q, k, v, ov, ws=workspace(q, k), **how)
    ob.rel_attention_forward(q.contiguous(), k.contiguous(), v.contiguous(), plain,
                             ws=workspace(q, k), **how)
    assert torch.equal(ov, plain) and bool((o[..., D:] == 5).all())


def test_values_past_the_length_and_nan_inputs():
    """NaN in a query reaches its own row alone."""
    dev = device()
    g = gen(9, dev)
    q, k, v = make("bf16", 1, 1, 1, 40, 100, 64, g, dev)
    clean = torch.empty_like(q)
    ob.rel_attention_forward(q, k, v, clean, ws=workspace(q, k))
    q[0, 7] = float("nan")
    o = torch.empty_like(q)
    ob.rel_attention_forward(q, k, v, o, ws=workspace(q, k))
    assert bool(o[0, 7].isnan().all())
    rest = [i for i in range(40) if i != 7]
    assert torch.equal(o[0, rest], clean[0, rest])


@pytest.mark.parametrize("dtype", TYPES)
def test_cache_places_that_no_query_sees(dtype):
    """Under the causal mask a cache may hold anything past the last query's
    position: the results are those of a cache that ends there, and its keys'
    gradients are 0."""
    dev = device()
    bmap = rel_bucket_map(32, 40, False, dev)
    for Tq, Tk, D, pos, k_len in ((1, 1000, 64, (700, 0), None), (5, 500, 128, (300, 64), None),
                                  (70, 400, 64, (200, -30), (400, 41)),
                                  (130, 256, 80, (0, 17), None),
                                  (40, 3000, 128, (1000, 2000), None)):
        g = gen(Tq + D, dev)
        q, k, v = make(dtype, 2, 4, 2, Tq, Tk, D, g, dev)
        do = torch.randn(q.shape, generator=g, device=dev).to(TYPES[dtype])
        table = torch.randn((32, 4), generator=g, device=dev)
        how = dict(causal=True, q_pos=torch.tensor(pos, dtype=torch.int32, device=dev),
                   table=table, bucket_map=bmap, p=0.1, seed=SEED, step=5)
        if k_len is not None:
            how["k_len"] = torch.tensor(k_len, dtype=torch.int32, device=dev)
        want = _backward(q, k, v, how, do, torch.empty_like(table))
        for b, n in enumerate(pos):
            for x in (k, v):
                x[b, max(0, n + Tq):] = float("nan")
        got = _backward(q, k, v, how, do, torch.empty_like(table))
        for n in want:
            assert torch.equal(got[n], want[n]), (Tq, Tk, n)
        for b, n in enumerate(pos):
            for x in ("dk", "dv"):
                assert bool((got[x][b, max(0, n + Tq):] == 0).all())


def test_lowest_bias_values():
    """A table holding the type's lowest number, or -inf, hides its distances
    without NaN."""
    dev = device()
    g = gen(2, dev)
    q, k, v = make("f16", 1, 2, 2, 50, 80, 64, g, dev)
    bmap = rel_bucket_map(8, 20, True, dev)
    for low in (torch.finfo(torch.float32).min, float("-inf")):
        table = torch.randn((8, 2), generator=g, device=dev)
        table[5:] = low                       # every key after the query
        o, lse = torch.empty_like(q), torch.empty((1, 2, 50), device=dev)
        ob.rel_attention_forward(q, k, v, o, lse=lse, table=table, bucket_map=bmap,
                                 ws=workspace(q, k))
        want = torch.empty_like(q)
        safe = torch.where(table == low, torch.zeros_like(table), table)
        ob.rel_attention_forward(q, k, v, want, table=safe, bucket_map=bmap, causal=True,
                                 ws=workspace(q, k))
        assert torch.equal(o, want) and bool(lse.isfinite().all())


@pytest.mark.parametrize("Tq", [1, 50])
def test_lowest_bias_values_backward(Tq):
    """... nor in the gradients: those of the keys it hides are 0, and so are
    all of a row that it hides whole.  One query goes through the kernel for
    few, whose bias comes another way."""
    dev = device()
    g = gen(4, dev)
    q, k, v = make("bf16", 1, 2, 2, Tq, 80, 64, g, dev)
    do = torch.randn(q.shape, generator=g, device=dev).bfloat16()
    bmap = rel_bucket_map(8, 20, True, dev)
    for low in (torch.finfo(torch.float32).min, -1e38, float("-inf")):
        table = torch.randn((8, 2), generator=g, device=dev)
        table[5:, 0] = low                    # every key after the query
        table[:, 1] = low                     # every key of the second head
        dtable = torch.full_like(table, 9)
        got = _backward(q, k, v, dict(table=table, bucket_map=bmap), do, dtable)
        for n in ("o", "dq", "dk", "dv"):
            assert bool(got[n].isfinite().all()) and bool((got[n][:, :, 1] == 0).all()), n
        assert bool((dtable[5:] == 0).all()) and bool((dtable[:, 1] == 0).all())
        assert bool(dtable.isfinite().all())
        assert bool((got["lse"][:, 1] == float("-inf")).all())
        assert bool((got["dk"][:, Tq:, 0] == 0).all()) and bool((got["dv"][:, Tq:, 0] == 0).all())
        safe = torch.where(table == low, torch.zeros_like(table), table)
        want = _backward(q, k, v, dict(table=safe, bucket_map=bmap, causal=True), do,
                         torch.empty_like(table))
        for n in ("o", "dq", "dk", "dv"):
            assert torch.equal(got[n][:, :, 0], want[n][:, :, 0]), n


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("p", [0.0, 0.4])
def test_a_row_of_one_key_has_no_score_gradient(dtype, p):
    """A softmax over one key is 1 whatever the score: dq and the row's parts of
    dk and dtable are zeros, not what two roundings leave."""
    dev = device()
    g = gen(31, dev)
    bmap = rel_bucket_map(32, 128, False, dev)
    for B, H, Hkv, Tq, Tk, causal, k_len in ((3, 4, 2, 1, 1, False, None),
                                             (2, 2, 2, 70, 70, True, None),
                                             (2, 2, 1, 130, 300, False, (1, 1))):
        q, k, v = make(dtype, B, H, Hkv, Tq, Tk, 64, g, dev)
        do = torch.randn(q.shape, generator=g, device=dev).to(TYPES[dtype])
        table = torch.randn((32, H), generator=g, device=dev)
        how = dict(table=table, bucket_map=bmap, p=p, seed=SEED, step=3, causal=causal)
        if k_len is not None:
            how["k_len"] = torch.tensor(k_len, dtype=torch.int32, device=dev)
        if causal:  # a row of one key beside rows of more
            do[:, 1:] = 0
        dtable = torch.full_like(table, 9)
        got = _backward(q, k, v, how, do, dtable)
        for n in ("dq", "dk", "dtable"):
            assert bool((got[n] == 0).all()), (Tq, Tk, n, float(got[n].abs().max()))
        assert bool((got["dv"] != 0).any())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("low", [-1e4, -1e6, -1e9, 1e9, 5e11, -1e12])
def test_rows_of_one_large_bias(low, dtype):
    """A softmax does not change when all its scores do: a head whose table
    holds one large number has the outputs and gradients of a head without a
    bias, and an lse further by that number.  The references of such rows are
    rounded, which leaves |low| 2^-22 of the number in the scores at most: the
    oracle gets a table of that much, and its bounds with it.  Single queries
    and many go through different kernels."""
    dev = device()
    rest = abs(low) * 2.0 ** -22
    for n, (Tq, Tk, D, p, k_len) in enumerate((
            (1, 300, 64, 0.0, None), (3, 2000, 128, 0.2, (1500,)), (50, 80, 64, 0.2, None),
            (150, 400, 128, 0.0, (333,)), (40, 1100, 64, 0.0, None), (130, 64, 80, 0.1, None),
            (1, 5000, 128, 0.1, None), (200, 300, 64, 0.1, None))):
        g = gen(Tq + D, dev)
        q, k, v = make(dtype, 1, 2, 1, Tq, Tk, D, g, dev)
        do = torch.randn(q.shape, generator=g, device=dev).to(TYPES[dtype])
        table = torch.randn((32, 2), generator=g, device=dev)
        how = dict(scale=D ** -0.5, causal=n % 2 == 1, q_pos=Tk - Tq if n < 7 else 40, k_len=None,
                   bucket_map=rel_bucket_map(32, 40, True, dev), p=p, seed=SEED, step=17)
        if k_len is not None:
            how["k_len"] = torch.tensor(k_len, dtype=torch.int32, device=dev)
        table[:, 1] = -rest
        want, tol = _oracle(q, k, v, do, dict(table=table, **how), dtype)
        want["lse"][:, 1] += low + rest
        tol["lse"][:, 1] += 4 * 2.0 ** -24 * abs(low)
        table[:, 1] = low
        dtable = torch.full_like(table, 9.0)
        got = _backward(q, k, v, dict(table=table, **how), do, dtable)
        print(f"[attention] {low} {dtype} {Tq}x{Tk}x{D}", flush=True)
        check(got, want, tol, ("o", "lse", "dq", "dk", "dv", "dtable"), _tiny(dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("low", [-2.0 ** 40, -1e15, -1e30])
def test_rows_hidden_whole(low, dtype):
    """From -2^40 on a bias counts as -inf: its keys have no weight, a row of
    nothing else no output and no gradient, in every kernel."""
    dev = device()
    for Tq, Tk, D in ((1, 300, 64), (4, 1500, 128), (50, 80, 64), (150, 400, 128)):
        g = gen(Tq + D, dev)
        q, k, v = make(dtype, 1, 2, 2, Tq, Tk, D, g, dev)
        do = torch.randn(q.shape, generator=g, device=dev).to(TYPES[dtype])
        table = torch.randn((8, 2), generator=g, device=dev)
        table[5:, 0] = low                    # every key after the query
        table[:, 1] = low
        how = dict(q_pos=Tk // 2, bucket_map=rel_bucket_map(8, 20, True, dev))
        dtable = torch.full_like(table, 9)
        got = _backward(q, k, v, dict(table=table, **how), do, dtable)
        for n in ("o", "dq", "dk", "dv"):
            assert bool(got[n].isfinite().all()) and bool((got[n][:, :, 1] == 0).all()), n
        assert bool((got["lse"][:, 1] == float("-inf")).all())
        assert bool((dtable[5:] == 0).all()) and bool((dtable[:, 1] == 0).all())
        table[table == low] = float("-inf")
        want = _backward(q, k, v, dict(table=table, **how), do, torch.full_like(table, 9))
        for n in want:
            assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Tq", [1, 40, 150])
def test_low_biases_over_lower_products(Tq, dtype):
    """Far keys of a low bias hold all the weight where the products with the
    near keys are lower still."""
    dev = device()
    g = gen(Tq, dev)
    Tk, D = 1500, 64
    q = torch.full((1, Tq, 2, D), 8.0, device=dev).to(TYPES[dtype])
    k = torch.randn((1, Tk, 2, D), generator=g, device=dev).to(TYPES[dtype]) / 8
    v = torch.randn((1, Tk, 2, D), generator=g, device=dev).to(TYPES[dtype])
    k[:, Tk - Tq - 40:] = -64.0  # scores of -4096
    do = torch.randn(q.shape, generator=g, device=dev).to(TYPES[dtype])
    bmap = rel_bucket_map(8, 20, False, dev)
    table = torch.randn((8, 2), generator=g, device=dev)
    table[bmap[0]] = -2000.0
    how = dict(scale=D ** -0.5, causal=True, q_pos=Tk - Tq, k_len=None, table=table,
               bucket_map=bmap, p=0.1, seed=SEED, step=17)
    want, tol = _oracle(q, k, v, do, how, dtype)
    assert float(np.abs(want["lse"] + 2000).max()) < 100
    got = _backward(q, k, v, how, do, torch.empty_like(table))
    check(got, want, tol, ("o", "lse", "dq", "dk", "dv", "dtable"), _tiny(dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("low", [-1e4, -1e9, -1e12])
def test_large_biases_far_away(low, dtype):
    """Keys that a low bias hides behind others of the row count as hidden ones,
    wherever they come: first (the far keys of a decoder), last, or as all that
    a part of a split row has."""
    dev = device()
    for Tq, Tk, D, two in ((1, 3000, 128, False), (3, 500, 64, False), (100, 700, 64, False),
                           (150, 300, 128, True), (40, 1500, 64, True)):
        g = gen(Tq + D, dev)
        q, k, v = make(dtype, 1, 2, 2, Tq, Tk, D, g, dev)
        do = torch.randn(q.shape, generator=g, device=dev).to(TYPES[dtype])
        bmap = rel_bucket_map(8, 20, two, dev)
        table = torch.randn((8, 2), generator=g, device=dev)
        table[bmap[0]] = low
        table[bmap[-1] if two else bmap[0]] = low
        how = dict(q_pos=Tk // 2 if two else Tk - Tq, causal=not two, bucket_map=bmap, p=0.1,
                   seed=SEED, step=17)
        dtable = torch.full_like(table, 9)
        got = _backward(q, k, v, dict(table=table, **how), do, dtable)
        table[table == low] = float("-inf")
        want = _backward(q, k, v, dict(table=table, **how), do, torch.full_like(table, 9))
        for n in want:
            assert torch.equal(got[n], want[n]), n


@pytest.mark.parametrize("dtype,far", [("bf16", 3e2), ("f16", 3e2), ("bf16", 1e4), ("f16", 1e4),
                                       ("bf16", 1e5)])
def test_large_products(dtype, far):
    """Scores of up to 10^10 and more: each row's weight lies on one key to more
    than binary32 shows (its margin is checked), so o is that key's value, dv
    takes the rows' gradients whole, and no score has a gradient but for the
    rounding of delta."""
    dev = device()
    e = 2.0 ** -24
    for Tq, Tk, D in ((1, 200, 64), (2, 2000, 128), (50, 80, 64), (150, 300, 128)):
        g = gen(Tq + D, dev)
        q, k, v = make(dtype, 1, 2, 1, Tq, Tk, D, g, dev)
        q, k = q * far, k * far
        do = torch.randn(q.shape, generator=g, device=dev).to(TYPES[dtype])
        q64, k64, v64, do64 = (x[0].double().transpose(0, 1) for x in (q, k, v, do))
        s = q64 @ k64.transpose(1, 2) * D ** -0.5
        size = q64.abs() @ k64.abs().transpose(1, 2) * D ** -0.5
        top = s.topk(2, 2)
        off = (D + 8) * e * size.amax(2)
        sure = top.values[..., 0] - top.values[..., 1] > 2 * off + 200
        do64 = do64 * sure[..., None]
        do = do64.to(do.dtype).transpose(0, 1)[None].contiguous()  # the other rows' count 0
        got = _backward(q, k, v, {}, do, None)
        best = top.indices[..., 0]
        want = v64[0][best]
        o = got["o"][0].double().transpose(0, 1)
        assert bool(sure.any())
        assert torch.equal(o[sure], want[sure])
        lse = got["lse"][0].double()
        assert bool(((lse - top.values[..., 0]).abs() <= off + 4 * e * lse.abs()).all())
        dv = torch.zeros_like(v64[0]).index_add_(0, best[sure], do64[sure])
        size_dv = torch.zeros_like(v64[0]).index_add_(0, best[sure], do64[sure].abs())
        err = (got["dv"][0, :, 0].double() - dv).abs()
        assert bool((err <= half_step(dtype) * dv.abs() + 2 * Tq * e * size_dv).all())
        # dP is known to (D + 2) e of its terms, and delta adds one of a few
        # roundings more: dS = dP - delta of that key alone.  The row's normaliser
        # lies above a base that lse gives: as far as the scores are off, times
        # log2 e, and lse is rounded; it is rounded itself, e of that in the
        # weight, which delta takes times the distance of two dP
        high = 1.5 * (off + 4 * e * lse.abs()) + 30
        ds = (4 * (D + 8) + 2 * high) * e * (do64.abs() @ v64.abs().transpose(1, 2)).amax(2)
        dq = got["dq"][0].double().transpose(0, 1)
        bound = D ** -0.5 * ds[..., None] * k64.abs().amax((1, 2))
        assert bool((dq.abs() <= bound + _tiny(dtype)).all())
        bound = D ** -0.5 * (ds.sum() * q64.abs().max())
        assert bool((got["dk"].double().abs() <= bound + _tiny(dtype)).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("Tk", [200, 300, 1100])
def test_rows_of_one_heavy_key(Tk, dtype):
    """A row whose weight lies on one key of many has next to no score gradient.
    The query pass over more than 256 keys takes delta from the rounded output:
    dq is off by half a step of the output times the gradient, times that key.
    Over fewer keys, and in the key pass always, delta is binary32's.  The weight
    is 1 but for what lse has rounded, less than 5 times 2^-24 |lse| (its
    reference, two constants and two products), of the distance between that
    key's dP and what delta starts from."""
    dev = device()
    e, Tq, D = 2.0 ** -24, 70, 64
    g = gen(Tk, dev)
    q, k, v = make(dtype, 1, 2, 1, Tq, Tk, D, g, dev)
    q, k = q * 8, k * 8
    do = torch.randn(q.shape, generator=g, device=dev).to(TYPES[dtype])
    q64, k64, v64, do64 = (x[0].double().transpose(0, 1) for x in (q, k, v, do))
    top = (q64 @ k64.transpose(1, 2) * D ** -0.5).topk(2, 2).values
    sure = top[..., 0] - top[..., 1] > 25  # the others weigh less than 2^-25 together
    assert bool(sure.any())
    do64 = do64 * sure[..., None]
    do = do64.to(do.dtype).transpose(0, 1)[None].contiguous()
    got = _backward(q, k, v, {}, do, None)
    o64 = got["o"][0].double().transpose(0, 1)
    exact = (4 * (D + 8) + 10 * top[..., 0].abs()) * e * (
        do64.abs() @ v64.abs().transpose(1, 2)).amax(2)
    rounded = exact + half_step(dtype) * (do64 * o64).abs().sum(2) * (1 if Tk > 256 else 0)
    dq = got["dq"][0].double().transpose(0, 1).abs()
    assert bool((dq <= D ** -0.5 * rounded[..., None] * k64.abs().amax() + _tiny(dtype)).all())
    dk = got["dk"].double().abs()
    assert bool((dk <= D ** -0.5 * exact.sum() * q64.abs().max() + _tiny(dtype)).all())


def test_two_streams_at_once():
    """Calls on two streams at once, each with its own workspace (split keys,
    and a backward pass with the table's gradient), equal the same calls one
    after the other."""
    dev = device()
    g = gen(21, dev)
    bmap = rel_bucket_map(32, 64, True, dev)
    work = []
    for Tq, Tk in ((1, 9000), (300, 900)):
        q, k, v = make("bf16", 2, 4, 2, Tq, Tk, 64, g, dev)
        do = torch.randn(q.shape, generator=g, device=dev).bfloat16()
        table = torch.randn((32, 4), generator=g, device=dev)
        how = dict(table=table, bucket_map=bmap, p=0.1, seed=SEED, step=2, q_pos=Tk - Tq)
        work.append((q, k, v, how, do, [workspace(q, k, 64, True) for _ in range(2)]))
    alone = [_backward(q, k, v, how, do, torch.empty_like(how["table"]), ws=ws[0])
             for q, k, v, how, do, ws in work]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in work]
    both = [[], []]
    for _ in range(5):
        for n, (q, k, v, how, do, ws) in enumerate(work):
            with torch.cuda.stream(streams[n]):
                both[n].append(_backward(q, k, v, how, do, torch.empty_like(how["table"]),
                                         ws=ws[1]))
    torch.cuda.synchronize()
    for want, gots in zip(alone, both):
        for got in gots:
            for n in want:
                assert torch.equal(got[n], want[n]), n


def test_two_graphs_share_a_workspace():
    """The workspace holds nothing between calls: two graphs captured with the
    same one, replayed in turn, give the eager results."""
    dev = device()
    g = gen(22, dev)
    bmap = rel_bucket_map(32, 64, True, dev)
    graphs, results, inputs = [], [], []
    q0, k0, _ = make("bf16", 2, 4, 4, 1, 6000, 64, g, dev)
    ws = torch.full((max(workspace(q0, k0, 64, True).numel(), 1 << 22),), 0xFF, dtype=torch.uint8,
                    device=dev)
    for Tq, Tk in ((1, 6000), (129, 130)):
        q, k, v = make("bf16", 2, 4, 4, Tq, Tk, 64, g, dev)
        table = torch.randn((32, 4), generator=g, device=dev)
        do = torch.randn(q.shape, generator=g, device=dev).bfloat16()
        inputs.append((q, k, v, dict(table=table, bucket_map=bmap), do))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            _backward(*inputs[-1], torch.empty_like(table), ws=ws)
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            results.append(_backward(*inputs[-1], torch.empty_like(table), ws=ws))
        graphs.append(graph)
    for t in range(4):
        for n, (q, k, v, how, do) in enumerate(inputs):
            q.copy_(torch.randn(q.shape, generator=g, device=dev))
            graphs[n].replay()
            torch.cuda.synchronize()
            want = _backward(q, k, v, how, do, torch.empty_like(how["table"]))
            torch.cuda.synchronize()
            for x in want:
                assert torch.equal(results[n][x], want[x]), (t, n, x)


def test_largest_token_strides():
    """Tokens 2^23 elements apart, the last of them past 32-bit offsets."""
    dev = device()
    g = gen(23, dev)
    store = torch.zeros(300 * (1 << 23), dtype=torch.bfloat16, device=dev)  # 5 GB
    apart = store.as_strided((1, 300, 2, 64), (0, 1 << 23, 64, 1))
    for Tq in (1, 40):
        q, k, v = make("bf16", 1, 2, 2, Tq, 300, 64, g, dev)
        apart.copy_(k)
        o, want = torch.empty_like(q), torch.empty_like(q)
        ob.rel_attention_forward(q, apart, v, o, ws=workspace(q, k))
        ob.rel_attention_forward(q, k, v, want, ws=workspace(q, k))
        assert torch.equal(o, want)


def test_nothing_to_attend_or_ask():
    dev = device()
    q = torch.randn((2, 5, 2, 16), device=dev).bfloat16()
    k = torch.empty((2, 0, 2, 16), device=dev).bfloat16()
    o, lse = torch.full_like(q, 7), torch.full((2, 2, 5), 7.0, device=dev)
    ob.rel_attention_forward(q, k, k, o, lse=lse)
    assert bool((o == 0).all()) and bool((lse == float("-inf")).all())
    dq, dk = torch.full_like(q, 7), torch.empty_like(k)
    bmap = rel_bucket_map(8, 20, True, dev)
    table = torch.randn((8, 2), device=dev)
    dtable = torch.full_like(table, 7)
    ob.rel_attention_backward(q, k, k, o, lse, q, dq, dk, dk, table=table, bucket_map=bmap,
                              dtable=dtable, ws=workspace(q, k, 20, True))
    assert bool((dq == 0).all()) and bool((dtable == 0).all())
    # no queries: the keys' gradients are zeros
    dkv = [torch.full_like(q, 7) for _ in range(2)]
    e, el = q[:, :0], lse[:, :, :0]
    dtable.fill_(7)
    ob.rel_attention_forward(e, q, q, e, lse=el.contiguous())
    ob.rel_attention_backward(e, q, q, e, el.contiguous(), e, e, *dkv, table=table,
                              bucket_map=bmap, dtable=dtable, ws=workspace(e, q, 20, True))
    assert all(bool((x == 0).all()) for x in dkv) and bool((dtable == 0).all())


@pytest.mark.parametrize("p", [0.0, 0.2])
def test_replayed_graph_matches_eager(p):
    """Forward and backward captured together; every replay, with eager work
    between, equals the eager calls, and the mask follows the device step."""
    dev = device()
    g = gen(12, dev)
    q, k, v = make("bf16", 2, 2, 2, 100, 100, 64, g, dev)
    do = torch.randn(q.shape, generator=g, device=dev).bfloat16()
    bmap = rel_bucket_map(32, 40, True, dev)
    table = torch.randn((32, 2), generator=g, device=dev)
    step = torch.zeros(1, dtype=torch.int32, device=dev)
    how = dict(table=table, bucket_map=bmap, p=p, seed=SEED)

    def both(out, ws, **more):
        ob.rel_attention_forward(q, k, v, out["o"], lse=out["lse"], ws=ws, **how, **more)
        ob.rel_attention_backward(q, k, v, out["o"], out["lse"], do, out["dq"], out["dk"],
                                  out["dv"], dtable=out["dtable"], ws=ws, **how, **more)

    def buffers():
        return dict(o=torch.empty_like(q), lse=torch.empty((2, 2, 100), device=dev),
                    dq=torch.empty_like(q), dk=torch.empty_like(k), dv=torch.empty_like(v),
                    dtable=torch.empty_like(table))

    mine, theirs = buffers(), buffers()
    ws, ws2 = workspace(q, k, 40, True), workspace(q, k, 40, True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both(mine, ws, step=5, step_dev=step)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both(mine, ws, step=5, step_dev=step)
    for t in range(4):
        step.fill_(t)
        q.copy_(torch.randn(q.shape, generator=g, device=dev))
        graph.replay()
        torch.cuda.synchronize()
        both(theirs, ws2, step=5 + t)
        torch.cuda.synchronize()
        for n in mine:
            assert torch.equal(mine[n], theirs[n]), (t, n)


@pytest.mark.parametrize("Tq", [1, 40])
def test_a_long_cache(Tq):
    """200 001 keys: a token's row and a few more against 64 bits."""
    dev = device()
    g = gen(24, dev)
    Tk, H, D = 200_001, 2, 128
    q, k, v = make("bf16", 1, H, 1, Tq, Tk, D, g, dev)
    bmap = rel_bucket_map(32, 128, False, dev)
    table = torch.randn((32, H), generator=g, device=dev)
    o, lse = torch.empty_like(q), torch.empty((1, H, Tq), device=dev)
    pos = Tk - Tq
    ob.rel_attention_forward(q, k, v, o, lse=lse, causal=True, q_pos=pos, table=table,
                             bucket_map=bmap, ws=workspace(q, k))
    kd, vd = k[0, :, 0].double(), v[0, :, 0].double()
    j = torch.arange(Tk, device=dev)
    for i in {0, Tq // 2, Tq - 1}:
        d = (j - i - pos).clamp(-128, 128) + 128
        for h in range(H):
            qd = q[0, i, h].double()
            s = kd @ qd * D ** -0.5 + table[bmap[d].long(), h].double()
            s[j > i + pos] = float("-inf")
            want = torch.softmax(s, 0)[None] @ vd
            # the row's scores are off by (D + 8) e (|scores| + |terms|) < 2^-15
            # in all, its sum by the additions of a split, a wave and a lane
            # (fewer than 2^10), so weights by 2^-12 beside their rounding
            bound = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * (
                torch.softmax(s, 0)[None] @ vd.abs())
            assert bool(((o[0, i, h].double() - want[0]).abs() <= bound[0]).all()), (i, h)
            assert abs(float(lse[0, h, i]) - float(torch.logsumexp(s, 0))) < 2.0 ** -12
