"""Pins of the block operators' plain forms: against torch's float64 operators,
differences, and the 8-bit formats as torch defines them."""

import numpy as np
import pytest
import torch

from oracle import block as ref

RNG = np.random.default_rng(7)


def test_layer_norm_and_its_gradient():
    x, dy, w, b = (RNG.standard_normal(s) for s in ((5, 33), (5, 33), (33,), (33,)))
    t = [torch.from_numpy(a).requires_grad_() for a in (x, w, b)]
    eps = float(np.float32(1e-3))
    y = torch.nn.functional.layer_norm(t[0], (33,), t[1], t[2], eps)
    y.backward(torch.from_numpy(dy))
    got, mean, rstd = ref.layer_norm(x, w, b, 1e-3)
    dx, dw, db = ref.layer_norm_grad(dy, x, mean, rstd, w)
    for a, want in ((got, y.detach()), (dx, t[0].grad), (dw, t[1].grad), (db, t[2].grad)):
        np.testing.assert_allclose(a, want.numpy(), rtol=1e-11, atol=1e-12)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
def test_linear_and_its_gradients(act):
    x, w, b, r, dy = (RNG.standard_normal(s) for s in ((6, 9), (7, 9), (7,), (6, 7), (6, 7)))
    f = {"none": lambda z: z, "relu": torch.relu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh"),
         "silu": torch.nn.functional.silu}[act]
    t = [torch.from_numpy(a).requires_grad_() for a in (x, w, b)]
    z = torch.nn.functional.linear(*t)
    y = f(z) + torch.from_numpy(r)
    y.backward(torch.from_numpy(dy))
    got, pre = ref.linear(x, w, b, act, r)
    dx, dw, db, _ = ref.linear_grad(dy, x, w, act, pre)
    for a, want in ((got, y.detach()), (pre, z.detach()), (dx, t[0].grad), (dw, t[1].grad),
                    (db, t[2].grad)):
        np.testing.assert_allclose(a, want.numpy(), rtol=1e-9, atol=1e-10)
    # the slope against differences of the activation
    u, h = np.linspace(-6, 6, 101) + 0.003, 1e-5
    d = (ref.activate(u + h, act) - ref.activate(u - h, act)) / (2 * h)
    np.testing.assert_allclose(ref.slope(u, act), d, atol=1e-8)


@pytest.mark.parametrize("digits,kind", [(3, torch.float8_e4m3fn), (2, torch.float8_e5m2)])
def test_formats(digits, kind):
    """Every code's value is torch's, and a value on the grid keeps its code for
    any draw."""
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(kind).float().numpy()
    got = ref.decode(codes, digits)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    assert np.array_equal(got[ok].view(np.uint32), want[ok].view(np.uint32))
    # codes below the block's top binade, with its first value as the largest
    top = {3: 0x70, 2: 0x74}[digits]  # 2^7, 2^14
    some = np.concatenate([[top], np.arange(top)]).astype(np.uint8)
    x = ref.decode(some, digits) * np.float32(2.0 ** -20)
    for draw in (0, 1, 32768, 65535):
        c, s = ref.encode(x, np.full(x.size, draw, np.uint32), digits, False)
        assert np.array_equal(c, some) and np.all(s == np.float32(2.0 ** -20))


def test_rounding_of_the_states():
    """Between two codes the share of the upper one is the distance to the lower
    one, to half a draw; a variance above 0 keeps a code above 0."""
    u = np.arange(65536, dtype=np.uint32)
    for digits, positive in ((3, False), (2, True)):
        base = ref.decode(np.array([33], np.uint8), digits)[0]
        up = ref.decode(np.array([34], np.uint8), digits)[0]
        big = np.float32(2.0 ** (7 if digits == 3 else 14))
        for share in (0.25, 0.5, 0.90625):
            x = np.full(65536, np.float32(base + share * (up - base)), np.float32)
            x[::256] = big
            c, s = ref.encode(x, u, digits, positive)
            assert np.all(s == 1)
            rest = np.arange(65536) % 256 != 0
            assert abs((c[rest] == 34).mean() - share) < 0.01
            assert set(c[rest]) == {33, 34}
            # the signs are alike
            if not positive:
                n, _ = ref.encode(-x, u, digits, positive)
                assert np.array_equal(n, c | 0x80)
    v = np.array([1.0] + [1e-30] * 7, np.float32)
    c, _ = ref.encode(v, np.zeros(8, np.uint32), 2, True)
    assert np.all(c[1:] == 1)
    c, _ = ref.encode(np.zeros(8, np.float32), np.full(8, 65535, np.uint32), 2, True)
    assert np.all(c == 0)


def test_adamw_is_adamw():
    """Against torch's optimizer in float64, over some steps, within binary32's
    roundings."""
    n = 50
    x = RNG.standard_normal(n).astype(np.float32)
    p = torch.from_numpy(x.astype(np.float64)).requires_grad_()
    hp = dict(lr=float(np.float32(1e-2)), betas=(float(np.float32(.9)), float(np.float32(.999))),
              eps=float(np.float32(1e-8)), weight_decay=float(np.float32(.1)))
    opt = torch.optim.AdamW([p], **hp)
    m = v = np.zeros(n, np.float32)
    for t in range(1, 8):
        g = RNG.standard_normal(n).astype(np.float32)
        p.grad = torch.from_numpy(g.astype(np.float64))
        opt.step()
        x, m, v = ref.adamw(x, g, m, v, 1e-2, .9, .999, 1e-8, t, weight_decay=.1)
        # a dozen roundings a step
        np.testing.assert_allclose(x, p.detach().numpy(), rtol=0, atol=t * 12 * 2.0 ** -24 * 3)


def test_draws_are_apart():
    """Tensors, steps and seeds have draws of their own, and a tensor's first draws
    do not depend on its length."""
    base = ref.draws(4096, 0, 1, 5)
    for other in (ref.draws(4096, 1, 1, 5), ref.draws(4096, 0, 2, 5), ref.draws(4096, 0, 1, 6)):
        assert (base == other).mean() < 0.01
    assert np.array_equal(ref.draws(100, 0, 1, 5), base[:100])
