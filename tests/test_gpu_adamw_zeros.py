"""AdamW where parameters and first moments are zeros of either sign: the signs are
those of the formula's operations, one rounding each."""

import numpy as np
import pytest
import torch

from momentum_compression_amd.state import AdamW
from oracle import block as ref
from tests._gpu import device

pytestmark = pytest.mark.gpu

HP = dict(lr=2e-3, beta1=0.9, beta2=0.999, eps=1e-8)


def bits_of(a):
    return a.cpu().numpy().view(np.uint32)


@pytest.mark.parametrize("decay", [0.0, 0.5])
@pytest.mark.parametrize("v0", [0.0, 1e-3])
def test_signs_of_zeros(decay, v0):
    dev = device()
    values = [(x, g, m) for x in (0.0, -0.0, 0.5) for g in (0.0, -0.0, 0.25) for m in (0.0, -0.0, -0.125)]
    n = 8192  # whole waves: elements past a tensor's end take the general division
    x, g, m = (np.resize(np.array([v[k] for v in values], np.float32), n) for k in range(3))
    v = np.full(n, v0, np.float32)
    to = lambda a: torch.from_numpy(a.copy()).to(dev)  # noqa: E731
    opt = AdamW.create([to(x)], [to(g)], weight_decay=decay, state={"m": [to(m)], "v": [to(v)]})
    opt.step(**HP)
    torch.cuda.synchronize()
    want = ref.adamw(x, g, m, v, step=1, weight_decay=decay, **HP)
    assert (np.signbit(want[0]) & (want[0] == 0)).any() and (~np.signbit(want[0]) & (want[0] == 0)).any()
    for got, w, name in zip((opt.params[0], opt.m[0], opt.v[0]), want, "xmv"):
        bad = bits_of(got) != w.view(np.uint32)
        assert not bad.any(), (name, int(bad.sum()), x[bad][0], g[bad][0], m[bad][0])
