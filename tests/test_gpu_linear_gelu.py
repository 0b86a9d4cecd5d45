"""GELU and its slope far below 0, where both are small: relative to themselves."""

import numpy as np
import pytest
import torch

from momentum_compression_amd import onebit as ob
from oracle import block as ref
from tests._gpu import device
from tests.test_gpu_linear import TYPES, close, h64, half, least, workspace

pytestmark = pytest.mark.gpu

# the tail and the exponential: 4e-6 of themselves, and the exponential's argument
# (up to 104 in powers of two at |z| = 12), whose two roundings give 2 104 2^-24 ln 2
REL = 4e-6 + 2 * 104 * 2.0 ** -24 * 0.7 + 4 * 2.0 ** -24


@pytest.mark.parametrize("dtype", TYPES)
def test_negative_sums(dtype):
    dev, t = device(), TYPES[dtype]
    z = torch.linspace(-12, -0.01, 20011, device=dev).to(t).view(-1, 1)
    w = torch.ones(1, 1, device=dev, dtype=t)
    y, dx, dy = torch.empty_like(z), torch.empty_like(z), torch.ones_like(z)
    ws = workspace(len(z), 1, 1, True, dev)
    ob.linear_forward(z, w, y, activation="gelu", ws=ws)
    Z = h64(z)
    want = ref.activate(Z, "gelu")
    close(y, want, (REL + half(t) * (1 + REL)) * np.abs(want) + least(t), "gelu")
    ob.linear_backward(dy, z, w, dx=dx, activation="gelu", pre=z, ws=ws)
    want = ref.slope(Z, "gelu")
    parts = ref._phi(Z) + np.abs(Z) * np.exp(-Z * Z / 2) / np.sqrt(2 * np.pi)
    # dz is taken in two parts: 2^-15 of it or 2^-25
    tol = REL * parts + 2.0 ** -15 * np.abs(want) + 2 * least(t)
    close(dx, want, tol + half(t) * (np.abs(want) + tol) + least(t), "slope")
