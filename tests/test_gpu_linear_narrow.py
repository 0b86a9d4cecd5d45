"""linear_backward where a matrix has fewer than eight columns and the others' rows
are not whole 16-byte chunks; the workspace lies inside a larger buffer, whose bytes
around it stay."""

import pytest
import torch

from momentum_compression_amd import onebit as ob
from tests._gpu import device
from tests.test_gpu_linear import TYPES, check_backward, inputs, workspace

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M,N,K", [(64, 12, 4), (300, 1003, 1), (40, 9, 7), (40, 4, 20), (33, 7, 9),
                                   (2, 11, 3), (1, 13, 5), (700, 259, 6), (513, 3, 1003)])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_few_columns(dtype, M, N, K, act):
    dev = device()
    print(f"[linear] narrow {dtype} {M}x{N}x{K} {act}", flush=True)
    x, w, _, dy, pre = inputs(M, N, K, dtype, dev)
    n = ob.linear_workspace_bytes(M, N, K, True)
    room = torch.full((n + 512,), 0xFF, dtype=torch.uint8, device=dev)
    dx, db = torch.empty_like(x), torch.empty(N, device=dev)
    for dw_type in (torch.float32, TYPES[dtype]):
        dw = torch.empty(N, K, dtype=dw_type, device=dev)
        ob.linear_backward(dy, x, w, dx=dx, dw=dw, dbias=db, activation=act, pre=pre,
                           ws=room[256:256 + n])
        check_backward(dy, x, w, act, pre, dx, dw, db, f"{M}x{N}x{K}")
        assert bool((room[:256] == 0xFF).all()) and bool((room[256 + n:] == 0xFF).all())
    # each alone, from views that start on no 16 bytes
    wide = torch.full((M, N + 3), float("nan"), dtype=dy.dtype, device=dev)
    wide[:, 1:1 + N] = dy
    for name, want in (("dx", dx), ("dw", dw), ("dbias", db)):
        got = torch.empty_like(want)
        ob.linear_backward(wide[:, 1:1 + N], x, w, **{name: got}, activation=act, pre=pre,
                           ws=workspace(M, N, K, True, dev))
        check_backward(dy, x, w, act, pre, got if name == "dx" else None,
                       got if name == "dw" else None, got if name == "dbias" else None, name)
