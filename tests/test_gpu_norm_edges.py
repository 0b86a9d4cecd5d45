"""Layer norm's backward pass over rows so long that one workgroup for each 64 columns
would be more threads than a launch holds."""

import pytest
import torch

from momentum_compression_amd import onebit as ob
from tests._gpu import device, gen

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,cols", [(1, (1 << 27) + 5), (2, (1 << 29) - 3)])
def test_longest_rows(rows, cols):
    dev = device()
    print(f"[norm] {rows}x{cols}", flush=True)
    g = gen(1, dev)
    x = torch.randn((rows, cols), generator=g, device=dev, dtype=torch.bfloat16)
    dy = torch.randn((rows, cols), generator=g, device=dev, dtype=torch.bfloat16)
    mean = torch.tensor([0.25, -0.5], device=dev)[:rows].contiguous()
    rstd = torch.tensor([1.5, 0.75], device=dev)[:rows].contiguous()
    dw, db = torch.full((cols,), 2.0, device=dev), torch.empty(cols, device=dev)
    ws = torch.empty(ob.layer_norm_workspace_bytes(rows, cols), dtype=torch.uint8, device=dev)
    ob.layer_norm_backward(dy, x, mean, rstd, rows, cols, dbias=db, ws=ws)
    ob.layer_norm_backward(dy, x, mean, rstd, rows, cols, dweight=dw, accumulate=True, ws=ws)
    # a row's terms in binary32, one rounding an operation; the rows' sum in binary64
    for at in range(0, cols, 1 << 26):
        s = slice(at, min(cols, at + (1 << 26)))
        G, X = dy[:, s].float(), x[:, s].float()
        h = (X - mean[:, None]) * rstd[:, None]
        assert torch.equal(db[s], G.double().sum(0).float()), at
        assert torch.equal(dw[s], (2.0 + (G * h).double().sum(0)).float()), at
