"""AdamW whose gradients are set anew while steps on another stream have not run."""

import pytest
import torch

from momentum_compression_amd.state import AdamW
from tests._gpu import device, gen

pytestmark = pytest.mark.gpu

HP = dict(lr=2e-3, beta1=0.9, beta2=0.999, eps=1e-8)


@pytest.mark.parametrize("given", ["object", "handle", "current"])
@pytest.mark.parametrize("bits", [32, 8])
def test_set_grads_behind_a_busy_stream(bits, given):
    """Steps that wait on their stream use the gradients that they were enqueued with,
    however often others are set in the meantime."""
    dev = device()
    sizes = [5000, 300, 1, 2049]
    g = gen(3, dev)
    params = [torch.randn(n, generator=g, device=dev) for n in sizes]
    sets = [[torch.randn(n, generator=g, device=dev) for n in sizes] for _ in range(5)]
    late = AdamW.create([p.clone() for p in params], sets[0], bits=bits, seed=3)
    plain = AdamW.create([p.clone() for p in params], sets[0], bits=bits, seed=3)
    big = torch.randn((8192, 8192), generator=g, device=dev)
    out = torch.empty_like(big)
    torch.mm(big, big, out=out)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    done = torch.cuda.Event()
    with torch.cuda.stream(side):
        for _ in range(8):  # tens of milliseconds
            torch.mm(big, big, out=out)
        done.record(side)
    seen = set()
    for k, grads in enumerate(sets):
        if k:
            late.set_grads(grads)
        assert late.plan.plan.data_ptr() not in seen or done.query()
        seen.add(late.plan.plan.data_ptr())
        if given == "current":
            with torch.cuda.stream(side):
                late.step(**HP)
        else:
            late.step(stream=side if given == "object" else side.cuda_stream, **HP)
    side.synchronize()
    for k, grads in enumerate(sets):
        if k:
            plain.set_grads(grads)
        plain.step(**HP)
    torch.cuda.synchronize()
    for a, b in zip(late.params + late.m + late.v, plain.params + plain.m + plain.v):
        assert torch.equal(a, b)
