"""rel_bias_expand (exact) and rel_bias_grad (within its binary32 sums)
against the 64-bit forms."""

import numpy as np
import pytest
import torch

from momentum_compression_amd import onebit as ob
from momentum_compression_amd.attention import rel_bucket_map
from oracle import training as ref
from tests._gpu import device, gen, host

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("H,Tq,Tk,pos,n,far", [(1, 1, 1, 0, 4, 8), (3, 1, 8191, 8190, 32, 128),
                                               (2, 37, 53, 0, 8, 20), (5, 130, 257, 127, 32, 128),
                                               (1, 70, 9, -40, 32, 40), (2, 64, 64, 5, 64, 1024),
                                               (2, 16, 40, 10 ** 8, 4, 8)])
def test_expand_is_the_table(dtype, H, Tq, Tk, pos, n, far):
    dev = device()
    print(f"[bias] {dtype} H={H} {Tq}x{Tk} pos={pos} n={n} far={far}", flush=True)
    bmap = rel_bucket_map(n, far, True, dev)
    table = torch.randn((n, H), generator=gen(n + Tk, dev), device=dev)
    out = torch.full((H * Tq * Tk + 1,), 3.0, dtype=TYPES[dtype], device=dev)
    ob.rel_bias_expand(table, bmap, out[:-1].view(H, Tq, Tk), q_pos=pos)
    want = ref.rel_bias(table.double().cpu().numpy(), bmap.cpu().numpy(), Tq, Tk, pos)
    want = torch.from_numpy(want).float().to(TYPES[dtype])
    assert torch.equal(out[:-1].view(H, Tq, Tk).cpu(), want)
    assert float(out[-1]) == 3.0


def test_expand_bucket_outside_the_table_is_no_bias():
    dev = device()
    bmap = torch.tensor([-1, 0, 5, 1, 2 ** 31 - 1], dtype=torch.int32, device=dev)
    table = torch.randn((2, 3), generator=gen(1, dev), device=dev)
    out = torch.empty((3, 9, 9), device=dev)
    ob.rel_bias_expand(table, bmap, out)
    want = ref.rel_bias(table.double().cpu().numpy(), bmap.cpu().numpy(), 9, 9)
    assert np.array_equal(out.double().cpu().numpy(), want)
    d = torch.empty_like(table)
    ds = torch.ones((1, 3, 9, 9), device=dev)
    ws = torch.empty(ob.rel_bias_workspace_bytes(1, 3, 9, 9, 2), dtype=torch.uint8, device=dev)
    ob.rel_bias_grad(ds, bmap, d, ws=ws)
    assert np.array_equal(d.double().cpu().numpy(),
                          ref.rel_bias_grad(ds.cpu().numpy(), bmap.cpu().numpy(), 2))


def _tolerance(ds, bmap, n, pos, B, Tq, Tk):
    """binary32 additions that a term passes through: 8 rows of each sequence
    of the part, 6 + 1 shuffles, the bins of Tq / 32 row groups (15 sums each
    where they all lie beyond the radius), 6 more shuffles and 2 waves; each
    off by at most 2^-24 of a sum that the terms' sizes bound."""
    depth = 8 * B + 15 * (Tq // 32 + 1) + 16
    size = ref.rel_bias_grad(np.abs(ds), bmap, n, pos)
    return depth * 2.0 ** -24 * 1.01 * size + 1e-30


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("B,H,Tq,Tk,pos,n,far", [
    (1, 1, 1, 1, 0, 4, 8), (3, 2, 1, 700, 699, 32, 128), (9, 3, 37, 37, 0, 8, 20),
    (5, 2, 64, 65, 0, 32, 128), (17, 1, 33, 129, 96, 32, 40), (2, 2, 130, 521, 0, 32, 128),
    (1, 3, 257, 1100, 843, 64, 1024), (2, 1, 100, 9, -40, 32, 40)])
def test_grad_sums(dtype, B, H, Tq, Tk, pos, n, far):
    dev = device()
    print(f"[bias grad] {dtype} B={B} H={H} {Tq}x{Tk} pos={pos} n={n} far={far}", flush=True)
    bmap = rel_bucket_map(n, far, True, dev)
    ds = torch.randn((B, H, Tq, Tk), generator=gen(B + Tk, dev), device=dev).to(TYPES[dtype])
    got = torch.full((n, H), 5.0, device=dev)
    ws = torch.empty(ob.rel_bias_workspace_bytes(B, H, Tq, Tk, far), dtype=torch.uint8, device=dev)
    ws.fill_(0xFF)  # scratch: whatever it held
    ob.rel_bias_grad(ds, bmap, got, q_pos=pos, ws=ws)
    ds64, m = ds.double().cpu().numpy(), bmap.cpu().numpy()
    want = ref.rel_bias_grad(ds64, m, n, pos)
    err = np.abs(got.double().cpu().numpy() - want)
    tol = _tolerance(ds64, m, n, pos, B, Tq, Tk) + 2.0 ** -24 * np.abs(want)
    assert (err <= tol).all(), f"{(err - tol).max()}"
    again = got.clone()
    ob.rel_bias_grad(ds, bmap, again, q_pos=pos, ws=ws)
    assert torch.equal(again, got)
    ob.rel_bias_grad(ds, bmap, again, q_pos=pos, accumulate=True, ws=ws)
    # want is added to the first result in binary64 and rounded once
    twice = np.abs(again.double().cpu().numpy() - 2 * want)
    assert (twice <= 2 * tol + 2.0 ** -24 * np.abs(2 * want)).all()


def test_grad_of_nothing_is_zero():
    dev = device()
    bmap = rel_bucket_map(8, 20, True, dev)
    got = torch.full((8, 3), 5.0, device=dev)
    ws = torch.empty(256, dtype=torch.uint8, device=dev)
    ob.rel_bias_grad(torch.empty((0, 3, 4, 4), device=dev), bmap, got, accumulate=True, ws=ws)
    assert bool((got == 5).all())
    ob.rel_bias_grad(torch.empty((2, 3, 4, 0), device=dev), bmap, got, ws=ws)
    assert bool((got == 0).all())


def test_more_scores_than_32_bits_count():
    """Ones over 2^31 scores and more: every bucket's sum is its count.  Counts
    of a workgroup stay below 2^24, so binary32 has them exactly."""
    dev = device()
    B, H, Tq, Tk, far = 9, 16, 4100, 3700, 128
    ds = torch.ones((B, H, Tq, Tk), dtype=torch.bfloat16, device=dev)
    assert ds.numel() > 2 ** 31
    bmap = rel_bucket_map(32, far, True, dev)
    dtable = torch.empty((32, H), device=dev)
    ws = torch.empty(ob.rel_bias_workspace_bytes(B, H, Tq, Tk, far), dtype=torch.uint8, device=dev)
    ob.rel_bias_grad(ds, bmap, dtable, ws=ws)
    d = np.arange(-Tq + 1, Tk)
    times = np.minimum.reduce([d + Tq, Tk - d, np.full(d.size, min(Tq, Tk))])
    count = np.bincount(bmap.cpu().numpy()[np.clip(d, -far, far) + far], weights=times,
                        minlength=32) * B
    assert count.sum() == B * Tq * Tk
    assert np.array_equal(host(dtable), np.repeat(count.astype(np.float32)[:, None], H, 1))


@pytest.mark.parametrize("B", [(1 << 30) + 1, (1 << 31) - 1])
def test_more_sequences_than_2_30(B):
    """Scores of one query and key: one bucket, whose sum takes in the first
    and the last sequence and those about the parts' middle (whole numbers, of
    which a part's sums stay exact)."""
    dev = device()
    ds = torch.zeros((B, 1, 1, 1), dtype=torch.bfloat16, device=dev)
    for at, x in ((0, 3.0), (1 << 28, 5.0), (B // 2, 7.0), (B - 2, 11.0), (B - 1, 13.0)):
        ds[at] = x
    bmap = rel_bucket_map(4, 8, True, dev)
    dtable = torch.full((4, 1), 9.0, device=dev)
    ws = torch.empty(ob.rel_bias_workspace_bytes(B, 1, 1, 1, 8), dtype=torch.uint8, device=dev)
    ob.rel_bias_grad(ds, bmap, dtable, ws=ws)
    assert dtable[:, 0].tolist() == [39.0, 0.0, 0.0, 0.0]
