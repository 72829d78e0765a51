"""Weight gradients grouped by expert where every expert ends inside a k-block and its neighbours' rows are no numbers:
more tiles than the device takes at once, so that every stage of the ring holds such blocks in turn.

Tolerance as for the products: (K + K/128 + 8) 2^-23 of the terms' magnitudes, K an expert's rows rounded up to whole
blocks."""

import pytest
import torch

from collective_fusedallreduce_gb300 import coco

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("top", [63, 130, 700])
def test_neighbours_that_are_no_numbers_stay_out(dtype, top):
    experts, k, n = 90, 520, 1032
    g = torch.Generator().manual_seed(701 + top)
    counts = torch.randint(1, top + 1, (experts,), generator=g)
    counts[counts % 64 == 0] += 1
    rows = int(counts.sum())
    off = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    g = torch.Generator(device=DEV).manual_seed(702)
    x = torch.randn(rows, k, generator=g, device=DEV).to(dtype)
    dy = torch.randn(rows, n, generator=g, device=DEV).to(dtype)
    bad_x, bad_dy = x.clone(), dy.clone()
    for e in range(1, experts, 2):
        bad_x[off[e]:off[e + 1]] = float("nan")
        bad_dy[off[e]:off[e + 1]] = float("inf")
    out = torch.empty(experts, k, n, device=DEV)
    for _ in range(3):
        out.fill_(float("nan"))
        coco.coco_grouped_einsum("tk,tn->ekn", coco.local([bad_x]), None, coco.local([bad_dy]), None,
                                 off.to(DEV, torch.int32), coco.local([out]))
        coco.coco_device_status()
        for e in range(0, experts, 2):
            a, b = x[off[e]:off[e + 1]].double(), dy[off[e]:off[e + 1]].double()
            depth = -(-int(counts[e]) // 64) * 64
            bound = (depth + depth // 128 + 8) * 2.0 ** -23 * (a.abs().T @ b.abs())
            assert bool(((out[e].double() - a.T @ b).abs() <= bound + 1e-30).all()), e


@pytest.mark.parametrize("valid", list(range(1, 64)))
def test_every_number_of_rows_in_the_last_block(valid):
    k, n = 136, 264
    g = torch.Generator(device=DEV).manual_seed(703)
    counts = [valid, 64 + valid, 5]
    rows = sum(counts)
    x = torch.randn(rows, k, generator=g, device=DEV).bfloat16()
    dy = torch.randn(rows, n, generator=g, device=DEV).bfloat16()
    off = torch.tensor([0, valid, 64 + 2 * valid, rows], dtype=torch.int32, device=DEV)
    out = torch.full((3, k, n), float("nan"), device=DEV)
    coco.coco_grouped_einsum("tk,tn->ekn", coco.local([x]), None, coco.local([dy]), None, off, coco.local([out]))
    coco.coco_device_status()
    for e in range(3):
        a, b = x[off[e]:off[e + 1]].double(), dy[off[e]:off[e + 1]].double()
        bound = (128 + 9) * 2.0 ** -23 * (a.abs().T @ b.abs())
        assert bool(((out[e].double() - a.T @ b).abs() <= bound + 1e-30).all()), e
