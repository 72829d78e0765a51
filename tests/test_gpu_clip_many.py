"""Clipping of lists with more buckets than the device has warps: every warp takes several, the next one's entries under way
while one is summed, from one table or from two. Compared on the device with float64.

Tolerances as test_gpu_clip's: the norm within 40 e; a scaled value 50 e and one rounding; a sum over n ranks (n + 1) e of its
terms' magnitudes and one rounding, and so its norm."""

import pytest
import torch

from collective_fusedallreduce_gb300 import coco
from test_gpu_clip import INF, Guarded, like, space
from test_gpu_llm_norm import DEV, E, TINY, U

pytestmark = pytest.mark.gpu
# some 12 600 buckets, tensors that end inside one among them (a device has up to 4864 warps for them)
SIZES = [3000017, 1, 2097152, 1023, 1024, 1025, 31, 4000003, 513, 2000000, 7, 1500001] + [1000 * k + 3 for k in range(24)]


def gradients(n, dtype, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return Guarded([[torch.randn(s, generator=g, device=DEV).to(dtype) for s in SIZES] for _ in range(n)])


def flat(row):
    return torch.cat(row).double()


def near(got, want, dtype, more=0.0):
    over = (got - want).abs() - (want.abs() * (U[dtype] * 1.01 + 50 * E) + TINY[dtype] + more)
    assert float(over.max()) <= 0, (float(over.max()), int(over.argmax()))


@pytest.mark.parametrize("dtype,out_dtype", [(torch.bfloat16, torch.float32), (torch.float16, torch.bfloat16),
                                             (torch.float32, torch.float16), (torch.float32, torch.float32)])
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 8, 11])
def test_allreduce_clip(dtype, out_dtype, n):
    g = gradients(n, dtype, 911)
    out = like(g.tensors, 2, out_dtype)
    total = sum(flat(row) for row in g.tensors) / n
    lost = (n + 2) * E * sum(flat(row).abs() for row in g.tensors) / n
    norm64 = float(total.norm())
    dn = 40 * E * norm64 + float((total.abs() * U[out_dtype] + lost + TINY[out_dtype]).norm())
    ws, norm = space()
    for share in (0.5, 2.0):
        coco.coco_scattered_allreduce_clip(g.plan, 1.0 / n, share * norm64, out.plan, norm, ws)
        coco.coco_device_status()
        g.check(), out.check()
        assert abs(float(norm) - norm64) <= dn
        want = total * min(1.0, share)
        more = want.abs() * (dn / norm64 + U[out_dtype]) * 1.01 + lost + TINY[out_dtype]
        near(flat(out.tensors[0]), want, out_dtype, more)
        assert all(torch.equal(x, y) for x, y in zip(*out.tensors))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n", [3, 5, 8])
def test_allreduce_clip_in_place(dtype, n):
    g, h = gradients(n, dtype, 912), gradients(n, dtype, 912)
    out = like(g.tensors, 1, dtype)
    ws, norm = space()
    for top in (INF, 3.0):
        coco.coco_scattered_allreduce_clip(g.plan, 1.0 / n, top, out.plan, norm, ws)
        again = torch.empty_like(norm)
        coco.coco_scattered_allreduce_clip(h.plan, 1.0 / n, top, None, again, ws)
        coco.coco_device_status()
        h.check()
        assert torch.equal(norm, again)
        for row in h.tensors:
            assert all(torch.equal(x, y) for x, y in zip(row, out.tensors[0]))
        h = gradients(n, dtype, 912)


@pytest.mark.parametrize("dtype,out_dtype", [(torch.bfloat16, torch.float32), (torch.float16, None), (torch.float32, torch.bfloat16),
                                             (torch.float32, None)])
@pytest.mark.parametrize("layout,n", [(coco.LOCAL, 1), (coco.LOCAL, 3), (coco.REPLICATED, 1), (coco.REPLICATED, 2)])
def test_clip(dtype, out_dtype, layout, n):
    g = gradients(n, dtype, 913)
    if layout == coco.REPLICATED:
        for row in g.tensors[1:]:
            for x, y in zip(row, g.tensors[0]):
                x.copy_(y)
    before = [flat(row) for row in g.tensors]
    norm64 = float(torch.cat(before if layout == coco.LOCAL else before[:1]).norm())
    out = g if out_dtype is None else like(g.tensors, n if layout == coco.LOCAL else 3, out_dtype)
    ws, norm = space()
    coco.coco_scattered_clip(g.plan, layout, norm64 / 3, None if out_dtype is None else out.plan, norm, ws)
    coco.coco_device_status()
    g.check(), out.check()
    assert abs(float(norm) - norm64) <= 40 * E * norm64
    for r, row in enumerate(out.tensors):
        near(flat(row), before[r if layout == coco.LOCAL else 0] / 3, out_dtype or dtype)
