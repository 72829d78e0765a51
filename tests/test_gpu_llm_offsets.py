"""Offsets that descend: the values are unspecified, but no access leaves the arrays, the call ends and reports nothing,
and what is computed after it is right."""

import pytest
import torch

from collective_fusedallreduce_gb300 import coco
from test_gpu_llm_norm import guarded

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
F8 = torch.float8_e4m3fn

DESCENDING = [[40, 0, 40, 0, 40], [0, 40, 0, 40, 0], [10, 5, 30, 7, 40], [40, 40, 40, 0, 0], [90, -5, 50, 2, 1],
              [2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 0, 40]]


def operands(rows, k, n, form, dtype, g):
    x = torch.randn(rows, k, generator=g, device=DEV).to(dtype)
    if form == "grad":
        return x, torch.randn(rows, n, generator=g, device=DEV).to(dtype)
    return x, torch.randn(4, *((k, n) if form == "kn" else (n, k)), generator=g, device=DEV).to(dtype)


@pytest.mark.parametrize("form,dtype", [("kn", torch.bfloat16), ("nk", torch.float16), ("kn", F8), ("nk", F8),
                                        ("grad", torch.bfloat16)])
@pytest.mark.parametrize("scale", [1, 30])  # 40 rows: the few-row kernels; 1200: the large tiles
@pytest.mark.parametrize("k,n", [(272, 528), (2048, 1040)])
def test_descending_offsets_stay_inside_the_arrays(form, dtype, scale, k, n):
    rows = 40 * scale
    g = torch.Generator(device=DEV).manual_seed(731)
    a, b = operands(rows, k, n, form, dtype, g)
    sa = sb = None
    if dtype is F8:
        sa = [torch.ones(rows, -(-k // 128), device=DEV)]
        sb = [torch.ones(4, -(-b.shape[1] // 128), -(-b.shape[2] // 128), device=DEV)]
    spec = "tk,tn->ekn" if form == "grad" else f"tk,e{form}->tn"
    shape = (4, k, n) if form == "grad" else (rows, n)
    for off in DESCENDING:
        out, check = guarded(shape, torch.float32)
        o = torch.tensor([max(-2 ** 31, min(2 ** 31 - 1, x * (scale if abs(x) < 100 else 1))) for x in off],
                         dtype=torch.int32, device=DEV)
        coco.coco_grouped_einsum(spec, coco.local([a]), sa, coco.local([b]), sb, o, coco.local([out]))
        coco.coco_device_status()
        check()
    out, check = guarded(shape, torch.float32)
    o = torch.tensor([0, rows, rows, rows, rows], dtype=torch.int32, device=DEV)
    coco.coco_grouped_einsum(spec, coco.local([a]), sa, coco.local([b]), sb, o, coco.local([out]))
    coco.coco_device_status()
    check()
    x, w = (a.double().T, b.double()) if form == "grad" else (a.double(), b[0].double().T if form == "nk" else b[0].double())
    got, depth = (out[0], rows) if form == "grad" else (out, k)
    bound = (depth + depth // 64 + 72) * 2.0 ** -23 * (x.abs() @ w.abs())
    assert bool(((got.double() - x @ w).abs() <= bound + 1e-30).all())


def test_more_units_than_32_bits_count():
    """65536 experts that by turns own all rows and none, on 18 ranks: 2.4e9 tiles, were they all taken."""
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 30 GB of device memory")
    ranks, experts, rows, k, n = 18, 65536, 16384, 8, 16384
    x = torch.ones(rows, k, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(experts, k, n, dtype=torch.bfloat16, device=DEV)
    line = torch.zeros(experts + 1, dtype=torch.int32)
    line[1::2] = rows
    outs, checks = zip(*[guarded((rows, n), torch.bfloat16) for _ in range(ranks)])
    coco.coco_grouped_einsum("tk,ekn->tn", coco.replicated([x] * ranks), None, coco.replicated([w] * ranks), None,
                             line.repeat(ranks, 1).to(DEV), coco.local(outs))
    coco.coco_device_status()
    for check in checks:
        check()
    del x, w, outs, checks
    torch.cuda.empty_cache()
