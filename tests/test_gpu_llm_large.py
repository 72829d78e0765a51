"""The 8-bit and expert-grouped operators where element indexes pass 32 bits: arrays of over 2^32 elements, sampled
rows (first, last, and around the 2^31st and 2^32nd element) against float64 on the device."""

import pytest
import torch

from collective_fusedallreduce_gb300 import coco

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
F8 = torch.float8_e4m3fn


@pytest.fixture(autouse=True)
def room():
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 100 GB of device memory")
    yield
    torch.cuda.empty_cache()


def sampled(rows, cols):
    at = [0, rows - 1, (1 << 31) // cols, (1 << 32) // cols]
    return torch.tensor(sorted({r for a in at for r in (a - 1, a, a + 1) if 0 <= r < rows}), device=DEV)


def half_step(x, scale):
    """How far an e4m3 value may be from x (half a step, and the rounding of x over its scale)."""
    return torch.maximum(x.abs() / 16, scale * 2.0 ** -10) * (1 + 2.0 ** -10)


def test_norm_and_quantiser():
    rows, cols = 131072 + 40, 32768
    x = torch.randn(rows, cols, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(cols, dtype=torch.bfloat16, device=DEV)
    q, sc = torch.empty(rows, cols, dtype=F8, device=DEV), torch.empty(rows, cols // 128, device=DEV)
    rstd = torch.empty(rows, device=DEV)
    coco.coco_allreduce_rmsnorm(coco.local([x]), None, w, 1e-5, None, coco.replicated([q]), [sc], rstd)
    coco.coco_device_status()
    at = sampled(rows, cols)
    h = x[at].double()
    r = (h.square().mean(-1) + 1e-5).rsqrt()
    assert torch.allclose(rstd[at].double(), r, rtol=1e-5, atol=0)
    spread = sc[at].double().repeat_interleave(128, -1)
    y = h * r[:, None]
    assert bool(((q[at].double() * spread - y).abs() <= half_step(y, spread) + 1e-5 * y.abs()).all())
    tiles = torch.empty((rows + 127) // 128, cols // 128, device=DEV)
    coco.coco_quantize_fp8(coco.local([x]), 128, coco.local([q]), [tiles])
    coco.coco_device_status()
    spread = tiles[at // 128].double().repeat_interleave(128, -1)
    assert bool(((q[at].double() * spread - h).abs() <= half_step(h, spread)).all())
    # the gradient: dy = x, hidden = x, so xhat^2 sums to the row's length and dx is nearly zero; dweight = sum x^2 rstd
    dx, dw = torch.empty_like(x), torch.empty(cols, device=DEV)
    ws = torch.empty(coco.coco_allreduce_rmsnorm_backward_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    coco.coco_allreduce_rmsnorm_backward(coco.local([x]), None, coco.replicated([x]), w, rstd, coco.replicated([dx]),
                                         dw, ws)
    coco.coco_device_status()
    xhat = h * rstd[at].double()[:, None]
    want = rstd[at].double()[:, None] * (h - xhat * (h * xhat).mean(-1, keepdim=True))
    # (differences of nearly equal terms: the bound goes by the terms)
    bound = want.abs() * 2.0 ** -8 + rstd[at].double()[:, None] * h.abs() * 2.0 ** -16
    assert bool(((dx[at].double() - want).abs() <= bound + 1e-30).all())
    # 131112 terms near 1 each in fp32, a few hundred per thread: far below 1e-4
    assert torch.allclose(dw.double().mean(), (x[:512].double().square() * rstd[:512, None].double()).mean() * rows,
                          rtol=2e-2)


def test_outputs_beyond_32_bits():
    m, k, n = 530000, 128, 8208  # 4.35e9 outputs
    a = torch.randn(m, k, device=DEV).to(F8)
    b = torch.randn(n, k, device=DEV).to(F8)
    sa, sb = torch.rand(m, 1, device=DEV) + 0.5, torch.rand((n + 127) // 128, 1, device=DEV) + 0.5
    out = torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
    coco.coco_einsum_fp8("mk,nk->mn", coco.local([a]), [sa], coco.local([b]), [sb], coco.local([out]))
    coco.coco_device_status()
    at = sampled(m, n)
    x = a[at].double() * sa[at].double()
    w = b.double() * sb.double().repeat_interleave(128, 0)[:n]
    want, mag = x @ w.T, x.abs() @ w.abs().T
    assert bool(((out[at].double() - want).abs() <= want.abs() * 2.0 ** -8 + mag * 200 * 2.0 ** -23 + 1e-30).all())
    off = torch.tensor([0, 5, m - 7, m], dtype=torch.int32, device=DEV)  # ragged: the last expert's rows lie past 2^32
    w16 = torch.randn(3, k, n, dtype=torch.bfloat16, device=DEV)
    a16 = a.to(torch.bfloat16)
    coco.coco_grouped_einsum("tk,ekn->tn", coco.local([a16]), None, coco.local([w16]), None, off, coco.local([out]))
    coco.coco_device_status()
    expert = (at >= 5).long() + (at >= m - 7).long()
    for i, r in enumerate(at.tolist()):
        x, w = a16[r].double(), w16[expert[i]].double()
        want, mag = x @ w, x.abs() @ w.abs()
        assert bool(((out[r].double() - want).abs() <= want.abs() * 2.0 ** -8 + mag * 200 * 2.0 ** -23 + 1e-30).all())


@pytest.mark.parametrize("form", ["kn", "nk"])
@pytest.mark.parametrize("per_expert", [3, 300])
def test_weights_beyond_32_bits(form, per_expert):
    experts, k, n = 66, 8192, 8192  # 4.43e9 weights
    counts = torch.zeros(experts, dtype=torch.int64)
    counts[[0, 31, 32, 33, 64, 65]] = per_expert
    rows = int(counts.sum())
    off = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(DEV, torch.int32)
    w = torch.empty(experts, k, n, dtype=torch.uint8, device=DEV).random_(0, 100).view(F8)
    sw = torch.rand(experts, k // 128, n // 128, device=DEV) + 0.5
    a = torch.randn(rows, k, device=DEV).to(F8)
    sa = torch.rand(rows, k // 128, device=DEV) + 0.5
    out = torch.empty(rows, n, device=DEV)
    coco.coco_grouped_einsum(f"tk,e{form}->tn", coco.local([a]), [sa], coco.local([w]), [sw], off, coco.local([out]))
    coco.coco_device_status()
    x = a.double() * sa.double().repeat_interleave(128, 1)
    for e in (0, 31, 32, 33, 64, 65):
        lo = int(off[e])
        we = w[e].double() * sw[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        we = we if form == "kn" else we.T
        rows_e = slice(lo, lo + 3)
        want, mag = x[rows_e] @ we, x[rows_e].abs() @ we.abs()
        assert bool(((out[rows_e].double() - want).abs() <= mag * (k + k // 128 + 8) * 2.0 ** -23).all()), e
