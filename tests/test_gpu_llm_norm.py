"""The norm after an AllReduce, its gradient and the quantiser, through the C-ABI, against the float64 oracle.

Tolerances. u(T) is half the spacing of the stored type's values at 1 (2^-24, 2^-11, 2^-8) and e = 2^-24. A sum of n fp32 terms
is within n e of its exact value times the terms' magnitudes; the row statistics sum at most 8 values in each
of up to 8 chunks, then 5 shuffles and 32 warps: below 128 roundings, and rsqrt, the division and the products
add a few, so a normalised value is within 160 e of exact, relative, plus what the sum over ranks lost.
"""

import numpy as np
import pytest
import torch

import oracle
from collective_fusedallreduce_gb300 import coco, synth

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
E = 2.0 ** -24
U = {t: torch.finfo(t).eps / 2 for t in (torch.float32, torch.float16, torch.bfloat16)}
TINY = {torch.float32: 2.0 ** -126, torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -126}  # a subnormal's half step
F8 = torch.float8_e4m3fn


def dev(ts):
    return [t.to(DEV) for t in ts]


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def within(got, want, bound, what):
    err = np.abs(got - want)
    assert got.shape == want.shape, what
    assert np.all(err <= bound), f"{what}: {np.max(err - bound)} over the bound, at {np.argmax(err - bound)}"


def guarded(shape, dtype, pad=256):
    """A tensor inside a buffer of sentinel bytes, and the check that these are untouched."""
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    raw = torch.full((n + 2 * pad,), 0xA5, dtype=torch.uint8, device=DEV)

    def check():
        assert bool((raw[:pad] == 0xA5).all()) and bool((raw[pad + n:] == 0xA5).all()), "wrote outside the output"

    return raw[pad:pad + n].view(dtype).view(shape), check


NORM_CASES = [  # ranks, rows, cols
    (1, 1, 16), (2, 1, 128), (3, 5, 144), (8, 7, 256), (8, 1, 4096), (4, 3, 1040), (8, 33, 2064), (5, 2, 8192),
    (1, 3, 16400), (2, 2, 32768), (1, 2, 20000), (8, 300, 512), (40, 3, 512),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n,rows,cols", NORM_CASES)
@pytest.mark.parametrize("fp8", [False, True])
def test_norm_matches_the_oracle(dtype, n, rows, cols, fp8):
    parts = synth.per_rank(601, 0, n, (rows, cols), dtype, std=n ** -0.5)
    res = synth.tensor(602, (rows, cols), dtype)
    w = synth.tensor(603, (cols,), dtype)
    copies = min(n, 2)
    hid, hc = zip(*[guarded((rows, cols), dtype) for _ in range(copies)])
    nrm, nc = zip(*[guarded((rows, cols), F8 if fp8 else dtype) for _ in range(copies)])
    nb = -(-cols // 128)
    sc, sg = zip(*[guarded((rows, nb), torch.float32) for _ in range(copies)])
    rstd, rc = guarded((rows,), torch.float32)
    cyc = lambda ts: [ts[r % copies] for r in range(n)]  # noqa: E731
    coco.coco_allreduce_rmsnorm(coco.local(dev(parts)), coco.replicated(dev([res]) * n), w.to(DEV), 1e-5,
                                coco.replicated(cyc(hid)), coco.replicated(cyc(nrm)), cyc(sc) if fp8 else None, rstd)
    coco.coco_device_status()
    for check in list(hc) + list(nc) + list(sg) + [rc]:
        check()
    p64, r64, w64 = [f64(p) for p in parts], f64(res), f64(w)
    h, y, rs = oracle.allreduce_rmsnorm(p64, r64, w64, 1e-5)
    lost = (n + 1) * E * (sum(np.abs(p) for p in p64) + np.abs(r64))  # the fp32 sum over ranks
    # the row's statistic moves by at most the root mean square of what the sum lost
    rel = 160 * E + np.sqrt(np.mean(lost ** 2, -1)) * rs
    within(f64(rstd), rs, rs * rel, "rstd")
    ybound = np.abs(y) * rel[:, None] * 1.01 + lost * rs[:, None] * np.abs(w64) * 1.01
    for c in range(copies):
        within(f64(hid[c]), h, np.abs(h) * U[dtype] * 1.01 + lost * 1.01 + TINY[dtype], "hidden")
        if fp8:
            s = oracle.scales_of(y, 1)
            got_s = f64(sc[c])
            block_bound = oracle.block_amax(ybound, 1) / 448
            within(got_s, s, block_bound + s * 2 * E, "scales")
            back = oracle.dequantize(f64(nrm[c]), got_s, 1)
            half = np.maximum(np.abs(y) / 16, oracle.spread(got_s, y.shape, 1) * 2.0 ** -10)
            within(back, y, half * (1 + 2.0 ** -10) + ybound * 2, "8-bit values")
        else:
            within(f64(nrm[c]), y, np.abs(y) * U[dtype] * 1.01 + ybound + TINY[dtype], "normed")


def test_norm_without_residual_hidden_or_rstd_and_in_place():
    n, rows, cols = 4, 9, 272
    parts = dev(synth.per_rank(604, 0, n, (rows, cols), torch.bfloat16))
    w = synth.tensor(605, (cols,), torch.bfloat16).to(DEV)
    want = [torch.empty_like(parts[0]) for _ in range(2)]
    coco.coco_allreduce_rmsnorm(coco.local(parts), None, w, 1e-5, coco.replicated([want[0]] * n),
                                coco.replicated([want[1]] * n), None, None)
    only = torch.empty_like(parts[0])
    coco.coco_allreduce_rmsnorm(coco.local(parts), None, w, 1e-5, None, coco.replicated([only] * n), None, None)
    # in place: the hidden rows where rank 0's partial was, the normed rows where rank 1's was
    coco.coco_allreduce_rmsnorm(coco.local(parts), None, w, 1e-5, coco.replicated([parts[0]] * n),
                                coco.replicated([parts[1]] * n), None, None)
    torch.cuda.synchronize()
    assert torch.equal(only, want[1]) and torch.equal(parts[0], want[0]) and torch.equal(parts[1], want[1])


def test_norm_groups_are_independent_and_share_the_weight():
    groups, n, rows, cols = 3, 2, 4, 160
    parts = synth.per_rank(606, 0, groups * n, (rows, cols), torch.float16)
    res = synth.per_rank(606, 1, groups, (rows, cols), torch.float16)
    w = synth.tensor(607, (cols,), torch.float16)
    hid = [torch.empty(rows, cols, dtype=torch.float16, device=DEV) for _ in range(groups)]
    nrm = [torch.empty(rows, cols, dtype=F8, device=DEV) for _ in range(groups * n)]
    sc = [torch.empty(rows, 2, device=DEV) for _ in range(groups * n)]
    rstd = torch.empty(groups, rows, device=DEV)
    rep = lambda ts: [t for t in ts for _ in range(n)]  # noqa: E731
    coco.coco_allreduce_rmsnorm(coco.local(dev(parts), groups), coco.replicated(rep(dev(res)), groups), w.to(DEV),
                                1e-5, coco.replicated(rep(hid), groups), coco.replicated(nrm, groups), sc, rstd)
    torch.cuda.synchronize()
    for g in range(groups):
        h, y, rs = oracle.allreduce_rmsnorm([f64(p) for p in parts[g * n:g * n + n]], f64(res[g]), f64(w), 1e-5)
        within(f64(hid[g]), h, np.abs(h) * 2.0 ** -10 + 1e-6, "hidden")
        within(f64(rstd[g]), rs, rs * 1e-5, "rstd")
        for r in range(n):
            assert torch.equal(nrm[g * n + r].view(torch.uint8), nrm[g * n].view(torch.uint8))
            back = oracle.dequantize(f64(nrm[g * n + r]), f64(sc[g * n + r]), 1)
            within(back, y, np.maximum(np.abs(y) / 16, oracle.spread(f64(sc[g * n]), y.shape, 1) / 1024) * 1.001
                   + 1e-5, "8-bit values")


@pytest.mark.parametrize("fp8", [False, True])
def test_norm_of_zero_rows_and_of_rows_that_are_no_numbers(fp8):
    rows, cols = 4, 256
    x = synth.tensor(608, (rows, cols), torch.float32).to(DEV)
    x[0] = 0.0
    x[1, 3] = float("inf")
    x[2, 200] = float("nan")
    w = torch.ones(cols, device=DEV)
    out = torch.empty(rows, cols, dtype=F8 if fp8 else torch.float32, device=DEV)
    sc = torch.empty(rows, 2, device=DEV)
    coco.coco_allreduce_rmsnorm(coco.local([x]), None, w, 1e-5, None, coco.replicated([out]), [sc] if fp8 else None,
                                None)
    torch.cuda.synchronize()
    got = f64(out) * np.repeat(f64(sc), 128, 1) if fp8 else f64(out)
    assert np.all(got[0] == 0.0)
    # an infinite row has 1 / rms zero: inf * 0 where the infinity stood; a NaN is in every value of its row
    assert np.isnan(got[1, 3]) and np.all(np.isnan(got[2]))
    assert np.all(np.isnan(got[1, :128])) if fp8 else np.all(got[1, np.arange(cols) != 3] == 0.0)
    want = oracle.allreduce_rmsnorm([f64(x)[3:]], None, np.ones(cols), 1e-5)[1][0]
    assert np.allclose(got[3], want, rtol=1 / 15 if fp8 else 1e-5, atol=1e-2 if fp8 else 0)


BWD_CASES = [(1, 1, 16), (2, 3, 144), (8, 700, 128), (3, 9, 1040), (8, 650, 4096), (2, 5, 8192), (1, 2, 32768),
             (4, 3, 20000), (40, 3, 512), (1, 5000, 256)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("n,rows,cols", BWD_CASES)
def test_norm_backward_matches_the_oracle(dtype, n, rows, cols):
    dn = synth.per_rank(611, 0, n, (rows, cols), dtype, std=n ** -0.5)
    dh = synth.tensor(612, (rows, cols), dtype) if rows % 2 else None
    hid = synth.tensor(613, (rows, cols), dtype)
    w = synth.tensor(614, (cols,), dtype)
    rstd = torch.from_numpy(1.0 / np.sqrt(np.mean(f64(hid) ** 2, -1) + 1e-5)).float()
    dx, c0 = guarded((rows, cols), dtype)
    dw, c1 = guarded((cols,), torch.float32)
    ws, c2 = guarded((coco.coco_allreduce_rmsnorm_backward_bytes(rows, cols),), torch.uint8)
    args = (coco.local(dev(dn)), None if dh is None else coco.replicated(dev([dh]) * n),
            coco.replicated(dev([hid]) * n), w.to(DEV), rstd.to(DEV), coco.replicated([dx] * n), dw, ws)
    coco.coco_allreduce_rmsnorm_backward(*args)
    coco.coco_device_status()
    for check in (c0, c1, c2):
        check()
    d64, h64, w64, r64 = [f64(d) for d in dn], f64(hid), f64(w), f64(rstd)
    want_x, want_w = oracle.allreduce_rmsnorm_backward(d64, None if dh is None else f64(dh), h64, r64, w64)
    mag = sum(np.abs(d) for d in d64)
    xhat = np.abs(h64 * r64[:, None])
    gm = mag * np.abs(w64)
    # every term's magnitude times the roundings it passes: the ranks' sum, the row's sum, a few products
    terms = r64[:, None] * (gm + xhat * np.mean(gm * xhat, -1, keepdims=True)) + (0 if dh is None else np.abs(f64(dh)))
    within(f64(dx), want_x, np.abs(want_x) * U[dtype] * 1.01 + (n + 160) * E * terms + TINY[dtype], "dx")
    within(f64(dw), want_w, (rows + n + 16) * E * (mag * xhat).sum(0), "dweight")
    first = (dx.clone(), dw.clone())
    coco.coco_allreduce_rmsnorm_backward(*args)
    torch.cuda.synchronize()
    assert torch.equal(dx, first[0]) and torch.equal(dw, first[1])  # fixed order: the same bits


def test_norm_backward_is_the_difference_quotient_of_the_forward():
    n, rows, cols, eps = 2, 6, 136, 1e-3
    parts = dev(synth.per_rank(615, 0, n, (rows, cols), torch.float32))
    w = synth.tensor(616, (cols,), torch.float32).to(DEV)
    dn = dev(synth.per_rank(615, 2, n, (rows, cols), torch.float32))
    dh = synth.tensor(617, (rows, cols), torch.float32).to(DEV)
    hid, nrm = torch.empty(rows, cols, device=DEV), torch.empty(rows, cols, device=DEV)
    rstd = torch.empty(rows, device=DEV)

    def forward(p0, weight):
        coco.coco_allreduce_rmsnorm(coco.local([p0, parts[1]]), None, weight, eps, coco.replicated([hid] * n),
                                    coco.replicated([nrm] * n), None, rstd)
        torch.cuda.synchronize()
        return float((nrm.double() * (dn[0].double() + dn[1].double())).sum() + (hid.double() * dh.double()).sum())

    forward(parts[0], w)
    dx, dw = torch.empty_like(hid), torch.empty_like(w)
    ws = torch.empty(coco.coco_allreduce_rmsnorm_backward_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    coco.coco_allreduce_rmsnorm_backward(coco.local(dn), coco.replicated([dh] * n), coco.replicated([hid.clone()] * n),
                                         w, rstd.clone(), coco.replicated([dx] * n), dw, ws)
    torch.cuda.synchronize()
    # step 2^-6: the quotient's own error is its square times third derivatives of order one (2.5e-4) plus the
    # forward's fp32 rounding (about 800 values of 1e-7) over the step; both small against the quotient's size
    t = 2.0 ** -6
    g = torch.Generator().manual_seed(618)
    for _ in range(4):
        d = torch.randn(rows, cols, generator=g).to(DEV)
        got = (forward(parts[0] + t * d, w) - forward(parts[0] - t * d, w)) / (2 * t)
        want = float((dx.double() * d.double()).sum())
        scale = float(dx.double().norm() * d.double().norm())
        assert abs(got - want) <= 2e-3 * scale, (got, want, scale)
        d = torch.randn(cols, generator=g).to(DEV)
        got = (forward(parts[0], w + t * d) - forward(parts[0], w - t * d)) / (2 * t)
        want = float((dw.double() * d.double()).sum())
        assert abs(got - want) <= 2e-3 * float(dw.double().norm() * d.double().norm()), (got, want)


def test_norm_backward_without_rows_zeroes_the_weight_gradient_and_takes_inputs_places():
    cols = 64
    dw = torch.full((cols,), 7.0, device=DEV)
    none = torch.empty(0, cols, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(cols, dtype=torch.bfloat16, device=DEV)
    coco.coco_allreduce_rmsnorm_backward(coco.local([none]), None, coco.replicated([none]), w,
                                         torch.empty(0, device=DEV), coco.replicated([none]), dw,
                                         torch.empty(0, dtype=torch.uint8, device=DEV))
    torch.cuda.synchronize()
    assert bool((dw == 0).all())
    rows = 5
    dn = dev(synth.per_rank(619, 0, 2, (rows, cols), torch.bfloat16))
    dh, hid = dev(synth.per_rank(619, 1, 2, (rows, cols), torch.bfloat16))
    rstd = torch.ones(rows, device=DEV)
    ws = torch.empty(coco.coco_allreduce_rmsnorm_backward_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(hid)

    def go(to):
        coco.coco_allreduce_rmsnorm_backward(coco.local(dn), coco.replicated([dh] * 2), coco.replicated([hid] * 2), w,
                                             rstd, coco.replicated([to] * 2), dw, ws)
        torch.cuda.synchronize()

    go(out)
    keep = dh.clone()
    go(dh)
    assert torch.equal(dh, out)
    dh.copy_(keep)
    go(dn[1])
    assert torch.equal(dn[1], out)


QUANT_CASES = [(1, 16), (1, 128), (3, 144), (33, 256), (127, 400), (128, 128), (130, 272), (300, 4096), (2, 32768)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", QUANT_CASES)
def test_quantiser_matches_the_definition_bit_for_bit(dtype, block_rows, rows, cols):
    n = 2
    xs = synth.per_rank(621, 0, n, (rows, cols), dtype)
    xs[0][0, :16] = 0.0
    q, qc = zip(*[guarded((rows, cols), F8) for _ in range(n)])
    sc, cc = zip(*[guarded((-(-rows // block_rows), -(-cols // 128)), torch.float32) for _ in range(n)])
    coco.coco_quantize_fp8(coco.local(dev(xs)), block_rows, coco.local(q), sc)
    coco.coco_device_status()
    for check in qc + cc:
        check()
    for r in range(n):
        x = f64(xs[r])
        # the scale is one fp32 division, and so is each value before its rounding to e4m3
        s = np.maximum(oracle.block_amax(x, block_rows), 2.0 ** -100).astype(np.float32) / np.float32(448)
        assert np.array_equal(sc[r].cpu().numpy(), s)
        quotient = x.astype(np.float32) / oracle.spread(s, x.shape, block_rows).astype(np.float32)
        want = oracle.to_e4m3(quotient.astype(np.float64))
        assert np.array_equal(f64(q[r]), want)


def test_quantiser_extremes_and_stacks():
    x = torch.zeros(3, 128, 256)
    x[0, 0, 0] = 2.0 ** -140        # below the floor: stands as zero
    x[0, 5, 130] = 3e38
    x[1, 0, 1] = float("inf")
    x[1, 3, 200] = float("nan")
    x[2, 127, 255] = -5.0
    q = torch.empty(3, 128, 256, dtype=F8, device=DEV)
    sc = torch.empty(3, 1, 2, device=DEV)
    coco.coco_quantize_fp8(coco.local([x.to(DEV)]), 128, coco.local([q]), [sc])
    rows_sc = torch.empty(3 * 128, 2, device=DEV)
    q1 = torch.empty_like(q)
    coco.coco_quantize_fp8(coco.local([x.to(DEV)]), 1, coco.local([q1]), [rows_sc])
    torch.cuda.synchronize()
    s, v = sc.cpu().view(3, 2), q.cpu().float()
    assert float(s[0, 0]) == float(np.float32(2.0 ** -100) / np.float32(448)) and not v[0, :, :128].any()
    assert v[0, 5, 130] == 448 and float(s[0, 1]) == float(np.float32(3e38) / np.float32(448))
    assert torch.isinf(s[1, 0]) and torch.isnan(v[1, 0, 1]) and float(v[1, 0, 0]) == 0.0  # 0 * inf reads as NaN
    assert torch.isnan(s[1, 1]) and torch.isnan(v[1, :, 128:]).all()
    assert v[2, 127, 255] == -448 and float(s[2, 1]) == float(np.float32(5) / np.float32(448))
    r1 = rows_sc.cpu().view(3, 128, 2)
    assert float(r1[0, 5, 1]) == float(np.float32(3e38) / np.float32(448)) and torch.isnan(r1[1, 3, 1])
    assert float(r1[2, 0, 0]) == float(np.float32(2.0 ** -100) / np.float32(448))


def test_calls_run_on_the_stream_they_are_given():
    rows, cols = 64, 4096
    side = torch.cuda.Stream()
    x = torch.randn(rows, cols, device=DEV).bfloat16()
    w = torch.ones(cols, dtype=torch.bfloat16, device=DEV)
    a, b = torch.empty_like(x), torch.empty_like(x)
    q, s = torch.empty(rows, cols, dtype=F8, device=DEV), torch.empty(rows, cols // 128, device=DEV)
    coco.coco_allreduce_rmsnorm(coco.local([x]), None, w, 1e-5, None, coco.replicated([a]), None, None)
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=side):  # nothing allocates or synchronises
        coco.coco_allreduce_rmsnorm(coco.local([x]), None, w, 1e-5, None, coco.replicated([b]), None, None, side)
        coco.coco_quantize_fp8(coco.local([b]), 1, coco.local([q]), [s], side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        coco.coco_allreduce_rmsnorm(coco.local([x]), None, w, 1e-5, None, coco.replicated([b]), None, None, side)
        coco.coco_quantize_fp8(coco.local([b]), 1, coco.local([q]), [s], side)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    want_q, want_s = oracle.quantize(f64(a), 1)
    within(oracle.dequantize(f64(q), f64(s), 1), f64(a),
           np.maximum(np.abs(f64(a)) / 16, oracle.spread(want_s, a.shape, 1) / 1024) * 1.001, "graph")
