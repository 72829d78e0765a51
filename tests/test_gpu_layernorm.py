"""The layer norm after an AllReduce and its gradient, through the C-ABI, against the float64 oracle.

Tolerances, with u the half step of the stored type and e = 2^-24. The sum over n ranks and the residual loses at most
`lost` = (n + 1) e of its terms' magnitudes. The mean adds 64 values a lane, 5 shuffles and 16 warps and divides: within 100
e of the mean magnitude, plus the mean of `lost`. So h - mean is off by D = lost + that + 2 e (|h| + |mean|), the root of
the mean square by at most that of D (the triangle inequality), plus 128 roundings of a sum of positive terms: relative
160 e + rms(D) rstd for rstd. A normalised value follows by the product's rule, and one rounding.
"""

import numpy as np
import pytest
import torch

import oracle
from collective_fusedallreduce_gb300 import coco, synth
from test_gpu_llm_norm import DEV, E, F8, TINY, U, BWD_CASES, NORM_CASES, dev, f64, guarded, within

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def bounds(p64, r64, w64, b64, h, mean, rs):
    """How far the sum over ranks, the mean, 1 / deviation (relative) and y may be."""
    n = len(p64)
    lost = (n + 1) * E * (sum(np.abs(p) for p in p64) + (0 if r64 is None else np.abs(r64)))
    dm = 100 * E * np.mean(np.abs(h), -1) + np.mean(lost, -1)
    d = lost + (dm + 2 * E * np.abs(mean))[:, None] + 2 * E * np.abs(h)
    rel = 160 * E + np.sqrt(np.mean(d * d, -1)) * rs
    part = np.abs((h - mean[:, None]) * rs[:, None] * w64)
    yb = 1.01 * (np.abs(w64) * d * rs[:, None] + part * rel[:, None]) + 4 * E * (part + np.abs(b64))
    return lost, dm, rel, yb


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,rows,cols", NORM_CASES)
@pytest.mark.parametrize("fp8", [False, True])
def test_norm_matches_the_oracle(dtype, n, rows, cols, fp8):
    parts = synth.per_rank(801, 0, n, (rows, cols), dtype, std=n ** -0.5)
    res = synth.tensor(802, (rows, cols), dtype)
    w, b = synth.tensor(803, (cols,), dtype), synth.tensor(804, (cols,), dtype)
    copies = min(n, 2)
    hid, hc = zip(*[guarded((rows, cols), dtype) for _ in range(copies)])
    nrm, nc = zip(*[guarded((rows, cols), F8 if fp8 else dtype) for _ in range(copies)])
    nb = -(-cols // 128)
    sc, sg = zip(*[guarded((rows, nb), torch.float32) for _ in range(copies)])
    mean, mc = guarded((rows,), torch.float32)
    rstd, rc = guarded((rows,), torch.float32)
    cyc = lambda ts: [ts[r % copies] for r in range(n)]  # noqa: E731
    coco.coco_allreduce_layernorm(coco.local(dev(parts)), coco.replicated(dev([res]) * n), w.to(DEV), b.to(DEV), 1e-5,
                                  coco.replicated(cyc(hid)), coco.replicated(cyc(nrm)), cyc(sc) if fp8 else None, mean,
                                  rstd)
    coco.coco_device_status()
    for check in list(hc) + list(nc) + list(sg) + [mc, rc]:
        check()
    p64, r64, w64, b64 = [f64(p) for p in parts], f64(res), f64(w), f64(b)
    h, y, m, rs = oracle.allreduce_layernorm(p64, r64, w64, b64, 1e-5)
    lost, dm, rel, yb = bounds(p64, r64, w64, b64, h, m, rs)
    within(f64(mean), m, dm * 1.01 + E * np.abs(m), "mean")
    within(f64(rstd), rs, rs * rel, "rstd")
    for c in range(copies):
        within(f64(hid[c]), h, np.abs(h) * U[dtype] * 1.01 + lost * 1.01 + TINY[dtype], "hidden")
        if fp8:
            s = oracle.scales_of(y, 1)
            got_s = f64(sc[c])
            within(got_s, s, oracle.block_amax(yb, 1) / 448 + s * 2 * E, "scales")
            back = oracle.dequantize(f64(nrm[c]), got_s, 1)
            half = np.maximum(np.abs(y) / 16, oracle.spread(got_s, y.shape, 1) * 2.0 ** -10)
            within(back, y, half * (1 + 2.0 ** -10) + yb * 2, "8-bit values")
        else:
            within(f64(nrm[c]), y, np.abs(y) * U[dtype] * 1.01 + yb + TINY[dtype], "normed")


@pytest.mark.parametrize("dtype,fp8", [(torch.bfloat16, False), (torch.float16, True), (torch.float32, False)])
@pytest.mark.parametrize("n,rows,cols", [(1, 1230, 4112), (1, 1230, 8208), (1, 1230, 12304), (2, 170, 6096), (2, 170, 12304),
                                         (3, 170, 6144), (3, 170, 16384), (4, 170, 10784), (8, 170, 9216), (8, 170, 16384)])
def test_many_wide_rows_match_the_oracle(dtype, fp8, n, rows, cols):
    """More rows than the device has multiprocessors (eight times as many, on one rank): three and four chunks a thread."""
    test_norm_matches_the_oracle(dtype, n, rows, cols, fp8)


@pytest.mark.parametrize("cols", [256, 4096, 5008])
def test_a_mean_far_from_zero(cols):
    """Rows whose mean is some 3000 times their deviation. h is exact here (multiples of 2^-11 near 4) and so are the sums of
    a warp (24 bits hold them); the mean takes some roundings of 2^-24 of 4 each, 8 at most, and the variance about it only
    their square, as a sum about a mean off by d is off by n d^2."""
    g = torch.Generator().manual_seed(811)
    x = 4.0 + torch.randint(-4, 5, (5, cols), generator=g) * 2.0 ** -11
    w, b = torch.ones(cols), torch.zeros(cols)
    out, mean, rstd = torch.empty(5, cols, device=DEV), torch.empty(5, device=DEV), torch.empty(5, device=DEV)
    coco.coco_allreduce_layernorm(coco.local([x.to(DEV)]), None, w.to(DEV), b.to(DEV), 0.0, None, coco.replicated([out]),
                                  None, mean, rstd)
    coco.coco_device_status()
    h, y, m, rs = oracle.allreduce_layernorm([f64(x)], None, f64(w), f64(b), 0.0)
    dm = 8 * E * 4
    within(f64(mean), m, np.full(5, dm), "mean")
    within(f64(rstd), rs, rs * (160 * E + (dm * rs) ** 2), "rstd")
    rel = 164 * E + (dm * rs) ** 2
    within(f64(out), y, (dm + E * 8) * rs[:, None] + np.abs(y) * rel[:, None], "normed")


def test_norm_without_what_may_be_left_out_and_in_place():
    n, rows, cols = 4, 9, 272
    parts = dev(synth.per_rank(821, 0, n, (rows, cols), torch.bfloat16))
    w, b = dev([synth.tensor(822, (cols,), torch.bfloat16), synth.tensor(823, (cols,), torch.bfloat16)])
    want = [torch.empty_like(parts[0]) for _ in range(2)]
    coco.coco_allreduce_layernorm(coco.local(parts), None, w, b, 1e-5, coco.replicated([want[0]] * n),
                                  coco.replicated([want[1]] * n), None, None, None)
    only, bare, zero = (torch.empty_like(parts[0]) for _ in range(3))
    coco.coco_allreduce_layernorm(coco.local(parts), None, w, b, 1e-5, None, coco.replicated([only] * n), None, None, None)
    coco.coco_allreduce_layernorm(coco.local(parts), None, w, None, 1e-5, None, coco.replicated([bare] * n), None, None,
                                  None)
    coco.coco_allreduce_layernorm(coco.local(parts), None, w, torch.zeros_like(b), 1e-5, None,
                                  coco.replicated([zero] * n), None, None, None)
    # in place: the hidden rows where rank 0's partial was, the normed rows where rank 1's was
    coco.coco_allreduce_layernorm(coco.local(parts), None, w, b, 1e-5, coco.replicated([parts[0]] * n),
                                  coco.replicated([parts[1]] * n), None, None, None)
    torch.cuda.synchronize()
    assert torch.equal(only, want[1]) and torch.equal(parts[0], want[0]) and torch.equal(parts[1], want[1])
    assert torch.equal(bare, zero)


def test_norm_groups_are_independent():
    groups, n, rows, cols = 3, 2, 4, 160
    parts = synth.per_rank(826, 0, groups * n, (rows, cols), torch.float16)
    res = synth.per_rank(826, 1, groups, (rows, cols), torch.float16)
    w, b = synth.tensor(827, (cols,), torch.float16), synth.tensor(828, (cols,), torch.float16)
    hid = [torch.empty(rows, cols, dtype=torch.float16, device=DEV) for _ in range(groups)]
    nrm = [torch.empty(rows, cols, dtype=torch.float16, device=DEV) for _ in range(groups * n)]
    mean, rstd = torch.empty(groups, rows, device=DEV), torch.empty(groups, rows, device=DEV)
    rep = lambda ts: [t for t in ts for _ in range(n)]  # noqa: E731
    coco.coco_allreduce_layernorm(coco.local(dev(parts), groups), coco.replicated(rep(dev(res)), groups), w.to(DEV),
                                  b.to(DEV), 1e-5, coco.replicated(rep(hid), groups), coco.replicated(nrm, groups), None,
                                  mean, rstd)
    torch.cuda.synchronize()
    for g in range(groups):
        mine = [f64(p) for p in parts[g * n:g * n + n]]
        h, y, m, rs = oracle.allreduce_layernorm(mine, f64(res[g]), f64(w), f64(b), 1e-5)
        lost, dm, rel, yb = bounds(mine, f64(res[g]), f64(w), f64(b), h, m, rs)
        within(f64(hid[g]), h, np.abs(h) * 2.0 ** -11 * 1.01 + lost * 1.01 + TINY[torch.float16], "hidden")
        within(f64(mean[g]), m, dm * 1.01 + E * np.abs(m), "mean")
        within(f64(rstd[g]), rs, rs * rel, "rstd")
        for r in range(n):
            within(f64(nrm[g * n + r]), y, np.abs(y) * 2.0 ** -11 * 1.01 + yb + TINY[torch.float16], "normed")


@pytest.mark.parametrize("fp8", [False, True])
def test_rows_of_one_value_and_rows_that_are_no_numbers(fp8):
    rows, cols = 5, 256
    x = synth.tensor(831, (rows, cols), torch.float32).to(DEV)
    x[0] = 0.0
    x[1, 3] = float("inf")
    x[2, 200] = float("nan")
    x[4] = -3.0  # no deviation: the bias alone
    w, b = torch.ones(cols, device=DEV), torch.full((cols,), 0.5, device=DEV)
    out = torch.empty(rows, cols, dtype=F8 if fp8 else torch.float32, device=DEV)
    sc = torch.empty(rows, 2, device=DEV)
    coco.coco_allreduce_layernorm(coco.local([x]), None, w, b, 1e-5, None, coco.replicated([out]), [sc] if fp8 else None,
                                  None, None)
    torch.cuda.synchronize()
    got = f64(out) * np.repeat(f64(sc), 128, 1) if fp8 else f64(out)
    assert np.allclose(got[0], 0.5, rtol=1e-6) and np.allclose(got[4], 0.5, rtol=1e-6)
    assert np.all(np.isnan(got[1])) and np.all(np.isnan(got[2]))  # the mean of either is no number
    want = oracle.allreduce_layernorm([f64(x)[3:4]], None, np.ones(cols), 0.5, 1e-5)[1][0]
    assert np.allclose(got[3], want, rtol=1 / 15 if fp8 else 1e-5, atol=1e-2 if fp8 else 1e-5)


def backward_case(dtype, n, rows, cols, seed=841):
    dn = synth.per_rank(seed, 0, n, (rows, cols), dtype, std=n ** -0.5)
    dh = synth.tensor(seed + 1, (rows, cols), dtype) if rows % 2 else None
    hid = synth.tensor(seed + 2, (rows, cols), dtype)
    w = synth.tensor(seed + 3, (cols,), dtype)
    h = f64(hid)
    mean = torch.from_numpy(np.mean(h, -1)).float()
    rstd = torch.from_numpy(1.0 / np.sqrt(np.var(h, -1) + 1e-5)).float()
    return dn, dh, hid, w, mean, rstd


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,rows,cols", BWD_CASES + [(2, 40, 16400), (2, 400, 32768), (1, 3, 16384), (3, 5, 5008)])
def test_backward_matches_the_oracle(dtype, n, rows, cols):
    dn, dh, hid, w, mean, rstd = backward_case(dtype, n, rows, cols)
    dx, c0 = guarded((rows, cols), dtype)
    dw, c1 = guarded((cols,), torch.float32)
    db, c2 = guarded((cols,), torch.float32)
    ws, c3 = guarded((coco.coco_allreduce_layernorm_backward_bytes(rows, cols),), torch.uint8)
    args = (coco.local(dev(dn)), None if dh is None else coco.replicated(dev([dh]) * n),
            coco.replicated(dev([hid]) * n), w.to(DEV), mean.to(DEV), rstd.to(DEV), coco.replicated([dx] * n), dw)
    coco.coco_allreduce_layernorm_backward(*args, db, ws)
    coco.coco_device_status()
    for check in (c0, c1, c2, c3):
        check()
    d64, h64, w64, m64, r64 = [f64(d) for d in dn], f64(hid), f64(w), f64(mean), f64(rstd)
    want_x, want_w, want_b = oracle.allreduce_layernorm_backward(d64, None if dh is None else f64(dh), h64, m64, r64, w64)
    mag = sum(np.abs(d) for d in d64)
    xhat = np.abs((h64 - m64[:, None]) * r64[:, None])
    gm = mag * np.abs(w64)
    # every term's magnitude times the roundings it passes: the ranks' sum, the row's sums, a few products
    terms = r64[:, None] * (gm + np.mean(gm, -1, keepdims=True) + xhat * np.mean(gm * xhat, -1, keepdims=True)) \
        + (0 if dh is None else np.abs(f64(dh)))
    within(f64(dx), want_x, np.abs(want_x) * U[dtype] * 1.01 + (n + 160) * E * terms + TINY[dtype], "dx")
    within(f64(dw), want_w, (rows + n + 16) * E * (mag * xhat).sum(0), "dweight")
    within(f64(db), want_b, (rows + n + 16) * E * mag.sum(0), "dbias")
    first = (dx.clone(), dw.clone(), db.clone())
    coco.coco_allreduce_layernorm_backward(*args, db, ws)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((dx, dw, db), first))  # fixed order: the same bits
    db.fill_(5.0)
    dw.fill_(5.0)
    coco.coco_allreduce_layernorm_backward(*args, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(dw, first[1]) and bool((db == 5.0).all())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n,rows,cols", [(1, 3100, 1024), (2, 640, 4000), (3, 1000, 2064), (4, 5000, 272), (8, 650, 4096)])
def test_backward_of_several_rows_a_block_matches_the_oracle(dtype, n, rows, cols):
    """More rows than the device holds at a time, the last ones for some blocks only."""
    test_backward_matches_the_oracle(dtype, n, rows, cols)


def test_backward_of_groups_joins_their_rows():
    groups, n, rows, cols = 3, 2, 7, 160
    g = torch.Generator().manual_seed(851)
    rnd = lambda *s: torch.randn(*s, generator=g).bfloat16()  # noqa: E731
    dn, hid = [rnd(rows, cols) for _ in range(groups * n)], [rnd(rows, cols) for _ in range(groups)]
    dh, w = [rnd(rows, cols) for _ in range(groups)], rnd(cols)
    mean = torch.stack([h.float().mean(-1) for h in hid])
    rstd = torch.stack([(h.float().var(-1, correction=0) + 1e-5).rsqrt() for h in hid])
    dx = [torch.empty(rows, cols, dtype=torch.bfloat16, device=DEV) for _ in range(groups * n)]
    dw, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    ws = torch.empty(coco.coco_allreduce_layernorm_backward_bytes(groups * rows, cols), dtype=torch.uint8, device=DEV)
    rep = lambda ts: [t for t in dev(ts) for _ in range(n)]  # noqa: E731
    coco.coco_allreduce_layernorm_backward(coco.local(dev(dn), groups), coco.replicated(rep(dh), groups),
                                           coco.replicated(rep(hid), groups), w.to(DEV), mean.to(DEV), rstd.to(DEV),
                                           coco.replicated(dx, groups), dw, db, ws)
    coco.coco_device_status()
    sw, sb, mw, mb = 0, 0, 0, 0
    for i in range(groups):
        mine = [f64(d) for d in dn[i * n:i * n + n]]
        h, m, r = f64(hid[i]), f64(mean[i]), f64(rstd[i])
        want, a, b = oracle.allreduce_layernorm_backward(mine, f64(dh[i]), h, m, r, f64(w))
        sw, sb = sw + a, sb + b
        mag = sum(np.abs(d) for d in mine)
        mw, mb = mw + (mag * np.abs((h - m[:, None]) * r[:, None])).sum(0), mb + mag.sum(0)
        for j in range(n):
            # terms of at most 40: fp32's part is below 200 e of them
            within(f64(dx[i * n + j]), want, np.abs(want) * 2.0 ** -8 * 1.01 + 200 * E * 40, "dx")
    within(f64(dw), sw, (groups * rows + n + 16) * E * mw, "dweight")
    within(f64(db), sb, (groups * rows + n + 16) * E * mb, "dbias")


def test_backward_is_the_difference_quotient_of_the_forward():
    n, rows, cols, eps = 2, 6, 136, 1e-3
    parts = dev(synth.per_rank(861, 0, n, (rows, cols), torch.float32))
    w, b = dev([synth.tensor(862, (cols,), torch.float32), synth.tensor(863, (cols,), torch.float32)])
    dn = dev(synth.per_rank(861, 2, n, (rows, cols), torch.float32))
    dh = synth.tensor(864, (rows, cols), torch.float32).to(DEV)
    hid, nrm = torch.empty(rows, cols, device=DEV), torch.empty(rows, cols, device=DEV)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)

    def forward(p0, weight, bias):
        coco.coco_allreduce_layernorm(coco.local([p0, parts[1]]), None, weight, bias, eps, coco.replicated([hid] * n),
                                      coco.replicated([nrm] * n), None, mean, rstd)
        torch.cuda.synchronize()
        return float((nrm.double() * (dn[0].double() + dn[1].double())).sum() + (hid.double() * dh.double()).sum())

    forward(parts[0], w, b)
    dx, dw, db = torch.empty_like(hid), torch.empty_like(w), torch.empty_like(b)
    ws = torch.empty(coco.coco_allreduce_layernorm_backward_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    coco.coco_allreduce_layernorm_backward(coco.local(dn), coco.replicated([dh] * n), coco.replicated([hid.clone()] * n),
                                           w, mean.clone(), rstd.clone(), coco.replicated([dx] * n), dw, db, ws)
    torch.cuda.synchronize()
    # step 2^-6: the quotient's own error is its square times third derivatives of order one (2.5e-4) plus the
    # forward's fp32 rounding (about 800 values of 1e-7) over the step; both small against the quotient's size
    t = 2.0 ** -6
    g = torch.Generator().manual_seed(865)
    for _ in range(4):
        for i, grad in enumerate((dx, dw, db)):
            at = [parts[0], w, b]
            d = torch.randn(at[i].shape, generator=g).to(DEV)
            up, down = list(at), list(at)
            up[i], down[i] = at[i] + t * d, at[i] - t * d
            got = (forward(*up) - forward(*down)) / (2 * t)
            want = float((grad.double() * d.double()).sum())
            assert abs(got - want) <= 2e-3 * float(grad.double().norm() * d.double().norm()), (i, got, want)


def test_backward_without_rows_and_in_inputs_places():
    cols = 64
    dw, db = torch.full((cols,), 7.0, device=DEV), torch.full((cols,), 7.0, device=DEV)
    none = torch.empty(0, cols, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(cols, dtype=torch.bfloat16, device=DEV)
    empty = torch.empty(0, device=DEV)
    coco.coco_allreduce_layernorm_backward(coco.local([none]), None, coco.replicated([none]), w, empty, empty,
                                           coco.replicated([none]), dw, db, torch.empty(0, dtype=torch.uint8, device=DEV))
    torch.cuda.synchronize()
    assert not dw.any() and not db.any()
    rows = 5
    dn = dev(synth.per_rank(871, 0, 2, (rows, cols), torch.bfloat16))
    dh, hid = dev(synth.per_rank(871, 1, 2, (rows, cols), torch.bfloat16))
    mean, rstd = torch.zeros(rows, device=DEV), torch.ones(rows, device=DEV)
    ws = torch.empty(coco.coco_allreduce_layernorm_backward_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(hid)

    def go(to):
        coco.coco_allreduce_layernorm_backward(coco.local(dn), coco.replicated([dh] * 2), coco.replicated([hid] * 2), w,
                                               mean, rstd, coco.replicated([to] * 2), dw, db, ws)
        torch.cuda.synchronize()

    go(out)
    for place in (dh, hid, dn[1]):
        keep = place.clone()
        go(place)
        assert torch.equal(place, out)
        place.copy_(keep)


def test_captured_and_replayed():
    rows, cols = 64, 4096
    side = torch.cuda.Stream()
    x = torch.randn(rows, cols, device=DEV).bfloat16()
    w, b = torch.ones(cols, dtype=torch.bfloat16, device=DEV), torch.zeros(cols, dtype=torch.bfloat16, device=DEV)
    mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    dw, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    ws = torch.empty(coco.coco_allreduce_layernorm_backward_bytes(rows, cols), dtype=torch.uint8, device=DEV)

    def step():
        coco.coco_allreduce_layernorm(coco.local([x]), None, w, b, 1e-5, None, coco.replicated([y]), None, mean, rstd)
        coco.coco_allreduce_layernorm_backward(coco.local([y]), None, coco.replicated([x]), w, mean, rstd,
                                               coco.replicated([dx]), dw, db, ws)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(2):
        x.copy_(torch.randn(rows, cols, device=DEV))
        step()
        torch.cuda.synchronize()
        want = [t.clone() for t in (y, dx, dw, db)]
        for t in (y, dx, dw, db):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, c) for a, c in zip((y, dx, dw, db), want))
