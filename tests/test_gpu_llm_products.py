"""Block-scaled products of 8-bit operands and products grouped by expert, through the C-ABI, against the float64
oracle.

Tolerance: the oracle takes the stored values (8-bit ones times their scales) as they are, so what remains is
the accumulation and the output's rounding. Tensor-core products of these types are exact in fp32; every
addition rounds or truncates to fp32, at most one ulp (2^-23) of the sum of the terms' magnitudes S. A sum of K
products in blocks has at most K + K/128 of them, plus two roundings for the scales:
|err| <= (K + K/128 + 8) 2^-23 S, and the output rounds once, u(T)|ref|.
"""

import numpy as np
import pytest
import torch

import oracle
from collective_fusedallreduce_gb300 import coco, synth
from test_gpu_llm_norm import DEV, F8, TINY, U, dev, f64, guarded, within

pytestmark = pytest.mark.gpu


def gamma(k):
    return (k + k // 128 + 8) * 2.0 ** -23


def close(got, lhs, rhs, k, dtype, what):
    """got against lhs @ rhs in 64 bits."""
    want, mag = lhs @ rhs, np.abs(lhs) @ np.abs(rhs)
    within(f64(got), want, np.abs(want) * U[dtype] * 1.01 + gamma(k) * mag + TINY[dtype], what)


def eight_bits(x, block_rows):
    """(values on the device, scales on the device, what they stand for) of the last two dimensions of a CPU tensor."""
    mats = x.reshape(-1, *x.shape[-2:]).numpy().astype(np.float64)
    qs = [oracle.quantize(m, block_rows) for m in mats]
    q = torch.from_numpy(np.stack([a for a, _ in qs])).to(F8).reshape(x.shape)
    s = torch.from_numpy(np.stack([b for _, b in qs])).float()
    back = np.stack([oracle.dequantize(a, s[i].double().numpy(), block_rows) for i, (a, _) in enumerate(qs)])
    return q.to(DEV), s.reshape(*x.shape[:-2], *s.shape[1:]).to(DEV), back.reshape(x.shape)


PRODUCTS = [  # ranks, m, k, n
    (1, 1, 16, 16), (1, 1, 128, 128), (2, 1, 4096, 512), (1, 7, 144, 272), (1, 16, 1024, 128), (3, 17, 528, 144),
    (1, 33, 400, 2064), (1, 64, 2048, 256), (1, 65, 256, 400), (2, 129, 640, 528), (1, 200, 1296, 1040),
    (1, 256, 512, 256), (1, 300, 384, 1552), (8, 333, 528, 272), (1, 1000, 768, 2048), (1, 2049, 272, 4112),
    # many blocks through the rings of the few-row kernels; more tiles than pairs of SMs with many blocks each
    (1, 5, 4096, 8208), (1, 50, 2064, 10256), (1, 2500, 1040, 2576),
]


@pytest.mark.parametrize("form", ["kn", "nk"])
@pytest.mark.parametrize("ranks,m,k,n", PRODUCTS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_product_matches_the_oracle(form, ranks, m, k, n, dtype):
    lhs = [eight_bits(x, 1) for x in synth.per_rank(631, 0, ranks, (m, k), torch.float32)]
    shape = (k, n) if form == "kn" else (n, k)
    rhs = [eight_bits(x, 128) for x in synth.per_rank(631, 1, ranks, shape, torch.float32, std=k ** -0.5)]
    out, checks = zip(*[guarded((m, n), dtype) for _ in range(ranks)])
    coco.coco_einsum_fp8("mk,kn->mn" if form == "kn" else "mk, nk -> mn", coco.local([a[0] for a in lhs]),
                         [a[1] for a in lhs], coco.local([b[0] for b in rhs]), [b[1] for b in rhs], coco.local(out))
    coco.coco_device_status()
    for r in range(ranks):
        checks[r]()
        close(out[r], lhs[r][2], rhs[r][2] if form == "kn" else rhs[r][2].T, k, dtype, f"rank {r}")


@pytest.mark.parametrize("m", [1, 20, 70, 300])
def test_scales_differ_by_block_and_land_where_they_belong(m):
    """Operands of ones: the result is the scales' own product, exact in every format."""
    k, n = 400, 656
    kb, nb = 4, 6
    g = torch.Generator().manual_seed(632)
    sa = 2.0 ** torch.randint(-3, 4, (m, kb), generator=g).float()
    sb = 2.0 ** torch.randint(-3, 4, (kb, nb), generator=g).float()
    ones_a, ones_b = torch.ones(m, k).to(F8).to(DEV), torch.ones(k, n).to(F8).to(DEV)
    lens = torch.tensor([128.0, 128.0, 128.0, 16.0])
    want = (sa * lens) @ sb.repeat_interleave(128, 1)[:, :n]
    for form in ("kn", "nk"):
        out = torch.empty(m, n, device=DEV)
        rhs, srhs = (ones_b, sb) if form == "kn" else (ones_b.t().contiguous(), sb.t().contiguous())
        coco.coco_einsum_fp8(f"mk,{form}->mn", coco.local([ones_a]), [sa.to(DEV)], coco.local([rhs]),
                             [srhs.to(DEV)], coco.local([out]))
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want), form


@pytest.mark.parametrize("m", [3, 200])
def test_layouts_and_groups(m):
    """A replicated lhs (column-parallel weights) and slices on k (row-parallel partials), two groups."""
    k, n, ranks, groups = 256, 144, 2, 2
    lhs = [eight_bits(x, 1) for x in synth.per_rank(633, 0, groups, (m, k), torch.float32)]
    rhs = [eight_bits(x, 128) for x in synth.per_rank(633, 1, groups * ranks, (k, n), torch.float32)]
    out = [torch.empty(m, n, device=DEV) for _ in range(groups * ranks)]
    rep = [lhs[p // ranks] for p in range(groups * ranks)]
    for layout in ("replicated", "sliced"):
        if layout == "replicated":
            a, b = coco.replicated([x[0] for x in rep], groups), coco.local([x[0] for x in rhs], groups)
        else:
            a, b = coco.sliced([x[0] for x in rep], 1, groups), coco.sliced([x[0] for x in rhs], 0, groups)
        for o in out:
            o.fill_(float("nan"))
        coco.coco_einsum_fp8("mk,kn->mn", a, [x[1] for x in rep], b, [x[1] for x in rhs], coco.local(out, groups))
        coco.coco_device_status()
        for p in range(groups * ranks):
            close(out[p], rep[p][2], rhs[p][2], k, torch.float32, f"{layout} {p}")


@pytest.mark.parametrize("m", [2, 160])
def test_what_is_no_number_stays_in_its_row_or_column(m):
    k, n = 272, 272
    a, sa, lhs = eight_bits(synth.tensor(634, (m, k), torch.float32), 1)
    b, sb, rhs = eight_bits(synth.tensor(635, (k, n), torch.float32), 128)
    a.view(torch.uint8)[1, 5] = 0x7F            # a NaN in row 1
    sb[2, 1] = float("inf")                     # the scale of k 256.., n 128..255
    out = torch.empty(m, n, device=DEV)
    coco.coco_einsum_fp8("mk,kn->mn", coco.local([a]), [sa], coco.local([b]), [sb], coco.local([out]))
    coco.coco_device_status()
    got = f64(out)
    assert np.all(np.isnan(got[1]))
    assert not np.any(np.isfinite(got[0, 128:256]))
    cols = np.r_[0:128, 256:n]
    rows = [r for r in range(m) if r != 1]
    want, mag = lhs @ rhs, np.abs(lhs) @ np.abs(rhs)
    within(got[np.ix_(rows, cols)], want[np.ix_(rows, cols)], gamma(k) * mag[np.ix_(rows, cols)] + 1e-30, "others")


def test_empty_extents():
    z = lambda *s: torch.empty(*s, dtype=F8, device=DEV)  # noqa: E731
    sc = lambda *s: torch.empty(*s, device=DEV)  # noqa: E731
    out = torch.full((3, 32), 5.0, device=DEV)
    coco.coco_einsum_fp8("mk,kn->mn", coco.local([z(3, 0)]), [sc(3, 0)], coco.local([z(0, 32)]), [sc(0, 1)],
                         coco.local([out]))
    torch.cuda.synchronize()
    assert not out.any()
    coco.coco_einsum_fp8("mk,kn->mn", coco.local([z(0, 16)]), [sc(0, 1)], coco.local([z(16, 32)]), [sc(1, 1)],
                         coco.local([torch.empty(0, 32, device=DEV)]))
    off = torch.zeros(3, dtype=torch.int32, device=DEV)
    out = torch.full((2, 16, 32), 5.0, device=DEV)
    coco.coco_grouped_einsum("tk,tn->ekn", coco.local([torch.empty(0, 16, dtype=torch.bfloat16, device=DEV)]), None,
                             coco.local([torch.empty(0, 32, dtype=torch.bfloat16, device=DEV)]), None, off,
                             coco.local([out]))
    torch.cuda.synchronize()
    assert not out.any()


def offsets_of(counts, head=0):
    return np.concatenate([[0], np.cumsum(counts)]) + head


GROUPED = [  # counts (rows of each expert), rows before the first and after the last, k, n
    ([1], 0, 0, 16, 16), ([1, 0, 2], 0, 0, 128, 128), ([0, 0, 5, 0], 2, 3, 144, 272), ([3] * 40, 0, 0, 256, 144),
    ([37, 0, 200, 1, 64], 0, 5, 528, 400), ([129, 255, 256, 257], 0, 0, 384, 528), ([1000, 3, 0, 77], 9, 0, 272, 1040),
    ([0, 0], 4, 4, 128, 256), ([16] * 65, 0, 0, 128, 144), ([640, 700], 0, 0, 1024, 512),
    # enough columns for 256-row tiles: experts that end after 1, 31, 33, 44, 65 and 256 rows of one
    ([300, 1, 515, 0, 77, 256, 31, 321], 3, 2, 272, 4112), ([289, 5, 0, 1121], 0, 1, 1040, 2064),
]


@pytest.mark.parametrize("form", ["kn", "nk"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, F8])
@pytest.mark.parametrize("case", range(len(GROUPED)))
def test_grouped_matches_the_oracle(form, dtype, case):
    counts, head, tail, k, n = GROUPED[case]
    off = offsets_of(counts, head)
    rows, experts = int(off[-1]) + tail, len(counts)
    x = synth.tensor(641, (rows, k), torch.float32)
    w = synth.tensor(642, (experts, k, n) if form == "kn" else (experts, n, k), torch.float32, std=k ** -0.5)
    if dtype is F8:
        a, sa, lhs = eight_bits(x, 1)
        b, sb, rhs = eight_bits(w, 128)
        sa, sb, odt = [sa], [sb], torch.bfloat16
    else:
        a, b = x.to(dtype).to(DEV), w.to(dtype).to(DEV)
        lhs, rhs, sa, sb, odt = f64(a), f64(b), None, None, dtype
    # rows of no expert hold what is no number: they may not reach any other row
    outside = torch.ones(rows, dtype=torch.bool)
    outside[int(off[0]):int(off[-1])] = False
    a.view(torch.uint8 if dtype is F8 else torch.int16)[outside.to(DEV)] = 0x7F if dtype is F8 else 0x7FFF
    lhs[outside.numpy()] = 0.0
    out, check = guarded((rows, n), odt)
    out.fill_(float("nan"))
    coco.coco_grouped_einsum(f"tk,e{form}->tn", coco.local([a]), sa, coco.local([b]), sb,
                             torch.from_numpy(off).to(DEV, torch.int32), coco.local([out]))
    coco.coco_device_status()
    check()
    want = oracle.grouped_einsum(form, lhs, rhs, off)
    mag = oracle.grouped_einsum(form, np.abs(lhs), np.abs(rhs), off)
    within(f64(out), want, np.abs(want) * U[odt] * 1.01 + gamma(k) * mag + TINY[odt], "grouped")


@pytest.mark.parametrize("dtype,odt", [(torch.bfloat16, torch.bfloat16), (torch.float16, torch.float32),
                                       (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("case", range(len(GROUPED)))
def test_weight_gradient_matches_the_oracle(dtype, odt, case):
    counts, head, tail, k, n = GROUPED[case]
    off = offsets_of(counts, head)
    rows, experts = int(off[-1]) + tail, len(counts)
    a = synth.tensor(643, (rows, k), dtype).to(DEV)
    b = synth.tensor(644, (rows, n), dtype).to(DEV)
    lhs, rhs = f64(a), f64(b)
    outside = torch.ones(rows, dtype=torch.bool)
    outside[int(off[0]):int(off[-1])] = False
    for x in (a, b):
        x.view(torch.int16)[outside.to(DEV)] = 0x7FFF
    out, check = guarded((experts, k, n), odt)
    out.fill_(float("nan"))
    coco.coco_grouped_einsum("tk,tn->ekn", coco.local([a]), None, coco.local([b]), None,
                             torch.from_numpy(off).to(DEV, torch.int32), coco.local([out]))
    coco.coco_device_status()
    check()
    want = oracle.grouped_einsum("grad", lhs, rhs, off)
    mag = oracle.grouped_einsum("grad", np.abs(lhs), np.abs(rhs), off)
    within(f64(out), want, np.abs(want) * U[odt] * 1.01 + gamma(max(counts) + 128) * mag + TINY[odt], "gradient")


def test_an_experts_infinities_stay_with_it():
    """Neighbouring experts' rows share tiles: a NaN or an infinity of one may not reach another."""
    counts, k, n = [70, 3, 0, 130, 61], 144, 272
    off = offsets_of(counts)
    rows = int(off[-1])
    offsets = torch.from_numpy(off).to(DEV, torch.int32)
    a, dy = synth.tensor(645, (rows, k), torch.bfloat16), synth.tensor(646, (rows, n), torch.bfloat16)
    w = synth.tensor(647, (5, k, n), torch.bfloat16)
    lo, hi = int(off[3]), int(off[4])
    bad_a, bad_dy = a.clone(), dy.clone()
    bad_a[lo:hi] = float("inf")
    bad_dy[lo:hi] = float("nan")
    for x, y, what in ((bad_a, dy, "lhs"), (a, bad_dy, "rhs")):
        grad = torch.empty(5, k, n, device=DEV)
        coco.coco_grouped_einsum("tk,tn->ekn", coco.local([x.to(DEV)]), None, coco.local([y.to(DEV)]), None, offsets,
                                 coco.local([grad]))
        coco.coco_device_status()
        want = oracle.grouped_einsum("grad", f64(a), f64(dy), off)
        mag = oracle.grouped_einsum("grad", np.abs(f64(a)), np.abs(f64(dy)), off)
        for e in (0, 1, 2, 4):
            within(f64(grad[e]), want[e], gamma(256) * mag[e] + 1e-30, f"{what} expert {e}")
        assert not torch.isfinite(grad[3]).any()
    out = torch.empty(rows, n, dtype=torch.bfloat16, device=DEV)
    coco.coco_grouped_einsum("tk,ekn->tn", coco.local([bad_a.to(DEV)]), None, coco.local([w.to(DEV)]), None, offsets,
                             coco.local([out]))
    coco.coco_device_status()
    keep = torch.ones(rows, dtype=torch.bool)
    keep[lo:hi] = False
    assert torch.isfinite(out.cpu()[keep]).all()


def test_gradients_are_the_products_adjoints():
    """<dy, x @ w> = <dx, x> = <dw, w>: the difference quotient of a bilinear map is the map itself."""
    counts, k, n = [33, 0, 129, 6], 256, 144
    off = offsets_of(counts)
    rows = int(off[-1])
    offsets = torch.from_numpy(off).to(DEV, torch.int32)
    x, dy = (synth.tensor(s, (rows, c), torch.bfloat16).to(DEV) for s, c in ((648, k), (649, n)))
    w = synth.tensor(650, (4, k, n), torch.bfloat16).to(DEV)
    y, dx, dw = torch.empty(rows, n, device=DEV), torch.empty(rows, k, device=DEV), torch.empty(4, k, n, device=DEV)
    coco.coco_grouped_einsum("tk,ekn->tn", coco.local([x]), None, coco.local([w]), None, offsets, coco.local([y]))
    coco.coco_grouped_einsum("tk,enk->tn", coco.local([dy]), None, coco.local([w]), None, offsets, coco.local([dx]))
    coco.coco_grouped_einsum("tk,tn->ekn", coco.local([x]), None, coco.local([dy]), None, offsets, coco.local([dw]))
    coco.coco_device_status()
    dot = lambda a, b: float((a.double() * b.double()).sum())  # noqa: E731
    scale = float(y.double().norm() * dy.double().norm())
    assert abs(dot(dy, y) - dot(dx, x)) <= 1e-6 * scale
    assert abs(dot(dy, y) - dot(dw, w)) <= 1e-6 * scale


def test_ranks_have_their_own_routing():
    ranks, k, n, experts, rows = 3, 128, 144, 4, 50
    offs = np.array([[0, 10, 10, 50, 50], [3, 3, 20, 21, 40], [0, 0, 0, 0, 50]])
    xs = dev(synth.per_rank(651, 0, ranks, (rows, k), torch.float16))
    ws = dev(synth.per_rank(651, 1, ranks, (experts, k, n), torch.float16))
    out = [torch.empty(rows, n, device=DEV) for _ in range(ranks)]
    coco.coco_grouped_einsum("tk,ekn->tn", coco.local(xs), None, coco.local(ws), None,
                             torch.from_numpy(offs).to(DEV, torch.int32), coco.local(out))
    coco.coco_device_status()
    for r in range(ranks):
        want = oracle.grouped_einsum("kn", f64(xs[r]), f64(ws[r]), offs[r])
        mag = oracle.grouped_einsum("kn", np.abs(f64(xs[r])), np.abs(f64(ws[r])), offs[r])
        within(f64(out[r]), want, gamma(k) * mag + 1e-30, f"rank {r}")


def test_offsets_out_of_range_stay_inside_the_arrays():
    """Offsets past the rows are read as the number of rows, negative ones as zero (the documented clamp)."""
    k, n, rows = 64, 64, 40
    x = synth.tensor(652, (rows, k), torch.bfloat16).to(DEV)
    w = synth.tensor(653, (3, k, n), torch.bfloat16).to(DEV)
    off = torch.tensor([-7, 12, 30, 1000], dtype=torch.int32, device=DEV)
    out, check = guarded((rows, n), torch.float32)
    coco.coco_grouped_einsum("tk,ekn->tn", coco.local([x]), None, coco.local([w]), None, off, coco.local([out]))
    coco.coco_device_status()
    check()
    want = oracle.grouped_einsum("kn", f64(x), f64(w), [0, 12, 30, 40])
    mag = oracle.grouped_einsum("kn", np.abs(f64(x)), np.abs(f64(w)), [0, 12, 30, 40])
    within(f64(out), want, gamma(k) * mag + 1e-30, "clamped")


@pytest.mark.parametrize("m", [1, 200])
def test_a_call_repeats_its_bits_and_runs_in_a_graph(m):
    k, n = 1024, 528
    a, sa, _ = eight_bits(synth.tensor(654, (m, k), torch.float32), 1)
    b, sb, _ = eight_bits(synth.tensor(655, (n, k), torch.float32), 128)
    outs = [torch.empty(m, n, dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    call = lambda o, s=None: coco.coco_einsum_fp8("mk,nk->mn", coco.local([a]), [sa], coco.local([b]), [sb],  # noqa: E731
                                                  coco.local([o]), s)
    call(outs[0])
    call(outs[1])
    torch.cuda.synchronize()
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call(outs[2], side)
    graph.replay()
    coco.coco_device_status()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
