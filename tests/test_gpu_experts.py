"""Rows to their experts and back, through the C-ABI, against the float64 oracle.

Tolerances, with u the half step of the stored type and e = 2^-24. Sorting and dispatching are exact. A combined value is an
fp32 sum of n ranks, a product, a sum of k choices and of the residual: within (n + k + 2) e of the terms' magnitudes,
then one rounding. A row's gradient is one fp32 product and one rounding. A gate's gradient sums the ranks, then at most 64
values a lane, 5 shuffles and 16 warps: within (n + 100) e of its terms' magnitudes.
"""

import numpy as np
import pytest
import torch

import oracle
from collective_fusedallreduce_gb300 import coco, synth
from test_gpu_llm_norm import DEV, E, F8, TINY, U, dev, f64, guarded, within

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def routing(seed, tokens, choices, experts, dropped=0.15):
    """Choices of uneven experts, some of none."""
    rng = np.random.default_rng(seed)
    e = np.minimum(rng.geometric(4 / (experts + 4), (tokens, choices)) - 1, max(experts - 1, 0))
    return np.where(rng.random(e.shape) < dropped, rng.choice([-1, -7, experts, experts + 9], e.shape), e)


def sort(expert_of, experts, groups=1, ranks=1, dtype=torch.int64, choice=True, stream=None):
    e = torch.from_numpy(np.ascontiguousarray(expert_of)).to(dtype).to(DEV)
    row, c0 = guarded(e.shape, torch.int32)
    of, c1 = guarded((groups, e.numel() // groups), torch.int32)
    off, c2 = guarded((groups * ranks, experts + 1), torch.int32)
    coco.coco_expert_sort(e, experts, row, of if choice else None, off, stream)
    coco.coco_device_status()
    for c in (c0, c1, c2):
        c()
    return row, of, off


SORTS = [(1, 1, 1), (1, 8, 64), (3, 2, 5), (16, 2, 64), (33, 1, 40), (1000, 3, 7), (2048, 2, 32), (2049, 2, 257),
         (4100, 1, 1), (9000, 8, 1024), (50000, 4, 128), (300, 2, 5000), (700, 3, 8192), (800, 2, 20000), (3000, 2, 65536),
         (40, 2, 0), (300001, 3, 64)]


@pytest.mark.parametrize("dtype", [torch.int64, torch.int32])
@pytest.mark.parametrize("tokens,choices,experts", SORTS)
def test_sorting(dtype, tokens, choices, experts):
    e = routing(701 + tokens, tokens, choices, experts)
    row, of, off = sort(e, experts, dtype=dtype)
    want = oracle.expert_sort(e, experts) if tokens * choices < 3000 else by_argsort(e, experts)
    assert np.array_equal(row.cpu().numpy(), want[0])
    assert np.array_equal(of.cpu().numpy()[0], want[1])
    assert np.array_equal(off.cpu().numpy()[0], want[2])


def by_argsort(e, experts):
    flat = e.reshape(-1)
    key = np.where((flat >= 0) & (flat < experts), flat, experts)
    order = np.argsort(key, kind="stable")
    live = int((key < experts).sum())
    row, of = np.full(flat.size, -1), np.full(flat.size, -1)
    row[order[:live]] = np.arange(live)
    of[:live] = order[:live]
    return row.reshape(e.shape), of, np.searchsorted(key[order], np.arange(experts + 1))


def test_sorting_all_to_one_expert_none_and_numbers_past_32_bits():
    for e, experts in [(np.full((5000, 2), 3), 9), (np.full((5000, 2), -1), 9), (np.zeros((70, 2), np.int64), 1)]:
        row, of, off = sort(e, experts)
        want = by_argsort(e, experts)
        assert np.array_equal(row.cpu().numpy(), want[0]) and np.array_equal(of.cpu().numpy()[0], want[1])
        assert np.array_equal(off.cpu().numpy()[0], want[2])
    e = np.array([[2 ** 32, 1], [2 ** 40 + 1, -2 ** 33], [1, 0]])  # experts 0 and 1 in their low 32 bits
    row, _, off = sort(e, 2)
    assert row.tolist() == [[-1, 1], [-1, -1], [2, 0]] and off.tolist() == [[0, 1, 3]]


def test_sorting_groups_and_without_the_rows_choices():
    groups, ranks, tokens, choices, experts = 3, 4, 2500, 2, 11
    e = routing(702, groups * tokens, choices, experts).reshape(groups, tokens, choices)
    row, of, off = sort(e, experts, groups, ranks)
    again = sort(e, experts, groups, ranks, choice=False)
    assert torch.equal(again[0], row) and torch.equal(again[2], off)
    for g in range(groups):
        want = by_argsort(e[g], experts)
        assert np.array_equal(row[g].cpu().numpy(), want[0]) and np.array_equal(of[g].cpu().numpy(), want[1])
        for r in range(ranks):
            assert np.array_equal(off[g * ranks + r].cpu().numpy(), want[2])


def test_sorting_nothing_writes_zero_offsets():
    for shape in [(0, 2), (3, 0)]:
        off = torch.full((2, 5), 7, dtype=torch.int32, device=DEV)
        none = torch.empty(shape, dtype=torch.int64, device=DEV)
        coco.coco_expert_sort(none, 4, torch.empty(shape, dtype=torch.int32, device=DEV), None, off)
        torch.cuda.synchronize()
        assert not off.any()


ROWS = [(1, 1, 16), (5, 2, 144), (1, 8, 4096), (33, 3, 272), (700, 2, 1040), (9, 4, 16400), (2, 2, 32768), (300, 1, 512)]


@pytest.mark.parametrize("dtype", TYPES + [F8])
@pytest.mark.parametrize("tokens,choices,cols", ROWS)
def test_dispatch(dtype, tokens, choices, cols):
    x = synth.tensor(703, (tokens, cols), torch.float32).to(dtype).to(DEV)
    nb = -(-cols // 128)
    s = synth.tensor(704, (tokens, nb), torch.float32).to(DEV) if dtype is F8 else None
    row_of = sort(routing(705, tokens, choices, 6), 6)[0]
    n = tokens * choices
    rows, c0 = guarded((n, cols), dtype)
    scales, c1 = guarded((n, nb), torch.float32)
    before, sbefore = rows.view(torch.uint8).clone(), scales.clone()
    coco.coco_expert_dispatch(coco.replicated([x]), None if s is None else [s], row_of, coco.replicated([rows]),
                              None if s is None else [scales])
    coco.coco_device_status()
    c0(), c1()
    bytes_of = lambda t: t.view(torch.uint8).cpu().numpy()  # noqa: E731
    at = row_of.cpu().numpy()
    assert np.array_equal(bytes_of(rows), oracle.expert_dispatch(bytes_of(x), at, before.cpu().numpy()))
    if s is None:
        assert torch.equal(scales.view(torch.int32), sbefore.view(torch.int32))
    else:
        assert np.array_equal(bytes_of(scales), oracle.expert_dispatch(bytes_of(s), at, bytes_of(sbefore)))


@pytest.mark.parametrize("dtype", [torch.bfloat16, F8])
def test_dispatch_to_groups_and_their_copies(dtype):
    groups, ranks, tokens, choices, cols = 2, 3, 20, 2, 144
    e = routing(706, groups * tokens, choices, 4).reshape(groups, tokens, choices)
    row_of = sort(e, 4, groups, ranks)[0]
    x = [t.to(dtype).to(DEV) for t in synth.per_rank(707, 0, groups, (tokens, cols), torch.float32)]
    s = dev(synth.per_rank(707, 1, groups, (tokens, 2), torch.float32))
    out = [torch.zeros(tokens * choices, cols, device=DEV).to(dtype) for _ in range(groups * ranks)]
    so = [torch.zeros(tokens * choices, 2, device=DEV) for _ in range(groups * ranks)]
    rep, fp8 = lambda ts: [t for t in ts for _ in range(ranks)], dtype is F8  # noqa: E731
    coco.coco_expert_dispatch(coco.replicated(rep(x), groups), rep(s) if fp8 else None, row_of,
                              coco.replicated(out, groups), so if fp8 else None)
    torch.cuda.synchronize()
    for g in range(groups):
        at = row_of[g].cpu().numpy()
        want = oracle.expert_dispatch(f64(x[g]), at, np.zeros((tokens * choices, cols)))
        for r in range(ranks):
            assert np.array_equal(f64(out[g * ranks + r]), want)
            if fp8:
                assert np.array_equal(f64(so[g * ranks + r]), oracle.expert_dispatch(f64(s[g]), at, np.zeros((len(want), 2))))


def combine_case(dtype, n, tokens, choices, cols, seed=711):
    rows = dev(synth.per_rank(seed, 0, n, (tokens * choices, cols), dtype, std=n ** -0.5))
    gates = synth.tensor(seed + 1, (tokens, choices), torch.float32).to(DEV)
    row_of = sort(routing(seed, tokens, choices, 6), 6)[0]
    return rows, gates, row_of


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 2, 5, 8])
@pytest.mark.parametrize("tokens,choices,cols", ROWS)
def test_combine(dtype, n, tokens, choices, cols):
    rows, gates, row_of = combine_case(dtype, n, tokens, choices, cols)
    res = synth.tensor(713, (tokens, cols), dtype).to(DEV)
    at, r64 = row_of.cpu().numpy(), [f64(r) for r in rows]
    for weights, residual in [(gates, res), (None, None)]:
        outs, checks = zip(*[guarded((tokens, cols), dtype) for _ in range(n)])
        one, check = guarded((tokens, cols), dtype)
        coco.coco_expert_combine(coco.local(rows), row_of, weights, None, coco.local(outs))
        coco.coco_expert_combine(coco.local(rows), row_of, weights,
                                 None if residual is None else coco.replicated([residual] * n), coco.replicated([one] * n))
        coco.coco_device_status()
        for c in checks + (check,):
            c()
        w = None if weights is None else f64(weights)
        mag = lambda ts, r: oracle.expert_combine([np.abs(t) for t in ts], at, None if w is None else np.abs(w), r)  # noqa: E731,B023
        for r in range(n):
            want = oracle.expert_combine([r64[r]], at, w, None)
            within(f64(outs[r]), want, np.abs(want) * U[dtype] * 1.01 + (choices + 3) * E * mag([r64[r]], None)
                   + TINY[dtype], "a rank's sum")
        rr = None if residual is None else f64(residual)
        want = oracle.expert_combine(r64, at, w, rr)
        within(f64(one), want, np.abs(want) * U[dtype] * 1.01 + TINY[dtype]
               + (n + choices + 2) * E * mag(r64, None if rr is None else np.abs(rr)), "the sum over ranks")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("n", [1, 2, 5, 8])
@pytest.mark.parametrize("tokens,choices,cols", ROWS)
def test_combine_backward(dtype, n, tokens, choices, cols):
    rows, gates, row_of = combine_case(dtype, n, tokens, choices, cols, 721)
    dout = synth.tensor(723, (tokens, cols), dtype).to(DEV)
    at, r64, d64 = row_of.cpu().numpy(), [f64(r) for r in rows], f64(dout)
    for weights, grads in [(gates, True), (None, True), (gates, False)]:
        drows, c0 = guarded((tokens * choices, cols), dtype)
        dgates, c1 = guarded((tokens, choices), torch.float32)
        before = f64(drows)
        coco.coco_expert_combine_backward(coco.replicated([dout] * n), coco.local(rows) if grads else None, row_of,
                                          weights, coco.replicated([drows] * n), dgates if grads else None)
        coco.coco_device_status()
        c0(), c1()
        w = None if weights is None else f64(weights)
        want, wantg = oracle.expert_combine_backward(d64, r64, at, w, before)
        named = np.zeros(tokens * choices, bool)
        named[at[at >= 0]] = True
        got = f64(drows)
        assert np.array_equal(got[~named], before[~named])
        bound = np.abs(want[named]) * (U[dtype] * 1.01 + 2 * E) + TINY[dtype]
        within(got[named], want[named], bound, "drows")
        if grads:
            mag = oracle.expert_combine_backward(np.abs(d64), [np.abs(r) for r in r64], at, None, np.zeros_like(r64[0]))[1]
            within(f64(dgates), wantg, (n + 100) * E * mag, "dgates")


def test_gradients_are_difference_quotients():
    """Combining is linear in the rows and in the gates: the quotient is exact but for the forward's fp32 rounding."""
    n, tokens, choices, cols = 2, 12, 3, 136
    rows, gates, row_of = combine_case(torch.float32, n, tokens, choices, cols, 731)
    dout = synth.tensor(733, (tokens, cols), torch.float32).to(DEV)
    out = torch.empty(tokens, cols, device=DEV)

    def loss(r0, g):
        coco.coco_expert_combine(coco.local([r0, rows[1]]), row_of, g, None, coco.replicated([out] * n))
        torch.cuda.synchronize()
        return float((out.double() * dout.double()).sum())

    drows, dgates = torch.zeros_like(rows[0]), torch.empty_like(gates)
    coco.coco_expert_combine_backward(coco.replicated([dout] * n), coco.local(rows), row_of, gates,
                                      coco.replicated([drows] * n), dgates)
    g = torch.Generator().manual_seed(734)
    at, d64 = row_of.cpu().numpy(), np.abs(f64(dout))
    for _ in range(3):
        # either forward's outputs are within (n + choices + 2) e of their terms' magnitudes (and the operand's own sum, e)
        d = torch.randn(rows[0].shape, generator=g).to(DEV)
        got, want = loss(rows[0] + d, gates) - loss(rows[0] - d, gates), 2 * float((drows.double() * d.double()).sum())
        mag = np.sum(d64 * oracle.expert_combine([np.abs(f64(r)) for r in (rows[0], rows[1], d)], at, np.abs(f64(gates)), None))
        assert abs(got - want) <= 2 * (n + choices + 3) * E * mag + 2 * E * mag
        d = torch.randn(gates.shape, generator=g).to(DEV)
        got, want = loss(rows[0], gates + d) - loss(rows[0], gates - d), 2 * float((dgates.double() * d.double()).sum())
        mag = np.sum(d64 * oracle.expert_combine([np.abs(f64(r)) for r in rows], at, np.abs(f64(gates)) + np.abs(f64(d)), None))
        assert abs(got - want) <= 2 * (n + choices + 3) * E * mag + 2 * (n + 100) * E * mag
    # the dispatch's gradient: <rows, dispatch(x)> = <combine(rows), x>
    x = synth.tensor(735, (tokens, cols), torch.float32).to(DEV)
    sent = torch.zeros_like(rows[0])
    coco.coco_expert_dispatch(coco.replicated([x]), None, row_of, coco.replicated([sent]), None)
    coco.coco_expert_combine(coco.local([rows[0]]), row_of, None, None, coco.local([out]))
    torch.cuda.synchronize()
    a, b = float((sent.double() * rows[0].double()).sum()), float((out.double() * x.double()).sum())
    mag = np.sum(np.abs(f64(x)) * oracle.expert_combine([np.abs(f64(rows[0]))], at, None, None))
    assert abs(a - b) <= (choices + 1) * E * mag


def test_what_no_choice_names_does_not_matter():
    """NaN in rows that nothing names and in the gates of choices without a row; tokens all of whose choices have none."""
    n, tokens, choices, cols = 3, 30, 2, 256
    rows, gates, row_of = combine_case(torch.bfloat16, n, tokens, choices, cols, 741)
    row_of[4] = -1
    row_of[7, 0], row_of[8, 1], row_of[9, 0] = tokens * choices, -5, 2 ** 31 - 1  # not rows
    lost = (row_of < 0) | (row_of >= tokens * choices)
    named = torch.zeros(tokens * choices, dtype=torch.bool, device=DEV)
    named[row_of[~lost].long()] = True
    gates[lost] = float("nan")
    for r in rows:
        r[~named] = float("nan")
    res = synth.tensor(743, (tokens, cols), torch.bfloat16).to(DEV)
    out = torch.empty_like(res)
    coco.coco_expert_combine(coco.local(rows), row_of, gates, coco.replicated([res] * n), coco.replicated([out] * n))
    dgates = torch.full_like(gates, 7.0)
    drows = torch.full_like(rows[0], 3.0)
    coco.coco_expert_combine_backward(coco.replicated([res] * n), coco.local(rows), row_of, gates,
                                      coco.replicated([drows] * n), dgates)
    coco.coco_device_status()
    assert bool(torch.isfinite(out).all()) and torch.equal(out[4], res[4])
    assert bool((dgates[lost] == 0).all()) and bool(torch.isfinite(dgates).all())
    assert bool((drows[~named] == 3.0).all()) and bool(torch.isfinite(drows).all())


def test_rows_without_choices_and_the_residuals_place():
    tokens, cols, n = 6, 144, 4
    res = dev([synth.tensor(751, (tokens, cols), torch.float16)])[0]
    none = [torch.empty(0, cols, dtype=torch.float16, device=DEV)] * n
    nowhere = torch.empty(tokens, 0, dtype=torch.int32, device=DEV)
    out = torch.full_like(res, 9.0)
    coco.coco_expert_combine(coco.local(none), nowhere, None, coco.replicated([res] * n), coco.replicated([out] * n))
    own = [torch.full_like(res, 9.0) for _ in range(n)]
    coco.coco_expert_combine(coco.local(none), nowhere, None, None, coco.local(own))
    torch.cuda.synchronize()
    assert torch.equal(out, res) and not any(bool(o.any()) for o in own)
    rows, gates, row_of = combine_case(torch.float16, n, tokens, 2, cols, 752)
    coco.coco_expert_combine(coco.local(rows), row_of, gates, coco.replicated([res] * n), coco.replicated([out] * n))
    coco.coco_expert_combine(coco.local(rows), row_of, gates, coco.replicated([res] * n), coco.replicated([res] * n))
    torch.cuda.synchronize()
    assert torch.equal(out, res)


def test_groups_of_ranks():
    groups, n, tokens, choices, cols = 2, 2, 11, 2, 272
    e = routing(761, groups * tokens, choices, 4).reshape(groups, tokens, choices)
    row_of = sort(e, 4, groups, n)[0]
    rows = dev(synth.per_rank(762, 0, groups * n, (tokens * choices, cols), torch.bfloat16))
    gates = synth.tensor(763, (groups, tokens, choices), torch.float32).to(DEV)
    dout = dev(synth.per_rank(764, 0, groups, (tokens, cols), torch.bfloat16))
    rep = lambda ts: [t for t in ts for _ in range(n)]  # noqa: E731
    out = [torch.empty_like(dout[0]) for _ in range(groups)]
    own = [torch.empty_like(dout[0]) for _ in range(groups * n)]
    drows = [torch.zeros_like(rows[0]) for _ in range(groups * n)]
    dgates = torch.empty_like(gates)
    coco.coco_expert_combine(coco.local(rows, groups), row_of, gates, coco.replicated(rep(dout), groups),
                             coco.replicated(rep(out), groups))
    coco.coco_expert_combine(coco.local(rows, groups), row_of, gates, None, coco.local(own, groups))
    coco.coco_expert_combine_backward(coco.replicated(rep(dout), groups), coco.local(rows, groups), row_of, gates,
                                      coco.replicated(drows, groups), dgates)
    torch.cuda.synchronize()
    # values of at most some ten, so fp32's part of a bf16 bound is below 1e-5
    for g in range(groups):
        at, w, d = row_of[g].cpu().numpy(), f64(gates[g]), f64(dout[g])
        mine = [f64(r) for r in rows[g * n:g * n + n]]
        want = oracle.expert_combine(mine, at, w, d)
        within(f64(out[g]), want, np.abs(want) * 2.0 ** -8 * 1.01 + 1e-5, "sum")
        for r in range(n):
            want = oracle.expert_combine([mine[r]], at, w, None)
            within(f64(own[g * n + r]), want, np.abs(want) * 2.0 ** -8 * 1.01 + 1e-5, "a rank's sum")
        want, wantg = oracle.expert_combine_backward(d, mine, at, w, np.zeros(mine[0].shape))
        for r in range(n):
            within(f64(drows[g * n + r]), want, np.abs(want) * 2.0 ** -8 * 1.001 + 1e-9, "drows")
        mag = oracle.expert_combine_backward(np.abs(d), [np.abs(m) for m in mine], at, None, np.zeros(mine[0].shape))[1]
        within(f64(dgates[g]), wantg, (n + 100) * E * mag, "dgates")


def test_captured_and_replayed_with_new_routings():
    """Routing, dispatch and combination in one graph, beside a second graph of the same calls on another stream."""
    tokens, choices, experts, cols = 500, 2, 16, 512

    def graph_of(stream):
        s = {"e": torch.zeros(tokens, choices, dtype=torch.int64, device=DEV), "x": torch.zeros(tokens, cols, device=DEV),
             "row": torch.empty(tokens, choices, dtype=torch.int32, device=DEV),
             "off": torch.empty(1, experts + 1, dtype=torch.int32, device=DEV),
             "rows": torch.zeros(tokens * choices, cols, device=DEV), "out": torch.empty(tokens, cols, device=DEV)}
        torch.cuda.synchronize()
        s["graph"] = torch.cuda.CUDAGraph()
        with torch.cuda.graph(s["graph"], stream=stream):
            coco.coco_expert_sort(s["e"], experts, s["row"], None, s["off"])
            coco.coco_expert_dispatch(coco.replicated([s["x"]]), None, s["row"], coco.replicated([s["rows"]]), None)
            coco.coco_expert_combine(coco.local([s["rows"]]), s["row"], None, None, coco.local([s["out"]]))
        return s

    streams = [torch.cuda.Stream() for _ in range(2)]
    both = [graph_of(st) for st in streams]
    for turn in range(3):
        for i, s in enumerate(both):
            e = routing(770 + 2 * turn + i, tokens, choices, experts)
            s["e"].copy_(torch.from_numpy(e))
            s["x"].copy_(synth.tensor(780 + 2 * turn + i, (tokens, cols), torch.float32))
            s["want"] = e
        torch.cuda.synchronize()
        for s, st in zip(both, streams):
            with torch.cuda.stream(st):
                s["graph"].replay()
        torch.cuda.synchronize()
        for s in both:
            want = by_argsort(s["want"], experts)
            assert np.array_equal(s["row"].cpu().numpy(), want[0]) and np.array_equal(s["off"].cpu().numpy()[0], want[2])
            live = torch.from_numpy((want[0] >= 0).sum(1)).to(DEV)[:, None]
            assert torch.equal(s["out"], s["x"] * live)  # a token's own row, once or twice: exact
