"""Clipping of gradients whose values are out of the ordinary, through the C-ABI: exact zeros, which are many in a real
model's gradients and may not cost more than other numbers, and values that are no numbers where only the norm is asked for."""

import pytest
import torch

from collective_fusedallreduce_gb300 import coco
from test_gpu_clip import INF, Guarded, like, space
from test_gpu_llm_norm import DEV

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]


def graph_times(*calls):
    """The shortest replay of each call, in ms; they take turns."""
    graphs = []
    for call in calls:
        call()
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            for _ in range(4):
                call()
    best = [float("inf")] * len(calls)
    for _ in range(12):
        for i, graph in enumerate(graphs):
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            start.record()
            graph.replay()
            end.record()
            torch.cuda.synchronize()
            best[i] = min(best[i], start.elapsed_time(end))
    return best


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("summed", [False, True])
def test_zeros_take_no_longer_than_other_numbers(dtype, summed):
    """The norm alone of 32 million values a rank, in and out of place: the same bytes whatever they are. (A walk over them
    that only lost squares need takes three to five times as long: half as long again is far from either.)"""
    ranks = 2 if summed else 1
    dense = [[torch.randn(32 << 20, device=DEV).to(dtype), torch.randn(1021, device=DEV).to(dtype)] for _ in range(ranks)]
    zeros = [[torch.zeros_like(t) for t in row] for row in dense]
    for row in zeros:
        for t in row:
            t[::3] *= -1.0  # (zeros of either sign)
    calls, norms, kept = [], [], []
    for row in (dense, zeros):
        g, (ws, norm) = Guarded(row), space()
        out = like(g.tensors, 1, torch.float32) if summed else None
        if summed:
            calls.append(lambda g=g, out=out, norm=norm, ws=ws: coco.coco_scattered_allreduce_clip(g.plan, 0.5, INF, out.plan,
                                                                                                   norm, ws))
        else:
            calls.append(lambda g=g, norm=norm, ws=ws: coco.coco_scattered_clip(g.plan, coco.LOCAL, INF, None, norm, ws))
        norms.append(norm)
        kept.append((g, out, ws))
    a, b = graph_times(*calls)
    assert float(norms[0]) > 1000 and float(norms[1]) == 0.0
    assert b <= 1.5 * a, (b, a)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_small_value_among_zeros_is_seen(dtype):
    """A value whose square fp32 loses, in a bucket of zeros and in a tensor's last one: the sum is taken in fp64."""
    x = 2.0 ** -90
    for at in (0, 517, 1023, 2047, 2050):
        for sign in (1.0, -1.0):
            g = Guarded([[torch.zeros(2051, dtype=dtype)]])
            g.tensors[0][0][at] = sign * x
            ws, norm = space()
            coco.coco_scattered_clip(g.plan, coco.LOCAL, INF, None, norm, ws)
            torch.cuda.synchronize()
            assert float(norm) == x, (at, sign)
            h = Guarded([[torch.zeros(2051, dtype=dtype)] for _ in range(3)])
            h.tensors[1][0][at] = sign * x
            coco.coco_scattered_allreduce_clip(h.plan, 1.0, INF, None, norm, ws)
            torch.cuda.synchronize()
            assert float(norm) == x and float(h.tensors[2][0][at]) == sign * x


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), INF, -INF])
def test_without_a_limit_values_stay_what_they_are(dtype, bad):
    """INFINITY asks for the norm alone (to skip a step whose gradients are no numbers, say): nothing is scaled."""
    def filled(n):
        rows = [[torch.randn(5003, device=DEV).to(dtype), torch.randn(9, device=DEV).to(dtype)] for _ in range(n)]
        rows[0][0][2050] = bad
        return rows

    def same(x, y):
        return torch.equal(x.isnan(), y.isnan()) and torch.equal(x[~x.isnan()], y[~y.isnan()])

    def seen(norm):
        return bool(torch.isnan(norm)) if bad != bad else float(norm) == INF

    rows, (ws, norm) = filled(2), space()
    for layout, ranks in ((coco.LOCAL, 2), (coco.REPLICATED, 1)):
        g, out = Guarded(rows[:ranks]), like(rows, ranks, torch.float32)
        before = [[t.clone() for t in row] for row in g.tensors]
        coco.coco_scattered_clip(g.plan, layout, INF, None, norm.zero_(), ws)
        torch.cuda.synchronize()
        assert seen(norm)
        coco.coco_scattered_clip(g.plan, layout, INF, out.plan, norm.zero_(), ws)
        torch.cuda.synchronize()
        assert seen(norm)
        g.check(), out.check()
        for b, t, o in zip(before, g.tensors, out.tensors):
            assert all(same(x, y) and same(x.float(), z) for x, y, z in zip(b, t, o))
    a, b = Guarded(rows), Guarded(rows)
    coco.coco_scattered_allreduce(a.plan, 0.5)
    coco.coco_scattered_allreduce_clip(b.plan, 0.5, INF, None, norm.zero_(), ws)
    torch.cuda.synchronize()
    assert seen(norm)
    for x, y in zip(a.tensors, b.tensors):
        assert all(same(s, t) for s, t in zip(x, y))
