"""Clipping scattered gradients by their global norm, through the C-ABI, against the float64 oracle.

Tolerances, with u the half step of the stored type and e = 2^-24. Squares of one lane's 32 values are summed in fp32, the rest in
fp64: the norm is within 40 e, relative. A scaled value has the norm's error, the factor's rounding and the product's:
50 e, and one rounding. The AllReduce's sum is within (n + 1) e of its terms' magnitudes and rounded once, and so is its norm
(the triangle inequality).
"""

import numpy as np
import pytest
import torch

import oracle
from collective_fusedallreduce_gb300 import coco, synth
from test_gpu_llm_norm import DEV, E, TINY, U, f64

pytestmark = pytest.mark.gpu
TYPES = [torch.bfloat16, torch.float16, torch.float32]
SIZES = [(7,), (1,), (0,), (1023,), (1024,), (1025,), (3, 5000), (64, 1000), (100003,), (2055,)]
INF = float("inf")


def gradients(seed, n, dtype, sizes=SIZES, std=1.0):
    return [[synth.tensor(synth.seed_of(seed, t, r), s, dtype, std=std).to(DEV) for t, s in enumerate(sizes)]
            for r in range(n)]


class Guarded:
    """Tensors inside buffers of sentinel bytes, a plan of them, and the check that these are untouched."""

    def __init__(self, per_rank):
        self.raw, self.tensors = [], []
        for row in per_rank:
            self.tensors.append([])
            for t in row:
                raw = torch.full((t.nbytes + 512,), 0xA5, dtype=torch.uint8, device=DEV)
                view = raw[256:256 + t.nbytes].view(t.dtype).view(t.shape)
                view.copy_(t)
                self.raw.append((raw, t.nbytes))
                self.tensors[-1].append(view)
        numels = [t.numel() for t in per_rank[0]]
        self.table = torch.empty(coco.coco_scattered_table_bytes(numels, len(per_rank)), dtype=torch.uint8, device=DEV)
        self.plan = coco.coco_scattered_table_build(self.tensors, self.table)

    def check(self):
        for raw, n in self.raw:
            assert bool((raw[:256] == 0xA5).all()) and bool((raw[256 + n:] == 0xA5).all()), "wrote outside a tensor"


def like(per_rank, ranks, dtype):
    return Guarded([[torch.zeros_like(t, dtype=dtype) for t in per_rank[0]] for _ in range(ranks)])


def space():
    return torch.full((coco.coco_scattered_clip_bytes(),), 0xFF, dtype=torch.uint8, device=DEV), torch.empty(1, device=DEV)


def flat(row):
    return np.concatenate([f64(t).ravel() for t in row])


def near(got, want, dtype, more=0.0):
    err = np.abs(got - want)
    bound = np.abs(want) * (U[dtype] * 1.01 + 50 * E) + TINY[dtype] + more
    assert np.all(err <= bound), (float(np.max(err - bound)), int(np.argmax(err - bound)))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("out_dtype", TYPES + [None])
@pytest.mark.parametrize("n", [1, 2, 5])
@pytest.mark.parametrize("share", [0.5, 1.5])
def test_clip_of_parts(dtype, out_dtype, n, share):
    g = Guarded(gradients(901, n, dtype))
    before = [flat(row) for row in g.tensors]
    want_norm = np.sqrt(sum(np.sum(b * b) for b in before))
    top = float(want_norm * share)
    want, norm64 = oracle.clip(before, top)
    out = g if out_dtype is None else like(g.tensors, n, out_dtype)
    ws, norm = space()
    coco.coco_scattered_clip(g.plan, coco.LOCAL, top, None if out_dtype is None else out.plan, norm, ws)
    coco.coco_device_status()
    g.check(), out.check()
    assert abs(float(norm) - norm64) <= 40 * E * norm64
    for r in range(n):
        near(flat(out.tensors[r]), want[r], out_dtype or dtype)
        if out_dtype is not None:
            assert np.array_equal(flat(g.tensors[r]), before[r])
        elif share > 1:
            assert np.array_equal(flat(out.tensors[r]), before[r])  # below the norm: as they were


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("out_ranks", [0, 1, 3])
def test_clip_of_copies(dtype, out_ranks):
    n = 2
    host = gradients(902, 1, dtype)[0]
    g = Guarded([[t.clone() for t in host] for _ in range(n)])
    top = 3.0
    want, norm64 = oracle.clip([flat(host)], top)
    out = like(g.tensors, out_ranks, dtype) if out_ranks else g
    ws, norm = space()
    coco.coco_scattered_clip(g.plan, coco.REPLICATED, top, out.plan if out_ranks else None, norm, ws)
    coco.coco_device_status()
    g.check(), out.check()
    assert abs(float(norm) - norm64) <= 40 * E * norm64
    for row in out.tensors:
        near(flat(row), want[0], dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("out_dtype", [torch.float32, torch.bfloat16, None])
@pytest.mark.parametrize("n,out_ranks", [(1, 1), (2, 1), (3, 3), (8, 1), (8, 2), (11, 1)])
@pytest.mark.parametrize("share", [0.5, 1.5])
def test_allreduce_clip(dtype, out_dtype, n, out_ranks, share):
    g = Guarded(gradients(903, n, dtype))
    before = [flat(row) for row in g.tensors]
    alpha = 1.0 / n
    total = sum(before) * alpha
    lost = (n + 2) * E * sum(np.abs(b) for b in before) * alpha
    kind = out_dtype or dtype
    norm64 = float(np.linalg.norm(total))
    top = norm64 * share
    out = g if out_dtype is None else like(g.tensors, out_ranks, out_dtype)
    ws, norm = space()
    coco.coco_scattered_allreduce_clip(g.plan, alpha, top, None if out_dtype is None else out.plan, norm, ws)
    coco.coco_device_status()
    g.check(), out.check()
    dn = 40 * E * norm64 + np.linalg.norm(np.abs(total) * U[kind] + lost + TINY[kind])
    assert abs(float(norm) - norm64) <= dn
    factor = min(1.0, share)
    want = total * factor
    more = np.abs(want) * (dn / norm64 + U[kind]) * 1.01 + lost + TINY[kind]
    for row in out.tensors:
        near(flat(row), want, kind, more)
        assert np.array_equal(flat(row), flat(out.tensors[0]))
    if out_dtype is not None:
        for r in range(n):
            assert np.array_equal(flat(g.tensors[r]), before[r])


def test_without_a_limit_it_is_the_allreduce_and_the_norm_alone():
    for dtype in TYPES:
        a, b = Guarded(gradients(904, 4, dtype)), Guarded(gradients(904, 4, dtype))
        ws, norm = space()
        coco.coco_scattered_allreduce(a.plan, 0.25)
        coco.coco_scattered_allreduce_clip(b.plan, 0.25, INF, None, norm, ws)
        coco.coco_device_status()
        for x, y in zip(a.tensors, b.tensors):
            assert all(torch.equal(s, t) for s, t in zip(x, y))
        keep = [t.clone() for t in b.tensors[0]]
        again = torch.empty(1, device=DEV)
        coco.coco_scattered_clip(b.plan, coco.REPLICATED, INF, None, again, ws)
        coco.coco_device_status()
        assert float(again) == float(norm) and all(torch.equal(s, t) for s, t in zip(keep, b.tensors[0]))


@pytest.mark.parametrize("size", [1e-30, 1e-22, 1e15, 1e25, 3e38])
def test_magnitudes_whose_squares_leave_fp32(size):
    host = [[torch.full((5000,), size), torch.zeros(3000), torch.full((3,), -size)]]
    g, ws_norm = Guarded(host), space()
    out = like(g.tensors, 1, torch.float32)
    coco.coco_scattered_clip(g.plan, coco.LOCAL, size, out.plan, ws_norm[1], ws_norm[0])
    coco.coco_device_status()
    x = float(np.float32(size))
    want = np.sqrt(5003.0) * x
    if want < 3.4e38:
        assert abs(float(ws_norm[1]) - want) <= 40 * E * want
    else:
        assert float(ws_norm[1]) == INF  # past fp32; the values are still clipped to it
    got = flat(out.tensors[0])
    assert np.allclose(got[:5000], x * (x / want), rtol=60 * E, atol=2.0 ** -149) and not got[5000:8000].any()


def test_zeros_no_numbers_and_a_limit_of_zero():
    sizes = [(3000,), (5,)]
    for value, top, norm_is, out_is in [(0.0, 1.0, 0.0, 0.0), (0.0, 0.0, 0.0, 0.0), (2.0, 0.0, None, 0.0)]:
        g = Guarded([[torch.full(s, value) for s in sizes]])
        ws, norm = space()
        coco.coco_scattered_clip(g.plan, coco.LOCAL, top, None, norm, ws)
        torch.cuda.synchronize()
        assert norm_is is None or float(norm) == norm_is
        assert bool((torch.cat(g.tensors[0]) == out_is).all())
    for bad in (float("nan"), INF, -INF):
        g = Guarded([[torch.ones(s) for s in sizes]])
        g.tensors[0][0][2047] = bad
        ws, norm = space()
        coco.coco_scattered_clip(g.plan, coco.LOCAL, 1.0, None, norm, ws)
        torch.cuda.synchronize()
        x = torch.cat(g.tensors[0])
        if bad != bad:
            assert bool(torch.isnan(norm).all()) and bool(torch.isnan(x).all())
        else:
            assert float(norm) == INF and bool(torch.isnan(x[2047])) and int((x == 0).sum()) == x.numel() - 1


def test_no_tensors():
    g = Guarded([[torch.empty(0)]])
    ws, norm = space()
    coco.coco_scattered_clip(g.plan, coco.LOCAL, 1.0, None, norm, ws)
    torch.cuda.synchronize()
    assert float(norm) == 0.0
    coco.coco_scattered_allreduce_clip(g.plan, 1.0, 1.0, g.plan, norm.fill_(3.0), ws)
    torch.cuda.synchronize()
    assert float(norm) == 0.0


def test_plans_of_other_tensors_are_left_alone():
    a = Guarded([[torch.ones(3000), torch.ones(1000)]])
    b = Guarded([[torch.zeros(1000), torch.zeros(3000)]])  # as many buckets
    ws, norm = space()
    for call in (lambda: coco.coco_scattered_clip(a.plan, coco.LOCAL, 1.0, b.plan, norm, ws),
                 lambda: coco.coco_scattered_clip(a.plan, coco.REPLICATED, 1.0, b.plan, norm, ws),
                 lambda: coco.coco_scattered_allreduce_clip(a.plan, 1.0, 1.0, b.plan, norm, ws)):
        norm.fill_(1.0)
        call()
        coco.coco_device_status()
        assert bool(torch.isnan(norm).all())
        a.check(), b.check()
        assert bool((torch.cat(a.tensors[0]) == 1).all())


def test_the_same_bits_again_and_from_a_graph():
    g = Guarded(gradients(905, 3, torch.bfloat16, SIZES + [(700, 1024)]))
    out = like(g.tensors, 1, torch.float32)
    ws, norm = space()
    call = lambda: coco.coco_scattered_allreduce_clip(g.plan, 1 / 3, 1.0, out.plan, norm, ws)  # noqa: E731
    call()
    torch.cuda.synchronize()
    first, n0 = flat(out.tensors[0]), float(norm)
    call()
    torch.cuda.synchronize()
    assert np.array_equal(flat(out.tensors[0]), first) and float(norm) == n0
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for t in out.tensors[0]:
        t.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert np.array_equal(flat(out.tensors[0]), first) and float(norm) == n0
