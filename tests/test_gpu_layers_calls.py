"""Calls of the experts', layer norm's and clipping's entry points that the parity tests do not make: a process's first
call under capture, two threads at once, a stream of the caller's beside work on another, arrays past 2^32 elements, and
graphs that share nothing but the device."""

import os
import subprocess
import sys
import threading

import pytest
import torch

from collective_fusedallreduce_gb300 import coco

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
F8 = torch.float8_e4m3fn


class Calls:
    """One call of every entry point on tensors of its own, and what it wrote."""

    def __init__(self, seed, tokens=700, choices=2, experts=16, cols=1040, ranks=2):
        g = torch.Generator(device=DEV).manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
        n = tokens * choices
        self.e = torch.randint(-1, experts, (tokens, choices), generator=g, device=DEV)
        self.row, self.of = torch.zeros(tokens, choices, dtype=torch.int32, device=DEV), torch.zeros(n, dtype=torch.int32, device=DEV)
        self.off = torch.zeros(ranks, experts + 1, dtype=torch.int32, device=DEV)
        self.x, self.w, self.b = rnd(tokens, cols).bfloat16(), rnd(cols).bfloat16(), rnd(cols).bfloat16()
        self.rows = [rnd(n, cols).bfloat16() for _ in range(ranks)]
        self.sent, self.out, self.dx = torch.zeros(n, cols, device=DEV).bfloat16(), torch.zeros_like(self.x), torch.zeros_like(self.x)
        self.drows, self.dgates = torch.zeros_like(self.sent), torch.zeros(tokens, choices, device=DEV)
        self.gates = torch.rand(tokens, choices, generator=g, device=DEV)
        self.y, self.h = torch.zeros_like(self.x), torch.zeros_like(self.x)
        self.mean, self.rstd = torch.zeros(tokens, device=DEV), torch.zeros(tokens, device=DEV)
        self.dw, self.db = torch.zeros(cols, device=DEV), torch.zeros(cols, device=DEV)
        self.ws = torch.empty(coco.coco_allreduce_layernorm_backward_bytes(tokens, cols), dtype=torch.uint8, device=DEV)
        grads = [[rnd(s) for s in (5000, 7, 100000)] for _ in range(ranks)]
        self.clipped = [[torch.zeros_like(t).bfloat16() for t in row] for row in grads]
        self.grads = grads
        self.tables = [torch.empty(coco.coco_scattered_table_bytes([t.numel() for t in grads[0]], ranks), dtype=torch.uint8,
                                   device=DEV) for _ in range(2)]
        self.plans = [coco.coco_scattered_table_build(p, t) for p, t in zip((grads, self.clipped), self.tables)]
        self.norm = torch.zeros(2, device=DEV)
        self.space = torch.empty(coco.coco_scattered_clip_bytes(), dtype=torch.uint8, device=DEV)
        self.ranks, self.experts = ranks, experts
        torch.cuda.synchronize()

    def __call__(self, stream=None):
        rep = lambda t: coco.replicated([t] * self.ranks)  # noqa: E731
        coco.coco_expert_sort(self.e, self.experts, self.row, self.of, self.off, stream)
        coco.coco_expert_dispatch(rep(self.x), None, self.row, rep(self.sent), None, stream)
        coco.coco_expert_combine(coco.local(self.rows), self.row, self.gates, rep(self.x), rep(self.out), stream)
        coco.coco_expert_combine_backward(rep(self.x), coco.local(self.rows), self.row, self.gates, rep(self.drows),
                                          self.dgates, stream)
        coco.coco_allreduce_layernorm(coco.local([self.out] * self.ranks), rep(self.x), self.w, self.b, 1e-5, rep(self.h),
                                      rep(self.y), None, self.mean, self.rstd, stream)
        coco.coco_allreduce_layernorm_backward(coco.local([self.y] * self.ranks), rep(self.x), rep(self.h), self.w, self.mean,
                                               self.rstd, rep(self.dx), self.dw, self.db, self.ws, stream)
        coco.coco_scattered_clip(self.plans[0], coco.LOCAL, 1.0, self.plans[1], self.norm[:1], self.space, stream)
        coco.coco_scattered_allreduce_clip(self.plans[0], 0.5, 2.0, self.plans[1], self.norm[1:], self.space, stream)

    def wrote(self):
        return [self.row, self.of, self.off, self.sent, self.out, self.drows, self.dgates, self.h, self.y, self.mean,
                self.rstd, self.dx, self.dw, self.db, self.norm] + [t for r in self.clipped for t in r]

    def taken(self):
        torch.cuda.synchronize()
        got = [t.clone() for t in self.wrote()]
        for t in self.wrote():
            t.zero_()
        torch.cuda.synchronize()
        return got


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def first_call_under_capture():
    c = Calls(901)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c()
    graph.replay()
    got = c.taken()
    c()
    assert same(got, c.taken())
    coco.coco_device_status()


def test_a_process_can_start_with_a_capture():
    here = os.path.dirname(os.path.abspath(__file__))
    code = f"import sys; sys.path[:0] = [{os.path.dirname(here)!r}, {here!r}]; " \
           "import test_gpu_layers_calls as t; t.first_call_under_capture()"
    subprocess.run([sys.executable, "-c", code], check=True, timeout=300)


def test_two_threads_at_once():
    calls = [Calls(911), Calls(912, tokens=3000, choices=3, experts=100, cols=272, ranks=3)]
    want = []
    for c in calls:
        c()
        want.append(c.taken())
    streams = [torch.cuda.Stream() for _ in calls]
    failed = []

    def go(c, s):
        try:
            for _ in range(20):
                c(s)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=go, args=a) for a in zip(calls, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for c, w in zip(calls, want):
        assert same(c.taken(), w)


def test_work_stays_on_the_callers_stream():
    """The inputs come from the caller's stream, late: a call on it sees them, and what follows on it sees the call's."""
    c = Calls(921)
    side = torch.cuda.Stream()
    new_x = torch.randn_like(c.x)
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        c.x.copy_(new_x)
        c()
        early = [t.clone() for t in c.wrote()]
    torch.cuda.synchronize()
    got = c.taken()
    assert same(early, got)
    c()
    assert same(c.taken(), got)


def test_two_graphs_on_two_streams():
    calls = [Calls(931), Calls(932)]
    want, graphs, streams = [], [], [torch.cuda.Stream() for _ in range(2)]
    for c, s in zip(calls, streams):
        c()
        want.append(c.taken())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1], stream=s):
            c()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    for c, w in zip(calls, want):
        assert same(c.taken(), w)


def test_a_call_behind_its_own_copy():
    """Repeated calls without a wait between: each kernel starts behind the one before it, though some are placed early."""
    c = Calls(941)
    c()
    want = c.taken()
    for _ in range(50):
        c()
    assert same(c.taken(), want)


def test_calls_behind_copies_events_and_other_kernels_in_a_graph():
    """The dispatch, the clip's second launch and the norm gradient's last sum may be placed early; what is ahead of them
    here are a copy, a memset, an event of another stream, and PyTorch's kernels."""
    tokens, cols = 4096, 1024
    x, new = torch.zeros(tokens, cols, device=DEV), torch.randn(tokens, cols, device=DEV)
    row = torch.randperm(tokens, device=DEV, dtype=torch.int32)[:, None].contiguous()
    out = [torch.zeros(tokens, cols, device=DEV) for _ in range(4)]
    side = torch.cuda.Stream()

    def send(to):
        coco.coco_expert_dispatch(coco.replicated([x]), None, row, coco.replicated([to]), None)

    def run():
        x.copy_(new)              # a copy
        send(out[0])
        x.mul_(2.0)               # a kernel
        send(out[1])
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            x.zero_()             # another stream's work, joined by an event
            x.add_(new)
        main.wait_stream(side)
        send(out[2])
        out[3].zero_()            # a memset of what is written
        send(out[3])

    def check():
        want = torch.empty_like(x)
        want[row[:, 0].long()] = new
        assert torch.equal(out[0], want) and torch.equal(out[1], 2 * want)
        assert torch.equal(out[2], want) and torch.equal(out[3], want)

    run()
    torch.cuda.synchronize()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for _ in range(3):
        new.normal_()
        for t in out + [x]:
            t.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check()


def test_sorting_many_groups_on_wide_clusters():
    groups, tokens, choices, experts = 9, 9000, 2, 50
    e = torch.randint(-1, experts + 1, (groups, tokens, choices), device=DEV)
    row = torch.empty(groups, tokens, choices, dtype=torch.int32, device=DEV)
    of = torch.empty(groups, tokens * choices, dtype=torch.int32, device=DEV)
    off = torch.empty(groups * 2, experts + 1, dtype=torch.int32, device=DEV)
    coco.coco_expert_sort(e, experts, row, of, off)
    coco.coco_device_status()
    for g in range(groups):
        flat = e[g].reshape(-1)
        key = torch.where((flat >= 0) & (flat < experts), flat, experts)
        order = torch.argsort(key, stable=True)
        live = int((key < experts).sum())
        assert torch.equal(of[g, :live].long(), order[:live]) and bool((of[g, live:] == -1).all())
        want = torch.full_like(flat, -1)
        want[order[:live]] = torch.arange(live, device=DEV)
        assert torch.equal(row[g].reshape(-1).long(), want)
        assert torch.equal(off[2 * g].long(), torch.searchsorted(key[order], torch.arange(experts + 1, device=DEV)))
        assert torch.equal(off[2 * g], off[2 * g + 1])


@pytest.fixture
def room():
    if torch.cuda.get_device_properties(0).total_memory < 100 << 30:
        pytest.skip("needs 100 GB of device memory")
    yield
    torch.cuda.empty_cache()


def test_arrays_past_32_bits_of_elements(room):
    """2^32 elements and more, sampled against float64 on the device. Rows go to places in reverse: the first token's row is
    the last one."""
    tokens, cols = 131072 + 40, 32768
    x = torch.randn(tokens, cols, dtype=torch.bfloat16, device=DEV)
    row = torch.arange(tokens - 1, -1, -1, dtype=torch.int32, device=DEV)[:, None].contiguous()
    rows = torch.empty_like(x)
    at = torch.tensor(sorted({t for a in (0, tokens - 1, (1 << 31) // cols, (1 << 32) // cols, tokens - 1 - (1 << 32) // cols)
                              for t in (a - 1, a, a + 1) if 0 <= t < tokens}), device=DEV)
    coco.coco_expert_dispatch(coco.replicated([x]), None, row, coco.replicated([rows]), None)
    coco.coco_device_status()
    assert torch.equal(rows[tokens - 1 - at], x[at])
    gates = torch.rand(tokens, 1, device=DEV)
    out = torch.empty_like(x)
    coco.coco_expert_combine(coco.local([rows]), row, gates, coco.replicated([x]), coco.replicated([out]))
    coco.coco_device_status()
    want = x[at].double() * (1 + gates[at].double())
    assert bool(((out[at].double() - want).abs() <= want.abs() * (2.0 ** -8 + 1e-6)).all())
    dgates = torch.empty_like(gates)
    coco.coco_expert_combine_backward(coco.replicated([x]), coco.local([rows]), row, gates, coco.replicated([out]), dgates)
    coco.coco_device_status()
    want = x[at].double() * gates[at].double()
    assert bool(((out[tokens - 1 - at].double() - want).abs() <= want.abs() * (2.0 ** -8 + 1e-6)).all())
    square = x[at].double().square().sum(-1)
    assert bool(((dgates[at, 0].double() - square).abs() <= square * 110 * 2.0 ** -24).all())
    w, b = torch.ones(cols, dtype=torch.bfloat16, device=DEV), torch.zeros(cols, dtype=torch.bfloat16, device=DEV)
    mean, rstd = torch.empty(tokens, device=DEV), torch.empty(tokens, device=DEV)
    coco.coco_allreduce_layernorm(coco.local([x]), None, w, b, 1e-5, None, coco.replicated([out]), None, mean, rstd)
    coco.coco_device_status()
    h = x[at].double()
    m = h.mean(-1, keepdim=True)
    want = (h - m) * ((h - m).square().mean(-1, keepdim=True) + 1e-5).rsqrt()
    assert bool(((out[at].double() - want).abs() <= want.abs() * (2.0 ** -8 + 3e-5) + 3e-5).all())
    dw, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
    ws = torch.empty(coco.coco_allreduce_layernorm_backward_bytes(tokens, cols), dtype=torch.uint8, device=DEV)
    coco.coco_allreduce_layernorm_backward(coco.local([rows]), None, coco.replicated([x]), w, mean, rstd,
                                           coco.replicated([out]), dw, db, ws)
    coco.coco_device_status()
    g, xhat, r = rows[at].double(), (h - mean[at, None].double()) * rstd[at, None].double(), rstd[at, None].double()
    want = r * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
    terms = r * (g.abs() + g.abs().mean(-1, keepdim=True) + xhat.abs() * (g * xhat).abs().mean(-1, keepdim=True))
    assert bool(((out[at].double() - want).abs() <= want.abs() * 2.0 ** -8 * 1.01 + 161 * 2.0 ** -24 * terms).all())
    # the parameters' gradients, over all rows, of a few columns
    some = torch.tensor([0, 1, 17, cols - 1], device=DEV)
    gs, hs = rows[:, some].double(), (x[:, some].double() - mean[:, None].double()) * rstd[:, None].double()
    for got, want, mag in ((dw[some], (gs * hs).sum(0), (gs * hs).abs().sum(0)), (db[some], gs.sum(0), gs.abs().sum(0))):
        assert bool(((got.double() - want).abs() <= (tokens + 17) * 2.0 ** -24 * mag).all())
    # clipping: one tensor of 2^32 - 8 elements (the table's largest)
    del rows, out
    flat = x.view(-1)[:(1 << 32) - 8]
    table = torch.empty(coco.coco_scattered_table_bytes([flat.numel()], 1), dtype=torch.uint8, device=DEV)
    plan = coco.coco_scattered_table_build([[flat]], table)
    norm, space = torch.empty(1, device=DEV), torch.empty(coco.coco_scattered_clip_bytes(), dtype=torch.uint8, device=DEV)
    ends = torch.cat([flat[:1000], flat[(1 << 31) - 500:(1 << 31) + 500], flat[-1000:]]).double()
    want = sum(float(c.double().square().sum()) for c in flat.split(1 << 28)) ** 0.5
    coco.coco_scattered_clip(plan, coco.LOCAL, 1.0, None, norm, space)
    coco.coco_device_status()
    assert abs(float(norm) - want) <= 40 * 2.0 ** -24 * want
    got = torch.cat([flat[:1000], flat[(1 << 31) - 500:(1 << 31) + 500], flat[-1000:]]).double()
    assert bool(((got - ends / want).abs() <= (ends / want).abs() * (2.0 ** -8 + 1e-5) + 1e-30).all())
    assert bool((x.view(-1)[(1 << 32) - 8:].abs() <= 10).all()) and float(x.view(-1)[(1 << 32) - 8:].abs().max()) > 1e-3
