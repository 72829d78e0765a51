"""A training step of an expert layer with a layer norm, weighted and dropped experts, and clipped gradients: the experts'
rows, the grouped products, the layer norm and the clipping together, against the same step in float64 and against
differences; the same step again from a graph; and the existing layers' routing by the library.

Tolerances are norms of the whole output's difference over the output's: every step rounds to bf16 (2^-8 at most, some
ten of them on the longest path, partly relu'd), 3 %, as in test_gpu_llm_layer.
"""

import numpy as np
import pytest
import torch

import oracle
from collective_fusedallreduce_gb300 import coco, synth, workloads
from test_gpu_llm_layer import far
from test_gpu_llm_norm import DEV, dev, f64

pytestmark = pytest.mark.gpu


def inputs(tokens, hid, f, experts, n, choices, seed):
    parts = synth.per_rank(seed, 0, n, (tokens, hid), torch.bfloat16, std=n ** -0.5)
    res = synth.tensor(seed + 1, (tokens, hid), torch.bfloat16)
    w = synth.tensor(seed + 2, (hid,), torch.bfloat16, std=0.1) + 1
    b = synth.tensor(seed + 3, (hid,), torch.bfloat16, std=0.1)
    up = synth.per_rank(seed, 3, n, (experts, hid, f), torch.bfloat16, std=hid ** -0.5)
    down = synth.per_rank(seed, 4, n, (experts, f, hid), torch.bfloat16, std=(f * n) ** -0.5)
    dout = synth.tensor(seed + 4, (tokens, hid), torch.bfloat16)
    g = torch.Generator().manual_seed(seed)
    expert_of = torch.rand(tokens, experts, generator=g).topk(choices, 1).indices
    expert_of[torch.rand(tokens, choices, generator=g) < 0.1] = -1
    gates = torch.rand(tokens, choices, generator=g) + 0.1
    return parts, res, w, b, up, down, expert_of, gates, dout


def step64(parts, res, w, b, up, down, expert_of, gates, dout, active=None):
    """The step in float64, a choice at a time: (out, dx, dgates, dweight, dbias, dup, ddown). ``active``: which hidden units
    are on, as decided by another forward."""
    h, x, mean, rstd = oracle.allreduce_layernorm(parts, res, w, b, 1e-5)
    out, dx, dgates = h.copy(), np.zeros_like(h), np.zeros(gates.shape)
    dup, ddown = [np.zeros_like(u) for u in up], [np.zeros_like(d) for d in down]
    for t, k in np.argwhere(expert_of >= 0):
        e, gate = expert_of[t, k], gates[t, k]
        for r, (u, d) in enumerate(zip(up, down)):
            mid = x[t] @ u[e]
            on = mid > 0 if active is None else active[r][t, k]
            y = (mid * on) @ d[e]
            out[t] += gate * y
            dgates[t, k] += y @ dout[t]
            dmid = (d[e] @ (gate * dout[t])) * on
            ddown[r][e] += np.outer(mid * on, gate * dout[t])
            dup[r][e] += np.outer(x[t], dmid)
            dx[t] += u[e] @ dmid
    dh, dw, db = oracle.allreduce_layernorm_backward([dx], dout, h, mean, rstd, w)
    return out, dh, dgates, dw, db, dup, ddown


def run(args, max_norm):
    parts, res, w, b, up, down, expert_of, gates, dout = args
    buffers = workloads.gradient_buffers([[torch.empty_like(u), torch.empty_like(d)] for u, d in zip(up, down)])
    call = lambda: workloads.moe_layer_step(parts, res, w, b, 1e-5, expert_of, gates, up, down, dout, buffers, max_norm)  # noqa: E731
    return buffers, call


def on_device(args):
    return tuple(dev(a) if isinstance(a, list) else a.to(DEV) for a in args)


@pytest.mark.parametrize("tokens,hid,f,experts,n", [(1, 128, 64, 4, 2), (50, 272, 144, 6, 2), (400, 256, 128, 8, 3)])
def test_step_against_float64(tokens, hid, f, experts, n):
    args = inputs(tokens, hid, f, experts, n, 2, 881)
    if tokens == 1:
        args[6][0] = torch.tensor([1, 3])  # (one token: both of its choices stay)
    buffers, call = run(on_device(args), float("inf"))
    got = call()
    coco.coco_device_status()
    row_of = got["row_of_choice"].cpu().numpy()
    active = [f64(m)[np.maximum(row_of, 0)] > 0 for m in got["mid"]]
    to64 = lambda a: [f64(t) for t in a] if isinstance(a, list) else f64(a)  # noqa: E731
    a64 = [to64(a) for a in args]
    a64[6] = args[6].numpy()
    out, dx, dgates, dw, db, dup, ddown = step64(*a64, active)
    assert np.array_equal(row_of < 0, a64[6] < 0)
    for name, want in [("out", out), ("dx", dx), ("dgates", dgates), ("dweight", dw), ("dbias", db)]:
        assert far(f64(got[name]), want) <= 0.03, name
    for r in range(n):
        assert far(f64(buffers["grads"][r][0]), dup[r]) <= 0.03 and far(f64(buffers["grads"][r][1]), ddown[r]) <= 0.03
    flat = lambda: np.concatenate([f64(g).ravel() for pair in buffers["grads"] for g in pair])  # noqa: E731
    whole = flat()
    assert np.isclose(float(got["norm"]), np.linalg.norm(whole), rtol=1e-5)  # of the stored values
    # clipped to a third: bf16 rounds each value once more
    buffers3, call3 = run(on_device(args), float(got["norm"]) / 3)
    got3 = call3()
    coco.coco_device_status()
    buffers = buffers3
    assert float(got3["norm"]) == float(got["norm"])
    assert np.all(np.abs(flat() - whole / 3) <= np.abs(whole / 3) * (2.0 ** -8 + 1e-5) + 1e-30)


def test_gates_gradient_is_the_difference_quotient():
    """Combining is linear in the gates: two forwards at gates +- 1/2 d differ by dgates . d, up to bf16's rounding of the
    outputs (2^-8 of each, independent: 2^-8 / sqrt(3) of the whole in the root mean square, twice)."""
    args = on_device(inputs(64, 256, 128, 4, 2, 2, 891))
    gates, dout = args[7], args[8]
    buffers, call = run(args, float("inf"))
    dgates = call()["dgates"].double()
    d = torch.randn(gates.shape, generator=torch.Generator().manual_seed(892)).to(DEV)
    ends, noise = [], 0.0
    for sign in (0.5, -0.5):
        moved = list(args)
        moved[7] = gates + sign * d
        o = run(tuple(moved), float("inf"))[1]()["out"].double()
        ends.append(float((o * dout.double()).sum()))
        noise += float((o * dout.double()).norm()) * 2.0 ** -8
    want = float((dgates * d.double()).sum())
    # (and the experts' rows, that both use, are exactly the same)
    assert abs(ends[0] - ends[1] - want) <= 4 * noise + 1e-3 * abs(want)


def test_step_from_a_graph_is_the_same():
    args = on_device(inputs(96, 256, 128, 8, 2, 2, 893))
    buffers, call = run(args, 0.5)
    call()
    torch.cuda.synchronize()
    first = call()
    torch.cuda.synchronize()
    keep = {k: v.clone() for k, v in first.items() if torch.is_tensor(v)}
    grads = [g.clone() for pair in buffers["grads"] for g in pair]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = call()
    for pair in buffers["grads"]:
        for g in pair:
            g.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    coco.coco_device_status()
    for k, v in keep.items():
        assert torch.equal(held[k], v), k
    assert all(torch.equal(a, b) for a, b in zip(grads, (g for pair in buffers["grads"] for g in pair)))


def test_data_parallel_replicas_averaged_and_clipped():
    """Two replicas' experts' gradients (unclipped), summed, halved and clipped in one call, against float64 of what they
    held: two roundings to bf16."""
    sets = [on_device(inputs(40, 128, 64, 4, 2, 2, 895 + i)) for i in range(2)]
    sets[1] = sets[0][:2] + sets[0][2:6] + sets[1][6:]  # the same layer, another routing and loss
    replicas = []
    for args in sets:
        buffers, call = run(args, float("inf"))
        call()
        replicas.append([g for pair in buffers["grads"] for g in pair])
    mean = [(f64(a) + f64(b)) / 2 for a, b in zip(*replicas)]
    kept = workloads.gradient_buffers(replicas)
    coco.coco_scattered_allreduce_clip(kept["plan"], 0.5, 1.0, None, kept["norm"], kept["space"])
    coco.coco_device_status()
    want, norm = oracle.clip(mean, 1.0)
    assert norm > 1.0 and abs(float(kept["norm"]) - norm) <= 2.0 ** -8 * norm
    for row in replicas:
        for g, m in zip(row, want):
            assert np.all(np.abs(f64(g) - m) <= np.abs(m) * 3 * 2.0 ** -8 + 1e-30)


def test_the_librarys_routing_is_pytorchs():
    expert_of = torch.randint(0, 9, (321, 3), device=DEV)
    token_of, row_of, offsets = workloads.route(expert_of, 9)
    got, lines = workloads.sort_by_expert(expert_of, 9, 4)
    assert torch.equal(got.long(), row_of) and all(torch.equal(line, offsets) for line in lines)
    x = torch.randn(321, 64, device=DEV).bfloat16()
    rows, _ = workloads.dispatch(x, got, 4)
    assert torch.equal(rows, x[token_of])
    gates = torch.rand(321, 3, device=DEV)
    for g in (gates, None):
        want = (rows[row_of].float() * (gates[..., None] if g is not None else 1.0)).sum(1).bfloat16()
        assert torch.equal(workloads.combine([rows], got, g, x)[0], want)  # as the layers did it before


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(37, 2), (37, 1), (1, 2), (2,), ()])
def test_combining_for_any_residual_stream_with_gates_that_broadcast(dtype, shape):
    """The experts' products are bf16 whatever the stream's type is, and one gate may stand for many choices."""
    x, y = torch.randn(37, 64, device=DEV).to(dtype), torch.randn(74, 64, device=DEV).bfloat16()
    row_of = torch.randperm(74, device=DEV, dtype=torch.int32).view(37, 2)
    for gates in (torch.rand(shape, device=DEV), torch.rand(shape, device=DEV).bfloat16()):
        want = (y[row_of.long()].float() * gates[..., None]).sum(1).to(dtype)
        got = workloads.combine([y], row_of, gates, x)[0]
        assert got.dtype == dtype and torch.equal(got, want)


@pytest.mark.parametrize("choices", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("ranks", [1, 2, 3, 4, 8, 5])
def test_combined_products_and_sums_are_rounded_one_by_one(choices, ranks):
    """In fp32, where nothing hides it: the ranks in order, the weight, then the choices in order."""
    tokens, cols = 301, 256
    rows = [torch.randn(tokens * choices, cols, device=DEV) for _ in range(ranks)]
    row_of = torch.randperm(tokens * choices, device=DEV, dtype=torch.int32).view(tokens, choices)
    gates, at = torch.rand(tokens, choices, device=DEV), row_of.long()

    def summed(values):
        total = torch.zeros(tokens, cols, device=DEV)
        for k in range(choices):
            total = total + values[at[:, k]] * gates[:, k, None]
        return total

    for r, got in zip(rows, workloads.combine(rows, row_of, gates, rows[0][:tokens])):
        assert torch.equal(got, summed(r))
    over = rows[0]
    for r in rows[1:]:
        over = over + r
    out, res = torch.empty(tokens, cols, device=DEV), torch.randn(tokens, cols, device=DEV)
    coco.coco_expert_combine(coco.local(rows), row_of, gates, coco.replicated([res] * ranks), coco.replicated([out] * ranks))
    coco.coco_device_status()
    assert torch.equal(out, summed(over) + res)


@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_serving_layer_with_other_residual_streams(dtype):
    """As test_gpu_llm_layer's, whose stream is bf16; its tolerances (the stream's own rounding is no coarser here)."""
    parts, res, w, _, up, down, expert_of, gates, _ = inputs(37, 400, 144, 5, 3, 2, 901)
    parts, res, w = [p.to(dtype) for p in parts], res.to(dtype), w.to(dtype)
    expert_of = expert_of.clamp(min=0)
    up8, down8 = workloads.quantize_weights(dev(up)), workloads.quantize_weights(dev(down))
    h2, q, s = workloads.moe_layer_fp8(dev(parts), res.to(DEV), w.to(DEV), 1e-5, expert_of.to(DEV), gates.to(DEV), *up8,
                                       *down8, torch.ones(400, dtype=dtype, device=DEV))
    coco.coco_device_status()
    h, _, y = oracle.moe_layer([f64(p) for p in parts], f64(res), f64(w), 1e-5, expert_of.numpy(), f64(gates),
                               [f64(u) for u in up], [f64(d) for d in down])
    assert h2.dtype == dtype and far(f64(h2) - h, y) <= 0.08
    x2 = oracle.allreduce_rmsnorm([h + y], None, np.ones(400), 1e-5)[1]
    assert far(oracle.dequantize(f64(q), f64(s), 1), x2) <= 0.09
