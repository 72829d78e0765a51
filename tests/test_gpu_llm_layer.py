"""The 8-bit and expert-grouped operators together, as a mixture-of-experts layer uses them: serving in 8 bits and a
training step in 16 bits, against the float64 oracle of the same layer.

Tolerances are norms of the whole output's difference over the output's. Serving: four roundings to e4m3 lie on
the way to y (the normalised rows, the weights of both products, the activation), each off by at most 2^-4 of a
value and by 2^-4 / sqrt(3) in the root mean square; being independent they add as squares: sqrt(4) 2^-4 / sqrt(3)
= 7.3 %, a few bf16 roundings aside. The residual stream carries h unrounded, so the same bound holds for h'.
Training: every step rounds to bf16 (2^-8 at most, about ten of them on the longest path, partly relu'd): 3 %.
"""

import numpy as np
import pytest
import torch

import oracle
from collective_fusedallreduce_gb300 import coco, synth, workloads
from test_gpu_llm_norm import dev, f64

pytestmark = pytest.mark.gpu


def far(got, want):
    return np.linalg.norm(got - want) / np.linalg.norm(want)


def inputs(tokens, hid, f, experts, n, choices, seed):
    parts = synth.per_rank(seed, 0, n, (tokens, hid), torch.bfloat16, std=n ** -0.5)
    res = synth.tensor(seed + 1, (tokens, hid), torch.bfloat16)
    w = synth.tensor(seed + 2, (hid,), torch.bfloat16, std=0.1) + 1
    up = synth.per_rank(seed, 3, n, (experts, hid, f), torch.bfloat16, std=hid ** -0.5)
    down = synth.per_rank(seed, 4, n, (experts, f, hid), torch.bfloat16, std=(f * n) ** -0.5)
    g = torch.Generator().manual_seed(seed)
    expert_of = torch.rand(tokens, experts, generator=g).topk(choices, 1).indices
    gates = torch.rand(tokens, choices, generator=g)
    return parts, res, w, up, down, expert_of, gates


@pytest.mark.parametrize("tokens,hid,f,experts,n", [(1, 256, 128, 8, 2), (37, 400, 144, 5, 3), (300, 512, 256, 16, 2)])
def test_serving_layer_in_8_bits(tokens, hid, f, experts, n):
    parts, res, w, up, down, expert_of, gates = inputs(tokens, hid, f, experts, n, 2, 661)
    uq, us = workloads.quantize_weights(dev(up))
    dq, ds = workloads.quantize_weights(dev(down))
    next_w = torch.ones(hid, dtype=torch.bfloat16, device="cuda")
    h2, q, s = workloads.moe_layer_fp8(dev(parts), res.cuda(), w.cuda(), 1e-5, expert_of.cuda(), gates.cuda(), uq, us,
                                       dq, ds, next_w)
    coco.coco_device_status()
    h, _, y = oracle.moe_layer([f64(p) for p in parts], f64(res), f64(w), 1e-5, expert_of.numpy(), f64(gates),
                               [f64(u) for u in up], [f64(d) for d in down])
    assert far(f64(h2) - h, y) <= 0.08
    assert far(f64(h2), h + y) <= 0.08
    x2 = oracle.allreduce_rmsnorm([h + y], None, np.ones(hid), 1e-5)[1]
    assert far(oracle.dequantize(f64(q), f64(s), 1), x2) <= 0.09


@pytest.mark.parametrize("tokens,hid,f,experts,n", [(1, 128, 64, 4, 2), (50, 272, 144, 6, 2), (400, 256, 128, 8, 3)])
def test_training_step_in_16_bits(tokens, hid, f, experts, n):
    parts, res, w, up, down, expert_of, _ = inputs(tokens, hid, f, experts, n, 2, 671)
    dout = synth.tensor(679, (tokens, hid), torch.bfloat16)
    got = workloads.moe_layer_train(dev(parts), res.cuda(), w.cuda(), 1e-5, expert_of.cuda(), dev(up), dev(down),
                                    dout.cuda())
    coco.coco_device_status()
    a = ([f64(p) for p in parts], f64(res), f64(w), 1e-5, expert_of.numpy())
    u, d = [f64(x) for x in up], [f64(x) for x in down]
    h, _, y = oracle.moe_layer(*a, np.ones(expert_of.shape), u, d)
    # the activation's kink: which units are on is the forward's decision, made on its rounded values
    active = [f64(m)[got["row_of_choice"].cpu().numpy()] > 0 for m in got["mid"]]
    dx, dw, dup, ddown = oracle.moe_layer_backward(*a, u, d, f64(dout), active)
    assert far(f64(got["out"]), h + y) <= 0.03
    assert far(f64(got["dx"]), dx) <= 0.03 and far(f64(got["dweight"]), dw) <= 0.03
    for r in range(n):
        assert far(f64(got["dup"][r]), dup[r]) <= 0.03 and far(f64(got["ddown"][r]), ddown[r]) <= 0.03


def test_routing_sorts_rows_and_keeps_the_host_out_of_it():
    expert_of = torch.tensor([[3, 0], [0, 3], [2, 0]], device="cuda")
    token_of, row_of, offsets = workloads.route(expert_of, 5)
    assert offsets.tolist() == [0, 3, 3, 4, 6, 6] and offsets.dtype == torch.int32
    assert token_of.tolist() == [0, 1, 2, 2, 0, 1]
    for t in range(3):
        for j in range(2):
            assert token_of[row_of[t, j]] == t
            row, e = int(row_of[t, j]), int(expert_of[t, j])
            assert int(offsets[e]) <= row < int(offsets[e + 1])
