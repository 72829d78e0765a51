"""Plans of the quantiser and the products that larger models reach: stacks of more matrices than one launch takes,
slices and replicas of operands in both storages."""

import numpy as np
import pytest
import torch

import oracle
from collective_fusedallreduce_gb300 import coco, synth
from test_gpu_llm_norm import DEV, F8, f64
from test_gpu_llm_products import close, eight_bits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("ranks,matrices", [(1, 65), (3, 43), (2, 130)])
def test_stacks_of_more_matrices_than_a_launch_takes(ranks, matrices):
    rows, cols = 130, 144
    g = torch.Generator().manual_seed(721)
    # (sizes that differ by matrix: a scale or a matrix in the wrong place shows)
    xs = [torch.randn(matrices, rows, cols, generator=g) * torch.logspace(-3, 3, matrices)[:, None, None]
          for _ in range(ranks)]
    q = [torch.empty(matrices, rows, cols, dtype=F8, device=DEV) for _ in range(ranks)]
    sc = [torch.empty(matrices, 2, 2, device=DEV) for _ in range(ranks)]
    coco.coco_quantize_fp8(coco.local([x.to(DEV) for x in xs]), 128, coco.local(q), sc)
    coco.coco_device_status()
    for r in range(ranks):
        for m in range(matrices):
            x = f64(xs[r][m])
            s = np.maximum(oracle.block_amax(x, 128), 2.0 ** -100).astype(np.float32) / np.float32(448)
            assert np.array_equal(sc[r][m].cpu().numpy(), s), (r, m)
            quotient = x.astype(np.float32) / oracle.spread(s, x.shape, 128).astype(np.float32)
            assert np.array_equal(f64(q[r][m]), oracle.to_e4m3(quotient.astype(np.float64))), (r, m)


@pytest.mark.parametrize("m", [3, 200])
@pytest.mark.parametrize("layouts", [("replicated", "local"), ("sliced", "sliced"), ("local", "replicated"),
                                     ("replicated", "replicated")])
def test_layouts_of_weights_stored_by_columns(m, layouts):
    k, n, ranks, groups = 256, 144, 2, 2
    total = ranks * groups
    lhs = [eight_bits(x, 1) for x in synth.per_rank(722, 0, total, (m, k), torch.float32)]
    rhs = [eight_bits(x, 128) for x in synth.per_rank(722, 1, total, (n, k), torch.float32)]
    first = lambda xs: [xs[p // ranks * ranks] for p in range(total)]  # noqa: E731
    if layouts[0] == "replicated":
        lhs = first(lhs)
    if layouts[1] == "replicated":
        rhs = first(rhs)
    make = {"local": coco.local, "replicated": coco.replicated, "sliced": lambda t, g: coco.sliced(t, 1, g)}
    out = [torch.full((m, n), float("nan"), device=DEV) for _ in range(total)]
    coco.coco_einsum_fp8("mk,nk->mn", make[layouts[0]]([x[0] for x in lhs], groups), [x[1] for x in lhs],
                         make[layouts[1]]([x[0] for x in rhs], groups), [x[1] for x in rhs], coco.local(out, groups))
    coco.coco_device_status()
    for p in range(total):
        close(out[p], lhs[p][2], rhs[p][2].T, k, torch.float32, f"{layouts} {p}")


@pytest.mark.parametrize("counts", [[3, 0, 5], [200, 31, 70]])
def test_grouped_with_replicated_weights(counts):
    """The same experts on every rank (data-parallel rows), in both storages and in the weight gradient's lhs."""
    k, n, ranks = 144, 272, 2
    rows, off = sum(counts), np.concatenate([[0], np.cumsum(counts)])
    x = [t.to(DEV) for t in synth.per_rank(723, 0, ranks, (rows, k), torch.bfloat16)]
    offsets = torch.from_numpy(np.stack([off] * ranks)).to(DEV, torch.int32)
    for form in ("kn", "nk"):
        w = synth.tensor(724, (3, k, n) if form == "kn" else (3, n, k), torch.bfloat16).to(DEV)
        out = [torch.full((rows, n), float("nan"), device=DEV) for _ in range(ranks)]
        coco.coco_grouped_einsum(f"tk,e{form}->tn", coco.local(x), None, coco.replicated([w] * ranks), None, offsets,
                                 coco.local(out))
        coco.coco_device_status()
        for r in range(ranks):
            for e in range(3):
                we = f64(w[e]) if form == "kn" else f64(w[e]).T
                a, b = off[e], off[e + 1]
                close(out[r][a:b], f64(x[r][a:b]), we, k, torch.float32, f"{form} rank {r} expert {e}")
    dy = [t.to(DEV) for t in synth.per_rank(723, 1, ranks, (rows, n), torch.bfloat16)]
    grad = [torch.full((3, k, n), float("nan"), device=DEV) for _ in range(ranks)]
    coco.coco_grouped_einsum("tk,tn->ekn", coco.replicated([x[0]] * ranks), None, coco.local(dy), None, offsets,
                             coco.local(grad))
    coco.coco_device_status()
    for r in range(ranks):
        for e in range(3):
            a, b = off[e], off[e + 1]
            close(grad[r][e], f64(x[0][a:b]).T, f64(dy[r][a:b]), max(counts) + 128, torch.float32, f"grad {r} {e}")
