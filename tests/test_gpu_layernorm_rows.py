"""The layer norm and its gradient on more rows than the device holds at a time, where blocks walk rows: the next row is loaded
(or copied to shared memory) while one is stored, pairs of chunks share a thread, and the last rows are some blocks' only. Against
the float64 oracle with test_gpu_layernorm's tolerances; in their inputs' places, the bits of a call with outputs of its own."""

import pytest
import torch

from collective_fusedallreduce_gb300 import coco, synth
from test_gpu_layernorm import backward_case, test_norm_matches_the_oracle as norm_matches
from test_gpu_llm_norm import DEV, dev

pytestmark = pytest.mark.gpu
HALVES = [torch.bfloat16, torch.float16]


@pytest.mark.parametrize("dtype", HALVES)
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,rows,cols", [(1, 5003, 272), (2, 2049, 272), (2, 2500, 1040), (1, 2048, 2048), (2, 4001, 512),
                                         (2, 1500, 4096), (3, 1001, 4096), (3, 4001, 272), (1, 701, 8192)])
def test_rows_walked_by_blocks_match_the_oracle(dtype, fp8, n, rows, cols):
    norm_matches(dtype, n, rows, cols, fp8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n,rows,cols", [(1, 1501, 2048), (1, 5003, 272), (1, 701, 4096)])
def test_fp32_rows_walked_by_blocks_match_the_oracle(fp8, n, rows, cols):
    norm_matches(torch.float32, n, rows, cols, fp8)


def test_rows_that_no_pair_of_chunks_fills():
    """264 columns: 33 chunks, of which one warp's lanes hold two and the rest one."""
    norm_matches(torch.bfloat16, 2, 2049, 264, False)
    norm_matches(torch.float16, 1, 2048, 264, False)


@pytest.mark.parametrize("dtype,n,rows,cols", [
    (torch.bfloat16, 1, 5003, 272), (torch.bfloat16, 2, 2500, 1040), (torch.float16, 2, 1500, 4096), (torch.bfloat16, 3, 1001, 4096),
    (torch.float32, 1, 1501, 2048), (torch.float32, 2, 1501, 2048), (torch.bfloat16, 1, 701, 8192), (torch.float16, 8, 1001, 4096),
    (torch.bfloat16, 2, 500, 12304), (torch.float16, 3, 500, 16384), (torch.float32, 2, 400, 20000), (torch.bfloat16, 5, 900, 4096)])
def test_forward_in_its_inputs_places(dtype, n, rows, cols):
    """The hidden rows where the last partial is, the normed ones where the residual (or the first partial) is."""
    parts = dev(synth.per_rank(841, 0, n, (rows, cols), dtype, std=n ** -0.5))
    res = synth.tensor(842, (rows, cols), dtype).to(DEV)
    w, b = dev([synth.tensor(843, (cols,), dtype), synth.tensor(844, (cols,), dtype)])
    rep = lambda t: coco.replicated([t] * n)  # noqa: E731

    def call(p, r, hidden, normed):
        mean, rstd = torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
        coco.coco_allreduce_layernorm(coco.local(p), rep(r), w, b, 1e-5, rep(hidden), rep(normed), None, mean, rstd)
        torch.cuda.synchronize()
        return hidden, normed, mean, rstd

    want = call(parts, res, torch.empty_like(res), torch.empty_like(res))
    for swap in (False, True):
        p, r = [t.clone() for t in parts], res.clone()
        if swap and n == 1:
            got = call(p, r, r, p[0])
        else:
            got = call(p, r, p[-1], p[0] if swap else r)
        assert all(torch.equal(x, y) for x, y in zip(got, want)), swap


@pytest.mark.parametrize("dtype,n,rows,cols", [
    (torch.bfloat16, 1, 5003, 272), (torch.bfloat16, 2, 1500, 4096), (torch.float16, 3, 1001, 4096), (torch.float16, 8, 1001, 4096),
    (torch.bfloat16, 5, 1001, 2064), (torch.bfloat16, 1, 701, 8192), (torch.float16, 2, 400, 16384), (torch.bfloat16, 1, 400, 32768),
    (torch.float32, 2, 1501, 2048), (torch.float32, 8, 701, 4096), (torch.float32, 1, 701, 8192), (torch.float32, 1, 400, 20000)])
def test_backward_in_its_inputs_places(dtype, n, rows, cols):
    """dx where each of its inputs is."""
    dn, dh, hid, w, mean, rstd = backward_case(dtype, n, rows, cols)
    dh = dh if dh is not None else synth.tensor(845, (rows, cols), dtype)
    dn, dh, hid, w, mean, rstd = dev(dn), dh.to(DEV), hid.to(DEV), w.to(DEV), mean.to(DEV), rstd.to(DEV)
    ws = torch.empty(coco.coco_allreduce_layernorm_backward_bytes(rows, cols), dtype=torch.uint8, device=DEV)
    rep = lambda t: coco.replicated([t] * n)  # noqa: E731

    def call(d, e, h, dx):
        dw, db = torch.empty(cols, device=DEV), torch.empty(cols, device=DEV)
        coco.coco_allreduce_layernorm_backward(coco.local(d), rep(e), rep(h), w, mean, rstd, rep(dx), dw, db, ws)
        torch.cuda.synchronize()
        return dx, dw, db

    want = call(dn, dh, hid, torch.empty_like(hid))
    for place in range(4):
        d, e, h = [t.clone() for t in dn], dh.clone(), hid.clone()
        got = call(d, e, h, (d[0], d[-1], e, h)[place])
        assert all(torch.equal(x, y) for x, y in zip(got, want)), place
