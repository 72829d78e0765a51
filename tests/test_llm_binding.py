"""What the binding refuses before the library, which gets addresses only: operands that are not dense (the transposed
storage invites ``w.t()``), ranks' tensors of different sizes, and tensors in host memory. Runs without a GPU."""

import pytest
import torch

from test_llm_host import SHAPE, UNSUPPORTED, coco  # noqa: F401 (the fixture)

F8, BF = torch.float8_e4m3fn, torch.bfloat16


def status(coco, f):  # noqa: F811
    with pytest.raises(coco.CocoError) as e:
        f()
    return e.value.status


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def calls(c):
    """Per entry point: a call and its tensors by name (each a list of one rank's, or a plain tensor)."""
    norm = dict(x=z(4, 256), res=z(4, 256), hid=z(4, 256), out=z(4, 256, dtype=F8), w=z(256), sc=z(4, 2, dtype=torch.float32),
                rstd=z(4, dtype=torch.float32))
    back = dict(dn=z(4, 256), dh=z(4, 256), hid=z(4, 256), dx=z(4, 256), w=z(256), rstd=z(4, dtype=torch.float32),
                dw=z(256, dtype=torch.float32), ws=z(4 * 256 * 4, dtype=torch.uint8))
    quant = dict(x=z(4, 256), q=z(4, 256, dtype=F8), sc=z(4, 2, dtype=torch.float32))
    prod = dict(a=z(4, 256, dtype=F8), b=z(128, 256, dtype=F8), out=z(4, 128), sa=z(4, 2, dtype=torch.float32),
                sb=z(1, 2, dtype=torch.float32))
    group = dict(a=z(4, 256), b=z(2, 128, 256), out=z(4, 128), off=z(3, dtype=torch.int32))
    one, rep = lambda t: c.local([t]), lambda t: c.replicated([t])  # noqa: E731
    return {
        "norm": (norm, {"x", "res", "hid", "out"}, lambda x, res, hid, out, w, sc, rstd: c.coco_allreduce_rmsnorm(
            one(x), rep(res), w, 1e-5, rep(hid), rep(out), [sc], rstd, 0)),
        "back": (back, {"dn", "dh", "hid", "dx"}, lambda dn, dh, hid, dx, w, rstd, dw, ws:
                 c.coco_allreduce_rmsnorm_backward(one(dn), rep(dh), rep(hid), w, rstd, rep(dx), dw, ws, 0)),
        "quant": (quant, {"x", "q"}, lambda x, q, sc: c.coco_quantize_fp8(one(x), 1, one(q), [sc], 0)),
        "prod": (prod, {"a", "b", "out"}, lambda a, b, out, sa, sb: c.coco_einsum_fp8(
            "mk,nk->mn", one(a), [sa], one(b), [sb], one(out), 0)),
        "group": (group, {"a", "b", "out"}, lambda a, b, out, off: c.coco_grouped_einsum(
            "tk,enk->tn", one(a), None, one(b), None, off, one(out), 0)),
    }


def transposed(t):
    """The same shape, the last two dimensions stored the other way round."""
    return t.mT.contiguous().mT


@pytest.mark.parametrize("name", ["norm", "back", "quant", "prod", "group"])
def test_operands_that_are_not_dense(coco, name):  # noqa: F811
    args, dists, call = calls(coco)[name]
    for k in dists:
        assert status(coco, lambda: call(**{**args, k: transposed(args[k])})) == SHAPE, k
        wide = torch.zeros(*args[k].shape[:-1], args[k].shape[-1] + 16, dtype=args[k].dtype)
        assert status(coco, lambda: call(**{**args, k: wide[..., :-16]})) == SHAPE, k


@pytest.mark.parametrize("name", ["norm", "back", "quant", "prod", "group"])
def test_host_memory(coco, name):  # noqa: F811
    args, _, call = calls(coco)[name]
    assert status(coco, lambda: call(**args)) == UNSUPPORTED


def test_ranks_tensors_of_different_sizes(coco):  # noqa: F811
    big, small = z(8, 256), z(4, 256)
    q = [z(8, 256, dtype=F8) for _ in range(2)]
    sc = [z(8, 2, dtype=torch.float32) for _ in range(2)]
    assert status(coco, lambda: coco.coco_quantize_fp8(coco.local([big, small]), 1, coco.local(q), sc, 0)) == SHAPE
    assert status(coco, lambda: coco.coco_quantize_fp8(coco.local([big, big.float()]), 1, coco.local(q), sc, 0)) == SHAPE
    w = z(256)
    assert status(coco, lambda: coco.coco_allreduce_rmsnorm(
        coco.local([big, big]), None, w, 1e-5, coco.replicated([big, small]), coco.replicated(q), sc, None, 0)) == SHAPE
