"""Host-side tests of the experts', layer norm's and clipping's entry points: invalid arguments are refused with the right
status before any CUDA call (all device pointers are fake and never dereferenced), and the binding refuses what the
library cannot see. No GPU is needed."""

import pytest
import torch

from test_abi_host import FAKE, mk
from test_llm_host import (ALIAS, ALIGN, DTYPE, LAYOUT, NULL, OK, SHAPE, UNSUPPORTED, VALUE, area, coco,  # noqa: F401
                           ptrs, ref)


def test_sort_refusals(coco):  # noqa: F811
    good = dict(e=area(0), ib=8, t=10, k=2, x=5, g=1, n=2, row=area(1), of=area(2), off=area(3))

    def call(**kw):
        a = {**good, **kw}
        return coco.raw_call("coco_expert_sort", a["e"], a["ib"], a["t"], a["k"], a["x"], a["g"], a["n"], a["row"],
                             a["of"], a["off"], None)

    for k in ("e", "row", "off"):
        assert call(**{k: None}) == NULL, k
    for ib in (0, 2, 16):
        assert call(ib=ib) == DTYPE
    for kw in (dict(t=-1), dict(k=-1), dict(x=-1), dict(g=0), dict(n=0), dict(g=9, n=8)):
        assert call(**kw) == SHAPE, kw
    assert call(t=1 << 31) == UNSUPPORTED and call(t=1 << 30, k=2) == UNSUPPORTED and call(x=65537) == UNSUPPORTED
    assert call(t=(1 << 31) - 1, k=(1 << 31) - 1) == UNSUPPORTED
    assert call(e=area(0) + 4) == ALIGN and call(e=area(0) + 2, ib=4) == ALIGN
    for k in ("row", "of", "off"):
        assert call(**{k: area(7) + 2}) == ALIGN, k
        assert call(**{k: area(0)}) == ALIAS, k
    assert call(row=area(2) + 76) == ALIAS and call(off=area(1) + 76) == ALIAS and call(of=area(3) + 44) == ALIAS


def test_dispatch_refusals(coco):  # noqa: F811
    B, F8, R, L, S = coco.BF16, coco.F8E4M3, coco.REPLICATED, coco.LOCAL, coco.SLICED
    t, k, h, n = 6, 2, 256, 2

    def call(x=mk(coco, B, R, (t, h), n), sx=None, row=area(1), rows=mk(coco, B, R, (t * k, h), n, base=area(2)), sr=None):
        return coco.raw_call("coco_expert_dispatch", ref(x), sx, row, ref(rows), sr, None)

    f8 = dict(x=mk(coco, F8, R, (t, h), n), sx=ptrs(coco, n, area(3)), sr=ptrs(coco, n, area(4)),
              rows=mk(coco, F8, R, (t * k, h), n, base=area(2)))
    for kw in (dict(x=None), dict(row=None), dict(rows=None), {**f8, "sx": None}, {**f8, "sr": None},
               {**f8, "sr": ptrs(coco, n, 0, area(4))}):
        assert call(**kw) == NULL
    assert call(sx=ptrs(coco, n, area(3))) == DTYPE and call(sr=ptrs(coco, n, area(4))) == DTYPE
    assert call(x=mk(coco, B, L, (t, h), n)) == LAYOUT and call(rows=mk(coco, B, L, (t * k, h), n, base=area(2))) == LAYOUT
    assert call(x=mk(coco, B, S, (t, h), n, slice_dim=1)) == LAYOUT
    assert call(rows=f8["rows"]) == DTYPE
    for rows in ((t * k + 1, h), (t * k, h + 8), (t, k, h)):
        assert call(rows=mk(coco, B, R, rows, n, base=area(2))) == SHAPE
    assert call(rows=mk(coco, B, R, (t * k, h), 3, base=area(2))) == SHAPE
    assert call(x=mk(coco, B, R, (0, h), n)) == SHAPE
    big = 1 << 31
    assert call(x=mk(coco, B, R, (big, 8), n), rows=mk(coco, B, R, (big, 8), n, base=area(2))) == UNSUPPORTED
    assert call(row=area(1) + 2) == ALIGN and call(**{**f8, "sx": ptrs(coco, n, area(3) + 1)}) == ALIGN
    assert call(rows=mk(coco, B, R, (t * k, h), n, base=FAKE)) == ALIAS and call(row=area(2)) == ALIAS
    for a in (0, 1, 2, 3):
        assert call(**{**f8, "sr": ptrs(coco, n, area(a))}) == ALIAS, a
    assert call(x=mk(coco, B, R, (t, 0), n), rows=mk(coco, B, R, (t * k, 0), n, base=area(2))) == OK
    # a buffer of two groups
    two = lambda base, rows, **kw: mk(coco, B, R, (rows, h), 1, 2, base=base, **kw)  # noqa: E731
    assert call(x=two(FAKE, t), rows=two(area(2), t * k, stride=0)) == ALIAS


def test_combine_refusals(coco):  # noqa: F811
    B, F8, R, L, S = coco.BF16, coco.F8E4M3, coco.REPLICATED, coco.LOCAL, coco.SLICED
    t, k, h, n = 6, 2, 256, 2
    rows = mk(coco, B, L, (t * k, h), n)
    res, own = mk(coco, B, R, (t, h), n, base=area(3)), mk(coco, B, L, (t, h), n, base=area(4))
    one = mk(coco, B, R, (t, h), n, base=area(4))

    def call(rows=rows, row=area(1), gates=area(2), res=res, out=one):
        return coco.raw_call("coco_expert_combine", ref(rows), row, gates, ref(res), ref(out), None)

    for kw in (dict(rows=None), dict(row=None), dict(out=None)):
        assert call(**kw) == NULL
    assert call(out=own) == LAYOUT  # a rank's own sum has no residual
    assert call(rows=mk(coco, B, R, (t * k, h), n)) == LAYOUT and call(res=mk(coco, B, L, (t, h), n, base=area(3))) == LAYOUT
    assert call(out=mk(coco, B, S, (t * n, h), n, slice_dim=0, base=area(4))) == LAYOUT
    assert call(rows=mk(coco, coco.F16, L, (t * k, h), n)) == DTYPE and call(rows=mk(coco, F8, L, (t * k, h), n)) == DTYPE
    assert call(res=mk(coco, coco.F32, R, (t, h), n, base=area(3))) == DTYPE
    for bad in ((t * k + 1, h), (t * k, h - 8)):
        assert call(rows=mk(coco, B, L, bad, n)) == SHAPE
    assert call(res=mk(coco, B, R, (t + 1, h), n, base=area(3))) == SHAPE
    assert call(out=mk(coco, B, R, (t, h), 3, base=area(4))) == SHAPE
    assert call(row=area(1) + 1) == ALIGN and call(gates=area(2) + 2) == ALIGN
    assert call(out=mk(coco, B, R, (t, h), n, base=FAKE)) == ALIAS and call(row=area(4)) == ALIAS
    assert call(gates=area(4) + 512) == ALIAS
    assert call(out=mk(coco, B, R, (t, h), n, base=area(3) + 16)) == ALIAS
    assert call(res=None, out=mk(coco, B, L, (t, h), n, base=area(4), stride=0)) == ALIAS  # two ranks' sums in one place
    assert call(out=mk(coco, B, R, (0, h), n, base=area(4)), res=None, rows=mk(coco, B, L, (0, h), n)) == OK
    groups = dict(rows=mk(coco, B, L, (t * k, h), 1, 2), res=mk(coco, B, R, (t, h), 1, 2, base=area(3)))
    swapped = mk(coco, B, R, (t, h), 1, 2, ptrs=[area(3) + (1 << 32), area(4)])  # the other group's residual
    assert call(**groups, out=swapped) == ALIAS


def test_combine_backward_refusals(coco):  # noqa: F811
    B, F8, R, L = coco.BF16, coco.F8E4M3, coco.REPLICATED, coco.LOCAL
    t, k, h, n = 6, 2, 256, 2
    good = dict(d=mk(coco, B, R, (t, h), n), rows=mk(coco, B, L, (t * k, h), n, base=area(1)), row=area(2), gates=area(3),
                dr=mk(coco, B, R, (t * k, h), n, base=area(4)), dg=area(5))

    def call(**kw):
        a = {**good, **kw}
        return coco.raw_call("coco_expert_combine_backward", ref(a["d"]), ref(a["rows"]), a["row"], a["gates"],
                             ref(a["dr"]), a["dg"], None)

    for x in ("d", "rows", "row", "dr", "dg"):  # (rows and dgates: both or neither)
        assert call(**{x: None}) == NULL, x
    assert call(d=mk(coco, B, L, (t, h), n)) == LAYOUT and call(dr=mk(coco, B, L, (t * k, h), n, base=area(4))) == LAYOUT
    assert call(rows=mk(coco, B, R, (t * k, h), n, base=area(1))) == LAYOUT
    assert call(d=mk(coco, coco.F16, R, (t, h), n)) == DTYPE and call(d=mk(coco, F8, R, (t, h), n)) == DTYPE
    assert call(rows=mk(coco, coco.F32, L, (t * k, h), n, base=area(1))) == DTYPE
    assert call(rows=mk(coco, B, L, (t, h), n, base=area(1))) == SHAPE
    assert call(dr=mk(coco, B, R, (t * k + 1, h), n, base=area(4))) == SHAPE
    wide = dict(d=mk(coco, B, R, (1, 32776), n), rows=mk(coco, B, L, (2, 32776), n, base=area(1)),
                dr=mk(coco, B, R, (2, 32776), n, base=area(4)))
    assert call(**wide) == UNSUPPORTED
    for x in ("row", "gates", "dg"):
        assert call(**{x: area(9) + 2}) == ALIGN, x
    for a in (0, 1):
        assert call(dr=mk(coco, B, R, (t * k, h), n, base=area(a))) == ALIAS
    for a in (0, 1, 2, 3, 4):
        assert call(dg=area(a)) == ALIAS, a
    assert call(row=area(4)) == ALIAS and call(gates=area(4)) == ALIAS
    none = dict(d=mk(coco, B, R, (0, h), n), rows=mk(coco, B, L, (0, h), n, base=area(1)),
                dr=mk(coco, B, R, (0, h), n, base=area(4)))
    assert call(**none) == OK


class Norm:
    """Valid arguments of coco_allreduce_layernorm; tests replace one at a time."""

    def __init__(self, coco, n=2, shape=(4, 256), dtype=None, out=None):  # noqa: F811
        self.coco = coco
        T = coco.BF16 if dtype is None else dtype
        out = coco.F8E4M3 if out is None else out
        self.partials = mk(coco, T, coco.LOCAL, shape, n, base=area(0))
        self.residual = mk(coco, T, coco.REPLICATED, shape, n, base=area(1))
        self.weight, self.bias, self.eps = area(2), area(7), 1e-5
        self.hidden = mk(coco, T, coco.REPLICATED, shape, n, base=area(3))
        self.normed = mk(coco, out, coco.REPLICATED, shape, n, base=area(4))
        self.scales = ptrs(coco, n, area(5)) if out == coco.F8E4M3 else None
        self.mean, self.rstd = area(8), area(6)

    def __call__(self, **kw):
        a = {**self.__dict__, **kw}
        return self.coco.raw_call("coco_allreduce_layernorm", ref(a["partials"]), ref(a["residual"]), a["weight"],
                                  a["bias"], a["eps"], ref(a["hidden"]), ref(a["normed"]), a["scales"], a["mean"],
                                  a["rstd"], None)


def test_norm_refusals(coco):  # noqa: F811
    B, H, R, L = coco.BF16, coco.F16, coco.REPLICATED, coco.LOCAL
    call = Norm(coco)
    s = (4, 256)
    for kw in (dict(partials=None), dict(normed=None), dict(weight=None), dict(scales=None)):
        assert call(**kw) == NULL
    for k, v in [("partials", mk(coco, B, R, s, 2)), ("normed", mk(coco, coco.F8E4M3, L, s, 2, base=area(4))),
                 ("residual", mk(coco, B, L, s, 2, base=area(1))), ("hidden", mk(coco, B, L, s, 2, base=area(3)))]:
        assert call(**{k: v}) == LAYOUT, k
    for k, v in [("partials", mk(coco, coco.F8E4M3, L, s, 2)), ("normed", mk(coco, H, R, s, 2, base=area(4))),
                 ("residual", mk(coco, H, R, s, 2, base=area(1))), ("hidden", mk(coco, H, R, s, 2, base=area(3))),
                 ("normed", mk(coco, B, R, s, 2, base=area(4)))]:
        assert call(**{k: v}) == DTYPE, k
    for k, i in [("residual", 1), ("hidden", 3)]:
        assert call(**{k: mk(coco, B, R, (8, 256), 2, base=area(i))}) == SHAPE
        assert call(**{k: mk(coco, B, R, s, 4, base=area(i))}) == SHAPE
    for eps in (-1.0, float("nan"), float("inf")):
        assert call(eps=eps) == VALUE
    for k, off in [("weight", 8), ("bias", 8), ("rstd", 2), ("mean", 2)]:
        assert call(**{k: area(9) + off}) == ALIGN, k
    assert Norm(coco, shape=(1, 32784))() == UNSUPPORTED
    assert call(hidden=mk(coco, B, R, s, 2, base=area(0) + 16)) == ALIAS
    assert call(normed=mk(coco, coco.F8E4M3, R, s, 2, base=area(0))) == ALIAS
    same = Norm(coco, out=B)
    assert same(normed=mk(coco, B, R, s, 2, base=area(0) + 512)) == ALIAS and same(normed=same.hidden) == ALIAS
    for k in ("weight", "bias", "mean", "rstd"):
        for a in (3, 4, 5):
            assert call(**{k: area(a)}) == ALIAS, (k, a)
    assert call(mean=area(6)) == ALIAS and call(mean=area(0)) == ALIAS and call(rstd=area(7)) == ALIAS
    assert call(scales=ptrs(coco, 2, area(1))) == ALIAS
    assert Norm(coco, shape=(0, 256))() == OK


def test_norm_backward_refusals(coco):  # noqa: F811
    B, R, L = coco.BF16, coco.REPLICATED, coco.LOCAL
    s, n = (6, 256), 2
    need = coco.coco_allreduce_layernorm_backward_bytes(6, 256)
    assert need == 2 * 6 * 256 * 4 and coco.coco_allreduce_layernorm_backward_bytes(4, 1 << 20) == 0
    good = dict(dn=mk(coco, B, L, s, n, base=area(0)), dh=mk(coco, B, R, s, n, base=area(1)),
                h=mk(coco, B, R, s, n, base=area(2)), w=area(3), m=area(8), rstd=area(4),
                dx=mk(coco, B, R, s, n, base=area(5)), dw=area(6), db=area(9), ws=area(7), nb=need)

    def call(**kw):
        a = {**good, **kw}
        return coco.raw_call("coco_allreduce_layernorm_backward", ref(a["dn"]), ref(a["dh"]), ref(a["h"]), a["w"], a["m"],
                             a["rstd"], ref(a["dx"]), a["dw"], a["db"], a["ws"], a["nb"], None)

    for k in ("dn", "h", "w", "m", "rstd", "dx", "dw", "ws"):
        assert call(**{k: None}) == NULL, k
    assert call(nb=need - 1) == SHAPE
    assert call(dn=mk(coco, B, R, s, n)) == LAYOUT and call(dh=mk(coco, B, L, s, n, base=area(1))) == LAYOUT
    assert call(h=mk(coco, coco.F32, R, s, n, base=area(2))) == DTYPE
    assert call(dx=mk(coco, B, R, (5, 256), n, base=area(5))) == SHAPE and call(dh=mk(coco, B, R, s, 3, base=area(1))) == SHAPE
    for k, off in (("w", 4), ("ws", 8), ("dw", 1), ("db", 2), ("m", 2)):
        assert call(**{k: area(10) + off}) == ALIGN, k
    assert call(dx=mk(coco, B, R, s, n, base=area(0) + 16)) == ALIAS
    for k in ("dw", "db", "ws"):
        for a in (0, 1, 2, 3, 4, 5, 8):
            assert call(**{k: area(a)}) == ALIAS, (k, a)
    assert call(ws=area(6)) == ALIAS and call(db=area(6)) == ALIAS and call(ws=area(9)) == ALIAS
    wide = (1, 32784)
    assert call(dn=mk(coco, B, L, wide, n), h=mk(coco, B, R, wide, n, base=area(2)), dh=None,
                dx=mk(coco, B, R, wide, n, base=area(5))) == UNSUPPORTED


def plan(coco, table, nb=10, n=2, dtype=None):  # noqa: F811
    p = coco.CocoScatteredPlan()
    p.table, p.nbuckets, p.nranks, p.dtype = table, nb, n, coco.BF16 if dtype is None else dtype
    return p


def test_clip_refusals(coco):  # noqa: F811
    need = coco.coco_scattered_clip_bytes()
    inf, nan = float("inf"), float("nan")
    good = dict(p=plan(coco, area(0)), layout=coco.LOCAL, alpha=1.0, top=1.0, out=None, norm=area(1), ws=area(2), nb=need)

    def clip(**kw):
        a = {**good, **kw}
        return coco.raw_call("coco_scattered_clip", ref(a["p"]), a["layout"], a["top"], ref(a["out"]), a["norm"], a["ws"],
                             a["nb"], None)

    def reduce_clip(**kw):
        a = {**good, **kw}
        return coco.raw_call("coco_scattered_allreduce_clip", ref(a["p"]), a["alpha"], a["top"], ref(a["out"]), a["norm"],
                             a["ws"], a["nb"], None)

    for layout in (coco.SLICED, 3, -1):
        assert clip(layout=layout) == LAYOUT
    assert reduce_clip(alpha=nan) == VALUE
    for call in (clip, reduce_clip):
        for k in ("p", "norm", "ws"):
            assert call(**{k: None}) == NULL, k
        assert call(p=plan(coco, None)) == NULL and call(out=plan(coco, None)) == NULL
        for top in (-1.0, nan, -inf):
            assert call(top=top) == VALUE
        assert call(nb=need - 1) == SHAPE
        for bad in (plan(coco, area(0), nb=-1), plan(coco, area(0), n=0), plan(coco, area(0), n=65),
                    plan(coco, area(0), nb=1 << 41)):
            assert call(p=bad) == SHAPE and call(out=bad) == SHAPE
        assert call(p=plan(coco, area(0), dtype=coco.F8E4M3)) == DTYPE and call(out=plan(coco, area(3), dtype=7)) == DTYPE
        assert call(out=plan(coco, area(3), nb=9)) == SHAPE
        assert call(out=plan(coco, area(0), dtype=coco.F32)) == SHAPE  # one table, another type
        assert call(p=plan(coco, area(0) + 8)) == ALIGN and call(norm=area(1) + 2) == ALIGN and call(ws=area(2) + 8) == ALIGN
        assert call(norm=area(2) + 64) == ALIAS and call(norm=area(0) + 64) == ALIAS and call(ws=area(0)) == ALIAS
        assert call(out=plan(coco, area(3)), ws=area(3) + 64) == ALIAS
    assert clip(out=plan(coco, area(3), n=1)) == SHAPE  # parts: as many ranks


def test_binding_refuses_what_the_library_cannot_see(coco):  # noqa: F811
    def status(f):
        with pytest.raises(coco.CocoError) as e:
            f()
        return e.value.status

    i32, f32, bf = torch.int32, torch.float32, torch.bfloat16
    z = lambda *s, dtype=bf: torch.zeros(*s, dtype=dtype)  # noqa: E731
    rep, loc = lambda t: coco.replicated([t]), lambda t: coco.local([t])  # noqa: E731
    space = z(coco.coco_allreduce_layernorm_backward_bytes(4, 256), dtype=torch.uint8)
    clip_space = z(coco.coco_scattered_clip_bytes(), dtype=torch.uint8)
    calls = {
        "sort": (dict(e=z(4, 2, dtype=torch.int64), row=z(4, 2, dtype=i32), of=z(8, dtype=i32), off=z(1, 4, dtype=i32)),
                 lambda e, row, of, off: coco.coco_expert_sort(e, 3, row, of, off, 0)),
        "dispatch": (dict(x=z(4, 256), row=z(4, 2, dtype=i32), rows=z(8, 256)),
                     lambda x, row, rows: coco.coco_expert_dispatch(rep(x), None, row, rep(rows), None, 0)),
        "combine": (dict(rows=z(8, 256), row=z(4, 2, dtype=i32), gates=z(4, 2, dtype=f32), res=z(4, 256), out=z(4, 256)),
                    lambda rows, row, gates, res, out: coco.coco_expert_combine(loc(rows), row, gates, rep(res), rep(out), 0)),
        "back": (dict(d=z(4, 256), rows=z(8, 256), row=z(4, 2, dtype=i32), gates=z(4, 2, dtype=f32), dr=z(8, 256),
                      dg=z(4, 2, dtype=f32)),
                 lambda d, rows, row, gates, dr, dg: coco.coco_expert_combine_backward(rep(d), loc(rows), row, gates,
                                                                                       rep(dr), dg, 0)),
        "norm": (dict(x=z(4, 256), w=z(256), b=z(256), out=z(4, 256), m=z(4, dtype=f32), r=z(4, dtype=f32)),
                 lambda x, w, b, out, m, r: coco.coco_allreduce_layernorm(loc(x), None, w, b, 1e-5, None, rep(out), None, m,
                                                                          r, 0)),
        "grad": (dict(dn=z(4, 256), h=z(4, 256), w=z(256), m=z(4, dtype=f32), r=z(4, dtype=f32), dx=z(4, 256),
                      dw=z(256, dtype=f32), db=z(256, dtype=f32), ws=space),
                 lambda dn, h, w, m, r, dx, dw, db, ws: coco.coco_allreduce_layernorm_backward(
                     loc(dn), None, rep(h), w, m, r, rep(dx), dw, db, ws, 0)),
        "clip": (dict(norm=z(1, dtype=f32), ws=clip_space),
                 lambda norm, ws: coco.coco_scattered_clip(plan(coco, area(0)), coco.LOCAL, 1.0, None, norm, ws, 0)),
    }
    for name, (args, call) in calls.items():
        assert status(lambda: call(**args)) == UNSUPPORTED, name  # host memory
        for k, t in args.items():
            strided = torch.zeros(*t.shape[:-1], 2 * t.shape[-1], dtype=t.dtype)[..., ::2]
            if t.shape[-1] > 1:
                assert status(lambda: call(**{**args, k: strided})) == SHAPE, (name, k)
            if t.dtype in (i32, f32):
                assert status(lambda: call(**{**args, k: t.double()})) == DTYPE, (name, k)
                assert status(lambda: call(**{**args, k: torch.cat([t, t], -1)})) == SHAPE, (name, k)
    sort = calls["sort"]
    assert status(lambda: sort[1](**{**sort[0], "e": z(4, 2, dtype=f32)})) == DTYPE
    assert status(lambda: sort[1](**{**sort[0], "e": z(4, 3, dtype=torch.int64)})) == SHAPE
