"""Host-side tests of the 8-bit and expert-grouped entry points: invalid arguments are refused with the right
status before any CUDA call (all device pointers are fake and never dereferenced; no GPU is needed)."""

import ctypes

import pytest

import __graft_entry__
from test_abi_host import FAKE, mk

OK, NULL, SHAPE, DTYPE, LAYOUT, ALIGN, ALIAS, UNSUPPORTED, VALUE = 0, 1, 2, 3, 4, 5, 6, 7, 10


@pytest.fixture(scope="module")
def coco():
    __graft_entry__.build()
    from collective_fusedallreduce_gb300 import coco as c
    return c


def area(i):
    """The base address of a memory area of its own."""
    return FAKE + (i << 40)


def ptrs(coco, n, base, stride=1 << 32):
    return (ctypes.c_void_p * n)(*[base + i * stride for i in range(n)])


def ref(t):
    return None if t is None else ctypes.byref(t)


class Norm:
    """Valid arguments of coco_allreduce_rmsnorm; tests replace one at a time."""

    def __init__(self, coco, n=2, shape=(4, 256), dtype=None, out=None):
        self.coco = coco
        T = coco.BF16 if dtype is None else dtype
        out = coco.F8E4M3 if out is None else out
        self.partials = mk(coco, T, coco.LOCAL, shape, n, base=area(0))
        self.residual = mk(coco, T, coco.REPLICATED, shape, n, base=area(1))
        self.weight, self.eps = area(2), 1e-5
        self.hidden = mk(coco, T, coco.REPLICATED, shape, n, base=area(3))
        self.normed = mk(coco, out, coco.REPLICATED, shape, n, base=area(4))
        self.scales = ptrs(coco, n, area(5)) if out == coco.F8E4M3 else None
        self.rstd = area(6)

    def __call__(self, **kw):
        a = {**self.__dict__, **kw}
        return self.coco.raw_call("coco_allreduce_rmsnorm", ref(a["partials"]), ref(a["residual"]), a["weight"],
                                  a["eps"], ref(a["hidden"]), ref(a["normed"]), a["scales"], a["rstd"], None)


def test_norm_refusals(coco):
    B, H, R, L = coco.BF16, coco.F16, coco.REPLICATED, coco.LOCAL
    call = Norm(coco)
    s, at = (4, 256), lambda i, o=0: area(i) + o  # noqa: E731
    assert call(partials=None) == NULL and call(normed=None) == NULL
    assert call(weight=None) == NULL and call(scales=None) == NULL
    assert call(scales=ptrs(coco, 2, 0, area(5))) == NULL
    for k, v in [("partials", mk(coco, B, R, s, 2)), ("normed", mk(coco, coco.F8E4M3, L, s, 2, base=area(4))),
                 ("residual", mk(coco, B, L, s, 2, base=area(1))), ("hidden", mk(coco, B, L, s, 2, base=area(3)))]:
        assert call(**{k: v}) == LAYOUT, k
    for k, v in [("partials", mk(coco, coco.F8E4M3, L, s, 2)), ("normed", mk(coco, H, R, s, 2, base=area(4))),
                 ("residual", mk(coco, H, R, s, 2, base=area(1))), ("hidden", mk(coco, H, R, s, 2, base=area(3)))]:
        assert call(**{k: v}) == DTYPE, k
    assert call(normed=mk(coco, B, R, s, 2, base=area(4))) == DTYPE  # scales without 8-bit rows
    for k, i in [("residual", 1), ("hidden", 3)]:
        assert call(**{k: mk(coco, B, R, (8, 256), 2, base=area(i))}) == SHAPE
        assert call(**{k: mk(coco, B, R, s, 4, base=area(i))}) == SHAPE
    assert call(normed=mk(coco, coco.F8E4M3, R, (4, 128), 2, base=area(4))) == SHAPE
    for eps in (-1.0, float("nan"), float("inf")):
        assert call(eps=eps) == VALUE
    assert call(weight=at(2, 8)) == ALIGN and call(rstd=at(6, 2)) == ALIGN
    assert call(scales=ptrs(coco, 2, at(5, 2))) == ALIGN
    odd = Norm(coco, shape=(4, 24))  # 8-bit rows of 24 bytes
    assert odd() == ALIGN
    assert Norm(coco, shape=(1, 32784))() == UNSUPPORTED
    # shared memory: between roles never; an input's place only exactly, and only for values of its type
    assert call(hidden=mk(coco, B, R, s, 2, base=at(0, 16))) == ALIAS
    assert call(normed=mk(coco, coco.F8E4M3, R, s, 2, base=area(0))) == ALIAS
    same = Norm(coco, out=B)
    assert same(normed=mk(coco, B, R, s, 2, base=at(0, 512))) == ALIAS
    assert same(normed=same.hidden) == ALIAS
    assert call(rstd=area(3)) == ALIAS and call(scales=ptrs(coco, 2, area(4))) == ALIAS
    assert call(weight=area(3)) == ALIAS and call(weight=area(5)) == ALIAS and call(rstd=area(5)) == ALIAS
    assert call(scales=ptrs(coco, 2, area(1))) == ALIAS and call(rstd=area(0)) == ALIAS
    assert Norm(coco, shape=(0, 256))() == OK  # nothing to do, nothing launched


def test_norm_backward_refusals(coco):
    B, R, L = coco.BF16, coco.REPLICATED, coco.LOCAL
    s, n = (6, 256), 2
    need = coco.coco_allreduce_rmsnorm_backward_bytes(6, 256)
    assert need == 6 * 256 * 4 and coco.coco_allreduce_rmsnorm_backward_bytes(10 ** 6, 64) == 304 * 64 * 4
    assert coco.coco_allreduce_rmsnorm_backward_bytes(-1, 8) == 0
    assert coco.coco_allreduce_rmsnorm_backward_bytes(4, 1 << 20) == 0
    good = dict(dn=mk(coco, B, L, s, n, base=area(0)), dh=mk(coco, B, R, s, n, base=area(1)),
                h=mk(coco, B, R, s, n, base=area(2)), w=area(3), rstd=area(4),
                dx=mk(coco, B, R, s, n, base=area(5)), dw=area(6), ws=area(7), nb=need)

    def call(**kw):
        a = {**good, **kw}
        return coco.raw_call("coco_allreduce_rmsnorm_backward", ref(a["dn"]), ref(a["dh"]), ref(a["h"]), a["w"],
                             a["rstd"], ref(a["dx"]), a["dw"], a["ws"], a["nb"], None)

    for k in ("dn", "h", "w", "rstd", "dx", "dw", "ws"):
        assert call(**{k: None}) == NULL, k
    assert call(nb=need - 1) == SHAPE
    assert call(dn=mk(coco, B, R, s, n)) == LAYOUT and call(dh=mk(coco, B, L, s, n, base=area(1))) == LAYOUT
    assert call(h=mk(coco, coco.F32, R, s, n, base=area(2))) == DTYPE
    assert call(dx=mk(coco, coco.F8E4M3, R, s, n, base=area(5))) == DTYPE
    assert call(dx=mk(coco, B, R, (5, 256), n, base=area(5))) == SHAPE
    assert call(dh=mk(coco, B, R, s, 3, base=area(1))) == SHAPE
    assert call(w=area(3) + 4) == ALIGN and call(ws=area(7) + 8) == ALIGN and call(dw=area(6) + 1) == ALIGN
    assert call(dx=mk(coco, B, R, s, n, base=area(0) + 16)) == ALIAS
    for k in ("dw", "ws"):
        for a in (0, 1, 2, 3, 4, 5):
            assert call(**{k: area(a)}) == ALIAS, (k, a)
    assert call(ws=area(6)) == ALIAS
    wide = (1, 32784)
    assert call(dn=mk(coco, B, L, wide, n), h=mk(coco, B, R, wide, n, base=area(2)), dh=None,
                dx=mk(coco, B, R, wide, n, base=area(5))) == UNSUPPORTED


def test_quantiser_refusals(coco):
    B, L, R, F8 = coco.BF16, coco.LOCAL, coco.REPLICATED, coco.F8E4M3
    s = (5, 256)

    def call(x=mk(coco, B, L, s, 2), rows=1, q=mk(coco, F8, L, s, 2, base=area(1)), sc=ptrs(coco, 2, area(2))):
        return coco.raw_call("coco_quantize_fp8", ref(x), rows, ref(q), sc, None)

    assert call(x=None) == NULL and call(q=None) == NULL and call(sc=None) == NULL
    assert call(sc=ptrs(coco, 2, 0, area(2))) == NULL
    assert call(x=mk(coco, B, R, s, 2)) == LAYOUT and call(q=mk(coco, F8, R, s, 2, base=area(1))) == LAYOUT
    assert call(x=mk(coco, F8, L, s, 2)) == DTYPE and call(q=mk(coco, B, L, s, 2, base=area(1))) == DTYPE
    assert call(q=mk(coco, F8, L, (5, 128), 2, base=area(1))) == SHAPE
    assert call(q=mk(coco, F8, L, s, 1, base=area(1))) == SHAPE
    for rows in (0, 2, 64, -1):
        assert call(rows=rows) == VALUE
    assert call(sc=ptrs(coco, 2, area(2) + 1)) == ALIGN
    assert call(x=mk(coco, B, L, (5, 24), 2), q=mk(coco, F8, L, (5, 24), 2, base=area(1))) == ALIGN
    assert call(q=mk(coco, F8, L, s, 2, base=FAKE)) == ALIAS
    assert call(q=mk(coco, F8, L, s, 2, base=area(1), stride=0)) == ALIAS  # two ranks' values in one place
    assert call(sc=ptrs(coco, 2, area(1))) == ALIAS and call(sc=ptrs(coco, 2, area(2), 0)) == ALIAS
    none = (0, 256)
    assert call(x=mk(coco, B, L, none, 2), q=mk(coco, F8, L, none, 2, base=area(1))) == OK


def test_product_refusals(coco):
    F8, B, L, R, S = coco.F8E4M3, coco.BF16, coco.LOCAL, coco.REPLICATED, coco.SLICED
    m, k, n = 6, 256, 144

    def call(spec=b"mk,kn->mn", a=mk(coco, F8, L, (m, k), 2), sa=ptrs(coco, 2, area(1)),
             b=mk(coco, F8, L, (k, n), 2, base=area(2)), sb=ptrs(coco, 2, area(3)),
             o=mk(coco, B, L, (m, n), 2, base=area(4))):
        return coco.raw_call("coco_einsum_fp8", spec, ref(a), sa, ref(b), sb, ref(o), None)

    for spec in (None, b"bmk,bkn->bmn", b"mk,kn", b"mk,kn->mnx", b""):
        assert call(spec=spec) == UNSUPPORTED
    assert call(a=None) == NULL and call(b=None) == NULL and call(o=None) == NULL
    assert call(sa=None) == NULL and call(sb=None) == NULL and call(sb=ptrs(coco, 2, 0, area(3))) == NULL
    assert call(a=mk(coco, B, L, (m, k), 2)) == DTYPE and call(b=mk(coco, B, L, (k, n), 2, base=area(2))) == DTYPE
    assert call(o=mk(coco, F8, L, (m, n), 2, base=area(4))) == DTYPE
    assert call(b=mk(coco, F8, L, (n, k), 2, base=area(2))) == SHAPE
    assert call(spec=b"mk,nk->mn") == SHAPE
    assert call(o=mk(coco, B, L, (m + 1, n), 2, base=area(4))) == SHAPE
    assert call(o=mk(coco, B, L, (m, n), 1, base=area(4))) == SHAPE
    assert call(a=mk(coco, F8, L, (2, m, k), 2)) == SHAPE
    assert call(o=mk(coco, B, R, (m, n), 2, base=area(4))) == LAYOUT
    assert call(a=mk(coco, F8, S, (2 * m, k), 2, slice_dim=0)) == LAYOUT
    assert call(b=mk(coco, F8, S, (k, 2 * n), 2, slice_dim=1, base=area(2))) == LAYOUT
    assert call(a=mk(coco, F8, L, (m, k), 2, base=FAKE + 8)) == ALIGN
    assert call(a=mk(coco, F8, L, (m, 8), 2), b=mk(coco, F8, L, (8, n), 2, base=area(2))) == ALIGN
    assert call(sa=ptrs(coco, 2, area(1) + 2)) == ALIGN
    assert call(o=mk(coco, B, L, (m, n), 2, base=FAKE)) == ALIAS
    assert call(o=mk(coco, B, L, (m, n), 2, base=area(1))) == ALIAS
    assert call(o=mk(coco, B, L, (m, n), 2, base=area(4), stride=0)) == ALIAS
    big = (1 << 31)
    assert call(a=mk(coco, F8, L, (big, 16), 2), b=mk(coco, F8, L, (16, n), 2, base=area(2)),
                o=mk(coco, B, L, (big, n), 2, base=area(4))) == UNSUPPORTED
    assert call(a=mk(coco, F8, L, (0, k), 2), o=mk(coco, B, L, (0, n), 2, base=area(4))) == OK


def test_grouped_refusals(coco):
    F8, B, F32, L, R, S = coco.F8E4M3, coco.BF16, coco.F32, coco.LOCAL, coco.REPLICATED, coco.SLICED
    t, k, n, e = 10, 256, 144, 3

    def call(spec=b"tk,ekn->tn", a=mk(coco, B, L, (t, k), 1), sa=None, b=mk(coco, B, L, (e, k, n), 1, base=area(1)),
             sb=None, off=area(2), o=mk(coco, B, L, (t, n), 1, base=area(3))):
        return coco.raw_call("coco_grouped_einsum", spec, ref(a), sa, ref(b), sb, off, ref(o), None)

    for spec in (None, b"tk,kn->tn", b"tk,tn->kn"):
        assert call(spec=spec) == UNSUPPORTED
    assert call(a=None) == NULL and call(off=None) == NULL
    assert call(sa=ptrs(coco, 1, area(4))) == DTYPE and call(sb=ptrs(coco, 1, area(4))) == DTYPE
    assert call(a=mk(coco, coco.F16, L, (t, k), 1)) == DTYPE
    assert call(a=mk(coco, F32, L, (t, k), 1), b=mk(coco, F32, L, (e, k, n), 1, base=area(1))) == UNSUPPORTED
    f8 = dict(a=mk(coco, F8, L, (t, k), 1), b=mk(coco, F8, L, (e, k, n), 1, base=area(1)))
    assert call(**f8) == NULL  # 8-bit operands without scales
    assert call(**f8, sa=ptrs(coco, 1, area(4)), sb=ptrs(coco, 1, area(3))) == ALIAS
    assert call(spec=b"tk,tn->ekn", a=f8["a"], b=mk(coco, F8, L, (t, n), 1, base=area(1)),
                o=mk(coco, B, L, (e, k, n), 1, base=area(3))) == UNSUPPORTED
    assert call(spec=b"tk,enk->tn") == SHAPE and call(b=mk(coco, B, L, (k, n), 1, base=area(1))) == SHAPE
    assert call(o=mk(coco, B, L, (t, n + 8), 1, base=area(3))) == SHAPE
    assert call(spec=b"tk,tn->ekn", b=mk(coco, B, L, (t + 1, n), 1, base=area(1)),
                o=mk(coco, B, L, (e, k, n), 1, base=area(3))) == SHAPE
    assert call(a=mk(coco, B, S, (t, k), 1, slice_dim=1)) == LAYOUT
    assert call(o=mk(coco, B, R, (t, n), 1, base=area(3))) == LAYOUT
    assert call(off=area(2) + 2) == ALIGN
    assert call(off=area(3)) == ALIAS and call(o=mk(coco, B, L, (t, n), 1, base=area(1))) == ALIAS
    many = 65537
    assert call(b=mk(coco, B, L, (many, k, n), 1, base=area(1))) == UNSUPPORTED
    assert call(a=mk(coco, B, L, (0, k), 1), o=mk(coco, B, L, (0, n), 1, base=area(3))) == OK


def test_other_entries_still_refuse_eight_bits(coco):
    F8, L, R = coco.F8E4M3, coco.LOCAL, coco.REPLICATED
    a, o = mk(coco, F8, L, (4, 16), 2), mk(coco, F8, R, (4, 16), 2, base=area(1))
    assert coco.raw_call("coco_allreduce", ref(a), ref(o), None) == DTYPE
    b = mk(coco, F8, L, (16, 16), 2, base=area(2))
    assert coco.raw_call("coco_einsum", b"mk,kn->mn", ref(a), ref(b), ref(mk(coco, F8, L, (4, 16), 2, base=area(3))),
                         None) == DTYPE


def test_binding_refuses_what_the_library_cannot_see(coco):
    """Types, sizes and strides of plain tensors (the library gets their addresses only)."""
    import torch

    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    q = torch.zeros(4, 256, dtype=torch.float8_e4m3fn)
    w, sc = torch.zeros(256, dtype=torch.bfloat16), torch.zeros(4, 2)
    norm = lambda w=w, sc=(sc,), rstd=None: coco.coco_allreduce_rmsnorm(  # noqa: E731
        coco.local([x]), None, w, 1e-5, None, coco.replicated([q]), list(sc), rstd, 0)
    for kw in (dict(w=w.float()), dict(w=w[:128]), dict(sc=(sc.double(),)), dict(sc=(sc[:2],)), dict(sc=(sc, sc)),
               dict(sc=(torch.zeros(2, 4).t(),)), dict(rstd=torch.zeros(3)), dict(rstd=w)):
        with pytest.raises(coco.CocoError):
            norm(**kw)
    b = torch.zeros(2, 256, 256, dtype=torch.float8_e4m3fn)
    sb, out = torch.zeros(2, 2, 2), torch.zeros(4, 256, dtype=torch.bfloat16)
    group = lambda off, sa=sc, sb=sb: coco.coco_grouped_einsum(  # noqa: E731
        "tk,ekn->tn", coco.local([q]), [sa], coco.local([b]), [sb], off, coco.local([out]), 0)
    for args in ((torch.zeros(3),), (torch.zeros(2, dtype=torch.int32),), (torch.zeros(3, dtype=torch.int64),),
                 (torch.zeros(3, dtype=torch.int32), sc[:1]), (torch.zeros(3, dtype=torch.int32), sc, sb[:1])):
        with pytest.raises(coco.CocoError):
            group(*args)
