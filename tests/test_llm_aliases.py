"""Groups run at the same time and each reads its own inputs only: what may share memory within a group may not across
groups. Host only (fake pointers, refused before any CUDA call)."""

import ctypes

import pytest

from test_abi_host import mk
from test_llm_host import ALIAS, Norm, area, coco, ptrs, ref  # noqa: F401 (coco: the fixture)

S = (4, 256)
GROUPS, N = 2, 2


def at(i, p):
    """Pointer p of memory area i, as mk lays them out."""
    return area(i) + p * (1 << 32)


def swapped(i, other, which=(0, 2)):
    """The pointers of area i with those at `which[0]` taken from area `other` at `which[1]`."""
    out = [at(i, p) for p in range(GROUPS * N)]
    out[which[0]] = at(other, which[1])
    return out


@pytest.fixture
def norm(coco):  # noqa: F811
    def build(out=None):
        B, L, R = coco.BF16, coco.LOCAL, coco.REPLICATED
        call = Norm(coco, n=GROUPS * N, out=out)
        call.partials = mk(coco, B, L, S, N, GROUPS, base=area(0))
        call.residual = mk(coco, B, R, S, N, GROUPS, base=area(1))
        call.hidden = mk(coco, B, R, S, N, GROUPS, base=area(3))
        call.normed = mk(coco, coco.F8E4M3 if out is None else out, R, S, N, GROUPS, base=area(4))
        return call
    return build


def test_norm_outputs_stay_out_of_other_groups(coco, norm):  # noqa: F811
    B, R = coco.BF16, coco.REPLICATED
    call, same = norm(), norm(coco.BF16)
    rep = lambda p, dt=B: mk(coco, dt, R, S, N, GROUPS, ptrs=p)  # noqa: E731
    for which in ((0, 2), (0, 3), (1, 2), (2, 0), (3, 1)):  # (an output of one group, an input of the other)
        assert call(hidden=rep(swapped(3, 0, which))) == ALIAS, which
        assert same(normed=rep(swapped(4, 0, which))) == ALIAS, which
    for which in ((0, 2), (2, 0)):  # (a group's residual is read from its first rank)
        assert call(hidden=rep(swapped(3, 1, which))) == ALIAS, which
        assert same(normed=rep(swapped(4, 1, which))) == ALIAS, which
    for which in ((0, 2), (1, 3), (1, 2)):  # (the two groups' outputs in one place)
        assert call(hidden=rep(swapped(3, 3, which))) == ALIAS, which
        assert call(normed=rep(swapped(4, 4, which), coco.F8E4M3)) == ALIAS, which
        assert same(normed=rep(swapped(4, 4, which))) == ALIAS, which
        sc = [at(5, p) for p in range(GROUPS * N)]
        sc[which[0]] = at(5, which[1])
        assert call(scales=(ctypes.c_void_p * len(sc))(*sc)) == ALIAS, which
    # one residual for both groups, where a group's hidden rows take its place
    both = [at(1, 0)] * (GROUPS * N)
    assert call(residual=rep(both), hidden=rep([at(1, 0), at(1, 0), at(3, 2), at(3, 3)])) == ALIAS


def test_norm_gradients_stay_out_of_other_groups(coco):  # noqa: F811
    B, L, R = coco.BF16, coco.LOCAL, coco.REPLICATED
    need = coco.coco_allreduce_rmsnorm_backward_bytes(4 * GROUPS, 256)
    good = [mk(coco, B, lay, S, N, GROUPS, base=area(i)) for lay, i in ((L, 0), (R, 1), (R, 2))]

    def call(dx):
        return coco.raw_call("coco_allreduce_rmsnorm_backward", ref(good[0]), ref(good[1]), ref(good[2]), area(3),
                             area(4), ref(mk(coco, B, R, S, N, GROUPS, ptrs=dx)), area(6), area(7), need, None)

    for other in (0, 1, 2):  # dnormed, dhidden, hidden
        for which in ((0, 2), (2, 0)):
            assert call(swapped(5, other, which)) == ALIAS, (other, which)
    assert call(swapped(5, 0, (1, 3))) == ALIAS
    for which in ((0, 2), (1, 3), (3, 0)):
        assert call(swapped(5, 5, which)) == ALIAS, which
