"""What the binding of the experts' entry points refuses before the library, which gets addresses only. Runs without a
GPU: what passes is refused as host memory, after every check of shapes."""

import pytest
import torch

from test_llm_host import SHAPE, UNSUPPORTED, coco  # noqa: F401 (the fixture)

TOKENS, CHOICES, COLS = 6, 2, 256


def status(coco, f):  # noqa: F811
    with pytest.raises(coco.CocoError) as e:
        f()
    return e.value.status


def calls(c, groups):
    """Per entry point: a call, and the shape and type of its tensors with a value a choice, by name."""
    rows = lambda: [torch.zeros(TOKENS * CHOICES, COLS, dtype=torch.bfloat16) for _ in range(groups)]  # noqa: E731
    toks = lambda: [torch.zeros(TOKENS, COLS, dtype=torch.bfloat16) for _ in range(groups)]  # noqa: E731
    rep, loc = lambda t: c.replicated(t, groups), lambda t: c.local(t, groups)  # noqa: E731
    e = torch.zeros(*([groups] if groups > 1 else []), TOKENS, CHOICES, dtype=torch.int64)
    off = torch.zeros(groups, 4, dtype=torch.int32)
    i, f = torch.int32, torch.float32
    return {
        "sort": (dict(row=i), lambda row: c.coco_expert_sort(e, 3, row, None, off, 0)),
        "dispatch": (dict(row=i), lambda row: c.coco_expert_dispatch(rep(toks()), None, row, rep(rows()), None, 0)),
        "combine": (dict(row=i, gates=f), lambda row, gates: c.coco_expert_combine(loc(rows()), row, gates, rep(toks()),
                                                                                   rep(toks()), 0)),
        "own": (dict(row=i, gates=f), lambda row, gates: c.coco_expert_combine(loc(rows()), row, gates, None,
                                                                               loc(toks()), 0)),
        "back": (dict(row=i, gates=f, dgates=f), lambda row, gates, dgates: c.coco_expert_combine_backward(
            rep(toks()), loc(rows()), row, gates, rep(rows()), dgates, 0)),
    }


@pytest.mark.parametrize("groups", [1, 3])
@pytest.mark.parametrize("name", ["sort", "dispatch", "combine", "own", "back"])
def test_values_of_choices_in_another_order(coco, name, groups):  # noqa: F811
    """As many elements, in the wrong order: the choices first, or the groups last."""
    kinds, call = calls(coco, groups)[name]
    good = (groups, TOKENS, CHOICES) if groups > 1 else (TOKENS, CHOICES)
    make = lambda shape: {k: torch.zeros(shape, dtype=t) for k, t in kinds.items()}  # noqa: E731
    fine = [good, (groups * TOKENS * CHOICES,), (groups * TOKENS, CHOICES), (groups, TOKENS, CHOICES),
            (groups, TOKENS * CHOICES), (groups, 1, TOKENS, CHOICES), (groups * TOKENS, CHOICES, 1)]
    for shape in fine:
        assert status(coco, lambda: call(**make(shape))) == UNSUPPORTED, shape
    wrong = [(CHOICES, TOKENS), (3, 4), (4, 3)] if groups == 1 else \
        [(groups, CHOICES, TOKENS), (TOKENS, groups, CHOICES), (TOKENS, CHOICES, groups), (CHOICES, groups * TOKENS),
         (TOKENS, groups * CHOICES)]
    for shape in wrong:
        for k, t in kinds.items():
            assert status(coco, lambda: call(**{**make(good), k: torch.zeros(shape, dtype=t)})) == SHAPE, (shape, k)
