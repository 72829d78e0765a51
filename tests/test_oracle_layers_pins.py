"""Pins of the oracle's experts' rows, layer norm and clipping to facts fixed outside it."""

import numpy as np
import torch

import oracle


def test_sorting_against_a_stable_sort():
    rng = np.random.default_rng(11)
    for tokens, choices, experts in [(1, 1, 1), (7, 3, 5), (40, 2, 64), (0, 2, 4), (5, 2, 0)]:
        e = rng.integers(-2, experts + 2, (tokens, choices))
        row_of, choice_of, offsets = oracle.expert_sort(e, experts)
        flat = e.reshape(-1)
        live = np.flatnonzero((flat >= 0) & (flat < experts))
        order = live[np.argsort(flat[live], kind="stable")]
        assert np.array_equal(choice_of[:len(order)], order) and np.all(choice_of[len(order):] == -1)
        assert np.array_equal(row_of.reshape(-1)[order], np.arange(len(order)))
        assert np.all(np.delete(row_of.reshape(-1), live) == -1)
        assert np.array_equal(np.diff(offsets), np.bincount(flat[live], minlength=experts)[:experts])


def test_combining_is_a_product_with_the_gates_and_its_gradient_the_difference_quotient():
    rng = np.random.default_rng(12)
    tokens, choices, cols = 6, 3, 10
    e = rng.integers(-1, 4, (tokens, choices))
    row_of, _, _ = oracle.expert_sort(e, 4)
    rows, gates = [rng.standard_normal((tokens * choices, cols)) for _ in range(2)], rng.standard_normal(e.shape)
    res, dout = rng.standard_normal((tokens, cols)), rng.standard_normal((tokens, cols))
    m = np.zeros((tokens, tokens * choices))
    for t, k in np.argwhere(row_of >= 0):
        m[t, row_of[t, k]] += gates[t, k]
    assert np.allclose(oracle.expert_combine(rows, row_of, gates, res), m @ (rows[0] + rows[1]) + res)
    drows, dgates = oracle.expert_combine_backward(dout, rows, row_of, gates, np.zeros_like(rows[0]))
    assert np.allclose(drows, m.T @ dout)
    loss = lambda r0, g: np.sum(oracle.expert_combine([r0, rows[1]], row_of, g, res) * dout)  # noqa: E731
    d, dg = rng.standard_normal(rows[0].shape), rng.standard_normal(gates.shape)
    assert np.isclose(loss(rows[0] + d, gates) - loss(rows[0], gates), np.sum(drows * d))  # linear in each
    assert np.isclose(loss(rows[0], gates + dg) - loss(rows[0], gates), np.sum(dgates * dg))
    # dispatching is the transpose of combining with ones
    x = rng.standard_normal((tokens, cols))
    sent = oracle.expert_dispatch(x, row_of, np.zeros_like(rows[0]))
    assert np.isclose(np.sum(sent * rows[0]), np.sum(x * oracle.expert_combine([rows[0]], row_of, None, None)))


def test_layer_norm_against_pytorch_and_the_difference_quotient():
    rng = np.random.default_rng(13)
    parts, res = [rng.standard_normal((5, 24)) + 3 for _ in range(3)], rng.standard_normal((5, 24))
    w, b = rng.standard_normal(24), rng.standard_normal(24)
    h, y, mean, rstd = oracle.allreduce_layernorm(parts, res, w, b, 1e-3)
    t = torch.from_numpy
    assert np.allclose(y, torch.nn.functional.layer_norm(t(h), (24,), t(w), t(b), 1e-3).numpy())
    assert np.allclose(mean, h.mean(-1)) and np.allclose(rstd, 1 / np.sqrt(h.var(-1) + 1e-3))
    dy, dh = [rng.standard_normal((5, 24)) for _ in range(2)], rng.standard_normal((5, 24))

    def loss(p0, weight, bias):
        hh, yy, _, _ = oracle.allreduce_layernorm([p0] + parts[1:], res, weight, bias, 1e-3)
        return np.sum(yy * (dy[0] + dy[1])) + np.sum(hh * dh)

    dx, dw, db = oracle.allreduce_layernorm_backward(dy, dh, h, mean, rstd, w)
    step = 1e-5
    for _ in range(4):
        for i, g in enumerate((dx, dw, db)):
            at = [parts[0], w, b]
            d = rng.standard_normal(at[i].shape)
            up, down = list(at), list(at)
            up[i], down[i] = at[i] + step * d, at[i] - step * d
            assert np.isclose((loss(*up) - loss(*down)) / (2 * step), np.sum(g * d), rtol=1e-7, atol=1e-7)


def test_clipping_reaches_the_norm_and_leaves_smaller_ones():
    rng = np.random.default_rng(14)
    ts = [rng.standard_normal(s) for s in (3, (4, 5), 0, 1)]
    out, norm = oracle.clip(ts, 0.5)
    params = [torch.nn.Parameter(torch.from_numpy(np.asarray(t))) for t in ts]
    assert np.isclose(norm, np.linalg.norm(np.concatenate([t.ravel() for t in ts])))
    assert np.isclose(np.linalg.norm(np.concatenate([t.ravel() for t in out])), 0.5)
    for p in params:
        p.grad = p.detach().clone()
    torch.nn.utils.clip_grad_norm_(params, 0.5)
    for p, o in zip(params, out):
        assert np.allclose(p.grad.numpy(), o, rtol=1e-5)
    same, _ = oracle.clip(ts, norm)
    assert all(np.array_equal(a, b) for a, b in zip(same, ts))
