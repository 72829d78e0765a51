"""Pins of the oracle's 8-bit and expert-grouped operators to facts fixed outside it."""

import numpy as np
import pytest
import torch

import oracle


def test_e4m3_codes_are_the_formats():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.e4m3_table(), codes, equal_nan=True)


def test_e4m3_rounding_against_an_independent_converter():
    rng = np.random.default_rng(1)
    x = np.concatenate([rng.standard_normal(4096) * 10.0 ** rng.uniform(-5, 2.6, 4096),
                        oracle.e4m3_table()[:127], (oracle.e4m3_table()[:126] + oracle.e4m3_table()[1:127]) / 2])
    x = np.clip(np.concatenate([x, -x]), -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(oracle.to_e4m3(x.astype(np.float64)), want)
    assert oracle.to_e4m3(np.array([1e9, -np.inf]))[0] == 448.0
    assert np.isnan(oracle.to_e4m3(np.array([np.nan]))[0])


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("shape", [(1, 16), (130, 272), (3, 128)])
def test_quantised_values_stand_within_half_a_step(shape, block_rows):
    x = np.random.default_rng(2).standard_normal(shape)
    q, s = oracle.quantize(x, block_rows)
    assert s.shape == (-(-shape[0] // block_rows), -(-shape[1] // 128))
    assert np.allclose(s * 448, oracle.block_amax(x, block_rows))
    back = oracle.dequantize(q, s, block_rows)
    half = np.maximum(np.abs(x) / 16, oracle.spread(s, x.shape, block_rows) * 2.0 ** -10)
    assert np.all(np.abs(back - x) <= half * (1 + 1e-12))
    i, j = np.unravel_index(np.argmax(np.abs(x)), x.shape)
    assert np.isclose(back[i, j], x[i, j])  # a block's largest value is held exactly
    assert np.array_equal(oracle.scales_of(np.zeros(shape), block_rows).ravel()[:1], [2.0 ** -100 / 448])


def test_norm_has_unit_mean_square_and_its_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(3)
    parts, res = [rng.standard_normal((5, 24)) for _ in range(3)], rng.standard_normal((5, 24))
    w = rng.standard_normal(24)
    h, y, rstd = oracle.allreduce_rmsnorm(parts, res, w, 0.0)
    assert np.allclose(h, parts[0] + parts[1] + parts[2] + res)
    assert np.allclose(np.mean((y / w) ** 2, -1), 1.0)
    dy, dh = [rng.standard_normal((5, 24)) for _ in range(2)], rng.standard_normal((5, 24))

    def loss(p0, weight):
        hh, yy, _ = oracle.allreduce_rmsnorm([p0] + parts[1:], res, weight, 1e-3)
        return np.sum(yy * (dy[0] + dy[1])) + np.sum(hh * dh)

    h, _, rstd = oracle.allreduce_rmsnorm(parts, res, w, 1e-3)
    dx, dw = oracle.allreduce_rmsnorm_backward(dy, dh, h, rstd, w)
    for _ in range(8):
        d, dwt, t = rng.standard_normal(h.shape), rng.standard_normal(24), 1e-5
        got = (loss(parts[0] + t * d, w) - loss(parts[0] - t * d, w)) / (2 * t)
        assert np.isclose(got, np.sum(dx * d), rtol=1e-7, atol=1e-7)
        got = (loss(parts[0], w + t * dwt) - loss(parts[0], w - t * dwt)) / (2 * t)
        assert np.isclose(got, np.sum(dw * dwt), rtol=1e-7, atol=1e-7)


def test_grouped_products_by_brute_force():
    rng = np.random.default_rng(4)
    off = np.array([1, 3, 3, 7])  # one expert without rows, one row of none at each end
    lhs, rhs, dy = rng.standard_normal((8, 5)), rng.standard_normal((3, 5, 4)), rng.standard_normal((8, 4))
    expert = {1: 0, 2: 0, 3: 2, 4: 2, 5: 2, 6: 2}
    out, grad = np.zeros((8, 4)), np.zeros((3, 5, 4))
    for t, e in expert.items():
        for n in range(4):
            for k in range(5):
                out[t, n] += lhs[t, k] * rhs[e, k, n]
                grad[e, k, n] += lhs[t, k] * dy[t, n]
    assert np.allclose(oracle.grouped_einsum("kn", lhs, rhs, off), out)
    assert np.allclose(oracle.grouped_einsum("nk", lhs, rhs.transpose(0, 2, 1), off), out)
    assert np.allclose(oracle.grouped_einsum("grad", lhs, dy, off), grad)


def test_moe_layer_by_grouped_products_and_its_gradient_by_differences():
    rng = np.random.default_rng(5)
    t, hid, f, e, n = 6, 8, 5, 3, 2
    parts, res = [rng.standard_normal((t, hid)) for _ in range(n)], rng.standard_normal((t, hid))
    w, dout = rng.standard_normal(hid), rng.standard_normal((t, hid))
    up, down = [rng.standard_normal((e, hid, f)) for _ in range(n)], [rng.standard_normal((e, f, hid)) for _ in range(n)]
    expert_of = rng.integers(0, e, (t, 2))
    gates = rng.uniform(0, 1, (t, 2))
    h, x, y = oracle.moe_layer(parts, res, w, 1e-3, expert_of, gates, up, down)
    order = np.argsort(expert_of.ravel(), kind="stable")
    off = np.concatenate([[0], np.cumsum(np.bincount(expert_of.ravel(), minlength=e))])
    want = np.zeros_like(y)
    for u, d in zip(up, down):
        o = oracle.grouped_einsum("kn", np.maximum(oracle.grouped_einsum("kn", x[order // 2], u, off), 0), d, off)
        np.add.at(want, order // 2, o * gates.ravel()[order][:, None])
    assert np.allclose(y, want)

    def loss(p0, weight, u0, d0):
        hh, _, yy = oracle.moe_layer([p0] + parts[1:], res, weight, 1e-3, expert_of, np.ones((t, 2)), [u0] + up[1:],
                                     [d0] + down[1:])
        return np.sum(dout * (hh + yy))

    grads = oracle.moe_layer_backward(parts, res, w, 1e-3, expert_of, up, down, dout)
    at = [parts[0], w, up[0], down[0]]
    for i, g in enumerate([grads[0], grads[1], grads[2][0], grads[3][0]]):
        d, s = rng.standard_normal(g.shape), 1e-6
        hi, lo = list(at), list(at)
        hi[i], lo[i] = at[i] + s * d, at[i] - s * d
        assert np.isclose((loss(*hi) - loss(*lo)) / (2 * s), np.sum(g * d), rtol=1e-6, atol=1e-6), i
