"""8-bit and expert-grouped operators, in float64 NumPy (test infrastructure only).

The pages have none of these; the definitions are the published ones: the
root-mean-square norm of Zhang and Sennrich ("Root Mean Square Layer
Normalization", 2019), the e4m3 format of the OCP "8-bit Floating Point
Specification" (four exponent bits of bias 7, three fraction bits, largest value
448, no infinity, code 0x7f for NaN), and products of block-scaled values and
of expert-sorted rows written out as sums.
"""

import numpy as np

BLOCK = 128
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100


def e4m3_table():
    """The value of each of the 256 codes."""
    out = np.empty(256)
    for code in range(256):
        sign = -1.0 if code & 0x80 else 1.0
        exp, frac = (code >> 3) & 15, code & 7
        if exp == 15 and frac == 7:
            out[code] = np.nan
        elif exp == 0:
            out[code] = sign * frac * 2.0 ** -9
        else:
            out[code] = sign * (1 + frac / 8) * 2.0 ** (exp - 7)
    return out


def to_e4m3(x):
    """x rounded to the nearest e4m3 value, ties to the even code, magnitudes above 448 to 448."""
    grid = e4m3_table()[:127]  # 0, 2^-9, ..., 448: ascending in the code
    a = np.minimum(np.abs(x), E4M3_MAX)
    hi = np.clip(np.searchsorted(grid, a), 1, 126)  # grid[hi - 1] <= a <= grid[hi]
    below, above = a - grid[hi - 1], grid[hi] - a
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    return np.where(np.isnan(x), np.nan, np.copysign(grid[np.where(up, hi, hi - 1)], x))


def block_amax(x, block_rows):
    """The largest magnitude of every block_rows x 128 block of a 2-D array (NaN where a block holds one)."""
    rows, cols = x.shape
    out = np.zeros((-(-rows // block_rows), -(-cols // BLOCK)))
    for i in range(out.shape[0]):
        for j in range(out.shape[1]):
            b = x[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK]
            out[i, j] = np.max(np.abs(b))
    return out


def scales_of(x, block_rows):
    return np.maximum(block_amax(x, block_rows), AMAX_FLOOR) / E4M3_MAX


def spread(scales, shape, block_rows):
    """The scale of every element of a `shape` array."""
    up = np.repeat(np.repeat(scales, block_rows, 0), BLOCK, 1)
    return up[:shape[0], :shape[1]]


def quantize(x, block_rows):
    """(e4m3 values, scales) of a 2-D array."""
    s = scales_of(x, block_rows)
    return to_e4m3(x / spread(s, x.shape, block_rows)), s


def dequantize(q, scales, block_rows):
    return q * spread(scales, q.shape, block_rows)


def allreduce_rmsnorm(partials, residual, weight, eps):
    """(h, y, 1 / rms) over the last dimension."""
    h = sum(partials) + (0.0 if residual is None else residual)
    rstd = 1.0 / np.sqrt(np.mean(h * h, -1) + eps)
    return h, h * rstd[..., None] * weight, rstd


def allreduce_rmsnorm_backward(dnormed, dhidden, h, rstd, weight):
    """(gradient of h, gradient of the weight) for sum(y * sum(dnormed)) + sum(h * dhidden)."""
    dy = sum(dnormed)
    xhat = h * rstd[..., None]
    g = dy * weight
    dh = rstd[..., None] * (g - xhat * np.mean(g * xhat, -1, keepdims=True))
    return dh + (0.0 if dhidden is None else dhidden), (dy * xhat).reshape(-1, h.shape[-1]).sum(0)


def grouped_einsum(form, lhs, rhs, offsets):
    """Products by expert: form "kn" / "nk" (rhs [e, k, n] / [e, n, k]) or "grad" (rhs [t, n], out [e, k, n])."""
    experts = len(offsets) - 1
    if form == "grad":
        out = np.zeros((experts, lhs.shape[1], rhs.shape[1]))
    else:
        out = np.zeros((lhs.shape[0], rhs.shape[2 if form == "kn" else 1]))
    for e in range(experts):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if form == "grad":
            out[e] = lhs[a:b].T @ rhs[a:b]
        else:
            out[a:b] = lhs[a:b] @ (rhs[e] if form == "kn" else rhs[e].T)
    return out


def moe_layer(partials, residual, weight, eps, expert_of, gates, up, down):
    """(h, x, sum of the ranks' outputs) of a mixture-of-experts layer: per token and choice, a loop."""
    h, x, _ = allreduce_rmsnorm(partials, residual, weight, eps)
    y = np.zeros_like(h)
    for t in range(h.shape[0]):
        for j in range(expert_of.shape[1]):
            e = int(expert_of[t, j])
            for u, d in zip(up, down):
                y[t] += gates[t, j] * (np.maximum(x[t] @ u[e], 0.0) @ d[e])
    return h, x, y


def moe_layer_backward(partials, residual, weight, eps, expert_of, up, down, dout, active=None):
    """Gradients of sum(dout * (h + y)) (gates of one): (of h, of the weight, of up per rank, of down per rank).

    ``active[r][t, j]``: which hidden units of rank r are positive for choice j of token t, where another forward
    decided that (a unit within rounding of zero has two gradients); by default this one's."""
    h, x, rstd = allreduce_rmsnorm(partials, residual, weight, eps)
    dx, dup, ddown = np.zeros_like(h), [np.zeros_like(u) for u in up], [np.zeros_like(d) for d in down]
    for t in range(h.shape[0]):
        for j in range(expert_of.shape[1]):
            e = int(expert_of[t, j])
            for r, (u, d) in enumerate(zip(up, down)):
                mid = x[t] @ u[e]
                on = mid > 0 if active is None else active[r][t, j]
                dmid = (d[e] @ dout[t]) * on
                ddown[r][e] += np.outer(mid * on, dout[t])
                dup[r][e] += np.outer(x[t], dmid)
                dx[t] += u[e] @ dmid
    dh, dw = allreduce_rmsnorm_backward([dx], dout, h, rstd, weight)
    return dh, dw, dup, ddown
