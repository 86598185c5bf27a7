"""float64 reference of the 8-bit integer format, and of what computes with it.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

A group of values x is held as codes q and a scale s: m = max(max |x|, 2^-100),
s = m / 127 rounded to fp32, q = 127 x / m rounded half to even. Where x is bf16
the quotient is a ratio of integers below 2^15 and 2^8, so in float64 it is a
half exactly or at least 2^-10 away from one: the codes have one right value.

The bounds are worst-case sums of the roundings the kernels make, as in
``backward_ref``: an fp32 sum of n terms, BF16 for a value rounded to bf16, EXP for
the exponential and the divide.
"""
from __future__ import annotations

import numpy as np

from .backward_ref import BF16, EXP, FP32, TINY, gate_grads_values

LEAST = 2.0 ** -100
BLOCK = 128


def quantise(x):
    """(codes, scales) of float64 rows x [..., n]; codes of rows with a NaN or an infinity mean nothing."""
    top = np.abs(x).max(-1)
    m = np.maximum(top, LEAST)
    with np.errstate(invalid="ignore"):
        codes = np.rint(127 * x / m[..., None])
    scale = np.where(np.isfinite(top), (m.astype(np.float32) / np.float32(127)).astype(np.float64), np.nan)
    return codes, scale


def blocks(n):
    return -(-n // BLOCK)


def wide(scale, n):
    """scales [blocks, M] as one per value, [M, n]."""
    return np.repeat(scale, BLOCK, 0)[:n].T


def block_largest(x):
    """Largest magnitudes of x [M, N] per token and 128 columns, [blocks, M]."""
    m, n = x.shape
    padded = np.zeros((m, blocks(n) * BLOCK))
    padded[:, :n] = np.abs(x)
    return padded.reshape(m, -1, BLOCK).max(2).T


def silu(g):
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g))


def product(q, sa, w, sw):
    """(value, bound) of (q w) sa sw: codes [M, K] and [K, N], a scale per row and per column.
    Products of codes are integers below 2^14 and exact; their fp32 sum errs as n terms do, and the
    two scales round twice."""
    exact = (q @ w) * sa[:, None] * sw
    err = (q.shape[1] * FP32 * (abs(q) @ abs(w))) * sa[:, None] * sw + 2 * FP32 * abs(exact)
    return exact, err


def gated(g, eg, u, eu):
    """(value, bound) of SiLU(g) u rounded to bf16, from g and u with bounds."""
    y = silu(g) * u
    e = 1.1 * eg * (abs(u) + eu) + abs(silu(g)) * eu + EXP * abs(y)
    return y, e + BF16 * (abs(y) + e) + TINY


def added(x, e, r):
    """(value, bound) of x + r rounded to bf16, from x with a bound."""
    y = x + r
    e = e + FP32 * abs(y)
    return y, e + BF16 * (abs(y) + e) + TINY


def checkpoint_grads(g, u, dy):
    """(dG, dU, bounds) of the checkpoint's values: fp32 arithmetic, one rounding to bf16. The value
    code * scale is rounded to fp32 too, which moves SiLU' by 0.5 |g| and SiLU by 1.1 |g| of that."""
    dg, du = gate_grads_values(g, u, dy)
    eg = FP32 * abs(g)
    edg = abs(dy) * (0.5 * abs(u) * eg + 1.1 * FP32 * abs(u)) + (BF16 + EXP) * abs(dg)
    edu = 1.1 * abs(dy) * eg + (BF16 + EXP) * abs(du)
    return dg, du, edg, edu


def backward_values(a, w1, w2, g, u, dy):
    dg, du = gate_grads_values(g, u, dy)
    return dg @ w1.T + du @ w2.T, a.T @ dg, a.T @ du


def backward_bounds(a, w1, w2, g, u, dy, a_err=0.0):
    """Bounds on (dA, dW1, dW2); a_err: what each of the input's values may be off by."""
    dg, du, edg, edu = checkpoint_grads(g, u, dy)
    n, m = w1.shape[1], a.shape[0]
    ea = (edg + 2 * n * FP32 * abs(dg)) @ abs(w1).T + (edu + 2 * n * FP32 * abs(du)) @ abs(w2).T
    aa = abs(a) + a_err
    e1 = aa.T @ (edg + m * FP32 * abs(dg)) + (a_err + 0 * a).T @ abs(dg)
    e2 = aa.T @ (edu + m * FP32 * abs(du)) + (a_err + 0 * a).T @ abs(du)
    return [e + BF16 * (abs(ref) + e) + TINY
            for e, ref in zip((ea, e1, e2), backward_values(a, w1, w2, g, u, dy))]
