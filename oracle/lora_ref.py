"""float64 projections with one low-rank adapter per token, and bounds on 16-bit kernels' errors.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The shared projections are those of "Tile-Level Activation Overlap for
Efficient LLM Inference" (gist.science, section "Problem Statement"); the pages
do not cover adapters. The reading is the usual one: a linear map W becomes
W + scale_a (Lb_a La_a)^T for the tokens of adapter a, so for token m with
a = index[m] (outside the table: no adapter)

    Gate[m] = A[m] W1 + scale_a (A[m] La[a, 0]^T) Lb[a, 0]^T    (Up with W2 and La, Lb [a, 1])
    Y[m]    = SiLU(Gate[m]) Up[m]
    Out[m]  = Y[m] W3 + R[m] + scale_a (Y[m] La[a]^T) Lb[a]^T

Adapters are taken one token group at a time, so a token meets no other
adapter's values. The bounds are worst-case sums of the roundings allowed:
fp32 sums, V rounded to bf16, the exponential, one rounding of the output.
"""
from __future__ import annotations

import numpy as np

from .backward_ref import BF16, EXP, FP32, TINY


def adapted_values(x, w, la, lb, index, scale):
    """(x W + each token's adapter, its bound before rounding); la [L, r, in], lb [L, out, r]."""
    out = x @ w
    err = x.shape[1] * FP32 * (abs(x) @ abs(w))
    for a in range(la.shape[0]):
        rows = np.nonzero(index == a)[0]
        if rows.size == 0:
            continue
        v = scale[a] * (x[rows] @ la[a].T)
        ev = abs(scale[a]) * (x.shape[1] + 2) * FP32 * (abs(x[rows]) @ abs(la[a]).T) + BF16 * abs(v)
        out[rows] += v @ lb[a].T
        # the delta joins the same sum: its terms and the whole sum once more per term
        err[rows] += (ev + (la.shape[1] + 2) * FP32 * abs(v)) @ abs(lb[a]).T
    err += 66 * FP32 * abs(out)
    return out, err


def forward_lora(a, w1, w2, la, lb, index, scale):
    """(Y, bound) in float64; la [L, 2, r, K], lb [L, 2, N, r]."""
    g, eg = adapted_values(a, w1, la[:, 0], lb[:, 0], index, scale)
    u, eu = adapted_values(a, w2, la[:, 1], lb[:, 1], index, scale)
    e = np.exp(-np.abs(g))
    silu = g * np.where(g >= 0, 1 / (1 + e), e / (1 + e))
    y = silu * u
    err = 1.1 * eg * (abs(u) + eu) + abs(silu) * eu + EXP * abs(y)
    return y, err + BF16 * (abs(y) + err) + TINY


def down_forward_lora(y, w3, r, la, lb, index, scale):
    """(Out, bound) in float64; r may be None; la [L, r, N], lb [L, H, r]."""
    out, err = adapted_values(y, w3, la, lb, index, scale)
    if r is not None:
        out = out + r
        err = err + 2 * FP32 * abs(out)
    return out, err + BF16 * (abs(out) + err) + TINY
