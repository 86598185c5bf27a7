"""float64 gradients of the gated MLP, and bounds on what 16-bit kernels may differ by.

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__.py``).

The forward's definition ("Tile-Level Activation Overlap for Efficient LLM
Inference", gist.science, section "Problem Statement") is
Y = SiLU(G) (.) U with G = A x W1, U = A x W2; the down-projection is
Out = Y x W3 + R. With s = 1 / (1 + exp(-G)) and SiLU(G) = G s,
SiLU'(G) = s + G s (1 - s), so for an incoming dY

    dU = dY G s,  dG = dY U SiLU'(G),
    dA = dG W1^T + dU W2^T,  dW1 = A^T dG,  dW2 = A^T dU,

and dY = dOut W3^T, dW3 = Y^T dOut, dR = dOut.

The bounds are worst-case sums of the roundings the kernels are allowed: fp32
products summed in any order (at most one part in 2^23 a term), dG and dU
rounded once to bf16, the exponential to a part in 2^16, the output rounded
once to bf16 (half a unit in the last of 8 bits: a part in 2^8).
"""
from __future__ import annotations

import numpy as np

BF16 = 2.0 ** -8    # largest relative error of one rounding to bf16 (8 significant bits)
FP32 = 2.0 ** -23   # per term of an fp32 sum (a truncating adder included)
EXP = 2.0 ** -16    # fast exponential and divide, for |G| up to some tens
TINY = 1e-30


def gate_grads_values(g, u, dy):
    """(dG, dU) in float64 from float64 G, U and dY."""
    s = np.where(g >= 0, 1 / (1 + np.exp(-np.abs(g))), np.exp(-np.abs(g)) / (1 + np.exp(-np.abs(g))))
    return dy * u * (s + g * s * (1 - s)), dy * g * s


def backward_values(a, w1, w2, dy):
    """(dA, dW1, dW2) in float64."""
    dg, du = gate_grads_values(a @ w1, a @ w2, dy)
    return dg @ w1.T + du @ w2.T, a.T @ dg, a.T @ du


def backward_bounds(a, w1, w2, dy):
    """Elementwise bounds on the errors of (dA, dW1, dW2)."""
    g, u = a @ w1, a @ w2
    dg, du = gate_grads_values(g, u, dy)
    k = a.shape[1]
    eg = k * FP32 * (abs(a) @ abs(w1))
    eu = k * FP32 * (abs(a) @ abs(w2))
    # |SiLU'| <= 1.1 and |SiLU''| <= 0.5
    edu = 1.1 * abs(dy) * eg + (BF16 + EXP) * abs(du)
    edg = abs(dy) * (0.5 * abs(u) * eg + 1.1 * eu) + (BF16 + EXP) * abs(dg)
    n, m = w1.shape[1], a.shape[0]
    ea = (edg + 2 * n * FP32 * abs(dg)) @ abs(w1).T + (edu + 2 * n * FP32 * abs(du)) @ abs(w2).T
    e1 = abs(a).T @ (edg + m * FP32 * abs(dg))
    e2 = abs(a).T @ (edu + m * FP32 * abs(du))
    out = []
    for e, ref in zip((ea, e1, e2), (dg @ w1.T + du @ w2.T, a.T @ dg, a.T @ du)):
        out.append(e + BF16 * (abs(ref) + e) + TINY)
    return out


def down_backward_values(dout, w3, y):
    """(dY, dW3) in float64."""
    return dout @ w3.T, y.T @ dout


def down_backward_bounds(dout, w3, y):
    """Elementwise bounds on the errors of (dY, dW3): fp32 sums and one rounding."""
    out = []
    for x, z, n in ((dout, w3.T, dout.shape[1]), (y.T, dout, dout.shape[0])):
        e = n * FP32 * (abs(x) @ abs(z))
        out.append(e + BF16 * (abs(x @ z) + e) + TINY)
    return out
