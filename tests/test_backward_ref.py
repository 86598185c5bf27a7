"""The float64 gradients against differences of the float64 forward, and worked values."""
import math

import numpy as np
import pytest

from oracle.backward_ref import (BF16, backward_bounds, backward_values, down_backward_bounds,
                                 down_backward_values, gate_grads_values)


def silu(x):
    return x / (1 + np.exp(-x))


def forward(a, w1, w2):
    return silu(a @ w1) * (a @ w2)


@pytest.mark.parametrize("M,K,N", [(1, 1, 1), (3, 5, 4), (7, 4, 9)])
def test_gradients_match_central_differences(M, K, N):
    # h = 1e-5: the difference's own error is about h^2 = 1e-10 and eps / h = 1e-11
    rng = np.random.default_rng(M + K + N)
    a, w1, w2 = rng.normal(size=(M, K)), rng.normal(size=(K, N)), rng.normal(size=(K, N))
    dy = rng.normal(size=(M, N))
    args, h = [a, w1, w2], 1e-5
    for which, grad in enumerate(backward_values(a, w1, w2, dy)):
        for at in np.ndindex(*grad.shape):
            vals = []
            for sign in (1, -1):
                moved = [x.copy() for x in args]
                moved[which][at] += sign * h
                vals.append(float((forward(*moved) * dy).sum()))
            assert abs((vals[0] - vals[1]) / (2 * h) - grad[at]) < 1e-7


@pytest.mark.parametrize("M,N,H", [(1, 1, 1), (3, 5, 4)])
def test_down_gradients_match_differences(M, N, H):
    rng = np.random.default_rng(M + N + H)
    y, w3, dout = rng.normal(size=(M, N)), rng.normal(size=(N, H)), rng.normal(size=(M, H))
    dy, dw3 = down_backward_values(dout, w3, y)
    for at in np.ndindex(*dy.shape):  # the map is linear: a unit step is exact
        step = np.zeros_like(y)
        step[at] = 1
        assert abs(((step @ w3) * dout).sum() - dy[at]) < 1e-12
    for at in np.ndindex(*dw3.shape):
        step = np.zeros_like(w3)
        step[at] = 1
        assert abs(((y @ step) * dout).sum() - dw3[at]) < 1e-12


def test_gate_gradients_at_worked_values():
    # s(ln 3) = 3/4: SiLU = 3/4 ln 3, SiLU' = 3/4 + 3/16 ln 3; at 0: 0 and 1/2
    g, u, dy = np.array([math.log(3), 0.0, -800.0, 800.0]), np.full(4, 2.0), np.full(4, 5.0)
    dg, du = gate_grads_values(g, u, dy)
    assert np.allclose(du, [5 * 0.75 * math.log(3), 0.0, 0.0, 4000.0], rtol=1e-15, atol=1e-300)
    assert np.allclose(dg, [10 * (0.75 + 3 / 16 * math.log(3)), 5.0, 0.0, 10.0], rtol=1e-15, atol=1e-300)


def test_bounds_are_a_few_roundings():
    # typical entries: the bound is a small multiple of one bf16 rounding of the terms' sum
    rng = np.random.default_rng(0)
    a, dy = rng.normal(size=(32, 64)), rng.normal(size=(32, 48))
    w1, w2 = (rng.normal(size=(64, 48)) / 8 for _ in range(2))
    for ref, bound in zip(backward_values(a, w1, w2, dy), backward_bounds(a, w1, w2, dy)):
        assert bound.shape == ref.shape and (bound > 0).all()
        assert np.median(bound) < 0.06 * np.sqrt((ref ** 2).mean())
    w3, dout = rng.normal(size=(48, 40)), rng.normal(size=(32, 40))
    for ref, bound in zip(down_backward_values(dout, w3, dy), down_backward_bounds(dout, w3, dy)):
        assert bound.shape == ref.shape
        assert np.median(bound) < 0.02 * np.sqrt((ref ** 2).mean())


def test_rounding_constant_is_that_of_bf16():
    # just above a power of two, half way between two bf16 values: 1 + 2^-8 rounds by 2^-8
    import torch
    x = torch.linspace(1, 2, 100001, dtype=torch.float64)
    rel = ((x.to(torch.bfloat16).double() - x).abs() / x).max().item()
    assert 0.99 * BF16 < rel <= BF16
