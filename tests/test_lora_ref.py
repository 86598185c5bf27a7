"""The float64 adapter projections against merged weights and worked values."""
import numpy as np
import pytest

from oracle.down_ref import down_f64_values
from oracle.lora_ref import down_forward_lora, forward_lora


def silu(x):
    return x / (1 + np.exp(-x))


@pytest.mark.parametrize("M,K,N,L,r", [(1, 3, 4, 1, 2), (7, 5, 6, 3, 2)])
def test_adapters_equal_merged_weights(M, K, N, L, r):
    # every token by itself, with W + scale (Lb La)^T written out
    rng = np.random.default_rng(M)
    a, w1, w2, w3 = (rng.normal(size=s) for s in ((M, K), (K, N), (K, N), (K, N)))
    la, lb = rng.normal(size=(L, 2, r, K)), rng.normal(size=(L, 2, N, r))
    scale, index = rng.normal(size=L), rng.integers(-1, L + 1, M)
    y, bound = forward_lora(a, w1, w2, la, lb, index, scale)
    out, _ = down_forward_lora(a, w3, rng.normal(size=(M, N)) * 0 + 2, la[:, 0], lb[:, 0], index, scale)
    assert (bound > 0).all()
    for m in range(M):
        i = index[m]
        d = [np.zeros((K, N))] * 2 if not 0 <= i < L else [scale[i] * (lb[i, h] @ la[i, h]).T for h in (0, 1)]
        assert np.allclose(y[m], silu(a[m] @ (w1 + d[0])) * (a[m] @ (w2 + d[1])), rtol=1e-12, atol=1e-12)
        assert np.allclose(out[m], a[m] @ (w3 + d[0]) + 2, rtol=1e-12, atol=1e-12)


def test_no_adapter_is_the_plain_projection():
    rng = np.random.default_rng(0)
    a, w, la, lb = (rng.normal(size=s) for s in ((4, 3), (3, 5), (2, 2, 3), (2, 5, 2)))
    for none in (-1, 2, -(2 ** 31), 2 ** 31 - 1):
        out, _ = down_forward_lora(a, w, None, la, lb, np.full(4, none), np.ones(2))
        assert np.array_equal(out, down_f64_values(a, w, None))


def test_a_worked_value():
    # x = 2, W = 3, La = 5, Lb = 7, scale = 1/2: 2 * 3 + (1/2) (2 * 5) 7 = 41
    one = lambda v: np.array([[float(v)]])  # noqa: E731
    out, _ = down_forward_lora(one(2), one(3), None, one(5)[None], one(7)[None], np.array([0]), np.array([0.5]))
    assert out[0, 0] == 41
