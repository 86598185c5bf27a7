"""Which gradients the example's block returns, with the library's calls replaced by torch's."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def example(monkeypatch):
    spec = importlib.util.spec_from_file_location("gated_mlp_block", os.path.join(ROOT, "examples", "gated_mlp.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)

    class Library:
        """The entry points that the block calls, on the CPU; a packed weight is a copy."""

        @staticmethod
        def swiglu_pack_weights(w1, w2):
            return torch.stack([w1, w2]).detach().clone()

        @staticmethod
        def swiglu_pack_down_weights(w3):
            return w3.detach().clone()

        @staticmethod
        def swiglu_forward(x, wp, n):
            return torch.nn.functional.silu(x @ wp[0]) * (x @ wp[1])

        @staticmethod
        def swiglu_down_forward(y, w3p, h, R):
            return y @ w3p + R

        @staticmethod
        def swiglu_backward(x, wp, dy, need_input=True, need_weight=True):
            g, u = x @ wp[0], x @ wp[1]
            s = torch.sigmoid(g)
            du, dg = dy * g * s, dy * u * (s + g * s * (1 - s))
            return (dg @ wp[0].t() + du @ wp[1].t() if need_input else None,
                    x.t() @ dg if need_weight else None, x.t() @ du if need_weight else None)

        @staticmethod
        def swiglu_down_backward(d_out, w3p, y, need_input=True, need_weight=True):
            return d_out @ w3p.t() if need_input else None, y.t() @ d_out if need_weight else None

    monkeypatch.setattr(module, "sg", Library)
    return module


@pytest.mark.parametrize("trained", range(1, 16))
def test_each_choice_of_trained_tensors(example, trained):
    # x, w1, w2, w3: those that are trained get torch's own gradient, the others none
    g = torch.Generator().manual_seed(5)
    shapes = ((6, 8), (8, 12), (8, 12), (12, 8))
    values = [torch.randn(*s, generator=g, dtype=torch.float64) for s in shapes]
    d_out = torch.randn(6, 8, generator=g, dtype=torch.float64)
    grads = []
    for block in (example.GatedMLP.apply,
                  lambda x, w1, w2, w3: x + (torch.nn.functional.silu(x @ w1) * (x @ w2)) @ w3):
        args = [v.clone().requires_grad_(bool(trained >> i & 1)) for i, v in enumerate(values)]
        block(*args).backward(d_out)
        grads.append([a.grad for a in args])
    for i, (got, want) in enumerate(zip(*grads)):
        assert (got is None) == (want is None), i
        if want is not None:
            assert torch.allclose(got, want, rtol=1e-12, atol=1e-12), i
