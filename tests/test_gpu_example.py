"""The example trains and serves through the gradients and adapters (needs a GB300)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(native_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    spec = importlib.util.spec_from_file_location("gated_mlp_example", os.path.join(ROOT, "examples", "gated_mlp.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_example_trains_and_serves(example):
    losses, off = example.main(["--hidden", "256", "--intermediate", "520", "--tokens", "300", "--steps", "40"])
    # Adam on a convex-near-the-teacher fit: the loss has to fall well below its start
    assert losses[-1] < 0.5 * losses[0]
    # Y and Out are rounded to bf16 (2^-8 each at most) and V enters as bf16
    assert off < 3 * 2.0 ** -8


def test_autograd_gradients_match_torch(example):
    # the whole block's gradients against float32 autograd on the same bf16 values; the chain
    # rounds Y, dY, dG, dU and the output to bf16 once each, 2^-8 at most, 2^-9 typical
    g = torch.Generator(device="cuda").manual_seed(2)
    shapes = ((200, 136), (136, 264), (136, 264), (264, 136))
    args = [(torch.randn(*s, generator=g, device="cuda") / s[0] ** 0.5).bfloat16() for s in shapes]
    args[0] = args[0] * 14
    d_out = torch.randn(200, 136, generator=g, device="cuda").bfloat16()
    got_args = [a.clone().requires_grad_() for a in args]
    got = torch.autograd.grad(example.GatedMLP.apply(*got_args), got_args, d_out)
    x, w1, w2, w3 = [a.float().requires_grad_() for a in args]
    want = torch.autograd.grad(x + (torch.nn.functional.silu(x @ w1) * (x @ w2)) @ w3, (x, w1, w2, w3),
                               d_out.float())
    for a, b in zip(got, want):
        assert ((a.float() - b).norm() / b.norm()).item() < 5 * 2.0 ** -9


def test_frozen_weights_need_no_weight_gradients(example):
    g = torch.Generator(device="cuda").manual_seed(3)
    w = [(torch.randn(*s, generator=g, device="cuda") / 8).bfloat16() for s in ((64, 128), (64, 128), (128, 64))]
    x = torch.randn(5, 64, generator=g, device="cuda").bfloat16().requires_grad_()
    example.GatedMLP.apply(x, *w).float().sum().backward()
    assert x.grad is not None and x.grad.isfinite().all()


@pytest.mark.parametrize("frozen", [1, 2])
def test_one_of_the_two_first_weights_frozen(example, frozen):
    # the other one's gradient is the one that it gets when both are trained
    g = torch.Generator(device="cuda").manual_seed(4)
    shapes = ((40, 64), (64, 136), (64, 136), (136, 64))
    values = [(torch.randn(*s, generator=g, device="cuda") / 8).bfloat16() for s in shapes]
    d_out = torch.randn(40, 64, generator=g, device="cuda").bfloat16()
    both = [v.clone().requires_grad_() for v in values]
    one = [v.clone().requires_grad_(i != frozen) for i, v in enumerate(values)]
    for args in (both, one):
        example.GatedMLP.apply(*args).backward(d_out)
    for i in range(4):
        assert one[i].grad is None if i == frozen else torch.equal(one[i].grad, both[i].grad)
