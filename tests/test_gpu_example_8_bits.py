"""The example's block with its activations kept in 8 bits, and served in 8 bits (needs a GB300)."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(native_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    spec = importlib.util.spec_from_file_location("gated_mlp_example_8", os.path.join(ROOT, "examples", "gated_mlp.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_it_runs(example):
    losses, _ = example.main(["--hidden", "256", "--intermediate", "528", "--tokens", "300", "--steps", "4",
                              "--kept-bits", "8"])
    assert len(losses) == 4 and all(x == x for x in losses)


def block_args(seed, shapes):
    g = torch.Generator(device="cuda").manual_seed(seed)
    args = [(torch.randn(*s, generator=g, device="cuda") / s[0] ** 0.5).bfloat16() for s in shapes]
    args[0] = args[0] * shapes[0][0] ** 0.5
    return args, torch.randn(*shapes[0], generator=g, device="cuda").bfloat16()


def test_gradients_match_torch(example):
    # float32 autograd on the same bf16 values. A kept value is off by a uniform rounding of a step
    # (its group's largest, at most 4.5 standard deviations here, / 127): 0.0103 of one at most, for x,
    # Gate and Up; SiLU' moves by at most half of Gate's; with the bf16 roundings of the chain
    # (2^-9 each, four of them) the norm of the error stays below 0.0103 * sqrt(3) + 4 * 2^-9.
    args, d_out = block_args(2, ((200, 136), (136, 264), (136, 264), (264, 136)))
    got_args = [a.clone().requires_grad_() for a in args]
    got = torch.autograd.grad(example.GatedMLP8.apply(*got_args), got_args, d_out)
    x, w1, w2, w3 = [a.float().requires_grad_() for a in args]
    want = torch.autograd.grad(x + (torch.nn.functional.silu(x @ w1) * (x @ w2)) @ w3, (x, w1, w2, w3),
                               d_out.float())
    for a, b in zip(got, want):
        assert ((a.float() - b).norm() / b.norm()).item() < 0.026


@pytest.mark.parametrize("trained", range(1, 16))
def test_each_choice_of_trained_tensors(example, trained):
    # those that are trained get the gradient that they get when all are, the others none
    args, d_out = block_args(3, ((40, 64), (64, 136), (64, 136), (136, 64)))
    every = [a.clone().requires_grad_() for a in args]
    some = [a.clone().requires_grad_(bool(trained >> i & 1)) for i, a in enumerate(args)]
    for a in (every, some):
        example.GatedMLP8.apply(*a).backward(d_out)
    for i in range(4):
        assert torch.equal(some[i].grad, every[i].grad) if trained >> i & 1 else some[i].grad is None


def test_served_in_8_bits(example):
    # x, the weights and Y each off by at most 4.5 / 127 / sqrt(12) = 0.0103 of a standard deviation
    # (Y, a product, has longer tails: a largest of at most 20 of them, 0.046), and x itself in Out
    args, _ = block_args(4, ((24, 256), (256, 528), (256, 528), (528, 256)))
    out, want = example.serve_8_bits(*args[1:])
    assert out.shape == want.shape == (24, 256)
    assert ((out.float() - want.float()).norm() / want.float().norm()).item() < 0.06
