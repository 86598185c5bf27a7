"""Relative norms of the errors of the gradients and adapters, beside the elementwise bounds (needs a GB300).

A worst-case bound on one element of a sum of thousands of terms is as large as
several of them, so a lost piece of a sum can stay inside it. Errors of rounding
are independent from element to element, so their norm is known much better.

Rounding x to bf16 moves it by a uniform error of at most 2^(e - 8) where
2^e <= |x| < 2^(e + 1): its root mean square is at most EPS |x| with
EPS = 2^-8 / sqrt(3). Through a sum of products variances add:
  dA   EPS^2 (dG^2 (W1^2)^T + dU^2 (W2^2)^T)   from the rounded dG and dU
  dW1  EPS^2 (A^2)^T dG^2                      (dW2 with dU)
  Gate EPS^2 V1^2 (Lb1^2)^T                    from the rounded V (Up with V2)
and every output's own rounding adds EPS^2 of its square. What is left (fp32 sums
of 2^-23 a term, the exponential's 2^-16) is under a hundredth of that; a
twentieth more is allowed for it and for the sample.
"""
import pytest
import torch

from swiglu_gated_mlp_gb300.workloads import make_inputs

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -8 / 3 ** 0.5
MARGIN = 1.05


@pytest.fixture(scope="module")
def native(native_lib):
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    return native_lib


def allowed(ref, variance=0.0):
    """The norm that the error of `ref` may have; `variance`: that of the rounded operands, over EPS^2."""
    return MARGIN * EPS * (variance + ref.square()).sum().sqrt().item()


def check(out, ref, variance=0.0):
    error, limit = (out.double() - ref).norm().item(), allowed(ref, variance)
    assert error <= limit, (error / ref.norm().item(), limit / ref.norm().item())


def silu_and_slope(g):
    s = torch.sigmoid(g)
    return g * s, s * (1 + g * (1 - s))


@pytest.mark.parametrize("M,K,N", [(128, 896, 4864), (1000, 1416, 5000), (4096, 3584, 18944)])
def test_backward_error_norms(native, M, K, N):
    a, w1, w2 = (t.cuda() for t in make_inputs(M, K, N, 21))
    dy = make_inputs(M, N, 8, 22)[0].cuda()
    da, dw1, dw2 = native.swiglu_backward(a, native.swiglu_pack_weights(w1, w2), dy)
    native.swiglu_check_device_status()
    x, p, q, d = (t.double() for t in (a, w1, w2, dy))
    u = x @ q
    silu, slope = silu_and_slope(x @ p)
    dg, du = d * u * slope, d * silu
    del u, silu, slope, d
    check(da, dg @ p.t() + du @ q.t(), dg.square() @ p.square().t() + du.square() @ q.square().t())
    for got, grad in ((dw1, dg), (dw2, du)):
        ref, variance = x.t() @ grad, x.square().t() @ grad.square()
        check(got, ref, variance)
        # what 16 tokens add would be missed by far
        assert (x[:16].t() @ grad[:16]).norm().item() > 10 * allowed(ref, variance)


@pytest.mark.parametrize("M,N,H", [(128, 4864, 896), (1000, 5000, 1416), (4096, 18944, 3584)])
def test_down_backward_error_norms(native, M, N, H):
    y, w3, _ = (t.cuda() for t in make_inputs(M, N, H, 23))
    dout = make_inputs(M, H, 8, 24)[0].cuda()
    dy, dw3 = native.swiglu_down_backward(dout, native.swiglu_pack_down_weights(w3), y)
    native.swiglu_check_device_status()
    d, w, x = (t.double() for t in (dout, w3, y))
    check(dy, d @ w.t())
    ref = x.t() @ d
    check(dw3, ref)
    assert (x[:16].t() @ d[:16]).norm().item() > 10 * allowed(ref)


def adapted(x, w, la, lb, index, scale):
    """x W + each token's adapter, and the variance that rounding V adds, over EPS^2."""
    out, variance = x @ w, torch.zeros(x.shape[0], w.shape[1], dtype=x.dtype, device=x.device)
    for i in range(la.shape[0]):
        rows = (index == i).nonzero().reshape(-1)
        v = scale[i] * (x[rows] @ la[i].t())
        out[rows] += v @ lb[i].t()
        variance[rows] = v.square() @ lb[i].square().t()
    return out, variance


def table(L, halves, r, K, N, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (L, 2) if halves == 2 else (L,)
    la = (torch.randn(*shape, r, K, generator=g, device="cuda") / K ** 0.5).bfloat16()
    lb = (torch.randn(*shape, N, r, generator=g, device="cuda") / r ** 0.5).bfloat16()
    return la, lb, 0.5 + torch.rand(L, generator=g, device="cuda")


LORA = [(16, 3584, 18944, 8, 16), (128, 896, 4864, 32, 16), (333, 1416, 5000, 5, 24), (4096, 3584, 18944, 8, 64)]


@pytest.mark.parametrize("M,K,N,L,r", LORA)
def test_forward_lora_error_norms(native, M, K, N, L, r):
    a, w1, w2 = (t.cuda() for t in make_inputs(M, K, N, 25))
    la, lb, scale = table(L, 2, r, K, N, 25)
    index = (torch.arange(M, device="cuda") * (L + 1) // M - 1).int()  # runs of tokens, the first without
    y = native.swiglu_forward_lora(a, native.swiglu_pack_weights(w1, w2), N, la, lb, index, scale)
    native.swiglu_check_device_status()
    x, p, q, s = (t.double() for t in (a, w1, w2, scale))
    g, vg = adapted(x, p, la[:, 0].double(), lb[:, 0].double(), index, s)
    u, vu = adapted(x, q, la[:, 1].double(), lb[:, 1].double(), index, s)
    silu, slope = silu_and_slope(g)
    check(y, silu * u, (slope * u).square() * vg + silu.square() * vu)


@pytest.mark.parametrize("M,H,N,L,r", LORA)
def test_down_forward_lora_error_norms(native, M, H, N, L, r):
    y, w3, _ = (t.cuda() for t in make_inputs(M, N, H, 26))
    res = make_inputs(M, H, 8, 27)[0].cuda()
    la, lb, scale = table(L, 1, r, N, H, 26)
    index = (torch.arange(M, device="cuda") * (L + 1) // M - 1).int()
    out = native.swiglu_down_forward_lora(y, native.swiglu_pack_down_weights(w3), H, la, lb, index, scale, R=res)
    native.swiglu_check_device_status()
    ref, variance = adapted(y.double(), w3.double(), la.double(), lb.double(), index, scale.double())
    check(out, ref + res.double(), variance)


@pytest.mark.parametrize("M,K,N,L,r,kernel", [
    (4096, 8192, 8192, 6, 64, "large_m_pair"),  # 14 rounds of tiles
    (1300, 8192, 520, 3, 16, "large_m_pair"),   # one, beside the kernel that makes V
    (300, 8192, 1032, 3, 16, "small_m"),
])
def test_adapters_of_a_long_hidden_size(native, M, K, N, L, r, kernel):
    # K >= 8192: the CTA pairs keep their rounds of tiles together and walk every second one backwards
    assert kernel in native.swiglu_lora_plan_string(M, K, N, r)
    for _ in range(2):  # the launch numbers of a second call
        test_forward_lora_error_norms(native, M, K, N, L, r)


def test_backward_of_a_long_hidden_size(native):
    test_backward_error_norms(native, 1024, 8192, 4096)
