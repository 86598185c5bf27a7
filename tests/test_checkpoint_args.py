"""Refusals of the 8-bit checkpoint's entry points: no kernel is launched here."""
import pytest
import torch

FAKE = 0x1000000  # never dereferenced: every call below fails its argument checks first


def at(i):
    return FAKE * (i + 1)


def quantise(lib, X=at(0), Q=at(1), scale=at(2), M=4, K=64):
    return lib.swiglu_quantize_int8(X, Q, scale, M, K, None)


def forward(lib, A=at(0), Wp=at(1), Y=at(2), gate=at(3), up=at(4), scale=at(5), M=4, K=64, N=64):
    return lib.swiglu_forward_checkpoint(A, Wp, Y, gate, up, scale, M, K, N, None)


def output(lib, gate=at(0), up=at(1), scale=at(2), Y=at(3), M=4, N=64):
    return lib.swiglu_checkpoint_output(gate, up, scale, Y, M, N, None)


def backward(lib, A=at(0), sa=at(10), Wp=at(1), dY=at(2), gate=at(3), up=at(4), scale=at(5), dA=at(6), dW1=at(7),
             dW2=at(8), M=4, K=64, N=64, ws=at(9), nbytes=1 << 20):
    return lib.swiglu_backward_checkpoint(A, sa, Wp, dY, gate, up, scale, dA, dW1, dW2, M, K, N, ws, nbytes, None)


@pytest.mark.parametrize("M,K,N,want", [(-1, 64, 64, 1), (4, 0, 64, 1), (4, 64, 0, 1), (4, 60, 64, 2),
                                        (4, 64, 12, 2), (4, 1 << 22, 64, 2), (1 << 31, 64, 64, 2)])
def test_bad_shapes(native_lib, M, K, N, want):
    lib = native_lib.lib
    assert forward(lib, M=M, K=K, N=N) == want
    assert backward(lib, M=M, K=K, N=N) == want
    if K != 64 or M in (-1, 1 << 31):
        assert quantise(lib, M=M, K=K) == want
    if N != 64 or M in (-1, 1 << 31):
        assert output(lib, M=M, N=N) == want
    assert native_lib.swiglu_backward_checkpoint_workspace_bytes(M, K, N) == 0


@pytest.mark.parametrize("call,change", [
    (quantise, {"X": None}), (quantise, {"Q": None}), (quantise, {"scale": None}), (quantise, {"X": at(0) + 2}),
    (quantise, {"Q": at(1) + 8}), (quantise, {"scale": at(2) + 2}), (quantise, {"Q": at(0) + 64}),
    (quantise, {"scale": at(1)}),
    (forward, {"A": None}), (forward, {"Wp": None}), (forward, {"Y": None}), (forward, {"gate": None}),
    (forward, {"up": None}), (forward, {"scale": None}), (forward, {"gate": at(3) + 8}), (forward, {"up": at(3)}),
    (forward, {"scale": at(0)}), (forward, {"Y": at(1) + 16}), (forward, {"scale": at(4) + 240}),
    (output, {"gate": None}), (output, {"scale": None}), (output, {"Y": None}), (output, {"Y": at(1)}),
    (output, {"Y": at(3) + 2}), (output, {"up": at(1) + 8}),
    (backward, {"A": None}), (backward, {"Wp": None}), (backward, {"dY": None}), (backward, {"gate": None}),
    (backward, {"up": None}), (backward, {"scale": None}), (backward, {"ws": None}), (backward, {"dW1": None}),
    (backward, {"dW2": None}), (backward, {"sa": at(10) + 2}), (backward, {"A": at(0) + 8}),
    (backward, {"dA": at(0)}), (backward, {"dA": at(3)}), (backward, {"dW1": at(10)}), (backward, {"ws": at(5)}),
    (backward, {"dW2": at(7) + 16}), (backward, {"ws": at(9) + 8}),
])
def test_bad_pointers(native_lib, call, change):
    assert call(native_lib.lib, **change) == native_lib.SWIGLU_ERR_INVALID_ARG


def test_no_ops(native_lib):
    lib = native_lib.lib
    assert backward(lib, dA=None, dW1=None, dW2=None) == native_lib.SWIGLU_OK
    assert backward(lib, M=0, dW1=None, dW2=None) == native_lib.SWIGLU_OK
    for call in (quantise, forward, output):
        assert call(lib, M=0) == native_lib.SWIGLU_OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_without_a_device(native_lib):
    lib = native_lib.lib
    for call in (quantise, forward, output, backward):
        assert call(lib) == native_lib.SWIGLU_ERR_NO_DEVICE
    # what is not asked for needs nothing
    assert backward(lib, dA=None, Wp=None) == native_lib.SWIGLU_ERR_NO_DEVICE
    assert backward(lib, dW1=None, dW2=None, A=None, sa=None) == native_lib.SWIGLU_ERR_NO_DEVICE


def test_binding_checks(native_lib):
    a = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(2, 1, 4)
    with pytest.raises(ValueError):
        native_lib.swiglu_quantize_int8(a)
    with pytest.raises(ValueError):
        native_lib.swiglu_forward_checkpoint(a, a, 64)
    with pytest.raises(ValueError):
        native_lib.swiglu_checkpoint_output(q, q, s)
    with pytest.raises(ValueError):
        native_lib.swiglu_backward_checkpoint(a, a, a, q, q, s)
