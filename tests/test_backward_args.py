"""Refusals of the gradient entry points: no kernel is launched here."""
import pytest
import torch

FAKE = 0x1000000  # never dereferenced: every call below fails its argument checks first


def at(i):
    return FAKE * (i + 1)


def backward(lib, A=at(0), Wp=at(1), dY=at(2), dA=at(3), dW1=at(4), dW2=at(5), M=4, K=64, N=64,
             ws=at(6), nbytes=1 << 20):
    return lib.swiglu_backward(A, Wp, dY, dA, dW1, dW2, M, K, N, ws, nbytes, None)


def down(lib, dOut=at(0), Wp=at(1), Y=at(2), dY=at(3), dW3=at(4), M=4, N=64, H=64, ws=at(6),
         nbytes=1 << 20):
    return lib.swiglu_down_backward(dOut, Wp, Y, dY, dW3, M, N, H, ws, nbytes, None)


@pytest.mark.parametrize("M,K,N,want", [(-1, 64, 64, 1), (4, 0, 64, 1), (4, 64, 0, 1), (4, 60, 64, 2),
                                        (4, 64, 12, 2), (4, 1 << 22, 64, 2), (1 << 31, 64, 64, 2)])
def test_bad_shapes(native_lib, M, K, N, want):
    assert backward(native_lib.lib, M=M, K=K, N=N) == want
    assert down(native_lib.lib, M=M, N=K, H=N) == want
    assert native_lib.swiglu_backward_workspace_bytes(M, K, N) == 0
    assert native_lib.swiglu_down_backward_workspace_bytes(M, K, N) == 0


@pytest.mark.parametrize("change", [
    {"A": None}, {"Wp": None}, {"dY": None}, {"dW1": None}, {"dW2": None}, {"ws": None},
    {"A": at(0) + 2}, {"Wp": at(1) + 8}, {"dY": at(2) + 4}, {"dA": at(3) + 2}, {"dW1": at(4) + 2},
    {"dW2": at(5) + 2}, {"ws": at(6) + 8},
    {"dA": at(0)}, {"dA": at(1) + 16}, {"dW1": at(2)}, {"dW2": at(4)}, {"dA": at(5)}, {"ws": at(2) - 64},
    {"ws": at(3)},
])
def test_bad_pointers(native_lib, change):
    assert backward(native_lib.lib, **change) == native_lib.SWIGLU_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    {"dOut": None}, {"Wp": None}, {"Y": None}, {"dOut": at(0) + 2}, {"Wp": at(1) + 2}, {"Y": at(2) + 2},
    {"dY": at(3) + 2}, {"dW3": at(4) + 2}, {"ws": at(6) + 2}, {"dY": at(0)}, {"dW3": at(1)},
    {"dY": at(4)}, {"ws": at(2)},
])
def test_bad_down_pointers(native_lib, change):
    assert down(native_lib.lib, **change) == native_lib.SWIGLU_ERR_INVALID_ARG


def test_nothing_asked_for_is_a_no_op(native_lib):
    assert backward(native_lib.lib, dA=None, dW1=None, dW2=None) == native_lib.SWIGLU_OK
    assert down(native_lib.lib, dY=None, dW3=None) == native_lib.SWIGLU_OK
    # no tokens and no weight gradient: nothing to write
    assert backward(native_lib.lib, M=0, dW1=None, dW2=None) == native_lib.SWIGLU_OK
    assert down(native_lib.lib, M=0, dW3=None) == native_lib.SWIGLU_OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_without_a_device(native_lib):
    assert backward(native_lib.lib) == native_lib.SWIGLU_ERR_NO_DEVICE
    assert down(native_lib.lib) == native_lib.SWIGLU_ERR_NO_DEVICE
    assert backward(native_lib.lib, M=0) == native_lib.SWIGLU_ERR_NO_DEVICE


def test_binding_checks(native_lib):
    a = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        native_lib.swiglu_backward(a, a, a)
    with pytest.raises(ValueError):
        native_lib.swiglu_down_backward(a, a, a)


def test_plan_strings_check_their_arguments(native_lib):
    import ctypes
    lib, buf = native_lib.lib, ctypes.create_string_buffer(64)
    for f in (lib.swiglu_backward_plan_string, lib.swiglu_down_backward_plan_string):
        assert f(16, 64, 64, None, 0) == native_lib.SWIGLU_ERR_INVALID_ARG
        assert f(16, 60, 64, buf, 64) == native_lib.SWIGLU_ERR_UNSUPPORTED
        if not torch.cuda.is_available():
            assert f(16, 64, 64, buf, 64) == native_lib.SWIGLU_ERR_NO_DEVICE
    for f in (lib.swiglu_lora_plan_string, lib.swiglu_down_lora_plan_string):
        assert f(16, 64, 64, 8, None, 0) == native_lib.SWIGLU_ERR_INVALID_ARG
        assert f(16, 60, 64, 8, buf, 64) == native_lib.SWIGLU_ERR_UNSUPPORTED
        assert f(16, 64, 64, 12, buf, 64) == native_lib.SWIGLU_ERR_UNSUPPORTED
        if not torch.cuda.is_available():
            assert f(16, 64, 64, 8, buf, 64) == native_lib.SWIGLU_ERR_NO_DEVICE
