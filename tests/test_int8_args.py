"""Refusals of the 8-bit projections' entry points: no kernel is launched here."""
import ctypes

import pytest
import torch

FAKE = 0x1000000  # never dereferenced: every call below fails its argument checks first


def at(i):
    return FAKE * (i + 1)


def pack(lib, W1=at(0), W2=at(1), Wp=at(2), K=64, N=64):
    return lib.swiglu_pack_weights_int8(W1, W2, Wp, K, N, None)


def pack_down(lib, W3=at(0), Wp=at(2), N=64, H=64):
    return lib.swiglu_pack_down_weights_int8(W3, Wp, N, H, None)


def forward(lib, A=at(0), sa=at(1), Wp=at(2), s1=at(3), s2=at(4), Y=at(5), M=4, K=64, N=64, ws=at(7), nbytes=1 << 16):
    return lib.swiglu_forward_int8(A, sa, Wp, s1, s2, Y, M, K, N, ws, nbytes, None)


def down(lib, Y=at(0), sy=at(1), Wp=at(2), s3=at(3), R=at(4), Out=at(5), M=4, N=64, H=64, ws=at(7), nbytes=1 << 16):
    return lib.swiglu_down_forward_int8(Y, sy, Wp, s3, R, Out, M, N, H, ws, nbytes, None)


@pytest.mark.parametrize("M,K,N,want", [(-1, 64, 64, 1), (4, 0, 64, 1), (4, 64, 0, 1), (4, 60, 64, 2),
                                        (4, 64, 12, 2), (4, 1 << 22, 64, 2), (1 << 31, 64, 64, 2)])
def test_bad_shapes(native_lib, M, K, N, want):
    lib = native_lib.lib
    assert forward(lib, M=M, K=K, N=N) == want
    assert down(lib, M=M, N=K, H=N) == want
    if 0 <= M < 1 << 31:
        assert pack(lib, K=K, N=N) == want
        assert pack_down(lib, N=K, H=N) == want
        assert native_lib.swiglu_packed_weight_bytes_int8(K, N) == native_lib.swiglu_down_packed_bytes_int8(K, N) == 0
    assert native_lib.swiglu_int8_workspace_bytes(M, K, N) == native_lib.swiglu_down_int8_workspace_bytes(M, K, N) == 0


def test_packed_sizes(native_lib):
    assert native_lib.swiglu_packed_weight_bytes_int8(16, 8) == 256 * 128
    assert native_lib.swiglu_packed_weight_bytes_int8(3584, 18944) == 2 * 3584 * 18944
    assert native_lib.swiglu_down_packed_bytes_int8(4864, 896) == 4864 * 1024


@pytest.mark.parametrize("call,change", [
    (pack, {"W1": None}), (pack, {"W2": None}), (pack, {"Wp": None}), (pack, {"W1": at(0) + 8}), (pack, {"Wp": at(1)}),
    (pack_down, {"W3": None}), (pack_down, {"Wp": at(0) + 1024}), (pack_down, {"Wp": at(2) + 4}),
    (forward, {"A": None}), (forward, {"sa": None}), (forward, {"Wp": None}), (forward, {"s1": None}),
    (forward, {"s2": None}), (forward, {"Y": None}), (forward, {"A": at(0) + 8}), (forward, {"sa": at(1) + 2}),
    (forward, {"s1": at(3) + 4}), (forward, {"Y": at(5) + 8}), (forward, {"ws": at(7) + 8}), (forward, {"Y": at(0)}),
    (forward, {"Y": at(4)}), (forward, {"ws": at(2) + 16}), (forward, {"ws": at(5)}),
    (down, {"Y": None}), (down, {"Out": None}), (down, {"s3": None}), (down, {"R": at(4) + 2}), (down, {"Out": at(4) + 16}),
    (down, {"Out": at(1)}), (down, {"Wp": at(2) + 8}),
])
def test_bad_pointers(native_lib, call, change):
    assert call(native_lib.lib, **change) == native_lib.SWIGLU_ERR_INVALID_ARG


def test_no_tokens_is_a_no_op(native_lib):
    assert forward(native_lib.lib, M=0) == down(native_lib.lib, M=0) == native_lib.SWIGLU_OK


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_without_a_device(native_lib):
    lib = native_lib.lib
    for call in (pack, pack_down, forward, down):
        assert call(lib) == native_lib.SWIGLU_ERR_NO_DEVICE
    assert down(lib, Out=at(4)) == native_lib.SWIGLU_ERR_NO_DEVICE  # in place is allowed
    assert down(lib, R=None, ws=None, nbytes=0) == native_lib.SWIGLU_ERR_NO_DEVICE


def test_plan_strings_check_their_arguments(native_lib):
    lib, buf = native_lib.lib, ctypes.create_string_buffer(64)
    for f in (lib.swiglu_plan_string_int8, lib.swiglu_down_plan_string_int8):
        assert f(16, 64, 64, None, 0) == native_lib.SWIGLU_ERR_INVALID_ARG
        assert f(16, 60, 64, buf, 64) == native_lib.SWIGLU_ERR_UNSUPPORTED
        if not torch.cuda.is_available():
            assert f(16, 64, 64, buf, 64) == native_lib.SWIGLU_ERR_NO_DEVICE


def test_binding_checks(native_lib):
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(64)
    for call in (lambda: native_lib.swiglu_pack_weights_int8(q, q), lambda: native_lib.swiglu_pack_down_weights_int8(q),
                 lambda: native_lib.swiglu_forward_int8(q, s[:4], q, 64, s, s),
                 lambda: native_lib.swiglu_down_forward_int8(q, s[:4], q, 64, s)):
        with pytest.raises(ValueError):
            call()
