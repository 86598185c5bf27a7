"""Refusals of the adapter entry points: no kernel is launched here."""
import pytest
import torch

FAKE = 0x1000000  # never dereferenced: every call below fails its argument checks first


def at(i):
    return FAKE * (i + 1)


def gate_up(lib, A=at(0), Wp=at(1), Y=at(2), M=4, K=64, N=64, La=at(3), Lb=at(4), index=at(5),
            scale=at(6), adapters=3, rank=8, ws=at(7), nbytes=1 << 20):
    return lib.swiglu_forward_lora(A, Wp, Y, M, K, N, La, Lb, index, scale, adapters, rank, ws, nbytes, None)


def down(lib, Y=at(0), Wp=at(1), R=at(8), Out=at(2), M=4, N=64, H=64, La=at(3), Lb=at(4), index=at(5),
         scale=at(6), adapters=3, rank=8, ws=at(7), nbytes=1 << 20):
    return lib.swiglu_down_forward_lora(Y, Wp, R, Out, M, N, H, La, Lb, index, scale, adapters, rank, ws,
                                        nbytes, None)


@pytest.mark.parametrize("M,K,N,rank,want", [
    (-1, 64, 64, 8, 1), (4, 0, 64, 8, 1), (4, 64, 0, 8, 1), (4, 60, 64, 8, 2), (4, 64, 12, 8, 2),
    (4, 1 << 22, 64, 8, 2), (1 << 31, 64, 64, 8, 2), (4, 64, 64, 0, 1), (4, 64, 64, -8, 1),
    (4, 64, 64, 12, 2), (4, 64, 64, 72, 2),
])
def test_bad_shapes(native_lib, M, K, N, rank, want):
    assert gate_up(native_lib.lib, M=M, K=K, N=N, rank=rank) == want
    assert down(native_lib.lib, M=M, N=K, H=N, rank=rank) == want
    assert native_lib.swiglu_lora_workspace_bytes(M, K, N, rank) == 0
    assert native_lib.swiglu_down_lora_workspace_bytes(M, K, N, rank) == 0


@pytest.mark.parametrize("change", [
    {"A": None}, {"Wp": None}, {"Y": None}, {"La": None}, {"Lb": None}, {"index": None}, {"scale": None},
    {"ws": None}, {"A": at(0) + 2}, {"Wp": at(1) + 2}, {"Y": at(2) + 2}, {"La": at(3) + 2},
    {"Lb": at(4) + 2}, {"index": at(5) + 2}, {"scale": at(6) + 2}, {"ws": at(7) + 2}, {"nbytes": 16},
    {"adapters": -1}, {"Y": at(0)}, {"Y": at(1) + 16}, {"Y": at(3)}, {"Y": at(4)}, {"Y": at(5)},
    {"Y": at(6)}, {"ws": at(0)}, {"ws": at(2)}, {"ws": at(4) - 64}, {"ws": at(5)},
])
def test_bad_arguments(native_lib, change):
    assert gate_up(native_lib.lib, **change) == native_lib.SWIGLU_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [
    {"Y": None}, {"Wp": None}, {"Out": None}, {"La": None}, {"Lb": None}, {"index": None},
    {"scale": None}, {"ws": None}, {"R": at(8) + 2}, {"R": at(2) + 16}, {"Out": at(0)}, {"Out": at(3)},
    {"ws": at(8)}, {"nbytes": 0}, {"adapters": -1},
])
def test_bad_down_arguments(native_lib, change):
    assert down(native_lib.lib, **change) == native_lib.SWIGLU_ERR_INVALID_ARG


def test_too_many_adapter_rows(native_lib):
    assert gate_up(native_lib.lib, adapters=1 << 40) == native_lib.SWIGLU_ERR_UNSUPPORTED
    assert down(native_lib.lib, adapters=1 << 40) == native_lib.SWIGLU_ERR_UNSUPPORTED


def test_no_tokens_is_a_no_op(native_lib):
    assert gate_up(native_lib.lib, A=None, Y=None, M=0, ws=None, nbytes=0) == native_lib.SWIGLU_OK
    assert down(native_lib.lib, Y=None, Out=None, M=0, ws=None, nbytes=0) == native_lib.SWIGLU_OK
    assert native_lib.swiglu_lora_workspace_bytes(0, 64, 64, 8) == 0


def test_workspace_sizes(native_lib):
    # bf16 V; above 128 tokens a list per 256 tokens too (256-byte parts)
    f, g = native_lib.swiglu_lora_workspace_bytes, native_lib.swiglu_down_lora_workspace_bytes
    assert f(16, 64, 64, 16) == 16 * 32 * 2 and g(16, 64, 64, 16) == 16 * 16 * 2
    assert f(1, 64, 64, 8) == 256
    assert f(512, 64, 64, 16) == 512 * 32 * 2 + 2 * 260 * 4


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
def test_without_a_device(native_lib):
    assert gate_up(native_lib.lib) == native_lib.SWIGLU_ERR_NO_DEVICE
    assert down(native_lib.lib) == native_lib.SWIGLU_ERR_NO_DEVICE


def test_binding_checks(native_lib):
    a = torch.zeros(4, 64, dtype=torch.bfloat16)
    la = torch.zeros(3, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        native_lib.swiglu_forward_lora(a, a, 64, la, la, torch.zeros(4, dtype=torch.int32), torch.ones(3))
    with pytest.raises(ValueError):
        native_lib.swiglu_down_forward_lora(a, a, 64, la[:, 0], la[:, 0], torch.zeros(4, dtype=torch.int32),
                                            torch.ones(3))
