"""Thin ctypes binding of libswiglu (include/swiglu.h), with the same names.

Argument marshalling only: every step of the computation runs in the library's
CUDA kernels. PyTorch supplies device memory and the current stream. There is
no fallback: if the library is not built, importing this module raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

from .build import LIB_PATH

SWIGLU_OK = 0
SWIGLU_ERR_INVALID_ARG = 1
SWIGLU_ERR_UNSUPPORTED = 2
SWIGLU_ERR_CUDA = 3
SWIGLU_ERR_TIMEOUT = 4
SWIGLU_ERR_NO_DEVICE = 5

SWIGLU_VARIANT_AUTO = 0
SWIGLU_VARIANT_LARGE_M = 1
SWIGLU_VARIANT_SMALL_M = 2
SWIGLU_VARIANT_LARGE_M_PAIR = 3
SWIGLU_VARIANT_SEQUENTIAL = 4
SWIGLU_VARIANT_SPLIT_K = 5
SWIGLU_VARIANT_RESIDENT_PAIR = 6

PACK_BLOCK_N = 128

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is not built; run `python -m swiglu_gated_mlp_gb300.build` "
        "(or __graft_entry__.build()) first")

lib = ctypes.CDLL(LIB_PATH)

_i64, _vp, _sz, _int, _u32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_uint32
lib.swiglu_packed_weight_bytes.argtypes = [_i64, _i64]
lib.swiglu_packed_weight_bytes.restype = _sz
lib.swiglu_pack_weights.argtypes = [_vp, _vp, _vp, _i64, _i64, _vp]
lib.swiglu_pack_weights.restype = _int
lib.swiglu_forward.argtypes = [_vp, _vp, _vp, _i64, _i64, _i64, _vp]
lib.swiglu_forward.restype = _int
lib.swiglu_forward_variant.argtypes = [_vp, _vp, _vp, _i64, _i64, _i64, _int, _vp]
lib.swiglu_forward_variant.restype = _int
lib.swiglu_forward_from_host.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp]
lib.swiglu_forward_from_host.restype = _int
lib.swiglu_check_device_status.argtypes = [_vp]
lib.swiglu_check_device_status.restype = _int
lib.swiglu_status_string.argtypes = [_int]
lib.swiglu_status_string.restype = ctypes.c_char_p
lib.swiglu_plan_string.argtypes = [_i64, _i64, _i64, _int, ctypes.c_char_p, _sz]
lib.swiglu_plan_string.restype = _int
lib.swiglu_packed_weight_bytes_fp8.argtypes = [_i64, _i64]
lib.swiglu_packed_weight_bytes_fp8.restype = _sz
lib.swiglu_pack_weights_fp8.argtypes = [_vp, _vp, _vp, _i64, _i64, _vp]
lib.swiglu_pack_weights_fp8.restype = _int
lib.swiglu_forward_fp8.argtypes = [_vp, _vp, _vp, _i64, _i64, _i64, ctypes.c_float, ctypes.c_float,
                                   ctypes.c_float, _vp]
lib.swiglu_forward_fp8.restype = _int
lib.swiglu_down_packed_bytes.argtypes = [_i64, _i64]
lib.swiglu_down_packed_bytes.restype = _sz
lib.swiglu_pack_down_weights.argtypes = [_vp, _vp, _i64, _i64, _vp]
lib.swiglu_pack_down_weights.restype = _int
lib.swiglu_down_forward.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp]
lib.swiglu_down_forward.restype = _int
lib.swiglu_down_plan_string.argtypes = [_i64, _i64, _i64, ctypes.c_char_p, _sz]
lib.swiglu_down_plan_string.restype = _int
lib.swiglu_down_workspace_bytes.argtypes = [_i64, _i64, _i64]
lib.swiglu_down_workspace_bytes.restype = _sz
lib.swiglu_down_forward_ws.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp]
lib.swiglu_down_forward_ws.restype = _int
lib.swiglu_down_plan_string_ws.argtypes = [_i64, _i64, _i64, ctypes.c_char_p, _sz]
lib.swiglu_down_plan_string_ws.restype = _int
lib.swiglu_plan_string_fp8.argtypes = [_i64, _i64, _i64, ctypes.c_char_p, _sz]
lib.swiglu_plan_string_fp8.restype = _int
lib.swiglu_packed_weight_bytes_mxfp8.argtypes = [_i64, _i64]
lib.swiglu_packed_weight_bytes_mxfp8.restype = _sz
lib.swiglu_pack_weights_mxfp8.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _vp]
lib.swiglu_pack_weights_mxfp8.restype = _int
lib.swiglu_act_scale_bytes_mxfp8.argtypes = [_i64, _i64]
lib.swiglu_act_scale_bytes_mxfp8.restype = _sz
lib.swiglu_pack_act_scales_mxfp8.argtypes = [_vp, _vp, _i64, _i64, _vp]
lib.swiglu_pack_act_scales_mxfp8.restype = _int
lib.swiglu_forward_mxfp8.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp]
lib.swiglu_forward_mxfp8.restype = _int
lib.swiglu_plan_string_mxfp8.argtypes = [_i64, _i64, _i64, ctypes.c_char_p, _sz]
lib.swiglu_plan_string_mxfp8.restype = _int
lib.swiglu_forward_noalloc.argtypes = [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp]
lib.swiglu_forward_noalloc.restype = _int
lib.swiglu_backward_workspace_bytes.argtypes = [_i64, _i64, _i64]
lib.swiglu_backward_workspace_bytes.restype = _sz
lib.swiglu_backward.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp]
lib.swiglu_backward.restype = _int
lib.swiglu_down_backward_workspace_bytes.argtypes = [_i64, _i64, _i64]
lib.swiglu_down_backward_workspace_bytes.restype = _sz
lib.swiglu_down_backward.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _sz, _vp]
lib.swiglu_down_backward.restype = _int
lib.swiglu_lora_workspace_bytes.argtypes = [_i64, _i64, _i64, _i64]
lib.swiglu_lora_workspace_bytes.restype = _sz
lib.swiglu_forward_lora.argtypes = [_vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _i64, _i64, _vp,
                                    _sz, _vp]
lib.swiglu_forward_lora.restype = _int
lib.swiglu_down_lora_workspace_bytes.argtypes = [_i64, _i64, _i64, _i64]
lib.swiglu_down_lora_workspace_bytes.restype = _sz
lib.swiglu_down_forward_lora.argtypes = [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _i64,
                                         _i64, _vp, _sz, _vp]
lib.swiglu_down_forward_lora.restype = _int
for _f in (lib.swiglu_backward_plan_string, lib.swiglu_down_backward_plan_string):
    _f.argtypes, _f.restype = [_i64, _i64, _i64, ctypes.c_char_p, _sz], _int
for _f in (lib.swiglu_lora_plan_string, lib.swiglu_down_lora_plan_string):
    _f.argtypes, _f.restype = [_i64, _i64, _i64, _i64, ctypes.c_char_p, _sz], _int
lib.swiglu_testing_inject_stall.argtypes = [_int, _u32]
lib.swiglu_testing_inject_stall.restype = None
lib.swiglu_testing_pace_run_out.argtypes = [ctypes.POINTER(ctypes.c_uint64)]
lib.swiglu_testing_pace_run_out.restype = _int


class SwigluError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {swiglu_status_string(code)}")


def _check(code: int, where: str) -> None:
    if code != SWIGLU_OK:
        raise SwigluError(code, where)


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_handle(stream, device) -> int:
    if stream is None:
        if _raw_stream is not None:  # the current stream's handle without a Stream object
            return _raw_stream(device.index if device.index is not None
                               else torch.cuda.current_device())
        stream = torch.cuda.current_stream(device)
    return int(stream.cuda_stream) if isinstance(stream, torch.cuda.Stream) else int(stream)


class _on_device:
    """Makes `device` current for the library call (a no-op when it already is)."""
    __slots__ = ("idx", "prev")

    def __init__(self, device):
        self.idx = device.index if device.index is not None else torch.cuda.current_device()

    def __enter__(self):
        self.prev = torch.cuda.current_device()
        if self.prev != self.idx:
            torch.cuda.set_device(self.idx)

    def __exit__(self, *exc):
        if self.prev != self.idx:
            torch.cuda.set_device(self.prev)
        return False


def _new_tensor(shape, dtype, device, stream=None, returned=True) -> torch.Tensor:
    """An uninitialised tensor for a call that runs on `stream` (None: the current one).

    The allocator hands a freed block out again in the order of one stream. So the
    memory of a tensor that another stream than the current one will write comes from
    that stream's blocks: one of the current stream's could still be in use by work
    queued there. A returned tensor that its owner frees is kept until the current
    stream is done with it too.
    """
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    index = device if isinstance(device, int) else device.index
    handle = int(stream.cuda_stream) if isinstance(stream, torch.cuda.Stream) else int(stream)
    if (0 if handle == 1 else handle) == _stream_handle(None, torch.device("cuda", index)):
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):  # 0 and 1 both name the default stream
        stream = (torch.cuda.ExternalStream(handle, device=index) if handle > 1
                  else torch.cuda.default_stream(index))
    with _on_device(torch.device("cuda", index)):
        current = torch.cuda.current_stream(index)
        torch.cuda.set_stream(stream)
        try:
            t = torch.empty(shape, dtype=dtype, device=device)
        finally:
            torch.cuda.set_stream(current)
    if returned:
        t.record_stream(current)
    return t


def _dev_bf16(t: torch.Tensor, name: str) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def padded_n(n: int) -> int:
    return -(-int(n) // PACK_BLOCK_N) * PACK_BLOCK_N


def swiglu_status_string(code: int) -> str:
    return lib.swiglu_status_string(int(code)).decode()


def swiglu_packed_weight_bytes(K: int, N: int) -> int:
    return int(lib.swiglu_packed_weight_bytes(int(K), int(N)))


def swiglu_pack_weights(W1: torch.Tensor, W2: torch.Tensor, Wpacked: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """Packed gate/up weight (flat bf16 buffer) from W1, W2 [K, N] (bf16, CUDA)."""
    _dev_bf16(W1, "W1")
    _dev_bf16(W2, "W2")
    if W1.dim() != 2 or W1.shape != W2.shape:
        raise ValueError("W1 and W2 must both be [K, N]")
    K, N = W1.shape
    if Wpacked is None:  # opaque buffer of swiglu_packed_weight_bytes(K, N) bytes
        Wpacked = _new_tensor(swiglu_packed_weight_bytes(K, N) // 2, torch.bfloat16, W1.device, stream)
    _dev_bf16(Wpacked, "Wpacked")
    if Wpacked.numel() * 2 < swiglu_packed_weight_bytes(K, N):
        raise ValueError("Wpacked is too small")
    with _on_device(W1.device):
        _check(lib.swiglu_pack_weights(W1.data_ptr(), W2.data_ptr(), Wpacked.data_ptr(), K, N,
                                       _stream_handle(stream, W1.device)), "swiglu_pack_weights")
    return Wpacked


def swiglu_forward_variant(A: torch.Tensor, Wpacked: torch.Tensor, N: int, variant: int,
                           Y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    _dev_bf16(A, "A")
    _dev_bf16(Wpacked, "Wpacked")
    if A.dim() != 2:
        raise ValueError("A must be [M, K]")
    M, K = A.shape
    if Wpacked.numel() * 2 < swiglu_packed_weight_bytes(K, N):
        raise ValueError("Wpacked does not hold a packed weight for this K and N")
    if Y is None:
        Y = _new_tensor((M, N), torch.bfloat16, A.device, stream)
    _dev_bf16(Y, "Y")
    if tuple(Y.shape) != (M, N):
        raise ValueError("Y must be [M, N]")
    with _on_device(A.device):
        _check(lib.swiglu_forward_variant(A.data_ptr(), Wpacked.data_ptr(), Y.data_ptr(), M, K, N,
                                          int(variant), _stream_handle(stream, A.device)),
               "swiglu_forward")
    return Y


def swiglu_forward(A: torch.Tensor, Wpacked: torch.Tensor, N: int, Y: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """Y [M, N] = SiLU(A W1) * (A W2) from A [M, K] and the packed weight."""
    return swiglu_forward_variant(A, Wpacked, N, SWIGLU_VARIANT_AUTO, Y=Y, stream=stream)


def pack(W1: torch.Tensor, W2: torch.Tensor) -> torch.Tensor:
    """Short name of swiglu_pack_weights: the packed gate/up weight Wp from W1, W2 [K, N]."""
    return swiglu_pack_weights(W1, W2)


def forward(A: torch.Tensor, Wp: torch.Tensor, N: int) -> torch.Tensor:
    """Short name of swiglu_forward: Y [M, N] = SiLU(A W1) * (A W2) on the current stream."""
    return swiglu_forward(A, Wp, N)


def _dev_fp8(t: torch.Tensor, name: str) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.float8_e4m3fn:
        raise ValueError(f"{name} must be float8_e4m3fn, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def swiglu_packed_weight_bytes_fp8(K: int, N: int) -> int:
    return int(lib.swiglu_packed_weight_bytes_fp8(int(K), int(N)))


def swiglu_pack_weights_fp8(W1: torch.Tensor, W2: torch.Tensor, Wpacked: torch.Tensor | None = None,
                            stream=None) -> torch.Tensor:
    """Packed FP8 gate/up weight (flat uint8 buffer) from E4M3 W1, W2 [K, N] (CUDA)."""
    _dev_fp8(W1, "W1")
    _dev_fp8(W2, "W2")
    if W1.dim() != 2 or W1.shape != W2.shape:
        raise ValueError("W1 and W2 must both be [K, N]")
    K, N = W1.shape
    if Wpacked is None:
        Wpacked = _new_tensor(swiglu_packed_weight_bytes_fp8(K, N), torch.uint8, W1.device, stream)
    if Wpacked.numel() * Wpacked.element_size() < swiglu_packed_weight_bytes_fp8(K, N):
        raise ValueError("Wpacked is too small")
    with _on_device(W1.device):
        _check(lib.swiglu_pack_weights_fp8(W1.data_ptr(), W2.data_ptr(), Wpacked.data_ptr(), K, N,
                                           _stream_handle(stream, W1.device)),
               "swiglu_pack_weights_fp8")
    return Wpacked


def swiglu_forward_fp8(A: torch.Tensor, Wpacked: torch.Tensor, N: int, scale_a: float,
                       scale_w1: float, scale_w2: float, Y: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    """Y [M, N] bf16 = SiLU(sa*A x s1*W1) * (sa*A x s2*W2) from E4M3 A [M, K] and the packed weight."""
    _dev_fp8(A, "A")
    if A.dim() != 2:
        raise ValueError("A must be [M, K]")
    M, K = A.shape
    if Wpacked.numel() * Wpacked.element_size() < swiglu_packed_weight_bytes_fp8(K, N):
        raise ValueError("Wpacked does not hold a packed FP8 weight for this K and N")
    if Y is None:
        Y = _new_tensor((M, N), torch.bfloat16, A.device, stream)
    _dev_bf16(Y, "Y")
    if tuple(Y.shape) != (M, N):
        raise ValueError("Y must be [M, N]")
    with _on_device(A.device):
        _check(lib.swiglu_forward_fp8(A.data_ptr(), Wpacked.data_ptr(), Y.data_ptr(), M, K, N,
                                      float(scale_a), float(scale_w1), float(scale_w2),
                                      _stream_handle(stream, A.device)),
               "swiglu_forward_fp8")
    return Y


def _dev_u8(t: torch.Tensor, name: str) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.uint8:
        raise ValueError(f"{name} must be uint8 (UE8M0 scale bytes), got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def swiglu_packed_weight_bytes_mxfp8(K: int, N: int) -> int:
    return int(lib.swiglu_packed_weight_bytes_mxfp8(int(K), int(N)))


def swiglu_act_scale_bytes_mxfp8(M: int, K: int) -> int:
    return int(lib.swiglu_act_scale_bytes_mxfp8(int(M), int(K)))


def swiglu_pack_weights_mxfp8(W1: torch.Tensor, S1: torch.Tensor, W2: torch.Tensor,
                              S2: torch.Tensor, Wpacked: torch.Tensor | None = None,
                              stream=None) -> torch.Tensor:
    """Packed block-scaled weight (flat uint8) from E4M3 W1, W2 [K, N] and UE8M0 S1, S2 [K/32, N]."""
    _dev_fp8(W1, "W1")
    _dev_fp8(W2, "W2")
    _dev_u8(S1, "S1")
    _dev_u8(S2, "S2")
    if W1.dim() != 2 or W1.shape != W2.shape:
        raise ValueError("W1 and W2 must both be [K, N]")
    K, N = W1.shape
    if tuple(S1.shape) != (K // 32, N) or tuple(S2.shape) != (K // 32, N):
        raise ValueError("S1 and S2 must be [K/32, N]")
    if Wpacked is None:
        Wpacked = _new_tensor(swiglu_packed_weight_bytes_mxfp8(K, N), torch.uint8, W1.device, stream)
    if Wpacked.numel() * Wpacked.element_size() < swiglu_packed_weight_bytes_mxfp8(K, N):
        raise ValueError("Wpacked is too small")
    with _on_device(W1.device):
        _check(lib.swiglu_pack_weights_mxfp8(W1.data_ptr(), S1.data_ptr(), W2.data_ptr(),
                                             S2.data_ptr(), Wpacked.data_ptr(), K, N,
                                             _stream_handle(stream, W1.device)),
               "swiglu_pack_weights_mxfp8")
    return Wpacked


def swiglu_pack_act_scales_mxfp8(SA: torch.Tensor, SAtiled: torch.Tensor | None = None,
                                 stream=None) -> torch.Tensor:
    """A's UE8M0 scales [M, K/32] in the 512-byte block layout the forward reads."""
    _dev_u8(SA, "SA")
    if SA.dim() != 2:
        raise ValueError("SA must be [M, K/32]")
    M, K = SA.shape[0], 32 * SA.shape[1]
    if SAtiled is None:
        SAtiled = _new_tensor(max(swiglu_act_scale_bytes_mxfp8(M, K), 16), torch.uint8, SA.device, stream)
    if SAtiled.numel() * SAtiled.element_size() < swiglu_act_scale_bytes_mxfp8(M, K):
        raise ValueError("SAtiled is too small")
    with _on_device(SA.device):
        _check(lib.swiglu_pack_act_scales_mxfp8(SA.data_ptr(), SAtiled.data_ptr(), M, K,
                                                _stream_handle(stream, SA.device)),
               "swiglu_pack_act_scales_mxfp8")
    return SAtiled


def swiglu_forward_mxfp8(A: torch.Tensor, SAtiled: torch.Tensor, Wpacked: torch.Tensor, N: int,
                         Y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y [M, N] bf16 = SiLU(A x W1) * (A x W2) from block-scaled E4M3 A [M, K] and the packed weight."""
    _dev_fp8(A, "A")
    if A.dim() != 2:
        raise ValueError("A must be [M, K]")
    M, K = A.shape
    if Wpacked.numel() * Wpacked.element_size() < swiglu_packed_weight_bytes_mxfp8(K, N):
        raise ValueError("Wpacked does not hold a packed block-scaled weight for this K and N")
    if SAtiled.numel() * SAtiled.element_size() < swiglu_act_scale_bytes_mxfp8(M, K):
        raise ValueError("SAtiled does not hold A's scales for this M and K")
    if Y is None:
        Y = _new_tensor((M, N), torch.bfloat16, A.device, stream)
    _dev_bf16(Y, "Y")
    if tuple(Y.shape) != (M, N):
        raise ValueError("Y must be [M, N]")
    with _on_device(A.device):
        _check(lib.swiglu_forward_mxfp8(A.data_ptr(), SAtiled.data_ptr(), Wpacked.data_ptr(),
                                        Y.data_ptr(), M, K, N, _stream_handle(stream, A.device)),
               "swiglu_forward_mxfp8")
    return Y


def swiglu_plan_string_mxfp8(M: int, K: int, N: int) -> str:
    buf = ctypes.create_string_buffer(256)
    _check(lib.swiglu_plan_string_mxfp8(int(M), int(K), int(N), buf, 256),
           "swiglu_plan_string_mxfp8")
    return buf.value.decode()


def swiglu_down_packed_bytes(N: int, H: int) -> int:
    return int(lib.swiglu_down_packed_bytes(int(N), int(H)))


def swiglu_pack_down_weights(W3: torch.Tensor, W3packed: torch.Tensor | None = None,
                             stream=None) -> torch.Tensor:
    """Packed down-projection weight (flat bf16 buffer) from W3 [N, H] (bf16, CUDA)."""
    _dev_bf16(W3, "W3")
    if W3.dim() != 2:
        raise ValueError("W3 must be [N, H]")
    N, H = W3.shape
    if W3packed is None:
        W3packed = _new_tensor(swiglu_down_packed_bytes(N, H) // 2, torch.bfloat16, W3.device, stream)
    _dev_bf16(W3packed, "W3packed")
    if W3packed.numel() * 2 < swiglu_down_packed_bytes(N, H):
        raise ValueError("W3packed is too small")
    with _on_device(W3.device):
        _check(lib.swiglu_pack_down_weights(W3.data_ptr(), W3packed.data_ptr(), N, H,
                                            _stream_handle(stream, W3.device)),
               "swiglu_pack_down_weights")
    return W3packed


def swiglu_plan_string_fp8(M: int, K: int, N: int) -> str:
    buf = ctypes.create_string_buffer(256)
    _check(lib.swiglu_plan_string_fp8(int(M), int(K), int(N), buf, 256), "swiglu_plan_string_fp8")
    return buf.value.decode()


def swiglu_down_plan_string(M: int, N: int, H: int) -> str:
    buf = ctypes.create_string_buffer(256)
    _check(lib.swiglu_down_plan_string(int(M), int(N), int(H), buf, 256),
           "swiglu_down_plan_string")
    return buf.value.decode()


def swiglu_down_plan_string_ws(M: int, N: int, H: int) -> str:
    buf = ctypes.create_string_buffer(256)
    _check(lib.swiglu_down_plan_string_ws(int(M), int(N), int(H), buf, 256),
           "swiglu_down_plan_string_ws")
    return buf.value.decode()


def swiglu_down_workspace_bytes(M: int, N: int, H: int) -> int:
    return int(lib.swiglu_down_workspace_bytes(int(M), int(N), int(H)))


def swiglu_down_workspace(M: int, N: int, H: int, device=None) -> torch.Tensor | None:
    """A zero-filled workspace for swiglu_down_forward(..., workspace=) at (M, N, H), or None.

    One workspace serves any number of calls in stream order (each call leaves
    its counters at zero); calls that may overlap in time need one each.
    """
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device())
    device = torch.device(device)
    with _on_device(device):
        n = swiglu_down_workspace_bytes(M, N, H)
    if n == 0:
        return None
    return torch.zeros(n, dtype=torch.uint8, device=device)


def swiglu_down_forward(Y: torch.Tensor, W3packed: torch.Tensor, H: int,
                        R: torch.Tensor | None = None, Out: torch.Tensor | None = None,
                        stream=None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Out [M, H] = Y [M, N] x W3 + R (R optional; Out may be R for an in-place add).

    With `workspace` (from swiglu_down_workspace, on Y's device) the decode
    kernel may also split K across clusters (swiglu_down_forward_ws).
    """
    _dev_bf16(Y, "Y")
    _dev_bf16(W3packed, "W3packed")
    if Y.dim() != 2:
        raise ValueError("Y must be [M, N]")
    M, N = Y.shape
    if W3packed.numel() * 2 < swiglu_down_packed_bytes(N, H):
        raise ValueError("W3packed does not hold a packed W3 for this N and H")
    if R is not None:
        _dev_bf16(R, "R")
        if tuple(R.shape) != (M, H):
            raise ValueError("R must be [M, H]")
    if Out is None:
        Out = _new_tensor((M, H), torch.bfloat16, Y.device, stream)
    _dev_bf16(Out, "Out")
    if tuple(Out.shape) != (M, H):
        raise ValueError("Out must be [M, H]")
    if workspace is not None:
        if not workspace.is_cuda or workspace.device != Y.device or not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous CUDA tensor on Y's device")
        with _on_device(Y.device):
            _check(lib.swiglu_down_forward_ws(
                Y.data_ptr(), W3packed.data_ptr(), R.data_ptr() if R is not None else None,
                Out.data_ptr(), M, N, H, workspace.data_ptr(),
                workspace.numel() * workspace.element_size(), _stream_handle(stream, Y.device)),
                "swiglu_down_forward_ws")
        return Out
    with _on_device(Y.device):
        _check(lib.swiglu_down_forward(Y.data_ptr(), W3packed.data_ptr(),
                                       R.data_ptr() if R is not None else None, Out.data_ptr(),
                                       M, N, H, _stream_handle(stream, Y.device)),
               "swiglu_down_forward")
    return Out


# The gradient and adapter calls take up to ten tensors, and a small one runs for
# less time on the GPU than checking them one property at a time takes here
# (Python on the Grace host: 0.1 us a property). So the checks below read each
# property once and look for the reason only when something is wrong.
_BF16 = torch.bfloat16


def _refuse(dev: int, tensors, names) -> None:
    for t, name in zip(tensors, names):
        _dev_bf16(t, name)
        if t.get_device() != dev:
            raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")


def _all_bf16(tensors, names: tuple) -> int:
    """The CUDA device that all the contiguous bf16 `tensors` are on."""
    try:
        dev = tensors[0].get_device()
        for t in tensors:
            if t.dtype is not _BF16 or t.get_device() != dev or dev < 0 or not t.is_contiguous():
                break
        else:
            return dev
    except AttributeError:
        dev = -1
    _refuse(dev, tensors, names)
    raise ValueError(f"{', '.join(names)} must be contiguous CUDA bfloat16 tensors on one device")


_cur_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _output(t, name: str, rows: int, cols: int, dev: int, stream) -> torch.Tensor:
    """A caller's output tensor, checked, or a new one."""
    if t is None:
        return _new_tensor((rows, cols), _BF16, dev, stream)
    if t.dtype is not _BF16 or t.get_device() != dev or not t.is_contiguous():
        _refuse(dev, (t,), (name,))
    if t.shape != (rows, cols):
        raise ValueError(f"{name} must be [{rows}, {cols}], got {list(t.shape)}")
    return t


def _scratch(ws, dev: int, stream, bytes_fn, *shape) -> torch.Tensor:
    """A caller's workspace, checked, or a new one of bytes_fn(*shape)."""
    if ws is None:
        return _new_tensor(bytes_fn(*shape), torch.uint8, dev, stream, returned=False)
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError(f"workspace must be a contiguous CUDA tensor on cuda:{dev}")
    return ws


def _handle(stream, dev: int) -> int:
    if stream is None:
        return _raw_stream(dev) if _raw_stream else torch.cuda.current_stream(dev).cuda_stream
    return int(stream.cuda_stream) if isinstance(stream, torch.cuda.Stream) else int(stream)


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _holds(packed: torch.Tensor, blocks: int, K: int, what: str) -> None:
    """Whether a packed weight has room for `blocks` tiles of 32 KB for every 64 of K."""
    if packed.numel() < blocks * -(-K // 64) * 16384:
        raise ValueError(f"{what} does not hold a packed weight of this shape")


def _new_workspace(bytes_fn, device, *shape) -> torch.Tensor:
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with _on_device(device):
        return torch.empty(bytes_fn(*shape), dtype=torch.uint8, device=device)


def swiglu_backward_workspace_bytes(M: int, K: int, N: int) -> int:
    return int(lib.swiglu_backward_workspace_bytes(int(M), int(K), int(N)))


def swiglu_backward_workspace(M: int, K: int, N: int, device=None) -> torch.Tensor:
    """A workspace for swiglu_backward at (M, K, N); one serves any number of calls in stream order."""
    return _new_workspace(swiglu_backward_workspace_bytes, device, M, K, N)


def _plan(name: str, *shape: int) -> str:
    buf = ctypes.create_string_buffer(256)
    _check(getattr(lib, name)(*(int(n) for n in shape), buf, 256), name)
    return buf.value.decode()


def swiglu_backward_plan_string(M: int, K: int, N: int) -> str:
    return _plan("swiglu_backward_plan_string", M, K, N)


def swiglu_down_backward_plan_string(M: int, N: int, H: int) -> str:
    return _plan("swiglu_down_backward_plan_string", M, N, H)


def swiglu_lora_plan_string(M: int, K: int, N: int, rank: int) -> str:
    return _plan("swiglu_lora_plan_string", M, K, N, rank)


def swiglu_down_lora_plan_string(M: int, N: int, H: int, rank: int) -> str:
    return _plan("swiglu_down_lora_plan_string", M, N, H, rank)


def swiglu_backward(A: torch.Tensor, Wpacked: torch.Tensor, dY: torch.Tensor,
                    dA: torch.Tensor | None = None, dW1: torch.Tensor | None = None,
                    dW2: torch.Tensor | None = None, need_input: bool = True,
                    need_weight: bool = True, workspace: torch.Tensor | None = None, stream=None):
    """(dA [M, K], dW1 [K, N], dW2 [K, N]) of Y = SiLU(A W1) * (A W2) from A [M, K] and dY [M, N].

    Gate and Up are recomputed from A and the packed weight. What need_input
    or need_weight turns off is None. Without `workspace` (from
    swiglu_backward_workspace) one is allocated for the call.
    """
    dev = _all_bf16((A, Wpacked, dY), ("A", "Wpacked", "dY"))
    if A.dim() != 2 or dY.dim() != 2 or A.shape[0] != dY.shape[0]:
        raise ValueError("A must be [M, K] and dY [M, N]")
    M, K = A.shape
    N = dY.shape[1]
    _holds(Wpacked, -(-N // 128), K, "Wpacked")
    if _cur_device() != dev:
        with torch.cuda.device(dev):
            return swiglu_backward(A, Wpacked, dY, dA, dW1, dW2, need_input, need_weight, workspace, stream)
    dA = _output(dA, "dA", M, K, dev, stream) if need_input else None
    dW1 = _output(dW1, "dW1", K, N, dev, stream) if need_weight else None
    dW2 = _output(dW2, "dW2", K, N, dev, stream) if need_weight else None
    ws = _scratch(workspace, dev, stream, swiglu_backward_workspace_bytes, M, K, N)
    rc = lib.swiglu_backward(A.data_ptr(), Wpacked.data_ptr(), dY.data_ptr(), _ptr(dA), _ptr(dW1),
                             _ptr(dW2), M, K, N, ws.data_ptr(), ws.nbytes, _handle(stream, dev))
    if rc:
        _check(rc, "swiglu_backward")
    return dA, dW1, dW2


def swiglu_down_backward_workspace_bytes(M: int, N: int, H: int) -> int:
    return int(lib.swiglu_down_backward_workspace_bytes(int(M), int(N), int(H)))


def swiglu_down_backward_workspace(M: int, N: int, H: int, device=None) -> torch.Tensor:
    """A workspace for swiglu_down_backward at (M, N, H), possibly of no bytes."""
    return _new_workspace(swiglu_down_backward_workspace_bytes, device, M, N, H)


def swiglu_down_backward(dOut: torch.Tensor, W3packed: torch.Tensor | None, Y: torch.Tensor | None,
                         dY: torch.Tensor | None = None, dW3: torch.Tensor | None = None,
                         N: int | None = None, need_input: bool = True, need_weight: bool = True,
                         workspace: torch.Tensor | None = None, stream=None):
    """(dY [M, N], dW3 [N, H]) of Out = Y W3 + R from dOut [M, H], the packed W3 and Y [M, N] (dR = dOut).

    W3packed is needed for dY only, Y for dW3 only; without Y, N says its width.
    """
    if need_weight and Y is None:
        raise ValueError("dW3 needs Y")
    if need_input and W3packed is None:
        raise ValueError("dY needs W3packed")
    if Y is None:
        dev = _all_bf16((dOut, W3packed), ("dOut", "W3packed")) if need_input else _all_bf16((dOut,), ("dOut",))
    elif W3packed is None:
        dev = _all_bf16((dOut, Y), ("dOut", "Y"))
    else:
        dev = _all_bf16((dOut, W3packed, Y), ("dOut", "W3packed", "Y"))
    if dOut.dim() != 2:
        raise ValueError("dOut must be [M, H]")
    M, H = dOut.shape
    if Y is not None:
        if Y.dim() != 2 or Y.shape[0] != M or (N is not None and Y.shape[1] != N):
            raise ValueError("Y must be [M, N]")
        N = Y.shape[1]
    if N is None:
        raise ValueError("N is needed without Y")
    if W3packed is not None:
        _holds(W3packed, -(-H // 256), N, "W3packed")
    if _cur_device() != dev:
        with torch.cuda.device(dev):
            return swiglu_down_backward(dOut, W3packed, Y, dY, dW3, N, need_input, need_weight, workspace,
                                        stream)
    dY = _output(dY, "dY", M, N, dev, stream) if need_input else None
    dW3 = _output(dW3, "dW3", N, H, dev, stream) if need_weight else None
    ws = _scratch(workspace, dev, stream, swiglu_down_backward_workspace_bytes, M, N, H)
    rc = lib.swiglu_down_backward(dOut.data_ptr(), _ptr(W3packed), _ptr(Y), _ptr(dY), _ptr(dW3), M, N, H,
                                  ws.data_ptr(), ws.nbytes, _handle(stream, dev))
    if rc:
        _check(rc, "swiglu_down_backward")
    return dY, dW3


def _adapters(La, Lb, index, scale, la_shape, lb_shape, M: int, dev: int) -> None:
    """Checks an adapter table against the shapes its projection asks for."""
    if La.shape != la_shape or Lb.shape != lb_shape:
        raise ValueError(f"La and Lb must be {list(la_shape)} and {list(lb_shape)}, "
                         f"got {list(La.shape)} and {list(Lb.shape)}")
    if (index.dtype is not torch.int32 or index.shape != (M,) or index.get_device() != dev
            or not index.is_contiguous()):
        raise ValueError(f"index must be a contiguous int32 tensor of one adapter per token on cuda:{dev}")
    if (scale.dtype is not torch.float32 or scale.shape != la_shape[:1] or scale.get_device() != dev
            or not scale.is_contiguous()):
        raise ValueError(f"scale must be a contiguous float32 tensor of one value per adapter on cuda:{dev}")


def swiglu_lora_workspace_bytes(M: int, K: int, N: int, rank: int) -> int:
    return int(lib.swiglu_lora_workspace_bytes(int(M), int(K), int(N), int(rank)))


def swiglu_lora_workspace(M: int, K: int, N: int, rank: int, device=None) -> torch.Tensor:
    """A workspace for swiglu_forward_lora; one serves any number of calls in stream order."""
    return _new_workspace(swiglu_lora_workspace_bytes, device, M, K, N, rank)


def swiglu_forward_lora(A: torch.Tensor, Wpacked: torch.Tensor, N: int, La: torch.Tensor,
                        Lb: torch.Tensor, index: torch.Tensor, scale: torch.Tensor,
                        Y: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        stream=None) -> torch.Tensor:
    """Y [M, N] = SiLU(A W1 + D1) * (A W2 + D2), Dh[m] = scale[a] A[m] La[a, h]^T Lb[a, h]^T, a = index[m].

    La [adapters, 2, rank, K] and Lb [adapters, 2, N, rank] hold the gate and
    up halves; index [M] int32 names each token's adapter (outside the table:
    none); scale [adapters] float32. Without `workspace` (from
    swiglu_lora_workspace) one is allocated for the call.
    """
    dev = _all_bf16((A, Wpacked, La, Lb), ("A", "Wpacked", "La", "Lb"))
    if A.dim() != 2 or La.dim() != 4:
        raise ValueError("A must be [M, K] and La [adapters, 2, rank, K]")
    M, K = A.shape
    count, _, rank, _ = La.shape
    _holds(Wpacked, -(-N // 128), K, "Wpacked")
    _adapters(La, Lb, index, scale, (count, 2, rank, K), (count, 2, N, rank), M, dev)
    if _cur_device() != dev:
        with torch.cuda.device(dev):
            return swiglu_forward_lora(A, Wpacked, N, La, Lb, index, scale, Y, workspace, stream)
    Y = _output(Y, "Y", M, N, dev, stream)
    ws = _scratch(workspace, dev, stream, swiglu_lora_workspace_bytes, M, K, N, rank)
    rc = lib.swiglu_forward_lora(A.data_ptr(), Wpacked.data_ptr(), Y.data_ptr(), M, K, N, La.data_ptr(),
                                 Lb.data_ptr(), index.data_ptr(), scale.data_ptr(), count, rank,
                                 ws.data_ptr(), ws.nbytes, _handle(stream, dev))
    if rc:
        _check(rc, "swiglu_forward_lora")
    return Y


def swiglu_down_lora_workspace_bytes(M: int, N: int, H: int, rank: int) -> int:
    return int(lib.swiglu_down_lora_workspace_bytes(int(M), int(N), int(H), int(rank)))


def swiglu_down_lora_workspace(M: int, N: int, H: int, rank: int, device=None) -> torch.Tensor:
    """A workspace for swiglu_down_forward_lora; one serves any number of calls in stream order."""
    return _new_workspace(swiglu_down_lora_workspace_bytes, device, M, N, H, rank)


def swiglu_down_forward_lora(Y: torch.Tensor, W3packed: torch.Tensor, H: int, La: torch.Tensor,
                             Lb: torch.Tensor, index: torch.Tensor, scale: torch.Tensor,
                             R: torch.Tensor | None = None, Out: torch.Tensor | None = None,
                             workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Out [M, H] = Y W3 + R + D, D[m] = scale[a] Y[m] La[a]^T Lb[a]^T, a = index[m].

    La [adapters, rank, N], Lb [adapters, H, rank]; index and scale as in
    swiglu_forward_lora; Out may be R (in-place add).
    """
    dev = _all_bf16((Y, W3packed, La, Lb), ("Y", "W3packed", "La", "Lb"))
    if Y.dim() != 2 or La.dim() != 3:
        raise ValueError("Y must be [M, N] and La [adapters, rank, N]")
    M, N = Y.shape
    count, rank, _ = La.shape
    _holds(W3packed, -(-H // 256), N, "W3packed")
    _adapters(La, Lb, index, scale, (count, rank, N), (count, H, rank), M, dev)
    if _cur_device() != dev:
        with torch.cuda.device(dev):
            return swiglu_down_forward_lora(Y, W3packed, H, La, Lb, index, scale, R, Out, workspace, stream)
    if R is not None:
        _output(R, "R", M, H, dev, stream)
    Out = _output(Out, "Out", M, H, dev, stream)
    ws = _scratch(workspace, dev, stream, swiglu_down_lora_workspace_bytes, M, N, H, rank)
    rc = lib.swiglu_down_forward_lora(Y.data_ptr(), W3packed.data_ptr(), _ptr(R), Out.data_ptr(), M, N, H,
                                      La.data_ptr(), Lb.data_ptr(), index.data_ptr(), scale.data_ptr(),
                                      count, rank, ws.data_ptr(), ws.nbytes, _handle(stream, dev))
    if rc:
        _check(rc, "swiglu_down_forward_lora")
    return Out


def swiglu_forward_from_host(A_host: torch.Tensor, Wpacked: torch.Tensor, N: int,
                             Y_host: torch.Tensor, A_dev: torch.Tensor, Y_dev: torch.Tensor,
                             stream=None) -> torch.Tensor:
    """Host A -> device, fused forward, device Y -> host, all enqueued on `stream`."""
    for t, name in ((A_host, "A_host"), (Y_host, "Y_host")):
        if t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bfloat16 host tensor")
    _dev_bf16(Wpacked, "Wpacked")
    _dev_bf16(A_dev, "A_dev")
    _dev_bf16(Y_dev, "Y_dev")
    M, K = A_host.shape
    if tuple(A_dev.shape) != (M, K) or tuple(Y_host.shape) != (M, N) or tuple(Y_dev.shape) != (M, N):
        raise ValueError("shape mismatch between host and device buffers")
    with _on_device(A_dev.device):
        _check(lib.swiglu_forward_from_host(A_host.data_ptr(), Wpacked.data_ptr(), Y_host.data_ptr(),
                                            A_dev.data_ptr(), Y_dev.data_ptr(), M, K, N,
                                            _stream_handle(stream, A_dev.device)),
               "swiglu_forward_from_host")
    return Y_host


def swiglu_forward_noalloc(A: torch.Tensor, Wpacked: torch.Tensor, N: int, Y: torch.Tensor,
                           status_out=None, stream=None) -> torch.Tensor:
    """Allocation-free decode forward (M <= 256) into a caller-provided Y.

    `status_out`: optional host buffer of 4 x 32-bit words that receives the
    kernel's status record once the stream synchronises: a ctypes uint32
    array, or a CPU int32 tensor (page-locked keeps the copy asynchronous).
    """
    _dev_bf16(A, "A")
    _dev_bf16(Wpacked, "Wpacked")
    _dev_bf16(Y, "Y")
    M, K = A.shape
    if tuple(Y.shape) != (M, N):
        raise ValueError("Y must be [M, N]")
    if status_out is None:
        ptr = None
    elif isinstance(status_out, torch.Tensor):
        if (status_out.is_cuda or status_out.dtype != torch.int32 or status_out.numel() < 4
                or not status_out.is_contiguous()):
            raise ValueError("status_out must be a contiguous host int32 tensor of 4 words")
        ptr = status_out.data_ptr()
    else:
        if ctypes.sizeof(status_out) < 16:
            raise ValueError("status_out must hold 4 x uint32")
        ptr = ctypes.addressof(status_out)
    with _on_device(A.device):
        _check(lib.swiglu_forward_noalloc(A.data_ptr(), Wpacked.data_ptr(), Y.data_ptr(), M, K, N,
                                          ptr, _stream_handle(stream, A.device)),
               "swiglu_forward_noalloc")
    return Y


def swiglu_check_device_status(stream=None, device=None) -> None:
    """Synchronises the stream; raises SwigluError if a kernel reported a timeout."""
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else device
    with torch.cuda.device(device):
        _check(lib.swiglu_check_device_status(_stream_handle(stream, device)),
               "swiglu_check_device_status")


def swiglu_plan_string(M: int, K: int, N: int, variant: int = SWIGLU_VARIANT_AUTO) -> str:
    buf = ctypes.create_string_buffer(256)
    _check(lib.swiglu_plan_string(int(M), int(K), int(N), int(variant), buf, 256),
           "swiglu_plan_string")
    return buf.value.decode()


def swiglu_testing_inject_stall(enable: bool, timeout_ms: int = 0) -> None:
    lib.swiglu_testing_inject_stall(1 if enable else 0, int(timeout_ms))


def swiglu_testing_pace_run_out() -> int:
    """Pacing waits of the CTA-pair kernel that ran out on the current device."""
    v = ctypes.c_uint64(0)
    _check(lib.swiglu_testing_pace_run_out(ctypes.byref(v)), "swiglu_testing_pace_run_out")
    return v.value
