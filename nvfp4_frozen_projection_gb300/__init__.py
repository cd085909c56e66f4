"""GB300-native NVFP4 LoRA linear (the hot path of PACT: "NVFP4 Data-Flow LoRA
Fine-Tuning on Consumer GPUs").

Thin Python binding over the C ABI of libpact (``include/pact.h``).  Every
function here has the same name as its C entry point and only marshals
arguments: torch provides device memory and the current stream, every step of
the computation runs in libpact's CUDA kernels.  There is no CPU fallback: if the
library is missing or the device is not sm_103, calls raise.
"""
from __future__ import annotations

import array
import ctypes
import itertools
import os
import threading
from dataclasses import dataclass

import torch

__all__ = [
    "NVFP4", "FP8", "FP8Weight", "PactError", "load_library", "library_path",
    "pact_quant_nvfp4", "pact_pack_weight_fwd", "pact_pack_weight_bwd",
    "pact_lora_linear_fwd", "pact_lora_linear_fwd_noalloc", "pact_lora_linear_dgrad",
    "pact_lora_linear_dgrad_q", "pact_lora_adapter_grad", "pact_rmsnorm_quant",
    "pact_silu_mul_quant", "pact_silu_mul_bwd", "pact_rmsnorm_bwd", "pact_test_pexp",
    "pact_pack_weight_fwd_gate_up", "pact_lora_linear_fwd_gate_up",
    "pact_quant_fp8", "pact_pack_weight_fp8_fwd", "pact_pack_weight_fp8_bwd",
    "pact_linear_fp8_fwd", "pact_linear_fp8_dgrad", "pact_add_rmsnorm_quant_fp8",
    "pact_add_rmsnorm_bwd",
    "GradList", "pact_rope_turns", "pact_qk_norm_rope", "pact_qk_norm_rope_bwd",
    "pact_attention_fwd", "pact_attention_bwd", "pact_grad_norm", "pact_clip_grad_norm",
    "pact_test_fp8_plan", "pact_test_wait_timeout", "pact_test_bounds_check", "pact_check_status",
    "pact_device_supported", "pact_launch_count", "pact_profile_next_gemm", "pact_version",
]

_HERE = os.path.dirname(os.path.abspath(__file__))


def library_path() -> str:
    """libpact.so, or with PACT_DEBUG=1 in the environment the bounds-checked debug
    build libpact_debug.so (built by build.build_debug())."""
    if os.environ.get("PACT_DEBUG") == "1":
        return os.path.join(_HERE, "libpact_debug.so")
    return os.path.join(_HERE, "libpact.so")


class PactError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libpact error {code}: {msg}")
        self.code = code


class _NVFP4Struct(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("sf", ctypes.c_void_p), ("g", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class _FP8Struct(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("s", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class _HeadsStruct(ctypes.Structure):
    _fields_ = [("p", ctypes.c_void_p), ("rows", ctypes.c_int64), ("heads", ctypes.c_int64),
                ("ld", ctypes.c_int64)]


class _ListStruct(ctypes.Structure):
    _fields_ = [("data", ctypes.c_void_p), ("numel", ctypes.c_void_p), ("first", ctypes.c_void_p),
                ("count", ctypes.c_int64), ("chunks", ctypes.c_int64)]


_LIB = None
_LIB_LOCK = threading.Lock()

_vp, _i64, _sz, _int, _f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t, ctypes.c_int, ctypes.c_float
_SP = ctypes.POINTER(_NVFP4Struct)
_SP8 = ctypes.POINTER(_FP8Struct)
_SPH = ctypes.POINTER(_HeadsStruct)
_SPL = ctypes.POINTER(_ListStruct)
_SIGNATURES = {
    "pact_nvfp4_codes_bytes": (_sz, [_i64, _i64]),
    "pact_nvfp4_sf_bytes": (_sz, [_i64, _i64]),
    "pact_quant_nvfp4_workspace_size": (_sz, [_i64, _i64]),
    "pact_quant_nvfp4": (_int, [_vp, _i64, _i64, _i64, _vp, _SP, _vp, _sz, _vp]),
    "pact_pack_weight_workspace_size": (_sz, [_i64, _i64]),
    "pact_pack_weight_fwd": (_int, [_vp, _i64, _i64, _SP, _vp, _sz, _vp]),
    "pact_pack_weight_bwd": (_int, [_vp, _i64, _i64, _SP, _vp, _sz, _vp]),
    "pact_pack_weight_fwd_gate_up": (_int, [_vp, _i64, _i64, _SP, _vp, _sz, _vp]),
    "pact_lora_linear_fwd_workspace_size": (_sz, [_i64, _i64, _i64, _int]),
    "pact_lora_linear_fwd": (_int, [_SP, _SP, _vp, _vp, _int, _f32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "pact_lora_linear_fwd_gate_up": (_int, [_SP, _SP, _vp, _vp, _int, _f32, _vp, _vp, _vp, _sz,
                                            _vp]),
    "pact_lora_linear_fwd_noalloc_max_scratch": (_sz, []),
    "pact_lora_linear_fwd_noalloc": (_int, [_SP, _SP, _vp, _vp, _int, _f32, _vp, _vp, _vp, _vp]),
    "pact_lora_linear_dgrad_workspace_size": (_sz, [_i64, _i64, _i64, _int]),
    "pact_lora_linear_dgrad": (_int, [_SP, _vp, _SP, _vp, _vp, _int, _f32, _int, _vp, _vp, _sz, _vp]),
    "pact_lora_linear_dgrad_q_workspace_size": (_sz, [_i64, _i64, _i64, _int]),
    "pact_lora_linear_dgrad_q": (_int, [_vp, _vp, _SP, _vp, _vp, _int, _f32, _int, _SP, _vp, _vp,
                                        _sz, _vp]),
    "pact_lora_adapter_grad_workspace_size": (_sz, [_i64, _i64, _i64, _int]),
    "pact_lora_adapter_grad": (_int, [_SP, _vp, _vp, _vp, _int, _f32, _i64, _vp, _vp, _vp, _sz, _vp]),
    "pact_rmsnorm_quant_workspace_size": (_sz, [_i64, _i64]),
    "pact_rmsnorm_quant": (_int, [_vp, _vp, _i64, _i64, _f32, _SP, _vp, _vp, _sz, _vp]),
    "pact_silu_mul_quant_workspace_size": (_sz, [_i64, _i64]),
    "pact_silu_mul_quant": (_int, [_vp, _i64, _i64, _vp, _SP, _SP, _SP, _vp, _sz, _vp]),
    "pact_silu_mul_bwd": (_int, [_SP, _SP, _vp, _vp, _vp, _vp]),
    "pact_rmsnorm_bwd": (_int, [_SP, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "pact_fp8_scale_count": (_sz, [_i64, _i64]),
    "pact_fp8_weight_scale_count": (_sz, [_i64, _i64]),
    "pact_quant_fp8": (_int, [_vp, _i64, _i64, _i64, _SP8, _vp]),
    "pact_pack_weight_fp8_fwd": (_int, [_vp, _i64, _i64, _SP8, _vp]),
    "pact_pack_weight_fp8_bwd": (_int, [_vp, _i64, _i64, _SP8, _vp]),
    "pact_linear_fp8_fwd": (_int, [_SP8, _SP8, _vp, _vp, _vp]),
    "pact_linear_fp8_dgrad": (_int, [_SP8, _SP8, _vp, _vp, _vp]),
    "pact_add_rmsnorm_quant_fp8": (_int, [_vp, _vp, _vp, _i64, _i64, _f32, _vp, _SP8, _vp, _vp]),
    "pact_add_rmsnorm_bwd_workspace_size": (_sz, [_i64, _i64]),
    "pact_add_rmsnorm_bwd": (_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _vp, _vp, _vp, _sz, _vp]),
    "pact_rope_turns": (_int, [_vp, _i64, _vp, _vp]),
    "pact_qk_norm_rope": (_int, [_SPH, _SPH, _i64, _i64, _vp, _vp, _int, _vp, _vp, _f32, _SPH, _SPH,
                                 _vp]),
    "pact_qk_norm_rope_bwd_workspace_size": (_sz, [_i64, _i64, _i64, _i64]),
    "pact_qk_norm_rope_bwd": (_int, [_SPH, _SPH, _SPH, _SPH, _i64, _i64, _vp, _vp, _int, _vp, _vp,
                                     _f32, _SPH, _SPH, _vp, _vp, _vp, _sz, _vp]),
    "pact_attention_fwd": (_int, [_SPH, _SPH, _SPH, _i64, _vp, _vp, _i64, _int, _f32, _SPH, _vp, _vp, _sz,
                                  _vp]),
    "pact_attention_fwd_workspace_size": (_sz, [_i64] * 6),
    "pact_attention_bwd_workspace_size": (_sz, [_i64] * 6),
    "pact_attention_bwd": (_int, [_SPH, _SPH, _SPH, _SPH, _SPH, _vp, _i64, _vp, _vp, _i64, _int, _f32,
                                  _SPH, _SPH, _SPH, _vp, _sz, _vp]),
    "pact_grad_chunks": (_i64, [_i64]),
    "pact_grad_norm_workspace_size": (_sz, []),
    "pact_grad_norm": (_int, [_SPL, _vp, _vp, _sz, _vp]),
    "pact_clip_grad_norm": (_int, [_SPL, _vp, ctypes.c_double, _vp, _vp, _sz, _vp]),
    "pact_test_fp8_plan": (_int, [_i64, _i64, _i64, _int, ctypes.POINTER(_i64)]),
    "pact_test_pexp": (_int, [_vp, _vp, _i64, _vp]),
    "pact_test_wait_timeout": (_int, [ctypes.c_uint32, _vp]),
    "pact_test_bounds_check": (_int, [_vp]),
    "pact_check_status": (_int, [_vp]),
    "pact_launch_count": (ctypes.c_uint64, []),
    "pact_profile_next_gemm": (_int, [_vp, _vp]),
    "pact_device_supported": (_int, []),
    "pact_last_error": (ctypes.c_char_p, []),
    "pact_version": (ctypes.c_char_p, []),
}


def load_library():
    """Load libpact.so (built in-tree by ``__graft_entry__.build()``)."""
    global _LIB
    with _LIB_LOCK:
        if _LIB is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(f"libpact.so is not built ({path}); run __graft_entry__.build()")
            lib = ctypes.CDLL(path)
            for name, (res, args) in _SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype = res
                fn.argtypes = args
            _LIB = lib
    return _LIB


def _check(rc: int):
    if rc != 0:
        raise PactError(rc, load_library().pact_last_error().decode())


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _need_cuda(t: torch.Tensor, dtype, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


# ------------------------------------------------------------------ NVFP4 tensor
def _pad(x, m):
    return (x + m - 1) // m * m


@dataclass
class NVFP4:
    """Device NVFP4 tensor [rows, cols]: codes u8 [rows, cols/2], sf u8 (128x4-atom
    layout, pad128(rows) * pad4(cols/16) bytes), g f32 [1] (per-tensor scale)."""
    codes: torch.Tensor
    sf: torch.Tensor
    g: torch.Tensor
    rows: int
    cols: int

    @staticmethod
    def empty(rows: int, cols: int, device=None) -> "NVFP4":
        device = device or torch.device("cuda", torch.cuda.current_device())
        # 128-byte alignment of codes and sf comes from torch's caching allocator
        codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=device)
        sf = torch.empty((_pad(rows, 128) * _pad(cols // 16, 4),), dtype=torch.uint8, device=device)
        g = torch.empty((1,), dtype=torch.float32, device=device)
        return NVFP4(codes, sf, g, rows, cols)

    def struct(self) -> _NVFP4Struct:
        return _NVFP4Struct(self.codes.data_ptr(), self.sf.data_ptr(), self.g.data_ptr(),
                            self.rows, self.cols)


# ------------------------------------------------------------------ FP8 tensors
@dataclass
class FP8:
    """Device FP8 activation or gradient [rows, cols]: q float8_e4m3fn [rows, cols] and
    s float32 [ceil(cols/128), rows], one scale per 128 values of a row."""
    q: torch.Tensor
    s: torch.Tensor

    @property
    def rows(self) -> int:
        return self.q.shape[0]

    @property
    def cols(self) -> int:
        return self.q.shape[1]

    @classmethod
    def scale_shape(cls, rows: int, cols: int) -> tuple:
        return (cols + 127) // 128, rows

    @classmethod
    def empty(cls, rows: int, cols: int, device=None):
        device = device or torch.device("cuda", torch.cuda.current_device())
        return cls(torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device=device),
                   torch.empty(cls.scale_shape(rows, cols), dtype=torch.float32, device=device))


class FP8Weight(FP8):
    """Device FP8 weight [rows, cols]: q float8_e4m3fn [rows, cols] and s float32
    [ceil(rows/128), ceil(cols/128)], one scale per 128 x 128 tile."""

    @classmethod
    def scale_shape(cls, rows: int, cols: int) -> tuple:
        return (rows + 127) // 128, (cols + 127) // 128


# The FP8 calls also serve single tokens, where a launch takes 3 us: their checks and the
# look-up of the stream are kept below that (torch.cuda.current_stream() alone takes 3).
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(
    torch._C, "_cuda_getCurrentRawStream") else (
        lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _need(t, dtype, shape, name, dev):
    """t is a contiguous tensor of this dtype and shape on the current device dev."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == dev and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")


def _need_2d(t, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 2:
        raise ValueError(f"{name} must be a 2-D CUDA tensor")
    return t.shape


def _need_fp8(t, kind, name, dev=None, shape=None) -> _FP8Struct:
    """t is an FP8 tensor of this kind (FP8 or FP8Weight) on the current device (dev, when
    it is known already), of this shape when given; its struct for the call."""
    if type(t) is not kind:
        raise ValueError(f"{name} must be an {kind.__name__}, got {type(t).__name__}")
    q, s = t.q, t.s
    rows, cols = shape = tuple(shape or _need_2d(q, name + ".q"))
    if dev is None:
        dev = torch.cuda.current_device()
    _need(q, torch.float8_e4m3fn, shape, name + ".q", dev)
    _need(s, torch.float32, kind.scale_shape(rows, cols), name + ".s", dev)
    return _FP8Struct(q.data_ptr(), s.data_ptr(), rows, cols)


def _addr(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------------ workspace
_WS = {}


def _workspace(nbytes: int, device) -> torch.Tensor:
    """Per-(device, stream) scratch buffer, grown on demand.  Calls on one stream run
    in order, so they can share it."""
    key = (device.index if device.index is not None else torch.cuda.current_device(),
           torch.cuda.current_stream(device).cuda_stream)
    buf = _WS.get(key)
    need = max(256, int(nbytes))
    if buf is None or buf.numel() < need:
        buf = torch.empty((_pad(need, 1 << 20),), dtype=torch.uint8, device=device)
        _WS[key] = buf
    return buf


# ------------------------------------------------------------------ entry points
def pact_quant_nvfp4(x: torch.Tensor, amax: torch.Tensor | None = None,
                     out: NVFP4 | None = None) -> NVFP4:
    """Quantise BF16 x [M, K] (row stride may exceed K) to NVFP4."""
    lib = load_library()
    if not (isinstance(x, torch.Tensor) and x.is_cuda and x.dtype == torch.bfloat16 and x.dim() == 2):
        raise ValueError("x must be a 2-D CUDA bfloat16 tensor")
    if x.stride(1) != 1:
        raise ValueError("x must have unit column stride")
    M, K = x.shape
    out = out or NVFP4.empty(M, K, x.device)
    ws = _workspace(lib.pact_quant_nvfp4_workspace_size(M, K), x.device)
    s = out.struct()
    _check(lib.pact_quant_nvfp4(_ptr(x), M, K, x.stride(0), _ptr(amax), ctypes.byref(s),
                                _ptr(ws), ws.numel(), _stream()))
    return out


def _pack(W: torch.Tensor, backward: bool, out: NVFP4 | None, gate_up: bool = False) -> NVFP4:
    lib = load_library()
    _need_cuda(W, torch.float32, "W")
    N, K = W.shape
    out = out or (NVFP4.empty(K, N, W.device) if backward else NVFP4.empty(N, K, W.device))
    ws = _workspace(lib.pact_pack_weight_workspace_size(N, K), W.device)
    s = out.struct()
    fn = (lib.pact_pack_weight_bwd if backward else
          (lib.pact_pack_weight_fwd_gate_up if gate_up else lib.pact_pack_weight_fwd))
    _check(fn(_ptr(W), N, K, ctypes.byref(s), _ptr(ws), ws.numel(), _stream()))
    return out


def pact_pack_weight_fwd(W: torch.Tensor, out: NVFP4 | None = None) -> NVFP4:
    """Pack the frozen FP32 weight W [N, K] into the forward NVFP4 layout [N, K]."""
    return _pack(W, False, out)


def pact_pack_weight_bwd(W: torch.Tensor, out: NVFP4 | None = None) -> NVFP4:
    """Pack the frozen FP32 weight W [N, K] into the backward NVFP4 layout [K, N]."""
    return _pack(W, True, out)


def pact_pack_weight_fwd_gate_up(W: torch.Tensor, out: NVFP4 | None = None) -> NVFP4:
    """Forward pack of a fused gate|up weight [2I, K] in the interleaved row order that
    pact_lora_linear_fwd_gate_up reads."""
    return _pack(W, False, out, gate_up=True)


def pact_lora_linear_fwd_gate_up(xq: NVFP4, w_fwd_gu: NVFP4, A: torch.Tensor, B: torch.Tensor,
                                 scale: float, y: torch.Tensor | None = None,
                                 amax3: torch.Tensor | None = None):
    """The fused gate|up forward (y [M, 2I] as pact_lora_linear_fwd) and amax3 =
    (max |silu(gate) up|, max |gate|, max |up|) of it.  Returns (y, amax3)."""
    lib = load_library()
    _need_cuda(A, torch.bfloat16, "A")
    _need_cuda(B, torch.bfloat16, "B")
    M, K, N = xq.rows, xq.cols, w_fwd_gu.rows
    r = A.shape[1]
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    if amax3 is None:
        amax3 = torch.empty(3, dtype=torch.float32, device=A.device)
    _need_cuda(y, torch.bfloat16, "y")
    _need_cuda(amax3, torch.float32, "amax3")
    ws = _workspace(lib.pact_lora_linear_fwd_workspace_size(M, N, K, r), A.device)
    sx, sw = xq.struct(), w_fwd_gu.struct()
    _check(lib.pact_lora_linear_fwd_gate_up(ctypes.byref(sx), ctypes.byref(sw), _ptr(A), _ptr(B), r,
                                            float(scale), _ptr(y), _ptr(amax3), _ptr(ws),
                                            ws.numel(), _stream()))
    return y, amax3


def pact_lora_linear_fwd(xq: NVFP4, w_fwd: NVFP4, A: torch.Tensor, B: torch.Tensor,
                         scale: float, residual: torch.Tensor | None = None,
                         y: torch.Tensor | None = None,
                         out_amax: torch.Tensor | None = None) -> torch.Tensor:
    """Y = Xhat What^T + scale (Xhat A) B [+ residual], BF16 [M, N]."""
    lib = load_library()
    _need_cuda(A, torch.bfloat16, "A")
    _need_cuda(B, torch.bfloat16, "B")
    M, K, N = xq.rows, xq.cols, w_fwd.rows
    r = A.shape[1]
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=A.device)
    _need_cuda(y, torch.bfloat16, "y")
    if residual is not None:
        _need_cuda(residual, torch.bfloat16, "residual")
    ws = _workspace(lib.pact_lora_linear_fwd_workspace_size(M, N, K, r), A.device)
    sx, sw = xq.struct(), w_fwd.struct()
    _check(lib.pact_lora_linear_fwd(ctypes.byref(sx), ctypes.byref(sw), _ptr(A), _ptr(B), r,
                                    float(scale), _ptr(residual), _ptr(y), _ptr(out_amax),
                                    _ptr(ws), ws.numel(), _stream()))
    return y


def pact_lora_linear_fwd_noalloc(xq: NVFP4, w_fwd: NVFP4, A: torch.Tensor, B: torch.Tensor,
                                 scale: float, y: torch.Tensor,
                                 residual: torch.Tensor | None = None,
                                 out_amax: torch.Tensor | None = None) -> torch.Tensor:
    """pact_lora_linear_fwd for callers that cannot allocate: the output y is
    preallocated by the caller and the library's fixed scratch array replaces the
    workspace (calls that overlap on the GPU race on it)."""
    lib = load_library()
    _need_cuda(A, torch.bfloat16, "A")
    _need_cuda(B, torch.bfloat16, "B")
    _need_cuda(y, torch.bfloat16, "y")
    sx, sw = xq.struct(), w_fwd.struct()
    _check(lib.pact_lora_linear_fwd_noalloc(ctypes.byref(sx), ctypes.byref(sw), _ptr(A), _ptr(B),
                                            A.shape[1], float(scale), _ptr(residual), _ptr(y),
                                            _ptr(out_amax), _stream()))
    return y


def pact_lora_linear_dgrad(dyq: NVFP4, dy: torch.Tensor, w_bwd: NVFP4, A: torch.Tensor,
                           B: torch.Tensor, scale: float, dx: torch.Tensor | None = None,
                           accumulate: bool = False) -> torch.Tensor:
    """dX = dYhat W + scale (dY B^T) A^T [+ dX if accumulate], BF16 [M, K]."""
    lib = load_library()
    _need_cuda(dy, torch.bfloat16, "dy")
    _need_cuda(A, torch.bfloat16, "A")
    _need_cuda(B, torch.bfloat16, "B")
    M, N, K = dyq.rows, dyq.cols, w_bwd.rows
    r = A.shape[1]
    if dx is None:
        if accumulate:
            raise ValueError("accumulate needs dx")
        dx = torch.empty((M, K), dtype=torch.bfloat16, device=dy.device)
    _need_cuda(dx, torch.bfloat16, "dx")
    ws = _workspace(lib.pact_lora_linear_dgrad_workspace_size(M, N, K, r), dy.device)
    sd, sw = dyq.struct(), w_bwd.struct()
    _check(lib.pact_lora_linear_dgrad(ctypes.byref(sd), _ptr(dy), ctypes.byref(sw), _ptr(A),
                                      _ptr(B), r, float(scale), int(bool(accumulate)), _ptr(dx),
                                      _ptr(ws), ws.numel(), _stream()))
    return dx


def pact_lora_linear_dgrad_q(dy: torch.Tensor, w_bwd: NVFP4, A: torch.Tensor, B: torch.Tensor,
                             scale: float, amax: torch.Tensor | None = None,
                             dyq: NVFP4 | None = None, dx: torch.Tensor | None = None,
                             accumulate: bool = False):
    """Quantise dY into dyq and run the LoRA-linear input gradient in one call:
    the same results as pact_quant_nvfp4 + pact_lora_linear_dgrad.  Returns (dx, dyq)."""
    lib = load_library()
    _need_cuda(dy, torch.bfloat16, "dy")
    _need_cuda(A, torch.bfloat16, "A")
    _need_cuda(B, torch.bfloat16, "B")
    M, N = dy.shape
    K = w_bwd.rows
    r = A.shape[1]
    if amax is not None:
        _need_cuda(amax, torch.float32, "amax")
    if dyq is None:
        dyq = NVFP4.empty(M, N, dy.device)
    if dx is None:
        if accumulate:
            raise ValueError("accumulate needs dx")
        dx = torch.empty((M, K), dtype=torch.bfloat16, device=dy.device)
    _need_cuda(dx, torch.bfloat16, "dx")
    ws = _workspace(lib.pact_lora_linear_dgrad_q_workspace_size(M, N, K, r), dy.device)
    sq, sw = dyq.struct(), w_bwd.struct()
    _check(lib.pact_lora_linear_dgrad_q(_ptr(dy), _ptr(amax), ctypes.byref(sw), _ptr(A), _ptr(B),
                                        r, float(scale), int(bool(accumulate)), ctypes.byref(sq),
                                        _ptr(dx), _ptr(ws), ws.numel(), _stream()))
    return dx, dyq


def pact_lora_adapter_grad(xq: NVFP4, dy: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                           scale: float, dA: torch.Tensor | None = None,
                           dB: torch.Tensor | None = None):
    """dA = scale Xhat^T (dY B^T) FP32 [K, r] and dB = scale (Xhat A)^T dY FP32 [r, N]."""
    lib = load_library()
    _need_cuda(dy, torch.bfloat16, "dy")
    _need_cuda(A, torch.bfloat16, "A")
    _need_cuda(B, torch.bfloat16, "B")
    M, K = xq.rows, xq.cols
    N = dy.shape[1]
    r = A.shape[1]
    if dA is None:
        dA = torch.empty((K, r), dtype=torch.float32, device=dy.device)
    if dB is None:
        dB = torch.empty((r, N), dtype=torch.float32, device=dy.device)
    _need_cuda(dA, torch.float32, "dA")
    _need_cuda(dB, torch.float32, "dB")
    ws = _workspace(lib.pact_lora_adapter_grad_workspace_size(M, N, K, r), dy.device)
    sx = xq.struct()
    _check(lib.pact_lora_adapter_grad(ctypes.byref(sx), _ptr(dy), _ptr(A), _ptr(B), r,
                                      float(scale), N, _ptr(dA), _ptr(dB), _ptr(ws), ws.numel(),
                                      _stream()))
    return dA, dB


def pact_rmsnorm_quant(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-5,
                       out: NVFP4 | None = None, rstd: torch.Tensor | None = None):
    """Fused RMSNorm -> NVFP4.  Returns (yq, rstd)."""
    lib = load_library()
    _need_cuda(x, torch.bfloat16, "x")
    _need_cuda(gamma, torch.bfloat16, "gamma")
    M, H = x.shape
    out = out or NVFP4.empty(M, H, x.device)
    if rstd is None:
        rstd = torch.empty((M,), dtype=torch.float32, device=x.device)
    ws = _workspace(lib.pact_rmsnorm_quant_workspace_size(M, H), x.device)
    s = out.struct()
    _check(lib.pact_rmsnorm_quant(_ptr(x), _ptr(gamma), M, H, float(eps), ctypes.byref(s),
                                  _ptr(rstd), _ptr(ws), ws.numel(), _stream()))
    return out, rstd


def pact_silu_mul_quant(gateup: torch.Tensor, amax3: torch.Tensor | None = None,
                        outs: tuple | None = None):
    """Fused SiLU-multiply -> NVFP4 on gateup [M, 2I].  Returns (hq, gate_q, up_q)."""
    lib = load_library()
    _need_cuda(gateup, torch.bfloat16, "gateup")
    M, I2 = gateup.shape
    I = I2 // 2
    hq, gq, uq = outs or tuple(NVFP4.empty(M, I, gateup.device) for _ in range(3))
    ws = _workspace(lib.pact_silu_mul_quant_workspace_size(M, I), gateup.device)
    sh, sg, su = hq.struct(), gq.struct(), uq.struct()
    _check(lib.pact_silu_mul_quant(_ptr(gateup), M, I, _ptr(amax3), ctypes.byref(sh),
                                   ctypes.byref(sg), ctypes.byref(su), _ptr(ws), ws.numel(),
                                   _stream()))
    return hq, gq, uq


def pact_silu_mul_bwd(gate_q: NVFP4, up_q: NVFP4, dh: torch.Tensor,
                      dgateup: torch.Tensor | None = None,
                      out_amax: torch.Tensor | None = None) -> torch.Tensor:
    """SiLU-multiply backward from the NVFP4 gate/up copies.  Returns dgateup [M, 2I]."""
    lib = load_library()
    _need_cuda(dh, torch.bfloat16, "dh")
    M, I = gate_q.rows, gate_q.cols
    if dgateup is None:
        dgateup = torch.empty((M, 2 * I), dtype=torch.bfloat16, device=dh.device)
    sg, su = gate_q.struct(), up_q.struct()
    _check(lib.pact_silu_mul_bwd(ctypes.byref(sg), ctypes.byref(su), _ptr(dh), _ptr(dgateup),
                                 _ptr(out_amax), _stream()))
    return dgateup


def pact_rmsnorm_bwd(yq: NVFP4, gamma: torch.Tensor, rstd: torch.Tensor, dy: torch.Tensor,
                     dres: torch.Tensor | None = None,
                     dx: torch.Tensor | None = None,
                     out_amax: torch.Tensor | None = None) -> torch.Tensor:
    """RMSNorm backward from the retained NVFP4 output and rstd [+ dres].  out_amax
    (FP32 [1], optional) receives max |dx| for a single-pass quantisation of dx."""
    lib = load_library()
    _need_cuda(dy, torch.bfloat16, "dy")
    if dx is None:
        dx = torch.empty_like(dy)
    if out_amax is not None:
        _need_cuda(out_amax, torch.float32, "out_amax")
    s = yq.struct()
    _check(lib.pact_rmsnorm_bwd(ctypes.byref(s), _ptr(gamma), _ptr(rstd), _ptr(dy), _ptr(dres),
                                _ptr(dx), _ptr(out_amax), _stream()))
    return dx


# ------------------------------------------------------------------ FP8, blocks of 128
def pact_quant_fp8(x: torch.Tensor, out: FP8 | None = None) -> FP8:
    """Quantise BF16 x [M, K] (row stride may exceed K) to FP8."""
    lib = _LIB or load_library()
    M, K = _need_2d(x, "x")
    if x.dtype != torch.bfloat16:
        raise ValueError(f"x must be torch.bfloat16, got {x.dtype}")
    if x.stride(1) != 1:
        raise ValueError("x must have unit column stride")
    dev = torch.cuda.current_device()
    if x.device.index != dev:
        raise ValueError(f"x is on {x.device}, the current device is cuda:{dev}")
    if out is None:
        out = FP8.empty(M, K, x.device)
    s = _need_fp8(out, FP8, "out", dev, (M, K))
    # the stride of a single row says nothing: torch may report any number there
    _check(lib.pact_quant_fp8(_addr(x), M, K, x.stride(0) if M > 1 else _pad(K, 8),
                              ctypes.byref(s), _raw_stream(dev)))
    return out


def _pack_fp8(W: torch.Tensor, backward: bool, out: FP8Weight | None) -> FP8Weight:
    lib = _LIB or load_library()
    N, K = _need_2d(W, "W")
    dev = torch.cuda.current_device()
    _need(W, torch.float32, (N, K), "W", dev)
    shape = (K, N) if backward else (N, K)
    if out is None:
        out = FP8Weight.empty(*shape, W.device)
    s = _need_fp8(out, FP8Weight, "out", dev, shape)
    fn = lib.pact_pack_weight_fp8_bwd if backward else lib.pact_pack_weight_fp8_fwd
    _check(fn(_addr(W), N, K, ctypes.byref(s), _raw_stream(dev)))
    return out


def pact_pack_weight_fp8_fwd(W: torch.Tensor, out: FP8Weight | None = None) -> FP8Weight:
    """Pack the frozen FP32 weight W [N, K] into the FP8 forward layout [N, K]."""
    return _pack_fp8(W, False, out)


def pact_pack_weight_fp8_bwd(W: torch.Tensor, out: FP8Weight | None = None) -> FP8Weight:
    """Pack the frozen FP32 weight W [N, K] into the FP8 backward layout [K, N]: the
    forward layout's codes and tile scales, transposed."""
    return _pack_fp8(W, True, out)


def _linear_fp8(fn, x, xname, w, wname, add, addname, y, yname):
    sx = _need_fp8(x, FP8, xname)
    dev = x.q.get_device()
    sw = _need_fp8(w, FP8Weight, wname, dev)
    shape = (sx.rows, sw.rows)
    if sw.cols != sx.cols:
        raise ValueError(f"{xname} has {sx.cols} columns, {wname} {sw.cols}")
    if y is None:
        y = torch.empty(shape, dtype=torch.bfloat16, device=x.q.device)
    _need(y, torch.bfloat16, shape, yname, dev)
    if add is not None:
        _need(add, torch.bfloat16, shape, addname, dev)
    _check(fn(ctypes.byref(sx), ctypes.byref(sw), _addr(add), _addr(y), _raw_stream(dev)))
    return y


def pact_linear_fp8_fwd(xq: FP8, w_fwd: FP8Weight, residual: torch.Tensor | None = None,
                        y: torch.Tensor | None = None) -> torch.Tensor:
    """Y = Xhat What^T [+ residual], BF16 [M, N]; any M from one token up.  residual may
    be y itself."""
    return _linear_fp8((_LIB or load_library()).pact_linear_fp8_fwd, xq, "xq", w_fwd, "w_fwd", residual,
                       "residual", y, "y")


def pact_linear_fp8_dgrad(dyq: FP8, w_bwd: FP8Weight, dx_prev: torch.Tensor | None = None,
                          dx: torch.Tensor | None = None) -> torch.Tensor:
    """dX = dYhat W [+ dX_prev], BF16 [M, K], on the backward layout.  dx_prev may be dx
    itself, to add to it."""
    return _linear_fp8((_LIB or load_library()).pact_linear_fp8_dgrad, dyq, "dyq", w_bwd, "w_bwd", dx_prev,
                       "dx_prev", dx, "dx")


def pact_add_rmsnorm_quant_fp8(x: torch.Tensor, residual: torch.Tensor | None,
                               gamma: torch.Tensor, eps: float = 1e-5,
                               h: torch.Tensor | None = None, out: FP8 | None = None,
                               rstd: torch.Tensor | None = None):
    """h = bf16(x + residual), RMSNorm of h to FP8.  Without a residual h is x itself.
    h may be x or residual, to add in place.  Returns (h, yq, rstd)."""
    lib = _LIB or load_library()
    M, H = _need_2d(x, "x")
    dev = torch.cuda.current_device()
    _need(x, torch.bfloat16, (M, H), "x", dev)
    _need(gamma, torch.bfloat16, (H,), "gamma", dev)
    if residual is not None:
        _need(residual, torch.bfloat16, (M, H), "residual", dev)
        if h is None:
            h = torch.empty_like(x)
        _need(h, torch.bfloat16, (M, H), "h", dev)
    elif h is not None and h is not x:
        raise ValueError("without a residual h is x itself: pass no other h")
    if out is None:
        out = FP8.empty(M, H, x.device)
    s = _need_fp8(out, FP8, "out", dev, (M, H))
    if rstd is None:
        rstd = torch.empty((M,), dtype=torch.float32, device=x.device)
    _need(rstd, torch.float32, (M,), "rstd", dev)
    _check(lib.pact_add_rmsnorm_quant_fp8(_addr(x), _addr(residual), _addr(gamma), M, H, float(eps),
                                          _addr(h) if residual is not None else None,
                                          ctypes.byref(s), _addr(rstd), _raw_stream(dev)))
    return (x if residual is None else h), out, rstd


def pact_add_rmsnorm_bwd(h: torch.Tensor, gamma: torch.Tensor, rstd: torch.Tensor,
                         dy: torch.Tensor, dres: torch.Tensor | None = None,
                         dh: torch.Tensor | None = None,
                         dgamma: torch.Tensor | bool | None = None):
    """Backward of pact_add_rmsnorm_quant_fp8 from h and rstd: dh [+ dres], the gradient
    of x and of the residual alike (dh may be dy, dres or h).  dgamma: an FP32 [H] tensor
    to overwrite, True for a new one, None to leave it out.  Returns (dh, dgamma)."""
    lib = _LIB or load_library()
    M, H = _need_2d(h, "h")
    dev = torch.cuda.current_device()
    _need(h, torch.bfloat16, (M, H), "h", dev)
    _need(gamma, torch.bfloat16, (H,), "gamma", dev)
    _need(rstd, torch.float32, (M,), "rstd", dev)
    _need(dy, torch.bfloat16, (M, H), "dy", dev)
    if dres is not None:
        _need(dres, torch.bfloat16, (M, H), "dres", dev)
    if dh is None:
        dh = torch.empty_like(dy)
    _need(dh, torch.bfloat16, (M, H), "dh", dev)
    ws = None
    if dgamma is False:
        dgamma = None
    if dgamma is not None:
        if dgamma is True:
            dgamma = torch.empty((H,), dtype=torch.float32, device=h.device)
        _need(dgamma, torch.float32, (H,), "dgamma", dev)
        # its own scratch in every call: a captured graph then keeps one of its own
        size = lib.pact_add_rmsnorm_bwd_workspace_size(M, H)
        if size:
            ws = torch.empty((size,), dtype=torch.uint8, device=h.device)
    _check(lib.pact_add_rmsnorm_bwd(_addr(h), _addr(gamma), _addr(rstd), _addr(dy), _addr(dres), M, H,
                                    _addr(dh), _addr(dgamma), _addr(ws),
                                    0 if ws is None else ws.numel(), _raw_stream(dev)))
    return dh, dgamma


# ------------------------------------------------------------------ heads and attention
def _heads(t, name, dev, like=None) -> tuple:
    """The fields of pact_heads for t: a BF16 tensor of heads [T, heads, D] on the current
    device, of this shape when given, whose tokens lie ld values apart and whose heads are
    contiguous."""
    try:
        rows, heads, d = shape = t.shape
        ld, sh, sd = t.stride()
        if (t.dtype is torch.bfloat16 and t.get_device() == dev and sd == 1 and sh == d
                and (like is None or shape == like)):
            # the stride of a single row says nothing: torch may report any number there
            return t.data_ptr(), rows, heads, ld if rows > 1 else heads * d
    except (AttributeError, TypeError, ValueError):
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dim() != 3:
        raise ValueError(f"{name} must be a 3-D CUDA tensor [tokens, heads, D]")
    if t.dtype is not torch.bfloat16:
        raise ValueError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
    if like is not None and shape != like:
        raise ValueError(f"{name} must have shape {list(like)}, got {list(shape)}")
    if (sd != 1 and d > 1) or (sh != d and heads > 1):
        raise ValueError(f"the heads of {name} must be contiguous")
    return t.data_ptr(), rows, heads, ld if rows > 1 else heads * d


# Several pact_heads at once: one array of their fields, whose addresses are passed.  A
# structure for each costs twice as much, which a call on one token would notice.
_HEADS = {n: _i64 * (4 * n) for n in (4, 6, 8)}
_FAST = {}
_DENSE = torch.contiguous_format  # outputs of inputs with strides have none


def _heads_call(lib, name):
    """The library's function with plain addresses for its pact_heads."""
    fn = _FAST.get(name)
    if fn is None:
        fn = lib[name]  # an object of its own, beside the attribute of that name
        res, args = _SIGNATURES[name]
        fn.restype, fn.argtypes = res, [_vp if a is _SPH else a for a in args]
        _FAST[name] = fn
    return fn


def pact_rope_turns(inv_freq: torch.Tensor, turns: torch.Tensor | None = None) -> torch.Tensor:
    """The table of a rotary embedding (int64 [n], fractions of a turn) from its frequencies
    in radians per position, float64 [n]."""
    lib = _LIB or load_library()
    n = inv_freq.shape[0] if isinstance(inv_freq, torch.Tensor) and inv_freq.dim() == 1 else 0
    dev = torch.cuda.current_device()
    _need(inv_freq, torch.float64, (n,), "inv_freq", dev)
    if turns is None:
        turns = torch.empty((n,), dtype=torch.int64, device=inv_freq.device)
    _need(turns, torch.int64, (n,), "turns", dev)
    _check(lib.pact_rope_turns(_addr(inv_freq), n, _addr(turns), _raw_stream(dev)))
    return turns


def _need_rope(positions, turns, gamma_q, gamma_k, T, D, dev):
    _need(positions, torch.int32, (T,), "positions", dev)
    n = turns.shape[0] if isinstance(turns, torch.Tensor) and turns.dim() == 1 else 0
    _need(turns, torch.int64, (n,), "turns", dev)
    if gamma_q is not None:
        _need(gamma_q, torch.bfloat16, (D,), "gamma_q", dev)
    if gamma_k is not None:
        _need(gamma_k, torch.bfloat16, (D,), "gamma_k", dev)
    return 2 * n


def pact_qk_norm_rope(q: torch.Tensor, k: torch.Tensor, positions: torch.Tensor,
                      turns: torch.Tensor, gamma_q: torch.Tensor | None = None,
                      gamma_k: torch.Tensor | None = None, eps: float = 1e-5,
                      interleaved: bool = False, q_out: torch.Tensor | None = None,
                      k_out: torch.Tensor | None = None):
    """RMSNorm of every head (with gammas) and the rotary embedding of the first
    2 len(turns) columns, for q [T, hq, D] and k [T, hk, D].  An output may be its own
    input.  Returns (q_out, k_out)."""
    lib = _LIB or load_library()
    dev = torch.cuda.current_device()
    hq, hk = _heads(q, "q", dev), _heads(k, "k", dev)
    T, _, D = q.shape
    if k.shape[2] != D:
        raise ValueError(f"q has heads of {D}, k of {k.shape[2]}")
    rot = _need_rope(positions, turns, gamma_q, gamma_k, T, D, dev)
    if q_out is None:
        q_out = torch.empty_like(q, memory_format=_DENSE)
    if k_out is None:
        k_out = torch.empty_like(k, memory_format=_DENSE)
    h = _HEADS[4](*hq, *hk, *_heads(q_out, "q_out", dev, q.shape), *_heads(k_out, "k_out", dev, k.shape))
    at = ctypes.addressof(h)
    _check(_heads_call(lib, "pact_qk_norm_rope")(
        at, at + 32, D, rot, positions.data_ptr(), turns.data_ptr(), 1 if interleaved else 0,
        _addr(gamma_q), _addr(gamma_k), float(eps), at + 64, at + 96, _raw_stream(dev)))
    return q_out, k_out


def pact_qk_norm_rope_bwd(dyq: torch.Tensor, dyk: torch.Tensor, positions: torch.Tensor,
                          turns: torch.Tensor, q: torch.Tensor | None = None,
                          k: torch.Tensor | None = None, gamma_q: torch.Tensor | None = None,
                          gamma_k: torch.Tensor | None = None, eps: float = 1e-5,
                          interleaved: bool = False, dq: torch.Tensor | None = None,
                          dk: torch.Tensor | None = None,
                          dgamma_q: torch.Tensor | bool | None = None,
                          dgamma_k: torch.Tensor | bool | None = None):
    """Backward of pact_qk_norm_rope; q and k are its inputs, needed with gammas.  dq may
    be dyq or q, dk dyk or k.  dgamma_q, dgamma_k: FP32 [D] tensors to overwrite, True for
    new ones, None to leave both out.  Returns (dq, dk, dgamma_q, dgamma_k)."""
    lib = _LIB or load_library()
    dev = torch.cuda.current_device()
    sq, sk = _heads(dyq, "dyq", dev), _heads(dyk, "dyk", dev)
    T, hq, D = dyq.shape
    if dyk.shape[2] != D:
        raise ValueError(f"dyq has heads of {D}, dyk of {dyk.shape[2]}")
    rot = _need_rope(positions, turns, gamma_q, gamma_k, T, D, dev)
    none = (0, 0, 0, 0)
    xq = _heads(q, "q", dev, dyq.shape) if q is not None else none
    xk = _heads(k, "k", dev, dyk.shape) if k is not None else none
    if dq is None:
        dq = torch.empty_like(dyq, memory_format=_DENSE)
    if dk is None:
        dk = torch.empty_like(dyk, memory_format=_DENSE)
    h = _HEADS[6](*sq, *sk, *xq, *xk, *_heads(dq, "dq", dev, dyq.shape), *_heads(dk, "dk", dev, dyk.shape))
    at = ctypes.addressof(h)
    grads = []
    for g, name in ((dgamma_q, "dgamma_q"), (dgamma_k, "dgamma_k")):
        if g is True:
            g = torch.empty((D,), dtype=torch.float32, device=dyq.device)
        elif g is False:
            g = None
        if g is not None:
            _need(g, torch.float32, (D,), name, dev)
        grads.append(g)
    ws = None
    if grads[0] is not None:
        # its own scratch in every call: a captured graph then keeps one of its own
        ws = torch.empty((lib.pact_qk_norm_rope_bwd_workspace_size(T, hq, dyk.shape[1], D),),
                         dtype=torch.uint8, device=dyq.device)
    _check(_heads_call(lib, "pact_qk_norm_rope_bwd")(
        at, at + 32, at + 64 if q is not None else None, at + 96 if k is not None else None, D, rot,
        positions.data_ptr(), turns.data_ptr(), 1 if interleaved else 0, _addr(gamma_q),
        _addr(gamma_k), float(eps), at + 128, at + 160, _addr(grads[0]), _addr(grads[1]), _addr(ws),
        0 if ws is None else ws.numel(), _raw_stream(dev)))
    return dq, dk, grads[0], grads[1]


def _need_attention(q, k, v, cu_q, cu_k, scale, dev):
    """The fields of q, k and v, the heads' width, the number of sequences and the scale."""
    fields = _heads(q, "q", dev) + _heads(k, "k", dev) + _heads(v, "v", dev, k.shape)
    D = q.shape[2]
    if k.shape[2] != D:
        raise ValueError(f"q has heads of {D}, k of {k.shape[2]}")
    if not isinstance(cu_q, torch.Tensor) or cu_q.dim() != 1 or cu_q.shape[0] < 2:
        raise ValueError("cu_q must be a 1-D tensor of at least two offsets")
    _need(cu_q, torch.int32, cu_q.shape, "cu_q", dev)
    _need(cu_k, torch.int32, cu_q.shape, "cu_k", dev)
    return fields, D, cu_q.shape[0] - 1, float(D ** -0.5 if scale is None else scale)


# Keys a sequence has on average below which pact_attention_fwd_workspace_size is 0 whatever
# else it is given: asking costs a small call 1 us.
_PARTS_KEYS = 2048


def pact_attention_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_q: torch.Tensor,
                       cu_k: torch.Tensor, causal: bool = True, scale: float | None = None,
                       o: torch.Tensor | None = None, lse: torch.Tensor | None = None):
    """Attention over packed sequences: q [Tq, hq, D], k and v [Tk, hk, D], sequence b at
    rows cu_q[b]:cu_q[b + 1] and cu_k[b]:cu_k[b + 1] (int32, on the device).  scale is
    1 / sqrt(D) by default.  o may be q.  Returns (o [Tq, hq, D], lse FP32 [hq, Tq]); rows of
    no sequence are left as they were (in new tensors: as the memory was)."""
    lib = _LIB or load_library()
    dev = torch.cuda.current_device()
    fields, D, n, scale = _need_attention(q, k, v, cu_q, cu_k, scale, dev)
    if o is None:
        o = torch.empty_like(q, memory_format=_DENSE)
    h = _HEADS[4](*fields, *_heads(o, "o", dev, q.shape))
    at = ctypes.addressof(h)
    shape = (q.shape[1], q.shape[0])
    if lse is None:
        lse = torch.empty(shape, dtype=torch.float32, device=q.device)
    _need(lse, torch.float32, shape, "lse", dev)
    Tk, size, ws = k.shape[0], 0, None
    if Tk >= _PARTS_KEYS * n:
        size = lib.pact_attention_fwd_workspace_size(shape[1], shape[0], Tk, k.shape[1], D, n)
        # its own in every call, as for the backward
        ws = torch.empty((size,), dtype=torch.uint8, device=q.device) if size else None
    _check(_heads_call(lib, "pact_attention_fwd")(
        at, at + 32, at + 64, D, cu_q.data_ptr(), cu_k.data_ptr(), n, 1 if causal else 0, scale,
        at + 96, lse.data_ptr(), _addr(ws), size, _raw_stream(dev)))
    return o, lse


def pact_attention_bwd(do: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                       o: torch.Tensor, lse: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor,
                       causal: bool = True, scale: float | None = None,
                       dq: torch.Tensor | None = None, dk: torch.Tensor | None = None,
                       dv: torch.Tensor | None = None):
    """Backward of pact_attention_fwd from its inputs, its o and lse and the gradient do of
    o.  Returns (dq, dk, dv), which share no memory with one another or an input; rows of no
    sequence are left as they were (in new tensors: as the memory was), so a padded batch whose
    gradients are summed over all rows wants tensors of zeros."""
    lib = _LIB or load_library()
    dev = torch.cuda.current_device()
    fields, D, n, scale = _need_attention(q, k, v, cu_q, cu_k, scale, dev)
    fields += _heads(do, "do", dev, q.shape) + _heads(o, "o", dev, q.shape)
    _need(lse, torch.float32, (q.shape[1], q.shape[0]), "lse", dev)
    dq, dk, dv = (torch.empty_like(x, memory_format=_DENSE) if g is None else g
                  for g, x in ((dq, q), (dk, k), (dv, v)))
    h = _HEADS[8](*fields, *_heads(dq, "dq", dev, q.shape), *_heads(dk, "dk", dev, k.shape),
                  *_heads(dv, "dv", dev, v.shape))
    at = ctypes.addressof(h)
    # its own scratch in every call: a captured graph then keeps one of its own
    size = lib.pact_attention_bwd_workspace_size(q.shape[0], q.shape[1], k.shape[0], k.shape[1], D, n)
    ws = torch.empty((size,), dtype=torch.uint8, device=q.device)
    _check(_heads_call(lib, "pact_attention_bwd")(
        at + 96, at, at + 32, at + 64, at + 128, lse.data_ptr(), D, cu_q.data_ptr(), cu_k.data_ptr(),
        n, 1 if causal else 0, scale, at + 160, at + 192, at + 224, ws.data_ptr(), size,
        _raw_stream(dev)))
    return dq, dk, dv


# ------------------------------------------------------------------ gradient norm
class GradList:
    """FP32 tensors whose norm is taken together, listed in device memory once; they keep
    their addresses while the list is in use.  Contiguous, all on the current device, no two
    sharing memory.

    Making a list takes longer than clipping with it (448 tensors 0.35 ms, 14 tensors 40 us, on
    the host, with a copy that waits for the device): it pays for gradients that stay where they
    are, as those that are zeroed or overwritten in place do, not for new tensors each step."""

    def __init__(self, tensors):
        lib = _LIB or load_library()
        self.tensors = tuple(tensors)
        if not self.tensors:
            raise ValueError("a gradient list needs at least one tensor")
        self.device = dev = torch.cuda.current_device()
        f32 = torch.float32
        for i, t in enumerate(self.tensors):
            if not (isinstance(t, torch.Tensor) and t.dtype is f32 and t.get_device() == dev
                    and t.is_contiguous()):
                _need(t, f32, tuple(t.shape) if isinstance(t, torch.Tensor) else (), f"tensor {i}", dev)
        ptrs = [t.data_ptr() for t in self.tensors]
        self.numels = tuple(t.numel() for t in self.tensors)
        spans = sorted((a, n) for a, n in zip(ptrs, self.numels) if n)
        if any(a + 4 * n > b for (a, n), (b, _) in zip(spans, spans[1:])):
            raise ValueError("the tensors of a gradient list must not share memory")
        chunks = {n: lib.pact_grad_chunks(n) for n in set(self.numels)}
        first = [0, *itertools.accumulate(chunks[n] for n in self.numels)]
        self.chunks = first.pop()
        table = array.array("q", itertools.chain(ptrs, self.numels, first))
        self._table = torch.frombuffer(table, dtype=torch.int64).to(f"cuda:{dev}")
        step = 8 * len(self.tensors)
        self.data = self._table.data_ptr()
        self._struct = _ListStruct(self.data, self.data + step, self.data + 2 * step,
                                   len(self.tensors), self.chunks)


def _need_list(g, name, dev):
    if not isinstance(g, GradList):
        raise ValueError(f"{name} must be a GradList, got {type(g).__name__}")
    if g.device != dev:
        raise ValueError(f"{name} is on cuda:{g.device}, the current device is cuda:{dev}")


def _grad_scratch(grads, norm, dev, lib):
    if norm is None:
        norm = torch.empty((1,), dtype=torch.float32, device=grads._table.device)
    _need(norm, torch.float32, (1,), "norm", dev)
    # its own scratch in every call: a captured graph then keeps one of its own
    return norm, torch.empty((lib.pact_grad_norm_workspace_size(),), dtype=torch.uint8,
                             device=norm.device)


def pact_grad_norm(grads: GradList, norm: torch.Tensor | None = None) -> torch.Tensor:
    """The square root of the sum of all values' squares, FP32 [1]."""
    lib = _LIB or load_library()
    dev = torch.cuda.current_device()
    _need_list(grads, "grads", dev)
    norm, ws = _grad_scratch(grads, norm, dev, lib)
    _check(lib.pact_grad_norm(grads._struct, _addr(norm), _addr(ws), ws.numel(), _raw_stream(dev)))
    return norm


def pact_clip_grad_norm(grads: GradList, max_norm: float, norm: torch.Tensor | None = None,
                        out: GradList | None = None) -> torch.Tensor:
    """Scale every value by min(1, max_norm / (norm + 1e-6)), in place or into `out`: a list
    of the same sizes, each of whose tensors is its counterpart in grads or shares no memory
    with any tensor of the two.  Returns the norm before clipping, FP32 [1]."""
    lib = _LIB or load_library()
    dev = torch.cuda.current_device()
    _need_list(grads, "grads", dev)
    if out is None:
        out = grads
    elif out is not grads:
        _need_list(out, "out", dev)
        if out.numels != grads.numels:
            raise ValueError("out must list tensors of the same sizes as grads")
    norm, ws = _grad_scratch(grads, norm, dev, lib)
    _check(lib.pact_clip_grad_norm(grads._struct, out.data, float(max_norm), _addr(norm), _addr(ws),
                                   ws.numel(), _raw_stream(dev)))
    return norm


def pact_test_fp8_plan(rows: int, n: int, k: int, sms: int = 152) -> tuple:
    """How the FP8 product runs these sizes on a device of so many SMs: (way, CTAs or warps,
    tiles before a last wave of halves).  Host arithmetic only."""
    plan = (_i64 * 3)()
    _check((_LIB or load_library()).pact_test_fp8_plan(rows, n, k, sms, plan))
    return ("few", "tiles", "shared", "pairs")[plan[0]], plan[1], plan[2]


def pact_test_pexp(x: torch.Tensor) -> torch.Tensor:
    """The FP32 exp recipe used inside the SiLU kernels, element-wise on the GPU."""
    lib = load_library()
    _need_cuda(x, torch.float32, "x")
    y = torch.empty_like(x)
    _check(lib.pact_test_pexp(_ptr(x), _ptr(y), x.numel(), _stream()))
    return y


def pact_test_wait_timeout(limit_us: int = 1000) -> None:
    """Launch a kernel whose bounded wait runs out after limit_us microseconds; the
    next pact_check_status() raises PactError with code PACT_ERR_TIMEOUT (6)."""
    _check(load_library().pact_test_wait_timeout(int(limit_us), _stream()))


def pact_test_bounds_check() -> None:
    """Evaluate one failing bounds check on the GPU (no memory access): with the debug
    library the next pact_check_status() raises PactError (PACT_ERR_DEVICE_STATUS);
    with the release library it passes."""
    _check(load_library().pact_test_bounds_check(_stream()))


def pact_version() -> str:
    return load_library().pact_version().decode()


def pact_check_status() -> None:
    """Synchronise the current stream and raise if a kernel recorded an error."""
    _check(load_library().pact_check_status(_stream()))


def pact_device_supported() -> bool:
    return load_library().pact_device_supported() == 0


def pact_launch_count() -> int:
    """Number of libpact kernels launched by this process so far."""
    return int(load_library().pact_launch_count())


def pact_profile_next_gemm(begin: torch.cuda.Event, end: torch.cuda.Event) -> None:
    """Record begin/end on the launch stream around the next NVFP4 GEMM kernel."""
    _check(load_library().pact_profile_next_gemm(ctypes.c_void_p(begin.cuda_event),
                                                 ctypes.c_void_p(end.cuda_event)))
