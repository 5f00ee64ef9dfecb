"""Python binding of libnvfp4.so (include/nvfp4.h): the NVFP4 W4A4 linear
and MLP hot path on one sm_103a GPU.

Argument marshalling only: every step of the path runs in the library's CUDA
kernels.  torch provides device memory and streams.  If the library has not
been built (``python -c "import __graft_entry__ as g; g.build()"``) every
call raises; there is no fallback.

Function names match the C ABI.  Tensors are CUDA torch tensors:
  bf16 matrices: torch.bfloat16, row-major (a row pitch is taken from
  ``stride(0)``); quantized matrices: :class:`NVFP4Tensor`.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from dataclasses import dataclass

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libnvfp4.so")

NVFP4_OK = 0
NVFP4_ERR_TIMEOUT = 6        # device-side: a bounded wait ran out (status word: 6 * 100 + site)
NVFP4_INTER_STATIC = 0
NVFP4_INTER_DYNAMIC = 1

_lock = threading.Lock()
_lib = None


class _TensorC(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("sf", ctypes.c_void_p), ("g", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("ld", ctypes.c_int64)]


class _RopeC(ctypes.Structure):
    _fields_ = [("pos", ctypes.c_void_p), ("cos_t", ctypes.c_void_p), ("sin_t", ctypes.c_void_p),
                ("table_ld", ctypes.c_int64), ("positions", ctypes.c_int64), ("col0", ctypes.c_int64),
                ("heads", ctypes.c_int64), ("head_dim", ctypes.c_int64), ("rope_dim", ctypes.c_int64),
                ("inverse", ctypes.c_int)]


class _StepC(ctypes.Structure):
    _fields_ = [("requests", ctypes.c_int64), ("tokens", ctypes.c_int64), ("q_len", ctypes.c_void_p),
                ("ctx_len", ctypes.c_void_p), ("cu_q", ctypes.c_void_p), ("kv_len", ctypes.c_void_p),
                ("pos", ctypes.c_void_p), ("page_size", ctypes.c_int64), ("block_table", ctypes.c_void_p),
                ("table_cols", ctypes.c_int64), ("table_ld", ctypes.c_int64), ("slot", ctypes.c_void_p),
                ("free_pages", ctypes.c_void_p), ("free_count", ctypes.c_int64), ("cursor", ctypes.c_void_p),
                ("cursor_out", ctypes.c_void_p), ("heads", ctypes.c_int64), ("kv_heads", ctypes.c_int64),
                ("window", ctypes.c_int64), ("schedule", ctypes.c_void_p), ("schedule_bytes", ctypes.c_size_t)]


class _CacheC(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("pages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("kv_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("page_stride", ctypes.c_int64)]


class _AttnIOC(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("ldq", ctypes.c_int64), ("hq", ctypes.c_int64), ("out", ctypes.c_void_p),
                ("ldo", ctypes.c_int64), ("ho", ctypes.c_int64), ("lse", ctypes.c_void_p),
                ("head_dim", ctypes.c_int64), ("scale", ctypes.c_float), ("zero_padding", ctypes.c_int32)]


class _Cache4C(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_sf", ctypes.c_void_p), ("v_sf", ctypes.c_void_p),
                ("k_g", ctypes.c_void_p), ("v_g", ctypes.c_void_p), ("pages", ctypes.c_int64),
                ("page_size", ctypes.c_int64), ("kv_heads", ctypes.c_int64), ("head_dim", ctypes.c_int64),
                ("page_stride", ctypes.c_int64), ("sf_stride", ctypes.c_int64)]


class _HeadsC(ctypes.Structure):
    _fields_ = [("tokens", ctypes.c_int64), ("heads", ctypes.c_int64), ("kv_heads", ctypes.c_int64),
                ("head_dim", ctypes.c_int64), ("q", ctypes.c_void_p), ("ldq", ctypes.c_int64), ("hq", ctypes.c_int64),
                ("q_out", ctypes.c_void_p), ("ldqo", ctypes.c_int64), ("hqo", ctypes.c_int64), ("k", ctypes.c_void_p),
                ("ldk", ctypes.c_int64), ("hk", ctypes.c_int64), ("k_out", ctypes.c_void_p), ("ldko", ctypes.c_int64),
                ("hko", ctypes.c_int64), ("q_norm", ctypes.c_void_p), ("k_norm", ctypes.c_void_p),
                ("eps", ctypes.c_float), ("pos", ctypes.c_void_p), ("cos_t", ctypes.c_void_p),
                ("sin_t", ctypes.c_void_p), ("table_ld", ctypes.c_int64), ("positions", ctypes.c_int64),
                ("rope_dim", ctypes.c_int64), ("halves", ctypes.c_int32), ("slot", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("ldv", ctypes.c_int64), ("hv", ctypes.c_int64),
                ("cache", ctypes.c_void_p), ("cache4", ctypes.c_void_p)]


# The bytes of a structure for less than making it (nvfp4_heads_t 0.3 us, 1.5).
_pack_io = struct.Struct("@PqqPqqPqfi").pack
_pack_plane = struct.Struct("@Pqq").pack
_pack_heads = struct.Struct("@4q" + 4 * "Pqq" + "PPfPPPqqqiPPqqPP").pack


class _PagesC(ctypes.Structure):
    _fields_ = [("block_table", ctypes.c_void_p), ("requests", ctypes.c_int64), ("table_cols", ctypes.c_int64),
                ("table_ld", ctypes.c_int64), ("ctx_len", ctypes.c_void_p), ("page_size", ctypes.c_int64),
                ("pages", ctypes.c_int64)]


class _PlaneC(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("page_bytes", ctypes.c_int64), ("page_stride", ctypes.c_int64)]


_SIGS = {
    "nvfp4_codes_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    "nvfp4_sf_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64]),
    "nvfp4_amax_workspace_bytes": (ctypes.c_size_t, []),
    "nvfp4_gemm_workspace_bytes": (ctypes.c_size_t, []),
    "nvfp4_swiglu_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int]),
    "nvfp4_mlp_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int]),
    "nvfp4_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "nvfp4_device_status": (ctypes.c_int, [ctypes.POINTER(ctypes.c_int), ctypes.c_int]),
    "nvfp4_mma_issue_rate": (ctypes.c_int, [ctypes.POINTER(ctypes.c_double)]),
    "nvfp4_noalloc_scratch": (ctypes.c_int, [ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ctypes.c_size_t)]),
    "nvfp4_experts_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                                        ctypes.c_int64]),
    "nvfp4_gemm_experts": (ctypes.c_int, [ctypes.POINTER(_TensorC), ctypes.POINTER(_TensorC), ctypes.c_int64,
                                          ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                          ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "nvfp4_amax_scale": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                        ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_size_t, ctypes.c_void_p]),
    "nvfp4_quantize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                      ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                                      ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "nvfp4_scale_quantize": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                            ctypes.c_void_p, ctypes.c_float, ctypes.c_void_p, ctypes.c_void_p,
                                            ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_size_t,
                                            ctypes.c_void_p]),
    "nvfp4_gemm": (ctypes.c_int, [ctypes.POINTER(_TensorC), ctypes.POINTER(_TensorC), ctypes.c_void_p,
                                  ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p,
                                  ctypes.c_size_t, ctypes.c_void_p]),
    "nvfp4_gemm_rope": (ctypes.c_int, [ctypes.POINTER(_TensorC), ctypes.POINTER(_TensorC), ctypes.c_void_p,
                                       ctypes.c_int64, ctypes.POINTER(_RopeC), ctypes.c_void_p, ctypes.c_size_t,
                                       ctypes.c_void_p]),
    "nvfp4_gemm_swiglu": (ctypes.c_int, [ctypes.POINTER(_TensorC), ctypes.POINTER(_TensorC),
                                         ctypes.POINTER(_TensorC), ctypes.c_int, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                         ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "nvfp4_mlp": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                 ctypes.c_void_p, ctypes.c_float, ctypes.POINTER(_TensorC),
                                 ctypes.POINTER(_TensorC), ctypes.POINTER(_TensorC), ctypes.c_int,
                                 ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                 ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "nvfp4_mlp_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                         ctypes.c_void_p, ctypes.c_float, ctypes.POINTER(_TensorC),
                                         ctypes.POINTER(_TensorC), ctypes.POINTER(_TensorC), ctypes.c_int,
                                         ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64, ctypes.c_int,
                                         ctypes.c_void_p]),
    "nvfp4_attn_schedule_bytes": (ctypes.c_size_t, [ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64]),
    "nvfp4_attn_workspace_bytes": (ctypes.c_size_t, []),
    "nvfp4_attn_plan": (ctypes.c_int, [ctypes.POINTER(_StepC), ctypes.c_void_p]),
    "nvfp4_kv_append": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                       ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                       ctypes.POINTER(_CacheC), ctypes.c_void_p]),
    "nvfp4_attn_prompt": (ctypes.c_int, [ctypes.POINTER(_StepC), ctypes.POINTER(_AttnIOC), ctypes.c_void_p,
                                         ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                         ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "nvfp4_attn_paged": (ctypes.c_int, [ctypes.POINTER(_StepC), ctypes.POINTER(_AttnIOC), ctypes.POINTER(_CacheC),
                                        ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "nvfp4_qk_norm_rope": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p]),
    "nvfp4_kv4_append": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                        ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p, ctypes.c_int64,
                                        ctypes.POINTER(_Cache4C), ctypes.c_void_p]),
    "nvfp4_kv4_expand": (ctypes.c_int, [ctypes.POINTER(_Cache4C), ctypes.POINTER(_StepC), ctypes.POINTER(_CacheC),
                                        ctypes.c_void_p]),
    "nvfp4_attn_paged4": (ctypes.c_int, [ctypes.POINTER(_StepC), ctypes.c_void_p, ctypes.POINTER(_Cache4C),
                                         ctypes.POINTER(_CacheC), ctypes.c_void_p, ctypes.c_size_t, ctypes.c_void_p]),
    "nvfp4_pages_fork": (ctypes.c_int, [ctypes.POINTER(_PagesC), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int64,
                                        ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "nvfp4_pages_free": (ctypes.c_int, [ctypes.POINTER(_PagesC), ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                        ctypes.c_int64, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "nvfp4_pages_copy": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64, ctypes.c_void_p,
                                        ctypes.c_void_p, ctypes.c_int64, ctypes.c_void_p]),
}

EXPORTED_FUNCTIONS = tuple(_SIGS)


def lib(path: str | None = None):
    """Load libnvfp4.so (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None or path is not None:
            p = path or LIB_PATH
            if not os.path.exists(p):
                raise RuntimeError(f"{p} is missing: build it with nvfp4_block_scaled_device_gb300.build.build()")
            L = ctypes.CDLL(p)
            for name, (res, args) in _SIGS.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            if path is not None:
                return L
            _lib = L
    return _lib


class NVFP4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        msg = lib().nvfp4_status_string(status).decode()
        super().__init__(f"{where}: {msg} (status {status})")
        self.status = status


def _check(status: int, where: str):
    if status != NVFP4_OK:
        raise NVFP4Error(status, where)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:               # the current stream's handle, without a Stream object around it (3 us)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return ctypes.c_void_p(stream.cuda_stream)


def _bf16_2d(x: torch.Tensor, name: str):
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.stride(1) != 1 or not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA bf16 matrix with unit column stride")
    return x.shape[0], x.shape[1], x.stride(0)


# ------------------------------------------------------------ host helpers
def codes_bytes(rows: int, cols: int) -> int:
    return int(lib().nvfp4_codes_bytes(rows, cols))


def sf_bytes(rows: int, cols: int) -> int:
    return int(lib().nvfp4_sf_bytes(rows, cols))


def amax_workspace_bytes() -> int:
    return int(lib().nvfp4_amax_workspace_bytes())


def gemm_workspace_bytes() -> int:
    return int(lib().nvfp4_gemm_workspace_bytes())


def swiglu_workspace_bytes(T: int, I: int, inter_mode: int) -> int:
    return int(lib().nvfp4_swiglu_workspace_bytes(T, I, inter_mode))


def mlp_workspace_bytes(T: int, H: int, I: int, inter_mode: int) -> int:
    return int(lib().nvfp4_mlp_workspace_bytes(T, H, I, inter_mode))


def device_status(clear: bool = True) -> int:
    """Device-side status word (synchronous; diagnostics and tests)."""
    v = ctypes.c_int(0)
    _check(lib().nvfp4_device_status(ctypes.byref(v), int(clear)), "nvfp4_device_status")
    return v.value


def mma_issue_rate() -> float:
    """Multiply-adds per SM per clock of the GEMMs' block-scaled MMA form,
    measured on the current device (synchronous; a measurement diagnostic)."""
    v = ctypes.c_double(0.0)
    _check(lib().nvfp4_mma_issue_rate(ctypes.byref(v)), "nvfp4_mma_issue_rate")
    return v.value


def workspace(nbytes: int, device=None) -> torch.Tensor:
    """A zero-filled workspace buffer (torch's allocator aligns to >= 256 B)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device or "cuda")


@dataclass
class NVFP4Tensor:
    """A quantized [rows x cols] matrix on the device: codes uint8 [rows, cols/2],
    swizzled scales uint8 [sf_bytes(rows, cols)], global scale float32 [1]."""
    codes: torch.Tensor
    sf: torch.Tensor
    g: torch.Tensor
    rows: int
    cols: int

    @staticmethod
    def empty(rows: int, cols: int, device=None) -> "NVFP4Tensor":
        device = device or "cuda"
        return NVFP4Tensor(
            codes=torch.empty((rows, cols // 2), dtype=torch.uint8, device=device),
            sf=torch.zeros((sf_bytes(rows, cols),), dtype=torch.uint8, device=device),
            g=torch.zeros((1,), dtype=torch.float32, device=device),
            rows=rows, cols=cols)

    def c(self) -> _TensorC:
        return _TensorC(self.codes.data_ptr(), self.sf.data_ptr(), self.g.data_ptr(),
                        self.rows, self.cols, self.codes.stride(0))


# -------------------------------------------------------------- the path
def nvfp4_amax_scale(x: torch.Tensor, g_out: torch.Tensor, ws: torch.Tensor, norm_w=None, eps=1e-6,
                     stream=None):
    rows, cols, ldx = _bf16_2d(x, "x")
    _check(lib().nvfp4_amax_scale(_ptr(x), rows, cols, ldx, _ptr(norm_w), eps, _ptr(g_out), _ptr(ws),
                                  ws.numel() * ws.element_size(), _stream(stream)), "nvfp4_amax_scale")


def nvfp4_quantize(x: torch.Tensor, g: torch.Tensor, out: NVFP4Tensor, norm_w=None, eps=1e-6, y_out=None,
                   stream=None):
    rows, cols, ldx = _bf16_2d(x, "x")
    _check(lib().nvfp4_quantize(_ptr(x), rows, cols, ldx, _ptr(norm_w), eps, _ptr(g), _ptr(out.codes),
                                out.codes.stride(0), _ptr(out.sf), _ptr(y_out), _stream(stream)),
           "nvfp4_quantize")


def nvfp4_scale_quantize(x: torch.Tensor, out: NVFP4Tensor, ws: torch.Tensor, norm_w=None, eps=1e-6, stream=None):
    """Global scale into out.g and quantization into out, in one launch."""
    rows, cols, ldx = _bf16_2d(x, "x")
    _check(lib().nvfp4_scale_quantize(_ptr(x), rows, cols, ldx, _ptr(norm_w), eps, _ptr(out.g), _ptr(out.codes),
                                      out.codes.stride(0), _ptr(out.sf), _ptr(ws), ws.numel() * ws.element_size(),
                                      _stream(stream)), "nvfp4_scale_quantize")


def quantize_new(x: torch.Tensor, ws: torch.Tensor, norm_w=None, eps=1e-6, stream=None) -> NVFP4Tensor:
    """Global scale + quantization of x into a newly allocated NVFP4Tensor."""
    t = NVFP4Tensor.empty(x.shape[0], x.shape[1], x.device)
    nvfp4_amax_scale(x, t.g, ws, norm_w, eps, stream)
    nvfp4_quantize(x, t.g, t, norm_w, eps, None, stream)
    return t


def nvfp4_gemm(A: NVFP4Tensor, W: NVFP4Tensor, out: torch.Tensor, residual=None, stream=None, workspace=None):
    """workspace: None, or a zero-filled uint8 tensor (see workspace()) of
    gemm_workspace_bytes() bytes that lets the GEMM split tiles over all SMs."""
    _, _, ldo = _bf16_2d(out, "out")
    ldr = _bf16_2d(residual, "residual")[2] if residual is not None else 0
    a, w = A.c(), W.c()
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().nvfp4_gemm(ctypes.byref(a), ctypes.byref(w), _ptr(out), ldo, _ptr(residual), ldr,
                            _ptr(workspace), nbytes, _stream(stream)), "nvfp4_gemm")


def nvfp4_gemm_rope(A: NVFP4Tensor, W: NVFP4Tensor, out: torch.Tensor, pos: torch.Tensor, cos_t: torch.Tensor,
                    sin_t: torch.Tensor, col0: int, heads: int, head_dim: int, rope_dim: int, inverse=False,
                    stream=None, workspace=None):
    """nvfp4_gemm with the rotary embedding in its epilogue.  pos: int32
    [M] on the device; cos_t, sin_t: float32 [positions, >= rope_dim/2] on
    the device (row-major, the same shape)."""
    _, _, ldo = _bf16_2d(out, "out")
    if pos.dtype != torch.int32 or cos_t.dtype != torch.float32 or sin_t.dtype != torch.float32:
        raise TypeError("pos must be int32, cos_t and sin_t float32")
    if cos_t.shape != sin_t.shape or cos_t.dim() != 2 or cos_t.stride(1) != 1 or sin_t.stride() != cos_t.stride():
        raise ValueError("cos_t and sin_t must be row-major 2-D tensors of one shape")
    r = _RopeC(pos.data_ptr(), cos_t.data_ptr(), sin_t.data_ptr(), cos_t.stride(0), cos_t.shape[0], col0, heads,
               head_dim, rope_dim, int(bool(inverse)))
    a, w = A.c(), W.c()
    nbytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().nvfp4_gemm_rope(ctypes.byref(a), ctypes.byref(w), _ptr(out), ldo, ctypes.byref(r),
                                 _ptr(workspace), nbytes, _stream(stream)), "nvfp4_gemm_rope")


def nvfp4_gemm_swiglu(A: NVFP4Tensor, W_gate: NVFP4Tensor, W_up: NVFP4Tensor, inter_mode: int,
                      g_inter: torch.Tensor, s_out: NVFP4Tensor, ws: torch.Tensor, s_bf16=None, stream=None):
    a, wg, wu = A.c(), W_gate.c(), W_up.c()
    _check(lib().nvfp4_gemm_swiglu(ctypes.byref(a), ctypes.byref(wg), ctypes.byref(wu), inter_mode,
                                   _ptr(g_inter), _ptr(s_out.codes), s_out.codes.stride(0), _ptr(s_out.sf),
                                   _ptr(s_bf16), _ptr(ws), ws.numel(), _stream(stream)), "nvfp4_gemm_swiglu")


def nvfp4_mlp_noalloc(x: torch.Tensor, norm_w: torch.Tensor, W_gate: NVFP4Tensor, W_up: NVFP4Tensor,
                      W_down: NVFP4Tensor, inter_mode: int, g_inter: torch.Tensor, out: torch.Tensor,
                      add_residual=True, eps=1e-6, stream=None):
    """nvfp4_mlp without a workspace (the library's fixed scratch array; for
    callers that cannot allocate device memory -- see include/nvfp4.h)."""
    T, H, ldx = _bf16_2d(x, "x")
    _, _, ldo = _bf16_2d(out, "out")
    wg, wu, wd = W_gate.c(), W_up.c(), W_down.c()
    _check(lib().nvfp4_mlp_noalloc(_ptr(x), T, H, ldx, _ptr(norm_w), eps, ctypes.byref(wg), ctypes.byref(wu),
                                   ctypes.byref(wd), inter_mode, _ptr(g_inter), _ptr(out), ldo,
                                   int(bool(add_residual)), _stream(stream)), "nvfp4_mlp_noalloc")


def noalloc_scratch():
    """(device address, bytes) of nvfp4_mlp_noalloc's fixed array on the
    current device (diagnostics and tests)."""
    p, n = ctypes.c_void_p(0), ctypes.c_size_t(0)
    _check(lib().nvfp4_noalloc_scratch(ctypes.byref(p), ctypes.byref(n)), "nvfp4_noalloc_scratch")
    return int(p.value or 0), int(n.value)


def nvfp4_mlp(x: torch.Tensor, norm_w: torch.Tensor, W_gate: NVFP4Tensor, W_up: NVFP4Tensor,
              W_down: NVFP4Tensor, inter_mode: int, g_inter: torch.Tensor, out: torch.Tensor,
              ws: torch.Tensor, add_residual=True, eps=1e-6, stream=None):
    T, H, ldx = _bf16_2d(x, "x")
    _, _, ldo = _bf16_2d(out, "out")
    wg, wu, wd = W_gate.c(), W_up.c(), W_down.c()
    _check(lib().nvfp4_mlp(_ptr(x), T, H, ldx, _ptr(norm_w), eps, ctypes.byref(wg), ctypes.byref(wu),
                           ctypes.byref(wd), inter_mode, _ptr(g_inter), _ptr(out), ldo, int(bool(add_residual)),
                           _ptr(ws), ws.numel(), _stream(stream)), "nvfp4_mlp")


def experts_workspace_bytes(T: int, topk: int, K: int, num_experts: int) -> int:
    return int(lib().nvfp4_experts_workspace_bytes(T, topk, K, num_experts))


def nvfp4_gemm_experts(A: NVFP4Tensor, W: NVFP4Tensor, num_experts: int, ids: torch.Tensor, out: torch.Tensor,
                       ws: torch.Tensor, stream=None):
    """Expert-indexed GEMM.  W: the experts' weights stacked (rows = E * N,
    W.g fp32[E]); ids: CUDA int32 [T, topk] (or [T * topk]); out: bf16
    [T * topk, N], row t * topk + j for token t, slot j."""
    if ids.dtype != torch.int32 or not ids.is_cuda or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous CUDA int32 tensor")
    topk = ids.shape[1] if ids.dim() == 2 else ids.numel() // A.rows
    _, _, ldo = _bf16_2d(out, "out")
    a, w = A.c(), W.c()
    _check(lib().nvfp4_gemm_experts(ctypes.byref(a), ctypes.byref(w), num_experts, _ptr(ids), topk, _ptr(out), ldo,
                                    _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)), "nvfp4_gemm_experts")


# ------------------------------------------------ attention over a KV cache
# (The calls of a decode step cost the host more than the GPU: these functions
# look at what they are given once and build nothing that they can do without.)
def _i32(t, n, name):
    if t.dtype is not _I32 or not t.is_cuda or not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"{name} must be a contiguous CUDA int32 tensor of at least {n} elements")
    return t.data_ptr()


_BF16, _I32 = torch.bfloat16, torch.int32


def _heads_3d(x: torch.Tensor, name: str, tokens: int, heads: int, head_dim: int):
    """(address, row pitch, head pitch) of bf16 [tokens, heads, head_dim] with unit column stride."""
    st = x.stride()
    if x.dtype is not _BF16 or x.shape != (tokens, heads, head_dim) or st[2] != 1 or not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA bf16 [{tokens}, {heads}, {head_dim}] tensor with unit column stride, "
                         f"not {x.dtype} {tuple(x.shape)} on {x.device}")
    return x.data_ptr(), st[0], st[1]


def attn_schedule_bytes(requests: int, tokens: int, heads: int, kv_heads: int) -> int:
    return int(lib().nvfp4_attn_schedule_bytes(requests, tokens, heads, kv_heads))


def attn_workspace_bytes() -> int:
    return int(lib().nvfp4_attn_workspace_bytes())


class KVCache:
    """A paged KV cache: bf16 ``k`` and ``v`` of shape [pages, kv_heads,
    page_size, head_dim].  Pages may be apart (stride(0), e.g. the two halves
    of one [pages, 2, ...] tensor); within a page they are contiguous."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        for name, t in (("k", k), ("v", v)):
            if t.dtype != torch.bfloat16 or t.dim() != 4 or not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA bf16 [pages, kv_heads, page_size, head_dim] tensor")
            if t.stride()[1:] != (t.shape[2] * t.shape[3], t.shape[3], 1):
                raise ValueError(f"{name}'s pages must be contiguous")
        if k.shape != v.shape or (k.stride(0) != v.stride(0) and k.shape[0] > 1):
            raise ValueError("k and v must have one shape and one page stride")
        self.k, self.v = k, v
        self.pages, self.kv_heads, self.page_size, self.head_dim = k.shape
        page = self.kv_heads * self.page_size * self.head_dim
        self._c = _CacheC(k.data_ptr(), v.data_ptr(), self.pages, self.page_size, self.kv_heads, self.head_dim,
                          k.stride(0) if self.pages > 1 else page)
        self._planes = b"".join(_pack_plane(t.data_ptr(), 2 * page, 2 * self._c.page_stride) for t in (k, v))
        self._device = k.get_device()

    @staticmethod
    def empty(pages: int, kv_heads: int, page_size: int, head_dim: int, device=None) -> "KVCache":
        k, v = (torch.empty((pages, kv_heads, page_size, head_dim), dtype=torch.bfloat16, device=device or "cuda")
                for _ in range(2))
        return KVCache(k, v)


class AttnPlan:
    """The tables of one serving step (see nvfp4_step_t), in buffers that
    stay: cu_q int32 [requests + 1], kv_len int32 [requests], pos and slot
    int32 [tokens], block_table int32 [requests, pages per request], cursor
    int32 [1] (the free list's cursor after the step), and the attention's
    schedule.  Filled by :func:`nvfp4_attn_plan`, once per step; read by every
    layer's :func:`nvfp4_kv_append`, :func:`nvfp4_attn_paged` and
    :func:`nvfp4_attn_prompt`, and ``pos`` by :func:`nvfp4_gemm_rope`.

    requests, tokens: the most a step has (tokens: the rows of its matrices).
    page_size and block_table: for a paged cache; block_table (or the
    columns of a new one, all -1) holds the pages of the cached tokens.
    window: keys a row sees, its own included (0: all up to its own)."""

    def __init__(self, requests: int, tokens: int, heads: int, kv_heads: int, page_size: int = 0, block_table=None,
                 window: int = 0, device=None):
        self.requests, self.tokens, self.heads, self.kv_heads = requests, tokens, heads, kv_heads
        self.page_size, self.window = page_size, window
        if isinstance(block_table, torch.Tensor):
            if block_table.dim() == 2 and requests > 1 and block_table.stride(0) < block_table.shape[1]:
                raise ValueError("block_table's rows overlap (an expanded tensor has to be made contiguous)")
            if block_table.dtype != torch.int32 or not block_table.is_cuda or block_table.dim() != 2 or \
                    block_table.shape[0] < requests or block_table.stride(1) != 1:
                raise ValueError("block_table must be a CUDA int32 [requests, pages] tensor with unit column stride")
            device = block_table.device
        device = device or "cuda"
        empty = lambda n: torch.empty((n,), dtype=torch.int32, device=device)
        self.cu_q, self.kv_len, self.pos = empty(requests + 1), empty(requests), empty(tokens)
        self.slot = self.block_table = self.cursor = None
        if page_size:
            if not isinstance(block_table, torch.Tensor):
                block_table = torch.full((requests, int(block_table)), -1, dtype=torch.int32, device=device)
            self.block_table = block_table
            self.slot, self.cursor = empty(tokens), torch.zeros((1,), dtype=torch.int32, device=device)
        nbytes = attn_schedule_bytes(requests, tokens, heads, kv_heads)
        self.schedule = torch.zeros((max(nbytes, 1),), dtype=torch.uint8, device=device)
        t = self.block_table
        self._c = _StepC(requests, tokens, None, None, self.cu_q.data_ptr(), self.kv_len.data_ptr(),
                         self.pos.data_ptr(), page_size, None if t is None else t.data_ptr(),
                         0 if t is None else t.shape[1], 0 if t is None else max(t.stride(0), t.shape[1]),
                         None if t is None else self.slot.data_ptr(), None, 0, None,
                         None if t is None else self.cursor.data_ptr(), heads, kv_heads, window,
                         self.schedule.data_ptr(), nbytes)


def nvfp4_attn_plan(plan: AttnPlan, q_len: torch.Tensor, ctx_len=None, free_pages=None, cursor=None, stream=None):
    """The step's tables from its lengths: q_len, ctx_len int32 [requests]
    on the device; free_pages int32 and cursor int32 [1] (the entries of
    free_pages already taken; None: 0) for the pages the new tokens open, or
    None where block_table holds them already."""
    c = plan._c
    c.q_len = _i32(q_len, plan.requests, "q_len")
    c.ctx_len = None if ctx_len is None else _i32(ctx_len, plan.requests, "ctx_len")
    if free_pages is not None:
        c.free_pages, c.free_count = _i32(free_pages, 0, "free_pages"), free_pages.numel()
    else:
        c.free_pages, c.free_count = None, 0
    c.cursor = None if cursor is None else _i32(cursor, 1, "cursor")
    _check((_lib or lib()).nvfp4_attn_plan(ctypes.byref(c), _stream(stream)), "nvfp4_attn_plan")


def nvfp4_kv_append(k: torch.Tensor, v: torch.Tensor, plan: AttnPlan, cache: KVCache, stream=None):
    """k, v: bf16 [tokens, kv_heads, head_dim] (any row and head pitch, e.g.
    column slices of a QKV projection's output) into the cache's slots plan.slot."""
    if plan.slot is None:
        raise ValueError("the plan has no paged cache (page_size 0)")
    if plan.page_size != cache.page_size:        # (a slot is page * page_size + row)
        raise ValueError(f"the plan's pages of {plan.page_size} tokens are not the cache's of {cache.page_size}")
    kp = _heads_3d(k, "k", plan.tokens, cache.kv_heads, cache.head_dim)
    vp = _heads_3d(v, "v", plan.tokens, cache.kv_heads, cache.head_dim)
    _check((_lib or lib()).nvfp4_kv_append(*kp, *vp, plan.slot.data_ptr(), plan.tokens, ctypes.byref(cache._c),
                                 _stream(stream)), "nvfp4_kv_append")


def _attn_io(plan: AttnPlan, q: torch.Tensor, out: torch.Tensor, scale, lse, zero_padding) -> _AttnIOC:
    d, tokens, heads = q.shape[-1], plan.tokens, plan.heads
    if lse is None:
        at = None
    elif lse.dtype is torch.float32 and lse.is_contiguous() and lse.is_cuda and lse.numel() == tokens * heads:
        at = lse.data_ptr()
    else:
        raise ValueError("lse must be a contiguous CUDA float32 [tokens, heads] tensor")
    return _AttnIOC(*_heads_3d(q, "q", tokens, heads, d), *_heads_3d(out, "out", tokens, heads, d), at, d,
                    d ** -0.5 if scale is None else scale, 1 if zero_padding else 0)


def nvfp4_attn_prompt(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, plan: AttnPlan, out: torch.Tensor,
                      ws: torch.Tensor, scale=None, lse=None, stream=None, zero_padding=False):
    """Causal attention within packed prompts.  q, out: bf16 [tokens, heads,
    head_dim]; k, v: bf16 [tokens, kv_heads, head_dim] (any row and head
    pitch); scale: head_dim ** -0.5 if None; lse: None or float32 [tokens,
    heads]; ws: a zero-filled workspace of attn_workspace_bytes(); zero_padding:
    rows past the step's last token become 0 in out and -inf in lse (else they
    are not written)."""
    io = _attn_io(plan, q, out, scale, lse, zero_padding)
    kp = _heads_3d(k, "k", plan.tokens, plan.kv_heads, q.shape[2])
    vp = _heads_3d(v, "v", plan.tokens, plan.kv_heads, q.shape[2])
    _check((_lib or lib()).nvfp4_attn_prompt(ctypes.byref(plan._c), ctypes.byref(io), *kp, *vp, ws.data_ptr(),
                                   ws.numel() * ws.element_size(), _stream(stream)), "nvfp4_attn_prompt")


def nvfp4_attn_paged(q: torch.Tensor, cache: KVCache, plan: AttnPlan, out: torch.Tensor, ws: torch.Tensor, scale=None,
                     lse=None, stream=None, zero_padding=False):
    """Attention of a step's new tokens over the paged cache, which holds
    their K and V already.  The rest as :func:`nvfp4_attn_prompt`."""
    io = _attn_io(plan, q, out, scale, lse, zero_padding)
    _check((_lib or lib()).nvfp4_attn_paged(ctypes.byref(plan._c), ctypes.byref(io), ctypes.byref(cache._c), ws.data_ptr(),
                                  ws.numel() * ws.element_size(), _stream(stream)), "nvfp4_attn_paged")


# ------------------------------- heads, the 4-bit cache, pages of a cache
# (These calls refuse tensors that are not on the current device, whose stream
# and library state they would use: get_device() is -1 on the CPU.)
_here, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
_F32 = torch.float32


def _elsewhere(name: str, t: torch.Tensor):
    raise ValueError(f"{name} must be on the current CUDA device, not on {t.device}")


def _stream_of(stream, here: int):
    return _raw_stream(here) if stream is None else stream.cuda_stream


def _rows_of(x: torch.Tensor, name: str, shape, here: int):
    """(address, row pitch, head pitch) of bf16 rows [tokens, heads, head_dim]."""
    st = x.stride()
    if x.dtype is not _BF16 or x.shape != shape or st[2] != 1 or x.get_device() != here:
        raise ValueError(f"{name} must be a bf16 {list(shape)} tensor on the current CUDA device with unit column stride, "
                         f"not {x.dtype} {tuple(x.shape)} on {x.device}")
    return x.data_ptr(), st[0], st[1]


def _ints_of(t, n: int, name: str, here: int):
    if t.dtype is not _I32 or t.get_device() != here or not t.is_contiguous() or t.numel() < n:
        raise ValueError(f"{name} must be a contiguous int32 tensor of at least {n} elements on the current CUDA device")
    return t.data_ptr()


class KVCache4:
    """A paged KV cache in 4 bits (nvfp4_kv4_cache_t): ``k`` and ``v`` uint8
    [pages, kv_heads, page_size, head_dim // 2] (two E2M1 codes to a byte),
    ``k_sf`` and ``v_sf`` uint8 [pages, kv_heads, page_size, head_dim // 16]
    (E4M3), ``k_g`` and ``v_g`` float32 [1], the scales of all keys and of all
    values.  Pages may be apart (stride(0)); within a page they are contiguous."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_sf: torch.Tensor, v_sf: torch.Tensor, k_g: torch.Tensor,
                 v_g: torch.Tensor):
        for name, t in (("k", k), ("v", v), ("k_sf", k_sf), ("v_sf", v_sf)):
            if t.dtype != torch.uint8 or t.dim() != 4 or not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA uint8 [pages, kv_heads, page_size, bytes of a row] tensor")
            if t.stride()[1:] != (t.shape[2] * t.shape[3], t.shape[3], 1):
                raise ValueError(f"{name}'s pages must be contiguous")
        for a, b in ((k, v), (k_sf, v_sf)):
            if a.shape != b.shape or (a.stride(0) != b.stride(0) and a.shape[0] > 1):
                raise ValueError("k and v must have one shape and one page stride")
        if k_sf.shape[:3] != k.shape[:3] or k_sf.shape[3] * 8 != k.shape[3]:
            raise ValueError("a scale for each 16 columns (8 bytes of codes)")
        for name, g in (("k_g", k_g), ("v_g", v_g)):
            if g.dtype != torch.float32 or g.numel() != 1 or not g.is_cuda:
                raise ValueError(f"{name} must be a CUDA float32 tensor of one element")
        self.k, self.v, self.k_sf, self.v_sf, self.k_g, self.v_g = k, v, k_sf, v_sf, k_g, v_g
        self.pages, self.kv_heads, self.page_size = k.shape[:3]
        self.head_dim = 2 * k.shape[3]
        stride = lambda t: t.stride(0) if self.pages > 1 else t.shape[1] * t.shape[2] * t.shape[3]
        self._c = _Cache4C(k.data_ptr(), v.data_ptr(), k_sf.data_ptr(), v_sf.data_ptr(), k_g.data_ptr(),
                           v_g.data_ptr(), self.pages, self.page_size, self.kv_heads, self.head_dim, stride(k),
                           stride(k_sf))
        self._planes = b"".join(_pack_plane(t.data_ptr(), t.shape[1] * t.shape[2] * t.shape[3], stride(t))
                                for t in (k, v, k_sf, v_sf))
        self._device = k.get_device()
        if any(t.get_device() != self._device for t in (v, k_sf, v_sf, k_g, v_g)):
            raise ValueError("k, v, their scales and k_g, v_g must be on one device")

    @staticmethod
    def empty(pages: int, kv_heads: int, page_size: int, head_dim: int, k_g=2.0 ** -6, v_g=2.0 ** -6,
              device=None) -> "KVCache4":
        """k_g, v_g: the scales (a power of two near the largest magnitude / 2688
        loses nothing by them); 2^-6 reaches to 42, with full precision down to
        blocks whose largest magnitude is 0.0015."""
        make = lambda n: torch.empty((pages, kv_heads, page_size, n), dtype=torch.uint8, device=device or "cuda")
        scale = lambda g: torch.full((1,), g, dtype=torch.float32, device=device or "cuda")
        return KVCache4(make(head_dim // 2), make(head_dim // 2), make(head_dim // 16), make(head_dim // 16), scale(k_g),
                        scale(v_g))


def _cache_fits(plan: AttnPlan, cache, name="cache"):
    if plan.slot is None:
        raise ValueError("the plan has no paged cache (page_size 0)")
    if plan.page_size != cache.page_size:        # (a slot is page * page_size + row)
        raise ValueError(f"the plan's pages of {plan.page_size} tokens are not the {name}'s of {cache.page_size}")


def nvfp4_qk_norm_rope(q, k, q_norm=None, k_norm=None, pos=None, cos_t=None, sin_t=None, q_out=None, k_out=None,
                       halves=False, eps=1e-6, rope_dim=None, v=None, plan=None, cache=None, stream=None):
    """RMSNorm of each head of q [tokens, heads, head_dim] and k [tokens,
    kv_heads, head_dim] (bf16, any row and head pitch; either may be None) and
    their rotation, in one pass.  q_norm, k_norm: bf16 [head_dim], None for no
    norm.  pos int32 [tokens], cos_t and sin_t float32 [positions, >= rope_dim /
    2]; None for no rotation.  rope_dim: the last columns of a head that are
    rotated (None: twice the tables' width); halves: pairs (i, i + rope_dim / 2)
    instead of (2i, 2i + 1).  q_out, k_out: where the rows go (None: in place).

    With v, plan and cache (KVCache or KVCache4) the rows of k, and those of v,
    go into the cache's slots plan.slot instead (and to k_out where it is given)."""
    ref = k if q is None else q
    if ref is None:
        raise ValueError("q or k")
    if ref.dim() != 3:
        raise ValueError("q and k must be [tokens, heads, head_dim]")
    tokens, _, D = ref.shape
    here = ref.get_device()
    if here < 0 or here != _here():
        _elsewhere("q and k", ref)
    if (cache is None) != (v is None) or (cache is None) != (plan is None):
        raise ValueError("v, plan and cache go together")
    heads = kv_heads = slot = at = at4 = 0
    qp = qo = kp = ko = vp = (0, 0, 0)
    if q is not None:
        heads = q.shape[1]
        shape = (tokens, heads, D)
        qp = qo = _rows_of(q, "q", shape, here)
        if q_out is not None:
            qo = _rows_of(q_out, "q_out", shape, here)
    if k is not None:
        kv_heads = k.shape[1]
        shape = (tokens, kv_heads, D)
        kp = _rows_of(k, "k", shape, here)
        if k_out is not None:
            ko = _rows_of(k_out, "k_out", shape, here)
        elif cache is None:
            ko = kp
    for name, w in (("q_norm", q_norm), ("k_norm", k_norm)):
        if w is not None and (w.dtype is not _BF16 or w.numel() != D or not w.is_contiguous() or w.get_device() != here):
            raise ValueError(f"{name} must be a contiguous bf16 [{D}] tensor on the current CUDA device")
    ld = rows = 0
    p = c = s = 0
    if pos is not None:
        if cos_t is None or sin_t is None:
            raise ValueError("a rotation takes cos_t and sin_t")
        shape, st = cos_t.shape, cos_t.stride()
        if cos_t.dtype is not _F32 or sin_t.dtype is not _F32 or len(shape) != 2 or shape != sin_t.shape or \
                st != sin_t.stride() or st[1] != 1 or cos_t.get_device() != here or sin_t.get_device() != here:
            raise ValueError("cos_t and sin_t must be row-major float32 2-D tensors of one shape on the current CUDA device")
        rows, width = shape
        p, c, s, ld = _ints_of(pos, tokens, "pos", here), cos_t.data_ptr(), sin_t.data_ptr(), st[0] if rows > 1 else width
        if rope_dim is None:
            rope_dim = 2 * width
        elif rope_dim > 2 * width:
            raise ValueError("the tables are narrower than half of rope_dim")
    if cache is not None:
        _cache_fits(plan, cache)
        if k is None or plan.tokens != tokens:
            raise ValueError("a cache takes the rows of k and v of all of the plan's tokens")
        if cache._device != here or plan.slot.get_device() != here:
            _elsewhere("cache and plan", cache.k)
        slot = plan.slot.data_ptr()
        vp = _rows_of(v, "v", (tokens, kv_heads, D), here)
        if isinstance(cache, KVCache4):
            at4 = ctypes.addressof(cache._c)
        else:
            at = ctypes.addressof(cache._c)
    h = _pack_heads(tokens, heads, kv_heads, D, *qp, *qo, *kp, *ko, 0 if q_norm is None else q_norm.data_ptr(),
                    0 if k_norm is None else k_norm.data_ptr(), eps, p, c, s, ld, rows, rope_dim or 0, 1 if halves else 0,
                    slot, *vp, at, at4)
    _check((_lib or lib()).nvfp4_qk_norm_rope(h, _stream_of(stream, here)), "nvfp4_qk_norm_rope")


def nvfp4_kv4_append(k: torch.Tensor, v: torch.Tensor, plan: AttnPlan, cache: KVCache4, stream=None):
    """k, v: bf16 [tokens, kv_heads, head_dim] (any row and head pitch) into the
    4-bit cache's slots plan.slot."""
    _cache_fits(plan, cache)
    here = cache._device
    if here != _here() or plan.slot.get_device() != here:
        _elsewhere("cache and plan", cache.k)
    shape = (plan.tokens, cache.kv_heads, cache.head_dim)
    _check((_lib or lib()).nvfp4_kv4_append(*_rows_of(k, "k", shape, here), *_rows_of(v, "v", shape, here),
                                            plan.slot.data_ptr(), plan.tokens, ctypes.byref(cache._c),
                                            _stream_of(stream, here)), "nvfp4_kv4_append")


def nvfp4_kv4_expand(cache: KVCache4, plan: AttnPlan, out: KVCache, stream=None):
    """The rows of the cache that the step's new tokens see, as bf16 in the same
    pages of out (a KVCache of the same sizes)."""
    _cache_fits(plan, cache)
    here = cache._device
    if here != _here() or plan.slot.get_device() != here or out._device != here:
        _elsewhere("cache, plan and out", cache.k)
    _check((_lib or lib()).nvfp4_kv4_expand(ctypes.byref(cache._c), ctypes.byref(plan._c), ctypes.byref(out._c),
                                            _stream_of(stream, here)), "nvfp4_kv4_expand")


def nvfp4_attn_paged4(q: torch.Tensor, cache: KVCache4, plan: AttnPlan, out: torch.Tensor, ws: torch.Tensor, scale=None,
                      lse=None, stream=None, zero_padding=False, expanded: KVCache | None = None):
    """:func:`nvfp4_attn_paged` over a 4-bit cache.  expanded: a KVCache of the
    same sizes as scratch, which steps with many rows per request (prompts) are
    faster with; one serves all layers that run one after the other."""
    here = cache._device
    if here != _here() or plan.kv_len.get_device() != here or ws.get_device() != here or \
            (expanded is not None and expanded._device != here):
        _elsewhere("cache, plan, ws and expanded", cache.k)
    tokens, heads, d = plan.tokens, plan.heads, cache.head_dim
    shape, at = (tokens, heads, d), 0
    if lse is not None:
        if lse.dtype is not _F32 or lse.get_device() != here or not lse.is_contiguous() or lse.numel() != tokens * heads:
            raise ValueError("lse must be a contiguous float32 [tokens, heads] tensor on the current CUDA device")
        at = lse.data_ptr()
    io = _pack_io(*_rows_of(q, "q", shape, here), *_rows_of(out, "out", shape, here), at, d,
                  d ** -0.5 if scale is None else scale, 1 if zero_padding else 0)
    _check((_lib or lib()).nvfp4_attn_paged4(ctypes.byref(plan._c), io, ctypes.byref(cache._c),
                                             None if expanded is None else ctypes.byref(expanded._c), ws.data_ptr(),
                                             ws.numel() * ws.element_size(), _stream_of(stream, here)),
           "nvfp4_attn_paged4")


class PageTable:
    """What the requests of a server hold (nvfp4_pages_t): block_table int32
    [requests, pages per request], ctx_len int32 [requests], in pages of
    page_size rows of caches of so many pages.  ctx_len 0: the request has ended."""

    def __init__(self, block_table: torch.Tensor, ctx_len: torch.Tensor, page_size: int, pages: int):
        _table(block_table, "block_table", block_table.shape)
        self.block_table, self.ctx_len, self.page_size, self.pages = block_table, ctx_len, page_size, pages
        self.requests, self.cols = block_table.shape
        self._c = _PagesC(block_table.data_ptr(), self.requests, self.cols, max(block_table.stride(0), self.cols),
                          _i32(ctx_len, self.requests, "ctx_len"), page_size, pages)


def _table(t: torch.Tensor, name: str, shape):
    if t.dtype is not _I32 or not t.is_cuda or t.dim() != 2 or t.stride(1) != 1 or t.shape != shape:
        raise ValueError(f"{name} must be a CUDA int32 [requests, pages] tensor with unit column stride")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{name}'s rows overlap (an expanded tensor has to be made contiguous)")


def nvfp4_pages_fork(table: PageTable, src: torch.Tensor, dst: torch.Tensor, free_pages: torch.Tensor, cursor, cursor_out,
                     copy_src: torch.Tensor, copy_dst: torch.Tensor, stream=None):
    """Requests dst become copies of requests src (int32 [n]), sharing their full
    pages; last pages that are not full become pages of free_pages (int32) from
    cursor (int32 [1] or None: 0) on.  (copy_src, copy_dst), int32 [n]: the pages
    for :func:`nvfp4_pages_copy`.  cursor_out: int32 [1] or None, may be cursor."""
    n = src.numel()
    here = table.block_table.get_device()
    if here != _here() or table.ctx_len.get_device() != here:
        _elsewhere("table", table.block_table)
    if dst.numel() != n:
        raise ValueError("as many dst as src")
    _check((_lib or lib()).nvfp4_pages_fork(
        ctypes.byref(table._c), _ints_of(src, n, "src", here), _ints_of(dst, n, "dst", here), n,
        _ints_of(free_pages, 0, "free_pages", here), free_pages.numel(),
        None if cursor is None else _ints_of(cursor, 1, "cursor", here),
        None if cursor_out is None else _ints_of(cursor_out, 1, "cursor_out", here),
        _ints_of(copy_src, n, "copy_src", here), _ints_of(copy_dst, n, "copy_dst", here), _stream_of(stream, here)),
        "nvfp4_pages_fork")


def nvfp4_pages_free(table: PageTable, free_pages: torch.Tensor, free_count: torch.Tensor, table_out=None, move_src=None,
                     move_dst=None, stream=None):
    """The pages that no request holds, ascending, then -1, into free_pages (int32
    [pages]), their number into free_count (int32 [1]).  With table_out (int32,
    block_table's shape; may be block_table) the pages in use are moved to the
    lowest ids: move_src and move_dst (int32 [pages // 2], -1 past the last) are
    the moves for :func:`nvfp4_pages_copy`."""
    if (table_out is None) != (move_src is None) or (table_out is None) != (move_dst is None):
        raise ValueError("table_out, move_src and move_dst go together")
    here = table.block_table.get_device()
    if here != _here() or table.ctx_len.get_device() != here:
        _elsewhere("table", table.block_table)
    out, ld, ms, md = None, 0, None, None
    if table_out is not None:
        _table(table_out, "table_out", table.block_table.shape)
        if table_out.get_device() != here:
            _elsewhere("table_out", table_out)
        out, ld = table_out.data_ptr(), max(table_out.stride(0), table.cols)
        ms, md = _ints_of(move_src, table.pages // 2, "move_src", here), _ints_of(move_dst, table.pages // 2, "move_dst", here)
    _check((_lib or lib()).nvfp4_pages_free(ctypes.byref(table._c), _ints_of(free_pages, table.pages, "free_pages", here),
                                            _ints_of(free_count, 1, "free_count", here), out, ld, ms, md,
                                            _stream_of(stream, here)), "nvfp4_pages_free")


def nvfp4_pages_copy(caches, src: torch.Tensor, dst: torch.Tensor, stream=None):
    """Page src[i] to page dst[i] (int32 [n]; pairs of -1 are skipped) in every
    one of caches (KVCache, KVCache4; one or a list, all of as many pages)."""
    if not isinstance(caches, (list, tuple)):
        caches = (caches,)
    if not caches:
        raise ValueError("no caches")
    n, pages, here = src.numel(), caches[0].pages, _here()
    planes = []
    for c in caches:
        if c.pages != pages:
            raise ValueError("caches of one number of pages")
        if c._device != here:
            _elsewhere("every cache", c.k)
        planes.append(c._planes)
    if dst.numel() != n:
        raise ValueError("as many dst as src")
    planes = b"".join(planes)
    _check((_lib or lib()).nvfp4_pages_copy(planes, len(planes) // 24, pages, _ints_of(src, n, "src", here),
                                            _ints_of(dst, n, "dst", here), n, _stream_of(stream, here)), "nvfp4_pages_copy")
