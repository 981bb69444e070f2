"""B200-native N:M semi-structured sparse weight x dense activation GEMM.

A thin binding over ``libnmspmm.so`` (C ABI in ``include/nmspmm.h``): ctypes, and a
small compiled module for the calls that are made on few tokens.
Every step of the path runs in the library's sm_100a kernels; this module only
marshals torch tensors (device memory and streams) into the C calls, with the
same names.  There is no fallback: if the library is missing or a call fails,
an exception is raised.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnmspmm.so")

NM_OK, NM_ERR_INVALID, NM_ERR_UNSUPPORTED, NM_ERR_CUDA, NM_ERR_OOM, NM_ERR_TIMEOUT = range(6)
STATUS_NAMES = {0: "NM_OK", 1: "NM_ERR_INVALID", 2: "NM_ERR_UNSUPPORTED", 3: "NM_ERR_CUDA",
                4: "NM_ERR_OOM", 5: "NM_ERR_TIMEOUT"}
NM_INT8, NM_FP16, NM_BF16, NM_FP32, NM_MXFP4 = 0, 1, 2, 3, 4
_TORCH_DT = {torch.int8: NM_INT8, torch.float16: NM_FP16, torch.bfloat16: NM_BF16}
_MX_DT = {torch.float16: NM_FP16, torch.bfloat16: NM_BF16, torch.float32: NM_FP32}
_ELEM = {NM_INT8: torch.int8, NM_FP16: torch.float16, NM_BF16: torch.bfloat16}

# Every symbol include/nmspmm.h declares.
EXPORTS = ("nm_compress", "nm_compress_tile", "nm_recompress", "nm_spmm", "nm_spmm_ex", "nm_spmm_gather",
           "nm_spmm_gather_ex", "nm_spmm_noalloc", "nm_decompress", "nm_export", "nm_export_sizes", "nm_query",
           "nm_plan_query", "nm_plan_for_shape", "nm_device_status", "nm_destroy", "nm_last_error", "nm_version",
           "nm_test_spmm_skip_stage", "nm_mx_scale_bytes", "nm_mx_quantize", "nm_mx_dequantize", "nm_compress_mx",
           "nm_spmm_mx", "nm_spmm_mx_gated", "nm_compress_gated", "nm_spmm_gated", "nm_gated_backward",
           "nm_gated_backward_workspace", "nm_gated_backward_plan_for_shape")


class NMPlanInfo(ctypes.Structure):
    """nm_plan_info of include/nmspmm.h."""
    _fields_ = [("pair", ctypes.c_int), ("bn", ctypes.c_int), ("splits", ctypes.c_int),
                ("cluster", ctypes.c_int), ("grid", ctypes.c_int), ("units", ctypes.c_int)]


class NMGradPlanInfo(ctypes.Structure):
    """nm_grad_plan_info of include/nmspmm.h."""
    _fields_ = [("bn", ctypes.c_int), ("grid", ctypes.c_int), ("splits_dx", ctypes.c_int), ("splits_dw", ctypes.c_int),
                ("runs_dx", ctypes.c_int), ("runs_dw", ctypes.c_int), ("stages", ctypes.c_int64),
                ("complete", ctypes.c_int)]


class NMError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"{STATUS_NAMES.get(status, status)}: {msg}")
        self.status = status


_lib = None


def lib() -> ctypes.CDLL:
    """Load libnmspmm.so (built in-tree by ``build.py``); raise if it is absent."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m structured_sparse_gemm_compress_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
        L.nm_compress.argtypes = [vp, i64, i64, i32, i32, i32, vp, ctypes.POINTER(vp)]
        L.nm_compress_tile.argtypes = [vp, i64, i64, i32, i32, i32, vp, ctypes.POINTER(vp)]
        L.nm_spmm_gather.argtypes = [vp, vp, i64, i64, vp, vp, vp]
        L.nm_spmm_gather_ex.argtypes = [vp, vp, i64, i64, vp, ctypes.POINTER(NMEpilogue), vp]
        L.nm_recompress.argtypes = [vp, vp, vp]
        L.nm_spmm.argtypes = [vp, vp, i64, vp, vp, vp]
        L.nm_spmm_noalloc.argtypes = [vp, vp, i64, vp, vp, vp]
        L.nm_spmm_ex.argtypes = [vp, vp, i64, vp, ctypes.POINTER(NMEpilogue), vp]
        L.nm_test_spmm_skip_stage.argtypes = [vp, vp, i64, vp, vp, vp, i32, i64]
        L.nm_decompress.argtypes = [vp, vp, vp]
        L.nm_export.argtypes = [vp, vp, vp]
        L.nm_export_sizes.argtypes = [vp, ctypes.POINTER(ctypes.c_size_t), ctypes.POINTER(ctypes.c_size_t)]
        L.nm_query.argtypes = [vp, ctypes.POINTER(i64), ctypes.POINTER(i64), ctypes.POINTER(i32),
                               ctypes.POINTER(i32), ctypes.POINTER(i32)]
        L.nm_plan_query.argtypes = [vp, i64, i32, ctypes.POINTER(NMPlanInfo)]
        L.nm_plan_for_shape.argtypes = [i32, i64, i64, i32, i32, i64, i32, ctypes.POINTER(i32), ctypes.POINTER(i32),
                                        ctypes.POINTER(NMPlanInfo)]
        L.nm_mx_scale_bytes.argtypes = [i64, i64, ctypes.POINTER(ctypes.c_size_t)]
        L.nm_mx_quantize.argtypes = [vp, i64, i64, i64, i32, vp, vp, vp]
        L.nm_mx_dequantize.argtypes = [vp, vp, i64, i64, i32, vp, vp]
        L.nm_compress_mx.argtypes = [vp, i64, i64, i32, i32, i32, i32, vp, ctypes.POINTER(vp)]
        L.nm_spmm_mx.argtypes = [vp, vp, vp, i64, vp, ctypes.POINTER(NMEpilogue), vp]
        L.nm_spmm_mx_gated.argtypes = [vp, vp, vp, i64, vp, ctypes.POINTER(NMEpilogue), vp]
        L.nm_compress_gated.argtypes = [vp, i64, i64, i32, i32, i32, vp, ctypes.POINTER(vp)]
        L.nm_spmm_gated.argtypes = [vp, vp, i64, vp, vp, ctypes.POINTER(NMEpilogue), vp]
        L.nm_gated_backward_workspace.argtypes = [vp, i64, ctypes.POINTER(ctypes.c_size_t)]
        L.nm_gated_backward.argtypes = [vp, vp, vp, vp, i64, i32, vp, vp, vp, vp, ctypes.c_size_t, vp]
        L.nm_gated_backward_plan_for_shape.argtypes = [i64, i64, i64, i32, i32, i32, ctypes.POINTER(NMGradPlanInfo)]
        L.nm_device_status.argtypes = [vp]
        L.nm_destroy.argtypes = [vp]
        L.nm_destroy.restype = None
        L.nm_last_error.restype = ctypes.c_char_p
        L.nm_version.restype = ctypes.c_char_p
        for name in ("nm_compress", "nm_compress_tile", "nm_recompress", "nm_spmm", "nm_spmm_gather",
                     "nm_spmm_gather_ex", "nm_spmm_noalloc",
                     "nm_test_spmm_skip_stage", "nm_decompress", "nm_export", "nm_export_sizes", "nm_query",
                     "nm_plan_query", "nm_plan_for_shape", "nm_device_status", "nm_mx_scale_bytes", "nm_mx_quantize",
                     "nm_mx_dequantize", "nm_compress_mx", "nm_spmm_mx", "nm_spmm_mx_gated",
                     "nm_compress_gated", "nm_spmm_gated", "nm_gated_backward", "nm_gated_backward_workspace",
                     "nm_gated_backward_plan_for_shape"):
            getattr(L, name).restype = i32
        _lib = L
    return _lib


def _check(status: int) -> None:
    if status != NM_OK:
        raise NMError(status, lib().nm_last_error().decode(errors="replace"))


# The current device and its current stream's raw handle, without building a
# torch.cuda.Stream object per call (3 us of an 8 us call).
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def _stream(stream) -> int | None:
    if stream is None:
        return _raw_stream(_current_device())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _check_tensor(name: str, t: torch.Tensor, dtype: torch.dtype, shape: tuple) -> None:
    """A contiguous tensor of this type and shape on the current CUDA device."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {list(shape)} {dtype} tensor")
    if not t.is_cuda or t.get_device() != _current_device():
        raise ValueError(f"{name} must be on the current CUDA device")


_module = None


def _native():
    """The compiled binding (csrc/nm_binding.cpp) of the feed-forward and microscaled
    calls, which spend a quarter of ctypes' time on the host; speaks to the same
    library as ``lib()``."""
    global _module
    if _module is None:
        L = lib()
        try:
            from . import _binding
        except ImportError as e:
            raise RuntimeError(f"the compiled binding is missing or does not load ({e}): build it with "
                               "`python -m structured_sparse_gemm_compress_b200.build`") from e
        _binding.init(_check, *(ctypes.cast(getattr(L, f), ctypes.c_void_p).value for f in (
            "nm_mx_quantize", "nm_mx_dequantize", "nm_spmm_mx", "nm_spmm_mx_gated", "nm_spmm_gated",
            "nm_gated_backward", "nm_gated_backward_workspace")))
        _module = _binding
    return _module


class NMHandle:
    """One compressed weight (owns the library handle and its device memory)."""

    def __init__(self, raw: int, n_out: int, k: int, N: int, M: int, dt: int, tile: bool = False,
                 gated: bool = False, src: torch.dtype | None = None):
        self._raw = ctypes.c_void_p(raw)
        self.n_out, self.k, self.N, self.M, self.dt = n_out, k, N, M, dt
        self.tile = tile  # one pattern per 128-channel tile (nm_compress_tile)
        self.gated = gated  # rows [0, n_out / 2) gate, the rest up
        self.src = src  # microscaled handles: the element type of the source weight

    @property
    def raw(self) -> ctypes.c_void_p:
        if not self._raw:
            raise RuntimeError("handle already destroyed")
        return self._raw

    @property
    def dtype(self) -> torch.dtype:
        """Element type of the weight it is made from."""
        return self.src if self.src is not None else _ELEM[self.dt]

    def destroy(self) -> None:
        if self._raw and _lib is not None:
            _lib.nm_destroy(self._raw)
        self._raw = ctypes.c_void_p(None)

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


def nm_compress(W: torch.Tensor, N: int, M: int, stream=None) -> NMHandle:
    """Prune W [n_out, k] (int8 / fp16 / bf16, on the GPU) to N:M and pack it."""
    if not W.is_cuda:
        raise ValueError("W must be a CUDA tensor")
    if W.dtype not in _TORCH_DT:
        raise ValueError(f"unsupported dtype {W.dtype}")
    W = W.contiguous()
    n_out, k = W.shape
    out = ctypes.c_void_p()
    _check(lib().nm_compress(_ptr(W), n_out, k, _TORCH_DT[W.dtype], N, M, _stream(stream), ctypes.byref(out)))
    return NMHandle(out.value, n_out, k, N, M, _TORCH_DT[W.dtype])


def nm_compress_tile(W: torch.Tensor, N: int, M: int, stream=None) -> NMHandle:
    """Prune W [n_out, k] (int8 / fp16, on the GPU) to N:M with one pattern per
    128-row tile (largest column mass) and pack it for ``nm_spmm_gather``."""
    if not W.is_cuda:
        raise ValueError("W must be a CUDA tensor")
    if W.dtype not in _TORCH_DT:
        raise ValueError(f"unsupported dtype {W.dtype}")
    W = W.contiguous()
    n_out, k = W.shape
    out = ctypes.c_void_p()
    _check(lib().nm_compress_tile(_ptr(W), n_out, k, _TORCH_DT[W.dtype], N, M, _stream(stream), ctypes.byref(out)))
    return NMHandle(out.value, n_out, k, N, M, _TORCH_DT[W.dtype], tile=True)


def nm_recompress(h: NMHandle, W: torch.Tensor, stream=None) -> NMHandle:
    """Re-prune and re-pack a new weight of the same shape/dtype into ``h`` (no allocation)."""
    if not W.is_cuda or W.dtype != h.dtype or tuple(W.shape) != (h.n_out, h.k) or not W.is_contiguous():
        raise ValueError("W must be a contiguous CUDA tensor of the handle's shape and dtype")
    _check(lib().nm_recompress(h.raw, _ptr(W), _stream(stream)))
    return h


def out_dtype(h: NMHandle, scaled: bool) -> torch.dtype:
    if h.dt == NM_INT8:
        return torch.float32 if scaled or h.gated else torch.int32
    return h.dtype


def nm_spmm(h: NMHandle, X: torch.Tensor, Y: torch.Tensor | None = None, scale: torch.Tensor | None = None,
            stream=None) -> torch.Tensor:
    """Y = X @ Wm^T for the compressed weight of ``h`` (see include/nmspmm.h)."""
    if X.dtype != h.dtype or not X.is_cuda or not X.is_contiguous() or X.dim() != 2 or X.shape[1] != h.k:
        raise ValueError("X must be a contiguous CUDA [T, k] tensor of the handle's dtype")
    T = X.shape[0]
    want = out_dtype(h, scale is not None)
    if Y is None:
        Y = torch.empty((T, h.n_out), dtype=want, device=X.device)
    elif Y.dtype != want or tuple(Y.shape) != (T, h.n_out) or not Y.is_contiguous():
        raise ValueError(f"Y must be a contiguous [{T}, {h.n_out}] {want} tensor")
    if scale is not None and (scale.dtype != torch.float32 or scale.numel() != h.n_out or not scale.is_cuda):
        raise ValueError("scale must be a CUDA float32 tensor of n_out elements")
    _check(lib().nm_spmm(h.raw, _ptr(X), T, _ptr(Y), _ptr(scale), _stream(stream)))
    return Y


def nm_spmm_gather(h: NMHandle, Xt: torch.Tensor, T: int | None = None, Y: torch.Tensor | None = None,
                   scale: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = X @ Wm^T for a tile-shared handle, X given feature-major as
    ``Xt`` [k, ldx] (``Xt[kk, t] = X[t, kk]``, rows contiguous, ldx = the row
    stride); T defaults to ``Xt.shape[1]``."""
    if Xt.dtype != h.dtype or not Xt.is_cuda or Xt.dim() != 2 or Xt.shape[0] != h.k or Xt.stride(1) != 1:
        raise ValueError("Xt must be a CUDA [k, T] tensor of the handle's dtype with contiguous rows")
    T = Xt.shape[1] if T is None else int(T)
    want = out_dtype(h, scale is not None)
    if Y is None:
        Y = torch.empty((T, h.n_out), dtype=want, device=Xt.device)
    elif Y.dtype != want or tuple(Y.shape) != (T, h.n_out) or not Y.is_contiguous():
        raise ValueError(f"Y must be a contiguous [{T}, {h.n_out}] {want} tensor")
    if scale is not None and (scale.dtype != torch.float32 or scale.numel() != h.n_out or not scale.is_cuda):
        raise ValueError("scale must be a CUDA float32 tensor of n_out elements")
    ldx = Xt.stride(0) if Xt.shape[0] > 1 else Xt.shape[1]
    _check(lib().nm_spmm_gather(h.raw, _ptr(Xt), ldx, T, _ptr(Y), _ptr(scale), _stream(stream)))
    return Y


class NMEpilogue(ctypes.Structure):
    """``nm_epilogue`` of include/nmspmm.h."""
    _fields_ = [("out", ctypes.c_int), ("act", ctypes.c_int), ("scale", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("out_scale", ctypes.c_float)]


OUT_TYPES = {"default": 0, "int32": 1, "float32": 2, "float16": 3, "bfloat16": 4, "int8": 5}
ACTS = {"none": 0, "gelu": 1, "silu": 2, "relu": 3}  # silu and relu: gated products only
_OUT_TORCH = {"int32": torch.int32, "float32": torch.float32, "float16": torch.float16,
              "bfloat16": torch.bfloat16, "int8": torch.int8}


def resolve_out(h: NMHandle, out: str, scale, bias, act: str) -> str:
    """The output type ``NM_OUT_DEFAULT`` stands for, by the header's rule."""
    if out != "default":
        return out
    if h.dtype == torch.int8:
        raw = scale is None and bias is None and act == "none" and not getattr(h, "gated", False)
        return "int32" if raw else "float32"
    return {torch.float16: "float16", torch.bfloat16: "bfloat16", torch.float32: "float32"}[h.dtype]


def nm_spmm_ex(h: NMHandle, X: torch.Tensor, Y: torch.Tensor | None = None, scale: torch.Tensor | None = None,
               bias: torch.Tensor | None = None, act: str = "none", out: str = "default",
               out_scale: float = 1.0, stream=None) -> torch.Tensor:
    """Y = out(act(X @ Wm^T * scale + bias)) with the fused output stage of
    ``nm_spmm_ex`` (include/nmspmm.h).  ``out`` is one of ``OUT_TYPES``, ``act``
    one of ``ACTS``.  Only argument marshalling happens here."""
    if X.dtype != h.dtype or not X.is_cuda or not X.is_contiguous() or X.dim() != 2 or X.shape[1] != h.k:
        raise ValueError("X must be a contiguous CUDA [T, k] tensor of the handle's dtype")
    if out not in OUT_TYPES or act not in ACTS:
        raise ValueError(f"out must be one of {tuple(OUT_TYPES)}, act one of {tuple(ACTS)}")
    for name, v in (("scale", scale), ("bias", bias)):
        if v is not None and (v.dtype != torch.float32 or v.numel() != h.n_out or not v.is_cuda):
            raise ValueError(f"{name} must be a CUDA float32 tensor of n_out elements")
    T = X.shape[0]
    res = resolve_out(h, out, scale, bias, act)
    want = _OUT_TORCH[res]
    if Y is None:
        Y = torch.empty((T, h.n_out), dtype=want, device=X.device)
    elif Y.dtype != want or tuple(Y.shape) != (T, h.n_out) or not Y.is_contiguous():
        raise ValueError(f"Y must be a contiguous [{T}, {h.n_out}] {want} tensor")
    ep = NMEpilogue(OUT_TYPES[out], ACTS[act], _ptr(scale), _ptr(bias), float(out_scale))
    _check(lib().nm_spmm_ex(h.raw, _ptr(X), T, _ptr(Y), ctypes.byref(ep), _stream(stream)))
    return Y


def nm_spmm_gather_ex(h: NMHandle, Xt: torch.Tensor, T: int | None = None, Y: torch.Tensor | None = None,
                      scale: torch.Tensor | None = None, bias: torch.Tensor | None = None, act: str = "none",
                      out: str = "default", out_scale: float = 1.0, stream=None) -> torch.Tensor:
    """``nm_spmm_gather`` (feature-major ``Xt`` [k, ldx], tile-shared handle)
    with the fused output stage of ``nm_spmm_ex``."""
    if Xt.dtype != h.dtype or not Xt.is_cuda or Xt.dim() != 2 or Xt.shape[0] != h.k or Xt.stride(1) != 1:
        raise ValueError("Xt must be a CUDA [k, T] tensor of the handle's dtype with contiguous rows")
    if out not in OUT_TYPES or act not in ACTS:
        raise ValueError(f"out must be one of {tuple(OUT_TYPES)}, act one of {tuple(ACTS)}")
    for name, v in (("scale", scale), ("bias", bias)):
        if v is not None and (v.dtype != torch.float32 or v.numel() != h.n_out or not v.is_cuda):
            raise ValueError(f"{name} must be a CUDA float32 tensor of n_out elements")
    T = Xt.shape[1] if T is None else int(T)
    want = _OUT_TORCH[resolve_out(h, out, scale, bias, act)]
    if Y is None:
        Y = torch.empty((T, h.n_out), dtype=want, device=Xt.device)
    elif Y.dtype != want or tuple(Y.shape) != (T, h.n_out) or not Y.is_contiguous():
        raise ValueError(f"Y must be a contiguous [{T}, {h.n_out}] {want} tensor")
    ep = NMEpilogue(OUT_TYPES[out], ACTS[act], _ptr(scale), _ptr(bias), float(out_scale))
    ldx = Xt.stride(0) if Xt.shape[0] > 1 else Xt.shape[1]
    _check(lib().nm_spmm_gather_ex(h.raw, _ptr(Xt), ldx, T, _ptr(Y), ctypes.byref(ep), _stream(stream)))
    return Y


def _codes(act: str, out: str) -> tuple[int, int]:
    if out not in OUT_TYPES or act not in ACTS:
        raise ValueError(f"out must be one of {tuple(OUT_TYPES)}, act one of {tuple(ACTS)}")
    return ACTS[act], OUT_TYPES[out]


def nm_compress_gated(W: torch.Tensor, N: int, M: int, stream=None) -> NMHandle:
    """Prune and pack the two projections of a gated block: W [2 n_ff, k] (int8 /
    fp16 / bf16), the gate rows first, for ``nm_spmm_gated``."""
    if W.dim() != 2 or W.dtype not in _TORCH_DT or W.shape[0] % 2:
        raise ValueError("W must be a [2 n_ff, k] int8/float16/bfloat16 tensor")
    _check_tensor("W", W, W.dtype, tuple(W.shape))
    n_out, k = W.shape
    out = ctypes.c_void_p()
    _check(lib().nm_compress_gated(W.data_ptr(), n_out // 2, k, _TORCH_DT[W.dtype], N, M, _stream(stream),
                                   ctypes.byref(out)))
    return NMHandle(out.value, n_out, k, N, M, _TORCH_DT[W.dtype], gated=True)


def nm_spmm_gated(h: NMHandle, X: torch.Tensor, Y: torch.Tensor | None = None, P: torch.Tensor | None = None,
                  scale: torch.Tensor | None = None, bias: torch.Tensor | None = None, act: str = "silu",
                  out: str = "default", out_scale: float = 1.0, stream=None) -> torch.Tensor:
    """Y [T, n_ff] = act(g) * u with g, u the halves of X @ Wm^T * scale + bias, in
    one kernel.  P [T, 2 n_ff] (the handle's type), if given, receives g and u for
    ``nm_gated_backward``."""
    act_code, out_code = _codes(act, out)
    return (_module or _native()).spmm_gated(h.raw.value, h.n_out, h.k, h.dt, X, Y, P, scale, bias, act_code, out_code,
                                             out_scale, stream)


def nm_gated_backward_workspace(h: NMHandle, T: int) -> int:
    """Bytes of device workspace one ``nm_gated_backward`` call for T tokens needs."""
    n = ctypes.c_size_t()
    _check(lib().nm_gated_backward_workspace(h.raw, int(T), ctypes.byref(n)))
    return n.value


def nm_gated_backward(h: NMHandle, X: torch.Tensor, P: torch.Tensor, dY: torch.Tensor, act: str = "silu",
                      bias_grad: bool = False, dX: torch.Tensor | None = None, dW: torch.Tensor | None = None,
                      dbias: torch.Tensor | None = None, workspace: torch.Tensor | None = None, stream=None):
    """Gradients of ``nm_spmm_gated`` (fp16 / bf16 handles): (dX [T, k], dW [2 n_ff,
    k], dbias [2 n_ff] fp32 or None).  dW is the gradient of the masked weight at
    every position.  ``workspace``: a uint8 CUDA tensor, else one is allocated."""
    if act not in ACTS:
        raise ValueError(f"act must be one of {tuple(ACTS)}")
    return (_module or _native()).gated_backward(h.raw.value, h.n_out, h.k, h.dt, X, P, dY, ACTS[act], int(bias_grad), dX,
                                                 dW, dbias, workspace, stream)


def nm_gated_backward_plan_for_shape(n_ff: int, k: int, T: int, sms: int, dx: bool = True, dw: bool = True) -> dict:
    """How ``nm_gated_backward`` would share out its products on a GPU with ``sms`` SMs.  Needs
    no GPU: a test and diagnostic hook."""
    info = NMGradPlanInfo()
    _check(lib().nm_gated_backward_plan_for_shape(int(n_ff), int(k), int(T), int(bool(dx)), int(bool(dw)), int(sms),
                                                  ctypes.byref(info)))
    return {f: getattr(info, f) for f, _ in NMGradPlanInfo._fields_}


def nm_mx_scale_bytes(rows: int, k: int) -> int:
    """Bytes of the scales of a microscaled [rows, k] matrix (layout in include/nmspmm.h)."""
    n = ctypes.c_size_t()
    _check(lib().nm_mx_scale_bytes(int(rows), int(k), ctypes.byref(n)))
    return n.value


def nm_mx_quantize(X: torch.Tensor, Q: torch.Tensor | None = None, S: torch.Tensor | None = None,
                   stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """X [T, k] (fp32 / fp16 / bf16, rows contiguous, any row stride that is a
    multiple of 16 bytes) to microscaled 4-bit codes Q [T, k / 2] and scales S (uint8)."""
    return (_module or _native()).mx_quantize(X, Q, S, stream)


def nm_mx_dequantize(Q: torch.Tensor, S: torch.Tensor, dtype: torch.dtype = torch.bfloat16,
                     X: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The values that codes and scales of ``nm_mx_quantize`` stand for."""
    if dtype not in _MX_DT:
        raise ValueError("dtype must be float32, float16 or bfloat16")
    return (_module or _native()).mx_dequantize(Q, S, _MX_DT[dtype], X, stream)


def nm_compress_mx(W: torch.Tensor, N: int = 4, M: int = 4, gated: bool = False, stream=None) -> NMHandle:
    """Prune W [n_out, k] (fp32 / fp16 / bf16) to N:M, quantise it to microscaled
    4-bit values and pack it for ``nm_spmm_mx`` (``gated``: rows [0, n_out / 2)
    gate, the rest up, for ``nm_spmm_mx_gated``)."""
    if W.dim() != 2 or W.dtype not in _MX_DT:
        raise ValueError("W must be a [n_out, k] float32/float16/bfloat16 tensor")
    _check_tensor("W", W, W.dtype, tuple(W.shape))
    n_out, k = W.shape
    out = ctypes.c_void_p()
    _check(lib().nm_compress_mx(W.data_ptr(), n_out, k, _MX_DT[W.dtype], N, M, int(bool(gated)), _stream(stream),
                                ctypes.byref(out)))
    return NMHandle(out.value, n_out, k, N, M, NM_MXFP4, gated=bool(gated), src=W.dtype)


def _mx_product(gated: int, h: NMHandle, Q, S, Y, scale, bias, act: str, out: str, stream) -> torch.Tensor:
    act_code, out_code = _codes(act, out)
    src = _MX_DT.get(h.dtype, NM_FP32)  # (a handle of another kind: the library refuses it)
    return (_module or _native()).spmm_mx(h.raw.value, h.n_out, h.k, src, gated, Q, S, Y, scale, bias, act_code, out_code,
                                          stream)


def nm_spmm_mx(h: NMHandle, Q: torch.Tensor, S: torch.Tensor, Y: torch.Tensor | None = None,
               scale: torch.Tensor | None = None, bias: torch.Tensor | None = None, act: str = "none",
               out: str = "default", stream=None) -> torch.Tensor:
    """Y = out(act(X @ Wm^T * scale + bias)) for a handle of ``nm_compress_mx`` and
    X given as the codes Q and scales S of ``nm_mx_quantize``."""
    return _mx_product(0, h, Q, S, Y, scale, bias, act, out, stream)


def nm_spmm_mx_gated(h: NMHandle, Q: torch.Tensor, S: torch.Tensor, Y: torch.Tensor | None = None,
                     scale: torch.Tensor | None = None, bias: torch.Tensor | None = None, act: str = "silu",
                     out: str = "default", stream=None) -> torch.Tensor:
    """Y [T, n_out / 2] = act(gate) * up for a gated handle of ``nm_compress_mx``."""
    return _mx_product(1, h, Q, S, Y, scale, bias, act, out, stream)


def nm_spmm_noalloc(h: NMHandle, X: torch.Tensor, Y: torch.Tensor, scale: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """nm_spmm for callers that cannot allocate: split-K scratch lives in a fixed
    array inside the library (limits and ordering rules in include/nmspmm.h)."""
    _check(lib().nm_spmm_noalloc(h.raw, _ptr(X), X.shape[0], _ptr(Y), _ptr(scale), _stream(stream)))
    return Y


def nm_test_spmm_skip_stage(h: NMHandle, X: torch.Tensor, Y: torch.Tensor, scale: torch.Tensor | None,
                            skip_stage: int, timeout_ns: int, stream=None) -> int:
    """Test hook: run the SpMM with one producer stage left unfilled; returns the launch status."""
    return lib().nm_test_spmm_skip_stage(h.raw, _ptr(X), X.shape[0], _ptr(Y), _ptr(scale), _stream(stream),
                                         skip_stage, timeout_ns)


def nm_decompress(h: NMHandle, stream=None) -> torch.Tensor:
    """Masked dense W decoded from the packed operand image the SpMM reads."""
    dtype = torch.bfloat16 if h.dt == NM_MXFP4 else h.dtype
    out = torch.empty((h.n_out, h.k), dtype=dtype, device="cuda")
    _check(lib().nm_decompress(h.raw, _ptr(out), _stream(stream)))
    return out


def nm_export_sizes(h: NMHandle) -> tuple[int, int]:
    vb, ib = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().nm_export_sizes(h.raw, ctypes.byref(vb), ctypes.byref(ib)))
    return vb.value, ib.value


def nm_export(h: NMHandle):
    """Canonical format on the host: (values [n_out, k/M, N], idx [n_out, pitch] uint8) as torch CPU tensors."""
    vb, ib = nm_export_sizes(h)
    values = torch.empty((h.n_out, h.k // h.M, h.N), dtype=h.dtype)
    idx = torch.empty((h.n_out, ib // h.n_out), dtype=torch.uint8)
    assert values.numel() * values.element_size() == vb
    _check(lib().nm_export(h.raw, _ptr(values), _ptr(idx)))
    return values, idx


def nm_query(h: NMHandle) -> dict:
    n, k, N, M, dt = ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _check(lib().nm_query(h.raw, ctypes.byref(n), ctypes.byref(k), ctypes.byref(N), ctypes.byref(M),
                          ctypes.byref(dt)))
    return {"n_out": n.value, "k": k.value, "N": N.value, "M": M.value, "dtype": dt.value}


def nm_plan_query(h: NMHandle, T: int, scaled: bool = False) -> dict:
    """The launch plan the SpMM call would use for T tokens (kernel, token tile, splits, cluster, grid)."""
    info = NMPlanInfo()
    _check(lib().nm_plan_query(h.raw, int(T), int(bool(scaled)), ctypes.byref(info)))
    return {f: getattr(info, f) for f, _ in NMPlanInfo._fields_}


def nm_plan_for_shape(dtype: torch.dtype, n_out: int, k: int, N: int, M: int, T: int, sms: int,
                      pair_clusters=(74, 74, 74), stream_clusters=(148, 74, 48, 37, 28, 24, 21, 18)) -> dict:
    """The plan nm_plan_query would report for a handle of this shape on a GPU
    with ``sms`` SMs and the given resident-cluster capacities (two-SM kernel
    pairs at token tiles 224/192/128; clusters of 1..8 one-SM CTAs).  Needs no
    GPU: a test and diagnostic hook of the planner."""
    if dtype not in _TORCH_DT or len(pair_clusters) != 3 or len(stream_clusters) != 8:
        raise ValueError("dtype must be int8/float16/bfloat16, pair_clusters 3 values, stream_clusters 8")
    pc = (ctypes.c_int * 3)(*[int(v) for v in pair_clusters])
    sc = (ctypes.c_int * 8)(*[int(v) for v in stream_clusters])
    info = NMPlanInfo()
    _check(lib().nm_plan_for_shape(_TORCH_DT[dtype], int(n_out), int(k), int(N), int(M), int(T), int(sms), pc, sc,
                                   ctypes.byref(info)))
    return {f: getattr(info, f) for f, _ in NMPlanInfo._fields_}


def nm_device_status(h: NMHandle) -> int:
    """NM_OK, or NM_ERR_TIMEOUT if a kernel gave up a bounded wait (clears the word)."""
    return lib().nm_device_status(h.raw)


def nm_last_error() -> str:
    return lib().nm_last_error().decode(errors="replace")


def nm_version() -> str:
    return lib().nm_version().decode()
