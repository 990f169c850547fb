"""Python binding of libqgemm (quantized GEMMs dequantized inside the kernel,
products of 8-bit integers, dense or grouped by expert, and the paged key-value
cache of a decode step).

Argument marshalling only: each function checks dtypes and shapes of torch
tensors, allocates outputs with torch, and calls the C entry point of the same
name on torch's current stream.  Every step of the computation runs in the
library's HIP kernels; there is no fallback.  If libqgemm.so is missing the
calls raise instead of computing anything.

The calls that a decode step makes for every layer (key-value cache, int8 and
expert products) marshal their usual arguments in native code (the module
_binding); what that does not take goes through the checks here, and everything
where it is not built.
"""

import ctypes
import os
import warnings

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libqgemm.so")

QGEMM_W4A16 = 1
QGEMM_W8A16 = 2
QGEMM_MXFP4 = 3
QGEMM_FP8 = 4
QGEMM_W4A16_GROUPED = 5
QGEMM_W8A16_GROUPED = 6
QGEMM_NVFP4 = 7

FORMATS = {"w4a16": QGEMM_W4A16, "w8a16": QGEMM_W8A16, "mxfp4": QGEMM_MXFP4, "fp8": QGEMM_FP8,
           "w4a16_grouped": QGEMM_W4A16_GROUPED, "w8a16_grouped": QGEMM_W8A16_GROUPED,
           "nvfp4": QGEMM_NVFP4}

# (name, restype, argtypes) of every symbol declared in include/qgemm.h
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_SIGNATURES = [
    ("qgemm_status_string", ctypes.c_char_p, [ctypes.c_int]),
    ("qgemm_abi_version", ctypes.c_int, []),
    ("qgemm_dispatch_kernel", ctypes.c_int, [ctypes.c_int, _I64, _I64, _I64, _I64]),
    ("qgemm_prepack_bytes", ctypes.c_int64, [ctypes.c_int, _I64, _I64]),
    ("qgemm_prepack", ctypes.c_int, [ctypes.c_int, _P, _P, _P, _I64, _I64, _P]),
    ("qgemm_quantize_mxfp4", ctypes.c_int, [_P, _I64, _I64, _P, _P, _P]),
    ("qgemm_quantize_fp8", ctypes.c_int, [_P, _I64, _P, _P, _P]),
    ("qgemm_w4a16", ctypes.c_int, [_P, _P, _P, _P, _I64, _I64, _I64, _P]),
    ("qgemm_w8a16", ctypes.c_int, [_P, _P, _P, _P, _I64, _I64, _I64, _P]),
    ("qgemm_mxfp4", ctypes.c_int, [_P, _P, _P, _P, _I64, _I64, _I64, _P]),
    ("qgemm_fp8", ctypes.c_int, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _P]),
    ("qgemm_prepack_grouped_bytes", ctypes.c_int64, [ctypes.c_int, _I64, _I64, _I64]),
    ("qgemm_prepack_grouped", ctypes.c_int,
     [ctypes.c_int, _P, _P, _P, _I64, _I64, _P, _I64, _I64, _P]),
    ("qgemm_w4a16_grouped", ctypes.c_int, [_P, _P, _P, _I64, _I64, _I64, _I64, _P]),
    ("qgemm_w8a16_grouped", ctypes.c_int, [_P, _P, _P, _I64, _I64, _I64, _I64, _P]),
    ("qgemm_nvfp4", ctypes.c_int, [_P, _P, _P, _P, _I64, _I64, _I64, _P]),
    ("qgemm_act_workspace_bytes", ctypes.c_int64, [ctypes.c_int, _I64, _I64]),
    ("qgemm_mxfp4_act", ctypes.c_int, [_P, _P, _P, _P, _I64, _I64, _I64, _P]),
    ("qgemm_fp8_act", ctypes.c_int, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _P]),
    ("qgemm_fp8_act_noalloc", ctypes.c_int, [_P, _P, _P, _P, _I64, _I64, _I64, _P]),
    ("qgemm_kv_plan", ctypes.c_int, [_P] * 8 + [_I64] * 6 + [_P]),
    ("qgemm_kv_append", ctypes.c_int,
     [ctypes.c_int, ctypes.c_int] + [_P] * 7 + [_I64] * 12 + [_P]),
    ("qgemm_paged_attention_workspace_bytes", ctypes.c_int64, [_I64] * 6),
    ("qgemm_paged_attention", ctypes.c_int,
     [ctypes.c_int, ctypes.c_int] + [_P] * 9 + [_I64] * 15 + [ctypes.c_float, _P]),
    ("qgemm_quantize_int8", ctypes.c_int, [ctypes.c_int, _P, _P, _P, _I64, _I64, _I64, _P]),
    ("qgemm_prepack_w8a8_bytes", ctypes.c_int64, [_I64, _I64, _I64, ctypes.c_int]),
    ("qgemm_prepack_w8a8", ctypes.c_int, [_P, _P, _I64, _I64, _I64, ctypes.c_int, _P]),
    ("qgemm_w8a8", ctypes.c_int,
     [ctypes.c_int] + [_P] * 5 + [_I64] * 3 + [ctypes.c_int, _P]),
    ("qgemm_w8a8_experts", ctypes.c_int,
     [ctypes.c_int] + [_P] * 7 + [_I64] * 5 + [ctypes.c_int, _P]),
    ("qgemm_w8a8_tile", ctypes.c_int, [_I64] * 4 + [ctypes.c_int] + [_P] * 3),
    ("qgemm_expert_plan_workspace_bytes", ctypes.c_int64, [_I64] * 2),
    ("qgemm_expert_plan", ctypes.c_int, [ctypes.c_int] + [_P] * 5 + [_I64] * 3 + [_P]),
    ("qgemm_expert_combine", ctypes.c_int, [ctypes.c_int] + [_P] * 4 + [_I64] * 4 + [_P]),
    ("qgemm_read_probe", ctypes.c_int, [_P, _I64, _P, _I64, _P]),
    ("qgemm_mfma_probe", ctypes.c_int, [ctypes.c_int, _P, _I64, _P, _I64, _P]),
]

# largest M * K that qgemm_fp8_act_noalloc accepts (its fixed scratch)
FP8_ACT_NOALLOC_MAX_ELEMS = 16 * 1024 * 1024

_lib = None
_native = None    # the native binding, once the library is loaded, if there is one


class QgemmError(RuntimeError):
    def __init__(self, status, where):
        self.status = status
        super().__init__(f"{where}: status {status} ({status_string(status)})")


def lib():
    """The loaded libqgemm.so (ctypes), loading it (and the native binding, if
    there is one) on first use."""
    global _lib, _native
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is not built; run `python -m bit_quantized_gemm_qgemm_amd.build`")
        handle = ctypes.CDLL(LIB_PATH)
        for name, res, args in _SIGNATURES:
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        try:
            from . import _binding
        except ImportError as e:
            _binding = None
            warnings.warn(f"the native binding is not built for this interpreter ({e}); the "
                          "calls of a decode step take 3 to 5 us longer.  Run "
                          "`python -m bit_quantized_gemm_qgemm_amd.build`", RuntimeWarning,
                          stacklevel=2)
        _lib, _native = handle, _binding
    return _lib


def status_string(status):
    return lib().qgemm_status_string(int(status)).decode()


def _check(status, where):
    if status != 0:
        raise QgemmError(status, where)


def _stream(t):
    """Handle of torch's current stream on t's device (as
    torch.cuda.current_stream gives it, without the Stream object: 0.1 us
    instead of 1.9)."""
    return torch._C._cuda_getCurrentRawStream(t.get_device())


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _need(t, dtype, ndim, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {t.dim()}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major, no padding)")


def _out(out, M, N, dtype, device):
    """The caller's output tensor, checked to be a contiguous [M, N] device
    tensor of `dtype` (the library writes M * N elements through its pointer),
    or a new one."""
    if out is None:
        return torch.empty((M, N), dtype=dtype, device=device)
    _need(out, dtype, 2, "out")
    if tuple(out.shape) != (M, N):
        raise ValueError(f"out must be [{M}, {N}], got {list(out.shape)}")
    return out


# qgemm_dispatch_kernel results: the kernel each launches, by its name in
# profiler traces
KERNELS = {0: None, 1: "decode_gemm_kernel", 2: "pipe256_kernel", 3: "mxw_kernel",
           4: "f8w_kernel", 5: "tile_gemm_kernel"}


def qgemm_dispatch_kernel(fmt, M, N, K, group_k=0):
    """Name of the kernel a GEMM call of this format and sizes launches (None
    when M or N is 0); host-only.  The fused-quantization calls dispatch as
    "mxfp4" / "fp8"."""
    st = lib().qgemm_dispatch_kernel(int(FORMATS.get(fmt, fmt)), int(M), int(N), int(K),
                                     int(group_k))
    if st < 0:
        raise QgemmError(int(st), "qgemm_dispatch_kernel")
    return KERNELS[st]


def qgemm_prepack_bytes(fmt, K, N):
    n = lib().qgemm_prepack_bytes(int(fmt), int(K), int(N))
    if n < 0:
        raise QgemmError(int(n), "qgemm_prepack_bytes")
    return int(n)


def qgemm_prepack(fmt, w, K, N, w_scales=None):
    """Canonical weight (device tensor) -> opaque packed uint8 device tensor."""
    fmt = FORMATS.get(fmt, fmt)
    if fmt == QGEMM_W4A16:
        _need(w, torch.uint8, 2, "w")
        if tuple(w.shape) != (K // 2, N) or K % 2:
            raise ValueError("W4A16 weight must be uint8 [K/2, N] with K even")
    elif fmt == QGEMM_W8A16:
        _need(w, torch.int8, 2, "w")
        if tuple(w.shape) != (K, N):
            raise ValueError("W8A16 weight must be int8 [K, N]")
    elif fmt == QGEMM_MXFP4:
        _need(w, torch.uint8, 2, "w")
        _need(w_scales, torch.uint8, 2, "w_scales")
        if tuple(w.shape) != (N, K // 2) or tuple(w_scales.shape) != (N, K // 32):
            raise ValueError("MXFP4 weight must be codes uint8 [N, K/2] and scales uint8 [N, K/32]")
    elif fmt == QGEMM_NVFP4:
        _need(w, torch.uint8, 2, "w")
        _need(w_scales, torch.uint8, 2, "w_scales")
        if tuple(w.shape) != (N, K // 2) or tuple(w_scales.shape) != (N, K // 16) or K % 16:
            raise ValueError("NVFP4 weight must be codes uint8 [N, K/2] and e4m3 scales "
                             "uint8 [N, K/16], K a multiple of 16")
    elif fmt == QGEMM_FP8:
        if w.dtype == torch.float8_e4m3fn:
            w = w.view(torch.uint8)
        _need(w, torch.uint8, 2, "w")
        if tuple(w.shape) != (K, N):
            raise ValueError("FP8 weight must be e4m3fn [K, N]")
    else:
        raise ValueError(f"unknown format {fmt}")
    nbytes = qgemm_prepack_bytes(fmt, K, N)
    out = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=w.device)
    _check(lib().qgemm_prepack(fmt, _ptr(w), _ptr(w_scales), _ptr(out), int(K), int(N),
                               _stream(w)), "qgemm_prepack")
    return out


def qgemm_quantize_mxfp4(x):
    """fp32 [rows, K] -> (codes uint8 [rows, K/2], e8m0 uint8 [rows, K/32])."""
    _need(x, torch.float32, 2, "x")
    rows, k = x.shape
    if k % 32:
        raise ValueError("K must be a multiple of 32")
    codes = torch.empty((rows, k // 2), dtype=torch.uint8, device=x.device)
    e8m0 = torch.empty((rows, k // 32), dtype=torch.uint8, device=x.device)
    _check(lib().qgemm_quantize_mxfp4(_ptr(x), rows, k, _ptr(codes), _ptr(e8m0), _stream(x)),
           "qgemm_quantize_mxfp4")
    return codes, e8m0


def qgemm_quantize_fp8(x):
    """fp32 tensor -> (e4m3fn codes as uint8 of the same shape, fp32 scale [1])."""
    if not isinstance(x, torch.Tensor) or x.dtype != torch.float32 or not x.is_cuda \
            or not x.is_contiguous():
        raise TypeError("x must be a contiguous float32 device tensor")
    codes = torch.empty(x.shape, dtype=torch.uint8, device=x.device)
    scale = torch.empty(1, dtype=torch.float32, device=x.device)
    _check(lib().qgemm_quantize_fp8(_ptr(x), x.numel(), _ptr(codes), _ptr(scale), _stream(x)),
           "qgemm_quantize_fp8")
    return codes, scale


def _weight_only(name, x, w_packed, scales, N, out):
    _need(x, torch.float16, 2, "x")
    _need(w_packed, torch.uint8, 1, "w_packed")
    _need(scales, torch.float16, 1, "scales")
    M, K = x.shape
    if scales.shape[0] != N:
        raise ValueError("scales must have N entries")
    fmt = QGEMM_W4A16 if name == "qgemm_w4a16" else QGEMM_W8A16
    if w_packed.numel() < qgemm_prepack_bytes(fmt, K, N):
        raise ValueError("w_packed is smaller than the packed size for this K, N")
    out = _out(out, M, N, torch.float16, x.device)
    fn = getattr(lib(), name)
    _check(fn(_ptr(x), _ptr(w_packed), _ptr(scales), _ptr(out), M, N, K, _stream(x)), name)
    return out


def qgemm_w4a16(x, w_packed, scales, N, out=None):
    """Y = X @ ((code - 8) * s) -> fp16 [M, N]."""
    return _weight_only("qgemm_w4a16", x, w_packed, scales, N, out)


def qgemm_w8a16(x, w_packed, scales, N, out=None):
    """Y = X @ (w * s) -> fp16 [M, N]."""
    return _weight_only("qgemm_w8a16", x, w_packed, scales, N, out)


def qgemm_mxfp4(a_codes, a_e8m0, w_packed, N, out=None):
    """C = A_deq @ W_deq^T -> bf16 [M, N]."""
    _need(a_codes, torch.uint8, 2, "a_codes")
    _need(a_e8m0, torch.uint8, 2, "a_e8m0")
    _need(w_packed, torch.uint8, 1, "w_packed")
    M, half_k = a_codes.shape
    K = 2 * half_k
    if tuple(a_e8m0.shape) != (M, K // 32):
        raise ValueError("a_e8m0 must be [M, K/32]")
    if w_packed.numel() < qgemm_prepack_bytes(QGEMM_MXFP4, K, N):
        raise ValueError("w_packed is smaller than the packed size for this K, N")
    out = _out(out, M, N, torch.bfloat16, a_codes.device)
    _check(lib().qgemm_mxfp4(_ptr(a_codes), _ptr(a_e8m0), _ptr(w_packed), _ptr(out), M, N, K,
                             _stream(a_codes)), "qgemm_mxfp4")
    return out


def qgemm_fp8(a, b_packed, scale_a, scale_b, N, out=None):
    """C = (A @ B) * scale_a * scale_b -> bf16 [M, N]; scales are device fp32 [1]."""
    if a.dtype == torch.float8_e4m3fn:
        a = a.view(torch.uint8)
    _need(a, torch.uint8, 2, "a")
    _need(b_packed, torch.uint8, 1, "b_packed")
    for s, nm in ((scale_a, "scale_a"), (scale_b, "scale_b")):
        if s.dtype != torch.float32 or not s.is_cuda or s.numel() != 1:
            raise TypeError(f"{nm} must be a one-element float32 device tensor")
    M, K = a.shape
    if b_packed.numel() < qgemm_prepack_bytes(QGEMM_FP8, K, N):
        raise ValueError("b_packed is smaller than the packed size for this K, N")
    out = _out(out, M, N, torch.bfloat16, a.device)
    _check(lib().qgemm_fp8(_ptr(a), _ptr(b_packed), _ptr(scale_a), _ptr(scale_b), _ptr(out), M,
                           N, K, _stream(a)), "qgemm_fp8")
    return out


def qgemm_prepack_grouped_bytes(fmt, K, N, group_k):
    n = lib().qgemm_prepack_grouped_bytes(int(FORMATS.get(fmt, fmt)), int(K), int(N), int(group_k))
    if n < 0:
        raise QgemmError(int(n), "qgemm_prepack_grouped_bytes")
    return int(n)


def qgemm_prepack_grouped(fmt, w, K, N, scales, zeros=None, group_k=128, group_n=1):
    """Codes + group-wise fp16 scales [ceil(K/group_k), ceil(N/group_n)] (+ zero
    points of the same shape: uint8 0..15 for W4, int8 for W8; None for the
    symmetric 8 / 0) -> opaque packed uint8 device tensor."""
    fmt = FORMATS.get(fmt, fmt)
    if fmt == QGEMM_W4A16_GROUPED:
        _need(w, torch.uint8, 2, "w")
        if tuple(w.shape) != (K // 2, N):
            raise ValueError("grouped W4A16 weight must be uint8 [K/2, N]")
        zdtype = torch.uint8
    elif fmt == QGEMM_W8A16_GROUPED:
        _need(w, torch.int8, 2, "w")
        if tuple(w.shape) != (K, N):
            raise ValueError("grouped W8A16 weight must be int8 [K, N]")
        zdtype = torch.int8
    else:
        raise ValueError(f"not a grouped format: {fmt}")
    shape = (-(-K // group_k), -(-N // group_n))
    _need(scales, torch.float16, 2, "scales")
    if tuple(scales.shape) != shape:
        raise ValueError(f"scales must be {shape}")
    if zeros is not None:
        _need(zeros, zdtype, 2, "zeros")
        if tuple(zeros.shape) != shape:
            raise ValueError(f"zeros must be {shape}")
    nbytes = qgemm_prepack_grouped_bytes(fmt, K, N, group_k)
    out = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=w.device)
    _check(lib().qgemm_prepack_grouped(fmt, _ptr(w), _ptr(scales), _ptr(zeros), int(group_k),
                                       int(group_n), _ptr(out), int(K), int(N), _stream(w)),
           "qgemm_prepack_grouped")
    return out


def _grouped(name, fmt, x, w_packed, N, group_k, out):
    _need(x, torch.float16, 2, "x")
    _need(w_packed, torch.uint8, 1, "w_packed")
    M, K = x.shape
    if w_packed.numel() < qgemm_prepack_grouped_bytes(fmt, K, N, group_k):
        raise ValueError("w_packed is smaller than the packed size for this K, N, group_k")
    out = _out(out, M, N, torch.float16, x.device)
    _check(getattr(lib(), name)(_ptr(x), _ptr(w_packed), _ptr(out), M, N, K, int(group_k),
                                _stream(x)), name)
    return out


def qgemm_w4a16_grouped(x, w_packed, N, group_k, out=None):
    """Y = X @ ((code - z) * s) with group-wise s, z -> fp16 [M, N]."""
    return _grouped("qgemm_w4a16_grouped", QGEMM_W4A16_GROUPED, x, w_packed, N, group_k, out)


def qgemm_w8a16_grouped(x, w_packed, N, group_k, out=None):
    """Y = X @ ((w - z) * s) with group-wise s, z -> fp16 [M, N]."""
    return _grouped("qgemm_w8a16_grouped", QGEMM_W8A16_GROUPED, x, w_packed, N, group_k, out)


def qgemm_nvfp4(x, w_packed, global_scale, N, out=None):
    """Y = X @ (e2m1 * e4m3 block scale * global)^T -> fp16 [M, N]; global_scale
    is a one-element float32 device tensor."""
    _need(x, torch.float16, 2, "x")
    _need(w_packed, torch.uint8, 1, "w_packed")
    if global_scale.dtype != torch.float32 or not global_scale.is_cuda or global_scale.numel() != 1:
        raise TypeError("global_scale must be a one-element float32 device tensor")
    M, K = x.shape
    if w_packed.numel() < qgemm_prepack_bytes(QGEMM_NVFP4, K, N):
        raise ValueError("w_packed is smaller than the packed size for this K, N")
    out = _out(out, M, N, torch.float16, x.device)
    _check(lib().qgemm_nvfp4(_ptr(x), _ptr(w_packed), _ptr(global_scale), _ptr(out), M, N, K,
                             _stream(x)), "qgemm_nvfp4")
    return out


def qgemm_act_workspace_bytes(fmt, M, K):
    n = lib().qgemm_act_workspace_bytes(int(FORMATS.get(fmt, fmt)), int(M), int(K))
    if n < 0:
        raise QgemmError(int(n), "qgemm_act_workspace_bytes")
    return int(n)


def _act_workspace(fmt, a, workspace):
    M, K = a.shape
    need = qgemm_act_workspace_bytes(fmt, M, K)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=a.device)
    else:
        _need(workspace, torch.uint8, 1, "workspace")
        if workspace.numel() < need:
            raise ValueError(f"workspace needs {need} bytes")
    return workspace


def qgemm_mxfp4_act(a, w_packed, N, workspace=None, out=None):
    """fp32 A [M, K] -> MXFP4 on the device, then C = A_deq @ W_deq^T (bf16).
    Returns (C, workspace); the workspace holds the quantized A."""
    _need(a, torch.float32, 2, "a")
    _need(w_packed, torch.uint8, 1, "w_packed")
    M, K = a.shape
    if w_packed.numel() < qgemm_prepack_bytes(QGEMM_MXFP4, K, N):
        raise ValueError("w_packed is smaller than the packed size for this K, N")
    workspace = _act_workspace(QGEMM_MXFP4, a, workspace)
    out = _out(out, M, N, torch.bfloat16, a.device)
    _check(lib().qgemm_mxfp4_act(_ptr(a), _ptr(w_packed), _ptr(out), _ptr(workspace), M, N, K,
                                 _stream(a)), "qgemm_mxfp4_act")
    return out, workspace


def qgemm_fp8_act(a, b_packed, scale_b, N, workspace=None, out=None):
    """fp32 A [M, K] -> per-tensor e4m3fn on the device, then C = (A_q @ B) *
    s_a * s_b (bf16).  Returns (C, workspace); the workspace holds the codes
    and, at round_up(M*K, 16), the fp32 scale."""
    _need(a, torch.float32, 2, "a")
    _need(b_packed, torch.uint8, 1, "b_packed")
    if scale_b.dtype != torch.float32 or not scale_b.is_cuda or scale_b.numel() != 1:
        raise TypeError("scale_b must be a one-element float32 device tensor")
    M, K = a.shape
    if b_packed.numel() < qgemm_prepack_bytes(QGEMM_FP8, K, N):
        raise ValueError("b_packed is smaller than the packed size for this K, N")
    workspace = _act_workspace(QGEMM_FP8, a, workspace)
    out = _out(out, M, N, torch.bfloat16, a.device)
    _check(lib().qgemm_fp8_act(_ptr(a), _ptr(b_packed), _ptr(scale_b), _ptr(out), _ptr(workspace),
                               M, N, K, _stream(a)), "qgemm_fp8_act")
    return out, workspace


def qgemm_fp8_act_noalloc(a, b_packed, scale_b, N, out):
    """As qgemm_fp8_act, with the quantized A in the library's fixed per-GPU
    scratch instead of a workspace: the entry point allocates nothing, so the
    caller passes the output.  M * K <= FP8_ACT_NOALLOC_MAX_ELEMS."""
    _need(a, torch.float32, 2, "a")
    _need(b_packed, torch.uint8, 1, "b_packed")
    if scale_b.dtype != torch.float32 or not scale_b.is_cuda or scale_b.numel() != 1:
        raise TypeError("scale_b must be a one-element float32 device tensor")
    M, K = a.shape
    if b_packed.numel() < qgemm_prepack_bytes(QGEMM_FP8, K, N):
        raise ValueError("b_packed is smaller than the packed size for this K, N")
    if out is None:
        raise ValueError("qgemm_fp8_act_noalloc needs a caller-allocated out [M, N]")
    out = _out(out, M, N, torch.bfloat16, a.device)
    _check(lib().qgemm_fp8_act_noalloc(_ptr(a), _ptr(b_packed), _ptr(scale_b), _ptr(out), M, N,
                                       K, _stream(a)), "qgemm_fp8_act_noalloc")
    return out


# ---- paged key-value cache ---------------------------------------------------
#
# A call that brings its outputs and workspace first offers its arguments to the
# native binding (which is there once the library is loaded); a None means that
# they are not of the usual kind, and the checks below say why or make the call.

# qgemm_dtype codes; uint8 holds e4m3fn codes, as qgemm_quantize_fp8 returns them
_HALF_TYPES = {torch.float16: 1, torch.bfloat16: 2}
_CACHE_TYPES = {torch.float16: 1, torch.bfloat16: 2, torch.float8_e4m3fn: 3, torch.uint8: 3}
_INT32 = (torch.int32,)
_INT64 = (torch.int64,)
_FLOAT32 = (torch.float32,)
_UINT8 = (torch.uint8,)


def _refuse(t, dtypes, ndim, name, device, dense):
    """Raise for a tensor that failed a check of _dense or _view."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {t.dim()}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if t.get_device() != device:
        raise ValueError(f"{name} is on device {t.get_device()}, the first tensor on {device}")
    raise ValueError(f"{name} must be contiguous (row-major, no padding)" if dense
                     else f"the last axis of {name} must be dense")


def _dense(t, dtypes, ndim, name, device):
    """A contiguous tensor of one of `dtypes` on device number `device`."""
    if not (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.dim() == ndim and t.is_cuda
            and t.get_device() == device and t.is_contiguous()):
        _refuse(t, dtypes, ndim, name, device, True)


def _view(t, dtypes, ndim, name, device=None):
    """A tensor of one of `dtypes` whose last axis is dense; the other axes may
    have any strides.  Returns (shape, strides of all axes but the last): 0
    where an axis has one entry or none, whose stride torch leaves arbitrary.
    With no `device` number given the tensor sets it."""
    if not (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.dim() == ndim and t.is_cuda
            and (device is None or t.get_device() == device)):
        _refuse(t, dtypes, ndim, name, device, False)
    shape, strides = t.shape, t.stride()
    if strides[-1] != 1 and shape[-1] > 1 and t.numel() > 0:
        _refuse(t, dtypes, ndim, name, t.get_device(), False)
    if 1 in shape or 0 in shape:
        return shape, [st if n > 1 else 0 for n, st in zip(shape[:-1], strides)]
    return shape, strides[:-1]


def _kv_pools(k_cache, v_cache, k_scale, v_scale, dtype, device):
    """Check both pools; returns (type code, [pages, kv_heads, page_size, dim],
    strides of the first three axes, addresses of the scales)."""
    shape, strides = _view(k_cache, _CACHE_TYPES, 4, "k_cache", device)
    v_shape, v_strides = _view(v_cache, _CACHE_TYPES, 4, "v_cache", device)
    if v_cache.dtype != k_cache.dtype or v_shape != shape or v_strides != strides:
        raise ValueError("k_cache and v_cache must agree in type, shape and strides")
    if shape[2] < 1:
        raise ValueError("pages must hold at least one token")
    code = _CACHE_TYPES[k_cache.dtype]
    if code == 3:
        for t, name in ((k_scale, "k_scale"), (v_scale, "v_scale")):
            if t is None:
                raise ValueError(f"an e4m3 cache needs {name} (float32, one per kv head)")
            _dense(t, _FLOAT32, 1, name, device)
            if t.shape[0] != shape[1]:
                raise ValueError(f"{name} must have {shape[1]} entries, one per kv head")
        return code, shape, strides, k_scale.data_ptr(), v_scale.data_ptr()
    if k_cache.dtype != dtype:
        raise TypeError(f"a 16-bit cache must be {dtype} like the tokens, got {k_cache.dtype}")
    if k_scale is not None or v_scale is not None:
        raise ValueError("a 16-bit cache takes no scales")
    return code, shape, strides, None, None


def qgemm_kv_plan(table, cached, added, free_pages, page_size, tokens, out=None):
    """Pages and slots for the tokens that enter a step, on the device.

    Request b holds cached[b] tokens and gains added[b].  table (int32
    [batch, width]) gets the pages that it gains from free_pages (int32), in
    place.  Returns (lens [batch], cu_tokens [batch + 1], cu_pages
    [batch + 1], all int32, and slots int64 [tokens]); `out` may be a tuple of
    those four tensors to write into, none of which may share memory with
    another or with an input, except that lens may be cached.  tokens: how
    many tokens the host counts on (the sum of added).  cu_pages[-1] is the
    number of pages taken; past the end of free_pages entries and slots become
    -1."""
    status = None
    if _native and out is not None:
        status = _native.kv_plan(table, cached, added, free_pages, page_size, tokens, out)
    if status is not None:
        _check(status, "qgemm_kv_plan")
        return out
    (batch, width), (table_stride,) = _view(table, _INT32, 2, "table")
    device = table.get_device()
    _dense(cached, _INT32, 1, "cached", device)
    _dense(added, _INT32, 1, "added", device)
    _dense(free_pages, _INT32, 1, "free_pages", device)
    if cached.shape[0] != batch or added.shape[0] != batch:
        raise ValueError(f"cached and added must have {batch} entries, one per request")
    if page_size < 1 or tokens < 0:
        raise ValueError("page_size must be at least 1 and tokens at least 0")
    if out is None:
        i32 = {"dtype": torch.int32, "device": table.device}
        out = (torch.empty(batch, **i32), torch.empty(batch + 1, **i32),
               torch.empty(batch + 1, **i32),
               torch.empty(tokens, dtype=torch.int64, device=table.device))
        lens, cu_tokens, cu_pages, slots = out
    else:
        out = tuple(out)
        if len(out) != 4:
            raise ValueError("out must be (lens, cu_tokens, cu_pages, slots)")
        lens, cu_tokens, cu_pages, slots = out
        _dense(lens, _INT32, 1, "lens", device)
        _dense(cu_tokens, _INT32, 1, "cu_tokens", device)
        _dense(cu_pages, _INT32, 1, "cu_pages", device)
        _dense(slots, _INT64, 1, "slots", device)
        if (lens.shape[0] != batch or cu_tokens.shape[0] != batch + 1
                or cu_pages.shape[0] != batch + 1 or slots.shape[0] != tokens):
            raise ValueError(f"lens, cu_tokens, cu_pages and slots must have {batch}, {batch + 1}, "
                             f"{batch + 1} and {tokens} entries")
    _check(lib().qgemm_kv_plan(
        table.data_ptr(), cached.data_ptr(), added.data_ptr(), free_pages.data_ptr(),
        lens.data_ptr(), cu_tokens.data_ptr(), cu_pages.data_ptr(), slots.data_ptr(), batch, width,
        table_stride, free_pages.shape[0], page_size, tokens, _stream(table)), "qgemm_kv_plan")
    return out


def qgemm_kv_append(k, v, slots, k_cache, v_cache, k_scale=None, v_scale=None):
    """Write new tokens' keys and values ([tokens, kv_heads, dim] views, fp16
    or bf16) into the slots (int64 [tokens]; page * page_size + offset, below
    0: skipped) of the pools [pages, kv_heads, page_size, dim], in place.
    Pools of the same type take a copy; float8_e4m3fn (or uint8 code) pools
    take e4m3fn(x / scale[head]), k_scale and v_scale float32 [kv_heads]."""
    status = None
    if _native:
        status = _native.kv_append(k, v, slots, k_cache, v_cache, k_scale, v_scale)
    if status is not None:
        return _check(status, "qgemm_kv_append")
    shape, k_strides = _view(k, _HALF_TYPES, 3, "k")
    device, dtype = k.get_device(), k.dtype
    v_shape, v_strides = _view(v, (dtype,), 3, "v", device)
    _dense(slots, _INT64, 1, "slots", device)
    code, (pages, kv_heads, page_size, dim), strides, k_scale, v_scale = _kv_pools(
        k_cache, v_cache, k_scale, v_scale, dtype, device)
    tokens = slots.shape[0]
    if shape != (tokens, kv_heads, dim) or v_shape != shape:
        raise ValueError(f"k and v must be [{tokens}, {kv_heads}, {dim}], got {list(shape)} "
                         f"and {list(v_shape)}")
    _check(lib().qgemm_kv_append(
        _HALF_TYPES[dtype], code, k.data_ptr(), v.data_ptr(), slots.data_ptr(),
        k_cache.data_ptr(), v_cache.data_ptr(), k_scale, v_scale, tokens, kv_heads, dim,
        *k_strides, *v_strides, pages, page_size, *strides, _stream(k)), "qgemm_kv_append")


def qgemm_paged_attention_workspace_bytes(batch, heads, kv_heads, dim, max_len, window=0):
    n = lib().qgemm_paged_attention_workspace_bytes(int(batch), int(heads), int(kv_heads),
                                                    int(dim), int(max_len), int(window))
    if n < 0:
        raise QgemmError(int(n), "qgemm_paged_attention_workspace_bytes")
    return n


def qgemm_paged_attention(q, k_cache, v_cache, table, lens, k_scale=None, v_scale=None, window=0,
                          max_len=None, scale=None, out=None, workspace=None):
    """Attention of one new token per request over its cached tokens.

    q: [batch, heads, dim] view, fp16 or bf16; the pools as in qgemm_kv_append
    with heads a multiple of kv_heads; table int32 [batch, width]; lens int32
    [batch], the tokens of each request, the new one included.  window > 0
    keeps the last `window` tokens of each.  max_len bounds lens on the host
    (default: what the table can name); scale defaults to dim ** -0.5.
    workspace: uint8, at least qgemm_paged_attention_workspace_bytes(batch,
    heads, kv_heads, dim, max_len, window); allocated if None.  Returns out,
    [batch, heads, dim] of q's type."""
    status = None
    if _native and out is not None and workspace is not None:
        status = _native.paged_attention(q, k_cache, v_cache, table, lens, k_scale, v_scale, window,
                                         max_len, scale, out, workspace)
    if status is not None:
        _check(status, "qgemm_paged_attention")
        return out
    shape, q_strides = _view(q, _HALF_TYPES, 3, "q")
    device, dtype = q.get_device(), q.dtype
    batch, heads, dim = shape
    code, (pages, kv_heads, page_size, cache_dim), strides, k_scale, v_scale = _kv_pools(
        k_cache, v_cache, k_scale, v_scale, dtype, device)
    if dim != cache_dim:
        raise ValueError(f"q has head size {dim}, the cache {cache_dim}")
    if kv_heads < 1 or heads % kv_heads:
        raise ValueError(f"{heads} heads do not divide over {kv_heads} kv heads")
    (rows, width), (table_stride,) = _view(table, _INT32, 2, "table", device)
    _dense(lens, _INT32, 1, "lens", device)
    if rows != batch or lens.shape[0] != batch:
        raise ValueError(f"table and lens must have {batch} rows, one per request")
    if max_len is None:
        max_len = min(width * page_size, 2 ** 30 - 1)
    need = qgemm_paged_attention_workspace_bytes(batch, heads, kv_heads, dim, max_len, window)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    else:
        _dense(workspace, _UINT8, 1, "workspace", device)
        if workspace.shape[0] < need:
            raise ValueError(f"workspace needs {need} bytes")
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=q.device)
    else:
        _dense(out, (dtype,), 3, "out", device)
        if out.shape != shape:
            raise ValueError(f"out must be {list(shape)}, got {list(out.shape)}")
    _check(lib().qgemm_paged_attention(
        _HALF_TYPES[dtype], code, q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
        table.data_ptr(), lens.data_ptr(), k_scale, v_scale, out.data_ptr(), workspace.data_ptr(),
        batch, heads, kv_heads, dim, *q_strides, pages, page_size, *strides, width, table_stride,
        max_len, window, dim ** -0.5 if scale is None else scale, _stream(q)),
        "qgemm_paged_attention")
    return out


# ---- int8 x int8 products, dense and by expert ---------------------------------
#
# As above: a call that brings its outputs and workspace tries the native binding.

_ROW_TYPES = {torch.float16: 1, torch.bfloat16: 2, torch.float32: 4}
_INT8 = (torch.int8,)
_ID_BYTES = {torch.int32: 4, torch.int64: 8}


def _launch(device, name, *args):
    """Call a library function with the tensors' device as the current one."""
    fn = getattr(lib(), name)
    if device < 0 or torch._C._cuda_getDevice() == device:
        status = fn(*args)
    else:
        with torch.cuda.device(device):
            status = fn(*args)
    _check(status, name)


def _result(out, shape, dtype, device, like):
    """The caller's output, checked, or a new one."""
    if out is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    _dense(out, (dtype,), len(shape), "out", device)
    if tuple(out.shape) != shape:
        raise ValueError(f"out must be {list(shape)}, got {list(out.shape)}")
    return out


def qgemm_quantize_int8(x, out=None):
    """Codes int8 [rows, K] and scales float32 [rows] of x [rows, K] (float16,
    bfloat16 or float32, rows any stride apart): scale = max |x| / 127 of the
    row, codes = x / scale to the nearest whole number.  A row with an infinity
    or a NaN gets the scale NaN and codes of 0.  `out` may be a tuple of those
    two tensors to write into."""
    status = None
    if _native and out is not None:
        status = _native.quantize_int8(x, out)
    if status is not None:
        _check(status, "qgemm_quantize_int8")
        return out
    (rows, K), (row_stride,) = _view(x, _ROW_TYPES, 2, "x")
    device = x.get_device()
    if out is None:
        out = (torch.empty((rows, K), dtype=torch.int8, device=x.device),
               torch.empty(rows, dtype=torch.float32, device=x.device))
        codes, scale = out
    else:
        out = tuple(out)
        if len(out) != 2:
            raise ValueError("out must be (codes, scale)")
        codes, scale = out
        _dense(codes, _INT8, 2, "codes", device)
        _dense(scale, _FLOAT32, 1, "scale", device)
        if codes.shape != x.shape or scale.shape[0] != rows:
            raise ValueError(f"codes must be [{rows}, {K}] and scale [{rows}]")
    _launch(device, "qgemm_quantize_int8", _ROW_TYPES[x.dtype], x.data_ptr(), codes.data_ptr(),
            scale.data_ptr(), rows, K, row_stride, _stream(x))
    return out


def qgemm_prepack_w8a8_bytes(experts, K, N, gated=False):
    n = lib().qgemm_prepack_w8a8_bytes(int(experts), int(K), int(N), int(gated))
    if n < 0:
        raise QgemmError(int(n), "qgemm_prepack_w8a8_bytes")
    return int(n)


def qgemm_prepack_w8a8(w, gated=False):
    """int8 weight [K, N], or [experts, K, N] -> opaque packed uint8 device tensor
    for qgemm_w8a8 / qgemm_w8a8_experts.  gated: the N columns are two halves,
    gate and up."""
    _need(w, torch.int8, 2 if isinstance(w, torch.Tensor) and w.dim() == 2 else 3, "w")
    experts, K, N = (1, *w.shape) if w.dim() == 2 else w.shape
    nbytes = qgemm_prepack_w8a8_bytes(experts, K, N, gated)
    out = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=w.device)
    _launch(w.get_device(), "qgemm_prepack_w8a8", w.data_ptr(), out.data_ptr(), experts, K, N,
            int(gated), _stream(w))
    return out


def _w8a8_operands(a, a_scale, w_packed, experts, N, gated):
    """Check what both products take; returns (device, rows of a, K)."""
    if not isinstance(a, torch.Tensor):
        raise TypeError("a must be a torch tensor")
    device = a.get_device()
    _dense(a, _INT8, 2, "a", device)
    _dense(a_scale, _FLOAT32, 1, "a_scale", device)
    _dense(w_packed, _UINT8, 1, "w_packed", device)
    a_rows, K = a.shape
    if a_scale.shape[0] != a_rows:
        raise ValueError(f"a_scale must have {a_rows} entries, one per row of a")
    if w_packed.shape[0] < qgemm_prepack_w8a8_bytes(experts, K, N, gated):
        raise ValueError("w_packed is smaller than the packed size for these experts, K, N")
    return device, a_rows, K


def qgemm_w8a8(a, a_scale, w_packed, w_scale, N, gated=False, dtype=torch.bfloat16, out=None):
    """Y = (A @ W) * a_scale[:, None] * w_scale -> `dtype` (float16 or bfloat16; that
    of out, if given) [M, N]; gated: silu(Y[:, :N/2]) * Y[:, N/2:], [M, N/2].

    a: int8 [M, K] codes and a_scale float32 [M], as qgemm_quantize_int8 gives
    them; w_packed from qgemm_prepack_w8a8 with the same `gated`; w_scale
    float32 [N]."""
    status = None
    if _native and out is not None:
        status = _native.w8a8(a, a_scale, w_packed, w_scale, N, gated, out)
    if status is not None:
        _check(status, "qgemm_w8a8")
        return out
    N = int(N)
    device, M, K = _w8a8_operands(a, a_scale, w_packed, 1, N, gated)
    _dense(w_scale, _FLOAT32, 1, "w_scale", device)
    if w_scale.shape[0] != N:
        raise ValueError(f"w_scale must have {N} entries")
    dtype = dtype if out is None else getattr(out, "dtype", None)
    if dtype not in _HALF_TYPES:
        raise TypeError(f"the output must be float16 or bfloat16, not {dtype}")
    out = _result(out, (M, N // 2 if gated else N), dtype, device, a)
    _launch(device, "qgemm_w8a8", _HALF_TYPES[dtype], a.data_ptr(), a_scale.data_ptr(),
            w_packed.data_ptr(), w_scale.data_ptr(), out.data_ptr(), M, N, K, int(gated), _stream(a))
    return out


def qgemm_w8a8_experts(a, a_scale, w_packed, w_scale, offsets, N, rows=None, gated=False,
                       dtype=torch.bfloat16, out=None):
    """qgemm_w8a8 with a weight for each stretch of rows: rows offsets[e] to
    offsets[e + 1] of the output take expert e's.

    w_packed is of [experts, K, N], w_scale float32 [experts, N], offsets int32
    [experts + 1].  rows, int32 [M], names the row of a (and a_scale) that each
    of the M output rows reads; without it row m reads row m.  Rows that no
    expert has are not written: in `out` they stay as they were, and in the new
    tensor that a call without `out` returns they hold whatever its memory held."""
    status = None
    if _native and out is not None:
        status = _native.w8a8_experts(a, a_scale, w_packed, w_scale, offsets, N, rows, gated, out)
    if status is not None:
        _check(status, "qgemm_w8a8_experts")
        return out
    N = int(N)
    if not isinstance(offsets, torch.Tensor):
        raise TypeError("offsets must be a torch tensor")
    experts = offsets.numel() - 1
    device, a_rows, K = _w8a8_operands(a, a_scale, w_packed, experts, N, gated)
    _dense(offsets, _INT32, 1, "offsets", device)
    _dense(w_scale, _FLOAT32, 2, "w_scale", device)
    if tuple(w_scale.shape) != (experts, N):
        raise ValueError(f"w_scale must be [{experts}, {N}]")
    M = a_rows
    if rows is not None:
        _dense(rows, _INT32, 1, "rows", device)
        M = rows.shape[0]
    dtype = dtype if out is None else getattr(out, "dtype", None)
    if dtype not in _HALF_TYPES:
        raise TypeError(f"the output must be float16 or bfloat16, not {dtype}")
    out = _result(out, (M, N // 2 if gated else N), dtype, device, a)
    _launch(device, "qgemm_w8a8_experts", _HALF_TYPES[dtype], a.data_ptr(), a_scale.data_ptr(),
            w_packed.data_ptr(), w_scale.data_ptr(), offsets.data_ptr(),
            None if rows is None else rows.data_ptr(), out.data_ptr(), a_rows, M, N, K, experts,
            int(gated), _stream(a))
    return out


def qgemm_w8a8_tile(M, N, K, experts=0, gated=False):
    """(rows, columns, parts of K) of a workgroup of qgemm_w8a8, or with
    experts > 0 of qgemm_w8a8_experts, with these sizes; host-only."""
    out = [_I64(), _I64(), _I64()]
    _check(lib().qgemm_w8a8_tile(int(M), int(N), int(K), int(experts), int(gated),
                                 *(ctypes.addressof(x) for x in out)), "qgemm_w8a8_tile")
    return tuple(x.value for x in out)


def qgemm_expert_plan_workspace_bytes(pairs, experts):
    n = lib().qgemm_expert_plan_workspace_bytes(int(pairs), int(experts))
    if n < 0:
        raise QgemmError(int(n), "qgemm_expert_plan_workspace_bytes")
    return int(n)


def qgemm_expert_plan(ids, experts, out=None, workspace=None):
    """The order of a batch's rows, on the device.

    ids: int32 or int64 [tokens, top], the experts that each token goes to; one
    outside 0 .. experts - 1 has no row.  Returns (offsets [experts + 1], rows
    [tokens * top], places [tokens, top]), all int32: the rows sorted by expert,
    in their own order within one; rows[m] is the token of row m (-1 from
    offsets[-1] on), places[t, j] the row of a token's choice (-1: none).
    `out` may be a tuple of those three to write into; workspace: uint8, at least
    qgemm_expert_plan_workspace_bytes(tokens * top, experts), allocated if None."""
    status = None
    if _native and out is not None and workspace is not None:
        status = _native.expert_plan(ids, experts, out, workspace)
    if status is not None:
        _check(status, "qgemm_expert_plan")
        return out
    if not isinstance(ids, torch.Tensor):
        raise TypeError("ids must be a torch tensor")
    device, experts = ids.get_device(), int(experts)
    _dense(ids, _ID_BYTES, 2, "ids", device)
    tokens, top = ids.shape
    need = qgemm_expert_plan_workspace_bytes(tokens * top, experts)
    if out is None:
        i32 = {"dtype": torch.int32, "device": ids.device}
        out = (torch.empty(experts + 1, **i32), torch.empty(tokens * top, **i32),
               torch.empty((tokens, top), **i32))
        offsets, rows, places = out
    else:
        out = tuple(out)
        if len(out) != 3:
            raise ValueError("out must be (offsets, rows, places)")
        offsets, rows, places = out
        _dense(offsets, _INT32, 1, "offsets", device)
        _dense(rows, _INT32, 1, "rows", device)
        _dense(places, _INT32, 2, "places", device)
        if (offsets.shape[0] != experts + 1 or rows.shape[0] != tokens * top
                or places.shape != ids.shape):
            raise ValueError(f"offsets, rows and places must be [{experts + 1}], [{tokens * top}] "
                             f"and {list(ids.shape)}")
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=ids.device)
    else:
        _dense(workspace, _UINT8, 1, "workspace", device)
        if workspace.shape[0] < need:
            raise ValueError(f"workspace needs {need} bytes")
    _launch(device, "qgemm_expert_plan", _ID_BYTES[ids.dtype], ids.data_ptr(), offsets.data_ptr(),
            rows.data_ptr(), places.data_ptr(), workspace.data_ptr(), tokens, top, experts,
            _stream(ids))
    return out


def qgemm_expert_combine(y, places, gates, out=None):
    """out[t] = sum over j of gates[t, j] * y[places[t, j]], in fp32 and in the
    order of j, rounded once: y [rows, N] float16 or bfloat16, places int32
    [tokens, top] (outside 0 .. rows - 1: left out), gates float32 [tokens, top].
    Returns out, [tokens, N] of y's type."""
    status = None
    if _native and out is not None:
        status = _native.expert_combine(y, places, gates, out)
    if status is not None:
        _check(status, "qgemm_expert_combine")
        return out
    if not isinstance(y, torch.Tensor):
        raise TypeError("y must be a torch tensor")
    device = y.get_device()
    _dense(y, _HALF_TYPES, 2, "y", device)
    _dense(places, _INT32, 2, "places", device)
    _dense(gates, _FLOAT32, 2, "gates", device)
    if gates.shape != places.shape:
        raise ValueError(f"gates must be {list(places.shape)} like places, got {list(gates.shape)}")
    rows, N = y.shape
    tokens, top = places.shape
    out = _result(out, (tokens, N), y.dtype, device, y)
    _launch(device, "qgemm_expert_combine", _HALF_TYPES[y.dtype], y.data_ptr(), places.data_ptr(),
            gates.data_ptr(), out.data_ptr(), rows, tokens, top, N, _stream(y))
    return out


def qgemm_read_probe(buf, sink, workgroups):
    """Read all of the uint8 device tensor `buf` once (the plain-read
    reference of the weight stream); sink is an int32 device tensor with at
    least `workgroups` entries."""
    _need(buf, torch.uint8, 1, "buf")
    _need(sink, torch.int32, 1, "sink")
    if sink.numel() < workgroups:
        raise ValueError("sink needs one entry per workgroup")
    _check(lib().qgemm_read_probe(_ptr(buf), buf.numel(), _ptr(sink), int(workgroups),
                                  _stream(buf)), "qgemm_read_probe")


def qgemm_mfma_probe(fmt, operands, iters, sink, workgroups):
    """Back-to-back scaled matrix instructions on register operands loaded from
    the uint8 device tensor `operands` (272 bytes per thread); sink is a
    float32 device tensor with at least `workgroups` entries."""
    _need(operands, torch.uint8, 1, "operands")
    _need(sink, torch.float32, 1, "sink")
    if operands.numel() < 272 * 256 * workgroups or sink.numel() < workgroups:
        raise ValueError("operands needs 272 bytes per thread, sink one entry per workgroup")
    _check(lib().qgemm_mfma_probe(int(FORMATS.get(fmt, fmt)), _ptr(operands), int(iters),
                                  _ptr(sink), int(workgroups), _stream(operands)),
           "qgemm_mfma_probe")
