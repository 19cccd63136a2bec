"""Thin Python binding of libfp4.so (include/fp4.h), same names as the C calls.

Argument marshalling only: every step of the path runs in the HIP kernels behind
the C ABI. torch supplies device memory (outputs are allocated with
``torch.empty`` on the input's device) and the current stream. There is no
fallback: if the library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "FP4_MXFP4",
    "FP4_NVFP4",
    "Fp4Error",
    "library_path",
    "load_library",
    "fp4_rotate_quantize",
    "fp4_quantize_weights",
    "fp4_linear",
    "fp4_rotate_quantize_linear",
    "fp4_rotate_quantize_linear_noalloc",
    "linear_workspace_bytes",
    "fp8_quantize",
    "fp8_quantize_weights",
    "fp8_add_rmsnorm_quantize",
    "fp8_linear",
    "fp4_moe_route",
    "fp4_moe_experts",
    "moe_workspace_bytes",
    "fp4_abi_version",
    "group_size",
]

FP4_MXFP4 = 0
FP4_NVFP4 = 1
_FMT = {"mxfp4": FP4_MXFP4, "nvfp4": FP4_NVFP4, FP4_MXFP4: FP4_MXFP4, FP4_NVFP4: FP4_NVFP4}
_STATUS = {0: "OK", -1: "NULLPTR", -2: "SHAPE", -3: "BLOCK", -4: "FORMAT", -5: "ALIGN", -6: "HIP"}

_HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None


class Fp4Error(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"[{_STATUS.get(status, status)}] {message}")
        self.status = status


def library_path() -> str:
    return os.path.join(_HERE, "libfp4.so")


def load_library() -> ctypes.CDLL:
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is not built; build it with `python -m microscaling_fp4_quantized_amd.build` "
            "(there is no fallback path)")
    lib = ctypes.CDLL(path)
    i64, vp, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    q_args = [vp, i64, i64, i64, i32, i32, vp, vp, vp, vp]
    for name in ("fp4_rotate_quantize", "fp4_quantize_weights"):
        f = getattr(lib, name)
        f.argtypes = q_args
        f.restype = i32
    qx_args = [vp, i64, i64, i64, i32, i32, i32, vp, vp, vp, vp, vp]
    for name in ("fp4_rotate_quantize_ex", "fp4_quantize_weights_ex"):
        f = getattr(lib, name)
        f.argtypes = qx_args
        f.restype = i32
    lib.fp4_rotate_quantize_linear.argtypes = [vp, i64, i64, i64, i32, vp, vp, i64, vp, i32, vp, ctypes.c_size_t, vp]
    lib.fp4_rotate_quantize_linear.restype = i32
    lib.fp4_rotate_quantize_linear_noalloc.argtypes = [vp, i64, i64, i64, i32, vp, vp, i64, vp, i32, vp]
    lib.fp4_rotate_quantize_linear_noalloc.restype = i32
    lib.fp4_linear.argtypes = [vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, i32, vp]
    lib.fp4_linear.restype = i32
    for name in ("fp8_quantize", "fp8_quantize_weights"):
        f = getattr(lib, name)
        f.argtypes = [vp, i64, i64, i64, vp, vp, vp]
        f.restype = i32
    lib.fp8_add_rmsnorm_quantize.argtypes = [vp, i64, i64, i64, vp, i64, vp, ctypes.c_float, vp, vp, vp, vp, vp]
    lib.fp8_add_rmsnorm_quantize.restype = i32
    lib.fp8_linear.argtypes = [vp, vp, vp, vp, i64, i64, i64, vp, vp]
    lib.fp8_linear.restype = i32
    lib.fp4_moe_route.argtypes = [vp, i64, i64, i64, vp, i64, i32, i32, vp, vp, vp, ctypes.c_size_t, vp]
    lib.fp4_moe_route.restype = i32
    lib.fp4_moe_experts.argtypes = [vp, i64, i64, i64, vp, vp, i32, i64, i64, i32, vp, vp, vp, vp, vp, vp,
                                    ctypes.c_size_t, vp]
    lib.fp4_moe_experts.restype = i32
    lib.fp4_last_error.argtypes = []
    lib.fp4_last_error.restype = ctypes.c_char_p
    lib.fp4_abi_version.argtypes = []
    lib.fp4_abi_version.restype = i32
    _LIB = lib
    return lib


def group_size(fmt) -> int:
    return 32 if _FMT[fmt] == FP4_MXFP4 else 16


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(dev):
    """The handle of the device's current stream. torch.cuda.current_stream builds a Stream object around it
    (1.7 us a call, a fifth of a small call's host time); the raw form returns the number (0.06 us)."""
    if _RAW_STREAM is not None:
        return _RAW_STREAM(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


_RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_FAST = None


class _Fast:
    """The compiled module's functions, bound to the library's entry points."""

    def __init__(self, module, lib):
        def bind(function, name):
            entry = ctypes.cast(getattr(lib, name), ctypes.c_void_p).value

            def call(*args):
                index = torch.cuda.current_device()
                return function(entry, index, _RAW_STREAM(index), *args)
            return call

        self.quantize = {name: bind(module.quantize, name) for name in ("fp8_quantize", "fp8_quantize_weights")}
        self.norm = bind(module.norm, "fp8_add_rmsnorm_quantize")
        self.linear = bind(module.linear, "fp8_linear")
        self.route = bind(module.route, "fp4_moe_route")
        self.experts = bind(module.experts, "fp4_moe_experts")


def _compiled(lib):
    """The compiled calls for this library, or False: not built, built for another ABI, or no raw stream handles."""
    try:
        from . import _torch_calls
    except ImportError:
        return False
    if getattr(_torch_calls, "ABI_VERSION", None) != lib.fp4_abi_version() or _RAW_STREAM is None:
        return False
    return _Fast(_torch_calls, lib)


def _fast(t):
    """The compiled calls (_torch_calls.so) for calls with given outputs on the GPU, where the interpreter's share of
    a small call counts; None without them. They return a status, or None for operands that they leave to the checks
    below, which launch or refuse."""
    global _FAST
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        return None
    if _FAST is None:
        _FAST = _compiled(load_library())
    return _FAST or None


def _launch(dev, fn, *args):
    """Call an entry point with the operands' device current (the library launches on the current
    device) and that device's current stream as the last argument."""
    for t in args:
        if isinstance(t, torch.Tensor):
            raise TypeError("pass data pointers, not tensors")
    if dev.index is not None and torch.cuda.current_device() != dev.index:
        with torch.cuda.device(dev):
            return fn(*args, _stream(dev))
    return fn(*args, _stream(dev))


def _enqueue(fn, dev, *args):
    """Call an entry point on the operands' device and its current stream; raise what it refuses."""
    index = dev.index
    if torch.cuda.current_device() == index:
        status = fn(*args, _stream(dev))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _stream(dev))
    if status:
        _check(status)


def _same_device(name, dev, *tensors):
    for t in tensors:
        if isinstance(t, torch.Tensor) and t.device != dev:
            raise ValueError(f"{name}: every operand must be on {dev}, got one on {t.device}")


def _check(status: int):
    if status:
        raise Fp4Error(status, load_library().fp4_last_error().decode())


SCALE_RULES = {"standard": 0, "ocp_floor": 1, "oas": 2, "fit": 3}
TENSOR_SCALE_IN = 0x10


def _expect(t, shape, dtype, name, what):
    """Refuse anything but a contiguous CUDA tensor of this shape and dtype: the kernels take plain
    pointers and trust the sizes they imply, so a short buffer would be read or written out of bounds."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or t.dtype != dtype or \
            t.shape != shape or not t.is_contiguous():
        got = repr(t) if not isinstance(t, torch.Tensor) else f"{tuple(t.shape)} {t.dtype} on {t.device}"
        raise ValueError(f"{name}: {what} must be a contiguous {dtype} CUDA tensor of shape {tuple(shape)}, got {got}")


def _quantize(name: str, x: torch.Tensor, block: int, fmt, out=None, rule=None, signs=None, tensor_scale=None):
    lib = load_library()
    f = _FMT[fmt]
    if x.dim() != 2 or x.dtype != torch.bfloat16 or not x.is_cuda or x.stride(1) != 1:
        raise ValueError(f"{name}: expects a 2-D bf16 CUDA tensor with unit column stride")
    M, K = x.shape
    g = group_size(f)
    if out is None:
        codes = torch.empty((M, K // 2), dtype=torch.uint8, device=x.device)
        scales = torch.empty((M, K // g), dtype=torch.uint8, device=x.device)
        ts = torch.empty((1,), dtype=torch.float32, device=x.device) if f == FP4_NVFP4 else None
    else:
        codes, scales, ts = out
        _expect(codes, (M, K // 2), torch.uint8, name, "codes")
        _expect(scales, (M, K // g), torch.uint8, name, "scales")
        if f == FP4_NVFP4:
            if tensor_scale is None:
                _expect(ts, (1,), torch.float32, name, "tensor scale")
        elif ts is not None:
            raise ValueError(f"{name}: MXFP4 has no tensor scale")
    if tensor_scale is not None:
        # a given s_t: a device float32 [1] that the call reads and leaves unchanged
        if tensor_scale.dtype != torch.float32 or not tensor_scale.is_cuda or tensor_scale.numel() != 1:
            raise ValueError(f"{name}: tensor_scale must be a float32 CUDA tensor of one element")
        ts = tensor_scale
    _same_device(name, x.device, codes, scales, ts, signs, tensor_scale)
    if rule is None and signs is None and tensor_scale is None:
        _check(_launch(x.device, getattr(lib, name), _ptr(x), M, K, x.stride(0), int(block), f, _ptr(codes),
                       _ptr(scales), _ptr(ts)))
    else:
        if signs is not None and (signs.dtype != torch.int8 or not signs.is_cuda or signs.numel() != K
                                  or not signs.is_contiguous()):
            raise ValueError(f"{name}: signs must be a contiguous int8 CUDA tensor of K entries")
        r = SCALE_RULES[rule or "standard"] | (TENSOR_SCALE_IN if tensor_scale is not None else 0)
        _check(_launch(x.device, getattr(lib, name + "_ex"), _ptr(x), M, K, x.stride(0), int(block), f, r,
                       _ptr(signs), _ptr(codes), _ptr(scales), _ptr(ts)))
    return codes, scales, ts


def fp4_rotate_quantize(x: torch.Tensor, block: int, fmt="mxfp4", out=None, rule=None, signs=None,
                        tensor_scale=None):
    """Online block-Hadamard rotation + FP4 quantization of bf16 activations.

    Returns (codes [M, K/2] uint8, scales [M, K/g] uint8, tensor_scale [1] float32 or None).
    ``out`` may pass preallocated (codes, scales, tensor_scale). ``rule`` ("standard",
    "ocp_floor", "oas", "fit"), ``signs`` (int8 [K] of +-1) and ``tensor_scale`` (NVFP4: a
    given s_t, float32 [1] on the device) select fp4_rotate_quantize_ex.
    """
    return _quantize("fp4_rotate_quantize", x, block, fmt, out, rule, signs, tensor_scale)


def fp4_quantize_weights(w: torch.Tensor, block: int, fmt="mxfp4", out=None, rule=None, signs=None,
                         tensor_scale=None):
    """Offline rotation + quantization of a weight matrix [N, K] (same contract)."""
    return _quantize("fp4_quantize_weights", w, block, fmt, out, rule, signs, tensor_scale)


def fp4_linear(xq, xs, wq, ws, fmt="mxfp4", x_ts=None, w_ts=None, out_dtype=torch.float32, out=None):
    """Y = dq(Xq) dq(Wq)^T, [M, N] in float32 or bf16."""
    lib = load_library()
    f = _FMT[fmt]
    for t in (xq, wq):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError("fp4_linear: Xq and Wq must be 2-D tensors of packed codes")
    M, N, K = xq.shape[0], wq.shape[0], 2 * xq.shape[1]
    if wq.shape[1] * 2 != K:
        raise ValueError("fp4_linear: X and W disagree on K")
    g = group_size(f)
    _expect(xq, (M, K // 2), torch.uint8, "fp4_linear", "Xq")
    _expect(wq, (N, K // 2), torch.uint8, "fp4_linear", "Wq")
    _expect(xs, (M, K // g), torch.uint8, "fp4_linear", "Xs")
    _expect(ws, (N, K // g), torch.uint8, "fp4_linear", "Ws")
    if f == FP4_NVFP4:
        _expect(x_ts, (1,), torch.float32, "fp4_linear", "x_ts")
        _expect(w_ts, (1,), torch.float32, "fp4_linear", "w_ts")
    elif x_ts is not None or w_ts is not None:
        raise ValueError("fp4_linear: MXFP4 has no tensor scales")
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("fp4_linear: out_dtype must be torch.float32 or torch.bfloat16")
    ydt = {torch.float32: 0, torch.bfloat16: 1}[out_dtype]
    if out is None:
        y = torch.empty((M, N), dtype=out_dtype, device=xq.device)
    else:
        _expect(out, (M, N), out_dtype, "fp4_linear", "out")
        y = out
    _same_device("fp4_linear", xq.device, xs, wq, ws, x_ts, w_ts, y)
    _check(_launch(xq.device, lib.fp4_linear, _ptr(xq), _ptr(xs), _ptr(x_ts), _ptr(wq), _ptr(ws), _ptr(w_ts), M, N,
                   K, f, _ptr(y), ydt))
    return y


def linear_workspace_bytes(M: int, K: int) -> int:
    """FP4_LINEAR_WORKSPACE_BYTES(M, K) of include/fp4.h: X's codes, then its scales at the next
    256-byte boundary."""
    return ((M * K // 2 + 255) // 256) * 256 + M * K // 32


def fp4_rotate_quantize_linear(x: torch.Tensor, wq, ws, block: int, out_dtype=torch.float32, out=None,
                               workspace="auto"):
    """Decode step (MXFP4, 1 <= M <= 16): Y = fp4_linear(fp4_rotate_quantize(x), wq, ws).

    workspace: "auto" allocates one of linear_workspace_bytes(M, K) bytes, which lets the library
    take two launches where that is faster; None forces the one-launch kernel; or a contiguous
    uint8 CUDA tensor of at least that size."""
    lib = load_library()
    if x.dim() != 2 or x.dtype != torch.bfloat16 or not x.is_cuda or x.stride(1) != 1:
        raise ValueError("fp4_rotate_quantize_linear: expects a 2-D bf16 CUDA tensor with unit column stride")
    for t in (wq, ws):
        if not t.is_cuda or t.dtype != torch.uint8 or not t.is_contiguous():
            raise ValueError("fp4_rotate_quantize_linear: weight codes and scales must be contiguous uint8 CUDA tensors")
    M, K = x.shape
    if wq.dim() != 2 or wq.shape[1] * 2 != K:
        raise ValueError("fp4_rotate_quantize_linear: X and W disagree on K")
    N = wq.shape[0]
    _expect(ws, (N, K // 32), torch.uint8, "fp4_rotate_quantize_linear", "Ws")
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("fp4_rotate_quantize_linear: out_dtype must be torch.float32 or torch.bfloat16")
    ydt = {torch.float32: 0, torch.bfloat16: 1}[out_dtype]
    if out is None:
        y = torch.empty((M, N), dtype=out_dtype, device=x.device)
    else:
        _expect(out, (M, N), out_dtype, "fp4_rotate_quantize_linear", "out")
        y = out
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError('fp4_rotate_quantize_linear: workspace must be "auto", None or a uint8 tensor')
        workspace = torch.empty(linear_workspace_bytes(M, K), dtype=torch.uint8, device=x.device)
    if workspace is None:
        wsp, wsb = None, 0
        _same_device("fp4_rotate_quantize_linear", x.device, wq, ws, y)
    else:
        if not workspace.is_cuda or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
            raise ValueError("fp4_rotate_quantize_linear: workspace must be a contiguous uint8 CUDA tensor")
        if workspace.numel() < linear_workspace_bytes(M, K):
            raise ValueError("fp4_rotate_quantize_linear: workspace too small")
        wsp, wsb = _ptr(workspace), workspace.numel()
        _same_device("fp4_rotate_quantize_linear", x.device, wq, ws, y, workspace)
    _check(_launch(x.device, lib.fp4_rotate_quantize_linear, _ptr(x), M, K, x.stride(0), int(block), _ptr(wq),
                   _ptr(ws), N, _ptr(y), ydt, wsp, wsb))
    return y


def fp4_rotate_quantize_linear_noalloc(x: torch.Tensor, wq, ws, block: int, out_dtype=torch.float32, out=None):
    """The decode step through the allocation-free entry point: where two launches pay off, the
    library uses its own per-GPU array instead of a workspace. Calls that overlap on one GPU race
    on that array. With `out` given, nothing is allocated here either."""
    lib = load_library()
    if x.dim() != 2 or x.dtype != torch.bfloat16 or not x.is_cuda or x.stride(1) != 1:
        raise ValueError("fp4_rotate_quantize_linear_noalloc: expects a 2-D bf16 CUDA tensor with unit column stride")
    for t in (wq, ws):
        if not t.is_cuda or t.dtype != torch.uint8 or not t.is_contiguous():
            raise ValueError("fp4_rotate_quantize_linear_noalloc: weight codes and scales must be contiguous uint8 "
                             "CUDA tensors")
    M, K = x.shape
    if wq.dim() != 2 or wq.shape[1] * 2 != K:
        raise ValueError("fp4_rotate_quantize_linear_noalloc: X and W disagree on K")
    N = wq.shape[0]
    _expect(ws, (N, K // 32), torch.uint8, "fp4_rotate_quantize_linear_noalloc", "Ws")
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("fp4_rotate_quantize_linear_noalloc: out_dtype must be torch.float32 or torch.bfloat16")
    ydt = {torch.float32: 0, torch.bfloat16: 1}[out_dtype]
    if out is None:
        y = torch.empty((M, N), dtype=out_dtype, device=x.device)
    else:
        _expect(out, (M, N), out_dtype, "fp4_rotate_quantize_linear_noalloc", "out")
        y = out
    _same_device("fp4_rotate_quantize_linear_noalloc", x.device, wq, ws, y)
    _check(_launch(x.device, lib.fp4_rotate_quantize_linear_noalloc, _ptr(x), M, K, x.stride(0), int(block),
                   _ptr(wq), _ptr(ws), N, _ptr(y), ydt))
    return y


FP8_GROUP = 128  # values along K (and rows of a weight matrix) that share an 8-bit scale


def _rows(t, name, what):
    """A 2-D bf16 CUDA tensor of rows with unit column stride: its shape and row stride."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or t.dtype != torch.bfloat16 or not t.is_cuda or t.stride(1) != 1:
        raise ValueError(f"{name}: {what} must be a 2-D bf16 CUDA tensor with unit column stride")
    # the stride of a single row says nothing: torch may give any
    return t.shape[0], t.shape[1], t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _quantize8(name, x, rows, out):
    fast = _fast(x) if out is not None else None
    if fast:
        codes, scales = out
        status = fast.quantize[name](x, rows, codes, scales)
        if status is not None:
            _check(status)
            return codes, scales
    lib = load_library()
    M, K, ld = _rows(x, name, "the input")
    shape = (-(-M // rows), K // FP8_GROUP)
    if out is None:
        codes = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=x.device)
        scales = torch.empty(shape, dtype=torch.float32, device=x.device)
    else:
        codes, scales = out
        _expect(codes, (M, K), torch.float8_e4m3fn, name, "codes")
        _expect(scales, shape, torch.float32, name, "scales")
        _same_device(name, x.device, codes, scales)
    _enqueue(getattr(lib, name), x.device, x.data_ptr(), M, K, ld, codes.data_ptr(), scales.data_ptr())
    return codes, scales


def fp8_quantize(x: torch.Tensor, out=None):
    """bf16 activations [M, K] -> (codes [M, K] float8_e4m3fn, scales [M, K/128] float32).

    One scale for 128 consecutive values of a row; K a multiple of 128. ``out`` may pass
    preallocated (codes, scales)."""
    return _quantize8("fp8_quantize", x, 1, out)


def fp8_quantize_weights(w: torch.Tensor, out=None):
    """bf16 weights [N, K] -> (codes [N, K] float8_e4m3fn, scales [ceil(N/128), K/128] float32), one scale
    for a block of 128 x 128."""
    return _quantize8("fp8_quantize_weights", w, FP8_GROUP, out)


def fp8_add_rmsnorm_quantize(x: torch.Tensor, weight: torch.Tensor, residual=None, eps: float = 1e-6,
                             normed: bool = False, out=None):
    """h = x + residual; n = h / sqrt(mean(h^2) + eps) * weight; n quantized as fp8_quantize does.

    Returns (codes, scales, h in bf16 or None without a residual, n in bf16 or None unless ``normed``).
    ``out`` may pass those four preallocated (None where there is none); h may be the residual itself,
    which is then updated in place."""
    name = "fp8_add_rmsnorm_quantize"
    fast = _fast(x) if out is not None else None
    if fast:
        codes, scales, h, n = out
        if (h is None) == (residual is None) and (n is None) != bool(normed):
            status = fast.norm(x, weight, residual, eps, codes, scales, h, n)
            if status is not None:
                _check(status)
                return codes, scales, h, n
    lib = load_library()
    M, K, ld = _rows(x, name, "x")
    dev = x.device
    _expect(weight, (K,), torch.bfloat16, name, "weight")
    ldr = 0
    if residual is not None:
        Mr, Kr, ldr = _rows(residual, name, "residual")
        if (Mr, Kr) != (M, K):
            raise ValueError(f"{name}: residual must have the shape of x, {(M, K)}, got {(Mr, Kr)}")
    if out is None:
        codes = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=dev)
        scales = torch.empty((M, K // FP8_GROUP), dtype=torch.float32, device=dev)
        h = torch.empty((M, K), dtype=torch.bfloat16, device=dev) if residual is not None else None
        n = torch.empty((M, K), dtype=torch.bfloat16, device=dev) if normed else None
    else:
        codes, scales, h, n = out
        _expect(codes, (M, K), torch.float8_e4m3fn, name, "codes")
        _expect(scales, (M, K // FP8_GROUP), torch.float32, name, "scales")
        if (h is None) != (residual is None) or (n is None) == bool(normed):
            raise ValueError(f"{name}: out must hold the residual's sum exactly with a residual, and the normed rows "
                             "exactly with normed")
        for t, what in ((h, "the residual's sum"), (n, "the normed rows")):
            if t is not None:
                _expect(t, (M, K), torch.bfloat16, name, what)
    _same_device(name, dev, weight, residual, codes, scales, h, n)
    _enqueue(lib.fp8_add_rmsnorm_quantize, dev, x.data_ptr(), M, K, ld,
             residual.data_ptr() if residual is not None else None, ldr, weight.data_ptr(), eps, codes.data_ptr(),
             scales.data_ptr(), h.data_ptr() if h is not None else None, n.data_ptr() if n is not None else None)
    return codes, scales, h, n


def fp8_linear(xq, xs, wq, ws, out=None):
    """Y = dq(Xq) dq(Wq)^T, [M, N] in bf16, from the outputs of fp8_quantize (or
    fp8_add_rmsnorm_quantize) and fp8_quantize_weights."""
    name = "fp8_linear"
    fast = _fast(xq) if out is not None else None
    if fast:
        status = fast.linear(xq, xs, wq, ws, out)
        if status is not None:
            _check(status)
            return out
    lib = load_library()
    for t in (xq, wq):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError(f"{name}: Xq and Wq must be 2-D tensors of codes")
    M, K = xq.shape
    N = wq.shape[0]
    _expect(xq, (M, K), torch.float8_e4m3fn, name, "Xq")
    _expect(wq, (N, K), torch.float8_e4m3fn, name, "Wq")
    _expect(xs, (M, K // FP8_GROUP), torch.float32, name, "Xs")
    _expect(ws, (-(-N // FP8_GROUP), K // FP8_GROUP), torch.float32, name, "Ws")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=xq.device)
    else:
        _expect(out, (M, N), torch.bfloat16, name, "out")
    _same_device(name, xq.device, xs, wq, ws, out)
    _enqueue(lib.fp8_linear, xq.device, xq.data_ptr(), xs.data_ptr(), wq.data_ptr(), ws.data_ptr(), M, N, K,
             out.data_ptr())
    return out


def _workspace(workspace, need, name, dev):
    if isinstance(workspace, str) and workspace == "auto":
        return torch.empty(need, dtype=torch.uint8, device=dev)
    if not isinstance(workspace, torch.Tensor) or not workspace.is_cuda or workspace.dtype != torch.uint8 or \
            not workspace.is_contiguous():
        raise ValueError(f'{name}: workspace must be "auto" or a contiguous uint8 CUDA tensor')
    if workspace.numel() < need:
        raise ValueError(f"{name}: workspace too small, {need} bytes needed")
    return workspace


def fp4_moe_route(x: torch.Tensor, router: torch.Tensor, k: int, renormalize: bool = True, out=None, workspace="auto"):
    """softmax(x router^T) in float32 and its k largest of each token: (ids [T, k] int32, weights [T, k] float32).

    x bf16 [T, D], T at most 1048560, router bf16 [E, D]. Of equal weights the lowest expert comes first. ``out`` may pass
    preallocated (ids, weights); workspace: "auto", or a uint8 CUDA tensor of at least 16 T E bytes."""
    name = "fp4_moe_route"
    if not isinstance(router, torch.Tensor) or router.dim() != 2:
        raise ValueError(f"{name}: router must be a 2-D tensor")
    E, k = router.shape[0], int(k)
    fast = _fast(x) if out is not None else None
    if fast and x.dim() == 2:
        ids, weights = out
        ws = _workspace(workspace, 16 * x.shape[0] * E, name, x.device)
        status = fast.route(x, router, k, bool(renormalize), ids, weights, ws)
        if status is not None:
            _check(status)
            return ids, weights
    lib = load_library()
    T, D, ld = _rows(x, name, "x")
    _expect(router, (E, D), torch.bfloat16, name, "router")
    if out is None:
        ids = torch.empty((T, k), dtype=torch.int32, device=x.device)
        weights = torch.empty((T, k), dtype=torch.float32, device=x.device)
    else:
        ids, weights = out
        _expect(ids, (T, k), torch.int32, name, "ids")
        _expect(weights, (T, k), torch.float32, name, "weights")
    ws = _workspace(workspace, 16 * T * E, name, x.device)
    _same_device(name, x.device, router, ids, weights, ws)
    _enqueue(lib.fp4_moe_route, x.device, x.data_ptr(), T, D, ld, router.data_ptr(), E, k, int(bool(renormalize)),
             ids.data_ptr(), weights.data_ptr(), ws.data_ptr(), ws.numel())
    return ids, weights


def moe_workspace_bytes(T: int, k: int, D: int, I: int) -> int:
    """FP4_MOE_WORKSPACE_BYTES(T, k, D, I) of include/fp4.h."""
    def pad(n):
        return (n + 255) // 256 * 256
    P = T * k
    return pad(T * 4 * D) + pad(T * D // 32) + pad(P * I * 4) + pad(P * 4 * I) + pad(P * I // 32) + pad(P * D * 4) + 84 * P


def fp4_moe_experts(x: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, w13q, w13s, w2q, w2s, block: int,
                    out=None, workspace="auto"):
    """y_t = sum_j weights[t, j] W2[e] H (silu(G[e] H x_t) * (U[e] H x_t)), e = ids[t, j]: the experts of a
    mixture-of-experts layer for up to 128 tokens (more go in slices of 128), [T, D] in bf16.

    x bf16 [T, D]; ids int32 and weights float32 [T, k] (fp4_moe_route); an id outside [0, E) leaves its slot out.
    The experts' matrices are MXFP4 from fp4_quantize_weights with this ``block``: w13q uint8 [E, 2I, D/2] and w13s
    [E, 2I, D/32], gate rows first, w2q [E, D, I/2] and w2s [E, D, I/32]. workspace: "auto", or a uint8 CUDA
    tensor of at least moe_workspace_bytes(T, k, D, I)."""
    name = "fp4_moe_experts"
    fast = _fast(x) if out is not None else None
    if fast and isinstance(ids, torch.Tensor) and isinstance(w2q, torch.Tensor) and \
            x.dim() == ids.dim() == 2 and w2q.dim() == 3:
        ws = _workspace(workspace, moe_workspace_bytes(*ids.shape, x.shape[1], 2 * w2q.shape[2]), name, x.device)
        status = fast.experts(x, ids, weights, w13q, w13s, w2q, w2s, block, out, ws)
        if status is not None:
            _check(status)
            return out
    lib = load_library()
    T, D, ld = _rows(x, name, "x")
    for t, what in ((w13q, "w13q"), (w2q, "w2q")):
        if not isinstance(t, torch.Tensor) or t.dim() != 3:
            raise ValueError(f"{name}: {what} must be a 3-D tensor of codes")
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError(f"{name}: ids must be a 2-D tensor")
    E, I, k = w13q.shape[0], 2 * w2q.shape[2], ids.shape[1]
    _expect(ids, (T, k), torch.int32, name, "ids")
    _expect(weights, (T, k), torch.float32, name, "weights")
    _expect(w13q, (E, 2 * I, D // 2), torch.uint8, name, "w13q")
    _expect(w13s, (E, 2 * I, D // 32), torch.uint8, name, "w13s")
    _expect(w2q, (E, D, I // 2), torch.uint8, name, "w2q")
    _expect(w2s, (E, D, I // 32), torch.uint8, name, "w2s")
    if out is None:
        out = torch.empty((T, D), dtype=torch.bfloat16, device=x.device)
    else:
        _expect(out, (T, D), torch.bfloat16, name, "out")
    ws = _workspace(workspace, moe_workspace_bytes(T, k, D, I), name, x.device)
    _same_device(name, x.device, ids, weights, w13q, w13s, w2q, w2s, out, ws)
    _enqueue(lib.fp4_moe_experts, x.device, x.data_ptr(), T, D, ld, ids.data_ptr(), weights.data_ptr(), k, E, I,
             int(block), w13q.data_ptr(), w13s.data_ptr(), w2q.data_ptr(), w2s.data_ptr(), out.data_ptr(),
             ws.data_ptr(), ws.numel())
    return out


def fp4_abi_version() -> int:
    return load_library().fp4_abi_version()
