"""Python binding of libpk: packed-sequence RoPE attention forward on GB300.

Argument marshalling only: every step of the computation runs in the CUDA library
(`libpk.so`, built from `csrc/` by `build.py`); there is no fallback of any kind. If the
library is missing or cannot load, every call raises.

The entry points mirror include/pk.h:
    attend(qkv, cos, sin, cu, H, window, scale, out=None, lse=None, stream=None, tuned=False)
    pk_attend(qkv, cos, sin, cu, S, T, H, window, scale, out, lse, stream)   (raw pointers)
    schedule(cu, T, window)      -> tile records [NT, 8]
    last_status(stream=None)     -> int

and, on the token rows of the same packed batch:
    linear(x, w, bias, residual, act, p, seed, offset)          linear_backward(x, w, dy, pre, act, p, seed, offset)
    dropout(x, p, seed, offset, residual)                       dropout_backward(dy, p, seed, offset)
    cross_entropy(x, w, labels, bias) -> loss, lse              cross_entropy_backward(x, w, labels, lse, dloss, bias)
    rms_norm(x, w, residual, eps) -> y, h                       rms_norm_backward(h, w, dy, dh, eps)
    gated_linear(x, w, bias, act)                               gated_linear_backward(x, w, dy, pre, act)
    token_logprobs(logits, labels, top)                         token_logprobs_backward(logits, labels, lse, entropy, dlogp, dentropy)
    distill(x, w, idx, values, bias, temperature)               distill_backward(x, w, idx, values, lse, dloss, bias, temperature)
    rms_norm_q8, quantize_rows -> rows in e4m3, scales          linear_q8(xq, xs, wq, ws, bias, residual, act, out_dtype)
"""

from __future__ import annotations

import ctypes
import functools
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpk.so")

PK_F32, PK_BF16, PK_F16 = 0, 1, 2
STATUS = {
    0: "PK_OK", 1: "PK_ERR_ARG", 2: "PK_ERR_ALIGN", 3: "PK_ERR_CUDA", 4: "PK_ERR_UNSUPPORTED",
    5: "PK_ERR_BAD_CU", 6: "PK_ERR_TIMEOUT", 7: "PK_ERR_NOMEM", 8: "PK_ERR_INTERNAL",
    9: "PK_ERR_TOO_LARGE", 10: "PK_ERR_CAPTURE", 11: "PK_ERR_BAD_LABEL",
}
ACTS = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}
NOALLOC_MAX_T = 1048576
NORM_MAX_D = 16384
LOGPROBS_MAX_TOP = 64
DISTILL_MAX_TOP = 64
LINEAR_FEW_T = 8  # include/pk.h: half as many rows of any type need no workspace in linear

# names declared in include/pk.h
EXPORTS = ("pk_attend", "pk_attend_bf16", "pk_attend_f16", "pk_attend_f32", "pk_attend_dt",
           "pk_schedule", "pk_schedule_capacity", "pk_last_status", "pk_status_string",
           "pk_version", "pk_release", "pk_profile_start", "pk_profile_stop", "pk_attend_noalloc", "pk_rope", "pk_attend_mixed",
           "pk_attend_backward", "pk_attend_tuned", "pk_tune_pick", "pk_tune_key", "pk_tune_clear",
           "pk_forward_kernel", "pk_kernel_name", "pk_attend_mixed_ops",
           "pk_linear", "pk_linear_workspace", "pk_linear_backward", "pk_linear_backward_workspace", "pk_dropout",
           "pk_cross_entropy", "pk_cross_entropy_backward", "pk_cross_entropy_workspace",
           "pk_rms_norm", "pk_rms_norm_q8", "pk_quantize_rows", "pk_rms_norm_backward", "pk_rms_norm_backward_workspace",
           "pk_token_logprobs", "pk_token_logprobs_backward",
           "pk_gated_linear", "pk_gated_linear_workspace", "pk_gated_linear_backward", "pk_gated_linear_backward_workspace",
           "pk_linear_q8", "pk_linear_q8_workspace", "pk_distill", "pk_distill_backward", "pk_distill_workspace")
KERNELS = {0: "band", 1: "f32", 2: "tc", 3: "q4", 4: "tc_single", 5: "split"}

_lib = None


class PKError(RuntimeError):
    def __init__(self, code: int, what: str = ""):
        self.code = code
        msg = f"{STATUS.get(code, code)}: {status_string(code) if _lib else ''}"
        super().__init__(f"{what}: {msg}" if what else msg)


def load(path: str | None = None):
    """Load libpk.so (raises if it is missing: there is no other implementation)."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"libpk.so not built ({p}); run __graft_entry__.build()")
    L = ctypes.CDLL(p)
    vp, i32, i64, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float
    sig = [vp, vp, vp, vp, i32, i64, i32, i32, f32, vp, vp, vp]
    for name in ("pk_attend", "pk_attend_bf16", "pk_attend_f16", "pk_attend_f32"):
        getattr(L, name).argtypes = sig
        getattr(L, name).restype = i32
    L.pk_attend_dt.argtypes = [i32] + sig
    L.pk_attend_dt.restype = i32
    L.pk_attend_noalloc.argtypes = [i32] + sig[:11] + [vp, vp]
    L.pk_attend_noalloc.restype = i32
    L.pk_attend_backward.argtypes = [i32, vp, vp, vp, vp, i32, i64, i32, i32, f32, vp, vp, vp, vp, vp]
    L.pk_attend_backward.restype = i32
    L.pk_attend_mixed.argtypes = [i32] + sig
    L.pk_attend_mixed.restype = i32
    L.pk_attend_mixed_ops.argtypes = [i32] + sig
    L.pk_attend_mixed_ops.restype = i32
    L.pk_attend_tuned.argtypes = [i32, vp, vp, vp, vp, i32, i64, i32, i32, f32, i64, vp, vp, vp]
    L.pk_attend_tuned.restype = i32
    L.pk_tune_pick.argtypes = [i32, i32, i32, i64, i64]
    L.pk_tune_pick.restype = i32
    L.pk_tune_key.argtypes = [i32, i32, i32, i64, i64, ctypes.c_char_p, i32]
    L.pk_tune_key.restype = i32
    L.pk_tune_clear.argtypes = []
    L.pk_tune_clear.restype = i32
    L.pk_forward_kernel.argtypes = [i32, i32]
    L.pk_forward_kernel.restype = i32
    L.pk_kernel_name.argtypes = [i32]
    L.pk_kernel_name.restype = ctypes.c_char_p
    L.pk_rope.argtypes = [i32, vp, vp, vp, vp, i64, vp, i32, i64, i32, i32, i32, i32, vp, vp]
    L.pk_rope.restype = i32
    L.pk_schedule.argtypes = [vp, i32, i64, i32, vp, i64, ctypes.POINTER(i64), vp]
    L.pk_schedule.restype = i32
    L.pk_schedule_capacity.argtypes = [i64]
    L.pk_schedule_capacity.restype = i64
    L.pk_last_status.argtypes = [vp]
    L.pk_last_status.restype = i32
    L.pk_status_string.argtypes = [i32]
    L.pk_status_string.restype = ctypes.c_char_p
    L.pk_version.argtypes = []
    L.pk_version.restype = i32
    L.pk_release.argtypes = []
    L.pk_release.restype = i32
    L.pk_profile_start.argtypes = [i32]
    L.pk_profile_start.restype = i32
    dp = ctypes.POINTER(ctypes.c_double)
    L.pk_profile_stop.argtypes = [dp, dp, ctypes.POINTER(i32)]
    L.pk_profile_stop.restype = i32
    u64, f64, pi64 = ctypes.c_uint64, ctypes.c_double, ctypes.POINTER(i64)
    tail = [vp, i64, vp, vp]  # workspace, its bytes, status, stream
    for name, args in {
        "pk_linear": [i32, vp, i64, vp, vp, vp, i64, i32, f64, u64, u64, i64, i32, i32, vp, i64, vp] + tail,
        "pk_linear_workspace": [i32, vp, i64, vp, i64, i32, i32, pi64],
        "pk_linear_backward": [i32, vp, i64, vp, vp, i64, vp, i32, f64, u64, u64, i64, i32, i32, vp, vp, vp] + tail,
        "pk_linear_backward_workspace": [i32, vp, i64, vp, vp, i64, i32, f64, i32, i32, i32, i64, i32, i32, pi64],
        "pk_dropout": [i32, vp, i64, vp, i64, f64, u64, u64, i64, i32, vp, i64, vp],
        "pk_cross_entropy": [i32, vp, i64, vp, vp, vp, i64, i32, i32, vp, vp] + tail,
        "pk_cross_entropy_backward": [i32, vp, i64, vp, vp, vp, vp, vp, i64, i32, i32, vp, vp, vp] + tail,
        "pk_cross_entropy_workspace": [i32, vp, i64, vp, i32, i32, i64, i32, i32, pi64],
        "pk_rms_norm": [i32, vp, i64, vp, i64, vp, f32, i64, i32, vp, i64, vp, i64, vp],
        "pk_rms_norm_q8": [i32, vp, i64, vp, i64, vp, f32, i64, i32, vp, i64, vp, vp, i64, vp],
        "pk_quantize_rows": [i32, vp, i64, i64, i32, vp, i64, vp, vp],
        "pk_rms_norm_backward": [i32, vp, i64, vp, vp, i64, vp, i64, f32, i64, i32, vp, i64, vp, vp, i64, vp],
        "pk_rms_norm_backward_workspace": [i32, i64, i32, i32, pi64],
        "pk_gated_linear": [i32, vp, i64, vp, vp, i32, i64, i32, i32, vp, i64, vp] + tail,
        "pk_gated_linear_workspace": [i32, vp, i64, vp, i64, i32, i32, pi64],
        "pk_gated_linear_backward": [i32, vp, i64, vp, vp, i64, vp, i32, i64, i32, i32, vp, vp, vp] + tail,
        "pk_gated_linear_backward_workspace": [i32, vp, i64, vp, i32, i32, i32, i64, i32, i32, pi64],
        "pk_linear_q8": [i32, vp, i64, vp, vp, vp, vp, vp, i64, i32, i64, i32, i32, vp, i64] + tail,
        "pk_linear_q8_workspace": [i64, i32, i32, pi64],
        "pk_distill": [i32, vp, i64, vp, vp, vp, vp, i32, f64, i64, i32, i32, vp, vp] + tail,
        "pk_distill_backward": [i32, vp, i64, vp, vp, vp, vp, i32, f64, vp, vp, i64, i32, i32, vp, vp, vp] + tail,
        "pk_distill_workspace": [i32, vp, i64, vp, i32, i32, i64, i32, i32, i32, pi64],
        "pk_token_logprobs": [i32, vp, i64, vp, i64, i32, i32, vp, vp, vp, vp, vp, vp, vp],
        "pk_token_logprobs_backward": [i32, vp, i64, vp, vp, vp, vp, vp, i64, i32, vp, i64, vp],
    }.items():
        getattr(L, name).argtypes = args
        getattr(L, name).restype = i32
    _lib = L
    return L


def status_string(code: int) -> str:
    return load().pk_status_string(int(code)).decode()


def _check(rc: int, what: str):
    if rc:
        raise PKError(rc, what)


# ------------------------------------------------------------------------------------------
# raw-pointer entry points (same names and argument order as the C ABI)


def pk_attend(qkv, cos, sin, cu, S, T, H, window, scale, out, lse, stream) -> int:
    return load().pk_attend(qkv, cos, sin, cu, S, T, H, window, scale, out, lse, stream)


def pk_attend_dt(dtype, qkv, cos, sin, cu, S, T, H, window, scale, out, lse, stream) -> int:
    return load().pk_attend_dt(dtype, qkv, cos, sin, cu, S, T, H, window, scale, out, lse, stream)


def pk_attend_noalloc(dtype, qkv, cos, sin, cu, S, T, H, window, scale, out, lse, status, stream) -> int:
    """The allocation-free variant (see include/pk.h): for callers that cannot let the library
    cudaMalloc a workspace; `status` is an optional device pointer to one int."""
    return load().pk_attend_noalloc(dtype, qkv, cos, sin, cu, S, T, H, window, scale, out, lse, status, stream)


def pk_attend_mixed_ops(op_dtype, qkv, cos, sin, cu, S, T, H, window, scale, out, lse, stream) -> int:
    """fp32 storage, 16-bit tensor-core operands, fp32 out (see include/pk.h)."""
    return load().pk_attend_mixed_ops(op_dtype, qkv, cos, sin, cu, S, T, H, window, scale, out, lse, stream)


def attend_mixed_ops(qkv, cos, sin, cu, H: int, window: int, scale: float, op_dtype, out=None, lse=None,
                     stream=None, max_len=None):
    """out [T, H*64] and lse [H, T], both float32, for float32 device tensors qkv [T, 3*H*64] and
    cos/sin [P, 32], the products on the tensor cores with operands of op_dtype
    (torch.float16 or torch.bfloat16)."""
    torch = _torch()
    if qkv.dtype != torch.float32:
        raise TypeError("qkv must be float32")
    _check_inputs(qkv, cos, sin, cu, H, 32)
    _check_stream(stream, qkv.device)
    code = {torch.float16: PK_F16, torch.bfloat16: PK_BF16}.get(op_dtype)
    if code is None:
        raise TypeError("op_dtype must be torch.float16 or torch.bfloat16")
    T = qkv.shape[0]
    with torch.cuda.device(qkv.device):
        _check_table_rows(cu, cos.shape[0], max_len)
        if out is None:
            out = torch.empty((T, H * 64), dtype=torch.float32, device=qkv.device)
        else:
            _need(out, (T, H * 64), torch.float32, "out")
        if lse is None:
            lse = torch.empty((H, T), dtype=torch.float32, device=qkv.device)
        else:
            _need(lse, (H, T), torch.float32, "lse")
        _same_device(qkv, out, lse)
        rc = pk_attend_mixed_ops(code, qkv.data_ptr(), cos.data_ptr(), sin.data_ptr(), cu.data_ptr(),
                                 cu.shape[0] - 1, T, H, window, float(scale), out.data_ptr(), lse.data_ptr(),
                                 _stream_handle(stream))
        _check(rc, "pk_attend_mixed_ops")
    return out, lse


def pk_attend_tuned(dtype, qkv, cos, sin, cu, S, T, H, window, scale, longest, out, lse, stream) -> int:
    """The forward pass at the fastest usable kernel for the shape, tuned once per key (see
    include/pk.h)."""
    return load().pk_attend_tuned(dtype, qkv, cos, sin, cu, S, T, H, window, scale, longest, out, lse, stream)


def pk_tune_pick(dtype, H, window, T, longest) -> int:
    return load().pk_tune_pick(dtype, H, window, T, longest)


def pk_tune_key(dtype, H, window, T, longest) -> str:
    buf = ctypes.create_string_buffer(128)
    _check(load().pk_tune_key(dtype, H, window, T, longest, buf, 128), "pk_tune_key")
    return buf.value.decode()


def pk_tune_clear() -> int:
    return load().pk_tune_clear()


def pk_forward_kernel(dtype, window) -> int:
    return load().pk_forward_kernel(dtype, window)


def pk_kernel_name(kernel) -> str:
    return load().pk_kernel_name(kernel).decode()


def pk_attend_backward(dtype, qkv, cos, sin, cu, S, T, H, window, scale, out, lse, dout, dqkv, stream) -> int:
    """The backward pass (see include/pk.h)."""
    return load().pk_attend_backward(dtype, qkv, cos, sin, cu, S, T, H, window, scale, out, lse, dout, dqkv, stream)


def pk_attend_mixed(out_dtype, qkv, cos, sin, cu, S, T, H, window, scale, out, lse, stream) -> int:
    """fp32 inputs and arithmetic, out in out_dtype (see include/pk.h)."""
    return load().pk_attend_mixed(out_dtype, qkv, cos, sin, cu, S, T, H, window, scale, out, lse, stream)


def pk_rope(dtype, x, y, cos, sin, P, cu, S, T, H, dims, traditional, inverse, status, stream) -> int:
    """The standalone rotation of the q and k head vectors of a packed qkv (see include/pk.h)."""
    return load().pk_rope(dtype, x, y, cos, sin, P, cu, S, T, H, dims, traditional, inverse, status, stream)


def pk_schedule(cu, S, T, window, tiles, cap, stream):
    nt = ctypes.c_int64(0)
    rc = load().pk_schedule(cu, S, T, window, tiles, cap, ctypes.byref(nt), stream)
    return rc, nt.value


def pk_last_status(stream) -> int:
    return load().pk_last_status(stream)


# ------------------------------------------------------------------------------------------
# torch-tensor front (torch only allocates and supplies the stream)


_torch_module = None
_codes = None  # enum pk_dtype of a torch type


def _torch():
    global _torch_module, _codes
    if _torch_module is None:
        import torch

        _codes = {torch.float32: PK_F32, torch.bfloat16: PK_BF16, torch.float16: PK_F16}
        _torch_module = torch
    return _torch_module


def _code(dtype) -> int:
    _torch()
    code = _codes.get(dtype)
    if code is None:
        raise TypeError(f"unsupported dtype {dtype}")
    return code


def dtype_code(t) -> int:
    return _code(t.dtype)


def _need(t, shape, dtype, what):
    """A caller's buffer must have exactly this shape and dtype and be a contiguous CUDA tensor:
    the C ABI receives only its address and writes the sizes the call implies."""
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype:
        raise ValueError(f"{what} must be {tuple(shape)} {dtype}, not {tuple(t.shape)} {t.dtype}")
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous CUDA tensor")


def _check_inputs(qkv, cos, sin, cu, H, half):
    """qkv [T, 3*H*64], cos/sin [P, half] of qkv's dtype, cu [S+1] int32/uint32; all contiguous
    CUDA tensors on one device."""
    torch = _torch()
    if qkv.dim() != 2 or qkv.shape[1] != 3 * H * 64:
        raise ValueError("qkv must be [T, 3*H*64]")
    if cos.dtype != qkv.dtype or sin.dtype != qkv.dtype or cos.shape != sin.shape:
        raise TypeError("cos/sin must have qkv's dtype and one shape")
    if cos.dim() != 2 or cos.shape[1] != half:
        raise ValueError(f"cos/sin must be [P, {half}]")
    if cu.dim() != 1 or cu.dtype not in (torch.int32, torch.uint32):
        raise TypeError("cu must be a 1-D int32 or uint32 tensor")
    for t in (qkv, cos, sin, cu):
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("inputs must be contiguous CUDA tensors")
    _same_device(qkv, cos, sin, cu)


def _same_device(first, *rest):
    """Every tensor on the device of the first: the library launches on one device and
    dereferences every address there."""
    for t in rest:
        if t.device != first.device:
            raise ValueError(f"tensors on different devices ({first.device} and {t.device})")


def _check_stream(stream, device):
    """A torch stream given for the call must belong to the tensors' device."""
    dev = getattr(stream, "device", None)
    if dev is not None and dev != device:
        raise ValueError(f"stream of {dev} for tensors on {device}")


def _check_table_rows(cu, rows: int, max_len):
    """The tables must hold a row for every in-sequence position: rows >= the longest sequence.
    Without max_len this reads the longest length back from the device (one reduction and a
    synchronisation; skipped while a CUDA graph is being captured, where the caller vouches
    for the tables)."""
    torch = _torch()
    if max_len is None:
        if cu.shape[0] < 2 or (cu.is_cuda and torch.cuda.is_current_stream_capturing()):
            return
        max_len = int((cu[1:].to(torch.int64) - cu[:-1].to(torch.int64)).max().item())
    if int(max_len) > rows:
        raise ValueError(f"cos/sin hold {rows} positions but a sequence has {int(max_len)} tokens")


def _stream_handle(stream):
    torch = _torch()
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def attend(qkv, cos, sin, cu, H: int, window: int, scale: float, out=None, lse=None, stream=None,
           out_dtype=None, max_len=None, tuned=False):
    """out [T, H*64] (qkv's dtype) and lse [H, T] float32 for device tensors qkv [T, 3*H*64],
    cos/sin [P, 32] (qkv's dtype) and cu [S+1] (int32 or uint32), all on one device. For
    float32 inputs, out_dtype=torch.float16 or torch.bfloat16 gives a 16-bit out
    (pk_attend_mixed). max_len: the longest sequence's length, if the caller knows it
    (otherwise it is read back from cu to check that the tables are long enough).
    tuned=True: pk_attend_tuned (the fastest usable kernel for the shape, tuned on the
    first call of each key; that call synchronizes the stream)."""
    torch = _torch()
    _check_inputs(qkv, cos, sin, cu, H, 32)
    _check_stream(stream, qkv.device)
    with torch.cuda.device(qkv.device):
        if tuned and max_len is None:
            max_len = _longest(cu)
        _check_table_rows(cu, cos.shape[0], max_len)
        return _attend(qkv, cos, sin, cu, H, window, scale, out, lse, stream, out_dtype,
                       max_len if tuned else None)


def _longest(cu) -> int:
    torch = _torch()
    if cu.shape[0] < 2:
        return 0
    return int((cu[1:].to(torch.int64) - cu[:-1].to(torch.int64)).max().item())


def _attend(qkv, cos, sin, cu, H, window, scale, out, lse, stream, out_dtype, tuned_longest=None):
    torch = _torch()
    T = qkv.shape[0]
    S = cu.shape[0] - 1
    # the output type: out_dtype, else a given out's, else qkv's
    odt = out_dtype if out_dtype is not None else (out.dtype if out is not None else qkv.dtype)
    if odt != qkv.dtype and qkv.dtype != torch.float32:
        raise TypeError("a different output type needs float32 inputs")
    if out is None:
        out = torch.empty((T, H * 64), dtype=odt, device=qkv.device)
    else:
        _need(out, (T, H * 64), odt, "out")
    if lse is None:
        lse = torch.empty((H, T), dtype=torch.float32, device=qkv.device)
    else:
        _need(lse, (H, T), torch.float32, "lse")
    _same_device(qkv, out, lse)
    if tuned_longest is not None and odt != qkv.dtype:
        raise TypeError("the tuned entry point writes out in qkv's type")
    if tuned_longest is not None:
        rc = pk_attend_tuned(dtype_code(qkv), qkv.data_ptr(), cos.data_ptr(), sin.data_ptr(), cu.data_ptr(),
                             S, T, H, window, float(scale), int(tuned_longest), out.data_ptr(), lse.data_ptr(),
                             _stream_handle(stream))
    elif odt != qkv.dtype:
        rc = pk_attend_mixed(dtype_code(out), qkv.data_ptr(), cos.data_ptr(), sin.data_ptr(), cu.data_ptr(),
                             S, T, H, window, float(scale), out.data_ptr(), lse.data_ptr(), _stream_handle(stream))
    else:
        rc = pk_attend_dt(dtype_code(qkv), qkv.data_ptr(), cos.data_ptr(), sin.data_ptr(), cu.data_ptr(),
                          S, T, H, window, float(scale), out.data_ptr(), lse.data_ptr(),
                          _stream_handle(stream))
    _check(rc, "pk_attend")
    return out, lse


def attend_backward(qkv, cos, sin, cu, H: int, window: int, scale: float, out, lse, dout, dqkv=None, stream=None,
                    max_len=None):
    """dqkv [T, 3*H*64] (qkv's dtype): the gradient of sum(dout * out) with respect to qkv, for
    the forward's out and lse (max_len as for attend)."""
    torch = _torch()
    T = qkv.shape[0]
    S = cu.shape[0] - 1
    _check_inputs(qkv, cos, sin, cu, H, 32)
    _need(out, (T, H * 64), qkv.dtype, "out")
    _need(dout, (T, H * 64), qkv.dtype, "dout")
    _need(lse, (H, T), torch.float32, "lse")
    if dqkv is not None:
        _need(dqkv, tuple(qkv.shape), qkv.dtype, "dqkv")
        _same_device(qkv, dqkv)
    _same_device(qkv, out, lse, dout)
    _check_stream(stream, qkv.device)
    with torch.cuda.device(qkv.device):
        _check_table_rows(cu, cos.shape[0], max_len)
        if dqkv is None:
            dqkv = torch.empty_like(qkv)
        return _attend_backward(qkv, cos, sin, cu, S, T, H, window, scale, out, lse, dout, dqkv, stream)


def _attend_backward(qkv, cos, sin, cu, S, T, H, window, scale, out, lse, dout, dqkv, stream):
    rc = pk_attend_backward(dtype_code(qkv), qkv.data_ptr(), cos.data_ptr(), sin.data_ptr(), cu.data_ptr(), S, T, H,
                            window, float(scale), out.data_ptr(), lse.data_ptr(), dout.data_ptr(), dqkv.data_ptr(),
                            _stream_handle(stream))
    _check(rc, "pk_attend_backward")
    return dqkv


def rope(qkv, cos, sin, cu, H: int, dims: int = 64, traditional: bool = False, inverse: bool = False,
         out=None, status=None, stream=None):
    """qkv [T, 3*H*64] with the first `dims` features of every q and k head vector rotated at
    their in-sequence positions (tables cos/sin [P, dims/2] in qkv's dtype); v copied. `out`
    may be qkv itself (in place). `status`: optional int32 device tensor of one element."""
    torch = _torch()
    T = qkv.shape[0]
    S = cu.shape[0] - 1
    _check_inputs(qkv, cos, sin, cu, H, dims // 2)
    _check_stream(stream, qkv.device)
    if out is None:
        out = torch.empty_like(qkv)
    else:
        _need(out, tuple(qkv.shape), qkv.dtype, "out")
        _same_device(qkv, out)
    if status is not None:
        _need(status, (1,), torch.int32, "status")
        _same_device(qkv, status)
    with torch.cuda.device(qkv.device):
        return _rope(qkv, cos, sin, cu, S, T, H, dims, traditional, inverse, out, status, stream)


def _rope(qkv, cos, sin, cu, S, T, H, dims, traditional, inverse, out, status, stream):
    rc = pk_rope(dtype_code(qkv), qkv.data_ptr(), out.data_ptr(), cos.data_ptr(), sin.data_ptr(),
                 cos.shape[0], cu.data_ptr(), S, T, H, int(dims), int(bool(traditional)), int(bool(inverse)),
                 status.data_ptr() if status is not None else None, _stream_handle(stream))
    _check(rc, "pk_rope")
    return out


# ------------------------------------------------------------------------------------------
# token-row operators (the projection, dropout, the vocabulary cross entropy)


def _on_stream(dev, stream, tensors, call):
    """call(raw stream) with the tensors' device current and, when the caller names a stream, that stream current, so that
    outputs and workspace are allocated for the stream that uses them (a workspace may then be freed as soon as the call
    returns: its memory is handed out again in the order of that stream); the given tensors are held back from reuse until
    the stream is past them."""
    torch = _torch()
    with torch.cuda.device(dev):
        if stream is None:
            return call(torch.cuda.current_stream().cuda_stream)
        if not hasattr(stream, "cuda_stream"):
            h = int(stream)
            stream = torch.cuda.ExternalStream(h, device=dev) if h else torch.cuda.default_stream(dev)
        if stream != torch.cuda.current_stream():
            for t in tensors:
                if t is not None:
                    t.record_stream(stream)
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)


def _here(dev, stream):
    """The raw current stream when the call runs on it and on the current device (the usual case), else None."""
    if stream is not None:
        return None
    torch = _torch()
    if torch.cuda.current_device() == dev.index:
        return torch._C._cuda_getCurrentRawStream(dev.index)
    return None


def _rows(t, cols, what, dtype=None, dev=None, rows=None):
    """The row stride of a [T, cols] CUDA matrix whose rows are contiguous (strided rows allowed, none overlapping)."""
    # (the usual cases in few steps: these checks are part of what a small call takes)
    shape = t.shape
    if len(shape) == 2 and t.is_cuda and t.is_contiguous():
        if cols is None and dtype is None and rows is None:
            return max(shape[1], 1)
        if shape[1] == cols and shape[0] == rows and t.dtype == dtype and t.device == dev:
            return max(cols, 1)
    if t.dim() != 2 or (cols is not None and t.shape[1] != cols) or (rows is not None and t.shape[0] != rows):
        raise ValueError(f"{what} must be [{'T' if rows is None else rows}, {'K' if cols is None else cols}], "
                         f"not {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{what} must be a CUDA tensor")
    if dev is not None and t.device != dev:
        raise ValueError(f"tensors on different devices ({dev} and {t.device})")
    n, (s0, s1) = t.shape[1], t.stride()
    if n > 1 and s1 != 1:
        raise ValueError(f"{what} must have contiguous rows")
    if t.shape[0] <= 1:
        return max(n, 1)
    if s0 < n:
        raise ValueError(f"{what} must not have overlapping rows")
    return s0


def _vector(t, n, what, dtype, dev):
    if t.dim() != 1 or t.shape[0] != n or t.dtype != dtype or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous [{n}] {dtype} CUDA tensor, not {tuple(t.shape)} {t.dtype}")
    if t.device != dev:
        raise ValueError(f"tensors on different devices ({dev} and {t.device})")


def _dense(t, rows, cols, what, dtype, dev):
    if tuple(t.shape) != (rows, cols) or t.dtype != dtype or not t.is_contiguous() or t.device != dev:
        _rows(t, cols, what, dtype, dev, rows)
        raise ValueError(f"{what} must be contiguous")


def _act_code(act):
    if act not in ACTS:
        raise ValueError(f"act must be one of {', '.join(ACTS)}, not {act!r}")
    return ACTS[act]


def _drop_check(p, seed, offset):
    if not 0.0 <= p < 1.0 - 2.0**-17:
        raise ValueError(f"p must be in [0, 1 - 2^-17), not {p}")
    if not 0 <= seed < 1 << 64 or not 0 <= offset < 1 << 64:
        raise ValueError("seed and offset must be unsigned 64-bit numbers")


def _workspace(name, device, *args):
    """(tensor or None, its address, its bytes) of the workspace that `name` asks for."""
    n = ctypes.c_int64(0)
    _check(getattr(load(), name)(*args, ctypes.byref(n)), name)
    if n.value == 0:
        return None, None, 0
    t = _torch().empty(n.value, dtype=_torch().uint8, device=device)
    return t, t.data_ptr(), n.value


def _ptr(t):
    return None if t is None else t.data_ptr()


def _disjoint(out, what, *inputs):
    """An output that the caller gives must not share memory with what the call reads while it writes it."""
    for t in inputs:
        if t is not None and _overlap(out, t):
            raise ValueError(f"{what} overlaps an input")


def _extent(t):
    if t.numel() == 0:
        return 0
    return (sum((n - 1) * s for n, s in zip(t.shape, t.stride())) + 1) * t.element_size()


def _overlap(a, b):
    """Whether two tensors can share an element: their address ranges meet and they are not different columns of rows of
    one stride (slices of one wider matrix)."""
    pa, pb = a.data_ptr(), b.data_ptr()
    if not (pa < pb + _extent(b) and pb < pa + _extent(a)):
        return False
    if a.dim() == 2 and b.dim() == 2 and a.stride(0) == b.stride(0) > 0 and a.element_size() == b.element_size():
        row = a.stride(0) * a.element_size()
        d = (pb - pa) % row  # b's first column, counted from a's
        if d >= a.shape[1] * a.element_size() and d + b.shape[1] * b.element_size() <= row:
            return False
    return True


def _same_place(a, b):
    return b is not None and a.data_ptr() == b.data_ptr() and a.stride() == b.stride()


def linear(x, w, bias=None, residual=None, act: str = "none", p: float = 0.0, seed: int = 0, offset: int = 0, out=None,
           return_pre: bool = False, status=None, stream=None):
    """y [T, N] = residual + dropout(act(x w^T + bias)) for x [T, K] and w [N, K] (float32, bfloat16 or float16, everything
    of one type); act "none", "relu", "gelu" or "silu"; dropout of probability p with the bits of (seed, offset), as
    `dropout`. x, residual and out may have strided rows; out may be residual itself. return_pre: also the
    pre-activation x w^T + bias [T, N], which linear_backward needs when act is not "none". `status`: optional int32
    device tensor of one element (otherwise last_status of the call's stream tells of device-detected errors; a captured
    call's are those of the stream it was captured on)."""
    torch = _torch()
    dt, dev = x.dtype, x.device
    code = dtype_code(x)
    ldx = _rows(x, None, "x")
    T, K = x.shape
    N = w.shape[0] if w.dim() == 2 else 0
    _dense(w, N, K, "w", dt, dev)
    if N < 1 or K < 1:
        raise ValueError("x and w must have at least one column, w at least one row")
    if bias is not None:
        _vector(bias, N, "bias", dt, dev)
    ldr = _rows(residual, N, "residual", dt, dev, T) if residual is not None else N
    a = _act_code(act)
    _drop_check(p, seed, offset)
    _check_stream(stream, dev)
    if status is not None:
        _vector(status, 1, "status", torch.int32, dev)
    ldy = N
    if out is not None:
        ldy = _rows(out, N, "out", dt, dev, T)
        _disjoint(out, "out", x, w, bias, None if _same_place(out, residual) else residual)

    def call(st):
        y = torch.empty((T, N), dtype=dt, device=dev) if out is None else out
        pre = torch.empty((T, N), dtype=dt, device=dev) if return_pre else None
        ws, wp, wb = (None, None, 0) if 2 * T <= LINEAR_FEW_T else _workspace("pk_linear_workspace", dev, code, x.data_ptr(), ldx,
                                                                          w.data_ptr(), T, N, K)
        _check(load().pk_linear(code, x.data_ptr(), ldx, w.data_ptr(), _ptr(bias), _ptr(residual), ldr, a, p, seed, offset, T,
                              N, K, y.data_ptr(), ldy, _ptr(pre), wp, wb, _ptr(status), st), "pk_linear")
        return (y, pre) if return_pre else y

    st = _here(dev, stream)
    return call(st) if st is not None else _on_stream(dev, stream, (x, w, bias, residual, out, status), call)


def linear_backward(x, w, dy, pre=None, act: str = "none", p: float = 0.0, seed: int = 0, offset: int = 0,
                    need_dx: bool = True, need_dw: bool = True, need_db: bool = True, status=None, stream=None):
    """(dx [T, K], dw [N, K], db [N]) of `linear` for the gradient dy [T, N] of its output, each None where not needed;
    pre is the forward's pre-activation (not needed for act "none"), act, p, seed and offset the forward's. The gradient
    of the residual is dy."""
    torch = _torch()
    dt, dev = x.dtype, x.device
    code = dtype_code(x)
    ldx = _rows(x, None, "x")
    T, K = x.shape
    N = w.shape[0] if w.dim() == 2 else 0
    _dense(w, N, K, "w", dt, dev)
    if N < 1 or K < 1:
        raise ValueError("x and w must have at least one column, w at least one row")
    lddy = _rows(dy, N, "dy", dt, dev, T)
    a = _act_code(act)
    if a and pre is None:
        raise ValueError(f"act {act!r} needs the forward's pre-activation")
    if pre is not None:
        _dense(pre, T, N, "pre", dt, dev)
    _drop_check(p, seed, offset)
    _check_stream(stream, dev)
    if status is not None:
        _vector(status, 1, "status", torch.int32, dev)

    def call(st):
        dx = torch.empty((T, K), dtype=dt, device=dev) if need_dx else None
        dw = torch.empty((N, K), dtype=dt, device=dev) if need_dw else None
        db = torch.empty(N, dtype=dt, device=dev) if need_db else None
        ws, wp, wb = _workspace("pk_linear_backward_workspace", dev, code, x.data_ptr(), ldx, w.data_ptr(), dy.data_ptr(), lddy,
                                a, p, bool(need_dx), bool(need_dw), bool(need_db), T, N, K)
        _check(_lib.pk_linear_backward(code, x.data_ptr(), ldx, w.data_ptr(), dy.data_ptr(), lddy, _ptr(pre), a, p, seed,
                                       offset, T, N, K, _ptr(dx), _ptr(dw), _ptr(db), wp, wb, _ptr(status), st),
               "pk_linear_backward")
        return dx, dw, db

    st = _here(dev, stream)
    return call(st) if st is not None else _on_stream(dev, stream, (x, w, dy, pre, status), call)


def dropout(x, p: float, seed: int, offset: int = 0, residual=None, out=None, stream=None):
    """y [T, N] = residual + x keep / (1 - p): each element of x [T, N] kept with probability 1 - p (p to the nearest
    multiple of 2^-16) by bits that depend on (seed, offset, row, column) alone, so nothing is stored for the backward
    pass. One (seed, offset) for each use: the same pair draws the same mask. out may be x or residual itself."""
    torch = _torch()
    dt, dev = x.dtype, x.device
    code = dtype_code(x)
    ldx = _rows(x, None, "x")
    T, N = x.shape
    if N < 1:
        raise ValueError("x must have at least one column")
    ldr = _rows(residual, N, "residual", dt, dev, T) if residual is not None else N
    _drop_check(p, seed, offset)
    _check_stream(stream, dev)
    ldy = N
    if out is not None:
        ldy = _rows(out, N, "out", dt, dev, T)
        _disjoint(out, "out", None if _same_place(out, x) else x, None if _same_place(out, residual) else residual)

    def call(st):
        y = torch.empty((T, N), dtype=dt, device=dev) if out is None else out
        _check(load().pk_dropout(code, x.data_ptr(), ldx, _ptr(residual), ldr, p, seed, offset, T, N, y.data_ptr(), ldy, st),
               "pk_dropout")
        return y

    st = _here(dev, stream)
    return call(st) if st is not None else _on_stream(dev, stream, (x, residual, out), call)


def dropout_backward(dy, p: float, seed: int, offset: int = 0, out=None, stream=None):
    """The gradient of `dropout` with respect to x: dy keep / (1 - p), with the forward's p, seed and offset."""
    return dropout(dy, p, seed, offset, out=out, stream=stream)


def _xent_inputs(x, w, labels, bias, status, stream):
    torch = _torch()
    dt, dev = x.dtype, x.device
    code = dtype_code(x)
    ldx = _rows(x, None, "x")
    T, D = x.shape
    V = w.shape[0] if w.dim() == 2 else 0
    _dense(w, V, D, "w", dt, dev)
    if V < 1 or D < 1:
        raise ValueError("x and w must have at least one column, w at least one row")
    _vector(labels, T, "labels", torch.int64, dev)
    if bias is not None:
        _vector(bias, V, "bias", dt, dev)
    if status is not None:
        _vector(status, 1, "status", torch.int32, dev)
    _check_stream(stream, dev)
    return code, dt, dev, ldx, T, D, V


def cross_entropy(x, w, labels, bias=None, status=None, stream=None):
    """(loss [T], lse [T]), float32: the softmax cross entropy of the logits x w^T + bias, x [T, D], w [V, D], against
    int64 labels [T], without storing the logits. A negative label leaves its row out (loss 0, no work); a label >= V
    gives a loss of NaN and PK_ERR_BAD_LABEL (in `status`, an int32 device tensor of one element, or last_status of the call's stream)."""
    torch = _torch()
    code, dt, dev, ldx, T, D, V = _xent_inputs(x, w, labels, bias, status, stream)

    def call(st):
        loss = torch.empty(T, dtype=torch.float32, device=dev)
        lse = torch.empty(T, dtype=torch.float32, device=dev)
        ws, wp, wb = _workspace("pk_cross_entropy_workspace", dev, code, x.data_ptr(), ldx, w.data_ptr(), 0, 0, T, D, V)
        _check(_lib.pk_cross_entropy(code, x.data_ptr(), ldx, w.data_ptr(), _ptr(bias), labels.data_ptr(), T, D, V,
                                     loss.data_ptr(), lse.data_ptr(), wp, wb, _ptr(status), st), "pk_cross_entropy")
        return loss, lse

    st = _here(dev, stream)
    return call(st) if st is not None else _on_stream(dev, stream, (x, w, labels, bias, status), call)


def cross_entropy_backward(x, w, labels, lse, dloss, bias=None, need_dx: bool = True, need_dw: bool = True, status=None,
                           stream=None):
    """(dx [T, D], dw [V, D], db [V] or None without a bias): the gradient of sum(dloss * loss) of `cross_entropy` for its
    lse [T]; dloss [T] float32 (1 / count for a mean). Rows without a label get a zero dx."""
    torch = _torch()
    code, dt, dev, ldx, T, D, V = _xent_inputs(x, w, labels, bias, status, stream)
    _vector(lse, T, "lse", torch.float32, dev)
    _vector(dloss, T, "dloss", torch.float32, dev)

    def call(st):
        dx = torch.empty((T, D), dtype=dt, device=dev) if need_dx else None
        dw = torch.empty((V, D), dtype=dt, device=dev) if need_dw else None
        db = torch.empty(V, dtype=dt, device=dev) if bias is not None else None
        ws, wp, wb = _workspace("pk_cross_entropy_workspace", dev, code, x.data_ptr(), ldx, w.data_ptr(), 1, bias is not None,
                                T, D, V)
        _check(_lib.pk_cross_entropy_backward(code, x.data_ptr(), ldx, w.data_ptr(), _ptr(bias), labels.data_ptr(),
                                              lse.data_ptr(), dloss.data_ptr(), T, D, V, _ptr(dx), _ptr(dw), _ptr(db), wp, wb,
                                              _ptr(status), st), "pk_cross_entropy_backward")
        return dx, dw, db

    st = _here(dev, stream)
    return call(st) if st is not None else _on_stream(dev, stream, (x, w, labels, lse, dloss, bias, status), call)


# ------------------------------------------------------------------------------------------
# norms and 8-bit rows


def _norm_inputs(x, w, residual, eps, stream):
    dt, dev = x.dtype, x.device
    code = dtype_code(x)
    ldx = _rows(x, None, "x")
    T, D = x.shape
    if not 1 <= D <= NORM_MAX_D:
        raise ValueError(f"x must have 1 to {NORM_MAX_D} columns, not {D}")
    _vector(w, D, "w", dt, dev)
    ldr = _rows(residual, D, "residual", dt, dev, T) if residual is not None else D
    _eps_check(eps)
    _check_stream(stream, dev)
    return code, dt, dev, ldx, ldr, T, D


def _eps_check(eps):
    if not 1e-45 < eps < 3.4e38:
        raise ValueError(f"eps must be positive and finite in fp32, not {eps}")


def _sum_rows(h_out, x, w, residual, T, D, dt, dev):
    """The row stride of a given h_out, which may be x or the residual itself."""
    ldh = _rows(h_out, D, "h_out", dt, dev, T)
    _disjoint(h_out, "h_out", None if _same_place(h_out, x) else x, w, None if _same_place(h_out, residual) else residual)
    return ldh


def rms_norm(x, w, residual=None, eps: float = 1e-6, out=None, h_out=None, stream=None):
    """y [T, D] = w h / sqrt(mean(h^2) + eps) with h = x + residual, for x [T, D] and w [D] (float32, bfloat16 or float16,
    everything of one type, D up to 16384). With a residual: (y, h), the sum being what the next layer adds to. x, residual, out
    and h_out may have strided rows; h_out may be x or residual itself (the residual stream updated in place)."""
    torch = _torch()
    code, dt, dev, ldx, ldr, T, D = _norm_inputs(x, w, residual, eps, stream)
    ldy = ldh = D
    if h_out is not None:
        if residual is None:
            raise ValueError("h_out needs a residual: without one h is x")
        ldh = _sum_rows(h_out, x, w, residual, T, D, dt, dev)
    if out is not None:
        ldy = _rows(out, D, "out", dt, dev, T)
        _disjoint(out, "out", x, w, residual, h_out)

    def call(st):
        y = torch.empty((T, D), dtype=dt, device=dev) if out is None else out
        h = h_out if h_out is not None or residual is None else torch.empty((T, D), dtype=dt, device=dev)
        _check(load().pk_rms_norm(code, x.data_ptr(), ldx, _ptr(residual), ldr, w.data_ptr(), eps, T, D, y.data_ptr(), ldy, _ptr(h),
                                  ldh, st), "pk_rms_norm")
        return y if residual is None else (y, h)

    st = _here(dev, stream)
    return call(st) if st is not None else _on_stream(dev, stream, (x, w, residual, out, h_out), call)


def rms_norm_q8(x, w, residual=None, eps: float = 1e-6, h_out=None, stream=None):
    """`rms_norm` with its rows in 8 bits, for `linear_q8`: (q [T, D] float8_e4m3fn, scale [T] float32), and h with a
    residual; row t stands for q[t] scale[t], scale being the row's largest magnitude / 448."""
    torch = _torch()
    code, dt, dev, ldx, ldr, T, D = _norm_inputs(x, w, residual, eps, stream)
    ldh = D
    if h_out is not None:
        if residual is None:
            raise ValueError("h_out needs a residual: without one h is x")
        ldh = _sum_rows(h_out, x, w, residual, T, D, dt, dev)

    def call(st):
        q = torch.empty((T, D), dtype=torch.float8_e4m3fn, device=dev)
        scale = torch.empty(T, dtype=torch.float32, device=dev)
        h = h_out if h_out is not None or residual is None else torch.empty((T, D), dtype=dt, device=dev)
        _check(load().pk_rms_norm_q8(code, x.data_ptr(), ldx, _ptr(residual), ldr, w.data_ptr(), eps, T, D, q.data_ptr(), D,
                                     scale.data_ptr(), _ptr(h), ldh, st), "pk_rms_norm_q8")
        return (q, scale) if residual is None else (q, scale, h)

    st = _here(dev, stream)
    return call(st) if st is not None else _on_stream(dev, stream, (x, w, residual, h_out), call)


def quantize_rows(x, stream=None):
    """(q [T, D] float8_e4m3fn, scale [T] float32) for x [T, D]: row t is q[t] scale[t] to 8 bits, scale the row's largest
    magnitude / 448. For the weights of `linear_q8` and for activations that come from no norm; D up to 16384."""
    torch = _torch()
    dev = x.device
    code = dtype_code(x)
    ldx = _rows(x, None, "x")
    T, D = x.shape
    if not 1 <= D <= NORM_MAX_D:
        raise ValueError(f"x must have 1 to {NORM_MAX_D} columns, not {D}")
    _check_stream(stream, dev)

    def call(st):
        q = torch.empty((T, D), dtype=torch.float8_e4m3fn, device=dev)
        scale = torch.empty(T, dtype=torch.float32, device=dev)
        _check(load().pk_quantize_rows(code, x.data_ptr(), ldx, T, D, q.data_ptr(), D, scale.data_ptr(), st), "pk_quantize_rows")
        return q, scale

    st = _here(dev, stream)
    return call(st) if st is not None else _on_stream(dev, stream, (x,), call)


@functools.lru_cache(maxsize=1024)
def _norm_workspace(dev, code, T, D) -> int:
    """Bytes that pk_rms_norm_backward needs (its sizes alone decide; asked for with the device current)."""
    n = ctypes.c_int64(0)
    _check(load().pk_rms_norm_backward_workspace(code, T, D, 1, ctypes.byref(n)), "pk_rms_norm_backward_workspace")
    return n.value


def rms_norm_backward(h, w, dy, dh=None, eps: float = 1e-6, need_dx: bool = True, need_dw: bool = True, out=None, stream=None):
    """(dx [T, D], dw [D]) of `rms_norm` for the gradient dy of its output, each None where not needed; h is the forward's sum
    (x where there was no residual), dh the gradient that arrives on h itself. dx is the gradient of x and of the residual
    alike; `out` for it may be dy or dh itself."""
    torch = _torch()
    dt, dev = h.dtype, h.device
    code = dtype_code(h)
    ldh = _rows(h, None, "h")
    T, D = h.shape
    if not 1 <= D <= NORM_MAX_D:
        raise ValueError(f"h must have 1 to {NORM_MAX_D} columns, not {D}")
    _vector(w, D, "w", dt, dev)
    lddy = _rows(dy, D, "dy", dt, dev, T)
    lddh = _rows(dh, D, "dh", dt, dev, T) if dh is not None else D
    _eps_check(eps)
    _check_stream(stream, dev)
    lddx = D
    if out is not None:
        if not need_dx:
            raise ValueError("out is dx's, which is not needed")
        lddx = _rows(out, D, "out", dt, dev, T)
        _disjoint(out, "out", h, w, None if _same_place(out, dy) else dy, None if dh is None or _same_place(out, dh) else dh)

    def call(st):
        dx = out if out is not None or not need_dx else torch.empty((T, D), dtype=dt, device=dev)
        dw = torch.empty(D, dtype=dt, device=dev) if need_dw else None
        wb = _norm_workspace(dev, code, T, D) if need_dw else 0
        ws = torch.empty(wb, dtype=torch.uint8, device=dev) if wb else None
        wp = _ptr(ws)
        _check(load().pk_rms_norm_backward(code, h.data_ptr(), ldh, w.data_ptr(), dy.data_ptr(), lddy, _ptr(dh), lddh, eps, T, D,
                                           _ptr(dx), lddx, _ptr(dw), wp, wb, st), "pk_rms_norm_backward")
        return dx, dw

    st = _here(dev, stream)
    return call(st) if st is not None else _on_stream(dev, stream, (h, w, dy, dh, out), call)


def linear_q8(x, x_scale, w, w_scale, bias=None, residual=None, act: str = "none", out_dtype=None, out=None, status=None, stream=None):
    """y [T, N] = residual + act(x_scale w_scale (x w^T) + bias) for rows in 8 bits: x [T, K] and w [N, K] float8_e4m3fn with a
    float32 scale a row, as `rms_norm_q8` and `quantize_rows` give them; K a multiple of 16. y is of out_dtype (or out's, the
    residual's or the bias's type; bfloat16 where none of them says), bias and residual too. x, residual and out may have
    strided rows (of x: by multiples of 16); out may be residual itself."""
    torch = _torch()
    dev = x.device
    ldx = _rows(x, None, "x", torch.float8_e4m3fn)
    T, K = x.shape
    N = w.shape[0] if w.dim() == 2 else 0
    _dense(w, N, K, "w", torch.float8_e4m3fn, dev)
    if N < 1 or K < 1 or K % 16:
        raise ValueError("w must have at least one row, and x and w a multiple of 16 columns")
    if ldx % 16 or x.data_ptr() % 16 or w.data_ptr() % 16:
        raise ValueError("x and w must have rows on 16-byte boundaries")
    _vector(x_scale, T, "x_scale", torch.float32, dev)
    _vector(w_scale, N, "w_scale", torch.float32, dev)
    dt = out_dtype
    if dt is None:
        dt = next((t.dtype for t in (out, residual, bias) if t is not None), torch.bfloat16)
    code = _code(dt)
    if bias is not None:
        _vector(bias, N, "bias", dt, dev)
    ldr = _rows(residual, N, "residual", dt, dev, T) if residual is not None else N
    a = _act_code(act)
    _check_stream(stream, dev)
    if status is not None:
        _vector(status, 1, "status", torch.int32, dev)
    ldy = N
    if out is not None:
        ldy = _rows(out, N, "out", dt, dev, T)
        _disjoint(out, "out", x, x_scale, w, w_scale, bias, None if _same_place(out, residual) else residual)

    def call(st):
        y = torch.empty((T, N), dtype=dt, device=dev) if out is None else out
        ws, wp, wb = (None, None, 0) if 2 * T <= LINEAR_FEW_T else _workspace("pk_linear_q8_workspace", dev, T, N, K)
        _check(load().pk_linear_q8(code, x.data_ptr(), ldx, x_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(), _ptr(bias),
                                   _ptr(residual), ldr, a, T, N, K, y.data_ptr(), ldy, wp, wb, _ptr(status), st), "pk_linear_q8")
        return y

    st = _here(dev, stream)
    return call(st) if st is not None else _on_stream(dev, stream, (x, x_scale, w, w_scale, bias, residual, out, status), call)


# ------------------------------------------------------------------------------------------
# the gated feed-forward


def _gated_inputs(x, w, act, status, stream):
    dt, dev = x.dtype, x.device
    code = dtype_code(x)
    ldx = _rows(x, None, "x")
    T, K = x.shape
    N = w.shape[0] if w.dim() == 2 else 0
    _dense(w, N, K, "w", dt, dev)
    if N < 2 or N % 2 or K < 1:
        raise ValueError("w must have an even number of rows (the gate's, then the other's), x and w at least one column")
    a = _act_code(act)
    _check_stream(stream, dev)
    if status is not None:
        _vector(status, 1, "status", _torch().int32, dev)
    return code, dt, dev, ldx, T, K, N // 2, a


def gated_linear(x, w, bias=None, act: str = "gelu", out=None, return_pre: bool = False, status=None, stream=None):
    """y [T, F] = act(g) u with [g | u] = x w^T + bias, for x [T, K] and w [2 F, K] (F rows of the gate, then F of what it
    multiplies; float32, bfloat16 or float16, everything of one type) in one product; act "none", "relu", "gelu" or "silu".
    return_pre: also [g | u] [T, 2 F], which gated_linear_backward needs. x and out may have strided rows. `status` as
    for `linear`."""
    torch = _torch()
    code, dt, dev, ldx, T, K, F, a = _gated_inputs(x, w, act, status, stream)
    if bias is not None:
        _vector(bias, 2 * F, "bias", dt, dev)
    ldy = F
    if out is not None:
        ldy = _rows(out, F, "out", dt, dev, T)
        _disjoint(out, "out", x, w, bias)

    def call(st):
        y = torch.empty((T, F), dtype=dt, device=dev) if out is None else out
        pre = torch.empty((T, 2 * F), dtype=dt, device=dev) if return_pre else None
        ws, wp, wb = (None, None, 0) if 2 * T <= LINEAR_FEW_T else _workspace("pk_gated_linear_workspace", dev, code, x.data_ptr(), ldx,
                                                                          w.data_ptr(), T, F, K)
        _check(load().pk_gated_linear(code, x.data_ptr(), ldx, w.data_ptr(), _ptr(bias), a, T, F, K, y.data_ptr(), ldy, _ptr(pre), wp,
                                      wb, _ptr(status), st), "pk_gated_linear")
        return (y, pre) if return_pre else y

    st = _here(dev, stream)
    return call(st) if st is not None else _on_stream(dev, stream, (x, w, bias, out, status), call)


def gated_linear_backward(x, w, dy, pre, act: str = "gelu", need_dx: bool = True, need_dw: bool = True, need_db: bool = True,
                          status=None, stream=None):
    """(dx [T, K], dw [2 F, K], db [2 F]) of `gated_linear` for the gradient dy [T, F] of its output, each None where not
    needed; pre [T, 2 F] is the forward's, act too."""
    torch = _torch()
    code, dt, dev, ldx, T, K, F, a = _gated_inputs(x, w, act, status, stream)
    lddy = _rows(dy, F, "dy", dt, dev, T)
    _dense(pre, T, 2 * F, "pre", dt, dev)

    def call(st):
        dx = torch.empty((T, K), dtype=dt, device=dev) if need_dx else None
        dw = torch.empty((2 * F, K), dtype=dt, device=dev) if need_dw else None
        db = torch.empty(2 * F, dtype=dt, device=dev) if need_db else None
        ws, wp, wb = _workspace("pk_gated_linear_backward_workspace", dev, code, x.data_ptr(), ldx, w.data_ptr(), bool(need_dx),
                                bool(need_dw), bool(need_db), T, F, K)
        _check(_lib.pk_gated_linear_backward(code, x.data_ptr(), ldx, w.data_ptr(), dy.data_ptr(), lddy, pre.data_ptr(), a, T, F, K,
                                             _ptr(dx), _ptr(dw), _ptr(db), wp, wb, _ptr(status), st), "pk_gated_linear_backward")
        return dx, dw, db

    st = _here(dev, stream)
    return call(st) if st is not None else _on_stream(dev, stream, (x, w, dy, pre, status), call)


# ------------------------------------------------------------------------------------------
# log probabilities of rows of logits


def token_logprobs(logits, labels, top: int = 0, status=None, stream=None):
    """(logp [T], lse [T], entropy [T], top_logp [T, top], top_idx [T, top]) of logits [T, V] and int64 labels [T]: the log
    probability of each row's label (0 for a negative label; NaN and PK_ERR_BAD_LABEL for one >= V, in `status` or last_status
    of the call's stream), the row's log-sum-exp and entropy (float32), and its `top` (at most 64) likeliest words, the
    likeliest first and equal ones by index (int64; None, None for top 0). logits may have strided rows. The last bits of logp, lse
    and entropy may depend on T and top, which say how a row's sums are shared out."""
    torch = _torch()
    dev = logits.device
    code = dtype_code(logits)
    ld = _rows(logits, None, "logits")
    T, V = logits.shape
    if V < 1:
        raise ValueError("logits must have at least one column")
    _vector(labels, T, "labels", torch.int64, dev)
    if not 0 <= top <= min(LOGPROBS_MAX_TOP, V):
        raise ValueError(f"top must be in [0, min({LOGPROBS_MAX_TOP}, V)], not {top}")
    if status is not None:
        _vector(status, 1, "status", torch.int32, dev)
    _check_stream(stream, dev)

    def call(st):
        logp, lse, entropy = torch.empty((3, T), dtype=torch.float32, device=dev).unbind(0)
        best = torch.empty((T, top), dtype=torch.float32, device=dev) if top else None
        idx = torch.empty((T, top), dtype=torch.int64, device=dev) if top else None
        _check(load().pk_token_logprobs(code, logits.data_ptr(), ld, labels.data_ptr(), T, V, top, logp.data_ptr(), lse.data_ptr(),
                                        entropy.data_ptr(), _ptr(best), _ptr(idx), _ptr(status), st), "pk_token_logprobs")
        return logp, lse, entropy, best, idx

    st = _here(dev, stream)
    return call(st) if st is not None else _on_stream(dev, stream, (logits, labels, status), call)


def token_logprobs_backward(logits, labels, lse, entropy, dlogp, dentropy=None, out=None, stream=None):
    """dlogits [T, V]: the gradient of sum(dlogp * logp) + sum(dentropy * entropy) of `token_logprobs` for its lse and entropy
    (entropy may be None without dentropy). `out` may be logits itself."""
    torch = _torch()
    dt, dev = logits.dtype, logits.device
    code = dtype_code(logits)
    ld = _rows(logits, None, "logits")
    T, V = logits.shape
    if V < 1:
        raise ValueError("logits must have at least one column")
    _vector(labels, T, "labels", torch.int64, dev)
    for name, t in (("lse", lse), ("dlogp", dlogp), ("entropy", entropy), ("dentropy", dentropy)):
        if t is not None:
            _vector(t, T, name, torch.float32, dev)
        elif name == "lse" or name == "dlogp" or (name == "entropy" and dentropy is not None):
            raise ValueError(f"{name} is needed")
    _check_stream(stream, dev)
    ldo = V
    if out is not None:
        ldo = _rows(out, V, "out", dt, dev, T)
        _disjoint(out, "out", None if _same_place(out, logits) else logits, labels, lse, entropy, dlogp, dentropy)

    def call(st):
        d = torch.empty((T, V), dtype=dt, device=dev) if out is None else out
        _check(load().pk_token_logprobs_backward(code, logits.data_ptr(), ld, labels.data_ptr(), lse.data_ptr(), _ptr(entropy),
                                                 dlogp.data_ptr(), _ptr(dentropy), T, V, d.data_ptr(), ldo, st),
               "pk_token_logprobs_backward")
        return d

    st = _here(dev, stream)
    return call(st) if st is not None else _on_stream(dev, stream, (logits, labels, lse, entropy, dlogp, dentropy, out), call)


# ------------------------------------------------------------------------------------------
# distillation


def _distill_inputs(x, w, idx, values, bias, temperature, status, stream):
    torch = _torch()
    dt, dev = x.dtype, x.device
    code = dtype_code(x)
    ldx = _rows(x, None, "x")
    T, D = x.shape
    V = w.shape[0] if w.dim() == 2 else 0
    _dense(w, V, D, "w", dt, dev)
    if V < 1 or D < 1:
        raise ValueError("x and w must have at least one column, w at least one row")
    top = idx.shape[1] if idx.dim() == 2 else 0
    if not 1 <= top <= DISTILL_MAX_TOP:
        raise ValueError(f"idx must be [T, 1 to {DISTILL_MAX_TOP}], not {tuple(idx.shape)}")
    _dense(idx, T, top, "idx", torch.int64, dev)
    _dense(values, T, top, "values", torch.float32, dev)
    if bias is not None:
        _vector(bias, V, "bias", dt, dev)
    if not 1e-3 <= temperature <= 1e3:
        raise ValueError(f"temperature must be in [1e-3, 1e3], not {temperature}")
    if status is not None:
        _vector(status, 1, "status", torch.int32, dev)
    _check_stream(stream, dev)
    return code, dt, dev, ldx, T, D, V, top


def distill(x, w, idx, values, bias=None, temperature: float = 1.0, status=None, stream=None):
    """(loss [T], lse [T]), float32: how far a student's probabilities softmax((x w^T + bias) / temperature), x [T, D], w [V, D],
    are from a teacher's q = softmax(values / temperature) over its top words idx [T, top] int64 (values [T, top] float32: its
    logits or log probabilities there, as `token_logprobs` gives them; top up to 64): loss = sum_k q_k (ln q_k - ln p_k), without
    storing the logits. An entry with a negative index or the value -inf is not there; a row without any has loss 0 and
    costs no work; an index >= V gives a loss of NaN and PK_ERR_BAD_LABEL (in `status`, or last_status of the call's stream)."""
    torch = _torch()
    code, dt, dev, ldx, T, D, V, top = _distill_inputs(x, w, idx, values, bias, temperature, status, stream)

    def call(st):
        loss = torch.empty(T, dtype=torch.float32, device=dev)
        lse = torch.empty(T, dtype=torch.float32, device=dev)
        ws, wp, wb = _workspace("pk_distill_workspace", dev, code, x.data_ptr(), ldx, w.data_ptr(), 0, 0, T, D, V, top)
        _check(_lib.pk_distill(code, x.data_ptr(), ldx, w.data_ptr(), _ptr(bias), idx.data_ptr(), values.data_ptr(), top, temperature, T,
                               D, V, loss.data_ptr(), lse.data_ptr(), wp, wb, _ptr(status), st), "pk_distill")
        return loss, lse

    st = _here(dev, stream)
    return call(st) if st is not None else _on_stream(dev, stream, (x, w, idx, values, bias, status), call)


def distill_backward(x, w, idx, values, lse, dloss, bias=None, temperature: float = 1.0, need_dx: bool = True, need_dw: bool = True,
                     status=None, stream=None):
    """(dx [T, D], dw [V, D], db [V] or None without a bias): the gradient of sum(dloss * loss) of `distill` with respect to the
    student, for its lse [T]; dloss [T] float32 (temperature ** 2 / count for a mean that keeps the gradients' size at any
    temperature). Rows without a target get a zero dx."""
    torch = _torch()
    code, dt, dev, ldx, T, D, V, top = _distill_inputs(x, w, idx, values, bias, temperature, status, stream)
    _vector(lse, T, "lse", torch.float32, dev)
    _vector(dloss, T, "dloss", torch.float32, dev)

    def call(st):
        dx = torch.empty((T, D), dtype=dt, device=dev) if need_dx else None
        dw = torch.empty((V, D), dtype=dt, device=dev) if need_dw else None
        db = torch.empty(V, dtype=dt, device=dev) if bias is not None else None
        ws, wp, wb = _workspace("pk_distill_workspace", dev, code, x.data_ptr(), ldx, w.data_ptr(), 1, bias is not None, T, D, V, top)
        _check(_lib.pk_distill_backward(code, x.data_ptr(), ldx, w.data_ptr(), _ptr(bias), idx.data_ptr(), values.data_ptr(), top,
                                        temperature, lse.data_ptr(), dloss.data_ptr(), T, D, V, _ptr(dx), _ptr(dw), _ptr(db), wp, wb,
                                        _ptr(status), st), "pk_distill_backward")
        return dx, dw, db

    st = _here(dev, stream)
    return call(st) if st is not None else _on_stream(dev, stream, (x, w, idx, values, lse, dloss, bias, status), call)


def schedule(cu, T: int, window: int, stream=None):
    """Tile records [NT, 8] (int32 tensor holding the uint32 fields) of the device scheduler."""
    torch = _torch()
    if cu.dim() != 1 or cu.dtype not in (torch.int32, torch.uint32) or not cu.is_cuda or not cu.is_contiguous():
        raise ValueError("cu must be a contiguous 1-D int32 or uint32 CUDA tensor")
    cap = int(load().pk_schedule_capacity(T))
    tiles = torch.zeros((max(cap, 1), 8), dtype=torch.int32, device=cu.device)
    rc, nt = pk_schedule(cu.data_ptr(), cu.shape[0] - 1, T, window, tiles.data_ptr(), cap,
                         _stream_handle(stream))
    _check(rc, "pk_schedule")
    return tiles[:nt]


def last_status(stream=None) -> int:
    return pk_last_status(_stream_handle(stream))


def profile_start(n: int):
    """Record kernel events around the next n attention calls (see pk_profile_start)."""
    _check(load().pk_profile_start(int(n)), "pk_profile_start")


def profile_stop():
    """(schedule_ms_total, attend_ms_total, calls) recorded since profile_start."""
    a, b, n = ctypes.c_double(0), ctypes.c_double(0), ctypes.c_int(0)
    _check(load().pk_profile_stop(ctypes.byref(a), ctypes.byref(b), ctypes.byref(n)), "pk_profile_stop")
    return a.value, b.value, n.value


def release():
    _check(load().pk_release(), "pk_release")
