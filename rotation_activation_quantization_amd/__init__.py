"""SignRot's online activation path on MI355X: Python binding of libsignrot.

Argument marshalling only: every step of the path runs in the HIP library
(`libsignrot.so`, built in-tree by `build.py`).  Torch supplies device memory
and the current stream; nothing here computes on the CPU, and every call fails
loudly when the library is missing.

The C ABI is declared in include/signrot.h; the functions here keep its names.
"""

from __future__ import annotations

import ctypes
import os
import struct

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libsignrot.so")

SIGNROT_OK = 0
SIGNROT_EINVAL = -1
SIGNROT_EUNSUPPORTED_N = -2
SIGNROT_EHIP = -3

_lib = None


class SignRotError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: status {status}: {detail}")
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libsignrot.so (raises when it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(
            f"{LIB_PATH} is missing: build it with "
            "`python -m rotation_activation_quantization_amd.build` (hipcc, gfx950)")
    L = ctypes.CDLL(LIB_PATH)
    i64, vp = ctypes.c_int64, ctypes.c_void_p
    L.signrot_supported_n.argtypes = [i64]
    L.signrot_supported_n.restype = ctypes.c_int
    L.signrot_calibrate.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp, vp]
    L.signrot_calibrate.restype = ctypes.c_int
    L.signrot_calibrate_noalloc.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp, vp]
    L.signrot_calibrate_noalloc.restype = ctypes.c_int
    L.signrot_rotate_quant_int4.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp, vp, vp]
    L.signrot_rotate_quant_int4.restype = ctypes.c_int
    L.signrot_rotate_quant_int4_outlier.argtypes = [vp, i64, i64, i64, i64, ctypes.c_int, vp, vp, vp, vp, vp]
    L.signrot_rotate_quant_int4_outlier.restype = ctypes.c_int
    L.signrot_swiglu_rotate_quant_int4.argtypes = [vp, vp, i64, i64, i64, i64, ctypes.c_int, vp, vp, vp, vp, vp]
    L.signrot_swiglu_rotate_quant_int4.restype = ctypes.c_int
    L.signrot_rotate_quant_int4_zint.argtypes = [vp, i64, i64, i64, i64, ctypes.c_int, vp, vp, vp, vp]
    L.signrot_rotate_quant_int4_zint.restype = ctypes.c_int
    L.signrot_dequant.argtypes = [vp, vp, vp, i64, i64, vp, vp]
    L.signrot_dequant.restype = ctypes.c_int
    L.signrot_fold_weights.argtypes = [vp, i64, i64, i64, vp, vp, vp]
    L.signrot_fold_weights.restype = ctypes.c_int
    L.signrot_weight_rowsum.argtypes = [vp, i64, i64, i64, vp, vp]
    L.signrot_weight_rowsum.restype = ctypes.c_int
    L.signrot_int4_linear.argtypes = [vp, vp, vp, i64, i64, vp, i64, vp, i64, vp, vp]
    L.signrot_int4_linear.restype = ctypes.c_int
    L.signrot_int4_linear_kernel_name.argtypes = [vp, i64, i64, vp, i64, i64]
    L.signrot_int4_linear_kernel_name.restype = ctypes.c_char_p
    L.signrot_quant_int8.argtypes = [vp, i64, i64, i64, vp, i64, vp, vp, vp]
    L.signrot_quant_int8.restype = ctypes.c_int
    L.signrot_int8_linear.argtypes = [vp, i64, vp, i64, i64, vp, i64, vp, vp, i64, vp, i64, ctypes.c_int, vp, i64, vp]
    L.signrot_int8_linear.restype = ctypes.c_int
    L.signrot_int4_w8_linear.argtypes = [vp, vp, vp, i64, i64, vp, i64, vp, vp, vp, i64, vp, i64, ctypes.c_int, vp,
                                         i64, vp]
    L.signrot_int4_w8_linear.restype = ctypes.c_int
    L.signrot_int8_linear_workspace.argtypes = [vp, i64, i64, i64, vp, i64, i64]
    L.signrot_int8_linear_workspace.restype = i64
    L.signrot_int4_w8_linear_workspace.argtypes = [vp, i64, i64, vp, i64, i64]
    L.signrot_int4_w8_linear_workspace.restype = i64
    L.signrot_int8_linear_kernel_name.argtypes = [vp, i64, i64, i64, vp, i64, i64]
    L.signrot_int8_linear_kernel_name.restype = ctypes.c_char_p
    L.signrot_int4_w8_linear_kernel_name.argtypes = [vp, i64, i64, vp, i64, i64]
    L.signrot_int4_w8_linear_kernel_name.restype = ctypes.c_char_p
    L.signrot_residual_norm.argtypes = [vp, vp]
    L.signrot_residual_norm.restype = ctypes.c_int
    ci = ctypes.c_int
    L.signrot_quant_mxfp4.argtypes = [vp, ci, i64, i64, i64, ci, vp, i64, vp, i64, vp]
    L.signrot_quant_mxfp4.restype = ci
    L.signrot_dequant_mxfp4.argtypes = [vp, i64, vp, i64, i64, i64, vp, ci, i64, vp]
    L.signrot_dequant_mxfp4.restype = ci
    L.signrot_mxfp4_linear.argtypes = [vp, i64, vp, i64, i64, i64, vp, i64, vp, i64, vp, i64, vp, i64, ci, vp, i64, vp]
    L.signrot_mxfp4_linear.restype = ci
    L.signrot_mxfp4_linear_workspace.argtypes = [vp, i64, vp, i64, i64, i64, vp, i64, vp, i64, i64]
    L.signrot_mxfp4_linear_workspace.restype = i64
    L.signrot_mxfp4_linear_kernel_name.argtypes = [vp, i64, vp, i64, i64, i64, vp, i64, vp, i64, i64]
    L.signrot_mxfp4_linear_kernel_name.restype = ctypes.c_char_p
    L.signrot_rotate_quant_mxfp4.argtypes = [vp, i64, i64, i64, i64, ci, ci, vp, i64, vp, i64, vp, i64, vp]
    L.signrot_rotate_quant_mxfp4.restype = ci
    L.signrot_rotate_quant_mxfp4_workspace.argtypes = [i64, i64]
    L.signrot_rotate_quant_mxfp4_workspace.restype = i64
    L.signrot_swiglu_rotate_quant_mxfp4.argtypes = [vp, vp, i64, i64, i64, i64, ci, ci, vp, i64, vp, i64, vp]
    L.signrot_swiglu_rotate_quant_mxfp4.restype = ci
    L.signrot_qk_norm_rope.argtypes = [vp, vp]
    L.signrot_qk_norm_rope.restype = ci
    L.signrot_stream_ceiling.argtypes = [vp, i64, i64, i64, vp, vp, vp, vp]
    L.signrot_stream_ceiling.restype = ctypes.c_int
    L.signrot_strerror.argtypes = [ctypes.c_int]
    L.signrot_strerror.restype = ctypes.c_char_p
    L.signrot_last_error.argtypes = []
    L.signrot_last_error.restype = ctypes.c_char_p
    L.signrot_debug_h28.argtypes = [vp]
    L.signrot_debug_h28.restype = ctypes.c_int
    L.signrot_debug_outer.argtypes = [ctypes.c_int, vp]
    L.signrot_debug_outer.restype = ctypes.c_int
    L.signrot_outer_order.argtypes = [i64]
    L.signrot_outer_order.restype = ctypes.c_int
    L.signrot_debug_outer_folded.argtypes = [ctypes.c_int, ctypes.c_int, vp]
    L.signrot_debug_outer_folded.restype = ctypes.c_int
    L.signrot_outer_fold.argtypes = [i64]
    L.signrot_outer_fold.restype = ctypes.c_int
    L.signrot_kernel_name.argtypes = [i64]
    L.signrot_kernel_name.restype = ctypes.c_char_p
    _lib = L
    return L


EXPORTED = (
    "signrot_supported_n",
    "signrot_calibrate",
    "signrot_calibrate_noalloc",
    "signrot_rotate_quant_int4",
    "signrot_rotate_quant_int4_outlier",
    "signrot_rotate_quant_int4_zint",
    "signrot_swiglu_rotate_quant_int4",
    "signrot_dequant",
    "signrot_fold_weights",
    "signrot_weight_rowsum",
    "signrot_int4_linear",
    "signrot_int4_linear_kernel_name",
    "signrot_quant_int8",
    "signrot_int8_linear",
    "signrot_int8_linear_workspace",
    "signrot_int8_linear_kernel_name",
    "signrot_int4_w8_linear",
    "signrot_int4_w8_linear_workspace",
    "signrot_int4_w8_linear_kernel_name",
    "signrot_residual_norm",
    "signrot_quant_mxfp4",
    "signrot_dequant_mxfp4",
    "signrot_mxfp4_linear",
    "signrot_mxfp4_linear_workspace",
    "signrot_mxfp4_linear_kernel_name",
    "signrot_rotate_quant_mxfp4",
    "signrot_rotate_quant_mxfp4_workspace",
    "signrot_swiglu_rotate_quant_mxfp4",
    "signrot_qk_norm_rope",
    "signrot_strerror",
    "signrot_last_error",
    "signrot_debug_h28",
    "signrot_debug_outer",
    "signrot_debug_outer_folded",
    "signrot_outer_order",
    "signrot_outer_fold",
    "signrot_kernel_name",
    "signrot_stream_ceiling",
)


def check(status: int, where: str) -> None:
    if status != SIGNROT_OK:
        L = lib()
        detail = (L.signrot_last_error() or b"").decode() or L.signrot_strerror(status).decode()
        raise SignRotError(status, where, detail)


def supported_n(n: int) -> bool:
    return bool(lib().signrot_supported_n(int(n)))


def kernel_name(n: int) -> str | None:
    r = lib().signrot_kernel_name(int(n))
    return r.decode() if r else None


def outer_order(n: int) -> int:
    """The outer Hadamard order m of n = m * 2^k (1 for n = 2^k, 0 if unsupported)."""
    return int(lib().signrot_outer_order(int(n)))


def debug_outer(m: int):
    """The library's outer factor H_m as an m x m list of +-1 rows (host only)."""
    buf = (ctypes.c_int8 * (m * m))()
    check(lib().signrot_debug_outer(int(m), ctypes.addressof(buf)), "signrot_debug_outer")
    return [list(buf[r * m:(r + 1) * m]) for r in range(m)]


def debug_outer_folded(m: int, fold: int):
    """The library's folded outer factor H_m (x) Syl_{2^fold} (host only)."""
    import numpy as np

    mm = int(m) << int(fold)
    buf = (ctypes.c_int8 * (mm * mm))()
    check(lib().signrot_debug_outer_folded(int(m), int(fold), ctypes.addressof(buf)), "signrot_debug_outer_folded")
    return np.frombuffer(buf, dtype=np.int8).reshape(mm, mm).copy()


def outer_fold(n: int) -> int:
    """Sylvester bits the rotate kernel for n folds into its outer factor."""
    return int(lib().signrot_outer_fold(int(n)))


def debug_h28():
    """The library's own H28 as a 28x28 list of +-1 rows."""
    buf = (ctypes.c_int8 * 784)()
    check(lib().signrot_debug_h28(ctypes.addressof(buf)), "signrot_debug_h28")
    return [list(buf[r * 28:(r + 1) * 28]) for r in range(28)]


_raw_stream = _current_device = None


def _direct_calls():
    """torch's look-ups of a device's current stream and of the current device
    by number, without the objects and checks of the public calls (2 us of a
    small call's 7) where torch has the direct ones."""
    global _raw_stream, _current_device
    import torch

    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run(name, t, *args):
    """Calls the library's function `name` with args and the current stream of
    t's GPU, and with that GPU as the current one: a device's default stream has
    no handle of its own, so it is the current device that the kernel runs on."""
    if _raw_stream is None:
        _direct_calls()
    gpu = t.get_device()
    if gpu < 0:
        raise ValueError(f"expected a tensor on a GPU, not on {t.device}")
    if gpu == _current_device():
        status = getattr(lib(), name)(*args, _raw_stream(gpu))
    else:
        import torch

        with torch.cuda.device(gpu):
            status = getattr(lib(), name)(*args, _raw_stream(gpu))
    if status != SIGNROT_OK:
        check(status, name)


def _rows(x):
    """(pointer, tokens, n, ld) of a [T, n] bf16 tensor whose rows are contiguous."""
    import torch

    if x.dtype != torch.bfloat16 or x.dim() != 2 or not x.is_cuda:
        raise ValueError("x must be a 2-D bfloat16 CUDA tensor")
    if x.shape[1] > 0 and x.stride(1) != 1:
        raise ValueError("x rows must be contiguous")
    ld = x.stride(0) if x.shape[0] > 1 else max(x.shape[1], (x.shape[1] + 7) // 8 * 8)
    return x.data_ptr(), x.shape[0], x.shape[1], ld


def signrot_calibrate(x):
    """Calibrate on a bf16 batch [T, n] -> (d int8 [n] on the device, c, t, M_c)."""
    import torch

    ptr, t, n, ld = _rows(x)
    d = torch.empty(n, dtype=torch.int8, device=x.device)
    c = ctypes.c_int32()
    tt = ctypes.c_int64()
    m = ctypes.c_float()
    _run("signrot_calibrate", x, ptr, t, n, ld, d.data_ptr(), ctypes.addressof(c), ctypes.addressof(tt),
         ctypes.addressof(m))
    return d, c.value, tt.value, m.value


def signrot_calibrate_noalloc(x, d_out):
    """signrot_calibrate into a caller-provided d (int8 [n] on the device),
    without any allocation in the library -> (c, t, M_c)."""
    import torch

    ptr, t, n, ld = _rows(x)
    if d_out.dtype != torch.int8 or d_out.numel() != n or not d_out.is_contiguous():
        raise ValueError("d_out must be a contiguous int8 tensor of n entries")
    c = ctypes.c_int32()
    tt = ctypes.c_int64()
    m = ctypes.c_float()
    _run("signrot_calibrate_noalloc", x, ptr, t, n, ld, d_out.data_ptr(), ctypes.addressof(c), ctypes.addressof(tt),
         ctypes.addressof(m))
    return c.value, tt.value, m.value


def signrot_rotate_quant_int4(x, d, y_out: bool = False, out=None):
    """bf16 [T, n] and d int8 [n] -> (codes u8 [T, n/2], scale f32 [T], zero f32 [T]
    [, y f32 [T, n]]).  `out` may pass preallocated (codes, scale, zero[, y])."""
    import torch

    ptr, t, n, ld = _rows(x)
    if d.dtype != torch.int8 or d.numel() != n or not d.is_contiguous():
        raise ValueError("d must be a contiguous int8 tensor of n entries")
    if out is None:
        codes = torch.empty((t, n // 2), dtype=torch.uint8, device=x.device)
        scale = torch.empty(t, dtype=torch.float32, device=x.device)
        zero = torch.empty(t, dtype=torch.float32, device=x.device)
        y = torch.empty((t, n), dtype=torch.float32, device=x.device) if y_out else None
    else:
        codes, scale, zero = out[:3]
        y = out[3] if len(out) > 3 else None
    _run("signrot_rotate_quant_int4", x, ptr, t, n, ld, d.data_ptr(), codes.data_ptr(), scale.data_ptr(),
         zero.data_ptr(), y.data_ptr() if y is not None else None)
    return (codes, scale, zero, y) if y is not None else (codes, scale, zero)


def signrot_rotate_quant_int4_outlier(x, c: int, sigma: int, y_out: bool = False, out=None):
    """Like signrot_rotate_quant_int4 for d = sigma * (row c of H), given as the
    outlier channel c and sigma = sign(M_c) (what signrot_calibrate returns)."""
    import torch

    ptr, t, n, ld = _rows(x)
    if out is None:
        codes = torch.empty((t, n // 2), dtype=torch.uint8, device=x.device)
        scale = torch.empty(t, dtype=torch.float32, device=x.device)
        zero = torch.empty(t, dtype=torch.float32, device=x.device)
        y = torch.empty((t, n), dtype=torch.float32, device=x.device) if y_out else None
    else:
        codes, scale, zero = out[:3]
        y = out[3] if len(out) > 3 else None
    _run("signrot_rotate_quant_int4_outlier", x, ptr, t, n, ld, int(c), int(sigma), codes.data_ptr(),
         scale.data_ptr(), zero.data_ptr(), y.data_ptr() if y is not None else None)
    return (codes, scale, zero, y) if y is not None else (codes, scale, zero)


def signrot_rotate_quant_int4_zint(x, c: int, sigma: int, out=None):
    """The integer zero-point variant: zero = rint(-mn / s) (integral floats),
    codes = clamp(rint(y / s) + zero, 0, 15); d given as (c, sigma)."""
    import torch

    ptr, t, n, ld = _rows(x)
    if out is None:
        codes = torch.empty((t, n // 2), dtype=torch.uint8, device=x.device)
        scale = torch.empty(t, dtype=torch.float32, device=x.device)
        zero = torch.empty(t, dtype=torch.float32, device=x.device)
    else:
        codes, scale, zero = out[:3]
    _run("signrot_rotate_quant_int4_zint", x, ptr, t, n, ld, int(c), int(sigma), codes.data_ptr(), scale.data_ptr(),
         zero.data_ptr())
    return codes, scale, zero


def signrot_swiglu_rotate_quant_int4(gate, up, c: int, sigma: int, y_out: bool = False, out=None):
    """The online path on x = bf16(SiLU(gate) * up), the producer fused in:
    gate and up bf16 [T, n] (same row stride) -> (codes, scale, zero[, y])."""
    import torch

    ptr, t, n, ld = _rows(gate)
    uptr, tu, nu, ldu = _rows(up)
    if (tu, nu) != (t, n) or (t > 1 and ldu != ld):
        raise ValueError("gate and up must have the same shape and row stride")
    if out is None:
        codes = torch.empty((t, n // 2), dtype=torch.uint8, device=gate.device)
        scale = torch.empty(t, dtype=torch.float32, device=gate.device)
        zero = torch.empty(t, dtype=torch.float32, device=gate.device)
        y = torch.empty((t, n), dtype=torch.float32, device=gate.device) if y_out else None
    else:
        codes, scale, zero = out[:3]
        y = out[3] if len(out) > 3 else None
    _run("signrot_swiglu_rotate_quant_int4", gate, ptr, uptr, t, n, ld, int(c), int(sigma), codes.data_ptr(),
         scale.data_ptr(), zero.data_ptr(), y.data_ptr() if y is not None else None)
    return (codes, scale, zero, y) if y is not None else (codes, scale, zero)


def signrot_dequant(codes, scale, zero, n: int | None = None):
    """codes u8 [T, n/2], scale/zero f32 [T] -> y_hat f32 [T, n]."""
    import torch

    t = codes.shape[0]
    n = codes.shape[1] * 2 if n is None else int(n)
    y = torch.empty((t, n), dtype=torch.float32, device=codes.device)
    _run("signrot_dequant", codes, codes.data_ptr(), scale.data_ptr(), zero.data_ptr(), t, n, y.data_ptr())
    return y


def signrot_fold_weights(w, d):
    """Weights bf16 [rows, n] (one row per output feature of x . W^T) and the
    activations' sign vector d -> W' = W . H . D / sqrt(n), float32 [rows, n]."""
    import torch

    ptr, rows, n, ld = _rows(w)
    if d.dtype != torch.int8 or d.numel() != n or not d.is_contiguous():
        raise ValueError("d must be a contiguous int8 tensor of n entries")
    out = torch.empty((rows, n), dtype=torch.float32, device=w.device)
    _run("signrot_fold_weights", w, ptr, rows, n, ld, d.data_ptr(), out.data_ptr())
    return out


def signrot_weight_rowsum(w):
    """bf16 [rows, n] -> rowsum f32 [rows], the exact sum of each row."""
    import torch

    ptr, rows, n, ld = _rows(w)
    out = torch.empty(rows, dtype=torch.float32, device=w.device)
    _run("signrot_weight_rowsum", w, ptr, rows, n, ld, out.data_ptr())
    return out


def _linear_operands(codes, w):
    import torch

    if codes.dtype != torch.uint8 or codes.dim() != 2 or not codes.is_contiguous():
        raise ValueError("codes must be a contiguous 2-D uint8 tensor")
    ptr, rows, n, ld = _rows(w)
    if codes.shape[1] * 2 != n:
        raise ValueError(f"codes hold {codes.shape[1] * 2} channels, w has {n}")
    return ptr, rows, n, ld


def signrot_int4_linear(codes, scale, zero, w, rowsum, out=None):
    """INT4 activations (codes u8 [T, n/2], scale/zero f32 [T]) times the folded
    weight w bf16 [rows, n] -> f32 [T, rows] = (scale * (q - zero)) . w^T,
    with rowsum = signrot_weight_rowsum(w)."""
    import torch

    wptr, rows, n, ld = _linear_operands(codes, w)
    t = codes.shape[0]
    for name, v, size in (("scale", scale, t), ("zero", zero, t), ("rowsum", rowsum, rows)):
        if v.dtype != torch.float32 or v.numel() != size or not v.is_contiguous():
            raise ValueError(f"{name} must be a contiguous float32 tensor of {size} entries")
    if out is None:
        out = torch.empty((t, rows), dtype=torch.float32, device=codes.device)
    _run("signrot_int4_linear", codes, codes.data_ptr(), scale.data_ptr(), zero.data_ptr(), t, n, wptr, ld,
         rowsum.data_ptr(), rows, out.data_ptr())
    return out


def int4_linear_kernel_name(codes, w) -> str | None:
    wptr, rows, n, ld = _linear_operands(codes, w)
    r = lib().signrot_int4_linear_kernel_name(codes.data_ptr(), codes.shape[0], n, wptr, ld, rows)
    return r.decode() if r else None


# ---- 8-bit products and the norms around a block -----------------------------

_F32, _BF16 = 0, 1
_NORMS = {"none": 0, "rms": 1, "layer": 2}


def _type_of(dtype, what):
    import torch

    if dtype is torch.bfloat16:
        return _BF16
    if dtype is torch.float32:
        return _F32
    raise ValueError(f"{what} must be bfloat16 or float32, not {dtype}")


def _matrix(v, name, rows, n, dtype, gpu):
    """(pointer, row stride) of a [rows, n] tensor with contiguous rows on GPU
    number `gpu`; None sizes are free."""
    shape = v.shape
    if v.dtype is not dtype or len(shape) != 2 or v.get_device() != gpu:
        raise ValueError(f"{name} must be a 2-D {dtype} tensor on GPU {gpu}")
    t, m = shape
    if (rows is not None and t != rows) or (n is not None and m != n):
        raise ValueError(f"{name} has shape {tuple(shape)}, not [{'*' if rows is None else rows}, "
                         f"{'*' if n is None else n}]")
    step, unit = v.stride()
    if unit != 1 and m > 1:
        raise ValueError(f"{name} rows must be contiguous")
    if t <= 1:
        step = max(step, m)
    elif step < m:
        raise ValueError(f"{name} rows overlap")
    return v.data_ptr(), step


def _vector(v, name, size, dtype, gpu):
    """Pointer of a contiguous vector of `size` entries, 0 for None."""
    if v is None:
        return 0
    if v.dtype is not dtype or v.numel() != size or v.get_device() != gpu or not v.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {size} entries on GPU {gpu}")
    return v.data_ptr()


def _on_gpu(v, name):
    """(device, its number) of a GPU tensor."""
    if not v.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return v.device, v.get_device()


def _empty_codes(t, n, device):
    """int8 [T, n] in rows that start on 16-byte boundaries.  The products take
    them as they are where n is a multiple of 16; else they read them through
    registers, or, when they lay out the weights anew, codes from where they are."""
    import torch

    if n % 16 == 0:
        return torch.empty(t, n, dtype=torch.int8, device=device), n
    pitch = (n + 15) // 16 * 16
    return torch.empty(t, pitch, dtype=torch.int8, device=device)[:, :n], pitch


def signrot_quant_int8(x, sums: bool = False, out=None):
    """bf16 [T, n] -> (codes int8 [T, n], scale f32 [T][, sum int32 [T]]): per
    row scale = max|x| / 127 and codes = rint(127 x / max|x|); sum holds the
    code sums.  On a weight [rows, n] the rows are the output channels.  The
    codes' rows start on 16-byte boundaries (a view of wider rows where n is no
    multiple of 16).  `out` may pass preallocated (codes, scale[, sum])."""
    import torch

    device, gpu = _on_gpu(x, "x")
    ptr, ld = _matrix(x, "x", None, None, torch.bfloat16, gpu)
    t, n = x.shape
    if out is None:
        codes, ldc = _empty_codes(t, n, device)
        scale = torch.empty(t, dtype=torch.float32, device=device)
        out = (codes, scale, torch.empty(t, dtype=torch.int32, device=device)) if sums else (codes, scale)
        qptr, sptr = codes.data_ptr(), scale.data_ptr()
    else:
        out = tuple(out[:3 if sums else 2])
        if len(out) < (3 if sums else 2):
            raise ValueError("out must hold (codes, scale[, sum])")
        qptr, ldc = _matrix(out[0], "codes", t, n, torch.int8, gpu)
        sptr = _vector(out[1], "scale", t, torch.float32, gpu)
    _run("signrot_quant_int8", x, ptr, t, n, ld, qptr, ldc, sptr,
         _vector(out[2], "sum", t, torch.int32, gpu) if sums else 0)
    return out


def _product_out(out, dtype, t, rows, device, gpu):
    """(out, its type, pointer, row stride), allocated when the caller gave none."""
    import torch

    if out is None:
        out = torch.empty(t, rows, dtype=torch.bfloat16 if dtype is None else dtype, device=device)
        return out, _type_of(out.dtype, "out"), out.data_ptr(), rows
    if dtype is not None and out.dtype is not dtype:
        raise ValueError(f"out is {out.dtype}, dtype {dtype}")
    ptr, ldo = _matrix(out, "out", t, rows, out.dtype, gpu)
    return out, _type_of(out.dtype, "out"), ptr, ldo


def _workspace(size, device):
    """(pointer, bytes, owner) of a call's scratch, from torch's allocator on the current stream."""
    import torch

    if size <= 0:
        return 0, 0, None
    w = torch.empty(size, dtype=torch.uint8, device=device)
    return w.data_ptr(), size, w


def signrot_int8_linear(codes, scale, w, w_scale, bias=None, dtype=None, out=None):
    """INT8 activations (codes int8 [T, n], scale f32 [T]) times INT8 weights
    (w int8 [rows, n], w_scale f32 [rows]) -> [T, rows] of `dtype` (bfloat16,
    the default, or float32): scale * w_scale * (codes . w^T) + bias, the sum
    exact in int32.  `out` may pass the result's tensor."""
    import torch

    device, gpu = _on_gpu(codes, "codes")
    aptr, lda = _matrix(codes, "codes", None, None, torch.int8, gpu)
    t, n = codes.shape
    wptr, ldw = _matrix(w, "w", None, n, torch.int8, gpu)
    rows = w.shape[0]
    sptr = _vector(scale, "scale", t, torch.float32, gpu)
    vptr = _vector(w_scale, "w_scale", rows, torch.float32, gpu)
    bptr = _vector(bias, "bias", rows, torch.float32, gpu)
    out, kind, optr, ldo = _product_out(out, dtype, t, rows, device, gpu)
    L = lib()
    ws, size, _owner = _workspace(L.signrot_int8_linear_workspace(aptr, lda, t, n, wptr, ldw, rows), device)
    _run("signrot_int8_linear", codes, aptr, lda, sptr, t, n, wptr, ldw, vptr, bptr, rows, optr, ldo, kind, ws, size)
    return out


def signrot_int4_w8_linear(codes, scale, zero, w, w_scale, w_sum, bias=None, dtype=None, out=None):
    """The rotated INT4 activations (codes u8 [T, n/2], scale and zero f32 [T],
    as signrot_rotate_quant_int4 returns them) times INT8 weights (w int8
    [rows, n], w_scale f32 [rows], w_sum int32 [rows] = w.sum(1)) ->
    [T, rows] of `dtype` (bfloat16, the default, or float32)."""
    import torch

    device, gpu = _on_gpu(codes, "codes")
    if codes.dtype is not torch.uint8 or codes.dim() != 2 or not codes.is_contiguous():
        raise ValueError("codes must be a contiguous 2-D uint8 tensor")
    t, n = codes.shape[0], codes.shape[1] * 2
    wptr, ldw = _matrix(w, "w", None, n, torch.int8, gpu)
    rows = w.shape[0]
    sptr = _vector(scale, "scale", t, torch.float32, gpu)
    zptr = _vector(zero, "zero", t, torch.float32, gpu)
    vptr = _vector(w_scale, "w_scale", rows, torch.float32, gpu)
    uptr = _vector(w_sum, "w_sum", rows, torch.int32, gpu)
    bptr = _vector(bias, "bias", rows, torch.float32, gpu)
    out, kind, optr, ldo = _product_out(out, dtype, t, rows, device, gpu)
    L = lib()
    aptr = codes.data_ptr()
    ws, size, _owner = _workspace(L.signrot_int4_w8_linear_workspace(aptr, t, n, wptr, ldw, rows), device)
    _run("signrot_int4_w8_linear", codes, aptr, sptr, zptr, t, n, wptr, ldw, vptr, uptr, bptr, rows, optr, ldo, kind,
         ws, size)
    return out


def int8_linear_kernel_name(codes, w) -> str | None:
    import torch

    aptr, lda = _matrix(codes, "codes", None, None, torch.int8, codes.get_device())
    wptr, ldw = _matrix(w, "w", None, codes.shape[1], torch.int8, codes.get_device())
    r = lib().signrot_int8_linear_kernel_name(aptr, lda, codes.shape[0], codes.shape[1], wptr, ldw, w.shape[0])
    return r.decode() if r else None


def int4_w8_linear_kernel_name(codes, w) -> str | None:
    import torch

    n = codes.shape[1] * 2
    wptr, ldw = _matrix(w, "w", None, n, torch.int8, codes.get_device())
    r = lib().signrot_int4_w8_linear_kernel_name(codes.data_ptr(), codes.shape[0], n, wptr, ldw, w.shape[0])
    return r.decode() if r else None


class _ResidualNormArgs(ctypes.Structure):
    """signrot_residual_norm_args."""

    _fields_ = [(name, kind) for names, kind in (
        (("tokens", "n"), ctypes.c_int64), (("h",), ctypes.c_void_p), (("ldh",), ctypes.c_int64),
        (("y",), ctypes.c_void_p), (("ldy",), ctypes.c_int64), (("h_out",), ctypes.c_void_p),
        (("ldho",), ctypes.c_int64), (("u",), ctypes.c_void_p), (("ldu",), ctypes.c_int64),
        (("codes",), ctypes.c_void_p), (("ldc",), ctypes.c_int64),
        (("code_scale", "post_weight", "post_bias", "gate"), ctypes.c_void_p), (("ldg",), ctypes.c_int64),
        (("pre_weight", "pre_bias", "mod_scale", "mod_shift"), ctypes.c_void_p), (("ldm",), ctypes.c_int64),
        (("mod_index",), ctypes.c_void_p), (("mod_rows",), ctypes.c_int64),
        (("alpha", "beta", "eps_post", "eps_pre"), ctypes.c_float),
        (("post_norm", "pre_norm", "h_type", "param_type"), ctypes.c_int32)) for name in names]


# the same struct packed in one call (None is no pointer: 0)
_pack_norm_args = struct.Struct("@" + "".join(
    {ctypes.c_int64: "q", ctypes.c_void_p: "P", ctypes.c_float: "f", ctypes.c_int32: "i"}[kind]
    for _, kind in _ResidualNormArgs._fields_)).pack


def _modulation(v, name, t, n, index, dtype, gpu):
    """(pointer, stride, rows) of a gate or modulation: [n] shared by all rows, or [m, n]."""
    if v is None:
        return 0, 0, None
    if v.dim() == 1:
        return _vector(v, name, n, dtype, gpu), 0, None
    ptr, step = _matrix(v, name, None, n, dtype, gpu)
    if v.shape[0] < (1 if index is not None else t):
        raise ValueError(f"{name} has {v.shape[0]} rows for {t} tokens")
    if v.shape[0] == 1 or (index is None and t == 1):
        step = 0  # row 0 is the only one taken
    return ptr, step, v.shape[0]


def _residual_norm(h, y, norm, post_norm, eps, post_eps, post_weight, post_bias, gate, alpha, beta, weight, bias,
                   mod_scale, mod_shift, mod_index, h_out, out, codes):
    """Checks, allocates what the caller did not give and launches; `codes`: out is (codes, scale), not u."""
    import torch

    device, gpu = _on_gpu(h, "h")
    h_type = _type_of(h.dtype, "h")
    hptr, ldh = _matrix(h, "h", None, None, h.dtype, gpu)
    t, n = h.shape
    yptr, ldy = (0, 0) if y is None else _matrix(y, "y", t, n, torch.bfloat16, gpu)
    post_norm = norm if post_norm is None else post_norm
    if norm not in _NORMS or post_norm not in _NORMS:
        raise ValueError(f"norm must be one of {sorted(_NORMS)}")
    param = torch.bfloat16
    for v in (weight, post_weight, bias, post_bias, gate, mod_scale, mod_shift):
        if v is not None:
            param = v.dtype
            break
    p_type = _type_of(param, "the norm's parameters")
    gptr, mptr, cptr, ldg, ldm, mod_rows = 0, 0, 0, 0, 0, 0
    if gate is not None or mod_scale is not None or mod_shift is not None:
        gptr, ldg, grows = _modulation(gate, "gate", t, n, mod_index, param, gpu)
        mptr, ldm, mrows = _modulation(mod_scale, "mod_scale", t, n, mod_index, param, gpu)
        cptr, ldm2, crows = _modulation(mod_shift, "mod_shift", t, n, mod_index, param, gpu)
        if not mptr:
            ldm = ldm2
        elif cptr and ldm != ldm2:
            raise ValueError("mod_scale and mod_shift must have the same row stride")
        counts = {r for r in (grows, mrows, crows) if r is not None}
        if mod_index is not None and len(counts) > 1:
            raise ValueError(f"gate, mod_scale and mod_shift have {sorted(counts)} rows for one mod_index")
        mod_rows = min(counts, default=0)
    if h_out is None:
        h_out = torch.empty(t, n, dtype=h.dtype, device=device)
        hoptr, ldho = h_out.data_ptr(), n
    else:
        hoptr, ldho = _matrix(h_out, "h_out", t, n, h.dtype, gpu)
    uptr, ldu, qptr, ldc, sptr = 0, 0, 0, 0, 0
    if not codes:
        if out is None:
            out = torch.empty(t, n, dtype=torch.bfloat16, device=device)
            uptr, ldu = out.data_ptr(), n
        else:
            uptr, ldu = _matrix(out, "u", t, n, torch.bfloat16, gpu)
    elif out is None:
        q, ldc = _empty_codes(t, n, device)
        out = (q, torch.empty(t, dtype=torch.float32, device=device))
        qptr, sptr = q.data_ptr(), out[1].data_ptr()
    else:
        qptr, ldc = _matrix(out[0], "codes", t, n, torch.int8, gpu)
        sptr = _vector(out[1], "scale", t, torch.float32, gpu)
    args = _pack_norm_args(
        t, n, hptr, ldh, yptr, ldy, hoptr, ldho, uptr, ldu, qptr, ldc, sptr,
        _vector(post_weight, "post_weight", n, param, gpu), _vector(post_bias, "post_bias", n, param, gpu),
        gptr, ldg, _vector(weight, "weight", n, param, gpu), _vector(bias, "bias", n, param, gpu),
        mptr, cptr, ldm, _vector(mod_index, "mod_index", t, torch.int32, gpu), mod_rows,
        alpha, beta, eps if post_eps is None else post_eps, eps, _NORMS[post_norm], _NORMS[norm], h_type, p_type)
    _run("signrot_residual_norm", h, args)
    return h_out, out


def signrot_residual_norm(h, y=None, norm: str = "rms", post_norm: str | None = None, eps: float = 1e-6,
                          post_eps: float | None = None, post_weight=None, post_bias=None, gate=None,
                          alpha: float = 1.0, beta: float = 1.0, weight=None, bias=None, mod_scale=None,
                          mod_shift=None, mod_index=None, h_out=None, out=None):
    """The norms around a block with its gate and residual scale, one pass:

        h' = beta h + alpha gate * Norm_post(y)
        u  = Norm(h') * (1 + mod_scale) + mod_shift

    h (bf16 or f32) and y (bf16, None: no branch) are [T, n]; norm and
    post_norm (default: the same) are "rms", "layer" or "none"; weights and
    biases are [n]; gate, mod_scale and mod_shift are [n], or [m, n] with a row
    per token, or one per sequence picked by mod_index (int32 [T]; the same m
    for all three then), mod_scale and mod_shift in the same layout; all of
    them bf16, or all f32.  Returns (h' of h's type, u bf16).  h_out may be h,
    to update the stream in place; `out` may pass u's tensor."""
    return _residual_norm(h, y, norm, post_norm, eps, post_eps, post_weight, post_bias, gate, alpha, beta, weight,
                          bias, mod_scale, mod_shift, mod_index, h_out, out, False)


def signrot_residual_norm_quant_int8(h, y=None, norm: str = "rms", post_norm: str | None = None, eps: float = 1e-6,
                                     post_eps: float | None = None, post_weight=None, post_bias=None, gate=None,
                                     alpha: float = 1.0, beta: float = 1.0, weight=None, bias=None, mod_scale=None,
                                     mod_shift=None, mod_index=None, h_out=None, out=None):
    """signrot_residual_norm with u quantized as signrot_quant_int8 does, from
    its binary32 values: returns (h', codes int8 [T, n], scale f32 [T]).
    `out` may pass (codes, scale)."""
    h_out, (codes, scale) = _residual_norm(h, y, norm, post_norm, eps, post_eps, post_weight, post_bias, gate, alpha,
                                           beta, weight, bias, mod_scale, mod_shift, mod_index, h_out, out, True)
    return h_out, codes, scale


# ---- microscaled 4-bit floating point (MXFP4) --------------------------------

_MX_RULES = {"floor": 0, "noclip": 1}


def _mx_rule(rule):
    if rule not in _MX_RULES:
        raise ValueError(f"rule must be one of {sorted(_MX_RULES)}")
    return _MX_RULES[rule]


def _mx_out(out, t, n, device, gpu):
    """(out, codes pointer, its row stride, scales pointer, their row stride) of the codes and scales of [T, n]
    values; allocated ones have rows of scales that start on 16-byte boundaries."""
    import torch

    nb = (n + 31) // 32
    if out is None:
        pitch = (nb + 15) // 16 * 16
        codes = torch.empty(t, 16 * nb, dtype=torch.uint8, device=device)
        scale = torch.empty(t, pitch, dtype=torch.uint8, device=device)
        return (codes, scale if pitch == nb else scale[:, :nb]), codes.data_ptr(), 16 * nb, scale.data_ptr(), pitch
    codes, scale = out
    qptr, ldc = _matrix(codes, "codes", t, 16 * nb, torch.uint8, gpu)
    sptr, lds = _matrix(scale, "scale", t, nb, torch.uint8, gpu)
    return (codes, scale), qptr, ldc, sptr, lds


def _mx_operand(codes, scale, names, gpu):
    """(codes pointer, stride, scales pointer, stride, blocks of a row) of an MXFP4 operand."""
    import torch

    qptr, ldc = _matrix(codes, names[0], None, None, torch.uint8, gpu)
    rows, size = codes.shape
    if size % 16 != 0:
        raise ValueError(f"{names[0]} rows hold {size} bytes, not whole blocks of 16")
    sptr, lds = _matrix(scale, names[1], rows, size // 16, torch.uint8, gpu)
    return qptr, ldc, sptr, lds, size // 16


def signrot_quant_mxfp4(x, rule: str = "floor", out=None):
    """bf16 or f32 [T, n] -> (codes u8 [T, 16 nb], scale u8 [T, nb]), nb =
    ceil(n / 32): MXFP4 in blocks of 32 channels along a row, channel 2m in the
    low nibble of byte m, codes beyond n zero, scales 2^(byte - 127) (255: the
    block holds an infinity or NaN).  rule "floor": the scale's exponent is
    floor(log2 max|x|) - 2 and values over 6 scales saturate; "noclip": one more
    where the largest would.  Rows of scales start on 16-byte boundaries (a view
    of wider rows where nb is no multiple of 16).  `out` may pass preallocated
    (codes, scale)."""
    device, gpu = _on_gpu(x, "x")
    kind = _type_of(x.dtype, "x")
    ptr, ld = _matrix(x, "x", None, None, x.dtype, gpu)
    t, n = x.shape
    out, qptr, ldc, sptr, lds = _mx_out(out, t, n, device, gpu)
    _run("signrot_quant_mxfp4", x, ptr, kind, t, n, ld, _mx_rule(rule), qptr, ldc, sptr, lds)
    return out


def signrot_dequant_mxfp4(codes, scale, n: int | None = None, dtype=None, out=None):
    """The values of MXFP4 codes and scales, [T, n] (n: all channels of the
    blocks) of `dtype` (float32, the default, or bfloat16), exact.  `out` may
    pass the result's tensor."""
    import torch

    device, gpu = _on_gpu(codes, "codes")
    qptr, ldc, sptr, lds, nb = _mx_operand(codes, scale, ("codes", "scale"), gpu)
    t = codes.shape[0]
    n = 32 * nb if n is None else int(n)
    if (n + 31) // 32 != nb:
        raise ValueError(f"codes hold {nb} blocks of 32 channels, not {n} channels")
    if out is None and dtype is None:
        dtype = torch.float32
    out, kind, optr, ldo = _product_out(out, dtype, t, n, device, gpu)
    _run("signrot_dequant_mxfp4", codes, qptr, ldc, sptr, lds, t, n, optr, kind, ldo)
    return out


def signrot_mxfp4_linear(codes, scale, w, w_scale, bias=None, dtype=None, out=None):
    """MXFP4 activations (codes u8 [T, 16 nb], scale u8 [T, nb]) times MXFP4
    weights (w u8 [rows, 16 nb], w_scale u8 [rows, nb]) -> [T, rows] of `dtype`
    (bfloat16, the default, or float32), plus bias f32 [rows].  Sums in binary32
    on the matrix cores, which apply the scales.  `out` may pass the result's
    tensor."""
    device, gpu = _on_gpu(codes, "codes")
    aptr, lda, sptr, lds, nb = _mx_operand(codes, scale, ("codes", "scale"), gpu)
    wptr, ldw, vptr, ldws, wb = _mx_operand(w, w_scale, ("w", "w_scale"), gpu)
    if wb != nb:
        raise ValueError(f"codes hold {nb} blocks of 32 channels, w {wb}")
    t, rows = codes.shape[0], w.shape[0]
    import torch

    bptr = _vector(bias, "bias", rows, torch.float32, gpu)
    out, kind, optr, ldo = _product_out(out, dtype, t, rows, device, gpu)
    sizes = (aptr, lda, sptr, lds, t, 32 * nb, wptr, ldw, vptr, ldws)
    ws, size, _owner = _workspace(lib().signrot_mxfp4_linear_workspace(*sizes, rows), device)
    _run("signrot_mxfp4_linear", codes, *sizes, bptr, rows, optr, ldo, kind, ws, size)
    return out


def mxfp4_linear_kernel_name(codes, scale, w, w_scale) -> str | None:
    gpu = codes.get_device()
    aptr, lda, sptr, lds, nb = _mx_operand(codes, scale, ("codes", "scale"), gpu)
    wptr, ldw, vptr, ldws, _ = _mx_operand(w, w_scale, ("w", "w_scale"), gpu)
    r = lib().signrot_mxfp4_linear_kernel_name(aptr, lda, sptr, lds, codes.shape[0], 32 * nb, wptr, ldw, vptr, ldws,
                                               w.shape[0])
    return r.decode() if r else None


def signrot_rotate_quant_mxfp4(x, c: int, sigma: int, rule: str = "floor", out=None):
    """bf16 [T, n] -> MXFP4 (codes, scale) of its rotation y = (x H / sqrt n) * d,
    d = sigma * (row c of H) (what signrot_calibrate returns): what
    signrot_quant_mxfp4 gives of the binary32 y.  `out` may pass preallocated
    (codes, scale), codes rows on 16-byte boundaries."""
    device, gpu = _on_gpu(x, "x")
    ptr, t, n, ld = _rows(x)
    size = lib().signrot_rotate_quant_mxfp4_workspace(t, n)
    if size < 0:
        check(SIGNROT_EUNSUPPORTED_N, "signrot_rotate_quant_mxfp4")
    out, qptr, ldc, sptr, lds = _mx_out(out, t, n, device, gpu)
    ws, size, _owner = _workspace(size, device)
    _run("signrot_rotate_quant_mxfp4", x, ptr, t, n, ld, int(c), int(sigma), _mx_rule(rule), qptr, ldc, sptr, lds, ws,
         size)
    return out


def signrot_swiglu_rotate_quant_mxfp4(gate, up, c: int, sigma: int, rule: str = "floor", out=None):
    """signrot_rotate_quant_mxfp4 of x = bf16(SiLU(gate) * up), the producer
    fused in: gate and up bf16 [T, n] with the same row stride, n one of the
    fused kernels' widths."""
    device, gpu = _on_gpu(gate, "gate")
    ptr, t, n, ld = _rows(gate)
    uptr, tu, nu, ldu = _rows(up)
    if (tu, nu) != (t, n) or (t > 1 and ldu != ld) or up.get_device() != gpu:
        raise ValueError("gate and up must have the same shape, row stride and GPU")
    out, qptr, ldc, sptr, lds = _mx_out(out, t, n, device, gpu)
    _run("signrot_swiglu_rotate_quant_mxfp4", gate, ptr, uptr, t, n, ld, int(c), int(sigma), _mx_rule(rule), qptr, ldc,
         sptr, lds)
    return out


# ---- the norm of each head and the position rotation --------------------------


class _QkNormRopeArgs(ctypes.Structure):
    """signrot_qk_norm_rope_args."""

    _fields_ = [(name, kind) for names, kind in (
        (("tokens", "head", "rotary"), ctypes.c_int64),
        (("q",), ctypes.c_void_p), (("ldq", "hsq"), ctypes.c_int64),
        (("q_out",), ctypes.c_void_p), (("ldqo", "hsqo"), ctypes.c_int64),
        (("k",), ctypes.c_void_p), (("ldk", "hsk"), ctypes.c_int64),
        (("k_out",), ctypes.c_void_p), (("ldko", "hsko"), ctypes.c_int64),
        (("cos", "sin"), ctypes.c_void_p), (("ldt", "places"), ctypes.c_int64),
        (("positions", "q_weight", "k_weight", "q_bias", "k_bias"), ctypes.c_void_p),
        (("q_heads", "k_heads"), ctypes.c_int32), (("eps",), ctypes.c_float),
        (("norm", "interleaved", "positions_64", "in_type", "out_type", "param_type"), ctypes.c_int32))
        for name in names]


_pack_qk_args = struct.Struct("@" + "".join(
    {ctypes.c_int64: "q", ctypes.c_void_p: "P", ctypes.c_float: "f", ctypes.c_int32: "i"}[kind]
    for _, kind in _QkNormRopeArgs._fields_) + "0q").pack  # the struct's size is a multiple of eight


def _heads_of(v, name, t, heads, d, dtype, gpu):
    """(its shape, pointer, token stride, head stride) of a [T, heads, d] tensor with contiguous heads; None sizes
    are free."""
    shape = v.shape
    if v.dtype is not dtype or len(shape) != 3 or v.get_device() != gpu:
        raise ValueError(f"{name} must be a 3-D {dtype} tensor on GPU {gpu}")
    if (t is not None and shape[0] != t) or (heads is not None and shape[1] != heads) or (
            d is not None and shape[2] != d):
        raise ValueError(f"{name} has shape {tuple(shape)}, not "
                         f"[{'*' if t is None else t}, {'*' if heads is None else heads}, {'*' if d is None else d}]")
    step, hop, unit = v.stride()
    if unit != 1:
        raise ValueError(f"{name} heads must be contiguous")
    return shape, v.data_ptr(), step, hop


def _heads_out(v, name, shape, dtype, device, gpu):
    """(out, pointer, strides) of the result of a [T, heads, d] shape, allocated when v is None."""
    import torch

    t, heads, d = shape
    if v is None:
        v = torch.empty(t, heads, d, dtype=dtype, device=device)
        return v, v.data_ptr(), heads * d, d
    _, ptr, step, hop = _heads_of(v, name, t, heads, d, dtype, gpu)
    reach = d  # elements of the axes so far: the next one has to step over them
    for stride, count in ((hop, heads), (step, t)) if hop <= step else ((step, t), (hop, heads)):
        if count > 1:
            if stride < reach:
                raise ValueError(f"{name} heads overlap")
            reach += stride * (count - 1)
    return v, ptr, step, hop


def signrot_qk_norm_rope(q, k=None, cos=None, sin=None, positions=None, norm: str = "rms", eps: float = 1e-6,
                         q_weight=None, k_weight=None, q_bias=None, k_bias=None, interleaved: bool = False, dtype=None,
                         q_out=None, k_out=None):
    """The norm of each head of the queries and keys, then the rotation of its
    first 2 R channels by the token's position, in one pass:

        v = Norm(x);  a' = a cos[p] - b sin[p],  b' = b cos[p] + a sin[p]

    q [T, heads, D] and k [T, kv_heads, D] (or None) are bf16 or f32, of any
    token and head stride, D even in [8, 512]; cos and sin are f32 [places, R]
    (None: no rotation), read at row positions[t] (int32 or int64 [T], clamped
    into the table) or t; the pair p is channels (p, p + R), or (2p, 2p + 1) when
    interleaved.  norm is "rms", "layer" or "none", weights and biases [D], all
    bf16 or all f32.  Returns (q', k') of `dtype` (default: the input's); q_out
    and k_out may pass their tensors, among them q and k themselves."""
    import torch

    device, gpu = _on_gpu(q, "q")
    in_type = _type_of(q.dtype, "q")
    q_shape, qptr, ldq, hsq = _heads_of(q, "q", None, None, None, q.dtype, gpu)
    t, heads, d = q_shape
    if norm not in _NORMS:
        raise ValueError(f"norm must be one of {sorted(_NORMS)}")
    for v in (q_out, k_out):
        if v is not None:
            if dtype is not None and v.dtype is not dtype:
                raise ValueError(f"an output is {v.dtype}, dtype {dtype}")
            dtype = v.dtype
    if dtype is None or dtype is q.dtype:
        dtype, out_type = q.dtype, in_type
    else:
        out_type = _type_of(dtype, "the result")
    param, p_type, vectors = None, _BF16, []
    for v, name in ((q_weight, "q_weight"), (k_weight, "k_weight"), (q_bias, "q_bias"), (k_bias, "k_bias")):
        if v is None:
            vectors.append(0)
            continue
        if param is None:
            param = v.dtype
            p_type = _type_of(param, "the norm's parameters")
        vectors.append(_vector(v, name, d, param, gpu))
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    cptr = zptr = pptr = ldt = places = rotary = wide = 0
    if cos is not None:
        cptr, ldt = _matrix(cos, "cos", None, None, torch.float32, gpu)
        places, half = cos.shape
        rotary = 2 * half
        zptr, lds = _matrix(sin, "sin", places, half, torch.float32, gpu)
        if places > 1 and ldt != lds:
            raise ValueError("cos and sin must have the same row stride")
        if positions is not None:
            wide = positions.dtype is torch.int64
            pptr = _vector(positions, "positions", t, torch.int64 if wide else torch.int32, gpu)
    kptr = ldk = hsk = koptr = ldko = hsko = kv = 0
    q_out, qoptr, ldqo, hsqo = _heads_out(q_out, "q_out", q_shape, dtype, device, gpu)
    if k is not None:
        k_shape, kptr, ldk, hsk = _heads_of(k, "k", t, None, d, q.dtype, gpu)
        kv = k_shape[1]
        k_out, koptr, ldko, hsko = _heads_out(k_out, "k_out", k_shape, dtype, device, gpu)
    elif k_out is not None:
        raise ValueError("k_out without k")
    args = _pack_qk_args(
        t, d, rotary, qptr, ldq, hsq, qoptr, ldqo, hsqo, kptr, ldk, hsk, koptr, ldko, hsko, cptr, zptr, ldt, places,
        pptr, *vectors, heads, kv, eps,
        _NORMS[norm], 1 if interleaved else 0, 1 if wide else 0, in_type, out_type, p_type)
    _run("signrot_qk_norm_rope", q, args)
    return q_out, k_out


def signrot_stream_ceiling(x, out=None):
    """The memory-traffic ceiling kernel (a measurement aid: the online path's
    bytes per token, no arithmetic) on bf16 [T, n] -> (u8 [T, n/2], f32 [T],
    f32 [T])."""
    import torch

    ptr, t, n, ld = _rows(x)
    if out is None:
        out = (torch.empty((t, n // 2), dtype=torch.uint8, device=x.device),
               torch.empty(t, dtype=torch.float32, device=x.device),
               torch.empty(t, dtype=torch.float32, device=x.device))
    _run("signrot_stream_ceiling", x, ptr, t, n, ld, out[0].data_ptr(), out[1].data_ptr(), out[2].data_ptr())
    return out


# short aliases
calibrate = signrot_calibrate
rotate_quant_int4 = signrot_rotate_quant_int4
rotate_quant_int4_outlier = signrot_rotate_quant_int4_outlier
rotate_quant_int4_zint = signrot_rotate_quant_int4_zint
swiglu_rotate_quant_int4 = signrot_swiglu_rotate_quant_int4
dequant = signrot_dequant
fold_weights = signrot_fold_weights
weight_rowsum = signrot_weight_rowsum
int4_linear = signrot_int4_linear
quant_int8 = signrot_quant_int8
int8_linear = signrot_int8_linear
int4_w8_linear = signrot_int4_w8_linear
residual_norm = signrot_residual_norm
residual_norm_quant_int8 = signrot_residual_norm_quant_int8
quant_mxfp4 = signrot_quant_mxfp4
dequant_mxfp4 = signrot_dequant_mxfp4
mxfp4_linear = signrot_mxfp4_linear
rotate_quant_mxfp4 = signrot_rotate_quant_mxfp4
swiglu_rotate_quant_mxfp4 = signrot_swiglu_rotate_quant_mxfp4
qk_norm_rope = signrot_qk_norm_rope
