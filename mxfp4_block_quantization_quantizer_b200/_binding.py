"""ctypes binding of libmxfp4 (include/mxfp4.h).

Argument marshalling only: tensors become device pointers and sizes, the
current torch stream becomes the cudaStream_t, output buffers are allocated
with torch. Every step of the computation runs in the library's kernels.
There is no fallback: if the library is missing, or a tensor is not on a CUDA
device, the call raises.
"""
import ctypes
import functools
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmxfp4.so")

F32, BF16 = 0, 1
ROWS, COLS = 0, 1
RNE, SR = 0, 1
# Bit of the tensor-core entry points' status word: a bounded wait ran out.
STATUS_WAIT_TIMEOUT = 1

# Every symbol include/mxfp4.h declares.
SYMBOLS = ("mxfp4_quantize", "mxfp4_quantize_oas", "mxfp4_dequantize",
           "mxfp4_double_quantize", "mxfp4_double_quantize_oas",
           "mxfp4_rht_quantize", "mxfp4_rht_quantize_oas", "mxfp4_osc_step",
           "mxfp4_osc_synthetic_update", "mxfp4_qramp_step", "mxfp4_qema_quantize",
           "mxfp4_scales_to_blocked", "mxfp4_gemm", "mxfp4_gemm_quantize_a",
           "mxfp4_gemv", "mxfp4_gemv_workspace", "mxfp4_newton_schulz", "mxfp4_newton_schulz_workspace",
           "mxfp4_layernorm", "mxfp4_layernorm_quantize", "mxfp4_layernorm_backward",
           "mxfp4_layernorm_backward_workspace", "mxfp4_status_string")


class Mxfp4Error(RuntimeError):
    def __init__(self, status, what):
        self.status = status
        super().__init__("%s: %s (status %d)" % (what, status_string(status), status))


_lib = None


def lib():
    """The loaded libmxfp4 (ctypes.CDLL). Raises if it was not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                "libmxfp4.so is not built (expected at %s); run "
                "__graft_entry__.build() or python -m "
                "mxfp4_block_quantization_quantizer_b200.build" % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, i64, u64, u32, i32 = (ctypes.c_void_p, ctypes.c_int64,
                                  ctypes.c_uint64, ctypes.c_uint32,
                                  ctypes.c_int)
        sig = {
            "mxfp4_quantize": [vp, i32, i64, i64, i32, i32, u64, vp, vp, vp],
            "mxfp4_quantize_oas": [vp, i32, i64, i64, i32, i32, u64, vp, vp, vp],
            "mxfp4_dequantize": [vp, vp, i64, i64, i32, vp, i32, vp],
            "mxfp4_double_quantize": [vp, i32, i64, i64, u64, vp, vp, vp, vp,
                                      vp],
            "mxfp4_double_quantize_oas": [vp, i32, i64, i64, u64, vp, vp, vp,
                                          vp, vp],
            "mxfp4_rht_quantize": [vp, i32, i64, i64, u64, i32, u64, vp, vp,
                                   vp, vp, vp],
            "mxfp4_rht_quantize_oas": [vp, i32, i64, i64, u64, i32, u64, vp,
                                       vp, vp, vp, vp],
            "mxfp4_osc_step": [vp, vp, vp, vp, i64, i64, i32, ctypes.c_float,
                               vp, vp],
            "mxfp4_osc_synthetic_update": [vp, i64, i64, u64, u32,
                                           ctypes.c_float, vp],
            "mxfp4_qema_quantize": [vp, vp, i64, i64, ctypes.c_float, vp, vp,
                                    vp],
            "mxfp4_qramp_step": [vp, vp, vp, vp, vp, vp, vp, i64, i64, i64, i64,
                                 ctypes.c_float, i64, vp, vp],
            "mxfp4_scales_to_blocked": [vp, i64, i64, vp, vp],
            "mxfp4_gemm": [vp, vp, vp, vp, i64, i64, i64, vp, vp, vp],
            "mxfp4_gemm_quantize_a": [vp, i64, i64, i64, i32, u64, vp, vp, vp, vp,
                                      vp, vp, vp],
        }
        f32 = ctypes.c_float
        sig.update({
            "mxfp4_gemv": [vp, i64, i64, i64, i64, vp, vp, vp, i32, vp, i64, vp, vp],
            "mxfp4_newton_schulz": [vp, i32, i64, i64, i32, f32, f32, f32, f32, f32, vp, i32, vp,
                                    i64, vp, vp],
            "mxfp4_layernorm": [vp, i32, i64, i64, i64, vp, vp, f32, vp, vp, vp, vp],
            "mxfp4_layernorm_quantize": [vp, i32, i64, i64, i64, vp, vp, f32, vp, vp, vp, vp,
                                         vp, vp],
            "mxfp4_layernorm_backward": [vp, vp, i32, i64, i64, i64, i64, vp, vp, vp, vp, vp,
                                         vp, vp, i64, vp],
        })
        for name, args in sig.items():
            f = getattr(L, name)
            f.argtypes, f.restype = args, i32
        for f in (L.mxfp4_layernorm_backward_workspace, L.mxfp4_newton_schulz_workspace):
            f.argtypes, f.restype = [i64, i64], i64
        L.mxfp4_gemv_workspace.argtypes = [i64, i64, i64]
        L.mxfp4_gemv_workspace.restype = i64
        L.mxfp4_status_string.argtypes = [i32]
        L.mxfp4_status_string.restype = ctypes.c_char_p
        _lib = L
    return _lib


def status_string(status):
    return lib().mxfp4_status_string(status).decode()


def _check(status, what):
    if status != 0:
        raise Mxfp4Error(status, what)


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return BF16
    if t.dtype == torch.float32:
        return F32
    raise TypeError("expected a bfloat16 or float32 tensor, got %s" % t.dtype)


def _on_device(t, name, device=None):
    """t is a CUDA tensor (on `device` when one is given)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError("%s must be a CUDA tensor" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))


def _cuda2d(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dim() != 2 or not t.is_contiguous():
        raise ValueError("%s must be a contiguous 2-D tensor" % name)
    _on_device(t, name)
    return t


def _buffer(t, name, dtype, numel, device):
    """Check a buffer before its pointer reaches the C ABI, which cannot see
    sizes: the library reads and writes exactly the bytes the header states
    for the given shape, so a smaller, strided, mistyped or foreign-device
    buffer would be read or written out of bounds. Raises before any launch."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if t.numel() != numel:
        raise ValueError("%s must hold %d elements, got %d" % (name, numel, t.numel()))
    _on_device(t, name, device)
    return t


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device, stream=None):
    s = stream if stream is not None else torch.cuda.current_stream(device)
    return ctypes.c_void_p(s.cuda_stream)


def _empty_u8(shape, device):
    return torch.empty(shape, dtype=torch.uint8, device=device)


def quantize(x, axis=ROWS, rounding=RNE, seed=0, out=None, stream=None,
             oas=False):
    """mxfp4_quantize (mxfp4_quantize_oas with oas=True): returns (codes,
    scales) in the layout of `axis`: ROWS -> codes [R, C/2], scales
    [R, C/32]; COLS -> codes [C, R/2], scales [C, R/32]."""
    _cuda2d(x, "x")
    R, C = x.shape
    if out is None:
        shape_c = (R, C // 2) if axis == ROWS else (C, R // 2)
        shape_s = (R, C // 32) if axis == ROWS else (C, R // 32)
        out = (_empty_u8(shape_c, x.device), _empty_u8(shape_s, x.device))
    codes, scales = out
    _buffer(codes, "codes", torch.uint8, R * C // 2, x.device)
    _buffer(scales, "scales", torch.uint8, R * C // 32, x.device)
    fn = lib().mxfp4_quantize_oas if oas else lib().mxfp4_quantize
    _check(fn(_ptr(x), _dtype_code(x), R, C, axis, rounding, seed, _ptr(codes),
              _ptr(scales), _stream(x.device, stream)), "mxfp4_quantize")
    return codes, scales


def dequantize(codes, scales, rows, cols, axis=ROWS, out_dtype=torch.bfloat16,
               out=None, stream=None):
    """mxfp4_dequantize: values [rows, cols] (ROWS) or [cols, rows] (COLS)."""
    _on_device(codes, "codes")
    n = int(rows) * int(cols)
    _buffer(codes, "codes", torch.uint8, n // 2, codes.device)
    _buffer(scales, "scales", torch.uint8, n // 32, codes.device)
    if out is None:
        shape = (rows, cols) if axis == ROWS else (cols, rows)
        out = torch.empty(shape, dtype=out_dtype, device=codes.device)
    _dtype_code(out)
    _buffer(out, "out", out.dtype, n, codes.device)
    _check(lib().mxfp4_dequantize(_ptr(codes), _ptr(scales), rows, cols, axis,
                                  _ptr(out), _dtype_code(out),
                                  _stream(codes.device, stream)),
           "mxfp4_dequantize")
    return out


def double_quantize(x, seed=0, out=None, stream=None, oas=False):
    """mxfp4_double_quantize (mxfp4_double_quantize_oas when oas):
    (row_codes, row_scales, col_codes, col_scales)."""
    _cuda2d(x, "x")
    R, C = x.shape
    if out is None:
        d = x.device
        out = (_empty_u8((R, C // 2), d), _empty_u8((R, C // 32), d),
               _empty_u8((C, R // 2), d), _empty_u8((C, R // 32), d))
    rc, rs, cc, cs = out
    for t, nm, n in ((rc, "row_codes", R * C // 2), (rs, "row_scales", R * C // 32),
                     (cc, "col_codes", R * C // 2), (cs, "col_scales", R * C // 32)):
        _buffer(t, nm, torch.uint8, n, x.device)
    name = "mxfp4_double_quantize_oas" if oas else "mxfp4_double_quantize"
    _check(getattr(lib(), name)(_ptr(x), _dtype_code(x), R, C, seed, _ptr(rc),
                                _ptr(rs), _ptr(cc), _ptr(cs),
                                _stream(x.device, stream)),
           name)
    return out


def _status_word(status, device):
    """The optional device status word of the tensor-core entry points: an
    int32 tensor of one element on `device` (the kernels OR
    MXFP4_STATUS_WAIT_TIMEOUT = 1 into it; the caller zeroes it)."""
    if status is not None:
        _buffer(status, "status", torch.int32, 1, device)
    return _ptr(status)


def rht_quantize(x, sign_seed=0, rounding=RNE, sr_seed=0, want_rotated=False,
                 out=None, stream=None, oas=False, status=None):
    """mxfp4_rht_quantize (mxfp4_rht_quantize_oas when oas): (codes, scales,
    rotated or None), ROWS layout. status: optional int32 CUDA tensor of one
    element, the timeout status word."""
    _cuda2d(x, "x")
    R, C = x.shape
    if out is None:
        d = x.device
        rot = torch.empty((R, C), dtype=torch.float32, device=d) if want_rotated else None
        out = (_empty_u8((R, C // 2), d), _empty_u8((R, C // 32), d), rot)
    codes, scales, rot = out
    _buffer(codes, "codes", torch.uint8, R * C // 2, x.device)
    _buffer(scales, "scales", torch.uint8, R * C // 32, x.device)
    if rot is not None:
        _buffer(rot, "rotated", torch.float32, R * C, x.device)
    st = _status_word(status, x.device)
    name = "mxfp4_rht_quantize_oas" if oas else "mxfp4_rht_quantize"
    _check(getattr(lib(), name)(_ptr(x), _dtype_code(x), R, C, sign_seed, rounding,
                                sr_seed, _ptr(codes), _ptr(scales), _ptr(rot), st,
                                _stream(x.device, stream)),
           name)
    return out


def osc_step(w, w_snap, d_w, d_q, window_end=False, threshold=4.0,
             n_flagged=None, stream=None):
    """mxfp4_osc_step on fp32 tensors, in place. n_flagged: optional int64
    CUDA tensor of one element to which the flag count is added."""
    for name, t in (("w", w), ("w_snap", w_snap), ("d_w", d_w), ("d_q", d_q)):
        _cuda2d(t, name)
        if t.dtype != torch.float32 or t.shape != w.shape:
            raise TypeError("%s must be float32 with the shape of w" % name)
        _on_device(t, name, w.device)
    if n_flagged is not None:
        _buffer(n_flagged, "n_flagged", torch.int64 if n_flagged.dtype != torch.uint64
                else torch.uint64, 1, w.device)
    R, C = w.shape
    _check(lib().mxfp4_osc_step(_ptr(w), _ptr(w_snap), _ptr(d_w), _ptr(d_q),
                                R, C, int(bool(window_end)), threshold,
                                _ptr(n_flagged), _stream(w.device, stream)),
           "mxfp4_osc_step")


def qramp_step(w, delta, w_snap, d_w, d_q, acc, flag, it, track_iters=30, k1=16.0,
               k2=5, n_flagged=None, stream=None):
    """mxfp4_qramp_step: one Q-Ramping iteration, in place. w, delta,
    w_snap, d_w, d_q, acc: fp32 CUDA tensors of one shape; flag: uint8 of
    that shape; n_flagged: optional int64 CUDA tensor of one element."""
    _cuda2d(w, "w")
    if w.dtype != torch.float32:
        raise TypeError("w must be float32")
    for name, t in (("delta", delta), ("w_snap", w_snap), ("d_w", d_w), ("d_q", d_q),
                    ("acc", acc)):
        _buffer(t, name, torch.float32, w.numel(), w.device)
    _buffer(flag, "flag", torch.uint8, w.numel(), w.device)
    if n_flagged is not None:
        _buffer(n_flagged, "n_flagged", torch.int64 if n_flagged.dtype != torch.uint64
                else torch.uint64, 1, w.device)
    R, C = w.shape
    _check(lib().mxfp4_qramp_step(_ptr(w), _ptr(delta), _ptr(w_snap), _ptr(d_w), _ptr(d_q),
                                  _ptr(acc), _ptr(flag), R, C, int(it), int(track_iters),
                                  float(k1), int(k2), _ptr(n_flagged),
                                  _stream(w.device, stream)),
           "mxfp4_qramp_step")


def osc_synthetic_update(w, seed, step, rel_step=1e-4, stream=None):
    """mxfp4_osc_synthetic_update on an fp32 CUDA tensor, in place."""
    _cuda2d(w, "w")
    if w.dtype != torch.float32:
        raise TypeError("w must be float32")
    R, C = w.shape
    _check(lib().mxfp4_osc_synthetic_update(_ptr(w), R, C, seed, step,
                                            rel_step, _stream(w.device, stream)),
           "mxfp4_osc_synthetic_update")


def qema_quantize(w, w_ema, beta=0.998, out=None, stream=None):
    """mxfp4_qema_quantize: update w_ema in place (fp32 CUDA tensors) and
    return the ROWS-layout (codes, scales) of the new w_ema."""
    for name, t in (("w", w), ("w_ema", w_ema)):
        _cuda2d(t, name)
        if t.dtype != torch.float32 or t.shape != w.shape:
            raise TypeError("%s must be float32 with the shape of w" % name)
    _on_device(w_ema, "w_ema", w.device)
    R, C = w.shape
    if out is None:
        out = (_empty_u8((R, C // 2), w.device), _empty_u8((R, C // 32), w.device))
    codes, scales = out
    _buffer(codes, "codes", torch.uint8, R * C // 2, w.device)
    _buffer(scales, "scales", torch.uint8, R * C // 32, w.device)
    _check(lib().mxfp4_qema_quantize(_ptr(w), _ptr(w_ema), R, C, beta,
                                     _ptr(codes), _ptr(scales),
                                     _stream(w.device, stream)),
           "mxfp4_qema_quantize")
    return codes, scales


def scales_to_blocked(scales, out=None, stream=None):
    """mxfp4_scales_to_blocked: the [rows, groups] uint8 CUDA scales in the
    blocked order of block-scaled GEMMs, returned as a
    [ceil(rows/128)*128, ceil(groups/4)*4] uint8 tensor (storage order)."""
    _cuda2d(scales, "scales")
    if scales.dtype != torch.uint8:
        raise TypeError("scales must be uint8")
    rows, groups = scales.shape
    if out is None:
        out = _empty_u8((-(-rows // 128) * 128, -(-groups // 4) * 4),
                        scales.device)
    _buffer(out, "out", torch.uint8, -(-rows // 128) * 128 * (-(-groups // 4) * 4),
            scales.device)
    _check(lib().mxfp4_scales_to_blocked(_ptr(scales), rows, groups, _ptr(out),
                                         _stream(scales.device, stream)),
           "mxfp4_scales_to_blocked")
    return out


def gemm(a_codes, a_blocked, b_codes, b_blocked, k, out=None, stream=None, status=None):
    """mxfp4_gemm: C = A B^T in fp32 for MXFP4 operands given as K-major
    codes [rows, k/2] and blocked scales (from scales_to_blocked). status:
    optional int32 CUDA tensor of one element, the timeout status word."""
    for name, t in (("a_codes", a_codes), ("a_blocked", a_blocked),
                    ("b_codes", b_codes), ("b_blocked", b_blocked)):
        _cuda2d(t, name)
        if t.dtype != torch.uint8:
            raise TypeError("%s must be uint8" % name)
    m, n = a_codes.shape[0], b_codes.shape[0]
    if a_codes.shape[1] * 2 != k or b_codes.shape[1] * 2 != k:
        raise ValueError("codes must have k/2 bytes per row")
    for name, t, rows in (("a_blocked", a_blocked, m), ("b_blocked", b_blocked, n)):
        need = -(-rows // 128) * 128 * (-(-k // 128) * 4)
        if t.numel() != need:
            raise ValueError("%s must hold %d bytes" % (name, need))
    for name, t in (("a_blocked", a_blocked), ("b_codes", b_codes),
                    ("b_blocked", b_blocked)):
        _on_device(t, name, a_codes.device)
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=a_codes.device)
    _buffer(out, "out", torch.float32, m * n, a_codes.device)
    st = _status_word(status, a_codes.device)
    _check(lib().mxfp4_gemm(_ptr(a_codes), _ptr(a_blocked), _ptr(b_codes),
                            _ptr(b_blocked), m, n, k, _ptr(out), st,
                            _stream(a_codes.device, stream)), "mxfp4_gemm")
    return out


def gemm_quantize_a(x, b_codes, b_blocked, rounding=RNE, seed=0, out=None, want_a=False,
                    stream=None, status=None):
    """mxfp4_gemm_quantize_a: C = Q(x) B^T in fp32, x bf16 [m, k] (k a
    multiple of 256) quantized 1x32 (rounding RNE, or SR keyed by seed)
    inside the GEMM's load stage, B given as K-major codes [n, k/2] and
    blocked scales. Returns C, or (C, a_codes, a_scales) with want_a (Q(x)
    in the ROWS layout)."""
    _cuda2d(x, "x")
    if x.dtype != torch.bfloat16:
        raise TypeError("x must be bfloat16")
    m, k = x.shape
    for name, t in (("b_codes", b_codes), ("b_blocked", b_blocked)):
        _cuda2d(t, name)
        if t.dtype != torch.uint8:
            raise TypeError("%s must be uint8" % name)
        _on_device(t, name, x.device)
    n = b_codes.shape[0]
    if b_codes.shape[1] * 2 != k:
        raise ValueError("b_codes must have k/2 bytes per row")
    need = -(-n // 128) * 128 * (-(-k // 128) * 4)
    if b_blocked.numel() != need:
        raise ValueError("b_blocked must hold %d bytes" % need)
    d = x.device
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=d)
        if want_a:
            out = (out, _empty_u8((m, k // 2), d), _empty_u8((m, k // 32), d))
    c, ac, as_ = (out if want_a else (out, None, None))
    _buffer(c, "out", torch.float32, m * n, d)
    if want_a:
        _buffer(ac, "a_codes", torch.uint8, m * k // 2, d)
        _buffer(as_, "a_scales", torch.uint8, m * k // 32, d)
    st = _status_word(status, d)
    _check(lib().mxfp4_gemm_quantize_a(_ptr(x), m, n, k, rounding, seed, _ptr(b_codes),
                                       _ptr(b_blocked), _ptr(c), _ptr(ac), _ptr(as_), st,
                                       _stream(d, stream)), "mxfp4_gemm_quantize_a")
    return out


def _addr(t):
    return None if t is None else t.data_ptr()


_entry = {}   # entry points by name, as they are first called


def _call(name, device, stream, *args):
    """Call the entry point `name` on `stream` (by default the current stream
    of `device`) with `device` as the current one, where its launches go."""
    fn = _entry.get(name)
    if fn is None:
        fn = _entry[name] = getattr(lib(), name)
    i = device.index
    s = torch._C._cuda_getCurrentRawStream(i) if stream is None else stream.cuda_stream
    if torch._C._cuda_getDevice() == i:
        status = fn(*args, s)
    else:
        with torch.cuda.device(i):
            status = fn(*args, s)
    if status != 0:
        raise Mxfp4Error(status, name)


def _f32(t, name, n, device):
    """_buffer for fp32, whose usual answer costs less."""
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.float32 and t.is_contiguous()
            and t.numel() == n and t.is_cuda and t.device == device):
        _buffer(t, name, torch.float32, n, device)


def _new(shape, dtype, device, stream):
    """A new tensor for work on `stream` (None: the current one). From the
    memory of that stream, where what used it before has ended in order, and
    kept until the caller's current stream is done with it too."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream(device))
    return t


def _like(x, stream):
    """A new contiguous tensor of x's shape and type."""
    if stream is None and x.is_contiguous():
        return torch.empty_like(x)
    return _new(x.shape, x.dtype, x.device, stream)


def _rows2d(t, name):
    """A 2-D tensor whose rows are contiguous (they may lie apart, as in a
    view of a wider tensor). Returns its row stride in elements."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a CUDA tensor" % name)
    if t.dim() != 2:
        raise ValueError("%s must be a 2-D tensor with contiguous rows" % name)
    rows, cols = t.shape
    ld, one = t.stride()
    if one != 1 and cols > 1:
        raise ValueError("%s must be a 2-D tensor with contiguous rows" % name)
    _on_device(t, name)
    if rows <= 1:
        return max(1, cols)
    if ld < cols:
        raise ValueError("the rows of %s overlap" % name)
    return ld


def _span(t):
    """First and last + 1 address of the elements of t."""
    last = sum((n - 1) * s for n, s in zip(t.shape, t.stride()))
    a = t.data_ptr()
    return (a, a + (last + 1) * t.element_size()) if t.numel() else (a, a)


def _apart(written, read=()):
    """Refuse written tensors, (name, tensor or None) pairs, whose memory meets
    that of a tensor that is read, or of one another."""
    taken = [_span(t) for t in read if t is not None]
    for name, t in written:
        if t is None:
            continue
        a0, a1 = _span(t)
        for b0, b1 in taken:
            if a0 < b1 and b0 < a1:
                raise ValueError("%s overlaps another argument" % name)
        taken.append((a0, a1))


def _used(workspace, need):
    """The part of a workspace that a call writes: its first `need` bytes."""
    return None if workspace is None else workspace.view(-1)[:need]


def gemv(x, b_codes, b_blocked, out_dtype=torch.bfloat16, out=None, workspace=None, stream=None,
         status=None):
    """mxfp4_gemv: Y = x B^T for a few bf16 rows x [m, k] (contiguous rows,
    any row stride that is a multiple of 8; not quantized) and an MXFP4
    weight B given as K-major codes [n, k/2] and blocked scales. Y is bf16 or
    fp32 [m, n]. workspace: optional uint8 CUDA tensor of
    mxfp4_gemv_workspace(m, n, k) bytes; status: optional int32 CUDA tensor
    of one element, the timeout status word."""
    ldx = _rows2d(x, "x")
    if x.dtype != torch.bfloat16:
        raise TypeError("x must be bfloat16")
    m, k = x.shape
    d = x.device
    if not isinstance(b_codes, torch.Tensor) or b_codes.dim() != 2 or b_codes.shape[1] * 2 != k:
        raise ValueError("b_codes must be a 2-D tensor with k/2 bytes per row")
    n = b_codes.shape[0]
    _buffer(b_codes, "b_codes", torch.uint8, n * k // 2, d)
    _buffer(b_blocked, "b_blocked", torch.uint8, -(-n // 128) * 128 * (-(-k // 128) * 4), d)
    given = out is not None or workspace is not None or status is not None
    if out is None:
        out = _new((m, n), out_dtype, d, stream)
    else:
        _buffer(out, "out", out.dtype, m * n, d)
    st = None if status is None else _addr(_buffer(status, "status", torch.int32, 1, d))
    need = _workspace_size("mxfp4_gemv_workspace", m, n, k)
    workspace = _workspace(workspace, need, d, stream) if need > 0 else None
    if given:
        _apart((("out", out), ("workspace", _used(workspace, need)), ("status", status)),
               (x, b_codes, b_blocked))
    _call("mxfp4_gemv", d, stream, x.data_ptr(), m, n, k, ldx, b_codes.data_ptr(),
          b_blocked.data_ptr(), out.data_ptr(), _dtype_code(out), _addr(workspace), max(need, 0),
          st)
    return out


def _norm_inputs(x, weight, bias):
    ldx = _rows2d(x, "x")
    if weight is not None:
        _f32(weight, "weight", x.shape[1], x.device)
    if bias is not None:
        _f32(bias, "bias", x.shape[1], x.device)
    return ldx, _dtype_code(x)


def layernorm(x, weight=None, bias=None, eps=1e-5, want_stats=False, out=None, stream=None):
    """mxfp4_layernorm: y = (x - mean) rstd weight + bias over the rows of x
    (bf16 or fp32, contiguous rows, any row stride), weight and bias fp32
    [cols] or None. Returns y, or (y, mean, rstd) with want_stats (out then
    holds the three). No autograd graph is recorded, whatever requires grad:
    layernorm_backward gives the gradients."""
    ldx, dt = _norm_inputs(x, weight, bias)
    R, C = x.shape
    d = x.device
    mean = rstd = None
    if out is None:
        out = y = _like(x, stream)
        if want_stats:
            mean = _new(R, torch.float32, d, stream)
            rstd = _new(R, torch.float32, d, stream)
            out = (y, mean, rstd)
    else:
        y = out
        if want_stats:
            y, mean, rstd = out
            _buffer(mean, "mean", torch.float32, R, d)
            _buffer(rstd, "rstd", torch.float32, R, d)
        _buffer(y, "out", x.dtype, R * C, d)
        _apart((("out", y), ("mean", mean), ("rstd", rstd)), (x, weight, bias))
    _call("mxfp4_layernorm", d, stream, x.data_ptr(), dt, R, C, ldx, _addr(weight), _addr(bias),
          eps, y.data_ptr(), _addr(mean), _addr(rstd))
    return out


def layernorm_quantize(x, weight=None, bias=None, eps=1e-5, want_y=False, want_stats=False,
                       out=None, stream=None):
    """mxfp4_layernorm_quantize: the ROWS-layout (codes, scales) of the
    nearest-even quantization of layernorm(x, weight, bias, eps), and y, mean
    and rstd where wanted: (codes, scales[, y][, mean, rstd]). No autograd
    graph is recorded."""
    ldx, dt = _norm_inputs(x, weight, bias)
    R, C = x.shape
    d = x.device
    given = out is not None
    if out is None:
        out = (_new((R, C // 2), torch.uint8, d, stream),
               _new((R, C // 32), torch.uint8, d, stream))
        if want_y:
            out += (_new((R, C), x.dtype, d, stream),)
        if want_stats:
            out += (_new(R, torch.float32, d, stream), _new(R, torch.float32, d, stream))
    if len(out) != 2 + bool(want_y) + 2 * bool(want_stats):
        raise ValueError("out must hold codes, scales and what is wanted beside them")
    codes, scales = out[:2]
    y = out[2] if want_y else None
    mean, rstd = out[-2:] if want_stats else (None, None)
    _buffer(codes, "codes", torch.uint8, R * C // 2, d)
    _buffer(scales, "scales", torch.uint8, R * C // 32, d)
    if want_y:
        _buffer(y, "y", x.dtype, R * C, d)
    if want_stats:
        _buffer(mean, "mean", torch.float32, R, d)
        _buffer(rstd, "rstd", torch.float32, R, d)
    if given:
        _apart((("codes", codes), ("scales", scales), ("y", y), ("mean", mean), ("rstd", rstd)),
               (x, weight, bias))
    _call("mxfp4_layernorm_quantize", d, stream, x.data_ptr(), dt, R, C, ldx, _addr(weight),
          _addr(bias), eps, _addr(y), _addr(mean), _addr(rstd), codes.data_ptr(),
          scales.data_ptr())
    return out


@functools.lru_cache(maxsize=4096)
def _workspace_size(name, *shape):
    """Bytes that the entry point `name` needs for a shape (its _workspace
    function: host arithmetic, the same answer every time)."""
    return getattr(lib(), name)(*shape)


def _workspace(workspace, need, device, stream):
    """A caller's workspace (uint8, at least `need` bytes) or a new one."""
    if workspace is None:
        return _new(max(need, 16), torch.uint8, device, stream)
    if not isinstance(workspace, torch.Tensor) or workspace.numel() < need:
        raise ValueError("workspace must be a uint8 tensor of at least %d bytes" % need)
    return _buffer(workspace, "workspace", torch.uint8, workspace.numel(), device)


def layernorm_backward(dy, x, mean, rstd, weight=None, want_params=True, out=None,
                       workspace=None, stream=None):
    """mxfp4_layernorm_backward: (dx, dw, db) of layernorm for the gradient
    dy of its output, with the forward pass's mean and rstd; dx alone with
    want_params=False. dx has x's type, dw and db are fp32 (the gradients of
    the weight and the bias). workspace: optional uint8 CUDA tensor."""
    ldx, dt = _norm_inputs(x, weight, None)
    lddy = _rows2d(dy, "dy")
    if dy.dtype != x.dtype or dy.shape != x.shape:
        raise ValueError("dy must have the type and shape of x")
    R, C = x.shape
    d = x.device
    _on_device(dy, "dy", d)
    _f32(mean, "mean", R, d)
    _f32(rstd, "rstd", R, d)
    dw = db = None
    given = out is not None or workspace is not None
    if out is None:
        out = dx = _like(x, stream)
        if want_params:
            dw = _new(C, torch.float32, d, stream)
            db = _new(C, torch.float32, d, stream)
            out = (dx, dw, db)
    else:
        dx = out
        if want_params:
            dx, dw, db = out
            _buffer(dw, "dw", torch.float32, C, d)
            _buffer(db, "db", torch.float32, C, d)
        _buffer(dx, "out", x.dtype, R * C, d)
    need = size = 0
    if want_params:
        need = _workspace_size("mxfp4_layernorm_backward_workspace", R, C)
        workspace = _workspace(workspace, need, d, stream)
        size = workspace.numel()
    else:
        workspace = None
    if given:
        # dw and db are written when all inputs have been read
        used = _used(workspace, need)
        _apart((("out", dx), ("workspace", used)), (x, dy, mean, rstd, weight))
        _apart((("out", dx), ("workspace", used), ("dw", dw), ("db", db)))
    _call("mxfp4_layernorm_backward", d, stream, dy.data_ptr(), x.data_ptr(), dt, R, C, lddy, ldx,
          _addr(weight), mean.data_ptr(), rstd.data_ptr(), dx.data_ptr(), _addr(dw), _addr(db),
          _addr(workspace), size)
    return out


def newton_schulz(g, steps=5, coeffs=(3.4445, -4.7750, 2.0315), eps=1e-7, scale=1.0,
                  out_dtype=None, out=None, workspace=None, stream=None, status=None):
    """mxfp4_newton_schulz: scale times the nearly orthogonal matrix that
    `steps` Newton-Schulz steps with coefficients (a, b, c) make of g (bf16
    or fp32, any sides), in out_dtype (g's by default). workspace: optional
    uint8 CUDA tensor of mxfp4_newton_schulz_workspace(rows, cols) bytes;
    status: optional int32 CUDA tensor of one element."""
    _cuda2d(g, "g")
    dt = _dtype_code(g)
    R, C = g.shape
    d = g.device
    given = out is not None or workspace is not None or status is not None
    if out is None:
        out = _new((R, C), out_dtype or g.dtype, d, stream)
    else:
        _buffer(out, "out", out.dtype, R * C, d)
    odt = _dtype_code(out)
    need = _workspace_size("mxfp4_newton_schulz_workspace", R, C)
    workspace = _workspace(workspace, need, d, stream)
    st = None if status is None else _addr(_buffer(status, "status", torch.int32, 1, d))
    if given:
        in_place = out.data_ptr() == g.data_ptr() and out.dtype == g.dtype
        _apart((("out", out), ("workspace", _used(workspace, need)), ("status", status)),
               () if in_place else (g,))
    a, b, c = coeffs
    _call("mxfp4_newton_schulz", d, stream, g.data_ptr(), dt, R, C, steps, a, b, c, eps, scale,
          out.data_ptr(), odt, workspace.data_ptr(), workspace.numel(), st)
    return out


# The C names, for callers that prefer them.
mxfp4_gemv = gemv
mxfp4_newton_schulz = newton_schulz
mxfp4_layernorm = layernorm
mxfp4_layernorm_quantize = layernorm_quantize
mxfp4_layernorm_backward = layernorm_backward
mxfp4_quantize = quantize


def mxfp4_quantize_oas(x, axis=ROWS, rounding=RNE, seed=0, out=None, stream=None):
    return quantize(x, axis, rounding, seed, out, stream, oas=True)


mxfp4_dequantize = dequantize
mxfp4_double_quantize = double_quantize
mxfp4_rht_quantize = rht_quantize
mxfp4_osc_step = osc_step
mxfp4_osc_synthetic_update = osc_synthetic_update
mxfp4_qramp_step = qramp_step
mxfp4_qema_quantize = qema_quantize
mxfp4_scales_to_blocked = scales_to_blocked
mxfp4_gemm = gemm
mxfp4_gemm_quantize_a = gemm_quantize_a
mxfp4_status_string = status_string
