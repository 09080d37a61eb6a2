"""ctypes binding of libif4.so.

The functions named like the C entry points take torch tensors, check that
their dtypes and strides describe what the C call expects, and pass raw
device pointers, sizes and a CUDA stream: the one given, or the current stream
of the tensors' device, which need not be the current device.  Every step of
the IF4 path runs in the library's kernels; torch only owns memory and streams.
The helpers (``quantize``, ``dequantize``, ``linear_nvfp4`` ...) allocate
outputs with torch and call the entry points.  A helper that is given a stream
allocates its results and workspaces on it, as under torch.cuda.stream: they
share no memory with what the current stream may still hand out.

There is no fallback: if libif4.so is missing or a call fails, an exception
is raised.  What only the device can see is reported in err_flag alone, an int32
tensor that the caller zeroes and reads after the stream's work (DEV_* bits).
"""
import ctypes
import os

import torch

from . import build as _build

LIB_PATH = _build.LIB

IF4_OK = 0
TS_COMPUTE = 0
TS_GIVEN = 1
DEV_NONFINITE = 1
DEV_BAD_SCALE = 2
DEV_TIMEOUT = 4

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int


class IF4Error(RuntimeError):
    pass


def _load():
    if not os.path.exists(LIB_PATH):
        raise IF4Error(f"{LIB_PATH} is not built; run `python -m adaptive_block_scaled_b200.build`")
    lib = ctypes.CDLL(LIB_PATH)
    sig = {
        "if4_tensor_amax": [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp],
        "if4_tensor_scale": [_vp, _vp, _vp],
        "if4_quantize": [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _int, _vp, _vp],
        "nvfp4_quantize": [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _int, _vp, _vp],
        "nvint4_quantize": [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _int, _vp, _vp],
        "nvfp4_4over6_quantize": [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _int, _vp, _vp],
        "if4_dequantize": [_vp, _vp, _vp, _i64, _i64, _vp, _int, _i64, _vp],
        "if4_tensor_amax_rht": [_vp, _int, _i64, _i64, _i64, ctypes.c_uint32, _vp, _vp, _vp],
        "if4_quantize_rht": [_vp, _int, _i64, _i64, _i64, ctypes.c_uint32, _vp, _vp, _vp, _int,
                             _vp, _vp],
        "if4_quantize_fused": [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                               _vp],
        "if4_quantize_fused_rht": [_vp, _int, _i64, _i64, _i64, ctypes.c_uint32, _vp, _vp, _vp,
                                   _vp, _vp, _vp, _vp, _vp],
        "if4_quantize_fused_shared": [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _vp,
                                      _int, _vp, _vp],
        "if4_quantize_fused_rht_shared": [_vp, _int, _i64, _i64, _i64, ctypes.c_uint32, _vp, _vp,
                                          _vp, _vp, _vp, _vp, _int, _vp, _vp],
        "if4_quantize_fused_dequant": [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp,
                                       _vp, _vp, _vp, _vp],
        "if4_quantize_fused_dequant_shared": [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _vp,
                                              _vp, _vp, _vp, _int, _vp, _vp],
        "if4_decode_f16": [_vp, _vp, _i64, _i64, _vp, _vp],
        "if4_gemm_f16": [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp],
        "if4_linear_workspace_bytes": [_i64, _i64, _i64],
        "if4_linear": [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, ctypes.c_size_t,
                       _vp, _vp, _vp],
        "if4_linear_noalloc": [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp],
        "if4_linear_fused": [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _vp],
        "if4_linear_quantized": [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp,
                                 ctypes.c_size_t, _vp, _vp, _vp, _vp, _vp, _vp],
        "if4_quantize_t": [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _int, _vp, _vp],
        "nvfp4_quantize_t": [_vp, _int, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _vp, _int, _vp,
                             _vp],
        "if4_rms_norm_quantize": [_vp, _i64, _vp, _i64, _vp, _int, _int, _i64, _i64,
                                  ctypes.c_float, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
        "nvfp4_rms_norm_quantize": [_vp, _i64, _vp, _i64, _vp, _int, _int, _i64, _i64,
                                    ctypes.c_float, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp],
        "if4_rms_norm_backward_workspace_bytes": [_i64, _i64],
        "if4_rms_norm_backward": [_vp, _i64, _vp, _i64, _vp, _int, _vp, _vp, _i64, _int, _i64,
                                  _i64, _vp, _i64, _vp, _vp, ctypes.c_size_t, _vp],
        "nvfp4_linear_workspace_bytes": [_i64, _i64, _i64],
        "nvfp4_linear": [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, ctypes.c_size_t,
                         _vp, _int, _vp, _vp],
        "if6_quantize": [_vp, _int, _i64, _i64, _i64, _int, _vp, _vp, _vp, _int, _vp, _vp],
        "if3_quantize": [_vp, _int, _i64, _i64, _i64, _int, _vp, _vp, _vp, _int, _vp, _vp],
        "if6_dequantize": [_vp, _vp, _vp, _i64, _i64, _vp, _int, _i64, _vp],
        "if3_dequantize": [_vp, _vp, _vp, _i64, _i64, _vp, _int, _i64, _vp],
        "if4_status_str": [_int],
        "if4_version": [],
    }
    for name, args in sig.items():
        fn = getattr(lib, name, None)
        if fn is None:
            continue
        fn.argtypes = args
        fn.restype = _int
    lib.if4_status_str.restype = ctypes.c_char_p
    if hasattr(lib, "if4_linear_workspace_bytes"):
        lib.if4_linear_workspace_bytes.restype = ctypes.c_size_t
    for name in ("nvfp4_linear_workspace_bytes", "if4_rms_norm_backward_workspace_bytes"):
        if hasattr(lib, name):
            getattr(lib, name).restype = ctypes.c_size_t
    return lib


lib = _load()


def _check(rc: int, name: str):
    if rc != IF4_OK:
        raise IF4Error(f"{name}: {lib.if4_status_str(rc).decode()} (status {rc})")


# the handle of a device's current stream, without the Stream object that
# torch.cuda.current_stream() makes (0.1 against 3.1 us per call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda dev: torch.cuda.current_stream(dev).cuda_stream)


def _device(name, *tensors):
    """Index of the CUDA device that every given tensor lives on (None skipped)."""
    dev = -2
    for t in tensors:
        if t is not None:
            d = t.get_device()
            if d != dev:
                if d < 0:                       # -1: not a CUDA tensor
                    raise ValueError(f"{name}: every tensor must be on a CUDA device")
                if dev >= 0:
                    raise ValueError(f"{name}: tensors on cuda:{dev} and cuda:{d}")
                dev = d
    return dev


def _same_device(stream, dev):
    if stream.device_index != dev:
        raise ValueError(f"the stream belongs to cuda:{stream.device_index}, the tensors to cuda:{dev}")


def _under(stream, t):
    """torch.cuda.stream(stream), a stream of t's device."""
    _same_device(stream, t.get_device())
    return torch.cuda.stream(stream)


def _call(name, dev, stream, *args):
    """The C entry point `name` with args and the stream (the device's current
    one by default), with the tensors' device current."""
    fn = getattr(lib, name)
    if stream is None:
        raw = _raw_stream(dev)
    else:
        _same_device(stream, dev)
        raw = stream.cuda_stream
    if dev == torch.cuda.current_device():
        rc = fn(*args, raw)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, raw)
    if rc != IF4_OK:
        _check(rc, name)


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _rows(t, name, dtype=None, shape=None):
    """A 2-D tensor whose rows are contiguous and do not overlap: its row
    stride in elements."""
    if t.dim() != 2 or (shape is not None and t.shape != shape):
        raise ValueError(f"{name} must be 2-D" + ("" if shape is None else f" of {tuple(shape)}"))
    if dtype is not None and t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}")
    rows, cols = t.shape
    ld, step = t.stride()
    if (cols > 1 and step != 1) or (rows > 1 and ld < cols):
        raise ValueError(f"{name} must have contiguous rows that do not overlap")
    return ld if rows > 1 and cols > 0 else cols


def _matrix(t, name):
    """Rows, columns and row stride of a 2-D tensor with contiguous rows that do
    not overlap (an expanded tensor's rows do: its memory ends after the first)."""
    ld = _rows(t, name)
    return t.shape[0], t.shape[1], ld


def _dtype(t, name):
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name}: unsupported dtype {t.dtype}")
    return _DTYPES[t.dtype]


def _u8(t, name, shape):
    if t.dtype is not torch.uint8 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous uint8 tensor of shape {tuple(shape)}")


def _word(t, name, dtype):
    if t is not None and (t.dtype is not dtype or t.numel() < 1):
        raise ValueError(f"{name} must be a {dtype} device tensor")


def _words(err_flag, **floats):
    """float32 words and an int32 error word that a call reads or writes."""
    for n, t in floats.items():
        _word(t, n, torch.float32)
    _word(err_flag, "err_flag", torch.int32)


def _workspace(t):
    """Address and bytes of a workspace; (None, 0) for None."""
    if t is None:
        return None, 0
    if not t.is_contiguous():             # an expanded one has less memory than elements
        raise ValueError("workspace must be contiguous")
    return t.data_ptr(), t.numel() * t.element_size()


# ------------------------------------------------------- C entry points ---

def if4_tensor_amax(x, amax, err_flag=None, stream=None):
    name = "if4_tensor_amax"
    rows, cols, ld = _matrix(x, "x")
    _words(err_flag, amax=amax)
    _call(name, _device(name, x, amax, err_flag), stream, _ptr(x), _dtype(x, "x"), rows, cols, ld,
          _ptr(amax), _ptr(err_flag))


def if4_tensor_scale(amax, ts, stream=None):
    name = "if4_tensor_scale"
    _words(None, amax=amax, ts=ts)
    _call(name, _device(name, amax, ts), stream, _ptr(amax), _ptr(ts))


def _quantize_call(name, x, codes, scales, ts, ts_mode, err_flag, stream):
    rows, cols, ld = _matrix(x, "x")
    _u8(codes, "codes", (rows, cols // 2))
    _u8(scales, "scales", (rows, cols // 16))
    _words(err_flag, ts=ts)
    _call(name, _device(name, x, codes, scales, ts, err_flag), stream, _ptr(x), _dtype(x, "x"), rows,
          cols, ld, _ptr(codes), _ptr(scales), _ptr(ts), int(ts_mode), _ptr(err_flag))


def if4_quantize(x, codes, scales, ts, ts_mode=TS_COMPUTE, err_flag=None, stream=None):
    _quantize_call("if4_quantize", x, codes, scales, ts, ts_mode, err_flag, stream)


def nvfp4_quantize(x, codes, scales, ts, ts_mode=TS_COMPUTE, err_flag=None, stream=None):
    _quantize_call("nvfp4_quantize", x, codes, scales, ts, ts_mode, err_flag, stream)


def if4_tensor_amax_rht(x, signs, amax, err_flag=None, stream=None):
    name = "if4_tensor_amax_rht"
    rows, cols, ld = _matrix(x, "x")
    _words(err_flag, amax=amax)
    _call(name, _device(name, x, amax, err_flag), stream, _ptr(x), _dtype(x, "x"), rows, cols, ld,
          int(signs) & 0xFFFF, _ptr(amax), _ptr(err_flag))


def if4_quantize_rht(x, signs, codes, scales, ts, ts_mode=TS_COMPUTE, err_flag=None, stream=None):
    name = "if4_quantize_rht"
    rows, cols, ld = _matrix(x, "x")
    _u8(codes, "codes", (rows, cols // 2))
    _u8(scales, "scales", (rows, cols // 16))
    _words(err_flag, ts=ts)
    _call(name, _device(name, x, codes, scales, ts, err_flag), stream, _ptr(x), _dtype(x, "x"), rows,
          cols, ld, int(signs) & 0xFFFF, _ptr(codes), _ptr(scales), _ptr(ts), int(ts_mode),
          _ptr(err_flag))


def _fused_args(x, codes, scales, nv_codes, nv_scales, sync_words):
    rows, cols, ld = _matrix(x, "x")
    _u8(codes, "codes", (rows, cols // 2))
    _u8(scales, "scales", (rows, cols // 16))
    if (nv_codes is None) != (nv_scales is None):
        raise ValueError("nv_codes and nv_scales go together")
    if nv_codes is not None:
        _u8(nv_codes, "nv_codes", (rows, cols // 2))
        _u8(nv_scales, "nv_scales", (rows, cols // 16))
    if (sync_words.dtype != torch.int32 or sync_words.numel() < FUSED_SYNC_WORDS
            or not sync_words.is_contiguous()):
        raise ValueError(f"sync_words must be a contiguous int32 device tensor of at least "
                         f"{FUSED_SYNC_WORDS} elements")
    return rows, cols, ld


def _fused_call(name, x, signs, codes, scales, nv_codes, nv_scales, ts, sync_words, share, err_flag,
                stream):
    """name (or its transform form, with signs) on 1/share of the device, or the
    whole of it for share=None."""
    rows, cols, ld = _fused_args(x, codes, scales, nv_codes, nv_scales, sync_words)
    _words(err_flag, ts=ts)
    dev = _device(name, x, codes, scales, nv_codes, nv_scales, ts, sync_words, err_flag)
    _call(name, dev, stream, _ptr(x), _dtype(x, "x"), rows, cols, ld,
          *(() if signs is None else (int(signs) & 0xFFFF,)), _ptr(codes), _ptr(scales),
          _ptr(nv_codes), _ptr(nv_scales), _ptr(ts), _ptr(sync_words),
          *(() if share is None else (int(share),)), _ptr(err_flag))


def if4_quantize_fused_shared(x, codes, scales, nv_codes, nv_scales, ts, sync_words, share,
                              err_flag=None, stream=None, signs=None):
    """The single-launch quantizer (signs=None) or its transform form on
    1/share of the device's resident blocks (if4_quantize_fused_shared /
    if4_quantize_fused_rht_shared); outputs byte-identical to the plain
    call."""
    _fused_call("if4_quantize_fused_shared" if signs is None else "if4_quantize_fused_rht_shared", x,
                signs, codes, scales, nv_codes, nv_scales, ts, sync_words, share, err_flag, stream)


def if4_quantize_fused(x, codes, scales, nv_codes, nv_scales, ts, sync_words, err_flag=None,
                       stream=None, signs=None):
    """signs=None: the plain single-launch quantizer; an int: the same on the
    random-sign Hadamard transform of x (if4_quantize_fused_rht)."""
    _fused_call("if4_quantize_fused" if signs is None else "if4_quantize_fused_rht", x, signs, codes,
                scales, nv_codes, nv_scales, ts, sync_words, None, err_flag, stream)


def nvint4_quantize(x, codes, scales, ts, ts_mode=TS_COMPUTE, err_flag=None, stream=None):
    _quantize_call("nvint4_quantize", x, codes, scales, ts, ts_mode, err_flag, stream)


def nvfp4_4over6_quantize(x, codes, scales, ts, ts_mode=TS_COMPUTE, err_flag=None, stream=None):
    _quantize_call("nvfp4_4over6_quantize", x, codes, scales, ts, ts_mode, err_flag, stream)


def if4_dequantize(codes, scales, ts, y, stream=None):
    name = "if4_dequantize"
    rows, cols, ld = _matrix(y, "y")
    _u8(codes, "codes", (rows, cols // 2))
    _u8(scales, "scales", (rows, cols // 16))
    _word(ts, "ts", torch.float32)
    _call(name, _device(name, codes, scales, ts, y), stream, codes.data_ptr(), scales.data_ptr(),
          ts.data_ptr(), rows, cols, y.data_ptr(), _dtype(y, "y"), ld)


def if4_decode_f16(codes, scales, y, stream=None):
    name = "if4_decode_f16"
    rows, cols = y.shape
    if y.dtype != torch.float16 or not y.is_contiguous():
        raise ValueError("y must be a contiguous float16 tensor")
    _u8(codes, "codes", (rows, cols // 2))
    _u8(scales, "scales", (rows, cols // 16))
    _call(name, _device(name, codes, scales, y), stream, _ptr(codes), _ptr(scales), rows, cols,
          _ptr(y))


def if4_gemm_f16(a, b, a_ts, b_ts, c, err_flag, stream=None):
    name = "if4_gemm_f16"
    M, K = a.shape
    N = b.shape[0]
    for t, n in ((a, "a"), (b, "b")):
        if t.dtype != torch.float16 or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous float16 tensor")
    if b.shape[1] != K or tuple(c.shape) != (M, N) or c.dtype != torch.bfloat16:
        raise ValueError("shapes: a [M,K], b [N,K], c bf16 [M,N]")
    _words(err_flag, a_ts=a_ts, b_ts=b_ts)
    _call(name, _device(name, a, b, a_ts, b_ts, c, err_flag), stream, _ptr(a), _ptr(b), _ptr(a_ts),
          _ptr(b_ts), M, N, K, _ptr(c), _ptr(err_flag))


def if4_linear_workspace_bytes(M, N, K):
    return int(lib.if4_linear_workspace_bytes(int(M), int(N), int(K)))


def _linear_sizes(a_codes, a_scales, b_codes, b_scales, M, N, c):
    """K of IF4 operands [M, K] and [N, K]; c, if given, dense bf16."""
    K = a_codes.shape[1] * 2
    _u8(a_codes, "a_codes", (M, K // 2))
    _u8(a_scales, "a_scales", (M, K // 16))
    _u8(b_codes, "b_codes", (N, K // 2))
    _u8(b_scales, "b_scales", (N, K // 16))
    if c is not None and (c.dtype != torch.bfloat16 or not c.is_contiguous()):
        raise ValueError("c must be a contiguous bf16 tensor")
    return K


def if4_linear(a_codes, a_scales, a_ts, b_codes, b_scales, b_ts, workspace, c, err_flag,
               stream=None):
    name = "if4_linear"
    M, N = c.shape
    K = _linear_sizes(a_codes, a_scales, b_codes, b_scales, M, N, c)
    _words(err_flag, a_ts=a_ts, b_ts=b_ts)
    dev = _device(name, a_codes, a_scales, a_ts, b_codes, b_scales, b_ts, workspace, c, err_flag)
    _call(name, dev, stream, _ptr(a_codes), _ptr(a_scales), _ptr(a_ts), _ptr(b_codes), _ptr(b_scales),
          _ptr(b_ts), M, N, K, *_workspace(workspace), _ptr(c),
          _ptr(err_flag))


def if4_linear_fused(a_codes, a_scales, a_ts, b_codes, b_scales, b_ts, c, err_flag,
                     stream=None):
    """The IF4 x IF4 linear with the operand decode inside the GEMM (no
    workspace); the same C as if4_linear, bit for bit."""
    name = "if4_linear_fused"
    M, N = c.shape
    K = _linear_sizes(a_codes, a_scales, b_codes, b_scales, M, N, c)
    _words(err_flag, a_ts=a_ts, b_ts=b_ts)
    dev = _device(name, a_codes, a_scales, a_ts, b_codes, b_scales, b_ts, c, err_flag)
    _call(name, dev, stream, _ptr(a_codes), _ptr(a_scales), _ptr(a_ts), _ptr(b_codes), _ptr(b_scales),
          _ptr(b_ts), M, N, K, _ptr(c), _ptr(err_flag))


def if4_linear_noalloc(a_codes, a_scales, a_ts, b_codes, b_scales, b_ts, c, err_flag,
                       stream=None):
    """if4_linear with the library's fixed device scratch instead of a
    caller workspace (problems up to IF4_LINEAR_NOALLOC_MAX_BYTES)."""
    name = "if4_linear_noalloc"
    M, N = c.shape
    K = _linear_sizes(a_codes, a_scales, b_codes, b_scales, M, N, c)
    _words(err_flag, a_ts=a_ts, b_ts=b_ts)
    dev = _device(name, a_codes, a_scales, a_ts, b_codes, b_scales, b_ts, c, err_flag)
    _call(name, dev, stream, _ptr(a_codes), _ptr(a_scales), _ptr(a_ts), _ptr(b_codes), _ptr(b_scales),
          _ptr(b_ts), M, N, K, _ptr(c), _ptr(err_flag))


def if4_linear_quantized(a_codes, a_scales, a_ts, b_codes, b_scales, b_ts, workspace, c_codes,
                         c_scales, c_ts, c=None, err_flag=None, stream=None):
    name = "if4_linear_quantized"
    M, N = a_codes.shape[0], b_codes.shape[0]
    K = _linear_sizes(a_codes, a_scales, b_codes, b_scales, M, N, c)
    _u8(c_codes, "c_codes", (M, N // 2))
    _u8(c_scales, "c_scales", (M, N // 16))
    _words(err_flag, a_ts=a_ts, b_ts=b_ts, c_ts=c_ts)
    dev = _device(name, a_codes, a_scales, a_ts, b_codes, b_scales, b_ts, workspace, c_codes,
                  c_scales, c_ts, c, err_flag)
    _call(name, dev, stream, _ptr(a_codes), _ptr(a_scales), _ptr(a_ts), _ptr(b_codes), _ptr(b_scales),
          _ptr(b_ts), M, N, K, *_workspace(workspace), _ptr(c),
          _ptr(c_codes), _ptr(c_scales), _ptr(c_ts), _ptr(err_flag))


# ------------------------------------------------- the NVFP4 linear layer ---
#
# These calls sit between single-token kernels of a few microseconds, so each
# one checks its tensors with as few Python operations as will do (an expected
# argument passes in one comparison chain; what is wrong is worked out only
# when something is).

def _new(rows, cols, dtype, device):
    # empty_strided: 1.5 us per call against torch.empty's 2.5
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=device)


def _new1(n, dtype, device):
    return torch.empty_strided((n,), (1,), dtype=dtype, device=device)


def _dense(t, name, dtype, shape):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}")


def nvfp4_linear_workspace_bytes(M, N, K):
    return lib.nvfp4_linear_workspace_bytes(M, N, K)


def _operand(codes, scales, ts, name):
    """Rows and code bytes per row of an NVFP4 operand."""
    if codes.dim() != 2:
        raise ValueError(f"{name}_codes must be 2-D")
    rows, kb = codes.shape
    if (codes.dtype is not torch.uint8 or scales.dtype is not torch.uint8
            or scales.shape != (rows, kb // 8) or not codes.is_contiguous()
            or not scales.is_contiguous() or ts.dtype is not torch.float32 or ts.numel() < 1):
        _dense(codes, f"{name}_codes", torch.uint8, (rows, kb))
        _dense(scales, f"{name}_scales", torch.uint8, (rows, kb // 8))
        _word(ts, f"{name}_ts", torch.float32)
    return rows, kb


def _nvfp4_linear(a, b, ws, c, err_flag, stream):
    """Checks the operands (not c and ws) and calls nvfp4_linear."""
    (a_codes, a_scales, a_ts), (b_codes, b_scales, b_ts) = a, b
    dev = _device("nvfp4_linear", a_codes, a_scales, a_ts, b_codes, b_scales, b_ts, c, err_flag)
    M, kb = _operand(a_codes, a_scales, a_ts, "a")
    N, kb_b = _operand(b_codes, b_scales, b_ts, "b")
    if kb_b != kb:
        raise ValueError(f"a_codes has rows of {kb} bytes, b_codes of {kb_b}")
    _word(err_flag, "err_flag", torch.int32)
    wp, wn = (None, 0) if ws is None else _workspace(ws)
    _call("nvfp4_linear", dev, stream, a_codes.data_ptr(), a_scales.data_ptr(), a_ts.data_ptr(),
          b_codes.data_ptr(), b_scales.data_ptr(), b_ts.data_ptr(), M, N, 2 * kb, wp, wn,
          c.data_ptr(), _dtype(c, "c"), _ptr(err_flag))


def nvfp4_linear(a_codes, a_scales, a_ts, b_codes, b_scales, b_ts, workspace, c, err_flag,
                 stream=None):
    """C = A B^T of NVFP4 operands on the block-scaled tensor cores, into the
    dense c [M, N] (bf16, f16 or f32).  workspace: a uint8 tensor of
    nvfp4_linear_workspace_bytes, or None where that is 0."""
    _device("nvfp4_linear", a_codes, workspace, c)
    _dense(c, "c", c.dtype, (a_codes.shape[0], b_codes.shape[0]))
    _nvfp4_linear((a_codes, a_scales, a_ts), (b_codes, b_scales, b_ts), workspace, c, err_flag,
                  stream)


def linear_nvfp4(a, b, dtype=torch.bfloat16, err_flag=None, stream=None):
    """a, b: (codes, scales, ts) of NVFP4 operands [M, K] and [N, K].  Returns
    A B^T [M, N] of dtype.

    err_flag: an int32 tensor that the caller zeroes and reads.  Without one the
    device's errors are lost: operands with INT4 groups (DEV_BAD_SCALE), or a wait
    that ran out (DEV_TIMEOUT), then give an unspecified result in silence."""
    if stream is not None:
        with _under(stream, a[0]):
            return linear_nvfp4(a, b, dtype, err_flag)
    (M, kb), N, dev = a[0].shape, b[0].shape[0], a[0].device
    c = _new(M, N, dtype, dev)
    if err_flag is None:
        err_flag = _new1(1, torch.int32, dev)        # nobody reads it
    need = lib.nvfp4_linear_workspace_bytes(M, N, 2 * kb)
    ws = _new1(need, torch.uint8, dev) if need else None
    _nvfp4_linear(a, b, ws, c, err_flag, None)
    return c


def _entry(mode, name):
    if mode not in ("if4", "nvfp4"):
        raise ValueError(f'{name}: mode must be "if4" or "nvfp4"')
    return f"{mode}_{name}"


def _quantize_t(entry, x, codes, scales, codes_t, scales_t, ts, ts_mode, err_flag, stream):
    """Checks x, ts and err_flag (not the outputs' shapes) and calls entry."""
    ld = _rows(x, "x")
    dev = _device(entry, x, codes, scales, codes_t, scales_t, ts, err_flag)
    rows, cols = x.shape
    _word(ts, "ts", torch.float32)
    _word(err_flag, "err_flag", torch.int32)
    _call(entry, dev, stream, x.data_ptr(), _dtype(x, "x"), rows, cols, ld, _ptr(codes),
          _ptr(scales), codes_t.data_ptr(), scales_t.data_ptr(), ts.data_ptr(), ts_mode,
          _ptr(err_flag))


def _quantize_t_into(entry, x, codes, scales, codes_t, scales_t, ts, ts_mode, err_flag, stream):
    _rows(x, "x")
    rows, cols = x.shape
    if (codes is None) != (scales is None):
        raise ValueError("codes and scales go together")
    u8 = torch.uint8
    if codes is not None:
        _dense(codes, "codes", u8, (rows, cols // 2))
        _dense(scales, "scales", u8, (rows, cols // 16))
    _dense(codes_t, "codes_t", u8, (cols, rows // 2))
    _dense(scales_t, "scales_t", u8, (cols, rows // 16))
    _quantize_t(entry, x, codes, scales, codes_t, scales_t, ts, ts_mode, err_flag, stream)


def if4_quantize_t(x, codes, scales, codes_t, scales_t, ts, ts_mode=TS_COMPUTE, err_flag=None,
                   stream=None):
    """IF4 of x^T (codes_t [cols, rows/2], scales_t [cols, rows/16]) and, when
    codes and scales are given, of x as well."""
    _quantize_t_into("if4_quantize_t", x, codes, scales, codes_t, scales_t, ts, ts_mode, err_flag,
                     stream)


def nvfp4_quantize_t(x, codes, scales, codes_t, scales_t, ts, ts_mode=TS_COMPUTE, err_flag=None,
                     stream=None):
    """NVFP4 of x^T and, when codes and scales are given, of x as well."""
    _quantize_t_into("nvfp4_quantize_t", x, codes, scales, codes_t, scales_t, ts, ts_mode,
                     err_flag, stream)


def quantize_t(x, mode="if4", ts=None, with_rows=False, err_flag=None, stream=None):
    """Quantize a 2-D tensor along its rows with mode "if4" or "nvfp4".
    Returns (codes_t, scales_t, ts) of x^T or, with_rows, (codes, scales,
    codes_t, scales_t, ts) of x and of x^T under one tensor scale.  ts=None
    computes it; a float32 tensor is used as given."""
    if stream is not None:
        with _under(stream, x):
            return quantize_t(x, mode, ts, with_rows, err_flag)
    entry = _entry(mode, "quantize_t")
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    (rows, cols), dev, u8 = x.shape, x.device, torch.uint8
    codes_t, scales_t = _new(cols, rows // 2, u8, dev), _new(cols, rows // 16, u8, dev)
    codes = scales = None
    if with_rows:
        codes, scales = _new(rows, cols // 2, u8, dev), _new(rows, cols // 16, u8, dev)
    if ts is None:
        ts, ts_mode = _new1(1, torch.float32, dev), TS_COMPUTE
    else:
        ts_mode = TS_GIVEN
    _quantize_t(entry, x, codes, scales, codes_t, scales_t, ts, ts_mode, err_flag, None)
    if with_rows:
        return codes, scales, codes_t, scales_t, ts
    return codes_t, scales_t, ts


def _norm_weight(weight, cols, dtype):
    if weight.shape != (cols,) or not weight.is_contiguous():
        raise ValueError(f"weight must be a contiguous tensor of {cols} elements")
    if weight.dtype is not dtype and weight.dtype is not torch.float32:
        raise ValueError(f"weight must be {dtype} or float32")


def _rms_norm(entry, x, residual, weight, eps, h, rstd, codes, scales, ts, amax, err_flag, stream):
    """Checks the inputs (of the outputs only h) and calls entry."""
    ld, shape, dtype = _rows(x, "x"), x.shape, x.dtype
    dev = _device(entry, x, residual, weight, h, rstd, codes, scales, ts, amax, err_flag)
    rows, cols = shape
    ld_res = 0 if residual is None else _rows(residual, "residual", dtype, shape)
    ld_h = 0 if h is None else _rows(h, "h", dtype, shape)
    _norm_weight(weight, cols, dtype)
    _word(ts, "ts", torch.float32)
    _word(amax, "amax", torch.float32)
    _word(err_flag, "err_flag", torch.int32)
    _call(entry, dev, stream, x.data_ptr(), ld, _ptr(residual), ld_res, weight.data_ptr(),
          _dtype(weight, "weight"), _dtype(x, "x"), rows, cols, eps, _ptr(h), ld_h, _ptr(rstd),
          codes.data_ptr(), scales.data_ptr(), ts.data_ptr(), _ptr(amax), _ptr(err_flag))


def _rms_norm_into(entry, x, residual, weight, eps, h, rstd, codes, scales, ts, amax, err_flag,
                   stream):
    _rows(x, "x")
    rows, cols = x.shape
    _dense(codes, "codes", torch.uint8, (rows, cols // 2))
    _dense(scales, "scales", torch.uint8, (rows, cols // 16))
    if rstd is not None:
        _dense(rstd, "rstd", torch.float32, (rows,))
    _rms_norm(entry, x, residual, weight, eps, h, rstd, codes, scales, ts, amax, err_flag, stream)


def if4_rms_norm_quantize(x, residual, weight, eps, h, rstd, codes, scales, ts, amax=None,
                          err_flag=None, stream=None):
    """RMS norm of x (+ residual) quantized to IF4 under the given ts; residual,
    h, rstd and amax may be None."""
    _rms_norm_into("if4_rms_norm_quantize", x, residual, weight, eps, h, rstd, codes, scales, ts,
                   amax, err_flag, stream)


def nvfp4_rms_norm_quantize(x, residual, weight, eps, h, rstd, codes, scales, ts, amax=None,
                            err_flag=None, stream=None):
    """RMS norm of x (+ residual) quantized to NVFP4 under the given ts."""
    _rms_norm_into("nvfp4_rms_norm_quantize", x, residual, weight, eps, h, rstd, codes, scales, ts,
                   amax, err_flag, stream)


def rms_norm_quantize(x, weight, ts, residual=None, eps=1e-6, mode="if4", amax=None,
                      err_flag=None, stream=None):
    """RMS norm of x (+ residual), quantized with mode "if4" or "nvfp4" under
    the float32 tensor ts.  Returns (codes, scales, h, rstd): h = x + residual
    (x itself without a residual) and rstd [rows] are what rms_norm_backward
    takes.  amax: a float32 tensor raised to max |y|, for the next ts."""
    if stream is not None:
        with _under(stream, x):
            return rms_norm_quantize(x, weight, ts, residual, eps, mode, amax, err_flag)
    entry = _entry(mode, "rms_norm_quantize")
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    (rows, cols), dev = x.shape, x.device
    codes, scales = _new(rows, cols // 2, torch.uint8, dev), _new(rows, cols // 16, torch.uint8, dev)
    rstd = _new1(rows, torch.float32, dev)
    h = None if residual is None else _new(rows, cols, x.dtype, dev)
    _rms_norm(entry, x, residual, weight, eps, h, rstd, codes, scales, ts, amax, err_flag, None)
    return codes, scales, x if h is None else h, rstd


def if4_rms_norm_backward_workspace_bytes(rows, cols):
    return lib.if4_rms_norm_backward_workspace_bytes(rows, cols)


def if4_rms_norm_backward(dy, h, weight, rstd, dres, dx, dweight, workspace, stream=None):
    """Gradient of the norm into dx (x's type) and dweight (float32 [cols])."""
    name = "if4_rms_norm_backward"
    dev = _device(name, dy, h, weight, rstd, dres, dx, dweight, workspace)
    ld_h, shape, dtype = _rows(h, "h"), h.shape, h.dtype
    rows, cols = shape
    ld_dy, ld_dx = _rows(dy, "dy", dtype, shape), _rows(dx, "dx", dtype, shape)
    ld_dres = 0 if dres is None else _rows(dres, "dres", dtype, shape)
    _norm_weight(weight, cols, dtype)
    _dense(rstd, "rstd", torch.float32, (rows,))
    _dense(dweight, "dweight", torch.float32, (cols,))
    wp, wn = _workspace(workspace)
    _call(name, dev, stream, dy.data_ptr(), ld_dy, h.data_ptr(), ld_h, weight.data_ptr(),
          _dtype(weight, "weight"), rstd.data_ptr(), _ptr(dres), ld_dres, _dtype(h, "h"), rows, cols,
          dx.data_ptr(), ld_dx, dweight.data_ptr(), wp, wn)


def rms_norm_backward(dy, h, weight, rstd, dres=None, stream=None):
    """Gradient of rms_norm_quantize (straight through the quantizer) from dy,
    the gradient of the norm's output, and dres, that of h past the norm.
    Returns (dx, dweight): dx for x and the residual alike, dweight float32."""
    if stream is not None:
        with _under(stream, dy):
            return rms_norm_backward(dy, h, weight, rstd, dres)
    (rows, cols), dev = h.shape, h.device
    dx, dweight = _new(rows, cols, h.dtype, dev), _new1(cols, torch.float32, dev)
    need = lib.if4_rms_norm_backward_workspace_bytes(rows, cols)
    ws = _new1(need, torch.uint8, dev) if need else None
    if4_rms_norm_backward(dy, h, weight, rstd, dres, dx, dweight, ws)
    return dx, dweight


# ------------------------------------------------------- IF6 and IF3 ---

W_ADAPTIVE, W_FP_ONLY, W_INT_ONLY = 0, 1, 2


def _width_names(bits):
    if bits == 6:
        return "if6_quantize", "if6_dequantize"
    if bits == 3:
        return "if3_quantize", "if3_dequantize"
    raise ValueError("bits must be 6 or 3")


def ifw_quantize(x, bits, mode, codes, scales, ts, ts_mode=TS_COMPUTE, err_flag=None,
                 stream=None):
    """if6_quantize / if3_quantize: codes uint8 [rows, cols*bits/8]."""
    name, _ = _width_names(bits)
    rows, cols, ld = _matrix(x, "x")
    _u8(codes, "codes", (rows, cols * bits // 8))
    _u8(scales, "scales", (rows, cols // 16))
    _words(err_flag, ts=ts)
    _call(name, _device(name, x, codes, scales, ts, err_flag), stream, _ptr(x), _dtype(x, "x"), rows,
          cols, ld, int(mode), _ptr(codes), _ptr(scales), _ptr(ts), int(ts_mode), _ptr(err_flag))


def ifw_dequantize(codes, scales, ts, bits, y, stream=None):
    """if6_dequantize / if3_dequantize into y [rows, cols] (f32, bf16 or f16)."""
    _, name = _width_names(bits)
    rows, cols, ld = _matrix(y, "y")
    _u8(codes, "codes", (rows, cols * bits // 8))
    _u8(scales, "scales", (rows, cols // 16))
    _word(ts, "ts", torch.float32)
    _call(name, _device(name, codes, scales, ts, y), stream, _ptr(codes), _ptr(scales), _ptr(ts),
          rows, cols, _ptr(y), _dtype(y, "y"), ld)


def quantize_w(x, bits, mode=W_ADAPTIVE, ts=None, err_flag=None, stream=None):
    """IF6 (bits=6) or IF3 (bits=3) of a 2-D tensor, or the FP-only / INT-only
    candidate (mode).  Returns (codes, scales, ts); ts=None computes it."""
    if stream is not None:
        with _under(stream, x):
            return quantize_w(x, bits, mode, ts, err_flag)
    rows, cols, _ = _matrix(x, "x")
    dev = x.device
    codes = torch.empty((rows, cols * bits // 8), dtype=torch.uint8, device=dev)
    scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=dev)
    if ts is None:
        ts_t, ts_mode = torch.empty(1, dtype=torch.float32, device=dev), TS_COMPUTE
    else:
        ts_t, ts_mode = ts, TS_GIVEN
    ifw_quantize(x, bits, mode, codes, scales, ts_t, ts_mode, err_flag)
    return codes, scales, ts_t


def dequantize_w(codes, scales, ts, bits, dtype=torch.bfloat16, stream=None):
    if stream is not None:
        with _under(stream, codes):
            return dequantize_w(codes, scales, ts, bits, dtype)
    rows, cols = scales.shape[0], scales.shape[1] * 16
    y = torch.empty((rows, cols), dtype=dtype, device=codes.device)
    ifw_dequantize(codes, scales, ts, bits, y)
    return y


LINEAR_NOALLOC_MAX_BYTES = 32 * 1024 * 1024
FUSED_SYNC_WORDS = 64


# ---------------------------------------------------- allocating helpers ---

def quantize(x, mode="if4", ts=None, err_flag=None, stream=None):
    """Quantize a 2-D tensor on its device with mode "if4", "nvfp4", "nvint4"
    or "4over6".  Returns (codes, scales, ts).  ts=None computes the tensor
    scale; a float32 tensor is used as given."""
    if stream is not None:
        with _under(stream, x):
            return quantize(x, mode, ts, err_flag)
    rows, cols, _ = _matrix(x, "x")
    dev = x.device
    codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=dev)
    if ts is None:
        ts_t, ts_mode = torch.empty(1, dtype=torch.float32, device=dev), TS_COMPUTE
    else:
        ts_t, ts_mode = ts, TS_GIVEN
    fn = {"if4": if4_quantize, "nvfp4": nvfp4_quantize, "nvint4": nvint4_quantize,
          "4over6": nvfp4_4over6_quantize}[mode]
    fn(x, codes, scales, ts_t, ts_mode, err_flag)
    return codes, scales, ts_t


def quantize_rht(x, signs, ts=None, err_flag=None, stream=None):
    """Random-sign Hadamard transform + IF4 quantize.  Returns (codes, scales, ts)."""
    if stream is not None:
        with _under(stream, x):
            return quantize_rht(x, signs, ts, err_flag)
    rows, cols, _ = _matrix(x, "x")
    dev = x.device
    codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=dev)
    if ts is None:
        ts_t, ts_mode = torch.empty(1, dtype=torch.float32, device=dev), TS_COMPUTE
    else:
        ts_t, ts_mode = ts, TS_GIVEN
    if4_quantize_rht(x, signs, codes, scales, ts_t, ts_mode, err_flag)
    return codes, scales, ts_t


def _fused_dequant_call(name, x, codes, scales, nv_codes, nv_scales, ts, sync_words, y, share,
                        err_flag, stream):
    rows, cols, ld = _fused_dequant_args(x, codes, scales, nv_codes, nv_scales, sync_words, y)
    _words(err_flag, ts=ts)
    dev = _device(name, x, codes, scales, nv_codes, nv_scales, ts, sync_words, y, err_flag)
    _call(name, dev, stream, _ptr(x), _dtype(x, "x"), rows, cols, ld, _ptr(codes), _ptr(scales),
          _ptr(nv_codes), _ptr(nv_scales), _ptr(ts), _ptr(sync_words), _ptr(y),
          *(() if share is None else (int(share),)), _ptr(err_flag))


def if4_quantize_fused_dequant(x, codes, scales, nv_codes, nv_scales, ts, sync_words, y,
                               err_flag=None, stream=None):
    """The single launch that also writes y, the bf16 decode of its IF4 codes
    (dense, 32-byte aligned)."""
    _fused_dequant_call("if4_quantize_fused_dequant", x, codes, scales, nv_codes, nv_scales, ts,
                        sync_words, y, None, err_flag, stream)


def if4_quantize_fused_dequant_shared(x, codes, scales, nv_codes, nv_scales, ts, sync_words, y,
                                      share, err_flag=None, stream=None):
    """The same launch on 1/share of the device's resident blocks, for
    `share` calls at once on different streams (each with its own
    sync_words); outputs byte-identical to if4_quantize_fused_dequant."""
    _fused_dequant_call("if4_quantize_fused_dequant_shared", x, codes, scales, nv_codes, nv_scales,
                        ts, sync_words, y, share, err_flag, stream)


def _fused_dequant_args(x, codes, scales, nv_codes, nv_scales, sync_words, y):
    rows, cols, ld = _fused_args(x, codes, scales, nv_codes, nv_scales, sync_words)
    if y.dtype != torch.bfloat16 or tuple(y.shape) != (rows, cols) or not y.is_contiguous():
        raise ValueError("y must be a dense bf16 tensor of the shape of x")
    return rows, cols, ld


def quantize_fused_dequant(x, with_nvfp4=True, sync_words=None, err_flag=None, stream=None):
    """The quantize-then-dequantize round trip in one launch.  Returns
    (codes, scales, ts, y) or (codes, scales, ts, nv_codes, nv_scales, y)."""
    if stream is not None:
        with _under(stream, x):
            return quantize_fused_dequant(x, with_nvfp4, sync_words, err_flag)
    rows, cols, _ = _matrix(x, "x")
    dev = x.device
    codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=dev)
    nv_codes = torch.empty_like(codes) if with_nvfp4 else None
    nv_scales = torch.empty_like(scales) if with_nvfp4 else None
    ts = torch.empty(1, dtype=torch.float32, device=dev)
    y = torch.empty((rows, cols), dtype=torch.bfloat16, device=dev)
    if sync_words is None:
        sync_words = torch.zeros(FUSED_SYNC_WORDS, dtype=torch.int32, device=dev)
    if4_quantize_fused_dequant(x, codes, scales, nv_codes, nv_scales, ts, sync_words, y, err_flag)
    if with_nvfp4:
        return codes, scales, ts, nv_codes, nv_scales, y
    return codes, scales, ts, y


def quantize_fused(x, with_nvfp4=True, sync_words=None, err_flag=None, stream=None, signs=None):
    """amax, tensor scale, IF4 quantize (and NVFP4) in one launch, of x or,
    with signs, of its random-sign Hadamard transform.  Returns (codes,
    scales, ts) or (codes, scales, ts, nv_codes, nv_scales)."""
    if stream is not None:
        with _under(stream, x):
            return quantize_fused(x, with_nvfp4, sync_words, err_flag, signs=signs)
    rows, cols, _ = _matrix(x, "x")
    dev = x.device
    codes = torch.empty((rows, cols // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((rows, cols // 16), dtype=torch.uint8, device=dev)
    nv_codes = torch.empty_like(codes) if with_nvfp4 else None
    nv_scales = torch.empty_like(scales) if with_nvfp4 else None
    ts = torch.empty(1, dtype=torch.float32, device=dev)
    if sync_words is None:
        sync_words = torch.zeros(FUSED_SYNC_WORDS, dtype=torch.int32, device=dev)
    if4_quantize_fused(x, codes, scales, nv_codes, nv_scales, ts, sync_words, err_flag, None, signs)
    return (codes, scales, ts, nv_codes, nv_scales) if with_nvfp4 else (codes, scales, ts)


def dequantize(codes, scales, ts, dtype=torch.bfloat16, stream=None):
    if stream is not None:
        with _under(stream, codes):
            return dequantize(codes, scales, ts, dtype)
    rows, cols = codes.shape[0], codes.shape[1] * 2
    y = _new(rows, cols, dtype, codes.device)
    if4_dequantize(codes, scales, ts, y)
    return y


def decode_f16(codes, scales, stream=None):
    if stream is not None:
        with _under(stream, codes):
            return decode_f16(codes, scales)
    rows, cols = codes.shape[0], codes.shape[1] * 2
    y = torch.empty((rows, cols), dtype=torch.float16, device=codes.device)
    if4_decode_f16(codes, scales, y)
    return y
