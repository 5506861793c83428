"""ctypes binding of libwq (argument marshalling only).

Each function has the name and argument order of the C entry point declared
in include/wq.h.  Buffers are torch tensors on the GPU (or raw device
addresses as ints, or None for a nullable pointer); sizes are ints; `stream`
defaults to torch's current stream on the current device.  Every step of the
computation runs in the HIP library; a non-OK status raises WQError.

The library is loaded from this package directory (built in-tree by
``weight_only_quantized_wq_amd.build``).  Loading fails loudly if it is
missing: there is no fallback implementation.
"""

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libwq.so")

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_I32 = ctypes.c_int32

_SIGNATURES = {
    "wq_quantize_int8": [_P, _I64, _I64, _P, _P, _P],
    "wq_quantize_int4g32": [_P, _I64, _I64, _P, _P, _P],
    "wq_quantize_int4": [_P, _I64, _I64, _I32, _P, _P, _P],
    "wq_gemv_bf16": [_P, _P, _I64, _I64, _P, _P, _P],
    "wq_gemv_int8": [_P, _P, _P, _I64, _I64, _P, _P, _P],
    "wq_gemv_int4g32": [_P, _P, _P, _I64, _I64, _P, _P, _P],
    "wq_gemv_int4": [_P, _P, _P, _I64, _I64, _I32, _P, _P, _P],
    "wq_gemm_smallM": [_P, _I64, _P, _P, _I64, _I64, _P, _P, _P],
    "wq_gemm_smallM_int8": [_P, _I64, _P, _P, _I64, _I64, _P, _P, _P],
    "wq_gemm_smallM_int4": [_P, _I64, _P, _P, _I64, _I64, _I32, _P, _P, _P],
    "wq_quantize_mxfp4": [_P, _P, _I64, _I64, _P, _P, _P],
    "wq_dequantize_mxfp4": [_P, _P, _I64, _I64, _P, _P, _P],
    "moe_top2_gemv": [_P, _P, _I64, _P, _P, _P, _P, _I64, _I64, _P, _P, _P, _P, _P, _P],
    "moe_top2_gemv_noalloc": [_P, _P, _I64, _P, _P, _P, _P, _I64, _I64, _P, _P, _P, _P, _P],
}

WQ_FORMAT = {"bf16": 1, "int8": 2, "int4g32": 3, "int4g64": 4, "int4g128": 5, "int4g256": 6, "int4pc": 7,
             "mxfp4": 8}


class wq_matrix(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("w", ctypes.c_void_p), ("aux", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("k", ctypes.c_int64), ("y_f32", ctypes.c_void_p), ("y_bf16", ctypes.c_void_p)]


class wq_step_plan(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("m", ctypes.c_int32), ("count", ctypes.c_int32),
                ("groups", ctypes.c_int32), ("total_batches", ctypes.c_int64), ("workspace", ctypes.c_void_p)]


class wq_moe_layer(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("logits", ctypes.c_void_p), ("w13", ctypes.c_void_p),
                ("s13", ctypes.c_void_p), ("w2", ctypes.c_void_p), ("s2", ctypes.c_void_p),
                ("work", ctypes.c_void_p), ("y_f32", ctypes.c_void_p), ("y_bf16", ctypes.c_void_p),
                ("sel", ctypes.c_void_p), ("gates", ctypes.c_void_p)]


class wq_moe_plan(ctypes.Structure):
    _fields_ = [("dim", ctypes.c_int64), ("f", ctypes.c_int64), ("e", ctypes.c_int32), ("count", ctypes.c_int32),
                ("grid13", ctypes.c_int32), ("grid2", ctypes.c_int32), ("workspace", ctypes.c_void_p)]


class wq_kv_cache(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("pages", _I64), ("page_size", _I64), ("page_stride", _I64),
                ("token_stride", _I64), ("head_stride", _I64), ("table", _P), ("table_width", _I64),
                ("table_stride", _I64), ("kv_heads", _I32), ("head_dim", _I32)]


class wq_batch(ctypes.Structure):
    _fields_ = [("starts", _P), ("lengths", _P), ("tokens", _I64), ("requests", _I64)]


class wq_qkv_rope(ctypes.Structure):
    _fields_ = [("cache", wq_kv_cache), ("batch", wq_batch), ("qkv_f32", _P), ("qkv_bf16", _P), ("qkv_stride", _I64),
                ("q", _P), ("q_stride", _I64), ("positions", _P), ("q_norm", _P), ("k_norm", _P), ("freq", _P),
                ("eps", ctypes.c_float), ("rot_scale", ctypes.c_float), ("rot_dim", _I32), ("interleaved", _I32),
                ("heads", _I32)]


class wq_tree_attention(ctypes.Structure):
    _fields_ = [("cache", wq_kv_cache), ("batch", wq_batch), ("q", _P), ("q_stride", _I64), ("y", _P),
                ("y_stride", _I64), ("tree", _P), ("scale", ctypes.c_float), ("heads", _I32), ("max_tokens", _I32)]


class wq_kv_accept(ctypes.Structure):
    _fields_ = [("cache", wq_kv_cache), ("layers", _I64), ("layer_stride", _I64), ("requests", _I64), ("lengths", _P),
                ("path", _P), ("path_width", _I64), ("path_stride", _I64), ("accepted", _P)]


class wq_lora(ctypes.Structure):
    _fields_ = [("x", _P), ("x_stride", _I64), ("base", _P), ("base_stride", _I64), ("y_f32", _P), ("y_bf16", _P),
                ("y_stride", _I64), ("a", _P), ("b", _P), ("adapter", _P), ("ranks", _P), ("scale", _P),
                ("tokens", _I64), ("k", _I64), ("n", _I64), ("adapters", _I64), ("rank", _I32)]


class wq_gemm_mxfp4(ctypes.Structure):
    _fields_ = [("x", _P), ("x_stride", _I64), ("xq", _P), ("x_scale", _P), ("q", _P), ("scale", _P), ("y_f32", _P),
                ("y_bf16", _P), ("y_stride", _I64), ("m", _I64), ("n", _I64), ("k", _I64)]


class wq_moe_ffn(ctypes.Structure):
    _fields_ = [("x", _P), ("x_stride", _I64), ("router", _P), ("logits", _P), ("w13", _P), ("s13", _P), ("w2", _P),
                ("s2", _P), ("y_f32", _P), ("y_bf16", _P), ("y_stride", _I64), ("sel", _P), ("gates", _P),
                ("tokens", _I64), ("dim", _I64), ("f", _I64), ("e", _I64), ("top", _I32), ("format", _I32),
                ("renormalize", _I32)]


class wq_block_norm(ctypes.Structure):
    _fields_ = [("h_f32", _P), ("h_bf16", _P), ("h_stride", _I64), ("out_f32", _P), ("out_bf16", _P),
                ("out_stride", _I64), ("f_f32", _P), ("f_bf16", _P), ("f_stride", _I64), ("f_norm", _P), ("gate", _P),
                ("gate_stride", _I64), ("norm", _P), ("u", _P), ("u_stride", _I64), ("q", _P), ("q_scale", _P),
                ("rows", _I64), ("dim", _I64), ("scale", ctypes.c_float), ("eps", ctypes.c_float), ("gate_kind", _I32)]


# Plans: ctypes instances take further attributes, and `keep` holds the tensors
# a plan's addresses point into for as long as the plan lives.
class wq_qkv_rope_plan(ctypes.Structure):
    _fields_ = [("made", _I64), ("device", _I32), ("reserved", _I32), ("a", wq_qkv_rope)]


class wq_tree_attention_plan(ctypes.Structure):
    _fields_ = [("made", _I64), ("device", _I32), ("variant", _I32), ("workspace", _P), ("a", wq_tree_attention)]


class wq_kv_accept_plan(ctypes.Structure):
    _fields_ = [("made", _I64), ("device", _I32), ("reserved", _I32), ("a", wq_kv_accept)]


class wq_lora_plan(ctypes.Structure):
    _fields_ = [("made", _I64), ("device", _I32), ("tiles", _I32), ("splits", _I32), ("reserved", _I32),
                ("workspace", _P), ("a", wq_lora)]


class wq_gemm_mxfp4_plan(ctypes.Structure):
    _fields_ = [("made", _I64), ("device", _I32), ("reserved", _I32), ("workspace", _P), ("a", wq_gemm_mxfp4)]


class wq_moe_ffn_plan(ctypes.Structure):
    _fields_ = [("made", _I64), ("device", _I32), ("reserved", _I32), ("workspace", _P), ("a", wq_moe_ffn)]


class wq_block_norm_plan(ctypes.Structure):
    _fields_ = [("made", _I64), ("device", _I32), ("reserved", _I32), ("a", wq_block_norm)]


WQ_GATE = {"plain": 0, "sigmoid": 1, "silu": 2}

WQ_ROPE = {"plain": 0, "linear": 1, "bands": 2, "ramp": 3}

WQ_STATUS = {0: "WQ_OK", 1: "WQ_ERR_NULL", 2: "WQ_ERR_SHAPE", 3: "WQ_ERR_ALIGN", 4: "WQ_ERR_DEVICE",
             5: "WQ_ERR_LAUNCH"}


class WQError(RuntimeError):
    def __init__(self, fn, status, detail):
        self.fn = fn
        self.status = status
        self.detail = detail
        super().__init__(f"{fn}: {WQ_STATUS.get(status, status)}: {detail}")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"libwq.so not found at {LIB_PATH}; build it first with "
            "`python -m weight_only_quantized_wq_amd.build` (hipcc, gfx950)")
    lib = ctypes.CDLL(LIB_PATH)
    for name, args in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.wq_decode_step_workspace_bytes.argtypes = [ctypes.c_int32]
    lib.wq_decode_step_workspace_bytes.restype = ctypes.c_int64
    lib.wq_decode_step_prepare.argtypes = [ctypes.c_int32, ctypes.c_int32, ctypes.POINTER(wq_matrix), ctypes.c_int32,
                                           _P, _I64, ctypes.POINTER(wq_step_plan)]
    lib.wq_decode_step_prepare.restype = ctypes.c_int
    lib.wq_decode_step_run.argtypes = [ctypes.POINTER(wq_step_plan), _P]
    lib.wq_decode_step_run.restype = ctypes.c_int
    lib.wq_moe_step_workspace_bytes.argtypes = [ctypes.c_int32]
    lib.wq_moe_step_workspace_bytes.restype = ctypes.c_int64
    lib.wq_moe_step_prepare.argtypes = [_I64, _I64, _I64, ctypes.POINTER(wq_moe_layer), ctypes.c_int32, _P, _I64,
                                        ctypes.POINTER(wq_moe_plan)]
    lib.wq_moe_step_prepare.restype = ctypes.c_int
    lib.wq_moe_step_run.argtypes = [ctypes.POINTER(wq_moe_plan), _P]
    lib.wq_moe_step_run.restype = ctypes.c_int
    lib.wq_rope_frequencies.argtypes = [_I32, _I32] + [ctypes.c_double] * 5 + [ctypes.POINTER(ctypes.c_float)] * 2
    lib.wq_tree_attention_workspace_bytes.argtypes = [_I64] + [_I32] * 4
    lib.wq_tree_attention_workspace_bytes.restype = _I64
    lib.wq_lora_workspace_bytes.argtypes = [_I64, _I64, _I64, _I32]
    lib.wq_lora_workspace_bytes.restype = _I64
    lib.wq_gemm_mxfp4_workspace_bytes.argtypes = [_I64] * 3
    lib.wq_gemm_mxfp4_workspace_bytes.restype = _I64
    lib.wq_moe_ffn_workspace_bytes.argtypes = [_I64] * 4 + [_I32]
    lib.wq_moe_ffn_workspace_bytes.restype = _I64
    # prepare and run are called with ctypes.byref of the structures above
    lib.wq_qkv_rope_prepare.argtypes = [_P, _P]
    lib.wq_qkv_rope_run.argtypes = [_P, _P]
    lib.wq_tree_attention_prepare.argtypes = [_P, _P, _I64, _P]
    lib.wq_tree_attention_run.argtypes = [_P, _P]
    lib.wq_kv_accept_prepare.argtypes = [_P, _P]
    lib.wq_kv_accept_run.argtypes = [_P, _P]
    lib.wq_lora_prepare.argtypes = [_P, _P, _I64, _P]
    lib.wq_lora_run.argtypes = [_P, _P]
    lib.wq_gemm_mxfp4_prepare.argtypes = [_P, _P, _I64, _P]
    lib.wq_gemm_mxfp4_run.argtypes = [_P, _P]
    lib.wq_moe_ffn_prepare.argtypes = [_P, _P, _I64, _P]
    lib.wq_moe_ffn_run.argtypes = [_P, _P]
    lib.wq_block_norm_prepare.argtypes = [_P, _P]
    lib.wq_block_norm_run.argtypes = [_P, _P]
    lib.wq_status_string.argtypes = [ctypes.c_int]
    lib.wq_status_string.restype = ctypes.c_char_p
    lib.wq_last_error.argtypes = []
    lib.wq_last_error.restype = ctypes.c_char_p
    return lib


lib = _load()


class _HostBuffer:
    """Stand-in returned by _ptr for a tensor that is not in device memory;
    _call (and the plan builders) refuse it after every buffer's extent has
    been checked."""


def _ptr(t, nbytes=None, what="buffer"):
    """Device address of a tensor (or None / int passthrough).

    With `nbytes`, a tensor must hold at least that many bytes (the extent the
    C call will read or write for the sizes it is given); a shorter one raises
    ValueError before any call, since the kernels would access memory past
    it.  Raw integer addresses are passed through unchecked.  A tensor that is
    not on the GPU yields a _HostBuffer, which the call refuses once all
    arguments have been checked."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if nbytes is not None and nbytes > 0:
        have = t.numel() * t.element_size()
        if have < nbytes:
            raise ValueError(f"libwq: {what} holds {have} bytes; the sizes given need {nbytes}")
    if not getattr(t, "is_cuda", False):
        return _HostBuffer()
    if not t.is_contiguous():
        raise ValueError(f"libwq: {what} must be contiguous")
    return t.data_ptr()


def _refuse_host(args):
    if any(isinstance(a, _HostBuffer) for a in args):
        raise ValueError("libwq buffers must be GPU tensors (device memory)")


def _nonneg(*v):
    """True when every size is a non-negative int (else the C call reports the error)."""
    return all(isinstance(a, int) and a >= 0 for a in v)


def _int4_sz_bytes(n, k, group):
    """Bytes of the (scale, zero) words of an int4 matrix with groups of `group` (0 if undefined)."""
    if not _nonneg(n, k, group) or group == 0 or k % group:
        return 0
    return n * (k // group) * 4


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _call(name, *args):
    _refuse_host(args)
    rc = getattr(lib, name)(*args)
    if rc != 0:
        raise WQError(name, rc, lib.wq_last_error().decode(errors="replace"))


def status_string(status):
    return lib.wq_status_string(int(status)).decode()


def last_error():
    return lib.wq_last_error().decode(errors="replace")


def wq_quantize_int8(w, n, k, q, scale, stream=None):
    ok = _nonneg(n, k)
    _call("wq_quantize_int8", _ptr(w, ok and 4 * n * k, "w"), n, k, _ptr(q, ok and n * k, "q"),
          _ptr(scale, ok and 2 * n, "scale"), _stream(stream))


def wq_quantize_int4g32(w, n, k, qpacked, sz, stream=None):
    ok = _nonneg(n, k)
    _call("wq_quantize_int4g32", _ptr(w, ok and 4 * n * k, "w"), n, k, _ptr(qpacked, ok and n * k // 2, "qpacked"),
          _ptr(sz, _int4_sz_bytes(n, k, 32), "sz"), _stream(stream))


def wq_quantize_int4(w, n, k, group, qpacked, sz, stream=None):
    ok = _nonneg(n, k)
    _call("wq_quantize_int4", _ptr(w, ok and 4 * n * k, "w"), n, k, group, _ptr(qpacked, ok and n * k // 2, "qpacked"),
          _ptr(sz, _int4_sz_bytes(n, k, group), "sz"), _stream(stream))


def wq_gemv_bf16(x, w, n, k, y_f32=None, y_bf16=None, stream=None):
    ok = _nonneg(n, k)
    _call("wq_gemv_bf16", _ptr(x, ok and 2 * k, "x"), _ptr(w, ok and 2 * n * k, "w"), n, k,
          _ptr(y_f32, ok and 4 * n, "y_f32"), _ptr(y_bf16, ok and 2 * n, "y_bf16"), _stream(stream))


def wq_gemv_int8(x, q, scale, n, k, y_f32=None, y_bf16=None, stream=None):
    ok = _nonneg(n, k)
    _call("wq_gemv_int8", _ptr(x, ok and 2 * k, "x"), _ptr(q, ok and n * k, "q"), _ptr(scale, ok and 2 * n, "scale"),
          n, k, _ptr(y_f32, ok and 4 * n, "y_f32"), _ptr(y_bf16, ok and 2 * n, "y_bf16"), _stream(stream))


def wq_gemv_int4g32(x, qpacked, sz, n, k, y_f32=None, y_bf16=None, stream=None):
    ok = _nonneg(n, k)
    _call("wq_gemv_int4g32", _ptr(x, ok and 2 * k, "x"), _ptr(qpacked, ok and n * k // 2, "qpacked"),
          _ptr(sz, _int4_sz_bytes(n, k, 32), "sz"), n, k, _ptr(y_f32, ok and 4 * n, "y_f32"),
          _ptr(y_bf16, ok and 2 * n, "y_bf16"), _stream(stream))


def wq_gemv_int4(x, qpacked, sz, n, k, group, y_f32=None, y_bf16=None, stream=None):
    ok = _nonneg(n, k)
    _call("wq_gemv_int4", _ptr(x, ok and 2 * k, "x"), _ptr(qpacked, ok and n * k // 2, "qpacked"),
          _ptr(sz, _int4_sz_bytes(n, k, group), "sz"), n, k, group, _ptr(y_f32, ok and 4 * n, "y_f32"),
          _ptr(y_bf16, ok and 2 * n, "y_bf16"), _stream(stream))


def wq_gemm_smallM(x, m, qpacked, sz, n, k, y_f32=None, y_bf16=None, stream=None):
    ok = _nonneg(m, n, k)
    _call("wq_gemm_smallM", _ptr(x, ok and 2 * m * k, "x"), m, _ptr(qpacked, ok and n * k // 2, "qpacked"),
          _ptr(sz, _int4_sz_bytes(n, k, 32), "sz"), n, k, _ptr(y_f32, ok and 4 * m * n, "y_f32"),
          _ptr(y_bf16, ok and 2 * m * n, "y_bf16"), _stream(stream))


def wq_gemm_smallM_int4(x, m, qpacked, sz, n, k, group, y_f32=None, y_bf16=None, stream=None):
    """m token rows x [m, k] through int4 weights with groups of `group` inputs -> y [m, n]."""
    ok = _nonneg(m, n, k)
    _call("wq_gemm_smallM_int4", _ptr(x, ok and 2 * m * k, "x"), m, _ptr(qpacked, ok and n * k // 2, "qpacked"),
          _ptr(sz, _int4_sz_bytes(n, k, group), "sz"), n, k, group, _ptr(y_f32, ok and 4 * m * n, "y_f32"),
          _ptr(y_bf16, ok and 2 * m * n, "y_bf16"), _stream(stream))


def wq_gemm_smallM_int8(x, m, q, scale, n, k, y_f32=None, y_bf16=None, stream=None):
    """m token rows x [m, k] through int8 per-row weights -> y [m, n]."""
    ok = _nonneg(m, n, k)
    _call("wq_gemm_smallM_int8", _ptr(x, ok and 2 * m * k, "x"), m, _ptr(q, ok and n * k, "q"),
          _ptr(scale, ok and 2 * n, "scale"), n, k, _ptr(y_f32, ok and 4 * m * n, "y_f32"),
          _ptr(y_bf16, ok and 2 * m * n, "y_bf16"), _stream(stream))


def _mx_call(fn, name, stream, n, k, *buffers):
    """A call over [n][k] values with two buffers (tensor, bytes, what) before and two behind the sizes.  They are checked
    as in _ptr and must be on the current device, and the current stream is asked for as in _run (a call on a few rows is
    bound by these lines)."""
    ok = _nonneg(n, k)
    at, devices = [], set()
    for t, nbytes, what in buffers:
        if t is None or isinstance(t, int):
            at.append(t)
            continue
        if ok and t.numel() * t.element_size() < nbytes:
            raise ValueError(f"libwq: {what} holds {t.numel() * t.element_size()} bytes; the sizes given need {nbytes}")
        if not t.is_contiguous():
            raise ValueError(f"libwq: {what} must be contiguous")
        devices.add(t.get_device())
        at.append(t.data_ptr())
    if -1 in devices:
        _refuse_host((_HostBuffer(),))
    device = _current_device() if devices or stream is None else None
    if devices and devices != {device}:
        raise ValueError(f"libwq: buffers on devices {sorted(devices)}, the current one is {device}")
    rc = fn(at[0], at[1], n, k, at[2], at[3], _raw_stream(device) if stream is None else _stream(stream))
    if rc != 0:
        raise WQError(name, rc, lib.wq_last_error().decode(errors="replace"))


def _current_device():
    global _current_device
    import torch
    torch.cuda.current_device()               # initialises the runtime where nothing has yet
    _current_device = torch._C._cuda_getDevice
    return _current_device()


def wq_quantize_mxfp4(w_f32, w_bf16, n, k, q, scale, stream=None):
    _mx_call(lib.wq_quantize_mxfp4, "wq_quantize_mxfp4", stream, n, k, (w_f32, 4 * n * k, "w_f32"),
             (w_bf16, 2 * n * k, "w_bf16"), (q, n * k // 2, "q"), (scale, n * k // 32, "scale"))


def wq_dequantize_mxfp4(q, scale, n, k, y_f32=None, y_bf16=None, stream=None):
    _mx_call(lib.wq_dequantize_mxfp4, "wq_dequantize_mxfp4", stream, n, k, (q, n * k // 2, "q"),
             (scale, n * k // 32, "scale"), (y_f32, 4 * n * k, "y_f32"), (y_bf16, 2 * n * k, "y_bf16"))


def _moe_bytes(e, dim, f):
    """Extent of each buffer of one MoE layer (zeros when the sizes are invalid: the C call reports them)."""
    if not _nonneg(e, dim, f):
        e = dim = f = 0
    return {"x": 2 * dim, "logits": 4 * e, "w13": e * 2 * f * dim, "s13": e * 2 * f * 2, "w2": e * dim * f,
            "s2": e * dim * 2, "work": 8 * f, "y_f32": 4 * dim, "y_bf16": 2 * dim, "sel": 8, "gates": 8}


def moe_top2_gemv(x, logits, e, w13, s13, w2, s2, dim, f, work, y_f32=None, y_bf16=None, sel=None,
                  gates=None, stream=None):
    b = _moe_bytes(e, dim, f)
    _call("moe_top2_gemv", _ptr(x, b["x"], "x"), _ptr(logits, b["logits"], "logits"), e, _ptr(w13, b["w13"], "w13"),
          _ptr(s13, b["s13"], "s13"), _ptr(w2, b["w2"], "w2"), _ptr(s2, b["s2"], "s2"), dim, f,
          _ptr(work, b["work"], "work"), _ptr(y_f32, b["y_f32"], "y_f32"), _ptr(y_bf16, b["y_bf16"], "y_bf16"),
          _ptr(sel, b["sel"], "sel"), _ptr(gates, b["gates"], "gates"), _stream(stream))


def moe_top2_gemv_noalloc(x, logits, e, w13, s13, w2, s2, dim, f, y_f32=None, y_bf16=None, sel=None,
                          gates=None, stream=None):
    """moe_top2_gemv with the SwiGLU intermediate in the library's static device scratch (f <= 16384)."""
    b = _moe_bytes(e, dim, f)
    _call("moe_top2_gemv_noalloc", _ptr(x, b["x"], "x"), _ptr(logits, b["logits"], "logits"), e,
          _ptr(w13, b["w13"], "w13"), _ptr(s13, b["s13"], "s13"), _ptr(w2, b["w2"], "w2"), _ptr(s2, b["s2"], "s2"),
          dim, f, _ptr(y_f32, b["y_f32"], "y_f32"), _ptr(y_bf16, b["y_bf16"], "y_bf16"), _ptr(sel, b["sel"], "sel"),
          _ptr(gates, b["gates"], "gates"), _stream(stream))


def wq_decode_step_workspace_bytes(count):
    return int(lib.wq_decode_step_workspace_bytes(count))


def wq_decode_step_prepare(format, m, mats, workspace, workspace_bytes=None):
    """mats: sequence of (x, w, aux, n, k, y_f32, y_bf16) with tensors (or None).
    `format` is a WQ_FORMAT code or name ("bf16", "int8", "int4g32", "int4g64",
    "int4g128", "int4g256", "int4pc": one group per row).  Returns the
    wq_step_plan."""
    fmt = WQ_FORMAT.get(format, format)
    name = {v: k for k, v in WQ_FORMAT.items()}.get(fmt)
    ptrs = []
    for i, (x, w, aux, n, k, y32, y16) in enumerate(mats):
        ok = name is not None and _nonneg(m, n, k)
        if ok and name == "bf16":
            wb, ab = 2 * n * k, 0
        elif ok and name == "int8":
            wb, ab = n * k, 2 * n
        elif ok:
            wb, ab = n * k // 2, _int4_sz_bytes(n, k, k if name == "int4pc" else int(name[5:]))
        else:
            wb = ab = 0
        ptrs.append((_ptr(x, ok and 2 * m * k, f"matrix {i} x"), _ptr(w, wb, f"matrix {i} w"),
                     _ptr(aux, ab, f"matrix {i} aux"), n, k, _ptr(y32, ok and 4 * m * n, f"matrix {i} y_f32"),
                     _ptr(y16, ok and 2 * m * n, f"matrix {i} y_bf16")))
    _refuse_host([a for p in ptrs for a in p] + [_ptr(workspace)])
    arr = (wq_matrix * len(mats))()
    for i, p in enumerate(ptrs):
        arr[i] = wq_matrix(*p)
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    plan = wq_step_plan()
    rc = lib.wq_decode_step_prepare(fmt, m, arr, len(mats), _ptr(workspace), workspace_bytes, ctypes.byref(plan))
    if rc != 0:
        raise WQError("wq_decode_step_prepare", rc, lib.wq_last_error().decode(errors="replace"))
    return plan


def wq_decode_step_run(plan, stream=None):
    rc = lib.wq_decode_step_run(ctypes.byref(plan), _stream(stream))
    if rc != 0:
        raise WQError("wq_decode_step_run", rc, lib.wq_last_error().decode(errors="replace"))


def wq_moe_step_workspace_bytes(count):
    return int(lib.wq_moe_step_workspace_bytes(count))


def wq_moe_step_prepare(e, dim, f, layers, workspace, workspace_bytes=None):
    """layers: sequence of (x, logits, w13, s13, w2, s2, work, y_f32, y_bf16, sel, gates) with tensors (or
    None).  Returns the wq_moe_plan."""
    b = _moe_bytes(e, dim, f)
    keys = ("x", "logits", "w13", "s13", "w2", "s2", "work", "y_f32", "y_bf16", "sel", "gates")
    ptrs = [[_ptr(t, b[kk], f"layer {i} {kk}") for t, kk in zip(L, keys)] for i, L in enumerate(layers)]
    _refuse_host([a for p in ptrs for a in p] + [_ptr(workspace)])
    arr = (wq_moe_layer * len(layers))()
    for i, p in enumerate(ptrs):
        arr[i] = wq_moe_layer(*p)
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    plan = wq_moe_plan()
    rc = lib.wq_moe_step_prepare(e, dim, f, arr, len(layers), _ptr(workspace), workspace_bytes, ctypes.byref(plan))
    if rc != 0:
        raise WQError("wq_moe_step_prepare", rc, lib.wq_last_error().decode(errors="replace"))
    return plan


def wq_moe_step_run(plan, stream=None):
    rc = lib.wq_moe_step_run(ctypes.byref(plan), _stream(stream))
    if rc != 0:
        raise WQError("wq_moe_step_run", rc, lib.wq_last_error().decode(errors="replace"))


# ---------------------------------------------------------------------------
# Between the linears of a verify pass, and the adapters beside them.  Sizes
# and strides are read off the tensors; each *_prepare returns a plan that
# keeps its tensors alive, each *_run enqueues it.  Keep a plan (and with it its
# workspace) until its runs on every stream are done.


def _view(t, what, dims, dtypes, device, unit=True):
    """A GPU tensor of one of `dtypes` with `dims` axes on `device`, its last axis contiguous (`unit`)."""
    if not hasattr(t, "data_ptr"):
        raise ValueError(f"libwq: {what} must be a tensor")
    names = [str(t.dtype).replace("torch.", "")]
    if names[0] not in dtypes:
        raise ValueError(f"libwq: {what} must be {' or '.join(dtypes)}, not {names[0]}")
    if t.dim() != dims:
        raise ValueError(f"libwq: {what} must have {dims} axes, not {t.dim()}")
    if unit and dims and t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"libwq: the last axis of {what} must be contiguous")
    if not t.is_cuda:
        raise ValueError("libwq buffers must be GPU tensors (device memory)")
    if device is not None and t.device != device:
        raise ValueError(f"libwq: {what} is on {t.device}, the plan's other buffers on {device}")
    return t


_BF16 = ("bfloat16", "int16", "uint16")      # bf16 values, or their bit patterns


def _at(t):
    """Address of a tensor; an empty one has none, and its call touches nothing."""
    return t.data_ptr() if t.numel() else 16


def _heads_view(t, what, heads, device):
    """[tokens, heads, dim] or [tokens, heads * dim] as (tensor, tokens, row stride, dim)."""
    if hasattr(t, "dim") and t.dim() == 3:
        _view(t, what, 3, _BF16, device)
        if t.shape[1] > 1 and t.stride(1) != t.shape[2]:
            raise ValueError(f"libwq: the heads of a row of {what} must be contiguous")
        if heads is not None and t.shape[1] != heads:
            raise ValueError(f"libwq: {what} has {t.shape[1]} heads, not {heads}")
        width = t.shape[1] * t.shape[2]
    else:
        _view(t, what, 2, _BF16, device)
        width = t.shape[1]
    return t.shape[0], _row_stride(t, width)


def _row_stride(t, width):
    """Stride of the first axis; of a single row, any that holds it."""
    return t.stride(0) if t.shape[0] > 1 else max(width, 8 * (-(-width // 8)))


def _cache_struct(k, v, table, requests, device, layers=False):
    dims = 5 if layers else 4
    _view(k, "k", dims, _BF16, device)
    _view(v, "v", dims, _BF16, device)
    if k.shape != v.shape or k.stride() != v.stride():
        raise ValueError("libwq: k and v must have the same shape and strides")
    _view(table, "table", 2, ("int32",), device)
    if table.shape[0] < requests:
        raise ValueError(f"libwq: table holds {table.shape[0]} requests; {requests} are needed")
    if any(s == 0 and n > 1 for n, s in zip(k.shape, k.stride())):
        raise ValueError("libwq: k and v must not be expanded tensors")
    pages, page_size, kv_heads, head_dim = k.shape[-4:]
    # the stride of an axis of length one is never used
    strides = [s if n > 1 else 0 for n, s in zip(k.shape[-4:-1], k.stride()[-4:-1])]
    return wq_kv_cache(_at(k), _at(v), pages, page_size, *strides, _at(table), table.shape[1],
                       table.stride(0) if table.shape[0] > 1 else table.shape[1], kv_heads, head_dim)


def _batch_struct(starts, lengths, tokens, device):
    _view(starts, "starts", 1, ("int32",), device)
    _view(lengths, "lengths", 1, ("int32",), device)
    if starts.shape[0] != lengths.shape[0] + 1:
        raise ValueError(f"libwq: starts holds {starts.shape[0]} values; {lengths.shape[0] + 1} are needed")
    return wq_batch(_at(starts), _at(lengths), tokens, lengths.shape[0])


def _vector(t, what, length, dtypes, device):
    """Address of an optional vector of at least `length` elements."""
    if t is None:
        return None
    _view(t, what, 1, dtypes, device)
    if t.shape[0] < length:
        raise ValueError(f"libwq: {what} holds {t.shape[0]} values; {length} are needed")
    return _at(t)


def _workspace(workspace, nbytes, device):
    if workspace is None:
        import torch
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=device)
    _view(workspace, "workspace", 1, ("uint8",), device)
    return workspace, workspace.numel()


def _raw_stream(device):
    """Address of torch's current stream on `device`: what _stream returns, without building the Stream object (3 us
    of a 6 us call)."""
    global _raw_stream
    import torch
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda d: torch.cuda.current_stream(d).cuda_stream)
    return _raw_stream(device)


def _prepare(name, plan, device, keep, *args):
    import torch
    with torch.cuda.device(device):
        rc = getattr(lib, name)(*args, ctypes.byref(plan))
    if rc != 0:
        raise WQError(name, rc, lib.wq_last_error().decode(errors="replace"))
    plan.keep = keep
    plan.at = ctypes.addressof(plan)
    return plan


def _run(name, fn, plan, stream):
    rc = fn(plan.at, _raw_stream(plan.device) if stream is None else _stream(stream))
    if rc != 0:
        raise WQError(name, rc, lib.wq_last_error().decode(errors="replace"))


def wq_rope_frequencies(rot_dim, base, kind="plain", factor=1.0, low=1.0, high=None, original=8192.0):
    """Rotary frequencies as a CPU tensor fp32 [rot_dim / 2], and the rot_scale that goes with them.  kind:
    "plain", "linear", "bands" or "ramp" (a WQ_ROPE name or code).  high None: what the kind is published with, 4
    turns for bands and 32 for a ramp."""
    import torch
    if high is None:
        high = 32.0 if WQ_ROPE.get(kind, kind) == WQ_ROPE["ramp"] else 4.0
    freq = torch.empty(max(int(rot_dim), 0) // 2, dtype=torch.float32)
    scale = ctypes.c_float()
    rc = lib.wq_rope_frequencies(WQ_ROPE.get(kind, kind), rot_dim, base, factor, low, high, original,
                                 ctypes.cast(freq.data_ptr() or None, ctypes.POINTER(ctypes.c_float)),
                                 ctypes.byref(scale))
    if rc != 0:
        raise WQError("wq_rope_frequencies", rc, lib.wq_last_error().decode(errors="replace"))
    return freq, scale.value


def wq_qkv_rope_prepare(qkv, q, k, v, table, starts, lengths, freq=None, positions=None, q_norm=None, k_norm=None,
                        eps=1e-6, rot_scale=1.0, interleaved=False):
    """qkv [tokens, (heads + 2 kv_heads) * dim] fp32 or bf16; q out, bf16 [tokens, heads, dim]; k, v the layer's
    cache [pages, page_size, kv_heads, dim]; table int32 [requests, pages per request]; freq fp32 [rot_dim / 2]."""
    _view(qkv, "qkv", 2, ("float32",) + _BF16, None)
    device = qkv.device
    requests = lengths.shape[0] if hasattr(lengths, "shape") and lengths.dim() == 1 else 0
    cache = _cache_struct(k, v, table, requests, device)
    dim = cache.head_dim
    tokens, q_stride = _heads_view(q, "q", None, device)
    heads = (q.shape[1] * q.shape[2] if q.dim() == 3 else q.shape[1]) // dim
    if qkv.shape[0] != tokens or qkv.shape[1] != (heads + 2 * cache.kv_heads) * dim or \
            q.numel() != tokens * heads * dim:
        raise ValueError(f"libwq: qkv {tuple(qkv.shape)} does not go with q {tuple(q.shape)} and "
                         f"{cache.kv_heads} key heads of {dim}")
    rot_dim = 0
    if freq is not None:
        _view(freq, "freq", 1, ("float32",), device)
        rot_dim = 2 * freq.shape[0]
    f32 = str(qkv.dtype) == "torch.float32"
    a = wq_qkv_rope(cache, _batch_struct(starts, lengths, tokens, device), _at(qkv) if f32 else None,
                    None if f32 else _at(qkv), _row_stride(qkv, qkv.shape[1]), _at(q), q_stride,
                    _vector(positions, "positions", tokens, ("int32",), device),
                    _vector(q_norm, "q_norm", dim, _BF16, device), _vector(k_norm, "k_norm", dim, _BF16, device),
                    _at(freq) if rot_dim else None, eps, rot_scale, rot_dim, 1 if interleaved else 0, heads)
    return _prepare("wq_qkv_rope_prepare", wq_qkv_rope_plan(), device,
                    (qkv, q, k, v, table, starts, lengths, freq, positions, q_norm, k_norm), ctypes.byref(a))


def wq_qkv_rope_run(plan, stream=None):
    _run("wq_qkv_rope_run", lib.wq_qkv_rope_run, plan, stream)


def wq_tree_attention_workspace_bytes(requests, heads, kv_heads, head_dim, max_tokens):
    return int(lib.wq_tree_attention_workspace_bytes(requests, heads, kv_heads, head_dim, max_tokens))


def wq_tree_attention_prepare(q, k, v, table, starts, lengths, y, tree=None, max_tokens=64, scale=None,
                              workspace=None):
    """q, y bf16 [tokens, heads, dim]; k, v, table as for wq_qkv_rope_prepare; tree int64 (or uint64) [tokens]; scale
    None: dim ** -0.5; workspace None: allocated here."""
    device = getattr(q, "device", None)
    tokens, q_stride = _heads_view(q, "q", None, None)
    requests = lengths.shape[0] if hasattr(lengths, "shape") and lengths.dim() == 1 else 0
    cache = _cache_struct(k, v, table, requests, device)
    dim = cache.head_dim
    width = q.numel() // tokens if tokens else (q.shape[1] * q.shape[2] if q.dim() == 3 else q.shape[1])
    heads = width // dim
    _, y_stride = _heads_view(y, "y", None, device)
    if heads * dim != width or y.shape[0] != tokens or y.numel() != q.numel():
        raise ValueError(f"libwq: q {tuple(q.shape)} and y {tuple(y.shape)} do not hold heads of {dim}")
    a = wq_tree_attention(cache, _batch_struct(starts, lengths, tokens, device), _at(q), q_stride, _at(y),
                          y_stride, _vector(tree, "tree", tokens, ("int64", "uint64"), device),
                          dim ** -0.5 if scale is None else scale, heads, max_tokens)
    workspace, nbytes = _workspace(
        workspace, wq_tree_attention_workspace_bytes(requests, heads, cache.kv_heads, dim, max_tokens), device)
    return _prepare("wq_tree_attention_prepare", wq_tree_attention_plan(), device,
                    (q, k, v, table, starts, lengths, y, tree, workspace), ctypes.byref(a), _at(workspace),
                    nbytes)


def wq_tree_attention_run(plan, stream=None):
    _run("wq_tree_attention_run", lib.wq_tree_attention_run, plan, stream)


def wq_kv_accept_prepare(k, v, table, lengths, path, accepted):
    """k, v [layers, pages, page_size, kv_heads, dim] (or one layer without the first axis); path int32 [requests, up
    to 64]; accepted int32 [requests]."""
    if hasattr(k, "dim") and k.dim() == 4:
        return wq_kv_accept_prepare(k.unsqueeze(0), v.unsqueeze(0) if hasattr(v, "dim") else v, table, lengths, path,
                                    accepted)
    device = getattr(k, "device", None)
    _view(lengths, "lengths", 1, ("int32",), device)
    requests = lengths.shape[0]
    cache = _cache_struct(k, v, table, requests, device, layers=True)
    _view(path, "path", 2, ("int32",), device)
    if path.shape[0] < requests:
        raise ValueError(f"libwq: path holds {path.shape[0]} requests; {requests} are needed")
    a = wq_kv_accept(cache, k.shape[0], k.stride(0) if k.shape[0] > 1 else 0, requests, _at(lengths),
                     _at(path), path.shape[1], path.stride(0) if path.shape[0] > 1 else path.shape[1],
                     _vector(accepted, "accepted", requests, ("int32",), device))
    return _prepare("wq_kv_accept_prepare", wq_kv_accept_plan(), device, (k, v, table, lengths, path, accepted),
                    ctypes.byref(a))


def wq_kv_accept_run(plan, stream=None):
    _run("wq_kv_accept_run", lib.wq_kv_accept_run, plan, stream)


def wq_lora_workspace_bytes(tokens, k, adapters, rank):
    return int(lib.wq_lora_workspace_bytes(tokens, k, adapters, rank))


def wq_lora_prepare(x, a, b, adapter, y, y2=None, base=None, ranks=None, scale=None, workspace=None):
    """x bf16 [tokens, k]; a bf16 [adapters, rank, k]; b bf16 [adapters, n, rank]; adapter int32 [tokens]; y fp32 or
    bf16 [tokens, n], y2 the other of the two (same row stride) or None; base fp32 [tokens, n] or None."""
    _view(x, "x", 2, _BF16, None)
    device, (tokens, k) = x.device, x.shape
    _view(a, "a", 3, _BF16, device)
    _view(b, "b", 3, _BF16, device)
    if not a.is_contiguous() or not b.is_contiguous():
        raise ValueError("libwq: a and b must be contiguous")
    adapters, rank, n = a.shape[0], a.shape[1], b.shape[1]
    if a.shape[2] != k or b.shape[0] != adapters or b.shape[2] != rank:
        raise ValueError(f"libwq: a {tuple(a.shape)} and b {tuple(b.shape)} do not go with x {tuple(x.shape)}")
    out = {"f32": None, "bf16": None}
    for t, what in ((y, "y"), (y2, "y2")):
        if t is None:
            continue
        _view(t, what, 2, ("float32",) + _BF16, device)
        if tuple(t.shape) != (tokens, n):
            raise ValueError(f"libwq: {what} must be {(tokens, n)}, not {tuple(t.shape)}")
        kind = "f32" if str(t.dtype) == "torch.float32" else "bf16"
        if out[kind] is not None:
            raise ValueError("libwq: y and y2 must be one fp32 and one bf16")
        out[kind] = t
    strides = {_row_stride(t, n) for t in out.values() if t is not None}
    if len(strides) > 1:
        raise ValueError("libwq: y and y2 must have the same row stride")
    if base is not None:
        _view(base, "base", 2, ("float32",), device)
        if tuple(base.shape) != (tokens, n):
            raise ValueError(f"libwq: base must be {(tokens, n)}, not {tuple(base.shape)}")
    desc = wq_lora(_at(x), _row_stride(x, k), None if base is None else _at(base),
                   0 if base is None else _row_stride(base, n), *(None if t is None else _at(t) for t in out.values()),
                   max(strides, default=0), _at(a), _at(b),
                   _vector(adapter, "adapter", tokens, ("int32",), device),
                   _vector(ranks, "ranks", adapters, ("int32",), device),
                   _vector(scale, "scale", adapters, ("float32",), device), tokens, k, n, adapters, rank)
    workspace, nbytes = _workspace(workspace, wq_lora_workspace_bytes(tokens, k, adapters, rank), device)
    return _prepare("wq_lora_prepare", wq_lora_plan(), device,
                    (x, a, b, adapter, y, y2, base, ranks, scale, workspace), ctypes.byref(desc), _at(workspace),
                    nbytes)


def wq_lora_run(plan, stream=None):
    _run("wq_lora_run", lib.wq_lora_run, plan, stream)


# ---------------------------------------------------------------------------
# MXFP4 products and the block around them: plans, as above.


def _outputs(y, y2, shape, device):
    """Addresses of an fp32 and a bf16 result (either may be missing) and their row stride."""
    out = {"f32": None, "bf16": None}
    for t, what in ((y, "y"), (y2, "y2")):
        if t is None:
            continue
        _view(t, what, 2, ("float32",) + _BF16, device)
        if tuple(t.shape) != shape:
            raise ValueError(f"libwq: {what} must be {shape}, not {tuple(t.shape)}")
        kind = "f32" if str(t.dtype) == "torch.float32" else "bf16"
        if out[kind] is not None:
            raise ValueError("libwq: y and y2 must be one fp32 and one bf16")
        out[kind] = t
    strides = {_row_stride(t, shape[1]) for t in out.values() if t is not None}
    if len(strides) > 1:
        raise ValueError("libwq: y and y2 must have the same row stride")
    return [None if t is None else _at(t) for t in out.values()], max(strides, default=0)


def _mx_view(q, scale, what, dims, device):
    """MXFP4 codes [..., n, k / 2] and scales [..., n, k / 32], contiguous; k."""
    _view(q, what, dims, ("uint8",), device)
    _view(scale, f"the scales of {what}", dims, ("uint8",), q.device)
    if not q.is_contiguous() or not scale.is_contiguous():
        raise ValueError(f"libwq: {what} and its scales must be contiguous")
    if q.shape[:-1] != scale.shape[:-1] or q.shape[-1] != 16 * scale.shape[-1]:
        raise ValueError(f"libwq: {what} {tuple(q.shape)} and its scales {tuple(scale.shape)} do not go together")
    return 2 * q.shape[-1]


def wq_gemm_mxfp4_workspace_bytes(m, n, k):
    return int(lib.wq_gemm_mxfp4_workspace_bytes(m, n, k))


def wq_gemm_mxfp4_prepare(x, q, scale, y, y2=None, x_scale=None, workspace=None):
    """x bf16 [m, k], or uint8 codes [m, k / 2] with x_scale uint8 [m, k / 32]; q uint8 [n, k / 2], scale uint8
    [n, k / 32]; y fp32 or bf16 [m, n], y2 the other of the two (same row stride) or None."""
    device = getattr(x, "device", None)
    k = _mx_view(q, scale, "q", 2, device)
    n = q.shape[0]
    if x_scale is None:
        _view(x, "x", 2, _BF16, device)
        if x.shape[1] != k:
            raise ValueError(f"libwq: x {tuple(x.shape)} does not go with q {tuple(q.shape)}")
        ins = (_at(x), _row_stride(x, k), None, None)
    else:
        if _mx_view(x, x_scale, "x", 2, device) != k:
            raise ValueError(f"libwq: x {tuple(x.shape)} does not go with q {tuple(q.shape)}")
        ins = (None, 0, _at(x), _at(x_scale))
    m = x.shape[0]
    outs, y_stride = _outputs(y, y2, (m, n), device)
    a = wq_gemm_mxfp4(*ins, _at(q), _at(scale), *outs, y_stride, m, n, k)
    workspace, nbytes = _workspace(workspace, wq_gemm_mxfp4_workspace_bytes(m, n, k), device)
    return _prepare("wq_gemm_mxfp4_prepare", wq_gemm_mxfp4_plan(), device, (x, q, scale, y, y2, x_scale, workspace),
                    ctypes.byref(a), _at(workspace), nbytes)


def wq_gemm_mxfp4_run(plan, stream=None):
    _run("wq_gemm_mxfp4_run", lib.wq_gemm_mxfp4_run, plan, stream)


def wq_moe_ffn_workspace_bytes(tokens, dim, f, e, top):
    return int(lib.wq_moe_ffn_workspace_bytes(tokens, dim, f, e, top))


def wq_moe_ffn_prepare(x, w13, s13, w2, s2, y, y2=None, router=None, logits=None, top=2, renormalize=True, sel=None,
                       gates=None, workspace=None):
    """x bf16 [tokens, dim]; w13 int8 [e, 2f, dim] with s13 bf16 [e, 2f] and w2 int8 [e, dim, f] with s2 bf16 [e, dim],
    or MXFP4: uint8 [e, 2f, dim / 2] with uint8 [e, 2f, dim / 32] and [e, dim, f / 2] with [e, dim, f / 32]; router bf16
    [e, dim] or logits fp32 [tokens, e]; y fp32 or bf16 [tokens, dim], y2 the other of the two; sel int32 and gates fp32
    [tokens, top], out."""
    _view(x, "x", 2, _BF16, None)
    device, (tokens, dim) = x.device, x.shape
    mx = str(getattr(w13, "dtype", "")) == "torch.uint8"
    if mx:
        up, f = _mx_view(w13, s13, "w13", 3, device), _mx_view(w2, s2, "w2", 3, device)
    else:
        for t, what, dims, kinds in ((w13, "w13", 3, ("int8",)), (s13, "s13", 2, _BF16), (w2, "w2", 3, ("int8",)),
                                     (s2, "s2", 2, _BF16)):
            _view(t, what, dims, kinds, device)
            if not t.is_contiguous():
                raise ValueError(f"libwq: {what} must be contiguous")
        up, f = w13.shape[2], w2.shape[2]
        if s13.shape != w13.shape[:2] or s2.shape != w2.shape[:2]:
            raise ValueError(f"libwq: scales {tuple(s13.shape)}, {tuple(s2.shape)} do not go with w13 "
                             f"{tuple(w13.shape)} and w2 {tuple(w2.shape)}")
    e = w13.shape[0]
    if up != dim or w13.shape[1] != 2 * f or tuple(w2.shape[:2]) != (e, dim):
        raise ValueError(f"libwq: w13 {tuple(w13.shape)} and w2 {tuple(w2.shape)} do not go with x {tuple(x.shape)}")
    for t, what, shape, kinds in ((router, "router", (e, dim), _BF16), (logits, "logits", (tokens, e), ("float32",)),
                                  (sel, "sel", (tokens, top), ("int32",)), (gates, "gates", (tokens, top), ("float32",))):
        if t is not None:
            _view(t, what, 2, kinds, device)
            if tuple(t.shape) != shape or not t.is_contiguous():
                raise ValueError(f"libwq: {what} must be {shape} and contiguous, not {tuple(t.shape)}")
    outs, y_stride = _outputs(y, y2, (tokens, dim), device)
    a = wq_moe_ffn(_at(x), _row_stride(x, dim), *(None if t is None else _at(t) for t in (router, logits)), _at(w13),
                   _at(s13), _at(w2), _at(s2), *outs, y_stride, *(None if t is None else _at(t) for t in (sel, gates)),
                   tokens, dim, f, e, top, WQ_FORMAT["mxfp4" if mx else "int8"], 1 if renormalize else 0)
    workspace, nbytes = _workspace(workspace, wq_moe_ffn_workspace_bytes(tokens, dim, f, e, top), device)
    return _prepare("wq_moe_ffn_prepare", wq_moe_ffn_plan(), device,
                    (x, w13, s13, w2, s2, y, y2, router, logits, sel, gates, workspace), ctypes.byref(a), _at(workspace),
                    nbytes)


def wq_moe_ffn_run(plan, stream=None):
    _run("wq_moe_ffn_run", lib.wq_moe_ffn_run, plan, stream)


def wq_block_norm_prepare(h, h_out=None, f=None, f_norm=None, gate=None, gate_kind="plain", scale=1.0, norm=None, u=None,
                          q=None, q_scale=None, eps=1e-6):
    """h, h_out and f fp32 or bf16 [rows, dim] (h_out may be h); f_norm and norm bf16 [dim]; gate bf16 [rows, dim] (a row
    expanded over all is read once) or [dim], gate_kind a WQ_GATE name or code; u bf16 [rows, dim]; q uint8
    [rows, dim / 2] with q_scale uint8 [rows, dim / 32]."""
    kinds = ("float32",) + _BF16
    _view(h, "h", 2, kinds, None)
    device, (rows, dim) = h.device, h.shape

    def rows_of(t, what, dtypes):
        """(fp32 address, bf16 address, row stride)"""
        if t is None:
            return None, None, 0
        _view(t, what, 2, dtypes, device)
        if tuple(t.shape) != (rows, dim):
            raise ValueError(f"libwq: {what} must be {(rows, dim)}, not {tuple(t.shape)}")
        f32 = str(t.dtype) == "torch.float32"
        return _at(t) if f32 else None, None if f32 else _at(t), _row_stride(t, dim)

    if gate is not None and hasattr(gate, "dim") and gate.dim() == 1:
        gate = gate.expand(rows, dim) if gate.shape[0] == dim else gate
    _, gate_at, gate_stride = rows_of(gate, "gate", _BF16)
    if gate is not None and rows > 1 and gate.stride(0) == 0:
        gate_stride = 0
    _, u_at, u_stride = rows_of(u, "u", _BF16)
    if (q is None) != (q_scale is None):
        raise ValueError("libwq: q and q_scale go together")
    if q is not None and _mx_view(q, q_scale, "q", 2, device) != dim or q is not None and q.shape[0] != rows:
        raise ValueError(f"libwq: q {tuple(q.shape)} does not go with h {tuple(h.shape)}")
    a = wq_block_norm(*rows_of(h, "h", kinds), *rows_of(h_out, "h_out", kinds), *rows_of(f, "f", kinds),
                      _vector(f_norm, "f_norm", dim, _BF16, device), gate_at, gate_stride,
                      _vector(norm, "norm", dim, _BF16, device), u_at, u_stride, None if q is None else _at(q),
                      None if q is None else _at(q_scale), rows, dim, scale, eps, WQ_GATE.get(gate_kind, gate_kind))
    return _prepare("wq_block_norm_prepare", wq_block_norm_plan(), device,
                    (h, h_out, f, f_norm, gate, norm, u, q, q_scale), ctypes.byref(a))


def wq_block_norm_run(plan, stream=None):
    _run("wq_block_norm_run", lib.wq_block_norm_run, plan, stream)
