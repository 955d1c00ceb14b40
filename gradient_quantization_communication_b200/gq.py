"""Python binding of the C ABI in ``include/gq.h`` (``libgq.so``): argument marshalling only.

Every function keeps the C name.  Tensors are passed as ``data_ptr()``; the stream defaults to
torch's current CUDA stream.  There is no fallback: if ``libgq.so`` is missing the import of the
library fails with an error that says how to build it.
"""
import ctypes
import functools
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgq.so")

GQ_QSGD, GQ_TERNGRAD, GQ_BINGRAD_B, GQ_BINGRAD_PB, GQ_ORQ, GQ_QSGD_NEAREST, GQ_SIGNSGD, GQ_QSGD_L2, GQ_TERNGRAD_LAYER = range(9)
GQ_OK, GQ_ERR_INVALID, GQ_ERR_UNSUPPORTED, GQ_ERR_CUDA, GQ_ERR_NONFINITE, GQ_ERR_NOMEM, GQ_ERR_TIMEOUT = 0, 1, 2, 3, 4, 5, 6
GQ_MAX_WORKERS = 64
GQ_FORMAT_DENSE, GQ_FORMAT_BASE_S = 0, 1
SCHEMES = {"qsgd": GQ_QSGD, "terngrad": GQ_TERNGRAD, "bingrad_b": GQ_BINGRAD_B,
           "bingrad_pb": GQ_BINGRAD_PB, "orq": GQ_ORQ, "qsgd_nearest": GQ_QSGD_NEAREST, "signsgd": GQ_SIGNSGD,
           "qsgd_l2": GQ_QSGD_L2, "terngrad_layer": GQ_TERNGRAD_LAYER}


GQ_FLOAT32, GQ_BFLOAT16, GQ_FLOAT16 = range(3)
GQ_FN_GELU, GQ_FN_GELU_TANH, GQ_FN_SILU = range(3)
GQ_FP8_E4M3, GQ_FP8_E5M2 = range(2)
FP8_FORMATS = {"e4m3": GQ_FP8_E4M3, "e5m2": GQ_FP8_E5M2}
FUNCTIONS = {"gelu": GQ_FN_GELU, "gelu_tanh": GQ_FN_GELU_TANH, "silu": GQ_FN_SILU}


class gq_config_t(ctypes.Structure):
    _fields_ = [("scheme", ctypes.c_int32), ("levels", ctypes.c_int32), ("bucket", ctypes.c_int32),
                ("workers", ctypes.c_int32), ("error_feedback", ctypes.c_int32),
                ("clip_sigma", ctypes.c_float), ("seed", ctypes.c_uint64), ("n", ctypes.c_int64)]


class gq_adamw_config_t(ctypes.Structure):
    _fields_ = [("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32), ("state_bits", ctypes.c_int32),
                ("seed", ctypes.c_uint64)]


class gq_adamw_tensor_t(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("m", ctypes.c_void_p), ("v", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("weight_decay", ctypes.c_float), ("lr_scale", ctypes.c_float)]


class gq_adamw_scalars_t(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_float), ("inv1", ctypes.c_float), ("inv2", ctypes.c_float), ("step", ctypes.c_uint32)]


class GQError(RuntimeError):
    def __init__(self, status, what):
        super().__init__("%s: %s (status %d)" % (what, gq_status_string(status), status))
        self.status = status


_lib = None


def lib():
    """The loaded libgq.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError("libgq.so is not built (%s); run gradient_quantization_communication_b200/build.py"
                              % LIB_PATH)
        L = ctypes.CDLL(LIB_PATH)
        vp, sz = ctypes.c_void_p, ctypes.c_size_t
        cfgp = ctypes.POINTER(gq_config_t)
        L.gq_config_check.argtypes = [cfgp]
        L.gq_message_layout.argtypes = [cfgp, ctypes.POINTER(sz), ctypes.POINTER(sz), ctypes.POINTER(sz)]
        L.gq_plan_create.argtypes = [cfgp, ctypes.POINTER(vp)]
        L.gq_plan_destroy.argtypes = [vp]
        L.gq_encode.argtypes = [vp, ctypes.c_uint32, ctypes.c_uint64, vp, vp, vp, vp]
        L.gq_decode_accumulate.argtypes = [vp, ctypes.POINTER(vp), ctypes.c_int, vp, vp]
        L.gq_fused_step.argtypes = [vp, ctypes.c_uint64, ctypes.POINTER(vp), ctypes.POINTER(vp),
                                    ctypes.POINTER(vp), vp, vp]
        L.gq_quant_error.argtypes = [vp, ctypes.c_uint32, ctypes.c_uint64, vp, vp, vp, vp]
        L.gq_quant_error_noalloc.argtypes = [cfgp, ctypes.c_uint32, ctypes.c_uint64, vp, vp, vp, vp]
        L.gq_plan_status.argtypes = [vp, vp]
        L.gq_plan_set_segments.argtypes = [vp, ctypes.POINTER(ctypes.c_int64), ctypes.c_int]
        L.gq_plan_set_format.argtypes = [vp, ctypes.c_int]
        L.gq_plan_message_layout.argtypes = [vp, ctypes.POINTER(sz), ctypes.POINTER(sz), ctypes.POINTER(sz)]
        L.gq_selftest_bounded_wait.argtypes = [vp, ctypes.c_int64, vp]
        L.gq_entropy_layout.argtypes = [cfgp, ctypes.POINTER(sz), ctypes.POINTER(sz), ctypes.POINTER(sz)]
        L.gq_entropy_pack.argtypes = [cfgp, vp, vp, vp]
        L.gq_entropy_unpack.argtypes = [cfgp, vp, vp, vp]
        L.gq_elias_layout.argtypes = [cfgp, ctypes.POINTER(sz), ctypes.POINTER(sz), ctypes.POINTER(sz),
                                      ctypes.POINTER(sz)]
        L.gq_elias_used_bytes.argtypes = [cfgp, ctypes.c_uint64, ctypes.POINTER(sz)]
        L.gq_elias_pack.argtypes = [cfgp, vp, vp, vp]
        L.gq_elias_unpack.argtypes = [cfgp, vp, vp, vp]
        i64, ci = ctypes.c_int64, ctypes.c_int
        L.gq_act_layout.argtypes = [i64, i64, ctypes.POINTER(sz), ctypes.POINTER(sz), ctypes.POINTER(sz)]
        L.gq_act_pack.argtypes = [ci, i64, i64, vp, i64, vp, vp]
        L.gq_act_unpack.argtypes = [ci, i64, i64, vp, vp, i64, vp]
        L.gq_act_fn_forward.argtypes = [ci, ci, i64, i64, vp, i64, vp, i64, vp, vp]
        L.gq_act_fn_backward.argtypes = [ci, ci, i64, i64, vp, vp, i64, vp, i64, vp]
        L.gq_act_weight_grad_workspace.argtypes = [ci, i64, i64, i64, i64, ci, ctypes.POINTER(sz)]
        L.gq_act_weight_grad.argtypes = [ci, i64, i64, i64, vp, vp, i64, vp, i64, vp, ci, vp, sz, vp]
        L.gq_layer_norm_forward.argtypes = [ci, ci, i64, i64, vp, i64, vp, vp, ctypes.c_float, vp, i64, vp, vp, vp, vp]
        L.gq_layer_norm_workspace.argtypes = [i64, i64, ctypes.POINTER(sz)]
        L.gq_layer_norm_backward.argtypes = [ci, ci, i64, i64, vp, i64, vp, i64, vp, vp, vp, vp, vp, i64, vp, vp, ci, vp,
                                             sz, vp]
        L.gq_fp8_layout.argtypes = [ci, i64, i64, ctypes.POINTER(sz), ctypes.POINTER(sz), ctypes.POINTER(sz)]
        L.gq_fp8_pack.argtypes = [ci, ci, ci, i64, i64, vp, i64, vp, vp, vp]
        L.gq_fp8_unpack.argtypes = [ci, ci, ci, i64, i64, vp, vp, i64, vp]
        L.gq_fp8_matmul_workspace.argtypes = [i64, i64, i64, ctypes.POINTER(sz)]
        L.gq_fp8_matmul.argtypes = [ci, i64, i64, i64, ci, ci, vp, ci, ci, vp, vp, vp, i64, ci, vp, sz, vp]
        f64 = ctypes.c_double
        L.gq_adamw_layout.argtypes = [i64, ctypes.POINTER(sz), ctypes.POINTER(sz)]
        L.gq_adamw_create.argtypes = [ctypes.POINTER(gq_adamw_config_t), ctypes.POINTER(gq_adamw_tensor_t), ci,
                                      ctypes.POINTER(vp)]
        L.gq_adamw_destroy.argtypes = [vp]
        L.gq_adamw_norm.argtypes = [vp, f64, vp, vp]
        L.gq_adamw_scalars.argtypes = [f64, f64, f64, i64, ctypes.POINTER(gq_adamw_scalars_t)]
        L.gq_adamw_step.argtypes = [vp, f64, f64, f64, f64, i64, vp, vp, vp]
        L.gq_adamw_moments.argtypes = [vp, ci, vp, vp, vp]
        L.gq_status_string.argtypes = [ctypes.c_int]
        L.gq_status_string.restype = ctypes.c_char_p
        L.gq_version.restype = ctypes.c_char_p
        for f in ("gq_config_check", "gq_message_layout", "gq_plan_create", "gq_plan_destroy", "gq_encode",
                  "gq_decode_accumulate", "gq_fused_step", "gq_quant_error", "gq_quant_error_noalloc",
                  "gq_plan_status", "gq_plan_set_segments", "gq_plan_message_layout", "gq_plan_set_format",
                  "gq_selftest_bounded_wait", "gq_entropy_layout", "gq_entropy_pack",
                  "gq_entropy_unpack", "gq_elias_layout", "gq_elias_used_bytes", "gq_elias_pack",
                  "gq_elias_unpack", "gq_act_layout", "gq_act_pack", "gq_act_unpack", "gq_act_fn_forward",
                  "gq_act_fn_backward", "gq_act_weight_grad_workspace", "gq_act_weight_grad",
                  "gq_layer_norm_forward", "gq_layer_norm_workspace", "gq_layer_norm_backward", "gq_fp8_layout",
                  "gq_fp8_pack", "gq_fp8_unpack", "gq_fp8_matmul_workspace", "gq_fp8_matmul", "gq_adamw_layout",
                  "gq_adamw_create", "gq_adamw_destroy", "gq_adamw_norm", "gq_adamw_scalars", "gq_adamw_step",
                  "gq_adamw_moments"):
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


# ---------------------------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------------------------
def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ptr_array(xs):
    if xs is None:
        return None
    return (ctypes.c_void_p * len(xs))(*[_ptr(x) for x in xs])


def _check(st, what):
    if st != GQ_OK:
        raise GQError(st, what)


def gq_config(scheme, levels=0, bucket=512, workers=1, error_feedback=True, clip_sigma=0.0, seed=0, n=0):
    if isinstance(scheme, str):
        scheme = SCHEMES[scheme]
    return gq_config_t(scheme, levels, bucket, workers, int(bool(error_feedback)), clip_sigma, seed, n)


# ---------------------------------------------------------------------------------------------
# the C entry points
# ---------------------------------------------------------------------------------------------
def gq_config_check(cfg):
    return lib().gq_config_check(ctypes.byref(cfg))


def gq_message_layout(cfg):
    b, c, l = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().gq_message_layout(ctypes.byref(cfg), ctypes.byref(b), ctypes.byref(c), ctypes.byref(l)),
           "gq_message_layout")
    return b.value, c.value, l.value


def gq_plan_create(cfg):
    h = ctypes.c_void_p()
    _check(lib().gq_plan_create(ctypes.byref(cfg), ctypes.byref(h)), "gq_plan_create")
    return h


def gq_plan_destroy(plan):
    _check(lib().gq_plan_destroy(plan), "gq_plan_destroy")


def gq_encode(plan, worker, step, grad, residual, msg, stream=None):
    _check(lib().gq_encode(plan, worker, step, _ptr(grad), _ptr(residual), _ptr(msg), _stream(stream)), "gq_encode")


def gq_decode_accumulate(plan, msgs, avg, stream=None):
    _check(lib().gq_decode_accumulate(plan, _ptr_array(msgs), len(msgs), _ptr(avg), _stream(stream)),
           "gq_decode_accumulate")


def gq_fused_step(plan, step, grads, residuals, msgs, avg, stream=None):
    _check(lib().gq_fused_step(plan, step, _ptr_array(grads), _ptr_array(residuals), _ptr_array(msgs), _ptr(avg),
                               _stream(stream)), "gq_fused_step")


def gq_quant_error(plan, worker, step, grad, residual, out, stream=None):
    _check(lib().gq_quant_error(plan, worker, step, _ptr(grad), _ptr(residual), _ptr(out), _stream(stream)),
           "gq_quant_error")


def gq_quant_error_noalloc(cfg, worker, step, grad, residual, out, stream=None):
    _check(lib().gq_quant_error_noalloc(ctypes.byref(cfg), worker, step, _ptr(grad), _ptr(residual), _ptr(out),
                                        _stream(stream)), "gq_quant_error_noalloc")


def gq_plan_set_segments(plan, offsets):
    arr = (ctypes.c_int64 * len(offsets))(*[int(x) for x in offsets])
    _check(lib().gq_plan_set_segments(plan, arr, len(offsets) - 1), "gq_plan_set_segments")


def gq_plan_set_format(plan, fmt):
    _check(lib().gq_plan_set_format(plan, int(fmt)), "gq_plan_set_format")


def gq_plan_message_layout(plan):
    b, c, l = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().gq_plan_message_layout(plan, ctypes.byref(b), ctypes.byref(c), ctypes.byref(l)),
           "gq_plan_message_layout")
    return b.value, c.value, l.value


def gq_plan_status(plan, stream=None):
    return lib().gq_plan_status(plan, _stream(stream))


def gq_selftest_bounded_wait(plan, limit_ns, stream=None):
    _check(lib().gq_selftest_bounded_wait(plan, int(limit_ns), _stream(stream)), "gq_selftest_bounded_wait")


def gq_entropy_layout(cfg):
    b, c, l = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().gq_entropy_layout(ctypes.byref(cfg), ctypes.byref(b), ctypes.byref(c), ctypes.byref(l)),
           "gq_entropy_layout")
    return b.value, c.value, l.value


def gq_entropy_pack(cfg, msg, emsg, stream=None):
    _check(lib().gq_entropy_pack(ctypes.byref(cfg), _ptr(msg), _ptr(emsg), _stream(stream)), "gq_entropy_pack")


def gq_entropy_unpack(cfg, emsg, msg, stream=None):
    _check(lib().gq_entropy_unpack(ctypes.byref(cfg), _ptr(emsg), _ptr(msg), _stream(stream)), "gq_entropy_unpack")


def gq_elias_layout(cfg):
    """(capacity bytes, offsets_off, tables_off, stream_off)."""
    v = [ctypes.c_size_t() for _ in range(4)]
    _check(lib().gq_elias_layout(ctypes.byref(cfg), *[ctypes.byref(x) for x in v]), "gq_elias_layout")
    return tuple(x.value for x in v)


def gq_elias_used_bytes(cfg, stream_bits):
    b = ctypes.c_size_t()
    _check(lib().gq_elias_used_bytes(ctypes.byref(cfg), int(stream_bits), ctypes.byref(b)), "gq_elias_used_bytes")
    return b.value


def gq_elias_pack(cfg, msg, emsg, stream=None):
    _check(lib().gq_elias_pack(ctypes.byref(cfg), _ptr(msg), _ptr(emsg), _stream(stream)), "gq_elias_pack")


def gq_elias_unpack(cfg, emsg, msg, stream=None):
    _check(lib().gq_elias_unpack(ctypes.byref(cfg), _ptr(emsg), _ptr(msg), _stream(stream)), "gq_elias_unpack")


# ---------------------------------------------------------------------------------------------
# activations kept in 8 bits: these take tensors, whose sizes, strides and types are the arguments
# ---------------------------------------------------------------------------------------------
_torch = _dtypes = _current_stream = _current_device = None


def _setup():
    """torch, looked up once: it is imported by the first call that takes tensors."""
    global _torch, _dtypes, _current_stream, _current_device
    import torch
    _dtypes = {torch.float32: GQ_FLOAT32, torch.bfloat16: GQ_BFLOAT16, torch.float16: GQ_FLOAT16}
    # the handle itself where torch offers it: building a Stream object around it takes a microsecond
    _current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda dev: torch.cuda.current_stream(dev).cuda_stream)
    _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    _torch = torch


def _dtype(t, what):
    if _dtypes is None:
        _setup()
    d = _dtypes.get(t.dtype)
    if d is None:
        raise TypeError("%s: float32, bfloat16 or float16 expected, got %s" % (what, t.dtype))
    return d


def _matrix(t, what, dtype=None, shape=None):
    """(pointer, row stride) of a 2-D tensor whose columns are adjacent."""
    st = t.stride()
    if len(st) != 2 or (st[1] != 1 and t.shape[1] > 1):
        raise ValueError("%s: a 2-D tensor with adjacent columns expected, got shape %s, strides %s"
                         % (what, tuple(t.shape), st))
    if dtype is not None and _dtype(t, what) != dtype:
        raise TypeError("%s: its type differs from the other tensors' (%s)" % (what, t.dtype))
    if shape is not None and t.shape != shape:
        raise ValueError("%s: shape %s expected, got %s" % (what, tuple(shape), tuple(t.shape)))
    return t.data_ptr(), st[0]


def _vector(t, what, n, dtype=GQ_FLOAT32):
    """Pointer of a contiguous vector of n values (None: NULL)."""
    if t is None:
        return None
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError("%s: a contiguous vector of %d values expected, got shape %s, strides %s"
                         % (what, n, tuple(t.shape), t.stride()))
    if _dtype(t, what) != dtype:
        raise TypeError("%s: wrong type %s" % (what, t.dtype))
    return t.data_ptr()


def _ckpt(t, rows, cols):
    """Pointer of a checkpoint buffer of rows x cols values (None: NULL)."""
    if t is None:
        return None
    need = (rows * ((cols + 31) // 32 * 32) + 15) // 16 * 16 + (rows * ((cols + 127) // 128 * 4) + 15) // 16 * 16
    if t.element_size() != 1 or t.dim() != 1 or t.shape[0] < need or not t.is_contiguous():
        raise ValueError("ckpt: a contiguous uint8 vector of at least %d bytes expected, got %s of shape %s"
                         % (need, t.dtype, tuple(t.shape)))
    return t.data_ptr()


def _launch(fn, what, stream, tensors, *args):
    """Call fn(*args, stream) on the tensors' device; the stream defaults to that device's current one."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and (t.get_device() != dev or dev < 0):
            raise ValueError("%s: CUDA tensors of one device expected, got %s"
                             % (what, ", ".join(str(x.device) for x in tensors if x is not None)))
    if stream is None:
        stream = _current_stream(dev)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if _current_device() == dev:
        st = fn(*args, stream)
    else:
        with _torch.cuda.device(dev):
            st = fn(*args, stream)
    if st != GQ_OK:
        raise GQError(st, what)


def _workspace(nbytes, device, stream=None):
    """nbytes on the device (None for 0), for use on `stream` (default: the current one)."""
    import torch
    if not nbytes:
        return None
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
    # from the stream's own pool: nothing else still uses the memory, and what reuses it comes after
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _space(workspace, what):
    """(pointer, bytes) of a workspace or None."""
    if workspace is None:
        return None, 0
    if not workspace.is_contiguous():
        raise ValueError("%s: a contiguous workspace expected" % what)
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def gq_act_layout(rows, cols):
    """(bytes, codes_off, exps_off) of a checkpoint."""
    b, c, e = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().gq_act_layout(rows, cols, ctypes.byref(b), ctypes.byref(c), ctypes.byref(e)), "gq_act_layout")
    return b.value, c.value, e.value


def gq_act_pack(x, ckpt, stream=None):
    px, sx = _matrix(x, "x")
    rows, cols = x.shape
    _launch(lib().gq_act_pack, "gq_act_pack", stream, (x, ckpt), _dtype(x, "x"), rows, cols, px, sx,
            _ckpt(ckpt, rows, cols))


def gq_act_unpack(ckpt, x, stream=None):
    px, sx = _matrix(x, "x")
    rows, cols = x.shape
    _launch(lib().gq_act_unpack, "gq_act_unpack", stream, (x, ckpt), _dtype(x, "x"), rows, cols,
            _ckpt(ckpt, rows, cols), px, sx)


def _kind(kind):
    k = FUNCTIONS.get(kind, kind)
    if not isinstance(k, int):
        raise ValueError("kind: one of %s expected, got %r" % (sorted(FUNCTIONS), kind))
    return k


def gq_act_fn_forward(kind, x, y, ckpt=None, stream=None):
    """kind: "gelu", "gelu_tanh", "silu" or the C constant."""
    dt = _dtype(x, "x")
    rows, cols = x.shape
    px, sx = _matrix(x, "x")
    py, sy = _matrix(y, "y", dt, (rows, cols))
    _launch(lib().gq_act_fn_forward, "gq_act_fn_forward", stream, (x, y, ckpt), _kind(kind), dt, rows, cols,
            px, sx, py, sy, _ckpt(ckpt, rows, cols))


def gq_act_fn_backward(kind, ckpt, dy, dx, stream=None):
    dt = _dtype(dy, "dy")
    rows, cols = dy.shape
    pdy, sdy = _matrix(dy, "dy")
    pdx, sdx = _matrix(dx, "dx", dt, (rows, cols))
    _launch(lib().gq_act_fn_backward, "gq_act_fn_backward", stream, (dy, dx, ckpt), _kind(kind), dt, rows,
            cols, _ckpt(ckpt, rows, cols), pdy, sdy, pdx, sdx)


def _weight_grad_bytes(dt, tokens, cin, cout, dy_stride, bias):
    b = ctypes.c_size_t()
    _check(lib().gq_act_weight_grad_workspace(dt, tokens, cin, cout, dy_stride, int(bias), ctypes.byref(b)),
           "gq_act_weight_grad_workspace")
    return b.value


def gq_act_weight_grad_workspace(ckpt, dy, dw, db=None):
    """A workspace tensor for gq_act_weight_grad on tensors of these sizes (None if it needs none)."""
    return _workspace(_weight_grad_bytes(_dtype(dy, "dy"), dy.shape[0], dw.shape[1], dw.shape[0], dy.stride(0),
                                         db is not None), dy.device)


def gq_act_weight_grad(ckpt, dy, dw, db=None, accumulate=False, workspace=None, stream=None):
    """dw: (out, in) float32, db: (out,) float32 or None.  Without a workspace one is allocated."""
    dt = _dtype(dy, "dy")
    pdy, sdy = _matrix(dy, "dy")
    pdw, sdw = _matrix(dw, "dw", GQ_FLOAT32)
    tokens, cout = dy.shape
    cin = dw.shape[1]
    if dw.shape[0] != cout:
        raise ValueError("dw: %d rows expected, got %d" % (cout, dw.shape[0]))
    if workspace is None:
        workspace = _workspace(_weight_grad_bytes(dt, tokens, cin, cout, sdy, db is not None), dy.device, stream)
    pws, nws = _space(workspace, "gq_act_weight_grad")
    _launch(lib().gq_act_weight_grad, "gq_act_weight_grad", stream, (dy, ckpt, dw, db, workspace), dt, tokens, cin, cout,
            _ckpt(ckpt, tokens, cin), pdy, sdy, pdw, sdw, _vector(db, "db", cout), int(bool(accumulate)), pws, nws)


def gq_layer_norm_forward(x, gamma, beta, eps, y, mean, rstd, ckpt=None, stream=None):
    """gamma, beta: vectors of x's type or float32 (both the same), or None."""
    dt = _dtype(x, "x")
    rows, cols = x.shape
    px, sx = _matrix(x, "x")
    py, sy = _matrix(y, "y", dt, (rows, cols))
    pdt = dt if gamma is None and beta is None else _dtype(gamma if gamma is not None else beta, "gamma")
    _launch(lib().gq_layer_norm_forward, "gq_layer_norm_forward", stream, (x, gamma, beta, y, mean, rstd, ckpt), dt, pdt,
            rows, cols, px, sx, _vector(gamma, "gamma", cols, pdt), _vector(beta, "beta", cols, pdt), eps, py, sy,
            _vector(mean, "mean", rows), _vector(rstd, "rstd", rows), _ckpt(ckpt, rows, cols))


def _layer_norm_bytes(rows, cols):
    b = ctypes.c_size_t()
    _check(lib().gq_layer_norm_workspace(rows, cols, ctypes.byref(b)), "gq_layer_norm_workspace")
    return b.value


def gq_layer_norm_workspace(dy):
    """A workspace tensor for gq_layer_norm_backward on a gradient of dy's size."""
    return _workspace(_layer_norm_bytes(dy.shape[0], dy.shape[1]), dy.device)


def gq_layer_norm_backward(dy, x, gamma, mean, rstd, dx, dgamma, dbeta, accumulate=False, workspace=None, stream=None):
    """x: the forward pass's input (2-D) or its checkpoint (a uint8 vector).  dgamma, dbeta: float32
    vectors or None.  Without a workspace one is allocated."""
    dt = _dtype(dy, "dy")
    rows, cols = dy.shape
    pdy, sdy = _matrix(dy, "dy")
    pdx, sdx = _matrix(dx, "dx", dt, (rows, cols))
    if x.dim() == 1:
        px, sx, pk = None, 0, _ckpt(x, rows, cols)
    else:
        (px, sx), pk = _matrix(x, "x", dt, (rows, cols)), None
    pdt = dt if gamma is None else _dtype(gamma, "gamma")
    if workspace is None and (dgamma is not None or dbeta is not None):
        workspace = _workspace(_layer_norm_bytes(rows, cols), dy.device, stream)
    pws, nws = _space(workspace, "gq_layer_norm_backward")
    _launch(lib().gq_layer_norm_backward, "gq_layer_norm_backward", stream,
            (dy, x, gamma, mean, rstd, dx, dgamma, dbeta, workspace), dt, pdt, rows, cols, pdy, sdy, px, sx, pk, _vector(gamma, "gamma", cols, pdt), _vector(mean, "mean", rows),
            _vector(rstd, "rstd", rows), pdx, sdx, _vector(dgamma, "dgamma", cols), _vector(dbeta, "dbeta", cols),
            int(bool(accumulate)), pws, nws)


def _format(fmt):
    f = FP8_FORMATS.get(fmt, fmt)
    if f not in (GQ_FP8_E4M3, GQ_FP8_E5M2):
        raise ValueError("fmt: one of %s expected, got %r" % (sorted(FP8_FORMATS), fmt))
    return f


@functools.lru_cache(maxsize=4096)
def _fp8_bytes(tile, rows, cols):
    return ((rows * ((cols + 127) // 128 * 128) + 15) // 16 * 16
            + (((rows + 127) // 128 if tile else rows) * ((cols + 511) // 512 * 4) + 15) // 16 * 16)


def _packed(t, what, tile, rows, cols):
    """Pointer of the packed form of rows x cols values (None: NULL)."""
    if t is None:
        return None
    need = _fp8_bytes(tile, rows, cols)
    if t.numel() < need or t.element_size() != 1 or t.dim() != 1 or not t.is_contiguous():
        raise ValueError("%s: a contiguous uint8 vector of at least %d bytes expected, got %s of shape %s"
                         % (what, need, t.dtype, tuple(t.shape)))
    return t.data_ptr()


def gq_fp8_layout(rows, cols, tile=False):
    """(bytes, codes_off, exps_off) of the packed form of rows x cols values."""
    b, c, e = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().gq_fp8_layout(int(bool(tile)), rows, cols, ctypes.byref(b), ctypes.byref(c), ctypes.byref(e)),
           "gq_fp8_layout")
    return b.value, c.value, e.value


def gq_fp8_pack(x, packed=None, packed_t=None, fmt="e4m3", tile=False, stream=None):
    """x (2-D) into packed (a uint8 vector) and its transpose into packed_t; either may be None.  fmt: "e4m3",
    "e5m2" or the C constant; tile: one exponent for 128 x 128 values instead of 128 of a row."""
    px, sx = _matrix(x, "x")
    rows, cols = x.shape
    tile = int(bool(tile))
    _launch(lib().gq_fp8_pack, "gq_fp8_pack", stream, (x, packed, packed_t), _dtype(x, "x"), _format(fmt), tile, rows,
            cols, px, sx, _packed(packed, "packed", tile, rows, cols), _packed(packed_t, "packed_t", tile, cols, rows))


def gq_fp8_unpack(packed, x, fmt="e4m3", tile=False, stream=None):
    px, sx = _matrix(x, "x")
    rows, cols = x.shape
    tile = int(bool(tile))
    _launch(lib().gq_fp8_unpack, "gq_fp8_unpack", stream, (x, packed), _dtype(x, "x"), _format(fmt), tile, rows, cols,
            _packed(packed, "packed", tile, rows, cols), px, sx)


@functools.lru_cache(maxsize=4096)
def _fp8_matmul_bytes(m, n, k):
    b = ctypes.c_size_t()
    _check(lib().gq_fp8_matmul_workspace(m, n, k, ctypes.byref(b)), "gq_fp8_matmul_workspace")
    return b.value


def gq_fp8_matmul_workspace(k, y):
    """A workspace tensor for gq_fp8_matmul over k columns into a tensor of y's size (None if it needs none)."""
    return _workspace(_fp8_matmul_bytes(y.shape[0], y.shape[1], k), y.device)


def gq_fp8_matmul(a, b, k, y, bias=None, fmt=("e4m3", "e4m3"), tile=(False, False), accumulate=False, workspace=None,
                  stream=None):
    """y (m, n) = a b^T + bias, a and b the packed forms of (m, k) and (n, k) values; fmt, tile: of a and of b.
    bias: a float32 vector.  Without a workspace one is allocated."""
    py, sy = _matrix(y, "y")
    m, n = y.shape
    ta, tb = int(bool(tile[0])), int(bool(tile[1]))
    if workspace is None:
        need = _fp8_matmul_bytes(m, n, k)
        if need:
            workspace = _workspace(need, y.device, stream)
    pws, nws = _space(workspace, "gq_fp8_matmul")
    _launch(lib().gq_fp8_matmul, "gq_fp8_matmul", stream, (y, a, b, bias, workspace), _dtype(y, "y"), m, n, k,
            _format(fmt[0]), ta, _packed(a, "a", ta, m, k), _format(fmt[1]), tb, _packed(b, "b", tb, n, k),
            _vector(bias, "bias", n), py, sy, int(bool(accumulate)), pws, nws)


def gq_adamw_layout(n):
    """(bytes, exps_off) of a moment of n elements in 8 bits."""
    b, e = ctypes.c_size_t(), ctypes.c_size_t()
    _check(lib().gq_adamw_layout(n, ctypes.byref(b), ctypes.byref(e)), "gq_adamw_layout")
    return b.value, e.value


class _AdamWHandle(ctypes.c_void_p):
    """A gq_adamw_t, with its device's index and the elements of all its tensors."""


def gq_adamw_create(params, grads, ms, vs, masters=None, weight_decay=0.0, lr_scale=1.0, state_bits=32, seed=0):
    """The optimizer of lists of contiguous tensors.  ms, vs: float32 tensors, or uint8 vectors of gq_adamw_layout
    bytes (state_bits = 8).  weight_decay, lr_scale: a number, or one for each tensor.  The tensors must outlive it."""
    count = len(params)
    lists = {"grads": grads, "ms": ms, "vs": vs, "masters": masters}
    for what, ts in lists.items():
        if ts is not None and len(ts) != count:
            raise ValueError("%s: %d tensors expected, got %d" % (what, count, len(ts)))
    per = {"weight_decay": weight_decay, "lr_scale": lr_scale}
    for what, v in per.items():
        per[what] = [float(v)] * count if isinstance(v, (int, float)) else [float(x) for x in v]
        if len(per[what]) != count:
            raise ValueError("%s: %d values expected, got %d" % (what, count, len(per[what])))
    device = params[0].device if count else None
    bits = int(state_bits)
    array = (gq_adamw_tensor_t * count)()
    total = 0
    for i in range(count):
        p, g, m, v = params[i], grads[i], ms[i], vs[i]
        x = masters[i] if masters is not None else None
        n = p.numel()
        total += n
        for what, t in (("params", p), ("grads", g), ("ms", m), ("vs", v), ("masters", x)):
            if t is None:
                continue
            if t.device != device or device.type != "cuda":
                raise ValueError("%s[%d]: CUDA tensors of one device expected, got %s" % (what, i, t.device))
            if not t.is_contiguous():
                raise ValueError("%s[%d]: a contiguous tensor expected, got strides %s" % (what, i, t.stride()))
        if _dtype(p, "params[%d]" % i) != _dtype(params[0], "params") or _dtype(g, "grads[%d]" % i) != _dtype(grads[0], "grads"):
            raise TypeError("tensor %d: its type differs from the first one's" % i)
        if g.numel() != n or (x is not None and (x.numel() != n or _dtype(x, "masters[%d]" % i) != GQ_FLOAT32)):
            raise ValueError("tensor %d: a gradient (and float32 master copy) of %d values expected" % (i, n))
        for what, t in (("ms", m), ("vs", v)):
            if bits == 8:
                if t.element_size() != 1 or t.numel() < gq_adamw_layout(n)[0]:
                    raise ValueError("%s[%d]: a uint8 vector of %d bytes expected" % (what, i, gq_adamw_layout(n)[0]))
            elif t.numel() != n or _dtype(t, "%s[%d]" % (what, i)) != GQ_FLOAT32:
                raise ValueError("%s[%d]: %d float32 values expected" % (what, i, n))
        ptr = [t.data_ptr() if t is not None else None for t in (p, g, x, m, v)]
        array[i] = gq_adamw_tensor_t(*ptr, n, per["weight_decay"][i], per["lr_scale"][i])
    cfg = gq_adamw_config_t(_dtype(params[0], "params") if count else GQ_FLOAT32,
                            _dtype(grads[0], "grads") if count else GQ_FLOAT32, bits, int(seed))
    if _torch is None:
        _setup()
    h = _AdamWHandle()
    h.device = device.index if count else _torch.cuda.current_device()
    h.total = total
    with _torch.cuda.device(h.device):
        _check(lib().gq_adamw_create(ctypes.byref(cfg), array, count, ctypes.byref(h)), "gq_adamw_create")
    return h


def gq_adamw_destroy(opt):
    _check(lib().gq_adamw_destroy(opt), "gq_adamw_destroy")


def _adamw_call(fn, what, opt, stream, tensors, *args):
    dev = opt.device
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError("%s: tensors on cuda:%d expected, got %s" % (what, dev, t.device))
    if stream is None:
        stream = _current_stream(dev)
    elif not isinstance(stream, int):
        stream = stream.cuda_stream
    if _current_device() == dev:
        st = fn(opt, *args, stream)
    else:
        with _torch.cuda.device(dev):
            st = fn(opt, *args, stream)
    if st != GQ_OK:
        raise GQError(st, what)


def gq_adamw_norm(opt, max_norm, out, stream=None):
    """out: two float32 values, the gradients' norm and the clipping factor."""
    _adamw_call(lib().gq_adamw_norm, "gq_adamw_norm", opt, stream, (out,), float(max_norm), _vector(out, "out", 2))


def gq_adamw_scalars(lr, beta1, beta2, step):
    """The 16 bytes that a step reads from device memory in the place of lr and step (a CPU uint8 tensor)."""
    import torch
    s = gq_adamw_scalars_t()
    _check(lib().gq_adamw_scalars(float(lr), float(beta1), float(beta2), int(step), ctypes.byref(s)), "gq_adamw_scalars")
    return torch.frombuffer(bytearray(bytes(s)), dtype=torch.uint8)


def gq_adamw_step(opt, lr, beta1, beta2, eps, step, scale=None, scalars=None, stream=None):
    """scale: one float32 value that multiplies the gradients; scalars: 16 bytes (gq_adamw_scalars), both on the device."""
    if scalars is not None and (scalars.numel() * scalars.element_size() != 16 or not scalars.is_contiguous()):
        raise ValueError("scalars: 16 contiguous bytes expected, got shape %s of %s" % (tuple(scalars.shape), scalars.dtype))
    if scale is not None and (scale.numel() != 1 or _dtype(scale, "scale") != GQ_FLOAT32):
        raise ValueError("scale: one float32 value expected, got shape %s of %s" % (tuple(scale.shape), scale.dtype))
    _adamw_call(lib().gq_adamw_step, "gq_adamw_step", opt, stream, (scale, scalars), float(lr), float(beta1), float(beta2),
                float(eps), int(step), _ptr(scale), _ptr(scalars))


def gq_adamw_moments(opt, m=None, v=None, stream=None):
    """The moments' values, all tensors one after another, into vectors of one type (either may be None)."""
    some = m if m is not None else v
    if some is None:
        raise ValueError("gq_adamw_moments: at least one of m and v expected")
    dt = _dtype(some, "m")
    _adamw_call(lib().gq_adamw_moments, "gq_adamw_moments", opt, stream, (m, v), dt, _vector(m, "m", opt.total, dt),
                _vector(v, "v", opt.total, dt))


class AdamW:
    """Owner of a gq_adamw_t and of references to its tensors (destroyed on close / exit of a ``with`` block)."""

    def __init__(self, params, grads, ms, vs, masters=None, weight_decay=0.0, lr_scale=1.0, state_bits=32, seed=0):
        self.handle = None
        self.tensors = (list(params), list(grads), list(ms), list(vs), None if masters is None else list(masters))
        self.handle = gq_adamw_create(*self.tensors, weight_decay, lr_scale, state_bits, seed)

    def norm(self, max_norm, out, stream=None):
        gq_adamw_norm(self.handle, max_norm, out, stream)

    def step(self, lr, beta1, beta2, eps, step, scale=None, scalars=None, stream=None):
        gq_adamw_step(self.handle, lr, beta1, beta2, eps, step, scale, scalars, stream)

    def moments(self, m=None, v=None, stream=None):
        gq_adamw_moments(self.handle, m, v, stream)

    def close(self):
        if self.handle:
            gq_adamw_destroy(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def gq_status_string(status):
    return lib().gq_status_string(status).decode()


def gq_version():
    return lib().gq_version().decode()


class Plan:
    """Owner of a gq_plan_t (destroyed on close / exit of a ``with`` block)."""

    def __init__(self, cfg, segments=None, fmt=GQ_FORMAT_DENSE):
        """segments: the tensors' offsets (nseg + 1 values) for GQ_TERNGRAD_LAYER; fmt: the
        message format (GQ_FORMAT_BASE_S: base-s messages written and read directly)."""
        self.cfg = cfg
        self.handle = gq_plan_create(cfg)
        if segments is not None:
            gq_plan_set_segments(self.handle, segments)
        if fmt != GQ_FORMAT_DENSE:
            gq_plan_set_format(self.handle, fmt)
        if cfg.scheme == GQ_TERNGRAD_LAYER and segments is None:
            self.msg_bytes = self.codes_off = self.levels_off = None
        else:
            self.msg_bytes, self.codes_off, self.levels_off = gq_plan_message_layout(self.handle)

    def close(self):
        if self.handle:
            gq_plan_destroy(self.handle)
            self.handle = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
