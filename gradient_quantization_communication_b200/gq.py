"""Python binding of the C ABI in ``include/gq.h`` (``libgq.so``): argument marshalling only.

Every function keeps the C name.  Tensors are passed as ``data_ptr()``; the stream defaults to
torch's current CUDA stream.  There is no fallback: if ``libgq.so`` is missing the import of the
library fails with an error that says how to build it.
"""
import ctypes
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
FUNCTIONS = {"gelu": GQ_FN_GELU, "gelu_tanh": GQ_FN_GELU_TANH, "silu": GQ_FN_SILU}


class gq_config_t(ctypes.Structure):
    _fields_ = [("scheme", ctypes.c_int32), ("levels", ctypes.c_int32), ("bucket", ctypes.c_int32),
                ("workers", ctypes.c_int32), ("error_feedback", ctypes.c_int32),
                ("clip_sigma", ctypes.c_float), ("seed", ctypes.c_uint64), ("n", ctypes.c_int64)]


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
                  "gq_layer_norm_forward", "gq_layer_norm_workspace", "gq_layer_norm_backward"):
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
_torch = _dtypes = _current_stream = None


def _setup():
    """torch, looked up once: it is imported by the first call that takes tensors."""
    global _torch, _dtypes, _current_stream
    import torch
    _dtypes = {torch.float32: GQ_FLOAT32, torch.bfloat16: GQ_BFLOAT16, torch.float16: GQ_FLOAT16}
    # the handle itself where torch offers it: building a Stream object around it takes a microsecond
    _current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                              lambda dev: torch.cuda.current_stream(dev).cuda_stream)
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
    if _torch.cuda.current_device() == dev:
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
