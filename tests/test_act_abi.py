"""The activation checkpoints' and layer norm's entry points without a GPU: layout, workspace sizes and
every refusal.  Refused calls return before anything is enqueued, so made-up addresses are safe."""
import ctypes

import pytest
import torch

import act_oracle as A
import gradient_quantization_communication_b200.gq as G

P = 1 << 40     # made-up, 16-byte aligned addresses, far apart
FAR = 1 << 36
BF16, F32, F16 = G.GQ_BFLOAT16, G.GQ_FLOAT32, G.GQ_FLOAT16


@pytest.mark.parametrize("rows,cols", [(0, 1), (1, 1), (3, 31), (3, 32), (3, 33), (5, 128), (7, 129), (1000, 4097),
                                       (2 ** 31 - 1, 1 << 24)])
def test_layout(rows, cols):
    size, off = A.layout(rows, cols)
    assert G.gq_act_layout(rows, cols) == (size, 0, off)


@pytest.mark.parametrize("rows,cols", [(-1, 8), (2 ** 31, 8), (8, 0), (8, -3), (8, (1 << 24) + 1)])
def test_sizes_refused(rows, cols):
    with pytest.raises(G.GQError) as e:
        G.gq_act_layout(rows, cols)
    assert e.value.status == G.GQ_ERR_INVALID
    b = ctypes.c_size_t()
    assert G.lib().gq_layer_norm_workspace(rows, cols, ctypes.byref(b)) == G.GQ_ERR_INVALID
    assert G.lib().gq_act_weight_grad_workspace(BF16, rows, cols, 8, 8, 1, ctypes.byref(b)) == G.GQ_ERR_INVALID
    assert G.lib().gq_act_weight_grad_workspace(BF16, rows, 8, cols, 8, 1, ctypes.byref(b)) == G.GQ_ERR_INVALID


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("tokens", [0, 1, 32, 33, 64, 65, 4096, 100000, 2 ** 31 - 1])
@pytest.mark.parametrize("cin,cout", [(1, 1), (256, 256), (257, 8), (1000, 2499), (4096, 16384), (1 << 24, 1 << 24)])
def test_weight_grad_workspace(dtype, tokens, cin, cout):
    """The workspace's size is worked out for every size, never negative, larger by the bias's partial rows
    with a bias, and 0 without tokens."""
    sizes = []
    for bias in (0, 1):
        b = ctypes.c_size_t(123)
        assert G.lib().gq_act_weight_grad_workspace(dtype, tokens, cin, cout, (cout + 7) // 8 * 8, bias,
                                                    ctypes.byref(b)) == G.GQ_OK
        sizes.append(b.value)
    assert 0 <= sizes[0] <= sizes[1] < 1 << 62
    if tokens == 0:
        assert sizes == [0, 0]
    if dtype == F32 and tokens > 32:   # three bf16 planes of dy
        assert sizes[0] >= 6 * tokens * cout


CALLS = {
    # name: (arguments in order, keyword -> position of each)
    "gq_act_pack": dict(dtype=BF16, rows=4, cols=40, x=P, x_stride=40, ckpt=P + FAR, stream=None),
    "gq_act_unpack": dict(dtype=BF16, rows=4, cols=40, ckpt=P, x=P + FAR, x_stride=40, stream=None),
    "gq_act_fn_forward": dict(kind=0, dtype=BF16, rows=4, cols=40, x=P, x_stride=40, y=P + FAR, y_stride=40,
                              ckpt=P + 2 * FAR, stream=None),
    "gq_act_fn_backward": dict(kind=0, dtype=BF16, rows=4, cols=40, ckpt=P, dy=P + FAR, dy_stride=40, dx=P + 2 * FAR,
                               dx_stride=40, stream=None),
    "gq_act_weight_grad": dict(dtype=F32, tokens=64, cin=40, cout=24, ckpt=P, dy=P + FAR, dy_stride=24, dw=P + 2 * FAR,
                               dw_stride=40, db=P + 3 * FAR, accumulate=0, workspace=P + 4 * FAR,
                               workspace_bytes=1 << 30, stream=None),
    "gq_layer_norm_forward": dict(dtype=BF16, param_dtype=F32, rows=4, cols=40, x=P, x_stride=40, gamma=P + FAR,
                                  beta=P + 2 * FAR, eps=1e-5, y=P + 3 * FAR, y_stride=40, mean=P + 4 * FAR,
                                  rstd=P + 5 * FAR, ckpt=P + 6 * FAR, stream=None),
    "gq_layer_norm_backward": dict(dtype=BF16, param_dtype=F32, rows=4, cols=40, dy=P, dy_stride=40, x=P + FAR,
                                   x_stride=40, ckpt=None, gamma=P + 2 * FAR, mean=P + 3 * FAR, rstd=P + 4 * FAR,
                                   dx=P + 5 * FAR, dx_stride=40, dgamma=P + 6 * FAR, dbeta=P + 7 * FAR, accumulate=0,
                                   workspace=P + 8 * FAR, workspace_bytes=1 << 30, stream=None),
}

REFUSED = [
    ("gq_act_pack", dict(dtype=3)), ("gq_act_pack", dict(dtype=-1)), ("gq_act_pack", dict(rows=-1)),
    ("gq_act_pack", dict(cols=0)), ("gq_act_pack", dict(x=None)), ("gq_act_pack", dict(ckpt=None)),
    ("gq_act_pack", dict(x=P + 2)), ("gq_act_pack", dict(ckpt=P + FAR + 8)), ("gq_act_pack", dict(x_stride=-40)),
    ("gq_act_pack", dict(ckpt=P)), ("gq_act_pack", dict(ckpt=P + 304)),
    ("gq_act_unpack", dict(x_stride=39)), ("gq_act_unpack", dict(x_stride=0)), ("gq_act_unpack", dict(x=P)),
    ("gq_act_unpack", dict(x=None)), ("gq_act_unpack", dict(ckpt=None)), ("gq_act_unpack", dict(dtype=7)),
    ("gq_act_fn_forward", dict(kind=-1)), ("gq_act_fn_forward", dict(kind=3)), ("gq_act_fn_forward", dict(y=P)),
    ("gq_act_fn_forward", dict(ckpt=P)), ("gq_act_fn_forward", dict(ckpt=P + FAR)), ("gq_act_fn_forward", dict(y=None)),
    ("gq_act_fn_forward", dict(y_stride=8)), ("gq_act_fn_forward", dict(y=P + FAR + 4)),
    ("gq_act_fn_forward", dict(x_stride=64, y=P + 48, y_stride=64)),    # the rows' last 16 columns overlap
    ("gq_act_fn_forward", dict(x_stride=96, y=P + 80, y_stride=88)),    # strides differ: their extents overlap
    ("gq_act_fn_backward", dict(kind=3)), ("gq_act_fn_backward", dict(dx=P + FAR)), ("gq_act_fn_backward", dict(dx=P)),
    ("gq_act_fn_backward", dict(ckpt=None)), ("gq_act_fn_backward", dict(dy=None)),
    ("gq_act_fn_backward", dict(dx_stride=1)),
    ("gq_act_weight_grad", dict(dtype=3)), ("gq_act_weight_grad", dict(tokens=-1)), ("gq_act_weight_grad", dict(cin=0)),
    ("gq_act_weight_grad", dict(cout=0)), ("gq_act_weight_grad", dict(ckpt=None)), ("gq_act_weight_grad", dict(dy=None)),
    ("gq_act_weight_grad", dict(dw=None)), ("gq_act_weight_grad", dict(dw=P + 2 * FAR + 2)),
    ("gq_act_weight_grad", dict(db=P + 3 * FAR + 1)), ("gq_act_weight_grad", dict(dw_stride=39)),
    ("gq_act_weight_grad", dict(dy=P + FAR + 8)), ("gq_act_weight_grad", dict(accumulate=2)),
    ("gq_act_weight_grad", dict(workspace=None)), ("gq_act_weight_grad", dict(workspace_bytes=8)),
    ("gq_act_weight_grad", dict(workspace=P + 4 * FAR + 4)), ("gq_act_weight_grad", dict(db=P + 2 * FAR + 400)),
    ("gq_act_weight_grad", dict(workspace=P)), ("gq_act_weight_grad", dict(dw=P + FAR)),
    ("gq_layer_norm_forward", dict(param_dtype=F16)), ("gq_layer_norm_forward", dict(param_dtype=5)),
    ("gq_layer_norm_forward", dict(eps=-1e-5)), ("gq_layer_norm_forward", dict(eps=float("nan"))),
    ("gq_layer_norm_forward", dict(eps=float("inf"))), ("gq_layer_norm_forward", dict(mean=None)),
    ("gq_layer_norm_forward", dict(rstd=None)), ("gq_layer_norm_forward", dict(mean=P + 4 * FAR + 2)),
    ("gq_layer_norm_forward", dict(gamma=P + FAR + 2)), ("gq_layer_norm_forward", dict(beta=P + 2 * FAR + 1)),
    ("gq_layer_norm_forward", dict(y=P)), ("gq_layer_norm_forward", dict(rstd=P + 4 * FAR + 12)),
    ("gq_layer_norm_forward", dict(ckpt=P + 6 * FAR + 4)), ("gq_layer_norm_forward", dict(y=P + FAR + 16)),
    ("gq_layer_norm_backward", dict(ckpt=P + 9 * FAR)), ("gq_layer_norm_backward", dict(x=None)),
    ("gq_layer_norm_backward", dict(x=None, ckpt=P + 9 * FAR + 4)), ("gq_layer_norm_backward", dict(dx=P)),
    ("gq_layer_norm_backward", dict(dx_stride=0)), ("gq_layer_norm_backward", dict(mean=None)),
    ("gq_layer_norm_backward", dict(rstd=None)), ("gq_layer_norm_backward", dict(param_dtype=F16)),
    ("gq_layer_norm_backward", dict(accumulate=-1)), ("gq_layer_norm_backward", dict(workspace=None)),
    ("gq_layer_norm_backward", dict(workspace_bytes=100)), ("gq_layer_norm_backward", dict(workspace=P + 8 * FAR + 8)),
    ("gq_layer_norm_backward", dict(dbeta=P + 6 * FAR + 156)), ("gq_layer_norm_backward", dict(dgamma=P + 6 * FAR + 3)),
    ("gq_layer_norm_backward", dict(dgamma=P + 2 * FAR)), ("gq_layer_norm_backward", dict(workspace=P + 5 * FAR)),
]


@pytest.mark.parametrize("name,change", REFUSED)
def test_refused(name, change):
    args = dict(CALLS[name])
    assert set(change) <= set(args)
    args.update(change)
    assert getattr(G.lib(), name)(*args.values()) == G.GQ_ERR_INVALID


@pytest.mark.parametrize("name", [n for n in CALLS if n not in ("gq_act_weight_grad", "gq_layer_norm_backward")])
def test_no_rows_is_a_no_op(name):
    args = {k: None if isinstance(v, int) and v >= P else v for k, v in CALLS[name].items()}
    args["rows"] = 0
    assert getattr(G.lib(), name)(*args.values()) == G.GQ_OK


# ------------------------------------------------------------------------------------------------
# the binding's own checks
# ------------------------------------------------------------------------------------------------
def _u8(n):
    return torch.zeros(n, dtype=torch.uint8)


def test_binding_refuses_cpu_tensors():
    x, ck = torch.zeros(4, 40), _u8(1024)
    for call in (lambda: G.gq_act_pack(x, ck), lambda: G.gq_act_unpack(ck, x), lambda: G.gq_act_fn_forward("gelu", x, x),
                 lambda: G.gq_act_fn_backward("gelu", ck, x, x),
                 lambda: G.gq_act_weight_grad(ck, x, torch.zeros(40, 40)),
                 lambda: G.gq_layer_norm_forward(x, None, None, 1e-5, x, torch.zeros(4), torch.zeros(4)),
                 lambda: G.gq_layer_norm_backward(x, x, None, torch.zeros(4), torch.zeros(4), x, None, None)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


def test_binding_refuses_types_and_shapes():
    x, ck = torch.zeros(4, 40), _u8(1024)
    m = torch.zeros(4)
    bad = [
        (TypeError, lambda: G.gq_act_pack(x.double(), ck)),
        (TypeError, lambda: G.gq_act_pack(x.int(), ck)),
        (ValueError, lambda: G.gq_act_pack(x[0], ck)),
        (ValueError, lambda: G.gq_act_pack(x.t(), ck)),
        (ValueError, lambda: G.gq_act_pack(x[:, ::2], ck)),
        (ValueError, lambda: G.gq_act_pack(x, _u8(G.gq_act_layout(4, 40)[0] - 1))),
        (ValueError, lambda: G.gq_act_pack(x, _u8(2048)[::2])),
        (ValueError, lambda: G.gq_act_pack(x, torch.zeros(1024))),
        (TypeError, lambda: G.gq_act_fn_forward("gelu", x, x.half())),
        (ValueError, lambda: G.gq_act_fn_forward("gelu", x, torch.zeros(4, 41))),
        (ValueError, lambda: G.gq_act_fn_backward("gelu", _u8(8), x, x.clone())),
        (ValueError, lambda: G.gq_act_fn_forward("relu", x, x.clone())),
        (ValueError, lambda: G.gq_act_fn_backward("relu", ck, x, x.clone())),
        (ValueError, lambda: G.gq_act_weight_grad(ck, x, torch.zeros(39, 40))),
        (TypeError, lambda: G.gq_act_weight_grad(ck, x, torch.zeros(40, 40).bfloat16())),
        (ValueError, lambda: G.gq_act_weight_grad(ck, x, torch.zeros(40, 40), torch.zeros(39))),
        (TypeError, lambda: G.gq_layer_norm_forward(x.half(), torch.zeros(40).half(), torch.zeros(40), 1e-5, x.half(), m, m)),
        (ValueError, lambda: G.gq_layer_norm_forward(x, torch.zeros(41), None, 1e-5, x, m, m)),
        (ValueError, lambda: G.gq_layer_norm_forward(x, None, None, 1e-5, x, torch.zeros(5), m)),
        (TypeError, lambda: G.gq_layer_norm_forward(x, None, None, 1e-5, x, m.half(), m)),
        (ValueError, lambda: G.gq_layer_norm_backward(x, x, None, m, m, torch.zeros(4, 39), None, None)),
        (ValueError, lambda: G.gq_layer_norm_backward(x, _u8(100), None, m, m, x.clone(), None, None)),
    ]
    for i, (err, call) in enumerate(bad):
        with pytest.raises(err):
            call()
            raise AssertionError(i)
