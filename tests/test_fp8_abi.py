"""The entry points on packed matrices of 8-bit floating point without a GPU: layout, workspace sizes and every
refusal.  Refused calls return before anything is enqueued, so made-up addresses are safe."""
import ctypes

import pytest
import torch

import fp8_oracle as O
import gradient_quantization_communication_b200.gq as G

P = 1 << 40     # made-up, 16-byte aligned addresses, far apart
FAR = 1 << 36
BF16, F32, F16 = G.GQ_BFLOAT16, G.GQ_FLOAT32, G.GQ_FLOAT16


@pytest.mark.parametrize("tile", [0, 1])
@pytest.mark.parametrize("rows,cols", [(0, 1), (1, 1), (3, 127), (3, 128), (3, 129), (128, 512), (129, 513), (1000, 4097),
                                       (2 ** 31 - 1, 1 << 24)])
def test_layout(tile, rows, cols):
    size, off = O.layout(tile, rows, cols)
    assert G.gq_fp8_layout(rows, cols, tile) == (size, 0, off)
    assert G._fp8_bytes(tile, rows, cols) == size


@pytest.mark.parametrize("rows,cols", [(-1, 8), (2 ** 31, 8), (8, 0), (8, -3), (8, (1 << 24) + 1)])
def test_sizes_refused(rows, cols):
    with pytest.raises(G.GQError) as e:
        G.gq_fp8_layout(rows, cols)
    assert e.value.status == G.GQ_ERR_INVALID
    assert G.lib().gq_fp8_layout(2, 8, 8, None, None, None) == G.GQ_ERR_INVALID
    b = ctypes.c_size_t()
    assert G.lib().gq_fp8_matmul_workspace(rows, 8, cols, ctypes.byref(b)) == G.GQ_ERR_INVALID
    assert G.lib().gq_fp8_matmul_workspace(8, rows, cols, ctypes.byref(b)) == G.GQ_ERR_INVALID


@pytest.mark.parametrize("m", [0, 1, 16, 33, 128, 8192, 2 ** 31 - 1])
@pytest.mark.parametrize("n,k", [(1, 1), (256, 256), (257, 129), (4096, 4096), (1 << 24, 1 << 24)])
def test_matmul_workspace(m, n, k):
    b = ctypes.c_size_t(123)
    assert G.lib().gq_fp8_matmul_workspace(m, n, k, ctypes.byref(b)) == G.GQ_OK
    assert 0 <= b.value < 1 << 34
    assert G.lib().gq_fp8_matmul_workspace(m, 0, k, ctypes.byref(b)) == G.GQ_ERR_INVALID
    assert G.lib().gq_fp8_matmul_workspace(m, n, k, None) == G.GQ_ERR_INVALID


CALLS = {
    "gq_fp8_pack": dict(dtype=BF16, format=0, tile=0, rows=4, cols=40, x=P, x_stride=40, packed=P + FAR,
                        packed_t=P + 2 * FAR, stream=None),
    "gq_fp8_unpack": dict(dtype=BF16, format=0, tile=0, rows=4, cols=40, packed=P, x=P + FAR, x_stride=40, stream=None),
    "gq_fp8_matmul": dict(dtype=F32, m=40, n=24, k=300, format_a=0, tile_a=0, a=P, format_b=0, tile_b=1, b=P + FAR,
                          bias=P + 2 * FAR, y=P + 3 * FAR, y_stride=24, accumulate=0, workspace=P + 4 * FAR,
                          workspace_bytes=1 << 30, stream=None),
}
REFUSED = [
    ("gq_fp8_pack", dict(dtype=3)), ("gq_fp8_pack", dict(dtype=-1)), ("gq_fp8_pack", dict(format=2)),
    ("gq_fp8_pack", dict(format=-1)), ("gq_fp8_pack", dict(tile=2)), ("gq_fp8_pack", dict(rows=-1)),
    ("gq_fp8_pack", dict(cols=0)), ("gq_fp8_pack", dict(x=None)), ("gq_fp8_pack", dict(packed=None, packed_t=None)),
    ("gq_fp8_pack", dict(x=P + 2)), ("gq_fp8_pack", dict(packed=P + FAR + 8)), ("gq_fp8_pack", dict(packed_t=P + 2 * FAR + 4)),
    ("gq_fp8_pack", dict(x_stride=-40)), ("gq_fp8_pack", dict(packed=P)), ("gq_fp8_pack", dict(packed_t=P + 304)),
    ("gq_fp8_pack", dict(packed_t=P + FAR + 512)), ("gq_fp8_pack", dict(rows=(1 << 24) + 1)),
    ("gq_fp8_pack", dict(rows=0, packed_t=P)),
    ("gq_fp8_unpack", dict(x_stride=39)), ("gq_fp8_unpack", dict(x_stride=0)), ("gq_fp8_unpack", dict(x=P)),
    ("gq_fp8_unpack", dict(x=None)), ("gq_fp8_unpack", dict(packed=None)), ("gq_fp8_unpack", dict(dtype=7)),
    ("gq_fp8_unpack", dict(tile=-1)), ("gq_fp8_unpack", dict(format=5)), ("gq_fp8_unpack", dict(packed=P + 8)),
    ("gq_fp8_matmul", dict(dtype=3)), ("gq_fp8_matmul", dict(m=-1)), ("gq_fp8_matmul", dict(n=0)),
    ("gq_fp8_matmul", dict(k=0)), ("gq_fp8_matmul", dict(k=(1 << 24) + 1)), ("gq_fp8_matmul", dict(m=1 << 31)),
    ("gq_fp8_matmul", dict(format_a=2)), ("gq_fp8_matmul", dict(format_b=-1)), ("gq_fp8_matmul", dict(tile_a=3)),
    ("gq_fp8_matmul", dict(tile_b=2)), ("gq_fp8_matmul", dict(a=None)), ("gq_fp8_matmul", dict(b=None)),
    ("gq_fp8_matmul", dict(y=None)), ("gq_fp8_matmul", dict(a=P + 8)), ("gq_fp8_matmul", dict(b=P + FAR + 1)),
    ("gq_fp8_matmul", dict(bias=P + 2 * FAR + 2)), ("gq_fp8_matmul", dict(y=P + 3 * FAR + 2)),
    ("gq_fp8_matmul", dict(y_stride=23)), ("gq_fp8_matmul", dict(y_stride=-24)), ("gq_fp8_matmul", dict(accumulate=2)),
    ("gq_fp8_matmul", dict(y=P)), ("gq_fp8_matmul", dict(y=P + FAR)), ("gq_fp8_matmul", dict(y=P + 2 * FAR)),
]


@pytest.mark.parametrize("name,change", REFUSED)
def test_refused(name, change):
    args = dict(CALLS[name])
    assert set(change) <= set(args)
    args.update(change)
    assert getattr(G.lib(), name)(*args.values()) == G.GQ_ERR_INVALID


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_adding_to_16_bits_is_unsupported(dtype):
    args = dict(CALLS["gq_fp8_matmul"], dtype=dtype, accumulate=1)
    assert G.lib().gq_fp8_matmul(*args.values()) == G.GQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("name,change", [("gq_fp8_pack", dict(rows=0, packed_t=None)), ("gq_fp8_unpack", dict(rows=0)),
                                         ("gq_fp8_matmul", dict(m=0))])
def test_nothing_to_do(name, change):
    args = dict(CALLS[name], **change)
    args.update({k: None for k in ("x", "packed", "a", "b", "y") if k in args})
    assert getattr(G.lib(), name)(*args.values()) == G.GQ_OK


def test_binding_refuses_what_it_can_see():
    x = torch.zeros(4, 40)
    buf = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError):
        G.gq_fp8_pack(x.t(), buf)                       # columns not adjacent
    with pytest.raises(TypeError):
        G.gq_fp8_pack(x.double(), buf)
    with pytest.raises(ValueError):
        G.gq_fp8_pack(x, buf[:100])                     # too small
    with pytest.raises(ValueError):
        G.gq_fp8_pack(x, buf, fmt="e3m4")
    with pytest.raises(ValueError):
        G.gq_fp8_pack(x, buf)                           # not on a GPU
    with pytest.raises(ValueError):
        G.gq_fp8_matmul(buf, buf, 40, torch.zeros(4, 4), bias=torch.zeros(5))
    with pytest.raises(ValueError):
        G.gq_fp8_matmul(buf[:64], buf, 40, torch.zeros(4, 4))
