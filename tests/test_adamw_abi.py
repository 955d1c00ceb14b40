"""AdamW's entry points without a GPU: the 8-bit moments' layout, the scalars and every refusal.  Refused calls return
before anything is allocated or enqueued, so made-up addresses are safe."""
import ctypes
import math
import struct

import numpy as np
import pytest
import torch

import fp8_oracle as O
import gradient_quantization_communication_b200.gq as G

P = 1 << 40
FAR = 1 << 32
BF16, F32, F16 = G.GQ_BFLOAT16, G.GQ_FLOAT32, G.GQ_FLOAT16


@pytest.mark.parametrize("n", [0, 1, 127, 128, 129, 2048, 2049, 10 ** 6, 2 ** 40 - 1])
def test_layout(n):
    assert G.gq_adamw_layout(n) == O.adam_layout(n)


@pytest.mark.parametrize("n", [-1, 1 << 40])
def test_layout_refused(n):
    with pytest.raises(G.GQError):
        G.gq_adamw_layout(n)


def tensors(count=3, n=1000, eight=False, **change):
    out = (G.gq_adamw_tensor_t * count)()
    for i in range(count):
        at = P + i * 16 * FAR
        t = dict(param=at, grad=at + FAR, master=None, m=at + 2 * FAR, v=at + 3 * FAR, n=n, weight_decay=0.1, lr_scale=1.0)
        if i == count - 1:
            t.update(change)
        out[i] = G.gq_adamw_tensor_t(*t.values())
    return out


def create(cfg=(F32, F32, 32, 1), array=None, count=3):
    h = ctypes.c_void_p(7)
    c = G.gq_adamw_config_t(*cfg)
    array = tensors() if array is None else array
    st = G.lib().gq_adamw_create(ctypes.byref(c), array, count, ctypes.byref(h))
    assert not h.value
    return st


@pytest.mark.parametrize("cfg", [(3, F32, 32, 1), (-1, F32, 32, 1), (F32, 5, 32, 1), (F32, F32, 16, 1), (F32, F32, 0, 1)])
def test_config_refused(cfg):
    assert create(cfg) == G.GQ_ERR_INVALID


@pytest.mark.parametrize("change", [
    dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(param=P + 2), dict(grad=P + 40 * FAR + 1),
    dict(m=P + 50 * FAR + 2), dict(v=P + 50 * FAR + 3), dict(n=-1), dict(n=1 << 40), dict(weight_decay=-0.1),
    dict(weight_decay=float("nan")), dict(weight_decay=float("inf")), dict(lr_scale=-1.0), dict(lr_scale=float("inf")),
    dict(master=P + 60 * FAR),                                  # of float32 parameters
    dict(param=P), dict(m=P), dict(v=P + 2 * FAR + 3996),       # another tensor's memory
    dict(grad=P), dict(m=P + 33 * FAR), dict(v=P + 34 * FAR),   # its own or another's
])
def test_tensors_refused(change):
    assert create(array=tensors(**change)) == G.GQ_ERR_INVALID


@pytest.mark.parametrize("change", [dict(m=P + 50 * FAR + 4), dict(v=P + 50 * FAR + 8), dict(v=P + 34 * FAR + 1024)])
def test_moments_in_8_bits_refused(change):
    assert create((F32, F32, 8, 1), tensors(**change)) == G.GQ_ERR_INVALID


def test_masters_of_all_or_none():
    assert create((BF16, F32, 32, 1), tensors(master=P + 60 * FAR)) == G.GQ_ERR_INVALID


@pytest.mark.parametrize("count", [-1, (1 << 20) + 1])
def test_count_refused(count):
    assert create(count=count) == G.GQ_ERR_INVALID


def test_null_refused():
    c, h = G.gq_adamw_config_t(F32, F32, 32, 1), ctypes.c_void_p()
    assert G.lib().gq_adamw_create(None, tensors(), 3, ctypes.byref(h)) == G.GQ_ERR_INVALID
    assert G.lib().gq_adamw_create(ctypes.byref(c), None, 3, ctypes.byref(h)) == G.GQ_ERR_INVALID
    assert G.lib().gq_adamw_create(ctypes.byref(c), tensors(), 3, None) == G.GQ_ERR_INVALID
    assert G.lib().gq_adamw_destroy(None) == G.GQ_ERR_INVALID
    assert G.lib().gq_adamw_norm(None, 1.0, P, None) == G.GQ_ERR_INVALID
    assert G.lib().gq_adamw_step(None, 1e-3, 0.9, 0.999, 1e-8, 1, None, None, None) == G.GQ_ERR_INVALID
    assert G.lib().gq_adamw_moments(None, F32, P, None, None) == G.GQ_ERR_INVALID


@pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses would be accepted")
@pytest.mark.parametrize("array", [
    tensors(), tensors(grad=P + FAR),                           # shared gradients
    tensors(n=0), tensors(n=1000, param=P + 4000),              # adjacent
])
def test_accepted_without_a_device(array):
    """What passes the checks reaches the allocation, which fails here."""
    assert create(array=array) == G.GQ_ERR_CUDA


@pytest.mark.parametrize("step", [1, 2, 100, 10 ** 6, 2 ** 32 - 1])
@pytest.mark.parametrize("lr,beta1,beta2", [(1e-3, 0.9, 0.999), (0.0, 0.0, 0.0), (3e-4, 0.95, 0.99999999)])
def test_scalars(lr, beta1, beta2, step):
    got = struct.unpack("fffI", G.gq_adamw_scalars(lr, beta1, beta2, step).numpy().tobytes())
    want = (np.float32(lr), np.float32(1 / (1 - beta1 ** step)), np.float32(1 / math.sqrt(1 - beta2 ** step)), step)
    assert got == want


@pytest.mark.parametrize("args", [(-1e-3, 0.9, 0.999, 1), (float("nan"), 0.9, 0.999, 1), (float("inf"), 0.9, 0.999, 1),
                                  (1e-3, 1.0, 0.999, 1), (1e-3, -0.1, 0.999, 1), (1e-3, 0.9, 1.0, 1),
                                  (1e-3, 0.9, float("nan"), 1), (1e-3, 0.9, 0.999, 0), (1e-3, 0.9, 0.999, 2 ** 32)])
def test_scalars_refused(args):
    with pytest.raises(G.GQError) as e:
        G.gq_adamw_scalars(*args)
    assert e.value.status == G.GQ_ERR_INVALID


def test_philox_is_the_published_one():
    """The oracle's generator against the known-answer vectors of the quantizer's."""
    import os
    path = os.path.join(os.path.dirname(__file__), "golden", "philox4x32_10_kat.txt")
    lines = [ln.split() for ln in open(path) if ln.strip() and not ln.startswith("#")]
    assert lines
    for ln in lines:
        w = [int(x, 16) for x in ln if len(x) == 8 or x.startswith("0x")][-10:]
        ctr, key, out = w[:4], w[4:6], w[6:10]
        got = [int(x[0]) for x in O.philox([np.array([c]) for c in ctr], key[0] | key[1] << 32)]
        assert got == out
