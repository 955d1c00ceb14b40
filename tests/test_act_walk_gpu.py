"""Tensors of many rows, each cut into several pieces, more of them than the device holds at once: every warp
of the pack, unpack and activation-function kernels then walks on from piece to piece and from row to row.
Outputs are filled with what no piece writes beforehand, and every element is compared, in 64 bits on the GPU."""
import numpy as np
import pytest
import torch

import act_oracle as A
import gradient_quantization_communication_b200.gq as G

TYPES = [torch.float32, torch.bfloat16, torch.float16]
FILL = 0xAB


def _pow2(e):
    """2^e, from its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def encode(x):
    """act_oracle.encode in torch, on x's device."""
    rows, cols = x.shape
    cp, ep = A.pitches(cols)
    v = torch.zeros(rows, cp, dtype=torch.float64, device=x.device)
    v[:, :cols] = x
    v = v.view(rows, cp // 32, 32)
    bad = ~torch.isfinite(v).all(2)
    m = torch.where(torch.isfinite(v), v.abs(), 0.0).amax(2)
    E = torch.where(m > 0, torch.frexp(m)[1].to(torch.int64) - 9 + 133, 0).clamp(0, 254)
    for _ in range(4):
        E = E + ((torch.round(m * _pow2(133 - E)) > 127) & (E < 254))
    q = torch.round(v * _pow2(133 - E)[:, :, None]).clamp(-127, 127)
    q = torch.where(bad[:, :, None], 0.0, q)
    exps = torch.zeros(rows, ep, dtype=torch.uint8, device=x.device)
    exps[:, :cp // 32] = torch.where(bad, 255, E)
    return q.view(rows, cp).to(torch.int8), exps


def decode(codes, exps, cols):
    rows, cp = codes.shape
    v = codes.double().view(rows, cp // 32, 32) * _pow2(exps[:, :cp // 32].to(torch.int64) - 133)[:, :, None]
    return v.view(rows, cp)[:, :cols]


def _values(rows, cols, seed, device="cpu"):
    g = torch.Generator(device=device).manual_seed(seed)
    x = torch.randn(rows, cols, generator=g, device=device)
    return x * torch.exp2(torch.randint(-6, 3, (rows, 1), generator=g, device=device).float())


@pytest.mark.parametrize("dtype", TYPES)
def test_the_two_oracles_agree(dtype):
    x = _values(40, 100, 1)
    x[3, 5], x[4, 77], x[5] = float("nan"), float("inf"), 0.0
    x[6, :32], x[7, 0], x[8, :4] = 127.5, torch.finfo(dtype).max, torch.finfo(dtype).smallest_normal / 4
    x = x.to(dtype)
    codes, exps = A.encode(x)
    c, e = encode(x)
    assert np.array_equal(c.numpy(), codes) and np.array_equal(e.numpy(), exps)
    keep = [i for i in range(40) if i not in (3, 4)]
    assert torch.equal(decode(c, e, 100)[keep], A.decode(codes, exps, 100)[keep])


def _wide(rows, cols, pad, dtype):
    buf = torch.full((rows, cols + pad), float("nan"), dtype=dtype, device="cuda")
    return buf, buf[:, :cols]


# Pieces are 512 or 1024 columns.  Nine pieces a row (17 of the aligned backward pass): a count that does not
# divide the warps of any grid of whole blocks on 148 SMs, so a step changes the place in the row and wraps.
# Eight: it does, and the place stays.
SHAPES = [(3001, 4607, 0), (2001, 8200, 8), (2501, 4095, 0)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,pad", SHAPES)
def test_pack_and_unpack(dtype, rows, cols, pad):
    buf, x = _wide(rows, cols, pad, dtype)
    x.copy_(_values(rows, cols, rows + cols, "cuda"))
    codes, exps = encode(x)
    (cp, ep), (size, off) = A.pitches(cols), A.layout(rows, cols)
    ck = torch.full((size,), FILL, dtype=torch.uint8, device="cuda")
    G.gq_act_pack(x, ck)
    assert torch.equal(ck[:rows * cp].view(torch.int8).view(rows, cp), codes)
    assert torch.equal(ck[off:off + rows * ep].view(rows, ep), exps)
    assert (ck[rows * cp:off] == FILL).all() and (ck[off + rows * ep:] == FILL).all()
    want = decode(codes, exps, cols)
    for out in TYPES:
        wide, y = _wide(rows, cols, pad, out)
        G.gq_act_unpack(ck, y)
        assert torch.equal(y, A.as_type(want, out))
        assert torch.isnan(wide[:, cols:]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,pad", SHAPES)
def test_functions(dtype, rows, cols, pad):
    from test_act_values_gpu import STEP, U, bounds, within
    _, x = _wide(rows, cols, pad, dtype)
    _, dy = _wide(rows, cols, pad, dtype)
    x.copy_(_values(rows, cols, 1, "cuda"))
    dy.copy_(_values(rows, cols, 2, "cuda"))
    codes, exps = encode(x)
    ck, packed = (torch.full((A.layout(rows, cols)[0],), FILL, dtype=torch.uint8, device="cuda") for _ in range(2))
    (wide, y), (wide2, y2), (wide3, dx) = (_wide(rows, cols, pad, dtype) for _ in range(3))
    G.gq_act_fn_forward("silu", x, y, ck)
    G.gq_act_fn_forward("silu", x, y2)
    G.gq_act_pack(x, packed)
    assert torch.equal(ck, packed) and torch.equal(y, y2)
    f, _, ef, _ = bounds("silu", x.double())
    within(y, f, ef, dtype)
    G.gq_act_fn_backward("silu", ck, dy, dx)
    _, df, _, edf = bounds("silu", decode(codes, exps, cols))
    d = dy.double()
    within(dx, d * df, d.abs() * (edf + U * df.abs()) + STEP, dtype)
    for w in (wide, wide2, wide3):
        assert torch.isnan(w[:, cols:]).all()
