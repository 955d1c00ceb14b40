"""The checkpoint's exponent rule at every largest value a group can have: all magnitudes of the 16-bit types,
and of binary32 those around each exponent's border, subnormal ones among them.  Byte for byte."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import act_oracle as A
import gradient_quantization_communication_b200.gq as G

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _largest(dtype):
    """Magnitudes of every kind, as a vector of dtype."""
    if dtype != torch.float32:
        return torch.arange(0, 32768, dtype=torch.int32).to(torch.int16).view(dtype)
    # mantissas around 127.5 / 128 of the next power of two (1.9921875 for normal values, half of its last place
    # for subnormal ones), around the powers of two, and some between
    low = [0, 1, 2, 0x10000, 0x3fffff, 0x400000, 0x7effff, 0x7f0000, 0x7f0001, 0x7f7fff, 0x7f8000, 0x7f8001, 0x7fffff]
    bits = (torch.arange(0, 256, dtype=torch.int32)[:, None] << 23) | torch.tensor(low, dtype=torch.int32)
    return bits.view(-1).view(dtype)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad", [0, 3])
def test_pack_of_every_largest_value(dtype, pad):
    m = _largest(dtype)
    g = torch.Generator().manual_seed(1)
    # the largest value anywhere in its group, of either sign, and parts of it beside it
    x = (m.double()[:, None] * (torch.rand(m.numel(), 32, generator=g, dtype=torch.float64) * 2 - 1)).to(dtype)
    x = torch.where(x.abs().double() > m.abs().double()[:, None], torch.zeros((), dtype=dtype), x)
    at = torch.randint(0, 32, (m.numel(),), generator=g)
    x[torch.arange(m.numel()), at] = torch.where(torch.rand(m.numel(), generator=g) < 0.5, m, -m)
    x = x.reshape(-1, 4 * 32) if m.numel() % 4 == 0 else x
    rows, cols = x.shape
    wide = torch.zeros(rows, cols + pad, dtype=dtype, device="cuda")
    wide[:, :cols] = x.cuda()
    codes, exps = A.encode(x)
    want = torch.from_numpy(A.to_buffer(codes, exps))
    ck, y = torch.zeros(want.numel(), dtype=torch.uint8, device="cuda"), torch.empty_like(wide)
    G.gq_act_pack(wide[:, :cols], ck)
    off = (ck.cpu() != want).nonzero()[:, 0]
    assert off.numel() == 0, (off[:8], ck.cpu()[off[:8]], want[off[:8]])
    G.gq_act_fn_forward("silu", wide[:, :cols], y[:, :cols], ck.zero_())
    assert torch.equal(ck.cpu(), want)
    m, r = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    G.gq_layer_norm_forward(wide[:, :cols], None, None, 1e-5, y[:, :cols], m, r, ck.zero_())
    assert torch.equal(ck.cpu(), want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_largest_subnormal_is_kept(dtype):
    """127 times bf16's smallest value is a code of its own, under the exponent byte 0."""
    x = torch.full((1, 32), 127 * 2.0 ** -133, dtype=torch.float64).to(dtype)
    ck, y = torch.zeros(48, dtype=torch.uint8, device="cuda"), torch.empty(1, 32, dtype=dtype, device="cuda")
    G.gq_act_pack(x.cuda(), ck)
    G.gq_act_unpack(ck, y)
    assert ck[32] == 0 and torch.equal(y.cpu(), x)
