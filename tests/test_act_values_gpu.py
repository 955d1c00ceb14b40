"""Activation functions at every value: all 65536 bit patterns of the 16-bit types, and of binary32 by their
upper halves, through the forward pass; every code under every exponent through the backward pass.  Against
64 bits, with tolerances that hold down to the types' smallest subnormals.

What the arithmetic may lose, in binary32 half steps U = 2^-24 (the 16-bit types use the approximate
exponential and reciprocal, 4 U and 2 U, and a polynomial of 9 U; binary32 calls erfcf, expf and a division of
at most 8 U each):
  * an exponential (or complementary error function) whose argument has size a: the argument's own roundings,
    at most 5 U of it for the tanh form's cubic and less for the others, the product with log2(e) and its
    constant, 2.3 U of it, and an offset of 24 added to it, 17 U.  With the steps above and the products after
    it, at most (40 + 7.5 a) U of the tail s(-|x|) or Phi(-|x|);
  * the other side, 1 - tail, that and 4 U of itself;
  * products with x and dy, U each;
  * subnormal results: 2^-147 in a tail (four of binary32's smallest steps), times the factors after it.  Tails
    are 0 in binary32 and in the kernels beyond |x| = 128, so these factors are bounded."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import act_oracle as A
import gradient_quantization_communication_b200.gq as G

TYPES = [torch.float32, torch.bfloat16, torch.float16]
KINDS = ["gelu", "gelu_tanh", "silu"]
U = 2.0 ** -24
STEP = 2.0 ** -149                                    # binary32's smallest
SMALLEST = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def bounds(kind, x):
    """f and f' at float64 x, and what binary32 may lose of each."""
    f, df, _ = A.fn(kind, x)
    ax, near = x.abs(), x.abs().clamp(max=128.0)
    if kind == "gelu":
        a, tail = x * x / 2, 0.5 * torch.special.erfc(ax / math.sqrt(2))
    elif kind == "silu":
        a, tail = ax, torch.sigmoid(-ax)
    else:
        a = 2 * math.sqrt(2 / math.pi) * (ax + 0.044715 * ax ** 3)
        tail = torch.sigmoid(-a)
    rel = (40 + 7.5 * a) * U
    lost = torch.where(tail > 0, tail * rel, 0.0)      # a may be huge where the tail is 0
    s, r = torch.where(x < 0, tail, 1 - tail), torch.where(x < 0, 1 - tail, tail)
    es, er = lost + 4 * U * s, lost + 4 * U * r
    ef = ax * es + 4 * STEP * near + U * f.abs() + STEP
    if kind == "gelu":
        slope = ax * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
        edf = torch.where(slope > 0, slope * rel, 0.0) + es + 4 * STEP * (1 + near)
    elif kind == "silu":
        edf = es * (1 + ax * r) + s * (ax * er + 2 * U * (1 + ax * r)) + 8 * STEP * (1 + near)
    else:
        slope, b = (df - s).abs(), ax.clamp(max=30.0)  # x s r c (1 + 0.134 x^2), both tails' errors in it
        edf = es + torch.where(slope > 0, slope * (rel + 20 * U), 0.0) + (4 * b + 2) * (2 + 0.22 * b * b) * STEP
    return f, df, ef, edf


def within(got, want, lost, dtype):
    tol = lost + A.HALF_STEP[dtype] * (want.abs() + lost) + SMALLEST[dtype] / 2
    off = (got.double() - want).abs() > tol
    assert not off.any(), (int(off.sum()), got[off][:4], want[off][:4], tol[off][:4])


def patterns(dtype):
    """256 x 256 values: every bit pattern (binary32: every upper half, the lower at random)."""
    bits = torch.arange(-32768, 32768, dtype=torch.int32)
    if dtype == torch.float32:
        low = torch.randint(0, 1 << 16, bits.shape, generator=torch.Generator().manual_seed(1), dtype=torch.int32)
        return ((bits << 16) | low).view(dtype).view(256, 256)
    return bits.to(torch.int16).view(dtype).view(256, 256)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad", [0, 3])
def test_forward_of_every_value(kind, dtype, pad):
    x = patterns(dtype)
    wide = torch.zeros(256, 256 + pad, dtype=dtype, device="cuda")
    wide[:, :256] = x.cuda()
    y, ck = torch.empty_like(wide), torch.zeros(G.gq_act_layout(256, 256)[0], dtype=torch.uint8, device="cuda")
    G.gq_act_fn_forward(kind, wide[:, :256], y[:, :256], ck)
    got = y[:, :256].cpu()
    number = torch.isfinite(x)
    v = x[number].double()
    f, _, ef, _ = bounds(kind, v)
    within(got[number], f, ef, dtype)
    # infinity times 1 and infinity times 0, as the formulas have it
    assert (got[x == float("inf")].float() == float("inf")).all()
    assert torch.isnan(got[(x == float("-inf")) | torch.isnan(x)].float()).all()
    assert np.array_equal(ck.cpu().numpy(), A.to_buffer(*A.encode(x)))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad", [0, 3])
def test_backward_of_every_code(kind, dtype, pad):
    """Row E holds every code under the exponent byte E; dy is 1, then random."""
    exps = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 8, 1)
    codes = np.tile(np.arange(-128, 128).astype(np.int8), (256, 1))
    codes[254, 0] = -127    # -128 * 2^121 is beyond binary32; pack writes no code -128
    ck = torch.from_numpy(A.to_buffer(codes, exps)).cuda()
    x = A.decode(codes, exps, 256)
    _, df, _, edf = bounds(kind, x[:255])
    for dy in (torch.ones(256, 256), torch.randn(256, 256, generator=torch.Generator().manual_seed(2))):
        dy = dy.to(dtype)
        wide = torch.zeros(256, 256 + pad, dtype=dtype, device="cuda")
        wide[:, :256] = dy.cuda()
        dx = torch.empty_like(wide)
        G.gq_act_fn_backward(kind, ck, wide[:, :256], dx[:, :256])
        got, d = dx[:, :256].cpu(), dy.double()[:255]
        within(got[:255], d * df, d.abs() * (edf + U * df.abs()) + STEP, dtype)
        assert torch.isnan(got[255].float()).all()
