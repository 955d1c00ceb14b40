"""Weight gradients by calls that the header allows besides the usual ones: one token of a wide layer, slices of
a wider matrix as outputs of tiles that are cut along the tokens, gradients whose rows repeat or overlap over many
tiles."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import gradient_quantization_communication_b200.gq as G
from test_act_walk_gpu import decode, encode

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _inputs(tokens, cin, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, cin, generator=g, device="cuda").to(dtype)
    ck = torch.zeros(G.gq_act_layout(tokens, cin)[0], dtype=torch.uint8, device="cuda")
    G.gq_act_pack(x, ck)
    return g, ck, decode(*encode(x), cin)


@pytest.mark.parametrize("dtype", TYPES)
def test_one_token_of_a_wide_layer(dtype):
    """More than a block a token's products are: the tiles, with one row whose stride means nothing."""
    g, ck, xh = _inputs(1, 8200, dtype, 1)
    row = torch.randn(8201, generator=g, device="cuda").to(dtype)
    dw, db = torch.full((8201, 8200), 7.0, device="cuda"), torch.empty(8201, device="cuda")
    G.gq_act_weight_grad(ck, row.as_strided((1, 8201), (3, 1)), dw, db)
    want = row.double()[:, None] * xh
    # 16-bit types: one exact product.  float32: three exact products, added with two steps' error each
    tol = 3 * 2.0 ** -22 * want.abs() if dtype == torch.float32 else 0.0
    assert ((dw.double() - want).abs() <= tol).all()
    assert torch.equal(db, row.float())


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("offset", [3, 4])
def test_cut_tiles_into_slices_of_a_wider_matrix(dtype, offset):
    g, ck, xh = _inputs(5000, 700, dtype, 2)
    dy = (0.01 * torch.randn(5000, 650, generator=g, device="cuda")).to(dtype)
    alone, wide = torch.empty(650, 700, device="cuda"), torch.full((650, 711), 3.0, device="cuda")
    G.gq_act_weight_grad(ck, dy, alone)
    d = dy.double()
    # runs of 512 tokens lose at most two steps every 16 tokens, their sums one rounding each
    steps = 512 / 16 * 2 + 3 * 5000 / 512 + 16
    assert ((alone.double() - d.t() @ xh).abs() <= steps * 2.0 ** -23 * (d.abs().t() @ xh.abs())).all()
    dw = wide[:, offset:offset + 700]
    G.gq_act_weight_grad(ck, dy, dw)
    assert torch.equal(dw, alone)
    before = torch.randn(650, 700, generator=g, device="cuda")
    dw.copy_(before)
    G.gq_act_weight_grad(ck, dy, dw, accumulate=True)
    assert torch.equal(dw, before + alone)
    assert (wide[:, :offset] == 3.0).all() and (wide[:, offset + 700:] == 3.0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("stride", [0, 5, 8])
def test_rows_that_repeat_or_overlap(dtype, stride):
    """As if copied out."""
    g, ck, _ = _inputs(3001, 1300, dtype, 3)
    flat = torch.randn(3000 * stride + 1100, generator=g, device="cuda").to(dtype)
    dy = flat.as_strided((3001, 1100), (stride, 1))
    outs = []
    for t in (dy, dy.contiguous()):
        dw, db = torch.empty(1100, 1300, device="cuda"), torch.empty(1100, device="cuda")
        G.gq_act_weight_grad(ck, t, dw, db)
        outs.append((dw, db))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens", [2, 40])
def test_every_value_of_a_gradient(dtype, tokens):
    """All 65536 patterns of a 16-bit gradient (of float32 the upper halves, the lower at random), in one token,
    against inputs 1, -2, 0.5 and 0: products as the formulas have them, infinities, NaN and subnormals included."""
    bits = torch.arange(-32768, 32768, dtype=torch.int32)
    if dtype == torch.float32:
        low = torch.randint(0, 1 << 16, bits.shape, generator=torch.Generator().manual_seed(4), dtype=torch.int32)
        v = ((bits << 16) | low).view(dtype)
    else:
        v = bits.to(torch.int16).view(dtype)
    if tokens == 2:      # a few tokens, few columns: another kernel
        v = v[::4]
    v = v.cuda()
    x = torch.zeros(tokens, 64, dtype=dtype, device="cuda")
    x[1, :3] = torch.tensor([1.0, -2.0, 0.5], dtype=dtype)
    ck = torch.zeros(G.gq_act_layout(tokens, 64)[0], dtype=torch.uint8, device="cuda")
    G.gq_act_pack(x, ck)
    dy = torch.zeros(tokens, v.numel(), dtype=dtype, device="cuda")
    dy[1] = v
    dw, db = torch.empty(v.numel(), 64, device="cuda"), torch.empty(v.numel(), device="cuda")
    G.gq_act_weight_grad(ck, dy, dw, db)
    d = v.double()
    number = torch.isfinite(d)
    # float32 in three bf16 planes: what lies below bf16's smallest value, 2^-133, is cut off
    cut = 2.0 ** -133 if dtype == torch.float32 and tokens > 2 else 0.0
    for k, f in enumerate((1.0, -2.0, 0.5)):
        want = (d * f).float().double()
        got = dw[:, k].double()
        fits = number & torch.isfinite(want)
        # half of the smallest values: a tie, rounded or cut
        assert ((got - want).abs()[fits] <= cut * abs(f) + (2.0 ** -149 if f == 0.5 else 0.0)).all()
        assert torch.equal(torch.isnan(got), torch.isnan(d))
        assert torch.equal(got[~number & ~torch.isnan(d)], want[~number & ~torch.isnan(d)])
    assert torch.equal(torch.isnan(dw[:, 3]), ~number) and (dw[:, 3][number] == 0).all()
    assert torch.equal(torch.nan_to_num(db, nan=-1.0), torch.nan_to_num(v.float(), nan=-1.0))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,cin,cout,pad", [(5072, 859, 3264, 1), (5992, 153, 1931, 24), (16384, 1024, 1024, 0)])
def test_repeats_give_equal_bits(dtype, tokens, cin, cout, pad):
    """Long contractions, whose warps wait for one another some hundred times a tile, over and over."""
    g, ck, xh = _inputs(tokens, cin, dtype, 5)
    dy = (0.05 * torch.randn(tokens, cout + pad, generator=g, device="cuda")).to(dtype)[:, :cout]
    first, again = torch.empty(cout, cin, device="cuda"), torch.empty(cout, cin, device="cuda")
    ws = G.gq_act_weight_grad_workspace(ck, dy, first)
    G.gq_act_weight_grad(ck, dy, first, workspace=ws)
    d = dy.double()
    total = tokens * (3 if dtype == torch.float32 else 1)
    # runs of 512 tokens (of three planes) lose at most two steps every 16 tokens, their sums one rounding each
    steps = 512 / 16 * 2 + 3 * total / 512 + 16
    assert ((first.double() - d.t() @ xh).abs() <= steps * 2.0 ** -23 * (d.abs().t() @ xh.abs())).all()
    for _ in range(100):
        again.fill_(float("nan"))
        G.gq_act_weight_grad(ck, dy, again, workspace=ws)
        assert torch.equal(first, again)
