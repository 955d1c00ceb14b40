"""Matrices in 8-bit floating point on the GPU: packing against the 64-bit oracle code for code, products against the
64-bit product of the decoded operands."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import fp8_oracle as O
import gradient_quantization_communication_b200.gq as G

TYPES = [torch.float32, torch.bfloat16, torch.float16]
SHAPES = [(1, 1), (1, 127), (3, 128), (7, 129), (128, 256), (129, 257), (255, 40), (300, 1030), (1, 4096), (513, 8)]


def packed(rows, cols, tile, fill=0xEE):
    return torch.full((G.gq_fp8_layout(rows, cols, tile)[0],), fill, dtype=torch.uint8, device="cuda")


def matrix(rows, cols, dtype, seed, pad=0, spread=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(rows, cols + pad, generator=g, device="cuda") * torch.exp(
        spread * torch.randn(rows, 1, generator=g, device="cuda"))
    x = x * (torch.rand(rows, cols + pad, generator=g, device="cuda") > 0.1)
    return x.to(dtype)[:, :cols]


def check(buf, x, fmt, tile):
    """Codes, exponents and their padding, byte for byte."""
    codes, exps = O.pack(x.cpu(), fmt, tile)
    got, off = buf.cpu().numpy(), O.layout(tile, *x.shape)[1]
    assert np.array_equal(got[:codes.size].reshape(codes.shape), codes)
    assert np.array_equal(got[off:off + exps.size].reshape(exps.shape), exps)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_pack(dtype, fmt, tile, rows, cols):
    for pad in (0, 8, 3):
        x = matrix(rows, cols, dtype, rows * 31 + cols + pad, pad)
        for ways in ("rows", "cols", "both"):
            p = packed(rows, cols, tile) if ways != "cols" else None
            t = packed(cols, rows, tile) if ways != "rows" else None
            G.gq_fp8_pack(x, p, t, fmt=fmt, tile=tile)
            if p is not None:
                check(p, x, fmt, tile)
            if t is not None:
                check(t, x.t(), fmt, tile)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("dtype", TYPES)
def test_pack_borders(dtype, fmt, tile):
    """Largest values at and next to the borders between exponents, all exponents, zeros, subnormals, the largest
    values, infinities and NaN."""
    rows = 128 * 3 if tile else 600
    g = torch.Generator().manual_seed(3)
    x = torch.rand(rows, 1024, generator=g) * 1.9 - 0.95
    e = torch.randint(-149 if dtype == torch.float32 else -24, 128 if dtype != torch.float16 else 16, (rows, 8), generator=g)
    e = e.repeat_interleave(128, 1)
    top = torch.tensor([1.75, 1.75 * (1 + 2 ** -7), 1.75 - 2 ** -6, 1.0, 1.99])[torch.randint(0, 5, (rows, 8), generator=g)]
    x = torch.ldexp(x.double(), e.double())
    x[:, ::128] = torch.ldexp(top.double(), e[:, ::128].double())
    x = x.to(dtype)
    big = torch.finfo(dtype).max
    for r, c, v in ((0, 5, float("nan")), (1, 300, float("inf")), (2, 600, -float("inf")), (3, 700, big), (4, 800, -big)):
        x[r * (rows // 6):r * (rows // 6) + 1, c] = v
    x[rows // 2:rows // 2 + (128 if tile else 2)] = 0.0
    x = x.cuda()
    p, t = packed(rows, 1024, tile), packed(1024, rows, tile)
    G.gq_fp8_pack(x, p, t, fmt=fmt, tile=tile)
    check(p, x, fmt, tile)
    check(t, x.t(), fmt, tile)
    one = packed(rows, 1024, tile)
    G.gq_fp8_pack(x, one, fmt=fmt, tile=tile)
    assert torch.equal(one, p)


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_pack_every_value(fmt):
    """Every bfloat16 and float16 value, each beside a largest value that puts it at all places of the code's range."""
    for dtype in (torch.bfloat16, torch.float16):
        v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype)
        v = v[torch.isfinite(v)]
        x = torch.zeros((v.numel() + 126) // 127, 128, dtype=dtype)
        flat = torch.zeros(x.shape[0] * 127, dtype=dtype)
        flat[:v.numel()] = v
        x[:, 1:] = flat.view(-1, 127)
        x = x.cuda()
        p, t = packed(x.shape[0], 128, False), packed(128, x.shape[0], False)
        G.gq_fp8_pack(x, p, t, fmt=fmt)
        check(p, x, fmt, False)
        check(t, x.t(), fmt, False)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_unpack_every_code_and_exponent(dtype, fmt):
    rows = 256
    codes = np.zeros((rows, 256), np.uint8)
    codes[:] = np.arange(256)
    exps = np.zeros((rows, 4), np.uint8)
    exps[:, 0] = exps[:, 1] = np.arange(256)
    # exponents that packing gives: a packed buffer holds no others
    keep = np.concatenate([np.arange(10, 255 - O.TOP[fmt]), [255]])
    codes, exps = codes[keep], exps[keep]
    codes[exps[:, 0] == 255] = 0x7F
    want = O.decode(codes, exps, fmt, False, 256)
    buf = torch.from_numpy(O.to_buffer(codes, exps)).cuda()
    for pad in (0, 3):
        x = torch.full((len(keep), 256 + pad), 5.0, dtype=dtype, device="cuda")
        G.gq_fp8_unpack(buf, x[:, :256], fmt=fmt)
        w = want.clamp(-65504, 65504).to(dtype) if dtype == torch.float16 else want.to(dtype)
        assert torch.equal(torch.nan_to_num(x[:, :256].cpu(), 7.0, 8.0, 9.0), torch.nan_to_num(w, 7.0, 8.0, 9.0))
        assert torch.equal(torch.isnan(x[:, :256].cpu()), torch.isnan(w))
        assert (x[:, 256:] == 5.0).all()


@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("rows,cols", [(1, 1), (129, 257), (300, 1030)])
def test_unpack_what_was_packed(tile, rows, cols):
    for dtype in TYPES:
        x = matrix(rows, cols, dtype, 4)
        p, t = packed(rows, cols, tile), packed(cols, rows, tile)
        G.gq_fp8_pack(x, p, t, tile=tile)
        for buf, src in ((p, x), (t, x.t())):
            out = torch.empty(src.shape, dtype=dtype, device="cuda")
            G.gq_fp8_unpack(buf, out, tile=tile)
            assert torch.equal(out.cpu(), O.decode(*O.pack(src.cpu(), "e4m3", tile), "e4m3", tile, src.shape[1]).to(dtype))
            # half a step of the largest exponent that a value of the block may have, and half the smallest code
            err = (out.double() - src.double()).abs().cpu()
            lim = 2.0 ** -4 * src.double().abs().cpu() + 2.0 ** -10 * 2.0 ** -7 * src.double().abs().max().cpu()
            assert (err <= lim).all()


# ----------------------------------------------------------------------------------------------------
# Products
# ----------------------------------------------------------------------------------------------------
def operand(rows, k, fmt, tile, seed, spread=1.0):
    x = matrix(rows, k, torch.float32, seed, spread=spread)
    buf = packed(rows, k, tile)
    G.gq_fp8_pack(x, buf, fmt=fmt, tile=tile)
    codes = buf.cpu().numpy()
    size, off = O.layout(tile, rows, k)
    cp, ep = O.pitches(k)
    er = -(-rows // 128) if tile else rows
    return buf, O.decode(codes[:rows * cp].reshape(rows, cp), codes[off:off + er * ep].reshape(er, ep), fmt, tile, k).cuda()


def steps(k, dtype=torch.float32):
    """Half-steps of binary32 that a sum over k columns may be off by, relative to the sum of absolute products: two
    steps for every 32 products while the tensor cores cut off (runs of 4096 columns at most, 16384 for a result of 16
    bits), three roundings a run, and a few for joining parts, the bias and adding."""
    run = 4096 if dtype == torch.float32 else 16384
    return 2 * (min(k, run) / 32 * 2 + 3 * (k / run + 1) + 16)


def check_product(y, da, db, k, bias=None, before=None):
    want = da @ db.t()
    size = da.abs() @ db.abs().t()
    if bias is not None:
        want = want + bias.double()
        size = size + bias.double().abs()
    if before is not None:
        want = want + before.double()
        size = size + before.double().abs()
    tol = steps(k, y.dtype) * 2.0 ** -24 * size + O.HALF_STEP[y.dtype] * want.abs() * 1.01
    if y.dtype == torch.float16:
        tol = tol + 2.0 ** -25
    err = (y.double() - want).abs()
    assert (err <= tol).all(), (float((err / tol).max()), int((err > tol).sum()), tuple(torch.nonzero(err > tol)[0].tolist()))


PRODUCTS = [(1, 1, 1), (1, 128, 128), (2, 7, 5), (16, 130, 500), (17, 257, 513), (33, 64, 1030), (64, 300, 4096),
            (65, 129, 640), (128, 256, 128), (129, 255, 384), (200, 1000, 1000), (300, 77, 2050), (515, 515, 515),
            (1, 4096, 4096), (8, 1000, 8200), (1100, 900, 260), (300, 300, 8200), (70, 40, 20000), (260, 260, 20000)]


@pytest.mark.parametrize("m,n,k", PRODUCTS)
@pytest.mark.parametrize("dtype", TYPES)
def test_matmul(m, n, k, dtype):
    for fa, fb, ta, tb in (("e4m3", "e4m3", False, True), ("e5m2", "e4m3", False, True), ("e4m3", "e5m2", False, False),
                           ("e5m2", "e5m2", True, True)):
        a, da = operand(m, k, fa, ta, m + k)
        b, db = operand(n, k, fb, tb, n + k + 1)
        y = torch.full((m, n), 9.0, dtype=dtype, device="cuda")
        G.gq_fp8_matmul(a, b, k, y, fmt=(fa, fb), tile=(ta, tb))
        # keep float16 in its range: the operands have unit scale and a spread of a few
        if dtype == torch.float16 and (da @ db.t()).abs().max() > 6e4:
            continue
        check_product(y, da, db, k)


@pytest.mark.parametrize("m,n,k", [(1, 130, 300), (33, 257, 1030), (300, 200, 520), (700, 515, 260)])
def test_matmul_bias_adding_and_slices(m, n, k):
    a, da = operand(m, k, "e4m3", False, 1)
    b, db = operand(n, k, "e4m3", False, 2)
    g = torch.Generator(device="cuda").manual_seed(3)
    flat = torch.randn(n + 1, generator=g, device="cuda")
    bias = flat[1:]                                     # 4-byte aligned
    for dtype in TYPES:
        for pad, off in ((0, 0), (8, 0), (5, 3), (1, 1)):
            wide = torch.full((m, n + pad), 3.0, dtype=dtype, device="cuda")
            y = wide[:, off:off + n]
            G.gq_fp8_matmul(a, b, k, y, bias)
            check_product(y, da, db, k, bias)
            assert (wide[:, :off] == 3.0).all() and (wide[:, off + n:] == 3.0).all()
            if dtype != torch.float32:
                continue
            alone = torch.empty(m, n, device="cuda")
            G.gq_fp8_matmul(a, b, k, alone)
            before = torch.randn(m, n, generator=g, device="cuda")
            y.copy_(before)
            G.gq_fp8_matmul(a, b, k, y, accumulate=True)
            assert torch.equal(y, before + alone)       # one rounding
            y.copy_(before)
            G.gq_fp8_matmul(a, b, k, y, bias, accumulate=True)
            check_product(y, da, db, k, bias, before)
            assert (wide[:, :off] == 3.0).all() and (wide[:, off + n:] == 3.0).all()


@pytest.mark.parametrize("m,n,k", [(3, 5, 700), (40, 300, 600), (300, 300, 900)])
def test_matmul_of_nan_infinite_and_tiny_blocks(m, n, k):
    """A NaN block makes its rows of y NaN and no others; scales at both ends of their range."""
    x, w = matrix(m, k, torch.float32, 5), matrix(n, k, torch.float32, 6)
    x[1, 200] = float("nan")
    w[n - 1, k - 1] = float("inf")
    x[0] *= 2.0 ** -100
    x[2] *= 2.0 ** 100
    w[0] *= 2.0 ** -20
    w[1] *= 2.0 ** 20
    a, b = packed(m, k, False), packed(n, k, False)
    G.gq_fp8_pack(x, a)
    G.gq_fp8_pack(w, b)
    y = torch.empty(m, n, device="cuda")
    G.gq_fp8_matmul(a, b, k, y)
    nan = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    nan[1, :] = True
    nan[:, n - 1] = True
    assert torch.equal(torch.isnan(y), nan)
    da = O.decode(*O.pack(x.cpu(), "e4m3", False), "e4m3", False, k).cuda()
    db = O.decode(*O.pack(w.cpu(), "e4m3", False), "e4m3", False, k).cuda()
    keep_m, keep_n = [i for i in range(m) if i != 1], list(range(n - 1))
    sub = y[keep_m][:, keep_n]
    want = da[keep_m] @ db[keep_n].t()
    size = da[keep_m].abs() @ db[keep_n].abs().t()
    # sums below 2^-126 may read as 0
    assert ((sub.double() - want).abs() <= steps(k) * 2.0 ** -24 * size + 2.0 ** -126).all()


def test_matmul_every_code_and_scale():
    """Every pair of codes exactly: one product a sum."""
    for fa, fb in (("e4m3", "e4m3"), ("e5m2", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e5m2")):
        va, vb = O.values(fa), O.values(fb)
        bufs = []
        for _ in range(2):
            codes = np.zeros((256, 128), np.uint8)
            codes[:, 5] = np.arange(256)
            exps = np.zeros((256, 4), np.uint8)
            exps[:, 0] = 100 + np.arange(256) % 41
            bufs.append(torch.from_numpy(O.to_buffer(codes, exps)).cuda())
        y = torch.empty(256, 256, device="cuda")
        G.gq_fp8_matmul(bufs[0], bufs[1], 128, y, fmt=(fa, fb))
        e = 100 + np.arange(256) % 41 - 127
        with np.errstate(invalid="ignore"):
            want = torch.from_numpy(np.ldexp(va, e)[:, None] * np.ldexp(vb, e)[None, :])
        y = y.cpu().double()
        assert torch.equal(torch.isnan(y), torch.isnan(want))
        ok = ~torch.isnan(want)
        assert torch.equal(y[ok], want[ok])


@pytest.mark.parametrize("m,n,k", [(16, 4096, 4096), (1000, 1000, 3000), (4096, 2048, 2048), (640, 8000, 700)])
def test_equal_calls_give_equal_bits(m, n, k):
    a, da = operand(m, k, "e4m3", False, 7, spread=0.3)
    b, db = operand(n, k, "e4m3", True, 8, spread=0.3)
    first, again = (torch.empty(m, n, device="cuda") for _ in range(2))
    ws = G.gq_fp8_matmul_workspace(k, first)
    G.gq_fp8_matmul(a, b, k, first, tile=(False, True), workspace=ws)
    check_product(first, da, db, k)
    for _ in range(30):
        if ws is not None:
            ws.fill_(0xFF)
        again.fill_(1.0)
        G.gq_fp8_matmul(a, b, k, again, tile=(False, True), workspace=ws)
        assert torch.equal(first, again)


def test_another_stream_and_a_captured_call():
    m, n, k = 300, 500, 1000
    x, w = matrix(m, k, torch.bfloat16, 9), matrix(n, k, torch.float32, 10)
    a, b = packed(m, k, False), packed(n, k, True)
    G.gq_fp8_pack(w, b, tile=True)
    G.gq_fp8_pack(x, a)
    y = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    G.gq_fp8_matmul(a, b, k, y, tile=(False, True))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    other_a, other_y = packed(m, k, False), torch.zeros_like(y)
    s.wait_stream(torch.cuda.current_stream())
    G.gq_fp8_pack(x, other_a, stream=s)
    G.gq_fp8_matmul(other_a, b, k, other_y, tile=(False, True), stream=s)
    s.synchronize()
    assert torch.equal(other_y, y)
    # captured, with new inputs at every replay
    ws = G.gq_fp8_matmul_workspace(k, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        G.gq_fp8_pack(x, a)
        G.gq_fp8_matmul(a, b, k, y, tile=(False, True), workspace=ws)
    for seed in (11, 12):
        x.copy_(matrix(m, k, torch.bfloat16, seed))
        graph.replay()
        G.gq_fp8_pack(x, other_a)
        G.gq_fp8_matmul(other_a, b, k, other_y, tile=(False, True))
        assert torch.equal(other_y, y)


def test_offsets_past_32_bits():
    """Rows of x and y whose offsets pass 32 bits, in a buffer that is mostly not touched."""
    rows, cols, stride = 3, 300, (1 << 31) + 16
    big = torch.empty(2 * stride + cols, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((rows, cols), (stride, 1))
    x.copy_(matrix(rows, cols, torch.bfloat16, 13))
    p, t = packed(rows, cols, False), packed(cols, rows, False)
    G.gq_fp8_pack(x, p, t)
    check(p, x, "e4m3", False)
    check(t, x.t(), "e4m3", False)
    want = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    G.gq_fp8_unpack(p, want)
    x.zero_()
    G.gq_fp8_unpack(p, x)
    assert torch.equal(x, want)
    b, db = operand(cols, cols, "e4m3", True, 14)
    G.gq_fp8_matmul(p, b, cols, x, tile=(False, True))
    G.gq_fp8_matmul(p, b, cols, want, tile=(False, True))
    assert torch.equal(x, want)
