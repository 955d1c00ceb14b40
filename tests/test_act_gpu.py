"""GPU tests of the 8-bit activation checkpoints and the operators that read them (gq_act_pack,
gq_act_unpack, gq_act_fn_*, gq_act_weight_grad) against 64-bit computations on the CPU.

Checkpoints are compared byte for byte.  Tolerances count roundings: half a step of the output's
type, plus the binary32 arithmetic's own, written beside each."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import act_oracle as A
import gradient_quantization_communication_b200.gq as G

TYPES = [torch.float32, torch.bfloat16, torch.float16]
FILL = 0xAB


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _padded(x, pad, fill=0.0):
    """x on the GPU, its rows `pad` elements further apart than they are wide."""
    rows, cols = x.shape
    buf = torch.full((rows, cols + pad), fill, dtype=x.dtype, device="cuda")
    buf[:, :cols] = x.cuda()
    return buf[:, :cols]


def _values(rows, cols, dtype, seed, scale=1.0):
    g = _gen(seed)
    x = torch.randn(rows, cols, generator=g, dtype=torch.float64) * scale
    x *= torch.exp2(torch.randint(-6, 7, (rows, 1), generator=g).double())
    return x.to(dtype)


def _special(dtype):
    """Rows of 96 columns, whose groups hold the values where the format can go wrong."""
    f = torch.finfo(dtype)
    tiny = f.smallest_normal * f.eps   # the smallest subnormal
    lists = [
        [0.0] * 32,
        [-0.0] * 32,
        [tiny] + [0.0] * 31,
        [f.smallest_normal, -f.smallest_normal / 2, tiny * 3] + [0.0] * 29,
        [f.max, -f.max, f.max / 2] + [1.0] * 29,
        [f.max / 128, f.max / 3] + [0.0] * 30,
        [127.0, 126.5, 125.5, -0.5, 0.5, 1.5, -1.5, 2.5] + [3.5] * 24,          # ties
        [127.5, 1.0, 0.5, -0.5, 1.5] + [63.0] * 27,                              # the next scale
        [127.0, 127.4375 if dtype != torch.bfloat16 else 127.0, 0.0, -127.0] + [1.0] * 28,
        [1.9921875, 0.0078125, 0.015625, -0.0234375] + [1.0] * 28,
        [1.984375] * 32,
        [float("nan")] + [1.0] * 31,
        [1.0] * 31 + [float("inf")],
        [float("-inf"), float("nan")] + [0.0] * 30,
        [float(i) for i in range(-16, 16)],
    ]
    v = torch.tensor(lists, dtype=torch.float64).reshape(-1)
    v = v.reshape(-1, 96) if v.numel() % 96 == 0 else torch.cat([v, torch.zeros(96 - v.numel() % 96)]).reshape(-1, 96)
    return v.to(dtype)


def _ckpt(x):
    codes, exps = A.encode(x)
    return torch.from_numpy(A.to_buffer(codes, exps)).cuda(), codes, exps


def _check_pack(x, pad):
    rows, cols = x.shape
    codes, exps = A.encode(x)
    size, off = A.layout(rows, cols)
    assert G.gq_act_layout(rows, cols) == (size, 0, off)
    buf = torch.full((size + 64,), FILL, dtype=torch.uint8, device="cuda")
    G.gq_act_pack(_padded(x, pad, 7.0), buf)
    got = buf.cpu().numpy()
    cp, ep = A.pitches(cols)
    assert np.array_equal(got[:rows * cp].view(np.int8).reshape(rows, cp), codes)
    assert np.array_equal(got[off:off + rows * ep].reshape(rows, ep), exps)
    assert (got[rows * cp:off] == FILL).all() and (got[off + rows * ep:] == FILL).all()
    return codes, exps


def _check_unpack(codes, exps, cols, dtype, pad):
    rows = codes.shape[0]
    buf = torch.from_numpy(A.to_buffer(codes, exps)).cuda()
    wide = torch.full((rows, cols + pad), 7.0, dtype=dtype, device="cuda")
    G.gq_act_unpack(buf, wide[:, :cols])
    want = A.as_type(A.decode(codes, exps, cols), dtype)
    got = wide.cpu()
    assert torch.equal(torch.nan_to_num(got[:, :cols].float(), nan=-1e30), torch.nan_to_num(want.float(), nan=-1e30))
    assert (got[:, cols:] == 7.0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (1, 32, 0), (3, 33, 0), (5, 31, 1), (2, 8, 8), (7, 100, 4),
                                           (16, 128, 0), (9, 257, 7), (33, 1000, 24), (4, 1024, 0), (300, 129, 0),
                                           (2, 70001, 0), (3000, 40, 0)])
def test_pack_and_unpack(dtype, rows, cols, pad):
    codes, exps = _check_pack(_values(rows, cols, dtype, rows * 7 + cols), pad)
    for out in TYPES:
        _check_unpack(codes, exps, cols, out, pad)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pad", [0, 3])
def test_pack_special_values(dtype, pad):
    x = _special(dtype)
    codes, exps = _check_pack(x, pad)
    for out in TYPES:
        _check_unpack(codes, exps, x.shape[1], out, pad)


@pytest.mark.parametrize("pad", [0, 3])
def test_unpack_every_code_and_exponent(pad):
    """Every code under every exponent byte, -128 (which pack never writes) among them."""
    exps = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 8, 1)
    codes = np.tile(np.arange(-128, 128).astype(np.int8), (256, 1))
    for out in TYPES:
        _check_unpack(codes, exps, 256, out, pad)


def test_pack_reads_repeated_and_overlapping_rows():
    row = _values(1, 300, torch.bfloat16, 3).cuda()
    want = torch.zeros(G.gq_act_layout(5, 300)[0], dtype=torch.uint8, device="cuda")
    got = torch.zeros_like(want)
    G.gq_act_pack(row.repeat(5, 1), want)
    G.gq_act_pack(row.expand(5, 300), got)
    assert torch.equal(got, want)
    flat = _values(1, 400, torch.float32, 4).cuda()[0]
    windows = flat.as_strided((6, 64), (5, 1))
    want = torch.zeros(G.gq_act_layout(6, 64)[0], dtype=torch.uint8, device="cuda")
    got = torch.zeros_like(want)
    G.gq_act_pack(windows.contiguous(), want)
    G.gq_act_pack(windows, got)
    assert torch.equal(got, want)


# ------------------------------------------------------------------------------------------------
# activation functions
# ------------------------------------------------------------------------------------------------
def _fn_inputs(rows, cols, dtype, seed):
    g = _gen(seed)
    x = (torch.randn(rows, cols, generator=g, dtype=torch.float64) * 3).to(dtype)
    dy = torch.randn(rows, cols, generator=g, dtype=torch.float64).to(dtype)
    return x, dy


@pytest.mark.parametrize("kind", ["gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (3, 40, 0), (5, 33, 0), (17, 1000, 8), (65, 515, 3), (4, 4096, 0)])
def test_fn(kind, dtype, rows, cols, pad):
    x, dy = _fn_inputs(rows, cols, dtype, rows + cols)
    size = G.gq_act_layout(rows, cols)[0]
    ck = torch.zeros(size, dtype=torch.uint8, device="cuda")
    gx, gdy = _padded(x, pad), _padded(dy, pad)
    y, y2, dx = _padded(x * 0, pad, 7.0), _padded(x * 0, pad, 7.0), _padded(x * 0, pad, 7.0)
    G.gq_act_fn_forward(kind, gx, y, ck)
    G.gq_act_fn_forward(kind, gx, y2)
    want_ck, codes, exps = _ckpt(x)
    assert torch.equal(ck, want_ck)
    assert torch.equal(y, y2)
    G.gq_act_fn_backward(kind, ck, gdy, dx)
    half = A.HALF_STEP[dtype]
    # binary32: about 8 roundings of results and an exponential whose argument, of size a, carries 4
    f, _, a = A.fn(kind, x.double())
    tol = f.abs() * (half + 2.0 ** -24 * (8 + 4 * a)) + torch.finfo(dtype).smallest_normal
    assert ((y.cpu().double() - f).abs() <= tol).all()
    xh = A.decode(codes, exps, cols)
    _, df, a = A.fn(kind, xh)
    # the derivative's two terms may cancel: their sizes are at most |x| + 1 times the exponentials'
    terms = torch.where(xh < 0, torch.exp(-torch.minimum(a / 2 if kind == "gelu" else a, torch.tensor(700.0).double())), 1.0)
    terms = terms * (1 + xh.abs()) * (1 + (xh * xh if kind == "gelu_tanh" else 0))
    want = dy.double() * df
    tol = want.abs() * half + dy.double().abs() * terms * 2.0 ** -24 * (8 + 4 * a) + torch.finfo(dtype).smallest_normal
    assert ((dx.cpu().double() - want).abs() <= tol).all()
    wide = y.as_strided((rows, cols + pad), (cols + pad, 1))
    assert (wide[:, cols:] == 7.0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", [64, 72])
def test_fn_between_halves_of_one_buffer(dtype, cols):
    """Input and output as column halves of one buffer share rows but no element; nothing else is touched."""
    x, dy = _fn_inputs(50, cols, dtype, 3)
    buf = torch.full((50, 2 * cols + 16), 7.0, dtype=dtype, device="cuda")
    a, b = buf[:, :cols], buf[:, cols + 8:2 * cols + 8]
    a.copy_(x)
    want, ck = torch.empty(50, cols, dtype=dtype, device="cuda"), torch.zeros(G.gq_act_layout(50, cols)[0], dtype=torch.uint8,
                                                                            device="cuda")
    G.gq_act_fn_forward("silu", x.cuda(), want)
    G.gq_act_fn_forward("silu", a, b, ck)
    assert torch.equal(b, want) and torch.equal(a.cpu(), x)
    assert (buf[:, cols:cols + 8] == 7.0).all() and (buf[:, 2 * cols + 8:] == 7.0).all()
    G.gq_act_fn_backward("silu", ck, dy.cuda(), want)
    a.copy_(dy)
    G.gq_act_fn_backward("silu", ck, a, b)
    assert torch.equal(b, want) and torch.equal(a.cpu(), dy)
    with pytest.raises(G.GQError):
        G.gq_act_fn_forward("silu", a, buf[:, cols - 8:2 * cols - 8])


@pytest.mark.parametrize("kind", ["gelu", "gelu_tanh", "silu"])
def test_fn_far_values(kind):
    """Far out the functions are 0 or x and their derivatives 0 or 1, also where x^2 or x^3 overflows."""
    x = torch.tensor([[-3e38, -1e20, -1e13, -200.0, 200.0, 1e13, 1e20, 3e38] + [0.0] * 24] * 4)
    for r in range(4):   # one large value per group, so that the codes keep it
        x[r] = torch.where(torch.arange(32) == 2 * r, x[r], 0.0)
    dy = torch.ones_like(x)
    ck = torch.zeros(G.gq_act_layout(4, 32)[0], dtype=torch.uint8, device="cuda")
    y, dx = torch.empty(4, 32, device="cuda"), torch.empty(4, 32, device="cuda")
    G.gq_act_fn_forward(kind, x.cuda(), y, ck)
    G.gq_act_fn_backward(kind, ck, dy.cuda(), dx)
    big = x.abs() >= 200
    assert torch.equal(y.cpu()[big], x.clamp(min=0.0)[big])
    assert torch.equal(dx.cpu()[big], (x > 0).float()[big])
    assert torch.equal(dx.cpu()[~big], torch.full_like(dx.cpu()[~big], 0.5))


@pytest.mark.parametrize("kind", ["gelu", "gelu_tanh", "silu"])
def test_fn_gradient_against_differences(kind):
    """The kernel's gradient against central differences of the 64-bit function at the kept values."""
    x, dy = _fn_inputs(4, 64, torch.float32, 9)
    ck, codes, exps = _ckpt(x)
    dx = torch.empty(4, 64, device="cuda")
    G.gq_act_fn_backward(kind, ck, dy.cuda(), dx)
    xh, h = A.decode(codes, exps, 64), 1e-4
    diff = dy.double() * (A.fn(kind, xh + h)[0] - A.fn(kind, xh - h)[0]) / (2 * h)
    # central differences are off by h^2 f'''/6, |f'''| < 2 here, and by 2^-52 |f| / h
    assert ((dx.cpu().double() - diff).abs() <= dy.double().abs() * (1e-8 + 1e-10 + 2.0 ** -24 * 100)).all()


# ------------------------------------------------------------------------------------------------
# the weight gradient
# ------------------------------------------------------------------------------------------------
def _wgrad_want(x, dy):
    """(ckpt, dw, sum |dy||xh|, db, sum |dy|) in 64 bits."""
    ck, codes, exps = _ckpt(x)
    xh = A.as_type(A.decode(codes, exps, x.shape[1]), dy.dtype if dy.dtype == torch.float16 else torch.float32).double()
    d = dy.double()
    return ck, d.t() @ xh, d.abs().t() @ xh.abs(), d.sum(0), d.abs().sum(0)


def _wgrad_tol(tokens, size):
    """The sums: every 16 products join the accumulator with at most two steps' error (2^-22 of the sum of
    sizes so far), and up to 8 parts of the tokens and 3 parts of a float32 gradient are joined after that."""
    return (tokens / 16 + 16) * 2.0 ** -22 * size + 1e-37


SHAPES = [(1, 16, 16, 0), (1, 1, 1, 0), (2, 33, 7, 0), (64, 128, 128, 0), (63, 100, 257, 0), (129, 40, 300, 5),
          (200, 1000, 130, 8), (515, 129, 65, 3), (1000, 256, 512, 0), (2049, 384, 264, 8), (40, 2048, 1024, 0)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,cin,cout,pad", SHAPES)
def test_weight_grad(dtype, tokens, cin, cout, pad):
    x = _values(tokens, cin, dtype, tokens + cin)
    dy = _values(tokens, cout, dtype, tokens + cout, 0.01)
    dy[tokens // 2] = 0.0
    ck, dw, size, db, dsize = _wgrad_want(x, dy)
    flat = torch.full((cout * cin + cout + 3,), 5.0, device="cuda")
    gdw, gdb = flat[1:1 + cout * cin].view(cout, cin), flat[1 + cout * cin:1 + cout * cin + cout]
    gdy = _padded(dy, pad)
    G.gq_act_weight_grad(ck, gdy, gdw, gdb)
    assert ((gdw.cpu().double() - dw).abs() <= _wgrad_tol(tokens, size)).all()
    assert ((gdb.cpu().double() - db).abs() <= (tokens + 16) * 2.0 ** -24 * dsize + 1e-37).all()
    first = flat.clone()
    # again, added: the same bits twice, one rounding more
    G.gq_act_weight_grad(ck, gdy, gdw, gdb, accumulate=True)
    assert torch.equal(flat[1:-2], first[1:-2] * 2)
    assert flat[0] == 5.0 and (flat[-2:] == 5.0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,cin,cout", [(700, 2600, 2500), (5000, 700, 650), (9001, 256, 256), (70, 5000, 4999)])
def test_weight_grad_many_tiles(dtype, tokens, cin, cout):
    """More tiles than CTA pairs, tiles cut along the tokens, long sums; the 64-bit product on the GPU."""
    x, dy = _values(tokens, cin, dtype, 1), _values(tokens, cout, dtype, 2, 0.01)
    ck, codes, exps = _ckpt(x)
    xh = A.as_type(A.decode(codes, exps, cin), torch.float16 if dtype == torch.float16 else torch.float32).double().cuda()
    d = dy.double().cuda()
    dw = torch.empty(cout, cin, device="cuda")
    G.gq_act_weight_grad(ck, dy.cuda(), dw)
    # runs of 512 tokens lose at most two steps every 16 tokens, their sums one rounding each
    steps = min(tokens, 512) / 16 * 2 + 3 * tokens / 512 + 16
    assert ((dw.double() - d.t() @ xh).abs() <= steps * 2.0 ** -23 * (d.abs().t() @ xh.abs())).all()


def test_weight_grad_strided_output_and_no_bias():
    x, dy = _values(70, 72, torch.bfloat16, 1), _values(70, 40, torch.bfloat16, 2)
    ck, dw, size, _, _ = _wgrad_want(x, dy)
    wide = torch.full((40, 91), 3.0, device="cuda")
    G.gq_act_weight_grad(ck, dy.cuda(), wide[:, 5:77])
    got = wide.cpu().double()
    assert ((got[:, 5:77] - dw).abs() <= _wgrad_tol(70, size)).all()
    assert (got[:, :5] == 3.0).all() and (got[:, 77:] == 3.0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_weight_grad_without_tokens(dtype):
    dw, db = torch.full((9, 40), 4.0, device="cuda"), torch.full((9,), 4.0, device="cuda")
    ck = torch.zeros(16, dtype=torch.uint8, device="cuda")
    dy = torch.empty(0, 9, dtype=dtype, device="cuda")
    G.gq_act_weight_grad(ck, dy, dw, db, accumulate=True)
    assert (dw == 4.0).all() and (db == 4.0).all()
    G.gq_act_weight_grad(ck, dy, dw, db)
    assert (dw == 0.0).all() and (db == 0.0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_weight_grad_of_repeated_rows(dtype):
    """A gradient whose rows are one row (what a sum over tokens passes back)."""
    x, row = _values(130, 96, dtype, 5), _values(1, 72, dtype, 6)
    dy = row.expand(130, 72)
    ck, dw, size, db, dsize = _wgrad_want(x, dy)
    gdw, gdb = torch.empty(72, 96, device="cuda"), torch.empty(72, device="cuda")
    G.gq_act_weight_grad(ck, row.cuda().expand(130, 72), gdw, gdb)
    assert ((gdw.cpu().double() - dw).abs() <= _wgrad_tol(130, size)).all()
    assert ((gdb.cpu().double() - db).abs() <= 150 * 2.0 ** -24 * dsize).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_weight_grad_non_finite(dtype):
    """A NaN group reaches its 32 columns of every row of dw, an infinite gradient its row."""
    x, dy = _values(100, 96, dtype, 7), _values(100, 20, dtype, 8)
    x[50, 40] = float("nan")
    dy[60, 3] = float("inf")
    ck, _, _, _, _ = _wgrad_want(x, dy)
    gdw = torch.empty(20, 96, device="cuda")
    G.gq_act_weight_grad(ck, dy.cuda(), gdw)
    bad = ~torch.isfinite(gdw.cpu())
    want = torch.zeros(20, 96, dtype=torch.bool)
    want[:, 32:64] = True
    want[3] = True
    assert torch.equal(bad, want)


@pytest.mark.parametrize("dtype", TYPES)
def test_weight_grad_sizes_of_values(dtype):
    """Inputs and gradients at the ends of their types' range."""
    f = torch.finfo(dtype)
    for sx, sdy in [(f.smallest_normal * 8, 1.0), (1.0, f.smallest_normal * 64), (f.max / 1e3, 2.0 ** -10)]:
        g = _gen(11)
        x = ((torch.rand(90, 64, generator=g, dtype=torch.float64) * 2 - 1) * sx).to(dtype)
        dy = ((torch.rand(90, 48, generator=g, dtype=torch.float64) * 2 - 1) * sdy).to(dtype)
        ck, dw, size, _, _ = _wgrad_want(x, dy)
        gdw = torch.empty(48, 64, device="cuda")
        G.gq_act_weight_grad(ck, dy.cuda(), gdw)
        # products below binary32's normal range lose up to its smallest step each
        assert ((gdw.cpu().double() - dw).abs() <= _wgrad_tol(90, size) + 90 * 2.0 ** -126).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens", [255, 25])
def test_weight_grad_decodes_every_code_and_exponent(dtype, tokens):
    """Token t holds every code under exponent byte E and dy is 1 at (t, t) and 0 elsewhere, so row t of dw
    is the decoded row, exactly; with all 255 finite exponents, and with some of them a few tokens at a time."""
    for lo in range(0, 255, tokens):
        n = min(tokens, 255 - lo)
        exps = np.repeat(np.arange(lo, lo + n, dtype=np.uint8)[:, None], 8, 1)
        codes = np.tile(np.arange(-128, 128).astype(np.int8), (n, 1))
        # -128 * 2^121 is -2^128, beyond binary32: no number, and no code that a pack writes
        codes[exps[:, 0] == 254, 0] = -127
        want = A.as_type(A.decode(codes, exps, 256), dtype if dtype == torch.float16 else torch.float32).float()
        dw = torch.empty(n, 256, device="cuda")
        G.gq_act_weight_grad(torch.from_numpy(A.to_buffer(codes, exps)).cuda(), torch.eye(n, dtype=dtype, device="cuda"), dw)
        assert torch.equal(dw.cpu(), want)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,cin,cout", [(32, 40, 70), (33, 40, 70), (32, 2048, 1024), (32, 2048, 1025), (8, 1000, 8389),
                                             (64, 256, 256), (65, 257, 255), (512, 64, 300), (513, 64, 301)])
def test_weight_grad_around_the_choice_of_kernel(dtype, tokens, cin, cout):
    x, dy = _values(tokens, cin, dtype, 3), _values(tokens, cout, dtype, 4, 0.1)
    ck, dw, size, db, dsize = _wgrad_want(x, dy)
    gdw, gdb = torch.empty(cout, cin, device="cuda"), torch.empty(cout, device="cuda")
    G.gq_act_weight_grad(ck, dy.cuda(), gdw, gdb)
    assert ((gdw.cpu().double() - dw).abs() <= _wgrad_tol(tokens, size)).all()
    assert ((gdb.cpu().double() - db).abs() <= (tokens + 16) * 2.0 ** -24 * dsize + 1e-37).all()


def test_weight_grad_against_differences():
    """dw against differences of the loss sum(dy * (xh W^T)), which is linear in W: exact up to rounding."""
    x, dy = _values(30, 40, torch.bfloat16, 12), _values(30, 8, torch.bfloat16, 13)
    ck, codes, exps = _ckpt(x)
    xh = A.decode(codes, exps, 40)
    gdw = torch.empty(8, 40, device="cuda")
    G.gq_act_weight_grad(ck, dy.cuda(), gdw)
    w = torch.randn(8, 40, generator=_gen(14), dtype=torch.float64)
    loss = lambda w: (dy.double() * (xh @ w.t())).sum()
    size = dy.double().abs().t() @ xh.abs()
    for n, k in [(0, 0), (3, 17), (7, 39)]:
        e = torch.zeros_like(w)
        e[n, k] = 0.5
        diff = loss(w + e) - loss(w - e)
        assert abs(gdw[n, k].item() - diff.item()) <= _wgrad_tol(30, size[n, k].item()) + 1e-9 * abs(loss(w).item() + 1)


@pytest.mark.parametrize("dtype", TYPES)
def test_weight_grad_first_in_a_capture_of_its_own_workspace(dtype):
    """A captured call that allocates its workspace itself (from the graph's pool), twice in one graph."""
    x, dy = _values(600, 520, dtype, 8), _values(600, 264, dtype, 9, 0.1)
    ck, _, _ = _ckpt(x)
    gdy = dy.cuda()
    want, wantb = torch.empty(264, 520, device="cuda"), torch.empty(264, device="cuda")
    G.gq_act_weight_grad(ck, gdy, want, wantb)
    outs = [(torch.zeros_like(want), torch.zeros_like(wantb)) for _ in range(2)]
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for dw, db in outs:
            G.gq_act_weight_grad(ck, gdy, dw, db)
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for dw, db in outs:
        assert torch.equal(dw, want) and torch.equal(db, wantb)


# ------------------------------------------------------------------------------------------------
# streams and graphs
# ------------------------------------------------------------------------------------------------
def _block(dtype, seed):
    x, dy = _values(200, 136, dtype, seed), _values(200, 72, dtype, seed + 1)
    return x.cuda(), dy.cuda()


@pytest.mark.parametrize("dtype", TYPES)
def test_side_stream_and_repeat(dtype):
    """On a stream passed explicitly (its workspace allocated by the call) and again: the same bits."""
    x, dy = _block(dtype, 20)
    ck = torch.zeros(G.gq_act_layout(200, 136)[0], dtype=torch.uint8, device="cuda")
    outs = []
    for k in range(3):
        s = torch.cuda.Stream() if k else torch.cuda.current_stream()
        s.wait_stream(torch.cuda.current_stream())
        dw, db = torch.empty(72, 136, device="cuda"), torch.empty(72, device="cuda")
        G.gq_act_pack(x, ck, stream=s)
        G.gq_act_weight_grad(ck, dy, dw, db, stream=s if k < 2 else s.cuda_stream)
        s.synchronize()
        outs.append((dw, db))
    for dw, db in outs[1:]:
        assert torch.equal(dw, outs[0][0]) and torch.equal(db, outs[0][1])


@pytest.mark.parametrize("dtype", TYPES)
def test_captured_and_replayed(dtype):
    """Two graphs with workspaces of their own, replayed on new inputs, in both orders."""
    x, dy = _block(dtype, 30)

    def capture():
        ck = torch.zeros(G.gq_act_layout(200, 136)[0], dtype=torch.uint8, device="cuda")
        y, dx = torch.empty_like(x), torch.empty_like(x)
        dw, db = torch.empty(72, 136, device="cuda"), torch.empty(72, device="cuda")
        ws = G.gq_act_weight_grad_workspace(ck, dy, dw, db)

        def step():
            G.gq_act_fn_forward("silu", x, y, ck)
            G.gq_act_weight_grad(ck, dy, dw, db, workspace=ws)
            G.gq_act_fn_backward("silu", ck, x, dx)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        return g, step, (y, dx, dw, db)

    graphs = [capture() for _ in range(2)]
    nx, ndy = _block(dtype, 40)
    x.copy_(nx)
    dy.copy_(ndy)
    for g, _, outs in reversed(graphs):
        for o in outs:
            o.zero_()
        g.replay()
    torch.cuda.synchronize()
    got = [[o.clone() for o in outs] for _, _, outs in graphs]
    graphs[0][1]()
    for outs in got:
        for a, b in zip(outs, graphs[0][2]):
            assert torch.equal(a, b)
