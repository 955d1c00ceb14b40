"""GPU tests of layer norm (gq_layer_norm_forward / gq_layer_norm_backward), with and without the
8-bit checkpoint of its input, against 64-bit computations on the CPU."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import act_oracle as A
import gradient_quantization_communication_b200.gq as G

TYPES = [torch.float32, torch.bfloat16, torch.float16]
U = 2.0 ** -24


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _inputs(rows, cols, dtype, param, seed, offset=0.3):
    g = _gen(seed)
    x = (torch.randn(rows, cols, generator=g, dtype=torch.float64) * torch.exp(torch.randn(rows, 1, generator=g)) + offset)
    dy = torch.randn(rows, cols, generator=g, dtype=torch.float64)
    dy[rows // 3] = 0.0
    gamma = 1 + 0.3 * torch.randn(cols, generator=g, dtype=torch.float64)
    beta = 0.2 * torch.randn(cols, generator=g, dtype=torch.float64)
    return x.to(dtype), dy.to(dtype), gamma.to(param), beta.to(param)


def _padded(x, pad, fill=0.0):
    rows, cols = x.shape
    buf = torch.full((rows, cols + pad), fill, dtype=x.dtype, device="cuda")
    buf[:, :cols] = x.cuda()
    return buf[:, :cols]


def _depth(cols):
    """Additions on the way of one value into a row's sum: at most cols / 32 in a thread (a warp or more take
    a row), 5 in the warp, 16 over the warps, and the division's two roundings."""
    return cols / 32 + 24


def _forward_tol(x, y, mean, rstd, gamma, beta, eps, dtype):
    """(y, mean, rstd) bounds.  The mean is off by depth roundings of mean |x|; the centred values by that and
    one rounding; the variance by twice its relative error (depth + 4 roundings) and the mean's square; rstd by
    half of the variance's relative error and 3 roundings; y by these, 3 roundings more and its type's."""
    d = _depth(x.shape[1])
    em = d * U * x.abs().mean(1, keepdim=True) + 1e-44
    var = ((x - mean) ** 2).mean(1, keepdim=True)
    ev = (d + 6) * U * var + 2 * em * (var.sqrt() + em) + U * em * x.abs().amax(1, keepdim=True)
    er = rstd * (0.5 * (ev + 2 * U * (var + eps)) / (var + eps) + 4 * U)
    ey = gamma.abs() * (rstd * (em + U * x.abs()) + (x - mean).abs() * er) + 4 * U * ((y - beta).abs() + beta.abs())
    return ey + A.HALF_STEP[dtype] * y.abs() * 1.01 + torch.finfo(dtype).smallest_normal, em, er


SHAPES = [(1, 1, 0), (3, 8, 0), (2, 7, 1), (5, 33, 0), (4, 256, 0), (7, 300, 8), (19, 1000, 0), (6, 1001, 0), (130, 768, 16),
          (300, 512, 0), (3, 2051, 5), (5, 4096, 0), (17, 4100, 12), (2, 8192, 0), (3, 8200, 0), (2, 16384, 0), (2, 20001, 0)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,pad", SHAPES)
@pytest.mark.parametrize("same", [True, False])
def test_forward_and_backward(dtype, rows, cols, pad, same):
    eps = 1e-5
    x, dy, gamma, beta = _inputs(rows, cols, dtype, dtype if same else torch.float32, rows + cols)
    X, DY, GA, BE = x.double(), dy.double(), gamma.double(), beta.double()
    y, mean, rstd = A.norm(X, GA, BE, eps)
    gx, gdy = _padded(x, pad), _padded(dy, pad)
    gy, gy2, gdx = (_padded(x * 0, pad, 7.0) for _ in range(3))
    stats = torch.full((2, rows + 2), 9.0, device="cuda")
    gm, gr = stats[0, 1:rows + 1], stats[1, 1:rows + 1]
    ck = torch.zeros(G.gq_act_layout(rows, cols)[0], dtype=torch.uint8, device="cuda")
    G.gq_layer_norm_forward(gx, gamma.cuda(), beta.cuda(), eps, gy2, gm, gr)
    G.gq_layer_norm_forward(gx, gamma.cuda(), beta.cuda(), eps, gy, gm, gr, ck)
    assert torch.equal(gy, gy2)
    codes, exps = A.encode(x)
    assert np.array_equal(ck.cpu().numpy(), A.to_buffer(codes, exps))
    ey, em, er = _forward_tol(X, y, mean, rstd, GA, BE, eps, dtype)
    m, r = gm.cpu().double()[:, None], gr.cpu().double()[:, None]
    assert ((m - mean).abs() <= em).all()
    assert ((r - rstd).abs() <= er).all()
    assert ((gy.cpu().double() - y).abs() <= ey).all()
    assert (gy.as_strided((rows, cols + pad), (cols + pad, 1))[:, cols:] == 7.0).all()
    assert (stats[:, 0] == 9.0).all() and (stats[:, -1] == 9.0).all()
    # backward, given the kernel's mean and rstd as data: from the input, then from the checkpoint
    for src, xs in ((gx, X), (ck, A.decode(codes, exps, cols))):
        dx, dg, db = A.norm_backward(DY, xs, GA, m, r)
        flat = torch.full((2 * cols + 3,), 5.0, device="cuda")
        gdg, gdb = flat[1:1 + cols], flat[1 + cols:1 + 2 * cols]
        G.gq_layer_norm_backward(gdy, src, gamma.cuda(), gm, gr, gdx, gdg, gdb)
        d = _depth(cols)
        xh, g = (xs - m) * r, DY * GA
        exh = 2 * U * xh.abs() + U * r * xs.abs()                         # xh: two roundings and the difference's
        s0, s1 = g.abs().mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True)
        e0 = (d + 2) * U * s0
        e1 = (d + 4) * U * s1 + (g.abs() * exh).mean(1, keepdim=True)
        c1 = (g * xh).mean(1, keepdim=True).abs()
        tol = r * (3 * U * g.abs() + e0 + U * s0 + xh.abs() * e1 + exh * c1 + 4 * U * xh.abs() * c1) + 3 * U * dx.abs()
        tol = tol + A.HALF_STEP[dtype] * (dx.abs() + tol) + torch.finfo(dtype).smallest_normal
        assert ((gdx.cpu().double() - dx).abs() <= tol).all()
        # sums over rows: at most rows + 64 additions of a value
        n = (rows + 64) * U
        assert ((gdg.cpu().double() - dg).abs() <= n * (DY * xh).abs().sum(0) + (DY.abs() * exh).sum(0) + 1e-37).all()
        assert ((gdb.cpu().double() - db).abs() <= n * DY.abs().sum(0) + 1e-37).all()
        first = flat.clone()
        G.gq_layer_norm_backward(gdy, src, gamma.cuda(), gm, gr, gdx, gdg, gdb, accumulate=True)
        assert torch.equal(flat[1:-2], first[1:-2] * 2)
        assert flat[0] == 5.0 and (flat[-2:] == 5.0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_many_rows(dtype):
    """More rows than partial sums, few columns."""
    rows, cols = 5003, 72
    x, dy, gamma, beta = _inputs(rows, cols, dtype, torch.float32, 5)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    y, dx = torch.empty_like(x, device="cuda"), torch.empty_like(x, device="cuda")
    dg, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    G.gq_layer_norm_forward(x.cuda(), gamma.cuda(), beta.cuda(), 1e-5, y, mean, rstd)
    G.gq_layer_norm_backward(dy.cuda(), x.cuda(), gamma.cuda(), mean, rstd, dx, dg, db)
    m, r = mean.cpu().double()[:, None], rstd.cpu().double()[:, None]
    _, wg, wb = A.norm_backward(dy.double(), x.double(), gamma.double(), m, r)
    xh = (x.double() - m) * r
    assert ((dg.cpu().double() - wg).abs() <= (rows + 64) * U * (dy.double() * xh).abs().sum(0)).all()
    assert ((db.cpu().double() - wb).abs() <= (rows + 64) * U * dy.double().abs().sum(0)).all()


@pytest.mark.parametrize("gamma,beta", [(True, False), (False, True), (False, False)])
def test_without_parameters(gamma, beta):
    x, dy, g, b = _inputs(9, 264, torch.bfloat16, torch.bfloat16, 1)
    gg, gb = (g.cuda() if gamma else None), (b.cuda() if beta else None)
    ones, zeros = torch.ones_like(g).cuda(), torch.zeros_like(b).cuda()
    outs = []
    for pg, pb in ((gg, gb), (gg if gamma else ones, gb if beta else zeros)):
        y, dx = torch.empty_like(x, device="cuda"), torch.empty_like(x, device="cuda")
        m, r = torch.empty(9, device="cuda"), torch.empty(9, device="cuda")
        G.gq_layer_norm_forward(x.cuda(), pg, pb, 1e-6, y, m, r)
        G.gq_layer_norm_backward(dy.cuda(), x.cuda(), pg, m, r, dx, None, None)
        outs.append((y, m, r, dx))
    for a, c in zip(*outs):
        assert torch.equal(a, c)


def test_one_gradient_wanted():
    x, dy, g, _ = _inputs(50, 200, torch.float32, torch.float32, 2)
    m, r = torch.zeros(50, device="cuda"), torch.ones(50, device="cuda")
    dx = torch.empty(50, 200, device="cuda")
    both = [torch.empty(200, device="cuda") for _ in range(2)]
    one = [torch.empty(200, device="cuda") for _ in range(2)]
    G.gq_layer_norm_backward(dy.cuda(), x.cuda(), g.cuda(), m, r, dx, *both)
    G.gq_layer_norm_backward(dy.cuda(), x.cuda(), g.cuda(), m, r, dx, one[0], None)
    G.gq_layer_norm_backward(dy.cuda(), x.cuda(), g.cuda(), m, r, dx, None, one[1])
    assert torch.equal(both[0], one[0]) and torch.equal(both[1], one[1])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("cols", [64, 1003, 30000])
def test_constant_rows_and_large_means(dtype, cols):
    """A constant row has variance 0 (y = beta); a row whose mean is far larger than its spread keeps its
    digits, since the squares are summed around the mean."""
    x = torch.zeros(4, cols, dtype=torch.float64)
    x[0] = 0.0
    x[1] = 3.0
    x[2] = 1024.0 + 4.0 * (torch.arange(cols) % 8).double()   # exact in bf16 (steps of 8) after rounding, in fp16 too
    x[3] = torch.randn(cols, generator=_gen(3), dtype=torch.float64) * 1e-3
    x = x.to(dtype)
    X = x.double()
    y, m, r = (torch.empty(4, cols, dtype=dtype, device="cuda"), torch.empty(4, device="cuda"), torch.empty(4, device="cuda"))
    G.gq_layer_norm_forward(x.cuda(), None, None, 1e-5, y, m, r)
    wy, wm, wr = A.norm(X, torch.ones(cols).double(), torch.zeros(cols).double(), 1e-5)
    ey, em, er = _forward_tol(X, wy, wm, wr, torch.ones(cols).double(), torch.zeros(cols).double(), 1e-5, dtype)
    assert ((m.cpu().double()[:, None] - wm).abs() <= em).all()
    assert ((r.cpu().double()[:, None] - wr).abs() <= er).all()
    assert ((y.cpu().double() - wy).abs() <= ey).all()


def test_non_finite_rows_stay_apart():
    x, dy, g, b = _inputs(8, 300, torch.bfloat16, torch.float32, 3)
    x[2, 7], x[5, 299] = float("nan"), float("inf")
    y, m, r = torch.empty_like(x, device="cuda"), torch.empty(8, device="cuda"), torch.empty(8, device="cuda")
    dx, dg, db = torch.empty_like(x, device="cuda"), torch.empty(300, device="cuda"), torch.empty(300, device="cuda")
    ck = torch.zeros(G.gq_act_layout(8, 300)[0], dtype=torch.uint8, device="cuda")
    G.gq_layer_norm_forward(x.cuda(), g.cuda(), b.cuda(), 1e-5, y, m, r, ck)
    G.gq_layer_norm_backward(dy.cuda(), ck, g.cuda(), m, r, dx, dg, db)
    good = torch.tensor([i not in (2, 5) for i in range(8)])
    for t in (y.cpu(), dx.cpu()):
        assert torch.isfinite(t[good].float()).all() and not torch.isfinite(t[~good].float()).any()
    assert torch.isfinite(db.cpu()).all()


def test_no_rows():
    e = torch.empty(0, 40, device="cuda")
    m = torch.empty(0, device="cuda")
    dg, db = torch.full((40,), 2.0, device="cuda"), torch.full((40,), 2.0, device="cuda")
    G.gq_layer_norm_forward(e, None, None, 1e-5, e.clone(), m, m.clone())
    G.gq_layer_norm_backward(e, e.clone(), None, m, m.clone(), e.clone(), dg, db, accumulate=True)
    assert (dg == 2.0).all() and (db == 2.0).all()
    G.gq_layer_norm_backward(e, e.clone(), None, m, m.clone(), e.clone(), dg, db)
    assert (dg == 0.0).all() and (db == 0.0).all()


def test_repeated_gradient_rows():
    """dy whose rows are one row (stride 0): as if copied out."""
    x, dy, g, _ = _inputs(33, 520, torch.bfloat16, torch.bfloat16, 6)
    m, r = x.double().mean(1).float().cuda(), (1 / x.double().std(1)).float().cuda()
    outs = []
    for d in (dy[:1].cuda().expand(33, 520), dy[:1].cuda().repeat(33, 1)):
        dx, dg, db = torch.empty_like(x, device="cuda"), torch.empty(520, device="cuda"), torch.empty(520, device="cuda")
        G.gq_layer_norm_backward(d, x.cuda(), g.cuda(), m, r, dx, dg, db)
        outs.append((dx, dg, db))
    for a, c in zip(*outs):
        assert torch.equal(a, c)


def test_gradient_against_differences():
    """dx, dgamma and dbeta against central differences of the 64-bit loss sum(dy * y)."""
    x, dy, g, b = _inputs(3, 40, torch.float32, torch.float32, 7)
    X, DY, GA, BE = x.double(), dy.double(), g.double(), b.double()
    y, m, r = torch.empty(3, 40, device="cuda"), torch.empty(3, device="cuda"), torch.empty(3, device="cuda")
    dx, dg, db = torch.empty(3, 40, device="cuda"), torch.empty(40, device="cuda"), torch.empty(40, device="cuda")
    G.gq_layer_norm_forward(x.cuda(), g.cuda(), b.cuda(), 1e-5, y, m, r)
    G.gq_layer_norm_backward(dy.cuda(), x.cuda(), g.cuda(), m, r, dx, dg, db)
    loss = lambda x, g, b: (DY * A.norm(x, g, b, 1e-5)[0]).sum()
    h = 1e-5
    for what, base, got in (("x", X, dx), ("g", GA, dg), ("b", BE, db)):
        for i in [0, 13, base.numel() - 1]:
            e = torch.zeros(base.numel(), dtype=torch.float64)
            e[i] = h
            e = e.view(base.shape)
            args = {"x": X, "g": GA, "b": BE}
            up, down = dict(args), dict(args)
            up[what], down[what] = base + e, base - e
            diff = (loss(**up) - loss(**down)) / (2 * h)
            # differences: h^2 of the third derivative (below 1e3 for spreads above 0.1) and 2^-52 loss / h;
            # the kernel: some 60 roundings of sums below 100
            assert abs(got.cpu().reshape(-1)[i].item() - diff.item()) <= 1e-7 + 1e-8 + 60 * U * 100


def test_captured_and_replayed():
    x, dy, g, b = _inputs(70, 1024, torch.bfloat16, torch.bfloat16, 8)
    x, dy, g, b = x.cuda(), dy.cuda(), g.cuda(), b.cuda()
    y, dx = torch.empty_like(x), torch.empty_like(x)
    m, r = torch.empty(70, device="cuda"), torch.empty(70, device="cuda")
    dg, db = torch.empty(1024, device="cuda"), torch.empty(1024, device="cuda")
    ck = torch.zeros(G.gq_act_layout(70, 1024)[0], dtype=torch.uint8, device="cuda")
    ws = G.gq_layer_norm_workspace(dy)

    def step():
        G.gq_layer_norm_forward(x, g, b, 1e-5, y, m, r, ck)
        G.gq_layer_norm_backward(dy, ck, g, m, r, dx, dg, db, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    nx, ndy, _, _ = _inputs(70, 1024, torch.bfloat16, torch.bfloat16, 9)
    x.copy_(nx)
    dy.copy_(ndy)
    outs = (y, m, r, dx, dg, db)
    for o in outs:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    got = [o.clone() for o in outs]
    step()
    for a, c in zip(got, outs):
        assert torch.equal(a, c)
