"""Layer norm over more rows than the device holds at once, at widths of every shape the kernels take (chunks a
warp, warps a row, rows a block), so that blocks walk from row to row: against 64 bits on the GPU.  Parameters
that do not start on 16 bytes."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import act_oracle as A
import gradient_quantization_communication_b200.gq as G
from test_act_walk_gpu import decode, encode
from test_norm_gpu import TYPES, U, _depth, _forward_tol

SMALLEST = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}


def _inputs(rows, cols, pad, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    wide = lambda v: torch.cat([v, torch.zeros(rows, pad, device="cuda")], 1).to(dtype)[:, :cols]
    x, dy = wide(r(rows, cols) * torch.exp(r(rows, 1)) + 0.3), wide(r(rows, cols))
    return x, dy, (1 + 0.3 * r(cols)).to(dtype), (0.2 * r(cols)).to(dtype)


def _filled(rows, cols, pad, dtype):
    return torch.full((rows, cols + pad), float("nan"), dtype=dtype, device="cuda")[:, :cols]


# The forward pass takes two chunks of 256 columns a warp up to 768 columns and four above, and one, two, three,
# four, eight or sixteen warps a row; each of them with whole chunks, with rows on 16 bytes, and anywhere.  The
# rows are more than eight blocks an SM hold (256 threads, or a row's warps, a block).
SHAPES = [(10001, 512, 0), (10001, 500, 4), (10001, 499, 0), (6001, 768, 0), (6001, 600, 8), (6001, 601, 0),
          (10001, 1024, 0), (9601, 1000, 0), (9601, 1001, 0), (4801, 2048, 0), (4801, 2000, 8), (4801, 1999, 0),
          (2403, 2600, 0), (2403, 4096, 0), (2403, 4090, 6), (2403, 4095, 0), (1203, 8192, 0), (1203, 7001, 0),
          (603, 16384, 0), (603, 12001, 0), (403, 20000, 0)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols,pad", SHAPES)
def test_many_rows(dtype, rows, cols, pad):
    eps = 1e-5
    x, dy, gamma, beta = _inputs(rows, cols, pad, dtype, rows + cols)
    X, DY, GA, BE = x.double(), dy.double(), gamma.double(), beta.double()
    y, mean, rstd = A.norm(X, GA, BE, eps)
    gy, gy2, gdx = (_filled(rows, cols, pad, dtype) for _ in range(3))
    m, r = (torch.full((rows,), float("nan"), device="cuda") for _ in range(2))
    m2, r2 = m.clone(), r.clone()
    ck, packed = (torch.zeros(A.layout(rows, cols)[0], dtype=torch.uint8, device="cuda") for _ in range(2))
    G.gq_layer_norm_forward(x, gamma, beta, eps, gy, m, r, ck)
    G.gq_layer_norm_forward(x, gamma, beta, eps, gy2, m2, r2)
    G.gq_act_pack(x, packed)
    assert torch.equal(ck, packed)
    assert torch.equal(gy, gy2) and torch.equal(m, m2) and torch.equal(r, r2)
    ey, em, er = _forward_tol(X, y, mean, rstd, GA, BE, eps, dtype)
    ey = ey - torch.finfo(dtype).smallest_normal + SMALLEST[dtype]   # down to subnormal results
    M, R = m.double()[:, None], r.double()[:, None]
    assert ((M - mean).abs() <= em).all()
    assert ((R - rstd).abs() <= er).all()
    assert ((gy.double() - y).abs() <= ey).all()
    del y, ey
    # backward, given the kernel's mean and rstd as data: from the input, then from the checkpoint
    d = _depth(cols)
    for src, xs in ((x, X), (ck, decode(*encode(x), cols))):
        dx, dg, db = A.norm_backward(DY, xs, GA, M, R)
        gdg, gdb = (torch.full((cols,), float("nan"), device="cuda") for _ in range(2))
        gdx.fill_(float("nan"))
        G.gq_layer_norm_backward(dy, src, gamma, m, r, gdx, gdg, gdb)
        xh, g = (xs - M) * R, DY * GA
        exh = 2 * U * xh.abs() + U * R * xs.abs()                        # xh: two roundings and the difference's
        s0, s1 = g.abs().mean(1, keepdim=True), (g * xh).abs().mean(1, keepdim=True)
        e0 = (d + 2) * U * s0
        e1 = (d + 4) * U * s1 + (g.abs() * exh).mean(1, keepdim=True)
        c1 = (g * xh).mean(1, keepdim=True).abs()
        tol = R * (3 * U * g.abs() + e0 + U * s0 + xh.abs() * e1 + exh * c1 + 4 * U * xh.abs() * c1) + 3 * U * dx.abs()
        tol = tol + A.HALF_STEP[dtype] * (dx.abs() + tol) + SMALLEST[dtype]
        assert ((gdx.double() - dx).abs() <= tol).all()
        n = (rows + 64) * U                                              # at most rows + 64 additions of a value
        assert ((gdg.double() - dg).abs() <= n * (DY * xh).abs().sum(0) + (DY.abs() * exh).sum(0) + 1e-37).all()
        assert ((gdb.double() - db).abs() <= n * DY.abs().sum(0) + 1e-37).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(3, 300), (3, 1001), (6001, 600), (2403, 2600), (5, 20001)])
@pytest.mark.parametrize("same", [True, False])
def test_parameters_anywhere(dtype, rows, cols, same):
    """gamma and beta as slices of a flat vector, on their element size only: the same bits as from 16 bytes."""
    x, dy, gamma, beta = _inputs(rows, cols, 0, dtype, 7)
    if not same:
        gamma, beta = gamma.float(), beta.float()
    outs = []
    for odd in (False, True):
        flat = torch.full((2 * cols + 2,), float("nan"), dtype=gamma.dtype, device="cuda")
        g, b = (flat[1:1 + cols], flat[1 + cols:1 + 2 * cols]) if odd else (gamma, beta)
        g.copy_(gamma)
        b.copy_(beta)
        m, r = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        y, dx = torch.empty_like(x), torch.empty_like(x)
        dg, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
        G.gq_layer_norm_forward(x, g, b, 1e-5, y, m, r)
        G.gq_layer_norm_backward(dy, x, g, m, r, dx, dg, db)
        outs.append((y, m, r, dx, dg, db))
    for a, c in zip(*outs):
        assert torch.isfinite(a.float()).all() and torch.equal(a, c)
