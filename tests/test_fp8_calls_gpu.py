"""8-bit floating point by calls that the header allows besides the usual ones: rows that repeat or overlap, several
streams and captured graphs at once, kernels that follow one another without a pause, products of every shape of the
kernels, and a wide range of sizes."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import fp8_oracle as O
import gradient_quantization_communication_b200.gq as G
from test_fp8_gpu import check, check_product, matrix, operand, packed

TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("stride", [0, 5, 8, 264])
def test_rows_that_repeat_or_overlap(dtype, stride):
    """As if copied out."""
    g = torch.Generator(device="cuda").manual_seed(stride)
    flat = torch.randn(300 * stride + 1100, generator=g, device="cuda").to(dtype)
    x = flat.as_strided((301, 1100), (stride, 1))
    for tile in (False, True):
        p, t = packed(301, 1100, tile), packed(1100, 301, tile)
        G.gq_fp8_pack(x, p, t, tile=tile)
        check(p, x.contiguous(), "e4m3", tile)
        check(t, x.contiguous().t(), "e4m3", tile)
        G.gq_fp8_pack(x, p, tile=tile)
        check(p, x.contiguous(), "e4m3", tile)


def test_slices_of_one_buffer():
    """Columns of one wider buffer are packed, and others written, in turn."""
    wide = matrix(200, 640, torch.bfloat16, 1).contiguous()
    x, y = wide[:, :300], wide[:, 304:604]
    kept = wide.clone()
    p = packed(200, 300, False)
    G.gq_fp8_pack(x, p)
    G.gq_fp8_unpack(p, y)
    assert torch.equal(y.cpu(), O.decode(*O.pack(kept[:, :300].cpu(), "e4m3", False), "e4m3", False, 300).bfloat16())
    assert torch.equal(wide[:, :304], kept[:, :304]) and torch.equal(wide[:, 604:], kept[:, 604:])


@pytest.mark.parametrize("rows,cols", [(5000, 1000), (1, 100000), (20000, 130), (148 * 16 * 2 + 1, 256)])
@pytest.mark.parametrize("dtype", TYPES)
def test_more_items_than_the_device_holds(rows, cols, dtype):
    x = matrix(rows, cols, dtype, 2, pad=1)
    p, t, q = packed(rows, cols, False), packed(cols, rows, False), packed(rows, cols, False)
    G.gq_fp8_pack(x, p, t, fmt="e5m2")
    G.gq_fp8_pack(x, q, fmt="e5m2")
    assert torch.equal(p, q)
    check(p, x, "e5m2", False)
    check(t, x.t(), "e5m2", False)
    out = torch.empty(rows, cols, dtype=dtype, device="cuda")
    G.gq_fp8_unpack(p, out, fmt="e5m2")
    back = torch.empty(cols, rows, dtype=dtype, device="cuda")
    G.gq_fp8_unpack(t, back, fmt="e5m2")
    # either way the values are near x: two mantissa bits, blocks of very different values aside
    for y in (out, back.t()):
        assert ((y.double() - x.double()).abs() <= 2.0 ** -3 * x.double().abs() + 2.0 ** -17 * x.double().abs().max()).all()


# tokens across the shapes' borders, features and columns odd
SHAPES = [(m, n, k) for m in (1, 31, 32, 33, 63, 64, 65, 127, 128, 129, 191, 225, 257, 480) for n, k in ((127, 129), (260, 640))]


@pytest.mark.parametrize("m,n,k", SHAPES + [(2000, 3000, 384), (4100, 515, 4224), (3001, 1000, 2499), (150, 20000, 300),
                                            (64, 9000, 1200), (90, 9000, 1200), (12, 38000, 300), (20, 300, 66000)])
def test_products_of_every_shape(m, n, k):
    a, da = operand(m, k, "e4m3", False, m + n)
    b, db = operand(n, k, "e4m3", True, m + k, spread=0.2)
    y = torch.empty(m, n, device="cuda")
    G.gq_fp8_matmul(a, b, k, y, tile=(False, True))
    check_product(y, da, db, k)
    h = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
    bias = torch.randn(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    G.gq_fp8_matmul(a, b, k, h, bias, tile=(False, True))
    check_product(h, da, db, k, bias)


def test_a_tile_exponent_for_rows_and_row_exponents_for_a_tile_agree():
    """The same codes under exponents kept either way give equal bits."""
    w = matrix(300, 700, torch.float32, 3)
    one = packed(300, 700, True)
    G.gq_fp8_pack(w, one, tile=True)
    buf = one.cpu().numpy()
    cp, ep = O.pitches(700)
    off = O.layout(True, 300, 700)[1]
    exps = np.repeat(buf[off:off + 3 * ep].reshape(3, ep), 128, 0)[:300]
    rows = torch.from_numpy(O.to_buffer(buf[:300 * cp].reshape(300, cp), exps)).cuda()
    for m in (16, 100, 300):
        a, _ = operand(m, 700, "e4m3", False, 4)
        y, z = (torch.empty(m, 300, device="cuda") for _ in range(2))
        G.gq_fp8_matmul(a, one, 700, y, tile=(False, True))
        G.gq_fp8_matmul(a, rows, 700, z, tile=(False, False))
        assert torch.equal(y, z)


@pytest.mark.parametrize("m", [16, 100, 700])
def test_two_streams_at_once(m):
    n, k = 1000, 2100
    a, _ = operand(m, k, "e4m3", False, 6)
    b, _ = operand(n, k, "e4m3", True, 7)
    want = torch.empty(m, n, device="cuda")
    G.gq_fp8_matmul(a, b, k, want, tile=(False, True))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [[torch.zeros(m, n, device="cuda") for _ in range(8)] for _ in streams]
    spaces = [G.gq_fp8_matmul_workspace(k, want) for _ in streams]
    torch.cuda.synchronize()
    for i in range(8):
        for s, o, w in zip(streams, outs, spaces):
            G.gq_fp8_matmul(a, b, k, o[i], tile=(False, True), workspace=w, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for o in outs for y in o)


def test_two_graphs_replayed_at_once():
    k = 2100
    x, w = matrix(300, k, torch.bfloat16, 8), matrix(500, k, torch.float32, 9)
    b = packed(500, k, True)
    G.gq_fp8_pack(w, b, tile=True)
    a = packed(300, k, False)
    want = torch.empty(300, 500, device="cuda")
    G.gq_fp8_pack(x, a)
    G.gq_fp8_matmul(a, b, k, want, tile=(False, True))
    graphs, outs, keep = [], [], []
    for _ in range(2):
        p, y = packed(300, k, False), torch.zeros(300, 500, device="cuda")
        ws = G.gq_fp8_matmul_workspace(k, y)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            G.gq_fp8_pack(x, p)
            G.gq_fp8_matmul(p, b, k, y, tile=(False, True), workspace=ws)
        graphs.append(g), outs.append(y), keep.append((p, ws))
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want) and torch.equal(outs[1], want)


@pytest.mark.parametrize("m", [8, 70, 300])
def test_calls_that_follow_one_another(m):
    """Each call reads what the one before has just written, and overwrites what it has just read, on one stream: as
    if the device were waited for after each."""
    n = 640
    b, _ = operand(n, n, "e4m3", True, 10, spread=0.1)
    runs = []
    for wait in (True, False):
        x = matrix(m, n, torch.bfloat16, 11, spread=0.1).contiguous()
        y, p = torch.empty_like(x), packed(m, n, False)
        for _ in range(20):
            G.gq_fp8_pack(x, p)
            if wait:
                torch.cuda.synchronize()
            G.gq_fp8_matmul(p, b, n, y, tile=(False, True))
            if wait:
                torch.cuda.synchronize()
            G.gq_fp8_pack(y, p)
            if wait:
                torch.cuda.synchronize()
            G.gq_fp8_unpack(p, x)
            x.mul_(0.04)
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        assert torch.isfinite(x).all() and float(x.abs().max()) > 0
        runs.append(x)
    assert torch.equal(runs[0], runs[1])


def test_workspaces_content_and_size():
    m, n, k = 3000, 3000, 4096
    a, _ = operand(m, k, "e4m3", False, 12, spread=0.1)
    b, _ = operand(n, k, "e4m3", False, 13, spread=0.1)
    y, z = (torch.empty(m, n, device="cuda") for _ in range(2))
    need = G._fp8_matmul_bytes(m, n, k)
    G.gq_fp8_matmul(a, b, k, y)
    if need:
        with pytest.raises(G.GQError) as e:
            G.gq_fp8_matmul(a, b, k, z, workspace=torch.empty(need - 16, dtype=torch.uint8, device="cuda"))
        assert e.value.status == G.GQ_ERR_INVALID
    ws = torch.full((need + 64,), 0xFF, dtype=torch.uint8, device="cuda")
    G.gq_fp8_matmul(a, b, k, z, workspace=ws)
    assert torch.equal(y, z) and bool((ws[need:] == 0xFF).all())
