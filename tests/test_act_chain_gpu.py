"""The activation checkpoints' operators run together, as a training step uses them: a block of layer
norm, linear, GELU, linear whose backward pass reads the checkpoints and writes the flat float32 gradient
vector, which gq_fused_step then quantizes.  And sizes whose offsets pass 32 bits."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import act_oracle as A
import gradient_quantization_communication_b200.gq as G
import oracle as O
from gpu_harness import assert_same_f32

U = 2.0 ** -24


class Block:
    """y = GELU(LN(x) W1^T + b1) W2^T + b2 with its parameters' gradients in slices of one flat vector."""

    def __init__(self, d, h, seed, dtype=torch.bfloat16):
        g = torch.Generator().manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g)
        self.d, self.h, self.dtype = d, h, dtype
        self.w1, self.w2 = (r(h, d) / d ** 0.5).to(dtype).cuda(), (r(d, h) / h ** 0.5).to(dtype).cuda()
        self.b1, self.b2 = (0.1 * r(h)).to(dtype).cuda(), (0.1 * r(d)).to(dtype).cuda()
        self.gamma, self.beta = (1 + 0.1 * r(d)).cuda(), (0.1 * r(d)).cuda()
        sizes = [("dgamma", (d,)), ("dbeta", (d,)), ("dw1", (h, d)), ("db1", (h,)), ("dw2", (d, h)), ("db2", (d,))]
        self.flat = torch.zeros(sum(int(np.prod(s)) for _, s in sizes), device="cuda")
        self.grads, at = {}, 0
        for name, s in sizes:
            n = int(np.prod(s))
            self.grads[name] = self.flat[at:at + n].view(s)
            at += n

    def step(self, x, dy, accumulate):
        t, gr = x.shape[0], self.grads
        keep = lambda cols: torch.zeros(G.gq_act_layout(t, cols)[0], dtype=torch.uint8, device="cuda")
        mean, rstd = torch.empty(t, device="cuda"), torch.empty(t, device="cuda")
        kx, kn, kh, ka = keep(self.d), keep(self.d), keep(self.h), keep(self.h)
        n = torch.empty_like(x)
        G.gq_layer_norm_forward(x, self.gamma, self.beta, 1e-5, n, mean, rstd, kx)
        G.gq_act_pack(n, kn)
        hid = torch.addmm(self.b1, n, self.w1.t())
        act = torch.empty_like(hid)
        G.gq_act_fn_forward("gelu", hid, act, kh)
        G.gq_act_pack(act, ka)
        # backward: from here on only the checkpoints, mean and rstd are used
        G.gq_act_weight_grad(ka, dy, gr["dw2"], gr["db2"], accumulate)
        da = dy @ self.w2
        dh = torch.empty_like(da)
        G.gq_act_fn_backward("gelu", kh, da, dh)
        G.gq_act_weight_grad(kn, dh, gr["dw1"], gr["db1"], accumulate)
        dn = dh @ self.w1
        dx = torch.empty_like(dn)
        G.gq_layer_norm_backward(dn, kx, self.gamma, mean, rstd, dx, gr["dgamma"], gr["dbeta"], accumulate)
        self.seen = dict(x=x, n=n, hid=hid, act=act, da=da, dh=dh, dn=dn, mean=mean, rstd=rstd, dy=dy)
        return dx


def _kept(t):
    codes, exps = A.encode(t.cpu())
    return A.decode(codes, exps, t.shape[1])


def _inputs(t, d, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(t, d, generator=g).bfloat16().cuda(), (0.01 * torch.randn(t, d, generator=g)).bfloat16().cuda()


@pytest.mark.parametrize("t,d,h", [(1, 64, 96), (200, 136, 264), (515, 256, 512)])
def test_block_step(t, d, h):
    """Every gradient in 64 bits, from what the step itself kept and passed back."""
    block = Block(d, h, 1)
    x, dy = _inputs(t, d, 2)
    dx = block.step(x, dy, False)
    s = block.seen
    c = lambda v: v.cpu().double()
    dw2, size2 = c(dy).t() @ _kept(s["act"]), c(dy).abs().t() @ _kept(s["act"]).abs()
    dw1, size1 = c(s["dh"]).t() @ _kept(s["n"]), c(s["dh"]).abs().t() @ _kept(s["n"]).abs()
    steps = (t / 16 + 16) * 4 * U
    gr = {k: v.cpu().double() for k, v in block.grads.items()}
    assert ((gr["dw2"] - dw2).abs() <= steps * size2 + 1e-37).all()
    assert ((gr["dw1"] - dw1).abs() <= steps * size1 + 1e-37).all()
    assert ((gr["db2"] - c(dy).sum(0)).abs() <= (t + 16) * U * c(dy).abs().sum(0)).all()
    assert ((gr["db1"] - c(s["dh"]).sum(0)).abs() <= (t + 16) * U * c(s["dh"]).abs().sum(0)).all()
    # GELU's backward: bf16's half step, and binary32's few (test_act_gpu counts them; 1e-5 covers |x| < 8)
    want = c(s["da"]) * A.fn("gelu", _kept(s["hid"]))[1]
    assert ((c(s["dh"]) - want).abs() <= want.abs() * 2.0 ** -8 + c(s["da"]).abs() * 1e-5 + 1e-37).all()
    m, r = c(s["mean"])[:, None], c(s["rstd"])[:, None]
    wdx, wg, wb = A.norm_backward(c(s["dn"]), _kept(s["x"]), c(block.gamma), m, r)
    xh = (_kept(s["x"]) - m) * r
    rows = (t + 64) * U
    assert ((gr["dgamma"] - wg).abs() <= rows * (c(s["dn"]) * xh).abs().sum(0) + 1e-30).all()
    assert ((gr["dbeta"] - wb).abs() <= rows * c(s["dn"]).abs().sum(0) + 1e-30).all()
    g = c(s["dn"]) * c(block.gamma)
    # three sums of d values each, (d / 32 + 24 additions), of terms no larger than |g| (1 + |xh|) (1 + |xh|)
    loose = (d / 32 + 32) * U * r * (g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    assert ((c(dx) - wdx).abs() <= wdx.abs() * 2.0 ** -8 + loose + 1e-37).all()


def test_micro_batches_then_quantized_step():
    """Two workers, two micro-batches each, accumulated in their flat vectors; then the fused quantized
    step on them, which must equal the oracle's on the same vectors bit for bit."""
    blocks = [Block(128, 320, 7), Block(128, 320, 7)]
    for w, block in enumerate(blocks):
        first = None
        for k in range(2):
            x, dy = _inputs(300, 128, 100 * w + k)
            block.step(x, dy, k > 0)
            if k == 0:
                first = block.flat.clone()
        x, dy = _inputs(300, 128, 100 * w + 1)
        alone = Block(128, 320, 7)
        alone.step(x, dy, False)
        # accumulated: each element one more rounding than the two sums
        assert torch.equal(block.flat, first + alone.flat)
    n = blocks[0].flat.numel()
    cfg = G.gq_config("orq", 5, 512, 2, True, 0.0, 3, n)
    res = [torch.zeros(n, device="cuda") for _ in range(2)]
    avg = torch.empty(n, device="cuda")
    with G.Plan(cfg) as plan:
        G.gq_fused_step(plan.handle, 0, [b.flat for b in blocks], res, None, avg)
        assert G.gq_plan_status(plan.handle) == G.GQ_OK
    ores = [np.zeros(n, np.float32) for _ in range(2)]
    want, _ = O.fused_step(O.Config(O.ORQ, 5, 512, 2, 1, 0.0, 3, n), 0, [b.flat.cpu().numpy() for b in blocks], ores)
    assert_same_f32(avg.cpu().numpy(), want, "average")
    for a, b in zip(res, ores):
        assert_same_f32(a.cpu().numpy(), b, "residual")


def test_captured_block_equals_the_eager_one():
    """The whole step in a graph, replayed on new inputs."""
    block, ref = Block(256, 512, 3), Block(256, 512, 3)
    x, dy = _inputs(130, 256, 1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.step(x, dy, False)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dx = block.step(x, dy, False)
    nx, ndy = _inputs(130, 256, 2)
    x.copy_(nx)
    dy.copy_(ndy)
    block.flat.zero_()
    g.replay()
    want = ref.step(nx, ndy, False)
    torch.cuda.synchronize()
    assert torch.equal(dx, want) and torch.equal(block.flat, ref.flat)


def test_two_streams_at_once():
    """Weight gradients and norms of different data on two streams at the same time, each call with a
    workspace of its own, give what they give alone."""
    data = []
    for k in range(2):
        x, dy = _inputs(3000, 1032, 50 + k)
        ck = torch.zeros(G.gq_act_layout(3000, 1032)[0], dtype=torch.uint8, device="cuda")
        G.gq_act_pack(x, ck)
        data.append((x, dy, ck, torch.zeros(3000, device="cuda"), torch.ones(3000, device="cuda")))

    def run(d, stream):
        x, dy, ck, mean, rstd = d
        dw, db = torch.empty(1032, 1032, device="cuda"), torch.empty(1032, device="cuda")
        dx, dg, dbeta = torch.empty_like(x), torch.empty(1032, device="cuda"), torch.empty(1032, device="cuda")
        for _ in range(5):
            G.gq_act_weight_grad(ck, dy, dw, db, stream=stream)
            G.gq_layer_norm_backward(dy, ck, None, mean, rstd, dx, dg, dbeta, stream=stream)
        return dw, db, dx, dg, dbeta

    alone = [run(d, None) for d in data]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    both = [run(d, s) for d, s in zip(data, streams)]
    torch.cuda.synchronize()
    for a, b in zip(alone, both):
        for u, v in zip(a, b):
            assert torch.equal(u, v)


# ------------------------------------------------------------------------------------------------
# offsets past 32 bits
# ------------------------------------------------------------------------------------------------
def test_offsets_past_32_bits():
    """2.2e9 elements: the last rows are packed, unpacked, normalised and passed back as on their own."""
    rows, cols, tail = 67000, 32896, 5
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    end = torch.randn(tail, cols, generator=torch.Generator().manual_seed(1)).bfloat16()
    x[-tail:] = end.cuda()
    ck = torch.zeros(G.gq_act_layout(rows, cols)[0], dtype=torch.uint8, device="cuda")
    G.gq_act_pack(x, ck)
    codes, exps = A.encode(end)
    cp, ep = A.pitches(cols)
    off = A.layout(rows, cols)[1]
    assert np.array_equal(ck[(rows - tail) * cp:rows * cp].cpu().numpy().view(np.int8).reshape(tail, cp), codes)
    assert np.array_equal(ck[off + (rows - tail) * ep:off + rows * ep].cpu().numpy().reshape(tail, ep), exps)
    y = torch.empty_like(x)
    G.gq_act_unpack(ck, y)
    assert torch.equal(y[-tail:].cpu().double(), A.decode(codes, exps, cols))
    G.gq_act_fn_forward("silu", x, y)
    one = torch.empty(tail, cols, dtype=torch.bfloat16, device="cuda")
    G.gq_act_fn_forward("silu", end.cuda(), one)
    assert torch.equal(y[-tail:], one)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    G.gq_layer_norm_forward(x, None, None, 1e-5, y, mean, rstd)
    want, wm, wr = A.norm(end.double(), torch.ones(cols).double(), torch.zeros(cols).double(), 1e-5)
    # the sums: (cols / 32 + 24) roundings of values of size 1, then bf16's half step
    e = (cols / 32 + 40) * U
    assert ((mean[-tail:].cpu().double()[:, None] - wm).abs() <= e).all()
    assert ((rstd[-tail:].cpu().double()[:, None] - wr).abs() <= e * wr).all()
    assert ((y[-tail:].cpu().double() - want).abs() <= want.abs() * 2.0 ** -8 + 6 * e).all()
    # backward: dy is zero but for the last rows, so the gradients are theirs
    mean.zero_()
    rstd.fill_(1.0)
    dg, db = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    G.gq_layer_norm_backward(x, ck, None, mean, rstd, y, dg, db)
    kept = A.decode(codes, exps, cols)
    wdx, wdg, wdb = A.norm_backward(end.double(), kept, torch.ones(cols).double(), torch.zeros(tail, 1).double(),
                                    torch.ones(tail, 1).double())
    assert ((dg.cpu().double() - wdg).abs() <= 400 * U * (end.double() * kept).abs().sum(0) + 1e-30).all()
    assert ((db.cpu().double() - wdb).abs() <= 400 * U * end.double().abs().sum(0) + 1e-30).all()
    del y
    # weight gradient with a wide dy and a narrow checkpoint, and the other way round
    kn = torch.zeros(G.gq_act_layout(rows, 40)[0], dtype=torch.uint8, device="cuda")
    G.gq_act_pack(x[:, :40], kn)
    dw = torch.empty(cols, 40, device="cuda")
    G.gq_act_weight_grad(kn, x, dw)
    narrow = _kept(end[:, :40])
    tol = (512 / 16 * 2 + 3 * rows / 512 + 16) * 2.0 ** -23
    assert ((dw.cpu().double() - end.double().t() @ narrow).abs() <= tol * (end.double().abs().t() @ narrow.abs())).all()
    dw2 = torch.empty(24, cols, device="cuda")
    G.gq_act_weight_grad(ck, x[:, :24], dw2)
    part = end[:, :24].double()
    assert ((dw2.cpu().double() - part.t() @ kept).abs() <= tol * (part.abs().t() @ kept.abs())).all()
