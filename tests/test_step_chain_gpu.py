"""A training step as its parts are used together: a linear layer's three products in 8-bit floating point for two
workers' micro-batches, their gradients through the quantized exchange, the norm, AdamW, and the new weight packed again."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import fp8_oracle as O
import gradient_quantization_communication_b200.gq as G

TOKENS, CIN, COUT = 300, 520, 264


def packed(rows, cols, tile=False):
    return torch.zeros(G.gq_fp8_layout(rows, cols, tile)[0], dtype=torch.uint8, device="cuda")


def decoded(x, fmt="e4m3", tile=False):
    return O.decode(*O.pack(x.cpu(), fmt, tile), fmt, tile, x.shape[1]).cuda()


class Layer:
    """y = x W^T + b: its weight, packed for both products, and its slices of a worker's flat gradient."""

    def __init__(self, weight, bias):
        self.w, self.b = weight, bias
        self.w8, self.wt8 = packed(COUT, CIN, True), packed(CIN, COUT, True)
        self.repack()

    def repack(self):
        G.gq_fp8_pack(self.w, self.w8, self.wt8, tile=True)

    def forward(self, x):
        self.x8, self.xt8 = packed(TOKENS, CIN), packed(CIN, TOKENS)
        G.gq_fp8_pack(x, self.x8, self.xt8)
        y = torch.empty(TOKENS, COUT, dtype=x.dtype, device="cuda")
        G.gq_fp8_matmul(self.x8, self.w8, CIN, y, self.b, tile=(False, True))
        return y

    def backward(self, dy, flat, accumulate):
        d8, dt8 = packed(TOKENS, COUT), packed(COUT, TOKENS)
        G.gq_fp8_pack(dy, d8, dt8, fmt="e5m2")
        dx = torch.empty(TOKENS, CIN, dtype=dy.dtype, device="cuda")
        G.gq_fp8_matmul(d8, self.wt8, COUT, dx, fmt=("e5m2", "e4m3"), tile=(False, True))
        dw = flat[:COUT * CIN].view(COUT, CIN)
        G.gq_fp8_matmul(dt8, self.xt8, TOKENS, dw, fmt=("e5m2", "e4m3"), accumulate=accumulate)
        db = flat[COUT * CIN:]
        s = dy.float().sum(0)
        db.add_(s) if accumulate else db.copy_(s)
        return dx


def inputs(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(TOKENS, CIN, generator=g, device="cuda").bfloat16()
    dy = (1e-2 * torch.randn(TOKENS, COUT, generator=g, device="cuda")).bfloat16()
    return x, dy


def make_layer():
    g = torch.Generator(device="cuda").manual_seed(0)
    w = torch.randn(COUT, CIN, generator=g, device="cuda") / CIN ** 0.5
    return Layer(w, 0.1 * torch.randn(COUT, generator=g, device="cuda"))


def cut(k):
    """Half-steps of binary32 of a sum over k products, as the tensor cores make it (see the header)."""
    return 2 * (2 * k / 32 + 20) * 2.0 ** -24


def test_the_layers_products():
    layer, (x, dy) = make_layer(), inputs(1)
    n = COUT * CIN + COUT
    flat = torch.full((n,), 3.0, device="cuda")
    y = layer.forward(x)
    dx = layer.backward(dy, flat, False)
    xh, wh, dh = decoded(x), decoded(layer.w, tile=True), decoded(dy, "e5m2")
    want = xh @ wh.t() + layer.b.double()
    size = xh.abs() @ wh.abs().t() + layer.b.double().abs()
    assert ((y.double() - want).abs() <= cut(CIN) * size + O.HALF_STEP[y.dtype] * 1.01 * want.abs()).all()
    want = dh @ wh
    assert ((dx.double() - want).abs() <= cut(COUT) * (dh.abs() @ wh.abs()) + O.HALF_STEP[y.dtype] * 1.01 * want.abs()).all()
    dt, xt = decoded(dy.t(), "e5m2"), decoded(x.t())
    dw = flat[:COUT * CIN].view(COUT, CIN).double()
    assert ((dw - dt @ xt.t()).abs() <= cut(TOKENS) * (dt.abs() @ xt.abs().t())).all()
    # a second micro-batch is added
    before = flat.clone()
    x2, dy2 = inputs(2)
    layer.forward(x2)
    layer.backward(dy2, flat, True)
    dt, xt = decoded(dy2.t(), "e5m2"), decoded(x2.t())
    want = before[:COUT * CIN].view(COUT, CIN).double() + dt @ xt.t()
    size = before[:COUT * CIN].view(COUT, CIN).double().abs() + dt.abs() @ xt.abs().t()
    assert ((flat[:COUT * CIN].view(COUT, CIN).double() - want).abs() <= cut(TOKENS) * size).all()


def test_gradients_against_differences():
    """L = sum(y * dy) is linear in W and x: its difference quotients in 64 bits, without 8-bit values, against the
    products.  An operand's value is off by half a step (e4m3: 2^-4, e5m2: 2^-3) or half the smallest code of its block
    (a block's largest value times 2^-10 / 448 * 2 or 2^-17 / 57344 * 2 at most, far below)."""
    layer, (x, dy) = make_layer(), inputs(3)
    flat = torch.empty(COUT * CIN + COUT, device="cuda")
    layer.forward(x)
    dx = layer.backward(dy, flat, False)
    dw = flat[:COUT * CIN].view(COUT, CIN).double()
    xd, dd, wd = x.double(), dy.double(), layer.w.double()
    loss = lambda w, v: float(((v @ w.t()) * dd).sum())  # noqa: E731
    rng = np.random.RandomState(4)
    small = 2.0 ** -16
    for _ in range(12):
        i, j, t = rng.randint(COUT), rng.randint(CIN), rng.randint(TOKENS)
        h = 1.0
        e = torch.zeros_like(wd)
        e[i, j] = h
        quotient = (loss(wd + e, xd) - loss(wd - e, xd)) / (2 * h)
        size = float((dd[:, i].abs() * xd[:, j].abs()).sum() + small * (dd[:, i].abs().max() * xd.abs().max()) * TOKENS)
        off = (1 + 2.0 ** -4) * (1 + 2.0 ** -3) - 1
        assert abs(float(dw[i, j]) - quotient) <= off * size
        e = torch.zeros_like(xd)
        e[t, j] = h
        quotient = (loss(wd, xd + e) - loss(wd, xd - e)) / (2 * h)
        size = float((dd[t].abs() * wd[:, j].abs()).sum() + small * dd.abs().max() * wd.abs().max() * COUT)
        assert abs(float(dx[t, j]) - quotient) <= (off + 2.0 ** -8) * size


@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_of_two_workers(bits):
    """Forward, backward, exchange, clipping and AdamW on one stream, twice, against the same step put together from the
    average that the exchange gives."""
    layer = make_layer()
    n = COUT * CIN + COUT
    flats = [torch.zeros(n, device="cuda") for _ in range(2)]
    residuals = [torch.zeros(n, device="cuda") for _ in range(2)]
    avg = torch.zeros(n, device="cuda")
    plan = G.Plan(G.gq_config("orq", 5, 512, 2, True, 0.0, 7, n))
    sizes = (COUT * CIN, COUT)
    grads = avg.split(sizes)
    if bits == 32:
        ms, vs = ([torch.zeros(s, device="cuda") for s in sizes] for _ in range(2))
    else:
        ms, vs = ([torch.zeros(G.gq_adamw_layout(s)[0], dtype=torch.uint8, device="cuda") for s in sizes] for _ in range(2))
    opt = G.AdamW([layer.w.view(-1), layer.b], grads, ms, vs, weight_decay=[0.1, 0.0], state_bits=bits, seed=3)
    norm = torch.empty(2, device="cuda")
    lr = float(np.float32(1e-3))
    try:
        for step in (1, 2):
            w0, b0 = layer.w.double().cpu().numpy().ravel(), layer.b.double().cpu().numpy()
            if step == 2 and bits == 32:
                state = [(m.double().cpu().numpy(), v.double().cpu().numpy()) for m, v in zip(ms, vs)]
            else:
                state = [(np.zeros(s), np.zeros(s)) for s in sizes]
            if step == 2 and bits == 8:
                m8, v8 = (torch.empty(n, device="cuda") for _ in range(2))
                opt.moments(m8, v8)
                state = list(zip((t.double().cpu().numpy() for t in m8.split(sizes)),
                                 (t.double().cpu().numpy() for t in v8.split(sizes))))
            for worker in range(2):
                x, dy = inputs(10 * step + worker)
                layer.forward(x)
                layer.backward(dy, flats[worker], False)
            G.gq_fused_step(plan.handle, step, flats, residuals, None, avg)
            opt.norm(1.0, norm)
            opt.step(1e-3, 0.9, 0.999, 1e-8, step, scale=norm[1:])
            layer.repack()
            assert G.gq_plan_status(plan.handle) == G.GQ_OK
            g = avg.double()
            want = float(torch.sqrt((g * g).sum()))
            assert want > 0 and abs(float(norm[0]) - want) <= 2.0 ** -23 * want
            for p0, p, gi, (m, v), decay in zip((w0, b0), (layer.w.view(-1), layer.b), grads, state, (0.1, 0.0)):
                wp, wm, wv = O.adam_update(p0, gi.double().cpu().numpy(), m, v, lr, 0.9, 0.999, 1e-8, step,
                                           decay=float(np.float32(decay)), scale=float(norm[1]))
                got = p.double().cpu().numpy()
                below = np.sqrt(wv) / np.sqrt(1 - 0.999 ** step) + 1e-8
                factor = lr / (1 - 0.9 ** step)
                size = 0.9 * np.abs(m) + 0.1 * np.abs(gi.double().cpu().numpy()) * float(norm[1])
                u = 2.0 ** -24
                tol = 4 * u * np.abs(p0) + factor / below * (6 * u * size + 16 * u * np.abs(wm))
                assert (np.abs(got - wp) <= tol).all()
            # the packed weight is the new one's
            assert torch.equal(layer.w8, torch.from_numpy(O.to_buffer(*O.pack(layer.w.cpu(), "e4m3", True))).cuda())
            assert torch.equal(layer.wt8, torch.from_numpy(O.to_buffer(*O.pack(layer.w.t().cpu(), "e4m3", True))).cuda())
    finally:
        plan.close()
        opt.close()
