"""AdamW with moments in 8 bits at every beta1: where nearest codes would stand still the first moment is rounded
stochastically, bit for bit as the header says, and follows the exact one over hundreds of steps."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import fp8_oracle as O
import gradient_quantization_communication_b200.gq as G
from test_adamw_gpu import Case, SIZES, f32

SEED = 99      # Case's


def spread(m, rnd):
    """Codes and exponents of float64 rows of 128 with random fractions rnd / 2^16 of a code's step."""
    E = O.exponent(np.abs(m).max(1), "e4m3")
    bad = E == 255
    x = np.ldexp(np.where(bad[:, None], 0.0, np.abs(m)), 127 - E[:, None])
    _, e = np.frexp(x)                                   # x = f * 2^e, f in [1/2, 1)
    step = np.maximum(e - 1, -6) - 3                     # the code's step is 2^step
    units = np.floor((np.floor(np.ldexp(x, 16 - step)) + rnd) / 65536.0)
    value = np.ldexp(units, step)
    code = O.nearest(value, "e4m3")
    assert (O.values("e4m3")[code] == value).all()
    code = code | np.where(np.signbit(m), 128, 0).astype(np.uint8)
    return np.where(bad[:, None], 0x7F, code).astype(np.uint8), E


def want_codes(c, before, i, step, beta1, stochastic):
    """Of tensor i after a step: (codes, exponents) of m and of v."""
    n, (p, g, m, v) = c.sizes[i], before[i]
    _, m32, v32 = O.adam_update(p, g, m, v, f32(2e-3), beta1, 0.999, 1e-8, step, dtype=np.float32)
    nb = -(-n // 128)
    rows = np.zeros((2, nb * 128))
    rows[0, :n], rows[1, :n] = m32, v32
    rnd = [O.noise(0, nb * 128, step, i + k, SEED).reshape(nb, 128) for k in (2 ** 30, 0)]
    if stochastic:
        first = spread(rows[0].reshape(nb, 128), rnd[0])
    else:
        cm, em = O.pack(torch.from_numpy(rows[0]).view(nb, 128), "e4m3", False)
        first = cm, em[:, 0]
    return first, O.squares_encode(rows[1].reshape(nb, 128), rnd[1])


def check_codes(c, before, step, beta1, stochastic):
    for i, n in enumerate(c.sizes):
        if n == 0:
            continue
        for buf, (codes, exps) in zip((c.m[i], c.v[i]), want_codes(c, before, i, step, beta1, stochastic)):
            gc, ge = c.codes(buf, n)
            assert np.array_equal(ge, exps), (i, n)
            assert np.array_equal(gc, codes), (i, n)
            nb = -(-n // 128)
            assert (buf[nb * 128 + nb:] == 0).all()


def hyper(beta1):
    return dict(lr=2e-3, beta1=beta1, beta2=0.999, eps=1e-8)


def check_params(c, before, step, beta1, eps):
    """The update's own arithmetic, from the moments in binary32: up to 16 roundings of it and 4 of the parameter, then
    the parameter's type."""
    for i, n in enumerate(c.sizes):
        if n == 0:
            continue
        p, g, m, v = before[i]
        _, m32, v32 = O.adam_update(p, g, m, v, f32(2e-3), beta1, 0.999, eps, step, dtype=np.float32)
        lr, b1 = f32(f32(2e-3) * c.lr_scale[i]), 1 / (1 - beta1 ** step)
        with np.errstate(all="ignore"):
            upd = lr * b1 * m32.astype(np.float64) / (np.sqrt(v32.astype(np.float64)) / np.sqrt(1 - 0.999 ** step) + f32(eps))
        want = p * (1 - lr * f32(c.decay[i])) - upd
        got = (c.masters if c.masters else c.params)[i].double().cpu().numpy()
        half = 0.0 if c.masters else O.HALF_STEP[c.params[i].dtype]
        tol = 16 * 2.0 ** -24 * np.abs(upd) + 4 * 2.0 ** -24 * np.abs(p) + half * np.abs(want) * 1.01 + 2.0 ** -25 * (half == 2.0 ** -11)
        ok = v32 > 0
        assert (np.abs(got - want) <= tol)[ok].all(), (i, n)
        if c.masters:
            assert torch.equal(c.params[i], c.masters[i].to(c.params[i].dtype))


@pytest.mark.parametrize("eps", [1e-8, 0.0])       # with the approximate root and quotient, and without
@pytest.mark.parametrize("beta1", [0.95, 0.99, 0.9999, 1 - 2.0 ** -30])
@pytest.mark.parametrize("param,grad,master", [(torch.float32, torch.float32, False), (torch.bfloat16, torch.bfloat16, False),
                                               (torch.bfloat16, torch.float32, True), (torch.float16, torch.float16, True)])
def test_codes_above_the_border(param, grad, master, beta1, eps):
    for gap in (0, 3):
        c = Case(SIZES + [40960], param, grad, master, 8, seed=2 + gap, gap=gap)
        for step in (1, 7, 1000):
            before = c.snapshot()
            c.opt.step(**dict(hyper(beta1), eps=eps), step=step)
            check_codes(c, before, step, beta1, True)
            check_params(c, before, step, beta1, eps)


def test_the_border():
    """17/18 is the largest beta1 at which every nearest code still moves without a gradient: 1.125 by a tie."""
    border = float(np.float32(17 / 18))
    if border * 18 > 17:
        border = float(np.nextafter(np.float32(border), np.float32(0)))
    above = float(np.nextafter(np.float32(border), np.float32(1)))
    for beta1, stochastic in ((border, False), (0.5, False), (0.0, False), (above, True)):
        c = Case([5000], torch.float32, torch.float32, False, 8, seed=4)
        before = c.snapshot()
        c.opt.step(**hyper(beta1), step=3)
        check_codes(c, before, 3, beta1, stochastic)
    # and every code from 1.125 down moves at it, in blocks whose largest value is that code's
    c = Case([128 * 8], torch.float32, torch.float32, False, 8, zero=True)
    codes = np.zeros((8, 128), np.uint8)
    codes[:, 0] = 0x38 + np.arange(8)                    # 1 .. 1.875
    c.m[0].copy_(torch.from_numpy(np.concatenate([codes.reshape(-1), np.array([120] * 8 + [0] * 8, np.uint8)])))
    c.flat["grad"].zero_()
    start = c.moments(0)[0].reshape(8, 128)[:, 0]
    c.opt.step(**hyper(border), step=5)
    assert (c.moments(0)[0].reshape(8, 128)[:, 0] < start).all()


@pytest.mark.parametrize("lo,hi", [(-149, -100), (-80, -60), (-30, 0), (-9, 0), (40, 63)])
def test_gradients_of_every_size(lo, hi):
    """Blocks that span more than the codes do, both signs, zeros, values among the smallest codes."""
    rng = np.random.RandomState(5)
    g = np.ldexp(rng.uniform(1, 2, 1280) * rng.choice([-1, 1], 1280), rng.randint(lo, hi, 1280)).astype(np.float32)
    g[::7] = 0.0
    g[256:384] = 0.0
    c = Case([1280], torch.float32, torch.float32, False, 8, zero=True)
    c.flat["grad"][:1280] = torch.from_numpy(g).cuda()
    for step in (1, 2, 3):
        before = c.snapshot()
        c.opt.step(**hyper(0.98), step=step)
        check_codes(c, before, step, 0.98, True)


def test_nan_and_infinity_above_the_border():
    c = Case([1000], torch.float32, torch.float32, False, 8)
    c.grads[0][200], c.grads[0][600] = float("nan"), float("inf")
    c.opt.step(**hyper(0.95), step=4)
    m, _ = c.moments(0)
    bad = np.zeros(1000, bool)
    bad[128:256] = bad[512:640] = True
    assert np.isnan(m[bad]).all() and np.isfinite(m[~bad]).all()


# An element's relative error grows by at most half a code's step, 1/16, a step, in either direction and independently:
# after T steps its standard deviation is below sqrt((1 + 1/256)^T - 1) of the exact value, and the mean's over n
# elements that, times the values' own root mean square over their mean, over sqrt(n).
def sigma(steps, values):
    return np.sqrt((1 + 1 / 256) ** steps - 1) * np.sqrt((values ** 2).mean()) / values.mean() / np.sqrt(values.size)


@pytest.mark.parametrize("beta1", [0.9, 0.94, 0.95, 0.98])
def test_moments_decay_without_a_gradient(beta1):
    n, steps = 1 << 16, 300
    c = Case([n], torch.float32, torch.float32, False, 8, zero=True, seed=12)
    c.flat["grad"][:] = torch.randn(n + 1, generator=torch.Generator(device="cuda").manual_seed(3), device="cuda") * 1e-3
    c.opt.step(**hyper(beta1), step=1)
    m0, v0 = (np.abs(x) for x in c.moments(0))
    c.flat["grad"].zero_()
    for step in range(2, steps + 2):
        c.opt.step(**hyper(beta1), step=step)
        if step in (21, 101):
            m, v = (np.abs(x) for x in c.moments(0))
            if beta1 > 17 / 18:
                t = step - 1
                # and a step's remainder, cut off to 2^-16 of the step
                assert abs(m.mean() / (m0.mean() * beta1 ** t) - 1) <= 5 * sigma(t, m0) + t * 2.0 ** -19
    m, v = (np.abs(x) for x in c.moments(0))
    assert m.mean() < 1e-2 * m0.mean()
    if beta1 < 17 / 18:
        assert m.max() < 1e-2 * m0.max()
    # the second moment keeps at least the smallest code, 2^-31 of its block's largest
    assert abs(v.mean() / (v0.mean() * 0.999 ** steps) - 1) <= 5 * sigma(steps, v0) + steps * 2.0 ** -19


@pytest.mark.parametrize("beta1", [0.95, 0.98])
def test_sparse_gradients(beta1):
    """A gradient in one step of 100: the first moment's sum over all steps is the exact recurrence's."""
    n, steps = 1 << 16, 250
    c = Case([n], torch.float32, torch.float32, False, 8, zero=True, seed=13)
    g = torch.rand(n + 1, generator=torch.Generator(device="cuda").manual_seed(5), device="cuda") * 1e-3
    exact, total, stored = np.zeros(n), 0.0, 0.0
    out = torch.empty(n, device="cuda")
    for step in range(1, steps + 1):
        hit = step % 100 == 1
        c.flat["grad"].copy_(g) if hit else c.flat["grad"].zero_()
        c.opt.step(**hyper(beta1), step=step)
        exact = beta1 * exact + (1 - beta1) * (g[:n].double().cpu().numpy() if hit else 0.0)
        total += exact.sum()
        c.opt.moments(out)
        stored += float(out.double().sum())
    assert abs(stored / total - 1) <= 5 * sigma(steps, g.double().cpu().numpy()) + steps * 2.0 ** -19


@pytest.mark.parametrize("eps", [1e-8, 0.5])
@pytest.mark.parametrize("beta1", [0.0, 1.1 * 2.0 ** -20, 1.1 * 2.0 ** -12, 2.0 ** -9, 0.9])
def test_small_beta1_on_the_smallest_moments(beta1, eps):
    """m beta1 rounds once in binary32 where a block's scale times beta1 would be subnormal: parameters of 0 show m."""
    n, nb = 1280, 10
    c = Case([n], torch.float32, torch.float32, False, 8, zero=True)
    codes = np.random.RandomState(3).randint(0, 127, n).astype(np.uint8)
    exps = np.zeros(16, np.uint8)
    exps[:nb] = 10 + np.arange(nb)
    c.m[0].copy_(torch.from_numpy(np.concatenate([codes, exps])))
    c.flat["grad"].zero_(), c.flat["param"].zero_()
    p, g, m, v = c.snapshot()[0]
    lr = 2.0 ** 120
    c.opt.step(lr, beta1, 0.999, eps, 2)
    _, m32, _ = O.adam_update(p, g, m, v, lr, beta1, 0.999, eps, 2, dtype=np.float32)
    # m / eps, its product with lr / (1 - beta1^2), both factors rounded, and the approximate quotient
    want = -lr / (1 - beta1 ** 2) * m32.astype(np.float64) / eps
    got = c.params[0].double().cpu().numpy()
    assert (np.abs(got - want) <= 8 * 2.0 ** -24 * np.abs(want)).all()


def test_norm_beyond_float32():
    """The factor is taken from the norm in binary64, which passes float32's largest value here and reads as infinity."""
    c = Case([300], torch.float32, torch.float32, False, 32)
    c.flat["grad"].zero_()
    c.grads[0][:2] = 3.0e38
    out = torch.empty(2, device="cuda")
    c.opt.norm(2.0 ** 100, out)
    norm = np.sqrt(2.0) * f32(3.0e38)
    assert np.isinf(float(out[0])) and abs(float(out[1]) - 2.0 ** 100 / norm) <= 2.0 ** -23 * 2.0 ** 100 / norm


def test_captured_step_above_the_border():
    """A captured step draws anew at every replay: its step number is read when it runs."""
    a, b = (Case([5000, 300, 77], torch.bfloat16, torch.float32, True, 8, seed=5) for _ in range(2))
    scalars = torch.zeros(16, dtype=torch.uint8, device="cuda")
    h = dict(beta1=0.95, beta2=0.999, eps=1e-8)
    b.opt.norm(0.5, torch.empty(2, device="cuda"))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.opt.step(lr=1.0, step=1, scalars=scalars, **h)
    for step in (1, 2, 3):
        a.opt.step(lr=1e-3 / step, step=step, **h)
        scalars.copy_(G.gq_adamw_scalars(1e-3 / step, h["beta1"], h["beta2"], step))
        graph.replay()
        for x, y in zip([a.flat[k] for k in a.flat] + a.m + a.v, [b.flat[k] for k in b.flat] + b.m + b.v):
            assert torch.equal(x, y), step


def test_two_streams_above_the_border():
    a, b = (Case([70000, 300, 8200], torch.float32, torch.float32, False, 8, seed=6) for _ in range(2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for step in (1, 2, 3):
        a.opt.step(**hyper(0.98), step=step)
        b.opt.step(**hyper(0.98), step=step, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(a.flat["param"], b.flat["param"])
    assert all(torch.equal(x, y) for x, y in zip(a.m + a.v, b.m + b.v))
