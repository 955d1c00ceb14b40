"""AdamW over many tensors on the GPU: 32-bit moments against the step in 64 bits, 8-bit moments bit for bit against
the formula in binary32 and the formats in 64 bits, the norm, captured steps, tensors that start anywhere."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import fp8_oracle as O
import gradient_quantization_communication_b200.gq as G

TYPES = [torch.float32, torch.bfloat16, torch.float16]
SIZES = [1, 7, 8, 127, 0, 128, 129, 255, 256, 257, 1000, 4095, 4096, 4097, 10000, 1]
HYPER = dict(lr=2e-3, beta1=0.9, beta2=0.999, eps=1e-8)


class Case:
    """Tensors one after another in flat buffers, `gap` elements between them."""

    def __init__(self, sizes, param, grad, master, bits, seed=1, gap=0, zero=False, skew=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.sizes, self.bits = sizes, bits
        at, self.at = 0, []
        for n in sizes:
            self.at.append(at)
            at += n + gap
        total = at + 1
        r = lambda: torch.randn(total, generator=g, device="cuda")  # noqa: E731
        scale = torch.exp(2 * r())
        self.flat = {"param": (0.1 * r()).to(param), "grad": (1e-3 * r() * scale).to(grad)}
        if master:
            self.flat["master"] = 0.1 * r()
            self.flat["param"] = self.flat["master"].to(param)
        if skew:  # the gradients begin elsewhere within 16 bytes
            self.flat["grad"] = torch.cat([self.flat["grad"][:skew], self.flat["grad"]])[skew:]
        self.params, self.grads = self.views("param"), self.views("grad")
        self.masters = self.views("master") if master else None
        if bits == 32:
            self.flat["m"], self.flat["v"] = 1e-3 * r() * scale, (1e-3 * r() * scale) ** 2
            if zero:
                self.flat["m"].zero_(), self.flat["v"].zero_()
            self.m, self.v = self.views("m"), self.views("v")
        else:
            self.m, self.v = ([torch.zeros(G.gq_adamw_layout(n)[0], dtype=torch.uint8, device="cuda") for n in sizes]
                              for _ in range(2))
            if not zero:
                rng = np.random.RandomState(seed)
                for n, m, v in zip(sizes, self.m, self.v):
                    nb = -(-n // 128)
                    for buf, e0 in ((m, 90), (v, 80)):
                        codes = rng.randint(0, 127, nb * 128).astype(np.uint8)
                        codes[n:] = 0
                        exps = np.zeros(-(-nb // 16) * 16, np.uint8)
                        exps[:nb] = e0 + rng.randint(0, 20, nb)
                        buf.copy_(torch.from_numpy(np.concatenate([codes, exps])))
        self.decay = [0.1 * (i % 3) for i in range(len(sizes))]
        self.lr_scale = [1.0 + 0.5 * (i % 2) for i in range(len(sizes))]
        self.opt = G.AdamW(self.params, self.grads, self.m, self.v, self.masters, self.decay, self.lr_scale, bits, seed=99)

    def views(self, what):
        return [self.flat[what][a:a + n] for a, n in zip(self.at, self.sizes)]

    def moments(self, i):
        """float64 m and v of a tensor."""
        n = self.sizes[i]
        if self.bits == 32:
            return self.m[i].double().cpu().numpy(), self.v[i].double().cpu().numpy()
        (cm, em), (cv, ev) = (self.codes(b, n) for b in (self.m[i], self.v[i]))
        m = np.where((em == 255)[:, None], np.nan, O.values("e4m3")[cm] * np.exp2(em.astype(float) - 127)[:, None])
        return m.reshape(-1)[:n], O.squares_decode(cv, ev).reshape(-1)[:n]

    def codes(self, buf, n):
        nb = -(-n // 128)
        b = buf.cpu().numpy()
        return b[:nb * 128].reshape(nb, 128), b[nb * 128:nb * 128 + nb]

    def snapshot(self):
        """What the next step starts from, per tensor."""
        out = []
        for i, n in enumerate(self.sizes):
            p = (self.masters if self.masters else self.params)[i]
            out.append((p.double().cpu().numpy(), self.grads[i].double().cpu().numpy(), *self.moments(i)))
        return out


def f32(x):
    return float(np.float32(x))


def check_step(c, before, step, scale=1.0):
    for i, n in enumerate(c.sizes):
        if n == 0:
            continue
        p, g, m, v = before[i]
        kw = dict(step=step, decay=f32(c.decay[i]), scale=scale)
        lr = f32(f32(HYPER["lr"]) * c.lr_scale[i])
        h = dict(HYPER, lr=lr)
        wp, wm, wv = O.adam_update(p, g, m, v, **h, **kw)
        gs = np.abs(g * scale)
        u = 2.0 ** -24
        # m: the factors' roundings, two products (three with the scale's) and a sum
        tm = 5 * u * (0.9 * np.abs(m) + 0.1 * gs) + 1e-45
        tv = 7 * u * (0.999 * np.abs(v) + 0.001 * gs * gs) + 1e-45
        below = np.sqrt(np.maximum(wv, 0)) / np.sqrt(1 - 0.999 ** step) + 1e-8
        factor = lr / (1 - 0.9 ** step)
        upd = np.abs(wm) * factor / below
        # the quotient: m's own error, half of v's, six roundings; then the parameter's three and the last difference
        tp = factor * tm / below + upd * (0.5 * tv / np.maximum(wv, 1e-300) + 8 * u) + 4 * u * (np.abs(p) + upd)
        got = (c.masters if c.masters else c.params)[i].double().cpu().numpy()
        half = 0 if c.masters else O.HALF_STEP[c.params[i].dtype]
        tiny = 2.0 ** -25 if c.params[i].dtype == torch.float16 else 0.0
        assert (np.abs(got - wp) <= tp + half * np.abs(wp) * 1.01 + (0 if c.masters else tiny)).all(), (i, n)
        if c.masters:
            assert torch.equal(c.params[i], c.masters[i].to(c.params[i].dtype))
        if c.bits == 32:
            gm, gv = c.moments(i)
            assert (np.abs(gm - wm) <= tm).all() and (np.abs(gv - wv) <= tv).all(), (i, n)
            continue
        # 8 bits: from the moments in binary32, each operation rounded alone
        _, m32, v32 = O.adam_update(p, g, m, v, **h, **kw, dtype=np.float32)
        assert (np.abs(m32 - wm) <= tm).all() and (np.abs(v32 - wv) <= tv).all()
        nb = -(-n // 128)
        rows = np.zeros((2, nb * 128))
        rows[0, :n], rows[1, :n] = m32, v32
        rnd = np.zeros(nb * 128, np.int64)
        rnd[:] = O.noise(0, nb * 128, step, i, 99)
        cm, em = O.pack(torch.from_numpy(rows[0]).view(nb, 128), "e4m3", False)
        cv, ev = O.squares_encode(rows[1].reshape(nb, 128), rnd.reshape(nb, 128))
        for buf, codes, exps in ((c.m[i], cm, em[:, 0]), (c.v[i], cv, ev)):
            gc, ge = c.codes(buf, n)
            assert np.array_equal(ge, exps), (i, n)
            assert np.array_equal(gc, codes), (i, n)
            assert (buf[nb * 128 + nb:] == 0).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("grad", TYPES)
@pytest.mark.parametrize("param,master", [(torch.float32, False), (torch.bfloat16, False), (torch.bfloat16, True),
                                          (torch.float16, False), (torch.float16, True)])
def test_step(param, grad, master, bits):
    for gap in (0, 3):      # slices that start anywhere
        c = Case(SIZES, param, grad, master, bits, seed=2 + gap, gap=gap)
        kept = {k: t.clone() for k, t in c.flat.items()}
        for step in (1, 7, 1000):
            before = c.snapshot()
            c.opt.step(**HYPER, step=step)
            check_step(c, before, step)
        # nothing between the tensors, and no gradient, is touched
        inside = torch.zeros(c.flat["param"].numel(), dtype=torch.bool, device="cuda")
        for a, n in zip(c.at, c.sizes):
            inside[a:a + n] = True
        for k, t in c.flat.items():
            assert torch.equal(t[~inside], kept[k][~inside])
        assert torch.equal(c.flat["grad"], kept["grad"])


def test_aligned_tensors():
    for bits in (32, 8):
        c = Case([4096, 8192 + 512, 64, 40960], torch.float32, torch.float32, False, bits)
        before = c.snapshot()
        c.opt.step(**HYPER, step=3)
        check_step(c, before, 3)


@pytest.mark.parametrize("bits", [32, 8])
def test_from_zero(bits):
    c = Case([300, 5000], torch.float32, torch.float32, False, bits, zero=True)
    before = c.snapshot()
    c.opt.step(**HYPER, step=1)
    check_step(c, before, 1)
    c.flat["grad"].zero_()
    for step in (2, 3):
        before = c.snapshot()
        c.opt.step(**HYPER, step=step)
        check_step(c, before, step)


def test_scale_and_norm():
    c = Case([5000, 7, 0, 130], torch.bfloat16, torch.float32, True, 32, gap=1)
    out = torch.full((4,), 5.0, device="cuda")
    for limit in (0.01, 1e9, float("inf")):
        G.gq_adamw_norm(c.opt.handle, limit, out[1:3])
        g = torch.cat([x.double() for x in c.grads])
        norm = float(torch.sqrt((g * g).sum()))
        assert abs(float(out[1]) - norm) <= 2.0 ** -23 * norm
        want = min(1.0, limit / norm)
        assert abs(float(out[2]) - want) <= 2.0 ** -23 * want
        assert float(out[0]) == 5.0 and float(out[3]) == 5.0
    G.gq_adamw_norm(c.opt.handle, 0.01, out[1:3])
    before = c.snapshot()
    c.opt.step(**HYPER, step=5, scale=out[2:3])
    check_step(c, before, 5, scale=float(out[2]))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("value", [float("nan"), float("inf"), "max", "tiny"])
def test_norm_of_any_gradient(dtype, value):
    c = Case([3000, 300], torch.float32, dtype, False, 32)
    v = {"max": torch.finfo(dtype).max, "tiny": torch.finfo(dtype).smallest_normal}.get(value, value)
    if value == "tiny":
        c.flat["grad"].zero_()
    c.grads[1][299] = v
    out = torch.empty(2, device="cuda")
    c.opt.norm(1.0, out)
    g = torch.cat([x.double() for x in c.grads])
    want = torch.sqrt((g * g).sum())
    if value in ("max", "tiny"):
        assert abs(float(out[0]) - float(want)) <= 2.0 ** -23 * float(want)
        assert abs(float(out[1]) - min(1.0, 1.0 / float(want))) <= 2.0 ** -23
        return
    assert not np.isfinite(float(out[0])) and np.isnan(float(out[1]))
    # a scale of NaN: the step leaves everything as it was
    kept = {k: t.clone() for k, t in c.flat.items()}
    c.opt.step(**HYPER, step=2, scale=out[1:])
    for k, t in c.flat.items():
        assert torch.equal(torch.nan_to_num(t, 7.0), torch.nan_to_num(kept[k], 7.0))


def test_norm_of_zero_and_of_nothing():
    c = Case([300], torch.float32, torch.float32, False, 32)
    c.flat["grad"].zero_()
    out = torch.empty(2, device="cuda")
    c.opt.norm(1.0, out)
    assert out.tolist() == [0.0, 1.0]
    empty = Case([0, 0], torch.float32, torch.float32, False, 8)
    empty.opt.norm(1.0, out.fill_(7.0))
    assert out.tolist() == [0.0, 1.0]
    empty.opt.step(**HYPER, step=1)


@pytest.mark.parametrize("bits", [32, 8])
def test_infinite_and_nan_gradients_stay_in_their_block(bits):
    c = Case([1000, 128], torch.float32, torch.float32, False, bits)
    c.grads[0][200], c.grads[0][600], c.grads[1][5] = float("nan"), float("inf"), 1e25   # its square overflows
    before = c.snapshot()
    c.opt.step(**HYPER, step=4)
    m, v = c.moments(0)
    width = 128 if bits == 8 else 1
    bad = np.zeros(1000, bool)
    for i in (200, 600):
        bad[i // width * width:(i // width + 1) * width] = True
    assert not np.isfinite(v[bad]).any() and np.isfinite(v[~bad]).all() and np.isfinite(m[~bad]).all()
    p = c.params[0].cpu().numpy()
    assert np.isnan(p[200]) and np.isnan(p[600]) and np.isfinite(np.delete(p, [200, 600])).all()
    assert not np.isfinite(c.moments(1)[1][5])
    wp, wm, wv = O.adam_update(*before[0], **dict(HYPER, lr=f32(HYPER["lr"])), step=4, decay=0.0)
    ok = np.isfinite(wp)
    assert np.abs(p[ok] - wp[ok]).max() < 1e-6


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype", TYPES)
def test_moments(bits, dtype):
    for gap in (0, 3):
        c = Case(SIZES, torch.float32, torch.float32, False, bits, gap=gap)
        c.opt.step(**HYPER, step=9)
        total = sum(SIZES)
        m, v = (torch.full((total + 8,), 5.0, dtype=dtype, device="cuda") for _ in range(2))
        c.opt.moments(m[:total], v[:total])
        for out, which in ((m, 0), (v, 1)):
            want = torch.from_numpy(np.concatenate([c.moments(i)[which] for i in range(len(SIZES))]))
            want = want.clamp(-65504, 65504).to(dtype) if dtype == torch.float16 else want.to(dtype)
            assert torch.equal(out[:total].cpu(), want)
            assert (out[total:] == 5.0).all()
        only = torch.empty(total, dtype=dtype, device="cuda")
        c.opt.moments(v=only)
        assert torch.equal(only, v[:total])


def test_second_moment_is_unbiased():
    """Equal gradients in every element: the stored values' mean is the second moment itself."""
    n = 1 << 20
    c = Case([n], torch.float32, torch.float32, False, 8, zero=True)
    for step, g in ((1, 0.37), (2, 0.0), (3, 0.0)):
        c.flat["grad"].fill_(g)
        before = c.moments(0)[1]
        c.opt.step(**HYPER, step=step)
        want = 0.999 * before + 0.001 * g * g
        got = c.moments(0)[1]
        # an element's deviation is at most half a code's step, an eighth of its power of two
        sigma = 0.5 * 0.125 * want.max() / np.sqrt(n)
        assert abs((got - want).mean()) < 5 * sigma
        assert np.abs(got - want).max() <= 0.125 * want.max()
    assert (got < before).any() and (got >= before).any()


def test_captured_step_with_scalars():
    """One captured step, replayed with the scalars of three steps, against three calls."""
    for bits in (32, 8):
        a, b = (Case([5000, 300, 77], torch.bfloat16, torch.float32, True, bits, seed=5) for _ in range(2))
        out = torch.empty(2, device="cuda")
        scalars = torch.zeros(16, dtype=torch.uint8, device="cuda")
        scalars.copy_(G.gq_adamw_scalars(0.0, 0.9, 0.999, 1))
        b.opt.norm(0.5, out)                           # the kernels are loaded before the capture
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b.opt.norm(0.5, out)
            b.opt.step(1.0, 0.9, 0.999, 1e-8, 1, scale=out[1:], scalars=scalars)
        mine = torch.empty(2, device="cuda")
        for step in (1, 2, 3):
            lr = 1e-3 / step
            a.opt.norm(0.5, mine)
            a.opt.step(lr, 0.9, 0.999, 1e-8, step, scale=mine[1:])
            scalars.copy_(G.gq_adamw_scalars(lr, 0.9, 0.999, step))
            graph.replay()
            for k in a.flat:
                assert torch.equal(a.flat[k], b.flat[k]), (bits, step, k)
            for x, y in zip(a.m + a.v, b.m + b.v):
                assert torch.equal(x, y)


def test_another_stream():
    a, b = (Case([70000, 300], torch.float32, torch.float32, False, 8, seed=6) for _ in range(2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a.opt.step(**HYPER, step=1)
    b.opt.step(**HYPER, step=1, stream=s)
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(a.flat["param"], b.flat["param"]) and torch.equal(a.v[0], b.v[0])


def test_refusals_that_need_an_optimizer():
    c = Case([1000, 300], torch.float32, torch.float32, False, 8)
    L, h = G.lib(), c.opt.handle
    out = torch.zeros(4, device="cuda")
    p = out.data_ptr()
    for args in ((0.0, p), (-1.0, p), (float("nan"), p), (1.0, None), (1.0, p + 2), (1.0, c.grads[0].data_ptr()),
                 (1.0, c.v[1].data_ptr())):
        assert L.gq_adamw_norm(h, *args, None) == G.GQ_ERR_INVALID
    good = [1e-3, 0.9, 0.999, 1e-8, 1, p, None]
    for at, bad in ((0, -1.0), (1, 1.0), (2, 1.5), (3, -1e-8), (3, float("nan")), (4, 0), (5, p + 1), (6, p + 4),
                    (5, c.params[0].data_ptr()), (6, c.m[0].data_ptr())):
        args = list(good)
        args[at] = bad
        assert L.gq_adamw_step(h, *args, None) == G.GQ_ERR_INVALID
    buf = torch.zeros(2600, device="cuda")
    q = buf.data_ptr()
    for args in ((5, q, None), (0, None, None), (0, q + 4, None), (0, q, q + 16), (0, c.m[0].data_ptr(), None),
                 (0, q, c.params[0].data_ptr())):
        assert L.gq_adamw_moments(h, *args, None) == G.GQ_ERR_INVALID
    with pytest.raises(ValueError):
        c.opt.norm(1.0, torch.zeros(2))
    with pytest.raises(ValueError):
        c.opt.step(**HYPER, step=1, scale=torch.zeros(2, device="cuda"))
    with pytest.raises(ValueError):
        c.opt.moments(torch.zeros(7, device="cuda"))
    with pytest.raises(ValueError):
        c.opt.moments()
    with pytest.raises(ValueError):
        G.AdamW(c.params, c.grads[:1], c.m, c.v, state_bits=8)
    with pytest.raises(ValueError):
        G.AdamW(c.params, c.grads, c.m, c.v)            # moments of 8 bits for an optimizer of 32
    with pytest.raises(ValueError):
        G.AdamW([x[::2] for x in c.params], c.grads, c.m, c.v, state_bits=8)
    with pytest.raises(G.GQError):
        G.AdamW([c.params[0], c.params[0]], [c.grads[0], c.grads[0]], [c.m[0], c.m[0]], [c.v[0], c.v[0]], state_bits=8)


@pytest.mark.parametrize("param,grad,master", [(torch.float32, torch.float32, False), (torch.bfloat16, torch.bfloat16, True),
                                               (torch.bfloat16, torch.float32, False), (torch.float32, torch.float16, False)])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("skew", [0, 1])
def test_tensors_that_start_anywhere(param, grad, master, bits, skew):
    """Every start within 32 bytes and every short length, pieces that end in a tensor's last elements, NaN between the
    tensors: it reaches neither the norm nor the step, and what lies between stays as it is."""
    sizes = [n for n in range(1, 20)] + [250, 251, 4093, 4096, 4099, 8189, 8192 + 5, 12000]
    c = Case(sizes, param, grad, master, bits, seed=3 + skew, gap=3, skew=skew)
    between = torch.ones(c.flat["param"].numel(), dtype=torch.bool, device="cuda")
    for at, n in zip(c.at, sizes):
        between[at:at + n] = False
    for t in c.flat.values():
        t[between] = float("nan")
    out = torch.empty(2, device="cuda")
    c.opt.norm(0.25, out)
    norm = float(torch.cat([g.double() for g in c.grads]).square().sum().sqrt())
    assert abs(float(out[0]) - norm) <= 2.0 ** -23 * norm
    before, held = c.snapshot(), {k: t.clone() for k, t in c.flat.items()}
    c.opt.step(**HYPER, step=5)
    check_step(c, before, 5)
    for k, t in c.flat.items():
        assert torch.isnan(t[between]).all(), k
    assert torch.equal(c.flat["grad"][~between], held["grad"][~between])
    m, v = (torch.empty(sum(sizes), device="cuda") for _ in range(2))
    c.opt.moments(m, v)
    got = [c.moments(i) for i in range(len(sizes))]
    for flat, k in ((m, 0), (v, 1)):
        assert np.array_equal(flat.double().cpu().numpy(), np.concatenate([x[k] for x in got]))


def test_elements_past_32_bits():
    """A tensor of more than 2^31 elements: its last ones, whose byte offsets pass 2^32, and their random bits."""
    n = (1 << 31) + 300
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    size, off = G.gq_adamw_layout(n)
    m, v = (torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(2))
    first = n - 300 - 128
    tail = torch.randn(428, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).to(torch.bfloat16)
    g[first:] = tail
    with G.AdamW([p], [g], [m], [v], state_bits=8, seed=5) as opt:
        opt.step(**HYPER, step=1)
        out = torch.empty(2, device="cuda")
        opt.norm(1.0, out)
    want = float(torch.sqrt((tail.double() ** 2).sum()))
    assert abs(float(out[0]) - want) <= 2.0 ** -23 * want
    h = dict(HYPER, lr=f32(HYPER["lr"]))
    z = np.zeros(428)
    _, m32, v32 = O.adam_update(z, tail.double().cpu().numpy(), z, z, **h, step=1, dtype=np.float32)
    rows = np.zeros((2, 512))
    rows[0, :428], rows[1, :428] = m32, v32
    cm, em = O.pack(torch.from_numpy(rows[0]).view(4, 128), "e4m3", False)
    cv, ev = O.squares_encode(rows[1].reshape(4, 128), O.noise(first, 512, 1, 0, 5).reshape(4, 128))
    for buf, codes, exps in ((m, cm, em[:, 0]), (v, cv, ev)):
        assert np.array_equal(buf[first:first + 512].cpu().numpy(), codes.reshape(-1))
        assert np.array_equal(buf[off + first // 128:off + first // 128 + 4].cpu().numpy(), exps)
        assert int(buf[:first].max()) == 0
    assert int((p[:first] != 0).sum()) == 0 and int((p[first:] != 0).sum()) > 420


def _run_gradients(values, bits, steps=2):
    """A step or two on gradients of any size, from zero moments."""
    n = values.numel()
    c = Case([n], torch.float32, torch.float32, False, bits, zero=True)
    c.flat["grad"][:n] = values.cuda()
    for step in range(1, steps + 1):
        before = c.snapshot()
        c.opt.step(**HYPER, step=step)
        yield c, before, step


@pytest.mark.parametrize("lo,hi", [(-149, -100), (-80, -60), (-70, -63), (20, 40), (60, 68), (-149, 63)])
def test_second_moments_of_every_size(lo, hi):
    """8 bits: gradients whose squares are subnormal, vanish, come near binary32's largest value or pass it, and blocks
    that span more than the codes do."""
    rng = np.random.RandomState(5)
    g = np.ldexp(rng.uniform(1, 2, 1280) * rng.choice([-1, 1], 1280), rng.randint(lo, hi, 1280)).astype(np.float32)
    g[::7] = 0.0
    g[256:384] = 0.0                                     # a block of nothing
    g[400] = np.float32(2.0) ** (hi - 1)
    for c, (before,), step in _run_gradients(torch.from_numpy(g), 8):
        p, g64, m, v = before
        h = dict(HYPER, lr=f32(HYPER["lr"]))
        _, m32, v32 = O.adam_update(p, g64, m, v, **h, step=step, dtype=np.float32)
        cm, em = O.pack(torch.from_numpy(m32.astype(np.float64)).view(10, 128), "e4m3", False)
        cv, ev = O.squares_encode(v32.astype(np.float64).reshape(10, 128), O.noise(0, 1280, step, 0, 99).reshape(10, 128))
        for buf, codes, exps in ((c.m[0], cm, em[:, 0]), (c.v[0], cv, ev)):
            gc, ge = c.codes(buf, 1280)
            assert np.array_equal(ge, exps) and np.array_equal(gc, codes)
        gm, gv = c.moments(0)
        # a second moment that is not 0 is kept above 0
        assert (gv[np.isfinite(gv) & (v32 > 0)] > 0).all() and (gv[v32 == 0] == 0)[np.isfinite(gv[v32 == 0])].all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [2.0 ** 64, 2.0 ** 65, 2.0 ** 125, 2.0 ** 126, 3e38])
def test_eps_beyond_every_root(bits, eps):
    """The update of parameters of 0 keeps its digits where the divisor's reciprocal is subnormal."""
    g = np.random.RandomState(8).uniform(2.0 ** 59, 2.0 ** 60, 1280).astype(np.float32)
    c = Case([1280], torch.float32, torch.float32, False, bits, zero=True)
    c.flat["grad"][:1280] = torch.from_numpy(g).cuda()
    c.params[0].zero_()
    p, g64, m, v = c.snapshot()[0]
    lr, e = 2.0 ** 60, f32(eps)
    c.opt.step(lr, 0.9, 0.999, eps, 1)
    _, m32, v32 = O.adam_update(p, g64, m, v, lr, 0.9, 0.999, e, 1, dtype=np.float32)
    below = np.sqrt(v32.astype(np.float64)) / np.sqrt(1 - 0.999) + e
    want = -lr / (1 - 0.9) * m32.astype(np.float64) / below
    got = c.params[0].double().cpu().numpy()
    assert (np.abs(got - want) <= 16 * 2.0 ** -24 * np.abs(want)).all()


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [0.0, 1e-30, 1e-12, 1.0])
def test_eps_of_every_size(bits, eps):
    """Small second moments, subnormal ones among them, beside no eps and a large one."""
    g = np.ldexp(np.random.RandomState(6).uniform(1, 2, 1280), np.random.RandomState(7).randint(-66, 0, 1280)).astype(np.float32)
    c = Case([1280], torch.float32, torch.float32, bits == 0, bits, zero=True)
    c.flat["grad"][:1280] = torch.from_numpy(g).cuda()
    p, g64, m, v = c.snapshot()[0]
    lr = f32(2e-3)
    c.opt.step(lr, 0.9, 0.999, eps, 1)
    e = f32(eps)
    _, m32, v32 = O.adam_update(p, g64, m, v, lr, 0.9, 0.999, e, 1, dtype=np.float32)
    # from the moments in binary32: what is asked for here is the update's own arithmetic
    below = np.sqrt(v32.astype(np.float64)) / np.sqrt(1 - 0.999) + e
    want = p - lr / (1 - 0.9) * m32.astype(np.float64) / below
    upd = np.abs(lr / (1 - 0.9) * m32.astype(np.float64) / below)
    got = c.params[0].double().cpu().numpy()
    ok = v32 > 0
    assert (np.abs(got - want)[ok] <= 16 * 2.0 ** -24 * upd[ok] + 4 * 2.0 ** -24 * np.abs(p[ok])).all()


def test_two_optimizers_on_two_streams():
    made = [Case([70000, 300, 8200], torch.bfloat16, torch.float32, True, 8, seed=7) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in made[1:]]
    outs = [torch.empty(2, device="cuda") for _ in made]
    torch.cuda.synchronize()
    for step in (1, 2, 3):
        for c, s, o in zip(made[1:], streams, outs[1:]):
            c.opt.norm(0.3, o, stream=s)
            c.opt.step(**HYPER, step=step, scale=o[1:], stream=s)
        torch.cuda.synchronize()
        made[0].opt.norm(0.3, outs[0])
        torch.cuda.synchronize()
        made[0].opt.step(**HYPER, step=step, scale=outs[0][1:])
        torch.cuda.synchronize()
        for c in made[1:]:
            for k in c.flat:
                assert torch.equal(c.flat[k], made[0].flat[k])
            for x, y in zip(c.m + c.v, made[0].m + made[0].v):
                assert torch.equal(x, y)


def test_gradients_written_just_before():
    """The norm and the step read what the kernel before them on the stream has just written."""
    runs = []
    for wait in (True, False):
        c = Case([300000, 1000], torch.float32, torch.float32, False, 32, seed=8)
        out = torch.empty(2, device="cuda")
        g0 = c.flat["grad"].clone()
        for step in range(1, 16):
            torch.mul(g0, 1.0 / step, out=c.flat["grad"])
            if wait:
                torch.cuda.synchronize()
            c.opt.norm(0.1, out)
            if wait:
                torch.cuda.synchronize()
            c.opt.step(**HYPER, step=step, scale=out[1:])
            if wait:
                torch.cuda.synchronize()
        torch.cuda.synchronize()
        runs.append(c)
    assert all(torch.equal(runs[0].flat[k], runs[1].flat[k]) for k in runs[0].flat)


def test_shared_gradients_and_noncontiguous_order():
    """Two parameters may take one gradient; tensors may lie in memory in any order."""
    buf = torch.randn(4000, device="cuda")
    g = 1e-2 * torch.randn(1000, device="cuda")
    params = [buf[2000:3000], buf[:1000]]
    ms, vs = ([torch.zeros(1000, device="cuda") for _ in range(2)] for _ in range(2))
    before = [p.double().cpu().numpy() for p in params]
    with G.AdamW(params, [g, g], ms, vs, weight_decay=0.0) as opt:
        opt.step(**HYPER, step=1)
    for p, b in zip(params, before):
        wp, _, _ = O.adam_update(b, g.double().cpu().numpy(), np.zeros(1000), np.zeros(1000),
                                 **dict(HYPER, lr=f32(HYPER["lr"])), step=1)
        assert np.abs(p.double().cpu().numpy() - wp).max() <= 2.0 ** -22 * np.abs(b).max()
