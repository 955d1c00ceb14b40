"""Measured cases of the 8-bit activation checkpoints and of the operators that read them.

A training step keeps a layer's input for its backward pass.  Kept in 8 bits (groups of 32 columns of
a row, int8 codes, one power-of-two scale per group) it takes 33/32 bytes an element.  The cases run

  checkpoint   pack a tensor and unpack it again;
  fn           an activation function's forward pass, which also writes the checkpoint of its input,
               and its backward pass from that checkpoint;
  norm         layer norm: the forward pass alone, the backward pass from the input alone, or a step
               (forward with the checkpoint of the input, backward from the checkpoint);
  weight_grad  a linear layer's weight and bias gradients, from its input's checkpoint.

``run`` computes them in elementary torch operations where ``own`` is false and calls the library
where it is true.
"""
import math

import torch

own = False

GROUP = 32
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5


def listed():
    return [
        # a small layer's input at a short sequence: latency
        {"name": "checkpoint_small", "op": "checkpoint", "dtype": "bf16", "rows": 32, "cols": 1024, "pad": 0},
        # fp32 activations whose rows are not aligned
        {"name": "checkpoint_odd", "op": "checkpoint", "dtype": "f32", "rows": 2049, "cols": 1001, "pad": 0},
        # a wide hidden layer of a long batch
        {"name": "checkpoint_large", "op": "checkpoint", "dtype": "bf16", "rows": 16384, "cols": 8192, "pad": 0},
        # the activation of a small hidden layer in fp16, its rows part of a wider buffer
        {"name": "fn_small", "op": "fn", "kind": "silu", "dtype": "f16", "rows": 128, "cols": 4096, "pad": 64},
        # the activation of a wide hidden layer of a long batch
        {"name": "fn_large", "op": "fn", "kind": "gelu", "dtype": "bf16", "rows": 16384, "cols": 8192, "pad": 0},
        # the norm of a few tokens: latency
        {"name": "norm_forward_small", "op": "norm", "part": "forward", "dtype": "bf16", "param": "bf16",
         "rows": 8, "cols": 1024, "pad": 0},
        # the norm of an ordinary layer, forward and backward through the checkpoint
        {"name": "norm_step", "op": "norm", "part": "step", "dtype": "bf16", "param": "f32",
         "rows": 16384, "cols": 4096, "pad": 0},
        # a backward pass from the input itself, odd sizes
        {"name": "norm_backward_odd", "op": "norm", "part": "backward", "dtype": "f16", "param": "f16",
         "rows": 4095, "cols": 1023, "pad": 0},
        # a few tokens: the gradient's own bytes are the work
        {"name": "weight_grad_few", "op": "weight_grad", "dtype": "bf16", "tokens": 16, "in": 1024, "out": 1024,
         "pad": 0, "bias": True},
        # an ordinary square layer
        {"name": "weight_grad_square", "op": "weight_grad", "dtype": "bf16", "tokens": 8192, "in": 4096, "out": 4096,
         "pad": 0, "bias": False},
        # the widest layer of a long batch
        {"name": "weight_grad_large", "op": "weight_grad", "dtype": "bf16", "tokens": 16384, "in": 4096,
         "out": 16384, "pad": 0, "bias": False},
        # fp32 gradients of odd sizes, with the bias
        {"name": "weight_grad_odd", "op": "weight_grad", "dtype": "f32", "tokens": 3001, "in": 1000, "out": 2499,
         "pad": 0, "bias": True},
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]; half of them multiples of 8, as layers' widths are."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        v = (v + 7) // 8 * 8
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["checkpoint", "fn", "norm", "weight_grad"])
    case = {"op": op, "dtype": rng.choice(["f32", "bf16", "f16"]), "pad": rng.choice([0, 0, 8, 24, 5])}
    if op == "weight_grad":
        t, k, n = _log(rng, 1, 16384), _log(rng, 16, 8192), _log(rng, 16, 8192)
        case.update({"tokens": t, "in": k, "out": n, "bias": rng.random() < 0.5})
        return case
    rows, cols = _log(rng, 1, 16384), _log(rng, 16, 8192)
    if rows * cols > 2 ** 26:
        rows = 2 ** 26 // cols
    case.update({"rows": rows, "cols": cols})
    if op == "fn":
        case["kind"] = rng.choice(["gelu", "gelu_tanh", "silu"])
    if op == "norm":
        case["part"] = rng.choice(["forward", "backward", "step"])
        case["param"] = rng.choice(["f32", case["dtype"]])
    return case


def _padded(t, dtype, pad):
    """t rounded to dtype, its rows pad elements further apart than they are wide."""
    rows, cols = t.shape
    buf = torch.zeros(rows, cols + pad, dtype=dtype, device=t.device)
    out = buf[:, :cols]
    out.copy_(t)
    return out


def _like(x, pad):
    return _padded(torch.zeros(x.shape, device=x.device), x.dtype, pad)


def _pitches(cols):
    return (cols + 31) // 32 * 32, (cols + 127) // 128 * 4


def _layout(rows, cols):
    """(bytes, offset of the exponents) of a checkpoint: rows of codes, each padded to whole groups, then
    rows of exponents, each padded to four groups; both regions in whole 16 bytes."""
    cp, ep = _pitches(cols)
    e_off = (rows * cp + 15) // 16 * 16
    return e_off + (rows * ep + 15) // 16 * 16, e_off


def _pow2(e):
    """2^e in 64 bits, from its bits: exp2 may be off by a rounding, which moves ties."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _plain_codes(x):
    """The codes (rows, groups, 32) and exponent bytes (rows, groups) of x."""
    rows, cols = x.shape
    groups = (cols + GROUP - 1) // GROUP
    v = torch.zeros(rows, groups * GROUP, dtype=torch.float32, device=x.device)
    v[:, :cols] = x
    v = v.view(rows, groups, GROUP)
    m = v.abs().amax(2)
    e = ((m.view(torch.int32) + 0x10000) >> 23).clamp(max=254)
    e = torch.where(torch.isfinite(v).all(2), e, torch.full_like(e, 255))
    # in 64 bits, where neither the scale nor its reciprocal leaves the range
    q = torch.round(v.double() * _pow2(133 - e).unsqueeze(2)).clamp(-127, 127)
    q = torch.where(e.unsqueeze(2) == 255, torch.zeros_like(q), q)
    return q.to(torch.int8), e.to(torch.uint8)


def _to_buffer(q, e, rows, cols):
    size, e_off = _layout(rows, cols)
    cp, ep = _pitches(cols)
    buf = torch.zeros(size, dtype=torch.uint8, device=q.device)
    buf[:rows * cp].view(rows, cp).copy_(q.reshape(rows, cp).view(torch.uint8))
    buf[e_off:e_off + rows * ep].view(rows, ep)[:, :e.shape[1]] = e
    return buf


def _plain_values(q, e, cols, dtype):
    """The values of codes and exponents, rounded to dtype (and, in fp16, saturated)."""
    v = q.double() * _pow2(e.to(torch.int64) - 133).unsqueeze(2)
    v = torch.where(e.unsqueeze(2) == 255, torch.full_like(v, float("nan")), v)
    v = v.reshape(q.shape[0], -1)[:, :cols]
    if dtype == torch.float16:
        v = v.clamp(-65504.0, 65504.0)
    return v.to(dtype)


def _from_buffer(buf, rows, cols, dtype):
    _, e_off = _layout(rows, cols)
    cp, ep = _pitches(cols)
    q = buf[:rows * cp].view(torch.int8).view(rows, cp // GROUP, GROUP)
    e = buf[e_off:e_off + rows * ep].view(rows, ep)[:, :cp // GROUP]
    return _plain_values(q, e, cols, dtype)


def _activations(gen, rows, cols, dev):
    """Hidden activations: unit scale, a few channels an order of magnitude larger, rows of their own scale."""
    x = torch.randn(rows, cols, generator=gen, device=dev)
    channel = torch.where(torch.rand(cols, generator=gen, device=dev) < 0.01, 12.0, 1.0)
    row = torch.exp(0.3 * torch.randn(rows, 1, generator=gen, device=dev))
    return x * channel * row + 0.1


def _gradients(gen, rows, cols, dev):
    """Output gradients: small, rows of very different sizes, every sixteenth row or so a masked token."""
    g = torch.randn(rows, cols, generator=gen, device=dev)
    row = torch.exp(torch.randn(rows, 1, generator=gen, device=dev)) * 1e-2
    keep = torch.rand(rows, 1, generator=gen, device=dev) > 1 / 16
    return g * row * keep


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 2 + 1)
    dtype, pad = DTYPES[case["dtype"]], case["pad"]
    s = {"case": case}
    if case["op"] == "weight_grad":
        t, k, n = case["tokens"], case["in"], case["out"]
        x = _activations(gen, t, k, dev).to(dtype)
        s["ckpt"] = _to_buffer(*_plain_codes(x), t, k)
        s["dy"] = _padded(_gradients(gen, t, n, dev), dtype, pad)
        # the layer's slices of the flat fp32 gradient vector
        flat = torch.zeros(n * k + n, device=dev)
        s["dw"] = flat[:n * k].view(n, k)
        s["db"] = flat[n * k:] if case["bias"] else None
        if own:
            from gradient_quantization_communication_b200 import gq as G
            s["workspace"] = G.gq_act_weight_grad_workspace(s["ckpt"], s["dy"], s["dw"], s["db"])
        return s
    rows, cols = case["rows"], case["cols"]
    s["x"] = _padded(_activations(gen, rows, cols, dev), dtype, pad)
    s["ckpt"] = torch.zeros(_layout(rows, cols)[0], dtype=torch.uint8, device=dev)
    s["y"] = _like(s["x"], pad)
    if case["op"] == "checkpoint":
        return s
    s["dy"] = _padded(_gradients(gen, rows, cols, dev), dtype, pad)
    s["dx"] = _like(s["x"], pad)
    if case["op"] == "norm":
        param = DTYPES[case["param"]]
        s["gamma"] = (1.0 + 0.2 * torch.randn(cols, generator=gen, device=dev)).to(param)
        s["beta"] = (0.1 * torch.randn(cols, generator=gen, device=dev)).to(param)
        s["mean"] = torch.zeros(rows, device=dev)
        s["rstd"] = torch.zeros(rows, device=dev)
        s["dgamma"] = torch.zeros(cols, device=dev)
        s["dbeta"] = torch.zeros(cols, device=dev)
        if case["part"] == "backward":
            v = s["x"].double()
            s["mean"].copy_(v.mean(1))
            s["rstd"].copy_(1.0 / torch.sqrt(v.var(1, unbiased=False) + EPS))
        if own and case["part"] != "forward":
            from gradient_quantization_communication_b200 import gq as G
            s["workspace"] = G.gq_layer_norm_workspace(s["dy"])
    return s


def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from gradient_quantization_communication_b200 import gq as G
    case = s["case"]
    if case["op"] == "checkpoint":
        G.gq_act_pack(s["x"], s["ckpt"])
        G.gq_act_unpack(s["ckpt"], s["y"])
        return s["y"]
    if case["op"] == "fn":
        G.gq_act_fn_forward(case["kind"], s["x"], s["y"], s["ckpt"])
        G.gq_act_fn_backward(case["kind"], s["ckpt"], s["dy"], s["dx"])
        return s["y"], s["dx"]
    if case["op"] == "weight_grad":
        G.gq_act_weight_grad(s["ckpt"], s["dy"], s["dw"], s["db"], workspace=s["workspace"])
        return (s["dw"], s["db"]) if case["bias"] else s["dw"]
    if case["part"] == "forward":
        G.gq_layer_norm_forward(s["x"], s["gamma"], s["beta"], EPS, s["y"], s["mean"], s["rstd"])
        return s["y"], s["mean"], s["rstd"]
    if case["part"] == "backward":
        G.gq_layer_norm_backward(s["dy"], s["x"], s["gamma"], s["mean"], s["rstd"], s["dx"], s["dgamma"], s["dbeta"],
                                 workspace=s["workspace"])
        return s["dx"], s["dgamma"], s["dbeta"]
    G.gq_layer_norm_forward(s["x"], s["gamma"], s["beta"], EPS, s["y"], s["mean"], s["rstd"], s["ckpt"])
    G.gq_layer_norm_backward(s["dy"], s["ckpt"], s["gamma"], s["mean"], s["rstd"], s["dx"], s["dgamma"], s["dbeta"],
                             workspace=s["workspace"])
    return s["y"], s["dx"], s["dgamma"], s["dbeta"]


def _plain_fn(kind, x):
    if kind == "gelu":
        # the normal distribution's tail through erfc: 1 + erf cancels for negative x
        return 0.5 * x * torch.special.erfc(-x * math.sqrt(0.5))
    if kind == "gelu_tanh":
        return x * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x))
    return x * torch.sigmoid(x)


def _plain_fn_grad(kind, x):
    if kind == "gelu":
        return 0.5 * torch.special.erfc(-x * math.sqrt(0.5)) + x * torch.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
    if kind == "gelu_tanh":
        c = 2.0 * math.sqrt(2.0 / math.pi)
        g = torch.sigmoid(c * (x + 0.044715 * x * x * x))
        return g + x * g * (1.0 - g) * c * (1.0 + 3.0 * 0.044715 * x * x)
    g = torch.sigmoid(x)
    return g * (1.0 + x * (1.0 - g))


def _plain_norm_backward(dy, x, s):
    xh = (x - s["mean"].unsqueeze(1)) * s["rstd"].unsqueeze(1)
    g = dy * s["gamma"].float()
    dx = (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)) * s["rstd"].unsqueeze(1)
    return dx.to(s["dy"].dtype), (dy * xh).sum(0), dy.sum(0)


def _run_plain(s):
    case = s["case"]
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "checkpoint":
        q, e = _plain_codes(s["x"])
        return _plain_values(q, e, case["cols"], dtype)
    if case["op"] == "fn":
        q, e = _plain_codes(s["x"])
        y = _plain_fn(case["kind"], s["x"].float()).to(dtype)
        x = _plain_values(q, e, case["cols"], torch.float32)
        return y, (s["dy"].float() * _plain_fn_grad(case["kind"], x)).to(dtype)
    if case["op"] == "weight_grad":
        # fp16 takes the decoded input in fp16, as it would be kept; bf16 and fp32 hold it exactly
        decoded = torch.float16 if dtype == torch.float16 else torch.float32
        x = _from_buffer(s["ckpt"], case["tokens"], case["in"], decoded).float()
        dy = s["dy"].float()
        dw = dy.t() @ x
        return (dw, dy.sum(0)) if case["bias"] else dw
    if case["part"] == "backward":
        return _plain_norm_backward(s["dy"].float(), s["x"].float(), s)
    x = s["x"].float()
    s["mean"] = x.mean(1)
    centred = x - s["mean"].unsqueeze(1)
    s["rstd"] = 1.0 / torch.sqrt((centred * centred).mean(1) + EPS)
    y = (centred * s["rstd"].unsqueeze(1) * s["gamma"].float() + s["beta"].float()).to(dtype)
    if case["part"] == "forward":
        return y, s["mean"], s["rstd"]
    q, e = _plain_codes(s["x"])
    return (y, *_plain_norm_backward(s["dy"].float(), _plain_values(q, e, case["cols"], torch.float32), s))


def work(case):
    size = SIZE[case["dtype"]]
    if case["op"] == "weight_grad":
        t, k, n = case["tokens"], case["in"], case["out"]
        groups = (k + 31) // 32
        return {"bytes": t * (k + groups) + t * n * size + 4 * n * k + (4 * n if case["bias"] else 0),
                "flops": 2 * t * k * n + (t * n if case["bias"] else 0)}
    rows, cols = case["rows"], case["cols"]
    tensor = rows * cols * size
    kept = rows * (cols + (cols + 31) // 32)
    if case["op"] == "checkpoint":
        # the tensor in, the checkpoint out and in again, the tensor out
        return {"bytes": 2 * tensor + 2 * kept, "flops": 4 * rows * cols}
    if case["op"] == "fn":
        return {"bytes": 4 * tensor + 2 * kept, "flops": 40 * rows * cols}
    params = 2 * cols * SIZE[case["param"]]
    if case["part"] == "forward":
        return {"bytes": 2 * tensor + params + 8 * rows, "flops": 8 * rows * cols}
    back = params // 2 + 8 * rows + 8 * cols
    if case["part"] == "backward":
        return {"bytes": 3 * tensor + back, "flops": 14 * rows * cols}
    return {"bytes": 4 * tensor + 2 * kept + params + 8 * rows + back, "flops": 26 * rows * cols}


# ----------------------------------------------------------------------------------------------------
# The definitions in 64 bits.
# ----------------------------------------------------------------------------------------------------
def _exact_checkpoint(x):
    """x through the checkpoint: in every run of 32 columns, the nearest multiples (ties to even) of the
    smallest power of two that keeps every code within 127."""
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for lo in range(0, x.shape[1], GROUP):
        part = x[:, lo:lo + GROUP].double()
        mant, exp = torch.frexp(part.abs().amax(1, keepdim=True))   # m = mant * 2^exp, mant in [1/2, 1)
        e = exp - 7 + (mant * 128 >= 127.5).to(exp.dtype)
        # the exponent is a byte: fp32's subnormal groups share the lowest scale
        table = torch.tensor([2.0 ** i for i in range(-133, 122)], dtype=torch.float64, device=x.device)
        step = table[e.clamp(-133, 121).long() + 133]
        out[:, lo:lo + GROUP] = torch.round(part / step).clamp(-127, 127) * step
    return out


def _exact_fn(kind, x):
    """The function and its derivative."""
    if kind == "silu":
        p = 1 / (1 + torch.exp(-x))
        return x * p, p + x * p * (1 - p)
    if kind == "gelu_tanh":
        a = math.sqrt(2 / math.pi)
        u = a * (x + 0.044715 * x ** 3)
        p = 1 / (1 + torch.exp(-2 * u))
        return x * p, p + x * 2 * p * (1 - p) * a * (1 + 3 * 0.044715 * x ** 2)
    p = torch.special.ndtr(x)
    return x * p, p + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "checkpoint":
        return _exact_checkpoint(s["x"])
    if case["op"] == "fn":
        y = _exact_fn(case["kind"], s["x"].double())[0]
        return y, s["dy"].double() * _exact_fn(case["kind"], _exact_checkpoint(s["x"]))[1]
    if case["op"] == "weight_grad":
        t, k = case["tokens"], case["in"]
        # the codes and exponents as the buffer holds them
        cp, ep = (k + 31) // 32 * 32, (k + 127) // 128 * 4
        e0 = -(-t * cp // 16) * 16
        codes = s["ckpt"][:t * cp].view(torch.int8).reshape(t, cp)[:, :k].double()
        scale = s["ckpt"][e0:e0 + t * ep].reshape(t, ep).repeat_interleave(32, 1)[:, :k].long()
        x = codes * torch.tensor([2.0 ** i for i in range(-133, 123)], dtype=torch.float64, device=codes.device)[scale]
        if case["dtype"] == "f16":
            x = x.clamp(-65504, 65504).half().double()
        dw = torch.einsum("tn,tk->nk", s["dy"].double(), x)
        return (dw, torch.einsum("tn->n", s["dy"].double())) if case["bias"] else dw
    x = s["x"].double()
    var, mean = torch.var_mean(x, dim=1, correction=0, keepdim=True)
    rstd = (var + EPS) ** -0.5
    if case["part"] == "backward":
        mean, rstd = s["mean"].double()[:, None], s["rstd"].double()[:, None]
    y = (x - mean) * rstd * s["gamma"].double() + s["beta"].double()
    if case["part"] == "forward":
        return y, mean[:, 0], rstd[:, 0]
    kept = x if case["part"] == "backward" else _exact_checkpoint(s["x"])
    n = (kept - mean) * rstd
    dy = s["dy"].double()
    g = dy * s["gamma"].double()
    dx = rstd * (g - torch.einsum("tc->t", g)[:, None] / x.shape[1]
                 - n * torch.einsum("tc,tc->t", g, n)[:, None] / x.shape[1])
    grads = dx, torch.einsum("tc,tc->c", dy, n), torch.einsum("tc->c", dy)
    return grads if case["part"] == "backward" else (y, *grads)
