"""Measured cases of the step around the gradient exchange: the optimizer that takes the averaged
gradient, and a linear layer's products in 8-bit floating point.

  adamw    one AdamW step over many tensors at once, from slices of the flat averaged gradient, with the
           moments in 32 bits or in 8 (blocks of 128, one power of two a block; the second moment rounded
           stochastically by Philox4x32-10 keyed on the seed, the step, the tensor and the element), with or
           without a 32-bit master copy of 16-bit parameters, with or without clipping by the global norm;
  pack     a matrix into 8-bit floating point with a power-of-two scale for every 128 columns of a row (or every
           128 x 128 tile), along its rows and along its columns in one pass, and back;
  linear   a linear layer's products from such operands: the forward pass (packs its input), the input's gradient
           (packs the output's gradient) and the weight's gradient (packs it along the tokens).

``run`` computes them in elementary torch operations where ``own`` is false and calls the library
where it is true.
"""
import itertools
import math
import random

import torch

own = False

BLOCK = 128
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
FORMATS = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
TOP = {"e4m3": 8, "e5m2": 15}       # the largest code of either format is 1.75 * 2^TOP
LR, BETA1, BETA2, EPS, DECAY, MAX_NORM = 3e-4, 0.9, 0.999, 1e-8, 0.1, 1.0
FIRST_STEP, SEED = 100, 42


def listed():
    return [
        # the few tensors of one small layer: latency
        {"name": "adamw_small", "op": "adamw", "tensors": "layer256", "param": "f32", "grad": "f32", "master": False,
         "bits": 32, "clip": False},
        # the 161 tensors of ResNet-50 (25.6M), fp32 throughout, the averaged gradient clipped by its norm
        {"name": "adamw_resnet50", "op": "adamw", "tensors": "resnet50", "param": "f32", "grad": "f32", "master": False,
         "bits": 32, "clip": True},
        # mixed precision: bf16 parameters and gradients, fp32 master copies, 268M in 64 matrices
        {"name": "adamw_master_large", "op": "adamw", "tensors": "equal:64:4194304", "param": "bf16", "grad": "bf16",
         "master": True, "bits": 32, "clip": False},
        # ResNet-18 (62 tensors, 11.7M) with the moments in 8 bits
        {"name": "adamw8_resnet18", "op": "adamw", "tensors": "resnet18", "param": "f32", "grad": "f32", "master": False,
         "bits": 8, "clip": True},
        # a quarter of the billion-element gradient: 250 tensors of 1e6 (no whole number of blocks), bf16 parameters
        {"name": "adamw8_blocks", "op": "adamw", "tensors": "equal:250:1000000", "param": "bf16", "grad": "f32",
         "master": False, "bits": 8, "clip": False},
        # fp32 activations whose rows are not aligned, both ways, in the format of gradients
        {"name": "pack_odd", "op": "pack", "dtype": "f32", "rows": 2049, "cols": 1001, "pad": 0, "fmt": "e5m2",
         "tile": False, "ways": "both"},
        # the input of a wide hidden layer of a long batch, both ways: for the forward pass and the weight's gradient
        {"name": "pack_large", "op": "pack", "dtype": "bf16", "rows": 16384, "cols": 8192, "pad": 0, "fmt": "e4m3",
         "tile": False, "ways": "both"},
        # a few tokens through an ordinary layer: the weight's bytes are the work
        {"name": "linear_few_tokens", "op": "linear", "part": "forward", "dtype": "bf16", "fmt": "e4m3", "tokens": 16,
         "in": 4096, "out": 4096, "bias": True},
        # an ordinary square layer
        {"name": "linear_square", "op": "linear", "part": "forward", "dtype": "bf16", "fmt": "e4m3", "tokens": 8192,
         "in": 4096, "out": 4096, "bias": True},
        # the widest layer of a long batch
        {"name": "linear_large", "op": "linear", "part": "forward", "dtype": "bf16", "fmt": "e4m3", "tokens": 16384,
         "in": 4096, "out": 16384, "bias": False},
        # the input's gradient at odd sizes, from a gradient in e5m2
        {"name": "linear_input_grad_odd", "op": "linear", "part": "input_grad", "dtype": "f16", "fmt": "e5m2",
         "tokens": 3001, "in": 1000, "out": 2499, "bias": False},
        # the weight's gradient, added to the layer's slice of the flat fp32 gradient
        {"name": "linear_weight_grad", "op": "linear", "part": "weight_grad", "dtype": "bf16", "fmt": "e4m3",
         "tokens": 8192, "in": 4096, "out": 4096, "bias": False},
    ]


def _log(rng, lo, hi):
    """An integer spread over the logarithm of [lo, hi]; half of them multiples of 8, as layers' widths are."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5:
        v = (v + 7) // 8 * 8
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["adamw", "adamw", "pack", "linear", "linear"])
    if op == "adamw":
        count = _log(rng, 1, 300)
        param = rng.choice(["f32", "bf16", "f16"])
        return {"op": op, "tensors": "odd:%d:%d:%d" % (count, _log(rng, 1000, 2 ** 26), rng.randrange(1 << 30)),
                "param": param, "grad": rng.choice(["f32", param]), "master": param != "f32" and rng.random() < 0.5,
                "bits": rng.choice([8, 32]), "clip": rng.random() < 0.5}
    case = {"op": op, "dtype": rng.choice(["f32", "bf16", "f16"]), "fmt": rng.choice(["e4m3", "e4m3", "e5m2"])}
    if op == "pack":
        rows, cols = _log(rng, 1, 16384), _log(rng, 16, 8192)
        if rows * cols > 2 ** 26:
            rows = 2 ** 26 // cols
        case.update({"rows": rows, "cols": cols, "pad": rng.choice([0, 0, 8, 24, 5]), "tile": rng.random() < 0.3,
                     "ways": rng.choice(["rows", "both", "cols"])})
        return case
    case.update({"part": rng.choice(["forward", "forward", "input_grad", "weight_grad"]), "tokens": _log(rng, 1, 16384),
                 "in": _log(rng, 16, 8192), "out": _log(rng, 16, 8192)})
    case["bias"] = case["part"] == "forward" and rng.random() < 0.5
    return case


# ----------------------------------------------------------------------------------------------------
# Tensors of a model
# ----------------------------------------------------------------------------------------------------
def _residual_block(planes, inplanes, expansion, first):
    out = planes * expansion
    convs = [planes * inplanes * 9, planes * planes * 9] if expansion == 1 else \
        [planes * inplanes, planes * planes * 9, out * planes]
    widths = [planes, planes] if expansion == 1 else [planes, planes, out]
    sizes = [v for c, w in zip(convs, widths) for v in (c, w, w)]
    return sizes + ([out * inplanes, out, out] if first and inplanes != out else [])


def _resnet(blocks, expansion):
    planes = [64, 128, 256, 512]
    return [9408, 64, 64] + [
        v for s, n in enumerate(blocks) for b in range(n)
        for v in _residual_block(planes[s], planes[s] * expansion if b else (planes[s - 1] * expansion if s else 64),
                                 expansion, b == 0)] + [1000 * 512 * expansion, 1000]


def _sizes(case):
    """Elements of each tensor."""
    what = case["tensors"].split(":")
    if what[0] == "layer256":
        return [256 * 256, 256, 256, 256, 1000 * 256, 1000]
    if what[0] == "resnet18":
        return _resnet([2, 2, 2, 2], 1)
    if what[0] == "resnet50":
        return _resnet([3, 4, 6, 3], 4)
    if what[0] == "equal":
        return [int(what[2])] * int(what[1])
    # matrices, vectors and single values, odd sizes among them
    count, total, rng = int(what[1]), int(what[2]), random.Random(int(what[3]))
    share = [math.exp(rng.uniform(0.0, 7.0)) for _ in range(count)]
    odd = [rng.random() < 0.5 for _ in range(count)]
    sizes = [max(1, int(total * s / sum(share))) for s in share]
    return [n if o else (n + 7) // 8 * 8 for n, o in zip(sizes, odd)]


def _up(n, to):
    return (n + to - 1) // to * to


def _moment_bytes(n):
    """Bytes of a moment of n elements in 8 bits: whole blocks of codes, then the blocks' exponents in whole 16s."""
    nb = (n + BLOCK - 1) // BLOCK
    return nb * BLOCK + _up(nb, 16)


def _moment_views(buf, sizes):
    """Each tensor's codes and exponents in a buffer that holds all tensors' moments one after another."""
    nbs = [(n + BLOCK - 1) // BLOCK for n in sizes]
    starts = list(itertools.accumulate((_moment_bytes(n) for n in sizes), initial=0))
    return ([buf[s:s + nb * BLOCK] for s, nb in zip(starts, nbs)],
            [buf[s + nb * BLOCK:s + nb * BLOCK + nb] for s, nb in zip(starts, nbs)])


def _blocks(flat, sizes):
    """A flat vector as rows of 128, each tensor padded with 0 to whole rows."""
    return torch.cat([torch.nn.functional.pad(t, (0, -t.numel() % BLOCK)) for t in flat.split(sizes)]).view(-1, BLOCK)


def _unblocks(rows, sizes):
    """The flat vector of rows of 128."""
    nbs = [(n + BLOCK - 1) // BLOCK for n in sizes]
    return torch.cat([t.reshape(-1)[:n] for t, n in zip(rows.split(nbs), sizes)])


# ----------------------------------------------------------------------------------------------------
# Formats.  A block's exponent byte E stands for 2^(E - 127); E = 255 marks one with a NaN or an infinity.
# ----------------------------------------------------------------------------------------------------
def _pow2(e):
    """2^(e - 127) in 32 bits, 1 <= e <= 254."""
    return (e.to(torch.int32) << 23).view(torch.float32)


def _float_exponent(largest, fmt):
    """The smallest E with largest <= 1.75 * 2^TOP * 2^(E - 127), at least 10."""
    bits = largest.view(torch.int32)
    e = (((bits + 0x1FFFFF) >> 23) - TOP[fmt]).clamp(10, 254 - TOP[fmt] + 1)
    return torch.where(torch.isfinite(largest), e, torch.full_like(e, 255))


def _float_codes(v, e, fmt):
    """The codes of v (fp32) under exponents e (broadcastable)."""
    scaled = v * _pow2((254 - e).clamp(min=1))
    codes = scaled.to(FORMATS[fmt]).view(torch.uint8)
    return torch.where(e == 255, torch.full_like(codes, 0x7F), codes)


def _float_values(codes, e, fmt):
    return codes.view(FORMATS[fmt]).float() * _pow2(e)


def _largest(v, dims):
    # amax passes NaN on
    return v.abs().amax(dims, keepdim=True)


def _square_codes(v, noise):
    """A second moment's codes and exponents, v rows of 128: 5 exponent and 3 mantissa bits, no sign, 16 random
    bits deciding whether the 20 bits below round up; 0 only for 0."""
    bits = v.view(torch.int32)
    top = _largest(v, 1)
    e = ((top.view(torch.int32) + 0xFFFFF) >> 23).clamp(32, 254)
    e = torch.where(torch.isfinite(top), e, torch.full_like(e, 255))
    code = ((bits + (noise << 4)) >> 20) - ((e - 31) << 3)
    code = torch.where(v > 0, code.clamp(1, 255), torch.zeros_like(code))
    return torch.where(e == 255, torch.zeros_like(code), code).to(torch.uint8), e


def _square_values(codes, e):
    c = codes.to(torch.int32)
    v = ((c + ((e.to(torch.int32) - 31) << 3)) << 20).view(torch.float32)
    v = torch.where(c == 0, torch.zeros_like(v), v)
    return torch.where(e == 255, torch.full_like(v, float("nan")), v)


def _philox(words, key):
    """Philox4x32-10: the counter's four words (int64 tensors of 32-bit values) under a 64-bit key."""
    def round_(c, k):
        p0, p1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57      # the low 64 bits, as the wrapped product has them
        return [((p1 >> 32) & 0xFFFFFFFF) ^ c[1] ^ k[0], p1 & 0xFFFFFFFF,
                ((p0 >> 32) & 0xFFFFFFFF) ^ c[3] ^ k[1], p0 & 0xFFFFFFFF]

    def rounds(c, k, left):
        return c if left == 0 else rounds(round_(c, k), ((k[0] + 0x9E3779B9) & 0xFFFFFFFF,
                                                         (k[1] + 0xBB67AE85) & 0xFFFFFFFF), left - 1)

    return rounds(list(words), (key & 0xFFFFFFFF, key >> 32), 10)


def _noise(sizes, step, dev):
    """16 random bits for each element of each tensor's rows of 128: a draw for every 8 elements, the tensor's
    number (and the top bit) in the counter's last word; even elements take the low halves."""
    nbs = torch.tensor([(n + BLOCK - 1) // BLOCK for n in sizes], device=dev)
    groups = nbs * (BLOCK // 8)
    tensor = torch.repeat_interleave(torch.arange(len(sizes), device=dev), groups)
    at = torch.arange(int(groups.sum()), device=dev) - torch.repeat_interleave(torch.cumsum(groups, 0) - groups, groups)
    words = _philox((at & 0xFFFFFFFF, at >> 32, torch.full_like(at, step & 0xFFFFFFFF), tensor | 0x80000000), SEED)
    w = torch.stack(words, 1)
    return torch.stack((w & 0xFFFF, w >> 16), 2).to(torch.int32).view(-1, BLOCK)


# ----------------------------------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------------------------------
def _padded(t, dtype, pad):
    """t rounded to dtype, its rows pad elements further apart than they are wide."""
    rows, cols = t.shape
    buf = torch.zeros(rows, cols + pad, dtype=dtype, device=t.device)
    out = buf[:, :cols]
    out.copy_(t)
    return out


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


def _packed_layout(rows, cols, tile):
    """(bytes, code pitch, offset of the exponents, rows of exponents, exponent pitch) of a packed matrix."""
    cp, ep, er = _up(cols, BLOCK), 4 * ((cols + 511) // 512), (rows + BLOCK - 1) // BLOCK if tile else rows
    off = _up(rows * cp, 16)
    return off + _up(er * ep, 16), cp, off, er, ep


def _plain_pack(x, fmt, tile):
    """(codes, exponents) of the rows' blocks: codes (rows, blocks, 128), exponents (rows or rows / 128, blocks)."""
    rows, cols = x.shape
    up = BLOCK if tile else 1
    v = torch.nn.functional.pad(x.float(), (0, -cols % BLOCK, 0, -rows % up))
    v = v.view(v.shape[0] // up, up, -1, BLOCK)
    e = _float_exponent(_largest(v, (1, 3)), fmt)
    codes = _float_codes(v, e, fmt).reshape(-1, v.shape[2], BLOCK)[:rows]
    return codes, e[:, 0, :, 0]


def _plain_values(codes, e, fmt, tile, cols):
    rows = codes.shape[0]
    if tile:
        e = e.repeat_interleave(BLOCK, 0)[:rows]
    return _float_values(codes, e.unsqueeze(2), fmt).reshape(rows, -1)[:, :cols]


def _to_buffer(codes, e, rows, cols, tile):
    size, cp, off, er, ep = _packed_layout(rows, cols, tile)
    buf = torch.zeros(size, dtype=torch.uint8, device=codes.device)
    buf[:rows * cp].view(rows, cp).copy_(codes.reshape(rows, cp))
    buf[off:off + er * ep].view(er, ep)[:, :e.shape[1]] = e.to(torch.uint8)
    return buf


def _from_buffer(buf, rows, cols, fmt, tile):
    _, cp, off, er, ep = _packed_layout(rows, cols, tile)
    codes = buf[:rows * cp].view(rows, cp // BLOCK, BLOCK)
    return _plain_values(codes, buf[off:off + er * ep].view(er, ep)[:, :cp // BLOCK], fmt, tile, cols)


def _empty_packed(rows, cols, tile, dev):
    return torch.zeros(_packed_layout(rows, cols, tile)[0], dtype=torch.uint8, device=dev)


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 2 + 1)
    s = {"case": case}
    if case["op"] == "adamw":
        return _prepare_adamw(s, case, gen, dev)
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "pack":
        rows, cols, tile = case["rows"], case["cols"], case["tile"]
        s["x"] = _padded(_activations(gen, rows, cols, dev), dtype, case["pad"])
        if case["ways"] != "cols":
            s["packed"] = _empty_packed(rows, cols, tile, dev)
            s["y"] = torch.zeros(rows, cols, dtype=dtype, device=dev)
        if case["ways"] != "rows":
            s["packed_t"] = _empty_packed(cols, rows, tile, dev)
            s["y_t"] = torch.zeros(cols, rows, dtype=dtype, device=dev)
        return s
    t, k, n = case["tokens"], case["in"], case["out"]
    if case["part"] == "weight_grad":
        # the input's columns, as the forward pass packed them
        x = _activations(gen, t, k, dev).to(dtype)
        s["x_t"] = _to_buffer(*_plain_pack(x.t(), "e4m3", False), k, t, False)
        s["dy"] = _gradients(gen, t, n, dev).to(dtype)
        s["dy_t"] = _empty_packed(n, t, False, dev)
        # the layer's slice of the flat fp32 gradient, which holds an earlier micro-batch's
        s["dw"] = 1e-2 * torch.randn(n * k, generator=gen, device=dev).view(n, k)
        out = s["dw"], t
    else:
        w = torch.randn(n, k, generator=gen, device=dev) / math.sqrt(k)
        if case["part"] == "forward":
            s["x"] = _activations(gen, t, k, dev).to(dtype)
            s["bias"] = torch.randn(n, generator=gen, device=dev) if case["bias"] else None
            s["w"] = _to_buffer(*_plain_pack(w, "e4m3", True), n, k, True)
            s["packed"], s["y"] = _empty_packed(t, k, False, dev), torch.zeros(t, n, dtype=dtype, device=dev)
        else:
            s["x"] = _gradients(gen, t, n, dev).to(dtype)
            s["bias"] = None
            s["w"] = _to_buffer(*_plain_pack(w.t(), "e4m3", True), k, n, True)
            s["packed"], s["y"] = _empty_packed(t, n, False, dev), torch.zeros(t, k, dtype=dtype, device=dev)
        out = s["y"], s["x"].shape[1]
    if own:
        from gradient_quantization_communication_b200 import gq as G
        s["workspace"] = G.gq_fp8_matmul_workspace(out[1], out[0])
    return s


def _prepare_adamw(s, case, gen, dev):
    sizes = _sizes(case)
    total = sum(sizes)
    s["sizes"], s["step"] = sizes, FIRST_STEP
    count = torch.tensor(sizes, device=dev)
    # tensors' gradients of very different sizes, as the averaged gradient's slices have
    scale = torch.exp(math.log(10.0) * (-2.0 - 3.0 * torch.rand(len(sizes), generator=gen, device=dev)))
    scale = torch.repeat_interleave(scale, count)
    s["grad"] = (torch.randn(total, generator=gen, device=dev) * scale).to(DTYPES[case["grad"]])
    param = 0.02 * torch.randn(total, generator=gen, device=dev)
    s["master"] = param if case["master"] else None
    s["param"] = param.to(DTYPES[case["param"]]).clone()
    m = 0.3 * torch.randn(total, generator=gen, device=dev) * scale
    # as after a hundred steps: about a tenth of the squares' mean, from element to element within a factor of some e
    v = 0.1 * torch.exp(0.5 * torch.randn(total, generator=gen, device=dev)) * scale * scale
    decays = [DECAY if n > 4096 else 0.0 for n in sizes]
    s["decay"] = torch.repeat_interleave(torch.tensor(decays, device=dev), count)
    s["norm"] = torch.zeros(2, device=dev)
    if case["bits"] == 32:
        s["m"], s["v"] = m, v
        moments = [t.split(sizes) for t in (m, v)]
    else:
        size = sum(_moment_bytes(n) for n in sizes)
        s["m8"], s["v8"] = (torch.zeros(size, dtype=torch.uint8, device=dev) for _ in range(2))
        _store_moments(s, _blocks(m, sizes), _blocks(v, sizes), 0)
        s["m_out"], s["v_out"] = (torch.zeros(total, dtype=torch.bfloat16, device=dev) for _ in range(2))
        moments = [t.split([_moment_bytes(n) for n in sizes]) for t in (s["m8"], s["v8"])]
    if own:
        from gradient_quantization_communication_b200 import gq as G
        masters = s["master"].split(sizes) if case["master"] else None
        s["opt"] = G.AdamW(s["param"].split(sizes), s["grad"].split(sizes), *moments, masters=masters,
                           weight_decay=decays, state_bits=case["bits"], seed=SEED)
    return s


# ----------------------------------------------------------------------------------------------------
# The passes
# ----------------------------------------------------------------------------------------------------
def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    from gradient_quantization_communication_b200 import gq as G
    case = s["case"]
    if case["op"] == "adamw":
        if case["clip"]:
            G.gq_adamw_norm(s["opt"].handle, MAX_NORM, s["norm"])
        G.gq_adamw_step(s["opt"].handle, LR, BETA1, BETA2, EPS, s["step"], scale=s["norm"][1:] if case["clip"] else None)
        s["step"] += 1
        if case["bits"] == 8:
            G.gq_adamw_moments(s["opt"].handle, s["m_out"], s["v_out"])
        return _adamw_outputs(s)
    if case["op"] == "pack":
        fmt, tile = case["fmt"], case["tile"]
        G.gq_fp8_pack(s["x"], s.get("packed"), s.get("packed_t"), fmt=fmt, tile=tile)
        if "packed" in s:
            G.gq_fp8_unpack(s["packed"], s["y"], fmt=fmt, tile=tile)
        if "packed_t" in s:
            G.gq_fp8_unpack(s["packed_t"], s["y_t"], fmt=fmt, tile=tile)
        return [s[y] for y in ("y", "y_t") if y in s]
    if case["part"] == "weight_grad":
        G.gq_fp8_pack(s["dy"], None, s["dy_t"], fmt=case["fmt"])
        G.gq_fp8_matmul(s["dy_t"], s["x_t"], case["tokens"], s["dw"], fmt=(case["fmt"], "e4m3"), accumulate=True,
                        workspace=s["workspace"])
        return s["dw"]
    G.gq_fp8_pack(s["x"], s["packed"], fmt=case["fmt"])
    G.gq_fp8_matmul(s["packed"], s["w"], s["x"].shape[1], s["y"], s["bias"], fmt=(case["fmt"], "e4m3"),
                    tile=(False, True), workspace=s["workspace"])
    return s["y"]


def _adamw_outputs(s):
    out = {"param": s["param"]}
    if s["case"]["master"]:
        out["master"] = s["master"]
    if s["case"]["clip"]:
        out["norm"] = s["norm"]
    out["m"], out["v"] = (s["m"], s["v"]) if s["case"]["bits"] == 32 else (s["m_out"], s["v_out"])
    return out


def _load_moments(s):
    codes, exps = _moment_views(s["m8"], s["sizes"])
    m = _float_values(torch.cat(codes).view(-1, BLOCK), torch.cat(exps).unsqueeze(1), "e4m3")
    codes, exps = _moment_views(s["v8"], s["sizes"])
    return m, _square_values(torch.cat(codes).view(-1, BLOCK), torch.cat(exps).unsqueeze(1))


def _store_moments(s, m, v, noise):
    nbs = [(n + BLOCK - 1) // BLOCK for n in s["sizes"]]
    e = _float_exponent(_largest(m, 1), "e4m3")
    codes, exps = _moment_views(s["m8"], s["sizes"])
    torch._foreach_copy_(codes, [c.reshape(-1) for c in _float_codes(m, e, "e4m3").split(nbs)])
    torch._foreach_copy_(exps, list(e.to(torch.uint8).view(-1).split(nbs)))
    c, e = _square_codes(v, torch.as_tensor(noise, device=v.device))
    codes, exps = _moment_views(s["v8"], s["sizes"])
    torch._foreach_copy_(codes, [x.reshape(-1) for x in c.split(nbs)])
    torch._foreach_copy_(exps, list(e.to(torch.uint8).view(-1).split(nbs)))


def _plain_adamw(s):
    case, sizes = s["case"], s["sizes"]
    eight = case["bits"] == 8
    g = s["grad"].float()
    if case["clip"]:
        norm = torch.sqrt((s["grad"].double() ** 2).sum())
        s["norm"] = torch.stack((norm, torch.clamp(MAX_NORM / norm, max=1.0))).float()
        g = g * s["norm"][1]
    p = s["master"] if case["master"] else s["param"].float()
    m, v = (_unblocks(t, sizes) for t in _load_moments(s)) if eight else (s["m"], s["v"])
    f32 = lambda x: torch.tensor(x, dtype=torch.float32, device=g.device)  # noqa: E731
    m = m * f32(BETA1) + g * f32(1.0 - BETA1)
    v = v * f32(BETA2) + (g * g) * f32(1.0 - BETA2)
    lr = f32(LR)
    size = lr * f32(1.0 / (1.0 - BETA1 ** s["step"]))
    below = torch.sqrt(v) * f32(1.0 / math.sqrt(1.0 - BETA2 ** s["step"])) + f32(EPS)
    p = p * (1.0 - lr * s["decay"]) - size * (m / below)
    if case["master"]:
        s["master"] = p
    s["param"] = p.to(s["param"].dtype)
    if eight:
        _store_moments(s, _blocks(m, sizes), _blocks(v, sizes), _noise(sizes, s["step"], g.device))
        s["m_out"], s["v_out"] = (_unblocks(t, sizes).to(torch.bfloat16) for t in _load_moments(s))
    else:
        s["m"], s["v"] = m, v
    s["step"] += 1
    return _adamw_outputs(s)


def _run_plain(s):
    case = s["case"]
    if case["op"] == "adamw":
        return _plain_adamw(s)
    fmt, dtype = case["fmt"], DTYPES[case["dtype"]]
    if case["op"] == "pack":
        through = lambda x: _plain_values(*_plain_pack(x, fmt, case["tile"]), fmt, case["tile"], x.shape[1])  # noqa: E731
        most = 65504.0 if dtype == torch.float16 else math.inf
        out = ([through(s["x"])] if case["ways"] != "cols" else []) + ([through(s["x"].t())] if case["ways"] != "rows" else [])
        return [y.clamp(-most, most).to(dtype) for y in out]
    if case["part"] == "weight_grad":
        dy_t = _plain_values(*_plain_pack(s["dy"].t(), fmt, False), fmt, False, case["tokens"])
        s["dw"] = s["dw"] + dy_t @ _from_buffer(s["x_t"], case["in"], case["tokens"], "e4m3", False).t()
        return s["dw"]
    k, n = s["x"].shape[1], s["y"].shape[1]
    y = _plain_values(*_plain_pack(s["x"], fmt, False), fmt, False, k) @ _from_buffer(s["w"], n, k, "e4m3", True).t()
    return (y if s["bias"] is None else y + s["bias"]).to(dtype)


def work(case):
    if case["op"] == "adamw":
        n = sum(_sizes(case))
        state = 8 if case["bits"] == 32 else 2 + 2 / BLOCK
        p, g = SIZE[case["param"]], SIZE[case["grad"]]
        # the parameters (read only where there is no master copy) and moments in and out, the gradient in
        step = (8 + p if case["master"] else 2 * p) + g + 2 * state
        shown = 4 if case["bits"] == 8 else 0  # the moments' values in bf16
        return {"bytes": n * (step + shown), "flops": n * (16 + (2 if case["clip"] else 0))}
    size = SIZE[case["dtype"]]
    if case["op"] == "pack":
        rows, cols = case["rows"], case["cols"]
        kept = sum(er * ((c + BLOCK - 1) // BLOCK) + r * c for way, r, c in (("rows", rows, cols), ("cols", cols, rows))
                   if case["ways"] in (way, "both") for er in [(r + BLOCK - 1) // BLOCK if case["tile"] else r])
        ways = 2 if case["ways"] == "both" else 1
        return {"bytes": rows * cols * size * (1 + ways) + kept, "flops": 4 * ways * rows * cols}
    t, k, n = case["tokens"], case["in"], case["out"]
    flops = 2 * t * k * n
    blocks = lambda c: (c + BLOCK - 1) // BLOCK  # noqa: E731
    if case["part"] == "weight_grad":
        # the gradient, the packed input, the sums in and out
        return {"bytes": t * n * size + k * (t + blocks(t)) + 8 * n * k, "flops": flops}
    c, r = (k, n) if case["part"] == "forward" else (n, k)
    return {"bytes": t * c * size + r * c + blocks(r) * blocks(c) + t * r * size
            + (4 * n if case["bias"] else 0), "flops": flops}


# ----------------------------------------------------------------------------------------------------
# The definitions in 64 bits.
# ----------------------------------------------------------------------------------------------------
def _two(e):
    """2^e in 64 bits, from its bits: pow may be off by a rounding, which moves ties."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_float(x, top, mantissa, lowest, dims):
    """x through 8-bit floating point with `mantissa` bits, in blocks that span `dims`: the nearest multiples (ties to
    even) of each value's step, under the smallest power of two with which the block's largest value passes no code."""
    frac, exp = torch.frexp(x.abs().amax(dims, keepdim=True))      # frac in [1/2, 1)
    e = (exp - 1 - top + (frac > 0.875).to(exp.dtype)).clamp(10 - 127, 127 - top + 1)
    scale = _two(e)
    u = x / scale
    step = _two((torch.frexp(u)[1] - 1).clamp(min=lowest) - mantissa)
    return torch.round(u / step) * step * scale


def _exact_packed(x, fmt, tile):
    rows, cols = x.shape
    up = BLOCK if tile else 1
    full = torch.zeros((rows + up - 1) // up * up, (cols + BLOCK - 1) // BLOCK * BLOCK, dtype=torch.float64, device=x.device)
    full[:rows, :cols] = x
    v = full.reshape(full.shape[0] // up, up, full.shape[1] // BLOCK, BLOCK)
    v = _exact_float(v, 8, 3, -6, (1, 3)) if fmt == "e4m3" else _exact_float(v, 15, 2, -14, (1, 3))
    return v.reshape(full.shape)[:rows, :cols]


def _exact_decoded(buf, rows, cols, tile):
    """The values that a packed e4m3 buffer holds."""
    sign_and_size = []
    for c in range(256):
        e, f = c >> 3 & 15, c & 7
        v = math.nan if c & 127 == 127 else f * 2.0 ** -9 if e == 0 else (8 + f) * 2.0 ** (e - 10)
        sign_and_size.append(-v if c & 128 else v)
    table = torch.tensor(sign_and_size, dtype=torch.float64, device=buf.device)
    cp, ep = (cols + 127) // 128 * 128, (cols + 511) // 512 * 4
    er = (rows + 127) // 128 if tile else rows
    at = (rows * cp + 15) // 16 * 16
    codes = buf[:rows * cp].reshape(rows, cp)[:, :cols].long()
    exps = buf[at:at + er * ep].reshape(er, ep).long() - 127
    exps = torch.repeat_interleave(torch.repeat_interleave(exps, 128, 1)[:, :cols], 128 if tile else 1, 0)[:rows]
    return table[codes] * _two(exps)


def _exact_noise(sizes, step, dev):
    """Each element's 16 random bits as a fraction of 1, tensors one after another: Philox4x32-10 by limbs of 16 bits."""
    def wide(a, b):
        """High and low words of the product of 32-bit a (tensor) and b (number)."""
        a1, a0, b1, b0 = a >> 16, a & 0xFFFF, b >> 16, b & 0xFFFF
        mid = a1 * b0 + (a0 * b0 >> 16)
        mid2 = (mid & 0xFFFF) + a0 * b1
        return a1 * b1 + (mid >> 16) + (mid2 >> 16), (mid2 & 0xFFFF) << 16 | (a0 * b0 & 0xFFFF)

    out = []
    for t, n in enumerate(sizes):
        i = torch.arange((n + 7) // 8, device=dev)
        a, b, c, d = i % 2 ** 32, i // 2 ** 32, torch.full_like(i, step), torch.full_like(i, t + 2 ** 31)
        k0, k1 = SEED % 2 ** 32, SEED // 2 ** 32
        for _ in range(10):
            h0, l0 = wide(a, 0xD2511F53)
            h1, l1 = wide(c, 0xCD9E8D57)
            a, b, c, d = h1 ^ b ^ k0, l1, h0 ^ d ^ k1, l0
            k0, k1 = (k0 + 0x9E3779B9) % 2 ** 32, (k1 + 0xBB67AE85) % 2 ** 32
        halves = [h for w in (a, b, c, d) for h in (w % 65536, w // 65536)]
        out.append(torch.stack(halves, 1).reshape(-1)[:n].double() / 65536)
    return torch.cat(out)


def _exact_adamw(case, s):
    g = s["grad"].double()
    out = {}
    if case["clip"]:
        norm = torch.linalg.vector_norm(g)
        scale = min(1.0, MAX_NORM / float(norm))
        out["norm"] = torch.stack((norm, torch.full_like(norm, scale)))
        g = g * scale
    sizes = s["sizes"]
    if case["bits"] == 8:
        ms, vs, at = [], [], 0
        for n in sizes:
            nb = (n + 127) // 128
            cm, cv = s["m8"][at:at + nb * 128].long(), s["v8"][at:at + nb * 128].long()
            em, ev = (torch.repeat_interleave(s[k][at + nb * 128:at + nb * 129].long() - 127, 128) for k in ("m8", "v8"))
            e, f = cm // 8 % 16, cm % 8
            size = torch.where(e == 0, f * 2.0 ** -9, (8 + f) * _two(e - 10))
            ms.append((torch.where(cm > 127, -size, size) * _two(em))[:n])
            vs.append(torch.where(cv == 0, 0.0, (8 + cv % 8) * _two(cv // 8 - 34 + ev))[:n])
            at += nb * 128 + (nb + 15) // 16 * 16
        m, v = torch.cat(ms), torch.cat(vs)
    else:
        m, v = s["m"].double(), s["v"].double()
    m = BETA1 * m + (1 - BETA1) * g
    v = BETA2 * v + (1 - BETA2) * g ** 2
    p = s["master"].double() if case["master"] else s["param"].double()
    decay = torch.repeat_interleave(torch.tensor([DECAY if n > 4096 else 0.0 for n in sizes], dtype=torch.float64,
                                                 device=g.device), torch.tensor(sizes, device=g.device))
    t = s["step"]
    p = p - LR * (decay * p + m / (1 - BETA1 ** t) / (torch.sqrt(v / (1 - BETA2 ** t)) + EPS))
    out["param"] = p
    if case["master"]:
        out["master"] = p
    if case["bits"] == 8:
        noise = _exact_noise(sizes, t, g.device)
        ms, vs = [], []
        for mt, vt, ut in zip(m.split(sizes), v.split(sizes), noise.split(sizes)):
            pad = (0, -mt.numel() % 128)
            rows = torch.nn.functional.pad(mt, pad).view(-1, 128)
            ms.append(_exact_float(rows, 8, 3, -6, 1).reshape(-1)[:mt.numel()])
            # the second moment: steps of an eighth of each value's power of two, up with the remainder's probability;
            # 32 powers of two below the block's largest, and nothing between the lowest and 0
            rows, u = torch.nn.functional.pad(vt, pad).view(-1, 128), torch.nn.functional.pad(ut, pad).view(-1, 128)
            frac, exp = torch.frexp(rows.amax(1, keepdim=True))
            low = (exp - 1 + (frac > 0.9375).to(exp.dtype) - 31).clamp(min=-126)
            step = _two(torch.frexp(rows)[1] - 4)
            up = torch.floor(rows / step + u) * step
            up = torch.where(rows > 0, torch.maximum(up, 1.125 * _two(low)), 0.0)
            vs.append(up.reshape(-1)[:vt.numel()])
        m, v = torch.cat(ms), torch.cat(vs)
    out["m"], out["v"] = m, v
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_adamw(case, s)
    if case["op"] == "pack":
        x = s["x"].double()
        out = ([_exact_packed(x, case["fmt"], case["tile"])] if case["ways"] != "cols" else []) + \
              ([_exact_packed(x.t(), case["fmt"], case["tile"])] if case["ways"] != "rows" else [])
        return [y.clamp(-65504, 65504) if case["dtype"] == "f16" else y for y in out]
    if case["part"] == "weight_grad":
        dy_t = _exact_packed(s["dy"].double().t(), case["fmt"], False)
        return s["dw"].double() + torch.einsum("nt,kt->nk", dy_t, _exact_decoded(s["x_t"], case["in"], case["tokens"], False))
    k, n = s["x"].shape[1], s["y"].shape[1]
    y = torch.einsum("tk,nk->tn", _exact_packed(s["x"].double(), case["fmt"], False), _exact_decoded(s["w"], n, k, True))
    return y if s["bias"] is None else y + s["bias"].double()
