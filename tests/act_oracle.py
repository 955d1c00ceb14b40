"""The 8-bit activation checkpoint and the operators that read it, in 64 bits on the CPU: what the
kernels of gq_act_* and gq_layer_norm_* are held to.  Independent of the package."""
import math

import numpy as np
import torch

HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def pitches(cols):
    return -(-cols // 32) * 32, -(-cols // 128) * 4


def layout(rows, cols):
    cp, ep = pitches(cols)
    off = -(-rows * cp // 16) * 16
    return off + -(-rows * ep // 16) * 16, off


def encode(x):
    """(codes int8 (rows, code pitch), exponents uint8 (rows, exponent pitch)) of a CPU tensor."""
    rows, cols = x.shape
    cp, ep = pitches(cols)
    v = np.zeros((rows, cp), np.float64)
    v[:, :cols] = x.double().numpy()
    v = v.reshape(rows, cp // 32, 32)
    bad = ~np.isfinite(v).all(2)
    m = np.abs(np.where(np.isfinite(v), v, 0.0)).max(2)
    # smallest E with every |rint(x * 2^(133 - E))| <= 127, tried one by one from frexp's exponent
    _, p = np.frexp(m)
    E = np.where(m > 0, np.clip(p.astype(np.int64) - 9 + 133, 0, 254), 0)
    for _ in range(4):
        E = np.where((np.rint(np.ldexp(m, 133 - E)) > 127) & (E < 254), E + 1, E)
    q = np.clip(np.rint(np.ldexp(v, (133 - E)[:, :, None])), -127, 127)
    q = np.where(bad[:, :, None], 0, q)
    E = np.where(bad, 255, E)
    exps = np.zeros((rows, ep), np.uint8)
    exps[:, :cp // 32] = E
    return q.reshape(rows, cp).astype(np.int8), exps


def to_buffer(codes, exps):
    rows, cp = codes.shape
    ep = exps.shape[1]
    off = -(-rows * cp // 16) * 16
    buf = np.zeros(off + -(-rows * ep // 16) * 16, np.uint8)
    buf[:rows * cp] = codes.view(np.uint8).reshape(-1)
    buf[off:off + rows * ep] = exps.reshape(-1)
    return buf


def decode(codes, exps, cols):
    """float64 values (rows, cols)."""
    rows, cp = codes.shape
    E = exps[:, :cp // 32].astype(np.int64)
    v = np.ldexp(codes.reshape(rows, cp // 32, 32).astype(np.float64), (E - 133)[:, :, None])
    v = np.where((E == 255)[:, :, None], np.nan, v)
    return torch.from_numpy(v.reshape(rows, cp)[:, :cols].copy())


def as_type(v, dtype):
    """float64 values rounded to dtype (fp16: saturated), as gq_act_unpack gives them."""
    if dtype == torch.float16:
        v = v.clamp(-65504.0, 65504.0)
    return v.to(dtype)


def fn(kind, x):
    """(f, f', size of the exponentials' argument) at float64 x."""
    if kind == "silu":
        s = torch.sigmoid(x)
        return x * s, s * (1 + x * torch.sigmoid(-x)), x.abs()
    if kind == "gelu_tanh":
        a = math.sqrt(2 / math.pi)
        u = a * (x + 0.044715 * x ** 3)
        s = torch.sigmoid(2 * u)
        return x * s, s + 2 * x * s * torch.sigmoid(-2 * u) * a * (1 + 3 * 0.044715 * x ** 2), 2 * u.abs()
    phi = torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    Phi = 0.5 * torch.erfc(-x / math.sqrt(2))
    return x * Phi, Phi + x * phi, x * x


def norm(x, gamma, beta, eps):
    mean = x.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + eps)
    return (x - mean) * rstd * gamma + beta, mean, rstd


def norm_backward(dy, x, gamma, mean, rstd):
    xh = (x - mean) * rstd
    g = dy * gamma
    dx = rstd * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)
