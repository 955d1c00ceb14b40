"""Matrices in 8-bit floating point, and AdamW with moments in 8 bits, on the CPU: what the kernels of gq_fp8_* and
gq_adamw_* are held to.  Independent of the package."""
import math

import numpy as np
import torch

HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TOP = {"e4m3": 8, "e5m2": 15}


def values(fmt):
    """The 256 codes' values."""
    man = 3 if fmt == "e4m3" else 2
    bias = 7 if fmt == "e4m3" else 15
    out = []
    for c in range(256):
        e, f = (c & 127) >> man, c & ((1 << man) - 1)
        if fmt == "e4m3" and c & 127 == 127:
            v = math.nan
        elif fmt == "e5m2" and e == 31:
            v = math.inf if f == 0 else math.nan
        else:
            v = f * 2.0 ** (1 - bias - man) if e == 0 else ((1 << man) + f) * 2.0 ** (e - bias - man)
        out.append(-v if c & 128 else v)
    return np.array(out)


def nearest(x, fmt):
    """Codes of the values nearest to x (within the largest code), ties to the even code."""
    table = values(fmt)[:128]
    table = table[np.isfinite(table)]
    a = np.abs(x)
    hi = np.clip(np.searchsorted(table, a), 0, len(table) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - table[lo], table[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return (code | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def exponent(m, fmt):
    """The smallest E, at least 10, with m <= 1.75 * 2^TOP * 2^(E - 127); 255 where m is not finite."""
    E = np.full(m.shape, 10)
    fine = np.where(np.isfinite(m), m, 0.0)
    for e in range(10, 255):
        E = np.where(fine > math.ldexp(1.75, TOP[fmt] + e - 127), e + 1, E)
    return np.where(np.isfinite(m), E, 255)


def pitches(cols):
    return -(-cols // 128) * 128, -(-cols // 512) * 4


def layout(tile, rows, cols):
    cp, ep = pitches(cols)
    er = -(-rows // 128) if tile else rows
    off = -(-rows * cp // 16) * 16
    return off + -(-er * ep // 16) * 16, off


def pack(x, fmt, tile):
    """(codes (rows, code pitch), exponents (exponent rows, exponent pitch)) of a CPU tensor."""
    rows, cols = x.shape
    cp, ep = pitches(cols)
    up = 128 if tile else 1
    er = -(-rows // up)
    v = np.zeros((er * up, cp))
    v[:rows, :cols] = x.double().numpy()
    v = v.reshape(er, up, cp // 128, 128)
    E = exponent(np.abs(v).max((1, 3)), fmt)     # max passes NaN on
    bad = (E == 255)[:, None, :, None]
    with np.errstate(invalid="ignore"):
        codes = nearest(np.where(bad, 0.0, np.ldexp(np.where(bad, 0.0, v), (127 - E)[:, None, :, None])), fmt)
    codes = np.where(bad, 0x7F, codes).reshape(er * up, cp)[:rows]
    exps = np.zeros((er, ep), np.uint8)
    exps[:, :cp // 128] = E
    return codes.astype(np.uint8), exps


def to_buffer(codes, exps):
    rows, cp = codes.shape
    off = -(-rows * cp // 16) * 16
    buf = np.zeros(off + -(-exps.size // 16) * 16, np.uint8)
    buf[:rows * cp] = codes.reshape(-1)
    buf[off:off + exps.size] = exps.reshape(-1)
    return buf


def decode(codes, exps, fmt, tile, cols):
    """float64 values (rows, cols)."""
    rows, cp = codes.shape
    E = exps[:, :cp // 128].astype(np.int64)
    E = np.repeat(E, 128, 0)[:rows] if tile else E
    with np.errstate(invalid="ignore"):
        v = np.ldexp(values(fmt)[codes].reshape(rows, cp // 128, 128), (E - 127)[:, :, None])
    v = np.where((E == 255)[:, :, None], np.nan, v)
    return torch.from_numpy(v.reshape(rows, cp)[:, :cols].copy())


# ----------------------------------------------------------------------------------------------------
# AdamW
# ----------------------------------------------------------------------------------------------------
def philox(words, key):
    """Philox4x32-10 on arrays of uint32 words."""
    c = [np.asarray(w, np.uint64) & np.uint64(0xFFFFFFFF) for w in words]
    k0, k1 = key & 0xFFFFFFFF, key >> 32
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        p0, p1 = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(p1 >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), p1 & low, (p0 >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), p0 & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c


def noise(first, n, step, number, seed):
    """The 16 random bits of elements first .. first + n - 1 of a tensor."""
    i = np.arange(first, first + n, dtype=np.uint64)
    g = i >> np.uint64(3)
    one = np.ones_like(g)
    w = np.stack(philox((g, g >> np.uint64(32), one * np.uint64(step), one * np.uint64(number + 2 ** 31)), seed))
    j = (i & np.uint64(7)).astype(np.int64)
    word = w[j // 2, np.arange(n)]
    return np.where(j % 2, word >> np.uint64(16), word & np.uint64(0xFFFF)).astype(np.int64)


def squares_encode(v, rnd):
    """Codes and exponents of v (float64 rows of 128) with random fractions rnd / 2^16."""
    top = v.max(1)
    frac, e = np.frexp(np.where(np.isfinite(top), top, 1.0))          # top = frac * 2^e, frac in [1/2, 1)
    E = np.clip(e - 1 + (frac > 1.875 / 2) + 127, 32, 254)
    E = np.where(top == 0, 32, E)
    E = np.where(np.isfinite(top), E, 255)
    fine = np.where(np.isfinite(v), v, 0.0)
    f, e = np.frexp(fine)                                             # eighths of the value's own power of two
    units = np.floor(f * 16 + rnd / 65536.0)                          # 8 .. 16
    carry = units == 16
    units, e = np.where(carry, 8, units), e + carry
    code = (e - 1 + 127 - E[:, None] + 31) * 8 + units - 8
    code = np.where(fine > 0, np.clip(code, 1, 255), 0)
    return np.where(E[:, None] == 255, 0, code).astype(np.uint8), E


def squares_decode(codes, E):
    c = codes.astype(np.int64)
    v = np.ldexp((8 + c % 8).astype(np.float64), c // 8 - 34 + E[:, None].astype(np.int64) - 127)
    return np.where(E[:, None] == 255, np.nan, np.where(c == 0, 0.0, v))


def adam_layout(n):
    nb = -(-n // 128)
    return nb * 128 + -(-nb // 16) * 16, nb * 128


def adam_update(p, g, m, v, lr, beta1, beta2, eps, step, decay=0.0, scale=1.0, dtype=np.float64):
    """(p, m, v) after a step, each operation in dtype."""
    t = dtype
    p, g, m, v = (np.asarray(x, t) for x in (p, g, m, v))
    with np.errstate(all="ignore"):
        g = g * t(scale)
        m = m * t(beta1) + g * t(1.0 - beta1)
        v = v * t(beta2) + (g * g) * t(1.0 - beta2)
        keep = t(1.0) - t(lr) * t(decay)
        size = t(lr) * t(1.0 / (1.0 - beta1 ** step))
        below = np.sqrt(v) * t(1.0 / math.sqrt(1.0 - beta2 ** step)) + t(eps)
        p = p * keep - size * (m / below)
    return p, m, v
