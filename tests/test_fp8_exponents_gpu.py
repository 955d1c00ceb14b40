"""Packed forms that gq_fp8_pack did not write: every code under every exponent byte, unpacked and multiplied, has the value
that the layout gives it."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

import fp8_oracle as O
import gradient_quantization_communication_b200.gq as G


def every(tile):
    """codes (rows, 256) and exponents of all pairs: row r's blocks hold the codes 0 .. 255 under exponent r (or r / 128)."""
    rows = 256 * 128 if tile else 256
    codes = np.zeros((rows, 256), np.uint8)
    codes[:] = np.arange(256)
    exps = np.zeros((256, 4), np.uint8)
    exps[:, 0] = exps[:, 1] = np.arange(256)
    return codes, exps


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("tile", [False, True])
def test_unpack_every_pair(dtype, fmt, tile):
    codes, exps = every(tile)
    want = O.decode(codes, exps, fmt, tile, 256)
    # binary32 first: values beyond its largest are infinite there, and saturate in float16
    w = want.float()
    w = w.clamp(-65504, 65504).to(dtype) if dtype == torch.float16 else w.to(dtype)
    buf = torch.from_numpy(O.to_buffer(codes, exps)).cuda()
    for pad in (0, 3):
        x = torch.full((codes.shape[0], 256 + pad), 5.0, dtype=dtype, device="cuda")
        G.gq_fp8_unpack(buf, x[:, :256], fmt=fmt, tile=tile)
        got = x[:, :256].cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(w))
        assert torch.equal(torch.nan_to_num(got, 7.0, float("inf"), -float("inf")), torch.nan_to_num(w, 7.0, float("inf"), -float("inf")))


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("m", [16, 256])
def test_product_under_every_exponent(fmt, m):
    """Codes under exponent E times ones under 254 - E are the codes' values; under 255 they are NaN."""
    table = O.values(fmt)
    for E in (0, 1, 5, 9, 10, 126, 127, 200, 244, 247, 250, 253, 254, 255):
        a = np.zeros((m, 128), np.uint8)
        a[:, 3] = np.arange(m) * (256 // m) + 1
        ea = np.zeros((m, 4), np.uint8)
        ea[:, 0] = E
        b = np.zeros((5, 128), np.uint8)
        b[:, 3] = 0x38                                    # 1 in e4m3
        eb = np.zeros((5, 4), np.uint8)
        eb[:, 0] = max(254 - E, 0)
        y = torch.empty(m, 5, device="cuda")
        G.gq_fp8_matmul(torch.from_numpy(O.to_buffer(a, ea)).cuda(), torch.from_numpy(O.to_buffer(b, eb)).cuda(), 128, y,
                        fmt=(fmt, "e4m3"))
        got = y.double().cpu().numpy()
        want = np.repeat(table[a[:, 3]][:, None], 5, 1)
        if E == 255:
            want[:] = np.nan
        assert np.array_equal(np.isnan(got), np.isnan(want)), E
        assert np.array_equal(np.nan_to_num(got, nan=7.0), np.nan_to_num(want, nan=7.0)), E


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("tile", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("rows,cols", [(5, 130), (200, 300), (129, 257)])
def test_padding_of_a_block_without_a_value(fmt, tile, bad, rows, cols):
    """All 128 codes of a block with E = 255 are 0x7f, its padding behind the matrix among them; other padding is 0."""
    x = torch.randn(rows, cols, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    x[rows - 1, cols - 1] = bad
    for src, buf_of in ((x, lambda p, t: p), (x.t(), lambda p, t: t)):
        r, c = src.shape
        p, t = (torch.full((G.gq_fp8_layout(*s, tile)[0],), 0xEE, dtype=torch.uint8, device="cuda") for s in ((rows, cols), (cols, rows)))
        G.gq_fp8_pack(x, p, t, fmt=fmt, tile=tile)
        got = buf_of(p, t).cpu().numpy()
        pitch = O.pitches(c)[0]
        codes = got[:r * pitch].reshape(r, pitch)
        last = c // 128 * 128                             # the cut block
        hit = np.zeros(r, bool)
        hit[(r - 1) // 128 * 128 if tile else r - 1:] = True
        assert (codes[hit, last:] == 0x7F).all() and (codes[~hit, c:] == 0).all()
        want, exps = O.pack(src.cpu(), fmt, tile)
        assert np.array_equal(codes, want)
        off = O.layout(tile, r, c)[1]
        assert np.array_equal(got[off:off + exps.size].reshape(exps.shape), exps)
