"""The products' float32 sums over many columns: what the tensor cores cut off ends with a run of 4096 of them."""
import pytest
import torch

pytestmark = pytest.mark.gpu

import gradient_quantization_communication_b200.gq as G


def packed(x):
    buf = torch.empty(G.gq_fp8_layout(*x.shape)[0], dtype=torch.uint8, device="cuda")
    G.gq_fp8_pack(x, buf)
    return buf


# One product of 2^26 among ones.  A sum of 2^26 cuts off what lies below 2^-25 of it, so that every 1 that a run adds to the
# large product is lost; every other run's sum of ones is exact, and adding it to the whole rounds by half a step of 2^26 ..
# 2^27, 4, at most.  So a result is at most 4096 + 4 (k / 4096 + 8 parts) too small, where one run of all columns would lose
# nearly k.
@pytest.mark.parametrize("m,n,k", [
    (256, 600, 16384), (300, 512, 32768), (2048, 4096, 16384), (1500, 3000, 20001),       # CTA pairs: cut tiles, whole ones
    (1, 19200, 16384), (16, 19200, 16384), (48, 19200, 16384), (100, 9728, 16384),        # single CTAs, each a whole tile
    (16, 4096, 32768)])                                                                  # clusters
@pytest.mark.parametrize("place", [0.0, 0.3, 0.6, 1.0])
def test_a_large_product_among_ones(m, n, k, place):
    at = int(place * (k - 1))
    x, w = (torch.ones(r, k, dtype=torch.bfloat16, device="cuda") for r in (m, n))
    x[:, at] = w[:, at] = 8192.0
    y = torch.empty(m, n, device="cuda")
    G.gq_fp8_matmul(packed(x), packed(w), k, y)
    short = 2.0 ** 26 + k - 1 - y.double()
    assert float(short.abs().max()) <= 4096 + 4 * (k / 4096 + 8), float(short.abs().max())
