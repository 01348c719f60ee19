"""The norm's codes are clamp(rint(y / z)) of the quotient that IEEE division gives, as nq_quantize_act_int8 takes it.

A row of one value c = 2^-e, e >= 13, under eps = 1 has mean(s^2) + eps = 1 (c^2 <= 2^-26 is less than half a step of
2^-23), of which the root and its inverse are 1: y = c w is one product, known on the host to the bit."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,M", [(4096, 300), (4096, 1200), (520, 40), (16384, 64)])      # both thread layouts
@pytest.mark.parametrize("seed", range(4))
def test_codes_to_the_bit(nq, K, M, seed):
    r = np.random.default_rng(seed)
    # quotients near k + 1/2, of a largest value with any mantissa; a quarter anywhere
    top = np.float32(r.uniform(1, 2))
    z = top / np.float32(127)
    k = r.integers(0, 127, K)
    w = ((k + np.float32(0.5)) * z).astype(np.float32)
    w = (w.view(np.int32) + r.integers(-4, 5, K).astype(np.int32)).view(np.float32)
    w[::4] = r.uniform(0, 1, len(w[::4])).astype(np.float32) * top
    w = np.minimum(w, top) * r.choice(np.float32([-1, 1]), K)
    w[r.integers(0, K)] = top
    scale = np.float32(2.0 ** r.integers(-100, 100))     # largest values over fp32's range, z near 1e-30 and below 2^-126 among them
    w *= scale
    e = r.integers(13, 50, M)
    e[:38] = np.arange(13, 51)
    x = np.broadcast_to(np.float32(2.0) ** -e.astype(np.float32)[:, None], (M, K)).copy()
    y = x * w                                             # fp32, one rounding
    zr = np.abs(y).max(1) / np.float32(127)
    with np.errstate(all="ignore"):
        want = np.where(zr[:, None] > 0, np.clip(np.rint(y / zr[:, None]), -127, 127), 0)
    assert y.dtype == zr.dtype == np.float32
    _, xq, sx = nq.rms_norm(torch.from_numpy(x).cuda(), torch.from_numpy(w).cuda(), eps=1.0, quantize=True)
    assert nq.device_status() == 0
    assert np.array_equal(sx.cpu().numpy(), zr)
    assert np.array_equal(xq.cpu().numpy(), want)
