"""Which rows attention over pages counts: pages that a window has left behind,
windows longer than any sequence, pages that are not there, rows that were not
finite.  The reference is attention64 (64 bits, its tolerance derived there)."""
import pytest
import torch

from test_gpu_page_attn import FORMATS, cache, check, i32, query

pytestmark = pytest.mark.gpu

# query vectors per kv head on every kernel: one tile of 8 per warp, two, a CTA's shared decoding, tensor cores
# (bf16: 64 columns per CTA)
VECTORS = [(2, 1), (4, 3), (4, 5), (8, 5)]


def kind(nq, fmt):
    return nq.KV_BF16 if fmt == "bf16" else nq.KV_NESTED44


@pytest.mark.parametrize("fmt,planes", FORMATS)
@pytest.mark.parametrize("g,M", VECTORS)
@pytest.mark.parametrize("D,G,P", [(64, 64, 16), (128, 128, 32), (128, 64, 16)])
def test_a_window_leaves_any_page_behind(nq, fmt, planes, g, M, D, G, P):
    """The first row that is seen lies at every eighth row of 128; every page before its own is released."""
    window, lens = 100, [300 + 8 * i for i in range(16)]
    pool, m = cache(nq, lens, 1, D, G, P, kind(nq, fmt), 300 + g)
    q = query(301 + M, len(lens), M, g, D)
    want = check(nq, pool, m, lens, q, planes, D ** -0.5, window=window)
    for b, n in enumerate(lens):
        m.table[b, :(n - M - window + 1) // P] = -1
    got = pool.attention(0, m, q, i32(lens), planes, D ** -0.5, window=window)
    assert nq.device_status() == 0
    assert torch.equal(got, want)


@pytest.mark.parametrize("fmt,planes", FORMATS)
@pytest.mark.parametrize("g", [1, 2, 6])
def test_the_longest_windows_hide_nothing(nq, fmt, planes, g):
    """More query rows than rows, under windows up to the largest int32: the same as without one."""
    lens, M = [3, 1, 8, 40, 0], 9
    pool, m = cache(nq, lens, 2, 64, 64, 16, kind(nq, fmt), 320)
    q = query(321, len(lens), M, 2 * g, 64)
    want = check(nq, pool, m, lens, q, planes, 0.125)
    for window in (2 ** 31 - 1, 2 ** 31 - 4, 2 ** 31 - 9, 2 ** 30, 48):
        assert torch.equal(check(nq, pool, m, lens, q, planes, 0.125, window=window), want)
