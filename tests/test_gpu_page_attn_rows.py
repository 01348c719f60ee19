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
