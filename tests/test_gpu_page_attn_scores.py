"""Scores of attention over pages where they are easily lost: long flat tails,
caps far above the scores, tiny scales, and queries with a stride of their own."""
import numpy as np
import pytest
import torch

from paged_helpers import HostPool, attention64
from test_gpu_page_attn import FORMATS, cache, check, i32, query
from test_gpu_page_attn_rows import VECTORS, kind

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("planes", [1, 2])
@pytest.mark.parametrize("heads,batch", [(1, 456), (20, 608), (32, 152)])
def test_a_long_flat_tail_keeps_its_weight(nq, planes, heads, batch):
    """2^20 rows of one value, the first with a weight of 1 and each other with 2.45 2^-24: the output is that
    value.  Weights are rounded to fp16 at 2^3 times the largest (2^-25 2^-3 each), sums of products in fp32
    (sixteen at a time; one step of 2^-23 of the sum), the output to bf16."""
    n, D, P = 1 << 20, 64, 256
    pool = nq.PagePool(1, n // P, P, 1, D, nq.KV_NESTED44, group=64)
    m = nq.PageMap(1, n // P, n // P, P, table=torch.arange(n // P, dtype=torch.int32, device="cuda")[None].contiguous())
    k, v = torch.zeros(n, 1, D, device="cuda"), torch.ones(n, 1, D, device="cuda")
    k[0, 0, 0] = 7.0
    pool.append(0, m, k, v, torch.zeros(n, dtype=torch.int32, device="cuda"), torch.arange(n, dtype=torch.int32, device="cuda"))
    q = torch.zeros(batch, 1, heads, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1.0
    scale = np.log(2.0 ** 24 / 2.45) / 7.0
    out = pool.attention(0, m, q, i32([n] * batch), planes, scale, seqs=i32([0] * batch)).double()
    one = HostPool(pool).row(0, 0, 0, 0, 1, planes)[0]
    tail = (n - 1) * 2.45 * 2.0 ** -24
    tol = 2.0 ** -8 + n * 2.0 ** -28 / (1 + tail) + n / 16 * 2.0 ** -23
    assert float((out - one).abs().max()) <= tol * one, float((out - one).abs().max())
    assert nq.device_status() == 0


@pytest.mark.parametrize("fmt,planes", FORMATS)
@pytest.mark.parametrize("g,M", VECTORS)
@pytest.mark.parametrize("cap", [2.0 ** 14, 2.0 ** 20, 2.0 ** 60, 2.0 ** 100])
def test_a_cap_far_above_the_scores_changes_none(nq, fmt, planes, g, M, cap):
    """cap tanh(x / cap) = x (1 - x^2 / (3 cap^2) ..): below 2^-18 of a score of 100.  The tolerance is that of no cap."""
    lens = [6, 40, 300, 17]
    pool, m = cache(nq, lens, 2, 64, 64, 16, kind(nq, fmt), 380)
    q = query(381, len(lens), M, 2 * g, 64)
    ref, tol = attention64(HostPool(pool), 0, m.table.cpu().numpy(), q.float().cpu().numpy(), lens, planes, 0.3)
    out = pool.attention(0, m, q, i32(lens), planes, 0.3, softcap=cap).double().cpu().numpy()
    assert (np.abs(out - ref) <= tol).all()
    assert nq.device_status() == 0


@pytest.mark.parametrize("fmt,planes", FORMATS)
@pytest.mark.parametrize("cap", [2.0 ** -100, 1e-3, 1.0, 5.0])
def test_a_cap_far_below_the_scores(nq, fmt, planes, cap):
    lens = [6, 40, 300, 17]
    pool, m = cache(nq, lens, 2, 64, 64, 16, kind(nq, fmt), 382)
    for g, M in VECTORS:
        check(nq, pool, m, lens, query(383, len(lens), M, 2 * g, 64), planes, 0.3, softcap=cap)


@pytest.mark.parametrize("fmt,planes", FORMATS)
@pytest.mark.parametrize("fill", [0x7BFF, 0x7F00, 0x7C00])
@pytest.mark.parametrize("g,M", VECTORS)
def test_a_far_cap_beside_huge_hidden_scores(nq, fmt, planes, fill, g, M):
    """Rows past the end hold the largest scale, or values of 10^38: they do not touch the scores beside them."""
    lens = [6, 41, 300, 17, 1]
    pool, m = cache(nq, lens, 2, 64, 64, 16, kind(nq, fmt), 390, fill=fill)
    q = query(391, len(lens), M, 2 * g, 64)
    for window in (0, 11):
        ref, tol = attention64(HostPool(pool), 0, m.table.cpu().numpy(), q.float().cpu().numpy(), lens, planes, 0.3, window=window)
        out = pool.attention(0, m, q, i32(lens), planes, 0.3, softcap=2.0 ** 60, window=window).double().cpu().numpy()
        assert (np.abs(out - ref) <= tol).all()


@pytest.mark.parametrize("fmt,planes", FORMATS)
@pytest.mark.parametrize("g,M", VECTORS + [(3, 1)])
def test_queries_with_a_stride_of_their_own(nq, fmt, planes, g, M):
    """The heads of a wider row, read where they lie."""
    lens = [6, 40, 300, 17]
    pool, m = cache(nq, lens, 2, 64, 64, 16, kind(nq, fmt), 384)
    wide = query(385, len(lens), M, 2 * g + 3, 64)
    q = wide[:, :, 1:1 + 2 * g]
    want = check(nq, pool, m, lens, q.contiguous(), planes, 0.3)
    got = pool.attention(0, m, q, i32(lens), planes, 0.3)
    assert got.is_contiguous() and torch.equal(got, want)
    bad = [wide[:, :, ::2][:, :, :2], wide.float()[:, :, :2 * g]]
    if M > 1:
        bad += [query(386, len(lens), M + 1, 2 * g, 64)[:, 1:], wide[:, :, :2 * g].transpose(0, 1)]
    for x in bad:
        with pytest.raises(ValueError):
            pool.attention(0, m, x, i32([1] * x.shape[0]), planes, 0.3)


@pytest.mark.parametrize("fmt,planes", FORMATS)
@pytest.mark.parametrize("scale", [1e-18, 1e-30, 1e-38])
def test_tiny_scales_and_queries_of_zero(nq, fmt, planes, scale):
    """All scores equal: the mean of the rows that are seen."""
    lens = [6, 40, 300, 17]
    pool, m = cache(nq, lens, 2, 64, 64, 16, kind(nq, fmt), 387)
    for g, M in VECTORS:
        q = query(388, len(lens), M, 2 * g, 64)
        q[:, :, ::2] = 0
        check(nq, pool, m, lens, q, planes, scale)
