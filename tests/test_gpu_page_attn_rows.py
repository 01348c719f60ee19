"""Which rows attention over pages counts: pages that a window has left behind,
windows longer than any sequence, pages that are not there, rows that were not
finite.  The reference is attention64 (64 bits, its tolerance derived there)."""
import numpy as np
import pytest
import torch

from paged_helpers import HostPool, attention64, rows_of
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


def without(hp, table, q, lens, planes, scale, gone, window=0):
    """attention64 and its tolerance over the rows that are not gone[b]."""
    B, M, Hq, D = q.shape
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    c = 2.0 ** -8 if hp.bf else 2.0 ** -11
    for b, n in enumerate(lens):
        K, V = rows_of(hp, 0, table[b], n, planes)
        for m in range(M):
            at = n - M + m
            seen = np.array([t for t in range(max(0, at - window + 1) if window else 0, at + 1) if not gone[b][t]], int)
            for h in range(Hq if len(seen) else 0):
                k, v, x = K[h * hp.H // Hq, seen], V[h * hp.H // Hq, seen], q[b, m, h].astype(np.float64)
                s = scale * (k @ x)
                e = 2.0 ** -17 * scale * (np.abs(k) @ np.abs(x)).max()
                p = np.exp(s - s.max())
                out[b, m, h] = p @ v / p.sum()
                tol[b, m, h] = (2.0 ** -8 * np.abs(out[b, m, h]) + (2 * c + 2 * e) * (p @ np.abs(v) / p.sum())
                                + len(p) * 2.0 ** -24 * np.abs(v).max() / p.sum())
    return out, tol


@pytest.mark.parametrize("fmt,planes", FORMATS)
@pytest.mark.parametrize("g,M", VECTORS)
@pytest.mark.parametrize("D,G,P,window", [(64, 64, 16, 0), (128, 128, 32, 0), (128, 64, 16, 70)])
def test_rows_of_a_page_outside_the_pool_do_not_count(nq, fmt, planes, g, M, D, G, P, window):
    """Entries that name no page: first, inner, side by side, last, all of them.  Their rows count as not there,
    and nothing of another page takes their place."""
    lens = [5 * P, 3 * P + 1, 7 * P + 5, 9, 4 * P, 6 * P - 3, 2 * P]
    broken = [[0], [1, 3], [2, 3, 4], [0], [3], [0, 1, 4], []]
    pool, m = cache(nq, lens, 2, D, G, P, kind(nq, fmt), 340)
    q = query(341, len(lens), M, 2 * g, D)
    table = m.table.cpu().numpy().copy()
    gone = [np.isin(np.arange(n) // P, broken[b]) for b, n in enumerate(lens)]
    ref, tol = without(HostPool(pool), table, q.float().cpu().numpy(), lens, planes, 0.125, gone, window)
    for bad in (-1, pool.n_pages, 2 ** 31 - 1, -2 ** 31):
        for b, js in enumerate(broken):
            for j in js:
                m.table[b, j] = bad
        out = pool.attention(0, m, q, i32(lens), planes, 0.125, window=window).double().cpu().numpy()
        assert nq.device_status() == nq.NQ_DEV_BAD_PAGE
        assert (np.abs(out - ref) <= tol).all()


@pytest.mark.parametrize("planes", [1, 2])
@pytest.mark.parametrize("g,M", VECTORS)
@pytest.mark.parametrize("D,G", [(64, 64), (128, 128), (128, 64)])
@pytest.mark.parametrize("value", [float("inf"), float("nan"), 1e30])
def test_a_row_that_was_not_finite_is_zeros_to_every_reader(nq, planes, g, M, D, G, value):
    """Appended to nested pages: its group is stored as zeros and reported, however many queries then read it."""
    lens = [70, 33]
    pool, m = cache(nq, lens, 1, D, G, 16, nq.KV_NESTED44, 360)
    rows = torch.ones(4, 1, D, device="cuda")
    bad = rows.clone()
    bad[1, 0, 5] = value
    bad[3, 0, D - 1] = -value
    seqs, pos = i32([0, 0, 1, 1]), i32([3, 40, 30, 31])
    for k, v in ((rows, bad), (bad, rows)):
        pool.append(0, m, k, v, seqs, pos)
        assert nq.device_status() == nq.NQ_DEV_NONFINITE
        got = pool.read(0, m, seqs, pos, planes=planes)
        x = got[0] if k is bad else got[1]
        assert (x[1, 0, :G] == 0).all() and (x[3, 0, D - G:] == 0).all() and (x[0] != 0).all() and (x[2] != 0).all()
        assert (x[1, 0, G:] != 0).all() and (x[3, 0, :D - G] != 0).all()
        check(nq, pool, m, lens, query(361, 2, M, g, D), planes, D ** -0.5)


@pytest.mark.parametrize("fmt,planes", FORMATS)
def test_lengths_up_to_the_largest(nq, fmt, planes):
    """2^27 - 1 pages that are all one and the same: row t is row t mod 16, wherever the window lies.  Lengths past
    2^31 - 4096 are clamped and reported."""
    W, P, D = (1 << 27) - 1, 16, 64
    pool, small = cache(nq, [P], 1, D, D, P, kind(nq, fmt), 370)
    one = int(small.table[0, 0])
    m = nq.PageMap(1, W, pool.n_pages, P, table=torch.full((1, W), one, dtype=torch.int32, device="cuda"))
    few = np.full((1, 20), one)
    most = 2 ** 31 - 4096
    for g, M in VECTORS:
        q = query(371, 1, M, g, D)
        for n in (most - 7, most - 64, most, most + 1, W * P - 9, W * P, 2 ** 31 - 1):
            at = min(n, most)
            n0 = 256 + at % 16
            ref, tol = attention64(HostPool(pool), 0, few, q.float().cpu().numpy(), [n0], planes, 0.125, window=70)
            out = pool.attention(0, m, q, i32([n]), planes, 0.125, window=70).double().cpu().numpy()
            assert nq.device_status() == (nq.NQ_DEV_SEQ_FULL if n > most else 0)
            assert (np.abs(out - ref) <= tol).all()
