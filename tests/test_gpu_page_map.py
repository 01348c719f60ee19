"""Calls on a page map and a pool at their edges: a slot named twice, requests
whose total passes 32 bits, empty lists, a pool made on a stream."""
import random

import pytest
import torch

from paged_helpers import HostMap
from test_gpu_pages import i32, same

pytestmark = pytest.mark.gpu


def test_requests_past_32_bits_of_pages(nq):
    """Seventeen requests of 2^27 - 1 pages: more than 2^31 in all.  None is served, nothing changes."""
    S, W, N, P = 18, (1 << 27) - 1, 50, 16
    m = nq.PageMap(S, W, N, P)
    seqs, zero = i32(list(range(S))), i32([0] * S)
    assert m.reserve(None, i32([17]), i32([0]), i32([40])).tolist() == [1]
    for n in (17, 18):
        got = m.reserve(None, seqs[:n].contiguous(), zero[:n].contiguous(), i32([W * P] * n))
        assert got.tolist() == [0] * n and nq.device_status() == nq.NQ_DEV_POOL_FULL
        assert m.held.tolist() == [0] * 17 + [3] and m.ref.tolist() == [1] * 3 + [0] * 47
        assert (m.table[:17, :100] == -1).all() and m.table[17, :4].tolist() == [0, 1, 2, -1]
    # what fits before the first that does not is served
    got = m.reserve(None, seqs[:17].contiguous(), zero[:17].contiguous(), i32([30] + [W * P] * 16))
    assert got.tolist() == [1] + [0] * 16 and m.table[0, :3].tolist() == [3, 4, -1]
    assert nq.device_status() == nq.NQ_DEV_POOL_FULL


def test_truncate_names_a_slot_twice(nq):
    """Each page is released once, and the least of the rows stays."""
    S, W, P = 40, 30, 16
    N = S * W
    r = random.Random(5)
    for step in range(12):
        m, h = nq.PageMap(S, W, N, P), HostMap(S, W, N, P)
        seqs = list(range(S // 2))
        last = [r.randint(1, W * P) for _ in seqs]
        m.reserve(None, i32(seqs), i32([0] * len(seqs)), i32(last))
        h.reserve(seqs, [0] * len(seqs), last)
        src, rows = [r.choice(seqs) for _ in seqs], [r.randint(0, W * P) for _ in seqs]
        rows = [min(x, last[s]) for x, s in zip(rows, src)]
        m.fork(i32(src), i32([s + S // 2 for s in seqs]), i32(rows))
        h.fork(src, [s + S // 2 for s in seqs], rows)
        same(m, h)
        names = [r.choice([0, 1, 5, 20, 21, r.randrange(S)]) for _ in range(S)]
        keep = [r.randint(0, W * P) for _ in names]
        m.truncate(i32(names), i32(keep))
        h.truncate(names, keep)
        same(m, h)
        assert nq.device_status() == 0


def test_a_pool_made_on_a_stream(nq):
    """Its clearing is ordered before what that stream appends, not by the current stream."""
    s = torch.cuda.Stream()
    seqs, pos = i32([0] * 16), torch.arange(16, dtype=torch.int32, device="cuda")
    x = torch.ones(16, 1, 64, device="cuda")
    m = nq.PageMap(1, 1, 1000, 16, table=i32([[999]]))
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)                       # the current stream is busy for some milliseconds
    pool = nq.PagePool(1, 1000, 16, 1, 64, nq.KV_BF16, stream=s)
    pool.append(0, m, x, x, seqs, pos, stream=s)
    k, v = pool.read(0, m, seqs, pos, stream=s)
    s.synchronize()
    early = (k == 1).all() and (v == 1).all()
    torch.cuda.synchronize()
    k, v = pool.read(0, m, seqs, pos)
    assert early and (k == 1).all() and (v == 1).all()
    assert (pool.data.view(torch.bfloat16) == 1).sum() == 2 * 16 * 64 and (pool.data == 0).sum() > 0


def test_empty_lists(nq):
    """No sequence, no request: nothing happens, as for rotation, append and read."""
    pool, m = nq.PagePool(1, 4, 16, 2, 64, group=64), nq.PageMap(2, 2, 4, 16)
    e = i32([])
    m.reserve(pool, i32([1]), i32([0]), i32([20]))
    table, held, ref = m.table.clone(), m.held.clone(), m.ref.clone()
    assert m.reserve(pool, e, e, e).shape == (0,)
    m.fork(e, e, e)
    m.truncate(e, e)
    pool.copy_pages(e, e)
    q = torch.empty(0, 3, 4, 64, dtype=torch.bfloat16, device="cuda")
    assert pool.attention(0, m, q, e, 2, 0.1).shape == (0, 3, 4, 64)
    assert pool.attention(0, m, q, e, 2, 0.1, seqs=e).shape == (0, 3, 4, 64)
    assert torch.equal(m.table, table) and torch.equal(m.held, held) and torch.equal(m.ref, ref)
    assert nq.device_status() == 0
    one = i32([1])
    for bad in (lambda: m.reserve(pool, e, one, e), lambda: m.fork(e, e, one), lambda: m.truncate(e, one),
                lambda: pool.copy_pages(e, one), lambda: pool.attention(0, m, q, one, 2, 0.1),
                lambda: pool.attention(0, m, q.float(), e, 2, 0.1)):
        with pytest.raises(ValueError):
            bad()
