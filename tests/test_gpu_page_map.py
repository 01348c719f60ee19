"""Calls on a page map and a pool at their edges: a slot named twice, requests
whose total passes 32 bits, empty lists, a pool made on a stream."""
import pytest
import torch

from test_gpu_pages import i32

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
