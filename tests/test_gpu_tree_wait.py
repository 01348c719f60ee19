"""The failure path of attention of trees, without a GPU fault (as test_gpu_page_wait.py): the feed of the cache stops
early, the waits run out, the call reports NQ_DEV_TIMEOUT, writes nothing beside its output and workspace, and the
next call is right."""
import ctypes as C

import pytest
import torch

import tree_helpers as T
from test_gpu_tree_attn import check, i32, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,G,P,fmt,planes", [(128, 128, 16, 0, 2), (128, 128, 64, 0, 1), (64, 64, 16, 0, 2), (128, 64, 32, 0, 2), (128, 128, 16, 1, 2)])
@pytest.mark.parametrize("M,Hq", [(5, 1), (12, 1), (20, 1), (40, 2), (50, 3), (90, 3)])       # every kernel; one and two groups, two tiles
def test_a_feed_that_stops(nq, D, G, P, fmt, planes, M, Hq):
    held = [9000, M, M + 4097]
    parents = T.trees(M, 3, M)
    pool, m, q3 = setup(nq, held, parents, P, 1, Hq, D, G, fmt, 400)
    seqs = [1, 2] + [0] * 100 + [2] * 5            # more steps for every warp than any feed below gives
    lens, q = [held[s] for s in seqs], q3[seqs].contiguous()
    ln, slots, tree = i32(lens), i32(seqs), nq.Tree(i32([parents[s] for s in seqs]))
    opts = nq.nq_attn_opts(0.1, 0.0, 0, 0, None)
    need = nq.lib().nq_page_attn_tree_workspace_bytes(M, Hq, 1, D)
    guard = 1 << 20
    ws = torch.empty(need + guard, dtype=torch.uint8, device="cuda")
    big = torch.empty(q.numel() + guard, dtype=torch.bfloat16, device="cuda")
    for steps in (0, 1, 2, 5):
        for fill in (0x7F, 0x01, 0xFF):           # what an unwritten workspace may hold
            ws.fill_(fill)
            big.fill_(3.0)
            st = nq.lib().nq_selftest_page_attn_tree(pool.ptr, 0, m.ptr, q.data_ptr(), Hq * D, Hq, slots.data_ptr(), ln.data_ptr(), planes, C.byref(opts),
                                                     tree.ref, big.data_ptr(), ws.data_ptr(), need, steps, 20000, nq._stream(None))
            assert st == 0
            assert nq.device_status() == nq.NQ_DEV_TIMEOUT
            assert (big[q.numel():] == 3.0).all() and (ws[need:] == fill).all()
    lens = [200 + M, 0, M + 1]
    pool, m, q = setup(nq, lens, parents, P, 1, Hq, D, G, fmt, 401)
    check(nq, pool, m, q, lens, parents, planes)


@pytest.mark.parametrize("M,Hq", [(5, 1), (20, 1), (50, 3)])
def test_a_feed_that_lasts(nq, M, Hq):
    """With steps enough the diagnostic is the call itself."""
    lens, parents = [900 + M, M + 3], T.trees(M, 2, M)
    pool, m, q = setup(nq, lens, parents, 16, 1, Hq, 128, 128, 0, 402)
    want = check(nq, pool, m, q, lens, parents, 2)
    tree, ln = nq.Tree(i32(parents)), i32(lens)
    opts, out = nq.nq_attn_opts(128 ** -0.5, 0.0, 0, 0, None), torch.empty_like(q)
    need = nq.lib().nq_page_attn_tree_workspace_bytes(M, Hq, 1, 128)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert nq.lib().nq_selftest_page_attn_tree(pool.ptr, 0, m.ptr, q.data_ptr(), Hq * 128, Hq, None, ln.data_ptr(), 2, C.byref(opts), tree.ref,
                                               out.data_ptr(), ws.data_ptr(), need, 1 << 20, 1000000, nq._stream(None)) == 0
    assert torch.equal(out, want) and nq.device_status() == 0
