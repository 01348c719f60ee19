"""The failure path of attention over pages, without a GPU fault: the feed of
the cache stops early, the waits run out, the call reports NQ_DEV_TIMEOUT,
writes nothing beside its output and workspace, and the next call is right."""
import ctypes as C

import pytest
import torch

from test_gpu_page_attn import FORMATS, cache, check, i32, query

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt,planes", FORMATS)
@pytest.mark.parametrize("D,G", [(64, 64), (128, 128), (128, 64)])
@pytest.mark.parametrize("g,M", [(2, 1), (4, 3), (4, 5), (8, 5)])       # every kernel
def test_a_feed_that_stops(nq, fmt, planes, D, G, g, M):
    held, H = [9000, 5, 0, 4097], 2
    pool, m = cache(nq, held, H, D, G, 64, nq.KV_BF16 if fmt == "bf16" else nq.KV_NESTED44, 400)
    seqs = [1, 2] + [0] * 40 + [3] * 5            # more steps for every warp than any feed below gives
    lens = [held[s] for s in seqs]
    q, ln, slots = query(401, len(lens), M, H * g, D), i32(lens), i32(seqs)
    opts = nq.nq_attn_opts(0.1, 0.0, 0, 0, None)
    need = nq.lib().nq_page_attn_workspace_bytes(M, H * g, H, D)
    guard = 1 << 20
    ws = torch.empty(need + guard, dtype=torch.uint8, device="cuda")
    big = torch.empty(q.numel() + guard, dtype=torch.bfloat16, device="cuda")
    for steps in (0, 1, 7):
        for fill in (0x7F, 0x01, 0xFF):          # what an unwritten workspace may hold
            ws.fill_(fill)
            big.fill_(3.0)
            st = nq.lib().nq_selftest_page_attn(pool.ptr, 0, m.ptr, q.data_ptr(), H * g * D, len(lens), M, H * g, slots.data_ptr(), ln.data_ptr(),
                                                planes, C.byref(opts), big.data_ptr(), ws.data_ptr(), need, steps, 20000, nq._stream(None))
            assert st == 0
            assert nq.device_status() == nq.NQ_DEV_TIMEOUT
            assert (big[q.numel():] == 3.0).all() and (ws[need:] == fill).all()
    few = [41, 42, 0, 1, 2]
    check(nq, pool, m, [lens[b] for b in few], q[few].contiguous(), planes, 0.1, seqs=[seqs[b] for b in few])


def test_a_feed_that_lasts(nq):
    """With steps enough the diagnostic is the call itself."""
    pool, m = cache(nq, [900, 40], 2, 128, 128, 16, nq.KV_NESTED44, 402)
    q, ln = query(403, 2, 5, 16, 128), i32([900, 40])
    want = check(nq, pool, m, [900, 40], q, 2, 0.1)
    opts, out = nq.nq_attn_opts(0.1, 0.0, 0, 0, None), torch.empty_like(q)
    need = nq.lib().nq_page_attn_workspace_bytes(5, 16, 2, 128)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    assert nq.lib().nq_selftest_page_attn(pool.ptr, 0, m.ptr, q.data_ptr(), 16 * 128, 2, 5, 16, None, ln.data_ptr(), 2, C.byref(opts),
                                          out.data_ptr(), ws.data_ptr(), need, 1 << 20, 1000000, nq._stream(None)) == 0
    assert torch.equal(out, want) and nq.device_status() == 0
