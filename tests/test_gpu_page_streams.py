"""Streams, graphs and threads of the rotary, paged-cache and attention calls:
what a call allocates belongs to its stream, and the workspaces that objects keep
are never shared by work that may overlap.  Every call gives the same bits on
every run, so results are compared for equality."""
import threading

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nq():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from quantized_self_speculative_gb300 import nq as m
    m.lib()
    return m


def cache(nq, B=6, rows=1500, H=4, D=128, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = (rows + 15) // 16
    pmap = nq.PageMap(B, W, B * W, 16)
    pool = nq.PagePool(1, B * W, 16, H, D)
    seqs = torch.arange(B, dtype=torch.int32, device="cuda")
    full = torch.full_like(seqs, rows)
    assert pmap.reserve(pool, seqs, torch.zeros_like(seqs), full).all()
    kv = torch.randn(B * rows, 2 * H, D, generator=g, device="cuda")
    pos = torch.arange(rows, dtype=torch.int32, device="cuda").repeat(B)
    pool.append(0, pmap, kv[:, :H], kv[:, H:], seqs.repeat_interleave(rows), pos)
    return pool, pmap, full


def queries(n, B=6, M=2, Hq=16, D=128):
    g = torch.Generator(device="cuda").manual_seed(99)
    return [torch.randn(B, M, Hq, D, generator=g, device="cuda").bfloat16() for _ in range(n)]


def busy_then_overwrite(shape, dtype):
    """The current stream works for some milliseconds, then writes a tensor that is already given back."""
    x = torch.empty(shape, dtype=dtype, device="cuda")
    torch.cuda._sleep(20_000_000)
    x.fill_(7)
    del x


def test_results_of_another_stream_keep_their_memory(nq):
    pool, pmap, lens = cache(nq)
    q = queries(1)[0]
    plan = nq.Rope(128)
    x, pos = torch.randn(64, 8, 128, device="cuda"), torch.arange(64, dtype=torch.int32, device="cuda")
    seqs = torch.zeros(64, dtype=torch.int32, device="cuda")
    calls = [lambda **k: (nq.rope(x, pos, plan, **k),),
             lambda **k: (pool.attention(0, pmap, q, lens, 2, 0.1, **k),),
             lambda **k: pool.read(0, pmap, seqs, pos, **k)]
    for call in calls:
        want = [t.clone() for t in call()]
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        for t in want:
            busy_then_overwrite(t.shape, t.dtype)
        got = call(stream=s)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert nq.device_status() == 0


def test_streams_side_by_side(nq):
    pool, pmap, lens = cache(nq)
    qs = queries(4)
    want = [pool.attention(0, pmap, q, lens, 2, 0.1) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for q, s in zip(qs, streams):
            with torch.cuda.stream(s):
                got.append(pool.attention(0, pmap, q, lens, 2, 0.1))
    torch.cuda.synchronize()
    assert all(torch.equal(want[i % 4], y) for i, y in enumerate(got))


def test_eager_calls_beside_a_replayed_graph(nq):
    pool, pmap, lens = cache(nq)
    qa, qb = queries(2)
    wa, wb = pool.attention(0, pmap, qa, lens, 2, 0.1), pool.attention(0, pmap, qb, lens, 2, 0.1)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ya = pool.attention(0, pmap, qa, lens, 2, 0.1)
    torch.cuda.synchronize()
    for _ in range(10):
        ya.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            g.replay()
        yb = pool.attention(0, pmap, qb, lens, 2, 0.1)
        torch.cuda.synchronize()
        assert torch.equal(ya, wa) and torch.equal(yb, wb)


def test_threads_on_one_stream(nq):
    pool, pmap, lens = cache(nq)
    qs = queries(4)
    want = [pool.attention(0, pmap, q, lens, 2, 0.1) for q in qs]
    torch.cuda.synchronize()
    got = [[] for _ in qs]

    def work(i):
        for _ in range(25):
            got[i].append(pool.attention(0, pmap, qs[i], lens, 2, 0.1))

    ts = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    torch.cuda.synchronize()
    for i, ys in enumerate(got):
        assert len(ys) == 25 and all(torch.equal(want[i], y) for y in ys)


def test_a_kept_workspace_grows(nq):
    """Few query vectors, then many (another kernel, a larger workspace), then few again."""
    pool, pmap, lens = cache(nq)
    few, many = queries(1, M=1)[0], queries(1, M=9)[0]
    a = pool.attention(0, pmap, few, lens, 2, 0.1)
    b = pool.attention(0, pmap, many, lens, 2, 0.1)
    big = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    assert torch.equal(a, pool.attention(0, pmap, few, lens, 2, 0.1))
    assert torch.equal(b, pool.attention(0, pmap, many, lens, 2, 0.1, ws=big))
    with pytest.raises(nq.NQError):
        pool.attention(0, pmap, few, lens, 2, 0.1, ws=big[:1024])


def test_bookkeeping_on_another_stream(nq):
    pool, pmap, _ = cache(nq, B=4, rows=64)
    s = torch.cuda.Stream()
    ints = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    seqs, rows, zero, last = ints(0, 1), ints(20, 0), ints(20, 0), ints(40, 16)
    torch.cuda.synchronize()
    busy_then_overwrite(2, torch.int32)
    pmap.truncate(seqs, rows, stream=s)
    granted = pmap.reserve(pool, seqs, zero, last, stream=s)
    pmap.fork(ints(0), ints(1), ints(30), stream=s)
    used = pmap.compact(pool, stream=s)
    torch.cuda.synchronize()
    assert granted.tolist() == [1, 1] and pmap.held.tolist()[:2] == [3, 2]
    table = pmap.table.cpu().numpy()
    assert list(table[1, :2]) == list(table[0, :2])          # shared
    live = np.unique(np.concatenate([table[b, :n] for b, n in enumerate(pmap.held.tolist())]))
    assert used.item() == len(live) == live.max() + 1
    assert nq.device_status() == 0
