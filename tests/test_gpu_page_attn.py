"""Attention over pages against the same rows in 64 bits (see attention64 for
how its tolerance comes about)."""
import numpy as np
import pytest
import torch

from paged_helpers import HostPool, attention64

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def cache(nq, lens, H, D, G, P, fmt, seed, layers=1, amp=1.0, extra=2, fill=-1):
    """Sequences of lens rows at shuffled pages.  Everything past their rows --
    the rest of their last pages, other pages, table entries -- is garbage."""
    g = torch.Generator().manual_seed(seed)
    need = [-(-n // P) for n in lens]
    W, N = max(need) + extra, sum(need) + 3
    pool = nq.PagePool(layers, N, P, H, D, fmt, group=G)
    pool.data.view(torch.int16).fill_(fill)      # -1: NaN as bf16, NaN scales
    ids = torch.randperm(N, generator=g).int()
    table = torch.full((len(lens), W), -7, dtype=torch.int32)
    at = 0
    for b, k in enumerate(need):
        table[b, :k] = ids[at:at + k]
        at += k
        table[b, k:] = 2 ** 30
    m = nq.PageMap(len(lens), W, N, P, table=table.cuda())
    seqs = i32([b for b, n in enumerate(lens) for _ in range(n)])
    pos = i32([t for n in lens for t in range(n)])
    if len(seqs):
        kv = torch.randn(len(seqs), 2 * H, D, generator=g).cuda()
        kv[:, :H] *= 1 + 3 * torch.rand(D, generator=g).cuda() ** 8
        kv[:, H:] *= amp
        pool.append(layers - 1, m, kv[:, :H], kv[:, H:], seqs, pos)
    return pool, m


def check(nq, pool, m, lens, q, planes, scale, seqs=None, **opts):
    layer = pool.layers - 1
    sl = opts.get("slopes")
    out = pool.attention(layer, m, q, i32(lens), planes, scale, seqs=None if seqs is None else i32(seqs), **opts)
    table = m.table.cpu().numpy()
    host = dict(opts, slopes=None if sl is None else sl.cpu().numpy())
    ref, tol = attention64(HostPool(pool), layer, table if seqs is None else table[seqs], q.float().cpu().numpy(), lens, planes, scale, **host)
    d = np.abs(out.double().cpu().numpy() - ref)
    assert np.isfinite(d).all() and (d <= tol).all(), (d / np.maximum(tol, 1e-300)).max()
    assert nq.device_status() == 0
    return out


def query(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


FORMATS = [("nested", 1), ("nested", 2), ("bf16", 2)]


@pytest.mark.parametrize("fmt,planes", FORMATS)
@pytest.mark.parametrize("H,g,D,G,P,M,lens", [
    (1, 1, 128, 128, 16, 1, [1]),
    (2, 1, 64, 64, 16, 1, [0, 1, 15, 16, 17, 31, 32, 33]),
    (4, 8, 128, 64, 32, 1, [700, 0, 3]),              # 8 query vectors per kv head
    (4, 7, 128, 128, 64, 1, [65, 128, 513]),          # 7
    (2, 4, 128, 128, 16, 5, [300, 2, 5, 0, 4]),       # lengths below M: the first queries see nothing
    (1, 2, 64, 64, 256, 9, [1000, 257]),              # 18 query vectors: more than two tiles of 8
    (2, 8, 128, 128, 128, 9, [411, 130]),             # 72
    (8, 1, 128, 64, 32, 2, [2050]),
    (3, 5, 128, 128, 16, 3, [77, 1500, 3, 640, 9]),
    (32, 1, 64, 64, 64, 4, [129, 64]),
])
def test_matches_64_bits(nq, fmt, planes, H, g, D, G, P, M, lens):
    pool, m = cache(nq, lens, H, D, G, P, getattr(nq, "KV_BF16" if fmt == "bf16" else "KV_NESTED44"), 7 * H + M, layers=2)
    check(nq, pool, m, lens, query(M + D, len(lens), M, H * g, D), planes, D ** -0.5)


@pytest.mark.parametrize("fmt,planes", FORMATS)
@pytest.mark.parametrize("cap,window,slopes", [(20.0, 0, False), (0.0, 1, False), (0.0, 40, False), (0.0, 0, True),
                                               (50.0, 333, True), (0.0, 5000, False)])
def test_cap_window_bias(nq, fmt, planes, cap, window, slopes):
    lens, H, g, D, M = [1, 47, 900, 2000, 0], 2, 4, 128, 3
    pool, m = cache(nq, lens, H, D, 128, 32, getattr(nq, "KV_BF16" if fmt == "bf16" else "KV_NESTED44"), 50)
    s = torch.tensor([2.0 ** -(i % 7 + 1) for i in range(H * g)], device="cuda") if slopes else None
    check(nq, pool, m, lens, 4 * query(51, len(lens), M, H * g, D), planes, 0.1, softcap=cap, window=window, slopes=s)


@pytest.mark.parametrize("fmt,planes", FORMATS)
def test_pages_before_the_window_are_never_used(nq, fmt, planes):
    """Pages that a window has left behind may be released: their entries may be anything."""
    lens, P, window, M = [1000, 530], 16, 100, 2
    pool, m = cache(nq, lens, 2, 64, 64, P, getattr(nq, "KV_BF16" if fmt == "bf16" else "KV_NESTED44"), 60)
    q = query(61, 2, M, 4, 64)
    want = check(nq, pool, m, lens, q, planes, 0.2, window=window)
    for b, n in enumerate(lens):
        m.table[b, :(n - M - window + 1) // P] = -1
    got = pool.attention(0, m, q, i32(lens), planes, 0.2, window=window)
    assert torch.equal(got, want) and nq.device_status() == 0


@pytest.mark.parametrize("fmt,planes", FORMATS)
def test_long_ragged_batch(nq, fmt, planes):
    """Sequences cut over many CTAs beside short ones, and more (sequence, head) pairs than CTAs."""
    pool, m = cache(nq, [9000, 5, 0, 4097, 31], 2, 128, 128, 64, getattr(nq, "KV_BF16" if fmt == "bf16" else "KV_NESTED44"), 70)
    check(nq, pool, m, [9000, 5, 0, 4097, 31], query(71, 5, 1, 4, 128), planes, 0.09)
    lens = [(37 * i) % 200 for i in range(150)]
    pool, m = cache(nq, lens, 8, 64, 64, 16, getattr(nq, "KV_BF16" if fmt == "bf16" else "KV_NESTED44"), 72)
    check(nq, pool, m, lens, query(73, 150, 1, 8, 64), planes, 0.125)


@pytest.mark.parametrize("fmt,planes", FORMATS)
def test_slots_strides_and_scales(nq, fmt, planes):
    """Slots in any order and repeated, tiny and huge values, a strongly peaked softmax."""
    kind = getattr(nq, "KV_BF16" if fmt == "bf16" else "KV_NESTED44")
    lens = [300, 45, 801]
    pool, m = cache(nq, lens, 2, 128, 128, 16, kind, 80, amp=1e-4)
    check(nq, pool, m, [801, 300, 300, 20], query(81, 4, 2, 4, 128), planes, 0.09, seqs=[2, 0, 0, 1])
    pool, m = cache(nq, lens, 2, 128, 128, 16, kind, 82, amp=1000.0)
    for f in (1e-3, 30.0):
        check(nq, pool, m, lens, f * query(83, 3, 1, 2, 128), planes, 0.09)
    check(nq, pool, m, lens, 2.0 ** 20 * query(84, 3, 1, 2, 128), planes, 0.09 * 2.0 ** -20)


def test_inner_values_of_later_rows_stay_out(nq):
    """bf16: a non-finite value row is seen by the queries at and after it, by no earlier one."""
    lens, M = [50], 4
    pool, m = cache(nq, lens, 1, 64, 64, 16, nq.KV_BF16, 90)
    q = query(91, 1, M, 2, 64)
    want = pool.attention(0, m, q, i32(lens), 2, 0.1)
    k, v = pool.read(0, m, i32([0]), i32([48]))
    v[:] = float("inf")
    pool.append(0, m, k, v, i32([0]), i32([48]))
    got = pool.attention(0, m, q, i32(lens), 2, 0.1)
    assert torch.equal(got[:, :2], want[:, :2]) and torch.isinf(got[:, 2:]).all()


@pytest.mark.parametrize("fmt,planes", FORMATS)
def test_bytes_past_32_bits(nq, fmt, planes):
    """Pages that lie beyond 4 GB in the pool."""
    kind = getattr(nq, "KV_BF16" if fmt == "bf16" else "KV_NESTED44")
    H, D, P = 8, 128, 64
    n = nq.PagePool(1, 1, P, H, D, kind, data=None).bytes
    N = (9 << 29) // n
    pool = nq.PagePool(1, N, P, H, D, kind)
    table = torch.tensor([[N - 1, 0, N - 5], [N // 2, N - 2, 1]], dtype=torch.int32, device="cuda")
    m = nq.PageMap(2, 3, N, P, table=table)
    lens = [150, 192]
    kv = torch.randn(sum(lens), 2 * H, D, generator=torch.Generator().manual_seed(3)).cuda()
    seqs, pos = i32([0] * 150 + [1] * 192), i32(list(range(150)) + list(range(192)))
    pool.append(0, m, kv[:, :H], kv[:, H:], seqs, pos)
    q = query(4, 2, 1, 2 * H, D)
    got = pool.attention(0, m, q, i32(lens), planes, 0.09)
    # the same rows in a small pool
    small = nq.PagePool(1, 6, P, H, D, kind)
    sm = nq.PageMap(2, 3, 6, P, table=i32([[0, 1, 2], [3, 4, 5]]))
    small.append(0, sm, kv[:, :H], kv[:, H:], seqs, pos)
    assert torch.equal(got, small.attention(0, sm, q, i32(lens), planes, 0.09)) and nq.device_status() == 0


def test_same_bits_again_side_stream_and_graph(nq):
    lens = [3000, 77, 512]
    pool, m = cache(nq, lens, 4, 128, 128, 16, nq.KV_NESTED44, 95)
    q, ln = query(96, 3, 5, 16, 128), i32(lens)
    want = pool.attention(0, m, q, ln, 2, 0.09)
    for _ in range(20):
        assert torch.equal(pool.attention(0, m, q, ln, 2, 0.09), want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, ws = torch.empty_like(want), torch.empty(nq.lib().nq_page_attn_workspace_bytes(5, 16, 4, 128), dtype=torch.uint8, device="cuda")
        got = pool.attention(0, m, q, ln, 2, 0.09, out=out, ws=ws)
        s.synchronize()
        assert torch.equal(got, want)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            pool.attention(0, m, q, ln, 2, 0.09, out=out, ws=ws)
    out.zero_()
    ln.copy_(i32([2000, 78 - 1, 400]))           # lengths are read on the device, at replay
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, pool.attention(0, m, q, i32([2000, 77, 400]), 2, 0.09))


def test_reports(nq):
    pool, m = cache(nq, [40, 20], 1, 64, 64, 16, nq.KV_NESTED44, 99, extra=1)
    q = query(98, 2, 1, 1, 64)
    pool.attention(0, m, q, i32([40, 2 ** 30]), 1, 0.1)                       # clamped to the table; its ids are garbage
    assert nq.device_status() == nq.NQ_DEV_SEQ_FULL | nq.NQ_DEV_BAD_PAGE
    pool.attention(0, m, q, i32([40, 20]), 1, 0.1, seqs=i32([0, 2]))
    assert nq.device_status() == nq.NQ_DEV_BAD_PAGE
    out = pool.attention(0, m, q, i32([-5, 0]), 1, 0.1)
    assert (out == 0).all() and nq.device_status() == 0
    for bad in (lambda: pool.attention(0, m, q.float(), i32([1, 1]), 1, 0.1), lambda: pool.attention(0, m, q, i32([1]), 1, 0.1),
                lambda: pool.attention(0, m, q, i32([1, 1]), 1, 0.1, slopes=torch.ones(3, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(nq.NQError):
        pool.attention(0, m, q, i32([1, 1]), 3, 0.1)


# more query vectors per kv head than one warp holds: 8 columns per warp, or rows of the tensor cores
MANY = [
    (1, 8, 64, 64, 16, 4, [0, 1, 63, 64, 65, 200, 3]),       # 32 vectors of small heads, lengths about a step
    (2, 8, 128, 128, 16, 5, [1, 4, 700, 129, 64]),           # 40
    (2, 8, 128, 64, 32, 5, [1, 4, 700, 129]),                # 40, two groups per row
    (1, 20, 128, 128, 64, 9, [333, 100, 9]),                 # 180: two tiles of the tensor cores, three of 64
    (2, 7, 128, 128, 128, 3, [80, 2000]),                    # 21
    (1, 13, 64, 64, 256, 2, [515, 31]),                      # 26
    (1, 128, 128, 128, 16, 1, [300]),                        # 128: a full tile
]


@pytest.mark.parametrize("fmt,planes", FORMATS)
@pytest.mark.parametrize("H,g,D,G,P,M,lens", MANY)
def test_many_query_vectors(nq, fmt, planes, H, g, D, G, P, M, lens):
    pool, m = cache(nq, lens, H, D, G, P, getattr(nq, "KV_BF16" if fmt == "bf16" else "KV_NESTED44"), 11 * H + M, layers=2)
    check(nq, pool, m, lens, query(M + D, len(lens), M, H * g, D), planes, D ** -0.5)


@pytest.mark.parametrize("fmt,planes", FORMATS)
@pytest.mark.parametrize("cap,window,slopes", [(20.0, 0, False), (0.0, 1, False), (0.0, 90, False), (0.0, 0, True), (50.0, 333, True)])
@pytest.mark.parametrize("D,G,g", [(128, 128, 8), (64, 64, 4), (128, 64, 4)])
def test_many_query_vectors_cap_window_bias(nq, fmt, planes, cap, window, slopes, D, G, g):
    lens, H, M = [1, 47, 900, 0, 130], 2, 7
    pool, m = cache(nq, lens, H, D, G, 32, getattr(nq, "KV_BF16" if fmt == "bf16" else "KV_NESTED44"), 150)
    s = torch.tensor([2.0 ** -(i % 7 + 1) for i in range(H * g)], device="cuda") if slopes else None
    check(nq, pool, m, lens, 4 * query(151, len(lens), M, H * g, D), planes, 0.1, softcap=cap, window=window, slopes=s)


@pytest.mark.parametrize("fmt,planes", FORMATS)
def test_many_query_vectors_long_and_many(nq, fmt, planes):
    """Segments cut over many CTAs, many short ones, peaked and tiny values; the same bits again."""
    kind = getattr(nq, "KV_BF16" if fmt == "bf16" else "KV_NESTED44")
    pool, m = cache(nq, [9000, 5, 0, 4097], 1, 128, 128, 64, kind, 170)
    q = query(171, 4, 5, 8, 128)
    want = check(nq, pool, m, [9000, 5, 0, 4097], q, planes, 0.09)
    for _ in range(30):
        assert torch.equal(pool.attention(0, m, q, i32([9000, 5, 0, 4097]), planes, 0.09), want)
    lens = [(53 * i) % 150 for i in range(90)]
    pool, m = cache(nq, lens, 4, 64, 64, 16, kind, 172)
    check(nq, pool, m, lens, query(173, 90, 4, 32, 64), planes, 0.125)
    pool, m = cache(nq, [900, 77], 1, 128, 128, 16, kind, 174, amp=1e-4)
    check(nq, pool, m, [900, 77], 30 * query(175, 2, 4, 8, 128), planes, 0.09)


def test_many_query_vectors_inner_values(nq):
    """bf16: a non-finite value row is seen by the queries at and after it, by no earlier one."""
    lens, M = [50], 4
    pool, m = cache(nq, lens, 1, 64, 64, 16, nq.KV_BF16, 190)
    q = query(191, 1, M, 8, 64)
    want = pool.attention(0, m, q, i32(lens), 2, 0.1)
    k, v = pool.read(0, m, i32([0]), i32([48]))
    v[:] = float("inf")
    pool.append(0, m, k, v, i32([0]), i32([48]))
    got = pool.attention(0, m, q, i32(lens), 2, 0.1)
    assert torch.equal(got[:, :2], want[:, :2]) and torch.isinf(got[:, 2:]).all()


@pytest.mark.parametrize("fmt,planes", FORMATS)
@pytest.mark.parametrize("fill", [-1, -1024, 0x7C00, -128, 0x7F80, 0x7BFF])
@pytest.mark.parametrize("g,M", [(1, 1), (4, 3), (4, 5), (8, 5)])
def test_rows_past_the_end_hold_anything(nq, fmt, planes, fill, g, M):
    """NaN, both infinities (of fp16, of bf16) and the largest scale in every row that no sequence has."""
    lens = [1, 18, 250, 65, 0, 33]
    pool, m = cache(nq, lens, 2, 64, 64, 32, getattr(nq, "KV_BF16" if fmt == "bf16" else "KV_NESTED44"), 200, fill=fill)
    check(nq, pool, m, lens, query(201 + M, len(lens), M, 2 * g, 64), planes, 0.125)
