"""Rows stored in pages and the pages' bookkeeping on the GPU, against the page
format read byte by byte and a sequential model of the bookkeeping."""
import random

import numpy as np
import pytest
import torch

import oracle as O
from paged_helpers import HostMap, HostPool

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def scattered(nq, S, W, P, N, seed):
    """A map whose slots hold W pages each at shuffled ids (the table alone)."""
    g = torch.Generator().manual_seed(seed)
    return nq.PageMap(S, W, N, P, table=torch.randperm(N, generator=g)[:S * W].reshape(S, W).int().cuda())


def tokens(S, rows, seed):
    """Every row of every slot once, in a shuffled order."""
    at = [(s, t) for s in range(S) for t in range(rows[s])]
    random.Random(seed).shuffle(at)
    return i32([s for s, _ in at]), i32([t for _, t in at])


@pytest.mark.parametrize("D,G,P,H,Hq", [(128, 128, 16, 3, 6), (128, 64, 32, 2, 2), (64, 64, 64, 1, 8), (128, 128, 256, 2, 14)])
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_append_nested_codes_and_read(nq, D, G, P, H, Hq, dtype):
    """Codes and scales are the weights' quantiser's bit for bit; rotated rows
    are those of the rotation alone; reading gives both views' values."""
    S, rows = 3, [P + 5, 1, 2 * P]
    pool, m = nq.PagePool(2, 11, P, H, D, nq.KV_NESTED44, group=G), scattered(nq, S, 3, P, 11, 1)
    seqs, pos = tokens(S, rows, 2)
    T = len(seqs)
    g = torch.Generator().manual_seed(D + P)
    x = (torch.randn(T, Hq + 2 * H, D, generator=g) * 3).to(getattr(torch, dtype)).cuda()
    x[T // 2, Hq] = 0                                   # a row of zeros: scale 0
    plan = nq.Rope(D, layout="interleaved" if D == 64 else "half")
    before = pool.data.clone()
    q = pool.append(1, m, x[:, Hq:Hq + H], x[:, Hq + H:], seqs, pos, rope=plan, q=x[:, :Hq])
    assert nq.device_status() == 0
    assert torch.equal(q, nq.rope(x[:, :Hq], pos, plan, out_dtype=torch.bfloat16))
    half = pool.data.numel() // 2
    assert torch.equal(pool.data[:half], before[:half])  # the other layer
    K = nq.rope(x[:, Hq:Hq + H], pos, plan, out_dtype=torch.float32).cpu().numpy()
    V = x[:, Hq + H:].float().cpu().numpy()
    hp, table = HostPool(pool), m.table.cpu().numpy()
    sq, ps = seqs.cpu().numpy(), pos.cpu().numpy()
    outs = {p: [t.double().cpu().numpy() for t in pool.read(1, m, seqs, pos, planes=p)] for p in (1, 2)}
    nib = lambda b: np.stack([(b & 15).astype(np.int8), (b >> 4).astype(np.int8)], -1).reshape(*b.shape[:-1], -1)  # noqa: E731
    for which, X in ((0, K), (1, V)):
        base, resid, scales = O.kv_rows_pack(np.ascontiguousarray(X), G)
        want = [np.where(nib(c.reshape(T, H, D // 2)) > 7, nib(c.reshape(T, H, D // 2)) - 16, nib(c.reshape(T, H, D // 2))) for c in (base, resid)]
        for t in range(T):
            page = table[sq[t], ps[t] // P]
            for h in range(H):
                q4, r, sc = hp.codes(1, page, h, ps[t] % P, which)
                assert np.array_equal(q4, want[0][t, h]) and np.array_equal(r, want[1][t, h])
                assert np.array_equal(sc, scales.reshape(T, H, -1)[t, h])
                for p in (1, 2):
                    v = hp.row(1, page, h, ps[t] % P, which, p)
                    assert (np.abs(outs[p][which][t, h] - v) <= 2.0 ** -8 * np.abs(v) + 1e-30).all()


@pytest.mark.parametrize("D,P,H", [(128, 16, 2), (64, 128, 3)])
def test_append_bf16_and_strides(nq, D, P, H):
    S, rows = 2, [P + 1, P]
    pool, m = nq.PagePool(1, 5, P, H, D, nq.KV_BF16), scattered(nq, S, 2, P, 5, 4)
    seqs, pos = tokens(S, rows, 5)
    T = len(seqs)
    x = torch.randn(T, 2 * H + 3, D, generator=torch.Generator().manual_seed(D)).cuda()
    assert pool.append(0, m, x[:, :H], x[:, H:2 * H], seqs, pos) is None
    k, v = pool.read(0, m, seqs, pos)
    assert torch.equal(k, x[:, :H].bfloat16()) and torch.equal(v, x[:, H:2 * H].bfloat16())
    hp, table = HostPool(pool), m.table.cpu().numpy()
    for t in (0, T - 1):
        page, row = table[int(seqs[t]), int(pos[t]) // P], int(pos[t]) % P
        assert np.array_equal(hp.row(0, page, H - 1, row, 1, 2), v[t, H - 1].double().cpu().numpy())
    assert nq.device_status() == 0


def test_append_and_read_bad_rows(nq):
    """Rows past the table, slots outside the map and pages outside the pool are
    dropped and reported; every other row is stored; nothing else is written."""
    P, H, D = 16, 1, 64
    pool = nq.PagePool(1, 4, P, H, D, nq.KV_BF16)
    table = i32([[0, 2], [1, -1], [9, 3]])
    m = nq.PageMap(3, 2, 4, P, table=table)
    x = torch.ones(7, 1, D, device="cuda")
    ok = [(0, 3), (1, 15), (2, 31)]
    for bad, bit in (((0, 32), nq.NQ_DEV_SEQ_FULL), ((3, 0), nq.NQ_DEV_BAD_PAGE), ((-1, 0), nq.NQ_DEV_BAD_PAGE),
                     ((0, -1), nq.NQ_DEV_BAD_PAGE), ((1, 16), nq.NQ_DEV_BAD_PAGE), ((2, 0), nq.NQ_DEV_BAD_PAGE)):
        pool.data.zero_()
        at = ok + [bad]
        seqs, pos = i32([s for s, _ in at]), i32([t for _, t in at])
        pool.append(0, m, x[:4], x[:4], seqs, pos)
        assert nq.device_status() == bit, bad
        k, v = pool.read(0, m, seqs, pos)
        assert nq.device_status() & bit
        assert (k[:3] == 1).all() and (v[:3] == 1).all() and (k[3] == 0).all() and (v[3] == 0).all()
        assert int((pool.data.view(torch.bfloat16) == 1).sum()) == 3 * 2 * D
    # non-finite rows are reported in the nested format
    pool = nq.PagePool(1, 4, P, H, D, nq.KV_NESTED44, group=64)
    for value in (float("nan"), float("inf"), 1e30):
        y = x[:1].clone()
        y[0, 0, 5] = value
        pool.append(0, m, y, x[:1], i32([0]), i32([0]))
        assert nq.device_status() == nq.NQ_DEV_NONFINITE


def same(m, h):
    assert np.array_equal(m.table.cpu().numpy(), h.table())
    assert np.array_equal(m.held.cpu().numpy(), h.held())
    assert m.ref.cpu().tolist() == h.ref


@pytest.mark.parametrize("S,W,N,P,seed", [(5, 6, 24, 16, 0), (40, 9, 190, 64, 1), (3, 70, 9000, 16, 2), (1100, 4, 2600, 16, 3)])
def test_bookkeeping_matches_model(nq, S, W, N, P, seed):
    """Random requests against the sequential model: tables, counts, what is
    served when pages run out, and the pages' contents through copies and moves."""
    r = random.Random(seed)
    H, D, layers = 1, 64, 3
    pool, m, h = nq.PagePool(layers, N, P, H, D, nq.KV_BF16), nq.PageMap(S, W, N, P), HostMap(S, W, N, P)
    same(m, h)
    content = torch.randint(0, 256, (layers, N, pool.data.numel() // layers // N), dtype=torch.uint8, generator=torch.Generator().manual_seed(seed))
    pool.data.copy_(content.reshape(-1))
    status = 0
    for step in range(14):
        n = r.randint(1, S)
        slots = r.sample(range(S), n)
        kind = r.choice(["reserve", "reserve", "fork", "truncate", "compact"]) if step else "reserve"
        top = lambda s: len(h.pages[s]) * P  # noqa: E731
        if kind == "reserve":
            first = [r.randint(0, top(s)) for s in slots]
            last = [f + r.randint(0, 3 * P) for f in first]
            got = m.reserve(pool, i32(slots), i32(first), i32(last))
            granted, copies = h.reserve(slots, first, last)
            assert got.cpu().tolist() == granted
            for a, b in copies:
                content[:, b] = content[:, a]
            # pages taken without a copy hold whatever they held
        elif kind == "fork":
            src = [r.randrange(S) for _ in slots]
            rows = [r.randint(0, top(s)) for s in src]
            m.fork(i32(src), i32(slots), i32(rows))
            h.fork(src, slots, rows)
        elif kind == "truncate":
            rows = [r.randint(0, top(s) + P) for s in slots]
            m.truncate(i32(slots), i32(rows))
            h.truncate(slots, rows)
        else:
            used, moves = h.compact()
            assert int(m.compact(pool)) == used
            for a, b in moves:
                content[:, b] = content[:, a]
        same(m, h)
        assert torch.equal(pool.data.cpu().view_as(content), content)
        status |= nq.device_status()
    assert status & ~(nq.NQ_DEV_POOL_FULL | nq.NQ_DEV_SEQ_FULL) == 0


def test_last_holder_keeps_its_page(nq):
    m = nq.PageMap(4, 4, 8, 16)
    pool = nq.PagePool(2, 8, 16, 1, 64, nq.KV_BF16)
    pool.data.copy_(torch.arange(pool.data.numel(), device="cuda") % 251)
    m.reserve(pool, i32([0]), i32([0]), i32([20]))
    m.fork(i32([0, 0]), i32([1, 2]), i32([20, 20]))
    old = pool.data.view(2, 8, -1).clone()
    assert m.reserve(pool, i32([2, 0, 1]), i32([20, 20, 20]), i32([21, 21, 21])).cpu().tolist() == [1, 1, 1]
    assert m.table[:3, :2].cpu().tolist() == [[0, 3], [0, 1], [0, 2]]
    new = pool.data.view(2, 8, -1)
    assert torch.equal(new[:, 2], old[:, 1]) and torch.equal(new[:, 3], old[:, 1]) and torch.equal(new[:, 4:], old[:, 4:])


def test_bookkeeping_reports(nq):
    m, pool = nq.PageMap(3, 2, 3, 16), nq.PagePool(1, 3, 16, 1, 64, nq.KV_BF16)
    # past the table, outside the map, before the first row: left out, the others served
    got = m.reserve(pool, i32([0, 1, 2]), i32([0, 0, -4]), i32([33, 5, 7]))
    assert got.cpu().tolist() == [0, 1, 0] and nq.device_status() == nq.NQ_DEV_SEQ_FULL | nq.NQ_DEV_BAD_PAGE
    assert m.reserve(pool, i32([7, 0]), i32([0, 0]), i32([1, 20])).cpu().tolist() == [0, 1]
    assert nq.device_status() == nq.NQ_DEV_BAD_PAGE and m.ref.cpu().tolist() == [1, 1, 1]
    # no page left: nothing changes
    table = m.table.clone()
    assert m.reserve(pool, i32([2]), i32([0]), i32([1])).cpu().tolist() == [0]
    assert nq.device_status() == nq.NQ_DEV_POOL_FULL and torch.equal(m.table, table)
    assert m.reserve(pool, i32([2]), i32([5]), i32([5])).cpu().tolist() == [1] and nq.device_status() == 0   # no rows
    m.fork(i32([0, 5]), i32([2, 1]), i32([40, 1]))           # more rows than held; a slot outside
    assert nq.device_status() == nq.NQ_DEV_BAD_PAGE and m.held.cpu().tolist() == [2, 1, 2]
    m.truncate(i32([0, -1]), i32([0, 0]))
    assert nq.device_status() == nq.NQ_DEV_BAD_PAGE and m.held.cpu().tolist() == [0, 1, 2]
    pool.copy_pages(i32([0, 3]), i32([2, 1]))
    assert nq.device_status() == nq.NQ_DEV_BAD_PAGE


def test_copy_pages(nq):
    pool = nq.PagePool(3, 40, 32, 5, 128, nq.KV_NESTED44, group=64)
    g = torch.Generator().manual_seed(9)
    pool.data.copy_(torch.randint(0, 256, (pool.data.numel(),), dtype=torch.uint8, generator=g))
    want = pool.data.view(3, 40, -1).clone()
    perm = torch.randperm(40, generator=g).int().cuda()
    src, dst = perm[:17].contiguous(), perm[20:37].contiguous()
    want[:, dst.long()] = want[:, src.long()]
    pool.copy_pages(src, dst)
    assert torch.equal(pool.data.view(3, 40, -1), want)
