"""Attention of trees of drafted tokens over pages, against 64 bits (tolerances:
tree_helpers.tree_attention64).  Everything that no query may see holds NaN: rows
past a sequence's end, rows of unused nodes, the queries of unused nodes."""
import numpy as np
import pytest
import torch

import tree_helpers as T
from paged_helpers import HostPool

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def setup(nq, lens, parents, P, H, Hq, D, G, fmt, seed, layers=1, layer=0, big=None):
    """A pool of NaN into which the rows that are there have been appended, a map, queries."""
    B, M = len(lens), len(parents[0])
    W = max(1, -(-max(lens) // P)) + 1
    N = B * W + 2
    g = torch.Generator(device="cuda").manual_seed(seed)
    pool = nq.PagePool(layers, N, P, H, D, fmt, group=G)
    pool.data.fill_(0xFF)                      # scales (or values) that are NaN
    m = nq.PageMap(B, W, N, P, table=torch.randperm(N, generator=g, device="cuda")[:B * W].reshape(B, W).int())
    at = []
    for b, n in enumerate(lens):
        used = [d >= 0 for d, _ in T.sets_of(parents[b])]
        at += [(b, t) for t in range(n) if t < n - M or used[t - (n - M)]]
    if at:
        ch = 1 + 3 * torch.rand(D, generator=g, device="cuda") ** 8
        kv = torch.randn(len(at), 2 * H, D, generator=g, device="cuda") * ch
        if big:
            kv[::7] *= big
        pool.append(layer, m, kv[:, :H], kv[:, H:], i32([b for b, _ in at]), i32([t for _, t in at]))
    q = (torch.randn(B, M, Hq, D, generator=g, device="cuda") * 2).bfloat16()
    for b in range(B):
        for j, (d, _) in enumerate(T.sets_of(parents[b])):
            if d < 0:
                q[b, j] = float("nan")
    assert nq.device_status() == 0
    return pool, m, q


def check(nq, pool, m, q, lens, parents, planes, layer=0, tables=None, **kw):
    scale = q.shape[-1] ** -0.5
    tree = nq.Tree(i32(parents), window=kw.get("window", 0))
    out = pool.attention(layer, m, q, i32(lens), planes, scale, tree=tree, **kw)
    assert nq.device_status() == 0
    table = m.table.cpu().numpy() if tables is None else tables
    kw = {k: v for k, v in kw.items() if k in ("softcap", "window", "slopes")}
    if kw.get("slopes") is not None:
        kw["slopes"] = kw["slopes"].cpu().numpy()
    ref, tol = T.tree_attention64(HostPool(pool), layer, table, q.float().nan_to_num(0).cpu().numpy(), lens, planes, scale, parents, **kw)
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    off = np.abs(got - ref)
    assert (off <= tol + 1e-30).all(), (off - tol).max()
    assert (got[(tol == 0).all(-1)] == 0).all()       # a node that sees nothing
    return out


GEO = [  # D, G, page, format
    (128, 128, 16, 0), (128, 64, 32, 0), (64, 64, 64, 0), (128, 128, 16, 1), (64, 64, 128, 1)]


@pytest.mark.parametrize("D,G,P,fmt", GEO)
@pytest.mark.parametrize("planes", [1, 2])
@pytest.mark.parametrize("M,Hq,H", [(1, 2, 2), (5, 2, 2), (8, 2, 1), (13, 1, 1), (16, 4, 4), (7, 6, 2), (33, 2, 2), (20, 7, 1), (40, 8, 2), (65, 5, 1), (150, 2, 1)])
def test_trees_over_ragged_sequences(nq, D, G, P, fmt, planes, M, Hq, H):
    """Lengths of none, less than the tree, the tree alone, and more; fans, chains, forests, unused nodes."""
    if fmt == 1 and planes == 1:
        pytest.skip("16-bit pages have one view")
    lens = [M + 37, 0, M, M + 1, max(0, M - 3), M + 130, M + 63]
    parents = T.trees(M + Hq, len(lens), M)
    pool, m, q = setup(nq, lens, parents, P, H, Hq, D, G, fmt, M + D)
    check(nq, pool, m, q, lens, parents, planes)


@pytest.mark.parametrize("D,G,P,fmt", GEO)
@pytest.mark.parametrize("M,Hq,H", [(6, 4, 2), (24, 2, 1), (40, 4, 2), (70, 4, 1)])
@pytest.mark.parametrize("cap,window,bias", [(20.0, 0, False), (0.0, 9, False), (0.0, 0, True), (15.0, 70, True), (0.0, 1, False), (0.0, 3, True)])
def test_caps_windows_and_biases_go_by_positions(nq, D, G, P, fmt, M, Hq, H, cap, window, bias):
    lens = [M + 150, M + 2, M - 1, M + 64]
    parents = T.trees(3 * M, len(lens), M)
    pool, m, q = setup(nq, lens, parents, P, H, Hq, D, G, fmt, M + D + window)
    slopes = torch.linspace(0.02, 0.7, Hq, device="cuda") if bias else None
    check(nq, pool, m, q, lens, parents, 2, softcap=cap, window=window, slopes=slopes)


@pytest.mark.parametrize("D,G,P,fmt", GEO)
@pytest.mark.parametrize("M,Hq,H", [(9, 1, 1), (16, 4, 2), (64, 4, 1)])
def test_long_sequences_are_cut_and_joined(nq, D, G, P, fmt, M, Hq, H):
    """Few segments of many steps: runs end inside them, and inside the tree's rows; rows of very unequal size."""
    lens = [2900, M + 2, 1411]
    parents = T.trees(M + 2, 3, M)
    pool, m, q = setup(nq, lens, parents, P, H, Hq, D, G, fmt, M, layers=2, layer=1, big=30.0)
    check(nq, pool, m, q, lens, parents, 2, layer=1)


@pytest.mark.parametrize("M,Hq,H,fmt", [(8, 2, 2, 0), (12, 4, 2, 0), (12, 8, 2, 0), (12, 4, 2, 1), (40, 8, 2, 0)])
def test_a_chain_is_causal_attention(nq, M, Hq, H, fmt):
    """A tree that is a chain gives attention()'s values, within both sides' bf16 and fp16 (bf16) probabilities: see attention64."""
    lens, parents = [M + 300, M, M + 17], [[j - 1 for j in range(M)]] * 3
    pool, m, q = setup(nq, lens, parents, 16, H, Hq, 128, 128, fmt, 5)
    for kw in (dict(), dict(window=40, softcap=30.0, slopes=torch.full((Hq,), 0.1, device="cuda"))):
        a = check(nq, pool, m, q, lens, parents, 2, **kw).double()
        b = pool.attention(0, m, q, i32(lens), 2, 128 ** -0.5, **kw).double()
        _, tol = T.tree_attention64(HostPool(pool), 0, m.table.cpu().numpy(), q.float().cpu().numpy(), lens, 2, 128 ** -0.5, parents,
                                    **{k: v.cpu().numpy() if k == "slopes" else v for k, v in kw.items()})
        assert ((a - b).abs().cpu().numpy() <= 2 * tol).all()


@pytest.mark.parametrize("M,Hq,H", [(6, 2, 1), (30, 4, 1), (50, 4, 1)])
@pytest.mark.parametrize("fmt", [0, 1])
def test_slots_strides_and_shared_sequences(nq, M, Hq, H, fmt):
    """Sequences by slot, one slot twice with different trees; queries that are columns of a wider tensor."""
    lens, parents = [M + 90, M + 20], T.trees(9, 2, M)
    pool, m, q = setup(nq, lens, [[-1] * M, [-1] * M], 32, H, Hq, 64, 64, fmt, 2)
    wide = torch.randn(3, M, Hq + 2, 64, device="cuda").bfloat16()
    slots, n = [1, 0, 1], [lens[1], lens[0], lens[1]]
    trees = [parents[0], parents[1], [j - 1 for j in range(M)]]
    qs = wide[:, :, 1:1 + Hq]
    a = check(nq, pool, m, qs, n, trees, 2, seqs=i32(slots), tables=m.table.cpu().numpy()[slots])
    b = pool.attention(0, m, qs.contiguous(), i32(n), 2, 64 ** -0.5, seqs=i32(slots), tree=nq.Tree(i32(trees)))
    assert torch.equal(a, b)


@pytest.mark.parametrize("fmt", [0, 1])
@pytest.mark.parametrize("Hq", [1, 4, 16])
def test_infinite_values_stay_with_who_sees_them(nq, fmt, Hq):
    """A V row that is infinite (16-bit pages) or a missing page reaches only the queries that see it."""
    M, D, P = 8, 64, 16
    parents, lens = [[-1, 0, 0, 1, 2, 2, 0, 6]], [16 + M]
    pool, m, q = setup(nq, lens, parents, P, 1, Hq, D, 64, fmt, 4)
    tree = nq.Tree(i32(parents))
    want = pool.attention(0, m, q, i32(lens), 2, 0.125, tree=tree)
    if fmt == 1:
        page = int(m.table[0, 1])
        v = pool.data.view(torch.bfloat16).view(pool.n_pages, 1, 1, 2, 16, D)
        v[page, 0, 0, 1, 2] = float("inf")     # node 2: seen by 2, 4 and 5
        got = pool.attention(0, m, q, i32(lens), 2, 0.125, tree=tree)
        for j in range(M):
            if j in (2, 4, 5):
                assert not torch.isfinite(got[0, j]).any()
            else:                               # summed in another order (2^-18 of the largest at most), then rounded to bf16
                a, b = got[0, j].double(), want[0, j].double()
                assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 2.0 ** -18 * b.abs().max()).all()
        v[page, 0, 0, 1, 2] = 0
    m.table[0, 1] = -1                          # all of the tree's rows lie there
    got = pool.attention(0, m, q, i32(lens), 2, 0.125, tree=tree)
    assert nq.device_status() == nq.NQ_DEV_BAD_PAGE and torch.isfinite(got).all()
    for j in range(1, M):                       # the committed rows alone are left: the same for every node with that query
        alone = pool.attention(0, m, q[:, j:j + 1].contiguous(), i32([16]), 2, 0.125).double()
        assert (got[:, j:j + 1].double() - alone).abs().max() <= 2.0 ** -6 * alone.abs().max()


@pytest.mark.parametrize("M,Hq,H", [(8, 2, 2), (20, 4, 2), (40, 4, 1)])
def test_streams_graphs_and_repetition(nq, M, Hq, H):
    lens, parents = [M + 700, M + 5, M + 90], T.trees(6, 3, M)
    pool, m, q = setup(nq, lens, parents, 16, H, Hq, 128, 128, 0, 9)
    n, tree = i32(lens), nq.Tree(i32(parents))
    call = lambda **kw: pool.attention(0, m, q, n, 2, 0.09, tree=tree, **kw)  # noqa: E731
    want = call()
    for _ in range(5):
        assert torch.equal(call(), want)
    side = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in side:                              # two calls at once
        s.wait_stream(torch.cuda.current_stream())
        got.append(call(stream=s))
    torch.cuda.synchronize()
    assert torch.equal(got[0], want) and torch.equal(got[1], want)
    out = torch.empty_like(want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t2 = nq.Tree(tree.parents)
        pool.attention(0, m, q, n, 2, 0.09, tree=t2, out=out)
    tree.parents.copy_(i32(T.trees(60, 3, M)))
    q.nan_to_num_(0.5)
    tree = nq.Tree(tree.parents)
    g.replay()
    new = call()
    seen = torch.isfinite(new) & torch.isfinite(out)   # rows that were unused before hold NaN for both
    assert torch.equal(out[seen], new[seen]) and torch.equal(torch.isfinite(out), torch.isfinite(new))


def test_refusals(nq):
    lens, parents = [20, 9], T.trees(6, 2, 6)
    pool, m, q = setup(nq, lens, parents, 16, 1, 2, 64, 64, 0, 1)
    n, tree = i32(lens), nq.Tree(i32(parents))
    with pytest.raises(ValueError):
        pool.attention(0, m, q[:, :5].contiguous(), n, 2, 0.1, tree=tree)
    with pytest.raises(ValueError):
        pool.attention(0, m, q[:1], n[:1], 2, 0.1, tree=tree)
    for kw in (dict(window=4), dict(scale=0.0), dict(planes=3), dict(softcap=-1.0)):
        a = dict(planes=2, scale=0.1)
        a.update(kw)
        with pytest.raises(nq.NQError) as e:
            pool.attention(0, m, q, n, tree=tree, **a)
        assert e.value.status == nq.NQ_ERR_ARG
    with pytest.raises(nq.NQError) as e:
        pool.attention(0, m, q, n, 2, 0.1, tree=tree, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == nq.NQ_ERR_WORKSPACE
    empty = nq.Tree(torch.empty(0, 6, dtype=torch.int32, device="cuda"))
    assert pool.attention(0, m, q[:0], n[:0], 2, 0.1, tree=empty).shape == (0, 6, 2, 64)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("planes", [1, 2])
@pytest.mark.parametrize("M,Hq", [(9, 1), (20, 1), (40, 1), (50, 3)])
@pytest.mark.parametrize("sizes", ["tiny", "large", "mixed", "mixed late", "zeros"])
def test_values_of_very_unequal_size(nq, D, planes, M, Hq, sizes):
    """V rows whose scales are near fp16's ends, span more than fp16's normal numbers within a step or from step to
    step, or are zero: the tensor-core kernel takes them as values relative to the step's largest, or as codes."""
    lens, parents = [M + 400, M + 70], T.trees(M, 2, M)
    pool, m, q = setup(nq, lens, parents, 16, 1, Hq, D, D, 0, M + D)
    g = torch.Generator(device="cuda").manual_seed(8)
    at = [(b, t) for b, n in enumerate(lens) for t in range(n) if t < n - M or T.sets_of(parents[b])[t - (n - M)][0] >= 0]
    kv = torch.randn(len(at), 2, D, generator=g, device="cuda")
    f = torch.ones(len(at), device="cuda")
    if sizes == "tiny":
        f *= 2e-5
    elif sizes == "large":
        f *= 5e4
    elif sizes == "mixed":
        f[::5], f[1::5], f[2::7] = 2e-4, 3e3, 1e-6
    elif sizes == "mixed late":
        f[:200], f[200:330], f[400:] = 1e-4, 1e2, 1e4
    else:
        f[::2] = 0
    kv[:, 1] *= f[:, None]
    pool.append(0, m, kv[:, :1], kv[:, 1:], i32([b for b, _ in at]), i32([t for _, t in at]))
    assert nq.device_status() == 0
    check(nq, pool, m, q, lens, parents, planes)


SIZES = [(5, 1), (14, 1), (20, 2), (20, 4), (40, 4)]            # nodes, query heads of one kv head: every kernel


@pytest.mark.parametrize("fmt,planes", [(0, 1), (0, 2), (1, 2)])
@pytest.mark.parametrize("M,Hq", SIZES)
def test_lengths_up_to_the_largest(nq, fmt, planes, M, Hq):
    """2^27 - 1 pages that are all one and the same: row t is row t mod 16, wherever the tree lies.  Lengths past
    2^31 - 4096 are clamped and reported."""
    W, P, D = (1 << 27) - 1, 16, 64
    parents = T.trees(4 * M, 1, M)
    assert all(p >= -1 for p in parents[0])
    pool, small, q = setup(nq, [P], [[-1] * M], P, 1, Hq, D, D, fmt, 12)
    g = torch.Generator(device="cuda").manual_seed(4)
    kv = torch.randn(P, 2, D, generator=g, device="cuda")
    pool.append(0, small, kv[:, :1], kv[:, 1:], i32([0] * P), torch.arange(P, device="cuda").int())
    one = int(small.table[0, 0])
    m = nq.PageMap(1, W, pool.n_pages, P, table=torch.full((1, W), one, dtype=torch.int32, device="cuda"))
    few, most = np.full((1, 24), one), 2 ** 31 - 4096
    tree = nq.Tree(i32(parents), window=70)
    for n in (most - 7, most - 64, most, most + 1, W * P - 9, 2 ** 31 - 1):
        n0 = 256 + min(n, most) % 16
        ref, tol = T.tree_attention64(HostPool(pool), 0, few, q.float().cpu().numpy(), [n0], planes, 0.125, parents, window=70)
        out = pool.attention(0, m, q, i32([n]), planes, 0.125, window=70, tree=tree).double().cpu().numpy()
        assert nq.device_status() == (nq.NQ_DEV_SEQ_FULL if n > most else 0)
        assert (np.abs(out - ref) <= tol).all()


@pytest.mark.parametrize("D,G,P,fmt", GEO)
@pytest.mark.parametrize("M,Hq", SIZES)
@pytest.mark.parametrize("window", [0, 50])
def test_pages_outside_the_pool_are_hidden(nq, D, G, P, fmt, M, Hq, window):
    """Their rows count as not there for every query, and nothing of another page takes their place."""
    lens = [5 * P + M, 3 * P + 1 + M, M, 7 * P + 3 + M]
    broken = [[0, 3], [1, 2], [0], [2, 4, 7]]
    parents = T.trees(5 * M, 4, M)
    pool, m, q = setup(nq, lens, parents, P, 1, Hq, D, G, fmt, M + P)
    table = m.table.cpu().numpy().copy()
    gone = [np.isin(np.arange(n) // P, broken[b]) for b, n in enumerate(lens)]
    ref, tol = T.tree_attention64(HostPool(pool), 0, table, q.float().nan_to_num(0).cpu().numpy(), lens, 2, 0.125, parents, window=window, gone=gone)
    tree = nq.Tree(i32(parents), window=window)
    for bad in (-1, pool.n_pages, 2 ** 31 - 1, -2 ** 31):
        for b, js in enumerate(broken):
            for j in js:
                m.table[b, j] = bad
        out = pool.attention(0, m, q, i32(lens), 2, 0.125, window=window, tree=tree).double().cpu().numpy()
        assert nq.device_status() == nq.NQ_DEV_BAD_PAGE
        assert (np.abs(out - ref) <= tol + 1e-30).all()


@pytest.mark.parametrize("M,Hq", SIZES)
def test_two_graphs_at_once(nq, M, Hq):
    """Captured on two streams and replayed together: each has a workspace of its own."""
    lens, parents = [M + 900, M + 40], T.trees(M, 2, M)
    pool, m, q = setup(nq, lens, parents, 16, 2, 2 * Hq, 128, 128, 0, 3)
    n, tree = i32(lens), nq.Tree(i32(parents))
    qs = [q, (q.float() * 0.5).bfloat16()]
    want = [pool.attention(0, m, x, n, 2, 0.09, tree=tree) for x in qs]
    outs, graphs = [torch.empty_like(q) for _ in qs], [torch.cuda.CUDAGraph() for _ in qs]
    for x, o, gr in zip(qs, outs, graphs):
        with torch.cuda.graph(gr):
            pool.attention(0, m, x, n, 2, 0.09, tree=tree, out=o)
    streams = [torch.cuda.Stream() for _ in qs]
    for _ in range(5):
        torch.cuda.synchronize()
        for s, gr in zip(streams, graphs):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
