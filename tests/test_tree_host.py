"""Refusals of the tree, norm and keep calls without a GPU: each is rejected on
the host before any CUDA call, and no pointer is dereferenced."""
import ctypes as C

import pytest


@pytest.fixture(scope="module")
def nq():
    from quantized_self_speculative_gb300 import build, nq
    build.build()
    nq.lib()
    return nq


P = 4096          # an address that nothing reads


def norm(nq, x=P, xt=0, xs=64, add=None, at=0, as_=64, w=None, wt=0, eps=1e-6, M=1, K=64, s=None, ss=64, y=P, xq=None, sx=None):
    return nq.lib().nq_rms_norm(x, xt, xs, add, at, as_, w, wt, eps, M, K, s, ss, y, xq, sx, None)


def test_norm(nq):
    A, S, L = nq.NQ_ERR_ARG, nq.NQ_ERR_SHAPE, nq.NQ_ERR_ALIGN
    for kw, st in [(dict(x=None), A), (dict(M=0), A), (dict(K=0), A), (dict(xt=2), A), (dict(eps=0.0), A), (dict(eps=-1.0), A),
                   (dict(eps=float("inf")), A), (dict(add=P), A), (dict(s=P), A), (dict(add=P, s=P, at=5), A), (dict(w=P, wt=-1), A),
                   (dict(y=None), A), (dict(xq=P), A), (dict(sx=P), A), (dict(K=68, xs=72), S), (dict(K=16392, xs=16392), S), (dict(xs=56), S),
                   (dict(xs=68), S), (dict(add=P, s=P, as_=8), S), (dict(add=P, s=P, ss=8), S), (dict(x=P + 8), L), (dict(w=P + 8), L),
                   (dict(add=P + 4, s=P), L), (dict(add=P, s=P + 8), L), (dict(y=P + 2), L), (dict(xq=P + 4, sx=P), L), (dict(xq=P, sx=P + 2), L)]:
        assert norm(nq, **kw) == st, kw


def tree(nq, batch=1, nodes=4, window=0, parents=P, depth=P, bits=P):
    return C.byref(nq.nq_tree(batch, nodes, window, 0, parents, depth, bits))


BAD_TREES = [(dict(batch=0), 1), (dict(nodes=0), 1), (dict(window=-1), 1), (dict(parents=None), 1), (dict(depth=None), 1),
             (dict(bits=None), 1), (dict(nodes=1025), 2), (dict(parents=P + 2), 3), (dict(depth=P + 1), 3), (dict(bits=P + 3), 3)]


def test_plan_and_acceptance(nq):
    L = nq.lib()
    for kw, st in BAD_TREES:
        assert L.nq_tree_plan(tree(nq, **kw), None) == st, kw
        assert L.spec_accept_tree(tree(nq, **kw), P, P, 100, 4, P, P, P, None) == st, kw
    assert L.nq_tree_plan(None, None) == nq.NQ_ERR_ARG
    good = [P, P, 100, 4, P, P, P]
    for i, v, st in [(0, None, 1), (1, None, 1), (2, 0, 1), (2, 524289, 1), (3, 0, 1), (3, 5, 1), (4, None, 1), (5, None, 1), (6, None, 1),
                     (0, P + 2, 3), (1, P + 8, 3), (4, P + 1, 3), (5, P + 2, 3), (6, P + 3, 3)]:
        a = list(good)
        a[i] = v
        assert L.spec_accept_tree(tree(nq), *a, None) == st, (i, v)
    assert L.spec_accept_tree(tree(nq, batch=65536), *good, None) == nq.NQ_ERR_SHAPE


def pool_map(nq, fmt=0, D=128, page=16, map_page=16, n=4, data=P, table=P):
    return (C.byref(nq.nq_page_pool(1, 4, page, 2, D, 128, fmt, 0, data)), C.byref(nq.nq_page_map(2, 4, n, map_page, table, None, None)))


def test_keep(nq):
    L = nq.lib()
    good = [P, P, P, P, 1, 3]
    for i, v, st in [(0, None, 1), (1, None, 1), (2, None, 1), (3, None, 1), (4, 0, 1), (5, 0, 1), (0, P + 2, 3), (1, P + 1, 3), (2, P + 2, 3), (3, P + 3, 3)]:
        a = list(good)
        a[i] = v
        assert L.nq_page_keep(*pool_map(nq), *a, None) == st, (i, v)
    for kw, st in [(dict(map_page=32), 2), (dict(n=5), 2), (dict(D=96), 2), (dict(data=None), 1), (dict(table=None), 1), (dict(fmt=7), 1), (dict(data=P + 8), 3)]:
        assert L.nq_page_keep(*pool_map(nq, **kw), *good, None) == st, kw


def test_append_at(nq):
    L = nq.lib()
    good = [None, None, P, P, 0, 256, P, P, P, 1, 0, None]           # rope, q, k, v, dtype, stride, seqs, rows, at, T, heads_q, q_out
    for i, v, st in [(2, None, 1), (6, None, 1), (7, None, 1), (8, None, 1), (9, 0, 1), (8, P + 2, 3), (5, 8, 2)]:
        a = list(good)
        a[i] = v
        assert L.nq_page_append_at(pool_map(nq)[0], 0, pool_map(nq)[1], *a, None) == st, (i, v)


def test_attention(nq):
    L = nq.lib()
    opts = lambda **kw: C.byref(nq.nq_attn_opts(*{**dict(scale=0.1, softcap=0.0, window=0, pad=0, slopes=None), **kw}.values()))  # noqa: E731
    call = lambda t, q=P, stride=256, hq=2, seqs=None, lens=P, planes=2, o=None, out=P, ws=P, n=1 << 40, layer=0: L.nq_page_attn_tree(  # noqa: E731
        pool_map(nq)[0], layer, pool_map(nq)[1], q, stride, hq, seqs, lens, planes, o or opts(), t, out, ws, n, None)
    for kw, st in BAD_TREES:
        assert call(tree(nq, **kw)) == st, kw
    good = tree(nq)
    for kw, st in [(dict(q=None), 1), (dict(lens=None), 1), (dict(out=None), 1), (dict(hq=3), 1), (dict(hq=0), 1), (dict(planes=0), 1),
                   (dict(o=opts(scale=-1.0)), 1), (dict(o=opts(window=3)), 1), (dict(layer=1), 1), (dict(stride=128), 2), (dict(stride=260), 2),
                   (dict(q=P + 8), 3), (dict(seqs=P + 2), 3), (dict(ws=P + 4), 3)]:
        assert call(good, **kw) == st, kw
    assert call(tree(nq, batch=3)) == nq.NQ_ERR_ARG          # more sequences than slots
    assert call(tree(nq, window=3)) == nq.NQ_ERR_ARG         # another window than the plan's
    assert L.nq_page_attn_tree_workspace_bytes(1025, 8, 2, 128) == 0 and L.nq_page_attn_tree_workspace_bytes(4, 3, 2, 128) == 0
