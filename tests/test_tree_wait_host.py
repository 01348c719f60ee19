"""Refusals of the diagnostic of starved tree attention, before any CUDA call."""
import ctypes as C

from test_tree_host import BAD_TREES, P, nq, pool_map, tree  # noqa: F401


def test_starved_attention_of_trees(nq):  # noqa: F811
    opts = C.byref(nq.nq_attn_opts(0.1, 0.0, 0, 0, None))
    pool, pmap = pool_map(nq)
    f = lambda steps, us, t=None, n=1 << 40: nq.lib().nq_selftest_page_attn_tree(  # noqa: E731
        pool, 0, pmap, P, 256, 2, None, P, 2, opts, t or tree(nq), P, P, n, steps, us, None)
    assert f(-1, 10) == f(0, 0) == f(0, 1000001) == nq.NQ_ERR_ARG
    assert f(0, 10, n=16) == nq.NQ_ERR_WORKSPACE
    for kw, st in BAD_TREES:
        assert f(0, 10, tree(nq, **kw)) == st, kw
