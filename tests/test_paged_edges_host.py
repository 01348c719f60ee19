"""Refusals of the paged-cache calls beyond their plain arguments, before any CUDA call."""
import ctypes as C
import math

import pytest

from test_paged_host import A, nq, pmap, pool  # noqa: F401


def test_starved_attention_refusals(nq):  # noqa: F811
    opts = C.byref(nq.nq_attn_opts(0.1, 0.0, 0, 0, None))
    f = lambda steps, us, B=3: nq.lib().nq_selftest_page_attn(pool(nq), 0, pmap(nq), A, 512, B, 2, 4, None, A, 1, opts, A, A, 1 << 40,   # noqa: E731
                                                             steps, us, None)
    assert f(-1, 10) == nq.NQ_ERR_ARG and f(0, 0) == nq.NQ_ERR_ARG and f(0, 1000001) == nq.NQ_ERR_ARG
    assert f(0, 10, 0) == nq.NQ_ERR_ARG


def test_scales_and_caps_that_are_not_finite(nq):  # noqa: F811
    def call(scale=0.1, cap=0.0):
        o = C.byref(nq.nq_attn_opts(scale, cap, 0, 0, None))
        return nq.lib().nq_page_attn(pool(nq), 0, pmap(nq), A, 512, 3, 2, 4, None, A, 1, o, A, A, 4, None)
    assert call() == call(cap=2.0 ** 100) == call(cap=2.0 ** -100) == nq.NQ_ERR_WORKSPACE       # all else is in order
    for bad in (math.inf, math.nan, 0.0, -1.0):
        assert call(scale=bad) == nq.NQ_ERR_ARG
    for bad in (math.inf, math.nan, -1.0, 2.0 ** 101, 2.0 ** -101):
        assert call(cap=bad) == nq.NQ_ERR_ARG
