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
