"""Refusals of the paged-cache calls beyond their plain arguments, before any CUDA call."""
import ctypes as C
import math
from decimal import Decimal, localcontext

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


def test_rope_factor_in_two_parts(nq):  # noqa: F811
    hi, lo = C.c_float(), C.c_float()
    f = nq.lib().nq_rope_mscale
    for factor in (1.0, 1.5, 2.0, 8.0, 16.0, 40.0, 1e6):
        assert f(3, factor, C.byref(hi), C.byref(lo)) == 0
        with localcontext() as high:
            high.prec = 40
            exact = Decimal(factor).ln() / 10 + 1
        # both parts to half a step: 2^-24 of what is left beyond 2^-24; the logarithm, its product and the sum in 64 bits
        off = abs(Decimal(hi.value) + Decimal(lo.value) - exact)
        assert off <= exact * (Decimal(2) ** -48 + 3 * Decimal(2) ** -53) and abs(Decimal(hi.value) - exact) <= exact * Decimal(2) ** -24
    for kind in (0, 1, 2):
        assert f(kind, 4.0, C.byref(hi), C.byref(lo)) == 0 and hi.value == 1.0 and lo.value == 0.0
    for args in ((4, 2.0), (-1, 2.0), (3, 0.5), (3, math.inf), (3, math.nan)):
        assert f(*args, C.byref(hi), C.byref(lo)) == nq.NQ_ERR_ARG
    assert f(3, 2.0, None, C.byref(lo)) == nq.NQ_ERR_ARG and f(3, 2.0, C.byref(hi), None) == nq.NQ_ERR_ARG
