"""Sizes, argument checks and rotation rates of the paged-cache calls: all of
it on the host, every rejected call before any CUDA call."""
import ctypes as C
import math

import numpy as np
import pytest

from paged_helpers import HostMap


@pytest.fixture(scope="module")
def nq():
    from quantized_self_speculative_gb300 import build, nq
    build.build()
    nq.lib()
    return nq


A = 1 << 20          # a 16-byte aligned address that no call dereferences


def pool(nq, **kw):
    d = dict(layers=2, n_pages=8, page_size=16, heads_kv=2, head_dim=128, group=128, format=nq.KV_NESTED44, pad=0, data=A)
    d.update(kw)
    return C.byref(nq.nq_page_pool(*d.values()))


def pmap(nq, **kw):
    d = dict(max_seqs=4, max_pages=6, n_pages=8, page_size=16, table=A, held=A, ref=A)
    d.update(kw)
    return C.byref(nq.nq_page_map(*d.values()))


def test_pool_bytes(nq):
    n = C.c_size_t()
    f = nq.lib().nq_page_pool_bytes
    # a nested row and head: D/2 bytes in each of 4 planes, 2 fp16 scales per group
    assert f(3, 10, 32, 4, 128, 64, nq.KV_NESTED44, C.byref(n)) == 0 and n.value == 3 * 10 * 4 * 32 * (4 * 64 + 8)
    assert f(1, 1, 16, 1, 64, 64, nq.KV_NESTED44, C.byref(n)) == 0 and n.value == 16 * (4 * 32 + 4)
    assert f(2, 5, 64, 3, 64, 0, nq.KV_BF16, C.byref(n)) == 0 and n.value == 2 * 5 * 3 * 64 * 256
    big = f(80, 1 << 20, 256, 64, 128, 128, nq.KV_BF16, C.byref(n))
    assert big == 0 and n.value == 80 * (1 << 20) * 64 * 256 * 512         # past 2^32
    for args, st in [((0, 1, 16, 1, 128, 128, 0), nq.NQ_ERR_ARG), ((1, 0, 16, 1, 128, 128, 0), nq.NQ_ERR_ARG),
                     ((1, 1, 16, 0, 128, 128, 0), nq.NQ_ERR_ARG), ((1, 1, 16, 1, 128, 128, 2), nq.NQ_ERR_ARG),
                     ((1, 1, 24, 1, 128, 128, 0), nq.NQ_ERR_SHAPE), ((1, 1, 16, 1, 96, 96, 0), nq.NQ_ERR_SHAPE),
                     ((1, 1, 16, 1, 64, 128, 0), nq.NQ_ERR_SHAPE), ((1, 1, 16, 1, 128, 32, 0), nq.NQ_ERR_SHAPE)]:
        assert f(*args, C.byref(n)) == st, args
    assert f(1, 1, 16, 1, 128, 128, 0, None) == nq.NQ_ERR_ARG


def test_workspace_bytes(nq):
    f = nq.lib().nq_page_workspace_bytes
    assert f(pmap(nq), 4) >= 4 * (3 * 8 + 5 * 4) and f(pmap(nq, max_pages=1000), 4) >= 4 * 4 * 1002
    assert f(pmap(nq), 0) == 0 and f(pmap(nq), 5) == 0 and f(pmap(nq, table=None), 1) == 0
    g = nq.lib().nq_page_attn_workspace_bytes
    assert g(1, 8, 2, 128) > 0
    for bad in [(0, 8, 2, 128), (1, 8, 3, 128), (1, 1, 2, 128), (1, 8, 2, 96), (1, 8, 0, 64)]:
        assert g(*bad) == 0


@pytest.mark.parametrize("rot,scaling,factor,old", [(128, "none", 1.0, 0), (8, "ntk", 4.0, 0), (64, "linear", 8.0, 0),
                                                   (120, "parts", 16.0, 4096)])
def test_rates(nq, rot, scaling, factor, old):
    theta = 500000.0
    rates = np.zeros(rot // 2, np.uint64)
    ms = C.c_float()
    kind = ("none", "linear", "ntk", "parts").index(scaling)
    assert nq.lib().nq_rope_rates(rot, theta, kind, factor, old, rates.ctypes.data, C.byref(ms)) == 0
    want = np.arange(rot // 2, dtype=np.float64)
    base = theta * factor ** (rot / (rot - 2)) if scaling == "ntk" else theta
    w = base ** (-2 * want / rot)
    if scaling == "linear":
        w /= factor
    if scaling == "parts":
        keep = np.clip((old * w / (2 * math.pi) - 1) / 31, 0, 1)
        assert keep.min() == 0 and keep.max() == 1
        w = w * keep + w / factor * (1 - keep)
        assert ms.value == np.float32(0.1 * math.log(factor) + 1)
    else:
        assert ms.value == 1.0
    # a few roundings of 64-bit arithmetic, and the rounding to a whole number of 2^-64 turns
    turns = w / (2 * math.pi) * 2.0 ** 64
    assert (np.abs(rates.astype(np.float64) - turns) <= 0.5 + 8 * 2.0 ** -53 * turns).all()


def test_rates_refusals(nq):
    r, ms = np.zeros(64, np.uint64), C.c_float()
    f = nq.lib().nq_rope_rates
    ok = (64, 10000.0, 0, 1.0, 0, r.ctypes.data, C.byref(ms))
    assert f(*ok) == 0
    for i, bad, st in [(0, 4, nq.NQ_ERR_SHAPE), (0, 12, nq.NQ_ERR_SHAPE), (0, 136, nq.NQ_ERR_SHAPE), (1, 1.0, nq.NQ_ERR_ARG),
                       (1, math.inf, nq.NQ_ERR_ARG), (1, math.nan, nq.NQ_ERR_ARG), (2, 4, nq.NQ_ERR_ARG), (2, -1, nq.NQ_ERR_ARG),
                       (5, None, nq.NQ_ERR_ARG), (6, None, nq.NQ_ERR_ARG)]:
        a = list(ok)
        a[i] = bad
        assert f(*a) == st, (i, bad)
    assert f(64, 10000.0, 1, 0.5, 0, r.ctypes.data, C.byref(ms)) == nq.NQ_ERR_ARG
    assert f(64, 10000.0, 3, 2.0, 0, r.ctypes.data, C.byref(ms)) == nq.NQ_ERR_ARG


def test_rope_refusals(nq):
    plan = lambda **kw: C.byref(nq.nq_rope_plan(*{**dict(rot_dim=64, layout=0, mscale=1.0, pad=0, rates=A), **kw}.values()))  # noqa: E731
    ok = dict(plan=plan(), x=A, xt=0, xs=256, pos=A, T=3, H=2, D=128, inv=0, out=A * 2, ot=1, os=256, stream=None)
    f = lambda **kw: nq.lib().nq_rope(*{**ok, **kw}.values())  # noqa: E731
    ARG, SHAPE, ALIGN = nq.NQ_ERR_ARG, nq.NQ_ERR_SHAPE, nq.NQ_ERR_ALIGN
    for kw, st in [(dict(x=None), ARG), (dict(pos=None), ARG), (dict(out=None), ARG), (dict(T=0), ARG), (dict(H=0), ARG),
                   (dict(xt=2), ARG), (dict(ot=-1), ARG), (dict(D=96), SHAPE), (dict(xs=255), SHAPE), (dict(xs=260), SHAPE),
                   (dict(os=128), SHAPE), (dict(x=A + 8), ALIGN), (dict(out=A + 4), ALIGN), (dict(pos=A + 2), ALIGN),
                   (dict(plan=None), ARG), (dict(plan=plan(rates=None)), ARG), (dict(plan=plan(layout=2)), ARG),
                   (dict(plan=plan(rot_dim=132)), SHAPE), (dict(plan=plan(rot_dim=136)), SHAPE), (dict(plan=plan(rates=A + 8)), ALIGN),
                   (dict(out=A, ot=1), ARG), (dict(out=A, ot=0, os=512), ARG)]:
        assert f(**kw) == st, kw


def test_map_refusals(nq):
    ARG, SHAPE, ALIGN, WS = nq.NQ_ERR_ARG, nq.NQ_ERR_SHAPE, nq.NQ_ERR_ALIGN, nq.NQ_ERR_WORKSPACE
    L, big = nq.lib(), 1 << 20
    maps = [(dict(max_seqs=0), ARG), (dict(max_pages=0), ARG), (dict(table=None), ARG), (dict(held=None), ARG),
            (dict(ref=None), ARG), (dict(page_size=48), SHAPE), (dict(max_pages=1 << 30), SHAPE), (dict(table=A + 2), ALIGN)]
    for kw, st in maps:
        m = pmap(nq, **kw)
        assert L.nq_page_map_init(m, None) == st, kw
        assert L.nq_page_truncate(m, A, A, 1, None) == st, kw
        assert L.nq_page_fork(m, A, A, A, 1, A, big, None) == st, kw
        assert L.nq_page_reserve(m, None, A, A, A, 1, None, A, big, None) == st, kw
    m, p = pmap(nq), pool(nq)
    for args, st in [((m, None, A, A, 1, A, big, None), ARG), ((m, A, A, A, 0, A, big, None), ARG),
                     ((m, A, A, A, 5, A, big, None), ARG), ((m, A, A, A, 1, None, big, None), WS),
                     ((m, A, A, A, 1, A, 8, None), WS), ((m, A, A, A, 1, A + 4, big, None), ALIGN),
                     ((m, A + 1, A, A, 1, A, big, None), ALIGN)]:
        assert L.nq_page_fork(*args) == st
        assert L.nq_page_reserve(args[0], None, *args[1:5], None, *args[5:]) == st
    assert L.nq_page_truncate(m, None, A, 1, None) == ARG and L.nq_page_truncate(m, A, A, 9, None) == ARG
    # a pool that is not the map's
    for kw, st in [(dict(n_pages=9), SHAPE), (dict(page_size=32), SHAPE), (dict(data=None), ARG), (dict(data=A + 8), ALIGN)]:
        q = pool(nq, **kw)
        assert L.nq_page_reserve(m, q, A, A, A, 1, None, A, big, None) == st
        assert L.nq_page_compact(m, q, A, A, big, None) == st
    assert L.nq_page_compact(m, None, A, A, big, None) == ARG and L.nq_page_compact(m, p, None, A, big, None) == ARG
    assert L.nq_page_compact(m, p, A, A, 8, None) == WS
    assert L.nq_page_copy(p, None, A, 1, None) == ARG and L.nq_page_copy(p, A, A, 0, None) == ARG
    assert L.nq_page_copy(p, A + 2, A, 1, None) == ALIGN


def test_append_read_refusals(nq):
    ARG, SHAPE, ALIGN = nq.NQ_ERR_ARG, nq.NQ_ERR_SHAPE, nq.NQ_ERR_ALIGN
    plan = C.byref(nq.nq_rope_plan(128, 0, 1.0, 0, A))
    ok = dict(pool=pool(nq), layer=1, m=pmap(nq, held=None, ref=None), rope=plan, q=A, k=A, v=A, dt=0, stride=1024, seqs=A,
              pos=A, T=3, Hq=4, out=A, stream=None)
    f = lambda **kw: nq.lib().nq_page_append(*{**ok, **kw}.values())  # noqa: E731
    for kw, st in [(dict(layer=2), ARG), (dict(layer=-1), ARG), (dict(k=None), ARG), (dict(v=None), ARG), (dict(seqs=None), ARG),
                   (dict(T=0), ARG), (dict(dt=2), ARG), (dict(out=None), ARG), (dict(q=None), ARG), (dict(q=None, Hq=0), ARG),
                   (dict(Hq=0), ARG), (dict(stride=504), SHAPE), (dict(stride=1025), SHAPE), (dict(k=A + 4), ALIGN),
                   (dict(q=A + 8), ALIGN), (dict(pos=A + 1), ALIGN), (dict(pool=pool(nq, page_size=64)), SHAPE),
                   (dict(rope=C.byref(nq.nq_rope_plan(128, 3, 1.0, 0, A))), ARG)]:
        assert f(**kw) == st, kw
    assert f(pool=pool(nq, head_dim=64, group=64)) == SHAPE       # 128 rotated values of a head of 64
    ok2 = dict(pool=pool(nq), layer=0, m=pmap(nq), seqs=A, pos=A, T=1, planes=2, k=A, v=A, stream=None)
    g = lambda **kw: nq.lib().nq_page_read(*{**ok2, **kw}.values())  # noqa: E731
    for kw, st in [(dict(planes=3), ARG), (dict(T=0), ARG), (dict(k=None), ARG), (dict(layer=5), ARG), (dict(v=A + 2), ALIGN)]:
        assert g(**kw) == st, kw


def test_attn_refusals(nq):
    ARG, SHAPE, ALIGN, WS = nq.NQ_ERR_ARG, nq.NQ_ERR_SHAPE, nq.NQ_ERR_ALIGN, nq.NQ_ERR_WORKSPACE
    o = lambda scale=0.1, cap=0.0, window=0, slopes=None: C.byref(nq.nq_attn_opts(scale, cap, window, 0, slopes))  # noqa: E731
    ok = dict(pool=pool(nq), layer=0, m=pmap(nq), q=A, qs=4 * 128, B=3, M=2, Hq=4, seqs=None, len=A, planes=1, o=o(), out=A,
              ws=A, wsb=1 << 40, stream=None)
    f = lambda **kw: nq.lib().nq_page_attn(*{**ok, **kw}.values())  # noqa: E731
    for kw, st in [(dict(q=None), ARG), (dict(len=None), ARG), (dict(out=None), ARG), (dict(o=None), ARG), (dict(B=0), ARG),
                   (dict(B=5), ARG), (dict(M=0), ARG), (dict(Hq=3), ARG), (dict(Hq=1), ARG), (dict(planes=0), ARG), (dict(layer=2), ARG),
                   (dict(o=o(scale=0.0)), ARG), (dict(o=o(scale=math.nan)), ARG), (dict(o=o(cap=-1.0)), ARG),
                   (dict(o=o(cap=math.nan)), ARG), (dict(o=o(window=-1)), ARG), (dict(qs=500), SHAPE), (dict(qs=513), SHAPE),
                   (dict(q=A + 2), ALIGN), (dict(out=A + 8), ALIGN), (dict(len=A + 2), ALIGN), (dict(o=o(slopes=A + 2)), ALIGN),
                   (dict(ws=None), WS), (dict(wsb=4), WS), (dict(m=pmap(nq, n_pages=7)), SHAPE)]:
        assert f(**kw) == st, kw


def test_host_map_model():
    """The sequential model that the GPU tests compare with, on a case worked by hand."""
    m = HostMap(4, 4, 8, 16)
    assert m.reserve([0], [0], [40]) == ([1], []) and m.pages[0] == [0, 1, 2]
    m.fork([0, 0], [1, 2], [40, 20])
    assert m.pages[1] == [0, 1, 2] and m.pages[2] == [0, 1] and m.ref[:3] == [3, 3, 2]
    # both holders of page 2 ask: the first is copied, the last keeps it
    assert m.reserve([0, 1], [40, 40], [41, 41]) == ([1, 1], [(2, 3)])
    assert m.pages[0] == [0, 1, 3] and m.pages[1] == [0, 1, 2] and m.ref[:4] == [3, 3, 1, 1]
    # slot 2 writes on page 1 that it shares with two others
    assert m.reserve([2], [20], [64])[1] == [(1, 4)] and m.pages[2] == [0, 4, 5, 6]
    # one page is free: the first request takes it, the second and all after it get none
    assert m.reserve([0, 1, 3], [48, 48, 0], [49, 49, 1])[0] == [1, 0, 0]
    m.truncate([0, 2], [16, 0])
    assert m.pages[0] == [0] and m.pages[2] == [] and m.ref == [2, 1, 1, 0, 0, 0, 0, 0]
