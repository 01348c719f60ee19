"""Root-mean-square norm with the residual's addition against 64 bits.

The sum s is one addition in fp32, rounded once more for bf16: exact to the bit.
Of y: the sum of squares adds at most 16 squares per thread and 5 + 5 levels of
trees, each off by 2^-24 of it, 26 2^-24 in all, which the root halves; the
division, eps, rsqrtf (2 steps of 2^-23), and two products add 8 2^-24: 21 2^-24 <
2^-19.  bf16 adds 2^-8.  The scale is max|y| / 127 within 2^-19 + 2^-24, and a code is
off from y / scale by half a step and by 127 times the two errors, 2^-18 each at most."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
E = 2.0 ** -19
TYPES = {"f": torch.float32, "b": torch.bfloat16}


def make(M, K, x, add, w, seed=0, spread=1.0):
    g = torch.Generator().manual_seed(seed + M * 7 + K)
    t = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    rows = torch.exp(spread * t(M, 1))
    d = lambda v, k: v.to(TYPES[k]).cuda() if k else None  # noqa: E731
    return d(t(M, K) * rows, x), d(t(M, K), add), d(1 + 0.3 * t(K), w)


def sum64(x, add):
    """The residual as it is kept, in 64 bits."""
    s = x if add is None else (x.float() + add.float()).to(x.dtype)
    return s


def norm64(s, w, eps):
    s = s.double()
    y = s / torch.sqrt(s.square().mean(-1, keepdim=True) + eps)
    return y if w is None else y * w.double()


def check(s, y, xq, sx, x, add, w, eps):
    want = sum64(x, add)
    assert torch.equal(s, want)
    ref = norm64(want, w, eps)
    if y is not None:
        off = (y.double() - ref).abs()
        assert (off <= (2.0 ** -8 + 2 * E) * ref.abs() + 1e-40).all()
    if xq is not None:
        z = ref.abs().amax(-1, keepdim=True) / 127
        assert ((sx.double() - z[:, 0]).abs() <= (E + 2.0 ** -23) * z[:, 0]).all()
        t = torch.where(z > 0, ref / z, 0)
        assert ((xq.double() - t).abs() <= 0.5 + 127 * 2.0 ** -17).all()
        assert (xq.abs().amax(-1) == torch.where(z[:, 0] > 0, 127, 0)).all()


@pytest.mark.parametrize("M,K", [(1, 8), (1, 64), (3, 1000), (5, 4096), (2, 8192), (7, 8200), (3, 16384), (500, 136), (305, 3584)])
@pytest.mark.parametrize("x,add,w", [("f", "f", "f"), ("f", "b", "b"), ("b", "f", "b"), ("b", "b", None), ("f", None, "f"), ("b", None, None)])
def test_against_64_bits(nq, M, K, x, add, w):
    X, A, W = make(M, K, x, add, w)
    keep = X.clone()
    s, y = nq.rms_norm(X, W, eps=1e-5, add=A)
    s2, xq, sx = nq.rms_norm(X, W, eps=1e-5, add=A, quantize=True)
    assert torch.equal(X, keep) and (s is X) == (A is None)
    check(s, y, xq, sx, X, A, W, 1e-5)
    assert torch.equal(s, s2) and nq.device_status() == 0


def test_rows_do_not_depend_on_the_batch(nq):
    X, A, W = make(400, 4096, "f", "f", "b")
    s, xq, sx = nq.rms_norm(X, W, add=A, quantize=True)
    y = nq.rms_norm(X, W, add=A)[1]
    for m in (0, 17, 399):
        s1, q1, z1 = nq.rms_norm(X[m:m + 1], W, add=A[m:m + 1], quantize=True)
        assert torch.equal(s1[0], s[m]) and torch.equal(q1[0], xq[m]) and torch.equal(z1[0], sx[m])
        assert torch.equal(nq.rms_norm(X[m:m + 1], W, add=A[m:m + 1])[1][0], y[m])


def test_strided_rows_and_in_place(nq):
    """Columns of a wider tensor, the sum written over the residual; the columns beside it stay."""
    X, A, W = make(9, 256, "b", "f", "f")
    wide, wa = torch.full((9, 512), 3.0, dtype=torch.bfloat16, device="cuda"), torch.randn(9, 264, device="cuda")
    wide[:, 64:320] = X
    wa[:, :256] = A
    x = wide[:, 64:320]
    s, y = nq.rms_norm(x, W, add=wa[:, :256], sum_out=x)
    assert s.data_ptr() == x.data_ptr()
    check(s.contiguous(), y, None, None, X, A, W, 1e-6)
    assert (wide[:, :64] == 3).all() and (wide[:, 320:] == 3).all()


def test_zero_rows_tiny_and_large_values(nq):
    X = torch.zeros(5, 512, device="cuda")
    X[1] = 1e-30                     # under eps: y = x / sqrt(eps)
    X[2] = torch.randn(512, device="cuda") * 1e15
    X[3, 7] = 5.0
    X[4] = -1e-42                    # below the normal numbers
    s, xq, sx = nq.rms_norm(X, None, eps=1e-6, quantize=True)
    y = nq.rms_norm(X, None, eps=1e-6)[1]
    assert nq.device_status() == 0
    assert (xq[0] == 0).all() and sx[0] == 0 and (y[0] == 0).all()
    ref = norm64(X[1:4], None, 1e-6)
    assert ((y[1:4].double() - ref).abs() <= (2.0 ** -8 + 2 * E) * ref.abs()).all()
    z = ref.abs().amax(-1) / 127
    assert ((sx[1:4].double() - z).abs() <= (E + 2.0 ** -23) * z).all()
    assert xq[3, 7] == 127 and xq[3].abs().sum() == 127
    assert (xq[4] <= 0).all()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 3e38])
def test_rows_that_are_not_finite_are_reported(nq, bad):
    X, A, W = make(4, 512, "f", "f", "f")
    X[2, 511] = bad
    s, xq, sx = nq.rms_norm(X, W, add=A, quantize=True)
    assert nq.device_status() == nq.NQ_DEV_NONFINITE
    assert (xq[2] == 0).all() and sx[2] == 0
    keep = [0, 1, 3]
    check(s[keep], None, xq[keep], sx[keep], X[keep], A[keep], W, 1e-6)
    W2 = W.clone()
    W2[5] = bad if bad != 3e38 else float("inf")
    X[2, 511] = 1.0
    _, xq, sx = nq.rms_norm(X, W2, add=A, quantize=True)
    assert nq.device_status() == nq.NQ_DEV_NONFINITE and (xq == 0).all() and (sx == 0).all()


def test_graph_stream_and_empty(nq):
    X, A, W = make(33, 1024, "f", "f", "f")
    want = nq.rms_norm(X, W, add=A, quantize=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = nq.rms_norm(X, W, add=A, quantize=True, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = torch.empty_like(X), torch.empty(33, 1024, dtype=torch.int8, device="cuda"), torch.empty(33, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        nq.rms_norm(X, W, add=A, quantize=True, sum_out=out[0], xq=out[1], sx=out[2])
    A.mul_(2)
    g.replay()
    want = nq.rms_norm(X, W, add=A, quantize=True)
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert nq.rms_norm(X[:0], W, add=A[:0])[1].shape == (0, 1024)


def test_refusals(nq):
    X, A, W = make(4, 512, "f", "f", "f")
    for args, kw in [((X[0], W), {}), ((X.half(), W), {}), ((X, W[:8]), {}), ((X, W.half()), {}), ((X, W), dict(add=A[:3])),
                     ((X, W), dict(sum_out=X)), ((X, W), dict(add=A, sum_out=A.bfloat16())), ((X.T, None), {}),
                     ((X, W), dict(xq=torch.empty(4, 512, dtype=torch.int8, device="cuda"))),
                     ((X, W), dict(y=torch.empty(4, 256, dtype=torch.bfloat16, device="cuda"))),
                     ((X, W), dict(quantize=True, sx=torch.empty(3, device="cuda")))]:
        with pytest.raises(ValueError):
            nq.rms_norm(*args, **kw)
    for x, kw, status in [(X[:, :4], {}, nq.NQ_ERR_SHAPE), (torch.zeros(1, 16392, device="cuda"), {}, nq.NQ_ERR_SHAPE),
                          (torch.zeros(4, 68, device="cuda")[:, :64], {}, nq.NQ_ERR_SHAPE), (X, dict(eps=0.0), nq.NQ_ERR_ARG),
                          (X, dict(eps=float("nan")), nq.NQ_ERR_ARG), (torch.zeros(4, 516, device="cuda")[:, 1:513], {}, nq.NQ_ERR_SHAPE)]:
        with pytest.raises(nq.NQError) as e:
            nq.rms_norm(x, **kw)
        assert e.value.status == status
    assert nq.device_status() == 0


def test_feeds_the_int8_linear(nq):
    """The codes go into LinearA8Batch: y = W (codes sx) within what the linear itself allows (1e-5 of its largest)."""
    X, A, W = make(9, 512, "f", "f", "f")
    w = torch.randn(320, 512, device="cuda") * 0.05
    lin = nq.pack_weights(w, nq.FMT_NESTED44, 128)
    _, xq, sx = nq.rms_norm(X, W, add=A, quantize=True)
    y = nq.linear_a8(lin, xq, sx, True).double()
    s = lin.scales.view(torch.float16).view(320, 4).double().repeat_interleave(128, 1) / 16
    nib = lambda t: torch.stack([t & 15, t >> 4], -1).view(320, 512).int()  # noqa: E731
    signed = lambda v: torch.where(v > 7, v - 16, v).double()  # noqa: E731
    full = s * (16 * signed(nib(lin.base.view(320, 256))) + signed(nib(lin.resid.view(320, 256))))
    ref = (xq.double() * sx.double()[:, None]) @ full.T
    assert (y - ref).abs().max() <= 1e-5 * ref.abs().max()
