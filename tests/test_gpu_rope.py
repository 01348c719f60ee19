"""Rotary positions on the GPU against the formula in 64 bits."""
import numpy as np
import pytest
import torch

from paged_helpers import turned64

pytestmark = pytest.mark.gpu


def data(seed, T, H, D, dtype, pad=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H + pad, D, generator=g).to(dtype).cuda()
    return x[:, :H]


def close(y, ref, amp, x, rot, layout, dtype):
    """sin and cos: 2 ulp each, and 2^-25 half turns of angle (pi 2^-25); one rounding of the factor (and of it in 32
    bits), of the product and of the sum: 7 steps of 2^-24 on each term.  Then half a step of the output's type."""
    x = np.abs(np.asarray(x.double().cpu()))
    near = np.zeros_like(x)
    for i in range(rot // 2):
        u, v = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
        near[..., u] = near[..., v] = x[..., u] + x[..., v]
    tol = 7 * 2.0 ** -24 * amp * near + (torch.finfo(dtype).eps / 2) * np.abs(ref) * (1 + 2.0 ** -20)
    return (np.abs(y.double().cpu().numpy() - ref) <= tol).all()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("D,rot,scaling,factor", [(128, 128, "none", 1.0), (128, 64, "linear", 8.0), (128, 72, "ntk", 4.0),
                                                  (64, 64, "parts", 16.0), (64, 8, "none", 1.0), (128, 120, "parts", 2.0)])
@pytest.mark.parametrize("src,dst", [("float32", "float32"), ("float32", "bfloat16"), ("bfloat16", "bfloat16"),
                                     ("bfloat16", "float32")])
def test_matches_formula(nq, layout, D, rot, scaling, factor, src, dst):
    src, dst = getattr(torch, src), getattr(torch, dst)
    for T, H, top in ((1, 1, 9), (7, 5, 5000), (131, 9, 2 ** 24)):
        x = data(T + rot, T, H, D, src, pad=2)
        pos = torch.randint(0, top, (T,), dtype=torch.int32)
        pos[0] = top - 1 if T > 1 else 0
        plan = nq.Rope(rot, theta=500000.0, layout=layout, scaling=scaling, factor=factor, old_len=4096)
        for inverse in (False, True):
            y = nq.rope(x, pos.cuda(), plan, inverse=inverse, out_dtype=dst)
            ref, amp = turned64(x.double().cpu(), pos, rot, 500000.0, layout, scaling, factor, 4096, inverse)
            assert close(y, ref, amp, x, rot, layout, dst)


def test_far_positions_exact(nq):
    """A rate of an exact fraction of a turn keeps its angles at any position:
    with rate 2^61 (an eighth of a turn) position 8 n + j turns by j / 8."""
    plan = nq.Rope(64)
    plan.rates.fill_(2 ** 61)
    x = data(3, 8, 2, 64, torch.float32)
    near = torch.arange(8, dtype=torch.int32, device="cuda")
    far = (2 ** 31 - 16) + near
    assert torch.equal(nq.rope(x, near, plan), nq.rope(x, far.int(), plan))


def test_in_place_inverse_and_gradient(nq):
    x = data(5, 33, 6, 128, torch.float32)
    x = x.contiguous()
    pos = torch.arange(33, dtype=torch.int32, device="cuda") * 117
    plan = nq.Rope(128, layout="half")
    y = nq.rope(x, pos, plan)
    z = x.clone()
    assert nq.rope(z, pos, plan, out=z) is z and torch.equal(z, y)
    back = nq.rope(y, pos, plan, inverse=True)
    # two rotations, each within 7 steps of the pair's magnitude
    assert (back - x).abs().max() <= 2 * 7 * 2.0 ** -24 * 2 * x.abs().max()
    # d<y, w>/dx is the rotation of w back: against central differences of the linear map (step 1, sums in 64 bits)
    w = data(6, 33, 6, 128, torch.float32).contiguous()
    grad = nq.rope(w, pos, plan, inverse=True)
    for t, h, i in ((0, 0, 0), (1, 5, 63), (32, 2, 64), (17, 3, 127)):
        d = torch.zeros_like(x)
        d[t, h, i] = 1.0
        diff = ((nq.rope(x + d, pos, plan).double() - nq.rope(x - d, pos, plan).double()) * w.double()).sum() / 2
        # each of the four rotated values of a pair is off by 7 steps of |x1| + |x2| + 1
        tol = 4 * 7 * 2.0 ** -24 * (2 * x[t, h].abs().max() + 1) * w[t, h].abs().max()
        assert (diff - grad[t, h, i].double()).abs() <= tol


def test_empty_side_stream_and_refusals(nq):
    plan = nq.Rope(64)
    assert nq.rope(torch.empty(0, 3, 64, device="cuda"), torch.empty(0, dtype=torch.int32, device="cuda"), plan).shape == (0, 3, 64)
    x, pos = data(8, 50, 4, 64, torch.bfloat16), torch.arange(50, dtype=torch.int32, device="cuda")
    want = nq.rope(x, pos, plan)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = nq.rope(x, pos, plan, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    for bad in (lambda: nq.rope(x.half(), pos, plan), lambda: nq.rope(x, pos[:3], plan), lambda: nq.rope(x, pos.long(), plan),
                lambda: nq.rope(x.transpose(0, 1), pos, plan), lambda: nq.rope(x.cpu(), pos.cpu(), plan),
                lambda: nq.rope(x[..., ::2], pos, plan), lambda: nq.Rope(64, layout="other")):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(nq.NQError):
        nq.rope(x, pos, nq.Rope(128))
