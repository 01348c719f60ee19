"""Sines of the rotation one by one, and keys against those rotated by 64-bit angles."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def angles(x):
    """sin, cos in extended precision of x / 2^64 turns (uint64): the nearest quarter turn taken off in integers."""
    k = (x + np.uint64(1 << 61)) >> np.uint64(62)
    rest = (x - (k << np.uint64(62))).view(np.int64).astype(np.longdouble)
    a = rest * (np.longdouble("6.28318530717958647692528676655900577") / np.longdouble(2.0) ** 64)
    s, c = np.sin(a), np.cos(a)
    k = (k % np.uint64(4)).astype(np.int64)
    return np.choose(k, [s, c, -s, -c]), np.choose(k, [c, -s, -c, s])


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("parts", 2.0), ("parts", 16.0)])
def test_sines_and_cosines(nq, layout, scaling, factor):
    """A pair (1, 0) turns into (m cos, m sin).  The rounded exact value in 996 of 1000 cases at least, else a step
    off.  The polynomials hold 32 bits, truncated a few times: 1.5 units of 2^-32 at most beside a value that one
    step of 2^-24 holds 256 times, and 0.3% were counted on the CPU with the same integers."""
    T, rot = 4000, 128
    r = np.random.default_rng(11)
    rates = r.integers(0, 1 << 64, rot // 2, dtype=np.uint64)
    rates[:6] = [0, 1, 1 << 61, (1 << 61) - 1, 1 << 62, 1 << 63]         # no turn, the least, eighths, a quarter, half
    plan = nq.Rope(rot, layout=layout, scaling=scaling, factor=factor, old_len=4096)
    plan.rates.copy_(torch.from_numpy(rates.view(np.int64)))
    pos = r.integers(0, 2 ** 31, T)
    pos[:40] = np.arange(40)
    x = torch.zeros(T, 1, rot, device="cuda")
    first, second = (slice(0, rot // 2), slice(rot // 2, rot)) if layout == "half" else (slice(0, rot, 2), slice(1, rot, 2))
    x[..., first] = 1.0
    y = nq.rope(x, torch.from_numpy(pos).int().cuda(), plan).cpu().numpy()[:, 0]
    with np.errstate(over="ignore"):
        sn, cs = angles(pos.astype(np.uint64)[:, None] * rates[None])
    m = np.longdouble(0.1 * math.log(factor) + 1.0 if scaling == "parts" else 1.0)
    for got, exact in ((y[:, first], m * cs), (y[:, second], m * sn)):
        want = exact.astype(np.float32)
        off = np.abs(got.astype(np.float64) - want) / np.spacing(np.abs(want)).astype(np.float64)
        off[want == 0] = np.abs(got[want == 0])
        assert off.max() <= 1.0, off.max()
        assert (off == 0).mean() >= 0.996, (off == 0).mean()


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("scaling,factor", [("none", 1.0), ("linear", 8.0), ("ntk", 4.0), ("parts", 16.0)])
def test_keys_and_their_codes_from_64_bit_angles(nq, layout, scaling, factor):
    """Keys equal those whose sines are rounded from 64-bit angles wherever both sines do: 992 of 1000.  The others
    are a step of a sine off; a code or scale of the cache changes with that once in some 10^7 values (a step is
    112 2^-24 of the width between two codes): at most 3 rows of some 15000."""
    T, H, D, P, theta, old = 4096, 4, 128, 256, 500000.0, 4096
    g = torch.Generator().manual_seed(12)
    k = (torch.randn(T, H, D, generator=g) * (1 + 3 * torch.rand(D, generator=g) ** 8)).cuda()
    pos = torch.randint(0, 32768, (T,), generator=g, dtype=torch.int32).cuda()
    i = torch.arange(0, D, 2, dtype=torch.float64, device="cuda") / D
    w = (theta * factor ** (D / (D - 2)) if scaling == "ntk" else theta) ** -i
    m = 1.0
    if scaling == "linear":
        w = w / factor
    if scaling == "parts":
        keep = ((old * w / (2 * math.pi) - 1) / 31).clamp(0, 1)
        w, m = w * keep + w / factor * (1 - keep), 0.1 * math.log(factor) + 1
    a = pos.double()[:, None] * w
    c, s = (m * a.cos()).float()[:, None], (m * a.sin()).float()[:, None]
    first, second = (slice(0, D // 2), slice(D // 2, D)) if layout == "half" else (slice(0, D, 2), slice(1, D, 2))
    u, v = k[..., first], k[..., second]
    want = torch.empty_like(k)
    want[..., first], want[..., second] = u * c - v * s, u * s + v * c
    plan = nq.Rope(D, theta=theta, layout=layout, scaling=scaling, factor=factor, old_len=old)
    got = nq.rope(k, pos, plan)
    same = (got == want).double().mean().item()
    assert same >= 0.992, same
    # what the cache holds of them: rotated before, at row t; rotated by the append, at the row of the position
    near = nq.PagePool(1, T // P, P, H, D, nq.KV_NESTED44)
    seqs = torch.zeros(T, dtype=torch.int32, device="cuda")
    rows = torch.arange(T, dtype=torch.int32, device="cuda")
    pmap = nq.PageMap(1, T // P, T // P, P, table=rows[:T // P].reshape(1, -1).contiguous())
    near.append(0, pmap, want, k, seqs, rows)
    far = nq.PagePool(1, 32768 // P, P, H, D, nq.KV_NESTED44)
    fmap = nq.PageMap(1, 32768 // P, 32768 // P, P, table=torch.arange(32768 // P, dtype=torch.int32, device="cuda")[None].contiguous())
    t = torch.from_numpy(np.unique(pos.cpu().numpy(), return_index=True)[1]).cuda()      # a token of each position
    far.append(0, fmap, k[t].contiguous(), k[t].contiguous(), seqs[:len(t)].contiguous(), pos[t].contiguous(), rope=plan)
    kg, _ = far.read(0, fmap, seqs[:len(t)].contiguous(), pos[t].contiguous())
    kw, _ = near.read(0, pmap, seqs[:len(t)].contiguous(), rows[t].contiguous())
    wrong = (kg != kw).reshape(-1, D).any(-1).sum().item()
    assert len(t) > 3500 and wrong <= 3, wrong
    assert nq.device_status() == 0
