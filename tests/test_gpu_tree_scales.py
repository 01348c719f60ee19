"""Attention of trees over V rows of zeros and of very unequal size: what a row adds nothing to may not take the
others' place in fp16's range.

Tolerance: tree_helpers.tree_attention64's, but with a tail that is counted against the largest contribution
p_t max|V_t| instead of the largest |V|.  The kernels hold P scaled so that the largest contribution is 2^3 or more
(2^(3 - span) where V's scales, which span at most 2^4 then, are in V already), and round P, or P times V's scale, by
2^-25 at most below fp16's normal numbers; a code is at most 136 / 105 of its row's largest: n 2^-22 of it in all."""
import numpy as np
import pytest
import torch

import tree_helpers as T
from paged_helpers import HostPool, rows_of
from test_gpu_tree_attn import check, i32, setup

pytestmark = pytest.mark.gpu

SIZES = [(9, 1), (20, 1), (40, 1), (50, 3)]            # nodes, query heads of one kv head: every kernel


def store(pool, m, lens, parents, k, v):
    """Rows k, v [B][rows][D] of one kv head, those of unused nodes left as they are."""
    at = [(b, t) for b, n in enumerate(lens) for t in range(n) if t < n - len(parents[b]) or T.sets_of(parents[b])[t - (n - len(parents[b]))][0] >= 0]
    b, t = i32([b for b, _ in at]), i32([t for _, t in at])
    pool.append(0, m, k[b.long(), t.long()][:, None].contiguous(), v[b.long(), t.long()][:, None].contiguous(), b, t)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("planes", [1, 2])
@pytest.mark.parametrize("M,Hq", SIZES)
@pytest.mark.parametrize("nats", [6.0, 10.0])
def test_steps_of_which_all_values_are_zero(nq, D, planes, M, Hq, nats):
    """The first 64 rows' values are zero, one of their scores is the highest by far; the other values are small."""
    lens, parents = [448 + M, 1500 + M], T.trees(M, 2, M)
    pool, m, _ = setup(nq, lens, parents, 16, 1, Hq, D, D, 0, M + D)
    g = torch.Generator(device="cuda").manual_seed(8)
    k = torch.randn(2, max(lens), D, generator=g, device="cuda") * 0.3
    v = torch.randn(2, max(lens), D, generator=g, device="cuda") * 2e-5
    u = torch.randn(D, generator=g, device="cuda")
    u *= D ** 0.5 / u.norm()                            # of 1 per dimension: scale q k = 1 sqrt(D) for q = k = u
    k[:, 10] = nats * u * D ** -0.5
    v[:, :64] = 0
    store(pool, m, lens, parents, k, v)
    q = (u + 0.05 * torch.randn(2, M, Hq, D, generator=g, device="cuda")).bfloat16()
    check(nq, pool, m, q, lens, parents, planes)


def small_tail(hp, table, q, lens, planes, scale, parents):
    """(out, tol), as derived above."""
    B, M, Hq, D = q.shape
    out, tol = np.zeros((B, M, Hq, D)), np.zeros((B, M, Hq, D))
    for b in range(B):
        K, V = rows_of(hp, 0, table[b], lens[b], planes)
        base = lens[b] - M
        for j, (d, up) in enumerate(T.sets_of(parents[b])):
            if d < 0:
                continue
            rows = np.array(list(range(base)) + [base + i for i in up])
            for h in range(Hq):
                k, v, x = K[0, rows], V[0, rows], q[b, j, h].astype(np.float64)
                s = scale * (k @ x)
                e = 2.0 ** -17 * scale * (np.abs(k) @ np.abs(x)).max()
                p = np.exp(s - s.max())
                l = p.sum()
                out[b, j, h] = p @ v / l
                tol[b, j, h] = (2.0 ** -8 * np.abs(out[b, j, h]) + (2 * 2.0 ** -11 + 2 * e) * (p @ np.abs(v)) / l
                                + len(p) * 2.0 ** -22 * (p * np.abs(v).max(1)).max() / l)
    return out, tol


def long_tail(nq, D, planes, M, Hq, value, bits, batch):
    """One key of 12000 has nearly all the weight, and `value` times the size of the others' values."""
    lens, parents = [12000 + M], T.trees(M, 1, M)
    pool, m, _ = setup(nq, lens, parents, 64, 1, Hq, D, D, 0, M + D)
    g = torch.Generator(device="cuda").manual_seed(9)
    k = torch.zeros(1, lens[0], D, device="cuda")        # scores of 0
    v = 0.5 + 0.5 * torch.rand(1, lens[0], D, generator=g, device="cuda")
    k[:, 5] = bits * np.log(2.0) * D ** -0.5             # against queries of ones
    v[:, 5] *= value
    store(pool, m, lens, parents, k, v)
    q = torch.ones(batch, M, Hq, D, device="cuda").bfloat16()
    scale = D ** -0.5
    out = pool.attention(0, m, q, i32(lens * batch), planes, scale, seqs=i32([0] * batch), tree=nq.Tree(i32(parents * batch)))
    assert nq.device_status() == 0
    ref, tol = small_tail(HostPool(pool), m.table.cpu().numpy(), q[:1].float().cpu().numpy(), lens, planes, scale, parents)
    off = np.abs(out.double().cpu().numpy() - ref)
    assert (off <= tol + 1e-30).all(), (off / (np.abs(ref) + 1e-30)).max()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("planes", [1, 2])
@pytest.mark.parametrize("M,Hq", SIZES)
@pytest.mark.parametrize("value,bits", [(0.0, 27.0), (0.0, 29.6)])
def test_a_long_tail_below_one_key(nq, D, planes, M, Hq, value, bits):
    """One key has nearly all the weight and a value of nothing: the many others carry the output."""
    long_tail(nq, D, planes, M, Hq, value, bits, 1)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("planes", [1, 2])
@pytest.mark.parametrize("M,Hq", SIZES)
@pytest.mark.parametrize("value,bits", [(0.0, 29.6), (2.0 ** -11, 27.0), (2.0 ** -11, 28.3), (2.0 ** -8, 28.3), (2.0 ** -4, 28.3)])
def test_a_long_tail_within_one_state(nq, D, planes, M, Hq, value, bits):
    """The same, or a value of little beside its neighbours', for more sequences than there are SMs: one running maximum
    goes over all of the rows, none of which may fall out of fp16's range beside it."""
    long_tail(nq, D, planes, M, Hq, value, bits, 160)
