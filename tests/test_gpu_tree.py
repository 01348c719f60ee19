"""Trees of drafted tokens on the GPU: masks and depths, greedy acceptance and
keeping the accepted path, against plain walks."""
import random

import numpy as np
import pytest
import torch

import tree_helpers as T
from paged_helpers import HostPool

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ plan
@pytest.mark.parametrize("B,M", [(1, 1), (5, 2), (8, 31), (8, 32), (9, 33), (6, 130), (5, 1000), (4, 1024), (300, 17)])
@pytest.mark.parametrize("window", [0, 1, 3])
def test_masks_and_depths(nq, B, M, window):
    p = T.trees(B + M, B, M)
    t = nq.Tree(i32(p), window=window)
    assert nq.device_status() == 0
    assert t.depth.cpu().tolist() == [[d for d, _ in T.sets_of(x)] for x in p]
    assert np.array_equal(t.bits.cpu().numpy().view(np.uint32), np.stack([T.bits_of(x, window) for x in p]))
    base = torch.arange(B, device="cuda", dtype=torch.int32) * 7
    assert torch.equal(t.positions(base), base[:, None] + t.depth.clamp(min=0))


@pytest.mark.parametrize("p", [[0, 0], [-1, 1], [-1, 5, 0], [-1, -2, 1], [-1, 2, 1, 0], [-1, 2147483647, 0], [-2147483648, 0]])
def test_a_parent_that_is_not_below_its_node_is_reported(nq, p):
    """Such nodes, and those that hang on them, are not used; the others are what they were."""
    t = nq.Tree(i32([p, [-1] * len(p)]))
    assert nq.device_status() == nq.NQ_DEV_BAD_TREE
    assert t.depth.cpu().tolist() == [[d for d, _ in T.sets_of(p)], [0] * len(p)]
    assert np.array_equal(t.bits.cpu().numpy().view(np.uint32)[0], T.bits_of(p))


def test_plan_refusals(nq):
    with pytest.raises(ValueError):
        nq.Tree(i32([-1, 0]))
    with pytest.raises(ValueError):
        nq.Tree(i32([[-1, 0]]).long())
    with pytest.raises(ValueError):
        nq.Tree(i32([[-1, 0], [-1, 0]]).T)
    for shape, kw, status in [((1, 1025), {}, nq.NQ_ERR_SHAPE), ((1, 0), {}, nq.NQ_ERR_ARG), ((1, 4), dict(window=-1), nq.NQ_ERR_ARG)]:
        with pytest.raises(nq.NQError) as e:
            nq.Tree(torch.full(shape, -1, dtype=torch.int32, device="cuda"), **kw)
        assert e.value.status == status
    assert nq.Tree(torch.empty(0, 4, dtype=torch.int32, device="cuda")).depth.shape == (0, 4)


# ------------------------------------------------------------------ acceptance
def accept_case(seed, B, M, V, likely=0.8):
    """Trees, tokens and logits where the target often agrees with some child; children with the same token among them."""
    r, g = random.Random(seed), torch.Generator().manual_seed(seed)
    p = T.trees(seed, B, M)
    logits = torch.randn(B, M, V, generator=g)
    tokens = torch.randint(0, V, (B, M), generator=g, dtype=torch.int32)
    for b in range(B):
        for m in range(M):
            kids = [c for c in range(m + 1, M) if p[b][c] == m]
            if kids and r.random() < likely:
                c = r.choice(kids)
                logits[b, m, tokens[b, c]] = 9.0
                if len(kids) > 1 and r.random() < 0.5:
                    tokens[b, r.choice(kids)] = tokens[b, c]         # a twin
    return p, tokens, logits


def check_accept(got, p, tokens, logits, width):
    tok, cnt, path = (t.cpu().tolist() for t in got)
    for b in range(len(p)):
        out, nodes = T.accept(p[b], tokens[b].tolist(), logits[b].numpy(), width)
        assert cnt[b] == len(out)
        assert tok[b] == out + [-1] * (width - len(out)) and path[b] == nodes + [-1] * (width - len(out))


@pytest.mark.parametrize("B,M,V", [(1, 1, 1), (1, 16, 32000), (7, 9, 3), (5, 33, 1001), (4, 64, 4099), (70, 12, 130), (3, 1024, 67), (2, 7, 152064), (1, 3, 524288)])
def test_acceptance_walks_the_tree(nq, B, M, V):
    p, tokens, logits = accept_case(B + M + V, B, M, V)
    tree = nq.Tree(i32(p))
    x = logits.cuda()
    for width in sorted({1, min(2, M), M}):
        got = nq.accept_tree(tokens.cuda(), x, tree, width=width)
        assert nq.device_status() == 0
        check_accept(got, p, tokens, logits, width)


def test_ties_take_the_lowest_index_and_zeros_are_alike(nq):
    V = 5000
    logits = torch.full((3, 2, V), -1.0)
    logits[0, 0, [17, 18, 4000]] = 2.0
    logits[1, 0] = 0.0
    logits[1, 0, 0::2] = -0.0
    logits[2, 0, [4999, 4996]] = 3.0
    tokens = i32([[0, 17], [0, 0], [0, 4996]])
    tok, cnt, path = nq.accept_tree(tokens, logits.cuda(), nq.Tree(i32([[-1, 0]] * 3)))
    assert tok.cpu().tolist() == [[17, 0], [0, 0], [4996, 0]] and cnt.cpu().tolist() == [2, 2, 2]


def test_a_chain_is_the_chain_acceptance(nq):
    """A tree that is a chain emits what spec_accept_greedy emits."""
    B, k, V = 6, 4, 3000
    p = [[m - 1 for m in range(k + 1)]] * B
    g = torch.Generator().manual_seed(5)
    logits = torch.randn(B, k + 1, V, generator=g)
    draft = torch.randint(0, V, (B, k), generator=g, dtype=torch.int32)
    for b in range(B):
        for j in range(min(b, k)):
            draft[b, j] = int(logits[b, j].argmax())
    tokens = torch.cat([torch.zeros(B, 1, dtype=torch.int32), draft], 1).cuda()
    tok, cnt, _ = nq.accept_tree(tokens, logits.cuda(), nq.Tree(i32(p)))
    want, wcnt = nq.accept_greedy(draft.cuda(), logits.cuda())
    assert torch.equal(tok, want) and torch.equal(cnt, wcnt)


def test_what_is_not_finite_and_tokens_outside_the_vocabulary(nq):
    tree = nq.Tree(i32([[-1, 0, 0], [-1, 0, 0]]))
    logits = torch.randn(2, 3, 500)
    logits[:, :, 7] = 9.0
    tokens = i32([[0, 7, 3], [0, 3, 2]])
    for bad in (float("nan"), float("inf"), -float("inf")):
        x = logits.clone()
        x[0, 2, 3] = bad                                # a node off the walk: not read
        nq.accept_tree(tokens, x.cuda(), tree)
        assert nq.device_status() == 0
        x[0, 1, 499] = bad
        tok, cnt, _ = nq.accept_tree(tokens, x.cuda(), tree)
        assert nq.device_status() == nq.NQ_DEV_NONFINITE
        assert tok[1].tolist() == [7, -1, -1] and int(cnt[1]) == 1 and 0 <= int(tok[0, 1]) < 500
    x = torch.full((2, 3, 500), float("nan"))
    tok, cnt, _ = nq.accept_tree(tokens, x.cuda(), tree)
    assert nq.device_status() == nq.NQ_DEV_NONFINITE and (tok < 500).all() and (cnt <= 3).all()
    for t in (500, -1):
        tokens[1, 2] = t
        tok, cnt, path = nq.accept_tree(tokens, logits.cuda(), tree)
        assert nq.device_status() == nq.NQ_DEV_BAD_TOKEN and tok.tolist() == [[7, 7, -1], [7, -1, -1]]
    # of an unused node nothing is asked
    tok, cnt, _ = nq.accept_tree(tokens, logits.cuda(), nq.Tree(i32([[-1, 0, -2], [-2, -2, -2]])))
    assert nq.device_status() == 0 and cnt.tolist() == [2, 0] and tok[1].tolist() == [-1, -1, -1]


def test_acceptance_goes_on_to_the_commit(nq):
    p, tokens, logits = accept_case(3, 4, 12, 400)
    tok, cnt, _ = nq.accept_tree(tokens.cuda(), logits.cuda(), nq.Tree(i32(p)), width=6)
    has = [b for b in range(4) if int(cnt[b]) > 0]
    seq, length, x0 = torch.full((4, 64), -5, dtype=torch.int32, device="cuda"), i32([3, 1, 0, 9]), i32([0] * 4)
    nq.round_commit(tok, cnt, seq, length, x0)
    nq.device_status()
    for b in has:
        n = int(cnt[b])
        at = [3, 1, 0, 9][b]
        assert seq[b, at:at + n].tolist() == tok[b, :n].tolist() and int(length[b]) == at + n and int(x0[b]) == int(tok[b, n - 1])


def test_accept_refusals_streams_and_graph(nq):
    p, tokens, logits = accept_case(11, 5, 20, 900)
    tree, tokens, x = nq.Tree(i32(p)), tokens.cuda(), logits.cuda()
    for a in [(tokens[:, :3], x, tree), (tokens, x[:, :3], tree), (tokens.long(), x, tree), (tokens, x.half(), tree)]:
        with pytest.raises(ValueError):
            nq.accept_tree(*a)
    for width in (0, 21):
        with pytest.raises(nq.NQError):
            nq.accept_tree(tokens, x, tree, width=width)
    want = nq.accept_tree(tokens, x, tree)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = nq.accept_tree(tokens, x, tree, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = [torch.empty_like(t) for t in want]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t2 = nq.Tree(tree.parents)
        nq.accept_tree(tokens, x, t2, out_tok=out[0], out_cnt=out[1], path=out[2])
    x.mul_(-1)
    g.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, nq.accept_tree(tokens, x, tree)))


# ------------------------------------------------------------------ keep
def filled(nq, layers, S, W, P, H, D, G, fmt, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    N = S * W + 2
    pool = nq.PagePool(layers, N, P, H, D, fmt, group=G)
    pool.data.copy_(torch.randint(0, 256, pool.data.shape, generator=g, device="cuda", dtype=torch.uint8))
    table = torch.randperm(N, generator=g, device="cuda")[:S * W].reshape(S, W).int()
    return pool, nq.PageMap(S, W, N, P, table=table)


def row_bytes(hp, layer, page, h, row):
    """What one row is, by the format's reader."""
    if hp.bf:
        return [hp.row(layer, page, h, row, w, 2).tobytes() for w in (0, 1)]
    return [tuple(x.tobytes() for x in hp.codes(layer, page, h, row, w)) for w in (0, 1)]


@pytest.mark.parametrize("D,G,P,H,fmt", [(128, 128, 16, 2, 0), (128, 64, 32, 1, 0), (64, 64, 16, 3, 0), (128, 128, 64, 2, 1), (64, 64, 16, 1, 1)])
def test_path_rows_move_and_nothing_else_does(nq, D, G, P, H, fmt):
    layers, S, W = 2, 5, 4
    pool, m = filled(nq, layers, S, W, P, H, D, G, fmt, D + P + fmt)
    paths = [[0, 3, 5, 6, 20], [], list(range(9)), [1, 2, 3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 16, 17, 18, 19, 24], [0, 2]]
    first, seqs = [P - 3, 5, 0, P + 1, 2 * P - 1], [3, 1, 0, 4, 2]
    width = max(map(len, paths))
    before = HostPool(pool)
    pool.keep(m, i32(seqs), i32(first), i32([p + [99] * (width - len(p)) for p in paths]), i32([len(p) for p in paths]))
    assert nq.device_status() == 0
    after, table = HostPool(pool), m.table.cpu().numpy()
    moved = {}
    for s, f, p in zip(seqs, first, paths):
        for j, x in enumerate(p):
            a, b = f + x, f + j
            moved[int(table[s, b // P]), b % P] = int(table[s, a // P]), a % P
    for layer in range(layers):
        for page in range(pool.n_pages):
            for r in range(P):
                a, b = moved.get((page, r), (page, r))
                for h in range(H):
                    assert row_bytes(after, layer, page, h, r) == row_bytes(before, layer, a, h, b), (layer, page, r, h)


def test_a_path_that_cannot_be_kept_is_left_out(nq):
    P = 16
    pool, m = filled(nq, 1, 4, 2, P, 1, 64, 64, 0, 1)
    before = pool.data.clone()
    one = lambda s, f, p, c: pool.keep(m, i32([s]), i32([f]), i32([p]), i32([c]))  # noqa: E731
    for s, f, p, c in [(4, 0, [1], 1), (-1, 0, [1], 1), (0, -1, [1], 1), (0, 0, [1, 1], 2), (0, 0, [3, 2], 2), (0, 0, [-1, 2], 2),
                       (0, 0, [1, 2], 3), (0, 0, [1, 2], -1)]:
        one(s, f, p, c)
        assert nq.device_status() == nq.NQ_DEV_BAD_PAGE
    one(0, 20, [0, 12], 2)
    assert nq.device_status() == nq.NQ_DEV_SEQ_FULL
    one(0, 2147483647, [1, 2147483647], 2)
    assert nq.device_status() == nq.NQ_DEV_SEQ_FULL
    m.table[1, 1] = -1
    one(1, 3, [0, 14], 2)
    m.table[1, 1] = 10000
    one(1, 3, [0, 14], 2)
    assert nq.device_status() == nq.NQ_DEV_BAD_PAGE
    one(2, 3, [2, 5], 0)
    assert nq.device_status() == 0 and torch.equal(pool.data, before)
    for a in [(i32([0]), i32([0]), i32([1]), i32([1])), (i32([0]), i32([0, 1]), i32([[1]]), i32([1])), (i32([0]), i32([0]), i32([[1]]).long(), i32([1]))]:
        with pytest.raises(ValueError):
            pool.keep(m, *a)
    pool.keep(m, i32([]), i32([]), torch.empty(0, 3, dtype=torch.int32, device="cuda"), i32([]))


# ------------------------------------------------------------------ rows and positions apart
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_append_rotates_by_the_positions_given(nq, dtype):
    """k and q as the rotation by `at` alone gives them, in the rows of pos."""
    H, Hq, D, P = 2, 4, 64, 16
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(21, Hq + 2 * H, D, generator=g, device="cuda").to(getattr(torch, dtype))
    seqs, pos = i32([0] * 21), torch.arange(5, 26, device="cuda").int()
    at = torch.randint(0, 9000, (21,), generator=g, device="cuda").int()
    plan = nq.Rope(D)
    pools = [nq.PagePool(1, 4, P, H, D, nq.KV_NESTED44, group=64) for _ in range(2)]
    m = nq.PageMap(1, 2, 4, P, table=i32([[3, 1]]))
    q = pools[0].append(0, m, x[:, Hq:Hq + H], x[:, Hq + H:], seqs, pos, rope=plan, q=x[:, :Hq], at=at)
    k = nq.rope(x[:, Hq:Hq + H], at, plan, out_dtype=torch.float32)
    pools[1].append(0, m, k, x[:, Hq + H:].float().contiguous(), seqs, pos)
    assert torch.equal(q, nq.rope(x[:, :Hq], at, plan, out_dtype=torch.bfloat16))
    assert torch.equal(pools[0].data, pools[1].data) and nq.device_status() == 0
    with pytest.raises(ValueError):
        pools[0].append(0, m, x[:, Hq:Hq + H], x[:, Hq + H:], seqs, pos, rope=plan, at=at[:3])
