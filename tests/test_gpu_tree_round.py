"""The tree calls together, as examples/tree_rounds.py uses them: norm, 8-bit
linears, append, attention, acceptance and keep, round after round."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("branch,depth,page", [(3, 3, 16), (5, 4, 32), (1, 2, 16)])
def test_rounds_leave_the_committed_rows(nq, branch, depth, page):
    """After each round the first layer's rows are, bit for bit, those that the committed tokens give at their positions:
    what was accepted lies where it belongs, whatever its node's row was."""
    from examples import tree_rounds as E
    model = E.Decoder(seed=3)
    seen = []

    def check(pool, pmap, slots, tokens, rows):
        for b, n in enumerate(rows.tolist()):
            assert len(tokens[b]) == n + 1
            ids = i32(tokens[b][:n])
            _, xq, sx = nq.rms_norm(model.table[ids.long()].float(), quantize=True)
            y = nq.linear_a8(model.qkv[0], xq, sx, True).view(n, model.Hq + 2 * model.H, model.D)
            alone = nq.PagePool(model.L, -(-n // page), page, model.H, model.D, nq.KV_NESTED44, group=64)
            m = nq.PageMap(1, -(-n // page), -(-n // page), page, table=torch.arange(-(-n // page), device="cuda").int()[None])
            pos = torch.arange(n, device="cuda").int()
            alone.append(0, m, y[:, model.Hq:model.Hq + model.H], y[:, model.Hq + model.H:], torch.zeros_like(pos), pos, rope=model.rope)
            for planes in (1, 2):
                want = alone.read(0, m, torch.zeros_like(pos), pos, planes=planes)
                got = pool.read(0, pmap, torch.full_like(pos, b), pos, planes=planes)
                assert all(torch.equal(x, z) for x, z in zip(want, got))
        seen.append(rows.tolist())

    tokens, accepted = E.run(prompts=(20, 1, 45), rounds=4, branch=branch, depth=depth, page_size=page, model=model, say=lambda *a: None, check=check)
    assert len(seen) == 4 and accepted >= 0


def test_a_round_in_a_graph(nq):
    """Plan, attention, acceptance and keep of a round, captured and replayed on other logits, as eager calls give them."""
    B, M, V, P, H, Hq, D = 3, 12, 700, 16, 2, 8, 64
    g = torch.Generator(device="cuda").manual_seed(1)
    parents = i32([[-1] + [(m - 1) // 2 for m in range(1, M)]] * B)
    pool = nq.PagePool(2, 12, P, H, D, nq.KV_NESTED44, group=64)
    pmap = nq.PageMap(B, 4, 12, P)
    slots, base = torch.arange(B, device="cuda").int(), i32([5, 17, 0])
    pmap.reserve(pool, slots, torch.zeros_like(base), base + M)
    seqs = torch.cat([torch.full((int(b) + M,), s, device="cuda").int() for s, b in enumerate(base)])
    pos = torch.cat([torch.arange(int(b) + M, device="cuda").int() for b in base])
    for l in range(2):
        kv = torch.randn(len(pos), 2 * H, D, generator=g, device="cuda")
        pool.append(l, pmap, kv[:, :H], kv[:, H:], seqs, pos)
    start = pool.data.clone()
    q = torch.randn(B, M, Hq, D, generator=g, device="cuda").bfloat16()
    tokens = torch.randint(0, V, (B, M), generator=g, device="cuda", dtype=torch.int32)
    logits = torch.randn(B, M, V, generator=g, device="cuda")
    out = [torch.empty(B, M, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda"),
           torch.empty(B, M, dtype=torch.int32, device="cuda"), torch.empty_like(q)]

    def work():
        tree = nq.Tree(parents)
        pool.attention(0, pmap, q, base + M, 2, 0.125, seqs=slots, tree=tree, out=out[3])
        nq.accept_tree(tokens, logits, tree, out_tok=out[0], out_cnt=out[1], path=out[2])
        pool.keep(pmap, slots, base, out[2], out[1])

    work()                                       # warm
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for k in range(3):
        logits.copy_(torch.randn(B, M, V, generator=g, device="cuda"))
        for b in range(B):
            logits[b, 0, tokens[b, 1 + (b + k) % 2].long()] = 9.0
        pool.data.copy_(start)
        graph.replay()
        got = [t.clone() for t in out] + [pool.data.clone()]
        pool.data.copy_(start)
        work()
        assert all(torch.equal(a, b) for a, b in zip(got, out + [pool.data])) and int(out[1].min()) >= 2
    assert nq.device_status() == 0
