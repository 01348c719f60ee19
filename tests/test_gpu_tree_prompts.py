"""Prompts longer than a tree may be, in examples/tree_rounds.py."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("prompts", [(1025, 3), (1026, 2049), (2500,)])
def test_prompts_of_more_rows_than_a_tree_has_nodes(nq, prompts):
    """Every row of the first layer's cache is, bit for bit, that of its token at its position."""
    from examples import tree_rounds as E
    model = E.Decoder(seed=3)
    seen = []

    def check(pool, pmap, slots, tokens, rows):
        for b, n in enumerate(rows.tolist()):
            pos = torch.arange(n, device="cuda").int()
            ids = torch.tensor(tokens[b][:n], device="cuda")
            _, xq, sx = nq.rms_norm(model.table[ids].float(), quantize=True)
            y = nq.linear_a8(model.qkv[0], xq, sx, True).view(n, model.Hq + 2 * model.H, model.D)
            alone = nq.PagePool(model.L, -(-n // 16), 16, model.H, model.D, nq.KV_NESTED44, group=64)
            m = nq.PageMap(1, -(-n // 16), -(-n // 16), 16, table=torch.arange(-(-n // 16), device="cuda").int()[None])
            alone.append(0, m, y[:, model.Hq:model.Hq + model.H], y[:, model.Hq + model.H:], torch.zeros_like(pos), pos, rope=model.rope)
            want, got = alone.read(0, m, torch.zeros_like(pos), pos), pool.read(0, pmap, torch.full_like(pos, b), pos)
            assert all(torch.equal(x, z) for x, z in zip(want, got))
        seen.append(rows.tolist())

    tokens, _ = E.run(prompts=prompts, rounds=1, branch=2, depth=2, model=model, say=lambda *a: None, check=check)
    assert len(seen) == 1 and all(len(t) > n for t, n in zip(tokens, prompts))
