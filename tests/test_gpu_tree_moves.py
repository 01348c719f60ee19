"""Rounds of examples/tree_rounds.py in which the accepted path does not lie next to the committed rows: what keep
moves, in every layer."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("branch,depth,page", [(3, 3, 16), (5, 4, 32), (4, 2, 16)])
def test_accepted_rows_move_in_every_layer(nq, monkeypatch, branch, depth, page):
    """The target is made to agree with the last child of node 0 and the node below it (its logits there are raised), so
    that rows of other nodes lie between the accepted ones; after keep they follow the committed rows, and the rows
    before them are as they were."""
    from examples import tree_rounds as E
    model = E.Decoder(seed=3)
    assert model.L > 1
    paths, keep, accept = [], nq.PagePool.keep, nq.accept_tree
    last, below = branch, 2 * branch                    # nodes: children of 0 are 1 .. branch, below each the next level's

    def forced(tokens, logits, tree, width=None, **kw):
        logits = logits.clone()
        for up, child in ((0, last), (last, below)):
            same = (tokens[:, 1:1 + branch] == tokens[:, child:child + 1]).sum(-1) if up == 0 else torch.ones_like(tokens[:, 0])
            assert (same == 1).all()                     # (of children with one token the lowest would go on)
            logits[:, up].scatter_(1, tokens[:, child:child + 1].long(), 1e4)
        return accept(tokens, logits, tree, width=width, **kw)

    def rows(pool, pmap, slot, at):
        n = torch.full_like(at, slot)
        return [t.clone() for l in range(pool.layers) for planes in (1, 2) for t in pool.read(l, pmap, n, at, planes=planes)]

    def watched(pool, pmap, seqs, first, path, count, **kw):
        want, told = [], []
        for s, f, p, c in zip(seqs.tolist(), first.tolist(), path.tolist(), count.tolist()):
            assert c >= 3 and p[:3] == [0, last, below]
            want.append((s, torch.arange(f + c, device="cuda").int(),
                         rows(pool, pmap, s, torch.cat([torch.arange(f, device="cuda").int(), i32([f + j for j in p[:c]])]))))
            told.append(p[:c])
        keep(pool, pmap, seqs, first, path, count, **kw)
        for s, at, before in want:
            assert all(torch.equal(a, b) for a, b in zip(before, rows(pool, pmap, s, at)))
        paths.append(told)

    monkeypatch.setattr(nq, "accept_tree", forced)
    monkeypatch.setattr(nq.PagePool, "keep", watched)
    E.run(prompts=(20, 1, 45), rounds=3, branch=branch, depth=depth, page_size=page, model=model, say=lambda *a: None)
    assert len(paths) == 3 and nq.device_status() == 0
