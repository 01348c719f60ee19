"""A plan made on a stream of its own, and what is taken from it there."""
import pytest
import torch

import tree_helpers as T

pytestmark = pytest.mark.gpu


def test_positions_on_the_plans_stream(nq):
    """The stream is still busy when the plan and the positions are asked for: they follow each other on it."""
    parents = T.trees(5, 4, 70)
    p = torch.tensor(parents, dtype=torch.int32, device="cuda")
    base = torch.tensor([0, 9, 100, 7], dtype=torch.int32, device="cuda")
    want = [[b + max(d, 0) for d, _ in T.sets_of(t)] for b, t in zip(base.tolist(), parents)]
    side = torch.cuda.Stream()
    for _ in range(3):
        junk = torch.full((4, 70), 12345, dtype=torch.int32, device="cuda")      # what fresh memory may hold
        del junk
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)                # some 10 ms
        tree = nq.Tree(p, stream=side)
        got = tree.positions(base, stream=side)
        side.synchronize()
        assert got.tolist() == want and got.dtype == torch.int32
    assert nq.Tree(p).positions(base).tolist() == want and nq.device_status() == 0
