"""The paged operators together: the example's speculative rounds."""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example(nq):
    spec = importlib.util.spec_from_file_location("paged_rounds", os.path.join(ROOT, "examples", "paged_rounds.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_rounds_keep_their_books(nq, example):
    said = []
    tokens, accepted, drafted, pmap = example.run(prompts=(33, 1, 70), samples=2, rounds=4, k=3, say=said.append)
    assert (pmap.ref == 0).all() and (pmap.held == 0).all() and (pmap.table == -1).all()
    # two rounds of six sequences, two of three: 1 .. k + 1 tokens each
    assert drafted == 3 * (2 * 6 + 2 * 3) and 0 <= accepted <= drafted
    assert sum(len(t) - 1 for t in tokens) == accepted + 2 * 6 + 2 * 3
    assert all(0 <= x < 2048 for t in tokens for x in t)


def test_a_shared_prompt_reads_like_an_own_one(nq, example):
    """Logits after a forked prompt (shared pages, the last one copied on write)
    are those after the same prompt stored alone."""
    model = example.Decoder(seed=3)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    ids = torch.randint(0, model.vocab, (1, 41), device="cuda", dtype=torch.int32)
    pool = nq.PagePool(model.L, 16, 16, model.H, model.D, nq.KV_NESTED44, group=64)
    m = nq.PageMap(3, 4, 16, 16)
    m.reserve(pool, i32([0]), i32([0]), i32([40]))
    model(ids[:, :40], i32([0]), i32([0]), pool, m, False)
    m.fork(i32([0, 0]), i32([1, 2]), i32([40, 40]))
    m.reserve(pool, i32([1, 2, 0]), i32([40] * 3), i32([41] * 3))
    # slots 1 and 2 write other rows on their copies of the last page first
    model(ids[:, :1], i32([1]), i32([40]), pool, m, False)
    model(ids[:, 5:6], i32([2]), i32([40]), pool, m, False)
    want = model(ids[:, 40:], i32([0]), i32([40]), pool, m, False)
    for s in (1, 2):
        assert torch.equal(model(ids[:, 40:], i32([s]), i32([40]), pool, m, False), want)
    assert nq.device_status() == 0
