"""Tree-drafted rounds on the paged cache with 8-bit activations, end to end on one GPU.

A small decoder of random weights answers a batch of prompts.  Every round drafts
a tree below the last token (the likeliest `branch` words below it, the likeliest
one below each of those, ..) on the 4-bit views of weights and cache, checks all
nodes in one pass on the 8-bit views, keeps the path that the target agrees
with, moves its rows next to the committed ones and gives back the others' pages.
Between the linears the norm adds the residual and writes int8 codes.

    python examples/tree_rounds.py --rounds 6 --branch 3 --depth 3
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from examples.paged_rounds import Decoder  # noqa: E402
from quantized_self_speculative_gb300 import nq  # noqa: E402


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def shape_of(branch, depth):
    """Parents of node 0 and `branch` chains of `depth` nodes below it, level by level."""
    return [-1] + [0 if level == 0 else 1 + (level - 1) * branch + b for level in range(depth) for b in range(branch)]


def step(model, tokens, slots, base, tree, pool, pmap, draft):
    """Logits [B][nodes][vocab] of a tree's tokens int32 [B][nodes], node m as row base[b] + m of the cache."""
    B, M = tokens.shape
    planes, D = (1 if draft else 2), model.D
    seqs = slots.repeat_interleave(M)
    rows = (base[:, None] + torch.arange(M, dtype=torch.int32, device="cuda")).reshape(-1)
    at = tree.positions(base).reshape(-1)
    x = model.table[tokens.long()].reshape(B * M, -1).float()
    add = None
    for l in range(model.L):
        x, xq, sx = nq.rms_norm(x, add=add, quantize=True)
        y = nq.linear_a8(model.qkv[l], xq, sx, not draft).view(B * M, model.Hq + 2 * model.H, D)
        q, k, v = y[:, :model.Hq], y[:, model.Hq:model.Hq + model.H], y[:, model.Hq + model.H:]
        q = pool.append(l, pmap, k, v, seqs, rows, rope=model.rope, q=q, at=at)
        a = pool.attention(l, pmap, q.view(B, M, model.Hq, D), base + M, planes, D ** -0.5, seqs=slots, tree=tree)
        add = nq.linear_a8(model.out[l], *nq.quantize_act_int8(a.view(B * M, -1)), not draft)
        x, xq, sx = nq.rms_norm(x, add=add, quantize=True)
        gu = nq.linear_a8(model.gate_up[l], xq, sx, not draft)
        h = (torch.nn.functional.silu(gu[:, :model.ffn]) * gu[:, model.ffn:]).bfloat16()
        add = nq.linear_a8(model.down[l], *nq.quantize_act_int8(h), not draft)
    _, xq, sx = nq.rms_norm(x, add=add, quantize=True)
    return nq.linear_a8(model.head, xq, sx, not draft).view(B, M, -1)


def run(prompts=(40, 7, 129), rounds=6, branch=3, depth=3, page_size=16, seed=0, model=None, say=print, check=None):
    """Returns (tokens per sequence, accepted drafts).  check(pool, pmap, slots, committed tokens, rows) is called
    after every round."""
    model = model or Decoder(seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    B, parents = len(prompts), shape_of(branch, depth)
    M = len(parents)
    W = -(-(max(prompts) + rounds * (depth + 1) + M) // page_size)
    pool = nq.PagePool(model.L, B * W, page_size, model.H, model.D, nq.KV_NESTED44, group=64)
    pmap = nq.PageMap(B, W, B * W, page_size)
    slots, base, last, tokens = torch.arange(B, dtype=torch.int32, device="cuda"), [], [], []
    for b, n in enumerate(prompts):              # a prompt is a chain, in pieces of what a tree holds
        ids = torch.randint(0, model.vocab, (1, n), generator=g, device="cuda", dtype=torch.int32)
        if n > 1:
            assert int(pmap.reserve(pool, i32([b]), i32([0]), i32([n - 1])))
            for at in range(0, n - 1, 1024):
                part = ids[:, at:min(at + 1024, n - 1)].contiguous()
                chain = nq.Tree(torch.arange(-1, part.shape[1] - 1, dtype=torch.int32, device="cuda")[None])
                step(model, part, i32([b]), i32([at]), chain, pool, pmap, False)
        base.append(n - 1)
        last.append(int(ids[0, -1]))
        tokens.append(ids[0].tolist())
    base, x0, accepted = i32(base), i32(last), 0
    levels = [i32([parents[:1 + k * branch]] * B) for k in range(depth + 1)]
    for r in range(rounds):
        granted = pmap.reserve(pool, slots, base, base + M)
        drawn = x0[:, None]
        for k in range(depth):                   # the tree so far, then one more level
            logits = step(model, drawn.contiguous(), slots, base, nq.Tree(levels[k]), pool, pmap, True)
            new = logits[:, 0].topk(branch).indices if k == 0 else logits[:, -branch:].argmax(-1)
            drawn = torch.cat([drawn, new.int()], 1)
        tree = nq.Tree(levels[depth])
        target = step(model, drawn.contiguous(), slots, base, tree, pool, pmap, False)
        out, count, path = nq.accept_tree(drawn.contiguous(), target.contiguous(), tree, width=depth + 1)
        pool.keep(pmap, slots, base, path, count)
        base = base + count
        pmap.truncate(slots, base)
        x0 = out.gather(1, count.long()[:, None] - 1)[:, 0].contiguous()
        assert bool((granted == 1).all())
        for t, o, c in zip(tokens, out.tolist(), count.tolist()):
            t += o[:c]
        accepted += int(count.sum()) - B
        if check is not None:
            check(pool, pmap, slots, tokens, base)
    status = nq.device_status()
    say(f"{rounds * B + accepted} tokens in {rounds} rounds, {accepted} drafted ones kept, status {status}")
    if status:
        raise RuntimeError(f"device status {status:#x}")
    return tokens, accepted


if __name__ == "__main__":
    a = argparse.ArgumentParser()
    for name, value in (("rounds", 6), ("branch", 3), ("depth", 3), ("seed", 0), ("page-size", 16)):
        a.add_argument("--" + name, type=int, default=value)
    a = a.parse_args()
    run(rounds=a.rounds, branch=a.branch, depth=a.depth, page_size=a.page_size, seed=a.seed)
