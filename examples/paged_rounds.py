"""Self-speculative rounds on the paged cache, end to end on one GPU.

A small decoder of random weights answers a batch of prompts of unequal length:
each prompt is stored once and forked into `samples` sequences that share its
pages; every round drafts k tokens on the 4-bit views of weights and cache,
checks them in one pass on the 8-bit views, keeps the accepted prefix and gives
back the rejected rows' pages.  Some sequences then end, the pool is compacted
and the others go on.

    python examples/paged_rounds.py --rounds 8 --k 4 --samples 3
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from quantized_self_speculative_gb300 import nq  # noqa: E402


class Decoder:
    """Grouped-query attention and a gated MLP per layer, nested 4+4-bit weights,
    rotary positions, a paged nested cache."""

    def __init__(self, layers=2, hidden=512, heads_q=8, heads_kv=2, head_dim=64, ffn=1024, vocab=2048, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        w = lambda n, k: nq.pack_weights(torch.randn(n, k, generator=g, device="cuda") * k ** -0.5, nq.FMT_NESTED44, 64)  # noqa: E731
        self.L, self.Hq, self.H, self.D, self.ffn, self.vocab = layers, heads_q, heads_kv, head_dim, ffn, vocab
        self.qkv = [w((heads_q + 2 * heads_kv) * head_dim, hidden) for _ in range(layers)]
        self.out = [w(hidden, heads_q * head_dim) for _ in range(layers)]
        self.gate_up = [w(2 * ffn, hidden) for _ in range(layers)]
        self.down = [w(hidden, ffn) for _ in range(layers)]
        self.table = (torch.randn(vocab, hidden, generator=g, device="cuda") * 2).bfloat16()
        self.head = w(vocab, hidden)
        self.rope = nq.Rope(head_dim, theta=10000.0)

    def __call__(self, tokens, slots, first, pool, pmap, draft):
        """Logits [B * M][vocab] of M new tokens per slot, tokens int32 [B][M] at rows first[b] .. of the cache."""
        B, M = tokens.shape
        lin = nq.draft_gemv if draft else nq.verify_gemm
        planes = 1 if draft else 2
        seqs = slots.repeat_interleave(M)
        pos = (first[:, None] + torch.arange(M, dtype=torch.int32, device="cuda")).reshape(-1)
        lens = first + M
        x = self.table[tokens.long()].reshape(B * M, -1).float()
        norm = lambda t: (t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6)).bfloat16()  # noqa: E731
        for l in range(self.L):
            y = lin(self.qkv[l], norm(x)).view(B * M, self.Hq + 2 * self.H, self.D)
            q, k, v = y[:, :self.Hq], y[:, self.Hq:self.Hq + self.H], y[:, self.Hq + self.H:]
            q = pool.append(l, pmap, k, v, seqs, pos, rope=self.rope, q=q)
            a = pool.attention(l, pmap, q.view(B, M, self.Hq, self.D), lens, planes, self.D ** -0.5, seqs=slots)
            x = x + lin(self.out[l], a.view(B * M, -1))
            gu = lin(self.gate_up[l], norm(x))
            x = x + lin(self.down[l], (torch.nn.functional.silu(gu[:, :self.ffn]) * gu[:, self.ffn:]).bfloat16())
        return lin(self.head, norm(x))


def run(prompts=(40, 7, 129), samples=3, rounds=8, k=4, page_size=16, seed=0, model=None, say=print):
    """Returns (tokens per sequence, accepted drafts, drafts, map)."""
    model = model or Decoder(seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    n_prompts, B = len(prompts), len(prompts) * samples
    longest = max(prompts) + (rounds + 1) * (k + 1) + 1
    W = -(-longest // page_size)
    N = B * W
    pool = nq.PagePool(model.L, N, page_size, model.H, model.D, nq.KV_NESTED44, group=64)
    pmap = nq.PageMap(B, W, N, page_size)
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731

    # prompts, one after another, in the slots of their first samples; the last token starts the first round
    last = []
    for i, n in enumerate(prompts):
        slot, zero = i32([i * samples]), i32([0])
        ids = torch.randint(0, model.vocab, (1, n), generator=g, device="cuda", dtype=torch.int32)
        if n > 1:
            assert int(pmap.reserve(pool, slot, zero, i32([n - 1])))
            model(ids[:, :n - 1], slot, zero, pool, pmap, False)
        last.append(int(ids[0, n - 1]))
    rows = i32([n - 1 for n in prompts for _ in range(samples)])
    src = i32([i * samples for i in range(n_prompts) for _ in range(samples)])
    slots = torch.arange(B, dtype=torch.int32, device="cuda")
    pmap.fork(src, slots, rows)
    x0 = i32([t for t in last for _ in range(samples)])
    # the samples of a prompt differ from their first token on
    x0 = ((x0 + torch.arange(samples, device="cuda").repeat(n_prompts).int()) % model.vocab).int()
    say(f"{B} sequences share {int((pmap.ref > 0).sum())} pages of {page_size} rows")

    tokens = [[int(t)] for t in x0]
    accepted = drafted = 0
    ws = nq.accept_workspace(B, k, model.vocab, torch.device("cuda"))
    for r in range(rounds):
        if r == rounds // 2 and samples > 1:      # half way, the last sample of each prompt ends
            done = torch.arange(samples - 1, B, samples, device="cuda").int()
            pmap.truncate(done, torch.zeros_like(done))
            used = int(pmap.compact(pool))
            keep = (slots % samples != samples - 1).nonzero()[:, 0]
            slots, rows, x0 = slots[keep].contiguous(), rows[keep].contiguous(), x0[keep].contiguous()
            say(f"round {r}: {len(done)} sequences end, the others lie in pages 0 .. {used - 1}")
        n = len(slots)
        granted = pmap.reserve(pool, slots, rows, rows + k + 1)
        draft = torch.empty(n, k, dtype=torch.int32, device="cuda")
        t = x0
        for j in range(k):
            t = model(t[:, None], slots, rows + j, pool, pmap, True).argmax(-1).int()
            draft[:, j] = t
        target = model(torch.cat([x0[:, None], draft], 1).contiguous(), slots, rows, pool, pmap, False)
        out, count = nq.accept_greedy(draft, target.view(n, k + 1, -1).contiguous(), ws if n == B else None)
        rows = (rows + count).contiguous()
        x0 = out.gather(1, count.long()[:, None] - 1)[:, 0].contiguous()
        pmap.truncate(slots, rows)                # the rejected rows' pages
        assert bool((granted == 1).all())
        for s, o, c in zip(slots.tolist(), out.tolist(), count.tolist()):
            tokens[s] += o[:c]
        accepted, drafted = accepted + int(count.sum()) - n, drafted + n * k
    pmap.truncate(slots, torch.zeros_like(slots))
    status = nq.device_status()
    say(f"{sum(len(t) - 1 for t in tokens)} tokens in {rounds} rounds, {accepted} of {drafted} drafts kept, status {status}")
    if status:
        raise RuntimeError(f"device status {status:#x}")
    return tokens, accepted, drafted, pmap


if __name__ == "__main__":
    a = argparse.ArgumentParser()
    for name, value in (("rounds", 8), ("k", 4), ("samples", 3), ("seed", 0), ("page-size", 16)):
        a.add_argument("--" + name, type=int, default=value)
    a = a.parse_args()
    run(samples=a.samples, rounds=a.rounds, k=a.k, page_size=a.page_size, seed=a.seed)
