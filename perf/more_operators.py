"""Measured cases of the operators of a tree-drafted round: the norm between two
linears (with the residual's addition and an 8-bit output), attention of a tree
of drafted tokens over the paged cache, greedy acceptance along the tree, and
keeping the accepted path's rows in the cache.

`run` computes a case in elementary torch operations (32 bits, rounded once at
the end) or, where `own` is true, through the package's entry points.  Both
read and write the same bytes, so the page format is written out here too:

A pool holds [layers][pages][heads_kv] records of `page` rows.  A NESTED44
record is page / 16 base blocks, then page / 16 refinement blocks.  A base
block is 16 rows of K base nibbles, 16 rows of V base nibbles, the fp16 K
scales [row][group] and the V scales; a refinement block is 16 rows of K
refinement nibbles, then of V.  Nibbles are offset by 8, element 2j in the low
half of byte j.  A BF16 record is page / 16 blocks of 16 K rows, 16 V rows.
Within 16 rows the 16-byte chunks are permuted (see `_nib_at`, `_bf_at`).

A tree is its parents: parents[m] < m is the node above node m, -1 the last
committed row, -2 marks a node that a padded batch does not use.
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------ cases
def listed():
    return [
        # between two linears of one decoding step: the linear's fp32 output joins the residual, int8 codes for the next
        {"name": "norm_step", "op": "norm", "M": 1, "K": 4096, "x": "float32", "add": "float32", "w": "float32", "int8": True},
        # the verify pass of a batched round, 16 sequences of 9 rows
        {"name": "norm_verify", "op": "norm", "M": 144, "K": 4096, "x": "float32", "add": "float32", "w": "bfloat16", "int8": True},
        # a prompt's rows, the residual kept in 16 bits, bf16 activations for the next linear
        {"name": "norm_prompt", "op": "norm", "M": 16381, "K": 3584, "x": "bfloat16", "add": "float32", "w": "bfloat16", "int8": False},
        # one conversation, a small tree on MHA heads: latency
        {"name": "tree_short", "op": "attend", "fmt": "nested", "planes": 2, "B": 1, "M": 16, "Hq": 32, "H": 32, "D": 128, "G": 128,
         "page": 16, "lo": 517, "hi": 517, "pad": False, "mix": 1, "cap": 0.0, "window": 0, "slopes": False},
        # the verify read of a batched round: 16 ragged sequences, trees of up to 32 nodes, grouped-query heads
        {"name": "tree_batch", "op": "attend", "fmt": "nested", "planes": 2, "B": 16, "M": 32, "Hq": 32, "H": 8, "D": 128, "G": 128,
         "page": 16, "lo": 301, "hi": 4099, "pad": True, "mix": 2, "cap": 0.0, "window": 0, "slopes": False},
        # long contexts, trees of 64 nodes, seven query heads share a kv head
        {"name": "tree_long", "op": "attend", "fmt": "nested", "planes": 2, "B": 4, "M": 64, "Hq": 28, "H": 4, "D": 128, "G": 128,
         "page": 64, "lo": 20001, "hi": 32768, "pad": False, "mix": 3, "cap": 0.0, "window": 0, "slopes": False},
        # 16-bit pages of small heads, capped scores with a distance bias in a sliding window
        {"name": "tree_capped_window", "op": "attend", "fmt": "bf16", "planes": 2, "B": 8, "M": 13, "Hq": 16, "H": 4, "D": 64, "G": 64,
         "page": 32, "lo": 900, "hi": 9001, "pad": True, "mix": 4, "cap": 30.0, "window": 4096, "slopes": True},
        # one conversation's tree against the target's logits
        {"name": "accept_one", "op": "accept", "B": 1, "M": 16, "V": 32000, "pad": False, "mix": 5},
        # a batched round over a large vocabulary
        {"name": "accept_batch", "op": "accept", "B": 64, "M": 32, "V": 152064, "pad": True, "mix": 6},
        # the accepted path of one conversation, all layers
        {"name": "keep_one", "op": "keep", "fmt": "nested", "layers": 32, "B": 1, "M": 16, "H": 8, "D": 128, "G": 128, "page": 16,
         "lo": 517, "hi": 517, "mix": 7},
        # the same for a batched round, MHA heads
        {"name": "keep_batch", "op": "keep", "fmt": "nested", "layers": 32, "B": 16, "M": 64, "H": 32, "D": 128, "G": 64, "page": 16,
         "lo": 40, "hi": 90, "mix": 8},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "attend", "attend", "accept", "keep"])
    types = ["float32", "bfloat16"]
    if op == "norm":
        K = 8 * _log(rng, 8, 2048)
        return {"op": op, "M": _log(rng, 1, max(2, 45000000 // K)), "K": K, "x": rng.choice(types), "add": rng.choice(types + [""]),
                "w": rng.choice(types + [""]), "int8": rng.random() < 0.5}
    D = rng.choice([64, 128, 128])
    G = rng.choice([64, D])
    fmt = rng.choice(["nested", "nested", "bf16"])
    H = rng.choice([1, 2, 4, 8, 32])
    page = rng.choice([16, 32, 64, 128])
    mix = rng.randrange(1 << 30)
    if op == "attend":
        g = rng.choice([1, 2, 4, 7, 8]) if H < 32 else 1
        B, M = _log(rng, 1, 24), _log(rng, 1, 130)
        hi = _log(rng, 1, max(2, min(32000, 200000000 // (B * M * H * g), 700000 // (B * H)) - M))
        return {"op": op, "fmt": fmt, "planes": rng.choice([1, 2]), "B": B, "M": M, "Hq": H * g, "H": H, "D": D, "G": G, "page": page,
                "lo": rng.choice([hi, max(0, hi // 7), 0]), "hi": hi, "pad": rng.random() < 0.5, "mix": mix,
                "cap": rng.choice([0.0, 0.0, 30.0]), "window": rng.choice([0, 0, max(1, hi // 3)]), "slopes": rng.random() < 0.3}
    B, M = _log(rng, 1, 64), _log(rng, 1, 100)
    if op == "accept":
        return {"op": op, "B": B, "M": M, "V": _log(rng, 1000, max(1001, min(200000, 250000000 // (B * M)))), "pad": rng.random() < 0.5, "mix": mix}
    c = {"op": op, "fmt": fmt, "layers": 1, "B": B, "M": M, "H": H, "D": D, "G": G, "page": page, "lo": 0, "hi": _log(rng, 1, 100), "mix": mix}
    c["layers"] = _log(rng, 1, max(1, min(32, 16384 // (B * H), 800000000 // (B * ((c["hi"] + M) // page + 2) * H * _record(c)))))
    return c


def _bases(c):
    """Committed rows of each sequence."""
    r = random.Random(c["mix"])
    got = [r.randint(c["lo"], c["hi"]) for _ in range(c["B"])]
    got[0] = c["hi"]
    return got


def _trees(c):
    """Parents of each sequence's nodes, and a path from node 0 downwards in each."""
    r = random.Random(c["mix"] + 1)
    trees, paths = [], []
    for _ in range(c["B"]):
        n = r.randint(max(1, c["M"] // 2), c["M"]) if c.get("pad") else c["M"]
        # likelier below the newest nodes, so that there are chains as well as fans
        p = [-1] + [max(r.randrange(m), r.randrange(m)) for m in range(1, n)]
        path = [0]
        while r.random() < 0.8:
            below = [m for m in range(n) if p[m] == path[-1]]
            if not below:
                break
            path.append(r.choice(below))
        trees.append(p + [-2] * (c["M"] - n))
        paths.append(path)
    return trees, paths


def _row_bytes(c, planes=2):
    """K and V bytes of one row of one head."""
    if c["fmt"] == "bf16":
        return 4 * c["D"]
    return c["D"] * planes + 4 * (c["D"] // c["G"])


def _record(c):
    return c["page"] * _row_bytes(c)


def work(c):
    el = {"float32": 4, "bfloat16": 2, "": 0}
    if c["op"] == "norm":
        n = c["M"] * c["K"]
        return {"bytes": n * (el[c["x"]] * (2 if c["add"] else 1) + el[c["add"]] + (1 if c["int8"] else 2)) + c["K"] * el[c["w"]] + 4 * c["M"],
                "flops": 5 * n}
    if c["op"] == "attend":
        rows = [(min(n, c["window"] - 1) if c["window"] else n) + c["M"] for n in _bases(c)]
        return {"bytes": sum(rows) * c["H"] * _row_bytes(c, c["planes"]) + 4 * c["B"] * c["M"] * c["Hq"] * c["D"] + 4 * sum(-(-n // c["page"]) for n in rows),
                "flops": 4 * sum(rows) * c["M"] * c["Hq"] * c["D"]}
    paths = _trees(c)[1]
    if c["op"] == "accept":           # the logits of the nodes on the path; parents, tokens, depths, path
        return {"bytes": 4 * sum(map(len, paths)) * c["V"] + 24 * c["B"] * c["M"], "flops": sum(map(len, paths)) * c["V"]}
    moved = sum(sum(j != m for j, m in enumerate(p)) for p in paths)
    return {"bytes": 2 * c["layers"] * c["H"] * moved * _row_bytes(c) + 12 * sum(map(len, paths)), "flops": 0}


# ------------------------------------------------------------------ page format
def _nib_at(D, dev):
    """Where byte (row, o) of 16 rows of nibbles lies among their 16 D / 2 bytes."""
    rb = D // 2
    r, o = torch.meshgrid(torch.arange(16, device=dev), torch.arange(rb, device=dev), indexing="ij")
    q = r * (rb // 16) + o // 16
    line = q // 8
    return line * 128 + (((q % 8) ^ (2 * (line % 4))) * 16) + o % 16


def _bf_at(D, dev):
    """Where element (row, i) of 16 rows of bf16 lies among their 16 D elements."""
    r, i = torch.meshgrid(torch.arange(16, device=dev), torch.arange(D, device=dev), indexing="ij")
    return r * D + (((i // 8) ^ (r % 8)) * 8) + i % 8


def _row_at(c, dev):
    """[page][row bytes]: where the bytes of a row lie in its record."""
    D, nb = c["D"], c["page"] // 16
    b = torch.arange(nb, device=dev)[:, None, None]
    if c["fmt"] == "bf16":
        e = 2 * _bf_at(D, dev)
        k = torch.stack([e, e + 1], -1).reshape(16, -1)
        return (b * 64 * D + torch.cat([k, k + 32 * D], -1)).reshape(c["page"], -1)
    rb, ng = D // 2, D // c["G"]
    at, bb = _nib_at(D, dev), 32 * rb + 64 * ng
    sc = 32 * rb + torch.arange(16, device=dev)[:, None] * 2 * ng + torch.arange(2 * ng, device=dev)
    return torch.cat([b * bb + torch.cat([at, at + 16 * rb, sc, sc + 32 * ng], -1), nb * bb + b * 32 * rb + torch.cat([at, at + 16 * rb], -1)],
                     -1).reshape(c["page"], -1)


def _quantise(x, G):
    """Codes (q4, r) and fp16 scales of rows x [..., D] in groups of G."""
    v = x.reshape(*x.shape[:-1], x.shape[-1] // G, G)
    s = (v.abs().amax(-1) / 7).half()
    f = s.to(v.dtype).unsqueeze(-1)
    t = torch.where(f == 0, torch.zeros_like(v), v / f)
    q = t.round().clamp(-8, 7)
    r = ((t - q) * 16).round().clamp(-8, 7)
    return q.reshape(x.shape), r.reshape(x.shape), s


def _pack_pages(K, V, c):
    """Records [n][H][record] of rows K, V fp32 [n][H][page][D]; rows with NaN get NaN scales."""
    n, H, P, D = K.shape
    nb = P // 16
    if c["fmt"] == "bf16":
        at = _bf_at(D, K.device).reshape(-1)
        got = torch.empty(n, H, nb, 2, 16 * D, dtype=torch.bfloat16, device=K.device)
        got[:, :, :, 0, at] = K.reshape(n, H, nb, 16 * D).bfloat16()
        got[:, :, :, 1, at] = V.reshape(n, H, nb, 16 * D).bfloat16()
        return got.view(torch.uint8).reshape(n, H, -1)
    at = _nib_at(D, K.device).reshape(-1)
    base, resid, sc = [], [], []
    for x in (K, V):
        q, r, s = _quantise(x, c["G"])
        put = []
        for code in (q, r):
            u = (code.nan_to_num(0.0) + 8).to(torch.uint8).reshape(n, H, nb, 16 * D // 2, 2)
            w = torch.empty(n, H, nb, 16 * D // 2, dtype=torch.uint8, device=K.device)
            w[..., at] = u[..., 0] | (u[..., 1] << 4)
            put.append(w)
        base.append(put[0])
        resid.append(put[1])
        sc.append(s.reshape(n, H, nb, -1).view(torch.uint8))
    b = torch.cat([base[0], base[1], sc[0], sc[1]], -1).reshape(n, H, -1)
    return torch.cat([b, torch.cat(resid, -1).reshape(n, H, -1)], -1)


def _unpack_pages(rec, c, planes):
    """K, V fp32 [..., page, D] of records uint8 [..., record]."""
    D, P, G = c["D"], c["page"], c["G"]
    nb, lead = P // 16, rec.shape[:-1]
    if c["fmt"] == "bf16":
        x = rec.view(torch.bfloat16).reshape(*lead, nb, 2, 16 * D)[..., _bf_at(D, rec.device).reshape(-1)].float()
        return x[..., 0, :].reshape(*lead, P, D), x[..., 1, :].reshape(*lead, P, D)
    rb, ng = D // 2, D // G
    bb = 32 * rb + 64 * ng
    base = rec[..., :nb * bb].reshape(*lead, nb, bb)
    more = rec[..., nb * bb:].reshape(*lead, nb, 2, 16 * rb)
    at = _nib_at(D, rec.device).reshape(-1)
    s = base[..., 32 * rb:].contiguous().view(torch.float16).float().reshape(*lead, nb, 2, 16, ng, 1)
    code = base[..., :32 * rb].reshape(*lead, nb, 2, 16 * rb)[..., at]
    v = torch.stack([code & 15, code >> 4], -1).float() - 8
    if planes == 2:
        code = more[..., at]
        v = v * 16 + (torch.stack([code & 15, code >> 4], -1).float() - 8)
        s = s / 16
    v = (v.reshape(*lead, nb, 2, 16, ng, G) * s).reshape(*lead, nb, 2, 16, D)
    return v[..., 0, :, :].reshape(*lead, P, D), v[..., 1, :, :].reshape(*lead, P, D)


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rows(shape, g, D):
    """Rows as a trained model's layers give them: a few channels larger than the rest."""
    ch = 1 + 3 * (torch.rand(D, generator=g, device="cuda") ** 8)
    return torch.randn(*shape, D, generator=g, device="cuda") * ch


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _table(c, rows, g):
    """Page ids [B][W] of sequences of `rows` rows, in any order, and how many pages the pool has."""
    need = [-(-n // c["page"]) for n in rows]
    W, N = max(max(need), 1) + 2, sum(need) + 3
    table = torch.full((len(rows), W), -1, dtype=torch.int32, device="cuda")
    there = torch.arange(W, device="cuda")[None] < torch.tensor(need, device="cuda")[:, None]
    table[there] = torch.randperm(N, generator=g, device="cuda").int()[:sum(need)]
    return table, there, W, N


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    dev = torch.device("cuda")
    if c["op"] == "norm":
        x = _rows((c["M"],), g, c["K"]) * torch.exp(torch.randn(c["M"], 1, generator=g, device=dev))
        kind = lambda t, name: t.to(getattr(torch, name)) if name else None  # noqa: E731
        return {"c": c, "x": kind(x, c["x"]), "add": kind(_rows((c["M"],), g, c["K"]), c["add"]),
                "w": kind(1 + 0.2 * torch.randn(c["K"], generator=g, device=dev), c["w"])}
    trees, paths = _trees(c)
    B, M = c["B"], c["M"]
    parents = _i32(trees)
    if c["op"] == "accept":
        tokens = torch.randint(0, c["V"], (B, M), generator=g, device=dev, dtype=torch.int32)
        logits = 3 * torch.randn(B, M, c["V"], generator=g, device=dev)
        # along each path the target's choice is the drafted token
        at = [(b, p[j], p[j + 1]) for b, p in enumerate(paths) for j in range(len(p) - 1)]
        if at:
            b, up, down = torch.tensor(at, device=dev).T
            logits[b, up, tokens[b, down].long()] = 30.0
        return {"c": c, "parents": parents, "tokens": tokens, "logits": logits}
    if c["op"] == "keep":
        bases = _bases(c)
        table, _, W, N = _table(c, [n + M for n in bases], g)
        L = max(map(len, paths))
        data = torch.randint(0, 256, (c["layers"] * N * c["H"] * _record(c),), generator=g, device=dev, dtype=torch.uint8)
        return {"c": c, "data": data, "table": table, "W": W, "N": N, "first": _i32(bases), "seqs": torch.arange(B, device=dev).int(),
                "path": _i32([p + [-1] * (L - len(p)) for p in paths]), "count": _i32([len(p) for p in paths])}
    lens = [n + M for n in _bases(c)]
    P = c["page"]
    table, there, W, N = _table(c, lens, g)
    # rows that a sequence has: those past its end, and the rows of unused nodes, hold NaN
    valid = torch.zeros(N, P, dtype=torch.bool, device=dev)
    row = torch.arange(W * P, device=dev)[None]
    node = row - (_i32(lens).long()[:, None] - M)
    fine = (node < 0) | ((node < M) & (parents.gather(1, node.clamp(0, M - 1)) >= -1))
    valid[table[there].long()] = fine.reshape(B, W, P)[there]
    data = torch.empty(N, c["H"], _record(c), dtype=torch.uint8, device=dev)
    step = max(1, (1 << 27) // (c["H"] * P * c["D"]))
    for a in range(0, N, step):     # a part of the pages at a time
        ok = valid[a:a + step, None, :, None]
        kv = [torch.where(ok, _rows((ok.shape[0], c["H"], P), g, c["D"]), torch.nan) for _ in range(2)]
        data[a:a + step] = _pack_pages(kv[0], kv[1], c)
    q = _rows((B, M, c["Hq"]), g, c["D"]).bfloat16()
    slopes = 2.0 ** (-8.0 * (torch.arange(c["Hq"], device=dev) + 1) / c["Hq"]) if c["slopes"] else None
    return {"c": c, "q": q, "data": data.reshape(-1), "table": table, "lens": _i32(lens), "N": N, "W": W, "parents": parents,
            "slopes": None if slopes is None else slopes.float(), "scale": c["D"] ** -0.5}


# ------------------------------------------------------------------ plain forms
def _closure(parents):
    """fp32 [B][M][M]: 1 where node j is node m or above it; and which nodes are used.  The inverse of
    I - (child, parent) sums that matrix' powers, whose entries are 0 or 1."""
    B, M = parents.shape
    up = (parents[..., None] == torch.arange(M, device=parents.device)).float()
    eye = torch.eye(M, device=parents.device)
    anc = torch.linalg.solve_triangular(eye - up, eye.expand(B, M, M), upper=False, unitriangular=True)
    used = parents >= -1
    return anc * used[..., None], used


def _plain_norm(s):
    c = s["c"]
    x = s["x"]
    got = {}
    if s["add"] is not None:
        x = got["sum"] = (x.float() + s["add"].float()).to(x.dtype)
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6)
    if s["w"] is not None:
        y = y * s["w"].float()
    if not c["int8"]:
        got["y"] = y.bfloat16()
        return got
    z = y.abs().amax(-1, keepdim=True) / torch.full((), 127.0, device=y.device)
    code = torch.where(z > 0, y / z, 0).round().clamp(-127, 127)
    return {**got, "y": (code * z).bfloat16(), "scale": z[:, 0]}


def _plain_attend(s):
    c = s["c"]
    B, M, Hq, H, D, P = c["B"], c["M"], c["Hq"], c["H"], c["D"], c["page"]
    W = s["W"] - 2
    rec = s["data"].view(s["N"], H, -1)[s["table"][:, :W].clamp(min=0).long()]        # [B][W][H][record]
    K, V = (t.transpose(1, 2).reshape(B, H, W * P, D) for t in _unpack_pages(rec, c, c["planes"]))
    key = torch.arange(W * P, device=K.device)
    anc, used = _closure(s["parents"])
    depth = anc.sum(-1) - 1                                                            # [B][M]
    base = s["lens"].long()[:, None] - M
    node = key[None] - base                                                            # [B][keys]
    inside = (node >= 0) & (node < M)
    at = node.clamp(0, M - 1)
    there = ((node < 0) | (inside & used.gather(1, at)))[:, None, :, None]
    K, V = K.masked_fill(~there, 0), V.masked_fill(~there, 0)
    q = s["q"].float().reshape(B, M, H, Hq // H, D).permute(0, 2, 3, 1, 4)            # [B][H][g][M][D]
    sc = s["scale"] * (q.reshape(B, H, -1, D) @ K.transpose(2, 3)).reshape(B, H, -1, M, W * P)
    if c["cap"]:
        sc = c["cap"] * torch.tanh(sc / c["cap"])
    pos = torch.where(inside, base + depth.gather(1, at), key[None].float())           # of the rows
    dist = base[..., None] + depth[..., None] - pos[:, None]                           # [B][M][keys]
    if s["slopes"] is not None:
        sc = sc - s["slopes"].reshape(1, H, -1, 1, 1) * dist[:, None, None]
    up = anc.gather(2, at[:, None].expand(B, M, -1)) > 0
    seen = torch.where(inside[:, None], up, (node < 0)[:, None] & used[..., None])
    if c["window"]:
        seen &= dist < c["window"]
    seen = seen[:, None, None]
    sc = sc.masked_fill(~seen, -math.inf)
    p = torch.exp(sc - sc.amax(-1, keepdim=True).clamp(min=-3e38))
    o = (p.reshape(B, H, -1, W * P) @ V).reshape(B, H, -1, M, D)
    o = torch.where(seen.any(-1, keepdim=True), o / p.sum(-1, keepdim=True), 0)
    return o.permute(0, 3, 1, 2, 4).reshape(B, M, Hq, D).bfloat16()


def _plain_accept(s):
    c = s["c"]
    B, M, V = c["B"], c["M"], c["V"]
    parents, tokens, x = s["parents"].long(), s["tokens"], s["logits"]
    word = torch.arange(V, device=x.device, dtype=torch.int32)
    t = torch.where(x == x.amax(-1, keepdim=True), word, V).amin(-1)                   # lowest index on ties
    anc, used = _closure(parents)
    m = torch.arange(M, device=x.device)
    hit = (parents >= 0) & (tokens == t.gather(1, parents.clamp(min=0)))
    # of several children that match, the lowest goes on
    twin = (parents[:, :, None] == parents[:, None]) & hit[:, None] & (m[None, :, None] > m[None, None])
    hit &= ~twin.any(-1)
    wrong = (~hit).float()
    wrong[:, 0] = 0
    on = used & (anc[..., 0] > 0) & ((anc * wrong[:, None]).sum(-1) == 0)
    path = torch.sort(torch.where(on, m, M), -1).values
    ok = path < M
    out = torch.where(ok, t.gather(1, path.clamp(max=M - 1)), -1)
    bits = torch.nn.functional.pad(anc, (0, -M % 32)).reshape(B, M, -1, 32).long() << torch.arange(32, device=x.device)
    return {"depth": torch.where(used, anc.sum(-1) - 1, -1).int(), "bits": bits.sum(-1).int(), "tok": out.int(),
            "count": on.sum(-1).int(), "path": torch.where(ok, path, -1).int()}


def _plain_keep(s):
    c = s["c"]
    P, H = c["page"], c["H"]
    j = torch.arange(s["path"].shape[1], device=s["path"].device)
    here = j[None] < s["count"][:, None]
    first = s["first"].long()[:, None]
    src, dst = (first + s["path"])[here], (first + j)[here]
    seq = s["seqs"].long()[:, None].expand(here.shape)[here]
    at = _row_at(c, j.device)

    def place(row):
        rec = s["table"][seq, row // P].long()[:, None] * H + torch.arange(H, device=row.device)
        return rec[..., None] * _record(c) + at[row % P][:, None]

    d = s["data"].view(c["layers"], -1)
    d[:, place(dst)] = d[:, place(src)]
    return s["data"].view(torch.int32)


def run(s):
    if own:
        return _own(s)
    return {"norm": _plain_norm, "attend": _plain_attend, "accept": _plain_accept, "keep": _plain_keep}[s["c"]["op"]](s)


# ------------------------------------------------------------------ through the package
def _own(s):
    from quantized_self_speculative_gb300 import nq
    c = s["c"]
    if c["op"] == "norm":
        got = nq.rms_norm(s["x"], s["w"], eps=1e-6, add=s["add"], quantize=c["int8"])
        out = {} if s["add"] is None else {"sum": got[0]}
        if not c["int8"]:
            return {**out, "y": got[1]}
        code, z = got[1], got[2]
        y = torch.empty(code.shape, dtype=torch.bfloat16, device=code.device)
        return {**out, "y": torch.mul(code, z[:, None], out=y), "scale": z}
    if c["op"] == "accept":
        tree = nq.Tree(s["parents"])
        tok, count, path = nq.accept_tree(s["tokens"], s["logits"], tree)
        return {"depth": tree.depth, "bits": tree.bits, "tok": tok, "count": count, "path": path}
    if "pool" not in s:                         # handles that a program keeps
        fmt = nq.KV_BF16 if c["fmt"] == "bf16" else nq.KV_NESTED44
        s["pool"] = nq.PagePool(c.get("layers", 1), s["N"], c["page"], c["H"], c["D"], fmt, group=c["G"], data=s["data"])
        s["map"] = nq.PageMap(s["table"].shape[0], s["W"], s["N"], c["page"], table=s["table"])
    if c["op"] == "keep":
        s["pool"].keep(s["map"], s["seqs"], s["first"], s["path"], s["count"])
        return s["data"].view(torch.int32)
    if "tree" not in s:                         # one plan serves all layers of a round
        s["tree"] = nq.Tree(s["parents"], window=c["window"])
    return s["pool"].attention(0, s["map"], s["q"], s["lens"], c["planes"], s["scale"], softcap=c["cap"], window=c["window"],
                               slopes=s["slopes"], tree=s["tree"])


# ------------------------------------------------------------------ 64 bits
def _cached(s, seq, row):
    """K, V [H][rows][D] in 64 bits of one sequence's rows, read byte by byte at their addresses."""
    c = s["c"]
    H, D, P, G = c["H"], c["D"], c["page"], c["G"]
    dev = s["data"].device
    rec = c["page"] * (4 * D if c["fmt"] == "bf16" else 2 * D + 4 * (D // G))
    base = (s["table"][seq].long()[row // P] * H + torch.arange(H, device=dev)[:, None]) * rec      # [H][n]
    r, b = row % 16, (row % P) // 16
    d = torch.arange(D, device=dev)
    got = []
    if c["fmt"] == "bf16":
        off = r[:, None] * D + (((d // 8)[None] ^ (r % 8)[:, None]) * 8) + d % 8
        for which in range(2):
            at = (base // 2 + b * 32 * D + which * 16 * D)[..., None] + off
            got.append(s["data"].view(torch.bfloat16)[at].double())
        return got
    unit = 32 * (D // 2) + 64 * (D // G)
    chunk = r[:, None] * (D // 32) + (d // 32)[None]
    line = torch.div(chunk, 8, rounding_mode="floor")
    off = line * 128 + ((chunk % 8) ^ (2 * (line % 4))) * 16 + (d // 2 % 16)
    for which in range(2):
        lo = s["data"][(base + b * unit + which * 8 * D)[..., None] + off]
        hi = s["data"][(base + (P // 16) * unit + b * 16 * D + which * 8 * D)[..., None] + off]
        nib = lambda u: (torch.where(d % 2 == 0, u & 15, u >> 4).double() - 8)  # noqa: E731
        sat = (base + b * unit + 16 * D + which * 32 * (D // G)) // 2 + r * (D // G)
        sc = s["data"].view(torch.float16)[sat[..., None] + d // G].double()
        got.append(sc * (nib(lo) + (nib(hi) / 16 if c["planes"] == 2 else 0)))
    return got


def exact(case, seed):
    if case["op"] in ("accept", "keep"):
        return None                     # whole numbers and bytes
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "norm":
        got, x = {}, s["x"].double()
        if s["add"] is not None:
            got["sum"] = x + s["add"].double()
            x = got["sum"].to(s["x"].dtype).double()         # the norm is that of the residual as it is kept
        y = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["K"] + 1e-6)
        if s["w"] is not None:
            y = y * s["w"].double()
        if not c["int8"]:
            return {**got, "y": y}
        z = y.abs().max(-1, keepdim=True).values / 127
        return {**got, "y": torch.nan_to_num(torch.round(y / z)) * z, "scale": z[:, 0]}
    B, M, Hq, H, D = c["B"], c["M"], c["Hq"], c["H"], c["D"]
    trees = _trees(c)[0]
    out = torch.zeros(B, M, Hq, D, dtype=torch.float64, device="cuda")
    for b, base in enumerate(_bases(c)):
        up = []                          # of each node: the nodes from the root down to it
        for m, p in enumerate(trees[b]):
            up.append([] if p < -1 else ([] if p < 0 else up[p]) + [m])
        K, V = _cached(s, b, torch.arange(base + M, device="cuda"))
        for m in range(M):
            if not up[m]:
                continue
            at = base + len(up[m]) - 1
            lo = max(0, at - c["window"] + 1) if c["window"] else 0
            pos = torch.arange(min(lo, base), base + len(up[m]), device="cuda")
            row = torch.cat([pos[:base - min(lo, base)], base + torch.tensor(up[m], device="cuda")])
            pos, row = pos[pos >= lo], row[pos >= lo]
            q = s["q"][b, m].double().reshape(H, Hq // H, D)
            x = s["scale"] * torch.einsum("hgd,hnd->hgn", q, K[:, row])
            if c["cap"]:
                x = c["cap"] * torch.tanh(x / c["cap"])
            if s["slopes"] is not None:
                x = x + s["slopes"].double().reshape(H, -1, 1) * (pos - at)
            out[b, m] = torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1), V[:, row]).reshape(Hq, D)
    return out
