"""Measured cases of the paged-cache operators: rotary positions, appending to
pages, attention over pages, and the bookkeeping of pages.

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
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decoding step of 16 sequences: the q and k heads of one layer, from the fused fp32 linear output
        {"name": "rope_step", "op": "rope", "T": 16, "H": 40, "D": 128, "rot": 128, "layout": "half", "scaling": "none",
         "theta": 500000.0, "factor": 1.0, "old": 0, "maxpos": 8192, "src": "float32", "dst": "bfloat16", "inverse": False},
        # a long prompt's queries, interleaved pairs on part of the head, positions far past the trained length
        {"name": "rope_prompt", "op": "rope", "T": 16384, "H": 32, "D": 128, "rot": 64, "layout": "interleaved", "scaling": "parts",
         "theta": 10000.0, "factor": 16.0, "old": 4096, "maxpos": 131072, "src": "bfloat16", "dst": "bfloat16", "inverse": False},
        # the verify pass of a batched round, 16 sequences of k + 1 = 9 rows: rotate q and k, quantise k and v into pages
        {"name": "append_verify", "op": "append", "fmt": "nested", "T": 144, "B": 16, "Hq": 32, "H": 8, "D": 128, "G": 128, "page": 16,
         "rot": 128, "layout": "half", "scaling": "none", "theta": 500000.0, "factor": 1.0, "old": 0, "start": 2000, "planes": 2},
        # prompts of several sequences entering the cache at once, groups of 64, MHA heads
        {"name": "append_prompt", "op": "append", "fmt": "nested", "T": 8191, "B": 5, "Hq": 32, "H": 32, "D": 128, "G": 64, "page": 64,
         "rot": 128, "layout": "half", "scaling": "linear", "theta": 10000.0, "factor": 8.0, "old": 0, "start": 0, "planes": 2},
        # the draft's single new token early in a conversation: latency
        {"name": "attend_draft_short", "op": "attend", "fmt": "nested", "planes": 1, "B": 1, "M": 1, "Hq": 32, "H": 32, "D": 128, "G": 128,
         "page": 16, "lo": 517, "hi": 517, "mix": 1, "cap": 0.0, "window": 0, "slopes": False},
        # the draft's single new token at 32K rows, MHA heads: the 4-bit view streamed once
        {"name": "attend_draft_32k", "op": "attend", "fmt": "nested", "planes": 1, "B": 1, "M": 1, "Hq": 32, "H": 32, "D": 128, "G": 128,
         "page": 64, "lo": 32768, "hi": 32768, "mix": 1, "cap": 0.0, "window": 0, "slopes": False},
        # the verify read of a batched round: 16 ragged sequences, k + 1 = 9 rows, grouped-query heads, the 8-bit view
        {"name": "attend_verify_batch", "op": "attend", "fmt": "nested", "planes": 2, "B": 16, "M": 9, "Hq": 32, "H": 8, "D": 128, "G": 128,
         "page": 16, "lo": 301, "hi": 4099, "mix": 2, "cap": 0.0, "window": 0, "slopes": False},
        # long contexts in 16 bits, one new token each
        {"name": "attend_bf16_long", "op": "attend", "fmt": "bf16", "planes": 2, "B": 4, "M": 1, "Hq": 32, "H": 8, "D": 128, "G": 128,
         "page": 128, "lo": 40001, "hi": 131072, "mix": 3, "cap": 0.0, "window": 0, "slopes": False},
        # capped scores with a distance bias in a sliding window, small heads
        {"name": "attend_capped_window", "op": "attend", "fmt": "nested", "planes": 2, "B": 8, "M": 2, "Hq": 16, "H": 4, "D": 64, "G": 64,
         "page": 32, "lo": 900, "hi": 9001, "mix": 4, "cap": 30.0, "window": 4096, "slopes": True},
        # after a round: drop the rejected rows of 16 sequences, make room for the next k + 1
        {"name": "pages_rollback", "op": "pages", "kind": "rollback", "layers": 1, "N": 4096, "S": 16, "W": 300, "H": 8, "D": 128, "G": 128,
         "fmt": "nested", "page": 16, "lo": 1000, "hi": 4000, "mix": 5, "new": 9},
        # 32 continuations of one prompt reordered by their parents; their shared last pages are copied before the next write
        {"name": "pages_beams", "op": "pages", "kind": "beams", "layers": 32, "N": 512, "S": 32, "W": 160, "H": 8, "D": 128, "G": 128,
         "fmt": "nested", "page": 16, "lo": 2050, "hi": 2120, "mix": 6, "new": 1},
        # a fragmented pool of all layers moved down to its lowest pages
        {"name": "pages_compact", "op": "pages", "kind": "compact", "layers": 32, "N": 2048, "S": 48, "W": 64, "H": 8, "D": 128, "G": 128,
         "fmt": "nested", "page": 16, "lo": 200, "hi": 700, "mix": 7, "new": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "pages"])
    D = rng.choice([64, 128, 128])
    G = rng.choice([64, D])
    fmt = rng.choice(["nested", "nested", "bf16"])
    H = rng.choice([1, 2, 4, 8, 32] if op in ("append", "attend") else [2, 4, 8])
    g = rng.choice([1, 2, 4, 7, 8]) if H < 32 else 1
    page = rng.choice([16, 32, 64, 128])
    ro = {"layout": rng.choice(["half", "interleaved"]), "scaling": rng.choice(["none", "linear", "ntk", "parts"]),
          "theta": rng.choice([10000.0, 500000.0]), "factor": rng.choice([2.0, 8.0]), "old": 4096, "rot": rng.choice([D, D, D // 2])}
    if op == "rope":
        return {"op": op, "T": _log(rng, 1, 12000), "H": rng.choice([1, 4, 8, 28, 32, 40]), "D": D, **ro, "maxpos": _log(rng, 100, 1000000),
                "src": rng.choice(["float32", "bfloat16"]), "dst": rng.choice(["float32", "bfloat16"]), "inverse": rng.random() < 0.3}
    if op == "append":
        B = _log(rng, 1, 24)
        return {"op": op, "fmt": fmt, "T": B + _log(rng, 1, 6000), "B": B, "Hq": H * g, "H": H, "D": D, "G": G, "page": page, **ro,
                "start": _log(rng, 1, 3000), "planes": rng.choice([1, 2])}
    if op == "attend":
        B = _log(rng, 1, 40)
        hi = _log(rng, 1, max(2, min(40000, 4000000 // (B * H))))
        return {"op": op, "fmt": fmt, "planes": rng.choice([1, 2]), "B": B, "M": rng.choice([1, 1, 2, 5, 9]), "Hq": H * g, "H": H, "D": D,
                "G": G, "page": page, "lo": rng.choice([hi, max(0, hi // 7), 0]), "hi": hi, "mix": rng.randrange(1 << 30),
                "cap": rng.choice([0.0, 0.0, 30.0]), "window": rng.choice([0, 0, max(1, hi // 3)]), "slopes": rng.random() < 0.3}
    lo = _log(rng, 20, 1500)
    hi = lo + _log(rng, 1, 400)
    S = _log(rng, 2, 40)
    W = (hi + 40) // page + 3
    c = {"op": op, "kind": rng.choice(["rollback", "beams", "compact"]), "layers": _log(rng, 1, 16), "N": 2 * S * W + 7, "S": S, "W": W,
         "H": H, "D": D, "G": G, "fmt": fmt, "page": page, "lo": lo, "hi": hi, "mix": rng.randrange(1 << 30), "new": rng.choice([1, 5, 9, 33])}
    c["layers"] = max(1, min(c["layers"], 2200000000 // (c["N"] * H * _record(c))))
    return c


def _lens(c):
    r = random.Random(c["mix"])
    n = c["B"] if "B" in c else c["S"]
    got = [r.randint(c["lo"], c["hi"]) for _ in range(n)]
    got[0] = c["hi"]
    return got


def _row_bytes(c, planes=2):
    """K and V bytes of one row of one head."""
    if c["fmt"] == "bf16":
        return 4 * c["D"]
    return c["D"] * planes + 4 * (c["D"] // c["G"])


def _record(c):
    return c["page"] * _row_bytes(c)


def work(c):
    el = {"float32": 4, "bfloat16": 2}
    if c["op"] == "rope":
        n = c["T"] * c["H"] * c["D"]
        return {"bytes": n * (el[c["src"]] + el[c["dst"]]) + 4 * c["T"], "flops": 3 * n}
    if c["op"] == "append":   # inputs, rotated q, cached rows written; then read and returned as values
        T, D = c["T"], c["D"]
        return {"bytes": T * (4 * D * (c["Hq"] + 2 * c["H"]) + 2 * D * c["Hq"] + c["H"] * (_row_bytes(c) + _row_bytes(c, c["planes"]) + 4 * D) + 16),
                "flops": T * D * (3 * c["Hq"] + 20 * c["H"])}
    if c["op"] == "attend":
        rows = [min(n, c["window"] + c["M"] - 1) if c["window"] else n for n in _lens(c)]
        return {"bytes": sum(rows) * c["H"] * _row_bytes(c, c["planes"]) + 4 * c["B"] * c["M"] * c["Hq"] * c["D"] + 4 * sum(-(-n // c["page"]) for n in rows),
                "flops": 4 * sum(rows) * c["M"] * c["Hq"] * c["D"]}
    page = c["layers"] * c["H"] * _record(c)
    book = 4 * (c["S"] * c["W"] + c["S"] + c["N"])
    if c["kind"] == "rollback":
        return {"bytes": 4 * c["N"] + 8 * c["S"] * (3 + c["new"] // c["page"]), "flops": 0}
    if c["kind"] == "beams":
        par = _parents(c)
        copied = sum(par.count(p) - 1 for p in set(par))
        return {"bytes": 2 * book + 2 * copied * page, "flops": 0}
    used = sum(-(-n // c["page"]) for n in _lens(c))
    return {"bytes": 2 * book + 2 * page * used * (c["N"] - used) // c["N"], "flops": 0}


def _parents(c):
    r = random.Random(c["mix"] + 1)
    return [r.randrange(c["S"]) for _ in range(c["S"])]


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
    base, resid = [], []
    sc = []
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
    """Rows as a trained model's heads give them: a few channels larger than the rest."""
    ch = 1 + 3 * (torch.rand(D, generator=g, device="cuda") ** 8)
    return torch.randn(*shape, D, generator=g, device="cuda") * ch


def prepare(case, seed):
    c, g = dict(case), _gen(seed)
    dev = torch.device("cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    if c["op"] == "rope":
        # the heads of one tensor among the columns of a fused linear's output
        wide = _rows((c["T"], c["H"] + 2), g, c["D"]).to(getattr(torch, c["src"]))
        pos = torch.randint(0, c["maxpos"], (c["T"],), generator=g, device=dev, dtype=torch.int32)
        return {"c": c, "x": wide[:, :c["H"]], "pos": pos}
    if c["op"] == "append":
        T, B, P = c["T"], c["B"], c["page"]
        r = random.Random(seed)
        cuts = sorted(r.sample(range(1, T), B - 1))
        n = [b - a for a, b in zip([0] + cuts, cuts + [T])]
        start = [r.randint(0, c["start"]) for _ in n]
        W = max(s + k for s, k in zip(start, n)) // P + 1
        seqs = torch.repeat_interleave(torch.arange(B, device=dev), torch.tensor(n, device=dev)).int()
        first = torch.tensor([0] + cuts, device=dev)
        pos = (torch.arange(T, device=dev) - first[seqs.long()] + torch.tensor(start, device=dev)[seqs.long()]).int()
        N = B * W + 3
        table = torch.randperm(N, generator=g, device=dev)[:B * W].reshape(B, W).int()
        data = torch.zeros(N * c["H"] * _record(c), dtype=torch.uint8, device=dev)
        qkv = _rows((T, c["Hq"] + 2 * c["H"]), g, c["D"])
        return {"c": c, "qkv": qkv, "seqs": seqs, "pos": pos, "table": table.contiguous(), "data": data, "N": N, "W": W}
    if c["op"] == "attend":
        lens, P = _lens(c), c["page"]
        need = [-(-n // P) for n in lens]
        W = max(max(need), 1) + 2
        N = sum(need) + 3
        ids = torch.randperm(N, generator=g, device=dev).int()
        table = torch.full((c["B"], W), -1, dtype=torch.int32, device=dev)
        held = torch.tensor(need, device=dev)
        there = torch.arange(W, device=dev)[None] < held[:, None]
        table[there] = ids[:sum(need)]
        valid = torch.zeros(N, P, dtype=torch.bool, device=dev)
        rows_in = (i32(lens).long()[:, None] - torch.arange(W, device=dev)[None] * P).clamp(0, P)
        valid[table[there].long()] = torch.arange(P, device=dev)[None] < rows_in[there][:, None]
        data = torch.empty(N, c["H"], _record(c), dtype=torch.uint8, device=dev)
        step = max(1, (1 << 27) // (c["H"] * P * c["D"]))
        for a in range(0, N, step):     # a part of the pages at a time: rows past a sequence's end hold NaN
            ok = valid[a:a + step, None, :, None]
            kv = [torch.where(ok, _rows((ok.shape[0], c["H"], P), g, c["D"]), torch.nan) for _ in range(2)]
            data[a:a + step] = _pack_pages(kv[0], kv[1], c)
        q = _rows((c["B"], c["M"], c["Hq"]), g, c["D"]).bfloat16()
        slopes = 2.0 ** (-8.0 * (torch.arange(c["Hq"], device=dev) + 1) / c["Hq"]) if c["slopes"] else None
        return {"c": c, "q": q, "data": data.reshape(-1), "table": table, "lens": i32(lens), "N": N, "W": W,
                "slopes": None if slopes is None else slopes.float(), "scale": c["D"] ** -0.5}
    N, S, W, P = c["N"], c["S"], c["W"], c["page"]
    lens = _lens(c)
    book = torch.full((S * W + S + N,), -1, dtype=torch.int32)
    table, held, ref = book[:S * W].view(S, W), book[S * W:S * W + S], book[S * W + S:]
    ref.zero_()
    r = random.Random(seed)
    ids = list(range(N))
    r.shuffle(ids)
    shared = (c["lo"] - 1) // P if c["kind"] == "beams" else 0
    head = [ids.pop() for _ in range(shared)]
    for s, n in enumerate(lens):
        own_pages = head + [ids.pop() for _ in range(-(-n // P) - shared)]
        table[s, :len(own_pages)] = torch.tensor(own_pages, dtype=torch.int32)
        held[s] = len(own_pages)
        ref += torch.bincount(torch.tensor(own_pages), minlength=N).int()
    par = _parents(c)
    after = [lens[p] for p in par] if c["kind"] == "beams" else [max(0, n - r.randint(0, 8)) for n in lens]
    order = list(range(S))
    if c["kind"] != "beams":
        r.shuffle(order)
    data = torch.randint(0, 256, (c["layers"] * N * c["H"] * _record(c),), generator=g, device=dev, dtype=torch.uint8)
    snap = book.to(dev)
    return {"c": c, "snap": snap, "book": snap.clone(), "data": data, "seqs": i32(order), "src": i32([par[s] for s in order]),
            "rows": i32([after[s] for s in order]), "last": i32([after[s] + c["new"] for s in order]), "N": N, "W": W}


# ------------------------------------------------------------------ plain forms
def _freqs(c):
    """Radians per position of each pair, and the factor on both rotated values."""
    i = torch.arange(c["rot"] // 2, dtype=torch.float64, device="cuda")
    theta, f = c["theta"], c["factor"]
    if c["scaling"] == "ntk":
        theta = theta * f ** (c["rot"] / (c["rot"] - 2))
    w = theta ** (-2 * i / c["rot"])
    if c["scaling"] == "linear":
        w = w / f
    if c["scaling"] == "parts":
        turns = c["old"] * w / (2 * math.pi)
        keep = ((turns - 1) / 31).clamp(0, 1)
        return w * keep + w / f * (1 - keep), 0.1 * math.log(f) + 1
    return w, 1.0


def _rotate(x, pos, c, inverse=False):
    """x fp32 [T][H][D] rotated by its positions; the angles in 64 bits."""
    w, a = _freqs(c)
    ang = pos.double()[:, None] * w
    cos, sin = (a * ang.cos()).float()[:, None], (a * ang.sin()).float()[:, None]
    if inverse:
        sin = -sin
    rot = c["rot"]
    head = x[..., :rot]
    if c["layout"] == "half":
        u, v = head[..., :rot // 2], head[..., rot // 2:]
        y = torch.cat([u * cos - v * sin, u * sin + v * cos], -1)
    else:
        u, v = head[..., 0::2], head[..., 1::2]
        y = torch.stack([u * cos - v * sin, u * sin + v * cos], -1).flatten(-2)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_append(s):
    c = s["c"]
    H, Hq, D, P = c["H"], c["Hq"], c["D"], c["page"]
    nb, rb, ng = P // 16, D // 2, D // c["G"]
    q = _rotate(s["qkv"][:, :Hq], s["pos"], c).bfloat16()
    k, v = _rotate(s["qkv"][:, Hq:Hq + H], s["pos"], c), s["qkv"][:, Hq + H:]
    pos = s["pos"].long()
    pg, row = s["table"][s["seqs"].long(), pos // P].long(), pos % P
    rec = (pg[:, None] * H + torch.arange(H, device=pg.device)) * _record(c)          # [T][H]
    blk, r16 = (row // 16)[:, None], row % 16
    if c["fmt"] == "bf16":
        at = (rec // 2 + blk * 32 * D)[..., None] + _bf_at(D, pg.device)[r16][:, None]
        d16 = s["data"].view(torch.bfloat16)
        k, v = k.bfloat16(), v.bfloat16()
        d16[at], d16[at + 16 * D] = k, v
        return {"q": q, "k": k, "v": v}
    bb = 32 * rb + 64 * ng
    at = _nib_at(D, pg.device)[r16][:, None]
    sat = (r16 * ng)[:, None, None] + torch.arange(ng, device=pg.device)
    out = {"q": q}
    kq, vq = _quantise(k, c["G"]), _quantise(v, c["G"])

    def put(name, codes, shift, sshift):
        q4, r, sc = codes
        nib = lambda t: (t[..., 0::2] + 8).to(torch.uint8) | ((t[..., 1::2] + 8).to(torch.uint8) << 4)  # noqa: E731
        s["data"][(rec + blk * bb)[..., None] + shift + at] = nib(q4)
        s["data"][(rec + nb * bb + blk * 32 * rb)[..., None] + shift + at] = nib(r)
        s["data"].view(torch.float16)[((rec + blk * bb + 32 * rb + sshift) // 2)[..., None] + sat] = sc
        f = sc.float().repeat_interleave(c["G"], -1)
        out[name] = (q4 * f if c["planes"] == 1 else (q4 * 16 + r) * (f / 16)).bfloat16()

    put("k", kq, 0, 0)
    put("v", vq, 16 * rb, 32 * ng)
    return out


def _plain_attend(s):
    c = s["c"]
    B, M, Hq, H, D, P = c["B"], c["M"], c["Hq"], c["H"], c["D"], c["page"]
    W = s["W"] - 2
    rec = s["data"].view(s["N"], H, -1)[s["table"][:, :W].clamp(min=0).long()]        # [B][W][H][record]
    K, V = (t.transpose(1, 2).reshape(B, H, W * P, D) for t in _unpack_pages(rec, c, c["planes"]))
    key = torch.arange(W * P, device=K.device)
    lens = s["lens"].long()
    there = (key[None] < lens[:, None])[:, None, :, None]
    K, V = K.masked_fill(~there, 0), V.masked_fill(~there, 0)
    q = s["q"].float().reshape(B, M, H, Hq // H, D).permute(0, 2, 3, 1, 4)            # [B][H][g][M][D]
    sc = s["scale"] * (q.reshape(B, H, -1, D) @ K.transpose(2, 3)).reshape(B, H, -1, M, W * P)
    if c["cap"]:
        sc = c["cap"] * torch.tanh(sc / c["cap"])
    at = lens[:, None] - M + torch.arange(M, device=K.device)                          # [B][M]
    dist = (at[..., None] - key)[:, None, None]
    if s["slopes"] is not None:
        sc = sc - s["slopes"].reshape(1, H, -1, 1, 1) * dist
    seen = (dist >= 0) & (dist < c["window"]) if c["window"] else dist >= 0
    sc = sc.masked_fill(~seen, -math.inf)
    p = torch.exp(sc - sc.amax(-1, keepdim=True).clamp(min=-3e38))
    o = (p.reshape(B, H, -1, W * P) @ V).reshape(B, H, -1, M, D)
    o = torch.where(seen.any(-1, keepdim=True), o / p.sum(-1, keepdim=True), 0)
    return o.permute(0, 3, 1, 2, 4).reshape(B, M, Hq, D).bfloat16()


def _views(s):
    c = s["c"]
    n = c["S"] * c["W"]
    return s["book"][:n].view(c["S"], c["W"]), s["book"][n:n + c["S"]], s["book"][n + c["S"]:]


def _plain_truncate(s, seqs, rows):
    table, held, ref = _views(s)
    keep = torch.minimum(-(-rows // s["c"]["page"]), held[seqs])
    t = table[seqs]
    gone = (torch.arange(s["W"], device=t.device) >= keep[:, None]) & (t >= 0)
    ref.scatter_add_(0, t.clamp(min=0).long().reshape(-1), -gone.int().reshape(-1))
    table[seqs] = t.masked_fill(gone, -1)
    held[seqs] = keep


def _plain_fork(s, src, dst, rows):
    table, held, ref = _views(s)
    n = torch.minimum(-(-rows // s["c"]["page"]), held[src])
    new, old = table[src], table[dst]
    new = new.masked_fill(torch.arange(s["W"], device=new.device) >= n[:, None], -1)
    ref.scatter_add_(0, new.clamp(min=0).long().reshape(-1), (new >= 0).int().reshape(-1))
    ref.scatter_add_(0, old.clamp(min=0).long().reshape(-1), -(old >= 0).int().reshape(-1))
    table[dst] = new
    held[dst] = n


def _plain_reserve(s, seqs, first, last):
    c = s["c"]
    P, W, N = c["page"], s["W"], s["N"]
    table, held, ref = _views(s)
    t, h = table[seqs], held[seqs]
    j = torch.arange(W, device=t.device)[None]
    need = (-(-last // P))[:, None]
    shared = (j >= (first // P)[:, None]) & (j < torch.minimum(h[:, None], need)) & (ref[t.clamp(min=0).long()] > 1)
    # of a page whose holders all ask for it, the last one keeps it: the others are copied before it
    pid = t[shared].long()
    order = torch.sort(pid, stable=True)
    run = torch.arange(len(pid), device=t.device) - torch.searchsorted(order.values, order.values)
    rank = torch.empty_like(run).scatter_(0, order.indices, run)
    cow = torch.zeros_like(shared)
    cow[shared] = rank < ref[pid] - 1
    fresh = (j >= h[:, None]) & (j < need)
    want = (cow | fresh) & (last <= W * P)[:, None]
    free = torch.nonzero(ref == 0)[:, 0]
    granted = (want.sum(1).cumsum(0) <= len(free)) & (last <= W * P)
    want &= granted[:, None]
    cow &= want
    at = torch.nonzero(want.reshape(-1))[:, 0]
    ids = free[:len(at)].int()
    full = torch.full((W * len(seqs),), -1, dtype=torch.int32, device=t.device).scatter_(0, at, ids).view_as(t)
    old, new = t[cow].long(), full[cow].long()
    d = s["data"].view(torch.int64).view(c["layers"], N, -1)
    d[:, new] = d[:, old]
    ref.scatter_add_(0, old, torch.full_like(old, -1, dtype=torch.int32))
    ref[ids.long()] = 1
    table[seqs] = torch.where(want, full, t)
    held[seqs] = torch.where(granted, torch.maximum(h, need[:, 0]), h)
    return granted.int()


def _plain_compact(s):
    table, held, ref = _views(s)
    used = ref > 0
    U = used.sum()
    ids = torch.arange(s["N"], device=ref.device)
    high, hole = ids[used & (ids >= U)], ids[~used & (ids < U)]
    d = s["data"].view(torch.int64).view(s["c"]["layers"], s["N"], -1)
    d[:, hole] = d[:, high]
    to = ids.clone()
    to[high] = hole
    ref[hole], ref[high] = ref[high], torch.zeros_like(ref[high])
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table))
    return U.int()


def run(s):
    if own:
        return _own(s)
    c = s["c"]
    if c["op"] == "rope":
        return _rotate(s["x"].float(), s["pos"], c, c["inverse"]).to(getattr(torch, c["dst"]))
    if c["op"] == "append":
        return _plain_append(s)
    if c["op"] == "attend":
        return _plain_attend(s)
    s["book"].copy_(s["snap"])          # every pass starts from the same pages
    got = {"book": s["book"]}
    seqs = s["seqs"].long()
    if c["kind"] == "compact":
        got["used"] = _plain_compact(s)
        got["data"] = s["data"].view(torch.int32)
    elif c["kind"] == "beams":
        _plain_fork(s, s["src"].long(), seqs, s["rows"])
        got["granted"] = _plain_reserve(s, seqs, s["rows"], s["last"])
        got["data"] = s["data"].view(torch.int32)
    else:
        _plain_truncate(s, seqs, s["rows"])
        got["granted"] = _plain_reserve(s, seqs, s["rows"], s["last"])
    return got


# ------------------------------------------------------------------ through the package
def _own(s):
    from quantized_self_speculative_gb300 import nq
    c = s["c"]
    if "rope" not in s and "rot" in c:          # plans and handles that a program keeps
        s["rope"] = nq.Rope(c["rot"], theta=c["theta"], layout=c["layout"], scaling=c["scaling"], factor=c["factor"], old_len=c["old"])
    if c["op"] == "rope":
        return nq.rope(s["x"], s["pos"], s["rope"], inverse=c["inverse"], out_dtype=getattr(torch, c["dst"]))
    if "pool" not in s:
        fmt = nq.KV_BF16 if c["fmt"] == "bf16" else nq.KV_NESTED44
        s["pool"] = nq.PagePool(c.get("layers", 1), s["N"], c["page"], c["H"], c["D"], fmt, group=c["G"], data=s["data"])
        if c["op"] == "pages":
            table, held, ref = _views(s)
            s["map"] = nq.PageMap(c["S"], c["W"], s["N"], c["page"], table=table, held=held, ref=ref)
        else:
            s["map"] = nq.PageMap(s["table"].shape[0], s["W"], s["N"], c["page"], table=s["table"])
    pool, pmap = s["pool"], s["map"]
    if c["op"] == "append":
        Hq, H = c["Hq"], c["H"]
        x = s["qkv"]
        q = pool.append(0, pmap, x[:, Hq:Hq + H], x[:, Hq + H:], s["seqs"], s["pos"], rope=s["rope"], q=x[:, :Hq])
        k, v = pool.read(0, pmap, s["seqs"], s["pos"], planes=c["planes"])
        return {"q": q, "k": k, "v": v}
    if c["op"] == "attend":
        return pool.attention(0, pmap, s["q"], s["lens"], c["planes"], s["scale"], softcap=c["cap"], window=c["window"], slopes=s["slopes"])
    s["book"].copy_(s["snap"])
    got = {"book": s["book"]}
    if c["kind"] == "compact":
        got["used"] = pmap.compact(pool).view(())
        got["data"] = s["data"].view(torch.int32)
    elif c["kind"] == "beams":
        pmap.fork(s["src"], s["seqs"], s["rows"])
        got["granted"] = pmap.reserve(pool, s["seqs"], s["rows"], s["last"])
        got["data"] = s["data"].view(torch.int32)
    else:
        pmap.truncate(s["seqs"], s["rows"])
        got["granted"] = pmap.reserve(pool, s["seqs"], s["rows"], s["last"])
    return got


# ------------------------------------------------------------------ 64 bits
def _turned(x, pos, c, sign=1.0):
    """Rows x [T][H][D] as complex pairs times e^(i angle), in 64 bits."""
    R = c["rot"]
    k = torch.arange(0, R, 2, dtype=torch.float64, device=x.device) / R
    base = c["theta"] * (c["factor"] ** (R / (R - 2.0)) if c["scaling"] == "ntk" else 1.0)
    w, amp = torch.exp(-k * math.log(base)), 1.0
    if c["scaling"] == "linear":
        w = w / c["factor"]
    elif c["scaling"] == "parts":
        share = torch.clamp((c["old"] * w / (2 * math.pi) - 1) / 31, 0, 1)
        w = share * w + (1 - share) * w / c["factor"]
        amp = 1 + 0.1 * math.log(c["factor"])
    z = torch.polar(torch.full_like(w, amp).expand(len(pos), -1).contiguous(), sign * pos.double()[:, None] * w)
    x = x.double()
    at = torch.arange(R, device=x.device)
    re, im = (at[:R // 2], at[R // 2:]) if c["layout"] == "half" else (at[0::2], at[1::2])
    t = torch.complex(x[..., re], x[..., im]) * z[:, None]
    y = x.clone()
    y[..., re], y[..., im] = t.real, t.imag
    return y


def _values(x, G, planes):
    """What the codes of rows x stand for."""
    T, H, D = x.shape
    w = x.reshape(T, H, -1, G)
    s = (w.abs().max(-1, keepdim=True).values / 7).to(torch.float16).double()
    t = torch.nan_to_num(w / s, nan=0.0)
    a = torch.clamp(torch.round(t), -8, 7)
    b = torch.clamp(torch.round(16 * (t - a)), -8, 7) if planes == 2 else 0
    return (s * (a + b / 16)).reshape(T, H, D)


def _cached(s, seq, n):
    """K, V [H][n][D] in 64 bits of one sequence's first n rows, read byte by byte at their addresses."""
    c = s["c"]
    H, D, P, G = c["H"], c["D"], c["page"], c["G"]
    dev = s["data"].device
    row = torch.arange(n, device=dev)
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
    if case["op"] == "pages":
        return None                     # whole numbers and bytes
    s = prepare(case, seed)
    c = s["c"]
    if c["op"] == "rope":
        return _turned(s["x"], s["pos"], c, -1.0 if c["inverse"] else 1.0)
    if c["op"] == "append":
        Hq, H = c["Hq"], c["H"]
        k, v = _turned(s["qkv"][:, Hq:Hq + H], s["pos"], c), s["qkv"][:, Hq + H:].double()
        if c["fmt"] == "nested":
            k, v = _values(k, c["G"], c["planes"]), _values(v, c["G"], c["planes"])
        return {"q": _turned(s["qkv"][:, :Hq], s["pos"], c), "k": k, "v": v}
    B, M, Hq, H, D = c["B"], c["M"], c["Hq"], c["H"], c["D"]
    out = torch.zeros(B, M, Hq, D, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_lens(c)):
        if n == 0:
            continue
        K, V = _cached(s, b, n)
        for m in range(M):
            at = n - M + m
            lo = max(0, at - c["window"] + 1) if c["window"] else 0
            if at < lo:
                continue
            q = s["q"][b, m].double().reshape(H, Hq // H, D)
            x = s["scale"] * torch.einsum("hgd,hnd->hgn", q, K[:, lo:at + 1])
            if c["cap"]:
                x = c["cap"] * torch.tanh(x / c["cap"])
            if s["slopes"] is not None:
                x = x + s["slopes"].double().reshape(H, -1, 1) * (torch.arange(lo, at + 1, device="cuda") - at)
            out[b, m] = torch.einsum("hgn,hnd->hgd", torch.softmax(x, -1), V[:, lo:at + 1]).reshape(Hq, D)
    return out
