"""Plain models of the paged KV cache for its tests: the page format read byte
by byte, attention in 64 bits, and the bookkeeping of pages as a sequential
program over Python lists."""
import math

import numpy as np
import torch


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.float32)).bfloat16()


class HostPool:
    """The rows of a pool's bytes (uint8 [layers][pages][heads][record])."""

    def __init__(self, pool):
        self.D, self.G, self.P, self.H = pool.head_dim, pool.group, pool.page_size, pool.heads_kv
        self.bf, self.N = pool.fmt == 1, pool.n_pages
        nb = self.P // 16
        self.bb = 64 * self.D if self.bf else 16 * self.D + 64 * (self.D // self.G)
        self.rec = nb * self.bb + (0 if self.bf else nb * 16 * self.D)
        self.a = pool.data.cpu().numpy().reshape(pool.layers, self.N, self.H, self.rec)

    def _nib(self, plane, r):
        """Unsigned nibbles of row r of 16 rows of D / 2 bytes."""
        rb = self.D // 2
        out = np.empty(self.D, np.int64)
        for o in range(rb):
            q = r * (rb // 16) + o // 16
            line = q // 8
            b = int(plane[line * 128 + ((q % 8) ^ (2 * (line % 4))) * 16 + o % 16])
            out[2 * o], out[2 * o + 1] = b & 15, b >> 4
        return out

    def codes(self, layer, page, h, row, which):
        """(q4, r, scale bits) of a NESTED44 row; which 0 = K, 1 = V."""
        rb, ng = self.D // 2, self.D // self.G
        rec, blk, r = self.a[layer, page, h], row // 16, row % 16
        base = rec[blk * self.bb:(blk + 1) * self.bb]
        more = rec[(self.P // 16) * self.bb + blk * 16 * self.D:]
        q = self._nib(base[which * 16 * rb:], r) - 8
        s = self._nib(more[which * 16 * rb:], r) - 8
        at = 32 * rb + which * 32 * ng + r * ng * 2
        return q, s, base[at:at + 2 * ng].copy().view(np.uint16)

    def row(self, layer, page, h, row, which, planes):
        """A row's values in 64 bits."""
        if self.bf:
            blk, r, D = row // 16, row % 16, self.D
            x = self.a[layer, page, h, blk * self.bb + which * 32 * D:][:32 * D].copy().view(np.uint16)
            at = [r * D + ((i // 8) ^ (r % 8)) * 8 + i % 8 for i in range(D)]
            return (x[at].astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        q, r, sc = self.codes(layer, page, h, row, which)
        s = np.repeat(sc.view(np.float16).astype(np.float64), self.G)
        return s * (q + (r / 16.0 if planes == 2 else 0))


def rows_of(hp, layer, table_row, n, planes):
    """K, V float64 [H][n][D] of one sequence, by whole-array indexing of the same addresses."""
    D, P, H = hp.D, hp.P, hp.H
    t = np.arange(n)
    rec = hp.a[layer][np.asarray(table_row)[t // P]]                 # [n][H][record]
    blk, r = (t % P) // 16, t % 16
    d = np.arange(D)
    got = []
    for which in range(2):
        if hp.bf:
            at = blk[:, None] * hp.bb + which * 32 * D + 2 * (r[:, None] * D + ((d // 8)[None] ^ (r % 8)[:, None]) * 8 + d % 8)
            lo = np.take_along_axis(rec, np.broadcast_to(at[:, None], (n, H, D)), 2).astype(np.uint32)
            hi = np.take_along_axis(rec, np.broadcast_to(at[:, None] + 1, (n, H, D)), 2).astype(np.uint32)
            x = ((lo << 16) | (hi << 24)).view(np.float32).astype(np.float64)
        else:
            rb, ng = D // 2, D // hp.G
            q = r[:, None] * (rb // 16) + (d // 32)[None]
            off = (q // 8) * 128 + ((q % 8) ^ (2 * (q // 8 % 4))) * 16 + (d // 2 % 16)
            nib = lambda at: np.where(d % 2 == 0, *(lambda b: (b & 15, b >> 4))(   # noqa: E731
                np.take_along_axis(rec, np.broadcast_to(at[:, None], (n, H, D)), 2).astype(np.int64))) - 8
            x = nib(blk[:, None] * hp.bb + which * 16 * rb + off).astype(np.float64)
            if planes == 2:
                x = x + nib((P // 16) * hp.bb + blk[:, None] * 16 * D + which * 16 * rb + off) / 16.0
            sat = blk[:, None] * hp.bb + 32 * rb + which * 32 * ng + 2 * (r[:, None] * ng + (d // hp.G)[None])
            sl = np.take_along_axis(rec, np.broadcast_to(sat[:, None], (n, H, D)), 2).astype(np.uint16)
            sh = np.take_along_axis(rec, np.broadcast_to(sat[:, None] + 1, (n, H, D)), 2).astype(np.uint16)
            x = x * (sl | (sh << 8)).astype(np.uint16).view(np.float16).astype(np.float64)
        got.append(x.transpose(1, 0, 2))
    return got


def attention64(hp, layer, table, q, lens, planes, scale, softcap=0.0, window=0, slopes=None):
    """(out, tol): attention in 64 bits and how far the kernel's bf16 output may be.

    The output is rounded to bf16 (2^-8).  Probabilities are rounded to fp16
    (2^-11; bf16 2^-8 for the bf16 format) in numerator and denominator; those
    below fp16's normal range by 2^-25 of the largest.  A score that is off by
    e moves its probability by e: fp32 products and sums (2^-17 of the sum of
    absolute products, 128 terms), the cap (2^-21 of it), the bias (2^-22)."""
    B, M, Hq, D = q.shape
    g = Hq // hp.H
    out, tol = np.zeros((B, M, Hq, D)), np.zeros((B, M, Hq, D))
    c = 2.0 ** -8 if hp.bf else 2.0 ** -11
    for b in range(B):
        n = int(lens[b])
        if n == 0:
            continue
        K, V = rows_of(hp, layer, table[b], n, planes)
        for m in range(M):
            at = n - M + m
            lo = max(0, at - window + 1) if window else 0
            if at < lo:
                continue
            for h in range(Hq):
                k, v = K[h // g, lo:at + 1], V[h // g, lo:at + 1]
                x = q[b, m, h].astype(np.float64)
                s = scale * (k @ x)
                e = 2.0 ** -17 * scale * (np.abs(k) @ np.abs(x)).max()
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                    e += 2.0 ** -21 * softcap
                if slopes is not None:
                    bias = float(slopes[h]) * (at - np.arange(lo, at + 1))
                    s = s - bias
                    e += 2.0 ** -22 * np.abs(bias).max()
                p = np.exp(s - s.max())
                l = p.sum()
                out[b, m, h] = p @ v / l
                near = p @ np.abs(v) / l
                tol[b, m, h] = (2.0 ** -8 * np.abs(out[b, m, h]) + (2 * c + 2 * e) * near
                                + len(p) * 2.0 ** -24 * np.abs(v).max() / l)
    return out, tol


class HostMap:
    """The page bookkeeping, one sequence after another."""

    def __init__(self, S, W, N, P):
        self.W, self.N, self.P = W, N, P
        self.pages = [[] for _ in range(S)]
        self.ref = [0] * N

    def table(self):
        return np.array([p + [-1] * (self.W - len(p)) for p in self.pages], np.int32)

    def held(self):
        return np.array([len(p) for p in self.pages], np.int32)

    def _need(self, rows):
        return max(0, -(-rows // self.P))

    def truncate(self, seqs, rows):
        for s, r in zip(seqs, rows):
            for p in self.pages[s][self._need(r):]:
                self.ref[p] -= 1
            self.pages[s] = self.pages[s][:self._need(r)]

    def fork(self, src, dst, rows):
        new = [self.pages[a][:self._need(r)] for a, r in zip(src, rows)]
        for b, pg in zip(dst, new):
            for p in pg:
                self.ref[p] += 1
            for p in self.pages[b]:
                self.ref[p] -= 1
        for b, pg in zip(dst, new):
            self.pages[b] = list(pg)

    def reserve(self, seqs, first, last):
        """(granted, [(from, to)] of the pages whose other rows are copied)."""
        start = list(self.ref)
        free = [p for p in range(self.N) if start[p] == 0]
        touch = {}
        for i, (s, f, l) in enumerate(zip(seqs, first, last)):
            if l > f and l <= self.W * self.P:
                for j in range(f // self.P, min(len(self.pages[s]), self._need(l))):
                    touch.setdefault(self.pages[s][j], []).append(i)
        granted, copies, open_ = [], [], True
        for i, (s, f, l) in enumerate(zip(seqs, first, last)):
            if l > self.W * self.P:
                granted.append(0)
                continue
            pg, need = list(self.pages[s]), self._need(l) if l > f else 0
            cow = [j for j in range(f // self.P, min(len(pg), need))
                   if start[pg[j]] > 1 and not (len(touch[pg[j]]) == start[pg[j]] and touch[pg[j]][-1] == i)]
            want = len(cow) + max(0, need - len(pg))
            open_ = open_ and want <= len(free)
            granted.append(int(open_))
            if not open_:
                continue
            for j in cow:
                p = free.pop(0)
                self.ref[pg[j]] -= 1
                self.ref[p] += 1
                if j * self.P < f or (j + 1) * self.P > l:
                    copies.append((pg[j], p))
                pg[j] = p
            while len(pg) < need:
                p = free.pop(0)
                self.ref[p] += 1
                pg.append(p)
            self.pages[s] = pg
        return granted, copies

    def compact(self):
        used = sum(r > 0 for r in self.ref)
        high = [p for p in range(used, self.N) if self.ref[p] > 0]
        hole = [p for p in range(used) if self.ref[p] == 0]
        to = dict(zip(high, hole))
        for a, b in to.items():
            self.ref[b], self.ref[a] = self.ref[a], 0
        self.pages = [[to.get(p, p) for p in pg] for pg in self.pages]
        return used, list(to.items())


def turned64(x, pos, rot, theta, layout, scaling, factor, old, inverse):
    """Rotation of x [T][H][D] in 64 bits, and the factor on it."""
    x = np.asarray(x, np.float64)
    y = x.copy()
    amp = 0.1 * math.log(factor) + 1 if scaling == "parts" else 1.0
    for i in range(rot // 2):
        base = theta * factor ** (rot / (rot - 2)) if scaling == "ntk" else theta
        w = base ** (-2 * i / rot)
        if scaling == "linear":
            w /= factor
        if scaling == "parts":
            keep = min(1.0, max(0.0, (old * w / (2 * math.pi) - 1) / 31))
            w = w * keep + w / factor * (1 - keep)
        a = np.asarray(pos, np.float64)[:, None] * w * (-1 if inverse else 1)
        u, v = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
        y[..., u] = amp * (x[..., u] * np.cos(a) - x[..., v] * np.sin(a))
        y[..., v] = amp * (x[..., u] * np.sin(a) + x[..., v] * np.cos(a))
    return y, amp
