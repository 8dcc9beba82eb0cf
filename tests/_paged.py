"""Plain models of the paged cache for its tests: records byte by byte,
page-table operations as Python loops, attention in 64 bits."""
from __future__ import annotations

import numpy as np


def record_bytes(D, page, bits, group):
    return page * (2 * D * bits // 8 + 8 * (D // group))


class Geometry:
    def __init__(self, KV, D, page, bits, group, layers=1):
        self.KV, self.D, self.page, self.bits, self.group, self.layers = KV, D, page, bits, group, layers
        self.rb, self.groups = D * bits // 8, D // group
        self.rec = record_bytes(D, page, bits, group)

    def spans(self, slot):
        """Byte ranges of one row in a record: K codes, V codes, K pairs, V pairs."""
        c, s = self.page * self.rb, self.page * self.groups * 4
        sb = 4 * self.groups
        return [(slot * self.rb, self.rb), (c + slot * self.rb, self.rb),
                (2 * c + slot * sb, sb), (2 * c + s + slot * sb, sb)]


def random_pool(rng, geo, n_pages):
    """uint8 [layers, n_pages, KV, rec]: any codes, pairs as a quantiser of rows of unit size leaves them."""
    pool = rng.integers(0, 256, size=(geo.layers, n_pages, geo.KV, geo.rec), dtype=np.uint8)
    at = 2 * geo.page * geo.rb
    shape = (geo.layers, n_pages, geo.KV, (geo.rec - at) // 4)
    s = (rng.random(shape) * 3.4 + 1.7) / 2 ** geo.bits
    b = -(2 ** (geo.bits - 1)) * s + 0.1 * rng.standard_normal(shape)
    pool[..., at:] = np.stack((s, b), -1).astype(np.float16).reshape(*shape[:-1], -1).view(np.uint8)
    return pool


def row_values(geo, record, which, slot):
    """(codes [D], values [D], biases [D]) of one row of one record, in 64 bits."""
    c0, n = geo.spans(slot)[which]
    p0, m = geo.spans(slot)[2 + which]
    bits = np.unpackbits(record[c0:c0 + n], bitorder="little").reshape(geo.D, geo.bits)
    codes = (bits.astype(np.int64) << np.arange(geo.bits)).sum(1)
    pair = record[p0:p0 + m].copy().view(np.float16).astype(np.float64).reshape(-1, 2)
    s, b = np.repeat(pair[:, 0], geo.group), np.repeat(pair[:, 1], geo.group)
    return codes, s * codes + b, b


def sequence_rows(geo, layer_pool, table_row, n, which):
    """[n][KV][D] values and biases of one sequence's first n tokens."""
    val = np.empty((n, geo.KV, geo.D))
    bias = np.empty((n, geo.KV, geo.D))
    at = 0
    while at < n:
        page = int(table_row[at // geo.page])
        m = min(geo.page, n - at)
        for kv in range(geo.KV):
            rec = layer_pool[page, kv]
            c = geo.page * geo.rb
            codes = rec[which * c:which * c + m * geo.rb].reshape(m, geo.rb)
            b = np.unpackbits(codes, axis=1, bitorder="little").reshape(m, geo.D, geo.bits)
            q = (b.astype(np.int64) << np.arange(geo.bits)).sum(-1)
            side = geo.page * geo.groups * 4
            p0 = 2 * c + which * side
            pair = rec[p0:p0 + m * geo.groups * 4].copy().view(np.float16).astype(np.float64)
            pair = pair.reshape(m, geo.groups, 2)
            s, o = np.repeat(pair[..., 0], geo.group, 1), np.repeat(pair[..., 1], geo.group, 1)
            val[at:at + m, kv], bias[at:at + m, kv] = s * q + o, o
        at += m
    return val, bias


def attention(geo, layer_pool, q, table, lens, scale):
    """q [B, L, H, D] float64 -> (o, sum_d |q k| (largest over keys), sum p |v|,
    largest |value bias|), each [B, L, H, ...]."""
    B, L, H, D = q.shape
    R = H // geo.KV
    o = np.zeros((B, L, H, D))
    vmag, bmax, smag = np.zeros((B, L, H, D)), np.zeros((B, L, H, D)), np.zeros((B, L, H, 1))
    for b in range(B):
        n = int(lens[b])
        if n <= 0:
            continue
        K, _ = sequence_rows(geo, layer_pool, table[b], n, 0)
        V, Vb = sequence_rows(geo, layer_pool, table[b], n, 1)
        for l in range(L):
            m = n - (L - 1 - l)
            if m <= 0:
                continue
            for h in range(H):
                kv = h // R
                s = scale * (K[:m, kv] @ q[b, l, h])
                p = np.exp(s - s.max())
                p /= p.sum()
                o[b, l, h] = p @ V[:m, kv]
                vmag[b, l, h] = p @ np.abs(V[:m, kv])
                bmax[b, l, h] = np.abs(Vb[:m, kv]).max(0)
                smag[b, l, h] = abs(scale) * (np.abs(K[:m, kv]) @ np.abs(q[b, l, h])).max()
    return o, smag, vmag, bmax


class Tables:
    """The page tables as lists, and the operations by their definitions."""

    def __init__(self, refs, table, lens, page):
        self.refs, self.lens, self.page = [int(x) for x in refs], [int(x) for x in lens], page
        self.table = [[int(x) for x in r] for r in table]
        self.width = len(self.table[0])

    def pages(self, n):
        return -(-n // self.page)

    def fork(self, parent, keep):
        bad, plan = 0, []
        for b, par in enumerate(parent):
            if par < 0:
                continue
            ok = par < len(self.lens) and par != b and self.lens[b] == 0 and parent[par] < 0
            if ok:
                n = self.lens[par] if keep[b] < 0 else keep[b]
                ok = n <= self.lens[par]
            if ok:
                plan.append((b, par, n))
            bad += not ok
        if bad:
            return [2, bad, 0, 0]
        total = 0
        for b, par, n in plan:
            for i in range(self.pages(n)):
                self.table[b][i] = self.table[par][i]
                self.refs[self.table[par][i]] += 1
                total += 1
            self.lens[b] = n
        return [0, 0, total, 0]

    def trim(self, keep):
        freed = 0
        for b, k in enumerate(keep):
            if k < 0 or k >= self.lens[b]:
                continue
            for i in range(self.pages(k), self.pages(self.lens[b])):
                p = self.table[b][i]
                self.table[b][i] = -1
                self.refs[p] -= 1
                freed += self.refs[p] == 0
            self.lens[b] = k
        return [0, 0, freed, 0]

    def grow(self, add):
        """Returns (status, copies): copies as (source, target, rows)."""
        bad = sum(a < 0 or self.pages(n + a) > self.width for n, a in zip(self.lens, add))
        if bad:
            return [2, bad, 0, 0], []
        growing = {}
        for b, a in enumerate(add):
            if a > 0 and self.lens[b] % self.page:
                growing.setdefault(self.table[b][self.lens[b] // self.page], []).append(b)
        copies = set()
        for p, rows in growing.items():
            if self.refs[p] > 1:
                copies |= set(rows if len(rows) < self.refs[p] else rows[:-1])
        need = [self.pages(n + a) - self.pages(n) + (b in copies)
                for b, (n, a) in enumerate(zip(self.lens, add))]
        free = [p for p, r in enumerate(self.refs) if r <= 0]
        if sum(need) > len(free):
            return [1, sum(need) - len(free), 0, 0], []
        at, done = 0, []
        for b in range(len(add)):
            mine = free[at:at + need[b]]
            at += need[b]
            for p in mine:
                self.refs[p] = 1
            if b in copies:
                old, new = self.table[b][self.lens[b] // self.page], mine.pop(0)
                self.table[b][self.lens[b] // self.page] = new
                self.refs[old] -= 1
                done.append((old, new, self.lens[b] % self.page))
            for i, p in enumerate(mine):
                self.table[b][self.pages(self.lens[b]) + i] = p
            self.lens[b] += add[b]
        return [0, 0, sum(need), len(done)], done

    def compact(self):
        """Returns (status, moves): moves as (source, target)."""
        n = sum(r > 0 for r in self.refs)
        holes = [p for p in range(n) if self.refs[p] <= 0]
        movers = [p for p in range(len(self.refs) - 1, n - 1, -1) if self.refs[p] > 0]
        to = dict(zip(movers, holes))
        for s, d in to.items():
            self.refs[d], self.refs[s] = self.refs[s], 0
        for b, row in enumerate(self.table):
            for i in range(self.pages(self.lens[b])):
                row[i] = to.get(row[i], row[i])
        return [0, 0, n, len(to)], list(to.items())
