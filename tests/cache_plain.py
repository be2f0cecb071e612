"""Plain 64-bit implementations of the cache-side operators, on CPU tensors, for the tests.

They loop over requests, rows and pages as the definitions read; nothing is shared with the
library.
"""
import math

import torch


def spans(num_drafts, row_offsets, lens, k_max):
    """(b, first row, rows, length) of each request with new tokens."""
    for b, k in enumerate(num_drafts.tolist()):
        row = int(row_offsets[b]) if row_offsets is not None else b * (k_max + 1)
        if k >= 0:
            yield b, row, k + 1, int(lens[b])


def turn(x, pos, inv_freq, interleaved, rope_scale):
    """x [heads, D] (float64) turned to position pos; also the sum of magnitudes of each pair."""
    half = inv_freq.numel()
    y, size = x.clone(), x.abs()
    for j in range(half):
        a, z = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        angle = pos * float(inv_freq[j])
        c, s = rope_scale * math.cos(angle), rope_scale * math.sin(angle)
        y[:, a], y[:, z] = x[:, a] * c - x[:, z] * s, x[:, a] * s + x[:, z] * c
        size[:, a] = size[:, z] = abs(rope_scale) * (x[:, a].abs() + x[:, z].abs())
    return y, size


def append(q, k, v, q_weight, k_weight, eps, inv_freq, k_cache, v_cache, table, lens, num_drafts, row_offsets, k_max,
           interleaved=False, rope_scale=1.0):
    """(q, k cache, v cache) in float64 and the magnitudes that their rounding errors scale with."""
    D, P = q.shape[-1], k_cache.shape[1]
    out, kc, vc = torch.zeros(q.shape, dtype=torch.float64), k_cache.double(), v_cache.double()
    out_size, kc_size = torch.zeros_like(out), torch.zeros_like(kc)
    freq = inv_freq if inv_freq is not None else torch.zeros(0)

    def head(x, w, pos):
        x = x.double()
        if w is not None:
            x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.double()
        return turn(x, pos, freq, interleaved, rope_scale)

    for b, row, n, L in spans(num_drafts, row_offsets, lens, k_max):
        for i in range(n):
            pos = L - n + i
            page, slot = int(table[b, pos // P]), pos % P
            out[row + i], out_size[row + i] = head(q[row + i], q_weight, pos)
            kc[page, slot], kc_size[page, slot] = head(k[row + i], k_weight, pos)
            vc[page, slot] = v[row + i].double()
    return out, kc, vc, out_size, kc_size


def visible(pos, window, sinks):
    """The keys that the row at position pos sees, ascending."""
    first = max(0, pos - window + 1) if window else 0
    return list(range(min(sinks if window else 0, first))) + list(range(first, pos + 1))


def attention(q, k_cache, v_cache, table, lens, num_drafts, row_offsets, k_max, scale, window, sinks):
    """(out, lse) in float64, sum_j p_j |v_j| per output, and the largest scale * sum |q k| per row."""
    R, Hq, D = q.shape
    P, Hk = k_cache.shape[1], k_cache.shape[2]
    out = torch.zeros(R, Hq, D, dtype=torch.float64)
    lse, size, score = torch.zeros(R, Hq, dtype=torch.float64), torch.zeros_like(out), torch.zeros(R, Hq)
    for b, row, n, L in spans(num_drafts, row_offsets, lens, k_max):
        for i in range(n):
            j = torch.tensor(visible(L - n + i, window, sinks))
            page, slot = table[b][j // P].long(), j % P
            k, v = k_cache[page, slot].double(), v_cache[page, slot].double()
            x = q[row + i].double().view(Hk, Hq // Hk, D)
            z = scale * torch.einsum("hgd,jhd->hgj", x, k)
            lse[row + i] = torch.logsumexp(z, -1).flatten()
            p = torch.softmax(z, -1)
            out[row + i] = torch.einsum("hgj,jhd->hgd", p, v).reshape(Hq, D)
            size[row + i] = torch.einsum("hgj,jhd->hgd", p, v.abs()).reshape(Hq, D)
            score[row + i] = (abs(scale) * torch.einsum("hgd,jhd->hgj", x.abs(), k.abs())).amax(-1).flatten()
    return out, lse, size, score


class Pages:
    """The page bookkeeping as a server would write it, one request and one page at a time."""

    def __init__(self, lens, table, ref, page_size):
        self.len, self.table, self.ref, self.P = lens.tolist(), table.tolist(), ref.tolist(), page_size
        self.errors = []

    def free(self):
        return [p for p, c in enumerate(self.ref) if c == 0]

    def reserve(self, num_drafts):
        free, asked = self.free(), 0
        for b, k in enumerate(num_drafts.tolist()):
            L = self.len[b]
            if k == -1:
                continue
            if k < -1 or L < 0 or L + k + 1 > len(self.table[b]) * self.P:
                self.fail(1, b)
                continue
            have, need = -(-L // self.P), -(-(L + k + 1) // self.P)
            if L % self.P:
                p = self.table[b][have - 1]
                if not 0 <= p < len(self.ref) or self.ref[p] < 1:
                    self.fail(9, b)
                    continue
                if self.ref[p] > 1:
                    self.fail(11, b)
                    continue
            first, asked = asked, asked + need - have
            if need > have and asked > len(free):
                self.fail(10, b)
                continue
            for x in range(have, need):
                p = free[first + x - have]
                self.table[b][x] = p
                self.ref[p] = 1
            self.len[b] = L + k + 1

    def fail(self, code, b):
        self.errors.append((code, b))
        if self.len[b] >= 0:
            self.len[b] = -1 - self.len[b]

    def fork(self, parents, children, fork_len):
        pairs, free, taken = [], self.free(), set()
        lens, table = list(self.len), [list(r) for r in self.table]
        asked = 0
        for f, (p, c) in enumerate(zip(parents.tolist(), children.tolist())):
            B = len(lens)
            pair, code, n = (-1, -1), 0, 0
            empty = 0 <= c < B and lens[c] == 0
            if not 0 <= p < B or not empty:
                code = 1
            else:
                n = int(fork_len[f]) if fork_len is not None else lens[p]
                if n < 1 or n > lens[p]:
                    code = 1
                elif n % self.P:
                    t = table[p][n // self.P]
                    if not 0 <= t < len(self.ref) or self.ref[t] < 1:
                        code = 9
            mine = empty and c not in taken
            if empty:
                taken.add(c)
            if not mine and not code:
                code = 1
            if not code and n % self.P:
                if asked >= len(free):
                    code = 10
                else:
                    pair = (table[p][n // self.P], free[asked])
                asked += 1
            if code:
                self.errors.append((code, f))
            else:
                row = table[p][:n // self.P] + ([pair[1]] if n % self.P else [])
                for t in table[p][:n // self.P]:
                    if t >= 0:
                        self.ref[t] += 1
                if pair[1] >= 0:
                    self.ref[pair[1]] = 1
                self.table[c] = row + [-1] * (len(table[c]) - len(row))
            if mine:
                self.len[c] = -1 if code else n
            pairs.append(pair)
        return pairs

    def release(self, window=0, sinks=0):
        for b, L in enumerate(self.len):
            if L < 0:
                continue
            for x, p in enumerate(self.table[b]):
                past = x * self.P >= L
                gone = window and x * self.P >= sinks and (x + 1) * self.P - 1 <= L - window
                if p >= 0 and (past or gone):
                    self.ref[p] -= 1
                    self.table[b][x] = -1

    def compact(self, capacity):
        used = [p for p, c in enumerate(self.ref) if c > 0]
        U = len(used)
        src = [p for p in used if p >= U]
        dst = [p for p in range(U) if self.ref[p] == 0]
        moves = list(zip(src, dst))[:capacity]
        for a, d in moves:
            self.ref[d], self.ref[a] = self.ref[a], 0
        to = dict(moves)
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        return moves + [(-1, -1)] * (capacity - len(moves))
