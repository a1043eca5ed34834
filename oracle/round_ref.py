"""Oracle of the operators of a verify round, on the CPU in 64 bits.

Plain definitions, row by row and token by token; tensors are torch CPU
tensors. Shares no code with the library.
"""

from __future__ import annotations

import math

import torch


def rope_frequencies(rot, base, scaling="none", factor=1.0, original_len=0):
    """(angle per position of each pair, factor on cosine and sine)."""
    half = rot // 2
    if scaling == "ntk" and rot > 2:
        base = base * factor ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(half)]
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling == "yarn":
        def pair(turns):
            return rot * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(base))
        lo, hi = max(math.floor(pair(32)), 0), min(math.ceil(pair(1)), rot - 1)
        out = []
        for i, x in enumerate(f):
            w = min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
            out.append(x * (1 - w) + x / factor * w)
        return out, 0.1 * math.log(factor) + 1.0 if factor > 1 else 1.0
    if scaling == "smooth":
        out = []
        for x in f:
            turns = original_len * x / (2 * math.pi)
            w = min(max((turns - 1) / 3, 0.0), 1.0)
            out.append(x * w + x / factor * (1 - w))
        return out, 1.0
    return f, 1.0


def rope_ref(x, pos, freqs, mscale, rot, interleaved):
    """x [heads, dim] (any type) turned for position pos, in 64 bits."""
    y = x.double().clone()
    for i, f in enumerate(freqs):
        c, s = mscale * math.cos(pos * f), mscale * math.sin(pos * f)
        e, o = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        a, b = x[:, e].double(), x[:, o].double()
        y[:, e], y[:, o] = a * c - b * s, a * s + b * c
    return y


def sequence_rows(row_start, kv_len):
    """(sequence, row, position) of every row."""
    for b in range(len(kv_len)):
        n = row_start[b + 1] - row_start[b]
        for i in range(n):
            yield b, row_start[b] + i, kv_len[b] - n + i


def visible(pos, kv_len, window, sinks):
    t = torch.arange(max(kv_len, 0))
    see = t <= pos
    if window > 0:
        see &= (t > pos - window) | (t < sinks)
    return see


def attn_ref(q, k, v, row_start, kv_len, table, scale, window=0, sinks=0):
    """q [rows, heads, dim], k and v [pages, page size, kv heads, dim]: outputs in 64 bits, the
    weighted mean of |v| of each output value, and the largest sum of |q k| * scale of a row."""
    pages, ps, hk, dim = k.shape
    g = q.shape[1] // hk
    out = torch.zeros(q.shape, dtype=torch.float64)
    mean = torch.zeros(q.shape, dtype=torch.float64)
    size = torch.zeros(q.shape[:2] + (1,), dtype=torch.float64)
    for b, r, pos in sequence_rows(row_start, kv_len):
        ids = [table[b][t // ps] if t // ps < len(table[b]) else -1 for t in range(kv_len[b])]
        paged = torch.tensor([0 <= p < pages for p in ids], dtype=torch.bool)
        see = visible(pos, kv_len[b], window, sinks) & paged
        at = see.nonzero()[:, 0]
        if not at.numel():
            continue
        page = torch.tensor(ids)[at]
        for e in range(q.shape[1]):
            kk, vv = k[page, at % ps, e // g].double(), v[page, at % ps, e // g].double()
            x = kk @ q[r, e].double() * scale
            p = torch.softmax(x, 0)
            out[r, e] = p @ vv
            mean[r, e] = p @ vv.abs()
            size[r, e] = (kk.abs() @ q[r, e].double().abs()).max() * scale
    return out, mean, size


class Book:
    """Pages of table rows, one operation after the other (lists of ints)."""

    def __init__(self, ref, table, held, length, page_size):
        self.ref, self.table, self.held, self.length = ref, table, held, length
        self.ps, self.width = page_size, len(table[0])

    def pages_for(self, tokens):
        return max(-(-tokens // self.ps), 0)

    def trim(self, keep, rows=None):
        for i, n in enumerate(keep):
            r = i if rows is None else rows[i]
            if not 0 <= r < len(self.table):
                continue
            n = max(n, 0)
            while self.held[r] > self.pages_for(n):
                self.held[r] -= 1
                p = self.table[r][self.held[r]]
                if 0 <= p < len(self.ref):
                    self.ref[p] -= 1
                self.table[r][self.held[r]] = -1
            self.length[r] = min(self.length[r], n)

    def reserve(self, goal):
        free = [p for p, n in enumerate(self.ref) if n == 0]
        ok, short = [], False
        for r, n in enumerate(goal):
            want = self.pages_for(n)
            if want > self.width:
                ok.append(0)
                continue
            last = self.length[r] // self.ps
            if n > self.length[r] and last < self.held[r]:
                p = self.table[r][last]
                if 0 <= p < len(self.ref) and self.ref[p] > 1:
                    ok.append(0)
                    continue
            need = max(want - self.held[r], 0)
            if need and (short or need > len(free)):
                short = True
                ok.append(0)
                continue
            for _ in range(need):
                p = free.pop(0)
                self.ref[p] = 1
                self.table[r][self.held[r]] = p
                self.held[r] += 1
            ok.append(1)
        return ok

    def fork(self, parent, child):
        """ok, and the pages to copy as (from, to)."""
        free = [p for p, n in enumerate(self.ref) if n == 0]
        ok, copies = [], []
        empty = [h <= 0 for h in self.held]
        rows = range(len(self.table))
        for i, (p, c) in enumerate(zip(parent, child)):
            if p not in rows or c not in rows or c in child[:i] or c in parent or not empty[c]:
                ok.append(0)
                continue
            full, rest = divmod(self.length[p], self.ps)
            full = min(full, self.held[p])
            part = rest != 0 and self.held[p] > full
            if part and (not 0 <= self.table[p][full] < len(self.ref) or not free):
                ok.append(0)
                continue
            for j in range(full):
                self.table[c][j] = self.table[p][j]
                if 0 <= self.table[p][j] < len(self.ref):
                    self.ref[self.table[p][j]] += 1
            if part:
                new = free.pop(0)
                self.ref[new] = 1
                self.table[c][full] = new
                copies.append((self.table[p][full], new))
            self.held[c] = full + part
            self.length[c] = self.length[p] if part else full * self.ps
            ok.append(1)
        return ok, copies


def logits_ref(logits, T, draft=None, counts=None, seen=None, repetition=None, frequency=None,
               presence=None, biases=None, allowed=None):
    """Edited logits in 64 bits and the sum of the sizes of the steps' results (each step of the
    library rounds once). seen [B, N] and allowed [B*T, N] are truth values, biases a list of
    (token, value) for each sequence."""
    rows, N = logits.shape
    out, size = logits.double().clone(), torch.zeros(rows, N, dtype=torch.float64)
    for r in range(rows):
        b, i = divmod(r, T)
        x = out[r]
        if repetition is not None or frequency is not None or presence is not None:
            n = counts[b].double().clone() if counts is not None else torch.zeros(N).double()
            if draft is not None:
                for t in draft[b][:i].tolist():
                    if 0 <= t < N:
                        n[t] += 1
            used = n > 0
            told = used | seen[b] if seen is not None else used
            if repetition is not None:
                rep = repetition[b].double()
                x = torch.where(told, torch.where(x > 0, x / rep, x * rep), x)
                size[r] += x.abs()
            if frequency is not None:
                step = frequency[b].double() * n
                x = x - step
                size[r] += step.abs() + x.abs()
            if presence is not None:
                x = torch.where(used, x - presence[b].double(), x)
                size[r] += x.abs()
        if biases is not None:
            for t, value in dict((t, value) for t, value in biases[b] if 0 <= t < N).items():
                x[t] += value
            size[r] += x.abs()
        if allowed is not None:
            x = torch.where(allowed[r], x, -math.inf)
        out[r] = x
    return out, size
