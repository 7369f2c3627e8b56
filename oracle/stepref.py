"""Plain references, in 64 bits, of what surrounds attention in a decoding step: pages, rotary positions, adapters, the draw."""
from __future__ import annotations

import numpy as np


def pages_of(tokens, page_size):
    return -(-max(0, int(tokens)) // page_size)


class Pool:
    """Pages of sequences, moved one by one."""

    def __init__(self, n_pages, page_size, sequences, width):
        self.n_pages, self.page_size, self.width = n_pages, page_size, width
        self.table = np.full((sequences, width), -1, dtype=np.int32)
        self.lengths = np.zeros(sequences, dtype=np.int32)
        self.free = list(range(n_pages - 1, -1, -1))

    def extend(self, counts, rows):
        seqs, positions, offsets, served = [], [], [], len(counts)
        for s, c in enumerate(counts):
            c, n = max(0, int(c)), int(self.lengths[s])
            if n < 0:
                c = 0
            need = pages_of(n + c, self.page_size) - pages_of(n, self.page_size) if c else 0
            wide = c and n + c > min(self.width * self.page_size, 2 ** 31 - 1)
            if served == len(counts) and (wide or need > len(self.free) or len(seqs) + c > rows):
                served = s
            offsets.append(len(seqs))
            if s >= served:
                continue
            for j in range(need):
                self.table[s, pages_of(n, self.page_size) + j] = self.free.pop()
            seqs += [s] * c
            positions += range(n, n + c)
            if c:
                self.lengths[s] = n + c
        offsets.append(len(seqs))
        pad = rows - len(seqs)
        return (np.array(seqs + [-1] * pad, dtype=np.int32), np.array(positions + [0] * pad, dtype=np.int32),
                np.array(offsets, dtype=np.int32), served)

    def trim(self, keep):
        back = []
        for s, k in enumerate(keep):
            n = int(self.lengths[s])
            if 0 <= k < n:
                for j in range(pages_of(k, self.page_size), pages_of(n, self.page_size)):
                    back.append(int(self.table[s, j]))
                    self.table[s, j] = -1
                self.lengths[s] = k
        self.free = (self.free + back[::-1])[:self.n_pages]   # no place for more: only of pages that it never gave out


def rotate(x, positions, rates, factor, rotary_dim, interleaved):
    """x [rows][heads][dim] turned, in 64 bits; rows with a negative position as they are."""
    x = np.asarray(x, dtype=np.float64)
    out = x.copy()
    half = rotary_dim // 2
    for r, p in enumerate(positions):
        if p < 0:
            continue
        for i in range(half):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            t = float(p) * float(rates[i])
            c, s = np.cos(t) * factor, np.sin(t) * factor
            with np.errstate(invalid="ignore"):   # infinities among the channels
                out[r, :, a] = x[r, :, a] * c - x[r, :, b] * s
                out[r, :, b] = x[r, :, a] * s + x[r, :, b] * c
    return out


def lora(x, ids, y, a, b, scales=None, ranks=None):
    """(out, S): out in 64 bits, and the sums of magnitudes S that its accuracy is stated by."""
    out = np.asarray(y, dtype=np.float64).copy()
    size = np.zeros_like(out)
    for r, i in enumerate(ids):
        if i < 0:
            continue
        if i >= len(a):
            out[r] = np.nan
            continue
        k = a.shape[1] if ranks is None else int(ranks[i])
        s = 1.0 if scales is None else float(scales[i])
        ai, bi, xr = a[i, :k].astype(np.float64), b[i, :, :k].astype(np.float64), np.asarray(x[r], dtype=np.float64)
        out[r] += s * (bi @ (ai @ xr))
        size[r] = abs(s) * (np.abs(bi) @ (np.abs(ai) @ np.abs(xr)))
    return out, size


def sample_row(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, logprob, the smallest distance of u times the sum to a border between two tokens, relative to the sum)."""
    l = np.asarray(logits, dtype=np.float64)
    if any(np.isnan(v) for v in (u, temperature, top_p, min_p)) or temperature < 0:
        return -1, np.nan, 1.0
    order = np.lexsort((np.arange(l.size), -np.where(np.isnan(l), -np.inf, l)))
    order = order[~np.isnan(l[order]) & (l[order] != -np.inf)]
    if not order.size:
        return -1, np.nan, 1.0
    if temperature == 0:
        return int(order[0]), 0.0, 1.0
    top = l[order[0]]
    with np.errstate(over="ignore", invalid="ignore"):
        z = np.where(l[order] == top, 0.0, (l[order] - top) / np.float64(temperature))
    w = np.where(np.isnan(z), 0.0, np.exp(z))
    if top_k > 0:
        order, w = order[:top_k], w[:top_k]
    if top_p < 1:
        sums = np.cumsum(w)
        order, w = (x[:max(1, 1 + int(np.searchsorted(sums, top_p * w.sum(), side="left")))] for x in (order, w))
    left = w >= min_p
    left[0] = True
    order, w = order[left], w[left]
    by = np.argsort(order)
    order, w = order[by], w[by]
    sums = np.cumsum(w)
    target = min(max(float(u), 0.0), np.nextafter(1.0, 0.0)) * w.sum()
    at = min(int(np.searchsorted(sums, target, side="right")), len(w) - 1)
    return int(order[at]), float(np.log(w[at] / w.sum())), float(np.min(np.abs(sums - target)) / w.sum())
