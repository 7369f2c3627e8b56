"""Plain reference of the paged key-value cache and of attention over it, in numpy and 64 bits.

Written from the layout and the quantizer in include/exq.h, one element's bit address at a time; shares no code with the
library.  Test infrastructure only.
"""
from __future__ import annotations

import numpy as np

GROUP, TILE = 32, 16


class Geometry:
    def __init__(self, page_size, kv_heads, head_dim, k_bits, v_bits):
        self.page_size, self.kv_heads, self.head_dim = page_size, kv_heads, head_dim
        self.bits = (k_bits, v_bits)
        G = head_dim // GROUP
        self.codes = [TILE * head_dim * b // 8 for b in self.bits]
        self.scales = [TILE * G * 2 if b < 16 else 0 for b in self.bits]
        self.tile_bytes = sum(self.codes) + sum(self.scales)
        self.page_bytes = kv_heads * (page_size // TILE) * self.tile_bytes

    def tile_base(self, page, head, token):
        """First byte of the tile that holds `token` (of the page)."""
        return page * self.page_bytes + (head * (self.page_size // TILE) + token // TILE) * self.tile_bytes

    def code_bit(self, part, token, d):
        """Bit of the tile where the code of channel d of `token` (of the tile) starts; part 0: keys, 1: values."""
        b, G = self.bits[part], self.head_dim // GROUP
        g, r = d // GROUP, d % GROUP
        gpc = 16 // b
        j = g // gpc
        n = np.minimum(gpc, G - j * gpc)
        if part == 0:
            lane, e = 16 * (r // 8) + token, r % 8
            inner = 4 * (e // 2) + 16 * (e % 2) if b == 4 else b * e
        else:
            lane, h, t = 16 * (token // 4) + r % 16, r // 16, token % 4
            inner = 16 * (t % 2) + 8 * (t // 2) + 4 * h if b == 4 else b * (4 * h + t)
        start = 0 if part == 0 else self.codes[0] + self.scales[0]
        return 8 * (start + 1024 * j + lane * n * b + (g - j * gpc) * b) + inner

    def scale_byte(self, part, token, g):
        G = self.head_dim // GROUP
        if part == 0:
            return self.codes[0] + 2 * (token * G + g)
        return self.codes[0] + self.scales[0] + self.codes[1] + 8 * G * (token // 4) + 8 * g + 2 * (token % 4)


def quantize(x, bits):
    """fp16 [..., dim] -> (codes int64 [..., dim], scales fp16 [..., dim / 32]); 16 bits: the bit patterns and None."""
    x = np.asarray(x, dtype=np.float16)
    if bits == 16:
        return x.view(np.uint16).astype(np.int64), None
    top = np.float32((1 << (bits - 1)) - 1)
    f = x.astype(np.float32).reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(all="ignore"):
        s = (np.abs(f).max(-1) / top).astype(np.float16)
        s = np.minimum(s, np.float16(9352 if bits == 4 else 515.5))   # top * s stays finite
        s = np.where(np.isfinite(f).all(-1), s, np.float16(np.nan))
        c = np.clip(np.rint(f / s.astype(np.float32)[..., None]), -top, top)
    c = np.where(s[..., None] > 0, c, 0).astype(np.int64) + (1 << (bits - 1))
    return c.reshape(x.shape), s


def dequantize(codes, scales, bits):
    """The fp16 values that codes and scales stand for."""
    if bits == 16:
        return codes.astype(np.uint16).view(np.float16)
    c = codes.reshape(*scales.shape, GROUP) - (1 << (bits - 1))
    with np.errstate(all="ignore"):
        return (c * scales.astype(np.float64)[..., None]).astype(np.float16).reshape(codes.shape)


def held(x, bits):
    """What x reads back as."""
    return dequantize(*quantize(x, bits), bits)


def resolve(geo, n_pages, table, seqs, positions):
    """(page, token of the page) of each row, or None: -1 for padding, -2 for a place outside."""
    out = []
    for s, p in zip(seqs, positions):
        if s < 0:
            out.append(-1)
        elif s >= table.shape[0] or p < 0 or p // geo.page_size >= table.shape[1]:
            out.append(-2)
        else:
            page = int(table[s, p // geo.page_size])
            out.append((page, int(p % geo.page_size)) if 0 <= page < n_pages else -2)
    return out


def append(geo, pages, k, v, table, seqs, positions):
    """Writes rows into `pages` (uint8, flat), in place."""
    n_pages = pages.size // geo.page_bytes
    d = np.arange(geo.head_dim)
    g = np.arange(geo.head_dim // GROUP)
    for r, place in enumerate(resolve(geo, n_pages, table, seqs, positions)):
        if not isinstance(place, tuple):
            continue
        page, token = place
        for h in range(geo.kv_heads):
            base = geo.tile_base(page, h, token)
            for part, x in enumerate((k, v)):
                b = geo.bits[part]
                codes, scales = quantize(x[r, h], b)
                bit = geo.code_bit(part, token % TILE, d)
                at = base + bit // 8
                if b == 4:
                    for sh, keep in ((0, 0xF0), (4, 0x0F)):   # a byte's two elements one after the other
                        i = bit % 8 == sh
                        pages[at[i]] = (pages[at[i]] & keep) | (codes[i] << sh)
                elif b == 8:
                    pages[at] = codes
                else:
                    pages[at], pages[at + 1] = codes & 255, codes >> 8
                if scales is not None:
                    sb = base + geo.scale_byte(part, token % TILE, g)
                    w = scales.view(np.uint16)
                    pages[sb], pages[sb + 1] = w & 255, w >> 8


def read_token(geo, pages, page, token, head):
    """(k, v) fp16 [dim] of one token and head."""
    base = geo.tile_base(page, head, token)
    d = np.arange(geo.head_dim)
    g = np.arange(geo.head_dim // GROUP)
    out = []
    for part in (0, 1):
        b = geo.bits[part]
        bit = geo.code_bit(part, token % TILE, d)
        at = base + bit // 8
        if b == 16:
            out.append((pages[at].astype(np.int64) | (pages[at + 1].astype(np.int64) << 8)).astype(np.uint16).view(np.float16))
            continue
        codes = (pages[at].astype(np.int64) >> (bit % 8)) & ((1 << b) - 1)
        sb = base + geo.scale_byte(part, token % TILE, g)
        s = (pages[sb].astype(np.uint16) | (pages[sb + 1].astype(np.uint16) << 8)).astype(np.uint16).view(np.float16)
        out.append(dequantize(codes, s, b))
    return out


def attend(q, k, v, scale):
    """One row: q fp16 [q_heads][dim], k and v fp16 [tokens][kv_heads][dim] (the tokens attended to) ->
    (out [q_heads][dim], lse [q_heads], bound of out, bound of lse), all float64.

    The bounds are those of include/exq.h: A is the largest magnitude sum of a score, P the weighted average of |v|."""
    heads, dim = q.shape
    per = heads // k.shape[1]
    qf, kf, vf = (x.astype(np.float64) for x in (q, k, v))
    out, lse = np.zeros((heads, dim)), np.full(heads, -np.inf)
    bo, bl = np.zeros((heads, dim)), np.zeros(heads)
    if k.shape[0] == 0:
        return out, lse, bo, bl
    with np.errstate(all="ignore"):
        for h in range(heads):
            kh, vh = kf[:, h // per], vf[:, h // per]
            s = scale * (kh @ qf[h])
            A = np.abs(scale) * (np.abs(kh) @ np.abs(qf[h])).max()
            m = s.max()
            w = np.exp(s - m)
            l = w.sum()
            out[h] = w @ vh / l
            lse[h] = m + np.log(l)
            P = w @ np.abs(vh) / l
            n = k.shape[0]
            bo[h] = ((2.0 ** -11 + 2.0 ** -14 + n * 2.0 ** -25 + (dim + 8) * 2.0 ** -23 * A) * P
                     + 2.0 ** -32 * np.abs(vh).sum(0) + 2.0 ** -11 * np.abs(out[h]) + 2.0 ** -24)
            bl[h] = (dim + 8) * 2.0 ** -24 * A + n * 2.0 ** -27 + 2.0 ** -19 + 2.0 ** -22 * np.abs(lse[h])
    return out, lse, bo, bl
