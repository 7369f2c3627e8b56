"""Cases of the key-value cache operators: writing a paged cache, reading it back, and attention of one new token over it.

`run` computes a case either in its plain form (elementary torch operations) or, with `own`, through the package's
`KVCache`.  Both work on the same pages, whose layout is the one that include/exq.h documents:

  a page is [kv head][tile of 16 tokens][tile bytes], a tile [key codes][key scales][value codes][value scales];
  with G = head_dim / 32 groups and gpc = 16 / bits groups to a chunk, chunk j of a code part starts at byte 1024 j and
  holds n_j = min(gpc, G - j gpc) groups: lane l of 64 owns bytes [l n_j bits, (l + 1) n_j bits) of it, `bits` bytes for
  each group (8 elements).  Keys: lane 16 q + t holds channels 32 g + 8 q + e of token t.  Values: lane 16 (t / 4) + c
  holds channels 32 g + c and 32 g + 16 + c of tokens 4 (t / 4) .. + 3.  Scales are fp16, keys [token][G], values
  [token / 4][G][token % 4].  16-bit parts hold fp16 values and have no scales.
"""
import math
import random

import torch

own = False

GROUP = 32
TILE = 16


# ------------------------------------------------------------------- cases

def _attend(name, batch, length, bits, q_heads=64, kv_heads=8, dim=128, page=256, ragged=False, window=0):
    k_bits, v_bits = bits
    return {"name": name, "op": "attend", "batch": batch, "length": length, "k_bits": k_bits, "v_bits": v_bits,
            "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "page": page, "ragged": ragged, "window": window}


def _rows(name, op, batch, length, new, bits, kv_heads=8, dim=128, page=256):
    k_bits, v_bits = bits
    return {"name": name, "op": op, "batch": batch, "length": length, "new": new, "k_bits": k_bits, "v_bits": v_bits,
            "kv_heads": kv_heads, "dim": dim, "page": page}


def listed():
    return [
        # One sequence of the 70B-shaped block (64 query heads, 8 key-value heads of 128) early in an answer: latency.
        _attend("attend 1x100 4bit", 1, 100, (4, 4)),
        # The same sequence at the end of its 2048-token context.
        _attend("attend 1x2048 4bit", 1, 2048, (4, 4)),
        # One long document: the only parallelism is along its length.
        _attend("attend 1x131072 4bit", 1, 131072, (4, 4)),
        # A serving batch of 16 with mixed lengths, keys held more finely than values.
        _attend("attend 16x8192 ragged k8v4", 16, 8192, (8, 4), page=64, ragged=True),
        # The same batch with an unquantized cache.
        _attend("attend 16x4096 16bit", 16, 4096, (16, 16)),
        # Odd sizes: 7 query heads to a key-value head, 96 channels, pages of one tile, a sliding window, an empty row.
        _attend("attend 5x1999 8bit window", 5, 1999, (8, 8), q_heads=14, kv_heads=2, dim=96, page=16, ragged=True,
                window=1023),
        # A full serving batch: the largest call.
        _attend("attend 32x16384 4bit", 32, 16384, (4, 4)),
        # One decoding step's new tokens, 16 sequences at odd positions, written and read back.
        _rows("write 16x1 4bit", "write", 16, 1000, 1, (4, 4)),
        # A prompt's chunk written behind an earlier one that ended inside a tile, and read back for its own attention.
        _rows("write 1x4096 k8v4", "write", 1, 1001, 4096, (8, 4)),
        # Whole prompts of a batch, from empty pages.
        _rows("write 4x4096 4bit", "write", 4, 0, 4096, (4, 4)),
        # A long shared prefix read back as fp16 for a prompt's attention.
        _rows("read 1x32768 4bit", "read", 1, 0, 32768, (4, 4)),
        # A few short tails read back, odd sizes.
        _rows("read 7x33 8bit", "read", 7, 21, 33, (8, 8), kv_heads=2, dim=64, page=32),
    ]


# What the largest listed case reads of its cache (144 bytes a token and head) and computes; a drawn one stays below both.
_MOST_BYTES = 32 * 16384 * 8 * 144
_MOST_FLOPS = 32 * 16384 * 4 * 64 * 128


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "write", "read"])
    bits = rng.choice([(4, 4), (8, 8), (8, 4), (4, 8), (16, 16)])
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    dim = rng.choice([64, 96, 128, 128, 256])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    batch = _log(rng, 1, 64)
    token = kv_heads * _row_bytes(dim, *bits)
    if op == "attend":
        q_heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8, 16])
        most = max(1, min(131072, _MOST_BYTES // (batch * token), _MOST_FLOPS // (4 * batch * q_heads * dim)))
        window = rng.choice([0, 0, 0, rng.randint(1, 4096)])
        c = _attend("", batch, _log(rng, 1, most), bits, q_heads, kv_heads, dim, page, rng.random() < 0.5, window)
    else:
        most = max(1, min(32768, 32768 * 8 * 144 // (batch * token)))
        c = _rows("", op, batch, rng.randint(0, 4096), _log(rng, 1, most), bits, kv_heads, dim, page)
    del c["name"]
    return c


def _lengths(case):
    """Tokens in the cache, by sequence: part of the case, not of the seed."""
    batch, length = case["batch"], case["length"]
    if not case.get("ragged"):
        return [length] * batch
    rng = random.Random(1000003 * length + batch)
    out = [length] + [rng.randint(1, length) for _ in range(batch - 1)]
    if batch >= 4:
        out[1] = 0
    return out


def _row_bytes(dim, k_bits, v_bits):
    scale = 2 * (dim // GROUP)
    return dim * k_bits // 8 + dim * v_bits // 8 + (scale if k_bits < 16 else 0) + (scale if v_bits < 16 else 0)


def work(case):
    dim, heads = case["dim"], case["kv_heads"]
    row = heads * _row_bytes(dim, case["k_bits"], case["v_bits"])
    if case["op"] == "attend":
        seen = [min(n, case["window"]) if case["window"] else n for n in _lengths(case)]
        io = 4 * case["batch"] * case["q_heads"] * dim
        table = sum(-(-n // case["page"]) for n in seen)
        return {"bytes": sum(seen) * row + io + 4 * table + 4 * case["batch"],
                "flops": 4 * case["q_heads"] * dim * sum(seen)}
    rows = case["batch"] * case["new"]
    values = 4 * rows * heads * dim            # fp16 keys and values on the user's side
    if case["op"] == "read":
        return {"bytes": rows * (row + 8) + values, "flops": 2 * rows * heads * dim}
    # written, and read back: the rows' values in and out, the cache's bytes written and read
    return {"bytes": 2 * rows * (row + 8) + 2 * values, "flops": 10 * rows * heads * dim}


# ------------------------------------------------------------------ layout

def _code_places(dim, bits, value, device):
    """Byte of a tile's code part for (token in the tile, byte of the token's row); int64 [16][dim * bits / 8]."""
    G, gpc = dim // GROUP, 16 // bits
    t = torch.arange(TILE, device=device)[:, None, None]
    g = torch.arange(G, device=device)[None, :, None]
    b = torch.arange(4 * bits, device=device)[None, None, :]      # the row's bytes in a group
    j = g // gpc
    n = torch.clamp(G - j * gpc, max=gpc)
    if not value:                      # (q, byte)
        lane, inner = 16 * (b // bits) + t, b % bits
    elif bits == 4:                    # c; the two channels share the byte, tokens in the order 0, 2, 1, 3
        lane, inner = 16 * (t // 4) + b, (t % 2) * 2 + (t % 4) // 2
    else:                              # (half of the group, c, byte of the value)
        w = bits // 8
        lane, inner = 16 * (t // 4) + b // w % 16, b // (16 * w) * 4 * w + (t % 4) * w + b % w
    at = 1024 * j + lane * (n * bits) + (g - j * gpc) * bits + inner
    return at.reshape(TILE, -1)


def _scale_places(dim, value, device):
    G = dim // GROUP
    t = torch.arange(TILE, device=device)[:, None, None]
    g = torch.arange(G, device=device)[None, :, None]
    b = torch.arange(2, device=device)[None, None, :]
    at = (t // 4) * 8 * G + g * 8 + (t % 4) * 2 + b if value else t * 2 * G + 2 * g + b
    return at.reshape(TILE, -1)


def _places(case, device):
    """Byte of the tile for (token, byte of its row), a row being [key codes][key scales][value codes][value scales]."""
    dim, base, parts = case["dim"], 0, []
    for bits, value in ((case["k_bits"], False), (case["v_bits"], True)):
        parts.append(base + _code_places(dim, bits, value, device))
        base += TILE * dim * bits // 8
        if bits < 16:
            parts.append(base + _scale_places(dim, value, device))
            base += TILE * 2 * (dim // GROUP)
    return torch.cat(parts, 1)


def _page_bytes(case):
    return case["page"] * case["kv_heads"] * _row_bytes(case["dim"], case["k_bits"], case["v_bits"])


def _pack(x, bits, value):
    """fp16 [..., dim] -> the row's bytes, uint8 [..., codes and scales]."""
    if bits == 16:
        return x.contiguous().view(torch.uint8)
    top = (1 << (bits - 1)) - 1
    f = x.float().reshape(*x.shape[:-1], -1, GROUP)
    s = (f.abs().amax(-1, keepdim=True) / top).half()
    c = torch.clamp(torch.round(f / s.float()), -top, top)
    c = (torch.where(s == 0, torch.zeros_like(c), c) + (top + 1)).to(torch.uint8)
    scales = s.squeeze(-1).contiguous().view(torch.uint8)
    if bits == 4 and value:
        c = c[..., :16] | (c[..., 16:] << 4)
    elif bits == 4:
        c = c.reshape(*c.shape[:-1], 4, 8)
        c = c[..., [0, 4, 1, 5]] | (c[..., [2, 6, 3, 7]] << 4)
    return torch.cat([c.reshape(*x.shape[:-1], -1), scales], -1)


def _unpack(codes, scales, bits, value):
    """A row's code and scale bytes -> its values, float32 [..., dim] (each one rounded to fp16)."""
    if bits == 16:
        return codes.contiguous().view(torch.float16).float()
    if bits == 4 and value:
        codes = codes.reshape(*codes.shape[:-1], -1, 16)
        codes = torch.cat([codes & 15, codes >> 4], -1)
    elif bits == 4:
        codes = codes.reshape(*codes.shape[:-1], -1, 4)
        codes = torch.cat([codes & 15, codes >> 4], -1)[..., [0, 2, 4, 6, 1, 3, 5, 7]]
    s = scales.contiguous().view(torch.float16).float()
    c = codes.reshape(*s.shape, GROUP).float() - (1 << (bits - 1))
    return (c * s[..., None]).half().float().reshape(*s.shape[:-1], -1)


def _split(row, case):
    """A row's bytes -> float32 keys and values."""
    out, base, dim = [], 0, case["dim"]
    for bits, value in ((case["k_bits"], False), (case["v_bits"], True)):
        n, m = dim * bits // 8, 2 * (dim // GROUP) if bits < 16 else 0
        out.append(_unpack(row[..., base:base + n], row[..., base + n:base + n + m], bits, value))
        base += n + m
    return out


def _row_places(st):
    """Byte of the pages for (row, head, byte of the row)."""
    case, page = st["case"], st["case"]["page"]
    pos = st["pos"].long()
    at = st["table"][st["seq"].long(), pos // page].long() * _page_bytes(case)
    tile_bytes = TILE * _row_bytes(case["dim"], case["k_bits"], case["v_bits"])
    head = torch.arange(case["kv_heads"], device=pos.device) * (page // TILE) * tile_bytes
    at = at + pos % page // TILE * tile_bytes
    return at[:, None, None] + head[None, :, None] + _places(case, pos.device)[pos % TILE][:, None, :]


def _write(st, k, v):
    case = st["case"]
    rows = torch.cat([_pack(k, case["k_bits"], False), _pack(v, case["v_bits"], True)], -1)
    st["pages"].view(-1)[_row_places(st)] = rows


def _read(st):
    return [x.half() for x in _split(st["pages"].view(-1)[_row_places(st)], st["case"])]


# ------------------------------------------------------------------ inputs

def _heads_values(gen, shape, spread, device):
    """Keys or values of (tokens, heads, dim): normal, a few channels of each head much larger than the rest."""
    x = torch.randn(shape, generator=gen, device=device, dtype=torch.float16)
    channel = torch.exp(spread * torch.randn(shape[-2:], generator=gen, device=device)).half()
    return x.mul_(channel)


def prepare(case, seed):
    device = "cuda"
    gen = torch.Generator(device).manual_seed(seed)
    batch, heads, dim, page = case["batch"], case["kv_heads"], case["dim"], case["page"]
    lengths = _lengths(case)
    total = max(lengths) + case.get("new", 0)
    width = -(-max(total, 1) // page)
    n_pages = batch * width
    st = {"case": case}
    # pages are handed out in any order
    st["table"] = torch.randperm(n_pages, generator=gen, device=device).to(torch.int32).view(batch, width)
    st["pages"] = torch.zeros((n_pages, _page_bytes(case)), dtype=torch.uint8, device=device)
    if case["op"] == "attend":
        st["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=device)
        st["q"] = torch.randn((batch, case["q_heads"], dim), generator=gen, device=device, dtype=torch.float16)
        st["scale"] = 1.0 / math.sqrt(dim)
        places = _places(case, device).view(-1)
        tiles = page // TILE
        pages = st["pages"].view(n_pages, heads, tiles, -1)
        for b in range(batch):
            k = _heads_values(gen, (width * page, heads, dim), 0.5, device)
            v = _heads_values(gen, (width * page, heads, dim), 0.3, device)
            rows = torch.cat([_pack(k, case["k_bits"], False), _pack(v, case["v_bits"], True)], -1)
            rows = rows.view(width, tiles, TILE, heads, -1).permute(0, 3, 1, 2, 4).reshape(width, heads, tiles, -1)
            laid = torch.empty_like(rows)
            laid[..., places] = rows
            pages[st["table"][b].long()] = laid
    else:
        new, start = case["new"], case["length"]
        st["seq"] = torch.arange(batch, device=device, dtype=torch.int32).repeat_interleave(new)
        st["pos"] = (start + torch.arange(new, device=device, dtype=torch.int32)).repeat(batch)
        k = _heads_values(gen, (batch * new, heads, dim), 0.5, device)
        v = _heads_values(gen, (batch * new, heads, dim), 0.3, device)
        if case["op"] == "write":
            st["k"], st["v"] = k, v
        else:
            _write(st, k, v)
    if own:   # the handle that a program keeps beside its pages
        import mixed_bitrate_quantized_amd as exq
        st["cache"] = exq.KVCache(n_pages, page, heads, dim, case["k_bits"], case["v_bits"], pages=st["pages"])
    return st


# --------------------------------------------------------------------- run

def _attend_plain(st):
    case = st["case"]
    batch, heads, dim, page = case["batch"], case["kv_heads"], case["dim"], case["page"]
    places = _places(case, st["pages"].device)
    x = st["pages"].view(-1, heads, page // TILE, TILE * places.shape[1])[st["table"].long()]
    rows = x[..., places.view(-1)].view(*x.shape[:-1], TILE, -1).transpose(1, 2).reshape(batch, heads, -1, places.shape[1])
    k, v = _split(rows, case)
    q = st["q"].float().view(batch, heads, -1, dim)
    s = torch.matmul(q, k.transpose(-1, -2)) * st["scale"]
    pos = torch.arange(k.shape[2], device=k.device)[None, :]
    n = st["lengths"].long()[:, None]
    seen = pos < n
    if case["window"]:
        seen = seen & (pos >= n - case["window"])
    seen = seen[:, None, None, :]
    s = torch.where(seen, s, torch.full_like(s, -1e30))
    m = s.amax(-1, keepdim=True)
    p = torch.where(seen, torch.exp(s - m), torch.zeros_like(s))
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(l > 0, l, torch.ones_like(l))
    lse = torch.where(l > 0, m + torch.log(l), torch.full_like(l, -math.inf))
    return [o.half().reshape(st["q"].shape), lse.view(batch, -1)]


def run(st):
    op = st["case"]["op"]
    if own:
        cache = st["cache"]
        if op == "attend":
            return list(cache.attend(st["q"], st["table"], st["lengths"], scale=st["scale"], window=st["case"]["window"],
                                     return_lse=True))
        if op == "write":
            cache.append(st["k"], st["v"], st["table"], st["seq"], st["pos"])
        return list(cache.read(st["table"], st["seq"], st["pos"]))
    if op == "attend":
        return _attend_plain(st)
    if op == "write":
        _write(st, st["k"], st["v"])
    return _read(st)


# ------------------------------------------------------------------- exact

def _value(at, pages, bits, scale_at, nibble):
    """Values in 64 bits of elements whose code lies in byte `at` (its high nibble where `nibble`), scale at `scale_at`."""
    if bits == 16:
        half = pages[at].to(torch.int32) | (pages[at + 1].to(torch.int32) << 8)
        return half.to(torch.int16).view(torch.float16).double()
    code = pages[at].long()
    if bits == 4:
        code = torch.where(nibble, code >> 4, code & 15)
    s = pages[scale_at].to(torch.int32) | (pages[scale_at + 1].to(torch.int32) << 8)
    s = s.to(torch.int16).view(torch.float16).double()
    return ((code - (1 << (bits - 1))) * s).half().double()   # the product is exact in 64 bits, the value is held in 16


def _elements(case, pages, base, token):
    """Keys and values in 64 bits, element by element: base is the tile's first byte and token its token, both [n][heads]."""
    dim = case["dim"]
    G = dim // GROUP
    d = torch.arange(dim, device=base.device)
    g, r = d // GROUP, d % GROUP
    out, start = [], base[..., None]
    t = token[..., None]
    for bits, value in ((case["k_bits"], False), (case["v_bits"], True)):
        gpc = 16 // bits
        j = g // gpc
        own_bytes = torch.minimum(torch.full_like(j, gpc), G - j * gpc) * bits
        if value:
            lane, half = 16 * (t // 4) + r % 16, r // 16
            if bits == 4:
                shift = 16 * (t % 2) + 8 * (t % 4 // 2) + 4 * half
            else:
                shift = bits * (4 * half + t % 4)
            scale = (t // 4) * 8 * G + 8 * g + 2 * (t % 4)
        else:
            lane, e = 16 * (r // 8) + t, r % 8
            shift = 4 * (e // 2) + 16 * (e % 2) if bits == 4 else bits * e
            scale = 2 * G * t + 2 * g
        at = start + 1024 * j + lane * own_bytes + (g % gpc) * bits + shift // 8
        scale_at = start + TILE * dim * bits // 8 + scale
        out.append(_value(at, pages, bits, scale_at, (shift % 8 == 4).expand(at.shape)))
        start = start + TILE * dim * bits // 8 + (TILE * 2 * G if bits < 16 else 0)
    return out


def _rounded(x, bits):
    """What x becomes when it is held in `bits` bits, from the definition: 64 bits but for the two stated roundings to fp16."""
    x = x.double()
    if bits == 16:
        return x
    top = 2 ** (bits - 1) - 1
    groups = x.unflatten(-1, (x.shape[-1] // GROUP, GROUP))
    s = (groups.abs().max(-1).values / top).half().double()[..., None]
    ratio = torch.where(s > 0, groups / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(groups))
    return (ratio.round().clamp(-top, top) * s).half().double().flatten(-2)


def exact(case, seed):
    st = prepare(case, seed)
    heads, dim, page = case["kv_heads"], case["dim"], case["page"]
    pages = st["pages"].view(-1)
    if case["op"] == "write":
        return [_rounded(st["k"], case["k_bits"]), _rounded(st["v"], case["v_bits"])]
    tile_bytes = TILE * _row_bytes(dim, case["k_bits"], case["v_bits"])
    head = torch.arange(heads, device=pages.device) * (page // TILE * tile_bytes)

    def rows(table_row, pos):
        base = table_row[pos // page].long() * _page_bytes(case) + pos % page // TILE * tile_bytes
        return _elements(case, pages, base[:, None] + head, (pos % TILE)[:, None].expand(-1, heads))

    if case["op"] == "read":
        parts = [rows(st["table"][b], st["pos"][st["seq"] == b].long()) for b in range(case["batch"])]
        return [torch.cat(x) for x in zip(*parts)]
    outs, lses = [], []
    per = case["q_heads"] // heads
    for b, n in enumerate(_lengths(case)):
        q = st["q"][b].double().view(heads, per, dim)
        o = torch.zeros((heads, per, dim), dtype=torch.float64, device=q.device)
        top = torch.full((heads, per), -math.inf, dtype=torch.float64, device=q.device)
        total = torch.zeros_like(top)
        first = max(0, n - case["window"]) if case["window"] else 0
        for a in range(first, n, 8192):
            k, v = rows(st["table"][b], torch.arange(a, min(n, a + 8192), device=q.device))
            s = (q @ k.permute(1, 2, 0).contiguous()) * st["scale"]
            new = torch.maximum(top, s.max(-1).values)
            p = torch.exp(s - new[..., None])
            keep = torch.exp(top - new)
            total = total * keep + p.sum(-1)
            o = o * keep[..., None] + p @ v.transpose(0, 1).contiguous()
            top = new
        outs.append((o / torch.where(total > 0, total, torch.ones_like(total))[..., None]).view(-1, dim))
        lses.append((top + torch.log(total)).view(-1))
    return [torch.stack(outs), torch.stack(lses)]
