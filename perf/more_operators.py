"""Cases of the operators around a decoding step: pages handed out to sequences, rotary positions, low-rank adapters beside a
shared projection, and the draw of the next token.

`run` computes a case either in its plain form (elementary torch operations) or, with `own`, through the package:

  pages   PagePool.trim and PagePool.extend: sequences give back the pages behind a length, then grow again; whole numbers only
  rotate  Rotary.rotate on queries and keys
  lora    Adapters.add: out = y + scale[id] * (x A[id]^T) B[id]^T, each row with an adapter of its own or none
  sample  sample: temperature, top-k, top-p and min-p from given random numbers
"""
import math
import random

import torch

own = False


# ------------------------------------------------------------------- cases

def _pages(name, seqs, page, length, new, ragged=True):
    return {"name": name, "op": "pages", "seqs": seqs, "page": page, "length": length, "new": new, "ragged": ragged}


def _rotate(name, rows, q_heads, kv_heads, dim, part, interleaved=False, farthest=2048, factor=1.0):
    return {"name": name, "op": "rotate", "rows": rows, "q_heads": q_heads, "kv_heads": kv_heads, "dim": dim, "part": part,
            "interleaved": interleaved, "farthest": farthest, "factor": factor}


def _sample(name, rows, vocab, wide, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, mixed=False, masked=False):
    return {"name": name, "op": "sample", "rows": rows, "vocab": vocab, "wide": wide, "temperature": temperature,
            "top_k": top_k, "top_p": top_p, "min_p": min_p, "mixed": mixed, "masked": masked}


def _lora(name, rows, k, n, rank, adapters, runs=False):
    return {"name": name, "op": "lora", "rows": rows, "k": k, "n": n, "rank": rank, "adapters": adapters, "runs": runs}


def listed():
    return [
        # A small batch drops the tokens that were drafted in vain and makes room for the next five: latency.
        _pages("pages 16 drafts of 5", 16, 256, 2000, 5, ragged=False),
        # A large serving batch, small pages, up to eight tokens to a sequence.
        _pages("pages 1024 of up to 8", 1024, 16, 4000, 8),
        # Prompts of a new batch, from nothing: 64 of up to 4096 tokens.
        _pages("pages 64 prompts", 64, 256, 0, 4096),
        # One decoding step of one sequence of the 70B-shaped block: 64 query and 8 key-value heads of 128.
        _rotate("rotate 1x72", 1, 64, 8, 128, 128),
        # Odd sizes: half of 96 channels, neighbours paired, far positions of a stretched context.
        _rotate("rotate 33x16 part", 33, 14, 2, 96, 48, interleaved=True, farthest=1000000, factor=32.0),
        # A prompt's chunk.
        _rotate("rotate 4096x72", 4096, 64, 8, 128, 128, farthest=131072),
        # One answer: a short list, then the nucleus of it.
        _sample("sample 1x32000 k40", 1, 32000, False, temperature=0.8, top_k=40, top_p=0.95),
        # A batch whose requests each bring their own settings, logits in 32 bits, some tokens forbidden.
        _sample("sample 16x50001 mixed", 16, 50001, True, mixed=True, masked=True),
        # A full serving batch over a large vocabulary, nucleus only.
        _sample("sample 256x131072 p0.9", 256, 131072, False, temperature=0.9, top_p=0.9),
        # One request with an adapter, 8192 x 8192 projection.
        _lora("lora 1x8192x8192 r16", 1, 8192, 8192, 16, 4),
        # A decoding batch in which requests use 16 adapters of different ranks, or none, beside the up projection.
        _lora("lora 48x8192x28672 r64", 48, 8192, 28672, 64, 16),
        # Prompts of several requests in one call.
        _lora("lora 2048x8192x8192 r32", 2048, 8192, 8192, 32, 6, runs=True),
    ]


_MOST_LOGITS = 256 * 131072
_MOST_ROWS = 64 * 4096
_MOST_HEADS = 4096 * 72 * 128
_MOST_LORA = 2048 * (8192 + 2 * 8192)


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["pages", "rotate", "sample", "sample", "lora", "lora"])
    if op == "pages":
        seqs = _log(rng, 1, 4096)
        new = _log(rng, 1, max(1, min(16384, _MOST_ROWS // seqs)))
        length = rng.randint(0, max(0, min(16384, 16 * _MOST_ROWS // seqs)))
        c = _pages("", seqs, rng.choice([16, 32, 48, 64, 128, 256]), length, new, rng.random() < 0.7)
    elif op == "rotate":
        dim = rng.choice([64, 80, 96, 128, 128, 256])
        kv = rng.choice([1, 2, 4, 5, 8])
        q = kv * rng.choice([1, 2, 4, 5, 7, 8, 16])
        rows = _log(rng, 1, max(1, min(16384, _MOST_HEADS // ((q + kv) * dim))))
        part = rng.choice([dim, dim, dim // 2, dim // 4])
        c = _rotate("", rows, q, kv, dim, part, rng.random() < 0.5, _log(rng, 1, 1 << 20), rng.choice([1.0, 1.0, 4.0, 32.0]))
    elif op == "sample":
        vocab = _log(rng, 1000, 262144)
        rows = _log(rng, 1, max(1, min(512, _MOST_LOGITS // 2 // vocab)))
        c = _sample("", rows, vocab, rng.random() < 0.5, rng.choice([0.0, 0.5, 0.7, 1.0, 1.0, 1.5]),
                    rng.choice([0, 0, 1, 20, 50, rng.randint(1, 1000), rng.randint(1, vocab)]),
                    rng.choice([1.0, 0.95, 0.9, rng.uniform(0.05, 1.0)]), rng.choice([0.0, 0.0, 0.05, 0.1, rng.uniform(0.0, 0.5)]),
                    rng.random() < 0.4, rng.random() < 0.4)
    else:
        k, n = rng.choice([1024, 2048, 4096, 8192, 28672, 1000]), rng.choice([1024, 2048, 4096, 8192, 28672, 1016])
        rows = _log(rng, 1, max(1, min(2048, _MOST_LORA // (k + 2 * n))))
        c = _lora("", rows, k, n, rng.choice([8, 16, 16, 32, 64, 128]), _log(rng, 1, 24), rng.random() < 0.5)
    del c["name"]
    return c


def _lengths(case):
    """(tokens kept, tokens added) by sequence: part of the case, not of the seed."""
    seqs, length, new = case["seqs"], case["length"], case["new"]
    if not case["ragged"]:
        return [length] * seqs, [new] * seqs
    rng = random.Random(1000003 * length + 101 * new + seqs)
    return ([length] + [rng.randint(0, length) for _ in range(seqs - 1)],
            [new] + [rng.randint(0, new) for _ in range(seqs - 1)])


def _ids(case):
    """The adapter of each row (-1: none), and each adapter's rank."""
    rng = random.Random(1000003 * case["rows"] + 101 * case["adapters"] + case["rank"])
    rows, n = case["rows"], case["adapters"]
    ids = [rng.randint(0, n - 1) if rng.random() < 0.9 or r == 0 else -1 for r in range(rows)]
    if case["runs"]:   # prompts: each row's adapter is its request's
        cuts = sorted(rng.randint(0, rows) for _ in range(min(rows, 12)))
        run = [rng.randint(0, n - 1) for _ in range(len(cuts) + 1)]
        ids = [run[sum(c <= r for c in cuts)] for r in range(rows)]
    return ids, [case["rank"] if i == 0 else rng.randint(max(1, case["rank"] // 2), case["rank"]) for i in range(n)]


def work(case):
    if case["op"] == "pages":
        kept, new = _lengths(case)
        page, moved = case["page"], 0
        for a, b in zip(kept, new):
            moved += -(-(a + b) // page) - -(-a // page)
        # a length, a kept length and a count read, lengths and an offset written; pages to the free list and back; two
        # numbers a row
        return {"bytes": 4 * 6 * case["seqs"] + 4 * 4 * moved + 8 * sum(new), "flops": 8 * case["seqs"] + 2 * sum(new)}
    if case["op"] == "rotate":
        values = case["rows"] * (case["q_heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": 4 * values + 4 * case["rows"] + 4 * case["part"], "flops": 3 * values}
    if case["op"] == "sample":
        values = case["rows"] * case["vocab"]
        return {"bytes": values * (4 if case["wide"] else 2) + 12 * case["rows"], "flops": 10 * values}
    ids, ranks = _ids(case)
    k, n = case["k"], case["n"]
    weights = sum(ranks[i] for i in set(ids) if i >= 0)
    return {"bytes": 2 * case["rows"] * (k + 2 * n) + 2 * weights * (k + n) + 4 * case["rows"],
            "flops": 2 * (k + n) * sum(ranks[i] for i in ids if i >= 0)}


# ------------------------------------------------------------------ inputs

def _rates(case):
    """Angles per token of a pair of channels, in 64 bits: the far half of a long wave's turns stretched by `factor`."""
    half = case["part"] // 2
    rate = [10000.0 ** (-2.0 * i / case["part"]) for i in range(half)]
    if case["factor"] == 1.0:
        return rate, 1.0
    out = []
    for f in rate:   # pairs that turn fewer than once in 4096 tokens are stretched, those with over 32 turns stay
        turns = 4096 * f / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1.0) / 31.0))
        out.append((1.0 - keep) * f / case["factor"] + keep * f)
    return out, 0.1 * math.log(case["factor"]) + 1.0


def prepare(case, seed):
    device = "cuda"
    gen = torch.Generator(device).manual_seed(seed)
    st = {"case": case}
    if case["op"] == "pages":
        _prepare_pages(st, gen, device)
    elif case["op"] == "rotate":
        rows, dim = case["rows"], case["dim"]
        heads = case["q_heads"] + 2 * case["kv_heads"]
        qkv = torch.randn((rows, heads, dim), generator=gen, device=device, dtype=torch.float16)
        # slices of the projections' common output
        st["q"], st["k"] = qkv[:, :case["q_heads"]], qkv[:, case["q_heads"]:case["q_heads"] + case["kv_heads"]]
        start = torch.randint(0, case["farthest"], (1,), generator=gen, device=device)
        st["positions"] = ((start + torch.arange(rows, device=device)) % case["farthest"]).to(torch.int32)
        rate, st["factor"] = _rates(case)
        st["rate"] = torch.tensor(rate, dtype=torch.float64, device=device)
    elif case["op"] == "sample":
        _prepare_sample(st, gen, device)
    else:
        ids, ranks = _ids(case)
        rows, k, n, rank, count = case["rows"], case["k"], case["n"], case["rank"], case["adapters"]
        st["ids"] = torch.tensor(ids, dtype=torch.int32, device=device)
        st["ranks"] = torch.tensor(ranks, dtype=torch.int32, device=device)
        st["scales"] = torch.rand((count,), generator=gen, device=device) + 0.5
        st["a"] = torch.randn((count, rank, k), generator=gen, device=device, dtype=torch.float16).mul_(k ** -0.5)
        st["b"] = torch.randn((count, n, rank), generator=gen, device=device, dtype=torch.float16).mul_(rank ** -0.5)
        st["x"] = torch.randn((rows, k), generator=gen, device=device, dtype=torch.float16)
        st["y"] = torch.randn((rows, n), generator=gen, device=device, dtype=torch.float16)
    if own:   # the handles that a program keeps
        import mixed_bitrate_quantized_amd as exq
        if case["op"] == "pages":
            st["pool"] = exq.PagePool(st["free"].numel(), case["page"], *st["table"].shape, device=device)
            for name in ("table", "lengths", "free", "free_count"):
                getattr(st["pool"], name).copy_(st[name])
        elif case["op"] == "rotate":
            st["rotary"] = exq.Rotary(case["dim"], case["part"], interleaved=case["interleaved"], rates=rate, factor=st["factor"],
                                      device=device)
        elif case["op"] == "lora":
            st["adapters"] = exq.Adapters(st["a"], st["b"], scales=st["scales"], ranks=st["ranks"])
    return st


def _prepare_pages(st, gen, device):
    """Sequences as they are after `new` tokens that are about to be dropped, their pages in any order."""
    case = st["case"]
    kept, new = (torch.tensor(x, dtype=torch.int64, device=device) for x in _lengths(case))
    page = case["page"]
    lengths = kept + new
    have = (lengths + page - 1) // page
    used = sum(-(-(a + b) // page) for a, b in zip(*_lengths(case)))
    width = max(-(-(a + b) // page) for a, b in zip(*_lengths(case))) + 1
    n_pages = used + 1 + used // 8
    order = torch.randperm(n_pages, generator=gen, device=device).to(torch.int32)
    col = torch.arange(width, device=device)
    holds = col < have[:, None]
    at = (torch.cumsum(holds.view(-1), 0) - 1).view(holds.shape)
    st["table"] = torch.where(holds, order[torch.clamp(at, min=0)], torch.full_like(at, -1, dtype=torch.int32))
    st["free"] = torch.cat([order[used:], torch.full((used,), -1, dtype=torch.int32, device=device)])
    st["free_count"] = torch.tensor([n_pages - used], dtype=torch.int32, device=device)
    st["lengths"] = lengths.to(torch.int32)
    st["kept"], st["new"] = kept.to(torch.int32), new.to(torch.int32)
    st["rows"] = max(1, sum(_lengths(case)[1]))


def _prepare_sample(st, gen, device):
    case = st["case"]
    rows, vocab = case["rows"], case["vocab"]
    # a few likely tokens and a long tail, anywhere in the vocabulary
    tail = -1.2 * torch.log1p(torch.arange(vocab, device=device, dtype=torch.float32)) + 12.0
    logits = torch.empty((rows, vocab), device=device, dtype=torch.float32 if case["wide"] else torch.float16)
    for r in range(rows):
        noise = 0.8 * torch.randn((vocab,), generator=gen, device=device)
        logits[r] = (tail + noise)[torch.randperm(vocab, generator=gen, device=device)].to(logits.dtype)
        if case["masked"]:
            logits[r, torch.rand((vocab,), generator=gen, device=device) < 0.1] = -math.inf
    st["logits"] = logits
    st["u"] = torch.rand((rows,), generator=gen, device=device)
    for name in ("temperature", "top_k", "top_p", "min_p"):
        st[name] = case[name]
    if case["mixed"]:   # requests with settings of their own
        rng = random.Random(1000003 * rows + vocab)
        st["temperature"] = torch.tensor([rng.choice([0.0, 0.6, 0.8, 1.0, 1.3]) for _ in range(rows)], device=device)
        st["top_k"] = torch.tensor([rng.choice([0, 0, 1, 20, 50, 200]) for _ in range(rows)], dtype=torch.int32, device=device)
        st["top_p"] = torch.tensor([rng.choice([1.0, 0.95, 0.8]) for _ in range(rows)], device=device)
        st["min_p"] = torch.tensor([rng.choice([0.0, 0.0, 0.02, 0.1]) for _ in range(rows)], device=device)


# --------------------------------------------------------------------- run

def _pages_plain(st):
    """Pages behind `kept` go to the free list, last one first; then each sequence takes what `new` tokens need from its end."""
    page, table, free = st["case"]["page"], st["table"], st["free"]
    col = torch.arange(table.shape[1], device=table.device)
    pages = lambda n: (n.long() + page - 1) // page
    old = torch.minimum(st["lengths"], st["kept"])
    given = (col >= pages(old)[:, None]) & (col < pages(st["lengths"])[:, None])
    at = (torch.cumsum(given.view(-1), 0) - 1).view(given.shape)
    total = given.sum()
    slots = torch.cat([free, free[:1]])   # one more, for what is not given back
    place = torch.where(given, st["free_count"] + total - 1 - at, torch.full_like(at, free.numel()))
    slots[place.view(-1)] = table.view(-1)
    top = st["free_count"] + total
    table = torch.where(given, torch.full_like(table, -1), table)
    lengths = old + st["new"]
    taken = (col >= pages(old)[:, None]) & (col < pages(lengths)[:, None])
    at = (torch.cumsum(taken.view(-1), 0) - 1).view(taken.shape)
    table = torch.where(taken, slots[torch.where(taken, top - 1 - at, torch.zeros_like(at))], table)
    ends = torch.cumsum(st["new"].long(), 0)
    offsets = torch.cat([torch.zeros_like(ends[:1]), ends]).to(torch.int32)
    r = torch.arange(st["rows"], device=table.device)
    s = torch.clamp(torch.searchsorted(ends, r, right=True), max=ends.numel() - 1)
    used = r < ends[-1]
    seqs = torch.where(used, s, torch.full_like(s, -1)).to(torch.int32)
    positions = torch.where(used, old[s] + r - offsets[s], torch.zeros_like(r)).to(torch.int32)
    count = (top - taken.sum()).to(torch.int32)
    st["table"].copy_(table)
    st["free"].copy_(slots[:-1])
    st["free_count"].copy_(count)
    st["lengths"].copy_(lengths)
    return [st["table"], st["lengths"], st["free_count"], seqs, positions, offsets]


def _turned(x, cos, sin, part, interleaved):
    a, rest = x[..., :part], x[..., part:]
    if interleaved:
        u, v = a[..., 0::2], a[..., 1::2]
        a = torch.stack([u * cos - v * sin, u * sin + v * cos], -1).flatten(-2)
    else:
        u, v = a[..., :part // 2], a[..., part // 2:]
        a = torch.cat([u * cos - v * sin, u * sin + v * cos], -1)
    return torch.cat([a, rest], -1)


def _rotate_plain(st):
    case = st["case"]
    angle = st["positions"].double()[:, None, None] * st["rate"]
    cos, sin = (torch.cos(angle) * st["factor"]).float(), (torch.sin(angle) * st["factor"]).float()
    return [_turned(st[x].float(), cos, sin, case["part"], case["interleaved"]).half() for x in ("q", "k")]


def _column(v, rows, like):
    return (v if isinstance(v, torch.Tensor) else torch.full((rows,), v, device=like.device)).double()[:, None]


def _sample_plain(st):
    logits = st["logits"].float()
    rows, vocab = logits.shape
    value, order = torch.sort(logits, dim=-1, descending=True, stable=True)
    t, p, m = (_column(st[x], rows, logits) for x in ("temperature", "top_p", "min_p"))
    k = _column(st["top_k"], rows, logits)
    z = (value.double() - value[:, :1].double()) / torch.where(t > 0, t, torch.ones_like(t))
    w = torch.exp(z)
    rank = torch.arange(vocab, device=logits.device)
    w = torch.where((k > 0) & (rank >= k), torch.zeros_like(w), w)
    before = torch.cumsum(w, -1) - w
    w = torch.where((p < 1) & (rank > 0) & (before >= p * w.sum(-1, keepdim=True)), torch.zeros_like(w), w)
    w = torch.where((w < m) & (rank > 0), torch.zeros_like(w), w)
    w = torch.where((t == 0) & (rank > 0), torch.zeros_like(w), w)
    w = torch.zeros_like(w).scatter(1, order, w)            # by token again
    sums = torch.cumsum(w, -1)
    total = w.sum(-1, keepdim=True)
    hit = (sums > st["u"].double()[:, None] * total) & (w > 0)
    token = hit.to(torch.uint8).argmax(-1)
    drawn = torch.gather(w, 1, token[:, None]) / total
    return [token.to(torch.int32), torch.log(drawn)[:, 0].float()]


def _lora_plain(st):
    """Every row times every adapter, then what is not the row's own is dropped."""
    x, a, b = st["x"].float(), st["a"].float(), st["b"].float()
    count, rank, k = a.shape
    mine = st["ids"].long()[:, None] == torch.arange(count, device=x.device)
    held = torch.arange(rank, device=x.device) < st["ranks"][:, None]
    weight = mine[:, :, None] * held * st["scales"][:, None]
    low = torch.matmul(x, a.view(count * rank, k).t()).view(-1, count, rank) * weight
    wide = b.permute(0, 2, 1).reshape(count * rank, -1)
    return [(st["y"].float() + torch.matmul(low.view(-1, count * rank), wide)).half()]


def run(st):
    op = st["case"]["op"]
    if own:
        import mixed_bitrate_quantized_amd as exq
        if op == "pages":
            pool = st["pool"]
            pool.trim(st["kept"])
            seqs, positions, offsets = pool.extend(st["new"], st["rows"])
            return [pool.table, pool.lengths, pool.free_count, seqs, positions, offsets]
        if op == "rotate":
            return list(st["rotary"].rotate(st["q"], st["positions"], k=st["k"]))
        if op == "sample":
            return list(exq.sample(st["logits"], st["u"], st["temperature"], st["top_k"], st["top_p"], st["min_p"],
                                   return_logprobs=True))
        return [st["adapters"].add(st["x"], st["ids"], st["y"])]
    return {"pages": _pages_plain, "rotate": _rotate_plain, "sample": _sample_plain, "lora": _lora_plain}[op](st)


# ------------------------------------------------------------------- exact

def _exact_row(logits, u, t, k, p, m):
    """The probability of the token drawn, and its number, from one row of logits in 64 bits."""
    z = logits.double()
    top = z.max()
    if t == 0:
        return 0.0, int((z == top).nonzero()[0])
    order = torch.argsort(-z, stable=True)
    w = torch.exp((z[order] - top) / t)
    if k > 0:
        w = w[:k]
    if p < 1:
        reach = torch.cumsum(w, 0) >= p * w.sum()
        first = reach.nonzero()
        w = w[:int(first[0]) + 1] if len(first) else w
    w = w[:max(1, int((w >= m).sum()))]
    keep, by = torch.sort(order[:w.numel()])
    w = w[by]
    sums = torch.cumsum(w, 0)
    at = int((sums > u * w.sum()).nonzero()[0])
    return float(torch.log(w[at] / w.sum())), int(keep[at])


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "pages":
        return None
    if case["op"] == "rotate":
        rows, half = case["rows"], case["part"] // 2
        angle = st["positions"].double()[:, None] * st["rate"][None, :]
        turn = torch.polar(torch.full_like(angle, st["factor"]), angle)[:, None, :]
        out = []
        for x in (st["q"], st["k"]):
            x = x.double().clone()
            i = torch.arange(half, device=x.device)
            first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + half)
            z = torch.complex(x[..., first].contiguous(), x[..., second].contiguous()) * turn
            x[..., first], x[..., second] = z.real, z.imag
            out.append(x)
        return out
    if case["op"] == "sample":
        at = lambda v, r: float(v[r]) if isinstance(v, torch.Tensor) else v
        found = [_exact_row(st["logits"][r], float(st["u"][r]), at(st["temperature"], r), int(at(st["top_k"], r)), at(st["top_p"], r),
                            at(st["min_p"], r)) for r in range(case["rows"])]
        logs, tokens = zip(*found)
        return [torch.tensor(tokens, dtype=torch.int32), torch.tensor(logs, dtype=torch.float64)]
    ids, ranks = _ids(case)
    out = st["y"].double()
    for i, rank in enumerate(ranks):
        rows = torch.tensor([r for r, j in enumerate(ids) if j == i], dtype=torch.int64, device=out.device)
        if not len(rows):
            continue
        low = st["x"][rows].double() @ st["a"][i, :rank].double().t().contiguous()
        out[rows] += st["scales"][i].double() * (low @ st["b"][i, :, :rank].double().t().contiguous())
    return [out]
