"""Pages, rotary positions, adapters and the draw on the CPU: refusals through the C-ABI and of tensors, rates, references.

No test here launches a kernel: every call fails validation first, or has no rows."""
import math

import numpy as np
import pytest

import mixed_bitrate_quantized_amd as exq
from oracle import stepref as ref

I, U = exq.EXQ_ERR_INVALID_ARG, exq.EXQ_ERR_UNSUPPORTED
B = 1 << 32   # apart by more than any call's arrays; never dereferenced


def at(i):
    return B * (i + 1)


def expect(status, fn, *args, **kw):
    with pytest.raises(exq.ExqError) as ei:
        fn(*args, **kw)
    assert ei.value.status == status, ei.value


# ------------------------------------------------------------------- pages

def pages_args(extend, **kw):
    a = dict(table=at(0), sequences=5, width=7, stride=7, page=16, lengths=at(1), change=at(2), free=at(3), count=at(4), n=40,
             seqs=at(5), positions=at(6), rows=9, offsets=at(7), served=at(8), ws=at(9), wsb=48)
    a.update(kw)
    head = [a[x] for x in ("table", "sequences", "width", "stride", "page", "lengths", "change", "free", "count", "n")]
    return head + ([a[x] for x in ("seqs", "positions", "rows", "offsets", "served")] if extend else []) + [a["ws"], a["wsb"], 0]


BAD_PAGES = [dict(table=0), dict(table=at(0) + 2), dict(sequences=0), dict(width=0), dict(stride=6), dict(stride=-7), dict(page=0),
             dict(lengths=0), dict(lengths=at(1) + 1), dict(change=0), dict(free=0), dict(count=0), dict(n=0), dict(ws=0),
             dict(wsb=47), dict(lengths=at(0)), dict(change=at(1) + 16), dict(free=at(2) - 4), dict(count=at(0) + 4 * 34),
             dict(ws=at(3) + 156), dict(ws=at(9) + 2)]


@pytest.mark.parametrize("bad", BAD_PAGES, ids=str)
def test_pages_reject(bad):
    expect(I, exq.exq_pages_extend, *pages_args(True, **bad))
    expect(I, exq.exq_pages_trim, *pages_args(False, **bad))


@pytest.mark.parametrize("bad", [dict(seqs=0), dict(positions=0), dict(rows=-1), dict(offsets=0), dict(served=0),
                                 dict(seqs=at(6) + 32), dict(offsets=at(1) - 20), dict(served=at(4)), dict(positions=at(9) + 44)],
                         ids=str)
def test_extend_rejects(bad):
    expect(I, exq.exq_pages_extend, *pages_args(True, **bad))


def test_pages_reject_tables_over_32_bits():
    big = dict(sequences=1 << 16, width=1 << 15, stride=1 << 15, wsb=1 << 30)
    far = {x: B * B.bit_length() * (i + 9) for i, x in enumerate(("lengths", "change", "free", "count", "ws"))}
    expect(U, exq.exq_pages_trim, *pages_args(False, **big, **far))
    assert exq.exq_pages_workspace_bytes(0) == 0 and exq.exq_pages_workspace_bytes(5) == 48


def test_reference_trim_undoes_extend():
    rng = np.random.default_rng(3)
    pool = ref.Pool(100, 16, 6, 20)
    for _ in range(4):
        pool.extend(rng.integers(0, 60, 6), 1000)
    table, lengths, free = pool.table.copy(), pool.lengths.copy(), list(pool.free)
    pool.extend(rng.integers(0, 40, 6), 1000)
    pool.trim(lengths)
    assert pool.free == free and np.array_equal(pool.lengths, lengths) and np.array_equal(pool.table, table)
    taken = [p for s in range(6) for p in pool.table[s][:ref.pages_of(lengths[s], 16)]]
    assert sorted(taken + free) == list(range(100))


# ------------------------------------------------------------------ rotate

def rotate_args(**kw):
    a = dict(q=at(0), qs=(512, 64), qo=at(1), qos=(512, 64), heads=8, k=at(2), ks=(128, 64), ko=at(3), kos=(128, 64), kheads=2,
             rows=3, dim=64, part=64, inter=False, rates=at(4), factor=1.0, pos=at(5))
    a.update(kw)
    return [a[x] for x in ("q", "qs", "qo", "qos", "heads", "k", "ks", "ko", "kos", "kheads", "rows", "dim", "part", "inter",
                           "rates", "factor", "pos")] + [0]


BAD_ROTATE = [dict(q=0), dict(q=at(0) + 8), dict(qo=0), dict(qs=(508, 64)), dict(qos=(512, -8)), dict(heads=-1),
              dict(heads=0, kheads=0), dict(heads=65536), dict(k=0), dict(ko=at(3) + 2), dict(kos=(0, 64)), dict(qos=(512, 32)),
              dict(rows=-1), dict(dim=60), dict(dim=0), dict(part=0), dict(part=3), dict(part=66), dict(rates=0),
              dict(rates=at(4) + 4), dict(pos=0), dict(pos=at(5) + 2), dict(factor=float("nan")), dict(factor=float("inf")),
              dict(qo=at(0) + 16), dict(qo=at(0), qos=(1024, 64)), dict(qo=at(3)), dict(qo=at(2)), dict(ko=at(0)), dict(rates=at(1)),
              dict(pos=at(3) + 8), dict(qo=at(0) - 1024)]


@pytest.mark.parametrize("bad", BAD_ROTATE, ids=str)
def test_rotate_rejects(bad):
    expect(I, exq.exq_rotate, *rotate_args(**bad))


def test_rotate_of_no_rows_and_of_too_many():
    exq.exq_rotate(*rotate_args(rows=0))
    exq.exq_rotate(*rotate_args(rows=0, q=0, qo=0, k=0, ko=0, rates=0, pos=0))
    step = 1 << 60
    far = dict(q=step, qo=2 * step, k=3 * step, ko=4 * step, rates=5 * step, pos=5 * step + 8192, dim=1024, part=512, rows=1 << 27,
               heads=1, kheads=1, qs=(1024, 1024), qos=(1024, 1024), ks=(1024, 1024), kos=(1024, 1024))
    expect(U, exq.exq_rotate, *rotate_args(**far))


def test_rates():
    rates, factor = exq.rotary_rates(8)
    assert factor == 1.0 and rates == [10000.0 ** (-i / 4) for i in range(4)]
    assert exq.rotary_rates(8, scaling={"kind": "linear", "factor": 4})[0] == [f / 4 for f in rates]
    based = exq.rotary_rates(8, scaling={"kind": "base", "factor": 8})[0]
    assert based[0] == 1.0 and math.isclose(based[-1], rates[-1] / 8, rel_tol=1e-14)
    parts, factor = exq.rotary_rates(64, scaling={"kind": "parts", "factor": 16, "context": 4096})
    plain = exq.rotary_rates(64)[0]
    assert math.isclose(factor, 0.1 * math.log(16) + 1)
    for f, g in zip(plain, parts):
        turns = 4096 * f / (2 * math.pi)
        want = f if turns > 32 else f / 16 if turns < 1 else f / 16 + (turns - 1) / 31 * (f - f / 16)
        assert math.isclose(g, want, rel_tol=1e-12)
    assert exq.rotary_rates(64, scaling={"kind": "parts", "factor": 8, "context": 8192, "low": 1, "high": 4, "attention": 1})[1] == 1.0
    for bad in (dict(kind="other"), dict(kind="linear", factor=0), dict(kind="parts", factor=2), dict(factor=2),
                dict(kind="linear", factor=2, context=3), dict(kind="parts", factor=2, context=9, low=3, high=3)):
        expect(I, exq.rotary_rates, 64, scaling=bad)
    for bad in (0, 7, -2):
        expect(I, exq.rotary_rates, bad)


# ---------------------------------------------------------------- adapters

@pytest.fixture()
def adapters():
    h = exq.exq_adapters_create(6, 256, 512, 16, at(0), at(1), at(2), at(3))
    yield h
    exq.exq_adapters_destroy(h)


@pytest.mark.parametrize("status,args", [
    (I, (0, 256, 512, 16, at(0), at(1))), (I, (6, 252, 512, 16, at(0), at(1))), (I, (6, 256, 4, 16, at(0), at(1))),
    (I, (6, 256, 512, 12, at(0), at(1))), (I, (6, 256, 512, 0, at(0), at(1))), (I, (6, 256, 512, 16, 0, at(1))),
    (I, (6, 256, 512, 16, at(0), at(1) + 8)), (I, (6, 256, 512, 16, at(0), at(1), at(2) + 2)),
    (I, (6, 256, 512, 16, at(0), at(1), None, at(2) + 1)), (U, (8193, 256, 512, 16, at(0), at(1))),
    (U, (6, 256, 512, 264, at(0), at(1))), (U, (6, (1 << 20) + 8, 512, 16, at(0), at(1)))], ids=str)
def test_adapters_reject(status, args):
    expect(status, exq.exq_adapters_create, *args)


def lora_args(h, **kw):
    a = dict(x=at(4), xs=256, rows=40, ids=at(5), y=at(6), ys=512, out=at(7), os=512, ws=at(8), wsb=1 << 20)
    a.update(kw)
    return [h] + [a[x] for x in ("x", "xs", "rows", "ids", "y", "ys", "out", "os", "ws", "wsb")] + [0]


BAD_LORA = [dict(x=0), dict(x=at(4) + 4), dict(xs=252), dict(xs=-256), dict(rows=-1), dict(ids=0), dict(ids=at(5) + 2), dict(y=0),
            dict(ys=260), dict(out=0), dict(os=504), dict(os=0), dict(out=at(4)), dict(out=at(6) + 1024), dict(out=at(6), os=1024),
            dict(ws=0), dict(ws=at(8) + 8), dict(wsb=64), dict(ids=at(7)), dict(out=at(0)), dict(out=at(1)), dict(out=at(2)),
            dict(out=at(3)), dict(ws=at(4)), dict(ws=at(6)), dict(ws=at(7)), dict(ws=at(0)), dict(ids=at(8) + 16)]


@pytest.mark.parametrize("bad", BAD_LORA, ids=str)
def test_lora_rejects(adapters, bad):
    expect(I, exq.exq_lora_add, *lora_args(adapters, **bad))


def test_lora_without_rows_or_adapters(adapters):
    exq.exq_lora_add(*lora_args(adapters, rows=0))
    exq.exq_lora_add(*lora_args(adapters, rows=0, x=0, ids=0, y=0, out=0, ws=0, wsb=0))
    expect(I, exq.exq_lora_add, *lora_args(None))
    assert exq.exq_lora_workspace_bytes(None, 3) == exq.exq_lora_workspace_bytes(adapters, 0) == 0
    assert exq.exq_lora_workspace_bytes(adapters, -1) == 0
    assert exq.exq_lora_workspace_bytes(adapters, 1) == exq.exq_lora_workspace_bytes(adapters, 16) == 0   # one launch, nothing between
    sizes = [exq.exq_lora_workspace_bytes(adapters, r) for r in (17, 64, 65, 500, 600, 5000)]
    assert 0 < min(sizes) and max(sizes) < 1 << 24
    exq.exq_adapters_destroy(None)


# ------------------------------------------------------------------ sample

def sample_args(**kw):
    a = dict(logits=at(0), bits=16, rows=4, vocab=1000, stride=1000, u=at(1), ts=None, t=1.0, ks=None, k=0, ps=None, p=1.0, ms=None,
             m=0.0, tokens=at(2), logs=at(3), ws=None, bytes=0)
    a.update(kw)
    return [a[x] for x in ("logits", "bits", "rows", "vocab", "stride", "u", "ts", "t", "ks", "k", "ps", "p", "ms", "m", "tokens",
                           "logs", "ws", "bytes")] + [0]


SPLIT = dict(rows=2, vocab=32000, stride=32000, ws=at(5), bytes=1 << 20)   # rows that a workspace shares out


NAN = float("nan")


@pytest.mark.parametrize("status,bad", [
    (I, dict(logits=0)), (I, dict(logits=at(0) + 1)), (I, dict(logits=at(0) + 2, bits=32)), (U, dict(bits=8)), (I, dict(rows=-1)),
    (I, dict(vocab=0)), (U, dict(vocab=(1 << 21) + 1)), (I, dict(stride=999)), (I, dict(stride=-1)), (I, dict(u=0)),
    (I, dict(u=at(1) + 2)), (I, dict(t=-1.0)), (I, dict(t=NAN)), (I, dict(p=NAN)), (I, dict(m=NAN)), (I, dict(ts=at(4) + 1)),
    (I, dict(ks=at(4) + 2)), (I, dict(tokens=0)), (I, dict(logs=at(3) + 2)), (I, dict(tokens=at(0) + 7996)), (I, dict(tokens=at(1))),
    (I, dict(logs=at(2) + 12)), (I, dict(ms=at(2) - 12)), (I, dict(ps=at(3))),
    (I, dict(SPLIT, ws=at(5) + 4)), (I, dict(SPLIT, bytes=1000)), (I, dict(SPLIT, ws=at(0) + 64)), (I, dict(SPLIT, ws=at(1))),
    (I, dict(SPLIT, ws=at(2) - 64)), (I, dict(SPLIT, ts=at(5) + 800))], ids=str)
def test_sample_rejects(status, bad):
    expect(status, exq.exq_sample, *sample_args(**bad))


def test_sample_of_no_rows():
    exq.exq_sample(*sample_args(rows=0))
    exq.exq_sample(*sample_args(rows=0, logits=0, u=0, tokens=0, logs=0))


def test_reference_draw():
    l = np.log([0.5, 0.2, 0.2, 0.1])
    for u, token in ((0.0, 0), (0.49, 0), (0.51, 1), (0.71, 2), (0.89, 2), (0.95, 3), (1.0, 3)):
        assert ref.sample_row(l, u)[0] == token
    assert ref.sample_row(l, 0.99, top_k=2)[0] == 1               # of equal ones the first
    assert ref.sample_row(l, 0.99, top_p=0.5)[0] == 0
    assert ref.sample_row(l, 0.99, top_p=0.51)[0] == 1
    assert ref.sample_row(l, 0.99, min_p=0.39)[0] == 2
    assert ref.sample_row(l, 0.99, temperature=0)[0] == 0
    assert ref.sample_row([-np.inf, np.nan], 0.5)[0] == -1
    token, log, _ = ref.sample_row([0, np.inf, -3, np.inf], 0.6)
    assert token == 3 and math.isclose(log, math.log(0.5))


# ----------------------------------------------------------------- tensors

def test_tensors_are_checked_before_the_library():
    torch = pytest.importorskip("torch")
    with pytest.raises(exq.ExqError):
        exq.sample(torch.zeros(2, 10), torch.zeros(2))
    with pytest.raises(exq.ExqError):
        exq.Adapters(torch.zeros(2, 8, 16, dtype=torch.float16), torch.zeros(2, 16, 8, dtype=torch.float16))
    with pytest.raises(exq.ExqError):
        exq.PagePool(0, 16, 4, 4, device="cpu")
    with pytest.raises(exq.ExqError):
        exq.Rotary(64, rates=[1.0] * 31, device="cpu")
    with pytest.raises(exq.ExqError):
        exq.Rotary(64, rates=[1.0] * 32, scaling={"kind": "linear", "factor": 2}, device="cpu")


def test_tensor_calls_refuse_before_the_library(adapters):
    """The checks of tensors (_exq_torch) with CPU tensors: every one is refused with the package's own error."""
    torch = pytest.importorskip("torch")
    calls = exq._tensor_calls()
    h = torch.zeros((3, 4, 64), dtype=torch.float16)
    n = torch.zeros(3, dtype=torch.int32)
    t = torch.zeros((3, 2), dtype=torch.int32)
    f = torch.zeros(32, dtype=torch.float64)
    for bad in ((n, 4, None, None, None), (None, 4, None, None, None), (n, -1, None, None, None), (n, 1 << 40, None, None, None)):
        expect(I, calls.extend, 0, 0, 16, t, n, n, n[:1], n[:1], n, *bad)
    for bad in (n, None, "n"):
        expect(I, calls.trim, 0, 0, 16, t, n, n, n[:1], n, bad)
    for bad in ((h, n, None, None, None), (None, n, None, None, None), (h[0], n, None, None, None), (h, None, h, None, None),
                (h, n, None, None, h), (h, n, h[0], None, None)):
        expect(I, calls.rotate, 0, 0, 64, 64, False, f, 1.0, *bad)
    x = torch.zeros((3, 256), dtype=torch.float16)
    for bad in ((x, n, x, None, None), (x[0], n, x, None, None), (None, n, x, None, None), (x, None, x, x, x)):
        expect(I, calls.lora_add, 0, 0, adapters, 256, 512, *bad)
    l, u = torch.zeros((3, 50)), torch.zeros(3)
    for bad in ((l, u), (None, u), (l.double(), u), (l[0], u), (l, 0.5)):
        expect(I, calls.sample, 0, 0, *bad, 1.0, 0, 1.0, 0.0, None, False, None)
    for wrong in (calls.extend, calls.trim, calls.rotate, calls.lora_add, calls.sample):
        with pytest.raises(TypeError):
            wrong(0, 0, n)
