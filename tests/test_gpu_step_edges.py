"""Borders of the calls around a decoding step that test_gpu_step.py leaves out: ties of a greedy draw in rows that begin
anywhere, objects dropped while another stream has their calls before it, adapters whose ranks differ by orders of magnitude,
angles up to 2^40, the largest list of pages.

The tolerances of adapters and angles are those that include/exq.h states."""
from decimal import Decimal, localcontext

import numpy as np
import pytest

from oracle import stepref as ref
from tests.gpu_helpers import note, to_dev as dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def exq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mixed_bitrate_quantized_amd as m
    return m


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def f32(x):
    return torch.tensor(np.asarray(x), dtype=torch.float32, device="cuda")


def host(x):
    return x.cpu().numpy()


# ------------------------------------------------------------------ sample

GREEDY = [dict(temperature=0.0), dict(top_k=1), dict(top_p=0.0), dict(top_p=-1.0), dict(min_p=2.0), dict(temperature=0.0, top_k=7)]


def tied_rows(rng, vocab, per, offset):
    """Rows of `vocab` logits whose largest value stands in several places, for rows that begin `offset` elements behind a border
    of 16 bytes (`per` elements)."""
    head = min(vocab, (per - offset) % per)
    rows = [np.zeros(vocab), np.full(vocab, -3.0), np.full(vocab, np.inf), rng.integers(0, 2, vocab) * 1.0,
            np.where(rng.random(vocab) < 0.5, -0.0, 0.0), np.where(rng.random(vocab) < 0.7, -np.inf, 5.0),
            np.where(rng.random(vocab) < 0.3, np.nan, rng.integers(-1, 1, vocab))]
    for t in range(head):     # a place before the border, and vectors of 16 bytes that the same thread may look at
        row = rng.standard_normal(vocab) - 10
        row[t] = 7.0
        for vector in (t, t + 1024, t + 2048):
            at = head + per * vector + int(rng.integers(0, per))
            if at < vocab:
                row[at] = 7.0
        rows.append(row)
        tail = row.copy()     # and the end of the row
        tail[:head] = -20
        tail[vocab - 1 - t] = 7.0
        rows.append(tail)
    return np.stack(rows)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("vocab", [1, 3, 17, 4097, 50257])
def test_greedy_draws_take_the_first_of_equal_logits(exq, vocab, wide):
    """The lowest index of the largest logit, wherever a row begins: at every offset from a border of 16 bytes."""
    rng = np.random.default_rng(vocab)
    kind, per = (np.float32, 4) if wide else (np.float16, 8)
    for offset in range(9):
        note("greedy %d offset %d" % (vocab, offset))
        rows = tied_rows(rng, vocab, per, offset % per).astype(kind)
        want = np.array([np.argmax(np.where(np.isnan(r), -np.inf, r)) for r in rows])
        want[[np.all(np.isnan(r) | (r == -np.inf)) for r in rows]] = -1
        pitch = (vocab + offset + per) // per * per          # so that all rows begin alike
        space = torch.full((len(rows), pitch), float("nan"), dtype=torch.float32 if wide else torch.float16, device="cuda")
        d = space[:, offset:offset + vocab]
        d.copy_(torch.from_numpy(rows))
        u = f32(rng.random(len(rows)))
        for settings in GREEDY:
            tokens, logs = exq.sample(d, u, return_logprobs=True, **settings)
            np.testing.assert_array_equal(host(tokens), want, "%d offset %d %s" % (vocab, offset, settings))
            assert np.all(host(logs)[want >= 0] == 0)


@pytest.mark.parametrize("wide", [False, True])
def test_greedy_rows_of_an_odd_vocabulary_and_settings_of_each(exq, wide):
    """Contiguous rows of an odd length each begin elsewhere."""
    rows, vocab = 16, 50257
    d = torch.zeros((rows, vocab), dtype=torch.float32 if wide else torch.float16, device="cuda")
    u = f32(np.linspace(0, 0.99, rows))
    for settings in GREEDY:
        assert torch.all(exq.sample(d, u, **settings) == 0), settings
    kinds = np.arange(rows) % 4
    each = dict(temperature=f32(np.where(kinds == 0, 0.0, 1.0)), top_k=i32(np.where(kinds == 1, 1, 0)),
                top_p=f32(np.where(kinds == 2, 0.0, 1.0)), min_p=f32(np.where(kinds == 3, 1.5, 0.0)))
    assert torch.all(exq.sample(d, u, **each) == 0)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("vocab,k", [(2400, 300), (8000, 899), (1334, 901), (5406, 2000), (20011, 1500), (40000, 4000), (70001, 4096)])
def test_a_top_k_that_ends_at_a_gap(exq, vocab, k, wide):
    """The first k logits far above the others, so that what is looked at more closely is exactly those k; at a high temperature
    the others would weigh as much."""
    rng = np.random.default_rng(vocab + k)
    rows = 24
    x = rng.uniform(-1, 1, (rows, vocab))
    for r, row in enumerate(x):
        # neighbours 16 bytes apart, where they fit so, or anywhere
        places = np.arange(k) * 8 if r % 2 and 8 * k <= vocab else rng.permutation(vocab)[:k]
        row[places] = 8 + rng.uniform(0, 1, k)
        if r % 3 == 2:
            row[rng.permutation(vocab)[:vocab // 5]] = -np.inf
    x = x.astype(np.float32 if wide else np.float16)
    u = rng.random(rows).astype(np.float32)
    note("top-k %d of %d at a gap" % (k, vocab))
    for settings in (dict(top_k=k), dict(top_k=k, min_p=1e-3), dict(top_k=k, top_p=0.999), dict(top_k=k, top_p=0.5)):
        got = host(exq.sample(dev(x), f32(u), temperature=10.0, **settings))
        one = {z: v if z == "top_k" else np.float32(v) for z, v in settings.items()}
        want = [ref.sample_row(l, v, np.float32(10.0), **one)[0] for l, v in zip(x, u)]
        np.testing.assert_array_equal(got, want, "%d of %d %s" % (k, vocab, settings))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("vocab", [351, 462, 1334, 5406])
def test_a_top_k_of_hundreds_in_short_rows(exq, vocab, wide):
    """Many rows of few logits: by chance the list ends at the k-th in some."""
    rng = np.random.default_rng(vocab)
    x = (3 * rng.standard_normal((140, vocab))).astype(np.float32 if wide else np.float16)
    u = rng.random(140).astype(np.float32)
    for k in (300, vocab // 2 + 100, vocab - 20):
        for t in (1.0, 10.0):
            got = host(exq.sample(dev(x), f32(u), temperature=t, top_k=k))
            np.testing.assert_array_equal(got, [ref.sample_row(l, v, np.float32(t), k)[0] for l, v in zip(x, u)], "%d of %d" % (k, vocab))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("vocab", [50, 3001, 40000])
def test_min_p_at_an_infinite_temperature(exq, vocab, wide):
    """Every logit weighs e^0 there: no min-p up to 1 drops any; a large finite one leaves the largest alone."""
    rng = np.random.default_rng(vocab)
    x = rng.standard_normal((6, vocab)).astype(np.float32 if wide else np.float16)
    x[1, ::3] = -np.inf
    x[2, 5:9] = np.inf
    u = rng.random(6).astype(np.float32)
    for min_p in (1.0, 0.5, 1e-30):
        for settings in (dict(), dict(top_k=40), dict(top_k=vocab // 2), dict(top_p=0.5)):
            for each in (False, True):
                t = f32([np.inf] * 6) if each else float("inf")
                m = f32([min_p] * 6) if each else min_p
                got = host(exq.sample(dev(x), f32(u), temperature=t, min_p=m, **settings))
                one = {z: v if z == "top_k" else np.float32(v) for z, v in settings.items()}
                want = [ref.sample_row(l, v, np.float32(np.inf), min_p=np.float32(min_p), **one)[0] for l, v in zip(x, u)]
                np.testing.assert_array_equal(got, want, "%d %g %s" % (vocab, min_p, settings))
    got = host(exq.sample(dev(x[3:]), f32(u[3:]), temperature=1e30, min_p=1.0))
    np.testing.assert_array_equal(got, [np.argmax(l) for l in x[3:]])


# ----------------------------------------------------------------- streams

@pytest.mark.parametrize("call", ["rotate", "add", "extend", "trim"])
def test_objects_dropped_after_a_call_on_another_stream_stay_until_it_is_through(exq, call):
    """What an object keeps for its calls (rates, adapters, a pool's arrays) is not given out again while a stream that a call
    named has that call still before it."""
    half = lambda *shape: torch.ones(shape, dtype=torch.float16, device="cuda")
    if call == "rotate":
        thing = exq.Rotary(65536)
        own = [thing.rates]
        q, p = half(3, 1, 65536), i32([1, 2, 3])
        run = lambda t: t.rotate(q, p, stream=side)
    elif call == "add":
        own = [half(7, 16, 4096), half(7, 4104, 16), torch.ones(7, device="cuda"), i32([16] * 7)]
        thing = exq.Adapters(*own)
        x, ids, y = half(40, 4096), i32(np.arange(40) % 7), half(40, 4104)
        run = lambda t: t.add(x, ids, y, stream=side)
    else:
        thing = exq.PagePool(70000, 16, 3000, 20)
        own = [thing.table, thing.lengths, thing.free, thing.free_count, thing.served, thing._workspace]
        change = i32([5] * 3000)
        run = lambda t: t.extend(change, 15000, stream=side) if call == "extend" else t.trim(change, stream=side)
    side = torch.cuda.Stream()
    run(thing)      # what the first call of a kind loads is loaded
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    note("objects on another stream: %s" % call)
    kept = run(thing)
    before = {x.data_ptr() for x in own}
    kinds = [(x.shape, x.dtype) for x in own]
    del thing, own
    after = [torch.empty(shape, dtype=dtype, device="cuda") for _ in range(20) for shape, dtype in kinds]
    waiting = not side.query()
    torch.cuda.synchronize()
    assert not (waiting and before & {x.data_ptr() for x in after})
    del kept


# ---------------------------------------------------------------- adapters

def check_lora(out, x, ids, y, a, b, scales, ranks, what):
    """Results that round past 65504 are infinite: 65536, the next step of fp16's grid, on both sides."""
    want, size = ref.lora(x, ids, y, a, b, scales, ranks)
    bound = 2.0 ** -11 * np.abs(want) + size * (a.shape[2] + a.shape[1] + 64) * 2.0 ** -23 + 2.0 ** -24
    got = host(out).astype(np.float64)
    got, want = np.where(np.isinf(got), np.copysign(65536.0, got), got), np.clip(want, -65536, 65536)
    e = np.abs(got - want) / bound
    assert e.max() <= 1, "%s: %.3g of the bound" % (what, e.max())


def uneven_stack(rng, count, K, N, rank):
    """Adapters whose ranks differ by up to 2^39: the largest inner products meet zeros of b in half of the columns, so that
    the small ones alone make the result there."""
    a = rng.uniform(0.5, 1, (count, rank, K)) * rng.choice([-1, 1], (count, rank, K))
    power = rng.integers(-22, 15, (count, rank, 1))
    power[:, 0], power[:, 1] = 15, -22
    a = (a * 2.0 ** power).astype(np.float16)
    b = rng.standard_normal((count, N, rank)).astype(np.float16)
    b[:, ::2, power[0, :, 0] > -12] = 0
    b[:, ::2] *= np.float16(2.0 ** 12)
    return a, b


@pytest.mark.parametrize("K,N,rank", [(8, 64, 8), (8, 520, 16), (256, 264, 16), (8192, 136, 16), (8, 264, 40), (520, 1032, 64), (72, 136, 128),
                                      (64, 72, 256)])
def test_lora_ranks_of_very_different_size(exq, K, N, rank):
    """What the largest inner product of a row leaves of the smallest, in one launch and in two, by every size of tile."""
    rng = np.random.default_rng(K + N + rank)
    a, b = uneven_stack(rng, 2, K, N, rank)
    if K == 8 and rank == 8:      # sums of one sign: by hand 3 * 2^-24 * 65504 * 8
        a[1], b[1] = 0, 0
        a[1, 0], a[1, 1], b[1, :, 1] = 32768, 3 * 2.0 ** -24, 65504
    adapters = exq.Adapters(dev(a), dev(b))
    for rows in (1, 2, 16, 17, 70, 600):
        note("lora of uneven ranks, %d rows" % rows)
        x = rng.standard_normal((rows, K)).astype(np.float16)
        x[0] = 1
        y = np.zeros((rows, N), dtype=np.float16)
        ids = rng.integers(0, 2, rows)
        ids[0] = 1
        check_lora(adapters.add(dev(x), i32(ids), dev(y)), x, ids, y, a, b, None, None, "%d rows" % rows)


@pytest.mark.parametrize("K,rank", [(256, 8), (256, 64)])
def test_a_row_of_uneven_products_leaves_the_others_alone(exq, K, rank):
    rng = np.random.default_rng(K + rank)
    a = (rng.standard_normal((1, rank, K)) * K ** -0.5).astype(np.float16)
    b = rng.standard_normal((1, 264, rank)).astype(np.float16)
    a[0, 1], a[0, 1, 0] = 0, 2.0 ** -24
    adapters = exq.Adapters(dev(a), dev(b))
    for rows in (5, 40, 600):
        x = rng.standard_normal((rows, K)).astype(np.float16)
        x[:, 0] = 0
        y = rng.standard_normal((rows, 264)).astype(np.float16)
        ids = i32([0] * rows)
        plain = host(adapters.add(dev(x), ids, dev(y)))
        x[3, 0] = 2.0 ** -3       # rank 1 of this row is 2^-27
        mixed = host(adapters.add(dev(x), ids, dev(y)))
        rest = np.arange(rows) != 3
        np.testing.assert_array_equal(mixed[rest], plain[rest])
        check_lora(adapters.add(dev(x), ids, dev(y)), x, [0] * rows, y, a, b, None, None, "%d rows" % rows)


@pytest.mark.parametrize("K,rank", [(4096, 16), (4096, 64)])
def test_lora_of_the_largest_scales(exq, K, rank):
    """Inner products of 2^44 by a scale of 2^100 and more: past fp16, but y where b is 0."""
    a = np.full((2, rank, K), 65504, dtype=np.float16)
    b = np.zeros((2, 264, rank), dtype=np.float16)
    b[:, 1::2] = np.float16(2.0 ** -24)
    adapters = exq.Adapters(dev(a), dev(b), f32([2.0 ** 100, -np.finfo(np.float32).max]))
    for rows in (1, 30, 600):
        x = np.full((rows, K), 65504, dtype=np.float16)
        y = np.random.default_rng(rows).standard_normal((rows, 264)).astype(np.float16)
        ids = np.arange(rows) % 2
        note("lora of the largest scales, %d rows" % rows)
        got = host(adapters.add(dev(x), i32(ids), dev(y)))
        np.testing.assert_array_equal(got[:, ::2], y[:, ::2])
        np.testing.assert_array_equal(got[:, 1::2], np.where(ids[:, None], -np.inf, np.inf) * np.ones((1, 132)))


# ------------------------------------------------------------------ rotate

TWO_PI = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")


def turned(x, positions, rates, interleaved):
    """x [rows][heads][2 * pairs] turned by the exact product of position and rate, and |u| + |v| of each channel's pair."""
    out, pair = np.zeros(x.shape), np.zeros(x.shape)
    half = len(rates)
    with localcontext() as context:
        context.prec = 120
        for r, p in enumerate(positions):
            for i, rate in enumerate(rates):
                t = float(Decimal(int(p)) * Decimal(float(rate)) % TWO_PI)
                a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
                u, v = x[r, :, a].astype(np.float64), x[r, :, b].astype(np.float64)
                out[r, :, a], out[r, :, b] = u * np.cos(t) - v * np.sin(t), u * np.sin(t) + v * np.cos(t)
                pair[r, :, a] = pair[r, :, b] = np.abs(u) + np.abs(v)
    return out, pair


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim", [32, 24])
def test_rotate_far_angles(exq, dim, interleaved):
    """Angles up to 2^40: those of the stated accuracy, 2^-20 of a pair beside the result's rounding.  fp16 results round at
    2^-11 of themselves, so pairs (1, 0) at the angles where a channel is small show the angle's error."""
    rng = np.random.default_rng(dim)
    rows = 60
    positions = np.concatenate([[2 ** 31 - 1, 2 ** 31 - 2, 2 ** 30 + 1, 1 << 30], rng.integers(1 << 29, 2 ** 31, rows - 4)])
    x = np.zeros((rows, 2, dim), dtype=np.float16)
    x[:, 0, :] = 1.0
    x[:, 1, 0::2] = 1.0
    for top in (2, 2 ** 3, 2 ** 6, 2 ** 9):       # angles up to 2^40
        rates = rng.uniform(0.5, 1, dim // 2) * top
        note("rotate by up to 2^%d" % (30 + np.log2(top)))
        # of many pairs, those that a turn takes within 2^-9 of an axis, where fp16 has 2^-20 and less
        rates[: dim // 4] = near_axis(positions[0], rates[: dim // 4])
        rotary = exq.Rotary(dim, interleaved=interleaved, rates=rates)
        got = host(rotary.rotate(dev(x), i32(positions))).astype(np.float64)
        want, pair = turned(x, positions, host(rotary.rates), interleaved)
        bound = 2.0 ** -11 * np.abs(want) + 2.0 ** -20 * pair + 2.0 ** -24
        assert np.all(np.abs(got - want) <= bound), "up to 2^%d: %.3g of the bound" % (30 + np.log2(top), np.max(np.abs(got - want) / bound))


def near_axis(position, rates):
    """The rates, each moved so that `position` times it lies within 2^-14 of a multiple of half a turn, or as near as doubles get."""
    out = []
    with localcontext() as context:
        context.prec = 120
        for rate in rates:
            turns = (Decimal(int(position)) * Decimal(float(rate)) / (TWO_PI / 2)).to_integral_value()
            out.append(float(turns * (TWO_PI / 2) / int(position)))
    return np.array(out)


# ------------------------------------------------------------------- pages

def test_a_row_too_long_for_the_table_is_not_served_from_the_largest_list(exq):
    """2^31 - 1 free pages: what does not fit a row of the table has to count as more."""
    note("a list of 2^31 - 1 pages")
    n = 2 ** 31 - 1
    pool = exq.PagePool(n, 16, 3, 2)
    for counts, served, rows in (([33, 1, 1], 0, 0), ([32, 2 ** 31 - 1, 1], 1, 32), ([1, 1, 1], 0, 0), ([0, 32, 33], 2, 32)):
        seqs, positions, offsets = pool.extend(i32(counts), 40)
        assert int(pool.served) == served and int(offsets[-1]) == rows, counts
        assert int((seqs >= 0).sum()) == rows
    np.testing.assert_array_equal(host(pool.table), [[0, 1], [2, 3], [-1, -1]])
    np.testing.assert_array_equal(host(pool.lengths), [32, 32, 0])
    assert int(pool.free_count) == n - 4 and int(pool.free[n - 5]) == 4
    pool.trim(i32([0, 0, 0]))
    assert int(pool.free_count) == n and host(pool.free[-4:]).tolist() == [3, 2, 1, 0]
    del pool
    torch.cuda.empty_cache()
