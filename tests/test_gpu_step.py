"""Pages, rotary positions, adapters and the draw on the GPU against references in 64 bits (oracle/stepref.py), each at the
sizes, strides and values where it can go wrong, and a decoding step made of all of them.

Tolerances are those that include/exq.h states: one rounding of the result to fp16 (2^-11 of it), 32-bit sums of the number
of terms, and for logprobs one rounding to fp32 of a value known to 2^-30.  Whole numbers are equal."""
import io

import numpy as np
import pytest

from oracle import cacheref, stepref as ref
from tests.gpu_helpers import note, to_dev

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


# ------------------------------------------------------------------- pages

def pool_pair(exq, n_pages, page, sequences, width):
    return exq.PagePool(n_pages, page, sequences, width), ref.Pool(n_pages, page, sequences, width)


def same_pool(pool, want, what=""):
    np.testing.assert_array_equal(host(pool.table), want.table, what)
    np.testing.assert_array_equal(host(pool.lengths), want.lengths, what)
    n = int(pool.free_count)
    assert n == len(want.free), what
    np.testing.assert_array_equal(host(pool.free)[:n], np.array(want.free, dtype=np.int32), what)


def extend_both(pool, want, counts, rows, what=""):
    seqs, positions, offsets = pool.extend(i32(counts), rows)
    a, b, c, served = want.extend(counts, rows)
    np.testing.assert_array_equal(host(seqs), a, what)
    np.testing.assert_array_equal(host(positions), b, what)
    np.testing.assert_array_equal(host(offsets), c, what)
    assert int(pool.served) == served, what
    same_pool(pool, want, what)


# one workgroup does all of a call, a second launch the rest of it, sequences in several passes
@pytest.mark.parametrize("sequences,page,width,most", [(1, 16, 8, 40), (3, 1, 50, 20), (64, 48, 9, 100), (255, 16, 6, 30),
                                                       (257, 16, 20, 90), (1100, 32, 4, 9), (1100, 16, 20, 40), (5000, 16, 3, 12), (9000, 64, 2, 3)])
def test_pages_of_a_changing_batch(exq, sequences, page, width, most):
    note("pages: %d sequences" % sequences)
    rng = np.random.default_rng(sequences)
    pool, want = pool_pair(exq, sequences * width + 5, page, sequences, width)
    for step in range(6):
        room = width * page - want.lengths
        counts = np.minimum(rng.integers(-2, most, sequences), room)
        total = int(np.maximum(counts, 0).sum())
        extend_both(pool, want, counts, total + (step % 2) * 7, "step %d" % step)
        keep = np.where(rng.random(sequences) < 0.5, rng.integers(-3, width * page + 3, sequences), rng.integers(0, 2, sequences) * 100000)
        pool.trim(i32(keep))
        want.trim(keep)
        same_pool(pool, want, "trim %d" % step)


@pytest.mark.parametrize("sequences", [5, 300, 4500])
@pytest.mark.parametrize("short", ["pages", "rows", "width"])
def test_what_does_not_fit_gets_nothing(exq, sequences, short):
    """The first sequence that does not fit and all after it keep their lengths; a later call serves them."""
    rng = np.random.default_rng(sequences)
    counts = rng.integers(0, 40, sequences)
    counts[3 * sequences // 5] = 40
    need = [ref.pages_of(c, 16) for c in counts]
    upto = 3 * sequences // 5
    pages = sum(need[:upto]) + 1 if short == "pages" else sum(need) + 9
    rows = int(sum(counts[:upto])) + 5 if short == "rows" else int(sum(counts)) + 5
    width = 2 if short == "width" else 3
    pool, want = pool_pair(exq, pages, 16, sequences, width)
    extend_both(pool, want, counts, rows)
    left = np.where(np.arange(sequences) < int(pool.served), 0, np.minimum(counts, 16))
    extend_both(pool, want, left, rows)
    pool.trim(torch.zeros(sequences, dtype=torch.int32, device="cuda"))
    want.trim([0] * sequences)
    same_pool(pool, want)


def test_pages_of_rows_not_in_use_and_wild_numbers(exq):
    pool, want = pool_pair(exq, 50, 16, 6, 8)
    want.lengths[:] = [-1, 20, 0, -5, 128, 7]
    pool.lengths.copy_(i32(want.lengths))
    for counts in ([3, 4, -7, 9, 0, 1], [2 ** 31 - 1, 1, 1, 1, 1, 1], [-2 ** 31, 1, 2 ** 31 - 1, 1, 1, 1], [0, 0, 0, 0, 1, 1]):
        extend_both(pool, want, counts, 20, str(counts))
    for keep in ([-1, -1, -1, -1, -1, -1], [0, 2 ** 31 - 1, 0, 0, 128, -2 ** 31], [0, 1, 0, 0, 17, 0]):
        pool.trim(i32(keep))
        want.trim(keep)
        same_pool(pool, want, str(keep))
    # a free list's count outside its bounds is taken as the nearest
    pool.free_count.fill_(-3)
    assert int(pool.extend(i32([0, 16, 0, 0, 0, 0]), 16)[2][-1]) == 0 and int(pool.served) == 1 and int(pool.free_count) == 0


def test_pages_into_given_tensors_and_rows_none(exq):
    pool, want = pool_pair(exq, 40, 16, 3, 9)
    out = [torch.full((n,), 77, dtype=torch.int32, device="cuda") for n in (12, 12, 4)]
    assert pool.extend(i32([5, 0, 6]), 12, *out) == tuple(out)
    a, b, c, _ = want.extend([5, 0, 6], 12)
    for x, y in zip(out, (a, b, c)):
        np.testing.assert_array_equal(host(x), y)
    extend_both(pool, want, [0, 0, 0], 0)
    extend_both(pool, want, [1, 0, 0], 0)     # no row fits
    with pytest.raises(exq.ExqError):
        pool.extend(i32([1, 1]), 4)
    with pytest.raises(exq.ExqError):
        pool.extend(i32([1, 1, 1]).float(), 4)
    with pytest.raises(exq.ExqError):
        pool.trim(i32([1, 1, 1, 1]))


# ------------------------------------------------------------------ rotate

def check_rotate(got, x, positions, rotary, what="", before=None):
    want = ref.rotate(x, positions, host(rotary.rates), rotary.factor, rotary.rotary_dim, rotary.interleaved)
    got, x = host(got).astype(np.float64), x.astype(np.float64)
    if before is not None:
        skipped = np.asarray(positions) < 0
        np.testing.assert_array_equal(got[skipped], np.broadcast_to(before, got.shape)[skipped], what)
        got, want, x = got[~skipped], want[~skipped], x[~skipped]
    part, half = rotary.rotary_dim, rotary.rotary_dim // 2
    pair = np.zeros_like(x)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if rotary.interleaved else (i, i + half)
        pair[..., a] = pair[..., b] = np.abs(x[..., a]) + np.abs(x[..., b])
    bound = 2.0 ** -11 * np.abs(want) + 2.0 ** -20 * abs(rotary.factor) * pair + 2.0 ** -24
    assert np.all(np.abs(got - want) <= bound), "%s: %.3f of the bound" % (what, np.max(np.abs(got - want) / bound))
    np.testing.assert_array_equal(got[..., part:], x[..., part:], what)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,part", [(64, 64), (128, 128), (256, 64), (96, 48), (80, 80), (80, 20), (72, 64), (40, 16), (8, 2), (24, 6)])
def test_rotate_matches_reference(exq, dim, part, interleaved):
    note("rotate %d of %d" % (part, dim))
    rng = np.random.default_rng(dim * 100 + part)
    scaling = {"kind": "parts", "factor": 8.0, "context": 4096}
    rotary = exq.Rotary(dim, part, interleaved=interleaved, scaling=scaling)
    for rows, heads, kv in ((1, 1, 1), (1, 40, 8), (7, 6, 2), (131, 9, 3)):
        q, k = (rng.standard_normal((rows, h, dim)).astype(np.float16) for h in (heads, kv))
        positions = rng.integers(0, 1 << 20, rows)
        positions[0] = 2 ** 31 - 1 if rows > 1 else 0
        dq, dk = to_dev(q), to_dev(k)
        q_out, k_out = rotary.rotate(dq, i32(positions), k=dk)
        check_rotate(q_out, q, positions, rotary, "q %d x %d" % (rows, heads))
        check_rotate(k_out, k, positions, rotary, "k %d x %d" % (rows, kv))
        alone = rotary.rotate(dq, i32(positions))
        assert torch.equal(alone, q_out)
        assert rotary.rotate(dq, i32(positions), k=dk, q_out=dq, k_out=dk)[0] is dq     # in place
        assert torch.equal(dq, q_out) and torch.equal(dk, k_out)


def test_rotate_strided_slices_padding_rows_and_infinities(exq):
    rng = np.random.default_rng(5)
    rows, dim = 19, 128
    rotary = exq.Rotary(dim, 96, interleaved=True)
    qkv = rng.standard_normal((rows, 24, dim)).astype(np.float16)
    qkv[2, 3, 5], qkv[4, 17, 100] = np.inf, np.nan
    positions = rng.integers(-2, 3, rows)
    positions[4], positions[2] = 1, 0
    d = to_dev(qkv)
    q_out = torch.full((rows, 20, dim), 7.0, dtype=torch.float16, device="cuda")[:, :16]
    k_out = torch.full((rows, 4, dim), 7.0, dtype=torch.float16, device="cuda")
    rotary.rotate(d[:, :16], i32(positions), k=d[:, 16:20], q_out=q_out, k_out=k_out)
    want = ref.rotate(qkv, positions, host(rotary.rates), 1.0, 96, True)
    assert np.isnan(host(k_out)[4, 1, 100]) and not np.isfinite(host(q_out)[2, 3, 4:6]).any()   # inf sin 0: NaN
    clean = qkv.copy()
    clean[2, 3, 4:6] = clean[4, 17, 100] = 0
    q, k = q_out.clone(), k_out.clone()
    q[2, 3, 4:6] = 0
    k[4, 1, 100] = 0
    check_rotate(q, clean[:, :16], positions, rotary, "q", before=7.0)
    check_rotate(k, clean[:, 16:20], positions, rotary, "k", before=7.0)
    # in place on slices of the projections' output: nothing else changes
    before = d.clone()
    rotary.rotate(d[:, :16], i32(positions), k=d[:, 16:20], q_out=d[:, :16], k_out=d[:, 16:20])
    live = torch.tensor(positions >= 0, device="cuda")
    assert torch.equal(d[live, :16].view(torch.int16), q_out[live].view(torch.int16))
    assert torch.equal(d[~live].view(torch.int16), before[~live].view(torch.int16))
    assert torch.equal(d[:, 20:], before[:, 20:])
    assert want.shape == qkv.shape


def test_rotate_refuses_tensors(exq):
    rotary = exq.Rotary(64)
    x = torch.zeros((3, 2, 64), dtype=torch.float16, device="cuda")
    p = i32([0, 1, 2])
    for bad in (dict(q=x.float()), dict(q=x[:, :, :32]), dict(q=x[0]), dict(q=x.transpose(1, 2)), dict(positions=p.long()),
                dict(positions=p[:2]), dict(k=x[:2]), dict(k=x, k_out=x[:, :1]), dict(q_out=x.cpu()), dict(k_out=x), dict(k=x, k_out=x)):
        a = dict(q=x, positions=p)
        a.update(bad)
        if bad.keys() == {"k", "k_out"} and bad["k_out"] is x:
            a["q_out"] = x      # both outputs over each other
        with pytest.raises(exq.ExqError):
            rotary.rotate(**a)
    assert rotary.rotate(x[:0], p[:0]).shape == (0, 2, 64)


# ---------------------------------------------------------------- adapters

def check_lora(out, x, ids, y, a, b, scales, ranks, what=""):
    want, size = ref.lora(x, ids, y, a, b, scales, ranks)
    got = host(out).astype(np.float64)
    bad = np.isnan(want)
    assert np.all(np.isnan(got[bad])), what
    bound = 2.0 ** -11 * np.abs(want) + size * (a.shape[2] + a.shape[1] + 64) * 2.0 ** -23 + 2.0 ** -24
    e = np.abs(got - want)[~bad] / bound[~bad]
    assert e.size == 0 or e.max() <= 1, "%s: %.3f of the bound" % (what, e.max())
    none = np.asarray(ids) < 0
    np.testing.assert_array_equal(got[none], np.asarray(y, dtype=np.float64)[none], what)


def stack(rng, count, K, N, rank):
    a = (rng.standard_normal((count, rank, K)) * K ** -0.5).astype(np.float16)
    b = (rng.standard_normal((count, N, rank)) * rank ** -0.5).astype(np.float16)
    return a, b, rng.uniform(-2, 2, count).astype(np.float32), rng.integers(0, rank + 1, count).astype(np.int32)


@pytest.mark.parametrize("K,N,rank,count", [(256, 512, 16, 3), (8, 8, 8, 1), (1000, 1016, 24, 7), (4096, 264, 64, 40), (520, 2056, 128, 2),
                                            (136, 72, 200, 3), (2048, 1024, 256, 2), (8192, 264, 16, 5), (4096, 4104, 8, 3),
                                            (4104, 520, 16, 2), (1000, 1016, 16, 7)])
def test_lora_matches_reference(exq, K, N, rank, count):
    note("lora K=%d N=%d rank=%d" % (K, N, rank))
    rng = np.random.default_rng(K + N + rank)
    a, b, scales, ranks = stack(rng, count, K, N, rank)
    ranks[0] = rank
    # behind an adapter's own rank anything may lie
    for i, r in enumerate(ranks):
        a[i, r:] = np.nan
        b[i, :, r:] = np.inf
    adapters = exq.Adapters(to_dev(a), to_dev(b), f32(scales), i32(ranks))
    for rows in (1, 2, 15, 16, 17, 63, 130, 600):
        x = rng.standard_normal((rows, K)).astype(np.float16)
        y = rng.standard_normal((rows, N)).astype(np.float16)
        ids = rng.integers(-1, count, rows)
        ids[-1] = 0
        if rows == 130:
            ids[:] = np.sort(ids)
        if rows > 16:
            ids[3], ids[11] = count, 2 ** 31 - 1
        dy = to_dev(y)
        out = adapters.add(to_dev(x), i32(ids), dy)
        check_lora(out, x, ids, y, a, b, scales, ranks, "rows %d" % rows)
        again = adapters.add(to_dev(x), i32(ids), dy, out=dy)      # in place
        assert again is dy and torch.equal(dy.view(torch.int16), out.view(torch.int16))


def test_lora_of_few_distinct_rows_and_one_adapter(exq):
    rng = np.random.default_rng(8)
    a, b, _, _ = stack(rng, 1, 640, 1280, 32)
    adapters = exq.Adapters(to_dev(a), to_dev(b))
    for rows, ids in ((5, [-1] * 5), (700, [-1] * 700), (700, [0] * 700), (700, [0, -1] * 350), (1, [5])):
        x, y = (rng.standard_normal((rows, n)).astype(np.float16) for n in (640, 1280))
        dy = to_dev(y)
        check_lora(adapters.add(to_dev(x), i32(ids), dy), x, ids, y, a, b, None, None, "%d rows" % rows)
        adapters.add(to_dev(x), i32(ids), dy, out=dy)
        check_lora(dy, x, ids, y, a, b, None, None, "%d rows in place" % rows)


@pytest.mark.parametrize("rows,count", [(64, 64), (65, 64), (511, 3), (512, 3), (9000, 5000), (20000, 2)])
def test_lora_of_many_rows_and_adapters(exq, rows, count):
    """On both sides of where rows are grouped and tiled otherwise; more rows than a thread keeps, more adapters than threads."""
    rng = np.random.default_rng(rows + count)
    K, N, rank = 72, 88, 8
    a, b, scales, ranks = stack(rng, count, K, N, rank)
    adapters = exq.Adapters(to_dev(a), to_dev(b), f32(scales), i32(ranks))
    x, y = (rng.standard_normal((rows, n)).astype(np.float16) for n in (K, N))
    for ids in (rng.permutation(np.arange(rows) % (count + 1) - 1), rng.integers(-1, count + 1, rows)):
        out = adapters.add(to_dev(x), i32(ids), to_dev(y))
        pick = np.unique(np.concatenate([np.arange(min(rows, 300)), rng.integers(0, rows, 700), np.arange(rows - 40, rows)]))
        check_lora(out[torch.tensor(pick, device="cuda")], x[pick], ids[pick], y[pick], a, b, scales, ranks, "%d rows of %d" % (rows, count))


def test_lora_large_small_and_non_finite_values(exq):
    """Inner products far beyond fp16, and far below; a row with an infinity leaves its neighbours alone."""
    rng = np.random.default_rng(9)
    a, b, _, _ = stack(rng, 2, 512, 256, 16)
    a[0] = (a[0].astype(np.float32) * 2e4).astype(np.float16)
    b[0] = (b[0].astype(np.float32) * 1e-4).astype(np.float16)
    a[1] = (a[1].astype(np.float32) * 1e-4).astype(np.float16)
    adapters = exq.Adapters(to_dev(a), to_dev(b), f32([1e-2, 1e6]))
    x = rng.standard_normal((20, 512)).astype(np.float16)
    x[:10] *= np.float16(100)
    x[12] = 0
    y = rng.standard_normal((20, 256)).astype(np.float16)
    ids = np.arange(20) // 10
    check_lora(adapters.add(to_dev(x), i32(ids), to_dev(y)), x, ids, y, a, b, np.array([1e-2, 1e6], dtype=np.float32), None)
    clean = host(adapters.add(to_dev(x), i32(ids), to_dev(y)))
    x[4, 100], x[15, 3], y[7, 9] = np.inf, np.nan, np.nan
    got = host(adapters.add(to_dev(x), i32(ids), to_dev(y)))
    rest = [r for r in range(20) if r not in (4, 7, 15)]
    np.testing.assert_array_equal(got[rest], clean[rest])
    assert not np.isfinite(got[[4, 15]].astype(np.float32)).any() and np.isnan(got[7, 9])


def test_lora_strides_and_refusals(exq):
    rng = np.random.default_rng(10)
    a, b, scales, ranks = stack(rng, 4, 128, 192, 8)
    adapters = exq.Adapters(to_dev(a), to_dev(b), f32(scales), i32(ranks))
    x, y = rng.standard_normal((33, 128)).astype(np.float16), rng.standard_normal((33, 192)).astype(np.float16)
    ids = rng.integers(0, 4, 33)
    dx, dy = torch.zeros((33, 136), dtype=torch.float16, device="cuda")[:, 8:], torch.zeros((33, 400), dtype=torch.float16, device="cuda")
    dx.copy_(to_dev(x))
    dy.fill_(9.0)
    dy[:, 200:392] = to_dev(y)
    adapters.add(dx, i32(ids), dy[:, 200:392], out=dy[:, :192])
    check_lora(dy[:, :192], x, ids, y, a, b, scales, ranks)
    assert torch.all(dy[:, 192:200] == 9) and torch.all(dy[:, 392:] == 9)
    wide = to_dev(x)[5:6].expand(33, 128)     # one row for all
    check_lora(adapters.add(wide, i32(ids), to_dev(y)), np.repeat(x[5:6], 33, 0), ids, y, a, b, scales, ranks)
    ok = dict(x=to_dev(x), ids=i32(ids), y=to_dev(y))
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    for bad in (dict(x=ok["x"].float()), dict(x=ok["x"][:, :64]), dict(x=ok["x"][:5]), dict(ids=ok["ids"].long()), dict(ids=ok["ids"][1:]),
                dict(y=ok["x"]), dict(out=ok["x"]), dict(out=ok["y"][:5]), dict(workspace=small), dict(y=ok["y"].cpu()),
                dict(out=ok["y"][:, :1].expand(33, 192))):
        with pytest.raises(exq.ExqError):
            adapters.add(**{**ok, **bad})
    assert adapters.add(ok["x"][:0], ok["ids"][:0], ok["y"][:0]).shape == (0, 192)
    for wrong in (dict(a=to_dev(a).float()), dict(b=to_dev(b)[:3]), dict(scales=f32(scales[:3])), dict(ranks=i32(ranks).long()),
                  dict(b=to_dev(b).transpose(1, 2)), dict(a=to_dev(a)[0])):
        with pytest.raises(exq.ExqError):
            exq.Adapters(**{**dict(a=to_dev(a), b=to_dev(b)), **wrong})


# ------------------------------------------------------------------ sample

def check_sample(exq, logits, u, what="", wide=False, **settings):
    logits = np.asarray(logits, dtype=np.float32 if wide else np.float16)
    dev = {k: (i32(v) if k == "top_k" else f32(v)) if isinstance(v, np.ndarray) else v for k, v in settings.items()}
    tokens, logs = exq.sample(to_dev(logits), f32(u), return_logprobs=True, **dev)
    tokens, logs = host(tokens), host(logs).astype(np.float64)
    for r, row in enumerate(logits):
        one = {k: v[r] if isinstance(v, np.ndarray) else np.float32(v) if k != "top_k" else v for k, v in settings.items()}
        token, log, _ = ref.sample_row(row, np.float32(u[r]), **one)
        assert tokens[r] == token, "%s row %d: %d, %d wanted" % (what, r, tokens[r], token)
        assert np.isnan(log) == np.isnan(logs[r]) and (np.isnan(log) or abs(logs[r] - log) <= 2.0 ** -23 * abs(log) + 2.0 ** -30), what
    return tokens


def likely(rng, rows, vocab, slope=1.2):
    x = -slope * np.log1p(np.arange(vocab)) + 12 + 0.8 * rng.standard_normal((rows, vocab))
    return rng.permuted(x, axis=1)


SETTINGS = [dict(), dict(top_k=1), dict(top_k=40), dict(top_p=0.9), dict(min_p=0.05), dict(temperature=0.0), dict(top_k=50, top_p=0.8),
            dict(temperature=0.7, top_k=300, top_p=0.95, min_p=0.01), dict(top_k=1500), dict(temperature=2.0, top_p=0.99),
            dict(top_k=10 ** 6, top_p=0.0), dict(min_p=1.0), dict(min_p=1.5), dict(top_p=1e-9), dict(temperature=1e-3)]


@pytest.mark.parametrize("settings", SETTINGS, ids=str)
@pytest.mark.parametrize("wide", [False, True])
def test_sample_matches_reference(exq, settings, wide):
    note("sample %s" % settings)
    rng = np.random.default_rng(11)
    for vocab in (1, 2, 7, 64, 1000, 5003, 32001, 131072):
        rows = 5
        check_sample(exq, likely(rng, rows, vocab), rng.random(rows), "vocab %d" % vocab, wide, **settings)


@pytest.mark.parametrize("wide", [False, True])
def test_sample_flat_rows_and_ties(exq, wide):
    """Equal logits, where the index alone decides and every border is exact, and rows so flat that the nucleus is most of them."""
    rng = np.random.default_rng(12)
    for vocab in (3, 1024, 4097, 40000):
        same = np.zeros((4, vocab))
        u = np.array([0.0, 0.25, 0.5, 0.999])
        for settings in (dict(), dict(top_k=vocab // 2 + 1), dict(top_p=0.5), dict(top_k=3), dict(min_p=0.5),
                         dict(top_k=vocab // 2, top_p=0.25)):
            check_sample(exq, same, u, "equal %d %s" % (vocab, settings), wide, **settings)
        few = rng.integers(0, 3, (4, vocab)) * 0.5
        for settings in (dict(), dict(top_k=vocab // 2), dict(top_p=0.7), dict(top_k=2 * vocab // 3, top_p=0.9), dict(top_p=0.97, min_p=0.3)):
            check_sample(exq, few, rng.random(4), "few values %d %s" % (vocab, settings), wide, **settings)
        flat = 0.3 * rng.standard_normal((4, vocab))
        for settings in (dict(), dict(top_p=0.95), dict(top_k=3 * vocab // 4), dict(top_k=vocab - 1, top_p=0.6)):
            check_sample(exq, flat, rng.random(4), "flat %d %s" % (vocab, settings), wide, **settings)


@pytest.mark.parametrize("wide", [False, True])
def test_sample_sorted_rows(exq, wide):
    """The likely tokens next to each other: one thread, or one wave, holds them all."""
    rng = np.random.default_rng(13)
    for vocab in (3000, 70001):
        x = np.sort(likely(rng, 3, vocab), axis=1)
        for row in (x, x[:, ::-1]):
            for settings in (dict(top_k=200), dict(top_p=0.9), dict(top_k=9000, top_p=0.999), dict()):
                check_sample(exq, row, rng.random(3), "sorted %d %s" % (vocab, settings), wide, **settings)


@pytest.mark.parametrize("wide", [False, True])
def test_sample_masked_infinite_and_nan_logits(exq, wide):
    rng = np.random.default_rng(14)
    x = likely(rng, 9, 5000)
    x[0, rng.random(5000) < 0.9] = -np.inf
    x[1, :] = -np.inf
    x[2, rng.random(5000) < 0.5] = np.nan
    x[3, :] = np.nan
    x[4, [17, 300, 4999]] = np.inf
    x[5, 1:] = -np.inf
    x[6, :4999] = np.nan
    x[7, :] = np.where(rng.random(5000) < 0.5, -0.0, 0.0)
    x[8, :] = -60000.0
    x[8, 77] = 60000.0
    for settings in (dict(), dict(top_k=30), dict(top_p=0.9), dict(top_k=2500, top_p=0.5), dict(min_p=0.1), dict(temperature=0.0),
                     dict(temperature=1e-30), dict(temperature=1e30), dict(temperature=np.inf)):
        check_sample(exq, x, rng.random(9), str(settings), wide, **settings)
    if wide:      # the largest finite value beside infinities is not drawn
        x[4, :200] = np.finfo(np.float32).max
        for settings in (dict(), dict(top_k=30), dict(top_p=0.9), dict(top_k=2500, top_p=0.5), dict(min_p=0.1)):
            check_sample(exq, x, rng.random(9), "beside infinities %s" % settings, wide, **settings)
    lowest = np.full((3, 2000), np.finfo(np.float32 if wide else np.float16).min)
    lowest[1, 1500] = 0.0
    check_sample(exq, lowest, np.array([0.3, 0.6, 0.9]), "lowest", wide, top_p=0.9)


def test_sample_settings_of_each_row_and_padding_rows(exq):
    rng = np.random.default_rng(15)
    rows, vocab = 40, 20011
    logits = likely(rng, rows, vocab).astype(np.float16)
    settings = dict(temperature=rng.choice([0.0, 0.5, 1.0, 1.7], rows).astype(np.float32), top_k=rng.choice([-4, 0, 1, 20, 900, 5000, vocab + 9], rows),
                    top_p=rng.choice([-1.0, 0.3, 0.95, 1.0, 7.0], rows).astype(np.float32), min_p=rng.choice([-1.0, 0.0, 0.02, 3.0], rows).astype(np.float32))
    settings["temperature"][3], settings["top_p"][5], settings["min_p"][6], settings["temperature"][7] = np.nan, np.nan, np.nan, -1.0
    u = rng.random(rows).astype(np.float32)
    u[8], u[9], u[10], u[11] = np.nan, 1.0, 5.0, np.inf
    check_sample(exq, logits, u, "each", **settings)
    u[::3] = -1.0
    tokens = torch.full((rows,), 99, dtype=torch.int32, device="cuda")
    logs = torch.full((rows,), 99.0, device="cuda")
    assert exq.sample(to_dev(logits), f32(u), out=tokens, logprobs=logs) is tokens
    assert torch.all(tokens[::3] == 99) and torch.all(logs[::3] == 99)
    np.testing.assert_array_equal(host(tokens)[1::3], [ref.sample_row(l, x)[0] for l, x in zip(logits[1::3], u[1::3])])


def test_sample_strides_offsets_and_refusals(exq):
    rng = np.random.default_rng(16)
    for wide in (False, True):
        x = likely(rng, 6, 3001).astype(np.float32 if wide else np.float16)
        u = rng.random(6)
        want = check_sample(exq, x, u, "plain", wide, top_p=0.9)
        for offset in range(9):
            d = torch.full((6, 3001 + 16), float("nan"), dtype=torch.float32 if wide else torch.float16, device="cuda")
            d[:, offset:offset + 3001] = to_dev(x)
            np.testing.assert_array_equal(host(exq.sample(d[:, offset:offset + 3001], f32(u), top_p=0.9)), want)
        same = exq.sample(to_dev(x)[:1].expand(6, 3001), f32([u[0]] * 6), top_p=0.9)
        assert torch.all(same == int(want[0]))
    l, u = to_dev(x), f32(u)
    for bad in (dict(logits=l.double()), dict(logits=l[0]), dict(logits=l[:, ::2]), dict(u=u[:3]), dict(u=u.double()), dict(temperature=-1.0),
                dict(temperature=u.half()), dict(top_k=u), dict(top_p=float("nan")), dict(top_p=u[:2]), dict(out=u), dict(out=i32([0])),
                dict(logprobs=u.double()), dict(logprobs=u), dict(logits=l.cpu())):
        with pytest.raises(exq.ExqError):
            exq.sample(**{**dict(logits=l, u=u), **bad})
    with pytest.raises(TypeError):
        exq.sample(l, u, top_k=0.5)
    assert exq.sample(l[:0], u[:0]).shape == (0,)


def test_sample_many_rows_and_the_largest_vocabulary(exq):
    rng = np.random.default_rng(17)
    check_sample(exq, likely(rng, 700, 999), rng.random(700), "many rows", top_p=0.9)
    big = likely(rng, 1, 1 << 21)
    for settings in (dict(), dict(top_p=0.9), dict(top_k=50), dict(top_k=1 << 20)):
        check_sample(exq, big, rng.random(1), "2^21 %s" % settings, True, **settings)


@pytest.mark.parametrize("wide", [False, True])
def test_sample_of_more_rows_than_are_shared_out(exq, wide):
    """Long rows that a workgroup has to itself."""
    rng = np.random.default_rng(18)
    x = likely(rng, 260, 20011)
    x[3, rng.random(20011) < 0.5] = -np.inf
    for settings in (dict(), dict(top_p=0.9), dict(temperature=3.0, top_p=0.98, min_p=0.01), dict(top_k=7000, top_p=0.95)):
        check_sample(exq, x, rng.random(260), "260 rows %s" % settings, wide, **settings)


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("rows,vocab", [(1, 16384), (2, 16391), (3, 70001), (17, 50001), (51, 16400), (85, 20001), (128, 16385), (129, 16385)])
def test_sample_rows_shared_out(exq, rows, vocab, wide):
    """Every number of parts, with rows that begin and end anywhere, masked ones and flat ones."""
    rng = np.random.default_rng(rows + vocab)
    x = likely(rng, rows, vocab)
    x[rng.integers(0, rows), :] *= 0.01
    x[rng.integers(0, rows), rng.random(vocab) < 0.99] = -np.inf
    x = x.astype(np.float32 if wide else np.float16)
    d = torch.full((rows, vocab + 5), float("nan"), dtype=torch.float32 if wide else torch.float16, device="cuda")
    for settings in (dict(), dict(top_p=0.9), dict(temperature=2.0, top_p=0.5, min_p=0.02)):
        u = rng.random(rows)
        want = check_sample(exq, x, u, "%d rows %s" % (rows, settings), wide, **settings)
        for offset in (1, 5):
            d[:, offset:offset + vocab] = to_dev(x)
            np.testing.assert_array_equal(host(exq.sample(d[:, offset:offset + vocab], f32(u), **settings)), want)


@pytest.mark.parametrize("wide", [False, True])
def test_sample_equal_logits_beyond_any_counter_and_list(exq, wide):
    """131072 equal logits: more than 16 bits count, than a list of candidates holds and than one power of two of bins tells apart."""
    rng = np.random.default_rng(19)
    same = np.zeros((3, 131072))
    same[1, :70000] = 1.0
    same[2, 5::2] = -np.inf
    u = np.array([0.1, 0.7, 0.999])
    for settings in (dict(), dict(top_p=0.5), dict(top_k=100000), dict(top_k=69999, top_p=0.9), dict(top_k=20), dict(top_k=901, top_p=0.5),
                     dict(top_p=0.9, min_p=0.5), dict(min_p=0.99)):
        check_sample(exq, same, u, "equal %s" % settings, wide, **settings)
    many = np.zeros((130, 131072), dtype=np.float16)      # a workgroup to a row
    many[:, 100000:] = rng.integers(-2, 1, (130, 31072))
    d = to_dev(many.astype(np.float32) if wide else many)
    for settings in (dict(top_p=0.5), dict()):
        got = host(exq.sample(d, f32([0.37] * 130), **settings))
        for r in (0, 64, 129):
            assert got[r] == ref.sample_row(many[r], np.float32(0.37), **{k: np.float32(v) for k, v in settings.items()})[0], (r, settings)


@pytest.mark.parametrize("vocab", [9000, 40000])
def test_sample_between_its_ways_to_find_the_top(exq, vocab):
    """A top-k on both sides of each way's limits, with ties at the end of it, nuclei that leave a list of any length, and min-p
    alone from one token to all."""
    rng = np.random.default_rng(vocab)
    x = likely(rng, 3, vocab)
    x[1] = np.round(x[1] * 4) / 4          # many ties
    x[2] = 0.02 * x[2]                     # flat
    for wide in (False, True):
        for settings in ([dict(top_k=k, top_p=p) for k in (127, 129, 899, 900, 901, 2048, 2049, 4096, 4097, 6000) for p in (1.0, 0.9)]
                         + [dict(min_p=p) for p in (1e-30, 1e-6, 1e-3, 0.3, 0.97, 1.0)] + [dict(temperature=2.0, top_k=3000, top_p=0.9, min_p=0.3)]):
            check_sample(exq, x, rng.random(3), "%d %s" % (vocab, settings), wide, **settings)


def test_sample_draws_the_shares(exq):
    """Evenly spaced numbers: each token as often as its share says, to one."""
    p = np.array([0.4, 0.3, 0.2, 0.07, 0.03])
    n = 2000
    logits = np.tile(np.log(p), (n, 1)).astype(np.float32)
    tokens = host(exq.sample(to_dev(logits), f32((np.arange(n) + 0.5) / n)))
    w = np.exp(logits[0].astype(np.float64))
    assert np.all(np.abs(np.bincount(tokens, minlength=5) - n * w / w.sum()) <= 1)


# --------------------------------------------------- streams, graphs, together

def small_step(exq):
    """The four operators' calls on small inputs: a function of a stream, and its tensors."""
    rng = np.random.default_rng(21)
    a, b, scales, ranks = stack(rng, 3, 256, 512, 16)
    t = dict(x=to_dev(rng.standard_normal((6, 256)).astype(np.float16)), y=to_dev(rng.standard_normal((6, 512)).astype(np.float16)),
             ids=i32([0, 2, -1, 1, 0, 2]), q=to_dev(rng.standard_normal((6, 4, 64)).astype(np.float16)), p=i32([4, 9, 0, 77, 3, 1]),
             logits=to_dev(likely(rng, 6, 5000).astype(np.float16)), u=f32(rng.random(6)), counts=i32([1, 0, 2, 1]), keep=i32([0, -1, 0, 0]))
    adapters = exq.Adapters(to_dev(a), to_dev(b), f32(scales), i32(ranks))
    rotary = exq.Rotary(64)
    pool = exq.PagePool(30, 16, 4, 6)

    def step(stream=None):
        out = [adapters.add(t["x"], t["ids"], t["y"], stream=stream), rotary.rotate(t["q"], t["p"], stream=stream)]
        out += exq.sample(t["logits"], t["u"], top_k=40, top_p=0.9, return_logprobs=True, stream=stream)
        pool.trim(t["keep"], stream=stream)
        out += pool.extend(t["counts"], 6, stream=stream)
        return out + [pool.table, pool.lengths]

    return step, t, (adapters, rotary, pool)


def test_calls_on_other_streams(exq):
    step, t, keep = small_step(exq)
    want = [x.clone() for x in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        got = step(stream)
        side.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_graphs_replay_with_new_values(exq):
    """Two captured graphs of the same calls, replayed in turn with new inputs and eager calls between."""
    step, t, (_, _, pool) = small_step(exq)
    nothing = i32([0, 0, 0, 0])
    rng = np.random.default_rng(22)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    graphs = []
    note("graph capture of a step")
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, step()))
    for rep in range(6):
        t["x"].copy_(to_dev(rng.standard_normal((6, 256)).astype(np.float16)))
        t["ids"].copy_(i32(rng.integers(-1, 3, 6)))
        t["p"].copy_(i32(rng.integers(0, 5000, 6)))
        t["logits"].copy_(to_dev(likely(rng, 6, 5000).astype(np.float16)))
        t["u"].copy_(f32(rng.random(6)))
        t["counts"].copy_(i32(rng.integers(0, 2, 4)))
        pool.trim(nothing)      # a step changes the pool: both start from the same
        want = [x.clone() for x in step()]
        pool.trim(nothing)
        g, got = graphs[rep % 2]
        g.replay()
        torch.cuda.synchronize()
        for i, (x, y) in enumerate(zip(got, want)):
            assert torch.equal(x, y), (rep, i)


def test_shared_out_draws_on_two_streams_and_in_graphs(exq):
    """Long rows on two streams at a time, eager and replayed: each call has a workspace of its own."""
    rng = np.random.default_rng(25)
    logits = [to_dev(likely(rng, 4, 50001).astype(np.float16)) for _ in range(2)]
    u = [f32(rng.random(4)) for _ in range(2)]
    note("graph capture of draws")
    draw = lambda i: exq.sample(logits[i], u[i], top_p=0.9, return_logprobs=True)
    streams, graphs = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(2):
        draw(i)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, draw(i)))
    for rep in range(5):
        for i in range(2):
            logits[i].copy_(to_dev(likely(rng, 4, 50001).astype(np.float16)))
            u[i].copy_(f32(rng.random(4)))
        want = [draw(i) for i in range(2)]
        torch.cuda.synchronize()
        got = []
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got.append([draw(i) for _ in range(8)])
                graphs[i][0].replay()
        torch.cuda.synchronize()
        for i in range(2):
            for tokens, logs in got[i] + [graphs[i][1]]:
                assert torch.equal(tokens, want[i][0]) and torch.equal(logs, want[i][1]), (rep, i)
            assert host(want[i][0]).tolist() == [ref.sample_row(l, x, top_p=np.float32(0.9))[0] for l, x in zip(host(logits[i]), host(u[i]))]


def test_offsets_past_32_bits(exq):
    """Rows 2^30 elements apart: the third lies past 2^31 elements and 2^32 bytes."""
    rng = np.random.default_rng(26)
    space = torch.empty(2 * (1 << 30) + (1 << 20), dtype=torch.float16, device="cuda")
    view = lambda offset, *shape: space.as_strided((3, *shape), (1 << 30, *([shape[-1], 1] if len(shape) == 2 else [1])), offset)
    logits = likely(rng, 3, 20000).astype(np.float16)
    l = view(8, 20000)
    l.copy_(to_dev(logits))
    u = rng.random(3)
    for settings in (dict(), dict(top_k=40), dict(top_p=0.9)):
        got = host(exq.sample(l, f32(u), **settings))
        assert got.tolist() == [ref.sample_row(x, np.float32(v), **{k: np.float32(p) if k == "top_p" else p for k, p in settings.items()})[0]
                                for x, v in zip(logits, u)], settings
    x = rng.standard_normal((3, 4, 64)).astype(np.float16)
    q, out, p = view(1 << 16, 4, 64), view(1 << 17, 4, 64), i32([7, -1, 1 << 20])
    q.copy_(to_dev(x))
    out.zero_()
    rotary = exq.Rotary(64)
    assert torch.equal(rotary.rotate(q, p, q_out=out)[::2], rotary.rotate(to_dev(x), p)[::2]) and not out[1].any()
    a, b, scales, ranks = stack(rng, 2, 64, 512, 16)
    adapters = exq.Adapters(to_dev(a), to_dev(b), f32(scales), i32(ranks))
    x, y, ids = rng.standard_normal((3, 64)).astype(np.float16), rng.standard_normal((3, 512)).astype(np.float16), i32([0, -1, 1])
    fx, fy = view(1 << 18, 64), view(1 << 19, 512)
    fx.copy_(to_dev(x))
    fy.copy_(to_dev(y))
    want = adapters.add(to_dev(x), ids, to_dev(y))
    assert torch.equal(adapters.add(fx, ids, fy), want)
    assert torch.equal(adapters.add(fx, ids, fy, out=fy), want)


def test_outputs_are_ordinary_tensors(exq):
    """Outputs of one call are chunks of an allocation: each can be changed, saved and used in a gradient by itself."""
    rng = np.random.default_rng(27)
    x, p = to_dev(rng.standard_normal((5, 3, 64)).astype(np.float16)), i32([0, 1, 2, 3, 4])
    rotary = exq.Rotary(64)
    q, k = rotary.rotate(x, p, k=x[:, :2])
    one = rotary.rotate(x, p)
    for t, shape in ((q, (5, 3, 64)), (k, (5, 2, 64))):
        assert t.shape == shape and t.is_contiguous() and t.device == x.device and not t.requires_grad and t.data_ptr() % 256 == 0
        assert torch.equal(t, one[:, :shape[1]])
    k.zero_()
    assert torch.equal(q, one)
    saved = io.BytesIO()
    torch.save(q, saved)
    saved.seek(0)
    assert torch.equal(torch.load(saved, weights_only=True), one)
    q.requires_grad_()
    (q.float() * 2).sum().backward()
    assert torch.all(q.grad == 2)
    tokens, logs = exq.sample(to_dev(likely(rng, 4, 1000).astype(np.float16)), f32(rng.random(4)), return_logprobs=True)
    kept = logs.clone()
    tokens.fill_(7)
    assert torch.equal(logs, kept)
    with torch.inference_mode():
        a, b = rotary.rotate(x, p, k=x)
        assert a.is_inference() and torch.equal(a, one)


def test_calls_are_deterministic(exq):
    rng = np.random.default_rng(23)
    a, b, _, _ = stack(rng, 5, 2048, 1024, 32)
    adapters = exq.Adapters(to_dev(a), to_dev(b))
    x, y, ids = to_dev(rng.standard_normal((600, 2048)).astype(np.float16)), to_dev(rng.standard_normal((600, 1024)).astype(np.float16)), i32(rng.integers(0, 5, 600))
    logits, u = to_dev(likely(rng, 30, 60000).astype(np.float16)), f32(rng.random(30))
    first = [adapters.add(x, ids, y), *exq.sample(logits, u, temperature=1.5, top_p=0.97, return_logprobs=True)]
    for _ in range(5):
        again = [adapters.add(x, ids, y), *exq.sample(logits, u, temperature=1.5, top_p=0.97, return_logprobs=True)]
        assert all(torch.equal(p, q) for p, q in zip(first, again))


def test_a_batch_decodes_with_all_of_it(exq):
    """Three sequences with pages from the pool: prompts of different lengths, then tokens one by one, one sequence ending and
    another taking its pages: projection with adapters, rotary positions, append, attention, logits, the draw."""
    rng = np.random.default_rng(24)
    S, H, KV, D, E, V = 3, 4, 2, 64, 256, 300
    weight = lambda n, k: (rng.standard_normal((n, k)) * k ** -0.5).astype(np.float16)
    qkv = exq.Layer.from_weight(weight((H + 2 * KV) * D, E).astype(np.float32), [8, 8])
    head = exq.Layer.from_weight(weight(304, H * D).astype(np.float32), [8, 8])
    w_qkv, w_head = host(qkv.dequant()).astype(np.float64), host(head.dequant()).astype(np.float64)
    a, b, scales, ranks = stack(rng, 2, E, (H + 2 * KV) * D, 8)
    adapters = exq.Adapters(to_dev(a), to_dev(b), f32(scales), i32(ranks))
    embed = rng.standard_normal((V, E)).astype(np.float16)
    d_embed = to_dev(embed)
    rotary = exq.Rotary(D, 32, interleaved=True)
    cache = exq.KVCache(12, 16, KV, D, 8, 8)
    pool, want = pool_pair(exq, 12, 16, S, 4)
    geo_held = lambda x: cacheref.held(x, 8)
    adapter_of = np.array([1, -1, 0])
    history = [[] for _ in range(S)]          # (k, v) fp16 of each token, as held
    feeds = [list(rng.integers(0, V, n)) for n in (20, 3, 33)]
    note("a batch decodes")
    for step in range(6):
        if step == 3:     # sequence 2 ends, a new prompt takes its place
            pool.trim(i32([-1, -1, 0]))
            want.trim([-1, -1, 0])
            history[2], feeds[2] = [], list(rng.integers(0, V, 18))
        counts = [len(f) for f in feeds]
        rows = sum(counts) + 2                # padded
        seqs, positions, offsets = pool.extend(i32(counts), rows)
        ps, pp, po, _ = want.extend(counts, rows)
        np.testing.assert_array_equal(host(seqs), ps)
        np.testing.assert_array_equal(host(positions), pp)
        same_pool(pool, want, "step %d" % step)
        ids = np.array([t for f in feeds for t in f] + [0, 0])
        x = d_embed[torch.tensor(ids, device="cuda")]
        row_adapter = np.where(ps >= 0, adapter_of[ps], -1)
        y = qkv.gemm(x)
        adapters.add(x, i32(row_adapter), y, out=y)
        y3 = y.view(rows, H + 2 * KV, D)
        rotary.rotate(y3[:, :H], positions, k=y3[:, H:H + KV], q_out=y3[:, :H], k_out=y3[:, H:H + KV])
        cache.append(y3[:, H:H + KV], y3[:, H + KV:], pool.table, seqs, positions)
        last = offsets[1:].long() - 1
        out = cache.attend(y3[last, :H], pool.table, pool.lengths)
        logits = head.gemm(out.view(S, H * D))[:, :V]
        u = rng.random(S).astype(np.float32)
        tokens = host(exq.sample(logits, f32(u), temperature=0.9, top_k=50, top_p=0.95))
        # the keys and values as the GPU rounded them, checked against the formulas, then the rest of the step from them
        base = embed[ids].astype(np.float64) @ w_qkv
        plain, size = ref.lora(embed[ids], row_adapter, base, a, b, scales, ranks)
        turned = np.concatenate([ref.rotate(plain.reshape(rows, -1, D)[:, :H + KV], pp, host(rotary.rates), 1.0, 32, True),
                                 plain.reshape(rows, -1, D)[:, H + KV:]], 1)
        got = host(y3).astype(np.float64)
        # gemm's rounding and bound, the adapters' and the rotation's: three roundings of values up to 1.5 times these
        sizes = np.abs(embed[ids].astype(np.float64)) @ np.abs(w_qkv) + size
        pair = sizes.reshape(rows, -1, D).max(-1, keepdims=True) + np.abs(plain).reshape(rows, -1, D).max(-1, keepdims=True)
        assert np.all(np.abs(got - turned) <= 5e-3 * pair + 1e-3)
        for r in range(rows):
            if ps[r] >= 0:
                history[ps[r]].append((geo_held(host(y3)[r, H:H + KV]), geo_held(host(y3)[r, H + KV:])))
        for s in range(S):
            k, v = (np.stack(z) for z in zip(*history[s]))
            o, _, bound, _ = cacheref.attend(host(y3)[po[s + 1] - 1, :H], k, v, D ** -0.5)
            assert np.all(np.abs(host(out)[s] - o) <= bound)
            assert tokens[s] == ref.sample_row(host(logits)[s], u[s], np.float32(0.9), 50, np.float32(0.95))[0]
            feeds[s] = [int(tokens[s])]
    qkv.close()
    head.close()
