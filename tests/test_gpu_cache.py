"""The paged key-value cache on the GPU against the plain reference (oracle/cacheref.py): appended bytes and values read
back bit for bit, attention within the bounds of include/exq.h, and what masks, strides, streams, graphs and bad tables do."""
import numpy as np
import pytest

import synth
from oracle import cacheref as ref
from tests.gpu_helpers import note, to_dev

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

BITS = [(4, 4), (8, 8), (8, 4), (4, 8), (16, 16)]


@pytest.fixture(scope="module")
def exq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mixed_bitrate_quantized_amd as m
    return m


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def values(rng, *shape, spread=1.0):
    x = rng.standard_normal(shape) * np.exp(spread * rng.standard_normal(shape[-2:]))
    return x.astype(np.float16)


class Case:
    """A cache of sequences with random pages in random order, filled through the reference."""

    def __init__(self, exq, seed, lengths, page, kv_heads, dim, bits, garbage=True, spare=1, spread=1.0):
        rng = np.random.default_rng(seed)
        self.rng, self.bits, self.lengths = rng, bits, list(lengths)
        self.geo = ref.Geometry(page, kv_heads, dim, *bits)
        width = max(1, -(-max(max(lengths), 1) // page)) + spare
        n_pages = len(lengths) * width
        self.table = rng.permutation(n_pages).astype(np.int32).reshape(len(lengths), width)
        # what lies where nothing was written: for 16-bit values NaN patterns, for scales too
        self.pages = np.full(n_pages * self.geo.page_bytes, 0xFF if garbage else 0, dtype=np.uint8)
        self.k, self.v = [], []
        for s, n in enumerate(lengths):
            n = max(n, 0)
            k, v = values(rng, n, kv_heads, dim, spread=spread), values(rng, n, kv_heads, dim, spread=spread)
            ref.append(self.geo, self.pages, k, v, self.table, [s] * n, range(n))
            self.k.append(ref.held(k, bits[0]) if n else k)
            self.v.append(ref.held(v, bits[1]) if n else v)
        self.dev = to_dev(self.pages)
        self.cache = exq.KVCache(n_pages, page, kv_heads, dim, *bits, pages=self.dev)
        self.dtable = i32(self.table)

    def check(self, out, lse, q, scale, window=0, lengths=None, what=""):
        out, lse = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        worst = 0.0
        for r, n in enumerate(self.lengths if lengths is None else lengths):
            if n < 0:
                continue
            lo = max(0, n - window) if window else 0
            o, l, bo, bl = ref.attend(q[r], self.k[r][lo:n], self.v[r][lo:n], scale)
            if n == 0:
                assert np.all(out[r] == 0) and np.all(lse[r] == -np.inf), what
                continue
            e = np.abs(out[r] - o) / bo
            f = np.abs(lse[r] - l) / bl
            assert e.max() <= 1 and f.max() <= 1, "%s row %d (n=%d): out %.3f lse %.3f of the bound" % (what, r, n, e.max(), f.max())
            worst = max(worst, e.max(), f.max())
        return worst


# ------------------------------------------------------------------ append, read

@pytest.mark.parametrize("bits", BITS, ids=str)
@pytest.mark.parametrize("dim,kv_heads,page", [(64, 3, 16), (96, 2, 48), (128, 1, 256), (256, 2, 32)])
def test_append_writes_exactly_the_references_bytes(exq, dim, kv_heads, page, bits):
    rng = np.random.default_rng(dim + page)
    geo = ref.Geometry(page, kv_heads, dim, *bits)
    n_pages, width = 9, 3
    table = rng.permutation(n_pages).astype(np.int32).reshape(3, width)
    pages = rng.integers(0, 256, n_pages * geo.page_bytes).astype(np.uint8)
    # a prompt from inside a tile over a page's end, single tokens, one whole aligned tile, padding
    spots = [(0, p) for p in range(page - 11, page + 26)] + [(1, 0), (2, 2 * page + 3), (-1, 5)] + [
        (1, p) for p in range(page, page + 16)] + [(-7, -3)]
    seqs, pos = np.array([s for s, _ in spots]), np.array([p for _, p in spots])
    k, v = values(rng, len(spots), kv_heads, dim), values(rng, len(spots), kv_heads, dim)
    k[3, 0, :32] = 0
    v[5, 0, 5] = 65504
    k[7, 0, 33] = np.float16(6e-8)
    note("append dim=%d page=%d bits=%s" % (dim, page, bits))
    dev = to_dev(pages)
    cache = exq.KVCache(n_pages, page, kv_heads, dim, *bits, pages=dev)
    cache.append(to_dev(k), to_dev(v), i32(table), i32(seqs), i32(pos))
    want = pages.copy()
    ref.append(geo, want, k, v, table, seqs, pos)
    np.testing.assert_array_equal(dev.cpu().numpy(), want)
    ko, vo = cache.read(i32(table), i32(seqs), i32(pos))
    live = seqs >= 0
    np.testing.assert_array_equal(ko.cpu().numpy()[live].view(np.uint16), ref.held(k, bits[0])[live].view(np.uint16))
    np.testing.assert_array_equal(vo.cpu().numpy()[live].view(np.uint16), ref.held(v, bits[1])[live].view(np.uint16))


@pytest.mark.parametrize("bits", [(4, 8), (8, 4)], ids=str)
def test_every_fp16_magnitude_as_a_groups_largest_and_ties(exq, bits):
    """Every finite fp16 as the largest of a group, beside the values nearest to the ties k + 1/2 of its scale (on the tie
    where fp16 has it) and random ones: all read back as the reference quantizes them."""
    rng = np.random.default_rng(11)
    top16 = np.arange(0x7C00, dtype=np.uint16).view(np.float16)
    n = top16.size
    x = np.zeros((n, 1, 64), dtype=np.float16)
    for g, b in enumerate((4, 8)):                      # the first group against 4-bit ties, the second against 8-bit ones
        top = (1 << (b - 1)) - 1
        s = (top16.astype(np.float32) / np.float32(top)).astype(np.float16).astype(np.float64)
        k = rng.integers(-top, top, size=(n, 28)) + 0.5
        ties = k * s[:, None]
        x[:, 0, 32 * g:32 * g + 28] = np.clip(ties, -top16[:, None].astype(np.float64), top16[:, None].astype(np.float64))
        x[:, 0, 32 * g + 28:32 * g + 31] = (rng.uniform(-1, 1, size=(n, 3)) * top16[:, None].astype(np.float64)).astype(np.float16)
        x[:, 0, 32 * g + 31] = top16 * np.where(rng.integers(0, 2, n), -1, 1)
    pages = -(-n // 256)
    cache = exq.KVCache(pages, 256, 1, 64, *bits)
    table, seqs, pos = i32(np.arange(pages)[None]), i32(np.zeros(n)), i32(np.arange(n))
    note("every fp16 magnitude bits=%s" % (bits,))
    cache.append(to_dev(x), to_dev(x), table, seqs, pos)
    ko, vo = cache.read(table, seqs, pos)
    np.testing.assert_array_equal(ko.cpu().numpy(), ref.held(x, bits[0]))
    np.testing.assert_array_equal(vo.cpu().numpy(), ref.held(x, bits[1]))


@pytest.mark.parametrize("bits", [(4, 8), (8, 4), (16, 16)], ids=str)
def test_the_largest_finite_values_stay_finite(exq, bits):
    x = torch.full((16, 1, 64), 65504.0, dtype=torch.float16, device="cuda")
    x[:, :, 1::2] = -65504.0
    cache = exq.KVCache(1, 16, 1, 64, *bits)
    table, seqs, pos = i32([[0]]), i32(np.zeros(16)), i32(np.arange(16))
    note("largest finite values bits=%s" % (bits,))
    cache.append(x, x, table, seqs, pos)
    for got, b in zip(cache.read(table, seqs, pos), bits):
        assert torch.all(got == torch.sign(x) * (65504 if b == 16 else 65472))   # 7 * 9352 and 127 * 515.5, in fp16


@pytest.mark.parametrize("bits", [(4, 4), (8, 8), (16, 16)], ids=str)
def test_aligned_prompt_and_long_read(exq, bits):
    """Whole tiles in order, from position 0: 2 sequences of 200 and 64 tokens, written in one call and read in two orders."""
    rng = np.random.default_rng(3)
    geo = ref.Geometry(64, 2, 128, *bits)
    table = rng.permutation(8).astype(np.int32).reshape(2, 4)
    seqs = np.repeat([0, 1], [200, 64])
    pos = np.concatenate([np.arange(200), np.arange(64)])
    k, v = values(rng, 264, 2, 128), values(rng, 264, 2, 128)
    want = np.zeros(8 * geo.page_bytes, dtype=np.uint8)
    ref.append(geo, want, k, v, table, seqs, pos)
    note("aligned prompt bits=%s" % (bits,))
    cache = exq.KVCache(8, 64, 2, 128, *bits)
    cache.append(to_dev(k), to_dev(v), i32(table), i32(seqs), i32(pos))
    np.testing.assert_array_equal(cache.pages.cpu().numpy().reshape(-1), want)
    for order in (np.arange(264), rng.permutation(264), np.concatenate([np.arange(1, 264), [5]])):
        ko, vo = cache.read(i32(table), i32(seqs[order]), i32(pos[order]))
        np.testing.assert_array_equal(ko.cpu().numpy(), ref.held(k, bits[0])[order])
        np.testing.assert_array_equal(vo.cpu().numpy(), ref.held(v, bits[1])[order])


@pytest.mark.parametrize("bits", [(4, 8), (16, 16)], ids=str)
def test_rows_outside_are_skipped_and_read_as_nan(exq, bits):
    rng = np.random.default_rng(4)
    geo = ref.Geometry(16, 2, 64, *bits)
    table = np.array([[1, 7, -1], [0, 2, 1 << 30]], dtype=np.int32)     # 4 pages: 7, -1 and 2^30 are none
    spots = [(0, 3), (0, 16), (0, 40), (1, 40), (2, 0), (1 << 30, 0), (1, 48), (1, 1 << 30), (1, -1), (1, 20), (-1, 0),
             (-(1 << 31), 1)]
    seqs, pos = np.array([s for s, _ in spots]), np.array([p for _, p in spots])
    k, v = values(rng, len(spots), 2, 64), values(rng, len(spots), 2, 64)
    pages = rng.integers(0, 256, 4 * geo.page_bytes).astype(np.uint8)
    want = pages.copy()
    ref.append(geo, want, k, v, table, seqs, pos)
    note("rows outside bits=%s" % (bits,))
    dev = to_dev(pages)
    cache = exq.KVCache(4, 16, 2, 64, *bits, pages=dev)
    cache.append(to_dev(k), to_dev(v), i32(table), i32(seqs), i32(pos))
    np.testing.assert_array_equal(dev.cpu().numpy(), want)
    ko, vo = (torch.full((len(spots), 2, 64), 7.0, dtype=torch.float16, device="cuda") for _ in range(2))
    cache.read(i32(table), i32(seqs), i32(pos), ko, vo)
    ko, vo = ko.cpu().numpy(), vo.cpu().numpy()
    for r in range(len(spots)):
        if r in (0, 9):
            np.testing.assert_array_equal(ko[r], ref.held(k[r], bits[0]))
            np.testing.assert_array_equal(vo[r], ref.held(v[r], bits[1]))
        elif seqs[r] < 0:
            assert np.all(ko[r] == 7) and np.all(vo[r] == 7)
        else:
            assert np.all(np.isnan(ko[r])) and np.all(np.isnan(vo[r]))


@pytest.mark.parametrize("bits", [(4, 8), (16, 16)], ids=str)
def test_infinities_and_nan_poison_their_group_only(exq, bits):
    rng = np.random.default_rng(5)
    k, v = values(rng, 3, 1, 64), values(rng, 3, 1, 64)
    k[0, 0, 3], k[1, 0, 40], v[2, 0, 0], v[2, 0, 63] = np.inf, np.nan, -np.inf, np.nan
    note("non-finite bits=%s" % (bits,))
    cache = exq.KVCache(1, 16, 1, 64, *bits)
    t, s, p = i32([[0]]), i32([0, 0, 0]), i32([0, 1, 15])
    cache.append(to_dev(k), to_dev(v), t, s, p)
    ko, vo = (x.cpu().numpy() for x in cache.read(t, s, p))
    np.testing.assert_array_equal(ko, ref.held(k, bits[0]))
    np.testing.assert_array_equal(vo, ref.held(v, bits[1]))


def test_strided_and_broadcast_rows(exq):
    """k and v as slices of one projection's rows and as [heads][rows] views; one value broadcast to all rows."""
    rng = np.random.default_rng(6)
    rows, heads, dim = 21, 2, 64
    fused = values(rng, rows, 6, dim)                       # [q q | k k | v v]
    d = to_dev(fused)
    t, s, p = i32([[1, 0]]), i32([0] * rows), i32(np.arange(rows) + 3)
    note("strided rows")
    cache = exq.KVCache(2, 16, heads, dim, 8, 4)
    cache.append(d[:, 2:4], d[:, 4:6], t, s, p)
    hold = to_dev(np.zeros((rows, 4, dim), dtype=np.float16))
    cache.read(t, s, p, hold[:, :2], hold[:, 2:])           # two slices of one buffer
    h = hold.cpu().numpy()
    np.testing.assert_array_equal(h[:, :2], ref.held(fused[:, 2:4], 8))
    np.testing.assert_array_equal(h[:, 2:], ref.held(fused[:, 4:6], 4))
    turned = to_dev(np.ascontiguousarray(fused[:, 2:4].transpose(1, 0, 2))).transpose(0, 1)
    one = to_dev(fused[0, 4:6])[None].expand(rows, heads, dim)
    cache.append(turned, one, t, s, p)
    ko, vo = (x.cpu().numpy() for x in cache.read(t, s, p))
    np.testing.assert_array_equal(ko, ref.held(fused[:, 2:4], 8))
    np.testing.assert_array_equal(vo, np.broadcast_to(ref.held(fused[0, 4:6], 4), vo.shape))


# ------------------------------------------------------------------ attend

@pytest.mark.parametrize("bits", BITS, ids=str)
@pytest.mark.parametrize("dim,kv_heads,group,page", [(64, 2, 1, 16), (96, 2, 7, 48), (128, 2, 8, 256), (256, 1, 16, 32),
                                                     (128, 1, 20, 64)])
def test_attend_matches_reference(exq, dim, kv_heads, group, page, bits):
    lengths = [1, 0, 15, 16, 17, 31, 33, 127, 128, 129, 513, 700]
    c = Case(exq, dim + group, lengths, page, kv_heads, dim, bits)
    q = values(c.rng, len(lengths), kv_heads * group, dim, spread=0.5)
    scale = dim ** -0.5
    note("attend dim=%d group=%d page=%d bits=%s" % (dim, group, page, bits))
    out, lse = c.cache.attend(to_dev(q), c.dtable, i32(lengths), scale=scale, return_lse=True)
    c.check(out, lse, q, scale, what="all rows")
    # the same rows alone: another split, within the same bounds
    for r in (0, 4, 11):
        o, l = c.cache.attend(to_dev(q[r:r + 1]), c.dtable[r:r + 1], i32(lengths[r:r + 1]), return_lse=True)
        one = Case.__new__(Case)
        one.k, one.v, one.lengths = [c.k[r]], [c.v[r]], [lengths[r]]
        one.check(o, l, q[r:r + 1], scale, what="alone")


@pytest.mark.parametrize("bits", BITS, ids=str)
@pytest.mark.parametrize("dim,kv_heads,group,page", [(64, 2, 5, 16), (96, 1, 3, 48), (128, 1, 8, 256), (256, 1, 2, 64)])
def test_attend_split(exq, dim, kv_heads, group, page, bits):
    """Rows long enough to be split and joined, in tables just wide enough and in ones of over 16384 tokens; with and
    without a window."""
    lengths = [1300, 5, 2100, 0, 1025]
    c = Case(exq, dim + group + 1, lengths, page, kv_heads, dim, bits, spread=0.7)
    wide = np.concatenate([c.table, np.full((5, -(-16384 // page)), -1, dtype=np.int32)], 1)
    q = values(c.rng, 5, kv_heads * group, dim, spread=0.5)
    for t in (c.table, wide):
        for window in (0, 1200):
            note("attend split dim=%d bits=%s width=%d window=%d" % (dim, bits, t.shape[1], window))
            assert exq.exq_attend_workspace_bytes(c.cache.handle, 5, kv_heads * group, t.shape[1]) > 0
            out, lse = c.cache.attend(to_dev(q), i32(t), i32(lengths), window=window, return_lse=True)
            c.check(out, lse, q, dim ** -0.5, window, what="window %d" % window)


@pytest.mark.parametrize("bits", [(4, 4), (16, 16)], ids=str)
@pytest.mark.parametrize("window", [1, 16, 100, 129, 400, 1000])
def test_window(exq, window, bits):
    lengths = [0, 1, 16, 99, 130, 300, 515]
    c = Case(exq, window, lengths, 32, 2, 64, bits)
    q = values(c.rng, len(lengths), 6, 64, spread=0.5)
    note("window=%d bits=%s" % (window, bits))
    # pages wholly before the window may have been given away: their entries are no pages
    t = c.table.copy()
    for r, n in enumerate(lengths):
        t[r, :max(0, n - window) // 32] = -1
        t[r, -(-n // 32):] = 1 << 30
    out, lse = c.cache.attend(to_dev(q), i32(t), i32(lengths), scale=0.2, window=window, return_lse=True)
    c.check(out, lse, q, 0.2, window, what="window %d" % window)


def test_long_sequence_split_and_ragged_batch(exq):
    """One long sequence over many workgroups, beside short ones: 9000, 40, 0 and 2500 tokens."""
    lengths = [9000, 40, 0, 2500]
    c = Case(exq, 9, lengths, 256, 1, 64, (8, 4), spread=0.5)
    q = values(c.rng, 4, 4, 64, spread=0.5)
    note("long ragged")
    out, lse = c.cache.attend(to_dev(q), c.dtable, i32(lengths), scale=0.125, return_lse=True)
    c.check(out, lse, q, 0.125)
    again, _ = c.cache.attend(to_dev(q), c.dtable, i32(lengths), scale=0.125, return_lse=True)
    assert torch.equal(out, again)


@pytest.mark.parametrize("bits", [(4, 4), (16, 16)], ids=str)
def test_sharp_and_rising_scores(exq, bits):
    """Scores that rise by far more than the reference's slack along the sequence, fall, and are all but one negligible."""
    n, dim = 700, 64
    for kind in ("rising", "falling", "spike"):
        c = Case(exq, 10, [n], 64, 1, dim, bits)
        ramp = {"rising": np.linspace(-40, 40, n), "falling": np.linspace(40, -40, n),
                "spike": np.where(np.arange(n) == 345, 60, -20)}[kind]
        k = np.ones((n, 1, dim)) * ramp[:, None, None] / 8
        k[:, 0, ::2] *= 0.5
        k = k.astype(np.float16)
        v = values(c.rng, n, 1, dim)
        ref.append(c.geo, c.pages, k, v, c.table, [0] * n, range(n))
        c.k, c.v = [ref.held(k, bits[0])], [ref.held(v, bits[1])]
        c.cache.pages.copy_(to_dev(c.pages))
        q = np.ones((1, 2, dim), dtype=np.float16)
        q[0, 1] = -1
        note("%s bits=%s" % (kind, bits))
        for scale in (0.125, 1.0, -0.5, 0.0):
            out, lse = c.cache.attend(to_dev(q), c.dtable, i32([n]), scale=scale, return_lse=True)
            c.check(out, lse, q, scale, what="%s scale %g" % (kind, scale))


def test_padding_rows_bad_pages_and_too_long_rows(exq):
    lengths = [40, -1, 33, 40, -(1 << 31), 200]
    for page, width_note in ((16, "split"), (48, "whole")):
        c = Case(exq, 12, [40, 40, 40, 40, 40, 40], page, 2, 64, (4, 4), spare=0 if page == 48 else 30)
        t = c.table.copy()
        t[3, 0] = c.cache.n_pages                 # read: not a page
        t[2, -(-33 // page):] = -5                # behind the end: never looked at
        n = [x if x != 200 else t.shape[1] * page + 1 for x in lengths]
        q = values(c.rng, 6, 4, 64)
        out = torch.full((6, 4, 64), 3.0, dtype=torch.float16, device="cuda")
        lse = torch.full((6, 4), 3.0, dtype=torch.float32, device="cuda")
        note("padding and bad pages, %s" % width_note)
        c.cache.attend(to_dev(q), i32(t), i32(n), out=out, lse=lse)
        assert torch.all(out[[1, 4]] == 3) and torch.all(lse[[1, 4]] == 3)
        assert torch.all(torch.isnan(out[[3, 5]])) and torch.all(torch.isnan(lse[[3, 5]]))
        c.check(out, lse, q, 0.125, lengths=[40, -1, 33, -1, -1, -1])


def test_only_padding_and_empty_rows(exq):
    c = Case(exq, 13, [5, 5, 5], 256, 1, 64, (8, 8), spare=4)
    q = to_dev(values(c.rng, 3, 1, 64))
    for n in ([-1, -1, -1], [0, 0, 0], [-1, 0, -1], [0, 3, -1]):
        out = torch.full((3, 1, 64), 3.0, dtype=torch.float16, device="cuda")
        note("lengths %s" % n)
        c.cache.attend(q, c.dtable, i32(n), out=out)
        for r in range(3):
            if n[r] < 0:
                assert torch.all(out[r] == 3)
            elif n[r] == 0:
                assert torch.all(out[r] == 0)
            else:
                assert torch.all(torch.isfinite(out[r])) and torch.any(out[r] != 0)


@pytest.mark.parametrize("bits", [(4, 4), (16, 16)], ids=str)
def test_infinite_and_nan_values_that_are_attended_to_show(exq, bits):
    """A NaN in a key makes its row NaN; a NaN in one group of a value only that group; other rows and heads stay."""
    n = 150
    c = Case(exq, 14, [n, n], 64, 2, 64, bits, spare=8)
    k, v = values(c.rng, n, 2, 64), values(c.rng, n, 2, 64)
    k[77, 0, 5] = np.nan
    v[140, 1, 40] = np.nan
    ref.append(c.geo, c.pages, k, v, c.table, [0] * n, range(n))
    c.cache.pages.copy_(to_dev(c.pages))
    q = values(c.rng, 2, 4, 64)
    note("attended NaN bits=%s" % (bits,))
    out, lse = c.cache.attend(to_dev(q), c.dtable, i32([n, n]), return_lse=True)
    o = out.cpu().numpy()
    assert np.all(np.isnan(o[0, :2])) and np.all(torch.isnan(lse[0, :2]).cpu().numpy())
    bad = slice(32, 64) if bits[1] < 16 else slice(40, 41)
    assert np.all(np.isnan(o[0, 2:, bad]))
    rest = np.ones(64, bool)
    rest[bad] = False
    assert np.all(np.isfinite(o[0, 2:][:, rest])) and np.all(np.isfinite(o[1]))


def test_averages_of_the_largest_values_stay_finite(exq):
    """Weights rounded to fp16 can sum to more than the sum they are divided by: an average of 65504s is still 65504."""
    lengths = [1, 2, 3, 7, 40, 333, 1024, 2500]
    c = Case(exq, 31, lengths, 64, 1, 64, (16, 16))
    for s, n in enumerate(lengths):
        c.v[s][:] = np.where(np.arange(64) % 2, np.float16(65504), np.float16(-65504))
        ref.append(c.geo, c.pages, c.k[s], c.v[s], c.table, [s] * n, range(n))
    c.cache.pages.copy_(to_dev(c.pages).view_as(c.cache.pages))
    q = values(c.rng, len(lengths), 16, 64)
    note("averages of the largest values")
    out, lse = c.cache.attend(to_dev(q), c.dtable, i32(lengths), return_lse=True)
    assert torch.all(torch.isfinite(out))
    c.check(out, lse, q, 0.125)


def test_scores_of_minus_infinity(exq):
    """Keys whose score is -infinity weigh nothing, whole steps of them at the front included; a row of nothing else is NaN."""
    n, dim = 2200, 64
    c = Case(exq, 23, [n, 60, 1100], 64, 1, dim, (16, 16), garbage=False)
    gone = [np.arange(n) < 900, np.ones(60, bool), np.arange(1100) >= 7]
    for s in range(3):
        c.k[s][gone[s], 0, 3] = -np.inf
        ref.append(c.geo, c.pages, c.k[s], c.v[s], c.table, [s] * len(c.k[s]), range(len(c.k[s])))
    c.cache.pages.copy_(to_dev(c.pages).view_as(c.cache.pages))
    q = np.abs(values(c.rng, 3, 2, dim)) + np.float16(0.01)
    note("scores of -infinity")
    out, lse = c.cache.attend(to_dev(q), c.dtable, i32(c.lengths), return_lse=True)
    out, lse = out.cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
    assert np.all(np.isnan(out[1])) and np.all(np.isnan(lse[1]) | (lse[1] == -np.inf))
    for s in (0, 2):
        o, l, bo, bl = ref.attend(q[s], c.k[s][~gone[s]], c.v[s][~gone[s]], 0.125)
        assert np.all(np.abs(out[s] - o) <= bo) and np.all(np.abs(lse[s] - l) <= bl)


def test_shared_pages_and_expanded_tables(exq):
    """Sequences that share a prefix's pages, through tables of their own and through one expanded table row."""
    c = Case(exq, 24, [96, 96], 32, 2, 64, (4, 4), garbage=False)
    t = c.table.copy()
    t[1, :2] = t[0, :2]                                   # 64 shared tokens, then each its own
    c.k[1][:64], c.v[1][:64] = c.k[0][:64], c.v[0][:64]
    q = values(c.rng, 2, 4, 64)
    note("shared pages")
    out, lse = c.cache.attend(to_dev(q), i32(t), i32([96, 90]), return_lse=True)
    c.check(out, lse, q, 0.125, lengths=[96, 90])
    c.k[1], c.v[1] = c.k[0], c.v[0]
    out, lse = c.cache.attend(to_dev(q), i32(t[:1]).expand(2, -1), i32([96, 40]), return_lse=True)
    c.check(out, lse, q, 0.125, lengths=[96, 40])


@pytest.mark.parametrize("rows", [65, 130, 257])
def test_rows_beyond_a_waves_lanes_with_long_ones_among_them(exq, rows):
    """More rows than a wave has lanes, most short, some long enough to be split (up to 256 rows), some padding."""
    rng = np.random.default_rng(rows)
    lengths = rng.integers(0, 40, rows)
    lengths[[0, 63, 64, rows - 1]] = [2500, 1, 2900, 2777]
    c = Case(exq, rows, list(lengths), 16, 1, 64, (8, 4), spare=0)
    n = np.where(rng.integers(0, 5, rows) == 0, -1, lengths)
    n[[0, 64, rows - 1]] = lengths[[0, 64, rows - 1]]
    q = values(c.rng, rows, 3, 64)
    note("%d rows, some long" % rows)
    out, lse = c.cache.attend(to_dev(q), c.dtable, i32(n), return_lse=True)
    c.check(out, lse, q, 0.125, lengths=list(n))


@pytest.mark.parametrize("dim,kv_heads,rows,bits", [(64, 4, 16, (16, 16)), (128, 8, 8, (8, 8)), (256, 1, 64, (4, 4)),
                                                    (64, 1, 128, (16, 16)), (96, 4, 24, (16, 16)),
                                                    (128, 4, 5, (4, 4)), (64, 3, 7, (8, 4)), (128, 7, 6, (16, 16)),
                                                    (128, 8, 11, (4, 8)), (64, 8, 12, (4, 4))])
def test_even_and_nearly_even_batches(exq, dim, kv_heads, rows, bits):
    """Rows of one length, whose chunks come out at one a CU, the same with a short, an empty and a padding row, and any."""
    c = Case(exq, 33, [1500], 32, kv_heads, dim, bits, spare=0)
    c.k, c.v = c.k * rows, c.v * rows
    table = c.dtable.expand(rows, -1)
    q = values(c.rng, rows, kv_heads, dim)
    ragged = [int(x) for x in c.rng.integers(1, 1501, rows)]
    for n in ([1500] * rows, [1400] * (rows - 1) + [130], [0, -1] + [1500] * (rows - 2), ragged):
        note("even batch dim=%d bits=%s lengths=%s.." % (dim, bits, n[:2]))
        out, lse = c.cache.attend(to_dev(q), table, i32(n), return_lse=True)
        c.check(out, lse, q, dim ** -0.5, lengths=n)


@pytest.mark.parametrize("dim", [64, 128])
def test_four_million_tokens_of_a_batch(exq, dim):
    """64 segments of over 2^16 tokens at 4 bits (a few pages over and over): even, and with one row short."""
    page, times, rows, kv_heads = 64, 260, 32, 2
    c = Case(exq, 34, [4 * page], page, kv_heads, dim, (4, 4), spare=0)
    c.k, c.v = [np.tile(c.k[0], (times, 1, 1))] * rows, [np.tile(c.v[0], (times, 1, 1))] * rows
    table = i32(np.tile(c.table, (1, times))).expand(rows, -1)
    q = values(c.rng, rows, kv_heads, dim)
    full = times * 4 * page
    for n in ([full] * rows, [full - 17] * (rows - 1) + [777]):
        note("four million tokens dim=%d last=%d" % (dim, n[-1]))
        out, lse = c.cache.attend(to_dev(q), table, i32(n), return_lse=True)
        keep = [n[r] if r in (0, 13, rows - 1) else -1 for r in range(rows)]
        c.check(out, lse, q, dim ** -0.5, lengths=keep)
        assert torch.all(torch.isfinite(out))


def test_many_rows_and_heads(exq):
    """More rows than a workgroup has threads, in both split and whole launches."""
    for spare in (0, 40):
        c = Case(exq, 15, [3 + r % 29 for r in range(300)], 16, 1, 64, (4, 4), spare=spare)
        q = values(c.rng, 300, 2, 64)
        note("300 rows, spare %d" % spare)
        out, lse = c.cache.attend(to_dev(q), c.dtable, i32(c.lengths), return_lse=True)
        c.check(out, lse, q, 0.125)


def test_strided_queries_and_outputs(exq):
    lengths = [70, 5, 260]
    c = Case(exq, 16, lengths, 32, 2, 64, (8, 8), spare=20)
    fused = values(c.rng, 3, 12, 64)                        # [4 query heads | something | 4 output heads]
    d = to_dev(fused)
    note("strided attend")
    lse = torch.empty((3, 4), dtype=torch.float32, device="cuda")
    c.cache.attend(d[:, :4], c.dtable, i32(lengths), out=d[:, 8:], lse=lse)
    c.check(d[:, 8:], lse, fused[:, :4], 0.125)
    np.testing.assert_array_equal(d[:, :8].cpu().numpy(), fused[:, :8])
    wide = i32(np.concatenate([c.table, np.full_like(c.table, 1 << 30)], 1))[:, :c.table.shape[1]]
    plain, lse = c.cache.attend(d[:, :4].contiguous(), wide, i32(lengths), return_lse=True)
    assert torch.equal(plain, d[:, 8:])
    turned = torch.zeros((4, 3, 64), dtype=torch.float16, device="cuda").transpose(0, 1)
    c.cache.attend(d[:, :4], c.dtable, i32(lengths), out=turned)
    assert torch.equal(turned, plain)
    same = to_dev(fused[0, :4])[None].expand(3, 4, 64)
    o, l = c.cache.attend(same, c.dtable, i32(lengths), return_lse=True)
    c.check(o, l, np.broadcast_to(fused[0, :4], (3, 4, 64)), 0.125)


def test_pages_beyond_32_bit_offsets(exq):
    """A cache of over 8 GiB whose used pages lie at its very end."""
    page, heads, dim, bits = 256, 8, 256, (16, 16)
    geo = ref.Geometry(page, heads, dim, *bits)
    n_pages = (9 << 30) // geo.page_bytes
    cache = exq.KVCache(n_pages, page, heads, dim, *bits, pages=torch.empty(n_pages * geo.page_bytes, dtype=torch.uint8, device="cuda"))
    rng = np.random.default_rng(17)
    n = 300
    k, v = values(rng, n, heads, dim, spread=0.3), values(rng, n, heads, dim, spread=0.3)
    t = i32([[n_pages - 1, n_pages - 2]])
    note("9 GiB of pages")
    cache.append(to_dev(k), to_dev(v), t, i32([0] * n), i32(np.arange(n)))
    ko, vo = cache.read(t, i32([0] * n), i32(np.arange(n)))
    np.testing.assert_array_equal(ko.cpu().numpy(), k)
    np.testing.assert_array_equal(vo.cpu().numpy(), v)
    q = values(rng, 1, heads, dim, spread=0.3)
    one = Case.__new__(Case)
    one.k, one.v, one.lengths = [k], [v], [n]
    out, lse = cache.attend(to_dev(q), t, i32([n]), return_lse=True)
    one.check(out, lse, q, dim ** -0.5)


# ------------------------------------------------- streams, graphs, guard bands, together

def test_guard_bands(exq):
    c = Case(exq, 18, [37, 2600], 64, 2, 96, (4, 8))
    q = to_dev(values(c.rng, 2, 6, 96))
    note("guard bands")
    buf = torch.full((2 * 6 * 96 + 128,), 9.0, dtype=torch.float16, device="cuda")
    lbuf = torch.full((2 * 6 + 64,), 9.0, dtype=torch.float32, device="cuda")
    need = exq.exq_attend_workspace_bytes(c.cache.handle, 2, 6, c.dtable.shape[1])
    ws = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
    counters = ws[256:256 + exq.ATTEND_COUNTER_BYTES]
    counters.zero_()
    out, lse = buf[64:-64].view(2, 6, 96), lbuf[32:-32].view(2, 6)
    assert need > exq.ATTEND_COUNTER_BYTES
    c.cache.attend(q, c.dtable, i32([37, 2600]), out=out, lse=lse, workspace=ws[256:256 + need])
    c.check(out, lse, q.cpu().numpy(), 96 ** -0.5)
    assert torch.all(counters == 0)
    assert torch.all(buf[:64] == 9) and torch.all(buf[-64:] == 9) and torch.all(lbuf[:32] == 9) and torch.all(lbuf[-32:] == 9)
    assert torch.all(ws[:256] == 77) and torch.all(ws[-256:] == 77)
    np.testing.assert_array_equal(c.cache.pages.cpu().numpy().reshape(-1), c.pages)


def test_calls_of_all_sizes_share_a_workspace(exq):
    """Many workgroups to a segment (two levels of joining), few, and none, one after another through one workspace."""
    lengths = [30000, 700]
    c = Case(exq, 22, lengths, 64, 1, 64, (8, 8), spread=0.5, garbage=False)
    ws = c.cache.workspace(max(exq.exq_attend_workspace_bytes(c.cache.handle, 2, h, c.dtable.shape[1]) for h in (1, 7, 16, 32)))
    for heads in (1, 32, 7, 16):
        q = values(c.rng, 2, heads, 64, spread=0.5)
        for lens in ([30000, 700], [130, -1], [17000, 0], [-1, -1], [5, 700], [30000, -1]):
            note("shared workspace heads=%d lengths=%s" % (heads, lens))
            out, lse = c.cache.attend(to_dev(q), c.dtable, i32(lens), return_lse=True, workspace=ws)
            if heads < 32:
                one = Case.__new__(Case)
                one.k, one.v, one.lengths = [x[:max(n, 0)] for x, n in zip(c.k, lens)], [
                    x[:max(n, 0)] for x, n in zip(c.v, lens)], lens
                one.check(out, lse, q, 0.125, what="%d heads %s" % (heads, lens))
            assert torch.all(ws[:exq.ATTEND_COUNTER_BYTES] == 0)


def test_a_new_cache_is_ready_for_any_stream(exq):
    x = to_dev(values(np.random.default_rng(32), 64, 8, 128))
    table, seqs, pos = i32([[0]]), i32(np.zeros(64)), i32(np.arange(64))
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    note("append on another stream than the cache's pages were zeroed on")
    cache = exq.KVCache(4096, 256, 8, 128, 16, 16)    # 4 GiB of zeros
    cache.append(x, x, table, seqs, pos, stream=other)
    torch.cuda.synchronize()
    k, v = cache.read(table, seqs, pos)
    assert torch.equal(k, x) and torch.equal(v, x)


def test_other_streams_at_once(exq):
    c = Case(exq, 19, [1500, 700, 20], 64, 2, 64, (4, 4))
    qs = [values(c.rng, 3, 4, 64) for _ in range(4)]
    dq, n = [to_dev(q) for q in qs], i32(c.lengths)
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    note("four streams")
    got = [c.cache.attend(dq[i], c.dtable, n, return_lse=True, stream=streams[i]) for i in range(4)]
    raw = c.cache.attend(dq[0], c.dtable, n, return_lse=True, stream=streams[1].cuda_stream)
    torch.cuda.synchronize()
    for i in range(4):
        c.check(*got[i], qs[i], 0.125)
    assert torch.equal(raw[0], got[0][0])


def test_graphs_replay_append_and_attend(exq):
    """Two captured graphs of one decoding step each, replayed several times with eager calls between: new tokens written,
    then attended to.  Lengths, tables and inputs are read at replay."""
    lengths = [700, 3, 120, 0]
    c = Case(exq, 20, lengths, 64, 2, 64, (8, 4), spare=2)
    rng = c.rng
    q, k, v = (torch.zeros((4, h, 64), dtype=torch.float16, device="cuda") for h in (6, 2, 2))
    seqs, pos, n = i32(np.arange(4)), i32([0] * 4), i32([0] * 4)

    def step():
        c.cache.append(k, v, c.dtable, seqs, pos)
        return c.cache.attend(q, c.dtable, n, return_lse=True)

    pos.copy_(i32(lengths))
    note("graph capture")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = step()
        graphs.append((g, res))
    held = [list(x) for x in zip(c.k, c.v)]
    now = list(lengths)
    for rep in range(6):
        g, (out, lse) = graphs[rep % 2]
        hq, hk, hv = values(rng, 4, 6, 64), values(rng, 4, 2, 64), values(rng, 4, 2, 64)
        q.copy_(to_dev(hq)); k.copy_(to_dev(hk)); v.copy_(to_dev(hv))
        pos.copy_(i32(now))
        now = [x + 1 for x in now]
        n.copy_(i32(now))
        g.replay()
        torch.cuda.synchronize()
        for s in range(4):
            held[s][0] = np.concatenate([held[s][0], ref.held(hk[s:s + 1], 8)])
            held[s][1] = np.concatenate([held[s][1], ref.held(hv[s:s + 1], 4)])
        c.k, c.v = [h[0] for h in held], [h[1] for h in held]
        c.check(out, lse, hq, 0.125, lengths=now, what="replay %d" % rep)
        eager, elog = c.cache.attend(q, c.dtable, n, return_lse=True)
        assert torch.equal(eager, out) and torch.equal(elog, lse)


def test_a_block_decodes_through_its_cache(exq):
    """The cache between a block's linears, as a decoding loop runs it: q/k/v in one plan, append, attend, output linear.
    Every step's attention is checked against the reference on the values the plan gave."""
    heads, kv_heads, dim, K, M, steps = 8, 2, 64, 512, 3, 20
    widths = [2, 4, 6, 8]
    mk = lambda tag, N: exq.Layer.from_weight(synth.weight(synth.seed_for("block", tag), N, K), widths)
    lq, lk, lv, lo = mk("q", heads * dim), mk("k", kv_heads * dim), mk("v", kv_heads * dim), mk("o", K)
    x = torch.empty((M, K), dtype=torch.float16, device="cuda")
    yq, yk, yv = (torch.empty((M, h * dim), dtype=torch.float16, device="cuda") for h in (heads, kv_heads, kv_heads))
    plan = exq.Plan([lq, lk, lv], [x, x, x], [yq, yk, yv], M)
    cache = exq.KVCache(M * 2, 16, kv_heads, dim, 4, 4)
    table = i32(np.arange(2 * M).reshape(M, 2)[:, ::-1].copy())
    seqs = i32(np.arange(M))
    ks, vs = [], []
    note("block decode")
    for t in range(steps):
        x.copy_(to_dev(synth.activations(synth.seed_for("block-x", t), M, K)))
        plan.run()
        cache.append(yk.view(M, kv_heads, dim), yv.view(M, kv_heads, dim), table, seqs, i32([t] * M))
        out, lse = cache.attend(yq.view(M, heads, dim), table, i32([t + 1] * M), return_lse=True)
        y = lo.gemm(out.view(M, heads * dim))
        torch.cuda.synchronize()
        ks.append(ref.held(yk.cpu().numpy().reshape(M, kv_heads, dim), 4))
        vs.append(ref.held(yv.cpu().numpy().reshape(M, kv_heads, dim), 4))
        one = Case.__new__(Case)
        one.k, one.v = list(np.stack(ks, 1)), list(np.stack(vs, 1))
        one.lengths = [t + 1] * M
        one.check(out, lse, yq.cpu().numpy().reshape(M, heads, dim), dim ** -0.5, what="step %d" % t)
        assert y.shape == (M, K) and torch.all(torch.isfinite(y))
    for l in (lq, lk, lv, lo):
        l.close()


def test_binding_checks_tensors(exq):
    c = Case(exq, 21, [5, 5], 16, 2, 64, (4, 4))
    q = to_dev(values(c.rng, 2, 4, 64))
    n = i32([5, 5])
    k = to_dev(values(c.rng, 2, 2, 64))
    s, p = i32([0, 1]), i32([5, 5])
    bad = [
        lambda: c.cache.attend(q.float(), c.dtable, n), lambda: c.cache.attend(q.cpu(), c.dtable, n),
        lambda: c.cache.attend(q[:, :3], c.dtable, n), lambda: c.cache.attend(q[:, :, ::2], c.dtable, n),
        lambda: c.cache.attend(q, c.dtable.long(), n), lambda: c.cache.attend(q, c.dtable[:1], n),
        lambda: c.cache.attend(q, c.dtable, n.long()), lambda: c.cache.attend(q, c.dtable, n[:1]),
        lambda: c.cache.attend(q, c.dtable, n, out=q), lambda: c.cache.attend(q, c.dtable, n, window=-1),
        lambda: c.cache.attend(q, c.dtable, n, scale=float("nan")),
        lambda: c.cache.attend(q, c.dtable, n, lse=torch.zeros((2, 3), device="cuda")),
        lambda: c.cache.append(k, k[:1], c.dtable, s, p), lambda: c.cache.append(k, k, c.dtable, s, p.long()),
        lambda: c.cache.append(k, k.bfloat16(), c.dtable, s, p), lambda: c.cache.append(k, k, c.dtable.T, s, p),
        lambda: c.cache.read(c.dtable, s, p, k, k), lambda: c.cache.read(c.dtable, s, p, k[:1], None),
    ]
    before = c.cache.pages.clone()
    note("binding checks")
    for i, f in enumerate(bad):
        with pytest.raises(exq.ExqError) as ei:
            f()
        assert ei.value.status == exq.EXQ_ERR_INVALID_ARG, i
    assert torch.equal(before, c.cache.pages)
    e = torch.empty((0, 4, 64), dtype=torch.float16, device="cuda")
    assert c.cache.attend(e, c.dtable[:0], n[:0]).shape == (0, 4, 64)
    c.cache.append(e[:, :2], e[:, :2], c.dtable, s[:0], p[:0])
    assert c.cache.read(c.dtable, s[:0], p[:0])[0].shape == (0, 2, 64)
    c.cache.close()
    with pytest.raises(exq.ExqError):
        c.cache.attend(q, c.dtable, n)


class RoomFor:
    """GPU memory that has room for so many bytes more, by the allocator's own limit."""

    def __init__(self, nbytes):
        self.nbytes = nbytes

    def __enter__(self):
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        total = torch.cuda.get_device_properties(0).total_memory
        torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + self.nbytes) / total)

    def __exit__(self, *_):
        torch.cuda.set_per_process_memory_fraction(1.0)


def calls_without_room(exq):
    """(what, room, call): a read and an attend whose first output of 1 GiB fits while the second does not."""
    cache = exq.KVCache(1, 16, 8, 64, 4, 4)
    rows = 1 << 20
    out = rows * 8 * 64 * 2
    table, zeros = i32([[0]]), i32(np.zeros(rows))
    q = torch.zeros((1, 8, 64), dtype=torch.float16, device="cuda").expand(rows, 8, 64)
    return [("read", 1.5 * out, lambda: cache.read(table, zeros, zeros)),
            ("attend", out + out // 64, lambda: cache.attend(q, table.expand(rows, 1), zeros, return_lse=True))]


def test_calls_that_run_out_of_memory_keep_nothing(exq):
    for what, room, call in calls_without_room(exq):
        before = torch.cuda.memory_allocated()
        note("out of memory: %s" % what)
        with RoomFor(room), pytest.raises(RuntimeError):
            call()
        assert torch.cuda.memory_allocated() <= before, what   # (less: what earlier tests left to the garbage collector)


def test_running_out_of_memory_is_pytorchs_own_error(exq):
    """As from any other allocation: a program that frees something and tries again catches that type."""
    for what, room, call in calls_without_room(exq):
        note("out of memory: %s" % what)
        with RoomFor(room), pytest.raises(torch.OutOfMemoryError):
            call()


@pytest.mark.parametrize("call", ["append", "read", "attend"])
def test_tensors_dropped_after_a_call_on_another_stream_stay_until_it_is_through(exq, call):
    """Temporaries handed to a call that names a stream: their memory is not given out again while that stream has the call
    still before it."""
    c = Case(exq, 40, [2000, 700], 64, 2, 64, (4, 4))
    side = torch.cuda.Stream()
    half = lambda *shape: torch.ones(shape, dtype=torch.float16, device="cuda")
    places = lambda: [c.dtable.clone(), i32(np.zeros(300)), i32(np.arange(300))]
    need = exq.exq_attend_workspace_bytes(c.cache.handle, 2, 4, c.dtable.shape[1])
    assert need > 0
    if call == "append":
        args = [half(300, 2, 64), half(300, 2, 64)] + places()
        run = lambda x: c.cache.append(*x, stream=side)
    elif call == "read":
        args = places() + [half(300, 2, 64), half(300, 2, 64)]
        run = lambda x: c.cache.read(*x, stream=side)
    else:
        args = [half(2, 4, 64), c.dtable.clone(), i32(c.lengths), half(2, 4, 64), torch.ones((2, 4), device="cuda"),
                c.cache.workspace(need)]
        run = lambda x: c.cache.attend(*x[:3], out=x[3], lse=x[4], workspace=x[5], stream=side)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)
    note("temporaries on another stream: %s" % call)
    run(args)
    before = {x.data_ptr() for x in args}
    kinds = [(x.shape, x.dtype) for x in args]
    del args
    after = [torch.empty(shape, dtype=dtype, device="cuda").data_ptr() for shape, dtype in kinds]
    waiting = not side.query()
    torch.cuda.synchronize()
    assert not (waiting and before & set(after))


# ------------------------------------------------- long chunks, two tiles of heads, raw stream handles

@pytest.mark.parametrize("bits", [(4, 4), (16, 16)], ids=str)
def test_whole_rows_of_many_steps(exq, bits):
    """More than 256 rows are not split: a wave takes 157 steps of the longest one, three looks at the page table.  A page
    number that is none makes only the rows NaN that read it, past the second look too."""
    rows, lengths = 257, {0: 20000, 5: 8193, 100: 8000, 256: 16500}
    c = Case(exq, 41, [20000], 64, 1, 64, bits, spare=0)
    n = np.full(rows, -1)
    n[list(lengths)] = list(lengths.values())
    c.k, c.v = c.k * rows, c.v * rows
    q = values(c.rng, rows, 2, 64)
    note("whole rows of many steps bits=%s" % (bits,))
    out, lse = c.cache.attend(to_dev(q), c.dtable.expand(rows, -1), i32(n), return_lse=True)
    c.check(out, lse, q, 0.125, lengths=list(n))
    for bad in (8192 // 64, 16384 // 64 + 1, 19999 // 64):
        t = c.table.copy()
        t[0, bad] = c.cache.n_pages
        out, lse = c.cache.attend(to_dev(q), i32(t).expand(rows, -1), i32(n), return_lse=True)
        hit = [r for r, x in lengths.items() if x > 64 * bad]
        assert hit and torch.all(torch.isnan(out[hit])) and torch.all(torch.isnan(lse[hit]))
        c.check(out, lse, q, 0.125, lengths=[-1 if r in hit else x for r, x in enumerate(n)])


@pytest.mark.parametrize("bits,unit", [((8, 8), 256), ((16, 16), 128)], ids=str)
def test_chunks_of_more_steps_than_one_look_at_the_page_table(exq, bits, unit):
    """One row so long that each of its 32 chunks has 66 units.  Seven pages over and over; all but a few places show the
    five whose scores are near 0, those few, in the last two units of a chunk among others, the two whose scores are 16."""
    page, dim = 48, 128 if bits[0] == 16 else 64
    c = Case(exq, 42, [7 * page], page, 1, dim, bits, spare=0)
    k = c.rng.standard_normal((7 * page, 1, dim)).astype(np.float16) * np.float16(0.05)
    k[5 * page:] = 1
    v = values(c.rng, 7 * page, 1, dim, spread=0.5)
    ref.append(c.geo, c.pages, k, v, c.table, [0] * len(k), range(len(k)))
    c.cache.pages.copy_(to_dev(c.pages).view_as(c.cache.pages))
    k, v = ref.held(k, bits[0]).reshape(7, page, 1, dim), ref.held(v, bits[1]).reshape(7, page, 1, dim)
    n = 32 * 66 * unit - 37
    order = np.arange(-(-n // page)) % 5
    chunk = 66 * unit
    special = [3 * chunk + 64 * unit + 60, 20 * chunk + 65 * unit + 50, 31 * chunk + 65 * unit + 10, 9 * chunk + 100]
    q = np.ones((1, 2, dim), dtype=np.float16)
    q[0, 1, ::2] = 0.5
    note("long chunks bits=%s" % (bits,))
    for at in [special] + [[x] for x in special]:
        here = order.copy()
        here[[x // page for x in at]] = [5 + i % 2 for i in range(len(at))]
        one = Case.__new__(Case)
        one.k, one.v = [k[here].reshape(-1, 1, dim)], [v[here].reshape(-1, 1, dim)]
        out, lse = c.cache.attend(to_dev(q), i32(c.table[:, here]), i32([n]), scale=16 / dim, return_lse=True)
        one.check(out, lse, q, 16 / dim, lengths=[n], what="at %s" % at)


def test_two_tiles_of_heads_through_a_shared_workspace(exq):
    """17 to 32 query heads to a key-value head: two segments, each with parts of its own, between calls of one."""
    c = Case(exq, 43, [2500, 700], 64, 1, 64, (8, 8), spread=0.5, garbage=False, spare=300)
    ws = c.cache.workspace(exq.exq_attend_workspace_bytes(c.cache.handle, 2, 32, c.dtable.shape[1]))
    for heads in (32, 5, 17, 32):
        q = values(c.rng, 2, heads, 64, spread=0.5)
        for lens in ([2500, 700], [2100, -1], [0, 650]):
            note("two tiles of heads, heads=%d lengths=%s" % (heads, lens))
            out, lse = c.cache.attend(to_dev(q), c.dtable, i32(lens), return_lse=True, workspace=ws)
            one = Case.__new__(Case)
            one.k, one.v = [x[:max(n, 0)] for x, n in zip(c.k, lens)], [x[:max(n, 0)] for x, n in zip(c.v, lens)]
            one.check(out, lse, q, 0.125, lengths=lens, what="%d heads %s" % (heads, lens))
            assert torch.all(ws[:exq.ATTEND_COUNTER_BYTES] == 0)


def test_a_stream_may_be_a_raw_handle(exq):
    """0, the default stream's, and another stream's, for all three calls."""
    c = Case(exq, 44, [900], 64, 2, 64, (8, 4))
    q, n = to_dev(values(c.rng, 1, 4, 64)), i32([900])
    seqs, pos = i32(np.zeros(40)), i32(np.arange(40) + 3)
    want = c.cache.attend(q, c.dtable, n)
    k, v = c.cache.read(c.dtable, seqs, pos)
    other = torch.cuda.Stream()
    for handle in (0, other.cuda_stream):
        torch.cuda.synchronize()
        note("raw stream handle")
        c.cache.append(k, v, c.dtable, seqs, pos, stream=handle)
        got = c.cache.read(c.dtable, seqs, pos, stream=handle)
        out = c.cache.attend(q, c.dtable, n, stream=handle)
        torch.cuda.synchronize()
        # (what was read back is written and read back again: a value's code and its group's scale may move by a rounding)
        assert torch.equal(out, c.cache.attend(q, c.dtable, n))
        assert all(torch.equal(a, b) for a, b in zip(got, c.cache.read(c.dtable, seqs, pos)))
    assert want.shape == out.shape


def test_a_captured_step_may_name_its_stream(exq):
    """append, read and attend captured with the capturing stream named, temporaries among their arguments; two graphs in
    turn, eager calls between."""
    c = Case(exq, 45, [700, 1500], 64, 2, 64, (4, 8), spare=10)
    q, k, v = (torch.zeros((2, h, 64), dtype=torch.float16, device="cuda") for h in (6, 2, 2))
    seqs, pos, n = i32([0, 1]), i32([700, 1500]), i32([701, 1501])
    assert exq.exq_attend_workspace_bytes(c.cache.handle, 2, 6, c.dtable.shape[1]) > 0

    def step(stream=None):
        c.cache.append(k.clone(), v.clone(), c.dtable, seqs, pos, stream=stream)
        return c.cache.read(c.dtable, seqs, pos, stream=stream) + c.cache.attend(q.clone(), c.dtable, n, return_lse=True, stream=stream)

    step()
    torch.cuda.synchronize()
    note("capture with a named stream")
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, step(torch.cuda.current_stream())))
    for rep in range(6):
        g, got = graphs[rep % 2]
        for x, h in ((q, 6), (k, 2), (v, 2)):
            x.copy_(to_dev(values(c.rng, 2, h, 64)))
        g.replay()
        torch.cuda.synchronize()
        want = step()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), rep
        torch.cuda.synchronize()
