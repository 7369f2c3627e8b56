"""Key-value cache on the CPU: sizes, argument checks of every entry point, and the reference's own pins.

No test here launches a kernel; addresses are made up and never dereferenced."""
import ctypes

import numpy as np
import pytest

import mixed_bitrate_quantized_amd as exq
from oracle import cacheref as ref

FAKE = 1 << 20


def expect(status, fn, *args, **kw):
    with pytest.raises(exq.ExqError) as ei:
        fn(*args, **kw)
    assert ei.value.status == status, ei.value
    assert exq.lib.exq_last_error() != b""


@pytest.mark.parametrize("dim", [64, 96, 128, 256])
@pytest.mark.parametrize("bits", [(4, 4), (8, 8), (8, 4), (4, 8), (16, 16)])
def test_page_bytes_and_layout_tile_every_byte_once(dim, bits):
    """Every byte of a tile belongs to exactly one (part, token): codes and scales cover it without overlap."""
    geo = ref.Geometry(32, 3, dim, *bits)
    assert exq.exq_cache_page_bytes(32, 3, dim, *bits) == geo.page_bytes
    owner = np.full(geo.tile_bytes * 8, -1, dtype=np.int64)
    for part in (0, 1):
        b = geo.bits[part]
        for t in range(16):
            for first, width in [(geo.code_bit(part, t, np.arange(dim)), b)] + (
                    [(8 * geo.scale_byte(part, t, np.arange(dim // 32)), 16)] if b < 16 else []):
                for x in first:
                    assert np.all(owner[x:x + width] == -1)
                    owner[x:x + width] = 2 * t + part
    assert np.all(owner >= 0)
    byte = owner.reshape(-1, 8)
    assert np.all(byte == byte[:, :1])   # no byte is shared by two tokens


def test_page_bytes_rejects():
    assert exq.exq_cache_page_bytes(256, 8, 128, 4, 4) == 256 * 8 * 144
    for bad in [(0, 8, 128, 4, 4), (24, 8, 128, 4, 4), (65552, 8, 128, 4, 4), (16, 0, 128, 4, 4), (16, 1 << 16, 128, 4, 4),
                (16, 8, 0, 4, 4), (16, 8, 100, 4, 4), (16, 8, 160, 4, 4), (16, 8, 128, 5, 4), (16, 8, 128, 16, 8),
                (16, 8, 128, 4, 16)]:
        assert exq.exq_cache_page_bytes(*bad) == 0


def test_create_rejects():
    I, U = exq.EXQ_ERR_INVALID_ARG, exq.EXQ_ERR_UNSUPPORTED
    expect(I, exq.exq_cache_create, None, 4, 16, 8, 128, 4, 4)
    expect(I, exq.exq_cache_create, FAKE + 8, 4, 16, 8, 128, 4, 4)
    expect(I, exq.exq_cache_create, FAKE, 0, 16, 8, 128, 4, 4)
    expect(I, exq.exq_cache_create, FAKE, 1 << 31, 16, 8, 128, 4, 4)
    expect(I, exq.exq_cache_create, FAKE, 4, 20, 8, 128, 4, 4)
    expect(U, exq.exq_cache_create, FAKE, 4, 16, 8, 192, 4, 4)
    expect(U, exq.exq_cache_create, FAKE, 4, 16, 8, 128, 3, 4)
    expect(U, exq.exq_cache_create, FAKE, 1 << 29, 16, 8, 128, 4, 4)        # 2^32 tiles
    exq.exq_cache_destroy(exq.exq_cache_create(FAKE, (1 << 29) - 1, 16, 8, 128, 4, 4))
    assert exq.lib.exq_cache_create(FAKE, 4, 16, 8, 128, 4, 4, None) == I
    exq.exq_cache_destroy(None)


@pytest.fixture()
def cache():
    h = exq.exq_cache_create(FAKE, 10, 32, 4, 64, 4, 8)
    yield h
    exq.exq_cache_destroy(h)


SIZE = 10 * 32 * 4 * (32 + 4 + 64 + 4)
K, V = FAKE + 2 * SIZE, FAKE + 4 * SIZE
T, S, P = 1 << 10, 1 << 11, 1 << 12


def rows_args(**kw):
    a = dict(k=K, ks=(256, 64), v=V, vs=(256, 64), rows=5, table=T, trows=3, width=4, tstride=4, seqs=S, pos=P)
    a.update(kw)
    return [a["k"], a["ks"], a["v"], a["vs"], a["rows"], a["table"], a["trows"], a["width"], a["tstride"], a["seqs"],
            a["pos"], 0]


BAD_ROWS = [dict(k=0), dict(v=0), dict(k=K + 2), dict(v=V + 8), dict(ks=(260, 64)), dict(vs=(256, 4)), dict(ks=(-256, 64)),
            dict(ks=((1 << 30) + 8, 64)), dict(rows=-1), dict(table=0), dict(table=T + 2), dict(trows=0), dict(width=0),
            dict(tstride=3), dict(tstride=-4), dict(seqs=0), dict(pos=0), dict(seqs=S + 1), dict(pos=P + 2),
            dict(k=FAKE + SIZE - 16), dict(v=FAKE), dict(k=FAKE - 16)]


@pytest.mark.parametrize("bad", BAD_ROWS, ids=str)
def test_append_and_read_reject(cache, bad):
    expect(exq.EXQ_ERR_INVALID_ARG, exq.exq_cache_append, cache, *rows_args(**bad))
    expect(exq.EXQ_ERR_INVALID_ARG, exq.exq_cache_read, cache, *rows_args(**bad))


@pytest.mark.parametrize("bad", [dict(ks=(0, 64)), dict(ks=(128, 64)), dict(vs=(256, 32)), dict(v=K), dict(v=K + 512),
                                 dict(ks=(256, 0))], ids=str)
def test_read_rejects_overlapping_outputs(cache, bad):
    expect(exq.EXQ_ERR_INVALID_ARG, exq.exq_cache_read, cache, *rows_args(**bad))


def test_rows_calls_reject_null_cache_and_too_many_rows(cache):
    expect(exq.EXQ_ERR_INVALID_ARG, exq.exq_cache_append, None, *rows_args())
    expect(exq.EXQ_ERR_INVALID_ARG, exq.exq_cache_read, None, *rows_args())
    big = exq.exq_cache_create(FAKE, 1, 16, 65535, 64, 4, 4)
    far = 1 << 50
    expect(exq.EXQ_ERR_UNSUPPORTED, exq.exq_cache_append, big, *rows_args(k=far, v=far, ks=(0, 0), vs=(0, 0), rows=1 << 20))
    exq.exq_cache_destroy(big)


def test_no_rows_is_a_no_op(cache):
    """Nothing is launched for no rows: this succeeds without a GPU."""
    exq.exq_cache_append(cache, *rows_args(rows=0))
    exq.exq_cache_read(cache, *rows_args(rows=0))
    exq.exq_attend(cache, *attend_args(rows=0)[:-1], stream=0)


@pytest.mark.parametrize("table", [dict(table=0, trows=0, tstride=0), dict(table=0, trows=0, width=0, tstride=0), dict(trows=0),
                                   dict(k=0, v=0, seqs=0, pos=0)], ids=str)
def test_no_rows_is_a_no_op_with_an_empty_table_too(cache, table):
    """A step without rows hands over empty tensors, whose pointers are NULL."""
    exq.exq_cache_append(cache, *rows_args(rows=0, **table))
    exq.exq_cache_read(cache, *rows_args(rows=0, **table))
    for bad in (dict(trows=-1), dict(width=-1)):
        expect(exq.EXQ_ERR_INVALID_ARG, exq.exq_cache_append, cache, *rows_args(rows=0, **{**table, **bad}))
        expect(exq.EXQ_ERR_INVALID_ARG, exq.exq_cache_read, cache, *rows_args(rows=0, **{**table, **bad}))


def test_attend_of_no_rows_with_an_empty_table(cache):
    for width in (400, 0):
        exq.exq_attend(cache, *attend_args(rows=0, table=0, width=width, tstride=0, q=0, out=0, lse=0, lengths=0, ws=0, wsb=0)[:-1],
                       stream=0)
        assert exq.exq_attend_workspace_bytes(cache, 0, 8, width) == 0
    expect(exq.EXQ_ERR_INVALID_ARG, exq.exq_attend, cache, *attend_args(rows=0, width=-1))


@pytest.mark.parametrize("over", [dict(table=K), dict(table=V + 64), dict(table=K - 4), dict(seqs=K + 128), dict(pos=V), dict(pos=K - 16),
                                  dict(table=K - 4 * 100, trows=2, tstride=100)], ids=str)
def test_read_rejects_outputs_over_its_own_indices(cache, over):
    expect(exq.EXQ_ERR_INVALID_ARG, exq.exq_cache_read, cache, *rows_args(**over))


@pytest.mark.parametrize("over", [dict(table=FAKE), dict(table=FAKE - 44), dict(seqs=FAKE + SIZE - 4), dict(pos=FAKE - 4),
                                  dict(table=FAKE - 4 * 100, trows=2, tstride=100)], ids=str)
def test_append_rejects_indices_in_the_pages(cache, over):
    expect(exq.EXQ_ERR_INVALID_ARG, exq.exq_cache_append, cache, *rows_args(**over))


Q, O, L, W = FAKE + 2 * SIZE, FAKE + 4 * SIZE, FAKE + 6 * SIZE, 1 << 40


def attend_args(**kw):
    a = dict(q=Q, qs=(512, 64), rows=3, heads=8, table=T, width=400, tstride=400, lengths=S, scale=0.125, window=0, out=O,
             os=(512, 64), lse=L, ws=W, wsb=1 << 30)
    a.update(kw)
    return [a["q"], a["qs"], a["rows"], a["heads"], a["table"], a["width"], a["tstride"], a["lengths"], a["scale"],
            a["window"], a["out"], a["os"], a["lse"], a["ws"], a["wsb"], 0]


BAD_ATTEND = [dict(q=0), dict(q=Q + 4), dict(qs=(508, 64)), dict(qs=(512, -8)), dict(rows=-1), dict(heads=0), dict(heads=6),
              dict(heads=-4), dict(table=0), dict(width=0), dict(tstride=399), dict(lengths=0), dict(lengths=S + 2),
              dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38), dict(window=-1), dict(out=0), dict(out=O + 2),
              dict(os=(0, 64)), dict(os=(512, 32)), dict(out=Q), dict(out=Q + 64), dict(out=FAKE), dict(lse=L + 2),
              dict(lse=O), dict(lse=Q), dict(lse=FAKE + 64), dict(ws=0), dict(ws=W + 8), dict(wsb=100), dict(ws=O), dict(ws=Q),
              dict(ws=FAKE), dict(ws=L)]


@pytest.mark.parametrize("bad", BAD_ATTEND, ids=str)
def test_attend_rejects(cache, bad):
    expect(exq.EXQ_ERR_INVALID_ARG, exq.exq_attend, cache, *attend_args(**bad))


@pytest.mark.parametrize("over", [
    dict(table=O), dict(table=O - 4796), dict(table=L), dict(table=W + 64), dict(table=O - 8000, tstride=2000), dict(lengths=O + 3064),
    dict(lengths=O - 8), dict(lengths=L + 4), dict(lengths=W), dict(lengths=L - 8)], ids=str)
def test_attend_rejects_outputs_and_a_workspace_over_its_table_or_lengths(cache, over):
    """Workgroups of one launch read the lengths and the table while others write."""
    expect(exq.EXQ_ERR_INVALID_ARG, exq.exq_attend, cache, *attend_args(**over))


def test_attend_rejects_null_cache_and_too_many_rows(cache):
    expect(exq.EXQ_ERR_INVALID_ARG, exq.exq_attend, None, *attend_args())
    expect(exq.EXQ_ERR_UNSUPPORTED, exq.exq_attend, cache, *attend_args(rows=(1 << 31) - 1, heads=64))
    expect(exq.EXQ_ERR_UNSUPPORTED, exq.exq_attend, cache, *attend_args(rows=1 << 22, heads=4))    # 2^24 workgroups of 256
    assert exq.exq_attend_workspace_bytes(None, 1, 8, 4) == 0
    assert exq.exq_attend_workspace_bytes(cache, 1, 6, 4) == 0
    assert exq.exq_attend_workspace_bytes(cache, 1, 8, 0) == 0


def test_workspace_is_bounded_and_grows_with_the_split(cache):
    one = exq.exq_attend_workspace_bytes(cache, 1, 8, 1)        # 32 tokens: nothing to split
    assert one == 0
    sizes = [exq.exq_attend_workspace_bytes(cache, r, 8, w) for r, w in ((1, 1000), (16, 1000), (256, 1 << 20))]
    assert 0 < sizes[0] <= sizes[1] <= sizes[2] < 1 << 28
    assert exq.exq_attend_workspace_bytes(cache, 4096, 8, 1 << 20) == 0      # rows enough to load the card unsplit
    for rows in (1, 16, 256, 257, 1 << 20):
        assert exq.exq_attend_workspace_bytes(cache, rows, 8, (1 << 31) - 1) < 1 << 28


def test_reference_reads_back_what_it_appends():
    rng = np.random.default_rng(1)
    for bits in [(4, 4), (8, 4), (16, 16)]:
        geo = ref.Geometry(16, 2, 96, *bits)
        pages = rng.integers(0, 256, 3 * geo.page_bytes).astype(np.uint8)
        before = pages.copy()
        table = np.array([[2, 0]], dtype=np.int32)
        k = rng.standard_normal((2, 2, 96)).astype(np.float16)
        v = rng.standard_normal((2, 2, 96)).astype(np.float16)
        ref.append(geo, pages, k, v, table, [0, -1], [21, 3])
        for h in range(2):
            a, b = ref.read_token(geo, pages, 0, 5, h)
            np.testing.assert_array_equal(a, ref.held(k[0, h], bits[0]))
            np.testing.assert_array_equal(b, ref.held(v[0, h], bits[1]))
        assert (pages != before).sum() <= 2 * geo.tile_bytes // 16
        np.testing.assert_array_equal(pages[geo.page_bytes:], before[geo.page_bytes:])


def test_reference_quantizer_pins():
    x = np.zeros(64, dtype=np.float16)
    x[:4] = [7.0, -3.5, 2.5, 0.5]       # scale 1: ties go to the even code
    c, s = ref.quantize(x, 4)
    assert list(c[:5]) == [15, 4, 10, 8, 8] and s[0] == 1 and s[1] == 0 and np.all(c[32:] == 8)
    x[40] = np.inf
    assert np.all(np.isnan(ref.held(x, 8)[32:])) and np.all(np.isfinite(ref.held(x, 8)[:32]))
    y = np.linspace(-2, 2, 32).astype(np.float16)
    for b in (4, 8):
        s = np.float64(ref.quantize(y, b)[1][0])
        # half a step, and the scale's and the product's roundings to fp16
        assert np.max(np.abs(ref.held(y, b).astype(np.float64) - y.astype(np.float64))) <= s / 2 + 2 * 2.0 ** -11 * 2


def test_reference_keeps_finite_values_finite():
    x = np.repeat(np.arange(0x7C00, dtype=np.uint16).view(np.float16)[:, None], 32, 1)
    for b in (4, 8):
        assert np.all(np.isfinite(ref.held(x, b))) and np.all(ref.held(x, b)[-1] == 65472)


def test_kvcache_checks_tensors_before_the_library():
    torch = pytest.importorskip("torch")
    with pytest.raises(exq.ExqError):
        exq.KVCache(4, 16, 2, 64, pages=torch.zeros(4, 16 * 2 * 72, dtype=torch.uint8))       # not on the GPU
    with pytest.raises(exq.ExqError) as ei:
        exq.KVCache(4, 17, 2, 64, device="cpu")
    assert ei.value.status == exq.EXQ_ERR_INVALID_ARG


def test_tensor_calls_refuse_before_the_library(cache):
    """The checks of tensors (_exq_torch) with CPU tensors: every one is refused with the package's own error."""
    torch = pytest.importorskip("torch")
    calls = exq._tensor_calls()
    head = (cache, 4, 64, 0, 0)
    k = torch.zeros((3, 4, 64), dtype=torch.float16)
    t = torch.zeros((3, 2), dtype=torch.int32)
    n = torch.zeros(3, dtype=torch.int32)
    I = exq.EXQ_ERR_INVALID_ARG
    for bad in ((k, k, t, n, n), (k[0, 0, 0], k, t, n, n), (None, k, t, n, n), (k, 3, t, n, n)):
        expect_call(I, calls.append, *head, *bad)
    for bad in ((t, n, n, None, None), (t, t, n, None, None), (None, n, n, None, None), (t, "n", n, k, k)):
        expect_call(I, calls.read, *head, *bad)
    q = torch.zeros((3, 8, 64), dtype=torch.float16)
    for bad in ((q, t, n), (q[0], t, n), (None, t, n), (q, n, n), (q, t, None)):
        expect_call(I, calls.attend, *head, *bad, 0.125, 0, None, False, None, None, None)
    expect_call(I, calls.attend, *head, q, t, n, 0.125, 1 << 40, None, False, None, None, None)
    for wrong in ((calls.append, head), (calls.read, head + (t,)), (calls.attend, head + (q,))):
        with pytest.raises(TypeError):
            wrong[0](*wrong[1])
    with pytest.raises(TypeError):
        calls.append("cache", 4, 64, 0, 0, k, k, t, n, n)
    with pytest.raises(TypeError):
        calls.attend(*head, q, t, n, "scale", 0, None, False, None, None, None)


def test_a_return_lse_without_a_truth_value_is_the_callers_error(cache):
    """Its error reaches the caller before anything is looked at or launched."""
    torch = pytest.importorskip("torch")
    calls = exq._tensor_calls()
    q = torch.zeros((3, 8, 64), dtype=torch.float16)
    t = torch.zeros((3, 2), dtype=torch.int32)
    with pytest.raises(ValueError):
        calls.attend(cache, 4, 64, 0, 0, q, t, t[:, 0], 0.125, 0, None, np.zeros(2), None, None, None)


def test_a_stream_of_another_device_is_refused():
    """A call that names a stream runs on it or not at all."""
    torch = pytest.importorskip("torch")

    class Stream:
        cuda_stream, device = 64, torch.device("cuda", 1)

    expect(exq.EXQ_ERR_INVALID_ARG, exq._on, Stream(), torch.device("cuda", 0))


def test_a_stream_handle_may_be_any_integer(monkeypatch):
    """numpy's integers have a device too, which is none of a stream's."""
    torch = pytest.importorskip("torch")

    class Reached(Exception):
        pass

    def device(_):
        raise Reached

    monkeypatch.setattr(torch.cuda, "device", device)
    for handle in (64, np.int64(64), np.uint64(64)):
        with pytest.raises(Reached):
            exq._on(handle, torch.device("cuda", 0))


def expect_call(status, fn, *args):
    with pytest.raises(exq.ExqError) as ei:
        fn(*args)
    assert ei.value.status == status
