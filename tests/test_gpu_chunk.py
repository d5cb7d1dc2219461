"""Attention of a chunk of new tokens over a paged cache against the plain 64-bit form, at the sizes and masks where it
can go wrong."""

import math

import numpy as np
import pytest
import torch

import chunk_ref as C
import block_ref as R
from test_gpu_attention import make_pages, poison, tables_for

pytestmark = pytest.mark.gpu

M = pytest.importorskip("w4a16_int4_mixture_grouped_gb300") if torch.cuda.is_available() else None
DEV = torch.device("cuda", 0) if torch.cuda.is_available() else None
BAD_INDEX, TIMEOUT = 8, 6


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def queries(rng, t, h, d, scale=1.0):
    return torch.from_numpy((rng.standard_normal((t, h, d)) * scale).astype(np.float32)).to(DEV).to(torch.bfloat16)


def starts_of(counts):
    return [0] + [int(x) for x in np.cumsum(counts)]


def compare(out, lse, ref, bound, rl, lb, rows=None):
    got, gl = out.double(), lse.double()
    if rows is not None:
        got, gl, ref, bound, rl, lb = got[rows], gl[rows], ref[rows], bound[rows], rl[rows], lb[rows]
    assert torch.isfinite(got).all()
    err = (got - ref).abs()
    assert (err <= bound).all(), f"out: {(err / bound.clamp(min=1e-300)).max().item()} of the bound"
    empty = rl == -math.inf
    assert torch.equal(gl == -math.inf, empty)
    assert (got[empty] == 0).all()
    d = (gl - rl).abs()[~empty]
    assert (d <= lb[~empty]).all(), f"lse: {(d / lb[~empty]).max().item()} of the bound"


def check(q, starts, k, v, tables, lens, scale=None, window=0, ks=1.0, vs=1.0, seq_ids=None, ws=None, want_err=0):
    t, h, d = q.shape
    scale = d ** -0.5 if scale is None else scale
    ws = ws if ws is not None else M.paged_chunk_workspace(h, k.shape[2], d)
    out = torch.full((t, h, d), 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((t, h), 7.0, dtype=torch.float32, device=DEV)
    M.paged_chunk_attention(q, i32(starts), k, v, i32(tables), i32(lens), ws, scale=scale, window=window, k_scale=ks,
                            v_scale=vs, seq_ids=None if seq_ids is None else i32(seq_ids), out=out, lse=lse)
    assert M.get_device_error(ws) == want_err
    ref = C.attention(q, starts, k, v, tables, lens, scale, window, ks, vs, seq_ids)
    mine = ~torch.isnan(ref[0][:, 0, 0])
    compare(out, lse, *ref, rows=mine)
    assert (out[~mine] == 7.0).all() and (lse[~mine] == 7.0).all()        # rows of no chunk: as they were
    return out, lse


# (new tokens, length with them); the last two: chunks longer than their sequences
CHUNKS = [(1, 1), (0, 50), (5, 5), (3, 130), (17, 17), (1, 300), (40, 333), (130, 130), (70, 190), (9, 4), (2, 0)]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dim,group,hkv,page", [(128, 4, 2, 16), (128, 8, 1, 64), (64, 1, 3, 32), (96, 5, 2, 48),
                                                (256, 2, 2, 16), (128, 16, 1, 1), (16, 3, 1, 7), (112, 20, 1, 40),
                                                (64, 33, 1, 128), (240, 9, 1, 24), (80, 12, 1, 200), (192, 1, 2, 64),
                                                (32, 130, 1, 16), (128, 257, 1, 64)])
def test_ragged_chunks(dim, group, hkv, page, e4m3):
    rng = np.random.default_rng(dim * 100 + group + e4m3)
    lens = [n for _, n in CHUNKS]
    tables, total = tables_for(rng, lens, page)
    k, v = make_pages(rng, total, page, hkv, dim, e4m3)
    poison(k, tables, lens, page)
    poison(v, tables, lens, page)
    starts = starts_of([n for n, _ in CHUNKS])
    ks, vs = (0.75, 1.5) if e4m3 else (1.0, 1.0)
    check(queries(rng, starts[-1], group * hkv, dim, 1.5), starts, k, v, tables, lens, ks=ks, vs=vs)


@pytest.mark.parametrize("window", [1, 5, 16, 100, 128, 200, 1000])
@pytest.mark.parametrize("e4m3,dim", [(False, 64), (True, 64), (False, 256)])
def test_window_with_the_pages_behind_it_freed(window, e4m3, dim):
    rng = np.random.default_rng(window)
    page, chunks = 16, [(1, 1), (5, 16), (17, 17), (99, 99), (100, 333), (1, 250), (300, 301)]
    lens = [n for _, n in chunks]
    tables, total = tables_for(rng, lens, page)
    for i, (c, n) in enumerate(chunks):
        tables[i, :max(0, n - c + 1 - window) // page] = -1
    k, v = make_pages(rng, total, page, 2, dim, e4m3)
    poison(k, tables, lens, page)
    poison(v, tables, lens, page)
    starts = starts_of([c for c, _ in chunks])
    check(queries(rng, starts[-1], 8, dim), starts, k, v, tables, lens, window=window)


@pytest.mark.parametrize("e4m3,dim", [(False, 128), (True, 128), (False, 256), (True, 256)])
def test_holes_in_the_table_and_rows_that_see_nothing(e4m3, dim):
    rng = np.random.default_rng(5)
    page, chunks = 16, [(50, 100), (30, 100), (64, 64), (16, 16), (20, 400)]
    lens = [n for _, n in chunks]
    tables, total = tables_for(rng, lens, page)
    tables[0, [0, 3, 6]] = -1            # freed here and there, the last page too
    tables[1, :] = -1                    # nothing left
    tables[2, :2] = -1                   # the chunk's first rows see nothing
    tables[3, 0] = -7                    # any negative entry is no page
    tables[4, 2:20] = -1                 # whole tiles of tokens
    k, v = make_pages(rng, total, page, 2, dim, e4m3)
    poison(k, tables, lens, page)
    poison(v, tables, lens, page)
    starts = starts_of([c for c, _ in chunks])
    check(queries(rng, starts[-1], 8, dim), starts, k, v, tables, lens)


def test_bad_ids_lengths_and_starts_are_skipped_and_recorded():
    rng = np.random.default_rng(6)
    page, lens = 16, [40, 33, 20]
    tables, total = tables_for(rng, lens, page, width=4)
    k, v = make_pages(rng, total, page, 1, 64, False)
    q = queries(rng, 30, 4, 64)
    starts = [0, 10, 22, 30]
    bad = tables.copy()
    bad[1, 1] = total                                            # past the pool
    check(q, starts, k, v, bad, lens, want_err=BAD_INDEX)
    check(q, starts, k, v, tables, [40, 33, -4], want_err=BAD_INDEX)
    full, total = tables_for(rng, [64, 64, 64], page, width=4)
    k, v = make_pages(rng, total, page, 1, 64, False)
    check(q, starts, k, v, full, [64, 1000, 30], want_err=BAD_INDEX)   # cut to the table's 64 tokens
    check(q, starts, k, v, full, [64, 64, 64], seq_ids=[2, 0, 1])
    check(q, starts, k, v, full, [64, 64, 64], seq_ids=[2, 3, -1], want_err=BAD_INDEX)
    for odd in ([0, 10, 22, 31], [-1, 10, 22, 30], [0, 22, 10, 30], [40, 50, 60, 70]):
        ws = M.paged_chunk_workspace(4, 1, 64)
        out = torch.full((30, 4, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        M.paged_chunk_attention(q, i32(odd), k, v, i32(full), i32([64, 64, 64]), ws, out=out)
        assert M.get_device_error(ws) == BAD_INDEX
        held = set()
        for a, b in zip(odd, odd[1:]):
            if 0 <= a <= b <= 30:
                held |= set(range(a, b))
        for t in range(30):
            assert (out[t] == 7.0).all().item() == (t not in held)


@pytest.mark.parametrize("first,last", [(0, 0), (3, 0), (0, 5), (4, 9)])
def test_rows_before_and_behind_the_chunks_stay(first, last):
    rng = np.random.default_rng(first + last)
    page, chunks = 32, [(20, 77), (0, 3), (45, 200)]
    lens = [n for _, n in chunks]
    tables, total = tables_for(rng, lens, page)
    k, v = make_pages(rng, total, page, 2, 128, False)
    starts = [first + x for x in starts_of([c for c, _ in chunks])]
    q = queries(rng, starts[-1] + last, 8, 128)
    q[:first], q[starts[-1]:] = math.nan, math.nan
    check(q, starts, k, v, tables, lens)


@pytest.mark.parametrize("e4m3", [False, True])
def test_strides_head_major_pages_and_query_slices(e4m3):
    rng = np.random.default_rng(7)
    page, chunks = 32, [(40, 77), (3, 3), (33, 200)]
    lens = [n for _, n in chunks]
    tables, total = tables_for(rng, lens, page)
    k, v = make_pages(rng, total, page, 4, 128, e4m3, head_major=True)
    starts = starts_of([c for c, _ in chunks])
    qkv = queries(rng, starts[-1], 24, 128)
    q = qkv[:, 2:18]                     # rows of a wider projection
    check(q, starts, k, v, tables, lens)
    wide = np.full((3, tables.shape[1] + 5), 10 ** 6, dtype=np.int32)
    wide[:, :tables.shape[1]] = tables
    ws = M.paged_chunk_workspace(16, 4, 128)
    a, la = M.paged_chunk_attention(q, i32(starts), k, v, i32(wide)[:, :tables.shape[1]], i32(lens), ws)
    b, lb = M.paged_chunk_attention(q.contiguous(), i32(starts), k, v, i32(tables), i32(lens), ws)
    assert torch.equal(a, b) and torch.equal(la, lb) and M.get_device_error(ws) == 0
    # a pool whose tokens lie apart, keys and values interleaved
    pool = torch.zeros((total, page, 4, 2, 128), dtype=k.dtype, device=DEV)
    pool.view(torch.uint8)[:, :, :, 0] = k.contiguous().view(torch.uint8).view(total, page, 4, -1)
    pool.view(torch.uint8)[:, :, :, 1] = v.contiguous().view(torch.uint8).view(total, page, 4, -1)
    c, lc = M.paged_chunk_attention(q, i32(starts), pool[:, :, :, 0], pool[:, :, :, 1], i32(tables), i32(lens), ws)
    assert torch.equal(a, c) and torch.equal(la, lc)


@pytest.mark.parametrize("batch,new,top,hkv,group", [(1, 3, 20011, 1, 8), (1, 40, 9000, 8, 4), (3, 300, 5000, 2, 16),
                                                      (200, 3, 90, 2, 2), (700, 1, 3, 1, 1), (1, 1000, 1000, 1, 1),
                                                      (2, 700, 2000, 2, 7)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_long_rows_are_split_and_joined(batch, new, top, hkv, group, e4m3):
    rng = np.random.default_rng(batch + top)
    page = 64
    counts = [new] + [int(x) for x in rng.integers(0, new + 1, batch - 1)]
    lens = [top] + [int(x) for x in rng.integers(0, top + 1, batch - 1)]
    tables, total = tables_for(rng, lens, page)
    k, v = make_pages(rng, total, page, hkv, 64, e4m3)
    starts = starts_of(counts)
    q = queries(rng, starts[-1], group * hkv, 64, 2.0)
    ws = M.paged_chunk_workspace(group * hkv, hkv, 64)
    a, la = check(q, starts, k, v, tables, lens, ws=ws)
    for _ in range(3):                   # the same workspace again: the same bits
        b, lb = M.paged_chunk_attention(q, i32(starts), k, v, i32(tables), i32(lens), ws)
        rows = starts[-1]
        assert torch.equal(a[:rows], b[:rows]) and torch.equal(la[:rows], lb[:rows])


@pytest.mark.parametrize("dim,e4m3", [(128, False), (128, True), (64, False), (256, False), (256, True)])
def test_many_chunks_of_odd_and_even_numbers_of_tiles(dim, e4m3):
    """Batches whose rows' tiles are shared by both halves of a CTA, beside ones that are not, over pages that come from
    HBM: no tile may be taken for another one's."""
    rng = np.random.default_rng(dim + e4m3)
    page, batch = 64, 40
    for most in (4, 300):
        chunks = [(int(rng.integers(1, most)) if rng.random() < 0.4 else 1, 0) for _ in range(batch)]
        chunks = [(c, c + int(rng.integers(0, 3000))) for c, _ in chunks]
        lens = [n for _, n in chunks]
        tables, total = tables_for(rng, lens, page)
        k, v = make_pages(rng, total, page, 4, dim, e4m3)
        starts = starts_of([c for c, _ in chunks])
        check(queries(rng, starts[-1], 16, dim, 1.5), starts, k, v, tables, lens)


@pytest.mark.parametrize("dim,e4m3", [(128, False), (128, True), (256, False), (256, True), (96, False)])
def test_wide_heads_split_and_joined(dim, e4m3):
    rng = np.random.default_rng(dim)
    page, chunks = 48, [(2, 6000), (150, 2500), (260, 260)]
    lens = [n for _, n in chunks]
    tables, total = tables_for(rng, lens, page)
    k, v = make_pages(rng, total, page, 2, dim, e4m3)
    starts = starts_of([c for c, _ in chunks])
    check(queries(rng, starts[-1], 10, dim, 1.5), starts, k, v, tables, lens)


@pytest.mark.parametrize("dim", [64, 256])
def test_scores_far_apart_and_scales(dim):
    """One token's score far above the others, in the first, a middle and the last tile; large and tiny scales."""
    rng = np.random.default_rng(8)
    page, lens, n = 16, [1000, 1000, 1000], 9
    tables, total = tables_for(rng, lens, page)
    k, v = make_pages(rng, total, page, 1, dim, False)
    q = queries(rng, 3 * n, 8, dim)
    for i, j in enumerate((0, 517, 999)):
        k[tables[i, j // page], j % page, 0] = (q[i * n + n - 1, 3].float() * 40).to(torch.bfloat16)
    for scale in (0.125, 4.0, 1e-4, -0.125, 0.0):
        check(q, [0, n, 2 * n, 3 * n], k, v, tables, lens, scale=scale)


@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("e4m3", [False, True])
def test_scores_that_rise_and_fall(e4m3, dim):
    """Scores that climb by a little from token to token, up to 2^40 of the first probabilities, and come down again:
    whatever the exponents are taken against has to follow."""
    rng = np.random.default_rng(31)
    page, n, new = 16, 1500, 200
    tables, total = tables_for(rng, [n, n], page)
    k, v = make_pages(rng, total, page, 1, dim, e4m3)
    q = queries(rng, 2 * new, 4, dim)
    steps = torch.from_numpy(np.concatenate([np.linspace(0.0, 1.0, 900), np.linspace(1.0, 0.2, n - 900)]).astype(np.float32)).to(DEV)
    for b in range(2):
        one = q[b * new, 0].float() / q[b * new, 0].float().norm()
        for j in range(n):
            k[tables[b, j // page], j % page, 0] = (one * steps[j] * 28.0).to(k.dtype)
        q[b * new:(b + 1) * new] = one.to(torch.bfloat16)
    check(q, [0, new, 2 * new], k, v, tables, [n, n], scale=1.0)


def test_wide_range_of_queries_over_an_8_bit_cache():
    """Queries far above and below the FP16 range: each row is scaled by its own power of two."""
    rng = np.random.default_rng(9)
    page, lens = 16, [50]
    tables, total = tables_for(rng, lens, page)
    k, v = make_pages(rng, total, page, 1, 64, True)
    for power in (40, -40):
        check(queries(rng, 6, 8, 64) * 2.0 ** power, [0, 6], k, v, tables, lens, scale=2.0 ** (-3 - power))
    q = queries(rng, 6, 8, 64)
    q[2, 1] = 0
    q[3] *= 2.0 ** 60
    q[4] *= 2.0 ** -60
    check(q, [0, 6], k, v, tables, lens, scale=2.0 ** -63)


def test_channels_far_apart_within_a_query_over_an_8_bit_cache():
    """One channel of each query far above the others and met by keys of zero, so that the small ones decide: they keep
    their bits down to 2^-32 of the largest."""
    rng = np.random.default_rng(41)
    page, n, dim = 16, 200, 64
    for power in (10, 17, 24, 30):
        tables, total = tables_for(rng, [n, n], page)
        k, v = make_pages(rng, total, page, 1, dim, True)
        k.view(torch.uint8)[..., 5] = 0
        q = queries(rng, 12, 4, dim, 0.3)
        q[q.float().abs() < 0.25] = 0.25             # within 2^-2 of each other: the row's span is the power's
        q[..., 5] = 2.0 ** power
        check(q, [0, 5, 12], k, v, tables, [n, n], scale=0.125)


@pytest.mark.parametrize("e4m3", [False, True])
def test_offsets_past_32_bits(e4m3):
    """Pages more than 2^32 bytes into a pool."""
    page, hkv, dim = 64, 8, 128
    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    pages = (1 << (32 if e4m3 else 31)) // (page * hkv * dim) + 8
    pool = torch.empty((2, pages, page, hkv, dim), dtype=kind, device=DEV)
    rng = np.random.default_rng(10)
    use = [pages - 1, 0, pages - 4]
    small = torch.empty((2, 3, page, hkv, dim), dtype=kind, device=DEV)
    for i, p in enumerate(use):
        small[:, i] = torch.from_numpy(rng.standard_normal((2, page, hkv, dim)).astype(np.float32)).to(DEV).to(kind)
        pool.view(torch.uint8)[:, p] = small.view(torch.uint8)[:, i]
    q = queries(rng, 40, 16, dim)
    ws = M.paged_chunk_workspace(16, hkv, dim)
    a = M.paged_chunk_attention(q, i32([0, 40]), pool[0], pool[1], i32([use]), i32([170]), ws)
    b = check(q, [0, 40], small[0], small[1], [[0, 1, 2]], [170])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dim,e4m3", [(64, False), (128, True), (256, False)])
def test_a_length_at_the_end_of_32_bits(dim, e4m3):
    """The longest table of pages of 64 tokens, its last columns alone with pages: a chunk that ends 2^31 - 64 tokens in
    with a window sees what a short sequence of the same last tokens does."""
    page, window, heads, n = 64, 100, 4, 30
    rng = np.random.default_rng(62)
    k, v = make_pages(rng, 4, page, 1, dim, e4m3)
    q = queries(rng, n, heads, dim)
    width = (1 << 25) - 1
    tables = torch.full((1, width), -1, dtype=torch.int32, device=DEV)              # 134 MB
    tables[0, -3:] = i32([2, 0, 3])
    ws = M.paged_chunk_workspace(heads, 1, dim)
    for short in (192, 181, 131):                                                   # tokens of the last three pages
        got = M.paged_chunk_attention(q, i32([0, n]), k, v, tables, i32([(width - 3) * page + short]), ws, window=window)
        assert M.get_device_error(ws) == 0
        want = check(q, [0, n], k, v, [[2, 0, 3]], [short], window=window)
        assert (got[0].float() - want[0].float()).abs().max() <= 2.0 ** -6 and torch.allclose(got[1], want[1], atol=2e-5)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("what", ["query", "key", "value", "later key", "later value"])
def test_a_number_that_is_none_stays_where_it_is_seen(what, e4m3):
    """A NaN query channel reaches its own row, a NaN key the rows of its cache head and sequence that see it, a NaN value
    their channel; what comes after a row's own token reaches it in no case."""
    rng = np.random.default_rng(61)
    page, hkv, group, dim = 16, 2, 4, 64
    chunks = [(20, 300), (60, 200), (5, 50)]
    lens = [n for _, n in chunks]
    tables, total = tables_for(rng, lens, page)
    k, v = make_pages(rng, total, page, hkv, dim, e4m3)
    starts = starts_of([c for c, _ in chunks])
    q = queries(rng, starts[-1], hkv * group, dim)
    nan = torch.zeros(q.shape, dtype=torch.bool, device=DEV)
    tok = 165 if what.startswith("later") else 70            # of sequence 1, whose chunk stands at 140 .. 199
    first = 20 + max(0, tok - 140)
    at = (int(tables[1, tok // page]), tok % page, 1)
    if what == "query":
        nan[25, 3] = True
        ref = C.attention(q, starts, k, v, tables, lens, dim ** -0.5)
        q[25, 3, 20] = math.nan
    else:
        pages = v if what.endswith("value") else k
        nan[first:80, group:2 * group, 33 if what.endswith("value") else slice(None)] = True
        ref = C.attention(q, starts, k, v, tables, lens, dim ** -0.5)
        (pages.view(torch.uint8) if e4m3 else pages)[at + (33 if what.endswith("value") else 9,)] = 0x7F if e4m3 else math.nan
    ws = M.paged_chunk_workspace(hkv * group, hkv, dim)
    out, lse = M.paged_chunk_attention(q, i32(starts), k, v, i32(tables), i32(lens), ws)
    assert M.get_device_error(ws) == 0
    assert torch.isnan(out[nan]).all() and ((out.double() - ref[0]).abs() <= ref[1])[~nan].all()
    rows = nan.all(2)
    assert torch.isnan(lse[rows]).all() and ((lse.double() - ref[2]).abs() <= ref[3])[~rows].all()


@pytest.mark.parametrize("dim,e4m3", [(64, False), (128, True), (128, False), (256, False), (256, True), (96, False)])
@pytest.mark.parametrize("length,new,group", [(200, 60, 4), (200, 200, 1), (6000, 90, 2)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_values_that_are_none_reach_the_rows_that_see_them_alone(bad, length, new, group, dim, e4m3):
    """Values of a token within the chunk, and of one that the window has passed for some rows: in the same tiles as the
    tokens that the other rows see, in blocks of one CTA and in blocks of several."""
    if e4m3 and not math.isnan(bad):
        pytest.skip("no infinities in the type")
    rng = np.random.default_rng(dim + length)
    page, window = 16, new // 2
    tables, total = tables_for(rng, [length], page)
    k, v = make_pages(rng, total, page, 1, dim, e4m3)
    q = queries(rng, new, group, dim)
    ws = M.paged_chunk_workspace(group, 1, dim)
    first = length - new
    for tok, w in ((length - 1, 0), (length - new // 3, 0), (first + new // 4, window), (max(0, first - window + 3), window)):
        ref = C.attention(q, [0, new], k, v, tables, [length], dim ** -0.5, w)
        keep = v.clone()
        at = (int(tables[0, tok // page]), tok % page, 0, 3)
        (v.view(torch.uint8) if e4m3 else v)[at] = 0x7F if e4m3 else bad
        out, lse = M.paged_chunk_attention(q, i32([0, new]), k, v, i32(tables), i32([length]), ws, window=w)
        assert M.get_device_error(ws) == 0
        pos = torch.arange(first, length, device=DEV)
        sees = (pos >= tok) & ((pos < tok + w) if w else True)
        hit = torch.zeros(q.shape, dtype=torch.bool, device=DEV)
        hit[sees, :, 3] = True
        got = out.double()
        assert (torch.isnan(got[hit]) if math.isnan(bad) else got[hit] == bad).all()
        assert ((got - ref[0]).abs() <= ref[1])[~hit].all() and ((lse.double() - ref[2]).abs() <= ref[3]).all()
        v = keep


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_an_infinite_key(sign):
    """A key that is infinite against a query makes its token's score -infinity or the row's result no number."""
    rng = np.random.default_rng(63)
    page, n, dim = 16, 150, 128
    tables, total = tables_for(rng, [n], page)
    k, v = make_pages(rng, total, page, 1, dim, False)
    q = queries(rng, 40, 2, dim)
    q[:, 0, 9], q[:, 1, 9] = sign, -sign
    tok = 20
    clean = tables.copy()
    k[tables[0, tok // page], tok % page, 0, 9] = math.inf
    ws = M.paged_chunk_workspace(2, 1, dim)
    out, lse = M.paged_chunk_attention(q, i32([0, 40]), k, v, i32(tables), i32([n]), ws)
    up, down = (0, 1) if sign > 0 else (1, 0)
    assert torch.isnan(out[:, up]).all() and torch.isnan(lse[:, up]).all()
    keep = [j for j in range(n) if j != tok]
    kk = torch.stack([k[clean[0, j // page], j % page, 0] for j in keep]).double()
    vv = torch.stack([v[clean[0, j // page], j % page, 0] for j in keep]).double()
    s = (q[:, down].double() @ kk.T * dim ** -0.5).masked_fill(torch.tensor(keep, device=DEV)[None] > torch.arange(110, 150, device=DEV)[:, None], -math.inf)
    want = torch.softmax(s, 1) @ vv
    assert ((out[:, down].double() - want).abs() <= 2.0 ** -6 * (1 + want.abs())).all()
    assert (lse[:, down].double() - torch.logsumexp(s, 1)).abs().max() <= 1e-4


def test_one_new_token_agrees_with_the_decode_call():
    rng = np.random.default_rng(12)
    page, lens = 32, [1, 40, 700, 0]
    tables, total = tables_for(rng, lens, page)
    k, v = make_pages(rng, total, page, 2, 128, False)
    q = queries(rng, 4, 8, 128)
    a, la = check(q, [0, 1, 2, 3, 4], k, v, tables, lens)
    b, lb = M.paged_attention(q, k, v, i32(tables), i32(lens), M.attention_workspace(4, 8, 2, 128))
    assert (a.float() - b.float()).abs().max() <= 2.0 ** -6 and torch.allclose(la, lb, atol=2e-5)


@pytest.mark.parametrize("chunk", [1, 37, 128, 500])
def test_a_prompt_in_chunks_is_the_prompt_in_one(chunk):
    rng = np.random.default_rng(chunk)
    page, n = 16, 500
    tables, total = tables_for(rng, [n], page)
    k, v = make_pages(rng, total, page, 2, 64, False)
    q = queries(rng, n, 4, 64)
    ref = C.attention(q, [0, n], k, v, tables, [n], 0.125)
    ws = M.paged_chunk_workspace(4, 2, 64)
    out, lse = torch.zeros_like(q), torch.zeros((n, 4), device=DEV)
    for at in range(0, n, chunk):
        to = min(n, at + chunk)
        M.paged_chunk_attention(q[at:to], i32([0, to - at]), k, v, i32(tables), i32([to]), ws, out=out[at:to], lse=lse[at:to])
    compare(out, lse, *ref)


@pytest.mark.parametrize("dim,e4m3", [(128, False), (64, True), (256, False)])
def test_another_stream_and_a_graph(dim, e4m3):
    rng = np.random.default_rng(11)
    page, lens = 16, [3330, 40]
    tables, total = tables_for(rng, lens, page)
    k, v = make_pages(rng, total, page, 2, dim, e4m3)
    q = queries(rng, 48, 8, dim)
    ws = M.paged_chunk_workspace(8, 2, dim)
    td, ld, sd = i32(tables), i32(lens), i32([0, 30, 48])
    want, wl = M.paged_chunk_attention(q, sd, k, v, td, ld, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, gl = M.paged_chunk_attention(q, sd, k, v, td, ld, ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want) and torch.equal(gl, wl)
    out, lse = torch.zeros_like(want), torch.zeros_like(wl)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.paged_chunk_attention(q, sd, k, v, td, ld, ws, out=out, lse=lse)
        M.paged_chunk_attention(q, sd, k, v, td, ld, ws, out=out, lse=lse)       # the next call behind this one's join
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)
    ld.copy_(i32([20, 0]))                                                       # a replay follows lengths and chunks
    sd.copy_(i32([0, 3, 48]))
    graph.replay()
    want, wl = M.paged_chunk_attention(q, sd, k, v, td, ld, ws)
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("e4m3", [False, True])
def test_more_sequences_than_a_cta_has_threads(e4m3):
    rng = np.random.default_rng(17)
    page, batch = 16, 1100
    counts = [int(x) for x in rng.integers(0, 12, batch)]
    lens = [c + int(x) for c, x in zip(counts, rng.integers(0, 700, batch))]
    ids = [int(x) for x in rng.permutation(batch)]
    tables, total = tables_for(rng, [lens[ids.index(i)] for i in range(batch)], page)
    k, v = make_pages(rng, total, page, 2, 64, e4m3)
    starts = starts_of(counts)
    rows = [0] * batch
    for b, i in enumerate(ids):
        rows[i] = lens[b]
    check(queries(rng, starts[-1] + 3, 6, 64), starts, k, v, tables, rows, seq_ids=ids)


@pytest.mark.parametrize("dims", [(128, 256), (64, 64), (128, 128)])
def test_two_calls_at_once(dims):
    """On two streams with a workspace each, over and over: the bits of each by itself."""
    calls, want = [], []
    for i, dim in enumerate(dims):
        rng = np.random.default_rng(18 + i)
        page, lens = 32, [5000, 333, 80]
        tables, total = tables_for(rng, lens, page)
        k, v = make_pages(rng, total, page, 4, dim, i == 1)
        q = queries(rng, 400, 16, dim)
        args = (q, i32([0, 5, 320, 400]), k, v, i32(tables), i32(lens), M.paged_chunk_workspace(16, 4, dim))
        calls.append(args)
        want.append(M.paged_chunk_attention(*args))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[], []]
    for _ in range(10):
        for i, (stream, args) in enumerate(zip(streams, calls)):
            with torch.cuda.stream(stream):
                got[i].append(M.paged_chunk_attention(*args))
    torch.cuda.synchronize()
    for i in range(2):
        assert M.get_device_error(calls[i][-1]) == 0
        for out, lse in got[i]:
            assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


def test_two_graphs_on_one_workspace():
    rng = np.random.default_rng(19)
    page, shapes = 16, [(8, 2, 64), (4, 1, 256)]
    ws = M.paged_chunk_workspace(4, 1, 256)
    graphs = []
    for h, hkv, dim in shapes:
        lens = [4000, 100]
        tables, total = tables_for(rng, lens, page)
        k, v = make_pages(rng, total, page, hkv, dim, False)
        args = queries(rng, 70, h, dim), i32([0, 60, 70]), k, v, i32(tables), i32(lens)
        want = M.paged_chunk_attention(*args, M.paged_chunk_workspace(h, hkv, dim))
        out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            M.paged_chunk_attention(*args, ws, out=out, lse=lse)
        graphs.append((graph, out, lse, want, args))
    for _ in range(4):
        for graph, *_ in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for _, out, lse, want, _ in graphs:
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert M.get_device_error(ws) == 0


@pytest.mark.parametrize("dim,e4m3", [(128, False), (64, True), (128, True), (256, False), (256, True)])
def test_a_wait_that_runs_out_is_recorded_and_the_next_call_is_right(dim, e4m3):
    """The limit lowered to zero: the first wait for a tile that is still on its way gives up (every copy and product does
    arrive, and is waited for before the kernel ends). Restored, the same workspace serves the next calls."""
    rng = np.random.default_rng(15)
    page, lens, starts = 32, [9000, 700], [0, 200, 700]
    tables, total = tables_for(rng, lens, page)
    k, v = make_pages(rng, total, page, 2, dim, e4m3)
    q = queries(rng, 700, 8, dim)
    ws = M.paged_chunk_workspace(8, 2, dim)
    td, ld, sd = i32(tables), i32(lens), i32(starts)
    torch.cuda.synchronize()
    try:
        M.set_wait_limit_ns(0)
        M.paged_chunk_attention(q, sd, k, v, td, ld, ws)
        code = M.get_device_error(ws)
    finally:
        M.set_wait_limit_ns(M.WAIT_LIMIT_NS)
    assert code == 6, f"expected the timed-out wait to be recorded, got error word {code}"
    M.workspace_init(ws)
    for _ in range(2):
        check(q, starts, k, v, tables, lens, ws=ws)


def test_one_workspace_for_the_calls_on_cache_and_attention():
    """Calls of different shapes, and the decode and append calls, on the largest of their workspaces in turn."""
    rng = np.random.default_rng(13)
    shapes = [(8, 2, 128), (4, 4, 64), (6, 1, 256), (16, 1, 80)]
    size = max(max(M.paged_chunk_workspace_size(*s), M.attention_workspace_size(*s)) for s in shapes)
    ws = torch.zeros(size, dtype=torch.uint8, device=DEV)
    page, lens = 32, [900, 64, 0, 333]
    for _ in range(2):
        for h, hkv, d in shapes:
            tables, total = tables_for(rng, lens, page)
            k, v = make_pages(rng, total, page, hkv, d, False)
            check(queries(rng, 80, h, d), [0, 40, 50, 52, 80], k, v, tables, lens, ws=ws)
            q = queries(rng, 4, h, d)
            got = M.paged_attention(q, k, v, i32(tables), i32(lens), ws)
            want = M.paged_attention(q, k, v, i32(tables), i32(lens), M.attention_workspace(4, h, hkv, d))
            assert torch.equal(got[0], want[0]) and M.get_device_error(ws) == 0


def test_empty_calls():
    k = torch.zeros((2, 16, 1, 64), dtype=torch.bfloat16, device=DEV)
    ws = M.paged_chunk_workspace(4, 1, 64)
    for t, starts in ((0, [0, 0]), (0, [0]), (3, [1])):
        out, lse = M.paged_chunk_attention(torch.zeros((t, 4, 64), dtype=torch.bfloat16, device=DEV), i32(starts), k, k,
                                           i32([[0]]), i32([3]), ws)
        assert out.shape == (t, 4, 64) and lse.shape == (t, 4) and M.get_device_error(ws) == 0


def test_refusals():
    q = torch.zeros((5, 8, 64), dtype=torch.bfloat16, device=DEV)
    k = torch.zeros((3, 16, 2, 64), dtype=torch.bfloat16, device=DEV)
    v, t, n, s = torch.zeros_like(k), i32([[0], [1]]), i32([1, 1]), i32([0, 2, 5])
    ws = M.paged_chunk_workspace(8, 2, 64)
    for error, args, kw in (
            (TypeError, (q.float(), s, k, v, t, n, ws), {}), (TypeError, (q, s.long(), k, v, t, n, ws), {}),
            (TypeError, (q, s, k.half(), v.half(), t, n, ws), {}), (ValueError, (q, s.cpu(), k, v, t, n, ws), {}),
            (ValueError, (q, s, k, None, t, n, ws), {}), (ValueError, (q, s[:0], k, v, t, n, ws), {}),
            (ValueError, (q, s, k, v[:2], t, n, ws), {}), (ValueError, (q, s, k, v, t, n[:1], ws), {}),
            (ValueError, (q[:, :, ::2], s, k, v, t, n, ws), {}), (ValueError, (q[..., :32].contiguous(), s, k, v, t, n, ws), {}),
            (ValueError, (q, s, k, v, t, n, ws), dict(out=torch.zeros((5, 8, 32), dtype=torch.bfloat16, device=DEV))),
            (ValueError, (q, s, k, v, t, n, ws), dict(lse=torch.zeros((4, 8), device=DEV))),
            (ValueError, (q, s, k, v, t, n, ws), dict(seq_ids=i32([0, 1, 0])))):
        with pytest.raises(error):
            M.paged_chunk_attention(*args, **kw)
    with pytest.raises(M.MoeW4A16Error) as e:
        M.paged_chunk_attention(q, s, k, v, t, n, ws, out=q)
    assert e.value.name == "ERR_INVALID_ARG"
    with pytest.raises(M.MoeW4A16Error) as e:
        M.paged_chunk_attention(q, s, k, v, t, n, ws, window=-1)
    assert e.value.name == "ERR_INVALID_ARG"
    with pytest.raises(M.MoeW4A16Error) as e:
        M.paged_chunk_attention(q, s, k, v, t, n, ws[:64])
    assert e.value.name == "ERR_WORKSPACE"


@pytest.mark.parametrize("dim,e4m3", [(64, False), (128, False), (128, True), (256, False), (256, True)])
def test_a_value_that_is_none_at_the_end_of_a_long_row(dim, e4m3):
    """The last of 70001 tokens has a value that is none: over a hundred tokens share its tiles and do not see it, each with
    all those before it to go through again. That is over far below the limit of the kernels' waits, no wait runs out, and
    the sequence beside it keeps its bits."""
    rng = np.random.default_rng(71)
    page, lens, starts, group = 64, [70001, 900], [0, 300, 360], 8
    tables, total = tables_for(rng, lens, page)
    k, v = make_pages(rng, total, page, 1, dim, e4m3)
    q = queries(rng, 360, group, dim)
    ws = M.paged_chunk_workspace(group, 1, dim)
    args = (q, i32(starts), k, v, i32(tables), i32(lens), ws)
    clean = M.paged_chunk_attention(*args)
    ref = C.attention(q[:300], [0, 300], k, v, tables[:1], lens[:1], dim ** -0.5)
    (v.view(torch.uint8) if e4m3 else v)[int(tables[0, 70000 // page]), 70000 % page, 0, 3] = 0x7F if e4m3 else math.inf
    times = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
    times[0].record()
    out, lse = M.paged_chunk_attention(*args)
    times[1].record()
    assert M.get_device_error(ws) == 0
    assert times[0].elapsed_time(times[1]) < 0.25e-6 * M.WAIT_LIMIT_NS           # (ms: a quarter of the limit)
    assert torch.equal(out[300:], clean[0][300:]) and torch.equal(lse, clean[1])
    compare(out[:299], lse[:299], *(x[:299] for x in ref))
    last = out[299].double()
    assert not torch.isfinite(last[:, 3]).any()
    last[:, 3] = ref[0][299, :, 3]
    assert ((last - ref[0][299]).abs() <= ref[1][299]).all()


@pytest.mark.parametrize("dim,e4m3", [(64, False), (128, True), (256, False)])
@pytest.mark.parametrize("lens", [[300, 7], [9001, 4000]])
def test_a_value_that_is_none_and_seen_by_all(lens, dim, e4m3):
    """No row has to be computed again: the channel is none in every row of the head, of one CTA and of several, and all else
    keeps its bits."""
    rng = np.random.default_rng(72)
    page, group, hkv = 32, 3, 2
    starts = [0, 150, 157]
    tables, total = tables_for(rng, lens, page)
    k, v = make_pages(rng, total, page, hkv, dim, e4m3)
    q = queries(rng, 157, group * hkv, dim)
    ws = M.paged_chunk_workspace(group * hkv, hkv, dim)
    args = (q, i32(starts), k, v, i32(tables), i32(lens), ws)
    clean = M.paged_chunk_attention(*args)
    (v.view(torch.uint8) if e4m3 else v)[int(tables[0, 0]), 5, 1, 20] = 0x7F if e4m3 else -math.inf
    out, lse = M.paged_chunk_attention(*args)
    assert M.get_device_error(ws) == 0 and torch.equal(lse, clean[1])
    hit = torch.zeros(q.shape, dtype=torch.bool, device=DEV)
    hit[:150, group:, 20] = True
    assert (torch.isnan(out[hit]) if e4m3 else out[hit] == -math.inf).all() and torch.equal(out[~hit], clean[0][~hit])


def test_values_that_are_none_in_a_graph_and_the_calls_after_it():
    """Flagged rows of one replay, none of the next: nothing is kept from call to call."""
    rng = np.random.default_rng(73)
    page, lens, starts, dim = 16, [5000, 400], [0, 60, 130], 128
    tables, total = tables_for(rng, lens, page)
    k, v = make_pages(rng, total, page, 2, dim, False)
    q = queries(rng, 130, 8, dim)
    ws = M.paged_chunk_workspace(8, 2, dim)
    args = (q, i32(starts), k, v, i32(tables), i32(lens), ws)
    clean = M.paged_chunk_attention(*args)
    places = [(int(tables[b, (n - 1) // page]), (n - 1) % page, 1, 7) for b, n in enumerate(lens)]
    kept = [v[at].clone() for at in places]
    for at in places:
        v[at] = math.nan
    want = M.paged_chunk_attention(*args)
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.paged_chunk_attention(*args, out=out, lse=lse)
    for _ in range(3):
        graph.replay()
        assert torch.equal(out.view(torch.int16), want[0].view(torch.int16)) and torch.equal(lse, want[1])
        for at, x in zip(places, kept):
            v[at] = x
        graph.replay()
        assert torch.equal(out, clean[0]) and torch.equal(lse, clean[1])
        for at in places:
            v[at] = math.nan
    assert M.get_device_error(ws) == 0


def test_outputs_between_the_queries_rows_and_over_them():
    """Outputs in a gap of the queries' buffer are theirs alone; any that share a byte with a query are refused."""
    rng = np.random.default_rng(74)
    page, n, heads, dim = 16, 9, 4, 64
    tables, total = tables_for(rng, [200], page)
    k, v = make_pages(rng, total, page, 2, dim, False)
    wide = torch.zeros((n, (n + 2) * heads * dim), dtype=torch.bfloat16, device=DEV)
    q = wide[:, :heads * dim].view(n, heads, dim)
    q.copy_(queries(rng, n, heads, dim))
    ws = M.paged_chunk_workspace(heads, 2, dim)
    args = (i32([0, n]), k, v, i32(tables), i32([200]), ws)
    want = M.paged_chunk_attention(q.contiguous(), *args)
    flat, size = wide.view(-1), n * heads * dim
    for at, fits in ((heads * dim, True), (2 * heads * dim, True), (2 * heads * dim + 8, False), (heads * dim - 8, False),
                     (wide.stride(0) * 8 + heads * dim, True), (wide.stride(0) * 8 - size + 8, False)):
        out = flat[at:at + size].view(n, heads, dim)
        if fits:
            M.paged_chunk_attention(q, *args, out=out)
            assert torch.equal(out, want[0])
        else:
            with pytest.raises(M.MoeW4A16Error) as e:
                M.paged_chunk_attention(q, *args, out=out)
            assert e.value.name == "ERR_INVALID_ARG"
    sums = flat[heads * dim:heads * dim + 2 * n * heads].view(torch.float32).view(n, heads)
    M.paged_chunk_attention(q, *args, lse=sums)
    assert torch.equal(sums, want[1])
    for lse in (flat[:2 * n * heads], flat[heads * dim - 2:heads * dim - 2 + 2 * n * heads]):
        with pytest.raises(M.MoeW4A16Error) as e:
            M.paged_chunk_attention(q, *args, lse=lse.view(torch.float32).view(n, heads))
        assert e.value.name == "ERR_INVALID_ARG"


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("n", [2000, 9000])
@pytest.mark.parametrize("gap", [8.0, 17.0, 20.0])
@pytest.mark.parametrize("sink", [0, 700])
def test_many_small_probabilities_behind_a_large_one_over_an_8_bit_cache(sink, gap, n, dim):
    """One token with a value of zero takes nearly all of the probability, thousands of equal ones `gap` nats below it make
    the output. Probabilities enter the product as FP16 numbers of 2^8 and more for the largest: off by 2^-11 of themselves, or
    half of the subnormals' spacing of 2^-24, which is 2^-33 of the largest."""
    rng = np.random.default_rng(n + dim)
    page, new, group = 32, 40, 2
    tables, total = tables_for(rng, [n], page)
    k = torch.zeros((total, page, 1, dim), dtype=torch.bfloat16, device=DEV)
    v = (torch.rand((total, page, 1, dim), generator=torch.Generator(device="cuda").manual_seed(n), device="cuda") * 1.5 + 0.5)
    at = int(tables[0, sink // page]), sink % page, 0
    k[at + (3,)] = 1.0
    v[at] = 0.0
    k, v = k.to(torch.float8_e4m3fn), v.to(torch.bfloat16).to(torch.float8_e4m3fn)
    q = torch.zeros((new, group, dim), dtype=torch.bfloat16, device=DEV)
    q[..., 3] = gap
    ws = M.paged_chunk_workspace(group, 1, dim)
    out, _ = M.paged_chunk_attention(q, i32([0, new]), k, v, i32(tables), i32([n]), ws, scale=1.0)
    assert M.get_device_error(ws) == 0
    values = v.float()[i32(tables)[0, :n // page + 1].long().clamp(min=0)].view(-1, dim)[:n].double()
    seen = torch.arange(n - new, n, device=DEV) + 1
    small = math.exp(-gap)
    sums = torch.cumsum(values, 0)[seen - 1] * small
    total_p = (1 + (seen - 1) * small)[:, None]
    want = sums / total_p
    # the scores' and the exponentials' errors as in chunk_ref: 2 e + 2^-16, and the sums'
    rel = 2.0 ** -11 + 2 * (dim + 8) * 2.0 ** -23 * gap + 2.0 ** -16 + (n / 16 + 64) * 2.0 ** -23
    bound = 2.0 ** -8 * 1.01 * want + rel * want + n * 2.0 ** -33 * 2.0 / total_p
    assert (bound <= 0.1 * want).all()
    for head in range(group):
        err = (out[:, head].double() - want).abs()
        assert (err <= bound).all(), (err / bound).max().item()


@pytest.mark.parametrize("dim,e4m3", [(64, False), (128, True), (256, False)])
def test_a_value_that_is_none_at_the_end_of_32_bits(dim, e4m3):
    """The last of 2^31 - 64 tokens, most of them without a page: the rows before it see what they do without it."""
    page, window, heads, n = 64, 100, 4, 30
    rng = np.random.default_rng(77)
    k, v = make_pages(rng, 4, page, 1, dim, e4m3)
    q = queries(rng, n, heads, dim)
    width = (1 << 25) - 1
    tables = torch.full((1, width), -1, dtype=torch.int32, device=DEV)
    tables[0, -3:] = i32([2, 0, 3])
    ws = M.paged_chunk_workspace(heads, 1, dim)
    args = (q, i32([0, n]), k, v, tables, i32([width * page]), ws)
    clean = M.paged_chunk_attention(*args, window=window)
    ref = C.attention(q, [0, n], k, v, [[2, 0, 3]], [192], dim ** -0.5, window)
    (v.view(torch.uint8) if e4m3 else v)[3, page - 1, 0, 3] = 0x7F if e4m3 else math.nan
    out, lse = M.paged_chunk_attention(*args, window=window)
    assert M.get_device_error(ws) == 0 and torch.equal(lse, clean[1])
    compare(out[:-1], lse[:-1], *(x[:-1] for x in ref))
    assert torch.isnan(out[-1, :, 3]).all() and torch.isfinite(out[-1, :, 4:]).all()
