"""Attention over a paged cache against the plain 64-bit form, at the sizes and masks where it can go wrong."""

import math

import numpy as np
import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu

M = pytest.importorskip("w4a16_int4_mixture_grouped_gb300") if torch.cuda.is_available() else None
DEV = torch.device("cuda", 0) if torch.cuda.is_available() else None


def f64(t):
    return t.detach().to(torch.float32).cpu().numpy().astype(np.float64)


def tables_for(rng, lens, page, extra=3, width=None):
    need = [R.pages_of(max(n, 0), page) for n in lens]
    width = width or max(1, max(need)) + 1
    total = sum(need) + extra
    order = rng.permutation(total)
    tables = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for i, c in enumerate(need):
        tables[i, :c] = order[at:at + c]
        at += c
    return tables, total


def poison(pages, tables, lens, page, page_dim=0):
    """NaN in every slot that holds no token: pages of no table, and the rest of each last page."""
    raw = pages.view(torch.uint8) if pages.dtype == torch.float8_e4m3fn else pages
    bad = 0x7F if pages.dtype == torch.float8_e4m3fn else float("nan")
    held = torch.zeros(pages.shape[:2], dtype=torch.bool)
    for row, n in zip(tables, lens):
        for j in range(max(0, n)):
            if row[j // page] >= 0:
                held[row[j // page], j % page] = True
    raw[~held.to(pages.device)] = bad


def make_pages(rng, total, page, heads, dim, e4m3, head_major=False):
    shape = (total, heads, page, dim) if head_major else (total, page, heads, dim)
    out = []
    for _ in range(2):
        t = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DEV).to(torch.bfloat16)
        t = t.to(torch.float8_e4m3fn) if e4m3 else t
        out.append(t.transpose(1, 2) if head_major else t)
    return out


def check(q, k, v, tables, lens, page, scale=None, window=0, ks=1.0, vs=1.0, seq_ids=None, ws=None, want_err=0):
    b, h, d = q.shape
    hkv = k.shape[2]
    scale = d ** -0.5 if scale is None else scale
    ws = ws if ws is not None else M.attention_workspace(b, h, hkv, d)
    sid = None if seq_ids is None else torch.tensor(seq_ids, dtype=torch.int32, device=DEV)
    td, ld = torch.from_numpy(tables).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, lse = M.paged_attention(q, k, v, td, ld, ws, scale=scale, window=window, k_scale=ks, v_scale=vs, seq_ids=sid)
    assert M.get_device_error(ws) == want_err
    kn, vn = f64(k), f64(v)
    ref, bound, rl, lb = R.attention(f64(q), lambda p, t: kn[p, t] * ks, lambda p, t: vn[p, t], h // hkv, tables, lens,
                                     page, k.shape[0], scale, window, vs, seq_ids)
    compare(out, lse, ref, bound, rl, lb)
    return out, lse


def compare(out, lse, ref, bound, rl, lb):
    got, gl = f64(out), f64(lse)
    assert np.isfinite(got).all()
    err = np.abs(got - ref)
    assert (err <= bound).all(), f"out: {(err / np.maximum(bound, 1e-300)).max()} of the bound"
    empty = np.isneginf(rl)
    assert np.array_equal(np.isneginf(gl), empty)
    assert (got[empty] == 0).all()
    d = np.abs(gl[~empty] - rl[~empty])
    assert (d <= lb[~empty]).all(), f"lse: {(d / lb[~empty]).max()} of the bound"


def queries(rng, b, h, d, scale=1.0):
    return torch.from_numpy((rng.standard_normal((b, h, d)) * scale).astype(np.float32)).to(DEV).to(torch.bfloat16)


LENS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 130, 300]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dim,group,hkv,page", [(128, 4, 2, 16), (128, 8, 1, 64), (64, 1, 3, 32), (96, 5, 2, 48),
                                                (256, 2, 2, 16), (128, 16, 1, 1), (16, 3, 1, 7), (112, 20, 1, 40),
                                                (64, 33, 1, 128), (240, 9, 1, 24)])
def test_ragged_lengths(dim, group, hkv, page, e4m3):
    rng = np.random.default_rng(dim * 100 + group + e4m3)
    tables, total = tables_for(rng, LENS, page)
    k, v = make_pages(rng, total, page, hkv, dim, e4m3)
    poison(k, tables, LENS, page)
    poison(v, tables, LENS, page)
    ks, vs = (0.75, 1.5) if e4m3 else (1.0, 1.0)
    check(queries(rng, len(LENS), group * hkv, dim, 1.5), k, v, tables, LENS, page, ks=ks, vs=vs)


@pytest.mark.parametrize("window", [1, 5, 16, 100, 1000])
@pytest.mark.parametrize("e4m3", [False, True])
def test_window_with_the_pages_behind_it_freed(window, e4m3):
    rng = np.random.default_rng(window)
    page, lens = 16, [0, 1, 5, 16, 17, 99, 100, 101, 333]
    tables, total = tables_for(rng, lens, page)
    for i, n in enumerate(lens):
        tables[i, :max(0, n - window) // page] = -1
    k, v = make_pages(rng, total, page, 2, 64, e4m3)
    poison(k, tables, lens, page)
    poison(v, tables, lens, page)
    check(queries(rng, len(lens), 8, 64), k, v, tables, lens, page, window=window)


def test_holes_in_the_table_and_rows_that_see_nothing():
    rng = np.random.default_rng(5)
    page, lens = 16, [100, 100, 64, 16]
    tables, total = tables_for(rng, lens, page)
    tables[0, [0, 3, 6]] = -1            # freed here and there, the last page too
    tables[1, :] = -1                    # nothing left
    tables[3, 0] = -7                    # any negative entry is no page
    k, v = make_pages(rng, total, page, 2, 128, False)
    poison(k, tables, lens, page)
    poison(v, tables, lens, page)
    check(queries(rng, 4, 8, 128), k, v, tables, lens, page)


def test_bad_ids_and_lengths_are_skipped_and_recorded():
    rng = np.random.default_rng(6)
    page, lens = 16, [40, 33, 20]
    tables, total = tables_for(rng, lens, page)
    k, v = make_pages(rng, total, page, 1, 64, False)
    q = queries(rng, 3, 4, 64)
    bad = tables.copy()
    bad[1, 1] = total                    # past the pool
    check(q, k, v, bad, lens, page, want_err=8)
    check(q, k, v, tables, [40, 33, -4], page, want_err=8)
    full, total = tables_for(rng, [64, 64, 64], page, width=4)
    k, v = make_pages(rng, total, page, 1, 64, False)
    check(q, k, v, full, [64, 1000, 3], page, want_err=8)      # cut to the table's 64 tokens
    check(q, k, v, full, [64, 64, 64], page, seq_ids=[2, 0, 1])
    ws = M.attention_workspace(3, 4, 1, 64)
    out, lse = M.paged_attention(q, k, v, torch.from_numpy(full).to(DEV), torch.full((3,), 9, dtype=torch.int32, device=DEV),
                                 ws, seq_ids=torch.tensor([0, 3, -1], dtype=torch.int32, device=DEV))
    assert M.get_device_error(ws) == 8
    assert (out[1:] == 0).all() and torch.isneginf(lse[1:]).all() and torch.isfinite(lse[0]).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_strides_head_major_pages_and_query_slices(e4m3):
    rng = np.random.default_rng(7)
    page, lens = 32, [77, 3, 200]
    tables, total = tables_for(rng, lens, page)
    k, v = make_pages(rng, total, page, 4, 128, e4m3, head_major=True)
    qkv = queries(rng, 3, 24, 128)
    q = qkv[:, 2:18]                     # rows of a wider projection
    wide = np.full((3, tables.shape[1] + 5), 10 ** 6, dtype=np.int32)
    wide[:, :tables.shape[1]] = tables
    check(q, k, v, tables, lens, page)
    ws = M.attention_workspace(3, 16, 4, 128)
    td = torch.from_numpy(wide).to(DEV)[:, :tables.shape[1]]
    ld = torch.tensor(lens, dtype=torch.int32, device=DEV)
    a, la = M.paged_attention(q, k, v, td, ld, ws)
    b, lb = M.paged_attention(q.contiguous(), k, v, td.contiguous(), ld, ws)
    assert torch.equal(a, b) and torch.equal(la, lb) and M.get_device_error(ws) == 0


@pytest.mark.parametrize("batch,top,hkv,group", [(1, 20011, 1, 8), (1, 9000, 8, 4), (3, 5000, 2, 16), (200, 90, 2, 2),
                                                  (700, 3, 1, 1)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_long_rows_are_split_and_joined(batch, top, hkv, group, e4m3):
    rng = np.random.default_rng(batch + top)
    page = 64
    lens = [top] + [int(x) for x in rng.integers(0, top + 1, batch - 1)]
    tables, total = tables_for(rng, lens, page)
    k, v = make_pages(rng, total, page, hkv, 64, e4m3)
    q = queries(rng, batch, group * hkv, 64, 2.0)
    ws = M.attention_workspace(batch, group * hkv, hkv, 64)
    a, la = check(q, k, v, tables, lens, page, ws=ws)
    for _ in range(3):                   # the same workspace again: the same bits
        b, lb = check(q, k, v, tables, lens, page, ws=ws)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_scores_far_apart_and_scales():
    """One token's score far above the others, in the first, a middle and the last tile; large and tiny scales."""
    rng = np.random.default_rng(8)
    page, lens = 16, [1000, 1000, 1000]
    tables, total = tables_for(rng, lens, page)
    k, v = make_pages(rng, total, page, 1, 64, False)
    q = queries(rng, 3, 8, 64)
    for i, j in enumerate((0, 517, 999)):
        k[tables[i, j // page], j % page, 0] = (q[i, 3].float() * 40).to(torch.bfloat16)
    for scale in (0.125, 4.0, 1e-4, -0.125, 0.0):
        check(q, k, v, tables, lens, page, scale=scale)


@pytest.mark.parametrize("group", [3, 8, 16])
@pytest.mark.parametrize("e4m3", [False, True])
def test_scores_that_rise_and_fall(group, e4m3):
    """Scores that climb by a little from token to token, up to 2^40 of the first probabilities, and come down again:
    whatever the exponents are taken against has to follow."""
    rng = np.random.default_rng(31)
    page, n, dim = 16, 1500, 64
    tables, total = tables_for(rng, [n, n], page)
    k, v = make_pages(rng, total, page, 1, dim, e4m3)
    q = queries(rng, 2, group, dim)
    steps = np.concatenate([np.linspace(0.0, 1.0, 900), np.linspace(1.0, 0.2, n - 900)])
    for b in range(2):
        one = q[b, 0].float() / q[b, 0].float().norm()
        for j in range(n):
            k[tables[b, j // page], j % page, 0] = (one * float(steps[j]) * 28.0).to(k.dtype)
    q[:] = q[:, :1] / q[:, :1].float().norm(dim=-1, keepdim=True).to(torch.bfloat16)
    check(q, k, v, tables, [n, n], page, scale=1.0)


def test_wide_range_of_queries_over_an_8_bit_cache():
    """Queries far above and below the FP16 range: each row is scaled by its own power of two."""
    rng = np.random.default_rng(9)
    page, lens = 16, [50, 50, 50]
    tables, total = tables_for(rng, lens, page)
    k, v = make_pages(rng, total, page, 1, 64, True)
    q = queries(rng, 3, 8, 64)
    q[0] *= 2.0 ** 40
    q[1] *= 2.0 ** -40
    q[2, 1] = 0
    check(q[:1], k, v, tables[:1], lens[:1], page, scale=2.0 ** -43)
    check(q[1:2], k, v, tables[1:2], lens[1:2], page, scale=2.0 ** 37)
    check(q[2:], k, v, tables[2:], lens[2:], page)


@pytest.mark.parametrize("group", [4, 16])
def test_channels_far_apart_within_a_query_over_an_8_bit_cache(group):
    """One channel of each query far above the others and met by keys of zero, so that the small ones decide: they keep
    their bits down to 2^-32 of the largest."""
    rng = np.random.default_rng(41)
    page, n, dim = 16, 200, 64
    for power in (10, 17, 24, 30):
        tables, total = tables_for(rng, [n, n], page)
        k, v = make_pages(rng, total, page, 1, dim, True)
        k.view(torch.uint8)[..., 5] = 0
        q = queries(rng, 2, group, dim, 0.3)
        small = q.float().abs() < 0.25               # within 2^-2 of each other: the row's span is the power's
        q[small] = 0.25
        q[..., 5] = 2.0 ** power
        check(q, k, v, tables, [n, n], page, scale=0.125)


def test_offsets_past_32_bits():
    """Pages more than 2^31 elements into a pool."""
    page, hkv, dim = 64, 8, 128
    pages = (1 << 31) // (page * hkv * dim) + 8
    pool = torch.empty((2, pages, page, hkv, dim), dtype=torch.bfloat16, device=DEV)
    rng = np.random.default_rng(10)
    use = [pages - 1, 0, pages - 4]
    for p in use:
        pool[:, p] = torch.from_numpy(rng.standard_normal((2, page, hkv, dim)).astype(np.float32)).to(DEV).to(torch.bfloat16)
    q = queries(rng, 1, 16, dim)
    small = pool[:, use].contiguous()
    ws = M.attention_workspace(1, 16, hkv, dim)
    ld = torch.tensor([170], dtype=torch.int32, device=DEV)
    a = M.paged_attention(q, pool[0], pool[1], torch.tensor([use], dtype=torch.int32, device=DEV), ld, ws)
    b = M.paged_attention(q, small[0], small[1], torch.tensor([[0, 1, 2]], dtype=torch.int32, device=DEV), ld, ws)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check(q, small[0], small[1], np.array([[0, 1, 2]], dtype=np.int32), [170], page)


@pytest.mark.parametrize("dim,e4m3", [(64, False), (128, True), (128, False)])
def test_a_length_at_the_end_of_32_bits(dim, e4m3):
    """The longest table of pages of 64 tokens, its last columns alone with pages: a window that ends 2^31 - 64 tokens in
    sees what a short sequence of the same last tokens does."""
    page, window, hkv, heads = 64, 100, 1, 4
    rng = np.random.default_rng(62)
    k, v = make_pages(rng, 4, page, hkv, dim, e4m3)
    q = queries(rng, 2, heads, dim)
    width = (1 << 25) - 1
    tables = torch.full((1, width), -1, dtype=torch.int32, device=DEV)              # 134 MB
    tables[0, -3:] = torch.tensor([2, 0, 3], dtype=torch.int32, device=DEV)
    ids = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = M.attention_workspace(1, heads, hkv, dim)
    for short in (192, 181, 131):                                                   # tokens of the last three pages
        lens = torch.tensor([(width - 3) * page + short], dtype=torch.int32, device=DEV)
        got = M.paged_attention(q[:1], k, v, tables, lens, ws, window=window, seq_ids=ids)
        assert M.get_device_error(ws) == 0
        want = check(q[:1], k, v, np.array([[2, 0, 3]], dtype=np.int32), [short], page, window=window)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("group", [4, 16])
@pytest.mark.parametrize("what", ["query", "key", "value", "infinite key"])
def test_a_number_that_is_none_stays_where_it_is_seen(what, group, e4m3):
    """A NaN query channel reaches its own head, a NaN key the heads of its cache head and sequence, a NaN value their
    channel. A key that is infinite against a query makes its token's score -infinity or the head's result no number."""
    if what == "infinite key" and e4m3:
        pytest.skip("no infinities in the type")
    rng = np.random.default_rng(61)
    page, lens, hkv, dim = 16, [300, 300, 50], 2, 64
    tables, total = tables_for(rng, lens, page)
    k, v = make_pages(rng, total, page, hkv, dim, e4m3)
    q = queries(rng, 3, hkv * group, dim)
    q[:, :, 9] = torch.where(torch.arange(hkv * group, device=DEV) % 2 == 0, 1.0, -1.0).to(torch.bfloat16)
    tok = (int(tables[1, 4]), 9)
    nan = np.zeros((3, hkv * group, dim), dtype=bool)
    first = slice(group, 2 * group)                          # the heads of cache head 1
    clean_k = k.clone()
    if what == "query":
        q0 = q.clone()
        q[1, 3, 20] = math.nan
        nan[1, 3] = True
    elif what == "value":
        (v.view(torch.uint8) if e4m3 else v)[tok[0], tok[1], 1, 33] = 0x7F if e4m3 else math.nan
        nan[1, first, 33] = True
    elif what == "key":
        (k.view(torch.uint8) if e4m3 else k)[tok[0], tok[1], 1, 9] = 0x7F if e4m3 else math.nan
        nan[1, first] = True
    else:
        k[tok[0], tok[1], 1, 9] = math.inf                   # heads with a negative channel there: the token is not seen
        nan[1, group:2 * group:2] = True
    ws = M.attention_workspace(3, hkv * group, hkv, dim)
    out, lse = M.paged_attention(q, k, v, torch.from_numpy(tables).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV), ws)
    assert M.get_device_error(ws) == 0
    kn, vn = f64(clean_k), np.nan_to_num(f64(v))
    qn = f64(q0 if what == "query" else q)
    ref, bound, rl, lb = R.attention(qn, lambda p, t: kn[p, t], lambda p, t: vn[p, t], group, tables, lens, page, total,
                                     dim ** -0.5, 0)
    if what == "infinite key":                               # the other heads of that cache head without the token
        unseen = tables.copy()
        keep = [j for j in range(300) if j != 4 * page + 9]
        k2, v2 = kn[unseen[1][np.array(keep) // page], np.array(keep) % page, 1], vn[unseen[1][np.array(keep) // page], np.array(keep) % page, 1]
        for h in range(group + 1, 2 * group, 2):
            s = k2 @ qn[1, h] * dim ** -0.5
            w = np.exp(s - s.max())
            ref[1, h], rl[1, h] = w @ v2 / w.sum(), s.max() + np.log(w.sum())
    got, gl = f64(out), f64(lse)
    assert np.isnan(got[nan]).all() and (np.abs(got - ref)[~nan] <= bound[~nan]).all()
    rows = nan.all(2)
    assert np.isnan(gl[rows]).all() and (np.abs(gl - rl)[~rows] <= lb[~rows]).all()


def test_another_stream_and_a_graph():
    rng = np.random.default_rng(11)
    page, lens = 16, [333, 40]
    tables, total = tables_for(rng, lens, page)
    k, v = make_pages(rng, total, page, 2, 128, False)
    q = queries(rng, 2, 8, 128)
    ws = M.attention_workspace(2, 8, 2, 128)
    td, ld = torch.from_numpy(tables).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    want, wl = M.paged_attention(q, k, v, td, ld, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, gl = M.paged_attention(q, k, v, td, ld, ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want) and torch.equal(gl, wl)
    out, lse = torch.zeros_like(want), torch.zeros_like(wl)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.paged_attention(q, k, v, td, ld, ws, out=out, lse=lse)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)
    ld.copy_(torch.tensor([20, 0], dtype=torch.int32))         # a replay follows the lengths
    graph.replay()
    want, wl = M.paged_attention(q, k, v, td, ld, ws)
    assert torch.equal(out, want) and torch.equal(lse, wl)


def test_empty_batch():
    k = torch.zeros((2, 16, 1, 64), dtype=torch.bfloat16, device=DEV)
    ws = M.attention_workspace(1, 4, 1, 64)
    out, lse = M.paged_attention(torch.zeros((0, 4, 64), dtype=torch.bfloat16, device=DEV), k, k,
                                 torch.zeros((1, 1), dtype=torch.int32, device=DEV),
                                 torch.zeros(1, dtype=torch.int32, device=DEV), ws)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


# ---------------------------------------------------------------------------
# latent cache
# ---------------------------------------------------------------------------

def check_latent(rng, lens, heads, page, window=0, holes=(), q_scale=1.0, scale=0.06, ws=None):
    tables, total = tables_for(rng, lens, page)
    for i, c in holes:
        tables[i, c] = -1
    if window:
        for i, n in enumerate(lens):
            tables[i, :max(0, n - window) // page] = -1
    pages = torch.from_numpy(rng.standard_normal((total, page, 576)).astype(np.float32)).to(DEV).to(torch.bfloat16)
    poison(pages, tables, lens, page)
    q = queries(rng, len(lens), heads, 576, q_scale)
    ws = ws if ws is not None else M.attention_workspace(len(lens), heads, 1, 576)
    td, ld = torch.from_numpy(tables).to(DEV), torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, lse = M.latent_attention(q, pages, td, ld, ws, scale=scale, window=window)
    assert M.get_device_error(ws) == 0
    c = f64(pages)
    compare(out, lse, *R.attention(f64(q), lambda p, t: c[p, t][None], lambda p, t: c[p, t][None, :512], heads, tables,
                                   lens, page, total, scale, window))
    again, al = M.latent_attention(q, pages, td, ld, ws, scale=scale, window=window)
    assert torch.equal(out, again) and torch.equal(lse, al)


@pytest.mark.parametrize("heads", [1, 8, 16, 24, 64, 80, 128])
@pytest.mark.parametrize("page", [16, 64])
def test_latent_ragged(heads, page):
    check_latent(np.random.default_rng(heads + page), LENS, heads, page)


@pytest.mark.parametrize("page", [1, 40, 128, 200])
def test_latent_page_sizes(page):
    check_latent(np.random.default_rng(page), [0, 1, 200, 129], 16, page)


@pytest.mark.parametrize("window", [1, 64, 100])
def test_latent_window(window):
    check_latent(np.random.default_rng(window), [0, 1, 64, 65, 300, 129], 16, 32, window=window)


def test_latent_holes():
    check_latent(np.random.default_rng(3), [300, 64, 128], 64, 32, holes=[(0, 0), (0, 4), (0, 9), (1, 0), (1, 1)])


@pytest.mark.parametrize("batch,top,heads", [(1, 9001, 64), (2, 3000, 128), (160, 200, 16), (33, 1000, 64)])
def test_latent_long_rows_are_split_and_joined(batch, top, heads):
    rng = np.random.default_rng(batch)
    check_latent(rng, [top] + [int(x) for x in rng.integers(0, top + 1, batch - 1)], heads, 64, q_scale=2.0)


def test_latent_one_workspace_for_many_shapes():
    ws = M.attention_workspace(1, 64, 1, 576)
    for i, lens in enumerate(([700], [0, 0], [64] * 40, [5000, 1])):
        check_latent(np.random.default_rng(i), lens, 64, 64, ws=ws)


# ---------------------------------------------------------------------------
# refusals
# ---------------------------------------------------------------------------

def _args():
    q = torch.zeros((2, 8, 64), dtype=torch.bfloat16, device=DEV)
    k = torch.zeros((3, 16, 2, 64), dtype=torch.bfloat16, device=DEV)
    t = torch.zeros((2, 1), dtype=torch.int32, device=DEV)
    n = torch.ones(2, dtype=torch.int32, device=DEV)
    return q, k, t, n, M.attention_workspace(2, 8, 2, 64)


def test_refusals():
    q, k, t, n, ws = _args()
    v = torch.zeros_like(k)
    with pytest.raises(TypeError):
        M.paged_attention(q.float(), k, v, t, n, ws)
    with pytest.raises(TypeError):
        M.paged_attention(q, k.half(), v.half(), t, n, ws)
    with pytest.raises(TypeError):
        M.paged_attention(q, k, v.to(torch.float8_e4m3fn), t, n, ws)
    with pytest.raises(TypeError):
        M.paged_attention(q, k, v, t.long(), n, ws)
    with pytest.raises(ValueError):
        M.paged_attention(q, k, v, t.cpu(), n, ws)
    with pytest.raises(ValueError):
        M.paged_attention(q, k, v[:2], t, n, ws)
    with pytest.raises(ValueError):
        M.paged_attention(q, k, v, t, n[:1], ws)
    with pytest.raises(ValueError):
        M.paged_attention(q[:, :, ::2], k, v, t, n, ws)
    with pytest.raises(ValueError):
        M.paged_attention(q, k, v, t, n, ws, out=torch.zeros((2, 8, 32), dtype=torch.bfloat16, device=DEV))

    def status(fn):
        with pytest.raises(M.MoeW4A16Error) as e:
            fn()
        return e.value.name

    assert status(lambda: M.paged_attention(q[:, :3].contiguous(), k, v, t, n, ws)) == "ERR_INVALID_ARG"
    assert status(lambda: M.paged_attention(q, k, v, t, n, ws[:64])) == "ERR_WORKSPACE"
    assert status(lambda: M.paged_attention(q, k, v, t, n, ws, window=-1)) == "ERR_INVALID_ARG"
    assert status(lambda: M.paged_attention(q, k, v, t, n, ws, scale=math.inf)) == "ERR_INVALID_ARG"
    assert status(lambda: M.paged_attention(q, k, v, t, n, ws, k_scale=2.0)) == "ERR_INVALID_ARG"
    assert status(lambda: M.paged_attention(q, k, v, t[:1], n[:1], ws)) == "ERR_INVALID_ARG"
    odd = torch.zeros((2, 8, 72), dtype=torch.bfloat16, device=DEV)
    ko = torch.zeros((3, 16, 2, 72), dtype=torch.bfloat16, device=DEV)
    assert status(lambda: M.paged_attention(odd, ko, ko, t, n, ws)) == "ERR_UNSUPPORTED"
    flat = torch.zeros(3 * 16 * 2 * 64 + 8, dtype=torch.bfloat16, device=DEV)
    off = flat[4:4 + k.numel()].view(k.shape)
    assert status(lambda: M.paged_attention(q, off, off, t, n, ws)) == "ERR_INVALID_ARG"      # not 16-byte aligned
    lat = torch.zeros((3, 16, 576), dtype=torch.bfloat16, device=DEV)
    ql = torch.zeros((2, 8, 576), dtype=torch.bfloat16, device=DEV)
    wl = M.attention_workspace(2, 8, 1, 576)
    assert status(lambda: M.latent_attention(ql, lat.to(torch.float8_e4m3fn), t, n, wl, 1.0)) == "ERR_UNSUPPORTED"
    with pytest.raises(ValueError):
        M.latent_attention(q, lat, t, n, wl, 1.0)
