"""Page operations against plain sequential forms (exact) and the rows they write."""

import numpy as np
import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu

M = pytest.importorskip("w4a16_int4_mixture_grouped_gb300") if torch.cuda.is_available() else None
DEV = torch.device("cuda", 0) if torch.cuda.is_available() else None


def dev(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def state(rng, pages, seqs, width, lens, page):
    """Sequences of the given lengths on random pages; the rest of the pool free."""
    tables = np.full((seqs, width), -1, dtype=np.int32)
    refs = np.zeros(pages, dtype=np.int32)
    order, at = rng.permutation(pages), 0
    for s, n in enumerate(lens):
        c = R.pages_of(n, page)
        tables[s, :c] = order[at:at + c]
        refs[order[at:at + c]] += 1
        at += c
    out = np.zeros(seqs, dtype=np.int32)
    out[:len(lens)] = lens
    return refs, tables, out


def pool_of(rng, planes, pages, *shape):
    return rng.integers(-30000, 30000, size=(planes, pages) + shape).astype(np.int16)


def on(pool):
    return torch.from_numpy(pool.copy()).to(DEV)


@pytest.mark.parametrize("page", [1, 16, 33])
@pytest.mark.parametrize("pages", [40, 1500, 5000])
def test_extend(page, pages):
    rng = np.random.default_rng(pages + page)
    seqs = 60
    lens = [int(x) for x in rng.integers(0, max(2, pages * page // 200), seqs)]
    refs, tables, ln = state(rng, pages, seqs, pages, lens, page) if sum(R.pages_of(n, page) for n in lens) <= pages \
        else state(rng, pages, seqs, pages, [0] * seqs, page)
    ws = M.cache_workspace(pages, seqs)
    dr, dt, dl = dev(refs), dev(tables), dev(ln)
    tight = False
    for step in range(6):
        ids = rng.permutation(seqs)[:rng.integers(1, seqs + 1)].astype(np.int32)
        counts = None if step % 2 else rng.integers(0, 3 * page + 1, len(ids)).astype(np.int32)
        pos = M.cache_extend(dr, dt, dl, dev(ids), page, ws, counts=None if counts is None else dev(counts))
        want = R.extend(refs, tables, ln, ids, [1] * len(ids) if counts is None else counts, page)
        assert np.array_equal(pos.cpu().numpy(), want)
        assert np.array_equal(dr.cpu().numpy(), refs) and np.array_equal(dt.cpu().numpy(), tables)
        assert np.array_equal(dl.cpu().numpy(), ln)
        tight |= bool((want < 0).any())
        assert M.get_device_error(ws) == (5 if (want < 0).any() else 0)
        M.clear_device_error(ws)
    assert tight or pages > 40


@pytest.mark.parametrize("offset", [0, 1])
def test_free_pages_far_into_a_large_pool(offset):
    """Free pages here and there behind thousands in use, counts at an address that 16 bytes do not divide; then compacted."""
    rng = np.random.default_rng(17)
    page, seqs, pages = 2, 50, 20011
    lens = [int(x) for x in rng.integers(700, 760, seqs)]
    refs, tables, ln = state(rng, pages, seqs, 600, lens, page)
    spare = np.setdiff1d(np.arange(pages), tables[tables >= 0])
    refs[spare] = 1                                                     # in use by others, all but a few
    refs[rng.permutation(spare[spare > 9000])[:40]] = 0
    store = torch.zeros(pages + 4, dtype=torch.int32, device=DEV)
    dr = store[offset:offset + pages]
    dr.copy_(torch.from_numpy(refs))
    dt, dl = dev(tables), dev(ln)
    ws = M.cache_workspace(pages, seqs)
    for _ in range(3):
        ids = rng.permutation(seqs)[:30].astype(np.int32)
        pos = M.cache_extend(dr, dt, dl, dev(ids), page, ws)
        want = R.extend(refs, tables, ln, ids, [1] * len(ids), page)
        assert np.array_equal(pos.cpu().numpy(), want)
        assert np.array_equal(dr.cpu().numpy(), refs) and np.array_equal(dt.cpu().numpy(), tables)
    drop = rng.permutation(pages)[:9000]
    drop = drop[~np.isin(drop, tables[tables >= 0])]
    refs[drop] = 0
    dr.copy_(torch.from_numpy(refs))
    pool = pool_of(rng, 1, pages, 8)
    dp = on(pool)
    new_refs, new_tables, page_map, live = M.cache_compact(dp, dr, dt, ws)
    want_refs, want_tables, want_map, want_live = R.compact(pool, refs, tables)
    assert int(live.item()) == want_live
    assert np.array_equal(page_map.cpu().numpy(), want_map) and np.array_equal(new_refs.cpu().numpy(), want_refs)
    assert np.array_equal(new_tables.cpu().numpy(), want_tables)
    assert np.array_equal(dp.cpu().numpy(), pool)


def test_extend_more_entries_than_a_block_and_bad_ids():
    rng = np.random.default_rng(1)
    page, seqs, pages = 4, 3000, 4000
    lens = [int(x) for x in rng.integers(0, 5, seqs)]
    refs, tables, ln = state(rng, pages, seqs, 3, lens, page)
    ids = rng.permutation(seqs).astype(np.int32)
    ids[[5, 1700]] = [-1, seqs]
    ws = M.cache_workspace(pages, seqs)
    dr, dt, dl = dev(refs), dev(tables), dev(ln)
    pos = M.cache_extend(dr, dt, dl, dev(ids), page, ws)
    want = R.extend(refs, tables, ln, ids, [1] * seqs, page)
    assert np.array_equal(pos.cpu().numpy(), want) and want[5] == -1 and want[1700] == -1
    assert np.array_equal(dr.cpu().numpy(), refs) and np.array_equal(dt.cpu().numpy(), tables)
    assert np.array_equal(dl.cpu().numpy(), ln)
    assert M.get_device_error(ws) in (5, 8)


@pytest.mark.parametrize("planes,page,shape,pages", [(1, 16, (16, 8), 50), (6, 16, (16, 2, 64), 300),
                                                     (2, 5, (5, 8), 2500), (3, 32, (32, 576), 64)])
def test_fork_extend_free(planes, page, shape, pages):
    rng = np.random.default_rng(planes * page)
    parents_n, forks = 7, 3
    seqs = parents_n * (1 + forks)
    lens = [0, 1, page, page + 1, 3 * page, 2 * page - 1, 4 * page + page // 2]
    refs, tables, ln = state(rng, pages, seqs, 8, lens, page)
    hole = tables[6, 1]
    refs[hole] -= 1
    tables[6, 1] = -1                      # a freed page in the middle of a parent
    pool = pool_of(rng, planes, pages, *shape)
    dp, dr, dt, dl = on(pool), dev(refs), dev(tables), dev(ln)
    parents = np.repeat(np.arange(parents_n), forks).astype(np.int32)
    children = np.arange(parents_n, seqs).astype(np.int32)
    ws = M.cache_workspace(pages, seqs)

    def same(err=0):
        assert M.get_device_error(ws) == err
        assert np.array_equal(dt.cpu().numpy(), tables) and np.array_equal(dl.cpu().numpy(), ln)
        assert np.array_equal(dr.cpu().numpy(), refs) and np.array_equal(dp.cpu().numpy(), pool)

    M.cache_fork(dp, dr, dt, dl, dev(parents), dev(children), page, ws)
    R.fork(pool, refs, tables, ln, parents, children, page)
    same()
    pos = M.cache_extend(dr, dt, dl, dev(children), page, ws)
    assert np.array_equal(pos.cpu().numpy(), R.extend(refs, tables, ln, children, [1] * len(children), page))
    same()
    keep = rng.integers(0, 2 * page, len(children)).astype(np.int32)
    M.cache_free(dr, dt, dl, dev(children), page, ws, keep=dev(keep))
    R.free(refs, tables, ln, children, page, keep)
    same()
    M.cache_free(dr, dt, dl, dev(np.concatenate([children, children[:3]])), page, ws)     # three named twice
    R.free(refs, tables, ln, children, page)
    same()
    assert (ln[parents_n:] == 0).all() and (tables[parents_n:] == -1).all()


def test_fork_without_room_and_onto_a_sequence_in_use():
    rng = np.random.default_rng(2)
    page, pages = 16, 6
    refs, tables, ln = state(rng, pages, 6, 4, [20, 40], page)       # five of six pages used
    pool = pool_of(rng, 2, pages, 16, 8)
    dp, dr, dt, dl = on(pool), dev(refs), dev(tables), dev(ln)
    ws = M.cache_workspace(pages, 4)
    ids, to = np.array([0, 1, 0], dtype=np.int32), np.array([2, 3, 4], dtype=np.int32)
    M.cache_fork(dp, dr, dt, dl, dev(ids), dev(to), page, ws)
    R.fork(pool, refs, tables, ln, ids, to, page)
    assert M.get_device_error(ws) == 5
    M.clear_device_error(ws)
    assert ln.tolist() == [20, 40, 20, 0, 0, 0]
    for a, b in ((dp, pool), (dr, refs), (dt, tables), (dl, ln)):
        assert np.array_equal(a.cpu().numpy(), b)
    M.cache_fork(dp, dr, dt, dl, dev(np.array([0], dtype=np.int32)), dev(np.array([1], dtype=np.int32)), page, ws)
    assert M.get_device_error(ws) == 8
    for a, b in ((dp, pool), (dr, refs), (dt, tables), (dl, ln)):
        assert np.array_equal(a.cpu().numpy(), b)


def test_free_of_a_page_without_a_count():
    ws = M.cache_workspace(4, 1)
    refs, tables, lens = dev(np.array([0, 1, 1, 0], dtype=np.int32)), dev(np.array([[0, 1, 9]], dtype=np.int32)), \
        dev(np.array([40], dtype=np.int32))
    M.cache_free(refs, tables, lens, dev(np.array([0], dtype=np.int32)), 16, ws)
    assert M.get_device_error(ws) == 8
    assert refs.tolist() == [0, 0, 1, 0] and tables.tolist() == [[-1, -1, -1]] and lens.tolist() == [0]


@pytest.mark.parametrize("pages,share,planes,shape", [(1, 1.0, 1, (8,)), (16, 0.0, 2, (8,)), (100, 0.5, 3, (5, 8)),
                                                      (1024, 0.3, 2, (16, 64)), (5003, 0.9, 1, (24,)),
                                                      (300, 0.6, 2, (64, 576))])
def test_compact(pages, share, planes, shape):
    rng = np.random.default_rng(pages)
    refs = np.where(rng.random(pages) < share, rng.integers(1, 4, pages), 0).astype(np.int32)
    used = np.nonzero(refs)[0]
    seqs, width = 9, 40
    tables = np.full((seqs, width), -1, dtype=np.int32)
    if len(used):
        picks = rng.choice(used, size=(seqs, width))
        tables = np.where(rng.random((seqs, width)) < 0.7, picks, -1).astype(np.int32)
    pool = pool_of(rng, planes, pages, *shape)
    dp, dr, dt = on(pool), dev(refs), dev(tables)
    ws = M.cache_workspace(pages, 0)
    new_refs, new_tables, page_map, live = M.cache_compact(dp, dr, dt, ws)
    wr, wt, wm, wl = R.compact(pool, refs, tables)
    assert M.get_device_error(ws) == 0 and live.item() == wl
    assert np.array_equal(new_refs.cpu().numpy(), wr) and np.array_equal(new_tables.cpu().numpy(), wt)
    assert np.array_equal(page_map.cpu().numpy(), wm) and np.array_equal(dp.cpu().numpy(), pool)
    assert np.array_equal(dr.cpu().numpy(), refs) and np.array_equal(dt.cpu().numpy(), tables)
    M.cache_compact(dp, dr, dt, ws, refs_out=dr, tables_out=dt)         # in place: the same counts and tables
    assert np.array_equal(dr.cpu().numpy(), wr) and np.array_equal(dt.cpu().numpy(), wt)


def test_copy_of_strided_pools_and_bad_pairs():
    rng = np.random.default_rng(3)
    whole = pool_of(rng, 4, 20, 8, 40)
    d = on(whole)
    view, ref = d[1:4:2, 2:18], whole[1:4:2, 2:18]       # planes 1 and 3, pages 2..17
    ws = M.cache_workspace(16, 8)
    src, dst = np.array([0, 5, 15, -1], dtype=np.int32), np.array([1, 14, 3, -1], dtype=np.int32)
    M.cache_copy(view, dev(src), dev(dst), ws)
    assert M.get_device_error(ws) == 0
    ref[:, dst[:3]] = ref[:, src[:3]]
    assert np.array_equal(d.cpu().numpy(), whole)
    M.cache_copy(view, dev(np.array([16, 2, 0], dtype=np.int32)), dev(np.array([4, -3, 16], dtype=np.int32)), ws)
    assert M.get_device_error(ws) == 8
    assert np.array_equal(d.cpu().numpy(), whole)


def test_copy_past_32_bits():
    pool = torch.empty((1, 70000, 64 * 1024), dtype=torch.int16, device=DEV)      # 9 GB
    pool[0, 69999] = torch.arange(65536, device=DEV).to(torch.int16)
    ws = M.cache_workspace(0, 1)
    M.cache_copy(pool, dev(np.array([69999], dtype=np.int32)), dev(np.array([68000], dtype=np.int32)), ws)
    assert torch.equal(pool[0, 69999], pool[0, 68000]) and M.get_device_error(ws) == 0


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("heads,dim,page,head_major", [(8, 128, 16, False), (1, 64, 7, False), (3, 96, 32, True),
                                                       (2, 16, 1, True)])
def test_append(heads, dim, page, head_major, e4m3):
    rng = np.random.default_rng(heads * dim + page)
    seqs, width, n = 5, 6, 37
    pages = seqs * width
    tables = rng.permutation(pages).reshape(seqs, width).astype(np.int32)
    slots = rng.permutation(seqs * width * page)[:n] if width * page * seqs >= n else np.arange(seqs * width * page)
    n = len(slots)
    seq, pos = (slots // (width * page)).astype(np.int32), (slots % (width * page)).astype(np.int32)
    pos[0] = -1                                                    # a skipped row
    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    shape = (pages, heads, page, dim) if head_major else (pages, page, heads, dim)
    qkv = torch.from_numpy(rng.standard_normal((n, 3 * heads, dim)).astype(np.float32) * 4).to(DEV).to(torch.bfloat16)
    qkv[1, :, 0] = float("nan")
    qkv[2, :, 0] = float("inf")
    qkv[3, :, 0] = -3e38
    qkv[4, :, :] = 0.0078125                                       # ties and subnormals of the 8-bit form
    k, v = qkv[:, heads:2 * heads], qkv[:, 2 * heads:]             # slices of a fused projection
    out, want = [], []
    for t, scale in ((k, 0.02), (v, 0.5)):
        store = torch.zeros(shape, dtype=torch.bfloat16, device=DEV).to(kind)
        out.append(store.transpose(1, 2) if head_major else store)
        ref = torch.zeros((pages, page, heads, dim), dtype=torch.bfloat16, device=DEV).to(kind).view(
            torch.uint8 if e4m3 else torch.bfloat16)
        rows = t
        if e4m3:
            rows = (t.double() / float(np.float32(scale))).float().clamp(-448, 448)   # the exact quotient, rounded once
            rows = rows.to(torch.float8_e4m3fn).view(torch.uint8)
        for i in range(n):
            if pos[i] >= 0:
                ref[tables[seq[i], pos[i] // page], pos[i] % page] = rows[i]
        want.append(ref)
    ws = M.cache_workspace(0, 0)
    ks, vs = (0.02, 0.5) if e4m3 else (1.0, 1.0)
    M.cache_append(k, out[0], dev(tables), dev(seq), dev(pos), ws, v=v, v_pages=out[1], k_scale=ks, v_scale=vs)
    assert M.get_device_error(ws) == 0
    for got, ref in zip(out, want):
        got = got.contiguous()
        raw = got.view(torch.uint8 if e4m3 else torch.int16)
        ref = ref if e4m3 else ref.contiguous().view(torch.int16)
        if e4m3:                                                   # either sign of NaN
            raw, ref = (torch.where((x & 0x7F) == 0x7F, torch.full_like(x, 0x7F), x) for x in (raw, ref))
        assert torch.equal(raw, ref)


def test_append_latent_and_positions_without_a_page():
    rng = np.random.default_rng(4)
    pages = torch.zeros((8, 16, 576), dtype=torch.bfloat16, device=DEV)
    rows = torch.from_numpy(rng.standard_normal((6, 576)).astype(np.float32)).to(DEV).to(torch.bfloat16)
    tables = np.array([[3, -1, 7], [0, 8, -1]], dtype=np.int32)
    seq = np.array([0, 0, 1, 1, 2, 0], dtype=np.int32)
    pos = np.array([5, 20, 15, 17, 0, 48], dtype=np.int32)          # rows 1, 3, 4, 5 have no page
    ws = M.cache_workspace(0, 0)
    M.cache_append(rows, pages, dev(tables), dev(seq), dev(pos), ws)
    assert M.get_device_error(ws) == 8
    want = torch.zeros_like(pages)
    want[3, 5], want[0, 15] = rows[0], rows[2]
    assert torch.equal(pages, want)


def test_append_then_attention_sees_the_rows():
    """What is written is what is read: append token by token, attend after each."""
    rng = np.random.default_rng(5)
    page, heads, dim, steps = 4, 2, 64, 11
    pool = torch.full((2, 8, page, heads, dim), float("nan"), dtype=torch.bfloat16, device=DEV)
    refs = torch.zeros(8, dtype=torch.int32, device=DEV)
    tables = torch.full((1, 4), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(1, dtype=torch.int32, device=DEV)
    ids = torch.zeros(1, dtype=torch.int32, device=DEV)
    ws, wa = M.cache_workspace(8, 1), M.attention_workspace(1, 4, heads, dim)
    ks, vs = [], []
    for _ in range(steps):
        k, v = (torch.from_numpy(rng.standard_normal((1, heads, dim)).astype(np.float32)).to(DEV).to(torch.bfloat16)
                for _ in range(2))
        pos = M.cache_extend(refs, tables, lens, ids, page, ws)
        M.cache_append(k, pool[0], tables, ids, pos, ws, v=v, v_pages=pool[1])
        ks.append(k), vs.append(v)
        q = torch.from_numpy(rng.standard_normal((1, 4, dim)).astype(np.float32)).to(DEV).to(torch.bfloat16)
        out, _ = M.paged_attention(q, pool[0], pool[1], tables, lens, wa)
        kk, vv = torch.cat(ks).double().repeat_interleave(2, 1), torch.cat(vs).double().repeat_interleave(2, 1)
        p = torch.softmax(torch.einsum("hd,lhd->hl", q[0].double(), kk) * dim ** -0.5, 1)
        ref, a = torch.einsum("hl,lhd->hd", p, vv), torch.einsum("hl,lhd->hd", p, vv.abs())
        assert ((out[0].double() - ref).abs() <= 2.0 ** -8 * 1.01 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * a).all()
    assert M.get_device_error(ws) == 0 and M.get_device_error(wa) == 0 and lens.item() == steps


def test_empty_calls_and_refusals():
    ws = M.cache_workspace(4, 2)
    refs, tables, lens = dev(np.zeros(4, dtype=np.int32)), dev(np.full((2, 2), -1, dtype=np.int32)), \
        dev(np.zeros(2, dtype=np.int32))
    none = torch.empty(0, dtype=torch.int32, device=DEV)
    pool = torch.zeros((1, 4, 64), dtype=torch.bfloat16, device=DEV)
    assert M.cache_extend(refs, tables, lens, none, 16, ws).numel() == 0
    M.cache_free(refs, tables, lens, none, 16, ws)
    M.cache_fork(pool, refs, tables, lens, none, none, 16, ws)
    M.cache_copy(pool, none, none, ws)
    one = dev(np.zeros(1, dtype=np.int32))

    def status(fn):
        with pytest.raises(M.MoeW4A16Error) as e:
            fn()
        return e.value.name

    assert status(lambda: M.cache_extend(refs, tables, lens, one, 0, ws)) == "ERR_INVALID_ARG"
    assert status(lambda: M.cache_extend(refs, tables, lens, one, 5000, ws)) == "ERR_INVALID_ARG"
    assert status(lambda: M.cache_extend(refs, tables, lens, one, 16, ws[:256])) == "ERR_WORKSPACE"
    assert status(lambda: M.cache_copy(torch.zeros((1, 4, 7), dtype=torch.bfloat16, device=DEV), one, one, ws)) == \
        "ERR_INVALID_ARG"                                          # pages are not a multiple of 16 bytes
    with pytest.raises(TypeError):
        M.cache_extend(refs.long(), tables, lens, one, 16, ws)
    with pytest.raises(ValueError):
        M.cache_fork(pool, refs[:3], tables, lens, one, one, 16, ws)
    with pytest.raises(ValueError):
        M.cache_copy(pool[:, :, ::2], one, one, ws)
    with pytest.raises(ValueError):
        M.cache_extend(refs, tables, lens[:1], one, 16, ws)
    k = torch.zeros((1, 2, 64), dtype=torch.bfloat16, device=DEV)
    kp = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        M.cache_append(k, kp, tables, one, one, ws)                # keys without values
    with pytest.raises(ValueError):
        M.cache_append(k[:, :1], kp, tables, one, one, ws, v=k[:, :1], v_pages=kp)
    assert status(lambda: M.cache_append(k, kp, tables, one, one, ws, v=k, v_pages=kp, k_scale=2.0)) == "ERR_INVALID_ARG"
