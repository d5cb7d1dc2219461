"""Rotation of positions, alone and on the way into the cache, against the plain 64-bit form."""

import numpy as np
import pytest
import torch

import chunk_ref as C

pytestmark = pytest.mark.gpu

M = pytest.importorskip("w4a16_int4_mixture_grouped_gb300") if torch.cuda.is_available() else None
DEV = torch.device("cuda", 0) if torch.cuda.is_available() else None

SCALINGS = {"none": {}, "linear": dict(factor=4.0), "base": dict(factor=8.0),
            "turns": dict(factor=8.0, trained_length=8192, low=1.0, high=4.0),
            "index": dict(factor=32.0, trained_length=4096, low=1.0, high=32.0)}
FAR = [0, 1, 2, 7, 100, 4095, 4096, 131071, 1 << 20, (1 << 31) - 1, -1, -5000, -(1 << 31)]


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def rows(rng, *shape, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(DEV).to(torch.bfloat16)


def f64(t):
    return t.detach().to(torch.float32).cpu().numpy().astype(np.float64)


def plain(dim, theta=10000.0, scaling="none", **kw):
    if "trained_length" in kw:
        kw["trained"] = kw.pop("trained_length")
    return C.frequencies(dim, theta, scaling, **kw)


def inside(got, ref, bound):
    """BF16: one rounding of a value within bound of ref."""
    err = np.abs(f64(got) - ref)
    limit = bound + 2.0 ** -8 * (np.abs(ref) + bound) + 2.0 ** -133
    assert (err <= limit).all(), (err / limit).max()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads,dim,rot,offset", [(4, 64, 64, 0), (3, 128, 64, 64), (1, 128, 128, 0), (2, 192, 64, 128),
                                                  (5, 96, 32, 0), (2, 256, 256, 0), (1, 576, 64, 512), (7, 80, 16, 8),
                                                  (3, 10, 6, 2), (2, 9, 4, 3), (1, 2, 2, 0), (3, 1500, 1024, 1)])
def test_layouts_and_parts(heads, dim, rot, offset, interleaved):
    rng = np.random.default_rng(dim + rot)
    pos = rng.integers(0, 1 << 20, 13)
    x = rows(rng, 13, heads, dim)
    rotation = M.Rotary(rot, offset=offset, interleaved=interleaved)
    ref, bound = C.rotate(f64(x), pos, plain(rot), offset, interleaved)
    before = x.clone()
    got = M.rotary(x, i32(pos), rotation)
    assert got.is_contiguous() and torch.equal(x, before)
    inside(got, ref, bound)
    still = torch.ones(dim, dtype=torch.bool)
    still[offset:offset + rot] = False
    assert torch.equal(got[:, :, still.to(DEV)], x[:, :, still.to(DEV)])
    same = M.rotary(x, i32(pos), rotation, out=x)                  # in place: the same bits
    assert same is x and torch.equal(x, got)


@pytest.mark.parametrize("scaling", list(SCALINGS))
@pytest.mark.parametrize("theta", [10000.0, 5e5])
def test_scaled_frequencies_at_far_positions(scaling, theta):
    rng = np.random.default_rng(3)
    x = rows(rng, len(FAR), 2, 128)
    kw = SCALINGS[scaling]
    ref, bound = C.rotate(f64(x), FAR, plain(128, theta, scaling, **kw), 0, False, 1.25)
    # frequencies that differ by 2^-50 (two ways of computing a power) turn by 2^-19 of a radian apart at position 2^31
    apart = np.abs(np.array(FAR, dtype=np.float64))[:, None, None] * 2.0 ** -50
    mag = np.abs(f64(x))
    pair = np.concatenate([mag[..., :64] + mag[..., 64:]] * 2, -1)
    inside(M.rotary(x, i32(FAR), M.Rotary(128, theta, scaling=scaling, magnitude=1.25, **kw)), ref, bound + 1.25 * apart * pair)


def test_given_frequencies():
    rng = np.random.default_rng(4)
    given = [3.0, -0.5, 0.0, 1e-9, 100.0, 2 * np.pi, 1e-30, 7.25]
    x = rows(rng, len(FAR), 3, 16)
    ref, bound = C.rotate(f64(x), FAR, np.array(given), 0, True)
    apart = np.abs(np.array(FAR, dtype=np.float64))[:, None, None] * 2.0 ** -45
    pair = np.repeat(np.abs(f64(x)).reshape(len(FAR), 3, 8, 2).sum(-1), 2, -1)
    inside(M.rotary(x, i32(FAR), M.Rotary(16, interleaved=True, scaling="given", given=given)), ref, bound + apart * pair)


@pytest.mark.parametrize("layout", ["slice", "head major", "odd", "odd heads", "broadcast", "strided out"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_strides(layout, interleaved):
    rng = np.random.default_rng(5)
    t, h, d = 9, 4, 64
    pos = rng.integers(0, 5000, t)
    out = None
    if layout == "slice":
        x = rows(rng, t, 10, d)[:, 3:7]
    elif layout == "head major":
        x = rows(rng, h, t, d).transpose(0, 1)
        out = torch.empty((h, t, d), dtype=torch.bfloat16, device=DEV).transpose(0, 1)
    elif layout == "odd":
        x = rows(rng, t * (h * d + 1) + 1)[1:].view(t, -1)[:, :h * d].view(t, h, d)
    elif layout == "odd heads":
        x = rows(rng, t, h, d + 3)[:, :, 2:2 + d]
    elif layout == "broadcast":
        x = rows(rng, t, 1, d).expand(t, h, d)
    else:
        x = rows(rng, t, h, d)
        out = torch.zeros((t, h + 2, d + 8), dtype=torch.bfloat16, device=DEV)[:, 1:1 + h, 4:4 + d]
    rotation = M.Rotary(32, offset=16, interleaved=interleaved)
    ref, bound = C.rotate(f64(x), pos, plain(32), 16, interleaved)
    got = M.rotary(x, i32(pos), rotation, out=out)
    inside(got, ref, bound)
    assert torch.equal(got.contiguous(), M.rotary(x.contiguous(), i32(pos), rotation))
    if layout != "broadcast":
        want = got.clone()
        M.rotary(x, i32(pos), rotation, out=x)
        assert torch.equal(x, want)


@pytest.mark.parametrize("t,h", [(0, 3), (1, 1), (1, 64), (300, 1), (5000, 2), (2, 4096)])
def test_token_and_head_counts(t, h):
    rng = np.random.default_rng(6)
    pos = rng.integers(0, 9000, t)
    x = rows(rng, t, h, 32)
    ref, bound = C.rotate(f64(x), pos, plain(32), 0, False)
    inside(M.rotary(x, i32(pos), M.Rotary(32)), ref, bound)


def test_turning_back_and_infinities():
    rng = np.random.default_rng(7)
    x = rows(rng, 8, 2, 64)
    pos = i32(rng.integers(0, 1 << 30, 8))
    rotation = M.Rotary(64)
    there = M.rotary(x, pos, rotation)
    back = M.rotary(there, -pos, rotation)
    # two roundings of each channel of a pair, turned by sine and cosine
    pair = torch.cat([(x[..., :32].float().square() + x[..., 32:].float().square()).sqrt()] * 2, -1)
    assert ((back.float() - x.float()).abs() <= (2.0 ** -8 * 2.5) * pair).all()
    x[3, 1, 5] = float("nan")
    x[4, 0, 7] = float("inf")
    got = M.rotary(x, pos, rotation)
    bad = ~torch.isfinite(got)
    want = torch.zeros_like(bad)
    want[3, 1, [5, 37]] = True
    want[4, 0, [7, 39]] = True
    assert torch.equal(bad, want)


# ---------------------------------------------------------------------------
# on the way into the cache
# ---------------------------------------------------------------------------

def cache_for(rng, pos, seqs, page, shape, e4m3, latent):
    """Tables of distinct pages for every sequence, pages filled with a marker value."""
    width = max(1, int(max(pos, default=0)) // page + 1)
    n = max(seqs, default=0) + 1
    tables = rng.permutation(n * width).astype(np.int32).reshape(n, width)
    full = (n * width, page) + shape
    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    return tables, [torch.full(full, 3.0, dtype=torch.float32, device=DEV).to(kind) for _ in range(1 if latent else 2)]


def check_append(rng, t, heads, kv, dim, rot, offset, interleaved, page, e4m3=False, latent=False, with_q=True, in_place=False,
                 skip=()):
    seqs = [int(x) for x in rng.integers(0, 3, t)]
    pos = np.zeros(t, dtype=np.int64)
    for s in range(3):                                   # distinct slots
        mine = [i for i in range(t) if seqs[i] == s]
        pos[mine] = rng.permutation(4 * max(1, len(mine)) + 3)[:len(mine)]
    tables, pages = cache_for(rng, pos, seqs, page, (dim,) if latent else (kv, dim), e4m3, latent)
    for i in skip:
        pos[i] = -1 - i
    x = rows(rng, t, heads + (1 if latent else 2 * kv), dim, scale=2.0)
    q = x[:, :heads] if with_q else None
    k, v = (x[:, heads], None) if latent else (x[:, heads:heads + kv], x[:, heads + kv:])
    k0, v0, q0 = f64(k), None if latent else f64(v), f64(q) if with_q else None
    ks, vs = (0.02, 0.03) if e4m3 else (1.0, 1.0)
    rotation = M.Rotary(rot, offset=offset, interleaved=interleaved, magnitude=0.75)
    ws = M.cache_workspace(0, 1)
    got = M.cache_append_rotary(q, k, pages[0], i32(tables), i32(seqs), i32(pos), rotation, ws, v=v,
                                v_pages=None if latent else pages[1], k_scale=ks, v_scale=vs, q_out=q if in_place else None)
    assert M.get_device_error(ws) == 0
    if with_q:
        assert (got is q) if in_place else got.is_contiguous()
        inside(got, *C.rotate(q0, pos, plain(rot), offset, interleaved, 0.75))
    else:
        assert got is None
    ref, bound = C.rotate(k0[:, None] if latent else k0, pos, plain(rot), offset, interleaved, 0.75)
    if latent:
        ref, bound = ref[:, 0], bound[:, 0]
    expect = [(pages[0], ref, bound, ks)] + ([] if latent else [(pages[1], v0, np.zeros_like(v0), vs)])
    for stored, want, off, scale in expect:
        held = f64(stored)
        untouched = np.ones(held.shape[:2], dtype=bool)
        for i in range(t):
            if pos[i] < 0:
                continue
            p, slot = tables[seqs[i], pos[i] // page], pos[i] % page
            untouched[p, slot] = False
            w, o = want[i] / scale, off[i] / scale
            if e4m3:
                w = np.clip(w, -448, 448)
                limit = o + 2.0 ** -4 * (np.abs(w) + o) + 2.0 ** -10
            else:
                limit = o + 2.0 ** -8 * (np.abs(w) + o) + 2.0 ** -133
            if not e4m3 and not off.any():
                limit = 0
            assert (np.abs(held[p, slot] - w) <= limit).all()
        assert (held[untouched] == 3.0).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads,kv,dim,rot,offset,page", [(8, 2, 128, 128, 0, 16), (4, 4, 64, 32, 32, 7), (5, 1, 96, 48, 0, 48),
                                                          (16, 2, 256, 64, 192, 64), (3, 3, 80, 16, 8, 1)])
def test_append(heads, kv, dim, rot, offset, page, interleaved, e4m3):
    rng = np.random.default_rng(dim + rot)
    for t in (1, 3, 70):
        check_append(rng, t, heads, kv, dim, rot, offset, interleaved, page, e4m3)
    check_append(rng, 9, heads, kv, dim, rot, offset, interleaved, page, e4m3, with_q=False)
    check_append(rng, 9, heads, kv, dim, rot, offset, interleaved, page, e4m3, in_place=True, skip=(0, 4, 8))


@pytest.mark.parametrize("interleaved", [False, True])
def test_append_latent(interleaved):
    rng = np.random.default_rng(8)
    for t in (1, 40):
        check_append(rng, t, 16, 1, 576, 64, 512, interleaved, 64, latent=True)
    check_append(rng, 700, 2, 1, 576, 64, 512, interleaved, 16, latent=True)


@pytest.mark.parametrize("t", [2431, 2437, 4864, 5003])
@pytest.mark.parametrize("e4m3,interleaved,in_place", [(False, False, False), (True, True, True), (True, False, False)])
def test_append_of_many_tokens(t, e4m3, interleaved, in_place):
    """Groups of tokens, the last one not full, rows without a place between them."""
    rng = np.random.default_rng(t)
    check_append(rng, t, 2, 1, 64, 32, 16, interleaved, 16, e4m3, in_place=in_place, skip=(0, 1, 2, 3, 6, 2000, t - 1))


@pytest.mark.parametrize("t", [2437, 4865])
def test_many_tokens(t):
    rng = np.random.default_rng(t)
    x, pos = rows(rng, t, 3, 96), i32(rng.integers(-5, 10 ** 6, t))
    rotation = M.Rotary(64, offset=16)
    want = M.rotary(x, pos, rotation)
    inside(want, *C.rotate(f64(x), pos.tolist(), plain(64), 16, False, 1.0))
    assert torch.equal(M.rotary(x, pos, rotation, out=x), want)


def test_append_is_rotary_then_append():
    """Bit for bit over BF16 pages, and the plain append's elements for the values."""
    rng = np.random.default_rng(9)
    t, page = 200, 32
    seqs = rng.integers(0, 4, t)
    pos = np.arange(t)
    tables, (ka, va) = cache_for(rng, pos, list(seqs), page, (2, 128), False, False)
    kb, vb = ka.clone(), va.clone()
    q, k, v = rows(rng, t, 8, 128), rows(rng, t, 2, 128), rows(rng, t, 2, 128)
    rotation, ws = M.Rotary(128, 5e5), M.cache_workspace(0, 1)
    args = i32(tables), i32(seqs), i32(pos)
    got = M.cache_append_rotary(q, k, ka, *args, rotation, ws, v=v, v_pages=va)
    M.cache_append(M.rotary(k, args[2], rotation), kb, *args, ws, v=v, v_pages=vb)
    assert torch.equal(got, M.rotary(q, args[2], rotation)) and torch.equal(ka, kb) and torch.equal(va, vb)


def test_append_slots_without_a_page_are_recorded():
    rng = np.random.default_rng(10)
    tables = np.array([[0, -1], [1, 9]], dtype=np.int32)
    rotation = M.Rotary(64)
    for seq, pos, bad in ((0, 3, False), (0, 20, True), (1, 20, True), (0, 40, True), (2, 0, True), (-1, 0, True), (5, -3, False)):
        k_pages = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16, device=DEV)
        v_pages, ws = torch.zeros_like(k_pages), M.cache_workspace(0, 1)
        q, k, v = rows(rng, 1, 4, 64), rows(rng, 1, 2, 64), rows(rng, 1, 2, 64)
        got = M.cache_append_rotary(q, k, k_pages, i32(tables), i32([seq]), i32([pos]), rotation, ws, v=v, v_pages=v_pages)
        assert M.get_device_error(ws) == (8 if bad else 0)
        assert torch.equal(got, M.rotary(q, i32([pos]), rotation))
        stored = not bad and pos >= 0
        assert bool((k_pages != 0).any()) == stored and bool((v_pages != 0).any()) == stored


def test_streams_and_graphs():
    rng = np.random.default_rng(11)
    x, pos, rotation = rows(rng, 30, 4, 64), i32(rng.integers(0, 900, 30)), M.Rotary(64, interleaved=True)
    want = M.rotary(x, pos, rotation)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = M.rotary(x, pos, rotation)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    tables, (kp, vp) = cache_for(rng, range(30), [0], 16, (4, 64), False, False)
    td, sd, ws = i32(tables), i32([0] * 30), M.cache_workspace(0, 1)
    at = i32(np.arange(30))
    out, q_out = torch.zeros_like(x), torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.rotary(x, pos, rotation, out=out)
        M.cache_append_rotary(x, x, kp, td, sd, at, rotation, ws, v=x, v_pages=vp, q_out=q_out)
    for step in range(2):
        pos.copy_(i32(rng.integers(0, 900, 30)))
        at.copy_(i32(rng.permutation(30)))
        x.copy_(rows(rng, 30, 4, 64))
        graph.replay()
        assert torch.equal(out, M.rotary(x, pos, rotation)) and torch.equal(q_out, M.rotary(x, at, rotation))
        page = td[0, (at // 16).long()].long()
        assert torch.equal(kp[page, (at % 16).long()], q_out) and torch.equal(vp[page, (at % 16).long()], x)


def test_refusals():
    rng = np.random.default_rng(12)
    x, pos, rotation = rows(rng, 4, 2, 64), i32([1, 2, 3, 4]), M.Rotary(64)
    for error, args, kw in ((TypeError, (x.float(), pos, rotation), {}), (TypeError, (x, pos.long(), rotation), {}),
                            (ValueError, (x, pos[:3], rotation), {}), (ValueError, (x[0], pos, rotation), {}),
                            (ValueError, (x, pos.cpu(), rotation), {}), (ValueError, (x, pos, rotation), dict(out=x[:3])),
                            (ValueError, (x[..., ::2], pos, M.Rotary(32)), {})):
        with pytest.raises(error):
            M.rotary(*args, **kw)
    for args, kw in (((x[..., :32], pos, rotation), {}), ((x, pos, M.Rotary(32, offset=34)), {}),
                     ((x, pos, rotation), dict(out=x[:1].expand(4, 2, 64))),
                     ((x, pos, rotation), dict(out=x.transpose(0, 1).contiguous().transpose(0, 1)[:, :1].expand(4, 2, 64)))):
        with pytest.raises(M.MoeW4A16Error) as e:
            M.rotary(*args, **kw)
        assert e.value.name == "ERR_INVALID_ARG"
    k_pages = torch.zeros((4, 16, 2, 64), dtype=torch.bfloat16, device=DEV)
    good = dict(q=x, k=x, k_pages=k_pages, tables=i32([[0]]), seq_ids=i32([0] * 4), positions=pos, rotary=rotation,
                ws=M.cache_workspace(0, 1), v=x, v_pages=k_pages)
    for error, kw in ((TypeError, dict(q=x.float())), (ValueError, dict(q=x[:3])), (ValueError, dict(v=None)),
                      (ValueError, dict(q=None, q_out=x)), (ValueError, dict(q_out=x[:, :1])), (ValueError, dict(k=x[..., :32].contiguous())),
                      (ValueError, dict(positions=pos[:2])), (TypeError, dict(seq_ids=pos.float()))):
        with pytest.raises(error):
            M.cache_append_rotary(**{**good, **kw})
    for kw, name in ((dict(rotary=M.Rotary(8)), "ERR_UNSUPPORTED"), (dict(rotary=M.Rotary(16, offset=4)), "ERR_UNSUPPORTED"),
                     (dict(rotary=M.Rotary(128)), "ERR_INVALID_ARG"), (dict(k_scale=2.0), "ERR_INVALID_ARG"),
                     (dict(ws=torch.zeros(16, dtype=torch.uint8, device=DEV)), "ERR_WORKSPACE")):
        with pytest.raises(M.MoeW4A16Error) as e:
            M.cache_append_rotary(**{**good, **kw})
        assert e.value.name == name


def test_append_turns_queries_beside_keys_and_values_of_one_buffer():
    """Queries in place, or to a free part of each row, beside the keys and values: refused only where they meet."""
    rng = np.random.default_rng(75)
    t, h, kv, d, page = 40, 4, 2, 64, 16
    pos = np.arange(t)
    tables, (ka, va) = cache_for(rng, pos, [0], page, (kv, d), False, False)
    kb, vb = ka.clone(), va.clone()
    buffer = rows(rng, t, 2 * h + 2 * kv, d)
    q, k, v, spare = buffer[:, :h], buffer[:, h:h + kv], buffer[:, h + kv:h + 2 * kv], buffer[:, h + 2 * kv:]
    rotation, ws = M.Rotary(d), M.cache_workspace(0, 1)
    args = i32(tables), i32([0] * t), i32(pos), rotation, ws
    want = M.cache_append_rotary(q.contiguous(), k.contiguous(), ka, *args, v=v.contiguous(), v_pages=va)
    for bad in (buffer[:, 1:1 + h], buffer[:, h + kv + 1:2 * h + kv + 1], buffer[:, h:2 * h], buffer.view(-1)[8:8 + t * h * d].view(t, h, d)):
        with pytest.raises(M.MoeW4A16Error) as e:
            M.cache_append_rotary(q, k, kb, *args, v=v, v_pages=vb, q_out=bad)
        assert e.value.name == "ERR_INVALID_ARG"
    for out in (spare, q):
        got = M.cache_append_rotary(q, k, kb, *args, v=v, v_pages=vb, q_out=out)
        assert got is out and torch.equal(got, want) and torch.equal(ka, kb) and torch.equal(va, vb)


def test_outputs_in_the_buffer_of_the_rows():
    """Both anywhere in one buffer, with strides of all kinds: refused where a byte is in both, else turned as from apart."""
    rng = np.random.default_rng(76)
    flat = rows(rng, 6000)
    kept, met, apart = flat.clone(), 0, 0
    for trial in range(600):
        t, h, d = (int(rng.integers(1, n)) for n in (7, 6, 5))
        d *= 2

        def strides():
            gaps = [int(x) * int(rng.integers(0, 2)) for x in rng.integers(0, 90, 2)]
            if rng.integers(0, 2):
                hs = d + gaps[0]
                return (h - 1) * hs + d + gaps[1], hs
            ts = d + gaps[0]
            return ts, (t - 1) * ts + d + gaps[1]

        so = strides()
        sx = [so, strides(), tuple(int(x) for x in rng.integers(0, 60, 2))][int(rng.integers(0, 3))]
        ax, ao = (int(x) for x in rng.integers(0, 400, 2))
        places = [{a + i * s[0] + j * s[1] + c for i in range(t) for j in range(h) for c in range(d)} for a, s in ((ax, sx), (ao, so))]
        x, out = (flat.as_strided((t, h, d), s + (1,), a) for a, s in ((ax, sx), (ao, so)))
        # in place: the same address, and the same strides where there is more than one
        same = ax == ao and (t == 1 or sx[0] == so[0]) and (h == 1 or sx[1] == so[1])
        rotation, pos = M.Rotary(2, offset=d - 2), i32(rng.integers(0, 99, t))
        if places[0] & places[1] and not same:
            met += 1
            with pytest.raises(M.MoeW4A16Error) as e:
                M.rotary(x, pos, rotation, out=out)
            assert e.value.name == "ERR_INVALID_ARG" and torch.equal(flat, kept)
        else:
            apart += 1
            want = M.rotary(x.contiguous(), pos, rotation)
            M.rotary(x, pos, rotation, out=out)
            assert torch.equal(out, want)
            kept.copy_(flat)
    assert met > 50 and apart > 50
