"""Chunks through the cache and the layer: prompts, drafts and single tokens as a serving loop sends them, against dense
attention of the whole sequences in 64 bits."""

import math
import os
import sys

import numpy as np
import pytest
import torch

import chunk_ref as C
from conftest import ROOT
from gpu_util import prepare_dev, random_weights

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    M = pytest.importorskip("w4a16_int4_mixture_grouped_gb300")
    from w4a16_int4_mixture_grouped_gb300 import pipeline
    from w4a16_int4_mixture_grouped_gb300.cache import PagedCache
    DEV = torch.device("cuda", 0)

HEADS, KV_HEADS, DIM, PAGE = 8, 2, 64, 16


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def rows(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


def compare(out, ref, bound):
    err = (out.double() - ref).abs()
    assert (err <= bound).all(), (err / bound.clamp(min=1e-300)).max().item()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("window", [0, 37])
def test_prompt_drafts_and_single_tokens(kind, window):
    """Three sequences: prompts in chunks (one of them padded), forks, drafts verified four at a time, single tokens, with
    the pages behind a window freed. Each step's attention is checked against the pages, the pages against the rows put in."""
    g = torch.Generator(device="cuda").manual_seed(5)
    e4m3 = kind == "e4m3"
    cache = PagedCache(2, 64, PAGE, 6, 16, HEADS, KV_HEADS, DIM, dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16,
                       **(dict(k_scale=0.02, v_scale=0.03) if e4m3 else {}))
    rotary = M.Rotary(DIM, 5e5, scaling="turns", factor=8.0, trained_length=64, low=1.0, high=4.0)
    freqs = C.frequencies(DIM, 5e5, "turns", 8.0, 64, 1.0, 4.0)
    sent = {s: [[], []] for s in range(6)}              # keys and values of every token, in 64 bits, keys turned
    plan = [("chunk", [0, 1, 2], [50, 7, 33], 0), ("chunk", [1, 0], [64, 1], 5), ("one", [0, 1, 2], None, 0), ("fork", [1, 2], [3, 4], 0),
            ("chunk", [0, 3, 4, 1], [4, 4, 4, 0], 2), ("one", [4, 3], None, 0), ("chunk", [2], [90], 0)]
    for what, seqs, counts, pad in plan:
        if what == "fork":
            cache.fork(i32(seqs), i32(counts))
            for a, b in zip(seqs, counts):
                sent[b] = [list(sent[a][0]), list(sent[a][1])]
            continue
        single = what == "one"
        counts = [1] * len(seqs) if single else counts
        starts = [0] + [int(x) for x in np.cumsum(counts)]
        t = starts[-1] + pad
        q, k, v = rows(g, t, HEADS, DIM), rows(g, t, KV_HEADS, DIM), rows(g, t, KV_HEADS, DIM)
        before = [len(sent[s][0]) for s in seqs]
        if single:
            seq_rows, pos = i32(seqs), cache.extend(i32(seqs))
        else:
            seq_rows, pos = cache.extend_chunk(i32(seqs), i32(starts), t)
        want = [b + j for b, c in zip(before, counts) for j in range(c)] + [-1] * pad
        assert pos.tolist() == want and seq_rows[:starts[-1]].tolist() == [s for s, c in zip(seqs, counts) for _ in range(c)]
        for layer in range(2):
            turned = cache.append_rotary(layer, q, k, v, seq_rows, pos, rotary)
            if window and layer == 1:
                # a chunk's first row still sees window - 1 tokens before it
                cache.free(i32(seqs), keep=i32([window + c for c in counts]))
            out = cache.attend(layer, turned, i32(seqs), 0.125, window) if single else \
                cache.attend_chunk(layer, turned, i32(starts), i32(seqs), 0.125, window)
            kp, vp = cache.pages(layer)
            ref = C.attention(turned[:starts[-1]], starts, kp, vp, cache.tables.tolist(), cache.lens.tolist(), 0.125, window,
                              cache.k_scale, cache.v_scale, seqs)
            compare(out[:starts[-1]], ref[0], ref[1])
            assert (out[starts[-1]:] == 0).all()
        cache.check()
        kt, kb = C.rotate(k.double().cpu().numpy(), pos.tolist(), freqs, 0, False)
        for i, s in enumerate(seqs):
            for j in range(starts[i], starts[i + 1]):
                sent[s][0].append((kt[j], kb[j]))
                sent[s][1].append(v[j].double().cpu().numpy())
        # the pages hold what was sent
        tables, (kp, vp) = cache.tables.tolist(), cache.pages(1)
        for s in seqs:
            for j in range(len(sent[s][0])):
                page = tables[s][j // PAGE]
                if page < 0:
                    continue
                key, off = sent[s][0][j]
                got_k = kp[page, j % PAGE].double().cpu().numpy() * cache.k_scale
                got_v = vp[page, j % PAGE].double().cpu().numpy() * cache.v_scale
                if e4m3:          # the element nearest to x / scale (half a step), or its last subnormal's
                    assert (np.abs(got_k - key) <= 2.0 ** -4 * np.abs(key) * 1.01 + off * 1.1 + 2.0 ** -10 * cache.k_scale).all()
                    assert (np.abs(got_v - sent[s][1][j]) <= 2.0 ** -4 * np.abs(sent[s][1][j]) * 1.01 + 2.0 ** -10 * cache.v_scale).all()
                else:
                    assert (np.abs(got_k - key) <= 2.0 ** -8 * np.abs(key) * 1.01 + off * 1.01 + 2.0 ** -133).all()
                    assert np.array_equal(got_v, sent[s][1][j])


def test_a_chunk_that_does_not_fit_stands_at_minus_one():
    cache = PagedCache(1, 4, PAGE, 3, 4, HEADS, KV_HEADS, DIM)
    seqs, pos = cache.extend_chunk(i32([0, 1, 2]), i32([0, 20, 60, 70]), 75)
    assert pos.tolist() == list(range(20)) + [-1] * 40 + [-1] * 10 + [-1] * 5 and seqs[:70].tolist() == [0] * 20 + [1] * 40 + [2] * 10
    assert cache.lens.tolist() == [20, 0, 0]
    with pytest.raises(M.MoeW4A16Error) as e:
        cache.check()
    assert e.value.name == "ERR_CAPACITY"


def test_no_chunks():
    cache = PagedCache(1, 4, PAGE, 3, 4, HEADS, KV_HEADS, DIM)
    seqs, pos = cache.extend_chunk(i32([]), i32([0]), 5)
    assert pos.tolist() == [-1] * 5 and seqs.shape == (5,)
    g = torch.Generator(device="cuda").manual_seed(7)
    q = cache.append_rotary(0, rows(g, 5, HEADS, DIM), *(rows(g, 5, KV_HEADS, DIM) for _ in range(2)), seqs, pos, M.Rotary(DIM))
    assert (cache.attend_chunk(0, q, i32([0]), i32([]), 0.125) == 0).all()
    seqs, pos = cache.extend_chunk(i32([1]), i32([0, 0]), 0)
    assert pos.shape == (0,) and cache.attend_chunk(0, q[:0], i32([0, 0]), i32([1]), 0.125).shape == (0, HEADS, DIM)
    cache.check()


def test_a_latent_cache_turns_its_rows_and_refuses_chunks():
    g = torch.Generator(device="cuda").manual_seed(6)
    cache = PagedCache(1, 8, PAGE, 2, 4, 4)
    rotary = M.Rotary(64, offset=512, interleaved=True)
    freqs = C.frequencies(64, 10000.0)
    kept = []
    for _ in range(20):
        q, k = rows(g, 2, 4, 576), rows(g, 2, 576)
        pos = cache.extend(i32([1, 0]))
        turned = cache.append_rotary(0, q, k, None, i32([1, 0]), pos, rotary)
        out = cache.attend(0, turned, i32([1, 0]), 0.07)
        kept.append(C.rotate(k.double().cpu().numpy()[:, None], pos.tolist(), freqs, 512, True)[0][:, 0])
    cache.check()
    # the last step, from the rows in 64 bits: a rounding of each row (2^-8) in the score and in the value
    keys = np.stack(kept)                                      # [20, 2, 576]
    qt = C.rotate(q.double().cpu().numpy(), [19, 19], freqs, 512, True)[0]
    for b in range(2):
        s = qt[b] @ keys[:, b].T * 0.07
        e = 2 * 2.0 ** -8 * 1.1 * (np.abs(qt[b]) @ np.abs(keys[:, b]).T * 0.07).max(1)
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        want, size = p @ keys[:, b, :512], p @ np.abs(keys[:, b, :512])
        assert (np.abs(out[b].double().cpu().numpy() - want) <= 2.0 ** -7 * size * 1.5 + 2 * np.expm1(e)[:, None] * size).all()
    with pytest.raises(ValueError):
        cache.attend_chunk(0, turned, i32([0, 2]), i32([0]), 0.07)


def layer_for(cache, batch, hidden=512, window=0, rotary=None, seed=3):
    rng = np.random.default_rng(seed)
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape, scale=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    inter, experts = 256, 8
    (q1, s1), (q2, s2) = random_weights(rng, experts, 2 * inter, hidden), random_weights(rng, experts, hidden, inter)
    w1, w2 = prepare_dev(q1, s1, M.MODE_GATE_UP, DEV), prepare_dev(q2, s2, M.MODE_PLAIN, DEV)
    weights = (rand(hidden, (HEADS + 2 * KV_HEADS) * DIM, scale=hidden ** -0.5), rand(HEADS * DIM, hidden, scale=(HEADS * DIM) ** -0.5),
               rand(hidden, experts, scale=0.1))
    norm = rand(hidden, scale=0.2) + 1
    return [pipeline.DecoderLayer(cache, 0, pipeline.MoEFFN(w1, w2, n, 2), HEADS, *weights, norm, window=window, rotary=rotary)
            for n in batch]


def test_the_layer_over_chunks_and_single_tokens():
    """DecoderLayer.forward over a padded batch of chunks: its attention sees turned queries and keys, and what it returns
    for a token is, to within its products' roundings, what the token gives by itself."""
    g = torch.Generator(device="cuda").manual_seed(8)
    rotary = M.Rotary(DIM)
    caches = [PagedCache(1, 32, PAGE, 2, 8, HEADS, KV_HEADS, DIM) for _ in range(2)]
    whole, = layer_for(caches[0], [48], rotary=rotary)
    single, = layer_for(caches[1], [2], rotary=rotary)
    starts, seqs = i32([0, 25, 45]), i32([1, 0])
    x, y = rows(g, 48, 512), rows(g, 48, 512)
    seq_rows, pos = caches[0].extend_chunk(seqs, starts, 48)
    seen = {}
    real = caches[0].attend_chunk
    caches[0].attend_chunk = lambda layer, q, *a: seen.setdefault("out", real(layer, seen.setdefault("q", q), *a))
    h, nxt = whole.forward(x, y, seq_rows, pos, chunk=(starts, seqs))
    assert nxt is None and h.shape == x.shape and torch.isfinite(h).all()
    q, k, v = whole.project(y, pos)
    assert torch.equal(seen["q"], M.rotary(q, pos, rotary))
    kp, vp = caches[0].pages(0)
    ref = C.attention(seen["q"], [0, 25, 45], kp, vp, caches[0].tables.tolist(), caches[0].lens.tolist(), DIM ** -0.5, seq_ids=[1, 0])
    compare(seen["out"][:45], ref[0][:45], ref[1][:45])
    # token by token: the last of each sequence's first 20
    for i in range(20):
        at = torch.stack([x[i], x[25 + i]]), torch.stack([y[i], y[25 + i]])
        one, _ = single.forward(*at, seqs, caches[1].extend(seqs))
        got = torch.stack([h[i], h[25 + i]])
        close = (one.float() - got.float()).abs() <= 0.02 * (1 + got.float().abs())
        assert close.float().mean() > 0.99                    # (a router's near tie may send a token elsewhere)
    for c in caches:
        c.check()


def test_a_captured_prompt_and_an_eager_one():
    """A prompt's chunk captured into a graph and replayed over other sequences and lengths."""
    g = torch.Generator(device="cuda").manual_seed(9)
    rotary = M.Rotary(DIM)
    cache = PagedCache(1, 64, PAGE, 4, 8, HEADS, KV_HEADS, DIM)
    q, k, v = rows(g, 40, HEADS, DIM), rows(g, 40, KV_HEADS, DIM), rows(g, 40, KV_HEADS, DIM)
    starts, seqs = i32([0, 30, 40]), i32([0, 1])
    out = torch.zeros_like(q)

    def step():
        seq_rows, pos = cache.extend_chunk(seqs, starts, 40)
        out.copy_(cache.attend_chunk(0, cache.append_rotary(0, q, k, v, seq_rows, pos, rotary), starts, seqs, 0.125))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    want = out.clone()
    cache.free(i32([0, 1]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    graph.replay()
    assert torch.equal(out, want) and cache.lens.tolist() == [30, 10, 0, 0]
    seqs.copy_(i32([2, 3]))
    starts.copy_(i32([0, 5, 40]))
    graph.replay()
    kp, vp = cache.pages(0)
    ref = C.attention(M.rotary(q, i32(list(range(5)) + list(range(35))), rotary), [0, 5, 40], kp, vp, cache.tables.tolist(),
                      cache.lens.tolist(), 0.125, seq_ids=[2, 3])
    compare(out, ref[0], ref[1])
    cache.check()


@pytest.mark.parametrize("latent,e4m3,prompt", [(False, False, 5), (False, True, 30), (True, False, 9)])
def test_the_example_with_a_prompt(latent, e4m3, prompt):
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import decode
    finally:
        sys.path.pop(0)
    decode.main(latent, e4m3, steps=20, prompt=prompt)


@pytest.mark.parametrize("e4m3", [False, True])
def test_a_chunk_that_does_not_fit_attends_to_nothing(e4m3):
    """Two sequences with tokens, one with a chunk that the pool has no room for: its rows are not the tokens that the
    sequence ends with, so they see none of them; the other sequence's are what they are without it. Then the chunk goes in,
    a page having been given back."""
    g = torch.Generator(device="cuda").manual_seed(12)
    cache = PagedCache(1, 8, PAGE, 3, 8, HEADS, KV_HEADS, DIM, dtype=torch.float8_e4m3fn if e4m3 else torch.bfloat16)
    rotary = M.Rotary(DIM)

    def step(counts, seqs):
        starts = i32([0] + [int(x) for x in np.cumsum(counts)])
        t = sum(counts) + 3
        q, k, v = rows(g, t, HEADS, DIM), rows(g, t, KV_HEADS, DIM), rows(g, t, KV_HEADS, DIM)
        seq_rows, pos = cache.extend_chunk(i32(seqs), starts, t)
        q = cache.append_rotary(0, q, k, v, seq_rows, pos, rotary)
        return q, starts, pos, cache.attend_chunk(0, q, starts, i32(seqs), 0.125, 0, pos)

    def right(q, starts, out, seqs, at):
        kp, vp = cache.pages(0)
        ref = C.attention(q, starts.tolist(), kp, vp, cache.tables.tolist(), cache.lens.tolist(), 0.125, seq_ids=seqs)
        compare(out[at], ref[0][at], ref[1][at])

    q, starts, pos, out = step([40, 20, 30], [0, 1, 2])                # 3 + 2 + 2 pages of 8
    right(q, starts, out, [0, 1, 2], slice(0, 90))
    cache.check()
    q, starts, pos, out = step([12, 30], [0, 1])                       # the last page, then two of none
    assert pos.tolist() == list(range(40, 52)) + [-1] * 33 and cache.lens.tolist() == [52, 20, 30]
    assert (out[12:] == 0).all()
    right(q, starts, out, [0, 1], slice(0, 12))
    kp, vp = cache.pages(0)
    for positions, lse_there in ((pos, False), (None, True)):
        lse = M.paged_chunk_attention(q, starts, kp, vp, cache.tables, cache.lens, cache.attn_ws, scale=0.125, seq_ids=i32([0, 1]),
                                      positions=positions)[1]
        assert torch.isfinite(lse[:12]).all()
        assert torch.isfinite(lse[32:42]).any() if lse_there else (lse[12:42] == -math.inf).all()
    assert M.get_device_error(cache.attn_ws) == 0                      # the append's error is the cache's
    with pytest.raises(M.MoeW4A16Error) as e:
        cache.check()
    assert e.value.name == "ERR_CAPACITY"
    cache.check()
    cache.free(i32([2]))
    q, starts, pos, out = step([30, 12], [1, 0])
    assert cache.lens.tolist() == [64, 50, 0]
    right(q, starts, out, [1, 0], slice(0, 42))
    cache.check()


def test_the_layer_leaves_a_chunk_out_that_does_not_fit():
    """DecoderLayer.forward: attention of zeros for it, so that its residual stream differs from its input by the FFN of its
    own norm alone; the same for a chunk of a sequence without tokens."""
    g = torch.Generator(device="cuda").manual_seed(13)
    cache = PagedCache(1, 6, PAGE, 2, 8, HEADS, KV_HEADS, DIM)
    layer, = layer_for(cache, [48], rotary=M.Rotary(DIM))
    seen = []
    real = cache.attend_chunk
    cache.attend_chunk = lambda *a: seen.append(real(*a)) or seen[-1]
    x, y = rows(g, 48, 512), rows(g, 48, 512)
    for counts, want in (([30, 18], [30, 18]), ([8, 40], [38, 18])):
        starts = i32([0, counts[0], sum(counts)])
        seq_rows, pos = cache.extend_chunk(i32([0, 1]), starts, 48)
        layer.forward(x, y, seq_rows, pos, chunk=(starts, i32([0, 1])))
        assert cache.lens.tolist() == want
    assert (seen[0] != 0).any(2).any(1).all() and (seen[1][:8] != 0).any(2).any(1).all() and (seen[1][8:] == 0).all()


def test_positions_of_another_kind_are_refused():
    q = torch.zeros((5, 8, 64), dtype=torch.bfloat16, device=DEV)
    k = torch.zeros((3, 16, 2, 64), dtype=torch.bfloat16, device=DEV)
    ws = M.paged_chunk_workspace(8, 2, 64)
    for error, positions in ((TypeError, torch.zeros(5, dtype=torch.int64, device=DEV)), (ValueError, i32([0] * 4)),
                             (ValueError, torch.zeros(5, dtype=torch.int32))):
        with pytest.raises(error):
            M.paged_chunk_attention(q, i32([0, 2, 5]), k, k.clone(), i32([[0], [1]]), i32([2, 3]), ws, positions=positions)


@pytest.mark.parametrize("accepted", [0, 2, 4])
def test_drafts_of_which_some_are_rejected(accepted):
    """Drafts go into a fork: if all are accepted it takes the sequence's place, else it is freed and the accepted ones' rows
    go into the sequence. No page is lost, and the attention of the next token is that of the accepted tokens alone."""
    g = torch.Generator(device="cuda").manual_seed(14)
    cache = PagedCache(1, 12, PAGE, 2, 8, HEADS, KV_HEADS, DIM)
    rotary = M.Rotary(DIM)

    def put(seq, q, k, v):
        starts = i32([0, q.shape[0]])
        seq_rows, pos = cache.extend_chunk(i32([seq]), starts, q.shape[0])
        return starts, cache.append_rotary(0, q, k, v, seq_rows, pos, rotary), pos

    def tokens(n):
        return rows(g, n, HEADS, DIM), rows(g, n, KV_HEADS, DIM), rows(g, n, KV_HEADS, DIM)

    prompt, drafts, last = tokens(46), tokens(4), tokens(1)           # the drafts end in a page of their own
    put(0, *prompt)
    cache.fork(i32([0]), i32([1]))
    starts, q, pos = put(1, *drafts)
    out = cache.attend_chunk(0, q, starts, i32([1]), 0.125, 0, pos)
    kp, vp = cache.pages(0)
    ref = C.attention(q, [0, 4], kp, vp, cache.tables.tolist(), cache.lens.tolist(), 0.125, seq_ids=[1])
    compare(out, ref[0], ref[1])
    seq = 1 if accepted == 4 else 0
    cache.free(i32([1 - seq]))
    if seq == 0 and accepted:
        put(0, *(x[:accepted] for x in drafts))
    starts, q, pos = put(seq, *last)
    assert cache.lens[seq] == 47 + accepted and int((cache.refs > 0).sum()) == -(-(47 + accepted) // PAGE)
    got = cache.attend_chunk(0, q, starts, i32([seq]), 0.125, 0, pos)
    # the same tokens in a cache that never held the rejected ones
    plain = PagedCache(1, 12, PAGE, 2, 8, HEADS, KV_HEADS, DIM)
    cache, kept = plain, cache
    for x in (prompt, [d[:accepted] for d in drafts], last):
        if x[0].shape[0]:
            starts, q, pos = put(0, *x)
    assert torch.equal(got, plain.attend_chunk(0, q, starts, i32([0]), 0.125, 0, pos))
    kept.free(i32([seq]))
    assert int((kept.refs != 0).sum()) == 0
    kept.check()
    plain.check()
