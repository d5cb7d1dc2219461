"""Cases that measure the attention of a chunk of new tokens over a paged cache and the rotation of positions.

A case is one call as a serving loop makes it:

  chunk    several new tokens of each sequence (a prompt's chunk, drafts to verify, both in one batch) over a paged
           K/V cache, causal, grouped heads (BF16 or e4m3 pages)
  rotary   queries (or keys) rotated by their positions: pairs half a rotation apart or side by side, part of a head,
           frequencies scaled for long contexts
  append   a step's queries rotated, its keys rotated into their pages, its values copied there (e4m3 pages: quantised;
           a latent cache: one row a token, its last channels rotated)
"""

import math
import random

import torch

own = False

LATENT = 576      # channels of a latent row, the last 64 of them rotated


def listed():
    return [
        # one user's five drafted tokens verified against a short chat: nothing but latency
        {"name": "chunk_verify_one", "kind": "chunk", "batch": 1, "new": 5, "past": 1507, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "e4m3": False, "window": 0, "single": 0, "lens_seed": 1},
        # four drafted tokens of each sequence of a serving batch: every key and value is read for few queries
        {"name": "chunk_verify_batch", "kind": "chunk", "batch": 64, "new": 4, "past": 8187, "heads": 64, "kv_heads": 8,
         "dim": 128, "page": 64, "e4m3": False, "window": 0, "single": 0, "lens_seed": 2},
        # whole prompts, nothing in the cache before them: products bound it
        {"name": "chunk_prefill", "kind": "chunk", "batch": 3, "new": 4096, "past": 0, "heads": 64, "kv_heads": 8,
         "dim": 128, "page": 64, "e4m3": False, "window": 0, "single": 0, "lens_seed": 3},
        # a chunk of a long document over an 8-bit cache: the largest
        {"name": "chunk_long_e4m3", "kind": "chunk", "batch": 1, "new": 1024, "past": 31744, "heads": 64, "kv_heads": 8,
         "dim": 128, "page": 32, "e4m3": True, "window": 0, "single": 0, "lens_seed": 4},
        # a batch that decodes while one prompt's chunk goes in: all sequences but one have a single new token
        {"name": "chunk_mixed", "kind": "chunk", "batch": 24, "new": 500, "past": 2047, "heads": 32, "kv_heads": 8,
         "dim": 128, "page": 16, "e4m3": False, "window": 0, "single": 100, "lens_seed": 5},
        # heads of 256 channels that see a window only, the pages behind it freed
        {"name": "chunk_window_wide", "kind": "chunk", "batch": 4, "new": 1000, "past": 6000, "heads": 16, "kv_heads": 4,
         "dim": 256, "page": 48, "e4m3": False, "window": 1024, "single": 0, "lens_seed": 6},
        # a decode step's queries at far positions of a long context
        {"name": "rotary_decode", "kind": "rotary", "tokens": 48, "heads": 64, "dim": 128, "rot": 128, "offset": 0,
         "interleaved": False, "scaling": "turns", "top": 131072},
        # a prefill's queries of which 64 channels of 192 turn
        {"name": "rotary_prefill_part", "kind": "rotary", "tokens": 8192, "heads": 64, "dim": 192, "rot": 64, "offset": 128,
         "interleaved": True, "scaling": "index", "top": 65536},
        # a decode step into an 8-bit cache
        {"name": "append_decode_e4m3", "kind": "append", "batch": 256, "tokens": 256, "heads": 64, "kv_heads": 8, "dim": 128,
         "page": 16, "e4m3": True, "latent": False, "rot": 128, "offset": 0, "interleaved": False, "scaling": "none",
         "top": 8192},
        # a prefill's rows
        {"name": "append_prefill", "kind": "append", "batch": 3, "tokens": 8191, "heads": 64, "kv_heads": 8, "dim": 128,
         "page": 64, "e4m3": False, "latent": False, "rot": 128, "offset": 0, "interleaved": False, "scaling": "linear",
         "top": 16384},
        # a prefill's rows of a latent cache and its queries in the latent space
        {"name": "append_prefill_latent", "kind": "append", "batch": 2, "tokens": 2048, "heads": 64, "kv_heads": 1,
         "dim": LATENT, "page": 64, "e4m3": False, "latent": True, "rot": 64, "offset": 512, "interleaved": True,
         "scaling": "index", "top": 32768},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["chunk", "chunk", "chunk", "rotary", "append", "append"])
    scaling = rng.choice(["none", "none", "linear", "base", "turns", "index"])
    if kind == "chunk":
        kv = rng.choice([1, 2, 4, 8])
        dim = rng.choice([64, 80, 96, 128, 128, 128, 192, 256])
        heads = kv * rng.choice([1, 2, 4, 5, 8, 8, 12, 16])
        e4m3 = rng.random() < 0.4
        batch = _log(rng, 1, 64)
        new = _log(rng, 1, 4096)
        # no more scores, and no more of a padded cache, than the largest listed case's
        most = min((1 << 31) // (batch * new * heads), (1 << 29) // (batch * kv * dim))
        while most < new:
            new = max(1, new // 2)
            most = min((1 << 31) // (batch * new * heads), (1 << 29) // (batch * kv * dim))
        past = rng.choice([0, _log(rng, 1, 32768), _log(rng, 1, 32768), _log(rng, 1, 32768)])
        return {"kind": kind, "batch": batch, "new": new, "past": max(0, min(past, most - new)), "heads": heads,
                "kv_heads": kv, "dim": dim, "page": rng.choice([16, 32, 48, 64, 128]), "e4m3": e4m3,
                "window": rng.choice([0, 0, 0, _log(rng, 1, 4096)]), "single": rng.choice([0, 0, 50, 100]),
                "lens_seed": rng.randrange(1 << 30)}
    if kind == "rotary":
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        rot = rng.choice([dim, dim, dim // 2, 32])
        return {"kind": kind, "tokens": _log(rng, 1, 8192), "heads": rng.choice([1, 2, 8, 10, 32, 64]), "dim": dim,
                "rot": rot, "offset": rng.choice([0, dim - rot]), "interleaved": rng.random() < 0.5, "scaling": scaling,
                "top": _log(rng, 1024, 1 << 20)}
    latent = rng.random() < 0.3
    batch, kv = _log(rng, 1, 256), 1 if latent else rng.choice([1, 2, 4, 8])
    dim = LATENT if latent else rng.choice([64, 96, 128, 256])
    rot = 64 if latent else rng.choice([dim, dim, dim // 2])
    heads = rng.choice([16, 32, 64]) if latent else kv * rng.choice([1, 4, 5, 8, 12])
    return {"kind": kind, "batch": batch, "tokens": max(batch, _log(rng, 1, (1 << 26) // (heads * dim))),
            "heads": heads, "kv_heads": kv, "dim": dim, "page": rng.choice([16, 32, 48, 64, 128]),
            "e4m3": (not latent) and rng.random() < 0.5, "latent": latent, "rot": rot, "offset": 512 if latent else 0,
            "interleaved": rng.random() < 0.5, "scaling": scaling, "top": _log(rng, 1024, 1 << 20)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(shape, g, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _pool(shape, g, e4m3=False):
    """Cache contents, drawn in BF16 so that a large pool needs no 32-bit copy of itself."""
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    return out.to(torch.float8_e4m3fn) if e4m3 else out


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _lens(case):
    """(new tokens, length with them) of each sequence: the case's own, whatever the seed. The first sequence has the
    most of both; of four or more, one has no new token and one nothing but a single one; `single` percent of the
    others have one new token (they decode)."""
    r = random.Random(case["lens_seed"])
    got = [(case["new"], case["past"] + case["new"])]
    for _ in range(case["batch"] - 1):
        n = 1 if r.random() * 100 < case["single"] else r.randint(max(1, case["new"] // 4), case["new"])
        got.append((n, n + r.randint(case["past"] // 4, case["past"])))
    if case["batch"] >= 4:
        got[1], got[2] = (0, got[1][1]), (1, 1)
    return got


def _tables(lens, seen_from, page, g):
    """Pages of every sequence, scattered over the pool; -1 past the end and wholly before the first seen token."""
    need = [-(-x // page) for x in lens]
    width, total = max(1, max(need)), max(1, sum(need))
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    n = torch.tensor(need, device="cuda")
    col = torch.arange(width, device="cuda")[None, :]
    at = (torch.cumsum(n, 0) - n)[:, None] + col
    keep = (col < n[:, None]) & (col >= torch.tensor(seen_from, device="cuda")[:, None] // page)
    return torch.where(keep, order[at.clamp(max=total - 1)], torch.full_like(at, -1, dtype=torch.int32)).contiguous(), total


#: theta, and what a scaling takes besides: (factor, trained length, low, high, magnitude)
THETA = 500000.0
SCALINGS = {"none": (1.0, 0, 0.0, 0.0, 1.0), "linear": (4.0, 0, 0.0, 0.0, 1.0), "base": (8.0, 0, 0.0, 0.0, 1.0),
            "turns": (8.0, 8192, 1.0, 4.0, 1.0), "index": (32.0, 4096, 1.0, 32.0, 1.25)}


def _frequencies(case):
    """Radians a token of each pair, from the definitions, in 64 bits."""
    rot, kind = case["rot"], case["scaling"]
    factor, trained, low, high, _ = SCALINGS[kind]
    i = torch.arange(rot // 2, dtype=torch.float64)
    if kind == "base":                  # a larger base, so that the slowest pair turns `factor` times slower
        return (THETA * factor ** (rot / (rot - 2))) ** (-2 * i / rot)
    f = THETA ** (-2 * i / rot)
    if kind == "linear":
        return f / factor
    if kind == "turns":                 # by the turns of a pair within the trained length
        keep = ((trained * f / (2 * math.pi) - low) / (high - low)).clamp(0, 1)
        return f * keep + f / factor * (1 - keep)
    if kind == "index":                 # by the pair's index, between those that turn `high` and `low` times
        def at(turns):
            return rot * math.log(trained / (turns * 2 * math.pi)) / (2 * math.log(THETA))
        first, last = max(0, math.floor(at(high))), min(rot - 1, math.ceil(at(low)))
        slow = ((i - first) / max(0.001, last - first)).clamp(0, 1)
        return f * (1 - slow) + f / factor * slow
    return f


def _module():
    import w4a16_int4_mixture_grouped_gb300 as M
    return M


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["kind"] == "chunk":
        pairs = _lens(c)
        lens = [x for _, x in pairs]
        first = [max(0, x - n - c["window"] + 1) if c["window"] else 0 for n, x in pairs]
        s["tables"], total = _tables(lens, first, c["page"], g)
        s["lens"] = _i32(lens)
        starts = [0]
        for n, _ in pairs:
            starts.append(starts[-1] + n)
        s["starts"] = _i32(starts)
        shape = (total, c["page"], c["kv_heads"], c["dim"])
        s["k"], s["v"] = _pool(shape, g, c["e4m3"]), _pool(shape, g, c["e4m3"])
        # scores with a standard deviation of 1.5: some tokens clearly ahead of the others
        s["q"] = _normal((starts[-1], c["heads"], c["dim"]), g) * 1.5
        s["scale"] = c["dim"] ** -0.5
        s["ks"], s["vs"] = (0.75, 1.25) if c["e4m3"] else (1.0, 1.0)
        if own:
            M = _module()
            s["ws"] = M.paged_chunk_workspace(c["heads"], c["kv_heads"], c["dim"])
        return s
    s["freqs"] = _frequencies(c).to("cuda")
    t = c["tokens"]
    if c["kind"] == "rotary":
        s["pos"] = torch.randint(0, c["top"], (t,), generator=g, device="cuda", dtype=torch.int32)
        s["x"] = _normal((t, c["heads"], c["dim"]), g)
    else:
        per = -(-t // c["batch"])
        # sequences that end anywhere up to `top`: their tables hold the pages of the last tokens alone
        end = torch.randint(per, max(per, c["top"]) + 1, (c["batch"],), generator=g, device="cuda")
        seq = torch.arange(t, device="cuda") // per
        s["seq"] = seq.to(torch.int32)
        s["pos"] = ((end - per)[seq] + torch.arange(t, device="cuda") % per).to(torch.int32)
        width, cols = -(-(max(per, c["top"]) + 1) // c["page"]), -(-per // c["page"]) + 1
        total = c["batch"] * cols
        order = torch.randperm(total, generator=g, device="cuda").to(torch.int32).reshape(c["batch"], cols)
        col = torch.arange(width, device="cuda")[None, :] - ((end - per) // c["page"])[:, None]
        s["tables"] = torch.where((col >= 0) & (col < cols), order.gather(1, col.clamp(0, cols - 1)),
                                  torch.full_like(col, -1, dtype=torch.int32)).contiguous()
        shape = (total, c["page"], LATENT) if c["latent"] else (total, c["page"], c["kv_heads"], c["dim"])
        # queries, keys and values are slices of one product, as a layer's projection gives them
        kv = 1 if c["latent"] else 2 * c["kv_heads"]
        x = _normal((t, c["heads"] + kv, c["dim"]), g)
        s["q"] = x[:, :c["heads"]]
        s["k"] = x[:, c["heads"]] if c["latent"] else x[:, c["heads"]:c["heads"] + c["kv_heads"]]
        s["v"] = None if c["latent"] else x[:, c["heads"] + c["kv_heads"]:]
        s["k_pages"] = _pool(shape, g, c["e4m3"])
        s["v_pages"] = None if c["latent"] else _pool(shape, g, c["e4m3"])
        s["ks"], s["vs"] = (0.015, 0.02) if c["e4m3"] else (1.0, 1.0)
    if own:
        M = _module()
        factor, trained, low, high, magnitude = SCALINGS[c["scaling"]]
        s["rotary"] = M.Rotary(c["rot"], theta=THETA, offset=c["offset"], interleaved=c["interleaved"],
                               scaling=c["scaling"], factor=factor, trained_length=trained, low=low, high=high,
                               magnitude=magnitude)
        if c["kind"] == "append":
            s["ws"] = M.cache_workspace(0, 1)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    kind = s["case"]["kind"]
    if own:
        return _run_own(s, kind)
    return {"chunk": _chunk, "rotary": _rotary, "append": _append}[kind](s)


def _run_own(s, kind):
    M, c = _module(), s["case"]
    if kind == "chunk":
        out, lse = M.paged_chunk_attention(s["q"], s["starts"], s["k"], s["v"], s["tables"], s["lens"], s["ws"],
                                           scale=s["scale"], window=c["window"], k_scale=s["ks"], v_scale=s["vs"])
        return {"out": out, "lse": lse}
    if kind == "rotary":
        return M.rotary(s["x"], s["pos"], s["rotary"])
    q = M.cache_append_rotary(s["q"], s["k"], s["k_pages"], s["tables"], s["seq"], s["pos"], s["rotary"], s["ws"],
                              v=s["v"], v_pages=s["v_pages"], k_scale=s["ks"], v_scale=s["vs"])
    return {"q": q, "k": s["k_pages"]} if c["latent"] else {"q": q, "k": s["k_pages"], "v": s["v_pages"]}


def _rows(pages, tables):
    """The pages of every table row as 32-bit rows in token order."""
    raw = pages.view(torch.uint8) if pages.dtype == torch.float8_e4m3fn else pages
    got = raw[tables.clamp(min=0).long()]
    if pages.dtype == torch.float8_e4m3fn:
        got = got.view(torch.float8_e4m3fn)
    return got.to(torch.float32).flatten(1, 2)


def _chunk(s):
    c = s["case"]
    b, kv, d, most = c["batch"], c["kv_heads"], c["dim"], c["new"]
    k, v = _rows(s["k"], s["tables"]), _rows(s["v"], s["tables"])              # [B, L, Hkv, D]
    length = k.shape[1]
    first, n = s["starts"][:-1, None].long(), (s["starts"][1:] - s["starts"][:-1])[:, None].long()
    i = torch.arange(most, device="cuda")[None, :]
    row = torch.where(i < n, first + i, torch.zeros_like(first))               # [B, new]: padded to the longest chunk
    q = s["q"].float()[row].reshape(b, most, kv, -1, d).permute(0, 2, 3, 1, 4).flatten(2, 3)    # [B, Hkv, G new, D]
    at, pos = torch.arange(length, device="cuda"), (s["lens"][:, None] - n + i)[:, :, None]
    seen = (at <= pos) & (torch.repeat_interleave(s["tables"], c["page"], 1) >= 0)[:, None, :]
    if c["window"]:
        seen &= at > pos - c["window"]
    seen = seen[:, None, None]                                                 # [B, 1, 1, new, L]
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)).unflatten(2, (-1, most))
    scores.mul_(s["scale"] * s["ks"]).masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p.flatten(2, 3), v.permute(0, 2, 1, 3)).unflatten(2, (-1, most))
    out = torch.where(total > 0, out / total, torch.zeros_like(out)) * s["vs"]
    lse = (top + torch.log(total)).squeeze(-1)
    # back to the rows: token t is the (t - first)-th of its sequence
    t = s["q"].shape[0]
    seq = torch.repeat_interleave(torch.arange(b, device="cuda"), n[:, 0], output_size=t)
    place = torch.arange(t, device="cuda") - first[seq, 0]
    out = out.permute(0, 3, 1, 2, 4)[seq, place].reshape(t, -1, d)
    return {"out": out.to(torch.bfloat16), "lse": lse.permute(0, 3, 1, 2)[seq, place].reshape(t, -1)}


def _turn(x, pos, freqs, c):
    """x [T, H, D] in 32 bits with its channels offset .. offset + rot turned; the angles in 64 bits."""
    angle = pos.to(torch.float64)[:, None] * freqs
    size = SCALINGS[c["scaling"]][4]
    cos, sin = (torch.cos(angle) * size).float()[:, None], (torch.sin(angle) * size).float()[:, None]
    lo, rot, half = c["offset"], c["rot"], c["rot"] // 2
    x = x.float()
    part = x[..., lo:lo + rot]
    a, b = (part[..., 0::2], part[..., 1::2]) if c["interleaved"] else (part[..., :half], part[..., half:])
    a, b = a * cos - b * sin, a * sin + b * cos
    part = torch.stack((a, b), -1).flatten(-2) if c["interleaved"] else torch.cat((a, b), -1)
    return torch.cat((x[..., :lo], part, x[..., lo + rot:]), -1)


def _rotary(s):
    return _turn(s["x"], s["pos"], s["freqs"], s["case"]).to(torch.bfloat16)


def _put(pages, rows, page, slot, scale):
    if pages.dtype == torch.float8_e4m3fn:
        rows = (rows.float() / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        pages.view(torch.uint8)[page, slot] = rows
    else:
        pages[page, slot] = rows.to(torch.bfloat16)


def _append(s):
    c = s["case"]
    pos = s["pos"].long()
    page, slot = s["tables"][s["seq"].long(), pos // c["page"]].long(), pos % c["page"]
    q = _turn(s["q"], s["pos"], s["freqs"], c).to(torch.bfloat16)
    k = _turn(s["k"][:, None] if c["latent"] else s["k"], s["pos"], s["freqs"], c)
    _put(s["k_pages"], k[:, 0] if c["latent"] else k, page, slot, s["ks"])
    if c["latent"]:
        return {"q": q, "k": s["k_pages"]}
    _put(s["v_pages"], s["v"], page, slot, s["vs"])
    return {"q": q, "k": s["k_pages"], "v": s["v_pages"]}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    if c["kind"] == "chunk":
        w = c["window"] or (1 << 40)
        read = scores = rows = 0
        for n, length in _lens(c):
            if n == 0:
                continue
            past = length - n
            read += length - max(0, past - w + 1)
            # the query at position p sees min(p + 1, window) tokens
            grow = max(0, min(n, w - past))
            scores += grow * past + grow * (grow + 1) // 2 + (n - grow) * min(w, length)
            rows += n
        row = 2 * c["kv_heads"] * c["dim"] * (1 if c["e4m3"] else 2)
        return {"bytes": read * row + rows * c["heads"] * (4 * c["dim"] + 4) + 4 * (read // c["page"] + 2 * c["batch"]),
                "flops": 4 * scores * c["heads"] * c["dim"]}
    t = c["tokens"]
    if c["kind"] == "rotary":
        return {"bytes": 4 * t * c["heads"] * c["dim"] + 4 * t + 4 * c["rot"], "flops": 3 * t * c["heads"] * c["rot"]}
    kv = c["kv_heads"] * c["dim"] * (1 if c["latent"] else 2)
    return {"bytes": t * (4 * c["heads"] * c["dim"] + kv * (2 + (1 if c["e4m3"] else 2)) + 12) + 4 * c["rot"],
            "flops": 3 * t * (c["heads"] + c["kv_heads"]) * c["rot"]}


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _rotated(x, pos, c):
    """x [T, H, D] as complex numbers times exp(i angle), the frequencies spelled out pair by pair."""
    factor, trained, low, high, size = SCALINGS[c["scaling"]]
    rot, lo = c["rot"], c["offset"]
    f = []
    for j in range(rot // 2):
        base = THETA * factor ** (rot / (rot - 2.0)) if c["scaling"] == "base" else THETA
        w = math.exp(-2.0 * j / rot * math.log(base))
        if c["scaling"] == "linear":
            w /= factor
        elif c["scaling"] == "turns":
            turns = trained * w / (2.0 * math.pi)
            share = 0.0 if turns <= low else 1.0 if turns >= high else (turns - low) / (high - low)
            w = share * w + (1.0 - share) * w / factor
        elif c["scaling"] == "index":
            edge = [rot / 2.0 * math.log(trained / (2.0 * math.pi * t), THETA) for t in (high, low)]
            start, stop = max(math.floor(edge[0]), 0), min(math.ceil(edge[1]), rot - 1)
            share = min(1.0, max(0.0, (j - start) / max(stop - start, 1e-3)))
            w = (1.0 - share) * w + share * w / factor
        f.append(w)
    turn = torch.outer(pos.to(torch.float64), torch.tensor(f, dtype=torch.float64, device=pos.device))
    turn = torch.polar(torch.full_like(turn, size), turn)[:, None, :]
    out = x.to(torch.float64).clone()
    part = out[:, :, lo:lo + rot]
    if c["interleaved"]:
        z = torch.complex(part[:, :, ::2], part[:, :, 1::2]) * turn
        part[:, :, ::2], part[:, :, 1::2] = z.real, z.imag
    else:
        z = torch.complex(part[:, :, :rot // 2], part[:, :, rot // 2:]) * turn
        part[:, :, :rot // 2], part[:, :, rot // 2:] = z.real, z.imag
    return out


def exact(case, seed):
    c = case
    global own
    was, own = own, False             # the inputs alone
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if c["kind"] == "rotary":
        return _rotated(s["x"], s["pos"], c)
    if c["kind"] == "append":
        seq, pos, table = s["seq"].tolist(), s["pos"].tolist(), s["tables"].tolist()
        at = torch.tensor([table[a][p // c["page"]] * c["page"] + p % c["page"] for a, p in zip(seq, pos)], device="cuda")
        rows = {"k": _rotated(s["k"][:, None] if c["latent"] else s["k"], s["pos"], c)}
        if not c["latent"]:
            rows["v"] = s["v"].to(torch.float64)
        got = {"q": _rotated(s["q"], s["pos"], c)}
        for name, new in rows.items():
            full = s[name + "_pages"].to(torch.float64)
            new = new / s["ks" if name == "k" else "vs"]
            if c["e4m3"]:
                new = new.clamp(-448, 448)
            full.view(-1, *full.shape[2:])[at] = new.reshape(len(at), *full.shape[2:])
            got[name] = full
        return got
    group, dim = c["heads"] // c["kv_heads"], c["dim"]
    table, starts = s["tables"].tolist(), s["starts"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, length in enumerate(s["lens"].tolist()):
        t0, t1 = starts[b], starts[b + 1]
        if t0 == t1:
            continue
        past = length - (t1 - t0)
        low = max(0, past - c["window"] + 1) if c["window"] else 0
        lead = low // c["page"]
        ids = torch.tensor(table[b][lead:-(-length // c["page"])], device="cuda")
        key_at = torch.arange(low, length, device="cuda")
        query_at = torch.arange(past, length, device="cuda")[:, None]
        hidden = key_at > query_at
        if c["window"]:
            hidden |= query_at - key_at >= c["window"]
        for j in range(c["kv_heads"]):
            k, v = (t.view(torch.uint8 if c["e4m3"] else torch.bfloat16)[ids, :, j].view(t.dtype).reshape(-1, dim)
                    [low - lead * c["page"]:length - lead * c["page"]].to(torch.float64) for t in (s["k"], s["v"]))
            for h in range(j * group, (j + 1) * group):
                z = s["q"][t0:t1, h].to(torch.float64) @ k.T * (s["scale"] * s["ks"])
                z[hidden] = -math.inf
                m = z.max(1, keepdim=True)[0]
                w = torch.exp(z - m)
                out[t0:t1, h] = w @ v / w.sum(1, keepdim=True) * s["vs"]
                lse[t0:t1, h] = m[:, 0] + torch.log(w.sum(1))
    return {"out": out, "lse": lse}
