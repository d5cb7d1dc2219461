"""Cases that measure the paged cache, the attention over it and the norms around a block.

A case is one call (or one short sequence of calls) as a serving loop makes it:

  attn     one new token per sequence over a paged K/V cache, grouped heads (BF16 or e4m3 pages)
  latent   the same over a shared latent cache (512 value + 64 position channels, all heads on one row)
  append   new tokens' rows written into their pages (e4m3 pages: quantised)
  fork     sequences forked, each fork grown by one token, the forks freed again (a beam or draft step)
  compact  the live pages moved to the front of the pool, tables and counts remapped
  norm     h' = rs * h + bs * gate * norm(x) * w_post, y = norm(h') * w_pre
"""

import math
import random

import torch

own = False

LATENT, VALUE = 576, 512      # channels of a latent row; the first VALUE of them are the values


def listed():
    return [
        # one user, a short chat turn: nothing but latency
        {"name": "attn_one", "kind": "attn", "batch": 1, "max_len": 517, "heads": 32, "kv_heads": 8, "dim": 128,
         "page": 16, "e4m3": False, "window": 0, "lens_seed": 1},
        # a serving batch with lengths from nothing to 8k, 8 query heads to a K/V head
        {"name": "attn_ragged", "kind": "attn", "batch": 96, "max_len": 8191, "heads": 64, "kv_heads": 8, "dim": 128,
         "page": 64, "e4m3": False, "window": 0, "lens_seed": 2},
        # a few long documents in an 8-bit cache: the largest
        {"name": "attn_long_e4m3", "kind": "attn", "batch": 8, "max_len": 131072, "heads": 64, "kv_heads": 8, "dim": 128,
         "page": 32, "e4m3": True, "window": 0, "lens_seed": 3},
        # one sequence of a few thousand tokens over the latent cache
        {"name": "latent_one", "kind": "latent", "batch": 1, "max_len": 4099, "heads": 64, "page": 64, "window": 0,
         "lens_seed": 4},
        # a serving batch over the latent cache
        {"name": "latent_ragged", "kind": "latent", "batch": 128, "max_len": 8192, "heads": 64, "page": 64,
         "window": 0, "lens_seed": 5},
        # a decode step's new rows into an 8-bit cache
        {"name": "append_decode_e4m3", "kind": "append", "batch": 256, "tokens": 256, "kv_heads": 8, "dim": 128,
         "page": 16, "e4m3": True, "latent": False},
        # a prefill's rows into the latent cache
        {"name": "append_prefill_latent", "kind": "append", "batch": 3, "tokens": 8192, "kv_heads": 1, "dim": LATENT,
         "page": 64, "e4m3": False, "latent": True},
        # four drafts of a batch's sequences over few cache planes
        {"name": "fork_drafts", "kind": "fork", "parents": 8, "forks": 4, "max_len": 2000, "pages": 4096, "planes": 2,
         "page": 16, "width": 1024},
        # a large batch forked once, every layer's planes in one pool
        {"name": "fork_batch", "kind": "fork", "parents": 192, "forks": 1, "max_len": 4000, "pages": 16384, "planes": 16,
         "page": 16, "width": 1024},
        # half the pool's pages freed here and there: the live ones to the front
        {"name": "compact_half", "kind": "compact", "pages": 2048, "planes": 16, "page": 64, "width": 1024, "live": 50,
         "seqs": 64},
        # one token's residual stream between two blocks, at the width of the FFN here
        {"name": "norm_one", "kind": "norm", "rows": 1, "n": 7168, "res32": False, "gate": 0, "post": True,
         "pre": True},
        # a prefill's rows, residual in 32 bits, one gate row per channel
        {"name": "norm_prefill", "kind": "norm", "rows": 8192, "n": 7168, "res32": True, "gate": 1, "post": True,
         "pre": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["attn", "attn", "latent", "append", "fork", "compact", "norm", "norm"])
    if kind == "attn":
        kv = rng.choice([1, 2, 4, 8])
        dim = rng.choice([64, 96, 128, 128, 256])
        e4m3 = rng.random() < 0.4
        batch = _log(rng, 1, 256)
        # no more padded cache than the largest listed case's
        most = (8 * 131072 * 8 * 128) // (batch * kv * dim) // (1 if e4m3 else 2)
        max_len = _log(rng, 1, max(1, min(131072, most)))
        return {"kind": kind, "batch": batch, "max_len": max_len, "heads": kv * rng.choice([1, 2, 4, 5, 8, 12, 16]),
                "kv_heads": kv, "dim": dim, "page": rng.choice([16, 32, 48, 64, 128]), "e4m3": e4m3,
                "window": rng.choice([0, 0, 0, _log(rng, 1, 4096)]), "lens_seed": rng.randrange(1 << 30)}
    if kind == "latent":
        batch = _log(rng, 1, 256)
        return {"kind": kind, "batch": batch, "max_len": _log(rng, 1, min(65536, (128 * 8192) // batch)),
                "heads": rng.choice([8, 16, 24, 32, 64]), "page": rng.choice([16, 32, 64, 128]),
                "window": rng.choice([0, 0, 0, _log(rng, 1, 4096)]), "lens_seed": rng.randrange(1 << 30)}
    if kind == "append":
        latent = rng.random() < 0.4
        batch = _log(rng, 1, 256)
        return {"kind": kind, "batch": batch, "tokens": max(batch, _log(rng, 1, 16384)),
                "kv_heads": 1 if latent else rng.choice([1, 2, 4, 8]), "dim": LATENT if latent else rng.choice([64, 96, 128, 256]),
                "page": rng.choice([16, 32, 48, 64, 128]), "e4m3": (not latent) and rng.random() < 0.5, "latent": latent}
    if kind == "fork":
        parents, planes = _log(rng, 1, 192), rng.choice([1, 2, 4, 8, 16])
        return {"kind": kind, "parents": parents, "forks": rng.choice([1, 2, 3, 4]), "max_len": _log(rng, 1, 4000),
                "pages": 16384, "planes": planes, "page": rng.choice([16, 24, 32]), "width": rng.choice([256, 512, 1024])}
    if kind == "compact":
        return {"kind": kind, "pages": _log(rng, 16, 2048), "planes": rng.choice([1, 2, 6, 16]),
                "page": rng.choice([16, 32, 64]), "width": rng.choice([576, 512, 1024]), "live": rng.randrange(1, 100),
                "seqs": _log(rng, 1, 64)}
    return {"kind": kind, "rows": _log(rng, 1, 8192), "n": rng.choice([_log(rng, 64, 7168), 8 * _log(rng, 8, 896)]),
            "res32": rng.random() < 0.5, "gate": rng.choice([0, 1, 2, 3]), "post": rng.random() < 0.7,
            "pre": rng.random() < 0.8}


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


def _lens(case):
    """Lengths of a batch: the case's own, whatever the seed. Single sequences have the full length; a batch
    has one full, one empty and one of a single token, the others spread between."""
    r = random.Random(case["lens_seed"])
    n, top = case["batch"], case["max_len"]
    lens = [top] + [r.randint(max(1, top // 4), top) for _ in range(n - 1)]
    if n >= 4:
        lens[1], lens[2] = 0, 1
    return lens


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _tables(lens, page, g, windows=0):
    """Pages of every sequence, scattered over the pool; -1 past the end and before the window."""
    need = [-(-x // page) for x in lens]
    width = max(1, max(need))
    total = max(1, sum(need))
    order = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    n = torch.tensor(need, device="cuda")
    col = torch.arange(width, device="cuda")[None, :]
    at = (torch.cumsum(n, 0) - n)[:, None] + col
    keep = col < n[:, None]
    if windows:
        first = (torch.tensor(lens, device="cuda") - windows).clamp(min=0) // page
        keep = keep & (col >= first[:, None])
    return torch.where(keep, order[at.clamp(max=total - 1)], torch.full_like(at, -1, dtype=torch.int32)).contiguous(), total


def _module():
    import w4a16_int4_mixture_grouped_gb300 as M
    return M


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["kind"] in ("attn", "latent"):
        lens = _lens(c)
        s["tables"], total = _tables(lens, c["page"], g, c["window"])
        s["lens"] = _i32(lens)
        if c["kind"] == "attn":
            shape = (total, c["page"], c["kv_heads"], c["dim"])
            s["k"], s["v"] = _pool(shape, g, c["e4m3"]), _pool(shape, g, c["e4m3"])
            # scores with a standard deviation of 1.5: some tokens clearly ahead of the others
            s["q"] = _normal((c["batch"], c["heads"], c["dim"]), g) * 1.5
            s["scale"] = c["dim"] ** -0.5
            s["ks"], s["vs"] = (0.75, 1.25) if c["e4m3"] else (1.0, 1.0)
        else:
            s["pages"] = _pool((total, c["page"], LATENT), g)
            s["q"] = _normal((c["batch"], c["heads"], LATENT), g)
            s["scale"] = 192 ** -0.5 * 0.6
    elif c["kind"] == "append":
        per = -(-c["tokens"] // c["batch"])
        start = torch.randint(0, 4 * c["page"], (c["batch"],), generator=g, device="cuda")
        seq = torch.arange(c["tokens"], device="cuda") // per
        s["seq"] = seq.to(torch.int32)
        s["pos"] = (start[seq] + torch.arange(c["tokens"], device="cuda") % per).to(torch.int32)
        width = -(-(per + 4 * c["page"]) // c["page"])
        total = c["batch"] * width
        s["tables"] = torch.randperm(total, generator=g, device="cuda").to(torch.int32).reshape(c["batch"], width)
        shape = (total, c["page"], LATENT) if c["latent"] else (total, c["page"], c["kv_heads"], c["dim"])
        rows = (c["tokens"],) + shape[2:]
        s["k_pages"], s["k"] = _pool(shape, g, c["e4m3"]), _normal(rows, g)
        s["v_pages"], s["v"] = (None, None) if c["latent"] else (_pool(shape, g, c["e4m3"]), _normal(rows, g))
        s["ks"], s["vs"] = (0.015, 0.02) if c["e4m3"] else (1.0, 1.0)
    elif c["kind"] == "fork":
        n = c["parents"]
        r = random.Random(c["parents"] * 131 + c["max_len"])
        lens = [r.randint(max(1, c["max_len"] // 2), c["max_len"]) for _ in range(n)]
        need = [-(-x // c["page"]) for x in lens]
        while sum(need) + 2 * n * c["forks"] > c["pages"]:     # the pool holds the parents and their forks
            lens = [max(1, x // 2) for x in lens]
            need = [-(-x // c["page"]) for x in lens]
        tables, total = _tables(lens, c["page"], g)
        spread = torch.randperm(c["pages"], generator=g, device="cuda").to(torch.int32)[:total]
        tables = torch.where(tables >= 0, spread[tables.clamp(min=0).long()], tables)
        width = tables.shape[1] + 1
        s["tables"] = torch.full((n * (1 + c["forks"]), width), -1, dtype=torch.int32, device="cuda")
        s["tables"][:n, :-1] = tables
        s["refs"] = torch.zeros(c["pages"], dtype=torch.int32, device="cuda")
        s["refs"][spread.long()] = 1
        s["lens"] = _i32(lens + [0] * (n * c["forks"]))
        s["parents"] = _i32([i for i in range(n) for _ in range(c["forks"])])
        s["children"] = _i32(list(range(n, n * (1 + c["forks"]))))
        s["pool"] = _pool((c["planes"], c["pages"], c["page"], c["width"]), g)
    elif c["kind"] == "compact":
        live = max(1, c["pages"] * c["live"] // 100)
        ids = torch.randperm(c["pages"], generator=g, device="cuda").to(torch.int32)[:live]
        s["refs"] = torch.zeros(c["pages"], dtype=torch.int32, device="cuda")
        s["refs"][ids.long()] = 1 + (torch.arange(live, device="cuda") % 3 == 0).to(torch.int32)
        width = -(-live // c["seqs"])
        s["tables"] = torch.full((c["seqs"], width), -1, dtype=torch.int32, device="cuda")
        s["tables"].view(-1)[:live] = ids
        s["moves"] = int((ids >= live).sum())      # the host's own count of pages to move
        s["pool"] = _pool((c["planes"], c["pages"], c["page"], c["width"]), g)
    else:
        t, n = c["rows"], c["n"]
        s["x"] = _normal((t, n), g)
        s["h"] = _normal((t, n), g, torch.float32 if c["res32"] else torch.bfloat16) * 3
        s["w_post"] = _normal((n,), g) * 0.1 + 1 if c["post"] else None
        s["w_pre"] = _normal((n,), g) * 0.1 + 1 if c["pre"] else None
        s["gate"] = (None, _normal((n,), g), _normal((t, n), g),
                     _normal((math.gcd(t, 64), n), g))[c["gate"]]
    if own:
        M = _module()
        if c["kind"] == "attn":
            s["ws"] = M.attention_workspace(c["batch"], c["heads"], c["kv_heads"], c["dim"])
        elif c["kind"] == "latent":
            s["ws"] = M.attention_workspace(c["batch"], c["heads"], 1, LATENT)
        elif c["kind"] != "norm":
            s["ws"] = M.cache_workspace(c.get("pages", 0), s["parents"].numel() if c["kind"] == "fork" else c.get("tokens", 1))
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    kind = s["case"]["kind"]
    if own:
        return _run_own(s, kind)
    return {"attn": _attn, "latent": _latent, "append": _append, "fork": _fork, "compact": _compact, "norm": _norm}[kind](s)


def _run_own(s, kind):
    M, c = _module(), s["case"]
    if kind == "attn":
        out, lse = M.paged_attention(s["q"], s["k"], s["v"], s["tables"], s["lens"], s["ws"], scale=s["scale"],
                                     window=c["window"], k_scale=s["ks"], v_scale=s["vs"])
        return {"out": out, "lse": lse}
    if kind == "latent":
        out, lse = M.latent_attention(s["q"], s["pages"], s["tables"], s["lens"], s["ws"], scale=s["scale"],
                                      window=c["window"])
        return {"out": out, "lse": lse}
    if kind == "append":
        M.cache_append(s["k"], s["k_pages"], s["tables"], s["seq"], s["pos"], s["ws"], v=s["v"], v_pages=s["v_pages"],
                       k_scale=s["ks"], v_scale=s["vs"])
        return {"k": s["k_pages"]} if c["latent"] else {"k": s["k_pages"], "v": s["v_pages"]}
    if kind == "fork":
        M.cache_fork(s["pool"], s["refs"], s["tables"], s["lens"], s["parents"], s["children"], c["page"], s["ws"])
        pos = M.cache_extend(s["refs"], s["tables"], s["lens"], s["children"], c["page"], s["ws"])
        M.cache_free(s["refs"], s["tables"], s["lens"], s["children"], c["page"], s["ws"])
        return {"pos": pos, "pool": s["pool"], "refs": s["refs"], "tables": s["tables"], "lens": s["lens"]}
    if kind == "compact":
        refs, tables, page_map, live = M.cache_compact(s["pool"], s["refs"], s["tables"], s["ws"])
        return {"refs": refs, "tables": tables, "map": page_map, "live": live, "pool": s["pool"]}
    h, y = M.block_norm(s["x"], s["h"], w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate"], eps=1e-6,
                        residual_scale=0.9, block_scale=1.2)
    return {"h": h, "y": y}


def _rows(pages, tables):
    """The pages of every table row as 32-bit rows in token order."""
    raw = pages.view(torch.uint8) if pages.dtype == torch.float8_e4m3fn else pages
    got = raw[tables.clamp(min=0).long()]
    if pages.dtype == torch.float8_e4m3fn:
        got = got.view(torch.float8_e4m3fn)
    return got.to(torch.float32).flatten(1, 2)


def _visible(s, length):
    c, at = s["case"], torch.arange(length, device="cuda")
    lens = s["lens"][:, None]
    seen = (at < lens) & (torch.repeat_interleave(s["tables"], c["page"], 1)[:, :length] >= 0)
    return seen & (at >= lens - c["window"]) if c["window"] else seen


def _softmax(scores, seen):
    """Probabilities (zero rows where nothing is seen) and the log of the sums."""
    scores = scores.masked_fill(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = e.sum(-1, keepdim=True)
    p = torch.where(total > 0, e / total, torch.zeros_like(e))
    return p, (top + torch.log(total)).squeeze(-1)


def _attn(s):
    c = s["case"]
    b, kv, d = c["batch"], c["kv_heads"], c["dim"]
    k, v = _rows(s["k"], s["tables"]), _rows(s["v"], s["tables"])              # [B, L, Hkv, D]
    seen = _visible(s, k.shape[1])
    q = s["q"].float().reshape(b, kv, -1, d)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)) * (s["scale"] * s["ks"])   # [B, Hkv, G, L]
    p, lse = _softmax(scores, seen[:, None, None, :])
    v = v.masked_fill(~seen[:, :, None, None], 0.0)
    out = torch.matmul(p, v.permute(0, 2, 1, 3)) * s["vs"]
    return {"out": out.reshape(b, -1, d).to(torch.bfloat16), "lse": lse.reshape(b, -1)}


def _latent(s):
    rows = _rows(s["pages"], s["tables"])                                      # [B, L, 576]
    seen = _visible(s, rows.shape[1])
    scores = torch.matmul(s["q"].float(), rows.transpose(1, 2)) * s["scale"]
    p, lse = _softmax(scores, seen[:, None, :])
    out = torch.matmul(p, rows[..., :VALUE].masked_fill(~seen[:, :, None], 0.0))
    return {"out": out.to(torch.bfloat16), "lse": lse}


def _put(pages, rows, page, slot, scale):
    if pages.dtype == torch.float8_e4m3fn:
        rows = (rows.float() / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        pages.view(torch.uint8)[page, slot] = rows
    else:
        pages[page, slot] = rows


def _append(s):
    c = s["case"]
    pos = s["pos"].long()
    page, slot = s["tables"][s["seq"].long(), pos // c["page"]].long(), pos % c["page"]
    _put(s["k_pages"], s["k"], page, slot, s["ks"])
    if c["latent"]:
        return {"k": s["k_pages"]}
    _put(s["v_pages"], s["v"], page, slot, s["vs"])
    return {"k": s["k_pages"], "v": s["v_pages"]}


def _free_ids(refs):
    """Page ids, the free ones first, each part ascending."""
    return torch.sort((refs > 0).to(torch.int32), stable=True)[1]


def _fork(s):
    page, refs, tables, lens, pool = s["case"]["page"], s["refs"], s["tables"], s["lens"], s["pool"]
    parents, children = s["parents"].long(), s["children"].long()
    # fork: the parent's pages shared, a partly filled last page copied
    n = lens[parents].long()
    need = n % page != 0
    col = n // page
    rows = tables[parents]
    src = rows.gather(1, col[:, None])[:, 0].long()
    fresh = _free_ids(refs)[(torch.cumsum(need, 0) - 1).clamp(min=0)]
    rows.scatter_(1, col[:, None], torch.where(need, fresh, src).to(torch.int32)[:, None])
    first = tables[parents, 0].long()              # where nothing is copied: a held page onto itself
    pool[:, torch.where(need, fresh, first)] = pool[:, torch.where(need, src, first)]
    tables[children] = rows
    lens[children] = n.to(torch.int32)
    refs.index_add_(0, rows.clamp(min=0).flatten().long(), (rows >= 0).flatten().to(torch.int32))
    # extend: one token each, a fresh page where the last one is full
    pos = lens[children]
    need = pos % page == 0
    col = (pos // page).long()
    fresh = _free_ids(refs)[(torch.cumsum(need, 0) - 1).clamp(min=0)]
    old = tables[children, col]
    tables[children, col] = torch.where(need, fresh.to(torch.int32), old)
    refs.index_add_(0, fresh, need.to(torch.int32))
    lens[children] = pos + 1
    # free
    rows = tables[children]
    refs.index_add_(0, rows.clamp(min=0).flatten().long(), -(rows >= 0).flatten().to(torch.int32))
    tables[children] = -1
    lens[children] = 0
    return {"pos": pos, "pool": pool, "refs": refs, "tables": tables, "lens": lens}


def _compact(s):
    refs, tables, pool = s["refs"], s["tables"], s["pool"]
    ids = torch.arange(refs.numel(), device="cuda")
    live = refs > 0
    count = live.sum()
    moved = live & (ids >= count)
    free = _free_ids(refs)
    to = torch.where(moved, free[(torch.cumsum(moved, 0) - 1).clamp(min=0)], torch.where(live, ids, -1))
    src = torch.nonzero_static(moved, size=s["moves"])[:, 0]
    pool[:, to[src]] = pool[:, src]
    # live pages first, in their new places: refs of page `to` are those of the page that came
    out = torch.zeros_like(refs).scatter_add_(0, to.clamp(min=0), torch.where(live, refs, torch.zeros_like(refs)))
    new = torch.where(tables >= 0, to[tables.clamp(min=0).long()].to(torch.int32), tables)
    return {"refs": out, "tables": new, "map": to.to(torch.int32), "live": count.to(torch.int32).reshape(1), "pool": pool}


def _norm(s):
    u, h = s["x"].float(), s["h"].float()
    if s["w_post"] is not None:
        u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + 1e-6) * s["w_post"].float()
    if s["gate"] is not None:
        gate = s["gate"].float().reshape(-1, u.shape[-1])
        u = u * torch.repeat_interleave(gate, u.shape[0] // gate.shape[0], 0, output_size=u.shape[0])
    h = 0.9 * h + 1.2 * u
    y = None
    if s["w_pre"] is not None:
        y = (h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * s["w_pre"].float()).to(torch.bfloat16)
    return {"h": h.to(s["h"].dtype), "y": y}


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------

def work(case):
    c = case
    if c["kind"] in ("attn", "latent"):
        seen = sum(min(x, c["window"]) if c["window"] else x for x in _lens(c))
        pages = sum(-(-x // c["page"]) for x in _lens(c))
        if c["kind"] == "attn":
            row = 2 * c["kv_heads"] * c["dim"] * (1 if c["e4m3"] else 2)
            ends = c["batch"] * c["heads"] * (4 * c["dim"] + 4)
            flops = 4 * seen * c["heads"] * c["dim"]
        else:
            row = LATENT * 2
            ends = c["batch"] * c["heads"] * (2 * LATENT + 2 * VALUE + 4)
            flops = 2 * seen * c["heads"] * (LATENT + VALUE)
        return {"bytes": seen * row + ends + 4 * pages + 4 * c["batch"], "flops": flops}
    if c["kind"] == "append":
        values = c["tokens"] * c["kv_heads"] * c["dim"] * (1 if c["latent"] else 2)
        return {"bytes": values * (2 + (1 if c["e4m3"] else 2)) + 8 * c["tokens"], "flops": 0}
    if c["kind"] == "fork":
        n = c["parents"] * c["forks"]
        # nearly every fork copies one partly filled page in every plane; its table row is written, then cleared
        table = n * (c["max_len"] * 3 // 4 // c["page"] + 1)
        return {"bytes": 2 * n * c["planes"] * c["page"] * c["width"] * 2 + 4 * 4 * table + 4 * c["pages"], "flops": 0}
    if c["kind"] == "compact":
        live = max(1, c["pages"] * c["live"] // 100)
        moves = live * (c["pages"] - live) // c["pages"]
        return {"bytes": 2 * moves * c["planes"] * c["page"] * c["width"] * 2 + 12 * c["pages"] + 8 * live, "flops": 0}
    t, n = c["rows"], c["n"]
    res = 4 if c["res32"] else 2
    gate = (0, 1, t, math.gcd(t, 64))[c["gate"]]
    bytes_ = t * n * (2 + 2 * res + (2 if c["pre"] else 0)) + 2 * n * (gate + c["post"] + c["pre"])
    return {"bytes": bytes_, "flops": 12 * t * n}


# ---------------------------------------------------------------------------
# the same from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    c = case
    if c["kind"] in ("fork", "compact") or (c["kind"] == "append" and not c["e4m3"]):
        return None                   # whole numbers and copies: nothing is computed
    global own
    was, own = own, False             # the inputs alone
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if c["kind"] == "append":
        got = {}
        for name, pages, rows, scale in (("k", s["k_pages"], s["k"], s["ks"]), ("v", s["v_pages"], s["v"], s["vs"])):
            full = pages.to(torch.float64)
            flat = full.reshape(-1, *full.shape[2:])
            seq, pos = s["seq"].tolist(), s["pos"].tolist()
            table = s["tables"].tolist()
            at = torch.tensor([table[a][p // c["page"]] * c["page"] + p % c["page"] for a, p in zip(seq, pos)], device="cuda")
            flat[at] = (rows.to(torch.float64) / scale).clamp(-448, 448)
            got[name] = full
        return got
    if c["kind"] == "norm":
        x, h = s["x"].to(torch.float64), s["h"].to(torch.float64)
        n = x.shape[1]
        if s["w_post"] is not None:
            x = x / torch.sqrt((x * x).sum(1, keepdim=True) / n + 1e-6) * s["w_post"].to(torch.float64)
        if s["gate"] is not None:
            g = s["gate"].to(torch.float64)
            g = g[None] if g.dim() == 1 else g
            x = (x.reshape(g.shape[0], -1, n) * g[:, None, :]).reshape(-1, n)
        h = h * 0.9 + x * 1.2
        if s["w_pre"] is None:
            return {"h": h, "y": None}
        return {"h": h, "y": h / torch.sqrt((h * h).sum(1, keepdim=True) / n + 1e-6) * s["w_pre"].to(torch.float64)}
    lens, table = s["lens"].tolist(), s["tables"].tolist()
    latent = c["kind"] == "latent"
    kv, width = (1, VALUE) if latent else (c["kv_heads"], c["dim"])
    group = c["heads"] // kv
    out = torch.zeros((c["batch"], c["heads"], width), dtype=torch.float64, device="cuda")
    lse = torch.full((c["batch"], c["heads"]), -math.inf, dtype=torch.float64, device="cuda")
    for b, n in enumerate(lens):
        first = max(0, n - c["window"]) if c["window"] else 0
        if first >= n:
            continue
        ids = torch.tensor(table[b][first // c["page"]:-(-n // c["page"])], device="cuda")
        lo = first - first // c["page"] * c["page"]
        for j in range(kv):
            if latent:
                k = s["pages"][ids].reshape(-1, LATENT)[lo:lo + n - first].to(torch.float64)
                v = k[:, :VALUE]
            else:
                k, v = (t.view(torch.uint8 if c["e4m3"] else torch.bfloat16)[ids, :, j].view(t.dtype).reshape(-1, width)
                        [lo:lo + n - first].to(torch.float64) for t in (s["k"], s["v"]))
            mine = slice(j * group, (j + 1) * group)
            z = s["q"][b, mine].to(torch.float64) @ k.T * (s["scale"] * (1.0 if latent else s["ks"]))
            top = z.max(1, keepdim=True)[0]
            w = torch.exp(z - top)
            out[b, mine] = w @ v / w.sum(1, keepdim=True) * (1.0 if latent else s["vs"])
            lse[b, mine] = top[:, 0] + torch.log(w.sum(1))
    return {"out": out, "lse": lse}
