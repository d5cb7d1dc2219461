"""Plain 64-bit references of the paged attention, the page operations and the block norms (numpy, host).

Attention bounds, derived from the arithmetic the header states, for one output element
out = sum_j p_j v_j with A = sum_j p_j |v_j|:
  * the output is rounded once to BF16 (8 significant bits, so at most 2^-8 relative): 2^-8 |out|, plus the
    BF16 subnormal spacing;
  * each probability enters the product rounded to BF16: at most 2^-8 relative, together 2^-8 A;
  * scores are FP32 sums of D products: |ds| <= (D + 8) 2^-24 scale sum_i |q_i k_ij| =: e_j, entering each
    probability (and their sum) as a relative error of at most e: together 2 e A;
  * exponentials, running maxima, sums and the joins of parts: a few FP32 roundings per part, 2^-18 A covers
    64 of them.
lse: e + 2^-20 (1 + |lse|).
"""

from __future__ import annotations

import numpy as np

LATENT, VALUE = 576, 512


def seen_tokens(table, n, page, window, num_pages):
    lo = max(0, n - window) if window else 0
    return [j for j in range(lo, n) if 0 <= table[j // page] < num_pages]


def attention(q, rows_k, rows_v, group, tables, lens, page, num_pages, scale, window, v_scale=1.0, seq_ids=None):
    """q [B, H, D] float64; rows_k(p, t) -> [Hkv, D], rows_v(p, t) -> [Hkv, Dv] float64 (k scaled, v unscaled).
    -> (out, out bound, lse, lse bound)."""
    b, h, d = q.shape
    out, bound, lse, lbound = [], [], np.full((b, h), -np.inf), np.zeros((b, h))
    for i in range(b):
        row = i if seq_ids is None else seq_ids[i]
        n = min(max(int(lens[row]), 0), tables.shape[1] * page)
        js = seen_tokens(tables[row], n, page, window, num_pages)
        if not js:
            dv = rows_v(0, 0).shape[1]
            out.append(np.zeros((h, dv)))
            bound.append(np.zeros((h, dv)))
            continue
        k = np.stack([rows_k(tables[row][j // page], j % page) for j in js])      # [L, Hkv, D]
        v = np.stack([rows_v(tables[row][j // page], j % page) for j in js])
        k, v = np.repeat(k, group, 1), np.repeat(v, group, 1)                     # [L, H, D]
        s = np.einsum("hd,lhd->hl", q[i], k) * scale
        e = ((d + 8) * 2.0 ** -24 * abs(scale) * np.einsum("hd,lhd->hl", np.abs(q[i]), np.abs(k))).max(1)
        m = s.max(1, keepdims=True)
        w = np.exp(s - m)
        l = w.sum(1, keepdims=True)
        p = w / l
        o = np.einsum("hl,lhd->hd", p, v) * v_scale
        a = np.einsum("hl,lhd->hd", p, np.abs(v)) * v_scale
        out.append(o)
        bound.append(2.0 ** -8 * 1.01 * np.abs(o) + (2.0 ** -8 + 2 * e[:, None] + 2.0 ** -18) * a + 2.0 ** -133)
        lse[i] = (m + np.log(l))[:, 0]
        lbound[i] = e + 2.0 ** -20 * (1 + np.abs(lse[i]))
    return np.stack(out), np.stack(bound), lse, lbound


# ---------------------------------------------------------------------------
# page operations, one entry after the other; tables, lens and refs are numpy arrays, changed in place
# ---------------------------------------------------------------------------

def _lowest_free(refs, n):
    return [int(p) for p in np.nonzero(refs <= 0)[0][:n]]


def pages_of(n, page):
    return -(-n // page)


def extend(refs, tables, lens, seq_ids, counts, page):
    """-> positions. Entry i gets its pages if the entries up to and including it need no more than are free."""
    free = _lowest_free(refs, len(refs))
    used, pos = 0, []
    for s, c in zip(seq_ids, counts):
        if not 0 <= s < len(lens) or lens[s] + c > tables.shape[1] * page:
            pos.append(-1)
            continue
        first, cols = pages_of(lens[s], page), pages_of(lens[s] + c, page)
        need = cols - first
        if need and used + need > len(free):
            used += need
            pos.append(-1)
            continue
        for k in range(need):
            tables[s, first + k] = free[used + k]
            refs[free[used + k]] = 1
        used += need
        pos.append(int(lens[s]))
        lens[s] += c
    return np.array(pos, dtype=np.int32)


def fork(pool, refs, tables, lens, parents, children, page):
    free = _lowest_free(refs, len(refs))
    used = 0
    for a, b in zip(parents, children):
        if lens[b] != 0:
            continue
        n = int(lens[a])
        cols = pages_of(n, page)
        row = tables[a, :cols].copy()
        if n % page and row[-1] >= 0:
            used += 1
            if used > len(free):
                continue
            dst = free[used - 1]
            pool[:, dst] = pool[:, row[-1]]
            row[-1] = dst
            refs[dst] = 0
        tables[b, :cols] = row
        for p in row:
            if p >= 0:
                refs[p] += 1
        lens[b] = n


def free(refs, tables, lens, seq_ids, page, keep=None):
    for i, s in enumerate(seq_ids):
        kept = 0 if keep is None else int(keep[i])
        cols = tables.shape[1] if kept <= 0 else max(0, int(lens[s]) - kept) // page
        for c in range(cols):
            if tables[s, c] >= 0:
                refs[tables[s, c]] -= 1
                tables[s, c] = -1
        if kept <= 0:
            lens[s] = 0


def compact(pool, refs, tables):
    """-> (refs, tables, map, live); pool changed in place."""
    live = int((refs > 0).sum())
    holes = [p for p in range(live) if refs[p] <= 0]
    to = np.where(refs > 0, np.arange(len(refs)), -1).astype(np.int32)
    for p in range(live, len(refs)):
        if refs[p] > 0:
            to[p] = holes.pop(0)
            pool[:, to[p]] = pool[:, p]
    out = np.zeros_like(refs)
    for p in range(len(refs)):
        if refs[p] > 0:
            out[to[p]] = refs[p]
    new = tables.copy()
    for i in np.ndindex(tables.shape):
        if tables[i] >= 0:
            new[i] = to[tables[i]]
    return out, new, to, live


# ---------------------------------------------------------------------------
# norms
# ---------------------------------------------------------------------------

def block_norm(x, h, w_post, w_pre, gate, eps, rs, bs, res32):
    """-> (h', its bound, y or None, its bound). FP32 bounds: a row's mean of squares is summed in at most
    log2(n) + n / 32 + 8 roundings of positive terms, so its root is off by at most half of that in 2^-24; the
    other steps are at most eight FP32 roundings each; a BF16 rounding is at most 2^-8 relative."""
    n = h.shape[1]
    mean = (np.log2(max(n, 2)) + n / 32 + 8) / 2 * 2.0 ** -24
    step = 8 * 2.0 ** -24
    u = None
    new, slack = rs * h, step * np.abs(rs * h)
    if x is not None:
        u = x
        if w_post is not None:
            u = x / np.sqrt((x * x).mean(1, keepdims=True) + eps) * w_post
        if gate is not None:
            g = gate.reshape(-1, n)
            u = u * np.repeat(g, h.shape[0] // g.shape[0], 0)
        new = new + bs * u
        slack = slack + (mean + step) * np.abs(bs * u)
    hb = slack + (2.0 ** -8 * np.abs(new) + 2.0 ** -133 if not res32 else 2.0 ** -24 * np.abs(new))
    if w_pre is None:
        return new, hb * 1.01, None, None
    root = np.sqrt((new * new).mean(1, keepdims=True) + eps)
    y = new / root * w_pre
    # an error of h' moves the element itself and, through the root, by at most the root mean square of the slacks
    shift = np.sqrt((slack * slack).mean(1, keepdims=True)) / root
    yb = np.abs(w_pre) * slack / root + (shift + mean + step + 2.0 ** -8) * np.abs(y) + 2.0 ** -133
    return new, hb * 1.01, y, yb * 1.01
