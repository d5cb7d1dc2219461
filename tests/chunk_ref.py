"""Plain 64-bit references of the chunk attention (torch, on the tensors' device) and of the position rotation (numpy).

Attention bounds, derived from the arithmetic the header states, for one output element out = sum_j p_j v_j with
A = sum_j p_j |v_j| over L seen tokens:
  * the output is rounded once to BF16: at most 2^-8 relative, plus the subnormal spacing;
  * each probability enters the product rounded: BF16 at most 2^-8 relative, FP16 (E4M3 pages) 2^-11, with an absolute
    floor of half its subnormal spacing, 2^-25 of the row's largest: together r A + L 2^-25 max|v| (FP16);
  * scores are FP32 sums of D products, each of whose additions is off by at most 2^-23 of the sum of magnitudes (a tensor
    core may cut instead of rounding): |ds| <= (D + 8) 2^-23 scale sum_i |q_i k_ij| =: e_j, entering each probability, and
    their sum, as a relative error of at most e: together 2 e A;
  * the exponent's argument (up to 2^7 where it matters) is rounded to FP32, 2^-17 relative at most after the
    exponential; the exponential itself, and the sum's additions: 2^-20; together 2^-16 A;
  * the value product adds L / 16 partial sums in FP32, each off by at most 2^-23 A, and 64 more for rescalings and joins.
lse: e + 2^-16 + 2^-22 (|lse| + L / 16).
"""

from __future__ import annotations

import math

import numpy as np
import torch


def attention(q, starts, k, v, tables, lens, scale, window=0, ks=1.0, vs=1.0, seq_ids=None):
    """q [T, H, D], pages k, v [P, S, Hkv, D], starts / tables / lens lists of numbers. -> (out, bound, lse, lse bound) in
    float64; rows of no chunk are NaN."""
    t, h, d = q.shape
    pages, page, hkv, _ = k.shape
    group = h // hkv
    e4m3 = k.dtype == torch.float8_e4m3fn
    out = torch.full((t, h, d), math.nan, dtype=torch.float64, device=q.device)
    bound, lse = out.clone(), out[:, :, 0].clone()
    lbound = lse.clone()
    for b in range(len(starts) - 1):
        t0, t1 = starts[b], starts[b + 1]
        if not 0 <= t0 < t1 <= t:
            continue
        out[t0:t1], bound[t0:t1], lse[t0:t1], lbound[t0:t1] = 0, 0, -math.inf, 0
        row = b if seq_ids is None else seq_ids[b]
        if not 0 <= row < len(lens):
            continue
        table = list(tables[row])
        n = min(max(int(lens[row]), 0), len(table) * page)
        js = [j for j in range(n) if 0 <= table[j // page] < pages]
        if not js:
            continue
        at = torch.tensor(js, device=q.device)
        ids = torch.tensor([table[j // page] for j in js], device=q.device)
        pos = torch.arange(n - (t1 - t0), n, device=q.device)[:, None]
        seen = at[None] <= pos
        if window:
            seen &= at[None] > pos - window
        count = seen.sum(1)[:, None].double()
        for j in range(hkv):
            kk = k[:, :, j].to(torch.float32)[ids, at % page].double() * ks
            vv = v[:, :, j].to(torch.float32)[ids, at % page].double()
            for head in range(j * group, (j + 1) * group):
                x = q[t0:t1, head].double()
                s = (x @ kk.T * scale).masked_fill(~seen, -math.inf)
                e = ((x.abs() @ kk.abs().T) * ((d + 8) * 2.0 ** -23 * abs(scale))).masked_fill(~seen, 0).amax(1, keepdim=True)
                m = s.amax(1, keepdim=True)
                m = torch.where(m == -math.inf, torch.zeros_like(m), m)
                w = torch.exp(s - m)
                l = w.sum(1, keepdim=True)
                p = torch.where(l > 0, w / l, torch.zeros_like(w))
                o, a = p @ vv * vs, p @ vv.abs() * vs
                r = 2.0 ** -11 if e4m3 else 2.0 ** -8
                rel = r + 2 * e + 2.0 ** -16 + (count / 16 + 64) * 2.0 ** -23
                floor = count * 2.0 ** -25 * (vv.abs() * seen.any(0)[:, None]).amax() * vs if e4m3 else 0.0
                out[t0:t1, head] = o
                bound[t0:t1, head] = 2.0 ** -8 * 1.01 * o.abs() + rel * a + floor + 2.0 ** -133
                ll = (m + torch.log(l))[:, 0]
                lse[t0:t1, head] = ll
                lbound[t0:t1, head] = e[:, 0] + 2.0 ** -16 + 2.0 ** -22 * (ll.abs() + count[:, 0] / 16).nan_to_num(posinf=0)
    return out, bound, lse, lbound


def frequencies(dim, theta, scaling="none", factor=1.0, trained=0, low=1.0, high=32.0, given=None):
    """Radians a token of each pair."""
    got = []
    for i in range(dim // 2):
        if scaling == "given":
            got.append(float(given[i]))
            continue
        base = theta * factor ** (dim / (dim - 2.0)) if scaling == "base" else theta
        f = base ** (-2.0 * i / dim)
        keep = 1.0
        if scaling == "linear":
            keep = 0.0
        elif scaling == "turns":
            keep = min(1.0, max(0.0, (trained * f / (2 * math.pi) - low) / (high - low)))
        elif scaling == "index":
            at = [dim * math.log(trained / (2 * math.pi * n)) / (2 * math.log(theta)) for n in (high, low)]
            first, last = max(0, math.floor(at[0])), min(dim - 1, math.ceil(at[1]))
            keep = 1.0 - min(1.0, max(0.0, (i - first) / max(0.001, last - first)))
        got.append(keep * f + (1 - keep) * f / factor)
    return np.array(got)


def rotate(x, pos, freqs, offset, interleaved, magnitude=1.0):
    """x [T, H, D] float64 -> (turned, bound before the output's rounding). FP32: the angle is off by at most 2^-25 turns
    (its 32 bits cut to 24, half a step) and 2^31 * 2^-53 of a turn times the frequency at most (positions below 2^20:
    2^-33); sine, cosine, the magnitude and the two products and their sum round five times: together less than
    2^-21 of the pair's magnitudes."""
    t, h, d = x.shape
    n = len(freqs)
    # the angle modulo a turn, in turns, with all bits: products of Python integers over 2^64
    two64 = 1 << 64
    turns = [int(math.floor((f / (2 * math.pi)) % 1.0 * two64)) for f in freqs]
    angle = np.array([[((int(p) * w) % two64) / two64 for w in turns] for p in pos]).reshape(t, n) * 2 * np.pi
    c, s = np.cos(angle)[:, None] * magnitude, np.sin(angle)[:, None] * magnitude
    out, bound = x.copy(), np.zeros_like(x)
    if interleaved:
        ia, ib = offset + 2 * np.arange(n), offset + 2 * np.arange(n) + 1
    else:
        ia, ib = offset + np.arange(n), offset + n + np.arange(n)
    a, b = x[:, :, ia], x[:, :, ib]
    out[:, :, ia], out[:, :, ib] = a * c - b * s, a * s + b * c
    bound[:, :, ia] = bound[:, :, ib] = 2.0 ** -21 * abs(magnitude) * (np.abs(a) + np.abs(b))
    return out, bound
