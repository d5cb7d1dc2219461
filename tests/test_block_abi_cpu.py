"""Host-side argument checks of the paged cache, its attention and the block norms: bad calls are rejected before
any CUDA work, and the binding's constants and structs are the header's (no GPU needed)."""

import ctypes
import os
import re

import pytest

from conftest import ROOT

import __graft_entry__

__graft_entry__.build()
import w4a16_int4_mixture_grouped_gb300 as M  # noqa: E402
from w4a16_int4_mixture_grouped_gb300 import block as B  # noqa: E402

HEADER = open(os.path.join(ROOT, "include", "moe_w4a16.h")).read()
FAKE = 0x10000          # never dereferenced: every call below fails its host-side checks
OK, ARG, UNSUPPORTED, WORKSPACE = 0, 1, 2, 4
BIG = 1 << 30


def pages(**kw):
    c = B.Pages(FAKE, FAKE, 0, 4, 16, 0, 16 * 2 * 64, 2 * 64, 64, 1.0, 1.0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def attend(c=None, q=FAKE, stride=8 * 64, batch=2, heads=8, kv=2, dim=64, table=FAKE, tstride=4, width=4, lens=FAKE,
           seqs=2, scale=0.125, window=0, out=FAKE, ws=FAKE, bytes_=BIG):
    return B._FN["paged_attention"](q, stride, batch, heads, kv, dim, ctypes.byref(c or pages()), table, tstride, width,
                                    lens, None, seqs, scale, window, out, None, ws, bytes_, None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), ARG), (dict(heads=7), ARG), (dict(heads=0), ARG), (dict(kv=0), ARG), (dict(dim=72), UNSUPPORTED),
    (dict(dim=272), UNSUPPORTED), (dict(dim=0), UNSUPPORTED), (dict(window=-1), ARG), (dict(scale=float("nan")), ARG),
    (dict(q=None), ARG), (dict(q=FAKE + 2), ARG), (dict(stride=8 * 64 - 8), ARG), (dict(stride=8 * 64 + 4), ARG),
    (dict(out=None), ARG), (dict(lens=None), ARG), (dict(table=None), ARG), (dict(width=0), ARG), (dict(tstride=3), ARG),
    (dict(seqs=1), ARG), (dict(ws=None), WORKSPACE), (dict(bytes_=100), WORKSPACE), (dict(width=1 << 28, tstride=1 << 28), ARG),
    (dict(batch=0), OK),
    (dict(c=pages(k=None)), ARG), (dict(c=pages(v=None)), ARG), (dict(c=pages(dtype=2)), ARG),
    (dict(c=pages(num_pages=0)), ARG), (dict(c=pages(page_size=0)), ARG), (dict(c=pages(page_size=4097)), ARG),
    (dict(c=pages(token_stride=32)), ARG), (dict(c=pages(head_stride=60)), ARG), (dict(c=pages(page_stride=-8)), ARG),
    (dict(c=pages(k=FAKE + 8)), ARG), (dict(c=pages(k_scale=0.5)), ARG), (dict(c=pages(dtype=1, v_scale=0.0)), ARG),
    (dict(c=pages(dtype=1, head_stride=72)), ARG), (dict(c=pages(reserved=1)), ARG),
])
def test_attention_refuses(kw, status):
    assert attend(**kw) == status


def test_latent_attention_refuses():
    def call(c, heads=64, stride=64 * 576):
        return B._FN["latent_attention"](FAKE, stride, 2, heads, ctypes.byref(c), FAKE, 4, 4, FAKE, None, 2, 0.1, 0,
                                         FAKE, None, FAKE, BIG, None)
    good = dict(v=None, page_stride=16 * 576, token_stride=576, head_stride=576)
    assert call(pages(**good, dtype=1)) == UNSUPPORTED
    assert call(pages(**{**good, "v": FAKE})) == ARG
    assert call(pages(**{**good, "token_stride": 512})) == ARG
    assert call(pages(**good), heads=0) == ARG
    assert call(pages(**good), stride=64 * 512) == ARG


def test_workspace_sizes():
    out = ctypes.c_size_t(0)
    f, g = B._FN["attention_workspace_size"], B._FN["cache_workspace_size"]
    assert f(64, 8, 128, ctypes.byref(out)) == OK and out.value >= 256
    assert f(64, 1, 576, ctypes.byref(out)) == OK and out.value >= 256
    assert f(64, 2, 576, ctypes.byref(out)) == UNSUPPORTED
    assert f(64, 7, 128, ctypes.byref(out)) == ARG
    assert f(64, 8, 128, None) == ARG
    assert g(1000, 10, ctypes.byref(out)) == OK and out.value >= 256 + 4000
    assert g(-1, 10, ctypes.byref(out)) == ARG


def append(c=None, k=FAKE, ks=128, v=FAKE, vs=128, n=3, heads=2, dim=64, seq=FAKE, ws=FAKE):
    return B._FN["cache_append"](k, ks, v, vs, n, heads, dim, ctypes.byref(c or pages()), FAKE, 4, 4, 2, seq, FAKE, ws,
                                 BIG, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), ARG), (dict(heads=0), ARG), (dict(dim=60), UNSUPPORTED), (dict(ks=64), ARG), (dict(vs=132), ARG),
    (dict(k=None), ARG), (dict(k=FAKE + 8), ARG), (dict(v=None), ARG), (dict(seq=None), ARG), (dict(ws=None), WORKSPACE),
    (dict(c=pages(v=None)), ARG), (dict(n=0), OK), (dict(c=pages(dtype=1, k_scale=float("inf"))), ARG),
])
def test_append_refuses(kw, status):
    assert append(**kw) == status


def test_page_calls_refuse():
    def extend(refs=FAKE, pages_=8, table=FAKE, stride=4, width=4, lens=FAKE, seqs=2, ids=FAKE, n=2, page=16, pos=FAKE,
               ws=FAKE, bytes_=BIG):
        return B._FN["cache_extend"](refs, pages_, table, stride, width, lens, seqs, ids, None, n, page, pos, ws, bytes_,
                                     None)
    for kw, status in ((dict(refs=None), ARG), (dict(pages_=0), ARG), (dict(table=None), ARG), (dict(stride=3), ARG),
                       (dict(lens=None), ARG), (dict(seqs=0), ARG), (dict(ids=None), ARG), (dict(n=-1), ARG),
                       (dict(page=0), ARG), (dict(pos=None), ARG), (dict(bytes_=256), WORKSPACE), (dict(n=0), OK),
                       (dict(n=1 << 20, width=1 << 12, stride=1 << 12), UNSUPPORTED)):
        assert extend(**kw) == status, kw

    def pool(**kw):
        p = B.Pool(FAKE, 2, 8, 8 * 1024, 1024, 1024)
        for k, v in kw.items():
            setattr(p, k, v)
        return ctypes.byref(p)

    def copy(p, src=FAKE, n=1):
        return B._FN["cache_copy"](p, src, FAKE, n, FAKE, BIG, None)
    for kw in (dict(base=None), dict(num_planes=0), dict(num_pages=0), dict(page_bytes=8), dict(page_stride=1000),
               dict(page_stride=512), dict(plane_stride=-16), dict(base=FAKE + 4)):
        assert copy(pool(**kw)) == ARG, kw
    assert copy(pool(page_bytes=1 << 34, page_stride=1 << 34)) == UNSUPPORTED
    assert copy(pool(), src=None) == ARG and copy(pool(), n=-1) == ARG and copy(pool(), src=None, n=0) == OK
    assert B._FN["cache_fork"](pool(), FAKE, FAKE, 4, 4, FAKE, 2, None, FAKE, 1, 16, FAKE, BIG, None) == ARG
    assert B._FN["cache_free"](FAKE, 8, FAKE, 4, 4, FAKE, 2, None, None, 1, 16, FAKE, BIG, None) == ARG
    assert B._FN["cache_compact"](pool(), FAKE, FAKE, 4, 4, 2, FAKE, None, FAKE, FAKE, FAKE, BIG, None) == ARG


def test_block_norm_refuses():
    def norm(x=FAKE, xs=64, h=FAKE, hs=64, kind=0, gate=None, grows=1, wpost=None, wpre=FAKE, rows=4, n=64, eps=1e-6,
             out=FAKE, outs=64, y=FAKE, ys=64):
        return B._FN["block_norm"](x, xs, h, hs, kind, gate, grows, wpost, wpre, rows, n, eps, 1.0, 1.0, out, outs, y, ys,
                                   None)
    for kw, status in ((dict(kind=2), ARG), (dict(rows=-1), ARG), (dict(n=0), ARG), (dict(n=32769), UNSUPPORTED),
                       (dict(eps=float("nan")), ARG), (dict(h=None), ARG), (dict(out=None, y=None, wpre=None), ARG),
                       (dict(y=None), ARG), (dict(wpre=None), ARG), (dict(x=None, wpost=FAKE), ARG),
                       (dict(x=None, gate=FAKE), ARG), (dict(gate=FAKE, grows=3), ARG), (dict(gate=FAKE, grows=0), ARG),
                       (dict(xs=63), ARG), (dict(hs=63), ARG), (dict(outs=63), ARG), (dict(ys=63), ARG),
                       (dict(h=FAKE + 1), ARG), (dict(kind=1, h=FAKE + 2), ARG), (dict(rows=0), OK)):
        assert norm(**kw) == status, kw


def test_constants_and_structs_match_the_header():
    vals = {n: int(v) for n, v in re.findall(r"\b(MOE_W4A16_[A-Z0-9_]+)\s*(?:=\s*|)(\d+)\b", HEADER)}
    for name in ("CACHE_BF16", "CACHE_E4M3", "RESIDUAL_BF16", "RESIDUAL_F32", "LATENT_DIM", "LATENT_VALUE_DIM",
                 "MAX_HEAD_DIM", "MAX_PAGE_SIZE", "MAX_NORM_WIDTH"):
        assert vals["MOE_W4A16_" + name] == getattr(M, name), name
    for struct, cls in (("pages", B.Pages), ("pool", B.Pool)):
        body = re.search(r"typedef struct moe_w4a16_%s \{(.*?)\}" % struct, HEADER, re.S).group(1)
        body = re.sub(r"/\*.*?\*/", "", body, flags=re.S)
        names = []
        for line in body.split(";"):
            line = line.strip()
            if line:
                names += [x.strip().lstrip("*").split()[-1].lstrip("*") for x in line.split(",")]
        assert names == [f[0] for f in cls._fields_]


def test_every_declared_entry_point_has_a_signature():
    declared = set(re.findall(r"\bmoe_w4a16_((?:cache|attention|paged|latent|block)_\w+)\s*\(", HEADER))
    assert declared == set(B._SIGNATURES)
