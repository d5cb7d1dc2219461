"""Host-side argument checks of the chunk attention and the position rotation, and the rotation's frequencies: no GPU
needed."""

import ctypes
import os
import re
from fractions import Fraction

import numpy as np
import pytest

from conftest import ROOT

import __graft_entry__

__graft_entry__.build()
import w4a16_int4_mixture_grouped_gb300 as M  # noqa: E402
from w4a16_int4_mixture_grouped_gb300 import block as B  # noqa: E402
from w4a16_int4_mixture_grouped_gb300 import positions as P  # noqa: E402

import chunk_ref as C  # noqa: E402
from test_block_abi_cpu import ARG, BIG, FAKE, OK, UNSUPPORTED, WORKSPACE, pages  # noqa: E402

HEADER = open(os.path.join(ROOT, "include", "moe_w4a16.h")).read()


def chunk(c=None, q=FAKE, stride=8 * 64, tokens=6, starts=FAKE, batch=2, heads=8, kv=2, dim=64, table=FAKE, tstride=4,
          width=4, lens=FAKE, seqs=2, scale=0.125, window=0, out=FAKE + (1 << 20), ws=FAKE, bytes_=BIG):
    return B._FN["paged_chunk_attention"](q, stride, tokens, starts, batch, heads, kv, dim, ctypes.byref(c or pages()), table,
                                          tstride, width, lens, None, seqs, scale, window, out, None, ws, bytes_, None)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), ARG), (dict(batch=-1), ARG), (dict(heads=7), ARG), (dict(heads=0), ARG), (dict(kv=0), ARG),
    (dict(dim=72), UNSUPPORTED), (dict(dim=272), UNSUPPORTED), (dict(dim=0), UNSUPPORTED), (dict(window=-1), ARG),
    (dict(scale=float("nan")), ARG), (dict(q=None), ARG), (dict(q=FAKE + 2), ARG), (dict(stride=8 * 64 - 8), ARG),
    (dict(stride=8 * 64 + 4), ARG), (dict(out=None), ARG), (dict(out=FAKE + 4), ARG), (dict(out=FAKE), ARG), (dict(lens=None), ARG),
    (dict(starts=None), ARG), (dict(table=None), ARG), (dict(width=0), ARG), (dict(tstride=3), ARG), (dict(seqs=1), ARG),
    (dict(ws=None), WORKSPACE), (dict(bytes_=100), WORKSPACE), (dict(width=1 << 28, tstride=1 << 28), ARG),
    (dict(tokens=1 << 29), UNSUPPORTED), (dict(tokens=0), OK), (dict(batch=0), OK),
    (dict(c=pages(k=None)), ARG), (dict(c=pages(v=None)), ARG), (dict(c=pages(dtype=2)), ARG),
    (dict(c=pages(token_stride=32)), ARG), (dict(c=pages(head_stride=60)), ARG), (dict(c=pages(k=FAKE + 8)), ARG),
    (dict(c=pages(k_scale=0.5)), ARG), (dict(c=pages(dtype=1, v_scale=0.0)), ARG),
])
def test_chunk_attention_refuses(kw, status):
    assert chunk(**kw) == status


def test_chunk_workspace():
    out = ctypes.c_size_t(0)
    f = B._FN["paged_chunk_workspace_size"]
    for heads, kv, dim in ((64, 8, 128), (1, 1, 16), (8, 8, 256), (300, 1, 64)):
        assert f(heads, kv, dim, ctypes.byref(out)) == OK and 256 <= out.value < 1 << 27
    assert f(64, 8, 576, ctypes.byref(out)) == UNSUPPORTED and f(64, 8, 24, ctypes.byref(out)) == UNSUPPORTED
    assert f(64, 7, 128, ctypes.byref(out)) == ARG and f(64, 8, 128, None) == ARG


def desc(**kw):
    d = P.RotaryDesc(FAKE, 64, 0, 0, 1.0)
    for k, v in kw.items():
        setattr(d, k, v)
    return ctypes.byref(d)


def turn(x=FAKE, xs=128, xh=64, pos=FAKE, tokens=3, heads=2, dim=64, r=None, out=FAKE + 4096, os_=128, oh=64):
    return P._FN["rotary"](x, xs, xh, pos, tokens, heads, dim, r or desc(), out, os_, oh, None)


@pytest.mark.parametrize("kw,status", [
    (dict(tokens=-1), ARG), (dict(heads=0), ARG), (dict(dim=62), ARG), (dict(x=None), ARG), (dict(out=None), ARG),
    (dict(pos=None), ARG), (dict(x=FAKE + 1), ARG), (dict(xs=-1), ARG), (dict(oh=32), ARG), (dict(os_=64), ARG),
    (dict(os_=0), ARG), (dict(out=FAKE, os_=256), ARG), (dict(r=desc(dim=63)), ARG), (dict(r=desc(dim=0)), ARG),
    (dict(r=desc(offset=2)), ARG), (dict(r=desc(offset=-2)), ARG), (dict(r=desc(turns=None)), ARG),
    (dict(r=desc(turns=FAKE + 4)), ARG), (dict(r=desc(interleaved=2)), ARG), (dict(r=desc(magnitude=float("inf"))), ARG),
    (dict(r=desc(dim=2048), dim=4096), ARG), (dict(tokens=0), OK), (dict(tokens=0, x=None), OK),
])
def test_rotary_refuses(kw, status):
    assert turn(**kw) == status


def append(c=None, q=FAKE, qs=8 * 64, qh=8, qo=FAKE, qos=8 * 64, k=FAKE, ks=128, v=FAKE, vs=128, n=3, heads=2, dim=64, r=None,
           seq=FAKE, pos=FAKE, ws=FAKE):
    return B._FN["cache_append_rotary"](q, qs, qh, qo, qos, k, ks, v, vs, n, heads, dim, r or desc(), ctypes.byref(c or pages()),
                                        FAKE, 4, 4, 2, seq, pos, ws, BIG, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), ARG), (dict(heads=0), ARG), (dict(dim=60), UNSUPPORTED), (dict(ks=64), ARG), (dict(vs=132), ARG),
    (dict(k=None), ARG), (dict(k=FAKE + 8), ARG), (dict(v=None), ARG), (dict(seq=None), ARG), (dict(pos=None), ARG),
    (dict(ws=None), WORKSPACE), (dict(c=pages(v=None)), ARG), (dict(q=None), ARG), (dict(qo=None), ARG), (dict(qh=0), ARG),
    (dict(qs=64), ARG), (dict(qos=8 * 64 + 2), ARG), (dict(qos=9 * 64), ARG), (dict(qs=9 * 64), ARG), (dict(q=FAKE + 2), ARG), (dict(qo=FAKE + 8), ARG),
    (dict(r=desc(dim=8)), UNSUPPORTED), (dict(r=desc(dim=32, offset=4)), UNSUPPORTED), (dict(r=desc(dim=128)), ARG),
    (dict(r=desc(dim=4, interleaved=1)), UNSUPPORTED), (dict(n=0), OK), (dict(n=0, q=None, qo=None, k=None, v=None), OK),
])
def test_append_rotary_refuses(kw, status):
    assert append(**kw) == status


def frequencies(dim=64, theta=10000.0, scaling=0, factor=2.0, trained=4096, low=1.0, high=32.0, given=None, out=True):
    buf = (ctypes.c_uint64 * 512)()
    values = None if given is None else (ctypes.c_double * len(given))(*given)
    return P._FN["rotary_frequencies"](dim, theta, scaling, factor, trained, low, high, values, buf if out else None)


@pytest.mark.parametrize("kw,status", [
    (dict(), OK), (dict(dim=0), ARG), (dict(dim=63), ARG), (dict(dim=1026), ARG), (dict(theta=0.0), ARG),
    (dict(theta=float("nan")), ARG), (dict(scaling=6), ARG), (dict(scaling=-1), ARG), (dict(scaling=1, factor=0.5), ARG),
    (dict(scaling=2, dim=2), ARG), (dict(scaling=3, trained=0), ARG), (dict(scaling=3, low=4.0, high=4.0), ARG),
    (dict(scaling=4, low=0.0), ARG), (dict(scaling=4, theta=1.0), ARG), (dict(scaling=5), ARG), (dict(out=False), ARG),
    (dict(scaling=5, dim=2, given=[float("inf")]), ARG), (dict(scaling=5, dim=2, given=[1.0], theta=0.0), OK),
    (dict(scaling=0, theta=1.0, dim=2), OK),
])
def test_frequencies_refuse(kw, status):
    assert frequencies(**kw) == status


@pytest.mark.parametrize("scaling,kw", [("none", {}), ("linear", dict(factor=4.0)), ("base", dict(factor=8.0)),
                                        ("turns", dict(factor=8.0, trained_length=8192, low=1.0, high=4.0)),
                                        ("index", dict(factor=32.0, trained_length=4096, low=1.0, high=32.0)),
                                        ("index", dict(factor=4.0, trained_length=64, low=0.001, high=0.002))])
@pytest.mark.parametrize("dim,theta", [(2, 10000.0), (16, 10000.0), (64, 5e5), (128, 1e6), (1024, 100.0)])
def test_frequencies(dim, theta, scaling, kw):
    if scaling == "base" and dim == 2:
        pytest.skip("refused: one pair has no other base")
    got = M.rotary_frequencies(dim, theta, scaling, **kw).numpy().view(np.uint64)
    plain = dict(kw)
    if "trained_length" in plain:
        plain["trained"] = plain.pop("trained_length")
    want = C.frequencies(dim, theta, scaling, **plain) / (2 * np.pi)
    # a few roundings of a double (a power's are up to a few 2^-53 of the exponent's size), and the fixed point's 2^-64
    assert (np.abs(got.astype(np.float64) / 2.0 ** 64 - want) <= 2.0 ** -48 * want + 2.0 ** -63).all()


def test_given_frequencies():
    given = [0.0, 1.0, -1.0, 2 * np.pi, 100.0, 1e-12]
    got = M.rotary_frequencies(12, scaling="given", given=given).numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64
    want = np.mod(np.array(given) / (2 * np.pi), 1.0)
    d = np.abs(got - want)
    assert (np.minimum(d, 1 - d) <= 2.0 ** -48).all()
    for kw in (dict(scaling="given", given=[1.0]), dict(scaling="none", given=given), dict(scaling="dynamic")):
        with pytest.raises(ValueError):
            M.rotary_frequencies(12, **kw)
    with pytest.raises(M.MoeW4A16Error):
        M.rotary_frequencies(12, scaling="given")


def test_constants_and_struct_match_the_header():
    vals = {n: int(v) for n, v in re.findall(r"\b(MOE_W4A16_[A-Z0-9_]+)\s*(?:=\s*|)(\d+)\b", HEADER)}
    for name in ("NONE", "LINEAR", "BASE", "TURNS", "INDEX", "GIVEN"):
        assert vals["MOE_W4A16_ROTARY_" + name] == getattr(M, "ROTARY_" + name)
    assert vals["MOE_W4A16_MAX_ROTARY_DIM"] == M.MAX_ROTARY_DIM
    body = re.search(r"typedef struct moe_w4a16_rotary_desc \{(.*?)\}", HEADER, re.S).group(1)
    names = [x.strip().split()[-1].lstrip("*") for x in re.sub(r"/\*.*?\*/", "", body, flags=re.S).split(";") if x.strip()]
    assert names == [f[0] for f in P.RotaryDesc._fields_]
    assert set(re.findall(r"\bmoe_w4a16_(rotary\w*)\s*\(", HEADER)) == set(P._SIGNATURES)


@pytest.mark.parametrize("out", [16, 8 * 64 * 2, 5 * 8 * 64 * 2 + 1008, -6 * 8 * 64 * 2 + 16, -16])
def test_chunk_attention_refuses_an_output_that_begins_within_its_queries(out):
    assert chunk(q=FAKE + (1 << 16), out=FAKE + (1 << 16) + out) == ARG


def test_chunk_attention_refuses_an_output_between_rows_that_it_does_not_fit():
    # rows of 1024 bytes, 4096 apart; outputs of 1024 behind each other run into the next query
    assert chunk(stride=4 * 8 * 64, out=FAKE + 1024) == ARG and chunk(stride=4 * 8 * 64, out=FAKE + 5 * 4096 - 16) == ARG


def test_chunk_attention_refuses_sums_over_its_queries_or_outputs():
    def call(lse):
        return B._FN["paged_chunk_attention"](FAKE, 512, 6, FAKE, 2, 8, 2, 64, ctypes.byref(pages()), FAKE, 4, 4, FAKE, None, 2, 0.125, 0,
                                              FAKE + (1 << 20), lse, FAKE, BIG, None)
    for lse in (FAKE, FAKE + 6 * 1024 - 4, FAKE + (1 << 20), FAKE + (1 << 20) + 6 * 1024 - 4, FAKE + (1 << 20) - 6 * 8 * 4 + 4):
        assert call(lse) == ARG


KEYS, VALUES = FAKE + (1 << 20), FAKE + (2 << 20)


@pytest.mark.parametrize("kw", [
    dict(qo=FAKE + 16), dict(qo=FAKE + 1024), dict(qo=FAKE - 1024), dict(q=FAKE + 2 * 1024, qo=FAKE), dict(qo=FAKE + 8192 - 2048, qs=4096),
    dict(qo=KEYS), dict(qo=KEYS + 2 * 256 + 240), dict(qo=KEYS - 2 * 1024 - 16), dict(qo=VALUES), dict(qo=VALUES + 16),
    dict(q=KEYS - 1024 + 16, qo=KEYS - 1024 + 16, qs=1024, qos=1024, ks=1024, k=KEYS)])
def test_append_rotary_refuses_turned_queries_over_its_other_rows(kw):
    args = dict(q=FAKE, qo=FAKE + (3 << 20), k=KEYS, v=VALUES)
    args.update(kw)
    assert append(**args) == ARG


def test_append_rotary_refuses_turned_queries_over_a_latent_row():
    args = dict(c=pages(v=None), v=None, vs=0, heads=1, dim=64, ks=64, qh=8, r=desc(dim=64), q=FAKE, k=KEYS)
    assert append(qo=KEYS + 64, **args) == ARG


@pytest.mark.parametrize("kw", [
    dict(out=FAKE + 2), dict(out=FAKE + 128), dict(out=FAKE + 256), dict(out=FAKE + 2 * 256 + 126), dict(out=FAKE - 2 * 256 - 126),
    dict(out=FAKE + 128, xs=128, xh=256), dict(xs=512, xh=64, out=FAKE + 256, os_=512, oh=64, heads=3),
    dict(xs=64, xh=3 * 64, out=FAKE + 6 * 128 - 2), dict(xs=0, xh=0, out=FAKE + 126, os_=128), dict(xs=1024, xh=0, out=FAKE + 2048 + 126)])
def test_rotary_refuses_outputs_over_other_rows(kw):
    assert turn(**kw) == ARG


PI = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)          # to 2^-160


@pytest.mark.parametrize("sign", [1, -1])
def test_frequencies_against_exact_turns(sign):
    """Each is off by a cut to 2^-64 turns and, for the division and two pi in double precision, 2^-52 of itself: small ones
    of either sign keep their own bits."""
    rng = np.random.default_rng(3)
    given = [1.0, 0.5, 1e-3, 1e-6, 1e-9, 1e-12, 1e-15, 1e-18, 3e-20, 1e-25, 0.0, 6.0, 7.0, 100.0, 12345.678, 2.0 ** -11]
    given += [float(x) for x in np.exp(rng.uniform(-50, 3, 200))]
    got = M.rotary_frequencies(2 * len(given), scaling="given", given=[sign * f for f in given]).numpy().view(np.uint64)
    for f, bits in zip(given, got):
        want = Fraction(f) / (2 * PI) * 2 ** 64
        off = (sign * int(bits) - want) % 2 ** 64
        assert min(off, 2 ** 64 - off) <= 1 + want / 2 ** 52, (sign * f, int(bits))


def test_scaled_frequencies_turn_as_far_as_exact_ones():
    """p f_i at far positions, from the frequency in double precision and exact numbers on: |p| (2^-64 + 2^-52 f / 2 pi)
    turns, and what two ways of computing a power differ by."""
    for dim, theta in ((128, 1e6), (64, 10000.0)):
        bits = M.rotary_frequencies(dim, theta).numpy().view(np.uint64)
        for w, f in zip(bits, C.frequencies(dim, theta)):
            t = Fraction(f) / (2 * PI)
            for p in (1, -1, 131071, 1 << 24, (1 << 31) - 1, -(1 << 31)):
                off = (Fraction(p * int(w), 2 ** 64) - p * t) % 1
                assert min(off, 1 - off) <= abs(p) * (Fraction(1, 2 ** 64) + t / 2 ** 50)
