"""The norms around a block against the plain 64-bit form."""

import numpy as np
import pytest
import torch

import block_ref as R

pytestmark = pytest.mark.gpu

M = pytest.importorskip("w4a16_int4_mixture_grouped_gb300") if torch.cuda.is_available() else None
DEV = torch.device("cuda", 0) if torch.cuda.is_available() else None


def bf16(rng, *shape, scale=1.0, shift=0.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale + shift).astype(np.float32)).to(DEV).to(torch.bfloat16)


def f64(t):
    return None if t is None else t.detach().to(torch.float64).cpu().numpy()


def check(x, h, w_post, w_pre, gate, rs=0.75, bs=1.5, eps=1e-6, **kw):
    hin = f64(h)
    out, y = M.block_norm(x, h, w_post=w_post, w_pre=w_pre, gate=gate, eps=eps, residual_scale=rs, block_scale=bs, **kw)
    nh, hb, ny, yb = R.block_norm(f64(x), hin, f64(w_post), f64(w_pre), f64(gate), eps, rs, bs,
                                  h.dtype == torch.float32)
    d = np.abs(f64(out) - nh)
    assert (d <= hb).all(), f"h': {(d / np.maximum(hb, 1e-300)).max()} of the bound"
    if w_pre is None:
        assert y is None
    else:
        d = np.abs(f64(y) - ny)
        assert (d <= yb).all(), f"y: {(d / np.maximum(yb, 1e-300)).max()} of the bound"
    return out, y


WIDTHS = [1, 2, 7, 8, 64, 129, 1000, 1024, 2047, 4096, 5003, 7168, 8200, 16384, 20000, 32768]


@pytest.mark.parametrize("n", WIDTHS)
@pytest.mark.parametrize("res32", [False, True])
def test_widths(n, res32):
    rng = np.random.default_rng(n)
    t = 5
    h = bf16(rng, t, n, scale=3.0)
    h = h.float() * 1.001 if res32 else h
    check(bf16(rng, t, n), h, bf16(rng, n, scale=0.1, shift=1.0), bf16(rng, n, scale=0.1, shift=1.0), bf16(rng, n))


@pytest.mark.parametrize("rows", [1, 2, 151, 1000, 3001])
def test_rows(rows):
    rng = np.random.default_rng(rows)
    check(bf16(rng, rows, 512), bf16(rng, rows, 512), bf16(rng, 512), bf16(rng, 512), None)


@pytest.mark.parametrize("n", [1032, 2048, 2056, 7168, 8192, 8200, 16384])
@pytest.mark.parametrize("res32", [False, True])
@pytest.mark.parametrize("gate", [None, "channel", "token", "sequence"])
def test_many_long_rows(n, res32, gate):
    rng = np.random.default_rng(n + res32)
    t = 1300 if n < 8000 else 1240
    h = bf16(rng, t, n, scale=2.0)
    g = {None: None, "channel": bf16(rng, n), "token": bf16(rng, t, n), "sequence": bf16(rng, 20, n)}[gate]
    check(bf16(rng, t, n), h.float() if res32 else h, bf16(rng, n), bf16(rng, n), g)


@pytest.mark.parametrize("n", [1, 3, 8, 57, 63, 64, 65, 121, 250, 256, 257, 505, 512, 513, 1021, 1026, 4100, 8185, 8191, 16377])
@pytest.mark.parametrize("res32", [False, True])
def test_widths_of_many_rows(n, res32):
    """Rows that start at every alignment; neighbours untouched (a guard column on each side of the outputs)."""
    rng = np.random.default_rng(n + res32)
    t = 701
    h = bf16(rng, t, n, scale=2.0)
    h = h.float() if res32 else h
    x, w1, w2 = bf16(rng, t, n), bf16(rng, n), bf16(rng, n)
    out, y = check(x, h, w1, w2, bf16(rng, n))
    flat_h = torch.full((t * n + 16,), 7.0, dtype=h.dtype, device=DEV)
    flat_y = torch.full((t * n + 16,), 7.0, dtype=torch.bfloat16, device=DEV)
    check(x, h, w1, w2, None, out=flat_h[8:8 + t * n].view(t, n), y=flat_y[8:8 + t * n].view(t, n))
    for f in (flat_h, flat_y):
        assert (f[:8] == 7).all() and (f[8 + t * n:] == 7).all()


@pytest.mark.parametrize("post,pre", [(False, False), (False, True), (True, False)])
def test_many_long_rows_without_a_norm(post, pre):
    rng = np.random.default_rng(post + 2 * pre)
    t, n = 1300, 1544
    check(bf16(rng, t, n), bf16(rng, t, n), bf16(rng, n) if post else None, bf16(rng, n) if pre else None, None)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("gate", [None, "channel", "sequence", "token"])
@pytest.mark.parametrize("n", [256, 261])
def test_forms(post, pre, gate, n):
    rng = np.random.default_rng(n + post * 2 + pre)
    t = 12
    g = {None: None, "channel": bf16(rng, n), "sequence": bf16(rng, 3, n), "token": bf16(rng, t, n)}[gate]
    check(bf16(rng, t, n), bf16(rng, t, n).float(), bf16(rng, n) if post else None, bf16(rng, n) if pre else None, g)


@pytest.mark.parametrize("n", [256, 261])
def test_first_norm_has_no_block_before_it(n):
    rng = np.random.default_rng(n)
    h, w = bf16(rng, 9, n), bf16(rng, n)
    out, y = check(None, h, None, w, None, rs=1.0)
    assert out is h
    out, _ = check(None, h, None, w, None, rs=0.5)
    assert out is not h


@pytest.mark.parametrize("n", [1024, 1021])
def test_in_place_strided_and_unaligned(n):
    rng = np.random.default_rng(n)
    t = 7
    wide = bf16(rng, t, 2 * n + 8)
    x = wide[:, 8:8 + n]
    res = bf16(rng, t, n + 24).float()
    h = res[:, 16:16 + n]
    w1, w2 = bf16(rng, n), bf16(rng, n)
    want, wy = check(x, h, w1, w2, None)
    keep = res.clone()
    got, y = M.block_norm(x, h, w_post=w1, w_pre=w2, eps=1e-6, residual_scale=0.75, block_scale=1.5, out=h)
    assert got is h and torch.equal(got, want) and torch.equal(y, wy)
    assert torch.equal(res[:, :16], keep[:, :16]) and torch.equal(res[:, 16 + n:], keep[:, 16 + n:])
    odd = bf16(rng, t * n + 1)[1:].view(t, n)                     # two bytes off any 16-byte boundary
    check(odd, h, w1, w2, None)


def test_extreme_rows():
    """Zero rows (eps alone under the root), tiny and large rows, and a row of one spike."""
    n = 640
    x = torch.zeros((5, n), dtype=torch.bfloat16, device=DEV)
    h = torch.zeros((5, n), dtype=torch.float32, device=DEV)
    rng = np.random.default_rng(1)
    x[1], h[1] = bf16(rng, n, scale=1e-6), bf16(rng, n, scale=1e-6).float()
    x[2], h[2] = bf16(rng, n, scale=1e12), bf16(rng, n, scale=1e12).float()
    x[3, 77], h[3, 5] = 1000.0, -2000.0
    w = bf16(rng, n)
    check(x, h, w, w, None)
    check(x, h, None, w, None)


def test_a_bad_row_stays_in_its_row():
    rng = np.random.default_rng(2)
    x, h, w = bf16(rng, 4, 96), bf16(rng, 4, 96), bf16(rng, 96)
    want = M.block_norm(x, h, w_post=w, w_pre=w)
    x[2, 3] = float("nan")
    got = M.block_norm(x, h, w_post=w, w_pre=w)
    for a, b in zip(got, want):
        assert torch.equal(a[[0, 1, 3]], b[[0, 1, 3]]) and torch.isnan(a[2].float()).all()


def test_repeats_are_bit_identical_and_empty_calls():
    rng = np.random.default_rng(3)
    x, h, w = bf16(rng, 300, 7168), bf16(rng, 300, 7168), bf16(rng, 7168)
    a = M.block_norm(x, h, w_post=w, w_pre=w)
    for _ in range(3):
        b = M.block_norm(x, h, w_post=w, w_pre=w)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    out, y = M.block_norm(x[:0], h[:0], w_post=w, w_pre=w)
    assert out.shape == (0, 7168) and y.shape == (0, 7168)


def test_refusals():
    rng = np.random.default_rng(4)
    x, h, w = bf16(rng, 4, 64), bf16(rng, 4, 64), bf16(rng, 64)
    with pytest.raises(TypeError):
        M.block_norm(x.float(), h, w_pre=w)
    with pytest.raises(TypeError):
        M.block_norm(x, h.half(), w_pre=w)
    with pytest.raises(ValueError):
        M.block_norm(x[:3], h, w_pre=w)
    with pytest.raises(ValueError):
        M.block_norm(x, h, w_pre=w[:32])
    with pytest.raises(ValueError):
        M.block_norm(x, h.cpu(), w_pre=w)
    with pytest.raises(ValueError):
        M.block_norm(x, h, y=torch.empty_like(x))

    def status(fn):
        with pytest.raises(M.MoeW4A16Error) as e:
            fn()
        return e.value.name

    assert status(lambda: M.block_norm(None, h)) == "ERR_INVALID_ARG"                 # nothing to do
    assert status(lambda: M.block_norm(None, h, w_post=w, w_pre=w)) == "ERR_INVALID_ARG"
    assert status(lambda: M.block_norm(x, h, w_pre=w, gate=bf16(rng, 3, 64))) == "ERR_INVALID_ARG"
    assert status(lambda: M.block_norm(x, h, w_pre=w, eps=-1.0)) == "ERR_INVALID_ARG"
    big = torch.zeros((1, 32769), dtype=torch.bfloat16, device=DEV)
    assert status(lambda: M.block_norm(big, big)) == "ERR_UNSUPPORTED"


@pytest.mark.parametrize("n", [1024, 1021, 509, 3, 8185, 12289])
@pytest.mark.parametrize("rows", [5, 701])
@pytest.mark.parametrize("where", ["w_post", "gate"])
def test_an_infinite_factor_of_an_edge_column(n, rows, where):
    """h' is infinite in that column alone, so its norm makes every other column of y zero: what lies past a row's ends
    takes no part, whatever the edge column's factor is."""
    rng = np.random.default_rng(n)
    x, h = bf16(rng, rows, n), bf16(rng, rows, n)
    f = {k: bf16(rng, n, scale=0.1, shift=1.0) for k in ("w_post", "gate", "w_pre")}
    for at in (0, n - 1):
        x[:, at] = 1.0
        plain, _ = M.block_norm(x, h, **f)
        bad = {k: v.clone() for k, v in f.items()}
        bad[where][at] = float("inf")
        got, y = M.block_norm(x, h, **bad)
        keep = [c for c in range(n) if c != at]
        assert torch.equal(got[:, keep], plain[:, keep]) and torch.isinf(got[:, at]).all()
        assert (y[:, keep] == 0).all() and torch.isnan(y[:, at]).all()
