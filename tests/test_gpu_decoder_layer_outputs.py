"""What DecoderLayer.forward returns, stage by stage in 64 bits from the tensors that pass between its stages."""

import numpy as np
import pytest
import torch

import block_ref as R
import oracle as O
from gpu_util import assert_close, combine_slack, dev_to_bits, prepare_dev, random_weights

pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    M = pytest.importorskip("w4a16_int4_mixture_grouped_gb300")
    from w4a16_int4_mixture_grouped_gb300 import pipeline
    from w4a16_int4_mixture_grouped_gb300.cache import PagedCache
    DEV = torch.device("cuda", 0)

HIDDEN, INTER, EXPERTS, TOP_K, HEADS, KV_HEADS, DIM, PAGE = 512, 256, 8, 2, 8, 2, 64, 16


def f64(t):
    return t.detach().to(torch.float64).cpu().numpy()


def product(a, w):
    """A BF16 product with FP32 sums: its value and bound."""
    a, w = f64(a), f64(w)
    ref = a @ w
    return ref, 2.0 ** -8 * 1.01 * np.abs(ref) + (a.shape[1] + 8) * 2.0 ** -24 * (np.abs(a) @ np.abs(w))


def inside(got, ref, bound, what):
    d = np.abs(f64(got) - ref)
    assert (d <= bound).all(), f"{what}: {(d / np.maximum(bound, 1e-300)).max()} of the bound"


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "latent"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("res32", [False, True])
def test_forward(kind, post, res32, monkeypatch):
    rng = np.random.default_rng(71)
    g = torch.Generator(device="cuda").manual_seed(9)

    def rand(*shape, scale=1.0, shift=0.0):
        return (torch.randn(shape, generator=g, device="cuda") * scale + shift).to(torch.bfloat16)

    batch, latent = 3, kind == "latent"
    cache = PagedCache(1, 32, PAGE, batch, 8, HEADS, *(() if latent else (KV_HEADS, DIM)),
                       dtype=torch.float8_e4m3fn if kind == "e4m3" else torch.bfloat16,
                       **(dict(k_scale=0.02, v_scale=0.02) if kind == "e4m3" else {}))
    (q1, s1), (q2, s2) = random_weights(rng, EXPERTS, 2 * INTER, HIDDEN), random_weights(rng, EXPERTS, HIDDEN, INTER)
    ffn = pipeline.MoEFFN(prepare_dev(q1, s1, M.MODE_GATE_UP, DEV), prepare_dev(q2, s2, M.MODE_PLAIN, DEV), batch, TOP_K)
    rows = (HEADS + 1) * 576 if latent else (HEADS + 2 * KV_HEADS) * DIM
    wide = HEADS * (512 if latent else DIM)
    # four norms that cannot be taken for one another
    after, before, last, following = (rand(HIDDEN, scale=0.2, shift=s) for s in (1.0, 2.0, 0.5, -1.5))
    layer = pipeline.DecoderLayer(cache, 0, ffn, HEADS, rand(HIDDEN, rows, scale=HIDDEN ** -0.5),
                                  rand(wide, HIDDEN, scale=wide ** -0.5), rand(HIDDEN, EXPERTS, scale=0.1), before,
                                  norm_post_attn=after if post else None, norm_post_ffn=last if post else None, eps=1e-5)
    seen = {"norm": [], "attend": [], "ffn": []}

    def record(name, fn):
        def call(*args, **kw):
            got = fn(*args, **kw)
            keep = got if isinstance(got, tuple) else (got,)
            seen[name].append((args, kw, tuple(x.clone() if x is not None else None for x in keep)))
            return got
        return call

    monkeypatch.setattr(pipeline, "block_norm", record("norm", pipeline.block_norm))
    monkeypatch.setattr(cache, "attend", record("attend", cache.attend))
    monkeypatch.setattr(ffn, "forward", record("ffn", ffn.forward))
    ids = torch.arange(batch, dtype=torch.int32, device="cuda")
    for step in range(20):
        for calls in seen.values():
            calls.clear()
        residual = rand(batch, HIDDEN).float() if res32 else rand(batch, HIDDEN)
        start = f64(residual)
        y0 = rand(batch, HIDDEN)
        nxt = following if step % 2 == 0 else None
        h, y = layer.forward(residual, y0, ids, cache.extend(ids), nxt)
        cache.check()
        (_, _, (o,)), = seen["attend"]
        (to_norm, _, (h1, y1)), (to_norm2, _, (h2, y2)) = seen["norm"]
        (to_ffn, _, (f,)), = seen["ffn"]
        # output projection
        a = to_norm[0]
        inside(a, *product(o.reshape(batch, wide), layer.w_o), "output projection")
        # norm after attention, the residual, norm before the FFN
        ref_h, hb, ref_y, yb = R.block_norm(f64(a), start, f64(after) if post else None, f64(before), None, 1e-5, 1.0, 1.0, res32)
        inside(h1, ref_h, hb, "residual after attention")
        inside(y1, ref_y, yb, "input of the FFN")
        # router: the experts of the highest logits (within the logits' rounding), softmax over all, renormalised
        assert torch.equal(to_ffn[0], y1)
        logits, lb = product(y1, layer.w_router)
        top, weights = to_ffn[1].cpu().numpy(), f64(to_ffn[2])
        for r in range(batch):
            chosen = set(top[r].tolist())
            assert len(chosen) == TOP_K
            others = [e for e in range(EXPERTS) if e not in chosen]
            assert min(logits[r, e] + lb[r, e] for e in chosen) >= max(logits[r, e] - lb[r, e] for e in others)
            w = np.exp(logits[r, top[r]] - logits[r].max())
            off = np.expm1(2 * lb[r].max()) + 2.0 ** -20
            assert (np.abs(weights[r] - w / w.sum()) <= off * w / w.sum()).all()
        # FFN from the packed weights
        ref = O.ffn(dev_to_bits(y1), top.astype(np.int32), weights.astype(np.float32), lambda x: (q1[x], s1[x]),
                    lambda x: (q2[x], s2[x]), 2 * INTER, HIDDEN)
        assert_close(dev_to_bits(f), ref["out"], "FFN", slack=combine_slack(ref["y2"], weights))
        # norm after the FFN, the residual, the next layer's norm
        assert torch.equal(to_norm2[0], f)
        ref_h, hb, ref_y, yb = R.block_norm(f64(f), f64(h1), f64(last) if post else None,
                                            None if nxt is None else f64(nxt), None, 1e-5, 1.0, 1.0, res32)
        assert torch.equal(h, h2) and h.dtype == residual.dtype
        inside(h, ref_h, hb, "residual after the FFN")
        if nxt is None:
            assert y is None
        else:
            inside(y, ref_y, yb, "input of the next layer")
        assert np.array_equal(f64(residual), start)
        for ws in ffn.workspaces:
            assert M.get_device_error(ws) == 0
