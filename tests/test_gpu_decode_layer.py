"""The decoder layer and the decode example: the operators together, as a serving loop runs them."""

import importlib.util
import os

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu

M = pytest.importorskip("w4a16_int4_mixture_grouped_gb300") if torch.cuda.is_available() else None


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decode_example", os.path.join(ROOT, "examples", "decode.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("latent,e4m3", [(False, False), (False, True), (True, False)])
def test_example(example, latent, e4m3, capsys):
    example.main(latent, e4m3, steps=37)
    assert "decode example ok" in capsys.readouterr().out


@pytest.mark.parametrize("latent", [False, True])
def test_layer_against_plain_attention_and_norms(example, latent):
    """One layer's steps with its attention and norms recomputed in 64 bits on the same projections."""
    batch, steps = 3, 20
    cache, stack, norms = example.build(batch, latent, False, seed=3, layers=1)
    layer = stack[0]
    ids = torch.arange(batch, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    rows = []
    for _ in range(steps):
        x = torch.randn((batch, example.HIDDEN), generator=g, device="cuda").to(torch.bfloat16)
        pos = cache.extend(ids)
        h, y = M.block_norm(None, x, w_pre=norms[0])
        assert h is x
        want = x.double() / torch.sqrt(x.double().square().mean(-1, keepdim=True) + 1e-6) * norms[0].double()
        assert ((y.double() - want).abs() <= want.abs() * 2.0 ** -7).all()
        q, k, v = layer.project(y, pos)
        rows.append((k.clone(), None if v is None else v.clone()))
        seen = []
        real = cache.attend
        cache.attend = lambda *a, **kw: seen.append(real(*a, **kw)) or seen[-1]
        try:
            layer.forward(h, y, ids, pos)
        finally:
            cache.attend = real
        keys = torch.stack([r[0] for r in rows], 1).double()                      # [B, L, (Hkv,) D]
        values = keys[..., :512] if latent else torch.stack([r[1] for r in rows], 1).double()
        if latent:
            keys, values = keys[:, :, None], values[:, :, None]
        group = example.HEADS // keys.shape[2]
        keys, values = keys.repeat_interleave(group, 2), values.repeat_interleave(group, 2)
        p = torch.softmax(torch.einsum("bhd,blhd->bhl", q.double(), keys) * layer.scale, -1)
        want = torch.einsum("bhl,blhd->bhd", p, values)
        bound = 2.0 ** -8 * 1.01 * want.abs() + (2.0 ** -8 + 2.0 ** -10) * torch.einsum("bhl,blhd->bhd", p, values.abs())
        assert ((seen[0].double() - want).abs() <= bound).all()
    cache.check()
