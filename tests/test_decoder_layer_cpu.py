"""DecoderLayer's score scale, from the cache's shape or as the caller says (no GPU needed)."""

from types import SimpleNamespace

import pytest
import torch

import __graft_entry__

__graft_entry__.build()
from w4a16_int4_mixture_grouped_gb300.pipeline import DecoderLayer  # noqa: E402


def layer(latent, **kw):
    cache = SimpleNamespace(latent=latent, pool=torch.empty((1, 2, 16, 576) if latent else (2, 2, 16, 4, 128)))
    return DecoderLayer(cache, 0, None, 8, None, None, None, None, **kw)


def test_defaults():
    assert layer(False).scale == 128 ** -0.5
    assert layer(True).scale == 192 ** -0.5


@pytest.mark.parametrize("latent", [False, True])
@pytest.mark.parametrize("scale", [256 ** -0.5, 1.0, 0.0])
def test_the_callers_scale(latent, scale):
    assert layer(latent, scale=scale).scale == scale
