"""Decode steps of a small two-layer model on the paged cache: fill, fork, window, free, compact.

    python examples/decode.py [--latent] [--e4m3] [--steps N]

Random weights. Sequences are prefilled token by token, one of them is forked, the fork and its parent get the same
next token (their outputs must be equal bit for bit), a finished sequence is freed, the pool is compacted (the next
step must not change by it) and decoding goes on. Prints the pages in use at each stage.
"""

from __future__ import annotations

import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import w4a16_int4_mixture_grouped_gb300 as M  # noqa: E402
from w4a16_int4_mixture_grouped_gb300.cache import PagedCache  # noqa: E402
from w4a16_int4_mixture_grouped_gb300.pipeline import DecoderLayer, MoEFFN  # noqa: E402

HIDDEN, INTER, EXPERTS, TOP_K, HEADS, KV_HEADS, DIM, PAGE = 512, 256, 8, 2, 8, 2, 64, 16


def build(batch: int, latent: bool, e4m3: bool, seed: int = 0, layers: int = 2, pages: int = 64):
    """(cache, layers, first norm) with random weights for a batch of that size."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape, scale):
        return (torch.randn(shape, generator=g, device="cuda") * scale).to(torch.bfloat16)

    kind = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    scales = dict(k_scale=0.02, v_scale=0.02) if e4m3 else {}
    cache = PagedCache(layers, pages, PAGE, 4 * batch, 8, HEADS, *(() if latent else (KV_HEADS, DIM)),
                       dtype=torch.bfloat16 if latent else kind, **({} if latent else scales))
    rows = HEADS * M.LATENT_DIM + M.LATENT_DIM if latent else (HEADS + 2 * KV_HEADS) * DIM
    out_rows = HEADS * (M.LATENT_VALUE_DIM if latent else DIM)
    stack = []
    for i in range(layers):
        packed = [torch.randint(-2 ** 31, 2 ** 31 - 1, (EXPERTS, n, k // 8), generator=g, device="cuda", dtype=torch.int64)
                  .to(torch.int32) for n, k in ((2 * INTER, HIDDEN), (HIDDEN, INTER))]
        groups = [torch.full((EXPERTS, n, k // 32), 0.01, device="cuda").to(torch.bfloat16)
                  for n, k in ((2 * INTER, HIDDEN), (HIDDEN, INTER))]
        ffn = MoEFFN(M.prepare(packed[0], groups[0], mode=M.MODE_GATE_UP), M.prepare(packed[1], groups[1]), batch, TOP_K)
        norms = [rand(HIDDEN, scale=0.1) + 1 for _ in range(3)]
        stack.append(DecoderLayer(cache, i, ffn, HEADS, rand(HIDDEN, rows, scale=HIDDEN ** -0.5),
                                  rand(out_rows, HIDDEN, scale=out_rows ** -0.5), rand(HIDDEN, EXPERTS, scale=0.1),
                                  norm_ffn=norms[0], norm_post_attn=norms[1], norm_post_ffn=norms[2]))
    return cache, stack, [rand(HIDDEN, scale=0.1) + 1 for _ in range(layers)]


def step(cache, stack, norms, tokens: torch.Tensor, seq_ids: torch.Tensor) -> torch.Tensor:
    """One decode step of the sequences on embedded tokens [B, hidden] -> the last layer's residual stream."""
    positions = cache.extend(seq_ids)
    h, y = M.block_norm(None, tokens, w_pre=norms[0])
    for i, layer in enumerate(stack):
        h, y = layer.forward(h, y, seq_ids, positions, norms[i + 1] if i + 1 < len(stack) else None)
    return h


def main(latent: bool = False, e4m3: bool = False, steps: int = 40) -> None:
    batch = 4
    cache, stack, norms = build(batch, latent, e4m3)
    g = torch.Generator(device="cuda").manual_seed(1)

    def ids(*values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    def tokens():
        return torch.randn((batch, HIDDEN), generator=g, device="cuda").to(torch.bfloat16)

    def used():
        return int((cache.refs > 0).sum())

    seqs = ids(0, 1, 2, 3)
    for _ in range(steps):
        step(cache, stack, norms, tokens(), seqs)
    print(f"after {steps} steps: {used()} pages in use")
    cache.fork(ids(1), ids(5))
    print(f"sequence 1 forked: {used()} pages")
    x = tokens()
    x[3] = x[1]
    h = step(cache, stack, norms, x, ids(0, 1, 2, 5))
    if not torch.equal(h[1], h[3]):
        raise AssertionError("a fork does not continue like its parent")
    cache.free(ids(0, 3))
    print(f"sequences 0 and 3 freed: {used()} pages")
    x = tokens()
    cache.fork(ids(1, 2, 5), ids(6, 7, 8))
    cache.fork(ids(1), ids(9))
    before = step(cache, stack, norms, x, ids(1, 2, 5, 9))
    live = int(cache.compact())
    if used() != live or int((cache.refs[live:] > 0).sum()):
        raise AssertionError("the pool is not compact")
    after = step(cache, stack, norms, x, ids(6, 7, 8, 9))
    if not torch.equal(before[:3], after[:3]):
        raise AssertionError("a step after compaction differs")
    print(f"compacted: pages 0..{live - 1}")
    cache.check()
    for layer in stack:
        for ws in layer.ffn.workspaces:
            if M.get_device_error(ws):
                raise AssertionError("device error in the FFN")
    print("decode example ok")


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--latent", action="store_true", help="latent cache (one 576-channel row a token for all heads)")
    ap.add_argument("--e4m3", action="store_true", help="8-bit cache (grouped heads)")
    ap.add_argument("--steps", type=int, default=40)
    a = ap.parse_args()
    main(a.latent, a.e4m3, a.steps)
