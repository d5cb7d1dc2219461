"""Decode steps of a small two-layer model on the paged cache: fill, fork, window, free, compact.

    python examples/decode.py [--latent] [--e4m3] [--steps N] [--prompt N]

Random weights. With --prompt the sequences' first N tokens go in as one chunk (two, if the prompt is longer than 8),
queries and keys turned by their positions (--latent: token by token). Sequences are filled token by token, one of them
is forked, the fork and its parent get the same next token (their outputs must be equal bit for bit), a finished
sequence is freed, the pool is compacted (the next step must not change by it) and decoding goes on. Prints the pages
in use at each stage.
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


def build(batch: int, latent: bool, e4m3: bool, seed: int = 0, layers: int = 2, pages: int = 64, rotary=None, chunks=()):
    """(cache, layers, first norm) with random weights for a batch of that size. For each of `chunks`, a number of rows,
    cache.stacks holds the same layers over that many."""
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
    cache.stacks = {rows: [] for rows in chunks}
    for i in range(layers):
        packed = [torch.randint(-2 ** 31, 2 ** 31 - 1, (EXPERTS, n, k // 8), generator=g, device="cuda", dtype=torch.int64)
                  .to(torch.int32) for n, k in ((2 * INTER, HIDDEN), (HIDDEN, INTER))]
        groups = [torch.full((EXPERTS, n, k // 32), 0.01, device="cuda").to(torch.bfloat16)
                  for n, k in ((2 * INTER, HIDDEN), (HIDDEN, INTER))]
        prepared = M.prepare(packed[0], groups[0], mode=M.MODE_GATE_UP), M.prepare(packed[1], groups[1])
        norms = [rand(HIDDEN, scale=0.1) + 1 for _ in range(3)]
        weights = (rand(HIDDEN, rows, scale=HIDDEN ** -0.5), rand(out_rows, HIDDEN, scale=out_rows ** -0.5),
                   rand(HIDDEN, EXPERTS, scale=0.1))
        for n, layers_of in [(batch, stack)] + list(cache.stacks.items()):
            layers_of.append(DecoderLayer(cache, i, MoEFFN(*prepared, n, TOP_K), HEADS, *weights, norm_ffn=norms[0],
                                          norm_post_attn=norms[1], norm_post_ffn=norms[2], rotary=rotary))
    return cache, stack, [rand(HIDDEN, scale=0.1) + 1 for _ in range(layers)]


def step(cache, stack, norms, tokens: torch.Tensor, seq_ids: torch.Tensor) -> torch.Tensor:
    """One decode step of the sequences on embedded tokens [B, hidden] -> the last layer's residual stream."""
    positions = cache.extend(seq_ids)
    h, y = M.block_norm(None, tokens, w_pre=norms[0])
    for i, layer in enumerate(stack):
        h, y = layer.forward(h, y, seq_ids, positions, norms[i + 1] if i + 1 < len(stack) else None)
    return h


def prefill(cache, norms, tokens: torch.Tensor, starts: torch.Tensor, seq_ids: torch.Tensor) -> torch.Tensor:
    """One chunk of embedded tokens [T, hidden], starts[b] .. starts[b + 1] - 1 of them sequence seq_ids[b]'s next."""
    rows, positions = cache.extend_chunk(seq_ids, starts, tokens.shape[0])
    stack = cache.stacks[tokens.shape[0]]
    h, y = M.block_norm(None, tokens, w_pre=norms[0])
    for i, layer in enumerate(stack):
        h, y = layer.forward(h, y, rows, positions, norms[i + 1] if i + 1 < len(stack) else None, chunk=(starts, seq_ids))
    return h


def main(latent: bool = False, e4m3: bool = False, steps: int = 40, prompt: int = 0) -> None:
    batch = 4
    pieces = [] if latent or prompt == 0 else [prompt] if prompt <= 8 else [prompt - 8, 8]
    rotary = None
    if prompt:
        rotary = M.Rotary(64, offset=512, interleaved=True) if latent else M.Rotary(DIM)
    cache, stack, norms = build(batch, latent, e4m3, rotary=rotary, chunks=sorted({batch * n for n in pieces}))
    g = torch.Generator(device="cuda").manual_seed(1)

    def ids(*values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    def tokens():
        return torch.randn((batch, HIDDEN), generator=g, device="cuda").to(torch.bfloat16)

    def used():
        return int((cache.refs > 0).sum())

    seqs = ids(0, 1, 2, 3)
    for n in pieces:
        chunk = torch.randn((batch * n, HIDDEN), generator=g, device="cuda").to(torch.bfloat16)
        h = prefill(cache, norms, chunk, ids(*range(0, batch * n + 1, n)), seqs)
        if not torch.isfinite(h).all():
            raise AssertionError("the prompt's outputs are not finite")
        print(f"prompt's chunk of {n} tokens a sequence: {used()} pages in use")
    for _ in range(steps + (prompt if latent else 0)):
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
    for layer in stack + [x for layers in cache.stacks.values() for x in layers]:
        for ws in layer.ffn.workspaces:
            if M.get_device_error(ws):
                raise AssertionError("device error in the FFN")
    print("decode example ok")


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--latent", action="store_true", help="latent cache (one 576-channel row a token for all heads)")
    ap.add_argument("--e4m3", action="store_true", help="8-bit cache (grouped heads)")
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--prompt", type=int, default=0, help="tokens of each sequence that go in as a prompt, with positions turned")
    a = ap.parse_args()
    main(a.latent, a.e4m3, a.steps, a.prompt)
