"""One workspace for calls of different shapes and kinds, one after the other on a stream."""

import numpy as np
import pytest
import torch

import oracle as O
from gpu_util import (assert_close, bits_to_dev, dev_to_bits, distinct_topk, i32_to_dev, prepare_dev, random_acts,
                      random_weights)

pytestmark = pytest.mark.gpu

M = pytest.importorskip("w4a16_int4_mixture_grouped_gb300") if torch.cuda.is_available() else None
DEV = torch.device("cuda", 0) if torch.cuda.is_available() else None


def test_gemm_calls_whose_regions_differ():
    """A combining call stages its routed rows where a plain call of a workspace of its own size has other things; both
    cut their last units into parts that a counter joins."""
    rng = np.random.default_rng(1900)
    e, kd, n, bm = 16, 256, 2048, 16
    qw, sc = random_weights(rng, e, n, kd)
    pw = prepare_dev(qw, sc, 1, DEV)
    flags = M.FLAG_COMBINE | M.FLAG_A_PER_ROW
    t1, k1 = 1000, 8
    ws = M.workspace(M.LAYOUT_INDEXED, t1, k1, e, n, kd, bm, flags, DEV)
    assert ws.numel() > M.workspace_size(M.LAYOUT_INDEXED, 24, 2, e, n, kd, bm, 0)
    ids1 = distinct_topk(rng, t1, e, k1)
    a1 = bits_to_dev(random_acts(rng, t1 * k1, kd), DEV)
    w1 = torch.from_numpy(rng.uniform(0, 1, size=(t1, k1)).astype(np.float32)).to(DEV)
    ids2 = distinct_topk(rng, 24, e, 2)
    a2 = random_acts(rng, 24, kd)
    want = O.indexed_gemm(a2, ids2, lambda x: (qw[x], sc[x]), n)
    first = None
    for _ in range(2):
        s_ids, e_ids, npp, _ = M.align(i32_to_dev(ids1, DEV), e, bm, ws)
        big = M.indexed(a1, pw, s_ids, e_ids, npp, t1, k1, bm, ws, flags=flags, topk_weights=w1)
        s_ids, e_ids, npp, _ = M.align(i32_to_dev(ids2, DEV), e, bm, ws)
        out = torch.full((48, n), float("nan"), dtype=torch.bfloat16, device=DEV)
        M.indexed(bits_to_dev(a2, DEV), pw, s_ids, e_ids, npp, 24, 2, bm, ws, out=out)
        assert M.get_device_error(ws) == 0
        assert_close(dev_to_bits(out), want, "a small call after a large one")
        first = big if first is None else first
        assert torch.equal(big, first)


def i32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def test_page_calls_and_attention_on_one_workspace():
    """Grouped attention joins its split rows by counters in the workspace; the page calls keep lists there, the latent
    form its parts."""
    g = torch.Generator(device=DEV).manual_seed(1)
    page, pages, seqs, width, heads, dim = 16, 2048, 128, 600, 8, 64
    pool = torch.randn((2, pages, page, 1, dim), generator=g, device=DEV).to(torch.bfloat16)
    latent = torch.randn((pages, page, 576), generator=g, device=DEV).to(torch.bfloat16)
    q = torch.randn((2, heads, dim), generator=g, device=DEV).to(torch.bfloat16)
    ql = torch.randn((2, heads, 576), generator=g, device=DEV).to(torch.bfloat16)
    long = torch.randperm(pages, generator=g, device=DEV).to(torch.int32)[:2 * width].view(2, width).contiguous()
    lens = i32([width * page, width * page - 37])

    def grouped(ws):
        return M.paged_attention(q, pool[0], pool[1], long, lens, ws)

    def one_latent(ws):
        return M.latent_attention(ql, latent, long, lens, ws, 0.05)

    def page_calls(ws):
        refs = torch.zeros(pages, dtype=torch.int32, device=DEV)
        tables = torch.full((2 * seqs, 8), -1, dtype=torch.int32, device=DEV)
        n = torch.zeros(2 * seqs, dtype=torch.int32, device=DEV)
        first, second = torch.arange(seqs, dtype=torch.int32, device=DEV), torch.arange(seqs, 2 * seqs, dtype=torch.int32, device=DEV)
        work = pool.clone()
        pos = M.cache_extend(refs, tables, n, first, page, ws, counts=torch.full_like(first, 70))
        M.cache_append(q[:1, :1], work[0], tables, first[:1], pos[:1], ws, v=q[1:, :1], v_pages=work[1])
        M.cache_fork(work, refs, tables, n, first, second, page, ws)
        M.cache_free(refs, tables, n, first[::3].contiguous(), page, ws)
        moved = M.cache_compact(work, refs, tables, ws)
        return (pos, work, refs, tables, n) + moved

    calls = [grouped, one_latent, page_calls]
    own = [M.attention_workspace(2, heads, 1, dim), M.attention_workspace(2, heads, 1, 576), M.cache_workspace(pages, seqs)]
    want = [call(ws) for call, ws in zip(calls, own)]
    assert [M.get_device_error(ws) for ws in own] == [0, 0, 0]
    ws = torch.zeros(max(x.numel() for x in own), dtype=torch.uint8, device=DEV)
    for order in ((2, 0, 1, 0), (1, 0, 2, 0), (2, 1, 2, 0, 0)):
        for i in order:
            for got, ref in zip(calls[i](ws), want[i]):
                assert torch.equal(got, ref)
    assert M.get_device_error(ws) == 0


@pytest.mark.parametrize("fill", [0x3F, 0xFF])
def test_counters_that_other_data_lies_on_are_recorded(fill):
    """A workspace that a call of another kind has used: reported, and right again once it is zeroed."""
    g = torch.Generator(device=DEV).manual_seed(2)
    k = torch.randn((200, 16, 1, 64), generator=g, device=DEV).to(torch.bfloat16)
    q = torch.randn((1, 8, 64), generator=g, device=DEV).to(torch.bfloat16)
    table, lens = torch.arange(200, dtype=torch.int32, device=DEV)[None], i32([3200])
    ws = M.attention_workspace(1, 8, 1, 64)
    want = M.paged_attention(q, k, k, table, lens, ws)
    ws[M.WS_HEADER_BYTES:] = fill
    M.paged_attention(q, k, k, table, lens, ws)
    assert M.get_device_error(ws) == 4
    M.workspace_init(ws)
    got = M.paged_attention(q, k, k, table, lens, ws)
    assert M.get_device_error(ws) == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])

    rng = np.random.default_rng(3)
    e, t, kd, n = 4, 16, 256, 512
    qw, sc = random_weights(rng, e, n, kd)
    pw, a = prepare_dev(qw, sc, 1, DEV), bits_to_dev(random_acts(rng, t, kd), DEV)
    ws = M.workspace(M.LAYOUT_INDEXED, t, 2, e, n, kd, 16, 0, DEV)
    s_ids, e_ids, npp, _ = M.align(i32_to_dev(distinct_topk(rng, t, e, 2), DEV), e, 16, ws)
    want = M.indexed(a, pw, s_ids, e_ids, npp, t, 2, 16, ws)
    assert M.get_device_error(ws) == 0
    ws[M.WS_HEADER_BYTES:] = fill
    M.indexed(a, pw, s_ids, e_ids, npp, t, 2, 16, ws)
    assert M.get_device_error(ws) == 4
    M.workspace_init(ws)
    assert torch.equal(M.indexed(a, pw, s_ids, e_ids, npp, t, 2, 16, ws), want) and M.get_device_error(ws) == 0
