"""Latent attention where the grouped form's tests do not reach: moving exponent bases over many tiles, long pools,
strides, scales, bad ids, batches past a block, other streams, graphs, and a wait that runs out."""

import math

import numpy as np
import pytest
import torch

from test_gpu_attention import compare, poison, queries, tables_for

pytestmark = pytest.mark.gpu

M = pytest.importorskip("w4a16_int4_mixture_grouped_gb300") if torch.cuda.is_available() else None
DEV = torch.device("cuda", 0) if torch.cuda.is_available() else None
TIMEOUT = 6   # MOE_W4A16_ERR_DEVICE_TIMEOUT


def reference(q, pages, tables, lens, scale, window=0, seq_ids=None):
    """(out, bound, lse, bound) in 64 bits, as block_ref.attention derives them, with products on the GPU."""
    page = pages.shape[1]
    b, h, _ = q.shape
    out, bound = np.zeros((b, h, 512)), np.zeros((b, h, 512))
    lse, lbound = np.full((b, h), -np.inf), np.zeros((b, h))
    for i in range(b):
        row = i if seq_ids is None else seq_ids[i]
        n = int(lens[row])
        at = np.arange(max(0, n - window) if window else 0, n)
        ids = tables[row][at // page]
        at, ids = at[ids >= 0], ids[ids >= 0]
        if not len(at):
            continue
        k = pages[torch.from_numpy(ids.astype(np.int64)).to(DEV), torch.from_numpy(at % page).to(DEV)].double()
        x = q[i].double()
        s = x @ k.T * scale
        e = (584 * 2.0 ** -24 * abs(scale) * (x.abs() @ k.abs().T)).amax(1)
        m = s.amax(1, keepdim=True)
        w = torch.exp(s - m)
        p = w / w.sum(1, keepdim=True)
        o, a = p @ k[:, :512], p @ k[:, :512].abs()
        out[i] = o.cpu().numpy()
        bound[i] = (2.0 ** -8 * 1.01 * o.abs() + (2.0 ** -8 + 2 * e[:, None] + 2.0 ** -18) * a + 2.0 ** -133).cpu().numpy()
        lse[i] = (m[:, 0] + torch.log(w.sum(1))).cpu().numpy()
        lbound[i] = e.cpu().numpy() + 2.0 ** -20 * (1 + np.abs(lse[i]))
    return out, bound, lse, lbound


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)


def normal(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DEV).to(torch.bfloat16)


@pytest.mark.parametrize("heads", [64, 24])
def test_scores_that_rise_and_fall_over_many_tiles(heads):
    """Heads' scores climb by up to 2^90 at different tokens, a little a tile, and come down again; a CTA takes about 13
    tiles of 64 tokens. Some rows begin with a tile of freed pages, or have a run of them further on."""
    rng = np.random.default_rng(51)
    page, n, batch, curves = 64, 8192, 16, 5
    tables, total = tables_for(rng, [n] * batch, page, width=n // page)
    tables[3, 0] = -1
    tables[4, :3] = -1
    tables[5, 20:31] = -1
    g = torch.Generator(device=DEV).manual_seed(3)
    axes = torch.linalg.qr(torch.randn((576, curves), generator=g, device=DEV))[0].T                  # orthonormal
    q = axes[torch.arange(heads, device=DEV) % curves].to(torch.bfloat16).expand(batch, heads, 576).contiguous()
    pages = torch.zeros((total, page, 576), dtype=torch.bfloat16, device=DEV)
    at = torch.arange(n, device=DEV, dtype=torch.float32)
    for b in range(batch):
        f = []
        for c in range(curves):
            top = n * (0.1 + 0.2 * ((b + c) % curves))                                                  # where it peaks
            f.append(62.0 * (1.0 - (at - top).abs() / n) ** (1 + c))
        rows = torch.stack(f, 1) @ axes + 0.02 * torch.randn((n, 576), generator=g, device=DEV)
        have = tables[b] >= 0
        ids = torch.from_numpy(tables[b][have].astype(np.int64)).to(DEV)
        pages[ids] = rows.view(n // page, page, 576)[torch.from_numpy(have).to(DEV)].to(torch.bfloat16)
    ws = M.attention_workspace(batch, heads, 1, 576)
    out, lse = M.latent_attention(q, pages, i32(tables), i32([n] * batch), ws, 1.0)
    assert M.get_device_error(ws) == 0
    compare(out, lse, *reference(q, pages, tables, [n] * batch, 1.0))


@pytest.mark.parametrize("scale", [-0.06, 0.0, 1e-4, 1.0])
def test_scales(scale):
    rng = np.random.default_rng(52)
    lens, page = [700, 1, 0, 64], 32
    tables, total = tables_for(rng, lens, page)
    pages, q = normal(rng, total, page, 576), queries(rng, 4, 24, 576)
    poison(pages, tables, lens, page)
    ws = M.attention_workspace(4, 24, 1, 576)
    out, lse = M.latent_attention(q, pages, i32(tables), i32(lens), ws, scale)
    assert M.get_device_error(ws) == 0
    compare(out, lse, *reference(q, pages, tables, lens, scale))


def test_offsets_past_32_bits():
    page = 64
    pages = (1 << 31) // (page * 576) + 8
    pool = torch.empty((pages, page, 576), dtype=torch.bfloat16, device=DEV)                          # 4.3 GB
    rng = np.random.default_rng(53)
    use = [pages - 1, 0, pages - 4]
    for p in use:
        pool[p] = normal(rng, page, 576)
    q, small = queries(rng, 1, 64, 576), pool[use].contiguous()
    ws = M.attention_workspace(1, 64, 1, 576)
    a = M.latent_attention(q, pool, i32([use]), i32([170]), ws, 0.05)
    b = M.latent_attention(q, small, i32([[0, 1, 2]]), i32([170]), ws, 0.05)
    assert M.get_device_error(ws) == 0
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    compare(*b, *reference(q, small, np.array([[0, 1, 2]]), [170], 0.05))


@pytest.mark.parametrize("batch", [513, 1100])
def test_batches_past_a_block_of_lengths(batch):
    rng = np.random.default_rng(batch)
    page = 16
    lens = [int(x) for x in rng.integers(0, 6, batch)]
    lens[-1] = 900
    lens[511] = 70
    tables, total = tables_for(rng, lens, page)
    pages, q = normal(rng, total, page, 576), queries(rng, batch, 8, 576)
    ws = M.attention_workspace(batch, 8, 1, 576)
    out, lse = M.latent_attention(q, pages, i32(tables), i32(lens), ws, 0.05)
    assert M.get_device_error(ws) == 0
    compare(out, lse, *reference(q, pages, tables, lens, 0.05))


def test_strided_pages_and_query_slices():
    rng = np.random.default_rng(54)
    page, lens = 24, [333, 20, 64]
    tables, total = tables_for(rng, lens, page)
    wide = normal(rng, total, 2 * page, 640)
    pages = wide[:, page:, 64:]                              # rows of 640 channels, every other half page
    q = queries(rng, 3, 40, 576)[:, 3:27]
    broad = np.full((3, tables.shape[1] + 5), 10 ** 6, dtype=np.int32)
    broad[:, :tables.shape[1]] = tables
    ws = M.attention_workspace(3, 24, 1, 576)
    out, lse = M.latent_attention(q, pages, i32(broad)[:, :tables.shape[1]], i32(lens), ws, 0.05)
    assert M.get_device_error(ws) == 0
    compare(out, lse, *reference(q, pages, tables, lens, 0.05))


def test_bad_ids_and_lengths_are_skipped_and_recorded():
    rng = np.random.default_rng(55)
    page, lens = 16, [90, 90, 40]
    tables, total = tables_for(rng, lens, page)
    pages, q = normal(rng, total, page, 576), queries(rng, 3, 8, 576)
    ws = M.attention_workspace(3, 8, 1, 576)

    def call(table, n, seq_ids=None):
        out = M.latent_attention(q, pages, i32(table), i32(n), ws, 0.05, seq_ids=None if seq_ids is None else i32(seq_ids))
        code = M.get_device_error(ws)
        M.clear_device_error(ws)
        return out, code

    bad = tables.copy()
    bad[1, 2] = total
    hole = tables.copy()
    hole[1, 2] = -1
    got, code = call(bad, lens)
    assert code == 8
    compare(*got, *reference(q, pages, hole, lens, 0.05))
    got, code = call(tables, [90, 90, -3])
    assert code == 8
    compare(*got, *reference(q, pages, tables, [90, 90, 0], 0.05))
    full, _ = tables_for(rng, [64, 64, 64], page, width=4, extra=0)
    got, code = call(full, [64, 5000, 7])
    assert code == 8
    compare(*got, *reference(q, pages, full, [64, 64, 7], 0.05))
    got, code = call(tables, lens, [2, 3, -1])
    assert code == 8
    assert (got[0][1:] == 0).all() and torch.isneginf(got[1][1:]).all()
    want = reference(q[:1], pages, tables, lens, 0.05, seq_ids=[2])
    compare(got[0][:1], got[1][:1], *want)


def test_another_stream_and_a_graph():
    rng = np.random.default_rng(56)
    page, lens = 64, [5000, 40]
    tables, total = tables_for(rng, lens, page)
    pages, q = normal(rng, total, page, 576), queries(rng, 2, 64, 576)
    ws = M.attention_workspace(2, 64, 1, 576)
    td, ld = i32(tables), i32(lens)
    want, wl = M.latent_attention(q, pages, td, ld, ws, 0.05)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, gl = M.latent_attention(q, pages, td, ld, ws, 0.05)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want) and torch.equal(gl, wl)
    out, lse = torch.zeros_like(want), torch.zeros_like(wl)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.latent_attention(q, pages, td, ld, ws, 0.05, out=out, lse=lse)
        M.latent_attention(q, pages, td, ld, ws, 0.05, out=out, lse=lse)      # the next call behind this one's join
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)
    ld.copy_(torch.tensor([20, 0], dtype=torch.int32))                        # a replay follows the lengths
    graph.replay()
    want, wl = M.latent_attention(q, pages, td, ld, ws, 0.05)
    assert torch.equal(out, want) and torch.equal(lse, wl)


@pytest.mark.parametrize("what", ["query", "key", "value"])
def test_a_number_that_is_none_stays_in_its_sequence(what):
    """A NaN query channel reaches its own head, a NaN row every head of its sequence; nothing reaches the others."""
    rng = np.random.default_rng(57)
    page, lens = 32, [300, 300, 100]
    tables, total = tables_for(rng, lens, page)
    pages, q = normal(rng, total, page, 576), queries(rng, 3, 24, 576)
    want = reference(q, pages, tables, lens, 0.05)
    hit = np.zeros((3, 24), dtype=bool)
    if what == "query":
        q[1, 7, 100] = math.nan
        hit[1, 7] = True
    else:
        pages[tables[1, 4], 9, 5 if what == "value" else 570] = math.nan
        hit[1] = True
    ws = M.attention_workspace(3, 24, 1, 576)
    out, lse = M.latent_attention(q, pages, i32(tables), i32(lens), ws, 0.05)
    keep = torch.from_numpy(~hit).to(DEV)
    assert torch.isnan(out[~keep]).all() and torch.isnan(lse[~keep]).all()
    compare(out[keep][:, None], lse[keep][:, None], *(x[~hit][:, None] for x in want))


@pytest.mark.parametrize("batch,top", [(1, 3000), (40, 900)])
def test_a_wait_that_runs_out_is_recorded_and_the_next_call_is_right(batch, top):
    """The limit lowered to zero: the first wait for a tile that is still on its way gives up (every copy and product does
    arrive, and is waited for before the kernel ends). Restored, the same workspace serves the next calls."""
    rng = np.random.default_rng(58)
    page = 64
    lens = [top] + [int(x) for x in rng.integers(1, top, batch - 1)]
    tables, total = tables_for(rng, lens, page)
    pages, q = normal(rng, total, page, 576), queries(rng, batch, 64, 576)
    ws = M.attention_workspace(batch, 64, 1, 576)
    td, ld = i32(tables), i32(lens)
    torch.cuda.synchronize()
    try:
        M.set_wait_limit_ns(0)
        M.latent_attention(q, pages, td, ld, ws, 0.05)
        code = M.get_device_error(ws)
    finally:
        M.set_wait_limit_ns(M.WAIT_LIMIT_NS)
    assert code == TIMEOUT, f"expected the timed-out wait to be recorded, got error word {code}"
    M.workspace_init(ws)
    for _ in range(2):
        out, lse = M.latent_attention(q, pages, td, ld, ws, 0.05)
        assert M.get_device_error(ws) == 0
        compare(out, lse, *reference(q, pages, tables, lens, 0.05))
