"""Binding of the paged cache, the attention that reads it and the block norms.

The half of a decoder layer's decode step beside the MoE FFN. As in the package
itself: argument marshalling only, names as in include/moe_w4a16.h without the
``moe_w4a16_`` prefix, MoeW4A16Error on a non-OK status. A call runs on the
current stream of its tensors' device; the page calls record what they find
wrong on the device (ids out of range, no free page) in the workspace, to be
read with get_device_error.

A cache's pages are tensors [num_pages, page_size, heads, dim] (latent:
[num_pages, page_size, 576]) of torch.bfloat16 or torch.float8_e4m3fn whose
last dimension is dense; tables int32 [num_seqs, max_pages] hold each sequence's
pages in order, -1 where there is none, lens int32 [num_seqs] the token counts,
refs int32 [num_pages] how many tables hold a page.
"""

from __future__ import annotations

import ctypes
import struct
from typing import Optional, Tuple

import torch

from . import MoeW4A16Error, WS_HEADER_BYTES, lib, workspace_init

CACHE_BF16, CACHE_E4M3 = 0, 1
RESIDUAL_BF16, RESIDUAL_F32 = 0, 1
LATENT_DIM, LATENT_VALUE_DIM = 576, 512
MAX_HEAD_DIM, MAX_PAGE_SIZE, MAX_NORM_WIDTH = 256, 4096, 32768

_CACHE_DTYPES = {torch.bfloat16: CACHE_BF16, torch.float8_e4m3fn: CACHE_E4M3}
_RESIDUALS = {torch.bfloat16: RESIDUAL_BF16, torch.float32: RESIDUAL_F32}
_BF16 = torch.bfloat16
_I32 = torch.int32


class Pages(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("reserved", ctypes.c_int32),
                ("page_stride", ctypes.c_int64), ("token_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64),
                ("k_scale", ctypes.c_float), ("v_scale", ctypes.c_float)]


class Pool(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("num_planes", ctypes.c_int32), ("num_pages", ctypes.c_int32),
                ("plane_stride", ctypes.c_int64), ("page_stride", ctypes.c_int64), ("page_bytes", ctypes.c_int64)]


_P, _I, _L, _F, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
# The structures of a call go over as their bytes (packing them is half as long as filling a ctypes structure).
_PAGES = _POOL = ctypes.c_void_p
_pack_pages = struct.Struct("@PPiiiiqqqff").pack
_pack_pool = struct.Struct("@Piiqqq").pack
assert struct.calcsize("@PPiiiiqqqff") == ctypes.sizeof(Pages) and struct.calcsize("@Piiqqq") == ctypes.sizeof(Pool)
_SIGNATURES = {
    "attention_workspace_size": [_I, _I, _I, ctypes.POINTER(_SZ)],
    "paged_attention": [_P, _L, _I, _I, _I, _I, _PAGES, _P, _L, _I, _P, _P, _I, _F, _I, _P, _P, _P, _SZ, _P],
    "latent_attention": [_P, _L, _I, _I, _PAGES, _P, _L, _I, _P, _P, _I, _F, _I, _P, _P, _P, _SZ, _P],
    "cache_append": [_P, _L, _P, _L, _I, _I, _I, _PAGES, _P, _L, _I, _I, _P, _P, _P, _SZ, _P],
    "cache_workspace_size": [_I, _I, ctypes.POINTER(_SZ)],
    "cache_extend": [_P, _I, _P, _L, _I, _P, _I, _P, _P, _I, _I, _P, _P, _SZ, _P],
    "cache_fork": [_POOL, _P, _P, _L, _I, _P, _I, _P, _P, _I, _I, _P, _SZ, _P],
    "cache_free": [_P, _I, _P, _L, _I, _P, _I, _P, _P, _I, _I, _P, _SZ, _P],
    "cache_copy": [_POOL, _P, _P, _I, _P, _SZ, _P],
    "cache_compact": [_POOL, _P, _P, _L, _I, _I, _P, _P, _P, _P, _P, _SZ, _P],
    "block_norm": [_P, _L, _P, _L, _I, _P, _I, _P, _P, _I, _I, _F, _F, _F, _P, _L, _P, _L, _P],
}
_FN = {}
for _name, _args in _SIGNATURES.items():
    _fn = getattr(lib, "moe_w4a16_" + _name)
    _fn.restype = ctypes.c_int
    _fn.argtypes = _args
    _FN[_name] = _fn


# The current stream's handle without a Stream object around it: a tenth of a decode call's host time otherwise.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _run(name: str, index: int, fn, *args) -> None:
    """The C entry point on the current stream of device `index` (made current for the launch where it is not)."""
    if _current_device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        raise MoeW4A16Error(status, name)


def _need(t: torch.Tensor, name: str, dtype, dim: int, index: Optional[int] = None) -> torch.Tensor:
    """A tensor of that type and rank on CUDA device `index` (None: any) whose last dimension is dense."""
    if (type(t) is torch.Tensor and t.dtype is dtype and t.dim() == dim and t.get_device() == index
            and (t.is_contiguous() or t.stride(-1) == 1)):
        return t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    where = t.get_device()
    if where < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if index is not None and where != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")
    if dtype is not None and t.dtype is not dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.dim() != dim:
        raise ValueError(f"{name} must have {dim} dimensions, not {t.dim()}")
    if t.stride(-1) != 1 and t.size(-1) > 1:
        raise ValueError(f"{name}: the last dimension must be dense")
    return t


def _vector(t: torch.Tensor, name: str, n: int, index: int, dtype=_I32) -> int:
    """Address of a dense 1-D tensor of n elements."""
    if _need(t, name, dtype, 1, index).size(0) != n:
        raise ValueError(f"{name} has {t.size(0)} elements, expected {n}")
    return t.data_ptr()


def _rows_dense(t: torch.Tensor, name: str) -> torch.Tensor:
    """The trailing two dimensions [heads, dim] lie dense behind each other."""
    if t.dim() == 3 and t.size(1) > 1 and t.stride(1) != t.size(2):
        raise ValueError(f"{name}: heads must be dense")
    return t


def _table(tables: torch.Tensor, index: int) -> Tuple[int, int, int, int]:
    """(address, row stride, max_pages, num_seqs)."""
    _need(tables, "tables", _I32, 2, index)
    s, m = tables.shape
    return tables.data_ptr(), (tables.stride(0) if s > 1 else m), m, s


def _pages(k: torch.Tensor, v: Optional[torch.Tensor], index: int, k_scale: float, v_scale: float) -> bytes:
    """A moe_w4a16_pages of k and v (None: a latent cache)."""
    dtype = k.dtype if isinstance(k, torch.Tensor) else None
    _need(k, "k_pages", dtype, 4 if v is not None else 3, index)
    kind = _CACHE_DTYPES.get(dtype)
    if kind is None:
        raise TypeError(f"pages have dtype {dtype}, expected torch.bfloat16 or torch.float8_e4m3fn")
    shape, st = k.shape, k.stride()
    if v is None:
        return _pack_pages(k.data_ptr(), 0, kind, shape[0], shape[1], 0, st[0], st[1], shape[2], k_scale, v_scale)
    _need(v, "v_pages", dtype, 4, index)
    if v.shape != shape or v.stride() != st:
        raise ValueError("k_pages and v_pages must have the same shape and strides")
    return _pack_pages(k.data_ptr(), v.data_ptr(), kind, shape[0], shape[1], 0, st[0], st[1], st[2], k_scale, v_scale)


def _pool(pool: torch.Tensor) -> Tuple[bytes, int]:
    """(moe_w4a16_pool, num_pages) of pool [planes, num_pages, ...], each page dense."""
    if not isinstance(pool, torch.Tensor) or not pool.is_cuda:
        raise ValueError("pool must be a CUDA tensor")
    shape, st = pool.shape, pool.stride()
    if len(shape) < 3:
        raise ValueError("pool must be [planes, num_pages, ...]")
    dense = 1
    for n, s in zip(reversed(shape[2:]), reversed(st[2:])):
        if n > 1 and s != dense:
            raise ValueError("pool: each page must be dense")
        dense *= n
    size = pool.element_size()
    return _pack_pool(pool.data_ptr(), shape[0], shape[1], st[0] * size, st[1] * size, dense * size), shape[1]


def _ws(ws: torch.Tensor, index: int) -> Tuple[int, int]:
    _need(ws, "ws", torch.uint8, 1, index)
    return ws.data_ptr(), ws.size(0)


def _alloc_ws(nbytes: int, device) -> torch.Tensor:
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    ws = torch.empty(max(nbytes, WS_HEADER_BYTES), dtype=torch.uint8, device=dev)
    workspace_init(ws)
    return ws


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

def attention_workspace_size(num_heads: int, num_kv_heads: int, head_dim: int) -> int:
    out = _SZ(0)
    status = _FN["attention_workspace_size"](num_heads, num_kv_heads, head_dim, ctypes.byref(out))
    if status != 0:
        raise MoeW4A16Error(status, "attention_workspace_size")
    return int(out.value)


def attention_workspace(batch: int, num_heads: int, num_kv_heads: int, head_dim: int, device=None) -> torch.Tensor:
    """Allocates (through torch) and zeroes a workspace for either attention call (latent: one head of 576). It
    does not depend on the lengths, and one made for a batch serves any other."""
    del batch
    return _alloc_ws(attention_workspace_size(num_heads, num_kv_heads, head_dim), device)


def _attention_out(q, b, h, width, index, out, lse):
    if out is None:
        out = torch.empty((b, h, width), dtype=_BF16, device=q.device)
    else:
        _need(out, "out", _BF16, 3, index)
        if out.shape != (b, h, width) or not out.is_contiguous():
            raise ValueError(f"out must be contiguous [{b}, {h}, {width}]")
    if lse is None:
        lse = torch.empty((b, h), dtype=torch.float32, device=q.device)
    else:
        _need(lse, "lse", torch.float32, 2, index)
        if lse.shape != (b, h) or not lse.is_contiguous():
            raise ValueError(f"lse must be contiguous [{b}, {h}]")
    return out, lse


def paged_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, tables: torch.Tensor,
                    lens: torch.Tensor, ws: torch.Tensor, scale: Optional[float] = None, window: int = 0,
                    k_scale: float = 1.0, v_scale: float = 1.0, seq_ids: Optional[torch.Tensor] = None,
                    out: Optional[torch.Tensor] = None,
                    lse: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """One new token per sequence over its pages: q [B, H, D] -> (out bf16 [B, H, D], lse float [B, H]).

    scale defaults to D ** -0.5; window counts the newest tokens seen (0: all); seq_ids [B] names the row of
    tables and lens of each query (default: row b)."""
    _rows_dense(_need(q, "q", _BF16, 3), "q")
    index = q.get_device()
    b, h, d = q.shape
    if v_pages is None:
        raise ValueError("v_pages is missing (a latent cache: latent_attention)")
    c = _pages(k_pages, v_pages, index, k_scale, v_scale)
    heads, dim = k_pages.shape[2:]
    if dim != d:
        raise ValueError(f"pages must hold keys and values of {d} channels")
    ta, ts, mp, ns = _table(tables, index)
    out, lse = _attention_out(q, b, h, d, index, out, lse)
    wa, wn = _ws(ws, index)
    _run("paged_attention", index, _FN["paged_attention"], q.data_ptr(), q.stride(0) if b > 1 else h * d, b, h, heads, d, c, ta, ts, mp,
          _vector(lens, "lens", ns, index), None if seq_ids is None else _vector(seq_ids, "seq_ids", b, index), ns,
          d ** -0.5 if scale is None else scale, window, out.data_ptr(), lse.data_ptr(), wa, wn)
    return out, lse


def latent_attention(q: torch.Tensor, pages: torch.Tensor, tables: torch.Tensor, lens: torch.Tensor, ws: torch.Tensor,
                     scale: float, window: int = 0, seq_ids: Optional[torch.Tensor] = None,
                     out: Optional[torch.Tensor] = None,
                     lse: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The same over a latent cache: q [B, H, 576], pages [P, S, 576] -> (out bf16 [B, H, 512], lse [B, H])."""
    _rows_dense(_need(q, "q", _BF16, 3), "q")
    index = q.get_device()
    b, h, d = q.shape
    c = _pages(pages, None, index, 1.0, 1.0)
    if d != LATENT_DIM or pages.size(2) != LATENT_DIM:
        raise ValueError(f"q and pages must have {LATENT_DIM} channels")
    ta, ts, mp, ns = _table(tables, index)
    out, lse = _attention_out(q, b, h, LATENT_VALUE_DIM, index, out, lse)
    wa, wn = _ws(ws, index)
    _run("latent_attention", index, _FN["latent_attention"], q.data_ptr(), q.stride(0) if b > 1 else h * d, b, h, c, ta, ts, mp,
          _vector(lens, "lens", ns, index), None if seq_ids is None else _vector(seq_ids, "seq_ids", b, index), ns, scale, window, out.data_ptr(),
          lse.data_ptr(), wa, wn)
    return out, lse


# ---------------------------------------------------------------------------
# cache
# ---------------------------------------------------------------------------

def cache_append(k: torch.Tensor, k_pages: torch.Tensor, tables: torch.Tensor, seq_ids: torch.Tensor,
                 positions: torch.Tensor, ws: torch.Tensor, v: Optional[torch.Tensor] = None,
                 v_pages: Optional[torch.Tensor] = None, k_scale: float = 1.0, v_scale: float = 1.0) -> None:
    """Writes rows k, v [T, heads, dim] (latent: k [T, 576] alone) to token positions[i] of sequence seq_ids[i]."""
    latent = v_pages is None
    if (v is None) != latent:
        raise ValueError("v and v_pages go together")
    _rows_dense(_need(k, "k", _BF16, 2 if latent else 3), "k")
    index = k.get_device()
    c = _pages(k_pages, v_pages, index, k_scale, v_scale)
    if tuple(k_pages.shape[2:]) != tuple(k.shape[1:]):
        raise ValueError(f"rows are {tuple(k.shape[1:])}, pages hold {tuple(k_pages.shape[2:])}")
    n = k.shape[0]
    heads, dim = (1, k.shape[1]) if latent else k.shape[1:]
    if not latent:
        _rows_dense(_need(v, "v", _BF16, 3, index), "v")
        if v.shape != k.shape:
            raise ValueError("k and v must have the same shape")
    ta, ts, mp, ns = _table(tables, index)
    wa, wn = _ws(ws, index)
    _run("cache_append", index, _FN["cache_append"], k.data_ptr(), k.stride(0) if n > 1 else heads * dim,
          None if latent else v.data_ptr(), 0 if latent else (v.stride(0) if n > 1 else heads * dim), n, heads, dim,
          c, ta, ts, mp, ns, _vector(seq_ids, "seq_ids", n, index),
          _vector(positions, "positions", n, index), wa, wn)


def cache_workspace_size(num_pages: int, count: int) -> int:
    out = _SZ(0)
    status = _FN["cache_workspace_size"](num_pages, count, ctypes.byref(out))
    if status != 0:
        raise MoeW4A16Error(status, "cache_workspace_size")
    return int(out.value)


def cache_workspace(num_pages: int, count: int, device=None) -> torch.Tensor:
    """Allocates (through torch) and zeroes a workspace for page calls of up to `count` entries on a pool of
    num_pages pages; it also serves cache_append and cache_copy."""
    return _alloc_ws(cache_workspace_size(num_pages, count), device)


def cache_extend(refs: torch.Tensor, tables: torch.Tensor, lens: torch.Tensor, seq_ids: torch.Tensor, page_size: int,
                 ws: torch.Tensor, counts: Optional[torch.Tensor] = None,
                 out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Grows the sequences by counts tokens (default one each), taking free pages; -> positions [n], each
    sequence's old length, -1 where it did not fit."""
    _need(refs, "refs", _I32, 1)
    index = refs.get_device()
    n = seq_ids.size(0)
    ta, ts, mp, ns = _table(tables, index)
    if out is None:
        out = torch.empty(n, dtype=_I32, device=refs.device)
    wa, wn = _ws(ws, index)
    _run("cache_extend", index, _FN["cache_extend"], refs.data_ptr(), refs.size(0), ta, ts, mp, _vector(lens, "lens", ns, index), ns,
          _vector(seq_ids, "seq_ids", n, index), None if counts is None else _vector(counts, "counts", n, index), n, page_size,
          _vector(out, "out", n, index), wa, wn)
    return out


def cache_fork(pool: torch.Tensor, refs: torch.Tensor, tables: torch.Tensor, lens: torch.Tensor, parents: torch.Tensor,
               children: torch.Tensor, page_size: int, ws: torch.Tensor) -> None:
    """Makes each (empty) children[i] a copy of parents[i]: full pages shared, a partly filled last page of pool
    [planes, num_pages, ...] copied in every plane."""
    p, pages = _pool(pool)
    index = pool.get_device()
    n = parents.size(0)
    ta, ts, mp, ns = _table(tables, index)
    wa, wn = _ws(ws, index)
    _run("cache_fork", index, _FN["cache_fork"], p, _vector(refs, "refs", pages, index), ta, ts, mp,
          _vector(lens, "lens", ns, index), ns, _vector(parents, "parents", n, index),
          _vector(children, "children", n, index), n, page_size, wa, wn)


def cache_free(refs: torch.Tensor, tables: torch.Tensor, lens: torch.Tensor, seq_ids: torch.Tensor, page_size: int,
               ws: torch.Tensor, keep: Optional[torch.Tensor] = None) -> None:
    """Frees the sequences' pages; with keep [n], only those wholly before the newest keep[i] tokens."""
    _need(refs, "refs", _I32, 1)
    index = refs.get_device()
    n = seq_ids.size(0)
    ta, ts, mp, ns = _table(tables, index)
    wa, wn = _ws(ws, index)
    _run("cache_free", index, _FN["cache_free"], refs.data_ptr(), refs.size(0), ta, ts, mp, _vector(lens, "lens", ns, index), ns,
          _vector(seq_ids, "seq_ids", n, index), None if keep is None else _vector(keep, "keep", n, index), n, page_size, wa, wn)


def cache_copy(pool: torch.Tensor, src: torch.Tensor, dst: torch.Tensor, ws: torch.Tensor) -> None:
    """pool[:, dst[i]] = pool[:, src[i]]; no destination is a source or another destination."""
    p, _ = _pool(pool)
    index = pool.get_device()
    n = src.size(0)
    wa, wn = _ws(ws, index)
    _run("cache_copy", index, _FN["cache_copy"], p, _vector(src, "src", n, index), _vector(dst, "dst", n, index), n, wa, wn)


def cache_compact(pool: torch.Tensor, refs: torch.Tensor, tables: torch.Tensor, ws: torch.Tensor,
                  refs_out: Optional[torch.Tensor] = None, tables_out: Optional[torch.Tensor] = None):
    """Moves the pages in use to the front of the pool -> (refs, tables, page_map [num_pages], num_live [1]).

    The new counts and tables are new tensors unless refs_out / tables_out (which may be refs / tables) are given."""
    p, pages = _pool(pool)
    index = pool.get_device()
    ra = _vector(refs, "refs", pages, index)
    ta, ts, mp, ns = _table(tables, index)
    if refs_out is None:
        refs_out = torch.empty(pages, dtype=_I32, device=refs.device)
    if tables_out is None:
        tables_out = torch.empty_strided(tables.shape, (ts, 1), dtype=_I32, device=refs.device)
    to, tos, _, _ = _table(tables_out, index)
    if tables_out.shape != tables.shape or tos != ts:
        raise ValueError("tables_out must have the shape and strides of tables")
    page_map = torch.empty(pages, dtype=_I32, device=refs.device)
    num_live = torch.empty(1, dtype=_I32, device=refs.device)
    wa, wn = _ws(ws, index)
    _run("cache_compact", index, _FN["cache_compact"], p, ra, ta, ts, mp, ns, _vector(refs_out, "refs_out", pages, index),
          to, page_map.data_ptr(), num_live.data_ptr(), wa, wn)
    return refs_out, tables_out, page_map, num_live


# ---------------------------------------------------------------------------
# norms
# ---------------------------------------------------------------------------

def block_norm(x: Optional[torch.Tensor], residual: torch.Tensor, w_post: Optional[torch.Tensor] = None,
               w_pre: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, eps: float = 1e-6,
               residual_scale: float = 1.0, block_scale: float = 1.0, out: Optional[torch.Tensor] = None,
               y: Optional[torch.Tensor] = None) -> Tuple[Optional[torch.Tensor], Optional[torch.Tensor]]:
    """The norms around a block, in one pass -> (h', y):

    h' = residual_scale * residual + block_scale * gate * norm(x) * w_post, y = norm(h') * w_pre.

    x bf16 [T, n] (None: the norm before the first block; h' is then the residual itself unless residual_scale
    changes it), residual bf16 or float32 [T, n]; without w_post x enters as it is, without w_pre y is None.
    gate bf16 [n], or [G, n] with G dividing T (row t takes gate row t // (T // G)). out may be residual."""
    kind = _RESIDUALS.get(residual.dtype) if isinstance(residual, torch.Tensor) else None
    if kind is None:
        raise TypeError(f"residual must be a torch.bfloat16 or torch.float32 tensor, got {getattr(residual, 'dtype', residual)}")
    _need(residual, "residual", residual.dtype, 2)
    index, shape = residual.get_device(), residual.shape
    t, n = shape
    xa = ga = oa = ya = wa = wb = None
    xs = os_ = ys = n
    gate_rows = 1
    if x is not None:
        if _need(x, "x", _BF16, 2, index).shape != shape:
            raise ValueError("x and residual must have the same shape")
        xa = x.data_ptr()
    if gate is not None:
        if _need(gate, "gate", _BF16, gate.dim(), index).shape[-1] != n or gate.dim() > 2 or not gate.is_contiguous():
            raise ValueError(f"gate must be contiguous [{n}] or [G, {n}]")
        ga, gate_rows = gate.data_ptr(), gate.size(0) if gate.dim() == 2 else 1
    if w_post is not None:
        wa = _vector(w_post, "w_post", n, index, _BF16)
    h = residual
    if x is not None or residual_scale != 1.0 or out is not None:    # else the residual passes through unchanged
        if out is None:
            out = torch.empty_like(residual)
        elif _need(out, "out", residual.dtype, 2, index).shape != shape:
            raise ValueError("out and residual must have the same shape")
        h, oa = out, out.data_ptr()
    if w_pre is not None:
        wb = _vector(w_pre, "w_pre", n, index, _BF16)
        if y is None:
            y = torch.empty_like(residual) if kind == RESIDUAL_BF16 else torch.empty(shape, dtype=_BF16, device=residual.device)
        elif _need(y, "y", _BF16, 2, index).shape != shape:
            raise ValueError("y and residual must have the same shape")
        ya = y.data_ptr()
    elif y is not None:
        raise ValueError("y needs w_pre")
    hs = n
    if t > 1:
        hs = residual.stride(0)
        if xa is not None:
            xs = x.stride(0)
        if oa is not None:
            os_ = out.stride(0)
        if ya is not None:
            ys = y.stride(0)
    _run("block_norm", index, _FN["block_norm"], xa, xs, residual.data_ptr(), hs, kind, ga, gate_rows, wa, wb, t, n, eps,
         residual_scale, block_scale, oa, os_, ya, ys)
    return h, y
