"""Python binding of libkda's latent-attention and cache-page entry points.

Argument marshalling only, as in :mod:`.api`: tensors are described by pointer,
sizes and strides and handed to the C entry points together with the current
HIP stream.  A non-OK status raises :class:`KDAError`.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Sequence

import torch

from . import _lib
from ._lib import KDA_BF16, KDAError, LatentDecodeArgs, LatentPrefillArgs, PagePool, PageStore
from .api import _device, _index_code, _on_stream, _stream_handle


def _bf16(what: str, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.dtype != torch.bfloat16:
            raise KDAError(what, 2, "%s must be bfloat16, got %s" % (name, t.dtype))


def _int32(what: str, name: str, t: torch.Tensor, dim: int) -> None:
    if t.dtype != torch.int32 or t.dim() != dim:
        raise KDAError(what, 2, "%s must be a %d-D int32 tensor" % (name, dim))


def _dense_last(what: str, **tensors) -> None:
    for name, t in tensors.items():
        if t is not None and t.shape[-1] > 1 and t.stride(-1) != 1:
            raise KDAError(what, 4, "the last dim of %s must be dense" % name)


def _out(what: str, name: str, t: Optional[torch.Tensor], shape, dtype, device, made: list) -> torch.Tensor:
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=device)
        made.append(t)
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise KDAError(what, 3, "%s must be a contiguous %s tensor of shape %s" % (name, dtype, tuple(shape)))
    return t


def kda_latent_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                       k_rope: Optional[torch.Tensor] = None, cu_seqlens_k: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                       scale: Optional[float] = None, causal: bool = True, with_lse: bool = False, stream=None):
    """Latent attention in the expanded form over a packed batch.

    q: [T,H,D+R]; k: [S,H,D]; v: [S,H,E]; k_rope: [S,R], the rotary part of the
    key shared by the heads (None: R = 0); all bf16 with a dense last dim and
    any strides that are multiples of 8 (views of a joint projection are
    fine).  cu_seqlens, cu_seqlens_k: [N+1] int32 offsets of the queries and
    of the keys (default: the same).  With ``causal``, a sequence's queries are
    the last of its key positions.  ``scale`` defaults to (D+R)^-1/2.
    Returns (out [T,H,E], lse [T,H] fp32 or None); a query that sees no key
    gets 0 and -inf.
    """
    what = "kda_latent_prefill"
    lib = _lib.load_library()
    if cu_seqlens_k is None:
        cu_seqlens_k = cu_seqlens
    dev = _device(q, k, v, cu_seqlens, k_rope, cu_seqlens_k, out, lse)
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3 or (k_rope is not None and k_rope.dim() != 2):
        raise KDAError(what, 3, "q, k, v must be 3-D and k_rope 2-D")
    T, H, S, D, E = int(q.shape[0]), int(q.shape[1]), int(k.shape[0]), int(k.shape[2]), int(v.shape[2])
    R = 0 if k_rope is None else int(k_rope.shape[1])
    if (int(q.shape[2]) != D + R or int(k.shape[1]) != H or tuple(v.shape[:2]) != (S, H)
            or (k_rope is not None and int(k_rope.shape[0]) != S)):
        raise KDAError(what, 3, "need q [T,H,D+R], k [S,H,D], k_rope [S,R], v [S,H,E]")
    _bf16(what, q=q, k=k, v=v, k_rope=k_rope)
    _dense_last(what, q=q, k=k, v=v, k_rope=k_rope)
    for name, t in (("cu_seqlens", cu_seqlens), ("cu_seqlens_k", cu_seqlens_k)):
        _int32(what, name, t, 1)
        if not t.is_contiguous():
            raise KDAError(what, 4, "%s must be contiguous" % name)
    N = int(cu_seqlens.numel()) - 1
    if N < 0 or int(cu_seqlens_k.numel()) != N + 1:
        raise KDAError(what, 3, "cu_seqlens and cu_seqlens_k must be [N+1]")
    made = []
    out = _out(what, "out", out, (T, H, E), q.dtype, q.device, made)
    if lse is not None or with_lse:
        lse = _out(what, "lse", lse, (T, H), torch.float32, q.device, made)
    _on_stream(stream, dev, *made)
    a = LatentPrefillArgs()
    a.T, a.S, a.N, a.H, a.D, a.R, a.E = T, S, N, H, D, R, E
    a.dtype = KDA_BF16
    a.q, a.k, a.v = q.data_ptr(), k.data_ptr(), v.data_ptr()
    for i in range(2):
        a.q_stride[i], a.k_stride[i], a.v_stride[i] = int(q.stride(i)), int(k.stride(i)), int(v.stride(i))
    if k_rope is not None:
        a.k_rope, a.k_rope_stride = k_rope.data_ptr(), int(k_rope.stride(0))
    a.cu_seqlens_q, a.cu_seqlens_k = cu_seqlens.data_ptr(), cu_seqlens_k.data_ptr()
    a.out = out.data_ptr()
    a.lse = lse.data_ptr() if lse is not None else None
    a.scale = float((D + R) ** -0.5 if scale is None else scale)
    a.causal = 1 if causal else 0
    with torch.cuda.device(dev):
        st = lib.kda_latent_prefill(ctypes.byref(a), _stream_handle(stream, dev))
    _lib.check(what, st)
    return out, lse


def kda_latent_decode_workspace_size(N: int, Q: int, H: int, L: int) -> int:
    return int(_lib.load_library().kda_latent_decode_workspace_size(N, Q, H, L))


def kda_latent_decode(cache: torch.Tensor, page_table: torch.Tensor, lengths: torch.Tensor, q: torch.Tensor,
                      q_rope: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                      out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                      with_lse: bool = False, workspace: Optional[torch.Tensor] = None, stream=None):
    """Latent attention in the absorbed form: new tokens against a paged cache.

    cache: [num_pages, page_size, L+R] bf16 (dense inner dims, any page stride):
    one row a token, its latent vector and its rotary key; page_table:
    [N, max_pages] int32; lengths: [N] int32 tokens in the cache, the new ones
    included; q: [N,H,L] or [N,Q,H,L] with the key up-projection folded in;
    q_rope: the same with R (None: R = 0).  Query i of Q sees the rows before
    lengths - (Q-1-i).  ``scale`` must be given: it is that of the expanded
    form.  Returns (out like q, lse fp32 without the last dim, or None).
    A call takes its workspace from PyTorch unless one is given
    (:func:`kda_latent_decode_workspace_size` bytes); calls that can overlap
    need workspaces of their own.
    """
    what = "kda_latent_decode"
    lib = _lib.load_library()
    if scale is None:
        raise KDAError(what, 3, "scale must be given: the expanded form's key dim is not known here")
    dev = _device(cache, page_table, lengths, q, q_rope, out, lse, workspace)
    if cache.dim() != 3 or q.dim() not in (3, 4) or (q_rope is not None and q_rope.dim() != q.dim()):
        raise KDAError(what, 3, "cache must be 3-D, q and q_rope 3-D or 4-D")
    _bf16(what, cache=cache, q=q, q_rope=q_rope)
    _dense_last(what, q=q, q_rope=q_rope)
    _int32(what, "page_table", page_table, 2)
    _int32(what, "lengths", lengths, 1)
    shape = tuple(q.shape)
    q4 = q.unsqueeze(1) if q.dim() == 3 else q
    N, Q, H, L = (int(x) for x in q4.shape)
    R = 0
    if q_rope is not None:
        r4 = q_rope.unsqueeze(1) if q_rope.dim() == 3 else q_rope
        R = int(r4.shape[3])
        if tuple(r4.shape[:3]) != (N, Q, H):
            raise KDAError(what, 3, "q_rope must be [N,(Q,)H,R]")
    num_pages, page_size, D = (int(x) for x in cache.shape)
    if D != L + R:
        raise KDAError(what, 3, "cache rows hold %d values, q and q_rope %d" % (D, L + R))
    if (page_size > 1 and cache.stride(1) != D) or (D > 1 and cache.stride(2) != 1):
        raise KDAError(what, 4, "cache pages must be dense")
    if int(page_table.shape[0]) != N or int(lengths.shape[0]) != N:
        raise KDAError(what, 3, "page_table must be [N,max_pages] and lengths [N]")
    if (page_table.shape[1] > 1 and page_table.stride(1) != 1) or not lengths.is_contiguous():
        raise KDAError(what, 4, "page_table rows and lengths must be dense")
    made = []
    out = _out(what, "out", out, shape, q.dtype, q.device, made)
    if lse is not None or with_lse:
        lse = _out(what, "lse", lse, shape[:-1], torch.float32, q.device, made)
    need = int(lib.kda_latent_decode_workspace_size(N, Q, H, L))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
        made.append(workspace)
    _on_stream(stream, dev, *made)
    a = LatentDecodeArgs()
    a.N, a.Q, a.H, a.L, a.R = N, Q, H, L, R
    a.dtype = KDA_BF16
    a.cache, a.num_pages, a.page_size = cache.data_ptr(), num_pages, page_size
    a.page_stride = int(cache.stride(0)) if num_pages > 1 else page_size * D
    a.page_table, a.max_pages = page_table.data_ptr(), int(page_table.shape[1])
    a.table_stride = int(page_table.stride(0))
    a.lengths = lengths.data_ptr()
    a.q = q4.data_ptr()
    for i in range(3):
        a.q_stride[i] = int(q4.stride(i))
    if R > 0:
        a.q_rope = r4.data_ptr()
        for i in range(3):
            a.q_rope_stride[i] = int(r4.stride(i))
    a.out = out.data_ptr()
    a.lse = lse.data_ptr() if lse is not None else None
    a.scale = float(scale)
    if workspace is not None:
        a.workspace = workspace.data_ptr()
        a.workspace_bytes = workspace.numel() * workspace.element_size() if workspace.is_contiguous() else 0
    with torch.cuda.device(dev):
        st = lib.kda_latent_decode(ctypes.byref(a), _stream_handle(stream, dev))
    _lib.check(what, st)
    return out, lse


def _pool(what: str, table: torch.Tensor, lengths: torch.Tensor, refs: torch.Tensor, page_size: int) -> PagePool:
    _int32(what, "table", table, 2)
    _int32(what, "lengths", lengths, 1)
    _int32(what, "refs", refs, 1)
    if int(lengths.shape[0]) != int(table.shape[0]):
        raise KDAError(what, 3, "table must be [num_seqs,max_pages] and lengths [num_seqs]")
    if (table.shape[1] > 1 and table.stride(1) != 1) or not lengths.is_contiguous() or not refs.is_contiguous():
        raise KDAError(what, 4, "table rows, lengths and refs must be dense")
    p = PagePool()
    p.table, p.table_stride = table.data_ptr(), int(table.stride(0))
    p.num_seqs, p.max_pages = int(table.shape[0]), int(table.shape[1])
    p.lengths, p.refs = lengths.data_ptr(), refs.data_ptr()
    p.num_pages, p.page_size = int(refs.shape[0]), int(page_size)
    return p


def _stores(what: str, caches: Sequence[torch.Tensor], num_pages: int):
    arr = (PageStore * max(1, len(caches)))()
    for s, c in zip(arr, caches):
        if c.dim() < 2 or int(c.shape[0]) != num_pages:
            raise KDAError(what, 3, "a cache must be [num_pages, ...] with the pool's %d pages" % num_pages)
        run = 1
        for d in range(c.dim() - 1, 0, -1):
            if c.shape[d] != 1 and c.stride(d) != run:
                raise KDAError(what, 4, "a cache's pages must be dense")
            run *= int(c.shape[d])
        b = c.element_size()
        s.data, s.page_bytes = c.data_ptr(), run * b
        s.page_stride = int(c.stride(0)) * b if num_pages > 1 else run * b
    return arr


def kda_page_fork(table: torch.Tensor, lengths: torch.Tensor, refs: torch.Tensor, src: torch.Tensor,
                  dst: torch.Tensor, page_size: int, caches: Sequence[torch.Tensor] = (), share: bool = True,
                  status: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                  stream=None) -> torch.Tensor:
    """Slots dst[i] become children of slots src[i].

    table: [num_seqs, max_pages] int32; lengths: [num_seqs] int32 tokens; refs:
    [num_pages] int32 (updated in place, as the caches are); src, dst: int32 or
    int64; caches: tensors [num_pages, ...] of any type whose pages are dense.
    With ``share`` the child holds the parent's full pages and gets a copy of a
    partly filled last one; without, copies of all.  Returns status [M] int32:
    0 served, 1 too few free pages, 2 bad entry (include/kda.h has the rules).
    """
    what = "kda_page_fork"
    lib = _lib.load_library()
    dev = _device(table, lengths, refs, src, dst, status, workspace, *caches)
    pool = _pool(what, table, lengths, refs, page_size)
    if src.dim() != 1 or src.shape != dst.shape or src.dtype != dst.dtype:
        raise KDAError(what, 3, "src and dst must be 1-D tensors of one size and type")
    if not src.is_contiguous() or not dst.is_contiguous():
        raise KDAError(what, 4, "src and dst must be contiguous")
    M = int(src.shape[0])
    stores = _stores(what, caches, int(refs.shape[0]))
    made = []
    status = _out(what, "status", status, (M,), torch.int32, table.device, made)
    need = int(lib.kda_page_fork_workspace_size(M, pool.max_pages, pool.num_pages, 1 if share else 0))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=table.device)
        made.append(workspace)
    _on_stream(stream, dev, *made)
    ws, wb = _span(workspace)
    with torch.cuda.device(dev):
        st = lib.kda_page_fork(ctypes.byref(pool), stores, len(caches), src.data_ptr(), dst.data_ptr(),
                               _index_code(src), M, 1 if share else 0, status.data_ptr(), ws, wb,
                               _stream_handle(stream, dev))
    _lib.check(what, st)
    return status


def _span(workspace):
    if workspace is None or not workspace.is_contiguous():
        return None, 0
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def kda_page_compact(table: torch.Tensor, lengths: torch.Tensor, refs: torch.Tensor, page_size: int,
                     caches: Sequence[torch.Tensor] = (), live: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Moves the pages in use to the front of the pool; returns their number
    ([1] int32, on the device).  Arguments as for :func:`kda_page_fork`."""
    what = "kda_page_compact"
    lib = _lib.load_library()
    dev = _device(table, lengths, refs, live, workspace, *caches)
    pool = _pool(what, table, lengths, refs, page_size)
    stores = _stores(what, caches, int(refs.shape[0]))
    made = []
    live = _out(what, "live", live, (1,), torch.int32, table.device, made)
    need = int(lib.kda_page_compact_workspace_size(pool.num_pages))
    if workspace is None and need > 0:
        workspace = torch.empty(need, dtype=torch.uint8, device=table.device)
        made.append(workspace)
    _on_stream(stream, dev, *made)
    ws, wb = _span(workspace)
    with torch.cuda.device(dev):
        st = lib.kda_page_compact(ctypes.byref(pool), stores, len(caches), live.data_ptr(), ws, wb,
                                  _stream_handle(stream, dev))
    _lib.check(what, st)
    return live


def kda_page_free(table: torch.Tensor, lengths: torch.Tensor, refs: torch.Tensor, release: torch.Tensor,
                  page_size: int, stream=None) -> None:
    """Empties the slots with release[s] != 0 ([num_seqs] bool or uint8): their
    pages lose one reference each and are free when none is left."""
    what = "kda_page_free"
    lib = _lib.load_library()
    dev = _device(table, lengths, refs, release)
    pool = _pool(what, table, lengths, refs, page_size)
    if release.dtype not in (torch.bool, torch.uint8) or release.dim() != 1 or not release.is_contiguous():
        raise KDAError(what, 2, "release must be a contiguous 1-D bool/uint8 tensor")
    if int(release.shape[0]) != pool.num_seqs:
        raise KDAError(what, 3, "release must have one entry a slot")
    with torch.cuda.device(dev):
        st = lib.kda_page_free(ctypes.byref(pool), release.data_ptr(), _stream_handle(stream, dev))
    _lib.check(what, st)
