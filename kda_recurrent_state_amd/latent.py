"""Python binding of libkda's latent-attention and cache-page entry points.

Argument marshalling only, as in :mod:`.api`: tensors are described by pointer,
sizes and strides and handed to the C entry points together with the current
HIP stream.  A non-OK status raises :class:`KDAError`.
"""
from __future__ import annotations

from typing import Optional, Sequence

import torch

from . import _lib
from ._lib import (KDA_BF16, KDA_E4M3, KDA_F32, KDA_I32, KDA_I64, KDAError, LatentDecodeArgs, LatentPrefillArgs,
                   LatentSharedArgs, LatentStore, PagePool, PageStore)
from .api import _device as _checked_device, _index_code, _on_stream, _stream_handle


def _device(first: torch.Tensor, *others) -> torch.device:
    """The one device of all given tensors (the slow check words the error)."""
    index = first.get_device()
    for t in others:
        if t is not None and t.get_device() != index:
            index = -1
            break
    return first.device if index >= 0 else _checked_device(first, *others)


def _int32(what: str, name: str, t: torch.Tensor, dim: int) -> None:
    if t.dtype != torch.int32 or t.dim() != dim:
        raise KDAError(what, 2, "%s must be a %d-D int32 tensor" % (name, dim))


def _operand(what: str, name: str, t: torch.Tensor) -> None:
    if t.dtype != torch.bfloat16:
        raise KDAError(what, 2, "%s must be bfloat16, got %s" % (name, t.dtype))
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        raise KDAError(what, 4, "the last dim of %s must be dense" % name)


def _out(what: str, name: str, t: Optional[torch.Tensor], shape, dtype, device, made: list) -> torch.Tensor:
    if t is None:
        t = torch.empty(shape, dtype=dtype, device=device)
        made.append(t)
    elif t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise KDAError(what, 3, "%s must be a contiguous %s tensor of shape %s" % (name, dtype, tuple(shape)))
    return t


def _workspace(workspace: Optional[torch.Tensor], need: int, device, made: list):
    """Address and bytes of the caller's workspace, or of one made here."""
    if workspace is None:
        if need == 0:
            return None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
        made.append(workspace)
    elif not workspace.is_contiguous():
        return None, 0
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def _call(what: str, dev: torch.device, stream, made: list, entry, *args) -> None:
    """entry(*args, stream) with the tensors' device current.  (The short
    calls are bound by the host, so the common case, the current stream of the
    current device, takes no context manager and makes no stream object.)"""
    index = dev.index
    if stream is None and index == torch.cuda.current_device():
        st = entry(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        _on_stream(stream, dev, *made)
        with torch.cuda.device(dev):
            st = entry(*args, _stream_handle(stream, dev))
    if st != 0:
        _lib.check(what, st)


def kda_latent_prefill(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                       k_rope: Optional[torch.Tensor] = None, cu_seqlens_k: Optional[torch.Tensor] = None,
                       out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                       scale: Optional[float] = None, causal: bool = True, with_lse: bool = False,
                       workspace: Optional[torch.Tensor] = None, stream=None):
    """Latent attention in the expanded form over a packed batch.

    q: [T,H,D+R]; k: [S,H,D]; v: [S,H,E]; k_rope: [S,R], the rotary part of the
    key shared by the heads (None: R = 0); all bf16 with a dense last dim and
    any strides that are multiples of 8 (views of a joint projection are
    fine).  cu_seqlens, cu_seqlens_k: [N+1] int32 offsets of the queries and
    of the keys (default: the same).  With ``causal``, a sequence's queries are
    the last of its key positions.  ``scale`` defaults to (D+R)^-1/2.
    Returns (out [T,H,E], lse [T,H] fp32 or None); a query that sees no key
    gets 0 and -inf.  Few queries over many keys take a workspace, from PyTorch
    unless one is given (:func:`kda_latent_prefill_workspace_size` bytes).
    """
    what = "kda_latent_prefill"
    lib = _lib.load_library()
    if cu_seqlens_k is None:
        cu_seqlens_k = cu_seqlens
    dev = _device(q, k, v, cu_seqlens, k_rope, cu_seqlens_k, out, lse, workspace)
    if q.dim() != 3 or k.dim() != 3 or v.dim() != 3 or (k_rope is not None and k_rope.dim() != 2):
        raise KDAError(what, 3, "q, k, v must be 3-D and k_rope 2-D")
    (T, H, DR), (S, Hk, D), (Sv, Hv, E) = q.shape, k.shape, v.shape
    R = 0 if k_rope is None else k_rope.shape[1]
    if DR != D + R or Hk != H or Hv != H or Sv != S or (k_rope is not None and k_rope.shape[0] != S):
        raise KDAError(what, 3, "need q [T,H,D+R], k [S,H,D], k_rope [S,R], v [S,H,E]")
    _operand(what, "q", q)
    _operand(what, "k", k)
    _operand(what, "v", v)
    rope = (None, 0)
    if k_rope is not None:
        _operand(what, "k_rope", k_rope)
        rope = (k_rope.data_ptr(), k_rope.stride(0))
    _int32(what, "cu_seqlens", cu_seqlens, 1)
    _int32(what, "cu_seqlens_k", cu_seqlens_k, 1)
    if not (cu_seqlens.is_contiguous() and cu_seqlens_k.is_contiguous()):
        raise KDAError(what, 4, "cu_seqlens and cu_seqlens_k must be contiguous")
    N = cu_seqlens.shape[0] - 1
    if N < 0 or cu_seqlens_k.shape[0] != N + 1:
        raise KDAError(what, 3, "cu_seqlens and cu_seqlens_k must be [N+1]")
    made = []
    out = _out(what, "out", out, (T, H, E), torch.bfloat16, dev, made)
    if lse is not None or with_lse:
        lse = _out(what, "lse", lse, (T, H), torch.float32, dev, made)
    ws = _workspace(workspace, lib.kda_latent_prefill_workspace_size(T, S, N, H, E), dev, made)
    a = LatentPrefillArgs(T, S, N, H, D, R, E, KDA_BF16, q.data_ptr(), q.stride()[:2], k.data_ptr(), k.stride()[:2],
                          *rope, v.data_ptr(), v.stride()[:2], cu_seqlens.data_ptr(), cu_seqlens_k.data_ptr(),
                          out.data_ptr(), None if lse is None else lse.data_ptr(),
                          DR ** -0.5 if scale is None else scale, 1 if causal else 0, *ws)
    _call(what, dev, stream, made, lib.kda_latent_prefill, a)
    return out, lse


def kda_latent_prefill_workspace_size(T: int, S: int, N: int, H: int, E: int) -> int:
    return int(_lib.load_library().kda_latent_prefill_workspace_size(T, S, N, H, E))


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
    if cache.dtype != torch.bfloat16:
        raise KDAError(what, 2, "cache must be bfloat16, got %s" % cache.dtype)
    _operand(what, "q", q)
    _int32(what, "page_table", page_table, 2)
    _int32(what, "lengths", lengths, 1)
    shape = q.shape
    q4 = q.unsqueeze(1) if len(shape) == 3 else q
    N, Q, H, L = q4.shape
    R, rope = 0, (None, (0, 0, 0))
    if q_rope is not None:
        _operand(what, "q_rope", q_rope)
        r4 = q_rope.unsqueeze(1) if len(shape) == 3 else q_rope
        R = r4.shape[3]
        if r4.shape[:3] != q4.shape[:3]:
            raise KDAError(what, 3, "q_rope must be [N,(Q,)H,R]")
        if R > 0:
            rope = (r4.data_ptr(), r4.stride()[:3])
    num_pages, page_size, D = cache.shape
    page_stride, row_stride, last = cache.stride()
    if D != L + R:
        raise KDAError(what, 3, "cache rows hold %d values, q and q_rope %d" % (D, L + R))
    if (page_size > 1 and row_stride != D) or (D > 1 and last != 1):
        raise KDAError(what, 4, "cache pages must be dense")
    if page_table.shape[0] != N or lengths.shape[0] != N:
        raise KDAError(what, 3, "page_table must be [N,max_pages] and lengths [N]")
    if (page_table.shape[1] > 1 and page_table.stride(1) != 1) or not lengths.is_contiguous():
        raise KDAError(what, 4, "page_table rows and lengths must be dense")
    made = []
    out = _out(what, "out", out, shape, torch.bfloat16, dev, made)
    if lse is not None or with_lse:
        lse = _out(what, "lse", lse, shape[:-1], torch.float32, dev, made)
    ws = _workspace(workspace, lib.kda_latent_decode_workspace_size(N, Q, H, L), dev, made)
    a = LatentDecodeArgs(N, Q, H, L, R, KDA_BF16, cache.data_ptr(), num_pages, page_size,
                         page_stride if num_pages > 1 else page_size * D, page_table.data_ptr(),
                         page_table.stride(0), page_table.shape[1], lengths.data_ptr(), q4.data_ptr(),
                         q4.stride()[:3], *rope, out.data_ptr(), None if lse is None else lse.data_ptr(), scale, *ws)
    _call(what, dev, stream, made, lib.kda_latent_decode, a)
    return out, lse


_CODES = (torch.float8_e4m3fn, torch.uint8)


def _pages(what: str, name: str, shape, stride, run: int, align: int) -> int:
    """Elements from page to page of a cache tensor [num_pages, page_size(, row)] whose pages, ``run`` elements, are
    dense (of the only page: any such number that is a multiple of ``align``)."""
    row = shape[2] if len(shape) == 3 else 1
    if (shape[1] != 1 and stride[1] != row) or (row != 1 and stride[-1] != 1):
        raise KDAError(what, 4, "%s: the pages must be dense" % name)
    return stride[0] if shape[0] > 1 else -(-run // align) * align


def _store(what: str, codes: torch.Tensor, scales: torch.Tensor, rope: Optional[torch.Tensor]):
    """The fields of a LatentStore for an 8-bit latent cache's tensors."""
    shape, near = codes.shape, scales.shape
    if len(shape) != 3 or len(near) != 2:
        raise KDAError(what, 3, "codes must be 3-D, scales 2-D")
    if codes.dtype not in _CODES or scales.dtype != torch.float32:
        raise KDAError(what, 2, "codes must be float8_e4m3fn or uint8 and scales float32, got %s and %s"
                       % (codes.dtype, scales.dtype))
    num_pages, page_size, L = shape
    R, rope_at, rope_page = 0, None, 0
    if near[0] != num_pages or near[1] != page_size:
        raise KDAError(what, 3, "need codes [num_pages,page_size,L] and scales [num_pages,page_size]")
    if rope is not None:
        rshape = rope.shape
        if len(rshape) != 3 or rshape[0] != num_pages or rshape[1] != page_size:
            raise KDAError(what, 3, "need rope [num_pages,page_size,R]")
        if rope.dtype != torch.bfloat16:
            raise KDAError(what, 2, "rope must be bfloat16, got %s" % rope.dtype)
        R = rshape[2]
        if R > 0:
            rope_at = rope.data_ptr()
            rope_page = _pages(what, "rope", rshape, rope.stride(), page_size * R, 8)
    return (codes.data_ptr(), scales.data_ptr(), rope_at, num_pages, page_size, L, R,
            _pages(what, "codes", shape, codes.stride(), page_size * L, 16),
            _pages(what, "scales", near, scales.stride(), page_size, 1), rope_page)


def _rows(what: str, name: str, t: torch.Tensor) -> int:
    row, last = t.stride()
    if last != 1 and t.shape[1] > 1:
        raise KDAError(what, 4, "the last dim of %s must be dense" % name)
    return row


def _index(what: str, slots: torch.Tensor) -> int:
    if slots.dtype == torch.int32:
        return KDA_I32
    if slots.dtype == torch.int64:
        return KDA_I64
    raise KDAError(what, 2, "slots must be int32 or int64, got %s" % slots.dtype)


_VALUES = {torch.float32: KDA_F32, torch.bfloat16: KDA_BF16}


def kda_latent_quantize_scatter(c: torch.Tensor, k_rope: Optional[torch.Tensor], slots: torch.Tensor,
                                codes: torch.Tensor, scales: torch.Tensor, rope: Optional[torch.Tensor] = None,
                                stream=None) -> None:
    """Writes token rows into an 8-bit latent cache.

    c: [T,L] latent vectors and k_rope: [T,R] rotary keys, both bf16 or both
    fp32, rows with any strides that are multiples of 8 (None: R = 0); slots: [T] int32 or
    int64, the token row (page * page_size + place) each goes to, entries
    outside the cache are skipped; codes: [num_pages, page_size, L]
    float8_e4m3fn (or uint8, the bits); scales: [num_pages, page_size] fp32; rope:
    [num_pages, page_size, R] bf16 (dense pages, any page stride that keeps 16 bytes' alignment).
    A row's scale is the smallest power of two under which its largest
    component is at most 448, its codes c / scale rounded to e4m3.  A row that
    is not finite gets the scale NaN.  Valid slots must be unique.
    """
    what = "kda_latent_quantize_scatter"
    lib = _lib.load_library()
    dev = _device(c, k_rope, slots, codes, scales, rope)
    store = _store(what, codes, scales, rope)
    shape, given = c.shape, slots.shape
    if len(shape) != 2 or len(given) != 1:
        raise KDAError(what, 3, "c must be 2-D, slots 1-D")
    T, R = shape[0], store[6]
    dtype = _VALUES.get(c.dtype)
    if dtype is None or (k_rope is not None and k_rope.dtype != c.dtype):
        raise KDAError(what, 2, "c and k_rope must both be bfloat16 or both float32")
    if shape[1] != store[5] or given[0] != T or (R > 0 if k_rope is None else tuple(k_rope.shape) != (T, R)):
        raise KDAError(what, 3, "need c [T,L], k_rope [T,R], slots [T] with the cache's L and R")
    if not slots.is_contiguous():
        raise KDAError(what, 4, "slots must be contiguous")
    _call(what, dev, stream, [], lib.kda_latent_quantize_scatter, LatentStore(*store), c.data_ptr(), _rows(what, "c", c),
          k_rope.data_ptr() if R > 0 else None, _rows(what, "k_rope", k_rope) if R > 0 else 0, dtype, slots.data_ptr(),
          _index(what, slots), T)


def kda_latent_dequantize_gather(codes: torch.Tensor, scales: torch.Tensor, rope: Optional[torch.Tensor],
                                 slots: torch.Tensor, out: Optional[torch.Tensor] = None,
                                 dtype: torch.dtype = torch.bfloat16, stream=None) -> torch.Tensor:
    """Reads token rows of an 8-bit latent cache: [T, L+R], the latent vector
    (code * scale) and the rotary key, in bf16 or fp32 (``dtype``, or that of
    ``out``); zeros for slots outside the cache.  The cache's tensors and slots
    as for :func:`kda_latent_quantize_scatter`; slots may repeat."""
    what = "kda_latent_dequantize_gather"
    lib = _lib.load_library()
    dev = _device(codes, scales, rope, slots, out)
    store = _store(what, codes, scales, rope)
    given = slots.shape
    if len(given) != 1:
        raise KDAError(what, 3, "slots must be 1-D")
    if not slots.is_contiguous():
        raise KDAError(what, 4, "slots must be contiguous")
    if out is not None:
        dtype = out.dtype
    if dtype not in _VALUES:
        raise KDAError(what, 2, "rows are read as bfloat16 or float32, not %s" % dtype)
    made = []
    out = _out(what, "out", out, (given[0], store[5] + store[6]), dtype, dev, made)
    _call(what, dev, stream, made, lib.kda_latent_dequantize_gather, LatentStore(*store), slots.data_ptr(),
          _index(what, slots), given[0], out.data_ptr(), _VALUES[dtype])
    return out


def kda_latent_shared_workspace_size(N: int, Q: int, H: int, L: int, G: int = 0) -> int:
    return int(_lib.load_library().kda_latent_shared_workspace_size(N, Q, H, L, G))


def _decode_shared(what: str, cache, page_table, lengths, cu_groups, shared, q, q_rope, scale, out, lse, with_lse,
                   workspace, stream):
    lib = _lib.load_library()
    if scale is None:
        raise KDAError(what, 3, "scale must be given: the expanded form's key dim is not known here")
    fp8 = isinstance(cache, (tuple, list))
    if fp8 and len(cache) != 3:
        raise KDAError(what, 3, "an 8-bit cache is (codes, scales, rope)")
    codes, scales, rope = cache if fp8 else (cache, None, None)
    dev = _device(codes, scales, rope, page_table, lengths, cu_groups, shared, q, q_rope, out, lse, workspace)
    if q.dim() not in (3, 4) or (q_rope is not None and q_rope.dim() != q.dim()):
        raise KDAError(what, 3, "q and q_rope must be 3-D or 4-D")
    _operand(what, "q", q)
    _int32(what, "page_table", page_table, 2)
    _int32(what, "lengths", lengths, 1)
    shape = q.shape
    q4 = q.unsqueeze(1) if len(shape) == 3 else q
    N, Q, H, L = q4.shape
    R, rope_q = 0, (None, (0, 0, 0))
    if q_rope is not None:
        _operand(what, "q_rope", q_rope)
        r4 = q_rope.unsqueeze(1) if len(shape) == 3 else q_rope
        R = r4.shape[3]
        if r4.shape[:3] != q4.shape[:3]:
            raise KDAError(what, 3, "q_rope must be [N,(Q,)H,R]")
        if R > 0:
            rope_q = (r4.data_ptr(), r4.stride()[:3])
    if fp8:
        store = _store(what, codes, scales, rope)
        if store[5] != L or store[6] != R:
            raise KDAError(what, 3, "cache rows hold %d + %d values, q and q_rope %d + %d" % (store[5], store[6], L, R))
        head = (KDA_E4M3, *store[:5], *store[7:])
    else:
        held = cache.shape
        if len(held) != 3 or held[2] != L + R:
            raise KDAError(what, 3, "cache must be [num_pages,page_size,%d] as q and q_rope are" % (L + R))
        if cache.dtype != torch.bfloat16:
            raise KDAError(what, 2, "cache must be bfloat16 or (codes, scales, rope), got %s" % cache.dtype)
        head = (KDA_BF16, cache.data_ptr(), None, None, held[0], held[1],
                _pages(what, "cache", held, cache.stride(), held[1] * held[2], 8), 0, 0)
    if page_table.shape[0] != N or lengths.shape[0] != N:
        raise KDAError(what, 3, "page_table must be [N,max_pages] and lengths [N]")
    if (page_table.shape[1] > 1 and page_table.stride(1) != 1) or not lengths.is_contiguous():
        raise KDAError(what, 4, "page_table rows and lengths must be dense")
    G, groups = 0, (None, None)
    if cu_groups is not None:
        _int32(what, "cu_groups", cu_groups, 1)
        _int32(what, "shared", shared, 1)
        G = shared.shape[0]
        if cu_groups.shape[0] != G + 1:
            raise KDAError(what, 3, "cu_groups must be [G+1] and shared [G]")
        if not (cu_groups.is_contiguous() and shared.is_contiguous()):
            raise KDAError(what, 4, "cu_groups and shared must be contiguous")
        groups = (cu_groups.data_ptr(), shared.data_ptr())
    made = []
    out = _out(what, "out", out, shape, torch.bfloat16, dev, made)
    if lse is not None or with_lse:
        lse = _out(what, "lse", lse, shape[:-1], torch.float32, dev, made)
    ws = _workspace(workspace, lib.kda_latent_shared_workspace_size(N, Q, H, L, G), dev, made)
    a = LatentSharedArgs(N, Q, H, L, R, G, *head, page_table.data_ptr(), page_table.stride(0), page_table.shape[1],
                         lengths.data_ptr(), *groups, q4.data_ptr(), q4.stride()[:3], *rope_q, out.data_ptr(),
                         None if lse is None else lse.data_ptr(), scale, *ws)
    _call(what, dev, stream, made, getattr(lib, what), a)
    return out, lse


def kda_latent_decode_fp8(codes: torch.Tensor, scales: torch.Tensor, rope: Optional[torch.Tensor],
                          page_table: torch.Tensor, lengths: torch.Tensor, q: torch.Tensor,
                          q_rope: Optional[torch.Tensor] = None, scale: Optional[float] = None,
                          out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                          with_lse: bool = False, workspace: Optional[torch.Tensor] = None, stream=None):
    """:func:`kda_latent_decode` over a cache in 8 bits.

    codes, scales, rope: the cache's tensors, as
    :func:`kda_latent_quantize_scatter` writes them; any scale is taken, not only
    powers of two.  The rest as for :func:`kda_latent_decode`, with the
    workspace of :func:`kda_latent_shared_workspace_size` (G = 0).
    """
    return _decode_shared("kda_latent_decode_fp8", (codes, scales, rope), page_table, lengths, None, None, q, q_rope,
                          scale, out, lse, with_lse, workspace, stream)


def kda_latent_decode_shared(cache, page_table: torch.Tensor, lengths: torch.Tensor, cu_groups: torch.Tensor,
                             shared: torch.Tensor, q: torch.Tensor, q_rope: Optional[torch.Tensor] = None,
                             scale: Optional[float] = None, out: Optional[torch.Tensor] = None,
                             lse: Optional[torch.Tensor] = None, with_lse: bool = False,
                             workspace: Optional[torch.Tensor] = None, stream=None):
    """:func:`kda_latent_decode` for sequences that share their first tokens,
    which are read and computed once for all of them.

    cache: a 16-bit cache's tensor, or (codes, scales, rope) of one in 8 bits;
    cu_groups: [G+1] int32, group g is the sequences cu_groups[g] ..
    cu_groups[g+1] - 1; shared: [G] int32, how many first tokens its sequences
    have in common (the same rows, as after a fork: they are read through the
    table of the group's first sequence).  Sequences of no group share
    nothing.  It pays for many sequences of few query rows behind a long prefix (64 with up
    to 32 rows each behind 8192 tokens, say); for few sequences, short prefixes or 128 rows
    and more :func:`kda_latent_decode` is as fast or faster.  The rest, and the results, as for :func:`kda_latent_decode`; the
    workspace has :func:`kda_latent_shared_workspace_size` bytes.
    """
    what = "kda_latent_decode_shared"
    if cu_groups is None or shared is None:
        raise KDAError(what, 1, "cu_groups and shared must be given")
    return _decode_shared(what, cache, page_table, lengths, cu_groups, shared, q, q_rope, scale, out, lse, with_lse,
                          workspace, stream)


def _pool(what: str, table: torch.Tensor, lengths: torch.Tensor, refs: torch.Tensor, page_size: int) -> PagePool:
    _int32(what, "table", table, 2)
    _int32(what, "lengths", lengths, 1)
    _int32(what, "refs", refs, 1)
    if lengths.shape[0] != table.shape[0]:
        raise KDAError(what, 3, "table must be [num_seqs,max_pages] and lengths [num_seqs]")
    if (table.shape[1] > 1 and table.stride(1) != 1) or not lengths.is_contiguous() or not refs.is_contiguous():
        raise KDAError(what, 4, "table rows, lengths and refs must be dense")
    return PagePool(table.data_ptr(), table.stride(0), table.shape[0], table.shape[1], lengths.data_ptr(),
                    refs.data_ptr(), refs.shape[0], page_size)


def _stores(what: str, caches: Sequence[torch.Tensor], num_pages: int):
    arr = (PageStore * max(1, len(caches)))()
    for s, c in zip(arr, caches):
        shape, stride = c.shape, c.stride()
        if len(shape) < 2 or shape[0] != num_pages:
            raise KDAError(what, 3, "a cache must be [num_pages, ...] with the pool's %d pages" % num_pages)
        run = 1
        for d in range(len(shape) - 1, 0, -1):
            if shape[d] != 1 and stride[d] != run:
                raise KDAError(what, 4, "a cache's pages must be dense")
            run *= shape[d]
        b = c.element_size()
        s.data, s.page_bytes = c.data_ptr(), run * b
        s.page_stride = stride[0] * b if num_pages > 1 else run * b
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
    M = src.shape[0]
    share = 1 if share else 0
    stores = _stores(what, caches, pool.num_pages)
    made = []
    status = _out(what, "status", status, (M,), torch.int32, dev, made)
    ws = _workspace(workspace, lib.kda_page_fork_workspace_size(M, pool.max_pages, pool.num_pages, share), dev, made)
    _call(what, dev, stream, made, lib.kda_page_fork, pool, stores, len(caches), src.data_ptr(), dst.data_ptr(),
          _index_code(src), M, share, status.data_ptr(), *ws)
    return status


def kda_page_compact(table: torch.Tensor, lengths: torch.Tensor, refs: torch.Tensor, page_size: int,
                     caches: Sequence[torch.Tensor] = (), live: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Moves the pages in use to the front of the pool; returns their number
    ([1] int32, on the device).  Arguments as for :func:`kda_page_fork`."""
    what = "kda_page_compact"
    lib = _lib.load_library()
    dev = _device(table, lengths, refs, live, workspace, *caches)
    pool = _pool(what, table, lengths, refs, page_size)
    stores = _stores(what, caches, pool.num_pages)
    made = []
    live = _out(what, "live", live, (1,), torch.int32, dev, made)
    ws = _workspace(workspace, lib.kda_page_compact_workspace_size(pool.num_pages), dev, made)
    _call(what, dev, stream, made, lib.kda_page_compact, pool, stores, len(caches), live.data_ptr(), *ws)
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
    if release.shape[0] != pool.num_seqs:
        raise KDAError(what, 3, "release must have one entry a slot")
    _call(what, dev, stream, [], lib.kda_page_free, pool, release.data_ptr())
