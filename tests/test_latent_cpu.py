"""Host-side refusals of the latent-attention and cache-page entry points: bad
arguments return the documented status before any HIP call is made.  Only
calls that fail validation, or that validate and enqueue nothing, are made."""
import ctypes
import math
import os

import pytest

NULL, DTYPE, SHAPE, LAYOUT, OVERLAP, UNSUPPORTED, WORKSPACE, ALIAS = 1, 2, 3, 4, 5, 6, 7, 8


@pytest.fixture(scope="module")
def lib():
    from kda_recurrent_state_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from kda_recurrent_state_amd import build
        build.build()
    return _lib.load_library()


def _set(struct, kw):
    for k, v in kw.items():
        if isinstance(v, (tuple, list)):
            for i, x in enumerate(v):
                getattr(struct, k)[i] = x
        else:
            setattr(struct, k, v)
    return struct


def _prefill(**kw):
    from kda_recurrent_state_amd._lib import LatentPrefillArgs
    a = LatentPrefillArgs()
    base = dict(T=10, S=20, N=2, H=2, D=16, R=8, E=24, dtype=1, q=0x10000, q_stride=(48, 24), k=0x20000,
                k_stride=(32, 16), k_rope=0x30000, k_rope_stride=8, v=0x40000, v_stride=(48, 24),
                cu_seqlens_q=0x50000, cu_seqlens_k=0x60000, out=0x70000, lse=0x80000, scale=0.2, causal=1)
    return _set(a, {**base, **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), SHAPE), (dict(S=-1), SHAPE), (dict(N=-1), SHAPE), (dict(H=0), SHAPE), (dict(D=0), SHAPE),
    (dict(R=-8), SHAPE), (dict(E=0), SHAPE), (dict(N=0), SHAPE),
    (dict(dtype=0), DTYPE), (dict(dtype=7), DTYPE),
    (dict(D=12), UNSUPPORTED), (dict(D=136), UNSUPPORTED), (dict(R=4), UNSUPPORTED), (dict(R=72), UNSUPPORTED),
    (dict(E=20), UNSUPPORTED), (dict(E=136), UNSUPPORTED), (dict(H=65536), UNSUPPORTED),
    (dict(T=1 << 31), UNSUPPORTED), (dict(T=1 << 30, H=65535), UNSUPPORTED),
    (dict(T=131072, N=131072, H=128, q_stride=(128 * 24, 24)), UNSUPPORTED), (dict(T=1 << 17, N=65408, H=256), UNSUPPORTED),
    (dict(T=(1 << 31) - 1, H=1), UNSUPPORTED), (dict(S=(1 << 31) - 1), UNSUPPORTED), (dict(S=(1 << 31) - 255), UNSUPPORTED),
    (dict(scale=0.0), UNSUPPORTED), (dict(scale=-1.0), UNSUPPORTED), (dict(scale=math.inf), UNSUPPORTED),
    (dict(scale=math.nan), UNSUPPORTED), (dict(scale=3e38), UNSUPPORTED),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL), (dict(k_rope=None), NULL), (dict(out=None), NULL),
    (dict(cu_seqlens_q=None), NULL), (dict(cu_seqlens_k=None), NULL),
    (dict(q_stride=(44, 24)), LAYOUT), (dict(q_stride=(48, -24)), LAYOUT), (dict(k_stride=(33, 16)), LAYOUT),
    (dict(v_stride=(48, 20)), LAYOUT), (dict(k_rope_stride=12), LAYOUT), (dict(k_stride=(1 << 50, 16)), LAYOUT),
    (dict(q=0x10008), LAYOUT), (dict(k=0x20002), LAYOUT), (dict(v=0x40008), LAYOUT), (dict(k_rope=0x30008), LAYOUT),
    (dict(out=0x70004), LAYOUT),
    (dict(S=1 << 16, H=1), WORKSPACE), (dict(S=1 << 16, H=1, workspace=0x10000000, workspace_bytes=64), WORKSPACE),
    (dict(S=1 << 16, H=1, workspace=0x10000008, workspace_bytes=1 << 30), LAYOUT),
    (dict(S=1 << 16, H=1, workspace=0x20000, workspace_bytes=1 << 30), ALIAS),
    (dict(k_stride=((1 << 24) + 8, 16)), UNSUPPORTED), (dict(v_stride=((1 << 24) + 8, 24)), UNSUPPORTED),
    (dict(k_rope_stride=(1 << 24) + 8), UNSUPPORTED),
    (dict(out=0x10000), ALIAS), (dict(out=0x20000 + 16), ALIAS), (dict(out=0x30000), ALIAS), (dict(out=0x40000), ALIAS),
    (dict(out=0x50000), ALIAS), (dict(out=0x60000), ALIAS), (dict(lse=0x70000 + 8), ALIAS), (dict(lse=0x10000), ALIAS),
])
def test_prefill_refusals(lib, kw, status):
    assert lib.kda_latent_prefill(ctypes.byref(_prefill(**kw)), None) == status


def test_prefill_workspace_is_for_few_queries_and_many_keys(lib):
    size = lib.kda_latent_prefill_workspace_size
    assert size(0, 100, 1, 8, 128) == 0 and size(100, 100, 1, 8, 136) == 0
    assert size(100, 512, 1, 8, 128) == 0 and size(1 << 16, 1 << 16, 1, 8, 128) == 0
    assert size(100, 1 << 16, 1, 8, 128) > 0


def test_prefill_nothing_to_do(lib):
    assert lib.kda_latent_prefill(None, None) == NULL
    assert lib.kda_latent_prefill(ctypes.byref(_prefill(T=0)), None) == 0
    assert lib.kda_latent_prefill(ctypes.byref(_prefill(T=0, N=0)), None) == 0


def _decode(lib, **kw):
    from kda_recurrent_state_amd._lib import LatentDecodeArgs
    a = LatentDecodeArgs()
    base = dict(N=3, Q=2, H=4, L=64, R=16, dtype=1, cache=0x1000000, num_pages=5, page_size=16, page_stride=16 * 80,
                page_table=0x20000, table_stride=4, max_pages=4, lengths=0x30000, q=0x40000, q_stride=(512, 256, 64),
                q_rope=0x50000, q_rope_stride=(128, 64, 16), out=0x60000, lse=0x70000, scale=0.2, workspace=0x10000000,
                workspace_bytes=lib.kda_latent_decode_workspace_size(3, 2, 4, 64))
    return _set(a, {**base, **kw})


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), SHAPE), (dict(Q=0), SHAPE), (dict(H=0), SHAPE), (dict(L=0), SHAPE), (dict(R=-8), SHAPE),
    (dict(num_pages=0), SHAPE), (dict(page_size=0), SHAPE), (dict(max_pages=0), SHAPE), (dict(dtype=0), DTYPE),
    (dict(L=60), UNSUPPORTED), (dict(L=520), UNSUPPORTED), (dict(R=12), UNSUPPORTED), (dict(R=72), UNSUPPORTED),
    (dict(Q=1025, H=1), UNSUPPORTED), (dict(Q=33, H=32), UNSUPPORTED), (dict(N=65536), UNSUPPORTED),
    (dict(scale=0.0), UNSUPPORTED), (dict(scale=math.nan), UNSUPPORTED), (dict(scale=3e38), UNSUPPORTED),
    (dict(scale=math.inf), UNSUPPORTED),
    (dict(max_pages=1 << 27, table_stride=1 << 27), UNSUPPORTED), (dict(page_size=1 << 31), UNSUPPORTED),
    (dict(N=65535, max_pages=1 << 21, table_stride=1 << 21), UNSUPPORTED),
    (dict(table_stride=3), OVERLAP), (dict(page_stride=16 * 80 - 8), OVERLAP), (dict(page_stride=16 * 80 + 4), LAYOUT),
    (dict(page_stride=1 << 45), SHAPE),
    (dict(cache=None), NULL), (dict(page_table=None), NULL), (dict(lengths=None), NULL), (dict(q=None), NULL),
    (dict(q_rope=None), NULL), (dict(out=None), NULL),
    (dict(q_stride=(512, 256, 60)), LAYOUT), (dict(q_rope_stride=(128, -64, 16)), LAYOUT),
    (dict(cache=0x1000008), LAYOUT), (dict(q=0x40004), LAYOUT), (dict(q_rope=0x50008), LAYOUT), (dict(out=0x60008), LAYOUT),
    (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=64), WORKSPACE), (dict(workspace=0x10000008), LAYOUT),
    (dict(out=0x1000000), ALIAS), (dict(out=0x40000), ALIAS), (dict(out=0x50000), ALIAS), (dict(lse=0x60000), ALIAS),
    (dict(workspace=0x60000), ALIAS), (dict(workspace=0x1000000), ALIAS), (dict(lse=0x30000), ALIAS),
])
def test_decode_refusals(lib, kw, status):
    assert lib.kda_latent_decode(ctypes.byref(_decode(lib, **kw)), None) == status


def test_decode_nothing_to_do_and_workspace(lib):
    assert lib.kda_latent_decode(None, None) == NULL
    assert lib.kda_latent_decode(ctypes.byref(_decode(lib, N=0)), None) == 0
    size = lib.kda_latent_decode_workspace_size
    assert size(0, 1, 32, 512) == 0 and size(1, 33, 32, 512) == 0 and size(1, 1, 32, 520) == 0
    assert size(4, 1, 32, 512) > 0


def _pool(**kw):
    from kda_recurrent_state_amd._lib import PagePool
    base = dict(table=0x10000, table_stride=8, num_seqs=6, max_pages=8, lengths=0x20000, refs=0x30000, num_pages=40,
                page_size=16)
    return _set(PagePool(), {**base, **kw})


def _stores(*stores):
    from kda_recurrent_state_amd._lib import PageStore
    arr = (PageStore * max(1, len(stores)))()
    for s, (data, stride, size) in zip(arr, stores):
        s.data, s.page_stride, s.page_bytes = data, stride, size
    return arr


def _fork(lib, pool=None, stores=((0x1000000, 256, 256),), src=0x40000, dst=0x50000, it=0, m=3, share=1, status=0x60000,
          ws=0x70000, wb=1 << 20):
    return lib.kda_page_fork(ctypes.byref(pool or _pool()), _stores(*stores), len(stores), src, dst, it, m, share,
                             status, ws, wb, None)


POOL_REFUSALS = [
    (dict(num_seqs=0), SHAPE), (dict(max_pages=0), SHAPE), (dict(num_pages=0), SHAPE), (dict(page_size=0), SHAPE),
    (dict(num_seqs=(1 << 24) + 1), UNSUPPORTED), (dict(max_pages=(1 << 20) + 1), UNSUPPORTED),
    (dict(num_pages=(1 << 30) + 1), UNSUPPORTED), (dict(page_size=(1 << 30) + 1), UNSUPPORTED),
    (dict(table_stride=7), OVERLAP), (dict(table=None), NULL), (dict(lengths=None), NULL), (dict(refs=None), NULL)]


@pytest.mark.parametrize("kw,status", POOL_REFUSALS + [
    (dict(table=0x20000), ALIAS), (dict(lengths=0x30000), ALIAS), (dict(refs=0x10000 + 8), ALIAS)])
def test_pool_refusals(lib, kw, status):
    pool = _pool(**kw)
    assert _fork(lib, pool) == status
    assert lib.kda_page_compact(ctypes.byref(pool), None, 0, None, 0x70000, 1 << 20, None) == status
    assert lib.kda_page_free(ctypes.byref(pool), 0x80000, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(it=3), DTYPE), (dict(m=-1), SHAPE), (dict(m=(1 << 24) + 1), UNSUPPORTED), (dict(m=(1 << 16) + 1), UNSUPPORTED), (dict(src=None), NULL),
    (dict(dst=None), NULL), (dict(status=None), NULL), (dict(ws=None), WORKSPACE), (dict(wb=8), WORKSPACE),
    (dict(ws=0x70002), LAYOUT),
    (dict(stores=((None, 256, 256),)), NULL), (dict(stores=((0x1000000, 255, 256),)), OVERLAP),
    (dict(stores=((0x1000000, 256, 0),)), SHAPE), (dict(stores=((0x1000000, 1 << 45, 256),)), SHAPE),
    (dict(stores=((0x1000000, 256, 256), (0x1000000 + 39 * 256, 256, 256))), ALIAS),
    (dict(stores=((0x1000000, 256, 256), (0x1000000 + 128, 256, 128))), ALIAS),
    (dict(stores=((0x10000 - 16, 64, 32),)), ALIAS), (dict(stores=((0x40000, 64, 32),)), ALIAS),
    (dict(status=0x70000), ALIAS), (dict(status=0x40000), ALIAS), (dict(ws=0x50000), ALIAS), (dict(dst=0x30000), ALIAS),
])
def test_fork_refusals(lib, kw, status):
    assert _fork(lib, **kw) == status


def test_page_calls_with_nothing_to_do(lib):
    assert _fork(lib, m=0, src=None, dst=None, status=None, ws=None) == 0
    assert lib.kda_page_fork(None, None, 0, 0x1000, 0x2000, 0, 1, 1, 0x3000, 0x4000, 64, None) == NULL
    assert lib.kda_page_compact(None, None, 0, None, None, 0, None) == NULL
    assert lib.kda_page_compact(ctypes.byref(_pool()), None, 0, None, None, 0, None) == WORKSPACE
    assert lib.kda_page_compact(ctypes.byref(_pool()), None, 0, 0x70000, 0x70000, 1 << 20, None) == ALIAS
    assert lib.kda_page_compact(ctypes.byref(_pool()), None, 1, None, 0x70000, 1 << 20, None) == NULL
    assert lib.kda_page_compact(ctypes.byref(_pool()), None, -1, None, 0x70000, 1 << 20, None) == SHAPE
    assert lib.kda_page_compact(ctypes.byref(_pool()), _stores((0x1000000, 8, 8)), 4097, None, 0x70000, 1 << 20,
                                None) == UNSUPPORTED
    assert lib.kda_page_free(ctypes.byref(_pool()), None, None) == NULL
    assert lib.kda_page_free(ctypes.byref(_pool()), 0x10000, None) == ALIAS
    assert lib.kda_page_fork_workspace_size(0, 8, 40, 1) == 0 and lib.kda_page_compact_workspace_size(0) == 0
    assert lib.kda_page_fork_workspace_size(3, 8, 40, 0) >= lib.kda_page_fork_workspace_size(3, 8, 40, 1) > 0


def test_bindings_refuse_host_tensors_and_missing_scale(lib):
    import torch
    import kda_recurrent_state_amd as kda
    x = torch.zeros(4, 2, 16, dtype=torch.bfloat16)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError):
        kda.kda_latent_prefill(x, x, x, cu)
    with pytest.raises(kda.KDAError):
        kda.kda_latent_decode(x, cu[None], cu, x)
    with pytest.raises(ValueError):
        kda.kda_page_free(cu[None], cu[:1], cu, cu[:1] > 0, 16)
