"""Host-side refusals of the 8-bit latent cache's and the shared-prefix decode's
entry points: bad arguments return the documented status before any HIP call
is made.  Only calls that fail validation, or that validate and enqueue
nothing, are made."""
import ctypes
import math

import pytest
import torch

from tests import latent8_ref as ref8
from tests.test_latent_cpu import (ALIAS, DTYPE, LAYOUT, NULL, OVERLAP, SHAPE, UNSUPPORTED, WORKSPACE, _set,  # noqa: F401
                                   lib)

BF16, F8, F32, I32, I64 = 1, 2, 0, 0, 1


def _store(**kw):
    from kda_recurrent_state_amd._lib import LatentStore
    base = dict(codes=0x100000, scales=0x200000, rope=0x300000, num_pages=10, page_size=16, L=64, R=16,
                codes_page_stride=16 * 64, scales_page_stride=16, rope_page_stride=16 * 16)
    return _set(LatentStore(), {**base, **kw})


BAD_STORES = [
    (dict(num_pages=0), SHAPE), (dict(page_size=0), SHAPE), (dict(L=0), SHAPE), (dict(R=-8), SHAPE),
    (dict(L=24), UNSUPPORTED), (dict(L=528, codes_page_stride=1 << 20), UNSUPPORTED), (dict(R=12), UNSUPPORTED),
    (dict(R=72, rope_page_stride=1 << 20), UNSUPPORTED), (dict(num_pages=1 << 27), UNSUPPORTED),
    (dict(num_pages=1 << 40), UNSUPPORTED),
    (dict(codes_page_stride=16 * 64 - 16), OVERLAP), (dict(scales_page_stride=15), OVERLAP),
    (dict(rope_page_stride=16 * 16 - 8), OVERLAP),
    (dict(codes_page_stride=16 * 64 + 8), LAYOUT), (dict(rope_page_stride=16 * 16 + 4), LAYOUT),
    (dict(codes_page_stride=1 << 45), SHAPE), (dict(scales_page_stride=1 << 45), SHAPE),
    (dict(codes=None), NULL), (dict(scales=None), NULL), (dict(rope=None), NULL),
    (dict(codes=0x100008), LAYOUT), (dict(scales=0x200002), LAYOUT), (dict(rope=0x300008), LAYOUT),
    (dict(scales=0x100100), ALIAS), (dict(rope=0x200010), ALIAS), (dict(rope=0x101000), ALIAS)]


@pytest.mark.parametrize("kw,status", BAD_STORES)
def test_store_refusals(lib, kw, status):  # noqa: F811
    s = ctypes.byref(_store(**kw))
    assert lib.kda_latent_quantize_scatter(s, 0x400000, 64, 0x500000, 16, BF16, 0x600000, I64, 5, None) == status
    assert lib.kda_latent_dequantize_gather(s, 0x600000, I64, 5, 0x700000, BF16, None) == status
    assert lib.kda_latent_quantize_scatter(s, 0x400000, 64, 0x500000, 16, BF16, 0x600000, I64, 0, None) == status


@pytest.mark.parametrize("change,status", [
    (dict(c=None), NULL), (dict(k_rope=None), NULL), (dict(slots=None), NULL), (dict(dtype=F8), DTYPE),
    (dict(dtype=5), DTYPE), (dict(index=2), DTYPE), (dict(n=-1), SHAPE), (dict(n=1 << 28), UNSUPPORTED),
    (dict(c_stride=60), LAYOUT), (dict(c_stride=-64), LAYOUT), (dict(k_rope_stride=20), LAYOUT),
    (dict(c=0x400008), LAYOUT), (dict(k_rope=0x500004), LAYOUT), (dict(c_stride=1 << 50), LAYOUT),
    (dict(c=0x100040), ALIAS), (dict(k_rope=0x300100), ALIAS), (dict(slots=0x200010), ALIAS),
    (dict(c=0x200000 - 64 * 4, dtype=F32), ALIAS)])
def test_quantize_scatter_refusals(lib, change, status):  # noqa: F811
    a = dict(c=0x400000, c_stride=64, k_rope=0x500000, k_rope_stride=16, dtype=BF16, slots=0x600000, index=I64, n=5)
    a.update(change)
    assert lib.kda_latent_quantize_scatter(ctypes.byref(_store()), a["c"], a["c_stride"], a["k_rope"], a["k_rope_stride"],
                                           a["dtype"], a["slots"], a["index"], a["n"], None) == status


@pytest.mark.parametrize("change,status", [
    (dict(out=None), NULL), (dict(slots=None), NULL), (dict(dtype=F8), DTYPE), (dict(index=7), DTYPE), (dict(n=-1), SHAPE),
    (dict(n=1 << 28), UNSUPPORTED), (dict(out=0x700008), LAYOUT), (dict(out=0x100000), ALIAS), (dict(out=0x300000), ALIAS),
    (dict(out=0x600000), ALIAS), (dict(out=0x200000 - 5 * 80 * 2 + 16), ALIAS)])
def test_dequantize_gather_refusals(lib, change, status):  # noqa: F811
    a = dict(out=0x700000, dtype=BF16, slots=0x600000, index=I64, n=5)
    a.update(change)
    assert lib.kda_latent_dequantize_gather(ctypes.byref(_store()), a["slots"], a["index"], a["n"], a["out"], a["dtype"],
                                            None) == status


def test_nothing_to_move_enqueues_nothing(lib):  # noqa: F811
    s = ctypes.byref(_store())
    assert lib.kda_latent_quantize_scatter(s, None, 0, None, 0, BF16, None, I32, 0, None) == 0
    assert lib.kda_latent_dequantize_gather(s, None, I32, 0, None, F32, None) == 0
    assert lib.kda_latent_quantize_scatter(None, None, 0, None, 0, BF16, None, I32, 0, None) == NULL
    assert lib.kda_latent_dequantize_gather(None, None, I32, 0, None, F32, None) == NULL


def _decode(**kw):
    from kda_recurrent_state_amd._lib import LatentSharedArgs
    base = dict(N=4, Q=2, H=8, L=64, R=16, G=2, cache_dtype=F8, cache=0x100000, scales=0x200000, rope=0x300000,
                num_pages=10, page_size=16, page_stride=16 * 64, scales_page_stride=16, rope_page_stride=16 * 16,
                page_table=0x400000, table_stride=8, max_pages=8, lengths=0x410000, cu_groups=0x420000, shared=0x430000,
                q=0x500000, q_stride=(2 * 8 * 64, 8 * 64, 64), q_rope=0x600000, q_rope_stride=(2 * 8 * 16, 8 * 16, 16),
                out=0x700000, lse=0x800000, scale=0.1, workspace=0x10000000, workspace_bytes=1 << 40)
    return _set(LatentSharedArgs(), {**base, **kw})


WIDE = dict(cache_dtype=BF16, cache=0x100000, page_stride=16 * 80)


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), SHAPE), (dict(Q=0), SHAPE), (dict(H=0), SHAPE), (dict(L=0), SHAPE), (dict(R=-8), SHAPE), (dict(G=-1), SHAPE),
    (dict(num_pages=0), SHAPE), (dict(page_size=0), SHAPE), (dict(max_pages=0), SHAPE),
    (dict(cache_dtype=F32), DTYPE), (dict(cache_dtype=3), DTYPE),
    (dict(L=24), UNSUPPORTED), (dict(L=520), UNSUPPORTED), (dict(R=4), UNSUPPORTED), (dict(R=72), UNSUPPORTED),
    (dict(Q=1025), UNSUPPORTED), (dict(Q=32, H=33), UNSUPPORTED), (dict(N=65536), UNSUPPORTED), (dict(G=65536), UNSUPPORTED),
    (dict(scale=0.0), UNSUPPORTED), (dict(scale=math.nan), UNSUPPORTED), (dict(scale=3e38), UNSUPPORTED),
    (dict(max_pages=1 << 27), UNSUPPORTED), (dict(N=65535, H=512, max_pages=1 << 20, table_stride=1 << 20), UNSUPPORTED),
    (dict(num_pages=1 << 27), UNSUPPORTED),
    # page strides of 2^32 bytes: the arrays would overlap, or lie apart
    (dict(page_stride=1 << 32), ALIAS), (dict(scales_page_stride=1 << 30), ALIAS), (dict(rope_page_stride=1 << 31), UNSUPPORTED),
    (dict(page_stride=1 << 32, cache=1 << 44), UNSUPPORTED), (dict(scales_page_stride=1 << 30, scales=1 << 44), UNSUPPORTED),
    (dict(**{**WIDE, "page_stride": 1 << 31, "cache": 1 << 44}), UNSUPPORTED),
    (dict(table_stride=7), OVERLAP), (dict(table_stride=1 << 45), SHAPE),
    (dict(page_stride=16 * 64 - 16), OVERLAP), (dict(scales_page_stride=15), OVERLAP), (dict(page_stride=16 * 64 + 8), LAYOUT),
    (dict(**{**WIDE, "page_stride": 16 * 80 - 8}), OVERLAP), (dict(**{**WIDE, "page_stride": 16 * 80 + 4}), LAYOUT),
    (dict(**{**WIDE, "page_stride": 1 << 45}), SHAPE), (dict(**{**WIDE, "cache": 0x100004}), LAYOUT),
    (dict(**{**WIDE, "cache": None}), NULL), (dict(**{**WIDE, "L": 20}), UNSUPPORTED),
    (dict(cache=None), NULL), (dict(scales=None), NULL), (dict(rope=None), NULL), (dict(page_table=None), NULL),
    (dict(lengths=None), NULL), (dict(q=None), NULL), (dict(q_rope=None), NULL), (dict(out=None), NULL),
    (dict(cu_groups=None), NULL), (dict(shared=None), NULL),
    (dict(q_stride=(1024, 512, 60)), LAYOUT), (dict(q_stride=(-1024, 512, 64)), LAYOUT), (dict(q=0x500008), LAYOUT),
    (dict(q_rope_stride=(256, 128, 12)), LAYOUT), (dict(q_rope=0x600002), LAYOUT), (dict(out=0x700008), LAYOUT),
    (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=64), WORKSPACE), (dict(workspace=0x10000008), LAYOUT),
    (dict(out=0x100000), ALIAS), (dict(out=0x300010), ALIAS), (dict(out=0x500000), ALIAS), (dict(lse=0x410000), ALIAS),
    (dict(lse=0x700000), ALIAS), (dict(workspace=0x80000), ALIAS), (dict(out=0x420000), ALIAS), (dict(lse=0x430000), ALIAS),
    (dict(**{**WIDE, "out": 0x100800}), ALIAS)])
def test_decode_shared_refusals(lib, kw, status):  # noqa: F811
    assert lib.kda_latent_decode_shared(ctypes.byref(_decode(**kw)), None) == status


def test_decode_fp8_refusals(lib):  # noqa: F811
    run = lib.kda_latent_decode_fp8
    assert run(None, None) == NULL and lib.kda_latent_decode_shared(None, None) == NULL
    assert run(ctypes.byref(_decode()), None) == SHAPE                                  # groups
    assert run(ctypes.byref(_decode(G=0, **WIDE)), None) == DTYPE
    assert run(ctypes.byref(_decode(G=0, scales=None)), None) == NULL
    assert run(ctypes.byref(_decode(G=0, workspace_bytes=4096)), None) == WORKSPACE
    assert run(ctypes.byref(_decode(G=0, N=0, page_table=None, q=None, out=None, workspace=None)), None) == 0
    assert lib.kda_latent_decode_shared(ctypes.byref(_decode(N=0, q=None)), None) == 0
    assert lib.kda_latent_decode_shared(ctypes.byref(_decode(N=0, q=None, lengths=None, **WIDE)), None) == 0


def test_workspace_sizes(lib):  # noqa: F811
    size = lib.kda_latent_shared_workspace_size
    for bad in ((0, 1, 8, 512, 0), (1, 0, 8, 512, 0), (1, 1, 0, 512, 0), (1, 1, 8, 0, 0), (1, 1, 8, 512, -1), (65536, 1, 8, 512, 0),
                (1, 1025, 1, 512, 0), (1, 32, 33, 512, 0), (1, 1, 8, 520, 0), (1, 1, 8, 512, 65536)):
        assert size(*bad) == 0, bad
    # two pieces a share of 16 query rows: 512 x 16 x (512 + 2) numbers at least
    assert size(1, 1, 8, 512, 0) >= 512 * 16 * 514 * 4
    # with groups also a row block's worth for each sequence and for the prefixes
    assert size(64, 1, 16, 512, 1) >= (512 + 64 + 16) * 64 * 514 * 4
    assert size(200, 1, 16, 512, 0) < size(200, 1, 16, 512, 3)


def test_shared_calls_need_their_groups():
    import kda_recurrent_state_amd as kda
    with pytest.raises(kda.KDAError):
        kda.kda_latent_decode_shared(None, None, None, None, None, None, scale=1.0)


def test_reference_codes():
    """The oracle's own codes: e4m3's values, the scale's rule at its edges and a hand-worked row."""
    v = ref8.VALUES
    assert v[0x7e] == 448 and v[0x08] == 2.0 ** -6 and v[0x01] == 2.0 ** -9 and v[0x80] == 0 and math.isnan(v[0x7f])
    assert torch.equal(v[:127], torch.sort(v[:127]).values)
    x = torch.tensor([[448.0, 0.0], [448.5, 0.0], [449.0, 1.0], [0.0, 0.0], [2.0 ** -140, 0.0], [3e38, 1.0]],
                     dtype=torch.float64)
    codes, scales = ref8.quantize(x)
    assert scales.tolist()[:3] == [1, 2, 2] and scales[3] == 2.0 ** -126 and scales[4] == 2.0 ** -126
    assert (x[:, 0] / scales <= 448).all() and (x[[0, 1, 2, 5], 0] / scales[[0, 1, 2, 5]] > 224).all()
    codes, scales = ref8.quantize(torch.tensor([[-400.0, 1.0625, 1.1875, 0.0009765625, -0.003]], dtype=torch.float64))
    # scale 1; ties 1.0625 -> 1 (even), 1.1875 -> 1.25 (even), 2^-10 -> 0 (even), -0.003 -> -2 2^-9
    assert scales[0] == 1 and codes[0].tolist() == [0x80 | 0x7c, 0x38, 0x3a, 0x00, 0x82]
