"""The 8-bit latent cache (written, read back, attended to) and latent decode
over shared prefixes on the GPU, against plain fp64 evaluations."""
import math

import pytest
import torch

from tests import latent8_ref as ref8
from tests import latent_ref as ref
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16
F8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _empty_store(pages, page, L, R, gap=False):
    """A cache whose bytes are all set to something; with ``gap`` the pages are views of longer ones."""
    more = 2 if gap else 1
    codes = torch.full((pages, more * page * L), 0x55, dtype=torch.uint8, device="cuda")
    scales = torch.full((pages, more * page), -7.0, device="cuda")
    rope = torch.full((pages, more * page * R), 3.0, dtype=BF16, device="cuda") if R else None
    return (codes[:, : page * L].unflatten(1, (page, L)), scales[:, :page],
            rope[:, : page * R].unflatten(1, (page, R)) if R else None)


def _rows(T, L, R, dtype, seed):
    """Rows of many sizes, with a zero row, ties, subnormal codes, the largest and the smallest magnitudes."""
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn(T, L, generator=gen) * torch.exp2(torch.randint(-20, 20, (T, 1), generator=gen).float())
    x[:, ::5] *= 2.0 ** -9
    if T > 4:
        x[0] = 0
        x[1] = torch.arange(L).float() * 0.5 + 0.25         # ties on the grid below 2^6
        x[2] = torch.where(torch.arange(L) % 2 == 0, 3e38, 1e-38)
        x[3] = 1e-39                                          # below the smallest scale's normal codes
        x[4] = 448.0                                          # exactly the largest code
        x[4, 0] = 447.9
    x = torch.cat([x, torch.randn(T, R, generator=gen)], 1).to(dtype).cuda()
    return x[:, :L], x[:, L:] if R else None


@pytest.mark.parametrize("T,L,R,page,dtype,index,gap", [
    (1, 512, 64, 64, BF16, torch.int64, False), (37, 512, 64, 16, BF16, torch.int32, True),
    (200, 256, 32, 1, torch.float32, torch.int64, False), (75, 128, 64, 48, BF16, torch.int32, False),
    (33, 384, 0, 64, torch.float32, torch.int32, True), (64, 16, 8, 7, BF16, torch.int64, False),
    (50, 272, 56, 5, BF16, torch.int64, True), (9, 512, 0, 128, torch.float32, torch.int64, False),
    (5000, 512, 64, 64, BF16, torch.int64, False), (20011, 128, 64, 16, torch.float32, torch.int32, False)])
def test_written_rows(T, L, R, page, dtype, index, gap):
    import kda_recurrent_state_amd as kda
    pages = T // page + 3
    codes, scales, rope = _empty_store(pages, page, L, R, gap)
    whole = [x._base if gap else x for x in (codes, scales, rope) if x is not None]
    before = [x.cpu().clone() for x in whole]
    c, k_rope = _rows(T, L, R, dtype, T)
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(1))[:T]
    bad = torch.arange(T) % 7 == 6
    slots[bad] = torch.tensor([-1, pages * page, -(2 ** 31), 2 ** 31 - 1])[torch.arange(int(bad.sum())) % 4]
    kda.kda_latent_quantize_scatter(c, k_rope, slots.to(index).cuda(), codes.view(F8), scales, rope)
    want, scale = ref8.quantize(c.cpu().double())
    at = slots[~bad]
    hit = torch.zeros(pages * page, dtype=torch.bool)
    hit[at] = True
    got = codes.cpu().reshape(-1, L), scales.cpu().reshape(-1), rope.cpu().reshape(-1, R) if R else None
    # every code's value, and its sign
    assert torch.equal(got[0][at], want[~bad])
    assert torch.equal(got[1][at].double(), scale[~bad])
    assert (got[0][~hit] == 0x55).all() and (got[1][~hit] == -7).all()
    if R:
        assert torch.equal(got[2][at], k_rope.to(BF16).cpu()[~bad]) and (got[2][~hit] == 3).all()
    if gap:  # nothing between the pages
        for x, y, n in zip(whole, before, (page * L, page, page * R)):
            assert torch.equal(x.cpu()[:, n:], y[:, n:])


def test_rows_that_are_not_finite():
    import kda_recurrent_state_amd as kda
    codes, scales, rope = _empty_store(2, 4, 128, 8)
    c = torch.randn(5, 128).to(BF16)
    k_rope = torch.randn(5, 8).to(BF16)
    c[1, 3], c[2, 127], c[3, 0] = math.nan, math.inf, -math.inf
    k_rope[4, 2] = math.nan
    kda.kda_latent_quantize_scatter(c.cuda(), k_rope.cuda(), _i32([0, 1, 2, 3, 4]), codes, scales, rope)
    assert torch.equal(scales.view(-1)[:5].isnan().cpu(), torch.tensor([False, True, True, True, False]))
    assert (codes.view(-1, 128)[1:4] == 0).all()
    out = kda.kda_latent_dequantize_gather(codes, scales, rope, _i32([0, 1, 2, 3, 4])).cpu()
    assert out[1:4, :128].isnan().all() and not out[[0, 4], :128].isnan().any()
    assert torch.equal(out[:, 128:].isnan(), k_rope.isnan())


@pytest.mark.parametrize("S,L,R,page,dtype,index", [
    (1, 512, 64, 64, BF16, torch.int64), (39, 256, 32, 16, torch.float32, torch.int32), (300, 128, 64, 1, BF16, torch.int32),
    (77, 384, 0, 48, BF16, torch.int64), (20, 16, 8, 3, torch.float32, torch.int64), (9000, 512, 64, 64, BF16, torch.int64),
    (18001, 128, 8, 64, torch.float32, torch.int32)])
def test_read_rows(S, L, R, page, dtype, index):
    """Any scales, and the same slot many times."""
    import kda_recurrent_state_amd as kda
    gen = torch.Generator().manual_seed(S)
    pages = 11
    codes = torch.randint(0, 255, (pages, page, L), generator=gen).to(torch.uint8)
    codes[(codes & 127) == 127] = 1
    scales = torch.rand(pages, page, generator=gen) + 0.1
    rope = torch.randn(pages, page, R, generator=gen).to(BF16) if R else None
    slots = torch.randint(-3, pages * page + 3, (S,), generator=gen)
    out = kda.kda_latent_dequantize_gather(codes.cuda().view(F8), scales.cuda(), None if rope is None else rope.cuda(),
                                           slots.to(index).cuda(), dtype=dtype)
    fine = (slots >= 0) & (slots < pages * page)
    at = slots.clamp(0, pages * page - 1)
    want = (ref8.VALUES[codes.long()].float() * scales[..., None]).view(-1, L)[at]
    if R:
        want = torch.cat([want, rope.float().view(-1, R)[at]], 1)
    assert torch.equal(out.cpu(), torch.where(fine[:, None], want, 0.0).to(dtype))


def test_written_and_read_and_written_again():
    """Powers of two as scales: reading to bf16 is exact, so the second cache holds the same values."""
    import kda_recurrent_state_amd as kda
    c, k_rope = _rows(300, 512, 64, BF16, 3)
    a, b = _empty_store(5, 64, 512, 64), _empty_store(5, 64, 512, 64)
    slots = torch.arange(300, device="cuda")
    kda.kda_latent_quantize_scatter(c, k_rope, slots, *a)
    rows = kda.kda_latent_dequantize_gather(*a, slots)
    assert torch.equal(rows.cpu().double(), ref8.values(*a).view(-1, 576)[:300])
    kda.kda_latent_quantize_scatter(rows[:, :512], rows[:, 512:], slots, *b)
    assert torch.equal(ref8.values(*b), ref8.values(*a))


# --- decode -----------------------------------------------------------------

def _cache8(gen, pages, page, L, R, spread=1.0):
    """A cache in 8 bits (CPU tensors) whose rows' scales are any numbers."""
    x = torch.randn(pages * page, L, generator=gen) * torch.exp2(spread * torch.randn(pages * page, 1, generator=gen))
    codes, scales = ref8.quantize(x.double())
    scales = scales.float() * (0.75 + 0.5 * torch.rand(pages * page, generator=gen))
    return (codes.view(pages, page, L), scales.view(pages, page),
            torch.randn(pages, page, R, generator=gen).to(BF16) if R else None)


def _gpu(store):
    return tuple(None if x is None else x.cuda() for x in store)


def _queries(gen, N, Q, H, L, R):
    return (torch.randn(N, Q, H, L, generator=gen).to(BF16), torch.randn(N, Q, H, R, generator=gen).to(BF16) if R else None)


def _table(gen, lens, page, extra=2, more=0):
    """A table whose pages lie anywhere, -1 behind the lengths; (table, number of pages)."""
    used = [max(0, -(-n // page)) for n in lens]
    pages = sum(used) + extra
    perm = torch.randperm(pages, generator=gen).tolist()
    table = torch.full((len(lens), max(used + [1]) + more), -1, dtype=torch.int32)
    at = 0
    for n, u in enumerate(used):
        table[n, :u] = torch.tensor(perm[at: at + u], dtype=torch.int32)
        at += u
    return table, pages


SCALE = 192 ** -0.5


@pytest.mark.parametrize("lens,Q,H,L,R,page", [
    ([1], 1, 1, 512, 64, 64), ([4000], 1, 32, 512, 64, 64), ([64, 65, 63, 128, 1, 0, 700], 1, 16, 512, 64, 16),
    ([300, 0, 17, 2, 1], 3, 20, 512, 64, 48), ([5000, 20], 2, 64, 512, 64, 64), ([900, 900, 30], 1, 128, 512, 64, 128),
    ([200, 129], 1, 8, 256, 32, 1), ([513, 64, 7], 2, 24, 256, 64, 16), ([333, 40], 1, 40, 128, 64, 5),
    ([1000, 10], 1, 17, 384, 0, 64), ([77, 640], 4, 33, 16, 8, 16), ([150], 1, 5, 272, 56, 7), ([222, 3], 1, 3, 128, 0, 3),
    ([90, 0, 0, 12], 1, 48, 256, 0, 64), ([0, 0], 2, 8, 512, 64, 64), ([2000] * 40, 1, 16, 512, 64, 64),
    ([30] * 300, 1, 8, 128, 64, 16)])
def test_decode8(lens, Q, H, L, R, page):
    import kda_recurrent_state_amd as kda
    gen = torch.Generator().manual_seed(len(lens) + H)
    table, pages = _table(gen, lens, page)
    store = _cache8(gen, pages, page, L, R)
    q, q_rope = _queries(gen, len(lens), Q, H, L, R)
    out, lse = kda.kda_latent_decode_fp8(*_gpu(store), table.cuda(), _i32(lens), q.cuda(),
                                         None if q_rope is None else q_rope.cuda(), scale=SCALE, with_lse=True)
    rows = ref8.values(*store)
    ref8.check(out, lse, ref8.decode(rows, table, torch.tensor(lens), q, q_rope, SCALE),
               ref8.score_error(rows, q, SCALE), "decode8")


def test_decode8_bad_pages_and_lengths():
    """Pages outside the cache are not seen, lengths are clamped, and what lies in rows that nobody sees does not matter."""
    import kda_recurrent_state_amd as kda
    gen = torch.Generator().manual_seed(5)
    lens, page = [200, 130, -5, 5000, 64], 32
    table, pages = _table(gen, [200, 130, 0, 224, 64], page)
    store = _cache8(gen, pages, page, 512, 64)
    table[0, 2], table[0, 6], table[1, :] = -1, pages, 2 ** 30
    table[4, 0] = -(2 ** 31)
    seen = torch.zeros(pages * page, dtype=torch.bool)
    for n, length in enumerate([200, 130, 0, 224, 64]):
        for j in range(length):
            if 0 <= table[n, j // page] < pages:
                seen[table[n, j // page] * page + j % page] = True
    store[1].view(-1)[~seen] = math.nan
    store[2].view(-1, 64)[~seen] = math.nan
    q, q_rope = _queries(gen, 5, 1, 24, 512, 64)
    out, lse = kda.kda_latent_decode_fp8(*_gpu(store), table.cuda(), _i32(lens), q.cuda(), q_rope.cuda(), scale=SCALE,
                                         with_lse=True)
    rows = ref8.values(*store).nan_to_num(0)
    ref8.check(out, lse, ref8.decode(rows, table, torch.tensor(lens), q, q_rope, SCALE),
               ref8.score_error(rows, q, SCALE), "bad pages")
    assert (out[1] == 0).all() and (out[2] == 0).all() and (lse[1] == -math.inf).all()


@pytest.mark.parametrize("what", ["scale", "rope"])
def test_decode8_row_that_is_not_finite_reaches_who_sees_it(what):
    """The last token of a sequence, with three query tokens: only the last one sees it; other sequences do not."""
    import kda_recurrent_state_amd as kda
    gen = torch.Generator().manual_seed(8)
    lens, page = [150, 90], 16
    table, pages = _table(gen, lens, page)
    store = _cache8(gen, pages, page, 512, 64)
    q, q_rope = _queries(gen, 2, 3, 12, 512, 64)
    rows = ref8.values(*store)
    want = ref8.decode(rows, table, torch.tensor(lens), q, q_rope, SCALE)
    place = table[0, 149 // page], 149 % page
    if what == "scale":
        store[1][place] = math.nan
    else:
        store[2][place][5] = math.nan
    out, lse = kda.kda_latent_decode_fp8(*_gpu(store), table.cuda(), _i32(lens), q.cuda(), q_rope.cuda(), scale=SCALE,
                                         with_lse=True)
    assert out[0, 2].isnan().all()
    delta = ref8.score_error(rows, q, SCALE)
    ref8.check(out[0, :2], lse[0, :2], [x[0, :2] for x in want], delta, "before it")
    ref8.check(out[1], lse[1], [x[1] for x in want], delta, "beside it")


# --- shared prefixes ----------------------------------------------------------

def _shared_inputs(gen, groups, page, L, R, fp8, Q, H, alone=()):
    """groups: (shared tokens, [lengths]); ``alone``: lengths of sequences of no group, before and behind.  Whole pages
    of the prefix are the same, the page that the prefix ends in is copied row by row up to there."""
    lens, cu, shared = list(alone[:1]), [len(alone[:1])], []
    for s, ls in groups:
        lens += ls
        cu.append(len(lens))
        shared.append(s)
    lens += list(alone[1:])
    table, pages = _table(gen, lens, page)
    if fp8:
        store = _cache8(gen, pages, page, L, R)
    else:
        store = (torch.randn(pages, page, L + R, generator=gen).to(BF16),)
    for g, (s, ls) in enumerate(groups):
        for n in range(cu[g] + 1, cu[g + 1]):
            for j in range(min(s, lens[n], lens[cu[g]])):
                a, b = int(table[cu[g], j // page]), int(table[n, j // page])
                if j % page == 0 and min(s, lens[n], lens[cu[g]]) - j >= page:
                    table[n, j // page] = a
                elif a != b:
                    for x in store:
                        if x is not None:
                            x[b, j % page] = x[a, j % page]
    q, q_rope = _queries(gen, len(lens), Q, H, L, R)
    return store, table, lens, cu, shared, q, q_rope


def _run_shared(store, table, lens, cu, shared, q, q_rope, **kw):
    import kda_recurrent_state_amd as kda
    cache = _gpu(store) if len(store) == 3 else store[0].cuda()
    return kda.kda_latent_decode_shared(cache, table.cuda(), _i32(lens), _i32(cu), _i32(shared), q.cuda(),
                                        None if q_rope is None else q_rope.cuda(), scale=SCALE, with_lse=True, **kw)


def _check_shared(store, table, lens, q, q_rope, got, name):
    fp8 = len(store) == 3
    rows = ref8.values(*store) if fp8 else store[0].double()
    want = ref8.decode(rows, table, torch.tensor(lens), q, q_rope, SCALE)
    ref8.check(*got, want, ref8.score_error(rows, q, SCALE) if fp8 else 0.0, name)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("groups,alone,Q,H,L,R,page", [
    ([(128, [130, 200])], (), 1, 8, 512, 64, 64),
    ([(2000, [2001, 2100, 2000, 2500])], (), 1, 16, 512, 64, 64),
    ([(100, [150, 101, 100, 333]), (64, [64, 64]), (0, [70, 80]), (500, [501])], (40, 300, 0), 1, 20, 512, 64, 16),
    ([(333, [400, 333, 500]), (777, [900, 778, 800, 779, 1000])], (5, 1), 3, 12, 256, 32, 48),
    ([(50, [60, 20, 0, 55])], (), 2, 33, 128, 64, 5),          # shorter than what is shared, and empty
    ([(50, [10, 60, 51])], (), 1, 7, 128, 0, 1),                # the first one is the short one
    ([(1000, [0, 1100, 1200])], (), 1, 16, 384, 0, 64),         # the first one is empty: nothing shared
    ([(4096, [4097 + i for i in range(40)])], (), 1, 16, 512, 64, 64),
    ([(4096, [4100, 4200, 4300])], (3000,), 2, 128, 512, 64, 64),
    ([(20000, [20010, 20400])], (), 1, 3, 512, 64, 128),
    ([(640, [700] * 5)] * 12, (), 1, 64, 272, 56, 16)])
def test_shared(groups, alone, Q, H, L, R, page, fp8):
    gen = torch.Generator().manual_seed(H + page)
    if fp8 and L % 16:
        pytest.skip("the 8-bit cache has L in multiples of 16")
    store, table, lens, cu, shared, q, q_rope = _shared_inputs(gen, groups, page, L, R, fp8, Q, H, alone)
    got = _run_shared(store, table, lens, cu, shared, q, q_rope)
    _check_shared(store, table, lens, q, q_rope, got, "shared")
