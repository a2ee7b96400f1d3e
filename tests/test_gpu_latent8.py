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


@pytest.mark.parametrize("T,L,R,page,dtype", [(60001, 512, 64, 64, BF16), (87501, 128, 64, 16, torch.float32),
                                              (64007, 256, 8, 64, torch.float32)])
def test_written_rows_of_a_large_batch(T, L, R, page, dtype):
    """Inputs of more than 64 MiB: 1999 rows many times over."""
    import kda_recurrent_state_amd as kda
    pages = T // page + 3
    codes, scales, rope = _empty_store(pages, page, L, R)
    c, k_rope = _rows(1999, L, R, dtype, T)
    row = (torch.arange(T) * 17 + 3) % 1999
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(2))[:T]
    bad = torch.arange(T) % 11 == 5
    slots[bad] = -1
    want, scale = ref8.quantize(c.cpu().double())
    kda.kda_latent_quantize_scatter(c[row.cuda()], k_rope[row.cuda()], slots.cuda(), codes, scales, rope)
    at, row = slots[~bad], row[~bad]
    hit = torch.zeros(pages * page, dtype=torch.bool)
    hit[at] = True
    got = codes.cpu().view(-1, L), scales.cpu().view(-1), rope.cpu().view(-1, R)
    assert torch.equal(got[0][at], want[row]) and torch.equal(got[1][at].double(), scale[row])
    assert torch.equal(got[2][at], k_rope.to(BF16).cpu()[row])
    assert (got[0][~hit] == 0x55).all() and (got[1][~hit] == -7).all() and (got[2][~hit] == 3).all()


def _at_the_ends(n, border):
    """Rows of a call of n: its first and last ones, and those around ``border``, where a second launch begins."""
    return torch.cat([torch.arange(4), torch.arange(border - 4, border + 4), torch.arange(n - 4, n)])


@pytest.mark.parametrize("n,L,R,index,dtype,rows", [
    ((1 << 27) + 5, 272, 8, torch.int32, BF16, 8), ((1 << 28) - 1, 144, 0, torch.int64, BF16, 16),
    ((1 << 26) + 5, 272, 8, torch.int32, torch.float32, 4)])
def test_written_rows_of_the_largest_calls(n, L, R, index, dtype, rows):
    """More rows than a launch of fewer than 2^32 threads takes, of ``rows`` a workgroup of 256.  The input's
    rows overlap (one begins 8 values behind the one before), and few of them are written."""
    import kda_recurrent_state_amd as kda
    at = _at_the_ends(n, ((1 << 24) - 1) * rows)
    codes, scales, rope = _empty_store(3, 16, L, R)
    base = torch.arange(1009, device="cuda").to(dtype).repeat((8 * n + L) // 1009 + 1)
    c = torch.as_strided(base, (n, L), (8, 1))
    k_rope = torch.as_strided(base, (n, R), (8, 1)) if R else None
    slots = torch.full((n,), -1, dtype=index, device="cuda")
    places = torch.randperm(48, generator=torch.Generator().manual_seed(1))[: len(at)]
    slots[at.cuda()] = places.to(index).cuda()
    kda.kda_latent_quantize_scatter(c, k_rope, slots, codes, scales, rope)
    rows = torch.stack([c[int(t)] for t in at]).cpu()
    want, scale = ref8.quantize(rows.double())
    hit = torch.zeros(48, dtype=torch.bool)
    hit[places] = True
    got = codes.cpu().view(-1, L), scales.cpu().view(-1)
    assert torch.equal(got[0][places], want) and torch.equal(got[1][places].double(), scale)
    assert (got[0][~hit] == 0x55).all() and (got[1][~hit] == -7).all()
    if R:
        assert torch.equal(rope.cpu().view(-1, R)[places], rows[:, :R].to(BF16)) and (rope.cpu().view(-1, R)[~hit] == 3).all()
    del base, c, k_rope, slots
    torch.cuda.empty_cache()


def test_read_rows_of_the_largest_calls():
    """The same of reading; most entries are no slot and give zeros."""
    import kda_recurrent_state_amd as kda
    n, L = (1 << 27) + 5, 272
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("needs 75 GB for the rows")
    gen = torch.Generator().manual_seed(4)
    at = _at_the_ends(n, ((1 << 24) - 1) * 8)
    codes, scales, _ = _cache8(gen, 3, 16, L, 0)
    places = torch.randint(0, 48, (len(at),), generator=gen)
    slots = torch.full((n,), -1, dtype=torch.int32, device="cuda")
    slots[at.cuda()] = places.int().cuda()
    out = kda.kda_latent_dequantize_gather(codes.cuda(), scales.cuda(), None, slots)
    want = (ref8.VALUES[codes.long()].float() * scales[..., None]).to(BF16).view(-1, L)[places]
    assert torch.equal(torch.stack([out[int(t)] for t in at]).cpu(), want)
    for t in at:
        out[int(t)].zero_()
    for part in out.split(1 << 23):
        assert not part.view(torch.int32).any()
    del out, part, slots
    torch.cuda.empty_cache()


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


def test_slots_that_are_rows_in_their_low_32_bits_alone():
    import kda_recurrent_state_amd as kda
    store = _empty_store(2, 16, 128, 8)
    c, k_rope = _rows(9, 128, 8, BF16, 7)
    slots = torch.tensor([3, 2 ** 32 + 4, -2 ** 32 + 5, 2 ** 62, -2 ** 62, 2 ** 62 + 6, -2 ** 62 + 7, 2 ** 63 - 1, 8])
    fine = torch.tensor([True] + [False] * 7 + [True])
    kda.kda_latent_quantize_scatter(c, k_rope, slots.cuda(), *store)
    want, _ = ref8.quantize(c.cpu().double())
    got, at = store[0].cpu().view(-1, 128), slots[fine]
    rest = torch.ones(32, dtype=torch.bool)
    rest[at] = False
    assert torch.equal(got[at], want[fine]) and (got[rest] == 0x55).all()
    assert (store[1].cpu().view(-1)[rest] == -7).all() and (store[2].cpu().view(-1, 8)[rest] == 3).all()
    rows = kda.kda_latent_dequantize_gather(*store, slots.cuda()).cpu()
    assert (rows[~fine] == 0).all()
    assert torch.equal(rows[fine].double(), ref8.values(*store).view(-1, 136)[at])


def test_rows_of_the_smallest_magnitudes():
    """fp32 rows down to the smallest subnormals, whose scale is 2^-126 to 2^-124: the fp32 read is exact, the bf16 read
    its rounding (a code can be worth 2^-135, bf16 ends at 2^-133), exact from the scale 2^-124 on; and rows whose small
    values lie 2^-13 below the largest keep four bits."""
    import kda_recurrent_state_amd as kda
    gen = torch.Generator().manual_seed(6)
    exps = torch.arange(-149, -114, dtype=torch.float64)
    x = torch.randn(len(exps), 128, generator=gen, dtype=torch.float64) * torch.exp2(exps)[:, None]
    x[-1] = 2.0 ** -117 * 225                                   # a largest one just above 224 scales
    x[-1, 1:] *= 2.0 ** -13 * (1 + torch.rand(127, generator=gen, dtype=torch.float64))
    x = x.float()
    store = _empty_store(4, 16, 128, 0)[:2]
    slots = torch.arange(len(x), device="cuda")
    kda.kda_latent_quantize_scatter(x.cuda(), None, slots, *store)
    codes, scales = ref8.quantize(x.double())
    assert torch.equal(store[0].cpu().view(-1, 128)[:len(x)], codes)
    assert torch.equal(store[1].cpu().view(-1)[:len(x)].double(), scales)
    want = ref8.VALUES[codes.long()] * scales[:, None]          # multiples of 2^-135: fp32 holds them
    assert torch.equal(want.float().double(), want)
    assert ((want[-1] - x[-1].double()).abs() <= 2.0 ** -4 * x[-1].double().abs()).all()
    assert torch.equal(kda.kda_latent_dequantize_gather(*store, None, slots, dtype=torch.float32).cpu(), want.float())
    got = kda.kda_latent_dequantize_gather(*store, None, slots).cpu()
    assert torch.equal(got, want.float().to(BF16))
    fine = scales >= 2.0 ** -124
    assert fine.any() and torch.equal(got[fine].double(), want[fine])
    assert not torch.equal(got[~fine].double(), want[~fine])


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
    ref.check(out, lse, ref.decode(rows, table, torch.tensor(lens), q, q_rope, SCALE), "decode8")


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
    ref.check(out, lse, ref.decode(rows, table, torch.tensor(lens), q, q_rope, SCALE), "bad pages")
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
    want = ref.decode(rows, table, torch.tensor(lens), q, q_rope, SCALE)
    place = table[0, 149 // page], 149 % page
    if what == "scale":
        store[1][place] = math.nan
    else:
        store[2][place][5] = math.nan
    out, lse = kda.kda_latent_decode_fp8(*_gpu(store), table.cuda(), _i32(lens), q.cuda(), q_rope.cuda(), scale=SCALE,
                                         with_lse=True)
    assert out[0, 2].isnan().all()
    ref.check(out[0, :2], lse[0, :2], [x[0, :2] for x in want], "before it")
    ref.check(out[1], lse[1], [x[1] for x in want], "beside it")


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
    rows = ref8.values(*store) if len(store) == 3 else store[0].double()
    ref.check(*got, ref.decode(rows, table, torch.tensor(lens), q, q_rope, SCALE), name)


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


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Q,H", [(1, 130), (5, 64), (2, 257), (7, 100), (3, 241), (1, 1024)])
def test_shared_rows_of_many_blocks(Q, H, fp8):
    """3, 5, 9, 11, 12 and 16 blocks of 64 query rows a sequence; a prefix's blocks are no multiple of those."""
    gen = torch.Generator().manual_seed(Q * H)
    groups, alone = [(700, [800, 720, 705, 700, 1200]), (64, [70, 200]), (130, [131, 150, 10])], (300, 0, 1)
    store, table, lens, cu, shared, q, q_rope = _shared_inputs(gen, groups, 16, 128, 64, fp8, Q, H, alone)
    got = _run_shared(store, table, lens, cu, shared, q, q_rope)
    _check_shared(store, table, lens, q, q_rope, got, "many blocks")
    got = _run_shared(store, table, lens, [0], [], q, q_rope)
    _check_shared(store, table, lens, q, q_rope, got, "many blocks, no groups")


@pytest.mark.parametrize("L,R", [(8, 0), (8, 56), (24, 8), (136, 0), (136, 64), (504, 56), (504, 0)])
@pytest.mark.parametrize("groups,Q,H", [
    ([(100, [130, 101])], 1, 8), ([(70, [71, 200])], 2, 8), ([(200, [260, 201, 199]), (64, [65, 300])], 1, 24)])
def test_shared_dims_of_8_more_than_16s(groups, Q, H, L, R):
    """The 16-bit cache takes any multiple of 8; with 1, 2 and 4 blocks of 16 query rows a workgroup."""
    gen = torch.Generator().manual_seed(L + R)
    store, table, lens, cu, shared, q, q_rope = _shared_inputs(gen, groups, 16, L, R, False, Q, H)
    got = _run_shared(store, table, lens, cu, shared, q, q_rope)
    _check_shared(store, table, lens, q, q_rope, got, "dims")
    got = _run_shared(store, table, lens, [0], [], q, q_rope)
    _check_shared(store, table, lens, q, q_rope, got, "dims, no groups")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seqs", [5, 9])
def test_shared_prefix_of_many_chunks(seqs, fp8):
    """Two and three row blocks behind 32768 tokens: shares of 4 and 6 of its 512 tiles, so 128 and 85 chunks, and the
    join looks up 64 at a time."""
    gen = torch.Generator().manual_seed(seqs)
    store, table, lens, cu, shared, q, q_rope = _shared_inputs(gen, [(32768, [32769 + 3 * i for i in range(seqs)])], 64, 128,
                                                               64, fp8, 1, 16)
    got = _run_shared(store, table, lens, cu, shared, q, q_rope)
    _check_shared(store, table, lens, q, q_rope, got, "many chunks")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("many", ["sequences", "groups", "room"])
def test_shared_plans_of_large_batches(many, fp8):
    """More sequences or groups than the kernels plan by themselves, and a table with more room than 31 bits of tiles."""
    gen = torch.Generator().manual_seed(3)
    if many == "sequences":
        groups, alone = [(100, [130 + i % 50 for i in range(30)]), (64, [70] * 200), (0, [5, 9])], [40 + i % 90 for i in range(400)]
    elif many == "groups":
        groups, alone = [(40 + i, [60 + i, 50 + i, 30]) for i in range(70)] + [(10, [])] * 5, (90, 1)
    else:
        groups, alone = [(300, [310, 400, 299])], (50, 200)
    Q, H, L, R, page = 2, 8, 128, 32, 16
    store, table, lens, cu, shared, q, q_rope = _shared_inputs(gen, groups, page, L, R, fp8, Q, H, alone)
    if many == "room":
        wide = torch.full((table.shape[0], 1 << 26), -1, dtype=torch.int32, device="cuda")
        wide[:, : table.shape[1]] = table.cuda()
        import kda_recurrent_state_amd as kda
        cache = _gpu(store) if fp8 else store[0].cuda()
        got = kda.kda_latent_decode_shared(cache, wide, _i32(lens), _i32(cu), _i32(shared), q.cuda(), q_rope.cuda(),
                                           scale=SCALE, with_lse=True)
    else:
        got = _run_shared(store, table, lens, cu, shared, q, q_rope)
    _check_shared(store, table, lens, q, q_rope, got, many)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("per", [1, 2, 3, 65535])
def test_shared_as_many_sequences_as_there_can_be(per, fp8):
    """65535 sequences, in as many groups, in pairs, in threes and in one group; with queries of 0 the output is the mean
    of the two rows that a sequence sees, the first one of which is that of its group's first sequence."""
    import kda_recurrent_state_amd as kda
    gen = torch.Generator().manual_seed(per)
    N, L, page = 65535, 16, 1
    G = -(-N // per)
    codes = torch.randint(0, 120, (2 * N, page, L), generator=gen).to(torch.uint8)
    scales = torch.exp2(torch.randint(-2, 2, (2 * N, page), generator=gen).float())
    values = ref8.values(codes, scales, None)
    store = (codes, scales, None) if fp8 else (values.to(BF16),)   # (4 bits: bf16 holds them)
    perm = torch.randperm(2 * N, generator=gen).int()
    table = torch.stack([perm[:N], perm[N:]], 1)
    cu = (torch.arange(G + 1) * per).clamp(max=N)
    if per > 1:                                                     # what the others' tables have there is not read
        table[torch.arange(N) % per != 0, 0] = -1
    q = torch.zeros(N, 2, L, dtype=BF16, device="cuda")
    out, lse = kda.kda_latent_decode_shared(_gpu(store) if fp8 else store[0].cuda(), table.cuda(), _i32([2] * N),
                                            cu.int().cuda(), _i32([1] * G), q, scale=1.0, with_lse=True)
    rows = values.view(-1, L)
    first = table[torch.arange(N) // per * per, 0].long()
    want = (rows[first] + rows[table[:, 1].long()]) / 2
    # the mean is rounded once to bf16 and four times in fp32
    assert ((out.cpu().double() - want[:, None]).abs() <= (2.0 ** -8 + 2.0 ** -20) * want[:, None]).all()
    assert (lse.cpu().double() - math.log(2)).abs().max() <= 2.0 ** -20


@pytest.mark.parametrize("fp8", [False, True])
def test_shared_groups_that_are_no_offsets(fp8):
    """Bounds that fall are raised to the largest before, and clamped to the batch; shared lengths are clamped."""
    gen = torch.Generator().manual_seed(11)
    groups = [(64, [100, 90, 80]), (32, [50, 60])]
    store, table, lens, cu, shared, q, q_rope = _shared_inputs(gen, groups, 16, 128, 64, fp8, 1, 16, (30, 40))
    for bad_cu, bad_shared in [([1, 4, 2, 6], [64, 7, 32]), ([-3, 1, 4, 6, 900], [0, 64, 32, -5]),
                               ([1, 4, 6], [64, -9]), ([9, 1, 4], [5, 5]), ([0, 0, 0], [1000, 1000])]:
        got = _run_shared(store, table, lens, bad_cu, bad_shared, q, q_rope)
        _check_shared(store, table, lens, q, q_rope, got, str(bad_cu))
    # as many shared as the first one has, or more: up to its length, which the others agree on as well
    store, table, lens, cu, shared, q, q_rope = _shared_inputs(gen, [(100, [100, 130, 101])], 16, 128, 64, fp8, 1, 16)
    got = _run_shared(store, table, lens, cu, [2 ** 31 - 1], q, q_rope)
    _check_shared(store, table, lens, q, q_rope, got, "long")


def test_shared_without_groups_and_as_latent_decode():
    """No groups: each for itself.  16 bits: as kda_latent_decode up to roundings."""
    import kda_recurrent_state_amd as kda
    gen = torch.Generator().manual_seed(12)
    store, table, lens, cu, shared, q, q_rope = _shared_inputs(gen, [(500, [700, 600, 501])], 64, 512, 64, False, 1, 32, (5, 900))
    none = _run_shared(store, table, lens, [0], [], q, q_rope)
    _check_shared(store, table, lens, q, q_rope, none, "no groups")
    some = _run_shared(store, table, lens, cu, shared, q, q_rope)
    one = kda.kda_latent_decode(store[0].cuda(), table.cuda(), _i32(lens), q.cuda(), q_rope.cuda(), scale=SCALE, with_lse=True)
    for x in (none, some):
        # each is off the true result by the bounds that _check_shared has
        assert ((x[0].float() - one[0].float()).norm() / one[0].float().norm()).item() < 2.0 ** -7
        assert (x[1] - one[1]).abs().max().item() <= 2e-4


@pytest.mark.parametrize("fp8", [False, True])
def test_shared_views_and_given_outputs(fp8):
    """Queries of a joint projection, a page table and caches that are views of larger ones, outputs and a workspace
    of exactly the size given; what lies around them stays."""
    import kda_recurrent_state_amd as kda
    gen = torch.Generator().manual_seed(13)
    Q, H, L, R, page = 2, 12, 256, 32, 16
    store, table, lens, cu, shared, q, q_rope = _shared_inputs(gen, [(160, [200, 170, 161])], page, L, R, fp8, Q, H, (70,))
    N = len(lens)
    joint = torch.randn(N, H, Q, L + R + 24).to(BF16).cuda()
    joint[..., :L], joint[..., L: L + R] = q.transpose(1, 2).cuda(), q_rope.transpose(1, 2).cuda()
    qv, rv = joint[..., :L].transpose(1, 2), joint[..., L: L + R].transpose(1, 2)
    wide = torch.full((N, table.shape[1] + 5), 2 ** 30, dtype=torch.int32, device="cuda")
    wide[:, : table.shape[1]] = table.cuda()
    views = []
    for x in _gpu(store):
        big = torch.full((x.shape[0], 3) + tuple(x.shape[1:]), 0x7f if x.dtype == torch.uint8 else math.nan, dtype=x.dtype,
                         device="cuda")
        big[:, 1] = x
        views.append(big[:, 1])
    need = kda.kda_latent_shared_workspace_size(N, Q, H, L, 1)
    room = torch.full((need + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    outs = torch.full((N + 2, Q, H, L), 7.0, dtype=BF16, device="cuda")
    lses = torch.full((N + 2, Q, H), 7.0, device="cuda")
    out, lse = kda.kda_latent_decode_shared(tuple(views) if fp8 else views[0], wide[:, : table.shape[1]], _i32(lens), _i32(cu),
                                            _i32(shared), qv, rv, scale=SCALE, out=outs[1: N + 1], lse=lses[1: N + 1],
                                            workspace=room[:need])
    assert out.data_ptr() == outs[1].data_ptr() and lse.data_ptr() == lses[1].data_ptr()
    _check_shared(store, table, lens, q, q_rope, (out, lse), "views")
    assert (room[need:] == 0x5a).all() and (outs[0] == 7).all() and (outs[-1] == 7).all()
    assert (lses[0] == 7).all() and (lses[-1] == 7).all()
    # one query row for all heads and queries: strides of 0
    one = q[:, :1, :1].cuda().expand(N, Q, H, L), q_rope[:, :1, :1].cuda().expand(N, Q, H, R)
    got = kda.kda_latent_decode_shared(tuple(views) if fp8 else views[0], wide[:, : table.shape[1]], _i32(lens), _i32(cu),
                                       _i32(shared), *one, scale=SCALE, with_lse=True)
    _check_shared(store, table, lens, q[:, :1, :1].expand(N, Q, H, L), q_rope[:, :1, :1].expand(N, Q, H, R), got, "broadcast")
    three = kda.kda_latent_decode_shared(tuple(views) if fp8 else views[0], wide[:, : table.shape[1]], _i32(lens), _i32(cu),
                                         _i32(shared), qv[:, 1], rv[:, 1], scale=SCALE)
    assert three[0].shape == (N, H, L) and three[1] is None
    _check_shared(store, table, lens, q[:, 1:], q_rope[:, 1:], (three[0], None), "3-D")


@pytest.mark.parametrize("fp8", [False, True])
def test_shared_twice_is_the_same(fp8):
    gen = torch.Generator().manual_seed(14)
    store, table, lens, cu, shared, q, q_rope = _shared_inputs(gen, [(3000, [3100 + 7 * i for i in range(9)])], 64, 512, 64, fp8,
                                                               1, 20, (900,))
    a = _run_shared(store, table, lens, cu, shared, q, q_rope)
    b = _run_shared(store, table, lens, cu, shared, q, q_rope)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("groups,alone,Q,H", [
    ([], (4000,), 1, 32), ([(700, [800, 720, 705, 700])], (300, 0, 1), 1, 4), ([(3000, [3100 + 7 * i for i in range(9)])], (900,), 1, 20),
    ([(640, [700, 1300, 641])] * 6, (), 1, 64), ([], tuple(range(20, 3000, 41)), 2, 40), ([(9000, [9001 + i for i in range(20)])], (), 1, 130)])
def test_shared_results_are_the_workspaces_own(groups, alone, Q, H, fp8):
    """Whatever a workspace holds before the call, the results are the same to the bit: nothing is read that the call has
    not written."""
    import kda_recurrent_state_amd as kda
    gen = torch.Generator().manual_seed(22 + H)
    store, table, lens, cu, shared, q, q_rope = _shared_inputs(gen, groups, 16, 128, 64, fp8, Q, H, alone)
    if not groups:
        cu = [0]
    need = kda.kda_latent_shared_workspace_size(len(lens), Q, H, 128, len(shared))
    got = []
    for fill in (0, 0xff, 0x7f, 0x01):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        got.append(_run_shared(store, table, lens, cu, shared, q, q_rope, workspace=ws))
    for out, lse in got[1:]:
        assert torch.equal(out, got[0][0]) and torch.equal(lse, got[0][1])
    _check_shared(store, table, lens, q, q_rope, got[0], "workspaces")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("size", [1e3, 1e6, 1e15, 2e37])  # (the query holds 13.86 times that: bf16 ends at 3.39e38)
def test_scores_of_any_size(size, fp8):
    """One component of the query and of some rows is so large that their scores stand alone, far beyond the step of
    fp32; the type's lowest value as the score of the others.  The weights are those of the large scores alone."""
    gen = torch.Generator().manual_seed(15)
    page, L, R, H = 16, 128, 64, 8
    lens = [400, 330, 300]
    table, pages = _table(gen, lens, page)
    rows = torch.randn(pages * page, L + R, generator=gen)
    # the rotary key is held in 16 bits in both caches: component 3 makes the scores 0 or -size or, of a few rows, size
    rows[:, L + 3] = -1.0
    few = [5, 100, 333]
    for n in range(3):
        for j in few:
            if j < lens[n]:
                rows[int(table[n, j // page]) * page + j % page, L + 3] = 1.0
    store = (*[x.view(pages, page, *x.shape[1:]) for x in ref8.quantize(rows[:, :L].double())],
             rows[:, L:].to(BF16).view(pages, page, R)) if fp8 else (rows.to(BF16).view(pages, page, L + R),)
    if fp8:
        store = (store[0], store[1].float(), store[2])
    q, q_rope = _queries(gen, 3, 1, H, L, R)
    q, q_rope = q * 0, q_rope * 0
    q_rope[..., 3] = size / SCALE
    got = _run_shared(store, table, lens, [0, 1], [10], q, q_rope)
    for n in range(3):
        seen = [j for j in few if j < lens[n]]
        at = [int(table[n, j // page]) * page + j % page for j in seen]
        values = (ref8.values(*store) if fp8 else store[0].double()).view(pages * page, -1)[at, :L]
        want = values.mean(0)
        bound = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -12) * values.abs().mean(0)
        assert ((got[0][n, 0].double().cpu() - want).abs() <= bound).all()
        top = float(q_rope[0, 0, 0, 3].double()) * SCALE
        assert (got[1][n].double().cpu() - (top + math.log(len(seen)))).abs().max() <= 2.0 ** -20 * top + 1e-4


@pytest.mark.parametrize("fp8", [False, True])
def test_values_as_large_as_documented(fp8):
    """500 tokens with values up to 2^109 (their product is below 2^119: 2^8 times it is fp32), and scores that rise by 7.6 units of log2, so
    that the maximum in use stays behind: the results are those of the formula."""
    gen = torch.Generator().manual_seed(21)
    N, page, L, R, H = 200, 64, 128, 8, 8
    lens = [500 - n % 3 for n in range(N)]
    table, pages = _table(gen, lens, page)
    latent = torch.randn(pages * page, L, generator=gen).clamp(-4, 4) * 2.0 ** 107
    k_rope = torch.zeros(pages * page, R)
    for n in range(N):
        j = torch.arange(lens[n])
        k_rope[table[n].long()[j // page] * page + j % page, 2] = j * (7.6 / 512)
    if fp8:
        codes, scales = ref8.quantize(latent.double())
        store = (codes.view(pages, page, L), scales.float().view(pages, page), k_rope.to(BF16).view(pages, page, R))
    else:
        store = (torch.cat([latent, k_rope], 1).to(BF16).view(pages, page, L + R),)
    q, q_rope = _queries(gen, N, 1, H, L, R)
    q = q * 0
    q_rope = q_rope * 0
    q_rope[..., 2] = math.log(2) / SCALE
    got = _run_shared(store, table, lens, [0], [], q, q_rope)
    _check_shared(store, table, lens, q, q_rope, got, "large values")


def test_decode8_query_that_is_not_finite():
    import kda_recurrent_state_amd as kda
    gen = torch.Generator().manual_seed(16)
    lens = [100, 200]
    table, pages = _table(gen, lens, 16)
    store = _cache8(gen, pages, 16, 128, 8)
    q, q_rope = _queries(gen, 2, 1, 8, 128, 8)
    rows = ref8.values(*store)
    want = ref.decode(rows, table, torch.tensor(lens), q, q_rope, SCALE)
    q[0, 0, 3, 5] = math.nan
    out, lse = kda.kda_latent_decode_fp8(*_gpu(store), table.cuda(), _i32(lens), q.cuda(), q_rope.cuda(), scale=SCALE, with_lse=True)
    assert out[0, 0, 3].isnan().all() and lse[0, 0, 3].isnan()
    keep = torch.ones(2, 1, 8, dtype=torch.bool)
    keep[0, 0, 3] = False
    assert torch.isfinite(out.cpu()[keep]).all()
    ref.check(out.cpu()[keep], lse.cpu()[keep], [x[keep] for x in want], "others")


@pytest.mark.parametrize("fp8", [False, True])
def test_pages_beyond_32_bits(fp8):
    """A cache of over 2^32 bytes (and 2^31 elements); the sequences' pages lie at its beginning and its end."""
    import kda_recurrent_state_amd as kda
    gen = torch.Generator().manual_seed(17)
    page, L, R, H = 64, 512, 64, 16
    lens = [130, 300, 64]
    table, few = _table(gen, lens, page, extra=0)
    pages = (1 << 32) // (page * L) + 1000 if fp8 else (1 << 32) // (page * (L + R) * 2) + 1000
    where = torch.cat([torch.arange(few // 2), torch.arange(pages - (few - few // 2), pages)])
    table = torch.where(table >= 0, where[table.clamp(min=0).long()].int(), table)
    small = _cache8(gen, few, page, L, R) if fp8 else (torch.randn(few, page, L + R, generator=gen).to(BF16),)
    big = []
    for x in small:
        y = torch.zeros((pages,) + tuple(x.shape[1:]), dtype=x.dtype, device="cuda")
        y[where.cuda()] = x.cuda()
        big.append(y)
    q, q_rope = _queries(gen, 3, 1, H, L, R)
    back = {int(w): i for i, w in enumerate(where)}
    near = torch.tensor([[back.get(int(p), -1) for p in row] for row in table], dtype=torch.int32)
    got = kda.kda_latent_decode_shared(tuple(big) if fp8 else big[0], table.cuda(), _i32(lens), _i32([0, 3]), _i32([0]), q.cuda(),
                                       q_rope.cuda(), scale=SCALE, with_lse=True)
    _check_shared(small, near, lens, q, q_rope, got, "far pages")
    if fp8:
        # written and read at both ends
        c, k_rope = _rows(40, L, R, BF16, 5)
        slots = torch.cat([torch.arange(20), torch.arange(pages * page - 20, pages * page)])
        kda.kda_latent_quantize_scatter(c, k_rope, slots.cuda(), *big)
        want, scale = ref8.quantize(c.cpu().double())
        assert torch.equal(big[0].view(-1, L)[slots.cuda()].cpu(), want)
        assert torch.equal(big[1].view(-1)[slots.cuda()].cpu().double(), scale)
        rows = kda.kda_latent_dequantize_gather(*big, slots.flip(0).cuda(), dtype=torch.float32).cpu()
        assert torch.equal(rows[:, :L].double(), (ref8.VALUES[want.long()] * scale[:, None]).flip(0).float().double())
        assert torch.equal(rows[:, L:], k_rope.cpu().float().flip(0))


def test_captured_calls_follow_their_inputs():
    """Two graphs with workspaces of their own, replayed in turn with eager work between; lengths, groups and the cache
    change between replays."""
    import kda_recurrent_state_amd as kda
    gen = torch.Generator().manual_seed(18)
    page, L, R, H, N = 16, 256, 64, 16, 5
    table, pages = _table(gen, [700] * N, page)
    store = _gpu(_cache8(gen, pages, page, L, R))
    q, q_rope = (x.cuda() for x in _queries(gen, N, 1, H, L, R))
    table[1:, : 400 // page] = table[0, : 400 // page]     # the first 400 tokens are shared
    lens, cu, shared = _i32([0] * N), _i32([0, N]), _i32([0])
    c, k_rope = torch.randn(N, L, generator=gen).to(BF16).cuda(), torch.randn(N, R, generator=gen).to(BF16).cuda()
    slots = torch.zeros(N, dtype=torch.int64, device="cuda")
    dtable = table.cuda()
    outs = []

    def step(i):
        kda.kda_latent_quantize_scatter(c, k_rope, slots, *store)
        if i == 0:
            kda.kda_latent_decode_shared(store, dtable, lens, cu, shared, q, q_rope, scale=SCALE, out=outs[i][0], lse=outs[i][1],
                                         workspace=outs[i][2])
        else:
            kda.kda_latent_decode_fp8(*store, dtable, lens, q, q_rope, scale=SCALE, out=outs[i][0], lse=outs[i][1],
                                      workspace=outs[i][2])
        outs[i][3].copy_(kda.kda_latent_dequantize_gather(*store, slots, out=outs[i][4]))

    graphs = []
    for i in range(2):
        need = kda.kda_latent_shared_workspace_size(N, 1, H, L, 1 - i)
        outs.append((torch.empty(N, 1, H, L, dtype=BF16, device="cuda"), torch.empty(N, 1, H, device="cuda"),
                     torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty(N, L + R, dtype=BF16, device="cuda"),
                     torch.empty(N, L + R, dtype=BF16, device="cuda")))
        stream = torch.cuda.Stream()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            step(i)
        torch.cuda.synchronize()
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[i]):
            step(i)
    for turn, (ls, share) in enumerate([([500, 450, 401, 699, 640], 400), ([100, 0, 700, 1, 50], 0), ([400, 500, 600, 650, 410], 333),
                                        ([0] * 5, 400), ([700] * 5, 400)]):
        lens.copy_(_i32(ls))
        shared.fill_(share)
        # each sequence's last token is written by the call itself (behind what is shared)
        at = [int(table[n, (ls[n] - 1) // page]) * page + (ls[n] - 1) % page if ls[n] > 400 else -1 for n in range(N)]
        slots.copy_(torch.tensor(at, device="cuda"))
        c.copy_(torch.randn(N, L, generator=gen))
        for i in (0, 1):
            graphs[i].replay()
        torch.cuda.synchronize()
        cpu = [x.cpu() for x in store]
        rows = ref8.values(*cpu)
        want = ref.decode(rows, table, torch.tensor(ls), q.cpu(), q_rope.cpu(), SCALE)
        for i in (0, 1):
            ref.check(outs[i][0], outs[i][1], want, "replay %d of graph %d" % (turn, i))
            flat = torch.where((slots >= 0)[:, None].cpu(), rows.view(-1, L + R)[slots.clamp(min=0).cpu()], 0.0)
            assert torch.equal(outs[i][3].cpu().double(), flat)
        torch.randn(1000, device="cuda").sum().item()         # eager work between


def test_other_streams_and_calls_at_once():
    import kda_recurrent_state_amd as kda
    gen = torch.Generator().manual_seed(19)
    sets = [_shared_inputs(gen, [(1000 + 500 * i, [1600 + 100 * i + 9 * j for j in range(6)])], 64, 512, 64, i == 1, 1, 16)
            for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    on = [(_gpu(s[0]) if i == 1 else s[0][0].cuda(), s[1].cuda(), _i32(s[2]), _i32(s[3]), _i32(s[4]), s[5].cuda(), s[6].cuda())
          for i, s in enumerate(sets)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i in range(2):
            got[i].append(kda.kda_latent_decode_shared(*on[i], scale=SCALE, with_lse=True, stream=streams[i]))
    torch.cuda.synchronize()
    for i, s in enumerate(sets):
        _check_shared(s[0], s[1], s[2], s[5], s[6], got[i][0], "stream %d" % i)
        for more in got[i][1:]:
            assert torch.equal(more[0], got[i][0][0]) and torch.equal(more[1], got[i][0][1])
    store = _empty_store(4, 16, 128, 8)
    c, k_rope = _rows(50, 128, 8, BF16, 2)
    slots = torch.arange(50, device="cuda")
    torch.cuda.synchronize()
    kda.kda_latent_quantize_scatter(c, k_rope, slots, *store, stream=streams[0])
    rows = kda.kda_latent_dequantize_gather(*store, slots, stream=streams[0])
    streams[0].synchronize()
    assert torch.equal(rows.cpu().double(), ref8.values(*store).view(-1, 136)[:50])


def test_a_serving_run():
    """Prompts written, forked with shared pages, continued one token at a time by the children, attended to with the
    prompt computed once, compacted, read back and freed: the rows and results are those of the tokens themselves."""
    import kda_recurrent_state_amd as kda
    gen = torch.Generator().manual_seed(20)
    page, L, R, H, seqs, per, pages = 16, 128, 64, 16, 8, 12, 60
    store = _empty_store(pages, page, L, R)
    for x in store:
        x.zero_()
    table = torch.full((seqs, per), -1, dtype=torch.int32, device="cuda")
    lens, refs = torch.zeros(seqs, dtype=torch.int32, device="cuda"), torch.zeros(pages, dtype=torch.int32, device="cuda")
    tokens = {}                                                    # of a slot: its rows in fp64

    def rows_of(n):
        x = torch.randn(n, L + R, generator=gen).to(BF16)
        codes, scales = ref8.quantize(x[:, :L].double())
        return x.cuda(), torch.cat([ref8.VALUES[codes.long()] * scales[:, None], x[:, L:].double()], 1)

    # two prompts, in pages from the end of the pool
    at = pages
    for s, n in ((0, 70), (4, 37)):
        used = -(-n // page)
        table[s, :used] = torch.arange(at - used, at, dtype=torch.int32, device="cuda")
        at -= used
        lens[s], refs[table[s, :used].long()] = n, 1
        x, tokens[s] = rows_of(n)
        j = torch.arange(n, device="cuda")
        kda.kda_latent_quantize_scatter(x[:, :L], x[:, L:], table[s].long()[j // page] * page + j % page, *store)
    status = kda.kda_page_fork(table, lens, refs, _i32([0, 0, 0, 4]), _i32([1, 2, 3, 5]), page, caches=list(store))
    assert status.tolist() == [0] * 4
    for child, parent in ((1, 0), (2, 0), (3, 0), (5, 4)):
        tokens[child] = tokens[parent]
    order = [0, 1, 2, 3, 4, 5]
    cu, shared = _i32([0, 4, 6]), _i32([70 // page * page, 37 // page * page])
    for turn in range(3):
        # one new token each; a page of its own where the last one is full (taken by hand: the pool's first free one)
        new, values = rows_of(len(order))
        slots = []
        for i, s in enumerate(order):
            n = int(lens[s])
            if n % page == 0:
                free = int((refs <= 0).nonzero()[0])
                table[s, n // page], refs[free] = free, 1
            slots.append(int(table[s, n // page]) * page + n % page)
            lens[s] = n + 1
            tokens[s] = torch.cat([tokens[s], values[i: i + 1]])
        kda.kda_latent_quantize_scatter(new[:, :L], new[:, L:], torch.tensor(slots, device="cuda"), *store)
        q, q_rope = _queries(gen, 6, 1, H, L, R)
        got = kda.kda_latent_decode_shared(store, table[:6], lens[:6], cu, shared, q.cuda(), q_rope.cuda(), scale=SCALE,
                                           with_lse=True)
        alone = kda.kda_latent_decode_fp8(*store, table[:6], lens[:6], q.cuda(), q_rope.cuda(), scale=SCALE, with_lse=True)
        for s in order:
            full = torch.cat([q[s, 0].double(), q_rope[s, 0].double()], -1)
            want = ref.attend(full, tokens[s], tokens[s][:, :L], torch.full((H,), len(tokens[s])), SCALE)
            ref.check(got[0][s, 0], got[1][s, 0], want, "turn %d, slot %d" % (turn, s))
            ref.check(alone[0][s, 0], alone[1][s, 0], want, "turn %d, slot %d alone" % (turn, s))
        if turn == 1:
            kda.kda_page_compact(table, lens, refs, page, caches=list(store))
    for s in order:
        j = torch.arange(len(tokens[s]), device="cuda")
        back = kda.kda_latent_dequantize_gather(*store, table[s].long()[j // page] * page + j % page)
        assert torch.equal(back.cpu().double(), tokens[s])
    kda.kda_page_free(table, lens, refs, torch.ones(seqs, dtype=torch.bool, device="cuda"), page)
    assert (refs == 0).all() and (lens == 0).all()


def test_python_refusals():
    import kda_recurrent_state_amd as kda
    codes, scales, rope = _empty_store(4, 16, 128, 8)
    c, k_rope = _rows(10, 128, 8, BF16, 2)
    slots = torch.arange(10, device="cuda")
    q, q_rope = (x.cuda() for x in _queries(torch.Generator().manual_seed(1), 1, 1, 8, 128, 8))
    table, lens, cu, sh = _i32([[0, 1]]), _i32([20]), _i32([0, 1]), _i32([0])
    write, read = kda.kda_latent_quantize_scatter, kda.kda_latent_dequantize_gather
    shared, fp8 = kda.kda_latent_decode_shared, kda.kda_latent_decode_fp8
    store = (codes, scales, rope)
    for call in [
            lambda: write(c, k_rope, slots, codes.float(), scales, rope), lambda: write(c, k_rope, slots, codes, scales.double(), rope),
            lambda: write(c, k_rope, slots, codes, scales, rope.float()), lambda: write(c, k_rope.float(), slots, *store),
            lambda: write(c.half(), k_rope.half(), slots, *store), lambda: write(c, None, slots, *store),
            lambda: write(c, k_rope, slots, codes, scales, None), lambda: write(c[:, :64], k_rope, slots, *store),
            lambda: write(c, k_rope, slots[:5], *store), lambda: write(c, k_rope, slots.float(), *store),
            lambda: write(c, k_rope, slots[::2], *store), lambda: write(c, k_rope[:9], slots, *store),
            lambda: write(c, k_rope, slots, codes[:, ::2], scales[:, ::2], rope[:, ::2]),
            lambda: write(c, k_rope, slots, codes[:3], scales, rope), lambda: write(c, k_rope, slots, codes.view(-1, 128), scales, rope),
            lambda: write(c.t().contiguous().t(), k_rope, slots, *store), lambda: write(c, k_rope, slots.cpu(), *store),
            lambda: read(*store, slots, dtype=torch.float16), lambda: read(*store, slots[None]), lambda: read(*store, slots.half()),
            lambda: read(*store, slots, out=torch.empty(10, 128, dtype=BF16, device="cuda")),
            lambda: read(codes[..., :120], scales, rope, slots),
            lambda: fp8(*store, table, lens, q, q_rope), lambda: fp8(*store, table, lens, q.float(), q_rope, scale=1.0),
            lambda: fp8(*store, table, lens, q[..., :64], q_rope, scale=1.0), lambda: fp8(*store, table, lens, q, None, scale=1.0),
            lambda: fp8(*store, table.long(), lens, q, q_rope, scale=1.0), lambda: fp8(*store, table, lens[:0], q, q_rope, scale=1.0),
            lambda: shared(store[:2], table, lens, cu, sh, q, q_rope, scale=1.0),
            lambda: shared(rope, table, lens, cu, sh, q, q_rope, scale=1.0),
            lambda: shared(store, table, lens, None, sh, q, q_rope, scale=1.0),
            lambda: shared(store, table, lens, cu, None, q, q_rope, scale=1.0),
            lambda: shared(store, table, lens, cu[:1], sh, q, q_rope, scale=1.0),
            lambda: shared(store, table, lens, cu.long(), sh, q, q_rope, scale=1.0),
            lambda: shared(store, table, lens, _i32([0, 9, 1])[::2], sh, q, q_rope, scale=1.0),
            lambda: shared(store, table, lens, cu, sh, q, q_rope, scale=-1.0),
            lambda: shared(store, table, lens, cu, sh, q, q_rope, scale=1.0, workspace=torch.empty(64, dtype=torch.uint8, device="cuda")),
            lambda: shared(store, table, lens, cu, sh, q, q_rope, scale=1.0, out=torch.empty(1, 1, 8, 64, dtype=BF16, device="cuda"))]:
        with pytest.raises((kda.KDAError, RuntimeError, ValueError)):
            call()
    write(c[:0], k_rope[:0], slots[:0], *store)                    # nothing to do
    assert read(*store, slots[:0]).shape == (0, 136)
    assert shared(store, table[:0], lens[:0], cu, sh, q[:0], q_rope[:0], scale=1.0)[0].shape == (0, 1, 8, 128)
