"""Fork, compact and free of cache pages on the GPU, bit for bit against plain
evaluations, one entry after the other."""
import math

import pytest
import torch

from tests import latent_ref as ref
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _i32(x):
    return torch.tensor(x, dtype=torch.int32)


def _pool(seed, seqs, per, pages, page, live, shared=0.3):
    """A pool in use, on the host: random lengths, scattered pages, some prefixes shared."""
    gen = torch.Generator().manual_seed(seed)
    rnd = lambda n: int(torch.randint(0, n, (1,), generator=gen))  # noqa: E731
    perm, at = torch.randperm(pages, generator=gen).tolist(), 0
    table, lens = torch.full((seqs, per), -1, dtype=torch.int32), [0] * seqs
    before = None
    for s in sorted(torch.randperm(seqs, generator=gen)[:live].tolist()):
        n = 1 + rnd(per * page)
        used, take = -(-n // page), 0
        if before is not None and torch.rand(1, generator=gen) < shared:
            take = min(n // page, lens[before] // page)
            table[s, :take] = table[before, :take]
        if at + used - take > pages - 2:
            table[s] = -1
            continue
        table[s, take:used] = torch.tensor(perm[at:at + used - take], dtype=torch.int32)
        at += used - take
        lens[s], before = n, s
    refs = torch.bincount(table[table >= 0].long(), minlength=pages).int()
    return table, _i32(lens), refs


def _dev(*ts):
    return [t.cuda() for t in ts]


def _caches(pages, page, seed=5):
    """Stores of several shapes, types, alignments and gaps."""
    gen = torch.Generator().manual_seed(seed)
    a = torch.randn(pages, page, 24, generator=gen).bfloat16()
    b = torch.randint(-128, 127, (pages, page * 13), generator=gen, dtype=torch.int8)
    flat = torch.randn(pages, page * 6 + 5, generator=gen)
    return a, b, flat


def _check_fork(pool, page, src, dst, share, idx=torch.int32, caches=(), view=None):
    import kda_recurrent_state_amd as kda
    table, lens, refs = pool
    dt, dl, dr = _dev(*pool)
    dc = _dev(*caches)
    src, dst = torch.tensor(src, dtype=idx), torch.tensor(dst, dtype=idx)
    status = kda.kda_page_fork(dt, dl, dr, src.cuda(), dst.cuda(), page, caches=[view(c) if view else c for c in dc],
                               share=share)
    t, n, r, c, s = ref.fork(table, lens, refs, src, dst, page, [view(c) if view else c for c in caches], share)
    if view:   # what lies around the pages stays
        whole = [c.clone() for c in caches]
        for w, x in zip(whole, c):
            view(w).copy_(x)
        c = whole
    assert torch.equal(status.cpu(), s), (status.tolist(), s.tolist())
    assert torch.equal(dt.cpu(), t) and torch.equal(dl.cpu(), n) and torch.equal(dr.cpu(), r)
    for got, want in zip(dc, c):
        assert torch.equal(got.cpu(), want)
    return s


@pytest.mark.parametrize("share", [True, False])
@pytest.mark.parametrize("idx", [torch.int32, torch.int64])
@pytest.mark.parametrize("seqs,per,pages,page,live", [(2, 1, 3, 1, 1), (8, 4, 40, 16, 4), (33, 7, 300, 5, 20),
                                                      (300, 12, 5000, 8, 150)])
def test_fork(seqs, per, pages, page, live, idx, share):
    pool = _pool(1, seqs, per, pages, page, live)
    full = [s for s in range(seqs) if pool[1][s] > 0]
    empty = [s for s in range(seqs) if pool[1][s] == 0]
    a, b, flat = _caches(pages, page)
    src = [full[i % len(full)] for i in range(len(empty))]
    s = _check_fork(pool, page, src, empty, share, idx, [a])
    assert (s == 0).any()
    _check_fork(pool, page, src, empty, share, idx, [a, b, flat[:, :page * 6].contiguous()])
    _check_fork(pool, page, src, empty, share, idx)


def test_fork_gaps_and_alignments():
    pool = _pool(2, 12, 3, 40, 4, 5)
    full = [s for s in range(12) if pool[1][s] > 0]
    empty = [s for s in range(12) if pool[1][s] == 0]
    flat = _caches(40, 4)[2]
    # pages of 24 floats with 5 floats between them; then one float further on; then odd bytes
    _check_fork(pool, 4, [full[0]] * len(empty), empty, False, caches=[flat], view=lambda c: c[:, :24])
    _check_fork(pool, 4, [full[0]] * len(empty), empty, False, caches=[flat], view=lambda c: c[:, 1:25])
    raw = torch.randint(0, 255, (40, 1031), dtype=torch.uint8, generator=torch.Generator().manual_seed(1))
    _check_fork(pool, 4, [full[-1]] * len(empty), empty, False, caches=[raw], view=lambda c: c[:, 3:1030])


def test_fork_bad_entries_and_full_pool():
    pool = _pool(3, 16, 4, 24, 4, 6, shared=0)
    table, lens, refs = pool
    full = [s for s in range(16) if lens[s] > 0]
    empty = [s for s in range(16) if lens[s] == 0]
    # bad slots, the same slot, a full target, a target twice, an empty parent, then real ones until the pages run out
    src = [-1, 16, full[0], full[0], full[1], full[1], empty[0]] + full
    dst = [empty[0], empty[0], full[0], full[1], empty[1], empty[1], empty[2]] + empty[3:3 + len(full)]
    src, dst = src[:len(dst)], dst[:len(src)]
    for share in (True, False):
        s = _check_fork(pool, 4, src, dst, share, caches=[_caches(24, 4)[0]])
        assert s.tolist()[:6] == [2, 2, 2, 2, s[4], 2] and s[6] == 0
    assert (s == 1).any()
    # a parent with a page outside the pool, one with a free page, lengths that no table row holds
    table[full[0], 0] = 24
    refs[table[full[1], 0].long()] = 0
    lens[full[2]] = 17
    lens[full[3]] = -1
    s = _check_fork((table, lens, refs), 4, full[:4], empty[:4], True)
    assert s.tolist() == [2, 2, 2, 2]


@pytest.mark.parametrize("entries", [7, 160])
@pytest.mark.parametrize("share", [True, False])
def test_fork_of_an_empty_slot_that_becomes_a_child(entries, share):
    """Every entry sees the pool as it was: a child of a slot that is empty before the call is empty, also where that
    slot is another entry's child."""
    pool = _pool(9, 400, 5, 1200, 8, 30, shared=0)
    full = [s for s in range(400) if pool[1][s] > 0]
    empty = [s for s in range(400) if pool[1][s] == 0][:2 * entries]
    a, b = empty[:entries], empty[entries:]
    src, dst = [full[i % len(full)] for i in range(entries)] + a, a + b
    order = [i // 2 + entries * (i % 2) for i in range(2 * entries)]
    status = _check_fork(pool, 8, [src[i] for i in order], [dst[i] for i in order], share, caches=[_caches(1200, 8)[0]])
    assert not status.any()


@pytest.mark.parametrize("entries", [60, 200, 1500])
@pytest.mark.parametrize("share", [True, False])
def test_fork_refusals_among_many_entries(entries, share):
    """Bad slots, full targets, repeated targets, parents with a bad or a free
    page or a length no row holds, among more entries than one workgroup checks
    and than one step of the plan sums; the pages run out before the end."""
    pool = _pool(14, 1800, 6, 4000, 4, 200, shared=0.2)
    table, lens, refs = pool
    full = [s for s in range(1800) if lens[s] > 0]
    empty = [s for s in range(1800) if lens[s] == 0]
    table[full[5], 0] = 4000
    refs[table[full[6], 0].long()] = 0
    lens[full[7]] = 25
    lens[full[8]] = -1
    refs[refs == 0] = -(torch.arange(int((refs == 0).sum())).int() % 2)
    gen = torch.Generator().manual_seed(entries)
    src = [full[int(torch.randint(0, len(full), (1,), generator=gen))] for _ in range(entries)]
    dst = empty[:entries]
    for i, (s, d) in enumerate([(-1, empty[0]), (1800, empty[1]), (full[0], full[1]), (full[2], full[2]),
                                (full[3], dst[0]), (full[5], dst[1]), (full[6], dst[2]), (full[7], dst[3]),
                                (full[8], dst[4]), (full[9], -7), (full[9], 1 << 20), (full[10], dst[5])]):
        for at in (10 + 3 * i, entries - 1 - 4 * i):
            src[at], dst[at] = s, d
    free = int((refs <= 0).sum())
    keep = torch.randperm(4000, generator=gen)
    taken = [p for p in keep.tolist() if refs[p] <= 0][:max(0, free - entries * (1 if share else 3) // 2)]
    refs[taken] = 1     # about half of the entries find pages
    s = _check_fork(pool, 4, src, dst, share, torch.int64 if share else torch.int32, [_caches(4000, 4)[0]])
    assert all((s == k).any() for k in (0, 1, 2))
    if entries > 1100 and not share:
        assert (s[1024:] == 1).any()


@pytest.mark.parametrize("entries", [5, 140])
@pytest.mark.parametrize("share", [True, False])
def test_fork_of_long_parents(entries, share):
    """Parents of 70 to 600 pages; one has a page outside the pool behind the
    64th, one a free page behind the 256th, one behind the 512th."""
    pages = 4000 + entries * (1 if share else 600)
    pool = _pool(15, 400, 600, pages, 2, 6, shared=0)
    table, lens, refs = pool
    full = [s for s in range(400) if lens[s] > 0]
    empty = [s for s in range(400) if lens[s] == 0]
    at = int(refs.sum())
    spare = [p for p in range(pages) if refs[p] == 0]
    for s, n in zip(empty[:5], (70, 129, 300, 513, 600)):
        for j in range(n):
            table[s, j] = spare.pop()
        lens[s] = 2 * n - 1
        refs[table[s, :n].long()] = 1
    assert int(refs.sum()) == at + 70 + 129 + 300 + 513 + 600
    parents = empty[:5]
    table[parents[1], 100] = -1
    refs[table[parents[2], 270].long()] = 0
    refs[table[parents[3], 512].long()] = -2
    src = [parents[(i + 4) % 5] for i in range(entries)]
    s = _check_fork(pool, 2, src, empty[5:5 + entries], share, caches=[_caches(pages, 2)[0]])
    assert s.tolist()[:5] == [0, 0, 2, 2, 2]


@pytest.mark.parametrize("share", [True, False])
def test_fork_runs_out_behind_entry_1024(share):
    """The plan's sums are carried over its steps of 1024 entries."""
    pool = _pool(16, 3200, 2, 2600, 4, 40, shared=0)
    table, lens, refs = pool
    full = [s for s in range(3200) if lens[s] == 5 or lens[s] == 6]
    empty = [s for s in range(3200) if lens[s] == 0]
    free = [p for p in range(2600) if refs[p] == 0]
    refs[free[(1030 if share else 2060):]] = 1
    s = _check_fork(pool, 4, [full[i % len(full)] for i in range(1300)], empty[:1300], share, caches=[_caches(2600, 4)[0]])
    assert not s[:1030].any() and (s[1030:] == 1).all()


def test_fork_of_state_rows_matches_gather_and_scatter():
    """Recurrent states (page size 1, one row a slot, rows with a gap): a fork
    without sharing equals gathering the parents' rows and scattering them."""
    import kda_recurrent_state_amd as kda
    rows, H, V, K = 40, 2, 32, 16
    gen = torch.Generator().manual_seed(6)
    flat = torch.randn(rows, H * V * K + 64, generator=gen).cuda()
    cache = torch.as_strided(flat, (rows, H, V, K), (H * V * K + 64, V * K, K, 1))
    perm = torch.randperm(rows, generator=gen)[:10]
    table = torch.full((30, 1), -1, dtype=torch.int32)
    table[:10, 0] = perm.int()
    lens = _i32([1] * 10 + [0] * 20)
    refs = torch.zeros(rows, dtype=torch.int32)
    refs[perm] = 1
    dt, dl, dr = _dev(table, lens, refs)
    before = flat.clone()
    status = kda.kda_page_fork(dt, dl, dr, _i32([0, 0, 7]).cuda(), _i32([10, 25, 11]).cuda(), 1, caches=[cache],
                               share=False)
    assert status.tolist() == [0, 0, 0]
    want = before.clone()
    view = torch.as_strided(want, (rows, H, V, K), (H * V * K + 64, V * K, K, 1))
    packed = kda.kda_state_gather(view, table[[0, 0, 7], 0].cuda())
    kda.kda_state_scatter(view, dt[[10, 25, 11], 0].contiguous(), packed)
    assert torch.equal(flat, want)


@pytest.mark.parametrize("many", [33, 70])
def test_fork_and_compact_many_layers(many):
    """More stores than one launch takes, sizes all different."""
    import kda_recurrent_state_amd as kda
    pool = _pool(4, 20, 3, 60, 4, 8)
    gen = torch.Generator().manual_seed(2)
    caches = [torch.randn(60, 4 * (1 + 8 * i % 37), generator=gen) for i in range(many)]
    full = [s for s in range(20) if pool[1][s] > 0]
    empty = [s for s in range(20) if pool[1][s] == 0]
    _check_fork(pool, 4, [full[2]] * len(empty), empty, False, caches=caches)
    dt, dl, dr = _dev(*pool)
    dc = _dev(*caches)
    live = kda.kda_page_compact(dt, dl, dr, 4, caches=dc)
    t, r, c, n = ref.compact(*pool, 4, caches)
    assert live.item() == n and torch.equal(dt.cpu(), t) and torch.equal(dr.cpu(), r)
    assert all(torch.equal(a.cpu(), b) for a, b in zip(dc, c))


@pytest.mark.parametrize("seqs,per,pages,page,live", [(1, 1, 1, 1, 1), (1, 1, 1, 1, 0), (8, 4, 40, 16, 4),
                                                      (33, 7, 300, 5, 20), (300, 12, 5000, 8, 150), (9, 5, 1500, 3, 9),
                                                      (64, 8, 70, 4, 64), (150, 300, 33000, 2, 110),
                                                      (150, 300, 70000, 2, 150)])
def test_compact(seqs, per, pages, page, live):
    import kda_recurrent_state_amd as kda
    pool = _pool(7, seqs, per, pages, page, live)
    if pages > 20:
        pool[2][pool[2] == 0] -= torch.arange(int((pool[2] == 0).sum())).int() % 3   # counts below zero are free too
    a, b, flat = _caches(pages, page)
    dt, dl, dr = _dev(*pool)
    dc = _dev(a, b, flat)
    got = kda.kda_page_compact(dt, dl, dr, page, caches=[dc[0], dc[1], dc[2][:, :page * 6]])
    keep = flat.clone()
    t, r, c, n = ref.compact(*pool, page, [a, b, flat[:, :page * 6]])
    keep[:, :page * 6] = c[2]
    assert got.item() == n and torch.equal(dt.cpu(), t) and torch.equal(dl.cpu(), pool[1])
    assert torch.equal(dr.cpu(), r)
    assert torch.equal(dc[0].cpu(), c[0]) and torch.equal(dc[1].cpu(), c[1]) and torch.equal(dc[2].cpu(), keep)
    assert (dr[:n] > 0).all() and (dr[n:] <= 0).all()
    # a compact pool stays as it is
    before = [x.clone() for x in (dt, dr, *dc)]
    kda.kda_page_compact(dt, dl, dr, page, caches=[dc[0], dc[1], dc[2][:, :page * 6]])
    assert all(torch.equal(x, y) for x, y in zip(before, (dt, dr, *dc)))


def test_compact_passes_over_entries_outside_the_pool():
    import kda_recurrent_state_amd as kda
    table, lens, refs = _pool(8, 10, 4, 50, 4, 6)
    s = [i for i in range(10) if lens[i] > 0][0]
    table[s, 0], lens[s] = 50, 1 << 20   # a bad entry, a length no row holds
    dt, dl, dr = _dev(table, lens, refs)
    kda.kda_page_compact(dt, dl, dr, 4)
    t, r, _, _ = ref.compact(table, lens, refs, 4, [])
    assert torch.equal(dt.cpu(), t) and torch.equal(dr.cpu(), r)


@pytest.mark.parametrize("dtype", [torch.bool, torch.uint8])
@pytest.mark.parametrize("seqs,per,pages,page,live", [(1, 1, 2, 1, 1), (8, 4, 40, 16, 5), (300, 40, 9000, 8, 200),
                                                      (5, 700, 4000, 1, 5)])
def test_free(seqs, per, pages, page, live, dtype):
    import kda_recurrent_state_amd as kda
    pool = _pool(9, seqs, per, pages, page, live, shared=0.6)
    gen = torch.Generator().manual_seed(1)
    release = (torch.rand(seqs, generator=gen) < 0.5).to(dtype)
    if live > 4:
        s = [i for i in range(seqs) if pool[1][i] > 0]
        pool[0][s[0], 0] = -7         # a bad entry
        pool[1][s[1]] = 1 << 29       # a length no row holds
        release[s[0]] = release[s[1]] = 1
    dt, dl, dr = _dev(*pool)
    kda.kda_page_free(dt, dl, dr, release.cuda(), page)
    t, n, r = ref.free(*pool, release, page)
    assert torch.equal(dt.cpu(), t) and torch.equal(dl.cpu(), n) and torch.equal(dr.cpu(), r)
    kda.kda_page_free(dt, dl, dr, release.cuda(), page)   # nothing is left to free
    assert torch.equal(dt.cpu(), t) and torch.equal(dr.cpu(), r)


@pytest.mark.parametrize("seqs", [1 << 24, (1 << 24) - 4000, (1 << 20) + 300])
def test_compact_and_free_of_very_many_slots(seqs):
    """More slots than a launch has workgroups for (2^24 is the most a pool may
    have); those in use lie at both ends and between."""
    import kda_recurrent_state_amd as kda
    pages = 700
    gen = torch.Generator().manual_seed(13)
    slots = torch.tensor([0, 1, (1 << 20) - 1, 1 << 20, (1 << 20) + 1, seqs // 2, seqs - 2, seqs - 1]).unique()
    perm = torch.randperm(pages, generator=gen)[:2 * len(slots)].int().view(-1, 2)
    table = torch.full((seqs, 2), -1, dtype=torch.int32, device="cuda")
    table[slots.cuda()] = perm.cuda()
    lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    lens[slots.cuda()] = 2
    refs = torch.bincount(perm.view(-1).long(), minlength=pages).int().cuda()
    cache = torch.arange(pages, dtype=torch.int32)[:, None].repeat(1, 5).cuda()
    small = perm.clone(), _i32([2] * len(slots)), refs.cpu()
    live = kda.kda_page_compact(table, lens, refs, 1, caches=[cache])
    t, r, c, n = ref.compact(*small, 1, [torch.arange(pages, dtype=torch.int32)[:, None].repeat(1, 5)])
    assert live.item() == n and torch.equal(table[slots.cuda()].cpu(), t) and torch.equal(refs.cpu(), r)
    assert torch.equal(cache.cpu(), c[0])
    release = torch.zeros(seqs, dtype=torch.bool, device="cuda")
    release[slots[1:].cuda()] = True
    kda.kda_page_free(table, lens, refs, release, 1)
    assert lens.sum().item() == 2 and lens[0].item() == 2 and int((table >= 0).sum()) == 2
    want = torch.zeros(pages, dtype=torch.int32)
    want[t[0].long()] = 1
    assert torch.equal(refs.cpu(), want)


def test_pool_in_rows_of_a_wider_table_on_a_side_stream():
    import kda_recurrent_state_amd as kda
    pool = _pool(10, 20, 6, 200, 4, 10)
    wide = torch.full((20, 9), 77, dtype=torch.int32)
    wide[:, :6] = pool[0]
    dw, dl, dr = _dev(wide, pool[1], pool[2])
    full = [s for s in range(20) if pool[1][s] > 0]
    empty = [s for s in range(20) if pool[1][s] == 0]
    src, dst = _i32(full[:3]), _i32(empty[:3])
    side = torch.cuda.Stream()
    src_d, dst_d, rel = src.cuda(), dst.cuda(), torch.zeros(20, dtype=torch.bool)
    rel[full[0]] = True
    rel_d = rel.cuda()
    side.wait_stream(torch.cuda.current_stream())
    kda.kda_page_fork(dw[:, :6], dl, dr, src_d, dst_d, 4, stream=side)
    kda.kda_page_free(dw[:, :6], dl, dr, rel_d, 4, stream=side)
    kda.kda_page_compact(dw[:, :6], dl, dr, 4, stream=side)
    torch.cuda.synchronize()
    t, n, r, _, _ = ref.fork(*pool, src, dst, 4, [], True)
    t, n, r = ref.free(t, n, r, rel, 4)
    t, r, _, _ = ref.compact(t, n, r, 4, [])
    assert torch.equal(dw[:, :6].cpu(), t) and (dw[:, 6:] == 77).all()
    assert torch.equal(dl.cpu(), n) and torch.equal(dr.cpu(), r)


def test_page_graph_replays():
    """Free, fork and compact captured together and replayed on changing pools."""
    import kda_recurrent_state_amd as kda
    pools = [_pool(s, 24, 6, 300, 4, 10 + s) for s in range(4)]
    dt, dl, dr = _dev(*pools[0])
    src, dst = torch.zeros(4, dtype=torch.int32, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    rel = torch.zeros(24, dtype=torch.bool, device="cuda")
    cache = torch.zeros(300, 32, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    kda.kda_page_compact(dt, dl, dr, 4, caches=[cache])   # loaded before the capture
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kda.kda_page_free(dt, dl, dr, rel, 4)
        kda.kda_page_fork(dt, dl, dr, src, dst, 4, caches=[cache], status=status)
        kda.kda_page_compact(dt, dl, dr, 4, caches=[cache])
    for i, pool in enumerate(pools):
        for d, h in zip((dt, dl, dr), pool):
            d.copy_(h)
        full = [s for s in range(24) if pool[1][s] > 0]
        empty = [s for s in range(24) if pool[1][s] == 0]
        hs, hd = _i32(full[1:5]), _i32(empty[:3] + [full[0]])
        hr = torch.zeros(24, dtype=torch.bool)
        hr[full[0]] = True
        hc = torch.randn(300, 32, generator=torch.Generator().manual_seed(i))
        src.copy_(hs), dst.copy_(hd), rel.copy_(hr), cache.copy_(hc)
        g.replay()
        torch.cuda.synchronize()
        t, n, r = ref.free(*pool, hr, 4)
        t, n, r, c, s = ref.fork(t, n, r, hs, hd, 4, [hc], True)
        t, r, c, _ = ref.compact(t, n, r, 4, c)
        assert torch.equal(status.cpu(), s) and torch.equal(dt.cpu(), t) and torch.equal(dl.cpu(), n)
        assert torch.equal(dr.cpu(), r) and torch.equal(cache.cpu(), c[0])


def test_serving_run():
    """The operators as they are used together: prompts are expanded and their
    latent rows scattered into pages, sequences are forked, one ends, the pool
    is compacted, and decoding goes on; the attention of every step must be
    that of the sequences' own rows."""
    import kda_recurrent_state_amd as kda
    gen = torch.Generator().manual_seed(12)
    page, L, R, H, D, E, pages, seqs, per = 16, 128, 64, 4, 64, 64, 64, 6, 8
    rows = [torch.randn(n, L + R, generator=gen).bfloat16() for n in (37, 64, 5)]
    cache = torch.zeros(pages, page, L + R, dtype=torch.bfloat16, device="cuda")
    table = torch.full((seqs, per), -1, dtype=torch.int32)
    lens, at, perm = [0] * seqs, 0, torch.randperm(pages, generator=gen).tolist()
    for s, x in enumerate(rows):
        used = -(-len(x) // page)
        table[s, :used] = torch.tensor(perm[at:at + used], dtype=torch.int32)
        at, lens[s] = at + used, len(x)
    refs = torch.bincount(table[table >= 0].long(), minlength=pages).int()
    dt, dl, dr = _dev(table, _i32(lens), refs)
    tokens = cache.view(pages * page, 1, 1, L + R)   # one token a row, for the state copies

    def put(slot_tokens, values):   # scatter latent rows to (slot, position) pairs
        where = [int(dt[s, p // page]) * page + p % page for s, p in slot_tokens]
        kda.kda_state_scatter(tokens, _i32(where).cuda(), values.cuda().view(-1, 1, 1, L + R))

    put([(s, p) for s, x in enumerate(rows) for p in range(len(x))], torch.cat(rows))
    # prefill of the prompts, keys and values expanded from the latent rows
    wk, wv = torch.randn(L, H * D, generator=gen) / 11, torch.randn(L, H * E, generator=gen) / 11
    lat = torch.cat(rows)
    k = (lat[:, :L].float() @ wk).bfloat16().view(-1, H, D).cuda()
    v = (lat[:, :L].float() @ wv).bfloat16().view(-1, H, E).cuda()
    q = torch.randn(len(lat), H, D + R, generator=gen).bfloat16().cuda()
    cu = [0, 37, 101, 106]
    got = kda.kda_latent_prefill(q, k, v, _i32(cu).cuda(), k_rope=lat[:, L:].cuda(), with_lse=True)
    ref.check(*got, ref.prefill(q, k, v, lat[:, L:], cu, cu, (D + R) ** -0.5, True), "prompts")

    have = {s: x for s, x in enumerate(rows)}
    status = kda.kda_page_fork(dt, dl, dr, _i32([0, 1]).cuda(), _i32([3, 5]).cuda(), page, caches=[cache])
    assert status.tolist() == [0, 0]
    have[3], have[5] = have[0], have[1]
    gone = torch.zeros(seqs, dtype=torch.bool)
    gone[0] = True
    kda.kda_page_free(dt, dl, dr, gone.cuda(), page)
    del have[0]
    live = kda.kda_page_compact(dt, dl, dr, page, caches=[cache])
    assert live.item() == int((dr > 0).sum()) and (dr[:live.item()] > 0).all()
    for step in range(3):   # slots 3 and 5 part from their parents, 1 stays inside its last page's end
        slots = sorted(s for s in have if s not in (1, 5) or step == 99)
        new = torch.randn(len(slots), L + R, generator=gen).bfloat16()
        put([(s, len(have[s])) for s in slots], new)
        for s, x in zip(slots, new):
            have[s] = torch.cat([have[s], x[None]])
            dl[s] += 1
        order = sorted(have)
        ql = torch.randn(len(order), H, L, generator=gen).bfloat16().cuda()
        qr = torch.randn(len(order), H, R, generator=gen).bfloat16().cuda()
        got = kda.kda_latent_decode(cache, dt[order], dl[order], ql, qr, scale=0.1, with_lse=True)
        flat = torch.cat([torch.cat([have[s], torch.zeros(-len(have[s]) % 16, L + R).bfloat16()]) for s in order])
        used = [-(-len(have[s]) // 16) for s in order]
        tb, a = torch.zeros(len(order), max(used), dtype=torch.int32), 0
        for i, u in enumerate(used):
            tb[i, :u] = torch.arange(a, a + u)
            a += u
        want = ref.decode(flat.view(-1, 16, L + R), tb, _i32([len(have[s]) for s in order]), ql[:, None], qr[:, None],
                          0.1)
        ref.check(*got, want, "step %d" % step)
    assert not math.isnan(float(cache.float().sum()))
