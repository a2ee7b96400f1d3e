"""Latent attention on the GPU (expanded varlen prefill, absorbed paged
decode) against plain fp64 evaluations."""
import math

import pytest
import torch

from tests import latent_ref as ref
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    ensure_built()


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen).to(BF16)


def _cu(lens):
    out = [0]
    for n in lens:
        out.append(out[-1] + n)
    return out


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# --- prefill ----------------------------------------------------------------

def _prefill_inputs(lq, lk, H, D, R, E, seed=1):
    gen = torch.Generator().manual_seed(seed)
    T, S = sum(lq), sum(lk)
    kv = _randn(gen, S, H, D + E).cuda()
    rows = _randn(gen, S, 64 + R).cuda() if R else None
    return dict(q=_randn(gen, T, H, D + R).cuda(), k=kv[..., :D], v=kv[..., D:],
                k_rope=rows[:, 64:] if R else None)


def _prefill(x, lq, lk, causal=True, scale=None, **kw):
    import kda_recurrent_state_amd as kda
    return kda.kda_latent_prefill(x["q"], x["k"], x["v"], _i32(_cu(lq)), k_rope=x["k_rope"],
                                  cu_seqlens_k=_i32(_cu(lk)), causal=causal, scale=scale, with_lse=True, **kw)


def _check_prefill(x, lq, lk, causal, got, scale=None):
    want = ref.prefill(x["q"], x["k"], x["v"], x["k_rope"], _cu(lq), _cu(lk),
                       x["q"].shape[2] ** -0.5 if scale is None else scale, causal)
    ref.check(*got, want, "prefill")


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lq,past", [
    ([1], [0]), ([1], [200]), ([64], [0]), ([65, 1, 63], [0, 0, 0]), ([128, 129, 127, 2], [0, 64, 1, 500]),
    ([0, 33, 0, 300, 0], [0, 31, 7, 0, 64]), ([517], [1])])
def test_prefill_lengths(lq, past, causal):
    lk = [a + b for a, b in zip(lq, past)]
    x = _prefill_inputs(lq, lk, 2, 128, 64, 128)
    _check_prefill(x, lq, lk, causal, _prefill(x, lq, lk, causal))


@pytest.mark.parametrize("H,D,R,E", [(1, 128, 64, 128), (5, 64, 32, 64), (3, 128, 0, 128), (2, 96, 32, 80),
                                     (2, 8, 0, 8), (4, 8, 8, 128), (3, 120, 56, 24), (2, 64, 64, 128)])
def test_prefill_dims(H, D, R, E):
    lq, lk = [70, 5, 200], [70, 90, 201]
    x = _prefill_inputs(lq, lk, H, D, R, E)
    _check_prefill(x, lq, lk, True, _prefill(x, lq, lk, True))


@pytest.mark.parametrize("lq,past,H,causal", [([1], [5000], 3, True), ([130], [4000], 8, True),
                                              ([70, 3], [2200, 9000], 2, True), ([200], [2100], 5, False),
                                              ([40, 0, 1], [0, 6000, 3000], 16, True), ([2300], [0], 1, True)])
def test_prefill_few_queries_over_many_keys(lq, past, H, causal):
    """The keys are split over workgroups and the pieces joined; a workspace of
    the caller's that holds NaN gives the same."""
    import kda_recurrent_state_amd as kda
    lk = [a + b for a, b in zip(lq, past)]
    need = kda.kda_latent_prefill_workspace_size(sum(lq), sum(lk), len(lq), H, 80)
    assert need > 0
    x = _prefill_inputs(lq, lk, H, 96, 32, 80)
    got = _prefill(x, lq, lk, causal)
    _check_prefill(x, lq, lk, causal, got)
    ws = torch.full((need // 4,), math.nan, device="cuda")
    again = _prefill(x, lq, lk, causal, workspace=ws)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


def test_prefill_split_keys_leave_other_rows():
    """Rows of q outside the sequences, with the keys split."""
    import kda_recurrent_state_amd as kda
    x = _prefill_inputs([50], [5000], 2, 64, 0, 64)
    cu_q, cu_k = [5, 5, 41], [100, 100, 4900]
    out = torch.full((50, 2, 64), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((50, 2), 7.0, device="cuda")
    kda.kda_latent_prefill(x["q"], x["k"], x["v"], _i32(cu_q), cu_seqlens_k=_i32(cu_k), out=out, lse=lse)
    want = ref.prefill(x["q"], x["k"], x["v"], None, cu_q, cu_k, 64 ** -0.5, True)
    ref.check(out[5:41], lse[5:41], [w[5:41] for w in want], "rows")
    assert (out[:5] == 7).all() and (out[41:] == 7).all() and (lse[:5] == 7).all() and (lse[41:] == 7).all()


def test_prefill_graph_follows_offsets():
    """A captured call whose offsets change between replays, keys split."""
    x = _prefill_inputs([60], [6000], 4, 64, 32, 64)
    import kda_recurrent_state_amd as kda
    cu_q, cu_k = _i32([0, 60, 60]), _i32([0, 6000, 6000])
    out, lse = torch.zeros(60, 4, 64, dtype=BF16, device="cuda"), torch.zeros(60, 4, device="cuda")
    ws = torch.empty(kda.kda_latent_prefill_workspace_size(60, 6000, 2, 4, 64), dtype=torch.uint8, device="cuda")
    call = lambda o, s, w: kda.kda_latent_prefill(x["q"], x["k"], x["v"], cu_q, k_rope=x["k_rope"],  # noqa: E731
                                                  cu_seqlens_k=cu_k, out=o, lse=s, workspace=w)
    call(out, lse, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(out, lse, ws)
    for a, b in (([0, 60, 60], [0, 6000, 6000]), ([0, 1, 60], [0, 4000, 6000]), ([0, 30, 60], [0, 10, 5000])):
        cu_q.copy_(_i32(a))
        cu_k.copy_(_i32(b))
        g.replay()
        torch.cuda.synchronize()
        eager = call(torch.zeros_like(out), torch.zeros_like(lse), None)
        torch.cuda.synchronize()
        assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])
        ref.check(out, lse, ref.prefill(x["q"], x["k"], x["v"], x["k_rope"], a, b, 96 ** -0.5, True), "graph %s" % a)


def test_nothing_to_do_and_empty_sides():
    import kda_recurrent_state_amd as kda
    z = lambda *s: torch.zeros(*s, dtype=BF16, device="cuda")  # noqa: E731
    out, lse = kda.kda_latent_prefill(z(0, 2, 64), z(5, 2, 64), z(5, 2, 64), _i32([0, 0]), cu_seqlens_k=_i32([0, 5]),
                                      with_lse=True)
    assert out.shape == (0, 2, 64) and lse.shape == (0, 2)
    out, lse = kda.kda_latent_prefill(z(3, 2, 64), z(0, 2, 64), z(0, 2, 64), _i32([0, 3]), cu_seqlens_k=_i32([0, 0]),
                                      with_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    out, lse = kda.kda_latent_decode(z(2, 16, 64), torch.zeros(0, 3, dtype=torch.int32, device="cuda"), _i32([]),
                                     z(0, 4, 64), scale=1.0, with_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_calls_on_two_streams_at_once():
    """Decode and split prefill of different inputs under way together: each
    call has a workspace of its own."""
    a = _decode_inputs([3000, 40, 900], 2, 32, 512, 64, 64, seed=21)
    b = _decode_inputs([100, 5000], 1, 64, 256, 32, 16, seed=22)
    c = _prefill_inputs([33], [7000], 4, 128, 64, 128, seed=23)
    alone = [_decode(a), _decode(b), _prefill(c, [33], [7000])]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = [_decode(a, stream=streams[0]), _decode(b, stream=streams[1]),
               _prefill(c, [33], [7000], stream=streams[2])]
        torch.cuda.synchronize()
        for x, y in zip(alone, got):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_prefill_rows_that_see_nothing():
    # more queries than keys: the first ones see none; and a sequence without keys
    lq, lk = [100, 40, 70], [30, 0, 70]
    x = _prefill_inputs(lq, lk, 3, 128, 64, 128)
    out, lse = _prefill(x, lq, lk, True)
    _check_prefill(x, lq, lk, True, (out, lse))
    assert (out[:70] == 0).all() and (lse[:70] == -math.inf).all()
    assert (out[100:140] == 0).all() and (lse[100:140] == -math.inf).all()


def test_prefill_large_scores_and_scale():
    # scores of several hundred: one weight takes all, the running maximum jumps
    lq = lk = [150, 90]
    x = _prefill_inputs(lq, lk, 2, 128, 64, 128)
    x["q"] = x["q"] * 8
    # (|s| reaches about 500: its fp32 rounding alone moves a weight by 2^-14,
    # inside the bound's 2^-12; lse is held to 1e-4 as 500 x 2^-24 = 3e-5)
    _check_prefill(x, lq, lk, True, _prefill(x, lq, lk, True, scale=0.5), scale=0.5)


def test_prefill_strides_and_other_rows():
    """Token and head strides of every tensor, a broadcast rotary key, and rows
    of q before and behind the sequences, whose outputs stay as they were."""
    import kda_recurrent_state_amd as kda
    gen = torch.Generator().manual_seed(3)
    H, D, R, E, T, S = 3, 64, 16, 40, 200, 180
    q = _randn(gen, H, T, 96).cuda().transpose(0, 1)[..., 8:8 + D + R]
    k = _randn(gen, H, S, D).cuda().transpose(0, 1)
    v = _randn(gen, S, 1, E).cuda().expand(S, H, E)
    kr = _randn(gen, 1, R).cuda().expand(S, R)
    cu_q, cu_k = [10, 60, 60, 187], [20, 70, 75, 180]
    out = torch.full((T, H, E), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((T, H), 7.0, device="cuda")
    kda.kda_latent_prefill(q, k, v, _i32(cu_q), k_rope=kr, cu_seqlens_k=_i32(cu_k), out=out, lse=lse, scale=0.1)
    want = ref.prefill(q, k, v, kr, cu_q, cu_k, 0.1, True)
    ref.check(out[10:187], lse[10:187], [w[10:187] for w in want], "strided")
    assert (out[:10] == 7).all() and (out[187:] == 7).all() and (lse[:10] == 7).all() and (lse[187:] == 7).all()


def test_prefill_unseen_keys_may_be_anything():
    """NaN and infinities in keys that a query does not see, in value rows
    behind a sequence, and in the padding between sequences."""
    import kda_recurrent_state_amd as kda
    lq, lk = [100, 30], [100, 50]
    x = _prefill_inputs(lq, [100, 50, 60], 2, 128, 64, 128)
    for t, bad in ((x["k"], math.nan), (x["v"], math.inf), (x["k_rope"], math.nan)):
        t[150:] = bad
    x["k"][80:100] = math.inf
    x["k_rope"][90:100] = math.nan
    out, lse = kda.kda_latent_prefill(x["q"], x["k"], x["v"], _i32(_cu(lq)), k_rope=x["k_rope"],
                                      cu_seqlens_k=_i32(_cu(lk)), with_lse=True)
    want = ref.prefill(x["q"], x["k"], x["v"], x["k_rope"], _cu(lq), _cu(lk), 192 ** -0.5, True)
    for a, b in ((0, 80), (100, 130)):
        ref.check(out[a:b], lse[a:b], [w[a:b] for w in want], "unseen %d" % a)


def test_prefill_bad_offsets_stay_inside():
    """Offsets outside the tensors are clamped: the call ends and the sound
    sequence is right."""
    import kda_recurrent_state_amd as kda
    x = _prefill_inputs([90], [90], 2, 64, 32, 64)
    out = torch.zeros(90, 2, 64, dtype=BF16, device="cuda")
    kda.kda_latent_prefill(x["q"], x["k"], x["v"], _i32([0, 50, 4000, -7, 90]), k_rope=x["k_rope"],
                           cu_seqlens_k=_i32([0, 50, 9000, 60, -1]), out=out)
    torch.cuda.synchronize()
    want = ref.prefill(x["q"][:50], x["k"][:50], x["v"][:50], x["k_rope"][:50], [0, 50], [0, 50], 96 ** -0.5, True)
    ref.check(out[:50], None, want, "clamped")


@pytest.mark.parametrize("cu_q", [[0, 50, 20, 90], [10, 5, 80, 80, 30, 90], [-4, 40, 400, 0, 90], [90, 0, 90],
                                  [0] + [30, 10] * 40 + [70, 60, 90], [(37 * i) % 91 for i in range(150)]])
def test_prefill_query_offsets_that_fall(cu_q):
    """A query offset below one before it is raised to it: no row has two
    writers, whatever the offsets, and rows of no sequence stay as they were."""
    import kda_recurrent_state_amd as kda
    x = _prefill_inputs([90], [90], 2, 64, 32, 64)
    cu_k = [(29 * i) % 60 + (40 if i % 2 else 0) for i in range(len(cu_q))]
    sound, k_ranges = [], []
    for i, c in enumerate(cu_q):
        sound.append(max([min(max(c, 0), 90)] + sound[-1:]))
        k0, k1 = min(cu_k[i], 90), min(cu_k[min(i + 1, len(cu_k) - 1)], 90)
        k_ranges.append((k0, max(k0, k1)))
    out = torch.full((90, 2, 64), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((90, 2), 7.0, device="cuda")
    kda.kda_latent_prefill(x["q"], x["k"], x["v"], _i32(cu_q), k_rope=x["k_rope"], cu_seqlens_k=_i32(cu_k), out=out,
                           lse=lse)
    torch.cuda.synchronize()
    seen = torch.zeros(90, dtype=torch.bool)
    for a, b, (c, d) in zip(sound, sound[1:], k_ranges):
        if a == b:
            continue
        seen[a:b] = True
        want = ref.prefill(x["q"][a:b], x["k"][c:d], x["v"][c:d], x["k_rope"][c:d], [0, b - a], [0, d - c], 96 ** -0.5,
                           True)
        ref.check(out[a:b], lse[a:b], want, "rows %d to %d" % (a, b))
    assert (out[~seen.cuda()] == 7).all() and (lse[~seen.cuda()] == 7).all()


@pytest.mark.parametrize("D,R,E", [(96, 32, 80), (64, 0, 128), (64, 32, 128), (120, 56, 24), (8, 8, 8), (64, 16, 64),
                                   (40, 0, 64), (128, 64, 128)])
@pytest.mark.parametrize("lq,past", [([70, 5, 130], [0, 85, 3]), ([40], [3000])])
def test_prefill_keys_with_infinite_components(D, R, E, lq, past):
    """A score bias in the last column of the keys (and of the rotary keys):
    -inf takes a key out, at every width; queries of which no key is left get 0
    and -inf."""
    lk = [a + b for a, b in zip(lq, past)]
    x = _prefill_inputs(lq, lk, 2, D, R, E)
    gen = torch.Generator().manual_seed(31)
    S = sum(lk)
    out = torch.rand(S, generator=gen) < 0.3
    out[:3] = True
    x["q"][..., D - 1] = 1
    x["k"][..., D - 1] = torch.where(out, -math.inf, 0.25).to(BF16).cuda()[:, None]
    if R:
        x["q"][..., D + R - 1] = 1
        x["k_rope"][..., R - 1] = torch.where(torch.rand(S, generator=gen) < 0.2, -math.inf, 0.0).to(BF16).cuda()
    _check_prefill(x, lq, lk, True, _prefill(x, lq, lk, True))


@pytest.mark.parametrize("low", [torch.finfo(BF16).min, -1e30, 1e30])
@pytest.mark.parametrize("lq,past,H", [([70, 5, 130], [0, 85, 3], 2), ([40], [1200], 3)])
def test_prefill_scores_of_the_types_range(lq, past, H, low):
    """A mask of the type's lowest value as a score bias.  Where nothing but
    such keys is seen, their scores are equal (the rest of the sum is below
    half a step) and the output is the mean of their values."""
    lk = [a + b for a, b in zip(lq, past)]
    x = _prefill_inputs(lq, lk, H, 128, 64, 128)
    gen = torch.Generator().manual_seed(32)
    masked = torch.rand(sum(lk), generator=gen) < 0.5
    masked[:40] = True
    masked[-sum(lk) // 3:] = True
    x["q"][..., 127] = 1
    x["q"][:, 0, 127] = 0   # a head without the bias
    x["k"][..., 127] = torch.where(masked, low, 0.0).to(BF16).cuda()[:, None]
    if past[0]:
        x["k"][..., 127] = low   # all of them
    out, lse = _prefill(x, lq, lk, True)
    want = ref.prefill(x["q"], x["k"], x["v"], x["k_rope"], _cu(lq), _cu(lk), 192 ** -0.5, True, ref.attend_far)
    ref.check(out, None, want, "range")
    _check_lse_range(lse, want[1])


def test_prefill_scores_of_the_types_range_over_many_tiles():
    """As above over several key tiles of a workgroup (no split): a mask over all
    keys, or over the first half of them."""
    import kda_recurrent_state_amd as kda
    lq = lk = [1100, 900]
    x = _prefill_inputs(lq, lk, 32, 64, 32, 64)
    assert kda.kda_latent_prefill_workspace_size(2000, 2000, 2, 32, 64) == 0
    x["q"][..., 95] = 1
    x["q"][:, 0, 95] = 0
    x["k_rope"][:, 31] = 0
    x["k_rope"][:1100, 31] = torch.finfo(BF16).min
    x["k_rope"][1100:1550, 31] = torch.finfo(BF16).min
    out, lse = _prefill(x, lq, lk, True)
    want = ref.prefill(x["q"], x["k"], x["v"], x["k_rope"], _cu(lq), _cu(lk), 96 ** -0.5, True, ref.attend_far)
    ref.check(out, None, want, "range")
    _check_lse_range(lse, want[1])


def _check_lse_range(lse, want):
    """Near scores of 1e30 and more lse is held relatively: the factor to base 2
    and back is rounded six times (the scale, its product with log2 e, log2 e,
    the score's product, ln 2 and its product), each by 2^-24 at most."""
    got = lse.cpu().double().reshape(want.shape)
    empty = want == -math.inf
    assert torch.equal(got == -math.inf, empty)
    got, want = got[~empty], want[~empty]
    assert ((got - want).abs() <= torch.where(want.abs() < 1e6, torch.full_like(want, 1e-4), want.abs() * 2.0 ** -21)).all()


def test_prefill_many_sequences():
    # more sequences than one scan step of a wave, most of them tiny
    lq = [(7 * i) % 5 for i in range(150)] + [140, 1]
    lk = [n + (i % 3) for i, n in enumerate(lq)]
    x = _prefill_inputs(lq, lk, 2, 64, 32, 64)
    _check_prefill(x, lq, lk, True, _prefill(x, lq, lk, True))


def test_prefill_is_repeatable_and_follows_a_side_stream():
    lq, lk = [300, 77], [400, 77]
    x = _prefill_inputs(lq, lk, 4, 128, 64, 128)
    one = _prefill(x, lq, lk)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    two = _prefill(x, lq, lk, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(one[0], two[0]) and torch.equal(one[1], two[1])


# --- decode -----------------------------------------------------------------

def _decode_inputs(lens, Q, H, L, R, page, seed=2, width=None, gap=0):
    gen = torch.Generator().manual_seed(seed)
    N = len(lens)
    used = [-(-max(n, 0) // page) for n in lens]
    width = width or max(used) + 1
    pages = sum(used) + 3
    perm = torch.randperm(pages, generator=gen).tolist()
    table = torch.full((N, width), -1, dtype=torch.int32)
    at = 0
    for n, u in enumerate(used):
        table[n, :u] = torch.tensor(perm[at:at + u], dtype=torch.int32)
        at += u
    flat = _randn(gen, pages, page * (L + R) + gap).cuda()
    cache = torch.as_strided(flat, (pages, page, L + R), (page * (L + R) + gap, L + R, 1))
    return dict(cache=cache, table=table.cuda(), lens=_i32(lens), q=_randn(gen, N, Q, H, L).cuda(),
                q_rope=_randn(gen, N, Q, H, R).cuda() if R else None)


def _decode(x, scale=0.07, **kw):
    import kda_recurrent_state_amd as kda
    return kda.kda_latent_decode(x["cache"], x["table"], x["lens"], x["q"], x["q_rope"], scale=scale, with_lse=True,
                                 **kw)


def _check_decode(x, got, scale=0.07, name="decode"):
    ref.check(*got, ref.decode(x["cache"], x["table"], x["lens"], x["q"], x["q_rope"], scale), name)


@pytest.mark.parametrize("lens", [[1], [64], [65], [0], [1000], [3, 0, 130, 64, 0, 1], [700, 63, 2000],
                                  [40] * 70, [1] * 300])
@pytest.mark.parametrize("H", [3, 32])
def test_decode_lengths(lens, H):
    x = _decode_inputs(lens, 1, H, 512, 64, 64)
    _check_decode(x, _decode(x))


@pytest.mark.parametrize("Q,H,L,R,page", [(1, 1, 512, 64, 16), (2, 8, 256, 32, 48), (3, 20, 128, 64, 1),
                                          (1, 128, 512, 64, 64), (1, 40, 384, 0, 128), (4, 5, 8, 8, 7),
                                          (2, 64, 504, 56, 33), (1, 16, 136, 0, 64), (5, 1, 256, 64, 200),
                                          (1, 17, 512, 64, 64)])
def test_decode_dims(Q, H, L, R, page):
    x = _decode_inputs([300, 1, 2, 77, 129], Q, H, L, R, page)
    _check_decode(x, _decode(x))


def test_decode_long_context_is_split():
    x = _decode_inputs([30000, 5], 1, 32, 512, 64, 64)
    _check_decode(x, _decode(x, scale=0.3), scale=0.3)


RAGGED = [700, 0, 63, 129, 2000, 1, 320, 64, 65, 0, 0, 1500, 128, 3, 900]


@pytest.mark.parametrize("lens,Q,H,L,R,page", [
    (RAGGED, 4, 256, 512, 64, 16),            # 16 row blocks and shares: 5 to 6 tiles a share
    (RAGGED * 2, 1, 1000, 256, 32, 48),       # 16 shares
    (RAGGED * 6, 1, 128, 512, 64, 64),        # two row blocks, 128 shares
    (RAGGED * 12, 2, 32, 512, 64, 64),        # 64 query rows, 256 shares, 4 tiles a share
    (RAGGED * 12, 1, 20, 504, 56, 33),        # 32 rows
    (RAGGED * 12, 1, 32, 512, 0, 128),
    (RAGGED * 16, 1, 7, 128, 64, 1),          # 16 rows
    (RAGGED * 16, 3, 3, 512, 64, 7),
    ([0, 20000, 0, 1] + [70] * 130 + [9000], 1, 5, 136, 8, 16)])
@pytest.mark.parametrize("grow", [0, 4])
def test_decode_many_tiles_a_share(lens, Q, H, L, R, page, grow):
    """Shares of several tiles, which end one sequence, hold others (empty ones
    among them) and begin another.  With ``grow`` a sequence's rows get larger
    to its end, so that the maxima grow by far more than 2^8 on the way: scores
    of up to about 400 before the scale of 0.07, whose fp32 rounding (576
    products, 24 x 2^-24 x 400 x 0.07 = 4e-5) the bound of lse holds."""
    x = _decode_inputs(lens, Q, H, L, R, page)
    if grow:
        for n, k in enumerate(lens):
            pages = x["table"][n, :-(-k // page)].long()
            f = torch.linspace(0, grow, pages.shape[0] * page, device="cuda").view(-1, page, 1)
            x["cache"][pages] = (x["cache"][pages].float() * f * (576 / (L + R)) ** 0.5).to(BF16)
    _check_decode(x, _decode(x))


def test_decode_queries_before_the_first_token():
    # three new tokens, lengths 0 .. 3: the first queries see nothing
    x = _decode_inputs([0, 1, 2, 3], 3, 4, 512, 64, 64)
    out, lse = _decode(x)
    _check_decode(x, (out, lse))
    assert (out[1, :2] == 0).all() and (lse[1, :2] == -math.inf).all() and (out[0] == 0).all()


def test_decode_bad_pages_and_lengths():
    """Table entries outside the pool are not seen (a whole tile of them too),
    lengths outside the table are clamped."""
    x = _decode_inputs([500, 300, 128, 90], 2, 8, 512, 64, 16)
    x["table"][0, 3] = -1
    x["table"][0, 8:12] = 1 << 30
    x["table"][2, :] = -5
    x["lens"][1] = 1 << 29
    x["lens"][3] = -4
    out, lse = _decode(x)
    _check_decode(x, (out, lse))
    assert (out[2] == 0).all() and (lse[2] == -math.inf).all() and (out[3] == 0).all()


def test_decode_rows_behind_the_length_may_be_anything():
    x = _decode_inputs([70, 130, 10], 1, 16, 512, 64, 64, gap=64)
    used = {(int(x["table"][n, j // 64]), j % 64) for n, k in enumerate([70, 130, 10]) for j in range(k)}
    mask = torch.ones(x["cache"].shape[:2], dtype=torch.bool)
    for p, s in used:
        mask[p, s] = False
    want = ref.decode(x["cache"], x["table"], x["lens"], x["q"], x["q_rope"], 0.07)
    x["cache"][mask.cuda()] = math.nan
    ref.check(*_decode(x), want, "behind")


@pytest.mark.parametrize("L,R", [(512, 56), (136, 24), (504, 56), (256, 32), (8, 8), (128, 8), (512, 64)])
@pytest.mark.parametrize("Q,H", [(1, 5), (2, 20), (1, 64)])
def test_decode_rotary_keys_with_infinite_components(L, R, Q, H):
    """A score bias in the last rotary column: -inf takes a row out, at every
    width; a sequence of which no row is left gets 0 and -inf."""
    lens = [300, 2, 70, 129]
    x = _decode_inputs(lens, Q, H, L, R, 16)
    gen = torch.Generator().manual_seed(33)
    x["q_rope"][..., R - 1] = 1
    x["cache"][..., L + R - 1] = torch.where(torch.rand(x["cache"].shape[:2], generator=gen) < 0.3, -math.inf, 0.5).to(BF16)
    x["cache"][x["table"][2, :5].long(), :, L + R - 1] = -math.inf
    out, lse = _decode(x)
    _check_decode(x, (out, lse))
    assert (out[2] == 0).all() and (lse[2] == -math.inf).all()


@pytest.mark.parametrize("L,R", [(384, 0), (136, 0), (504, 56), (40, 8), (264, 64)])
def test_decode_latents_with_infinite_components(L, R):
    """-inf in a latent row's last value, which the queries take as it is: the
    row has weight 0, and the other columns of the output do not see it."""
    x = _decode_inputs([200, 65, 3], 1, 6, L, R, 64)
    gen = torch.Generator().manual_seed(34)
    x["q"][..., L - 1] = 1
    bad = torch.rand(x["cache"].shape[:2], generator=gen) < 0.3
    x["cache"][..., L - 1] = torch.where(bad, -math.inf, 0.5).to(BF16)
    out, lse = _decode(x)
    want = ref.decode(x["cache"], x["table"], x["lens"], x["q"], x["q_rope"], 0.07)
    ref.check(out[..., :L - 1], lse, [want[0][..., :L - 1], want[1], want[2][..., :L - 1]], "latent bias")


@pytest.mark.parametrize("low", [torch.finfo(BF16).min, -1e30, 1e30])
@pytest.mark.parametrize("Q,H", [(1, 3), (2, 32)])
@pytest.mark.parametrize("lens", [[64, 40, 9, 17], [130, 300, 70, 2000]])
def test_decode_scores_of_the_types_range(lens, Q, H, low):
    """As test_prefill_scores_of_the_types_range: rows masked by the type's
    lowest value, all of a sequence's or some; longer sequences are in pieces of
    unequal length."""
    x = _decode_inputs(lens, Q, H, 512, 64, 16)
    gen = torch.Generator().manual_seed(35)
    x["q_rope"][..., 63] = 1
    x["q_rope"][:, :, 0, 63] = 0   # a head without the bias
    x["cache"][..., 575] = torch.where(torch.rand(x["cache"].shape[:2], generator=gen) < 0.5, low, 0.0).to(BF16)
    for n in (0, 3):
        x["cache"][x["table"][n, :-(-lens[n] // 16)].long(), :, 575] = low
    out, lse = _decode(x)
    want = ref.decode(x["cache"], x["table"], x["lens"], x["q"], x["q_rope"], 0.07, ref.attend_far)
    ref.check(out, None, want, "range")
    _check_lse_range(lse, want[1])


@pytest.mark.parametrize("Q,H,L,R", [(4, 256, 512, 64), (1, 1000, 136, 24)])
def test_decode_scores_of_the_types_range_over_many_tiles(Q, H, L, R):
    """Rows masked by the type's lowest value over several tiles of a share: all
    of every third sequence, the first half of the next, every other row of the
    last."""
    low = torch.finfo(BF16).min
    x = _decode_inputs(RAGGED, Q, H, L, R, 16)
    x["q_rope"][..., R - 1] = 1
    x["q_rope"][:, :, 0, R - 1] = 0
    x["cache"][..., L + R - 1] = 0
    for n, k in enumerate(RAGGED):
        pages = x["table"][n, :-(-k // 16)].long()
        bias = torch.zeros(pages.shape[0] * 16)
        bias[:[k, k // 2, k][n % 3]:[1, 1, 2][n % 3]] = low
        x["cache"][pages, :, L + R - 1] = bias.view(-1, 16).to(BF16).cuda()
    out, lse = _decode(x)
    want = ref.decode(x["cache"], x["table"], x["lens"], x["q"], x["q_rope"], 0.07, ref.attend_far)
    ref.check(out, None, want, "range")
    _check_lse_range(lse, want[1])


def test_decode_strides():
    """q as the transposed result of a product by head, q_rope as the end of a
    joint projection, pages with a gap, rows of a wider table, 3-D q."""
    import kda_recurrent_state_amd as kda
    x = _decode_inputs([100, 217, 64], 1, 12, 256, 32, 16, gap=24, width=40)
    gen = torch.Generator().manual_seed(9)
    q = _randn(gen, 12, 3, 256).cuda().transpose(0, 1)
    q_rope = _randn(gen, 3, 12, 96).cuda()[..., 64:]
    table = x["table"][:, :20]
    out, lse = kda.kda_latent_decode(x["cache"], table, x["lens"], q, q_rope, scale=0.1, with_lse=True)
    assert out.shape == (3, 12, 256) and lse.shape == (3, 12)
    ref.check(out, lse, ref.decode(x["cache"], table, x["lens"], q[:, None], q_rope[:, None], 0.1), "strided")


def test_decode_cache_beyond_four_gib():
    """Pages far apart: row addresses pass 32 bits."""
    stride = (1 << 31) // 2 + 8 * 64   # elements: 2 GiB and a gap from page to page
    flat = torch.zeros(5 * stride + 16 * 144, dtype=BF16, device="cuda")
    cache = torch.as_strided(flat, (6, 16, 144), (stride, 144, 1))
    gen = torch.Generator().manual_seed(4)
    cache.copy_(_randn(gen, 6, 16, 144))
    x = dict(cache=cache, table=_i32([[5, 0, 3], [4, 1, 2]]), lens=_i32([48, 33]),
             q=_randn(gen, 2, 1, 4, 128).cuda(), q_rope=_randn(gen, 2, 1, 4, 16).cuda())
    _check_decode(x, _decode(x))


def test_decode_graph_follows_lengths_and_table():
    """A captured call replayed with other lengths, pages and queries between
    eager calls; two graphs with workspaces of their own."""
    import kda_recurrent_state_amd as kda
    x = _decode_inputs([300, 20, 700], 1, 32, 512, 64, 64, width=32)
    out = torch.empty_like(x["q"])
    ws = [torch.empty(kda.kda_latent_decode_workspace_size(3, 1, 32, 512), dtype=torch.uint8, device="cuda")
          for _ in range(2)]
    outs = [torch.empty_like(x["q"]) for _ in range(2)]
    _decode(x, out=out)
    graphs = []
    for w, o in zip(ws, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kda.kda_latent_decode(x["cache"], x["table"], x["lens"], x["q"], x["q_rope"], scale=0.07, out=o,
                                  workspace=w)
        graphs.append(g)
    gen = torch.Generator().manual_seed(8)
    for lens in ([300, 20, 700], [1, 0, 64], [901, 65, 3], [500, 500, 500]):
        x["lens"].copy_(_i32(lens))
        x["table"].copy_(torch.randint(0, x["cache"].shape[0], x["table"].shape, generator=gen, dtype=torch.int32))
        x["q"].copy_(_randn(gen, *x["q"].shape))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        eager = _decode(x, out=out)[0].clone()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], eager) and torch.equal(outs[1], eager)
        _check_decode(x, (eager, None), name="graph %s" % lens)


def test_decode_on_a_side_stream_and_shared_pages():
    # two sequences share pages (a forked prefix); the binding allocates on the side stream's behalf
    x = _decode_inputs([200, 260], 1, 32, 512, 64, 64)
    x["table"][1, :3] = x["table"][0, :3]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = _decode(x, stream=side)
    torch.cuda.synchronize()
    _check_decode(x, got)


def test_decode_matches_the_expanded_form():
    """One head's up-projections applied on either side: absorbed decode of the
    last token equals expanded prefill of it, up to both roundings."""
    import kda_recurrent_state_amd as kda
    gen = torch.Generator().manual_seed(11)
    T, H, L, R, D, E = 150, 4, 512, 64, 128, 128
    c = torch.randn(T, L, generator=gen).to(BF16)
    kr = _randn(gen, T, R)
    uk = (torch.randn(H, D, L, generator=gen) * L ** -0.5)
    uv = (torch.randn(H, E, L, generator=gen) * L ** -0.5)
    qn, qr = torch.randn(1, H, D, generator=gen), _randn(gen, 1, H, R)
    scale = (D + R) ** -0.5
    k = torch.einsum("tl,hdl->thd", c.float(), uk)
    v = torch.einsum("tl,hel->the", c.float(), uv)
    exp_out, _ = kda.kda_latent_prefill(torch.cat([qn.to(BF16), qr], -1).cuda(), k.to(BF16).cuda(), v.to(BF16).cuda(),
                                        _i32([0, 1]), k_rope=kr.cuda(), cu_seqlens_k=_i32([0, T]))
    ql = torch.einsum("nhd,hdl->nhl", qn.to(BF16).float(), uk).to(BF16)
    cache = torch.zeros(3, 64, L + R, dtype=BF16)
    cache.view(192, L + R)[:T] = torch.cat([c, kr], -1)
    lat, _ = kda.kda_latent_decode(cache.cuda(), _i32([[0, 1, 2]]), _i32([T]), ql.cuda(), qr.cuda(), scale=scale)
    abs_out = torch.einsum("nhl,hel->nhe", lat.float().cpu(), uv)
    # roundings to bf16 (2^-8 each at most) on the way: k or q_latent (moves a
    # score by up to 2^-8 of sum |q k| / ..., here under 0.02), v, weights, latent
    # output, output: 5 x 2^-8 = 0.02 and the scores' 0.02 of |v| of order 1
    assert (abs_out - exp_out.float().cpu()).abs().max() <= 0.04
