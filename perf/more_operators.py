"""Timed cases of the 8-bit latent cache (written, read back, attended to) and of
latent decode over a prefix that sequences share.

Each case is one call of an operator on work of a real size: ``listed()`` names
the fixed ones, ``draw()`` gives more of the same ranges, ``prepare()`` makes the
inputs a serving program has in hand, ``run()`` makes one call (the library's
with ``own`` set, otherwise the operator's formula in elementary torch
operations in fp32), ``work()`` says what the call cannot do without and
``exact()`` evaluates the definition in fp64.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16
F8 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # the new tokens of a decode step
        dict(name="write_step", op="write", t=64, l=512, r=64, page=64, pool=40000, bad=0.0, wide=False),
        # the tokens of a large prefill batch, some of them padding (slot -1)
        dict(name="write_prompts", op="write", t=98304, l=512, r=64, page=64, pool=140000, bad=0.03, wide=False),
        # one cached prefix, expanded for the prefill that continues it
        dict(name="read_prefix", op="read", t=1500, l=512, r=64, page=64, pool=40000, bad=0.0),
        # the prefixes of a whole batch
        dict(name="read_prefixes", op="read", t=120000, l=512, r=64, page=64, pool=140000, bad=0.01),
        # one sequence, one new token: the latency of a decode step
        dict(name="fp8_one", op="fp8", n=1, q=1, h=32, l=512, r=64, page=64, lo=4000, hi=4000),
        # a serving batch with the length spread of the prefill workload (64..8192), two tokens a step
        dict(name="fp8_ragged", op="fp8", n=200, q=2, h=32, l=512, r=64, page=64, lo=64, hi=8192),
        # many heads over long contexts
        dict(name="fp8_long", op="fp8", n=64, q=1, h=128, l=512, r=64, page=64, lo=12000, hi=20000),
        # a few samples of one short prompt
        dict(name="shared_few", op="shared", cache="bf16", n=4, g=1, q=1, h=16, l=512, r=64, page=64, pre=2048, lo=1,
             hi=128),
        # a batch behind one long system prompt
        dict(name="shared_one", op="shared", cache="bf16", n=64, g=1, q=1, h=16, l=512, r=64, page=64, pre=32768, lo=64,
             hi=2048),
        # eight documents with several questions each
        dict(name="shared_groups", op="shared", cache="fp8", n=96, g=8, q=1, h=32, l=512, r=64, page=64, pre=8192, lo=16,
             hi=1024),
        # many heads, a drafted token checked with the new one
        dict(name="shared_heads", op="shared", cache="fp8", n=40, g=1, q=2, h=128, l=512, r=64, page=64, pre=16384, lo=64,
             hi=1024),
        # the same in the 16-bit cache
        dict(name="shared_heads16", op="shared", cache="bf16", n=40, g=1, q=2, h=128, l=512, r=64, page=64, pre=16384,
             lo=64, hi=1024),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "fp8", "fp8", "shared", "shared", "shared"])
    l, r = rng.choice([(512, 64), (512, 64), (512, 64), (256, 32), (128, 64), (384, 0)])
    page = rng.choice([1, 16, 16, 48, 64, 64, 128])
    if op in ("write", "read"):
        t = _log(rng, 1, 98304)
        c = dict(op=op, t=t, l=l, r=r, page=page, pool=int(t * rng.uniform(1.05, 1.5)) + 200,
                 bad=rng.choice([0.0, 0.0, 0.02, 0.1]))
        if op == "write":
            c.update(wide=rng.random() < 0.25)
        return c
    h, q = rng.choice([8, 16, 20, 32, 32, 48, 64, 128]), rng.choice([1, 1, 2, 3])
    if op == "fp8":
        n = _log(rng, 1, 160)
        hi = _log(rng, 20, max(40, min(20000, 1000000 // n, 64 * 16000 * 128 // (n * q * h))))
        return dict(op=op, n=n, q=q, h=h, l=l, r=r, page=page, lo=max(1, int(hi * rng.uniform(0.01, 1))), hi=hi)
    n = _log(rng, 2, 128)
    g = min(n, rng.choice([1, 1, 2, 3, 8]))
    hi = _log(rng, 8, max(16, min(2048, 120000 // n, 40 * 1024 * 256 // (n * q * h))))
    pre = _log(rng, 128, max(256, min(32768, 140000 // g, 40 * 14336 * 256 // (n * q * h))))
    return dict(op=op, cache=rng.choice(["bf16", "fp8"]), n=n, g=g, q=q, h=h, l=l, r=r, page=page, pre=pre,
                lo=max(1, int(hi * rng.uniform(0.02, 1))), hi=hi)


# ---------------------------------------------------------------------------------------------------------------
# inputs

def _normal(gen, shape, dtype=BF16):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _rows(gen, n, l):
    """n latent vectors: normalised ones of somewhat different sizes, a few components larger than the others."""
    x = torch.randn((n, l), generator=gen, device=DEV)
    x *= torch.exp2(0.5 * torch.randn((n, 1), generator=gen, device=DEV))
    return x * torch.exp2(torch.randn((1, l), generator=gen, device=DEV))


def _lengths(rs, n, lo, hi):
    """n lengths, log-uniform in [lo, hi]."""
    if lo == hi:
        return np.full(n, lo, np.int64)
    return np.clip(np.round(np.exp(rs.uniform(np.log(lo), np.log(hi), n))), lo, hi).astype(np.int64)


def _int(x, dtype=np.int32):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=dtype)).to(DEV)


def _power(e):
    """2^e of whole e in [-126, 127], exactly"""
    return ((e + 127) << 23).view(torch.float32)


def _quantize(x):
    """Rows in 8 bits: the scale is the smallest power of two, 2^-126 at least, under which the largest component is at
    most 448; a row that is not finite has the scale NaN and the codes 0."""
    top = x.abs().amax(-1)
    m, e = torch.frexp(top)                                                   # top = m 2^e, 0.5 <= m < 1
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-126)                 # 448 = 0.875 2^9
    fine = torch.isfinite(top)
    e = torch.where(fine, e, 0).int()
    codes = torch.where(fine[:, None], x * _power(-e)[:, None], 0.0).to(F8)
    return codes, torch.where(fine, _power(e), math.nan)


def _store(c, gen, rows):
    """An 8-bit cache of ``rows`` tokens whose rows hold values."""
    page, l, r = c["page"], c["l"], c["r"]
    codes, scales = torch.empty((rows, l), dtype=F8, device=DEV), torch.empty(rows, device=DEV)
    for a in range(0, rows, 1 << 18):
        b = min(rows, a + (1 << 18))
        codes[a:b], scales[a:b] = _quantize(_rows(gen, b - a, l).to(BF16).float())
    return dict(codes=codes.view(-1, page, l), scales=scales.view(-1, page),
                rope=_normal(gen, (rows // page, page, r)) if r else None)


def _slots(c, rs):
    """Token rows of a pool: consecutive ones inside a page, pages anywhere; some are no row."""
    page, pages = c["page"], -(-c["pool"] // c["page"])
    rows = (rs.permutation(pages)[:, None] * page + np.arange(page)[None, :]).reshape(-1)[: c["t"]]
    return np.where(rs.uniform(size=c["t"]) < c["bad"], -1, rows), pages * page


def _prepare_write(c, rs, gen):
    slots, rows = _slots(c, rs)
    x = _rows(gen, c["t"], c["l"])
    kind = torch.float32 if c["wide"] else BF16
    # latent and rotary key lie side by side, as one projection gives them
    both = torch.cat([x, torch.randn((c["t"], c["r"]), generator=gen, device=DEV)], 1).to(kind)
    return dict(_store(c, gen, rows), slots=_int(slots, np.int64), c=both[:, : c["l"]],
                k_rope=both[:, c["l"]:] if c["r"] else None)


def _prepare_read(c, rs, gen):
    slots, rows = _slots(c, rs)
    return dict(_store(c, gen, rows), slots=_int(slots, np.int64))


def _queries(c, gen):
    n, q, h = c["n"], c["q"], c["h"]
    # as large as scores of a few units need them to be beside the rows' values
    return dict(q=(0.4 * torch.randn((n, q, h, c["l"]), generator=gen, device=DEV)).to(BF16),
                q_rope=_normal(gen, (n, q, h, c["r"])) if c["r"] else None, scale=192.0 ** -0.5)


def _cache(c, gen, pages):
    if c.get("cache") == "bf16":
        rows = pages * c["page"]
        x = torch.cat([_rows(gen, rows, c["l"]), torch.randn((rows, c["r"]), generator=gen, device=DEV)], 1)
        return dict(cache=x.to(BF16).view(pages, c["page"], -1))
    return _store(c, gen, pages * c["page"])


def _prepare_fp8(c, rs, gen):
    n, page = c["n"], c["page"]
    lens = np.maximum(_lengths(rs, n, c["lo"], c["hi"]), 1)
    used = -(-lens // page)
    pages = int(used.sum()) + 7
    table = np.full((n, int(used.max()) + 1), -1, np.int32)
    table[np.arange(table.shape[1])[None, :] < used[:, None]] = rs.permutation(pages)[: int(used.sum())]
    return dict(_cache(c, gen, pages), **_queries(c, gen), table=_int(table), lens=_int(lens), longest=int(lens.max()))


def _prepare_shared(c, rs, gen):
    """Groups of sequences as a fork leaves them: whole pages of the prefix are one and the same, the rest is their own."""
    n, g, page = c["n"], c["g"], c["page"]
    cuts = np.sort(rs.permutation(np.arange(1, n))[: g - 1]) if g > 1 else np.zeros(0, np.int64)
    cu = np.concatenate([[0], cuts, [n]])
    group = np.repeat(np.arange(g), np.diff(cu))
    pre = np.round(c["pre"] * rs.uniform(0.7, 1, g)).astype(np.int64) if g > 1 else np.full(1, c["pre"])
    full = pre // page
    rest = np.maximum(_lengths(rs, n, c["lo"], c["hi"]), 1)
    lens = full[group] * page + rest
    used, pages = -(-rest // page), int(full.sum() + (-(-rest // page)).sum()) + 7
    perm = rs.permutation(pages)
    first = np.concatenate([[0], np.cumsum(full)])
    begin = int(full.sum()) + np.concatenate([[0], np.cumsum(used)])
    table = np.full((n, int((full[group] + used).max()) + 1), -1, np.int32)
    for a in range(n):
        f = int(full[group[a]])
        table[a, :f] = perm[first[group[a]]: first[group[a]] + f]
        table[a, f: f + used[a]] = perm[begin[a]: begin[a] + used[a]]
    return dict(_cache(c, gen, pages), **_queries(c, gen), table=_int(table), lens=_int(lens), cu=_int(cu),
                shared=_int(full * page), group=_int(group, np.int64), longest=int(rest.max()),
                longest_pre=int(full.max()) * page, most=int(np.diff(cu).max()))


def prepare(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    make = {"write": _prepare_write, "read": _prepare_read, "fp8": _prepare_fp8, "shared": _prepare_shared}
    return dict(make[case["op"]](case, rs, gen), op=case["op"])


# ---------------------------------------------------------------------------------------------------------------
# the formulas in elementary operations

def _plain_write(st):
    codes, scales, rope, slots = st["codes"], st["scales"], st["rope"], st["slots"]
    l, rows = codes.shape[-1], scales.numel()
    fine = (slots >= 0) & (slots < rows)
    at = slots[fine]
    new, scale = _quantize(st["c"].float())
    codes.view(torch.uint8).view(rows, l)[at] = new.view(torch.uint8)[fine]
    scales.view(rows)[at] = scale[fine]
    if rope is not None:
        rope.view(rows, -1)[at] = st["k_rope"].to(BF16)[fine]
    return dict(codes=codes, scales=scales, rope=rope)


def _values(st, at):
    """rows ``at`` of the cache in fp32"""
    if "cache" in st:
        return st["cache"].view(-1, st["cache"].shape[-1])[at].float()
    l = st["codes"].shape[-1]
    x = st["codes"].view(torch.uint8).view(-1, l)[at].view(F8).float() * st["scales"].view(-1)[at][..., None]
    return x if st["rope"] is None else torch.cat([x, st["rope"].view(-1, st["rope"].shape[-1])[at].float()], -1)


def _plain_read(st):
    slots = st["slots"]
    fine = (slots >= 0) & (slots < st["scales"].numel())
    return torch.where(fine[:, None], _values(st, torch.where(fine, slots, 0)), 0.0).to(BF16)


def _place(st, table, j):
    """rows of tokens j of the table's sequences"""
    page = (st["cache"] if "cache" in st else st["codes"]).shape[1]
    col = (j // page).clamp(max=table.shape[1] - 1)
    return (table.long()[:, col] * page + j % page).clamp(min=0)


def _part(q, kv, l, scale, seen):
    """Of queries [B, M, D] over rows [B, J, D]: outputs, maxima and sums before the division."""
    s = torch.matmul(q, kv.transpose(1, 2)).mul_(scale).masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(top.clamp(min=-3e38)).exp_()
    return torch.matmul(p, kv[..., :l]), top, p.sum(-1, keepdim=True)


def _full(st):
    q = st["q"].float()
    return q if st["q_rope"] is None else torch.cat([q, st["q_rope"].float()], -1)


def _plain_fp8(st):
    n, nq, h, l = st["q"].shape
    j = torch.arange(st["longest"], device=DEV)
    kv = _values(st, _place(st, st["table"], j))                              # [N, J, L+R]
    sees = st["lens"][:, None] - (nq - 1 - torch.arange(nq, device=DEV))      # [N, Q]
    seen = (j < sees[..., None])[:, :, None, :].expand(-1, -1, h, -1).reshape(n, nq * h, -1)
    out, top, total = _part(_full(st).view(n, nq * h, -1), kv, l, st["scale"], seen)
    out, lse = out / total.clamp(min=1e-38), top + total.log()
    return dict(out=out.view(n, nq, h, l).to(BF16), lse=lse.view(n, nq, h))


def _plain_shared(st):
    n, nq, h, l = st["q"].shape
    cu, shared, group, lens = st["cu"].long(), st["shared"].long(), st["group"], st["lens"].long()
    q, m = _full(st).view(n, nq * h, -1), st["most"]
    less = (nq - 1 - torch.arange(nq, device=DEV)).repeat_interleave(h)       # [Q H]
    # the prefixes: all queries of a group at once, groups padded to the largest
    who = (cu[:-1, None] + torch.arange(m, device=DEV)).clamp(max=n - 1)      # [G, M]
    j = torch.arange(max(1, st["longest_pre"]), device=DEV)
    kv = _values(st, _place(st, st["table"][cu[:-1]], j))                     # [G, J, L+R]
    g = cu.numel() - 1
    sees = torch.minimum((lens[:, None] - less)[who], shared[:, None, None])  # [G, M, Q H]
    seen = j < sees.view(g, m * nq * h, 1)
    pre = _part(q[who].view(g, m * nq * h, -1), kv, l, st["scale"], seen)
    a = torch.arange(n, device=DEV) - cu[group]
    o0, t0, s0 = (x.view(g, m, nq * h, -1)[group, a] for x in pre)
    # the sequences' own tokens
    j = torch.arange(st["longest"], device=DEV)
    at = shared[group][:, None] + j                                           # [N, J]
    page = (st["cache"] if "cache" in st else st["codes"]).shape[1]
    col = (at // page).clamp(max=st["table"].shape[1] - 1)
    kv = _values(st, (torch.gather(st["table"].long(), 1, col) * page + at % page).clamp(min=0))
    seen = at[:, None, :] < (lens[:, None] - less)[..., None]
    o1, t1, s1 = _part(q, kv, l, st["scale"], seen)
    top = torch.maximum(t0, t1).clamp(min=-3e38)
    f0, f1 = torch.exp(t0 - top), torch.exp(t1 - top)
    total = s0 * f0 + s1 * f1
    out, lse = (o0 * f0 + o1 * f1) / total.clamp(min=1e-38), top + total.log()
    return dict(out=out.view(n, nq, h, l).to(BF16), lse=lse.view(n, nq, h))


# ---------------------------------------------------------------------------------------------------------------
# the library's calls

def _own(st):
    import kda_recurrent_state_amd as kda
    op = st["op"]
    if op == "write":
        kda.kda_latent_quantize_scatter(st["c"], st["k_rope"], st["slots"], st["codes"], st["scales"], st["rope"])
        return dict(codes=st["codes"], scales=st["scales"], rope=st["rope"])
    if op == "read":
        return kda.kda_latent_dequantize_gather(st["codes"], st["scales"], st["rope"], st["slots"])
    if op == "fp8":
        out, lse = kda.kda_latent_decode_fp8(st["codes"], st["scales"], st["rope"], st["table"], st["lens"], st["q"],
                                             st["q_rope"], scale=st["scale"], with_lse=True)
        return dict(out=out, lse=lse)
    cache = st["cache"] if "cache" in st else (st["codes"], st["scales"], st["rope"])
    out, lse = kda.kda_latent_decode_shared(cache, st["table"], st["lens"], st["cu"], st["shared"], st["q"],
                                            st["q_rope"], scale=st["scale"], with_lse=True)
    return dict(out=out, lse=lse)


def run(state):
    if own:
        return _own(state)
    plain = {"write": _plain_write, "read": _plain_read, "fp8": _plain_fp8, "shared": _plain_shared}
    return plain[state["op"]](state)


# ---------------------------------------------------------------------------------------------------------------
# what a call cannot do without

def _mean_length(lo, hi):
    return lo if lo == hi else (hi - lo) / math.log(hi / lo)


def work(case):
    c, op = case, case["op"]
    l, r = c["l"], c["r"]
    if op in ("write", "read"):
        good = c["t"] * (1 - c["bad"])
        wide = (l + r) * (4 if c.get("wide") else 2)
        return dict(bytes=good * (wide + l + 2 * r + 4) + 8 * c["t"] + (c["t"] * c["bad"] * wide if op == "read" else 0),
                    flops=0)
    row = (l + r) * 2 if c.get("cache") == "bf16" else l + 2 * r + 4
    own_rows, queries = c["n"] * _mean_length(c["lo"], c["hi"]), c["n"] * c["q"] * c["h"]
    rows, pairs = own_rows, own_rows * c["q"] * c["h"]
    if op == "shared":
        pre = c["pre"] // c["page"] * c["page"] * (0.85 if c["g"] > 1 else 1)
        rows, pairs = rows + c["g"] * pre, pairs + queries * pre
    return dict(bytes=rows * row + queries * (2 * l + r) * 2 + queries * 4 + 4 * rows / c["page"],
                flops=2 * pairs * (2 * l + r))


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits

def _exact_codes(x):
    """(codes, scale) of a finite row's components: multiples of 2^(floor(log2) - 3), of 2^-9 at the least, ties to even"""
    top = x.abs().amax(-1, keepdim=True).clamp(min=2.0 ** -130)
    e = torch.floor(torch.log2(top)) - 8
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e).clamp(min=-126)
    y = x / torch.exp2(e)
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step, torch.exp2(e)


def _exact_rows(st, pages, begin, end):
    page = (st["cache"] if "cache" in st else st["codes"]).shape[1]
    ids = torch.tensor(pages[begin // page: -(-end // page)], device=DEV, dtype=torch.long)
    a, b = begin % page, begin % page + end - begin
    if "cache" in st:
        return st["cache"][ids].flatten(0, 1)[a:b].double()
    x = st["codes"].view(torch.uint8)[ids].view(F8).flatten(0, 1)[a:b].double()
    x = x * st["scales"][ids].flatten()[a:b, None].double()
    return x if st["rope"] is None else torch.cat([x, st["rope"][ids].flatten(0, 1)[a:b].double()], 1)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "write":
        slots = st["slots"]
        rows, l = st["scales"].numel(), case["l"]
        codes, scales = st["codes"].double().view(rows, l), st["scales"].double().view(rows)
        fine = (slots >= 0) & (slots < rows)
        new, scale = _exact_codes(st["c"].double())
        codes[slots[fine]], scales[slots[fine]] = new[fine], scale[fine, 0]
        return dict(codes=codes.view(st["codes"].shape), scales=scales.view(st["scales"].shape), rope=None)
    if case["op"] == "read":
        out = torch.zeros(case["t"], case["l"] + case["r"], dtype=torch.float64, device=DEV)
        slots = st["slots"]
        fine = (slots >= 0) & (slots < st["scales"].numel())
        at = slots[fine]
        out[fine, : case["l"]] = (st["codes"].double().view(-1, case["l"])[at] * st["scales"].double().view(-1, 1)[at])
        if case["r"]:
            out[fine, case["l"]:] = st["rope"].double().view(-1, case["r"])[at]
        return out
    n, nq, h, l = st["q"].shape
    out = torch.zeros(n, nq, h, l, dtype=torch.float64, device=DEV)
    lse = torch.full((n, nq, h), -math.inf, dtype=torch.float64, device=DEV)
    for a, (length, pages) in enumerate(zip(st["lens"].tolist(), st["table"].tolist())):
        rows = _exact_rows(st, pages, 0, length)
        for b in range(nq):
            sees = length - (nq - 1 - b)
            if sees > 0:
                s = st["q"][a, b].double() @ rows[:sees, :l].T
                if st["q_rope"] is not None:
                    s = s + st["q_rope"][a, b].double() @ rows[:sees, l:].T
                lse[a, b] = torch.logsumexp(s * st["scale"], -1)
                out[a, b] = torch.exp(s * st["scale"] - lse[a, b][:, None]) @ rows[:sees, :l]
    return dict(out=out, lse=lse)
