"""Timed cases of the latent-attention and cache-page operators.

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


# ---------------------------------------------------------------------------------------------------------------
# cases

def listed():
    return [
        # one sequence, one new token: the latency of a decode step
        dict(name="decode_one", op="decode", n=1, q=1, h=32, l=512, r=64, page=64, lo=4000, hi=4000),
        # a serving batch with the length spread of the prefill workload (64..8192), two tokens a step (a drafted
        # one is checked)
        dict(name="decode_ragged", op="decode", n=200, q=2, h=32, l=512, r=64, page=64, lo=64, hi=8192),
        # many heads over long contexts: the latent row is shared by 128 heads
        dict(name="decode_long", op="decode", n=64, q=1, h=128, l=512, r=64, page=64, lo=12000, hi=20000),
        # a handful of short prompts
        dict(name="prefill_short", op="prefill", n=4, h=32, d=128, r=64, e=128, lo=1, hi=100, past=0, causal=True),
        # prompts continued over cached prefixes: more keys than queries
        dict(name="prefill_prefix", op="prefill", n=12, h=32, d=128, r=64, e=128, lo=1, hi=1024, past=1500, causal=True),
        # one long prompt
        dict(name="prefill_long", op="prefill", n=1, h=16, d=128, r=64, e=128, lo=16384, hi=16384, past=0, causal=True),
        # beams: children share the parent's full pages, the last page is copied
        dict(name="fork_beams", op="fork", cache="latent", seqs=256, live=96, per=128, pages=8192, page=64, d=576,
             forks=96, share=True, lo=64, hi=8000),
        # recurrent-state rows (fp32, H=32, K=V=128, with a page gap) change in place: a fork copies them
        dict(name="fork_states", op="fork", cache="state", seqs=1024, live=512, per=1, pages=1024, page=1, d=524288,
             forks=256, share=False, lo=1, hi=1),
        # a latent cache after many sequences have ended
        dict(name="compact_pages", op="compact", cache="latent", seqs=256, live=100, per=128, pages=8192, page=64, d=576,
             lo=64, hi=8000),
        # state rows after half of the sequences have ended
        dict(name="compact_states", op="compact", cache="state", seqs=1024, live=512, per=1, pages=1024, page=1,
             d=524288, lo=1, hi=1),
        # a few sequences of a batch end
        dict(name="free_few", op="free", seqs=256, live=200, per=128, pages=16384, page=64, ended=24, lo=64, hi=8000),
        # a large pool is drained
        dict(name="free_many", op="free", seqs=4096, live=4096, per=512, pages=600000, page=16, ended=3000, lo=16,
             hi=8192),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["decode", "decode", "prefill", "prefill", "fork", "compact", "free"])
    if op == "decode":
        l, r = rng.choice([(512, 64), (512, 64), (512, 64), (256, 32), (128, 64), (384, 0)])
        n, q = _log(rng, 1, 160), rng.choice([1, 1, 2, 3])
        h = rng.choice([8, 16, 20, 32, 32, 48, 64, 128])
        hi = _log(rng, 20, max(40, min(20000, 1000000 // n, 64 * 16000 * 128 // (n * q * h))))
        return dict(op=op, n=n, q=q, h=h, l=l, r=r, page=rng.choice([1, 16, 16, 48, 64, 64, 128]),
                    lo=max(1, int(hi * rng.uniform(0.01, 1))), hi=hi)
    if op == "prefill":
        d, r, e = rng.choice([(128, 64, 128), (128, 64, 128), (64, 32, 64), (128, 0, 128), (96, 32, 80)])
        n, h = _log(rng, 1, 16), rng.choice([4, 8, 16, 21, 32])
        hi = _log(rng, 16, max(32, min(16384, int(16384 * math.sqrt(5 / (n * h))))))
        return dict(op=op, n=n, h=h, d=d, r=r, e=e, lo=max(1, int(hi * rng.uniform(0.02, 1))), hi=hi,
                    past=rng.choice([0, 0, hi // 3, hi // 2]), causal=rng.random() < 0.8)
    if op == "free":
        seqs, per, page = _log(rng, 16, 4096), _log(rng, 8, 512), rng.choice([16, 32, 64])
        live = max(1, int(seqs * rng.uniform(0.3, 1)))
        return dict(op=op, seqs=seqs, live=live, per=per, pages=int(1.1 * live * per) + 64, page=page,
                    ended=max(1, int(live * rng.uniform(0.05, 1))), lo=1, hi=per * page)
    kind = rng.choice(["latent", "latent", "state"])
    if kind == "state":
        seqs = _log(rng, 16, 1000)
        live = max(1, int(seqs * rng.uniform(0.2, 0.6)))
        c = dict(op=op, cache=kind, seqs=seqs, live=live, per=1, pages=seqs, page=1,
                 d=rng.choice([524288, 262144, 131072]), lo=1, hi=1)
        forks, share = max(1, int((seqs - live) * rng.uniform(0.1, 0.6))), False
    else:
        seqs, per, page = _log(rng, 8, 256), _log(rng, 4, 120), rng.choice([16, 32, 64])
        live = max(1, int(seqs * rng.uniform(0.2, 0.5)))
        c = dict(op=op, cache=kind, seqs=seqs, live=live, per=per, pages=live * per * 2 + 64, page=page,
                 d=rng.choice([576, 576, 288, 264]), lo=1, hi=per * page)
        share = rng.random() < 0.7
        forks = max(1, int((seqs - live) * rng.uniform(0.1, 1 if share else 0.4)))
    if op == "fork":
        c.update(forks=forks, share=share)
    return c


# ---------------------------------------------------------------------------------------------------------------
# inputs

def _normal(gen, shape, dtype=BF16):
    return torch.randn(shape, generator=gen, device=DEV, dtype=torch.float32).to(dtype)


def _lengths(rs, n, lo, hi):
    """n lengths, log-uniform in [lo, hi]."""
    if lo == hi:
        return np.full(n, lo, np.int64)
    return np.clip(np.round(np.exp(rs.uniform(np.log(lo), np.log(hi), n))), lo, hi).astype(np.int64)


def _i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)


def _prepare_decode(c, rs, gen):
    n, q, h, l, r, page = c["n"], c["q"], c["h"], c["l"], c["r"], c["page"]
    lens = np.maximum(_lengths(rs, n, c["lo"], c["hi"]), 1)
    used = -(-lens // page)
    pages = int(used.sum()) + 7
    width = int(used.max()) + 1
    perm = rs.permutation(pages)
    table = np.full((n, width), -1, np.int32)
    mask = np.arange(width)[None, :] < used[:, None]
    table[mask] = perm[: int(used.sum())]
    return dict(cache=_normal(gen, (pages, page, l + r)), table=_i32(table), lens=_i32(lens),
                q=_normal(gen, (n, q, h, l)), q_rope=_normal(gen, (n, q, h, r)) if r else None,
                scale=192.0 ** -0.5, longest=int(lens.max()))


def _prepare_prefill(c, rs, gen):
    n, h, d, r, e = c["n"], c["h"], c["d"], c["r"], c["e"]
    # log-spaced over the range, in an order of the seed: the number of tokens is the case's own
    lq = rs.permutation(np.round(np.geomspace(c["lo"], c["hi"], n)).astype(np.int64))
    lk = lq + (rs.randint(0, c["past"] + 1, n) if c["past"] else 0)
    cu_q, cu_k = np.concatenate([[0], np.cumsum(lq)]), np.concatenate([[0], np.cumsum(lk)])
    t, s = int(cu_q[-1]), int(cu_k[-1])
    # keys and values come out of one up-projection: views of a [S, H, D + E] tensor; the rotary key is the end of
    # the latent rows
    kv = _normal(gen, (s, h, d + e))
    rows = _normal(gen, (s, 512 + r)) if r else None
    return dict(q=_normal(gen, (t, h, d + r)), k=kv[..., :d], v=kv[..., d:], k_rope=rows[:, 512:] if r else None,
                cu_q=_i32(cu_q), cu_k=_i32(cu_k), scale=(d + r) ** -0.5, max_q=int(lq.max()), max_k=int(lk.max()),
                causal=bool(c["causal"]))


def _prepare_pool(c, rs, gen):
    """A pool in use: ``live`` of ``seqs`` slots hold sequences, neighbours share prefixes, pages lie anywhere."""
    seqs, per, pages, page = c["seqs"], c["per"], c["pages"], c["page"]
    lens = np.zeros(seqs, np.int64)
    slots = np.sort(rs.permutation(seqs)[: c["live"]])
    lens[slots] = np.minimum(np.maximum(_lengths(rs, c["live"], c["lo"], min(c["hi"], per * page)), 1), per * page)
    used = -(-lens // page)
    shared = np.zeros(seqs, np.int64)
    if per > 1:  # every third sequence shares half of its predecessor's full pages
        full = lens // page
        a, b = slots[1::3], slots[0::3][: len(slots[1::3])]
        shared[a] = np.minimum(full[a], full[b]) // 2
    fresh = np.concatenate([[0], np.cumsum(used - shared)])
    fresh, room = fresh[:-1], int(fresh[-1])
    if room > pages:
        raise ValueError("the pool has too few pages for its sequences")
    perm = rs.permutation(pages)
    table = np.full((seqs, per), -1, np.int32)
    col = np.arange(per)[None, :]
    own_part = (col >= shared[:, None]) & (col < used[:, None])
    table[own_part] = perm[(fresh[:, None] + col - shared[:, None])[own_part]]
    if per > 1:
        a, b = slots[1::3], slots[0::3][: len(slots[1::3])]
        part = col < shared[a][:, None]
        rows = table[a]
        rows[part] = table[b][part]
        table[a] = rows
    refs = np.bincount(table[table >= 0], minlength=pages)
    # one buffer, put back before every pass: table, lengths, reference counts
    first = _i32(np.concatenate([table.reshape(-1), lens, refs]))
    now = torch.empty_like(first)
    a, b = seqs * per, seqs * per + seqs
    st = dict(first=first, now=now, table=now[:a].view(seqs, per), lens=now[a:b], refs=now[b:], page=page)
    if c["op"] == "fork":
        empty = np.setdiff1d(np.arange(seqs), slots)
        st["src"] = _i32(rs.choice(slots, c["forks"]))
        st["dst"] = _i32(rs.permutation(empty)[: c["forks"]])
        st["share"] = bool(c["share"])
    if c["op"] == "free":
        gone = np.zeros(seqs, bool)
        gone[rs.permutation(slots)[: c["ended"]]] = True
        st["release"] = torch.from_numpy(gone).to(DEV)
    if c["op"] != "free":
        if c["cache"] == "state":  # [rows, H, 128, 128] fp32 with 4096 elements between the rows
            heads, stride = c["d"] // 16384, c["d"] + 4096
            flat = torch.randn(pages * stride, generator=gen, device=DEV)
            st["cache"] = torch.as_strided(flat, (pages, heads, 128, 128), (stride, 16384, 128, 1))
            st["bits"] = flat.view(torch.int32)
        else:
            st["cache"] = _normal(gen, (pages, page, c["d"]))
            st["bits"] = st["cache"].view(torch.int16)
    return st


def prepare(case, seed):
    rs = np.random.RandomState(seed % (1 << 31))
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    make = {"decode": _prepare_decode, "prefill": _prepare_prefill}.get(case["op"], _prepare_pool)
    return dict(make(case, rs, gen), op=case["op"])


# ---------------------------------------------------------------------------------------------------------------
# the formulas in elementary operations

def _softmax_products(s, seen, values):
    """softmax over the seen scores, times values, and the log of the softmax's sum; no seen score: 0 and -inf."""
    s.masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(top.clamp(min=-3e38)).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, values) / total.clamp(min=1e-38)
    return out, (top + total.log()).squeeze(-1)


def _plain_decode(st):
    cache, table, lens, q = st["cache"], st["table"], st["lens"], st["q"]
    pages, page, d = cache.shape
    n, nq, h, l = q.shape
    at = torch.arange(st["longest"], device=DEV)
    rows = (table.long()[:, at // page] * page + at % page).clamp(min=0)
    kv = cache.view(pages * page, d)[rows].float()                            # [N, J, L+R]
    full = q.float() if st["q_rope"] is None else torch.cat([q.float(), st["q_rope"].float()], -1)
    s = torch.matmul(full.view(n, nq * h, d), kv.transpose(1, 2)).mul_(st["scale"]).view(n, nq, h, -1)
    sees = lens[:, None] - (nq - 1 - torch.arange(nq, device=DEV))            # [N, Q]
    seen = (at < sees[..., None])[:, :, None, :]
    out, lse = _softmax_products(s, seen, kv[:, None, :, :l])
    return dict(out=out.to(q.dtype), lse=lse)


def _plain_prefill(st):
    q, k, v, cu_q, cu_k = st["q"], st["k"], st["v"], st["cu_q"].long(), st["cu_k"].long()
    i, j = torch.arange(st["max_q"], device=DEV), torch.arange(st["max_k"], device=DEV)
    keys = k.float()
    if st["k_rope"] is not None:
        keys = torch.cat([keys, st["k_rope"].float()[:, None, :].expand(-1, k.shape[1], -1)], -1)
    qi = (cu_q[:-1, None] + i).clamp(max=q.shape[0] - 1)
    kj = (cu_k[:-1, None] + j).clamp(max=k.shape[0] - 1)
    qs, ks, vs = (x.transpose(1, 2).contiguous() for x in (q.float()[qi], keys[kj], v.float()[kj]))   # [N, H, *, D]
    lq, lk = cu_q.diff()[:, None, None], cu_k.diff()[:, None, None]
    seen = (j < lk) & (i[:, None] < lq)
    if st["causal"]:
        seen = seen & (j < lk - (lq - 1 - i[:, None]))
    out, lse = _softmax_products(torch.matmul(qs, ks.transpose(2, 3)).mul_(st["scale"]), seen[:, None], vs)
    t = torch.arange(q.shape[0], device=DEV)
    seq = torch.searchsorted(cu_q[1:], t, right=True)
    return dict(out=out[seq, :, t - cu_q[seq]].to(q.dtype), lse=lse[seq, :, t - cu_q[seq]])


def _plain_fork(st):
    table, lens, refs, page = st["table"], st["lens"], st["refs"], st["page"]
    src, dst = st["src"].long(), st["dst"].long()
    seqs, per = table.shape
    ok = (src >= 0) & (src < seqs) & (dst >= 0) & (dst < seqs) & (src != dst)
    earlier = (dst[:, None] == dst[None, :]).tril(-1).any(1)
    s, d = src.clamp(0, seqs - 1), dst.clamp(0, seqs - 1)
    n, rows, col = lens[s].long(), table[s].long(), torch.arange(per, device=DEV)
    used = (n + page - 1) // page
    inside = col < used[:, None]
    sound = (rows >= 0) & (rows < refs.numel()) & (refs[rows.clamp(0, refs.numel() - 1)] > 0)
    ok = ok & ~earlier & (lens[d] == 0) & (n >= 0) & (used <= per) & (sound | ~inside).all(1)
    need = (n % page != 0).long() if st["share"] else used
    upto = torch.where(ok, need, 0).cumsum(0)
    taken = refs > 0
    served = ok & (upto <= (~taken).sum())
    free = torch.sort(taken.to(torch.int8), stable=True).indices            # the free pages first, in order
    fresh = inside & (col >= (used - need)[:, None]) & served[:, None]
    new = free[(upto[:, None] - need[:, None] + col - (used - need)[:, None]).clamp(0, free.numel() - 1)]
    child = torch.where(fresh, new, torch.where(inside, rows, -1)).int()
    kept = inside & ~fresh & served[:, None]
    st["cache"][new[fresh]] = st["cache"][rows[fresh]]
    refs.scatter_add_(0, torch.where(kept, rows, 0).view(-1), kept.int().view(-1))
    refs[new[fresh]] = 1
    table[d[served]] = child[served]
    lens[d[served]] = n[served].int()
    status = torch.where(served, 0, torch.where(ok, 1, 2)).int()
    return dict(table=table, lens=lens, refs=refs, status=status, cache=st["bits"])


def _plain_compact(st):
    table, lens, refs, page = st["table"], st["lens"], st["refs"], st["page"]
    taken, at = refs > 0, torch.arange(refs.numel(), device=DEV)
    live = taken.sum()
    src, dst = (taken & (at >= live)).nonzero().view(-1), (~taken & (at < live)).nonzero().view(-1)
    st["cache"][dst] = st["cache"][src]
    to = at.int()
    to[src] = dst.int()
    refs[dst] = refs[src]
    refs[src] = 0
    inside = torch.arange(table.shape[1], device=DEV) < ((lens + page - 1) // page)[:, None]
    sound = inside & (table >= 0) & (table < refs.numel())
    table.copy_(torch.where(sound, to[table.long().clamp(0, refs.numel() - 1)], table))
    return dict(table=table, lens=lens, refs=refs, live=live.int().view(1), cache=st["bits"])


def _plain_free(st):
    table, lens, refs, page = st["table"], st["lens"], st["refs"], st["page"]
    gone = st["release"][:, None] & (torch.arange(table.shape[1], device=DEV) < ((lens + page - 1) // page)[:, None])
    sound = gone & (table >= 0) & (table < refs.numel())
    refs.scatter_add_(0, torch.where(sound, table, 0).long().view(-1), -sound.int().view(-1))
    table.masked_fill_(gone, -1)
    lens.masked_fill_(st["release"], 0)
    return dict(table=table, lens=lens, refs=refs)


# ---------------------------------------------------------------------------------------------------------------
# the library's calls

def _own(st):
    import kda_recurrent_state_amd as kda
    op = st["op"]
    if op == "decode":
        out, lse = kda.kda_latent_decode(st["cache"], st["table"], st["lens"], st["q"], st["q_rope"],
                                         scale=st["scale"], with_lse=True)
        return dict(out=out, lse=lse)
    if op == "prefill":
        out, lse = kda.kda_latent_prefill(st["q"], st["k"], st["v"], st["cu_q"], k_rope=st["k_rope"],
                                          cu_seqlens_k=st["cu_k"], scale=st["scale"], causal=st["causal"],
                                          with_lse=True)
        return dict(out=out, lse=lse)
    table, lens, refs, page = st["table"], st["lens"], st["refs"], st["page"]
    if op == "fork":
        status = kda.kda_page_fork(table, lens, refs, st["src"], st["dst"], page, caches=[st["cache"]],
                                   share=st["share"])
        return dict(table=table, lens=lens, refs=refs, status=status, cache=st["bits"])
    if op == "compact":
        live = kda.kda_page_compact(table, lens, refs, page, caches=[st["cache"]])
        return dict(table=table, lens=lens, refs=refs, live=live, cache=st["bits"])
    kda.kda_page_free(table, lens, refs, st["release"], page)
    return dict(table=table, lens=lens, refs=refs)


def run(state):
    if "first" in state:
        state["now"].copy_(state["first"])  # the pool as it was: the page operators change it
    if own:
        return _own(state)
    plain = {"decode": _plain_decode, "prefill": _plain_prefill, "fork": _plain_fork, "compact": _plain_compact,
             "free": _plain_free}
    return plain[state["op"]](state)


# ---------------------------------------------------------------------------------------------------------------
# what a call cannot do without

def _mean_length(lo, hi):
    return lo if lo == hi else (hi - lo) / math.log(hi / lo)


def work(case):
    c, op = case, case["op"]
    if op == "decode":
        m = _mean_length(c["lo"], c["hi"])
        rows, nq = c["n"] * m, c["n"] * c["q"] * c["h"]
        return dict(bytes=rows * (c["l"] + c["r"]) * 2 + nq * (2 * c["l"] + c["r"]) * 2 + nq * 4 + 4 * rows / c["page"],
                    flops=2 * rows * c["q"] * c["h"] * (2 * c["l"] + c["r"]))
    if op == "prefill":
        m, past = _mean_length(c["lo"], c["hi"]), c["past"] / 2
        if c["lo"] == c["hi"]:
            square = m * m
        else:
            square = (c["hi"] ** 2 - c["lo"] ** 2) / (2 * math.log(c["hi"] / c["lo"]))
        pairs = c["n"] * ((square + m) / 2 + m * past if c["causal"] else square + m * past)
        t, s = c["n"] * m, c["n"] * (m + past)
        return dict(bytes=2 * (t * c["h"] * (c["d"] + c["r"] + c["e"]) + s * (c["h"] * (c["d"] + c["e"]) + c["r"]))
                    + 4 * t * c["h"], flops=2 * pairs * c["h"] * (c["d"] + c["r"] + c["e"]))
    per_seq = min(c["per"], _mean_length(c["lo"], c["hi"]) / c["page"] + 0.5) if c["page"] > 1 else 1
    if op == "free":
        return dict(bytes=c["ended"] * per_seq * (4 + 4 + 8) + c["seqs"] * 5, flops=0)
    payload = c["d"] * 4 if c["cache"] == "state" else c["page"] * c["d"] * 2
    if op == "fork":
        moved = c["forks"] * (per_seq if not c["share"] else 1 - 1 / c["page"])
        return dict(bytes=2 * moved * payload + c["pages"] * 4 + c["forks"] * per_seq * 16, flops=0)
    owned = c["live"] * per_seq * (1 if c["per"] == 1 else 0.9)
    moved = owned * (1 - owned / c["pages"])
    return dict(bytes=2 * moved * payload + c["pages"] * 4 + c["live"] * per_seq * 8 + moved * 8, flops=0)


# ---------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits, one sequence (and head) at a time

def _exact_row(scores, values):
    lse = torch.logsumexp(scores, -1)
    return torch.exp(scores - lse[..., None]) @ values, lse


def exact(case, seed):
    if case["op"] == "decode":
        st = prepare(case, seed)
        n, nq, h, l = st["q"].shape
        page = case["page"]
        out = torch.zeros(n, nq, h, l, dtype=torch.float64, device=DEV)
        lse = torch.full((n, nq, h), -math.inf, dtype=torch.float64, device=DEV)
        for a, (length, pages) in enumerate(zip(st["lens"].tolist(), st["table"].tolist())):
            rows = torch.cat([st["cache"][p] for p in pages[: -(-length // page)]])[:length].double()
            for b in range(nq):
                sees = length - (nq - 1 - b)
                if sees > 0:
                    s = st["q"][a, b].double() @ rows[:sees, :l].T
                    if st["q_rope"] is not None:
                        s = s + st["q_rope"][a, b].double() @ rows[:sees, l:].T
                    out[a, b], lse[a, b] = _exact_row(s * st["scale"], rows[:sees, :l])
        return dict(out=out, lse=lse)
    if case["op"] == "prefill":
        st = prepare(case, seed)
        t, h, _ = st["q"].shape
        d, e = case["d"], case["e"]
        out = torch.zeros(t, h, e, dtype=torch.float64, device=DEV)
        lse = torch.full((t, h), -math.inf, dtype=torch.float64, device=DEV)
        cu_q, cu_k = st["cu_q"].tolist(), st["cu_k"].tolist()
        for a in range(case["n"]):
            q0, q1, k0, k1 = cu_q[a], cu_q[a + 1], cu_k[a], cu_k[a + 1]
            hidden = None
            if st["causal"]:
                hidden = torch.ones(q1 - q0, k1 - k0, dtype=torch.bool, device=DEV).triu(k1 - k0 - (q1 - q0) + 1)
            for b in range(h):
                q = st["q"][q0:q1, b].double()
                s = q[:, :d] @ st["k"][k0:k1, b].double().T
                if st["k_rope"] is not None:
                    s = s + q[:, d:] @ st["k_rope"][k0:k1].double().T
                s = s * st["scale"]
                if hidden is not None:
                    s.masked_fill_(hidden, -math.inf)
                out[q0:q1, b], lse[q0:q1, b] = _exact_row(s, st["v"][k0:k1, b].double())
        return dict(out=out, lse=lse)
    return None  # the page operators copy bits and count
