"""Plain fp64 evaluations of latent attention and of the page operators, one
sequence (slot) at a time, for the tests."""
import math

import torch


def attend(q, keys, values, sees, scale):
    """q [I, D], keys [J, D], values [J, E] in fp64, sees [I] (query i sees the
    keys j < sees[i]) or a truth table [I, J].  Returns out [I, E], lse [I] and
    the sum of p |v| [I, E]; a query that sees nothing gets 0 and -inf."""
    if sees.dim() == 1:
        sees = torch.arange(keys.shape[0])[None, :] < sees[:, None]
    s = (q @ keys.T) * scale
    s = s.masked_fill(~sees, -math.inf)
    lse = torch.logsumexp(s, -1)
    p = torch.exp(s - torch.where(torch.isinf(lse), 0.0, lse)[:, None])
    p = torch.where(sees, p, 0.0)
    v = torch.where(sees.any(0)[:, None], values, 0.0)   # unseen rows may hold anything
    return p @ v, lse, p @ v.abs()


def attend_far(q, keys, values, sees, scale):
    """As attend, for scores whose step in fp64 is above 1: lse is the maximum
    there and exp(s - lse) no weight, so the maximum is subtracted and the
    weights are divided by their sum."""
    if sees.dim() == 1:
        sees = torch.arange(keys.shape[0])[None, :] < sees[:, None]
    s = ((q @ keys.T) * scale).masked_fill(~sees, -math.inf)
    top = s.amax(-1)
    p = torch.exp(s - torch.where(torch.isinf(top), 0.0, top)[:, None])
    total = p.sum(-1)
    p = p / total.clamp(min=1e-300)[:, None]
    return p @ values, top + total.log(), p @ values.abs()


def prefill(q, k, v, k_rope, cu_q, cu_k, scale, causal, attend=attend):
    T, H, _ = q.shape
    out = torch.zeros(T, H, v.shape[2], dtype=torch.float64)
    mag = torch.zeros_like(out)
    lse = torch.full((T, H), -math.inf, dtype=torch.float64)
    q, k, v = q.cpu().double(), k.cpu().double(), v.cpu().double()
    for n in range(len(cu_q) - 1):
        a, b, c, d = cu_q[n], cu_q[n + 1], cu_k[n], cu_k[n + 1]
        lq, lk = b - a, d - c
        if lq == 0:
            continue
        sees = torch.full((lq,), lk)
        if causal:
            sees = lk - (lq - 1 - torch.arange(lq))
        for h in range(H):
            keys = k[c:d, h]
            if k_rope is not None:
                keys = torch.cat([keys, k_rope[c:d].cpu().double()], -1)
            if lk:
                out[a:b, h], lse[a:b, h], mag[a:b, h] = attend(q[a:b, h], keys, v[c:d, h], sees, scale)
    return out, lse, mag


def decode(cache, table, lengths, q, q_rope, scale, attend=attend):
    """q [N, Q, H, L]"""
    N, Q, H, L = q.shape
    pages, page, _ = cache.shape
    out = torch.zeros(N, Q, H, L, dtype=torch.float64)
    mag = torch.zeros_like(out)
    lse = torch.full((N, Q, H), -math.inf, dtype=torch.float64)
    cache, table, lengths, q = cache.cpu(), table.cpu(), lengths.tolist(), q.cpu().double()
    if q_rope is not None:
        q = torch.cat([q, q_rope.cpu().double()], -1)
    for n in range(N):
        length = max(0, min(lengths[n], table.shape[1] * page))
        if length == 0:
            continue
        j = torch.arange(length)
        pg = table[n, j // page].long()
        ok = (pg >= 0) & (pg < pages)
        rows = cache[pg.clamp(0, pages - 1), j % page].double()
        rows[~ok] = 0
        for i in range(Q):
            sees = ((j < length - (Q - 1 - i)) & ok)[None, :].expand(H, -1)
            out[n, i], lse[n, i], mag[n, i] = attend(q[n, i], rows, rows[:, :L], sees, scale)
    return out, lse, mag


def check(out, lse, want, name=""):
    """Both outputs against the fp64 ones.

    out: the result is rounded to bf16 (off by at most 2^-8 of itself), and
    each softmax weight was (2^-8 of sum p |v|); the weights' fp32 scores,
    exponentials and sums add under 2^-12 of sum p |v|.  lse: a sum of up to
    576 fp32 products of size up to about 4 after scaling, each rounding 2^-24
    of the running sum (below 64), so their root-mean-square stays under
    sqrt(576) 2^-24 64 = 1e-4."""
    ref, ref_lse, mag = want
    o = out.detach().cpu().double().reshape(ref.shape)
    assert torch.isfinite(o).all(), name
    bound = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * mag + 1e-30
    over = ((o - ref).abs() / bound).max().item()
    rel = ((o - ref).norm() / ref.norm().clamp(min=1e-30)).item()
    print("  %s out: worst %.2f of its bound, relative L2 %.2e" % (name, over, rel), flush=True)
    assert over <= 1.0, (name, over)
    if lse is not None:
        s = lse.detach().cpu().double().reshape(ref_lse.shape)
        empty = torch.isinf(ref_lse)
        assert torch.equal(torch.isinf(s) & (s < 0), empty), name
        off = (s - ref_lse)[~empty].abs().max().item() if (~empty).any() else 0.0
        assert off <= 1e-4, (name, off)


# --- pages ------------------------------------------------------------------

def fork(table, lengths, refs, src, dst, page_size, caches, share):
    """Entry after entry, on copies; returns (table, lengths, refs, caches, status)."""
    t0, l0, r0 = table.tolist(), lengths.tolist(), refs.tolist()
    t, n, r = [list(x) for x in t0], list(l0), list(r0)
    caches = [c.clone() for c in caches]
    free = [p for p in range(len(r0)) if r0[p] <= 0]
    at, asked, seen, status = 0, 0, set(), []
    for s, d in zip(src.tolist(), dst.tolist()):
        ok = 0 <= s < len(l0) and 0 <= d < len(l0) and s != d and d not in seen
        seen.add(d)
        if ok:
            used = -(-l0[s] // page_size)
            ok = l0[d] == 0 and l0[s] >= 0 and used <= len(t0[0])
            ok = ok and all(0 <= p < len(r0) and r0[p] > 0 for p in t0[s][:used])
        if not ok:
            status.append(2)
            continue
        need = (1 if l0[s] % page_size else 0) if share else used
        asked += need
        if asked > len(free):
            status.append(1)
            continue
        status.append(0)
        row = t0[s][:used - need] + free[at:at + need]
        for p in row[:used - need]:
            r[p] += 1
        for p, q in zip(t0[s][used - need:used], row[used - need:]):
            r[q] = 1
            for c, c0 in zip(caches, caches):
                c[q] = c0[p]
        at += need
        t[d] = row + [-1] * (len(t0[0]) - used)
        n[d] = l0[s]
    mk = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return mk(t), mk(n), mk(r), caches, mk(status)


def compact(table, lengths, refs, page_size, caches):
    t, n, r = [list(x) for x in table.tolist()], lengths.tolist(), refs.tolist()
    caches = [c.clone() for c in caches]
    live = sum(x > 0 for x in r)
    src = [p for p in range(live, len(r)) if r[p] > 0]
    dst = [p for p in range(live) if r[p] <= 0]
    to = dict(zip(src, dst))
    for a, b in to.items():
        r[b], r[a] = r[a], 0
        for c in caches:
            c[b] = c[a]
    for s, row in enumerate(t):
        for j in range(min(len(row), -(-max(n[s], 0) // page_size))):
            row[j] = to.get(row[j], row[j])
    return torch.tensor(t, dtype=torch.int32), torch.tensor(r, dtype=torch.int32), caches, live


def free(table, lengths, refs, release, page_size):
    t, n, r = [list(x) for x in table.tolist()], lengths.tolist(), refs.tolist()
    for s, gone in enumerate(release.tolist()):
        if gone:
            for j in range(min(len(t[s]), -(-max(n[s], 0) // page_size))):
                if 0 <= t[s][j] < len(r):
                    r[t[s][j]] -= 1
                t[s][j] = -1
            n[s] = 0
    mk = lambda x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    return mk(t), mk(n), mk(r)
