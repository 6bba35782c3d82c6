"""Plain 64-bit implementations of the token statistics, of drafted trees and of branching
pages (numpy, on the host), with the error bounds that the GPU tests hold the kernels to."""
from __future__ import annotations

import numpy as np

U32 = 2.0 ** -24   # half a step of fp32, relative
U16 = 2.0 ** -8    # half a step of bf16
TINY = 2.0 ** -126  # exponentials below it are zero on the GPU


def log_probs(z, temperature):
    """(log p, lse) of the rows of z."""
    x = np.asarray(z, np.float64) / temperature
    with np.errstate(invalid="ignore", divide="ignore"):
        m = x.max(-1, keepdims=True)
        lse = m + np.log(np.exp(x - m).sum(-1, keepdims=True))
        return x - lse, lse[:, 0]


def entropy(lp):
    with np.errstate(invalid="ignore"):
        return -np.where(lp == -np.inf, 0, np.exp(lp) * lp).sum(-1)


def top(z, k):
    """Ids of the k largest, equal ones by the lowest id."""
    return np.argsort(-np.asarray(z, np.float64), axis=-1, kind="stable")[:, :k]


def stat_bounds(z, temperature):
    """Bounds of lse (and, with their own rounding, of log probabilities) and of the entropy.

    A term 2^t of t = (z - m) c carries t's three roundings (3 |t| half steps, times ln 2) and
    the exponential's 2^-21; a sum over V terms is a chain of V / 512, or, where a warp takes a
    row, of V / 64, 512 at most (one more for each of its rescales, one per 8 terms at most), and a
    tree.  The last steps are in 64 bits but for a
    logarithm of 2^-22 and the result's rounding."""
    lp, lse = log_probs(z, temperature)
    V = z.shape[1]
    p = np.exp(lp)
    with np.errstate(invalid="ignore"):
        u = np.where(p > 0, lp - lp.max(-1, keepdims=True), 0)  # = t ln 2
    a1, a2 = (p * np.abs(u)).sum(-1), (p * u * u).sum(-1)
    chain = 1.5 * max(V / 512, min(V / 64, 512)) + 80
    es = 2.0 ** -21 + chain * U32 + 3 * U32 * a1
    h = entropy(lp)
    e_lse = es + 2.0 ** -21 + U32 * np.abs(lse)
    e_h = es + 2.0 ** -21 + a1 * (2.0 ** -21 + es + (chain + 8) * U32) + 3 * U32 * a2 + 4 * U32 * np.abs(h)
    return lp, lse, h, e_lse, e_h


def token_logp_bwd(z, targets, lse, h, d_logp, d_entropy, temperature, ids=None, d_top=None):
    """Gradient of the logits from the forward's lse and entropy, and its bound before the
    rounding to the logits' type (fp32: U32, bf16: U16 of the value)."""
    z = np.asarray(z, np.float64)
    T, V = z.shape
    u = z / temperature - np.asarray(lse, np.float64)[:, None]
    p = np.exp(u)
    with np.errstate(invalid="ignore"):
        u = np.where(p > 0, u, 0)
    zero = np.zeros(T)
    g = zero if d_logp is None else np.asarray(d_logp, np.float64)
    dh = zero if d_entropy is None else np.asarray(d_entropy, np.float64)
    h = zero if h is None else np.asarray(h, np.float64)
    total, size = g.copy(), np.abs(g)
    if ids is not None:
        total += np.asarray(d_top, np.float64).sum(-1)
        size = size + np.abs(d_top).sum(-1)
    dz = -p * (total[:, None] + dh[:, None] * (u + h[:, None]))
    mag = p * (size[:, None] + np.abs(dh[:, None]) * (np.abs(u) + np.abs(h[:, None])))
    # the exponent: its roundings and the temperature's reciprocal's (at the logit's size)
    rel = 2.0 ** -21 + U32 * (44 + 4 * np.abs(u) + 4 * np.abs(np.where(p > 0, z, 0) / temperature))
    err = np.nan_to_num(mag * rel)
    rows = np.arange(T)
    if targets is not None and d_logp is not None:
        np.add.at(dz, (rows, targets), g)
        np.add.at(err, (rows, targets), 40 * U32 * np.abs(g))
    if ids is not None:
        for j in range(ids.shape[1]):
            np.add.at(dz, (rows, ids[:, j]), d_top[:, j])
            np.add.at(err, (rows, ids[:, j]), 40 * U32 * np.abs(d_top[:, j]))
    return dz / temperature, err / temperature + 64 * TINY * (1 + size[:, None])


# ------------------------------------------------------------------------------- drafts

def draft(lens, drafted, n):
    """First drafted row of every member."""
    d = np.full(len(lens), n) if drafted is None else np.asarray(drafted)
    return np.where(np.asarray(lens) < 0, n, n - d)


def draft_tree(parents, lens, drafted, pos0):
    """(sees [M][n][n] truth values, words, positions [M][n])."""
    parents = np.asarray(parents)
    M, n = parents.shape
    first = draft(lens, drafted, n)
    see = np.zeros((M, n, n), bool)
    pos = np.zeros((M, n), np.int64)
    for m in range(M):
        for r in range(first[m], n):
            see[m, r, r] = True
            depth = 0
            if parents[m, r] >= 0:
                see[m, r] |= see[m, parents[m, r]]
                depth = see[m, r].sum() - 1
            pos[m, r] = pos0 + lens[m] - (n - first[m]) + depth
    W = (n + 31) // 32
    bits = np.zeros((M, n, W * 32), np.uint64)
    bits[..., :n] = see
    words = (bits.reshape(M, n, W, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
    return see, words.view(np.int32), pos.astype(np.int32)


def accept(parents, tokens, chosen, lens, drafted):
    M, n = np.asarray(parents).shape
    first = draft(lens, drafted, n)
    rows = np.full((M, n), -1)
    count, follow, ends = np.zeros(M, int), np.full(M, -1), np.array(lens, int)
    for m in range(M):
        at = first[m]
        path = []
        while at is not None and at < n:
            path.append(at)
            follow[m] = chosen[m][at]
            at = next((c for c in range(at + 1, n) if parents[m][c] == at and tokens[m][c] >= 0
                       and tokens[m][c] == chosen[m][at]), None)
        rows[m, :len(path)] = path
        count[m] = len(path)
        if lens[m] >= 0:
            ends[m] = lens[m] - (n - first[m]) + len(path)
    return rows, count, follow, ends


def compact(pool, table, lens, drafted, rows, count, ps):
    """pool [pages][Hkv][ps][...], one layer; returns a new one."""
    out = pool.copy()
    n = np.asarray(rows).shape[1]
    first = draft(lens, drafted, n)
    for m in range(len(lens)):
        base = lens[m] - (n - first[m])
        for i in range(count[m]):
            a, b = base + rows[m][i] - first[m], base + i
            out[table[m][b // ps], :, b % ps] = pool[table[m][a // ps], :, a % ps]
    return out


# ------------------------------------------------------------------------------- pages

def pages_of(n, ps):
    return -(-max(int(n), 0) // ps)


def trim(table, lens, new, free, used, shared, ps, num_pages):
    """Member by member; None when the call has to be refused."""
    table, free = np.asarray(table), np.array(free)
    shared = None if shared is None else np.array(shared)
    back, out = [], []
    owners = {}
    for m, (a, b) in enumerate(zip(lens, new)):
        if (a < 0 and b >= 0) or b > a or pages_of(a, ps) > table.shape[1]:
            return None
        out.append(a if a < 0 else max(b, -1))
        for blk in range(pages_of(b, ps), pages_of(a, ps)):
            page = table[m, blk]
            if not 0 <= page < num_pages:
                return None
            owners.setdefault(page, []).append(len(owners))
    if not 0 <= used <= len(free):
        return None
    drops = {}
    for m, (a, b) in enumerate(zip(lens, new)):
        for blk in range(pages_of(b, ps), pages_of(a, ps)):
            page = table[m, blk]
            first = page not in drops
            drops[page] = drops.get(page, 0) + 1
            if shared is None or (first and shared[page] + 1 == len(owners[page])):
                back.append(page)
    if shared is not None:
        for page, n in drops.items():
            if n > shared[page] + 1:
                return None
            shared[page] = max(shared[page] - n, 0)
        for m, (a, b) in enumerate(zip(lens, new)):
            if 0 < b < a and b % ps:
                page = table[m, b // ps]
                if 0 <= page < num_pages and shared[page] > 0 and page not in back:
                    return None
    if len(back) > used:
        return None
    free[used - len(back):used] = back
    return np.array(out), free, used - len(back), shared


def fork(table, lens, src, keep, free, used, shared, ps, num_pages):
    table, shared, out = np.array(table), np.array(shared), np.array(lens)
    M = len(lens)
    copies = np.stack([np.full(M, -1), np.full(M, -1), np.zeros(M, int)])
    for m in range(M):
        s = src[m]
        if s < 0:
            continue
        if s >= M or s == m or lens[m] > 0 or lens[s] < 0 or src[s] >= 0:
            return None
        n = lens[s] if keep is None else keep[m]
        if not 0 <= n <= lens[s] or pages_of(lens[s], ps) > table.shape[1]:
            return None
        whole, part = divmod(int(n), ps)
        for b in range(whole + (part > 0)):
            if not 0 <= table[s, b] < num_pages:
                return None
        for b in range(whole):
            table[m, b] = table[s, b]
            shared[table[s, b]] += 1
        if part:
            if used >= len(free) or not 0 <= free[used] < num_pages:
                return None
            copies[:, m] = table[s, whole], free[used], part
            table[m, whole] = free[used]
            used += 1
        out[m] = n
    return table, out, used, shared, copies
