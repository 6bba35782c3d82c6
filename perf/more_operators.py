"""The operators of drafted and branching rollouts and of token statistics, as they are measured.

Log probabilities of given tokens with entropy and top alternatives and their backward; the
attention of a tree of drafted tokens over the captured prompt and each member's own pages,
with the plan it reads; what follows the drafts' verification (the accepted path, its keys and
values moved together in every layer, pages given back); and the branching of responses (pages
shared, the partial one copied in every layer).

Every case is run in its plain form (elementary torch operations, in 32 bits where numbers are
computed) or, with ``own`` set, through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

D = 128          # head dimension
DEV = "cuda"


def listed():
    return [
        # One decode step of an 8-member group: the sampled tokens' log probabilities, the
        # entropies and 20 alternatives to log.  Latency counts.
        {"name": "logp decode step", "op": "logp", "T": 8, "V": 151936, "pad": 0, "dtype": "bf16",
         "top": 20, "temp": 1.0},
        # One 4,096-token response scored with entropies and a few alternatives.
        {"name": "logp response", "op": "logp", "T": 4096, "V": 151936, "pad": 0, "dtype": "bf16",
         "top": 5, "temp": 1.0},
        # A ragged batch over a vocabulary of odd size in padded fp32 rows, sampled at 0.7.
        {"name": "logp odd vocabulary", "op": "logp", "T": 1531, "V": 50257, "pad": 47, "dtype": "fp32",
         "top": 0, "temp": 0.7},
        # The backward of one response's objective (log probabilities and entropy).
        {"name": "logp_bwd response", "op": "logp_bwd", "T": 4096, "V": 151936, "pad": 0,
         "dtype": "bf16", "top": 0, "temp": 1.0},
        # The same with gradients of the alternatives (distillation), odd fp32 rows, a temperature.
        {"name": "logp_bwd alternatives", "op": "logp_bwd", "T": 513, "V": 32003, "pad": 0,
         "dtype": "fp32", "top": 8, "temp": 1.3},
        # Drafts of a two-member group over a short prompt: latency.
        {"name": "tree short prompt", "op": "tree", "P": 4096, "M": 2, "n": 8, "hq": 8, "hkv": 2,
         "ps": 64, "len": 100, "ragged": False},
        # 8 members with 16 drafted tokens each over the 2,097,152-token prompt.
        {"name": "tree 2M prompt", "op": "tree", "P": 2097152, "M": 8, "n": 16, "hq": 24, "hkv": 4,
         "ps": 64, "len": 4096, "ragged": False},
        # 64 members with ragged drafts of up to 24 tokens and long responses over a prompt of
        # odd length: a member's rows pass one tile.
        {"name": "tree 64 members", "op": "tree", "P": 32749, "M": 64, "n": 24, "hq": 24, "hkv": 4,
         "ps": 256, "len": 8192, "ragged": True},
        # After the verification of an 8-member group's 16-token drafts, 16 layers.
        {"name": "settle drafts", "op": "settle", "M": 8, "n": 16, "L": 16, "hkv": 4, "ps": 64,
         "len": 2048, "deep": 5},
        # 256 members with drafts of 64 tokens and long accepted paths, small pages.
        {"name": "settle large group", "op": "settle", "M": 256, "n": 64, "L": 16, "hkv": 4, "ps": 16,
         "len": 200, "deep": 24},
        # A short response branched seven times in a small model.
        {"name": "branch one response", "op": "branch", "B": 1, "M": 8, "L": 4, "hkv": 2, "ps": 16,
         "len": 300},
        # The branches of 8 long responses pruned and grown anew, 56 of them, 16 layers.
        {"name": "branch group", "op": "branch", "B": 8, "M": 64, "L": 16, "hkv": 4, "ps": 256,
         "len": 4096},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["logp", "logp", "logp_bwd", "tree", "tree", "settle", "branch"])
    if op in ("logp", "logp_bwd"):
        V = _log(rng, 1000, 200000)
        T = _log(rng, 1, min(4096, 400000000 // V))
        return {"op": op, "T": T, "V": V, "pad": rng.choice([0, 0, rng.randrange(1, 128)]),
                "dtype": rng.choice(["bf16", "bf16", "fp32"]), "top": rng.choice([0, 1, 5, 20, 32]),
                "temp": rng.choice([1.0, 0.6, 1.4])}
    if op == "tree":
        hkv, g = rng.choice([(1, 8), (2, 4), (4, 6), (8, 2), (5, 1), (2, 7), (3, 5)])
        M = _log(rng, 1, 64)
        n = min(rng.choice([2, 5, 8, 13, 16, 24, 32, 48, 64]), 19000 // (M * g))
        c = {"op": op, "P": _log(rng, 1, 500000), "M": M, "n": n, "hq": hkv * g, "hkv": hkv,
             "ps": rng.choice([16, 64, 256]), "len": _log(rng, 80, 8192), "ragged": rng.random() < 0.5}
        most = 2097152 * 8 * 16 * 24 // 4
        if c["P"] * M * n * hkv * g > most:
            c["P"] = max(1, most // (M * n * hkv * g) - rng.randrange(1000))
        return c
    c = {"op": op, "L": rng.choice([1, 4, 16]), "hkv": rng.choice([1, 2, 4, 8]), "ps": rng.choice([16, 64, 256])}
    if op == "settle":
        M, n = _log(rng, 1, 256), rng.choice([4, 8, 13, 16, 32, 64])
        c.update(M=M, n=n, len=_log(rng, 70, 4096), deep=rng.randint(1, n // 2))
        while M * (c["len"] + n) * c["L"] * c["hkv"] > 256 * 400 * 64:
            c["len"] = c["len"] // 2 + 1
            if c["len"] < 100:
                c["L"] = 1
                break
    else:
        B = _log(rng, 1, 16)
        c.update(B=B, M=B + _log(rng, 1, 60), len=_log(rng, 20, 4096))
    return c


# ------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 13)
    return g


def _perm(n, g):
    return torch.randperm(n, generator=g, device=DEV).to(torch.int32)


def _int(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)


def _prepare_logp(case, seed):
    g = _gen(seed)
    T, V, top = case["T"], case["V"], case["top"]
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    # a trained model's logits: a broad bulk and a few likely tokens a row
    z = torch.empty(T, V + case["pad"], device=DEV, dtype=dt).normal_(0, 2, generator=g)
    likely = torch.randint(0, V, (T, 8), generator=g, device=DEV)
    lift = torch.rand(T, 8, generator=g, device=DEV) * 8 + 6
    rows = torch.arange(T, device=DEV)[:, None]
    z[rows, likely] = lift.to(dt)
    pick = torch.randint(0, 8, (T, 1), generator=g, device=DEV)
    y = torch.where(torch.rand(T, generator=g, device=DEV) < 0.8, likely.gather(1, pick)[:, 0],
                    torch.randint(0, V, (T,), generator=g, device=DEV))
    s = dict(case)
    s["logits"], s["targets"] = z[:, :V], y.to(torch.int32)
    if case["op"] == "logp_bwd":
        # the forward's statistics and what an objective sends back
        x = s["logits"].float() / case["temp"]
        m = x.amax(-1, keepdim=True)
        e = torch.exp(x - m)
        den = e.sum(-1, dtype=torch.float64)
        s["lse"] = (m[:, 0].double() + torch.log(den)).float()
        s["entropy"] = (torch.log(den) - (e.double() * (x - m)).sum(-1) / den).float()
        s["d_logp"] = torch.randn(T, generator=g, device=DEV)
        s["d_entropy"] = torch.randn(T, generator=g, device=DEV) * 0.1
        s["ids"] = s["d_top"] = None
        if top:
            s["ids"] = _keys(s["logits"]).topk(top, -1).values.remainder(1 << 31).neg().add(V - 1).to(torch.int32)
            s["d_top"] = torch.randn(T, top, generator=g, device=DEV) * 0.3
    return s


def _prepare_tree(case, seed):
    g = _gen(seed)
    P, M, n, hq, hkv, ps = (case[k] for k in ("P", "M", "n", "hq", "hkv", "ps"))
    top = max(n, case["len"])
    lens = torch.randint(max(n, case["len"] // 16), top + 1, (M,), generator=g, device=DEV)
    s = dict(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)

    npg = -(-P // ps) + 2
    s["k_prompt"], s["v_prompt"] = normal(npg, hkv, ps, D), normal(npg, hkv, ps, D)
    s["table"] = _perm(npg, g)[:-(-P // ps)].contiguous()
    nb = -(-top // ps)
    s["k_resp"], s["v_resp"] = normal(M * nb, hkv, ps, D), normal(M * nb, hkv, ps, D)
    s["blocks"] = _perm(M * nb, g).view(M, nb).contiguous()
    s["lens"] = lens.to(torch.int32)
    s["q"] = (normal(M, n, hq, D) * 2).contiguous()
    s["scale"] = D ** -0.5
    # drafts: the first node follows the context, later ones one of the four before them; the
    # nodes are the last rows of a member
    drafted = (torch.randint((n + 1) // 2, n + 1, (M,), generator=g, device=DEV) if case["ragged"]
               else torch.full((M,), n, device=DEV))
    i = torch.arange(n, device=DEV)[None] - (n - drafted[:, None])
    back = (torch.rand(M, n, generator=g, device=DEV) * i.clamp(1, 4)).long()
    row = torch.arange(n, device=DEV)[None]
    s["parents"] = torch.where(i > 0, row - 1 - back, -1).to(torch.int32)
    s["drafted"] = drafted.to(torch.int32) if case["ragged"] else None
    s["visible"] = torch.zeros(M, n, (n + 31) // 32, dtype=torch.int32, device=DEV)
    s["pos"] = torch.zeros(1, M, n, dtype=torch.int32, device=DEV)
    s["o"] = torch.zeros_like(s["q"])
    s["lse"] = torch.zeros(M, n, hq, device=DEV)
    if own:
        from response_replay_gb300 import torch_api as api
        s["cache"] = api.PagedKVCache(npg, s["table"], ps, hkv, P, k_pool=s["k_prompt"],
                                      v_pool=s["v_prompt"])
        s["resp"] = api.ResponseCache(api.PagePool(s["k_resp"], s["v_resp"]), s["blocks"], s["lens"])
    return s


def _pools(case, pages, g):
    shape = (case["L"], pages, case["hkv"], case["ps"], D)
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16),
            torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16))


def _prepare_settle(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    M, n, ps, deep = case["M"], case["n"], case["ps"], case["deep"]
    lens = rng.integers(max(n, case["len"] // 16), max(n, case["len"]) + 1, M)
    have = -(-lens // ps)
    nb = int(-(-max(n, case["len"]) // ps)) + 1
    pages = M * nb
    free = rng.permutation(pages)
    table = np.full((M, nb), -1)
    cols = np.arange(nb)[None]
    first = np.cumsum(have) - have
    table = np.where(cols < have[:, None], free[np.minimum(first[:, None] + cols, pages - 1)], -1)
    parents = np.full((M, n), -1)
    back = (rng.random((M, n)) * np.minimum(np.maximum(np.arange(n), 1), 6)).astype(np.int64)
    parents[:, 1:] = np.arange(n - 1)[None] - back[:, 1:]
    tokens = np.stack([rng.permutation(151936)[:n] for _ in range(M)])
    chosen = 160000 + rng.integers(0, 1000, (M, n))  # no drafted token follows these
    for m in range(M):
        c = int(rng.integers(0, deep))
        path = [0, *sorted(rng.choice(np.arange(deep, n), c, replace=False))]
        for a, b in zip(path, path[1:]):
            parents[m, b] = a
            chosen[m, a] = tokens[m, b]
    s = dict(case)
    s["k"], s["v"] = _pools(case, pages, g)
    s.update(lens=_int(lens), table=_int(table), free=_int(free), used=_int([have.sum()]),
             parents=_int(parents), tokens=_int(tokens), chosen=_int(chosen),
             lens_out=_int(lens), used_out=_int([0]))
    if own:
        from response_replay_gb300 import torch_api as api
        s["alloc"] = api.PageAllocator(s["table"], s["lens"], s["free"], s["used"], ps)
        s["pools"] = api.LayerPools(s["k"], s["v"])
    return s


def _prepare_branch(case, seed):
    g, rng = _gen(seed), np.random.default_rng(seed)
    B, M, ps = case["B"], case["M"], case["ps"]
    lens = np.full(M, -1)
    lens[:B] = rng.integers(max(1, case["len"] // 2), case["len"] + 1, B)
    nb = -(-case["len"] // ps) + 1
    have = np.where(lens > 0, -(-lens // ps), 0)
    base = int(have.sum())
    pages = B * nb + M - B + 3
    free = rng.permutation(pages)
    cols = np.arange(nb)[None]
    first = np.cumsum(have) - have
    table = np.where(cols < have[:, None], free[np.minimum(first[:, None] + cols, pages - 1)], -1)
    src, keep, shared, used = np.full(M, -1), np.zeros(M, np.int64), np.zeros(pages, np.int64), base
    # branches at random points of the responses, as they stand before the pass; the pass
    # prunes them and grows the same number anew, at the same points
    for m in range(B, M):
        b = m % B
        src[m], keep[m] = b, int(rng.integers(1, lens[b] + 1))
        whole = keep[m] // ps
        table[m, :whole] = table[b, :whole]
        shared[table[b, :whole]] += 1
        if keep[m] % ps:
            table[m, whole] = free[used]
            used += 1
    pruned = lens.copy()
    lens[B:] = keep[B:]
    s = dict(case)
    s["k"], s["v"] = _pools(case, pages, g)
    s.update(lens=_int(lens), table=_int(table), free=_int(free), used=_int([used]), src=_int(src),
             keep=_int(keep), shared=_int(shared), pruned=_int(pruned),
             copies=torch.zeros(3, M, dtype=torch.int32, device=DEV))
    if own:
        from response_replay_gb300 import torch_api as api
        s["alloc"] = api.PageAllocator(s["table"], s["lens"], s["free"], s["used"], ps,
                                       shared=s["shared"])
        s["pools"] = api.LayerPools(s["k"], s["v"])
    return s


def prepare(case, seed):
    return {"logp": _prepare_logp, "logp_bwd": _prepare_logp, "tree": _prepare_tree,
            "settle": _prepare_settle, "branch": _prepare_branch}[case["op"]](case, seed)


def _bits(s):
    return s["k"].view(torch.int16), s["v"].view(torch.int16)  # copies are exact


# ------------------------------------------------------------------------- plain forms

def _keys(x):
    """Whole numbers that order a row's logits, ties to the lowest index."""
    b = (x.float() + 0.0).contiguous().view(torch.int32)  # one zero
    b = torch.where(b < 0, b ^ 0x7FFFFFFF, b).long()
    return (b << 31) + torch.arange(x.shape[-1] - 1, -1, -1, device=x.device)


def _plain_logp(s):
    x = s["logits"].float() / s["temp"]
    V = x.shape[1]
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    den = e.sum(-1, dtype=torch.float64)
    log_den = torch.log(den)
    lse = m[:, 0].double() + log_den
    entropy = log_den - (e.mul_(x - m)).sum(-1, dtype=torch.float64) / den
    logp = x.gather(1, s["targets"].long()[:, None])[:, 0].double() - lse
    out = [logp.float(), lse.float(), entropy.float()]
    if s["top"]:
        ids = V - 1 - _keys(s["logits"]).topk(s["top"], -1).values.remainder(1 << 31)
        out += [(x.gather(1, ids).double() - lse[:, None]).float(), ids.to(torch.int32)]
    return out


def _plain_logp_bwd(s):
    x = s["logits"].float() / s["temp"]
    lp = x - s["lse"][:, None]
    p = torch.exp(lp)
    total = s["d_logp"] if s["d_top"] is None else s["d_logp"] + s["d_top"].sum(-1)
    dx = p * (-total[:, None] - s["d_entropy"][:, None] * (lp + s["entropy"][:, None]))
    dx.scatter_add_(1, s["targets"].long()[:, None], s["d_logp"][:, None])
    if s["d_top"] is not None:
        dx.scatter_add_(1, s["ids"].long(), s["d_top"])
    return dx.div_(s["temp"]).to(s["logits"].dtype)


def _plain_plan(s):
    """Visible rows of every row as truth values [M][n][n], as words, and positions."""
    M, n = s["parents"].shape
    row = torch.arange(n, device=DEV)
    drafted = torch.full((M,), n, device=DEV) if s["drafted"] is None else s["drafted"].long()
    real = row[None] >= n - drafted[:, None]
    step = (s["parents"].long()[..., None] == row) & real[..., None]
    reach = step | (torch.eye(n, dtype=torch.bool, device=DEV) & real[..., None])
    reach = reach.float()
    for _ in range(max(1, (n - 1).bit_length())):
        reach = (reach @ reach).clamp_(max=1)
    see = reach > 0.5
    depth = see.sum(-1) - 1
    base = s["P"] + s["lens"].long() - drafted
    pos = torch.where(real, base[:, None] + depth, 0).to(torch.int32)[None]
    W = (n + 31) // 32
    bits = torch.nn.functional.pad(see, (0, W * 32 - n)).view(M, n, W, 32).long()
    words = (bits << torch.arange(32, device=DEV)).sum(-1)
    words = torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)
    return see, words, pos, real, drafted


def _plain_tree(s):
    P, M, n, hq, hkv, ps = (s[k] for k in ("P", "M", "n", "hq", "hkv", "ps"))
    see, words, pos, real, drafted = _plain_plan(s)
    g = hq // hkv
    table, blocks = s["table"].long(), s["blocks"].long()
    q = (s["q"].float() * s["scale"]).view(M, n, hkv, g, D)
    L = blocks.shape[1] * ps
    lens = s["lens"].long()
    key = torch.arange(L, device=DEV)[None] - (lens - n)[:, None]      # a key's row, if it is a draft
    context = key < (n - drafted)[:, None]
    mine = see.gather(2, key.clamp(0, n - 1)[:, None].expand(M, n, L))
    sees = context[:, None] | (mine & (key < n)[:, None])              # [M][n][L]
    gone = torch.arange(L, device=DEV)[None] >= lens[:, None]
    os, ls = [], []
    for h in range(hkv):
        qh = q[:, :, h].reshape(M * n * g, D)
        kp = s["k_prompt"][table, h].reshape(-1, D)[:P].float()
        vp = s["v_prompt"][table, h].reshape(-1, D)[:P].float()
        a = qh @ kp.T
        del kp
        kr = s["k_resp"][blocks, h].reshape(M, L, D).float()
        vr = s["v_resp"][blocks, h].reshape(M, L, D).float().masked_fill(gone[..., None], 0)
        b = torch.einsum("mxd,mld->mxl", qh.view(M, n * g, D), kr).view(M, n, g, L)
        b = b.masked_fill(~sees[:, :, None], -math.inf).view(M * n * g, L)
        mx = torch.maximum(a.amax(-1), b.amax(-1))[:, None]
        a, b = torch.exp(a.sub_(mx)), torch.exp(b.sub_(mx))
        den = (a.sum(-1, dtype=torch.float64) + b.sum(-1, dtype=torch.float64)).float()[:, None]
        o = a @ vp + torch.einsum("mxl,mld->mxd", b.view(M, n * g, L), vr).reshape(M * n * g, D)
        os.append((o / den).view(M, n, g, D))
        ls.append((mx + torch.log(den)).view(M, n, g))
    o = torch.cat(os, 2).masked_fill(~real[..., None, None], 0)
    return words, pos, o.to(torch.bfloat16), torch.cat(ls, 2).masked_fill(~real[..., None], 0)


def _plain_settle(s):
    M, n, ps = s["M"], s["n"], s["ps"]
    parents, tokens, chosen = (s[k].long() for k in ("parents", "tokens", "chosen"))
    row = torch.arange(n, device=DEV)
    par = parents.clamp(min=0)
    match = (parents >= 0) & (tokens == chosen.gather(1, par))
    # the lowest of the matching children of a node
    same = (parents[:, :, None] == parents[:, None]) & match[:, None] & (row < row[:, None])
    match &= ~same.any(-1)
    match[:, 0] = True
    step = torch.eye(n, device=DEV) + (parents[..., None] == row).float()
    for _ in range(max(1, (n - 1).bit_length())):
        step = (step @ step).clamp_(max=1)
    kept = ~((step > 0.5) & ~match[:, None]).any(-1)
    count = kept.sum(-1)
    order = torch.where(kept, row, n + row).sort(-1).values
    rows = torch.where(order < n, order, -1)
    last = rows.gather(1, count[:, None] - 1)
    follow = chosen.gather(1, last)[:, 0]
    lens = s["lens"].long()
    base = lens - n
    ends = base + count
    m, i = (rows >= 0).nonzero(as_tuple=True)
    at_from, at_to = base[m] + rows[m, i], base[m] + i
    table = s["table"].long()
    pf, of, pt, ot = table[m, at_from // ps], at_from % ps, table[m, at_to // ps], at_to % ps
    for pool in (s["k"], s["v"]):
        pool[:, pt, :, ot] = pool[:, pf, :, of]
    have, need = (lens + ps - 1) // ps, (ends + ps - 1) // ps
    cols = torch.arange(table.shape[1], device=DEV)[None]
    back = (cols >= need[:, None]) & (cols < have[:, None])
    pages = s["table"][back]
    used = s["used"] - pages.numel()
    free = s["free"]
    free[used.long() + torch.arange(pages.numel(), device=DEV)] = pages
    return (rows.to(torch.int32), count.to(torch.int32), follow.to(torch.int32), ends.to(torch.int32),
            used, free, *_bits(s))


def _plain_branch(s):
    ps, B = s["ps"], s["B"]
    table, lens, free, shared, used = (s[k] for k in ("table", "lens", "free", "shared", "used"))
    cols = torch.arange(table.shape[1], device=DEV)[None]
    # the branches pruned: shared pages lose an owner, the others go back
    have = (lens.long().clamp(min=0) + ps - 1) // ps
    need = (s["pruned"].long().clamp(min=0) + ps - 1) // ps
    pages = table[(cols >= need[:, None]) & (cols < have[:, None])].long()
    drops = torch.zeros_like(shared).index_add_(0, pages, torch.ones_like(pages, dtype=torch.int32))
    gone = (shared - drops)[pages] < 0
    shared.sub_(drops).clamp_(min=0)
    back = pages[gone].to(torch.int32)
    used -= back.numel()
    free[used.long() + torch.arange(back.numel(), device=DEV)] = back
    lens.copy_(s["pruned"])
    # and grown anew
    src, keep = s["src"].long(), s["keep"].long()
    new = src >= 0
    of = src.clamp(min=0)
    whole, part = keep // ps, keep % ps
    take = cols < whole[:, None]
    table.copy_(torch.where(new[:, None] & take, table[of], table))
    mine = table[new[:, None] & take].long()
    shared.index_add_(0, mine, torch.ones_like(mine, dtype=torch.int32))
    fresh = new & (part > 0)
    at = used.long() + torch.cumsum(fresh, 0) - 1
    page = torch.where(fresh, free[at.clamp(0, free.numel() - 1)], -1)
    m = fresh.nonzero()[:, 0]
    table[m, whole[m]] = page[m]
    source = table[of, whole.clamp(max=table.shape[1] - 1)]
    copies = torch.stack([torch.where(fresh, source, -1), page, torch.where(fresh, part, 0).to(torch.int32)])
    row = torch.arange(ps, device=DEV)
    live = (row < part[m][:, None])[None, :, None, :, None]
    for pool in (s["k"], s["v"]):
        a, b = pool[:, source[m].long()], pool[:, page[m].long()]
        pool[:, page[m].long()] = torch.where(live, a, b)
    lens.copy_(torch.where(new, s["keep"], lens))
    used += fresh.sum().to(torch.int32)
    return table, lens, shared, used, free, copies.to(torch.int32), *_bits(s)


def run(s):
    op = s["op"]
    if not own:
        return {"logp": _plain_logp, "logp_bwd": _plain_logp_bwd, "tree": _plain_tree,
                "settle": _plain_settle, "branch": _plain_branch}[op](s)
    from response_replay_gb300 import torch_api as api
    if op == "logp":
        out = api.token_logp_fwd(s["logits"], s["targets"], temperature=s["temp"], top=s["top"])
        return [x for x in out if x is not None]
    if op == "logp_bwd":
        return api.token_logp_bwd(s["logits"], s["targets"], s["lse"], s["entropy"], s["d_logp"],
                                  s["d_entropy"], temperature=s["temp"], top_ids=s["ids"],
                                  d_top=s["d_top"])
    if op == "tree":
        api.draft_tree(s["parents"], s["lens"], s["P"], drafted=s["drafted"], visible=s["visible"],
                       positions=s["pos"])
        api.decode_attn_tree(s["cache"], s["resp"], s["q"], s["visible"], s["scale"],
                             drafted=s["drafted"], o=s["o"], lse=s["lse"])
        return s["visible"], s["pos"], s["o"], s["lse"]
    if op == "settle":
        rows, count, follow, ends = api.accept_draft(s["parents"], s["tokens"], s["chosen"], s["lens"])
        api.compact_rows(s["alloc"], s["pools"], rows, count)
        api.trim_pages(s["alloc"], ends, lens_out=s["lens_out"], used_out=s["used_out"])
        return rows, count, follow, s["lens_out"], s["used_out"], s["free"], *_bits(s)
    api.trim_pages(s["alloc"], s["pruned"])
    api.fork_pages(s["alloc"], s["src"], s["keep"], copies=s["copies"])
    api.copy_pages(s["pools"], s["copies"])
    return s["table"], s["lens"], s["shared"], s["used"], s["free"], s["copies"], *_bits(s)


# ------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op in ("logp", "logp_bwd"):
        T, V, top = case["T"], case["V"], case["top"]
        e = 2 if case["dtype"] == "bf16" else 4
        if op == "logp":
            return {"bytes": T * (V * e + 16 + 8 * top), "flops": 6.0 * T * V}
        return {"bytes": T * (2 * V * e + 20 + 8 * top), "flops": 8.0 * T * V}
    if op == "tree":
        P, M, n, hq, hkv = (case[k] for k in ("P", "M", "n", "hq", "hkv"))
        part = 0.75 if case["ragged"] else 1.0
        resp = M * (max(n, case["len"] // 16) + max(n, case["len"])) / 2
        rows = M * n * hq * part
        return {"bytes": (P + resp) * hkv * D * 4 + rows * (D * 4 + 4),
                "flops": 4.0 * D * hq * n * part * (M * P + resp)}
    page = case["hkv"] * D * 4 * case["L"]  # a token's keys and values in every layer
    if op == "settle":
        moved = case["M"] * (case["deep"] - 1) / 2
        return {"bytes": 2 * moved * page + case["M"] * case["n"] * 16, "flops": 0}
    new = case["M"] - case["B"]
    blocks = 0.375 * case["len"] / case["ps"]  # of a branch, shared
    return {"bytes": new * (page * case["ps"] + blocks * 24), "flops": 0}


# ------------------------------------------------------------------------------ exact

def _exact_logp(s):
    T, V = s["logits"].shape
    outs = [[], [], [], [], []]
    for at in range(0, T, 256):
        x = s["logits"][at:at + 256].double() / s["temp"]
        y = s["targets"][at:at + 256].long()
        lp = x - torch.logsumexp(x, -1, keepdim=True)
        outs[0].append(lp[torch.arange(len(y), device=DEV), y])
        outs[1].append(torch.logsumexp(x, -1))
        outs[2].append(-(lp.exp() * lp).sum(-1))
        if s["top"]:
            v, i = lp.sort(stable=True, dim=-1, descending=True)
            outs[3].append(v[:, :s["top"]])
            outs[4].append(i[:, :s["top"]].to(torch.int32))
    return [torch.cat(o) for o in outs if o]


def _exact_logp_bwd(s):
    T, V = s["logits"].shape
    out = torch.empty(T, V, dtype=torch.float64, device=DEV)
    for at in range(0, T, 256):
        r = slice(at, at + 256)
        x = s["logits"][r].double() / s["temp"]
        lp = x - torch.logsumexp(x, -1, keepdim=True)
        p = lp.exp()
        h = -(p * lp).sum(-1, keepdim=True)
        up = torch.zeros_like(p)  # the gradient of the log probabilities
        up.scatter_add_(1, s["targets"][r].long()[:, None], s["d_logp"][r].double()[:, None])
        if s["top"]:
            up.scatter_add_(1, s["ids"][r].long(), s["d_top"][r].double())
        dz = up - p * up.sum(-1, keepdim=True) - s["d_entropy"][r].double()[:, None] * p * (lp + h)
        out[r] = dz / s["temp"]
    return out


def _exact_tree(s):
    P, M, n, hq, hkv = (s[k] for k in ("P", "M", "n", "hq", "hkv"))
    if M * n * P * hq > 8e9:
        return None
    g = hq // hkv
    o = torch.zeros(M, n, hq, D, dtype=torch.float64, device=DEV)
    lse = torch.zeros(M, n, hq, dtype=torch.float64, device=DEV)
    lens, parents = s["lens"].tolist(), s["parents"].tolist()
    drafted = [n] * M if s["drafted"] is None else s["drafted"].tolist()
    for h in range(hkv):
        k0 = s["k_prompt"][:, h][s["table"].long()].flatten(0, 1)[:P].double()
        v0 = s["v_prompt"][:, h][s["table"].long()].flatten(0, 1)[:P].double()
        for m in range(M):
            pg = s["blocks"][m].long()
            k1 = s["k_resp"][pg, h].flatten(0, 1)[:lens[m]].double()
            v1 = s["v_resp"][pg, h].flatten(0, 1)[:lens[m]].double()
            for i in range(n - drafted[m], n):
                seen, a = [], i
                while a >= 0:
                    seen.append(lens[m] - n + a)
                    a = parents[m][a]
                hide = torch.ones(lens[m], dtype=torch.bool, device=DEV)
                hide[:lens[m] - drafted[m]] = False
                hide[seen] = False
                qq = s["q"][m, i, h * g:(h + 1) * g].double()
                sc = torch.cat([qq @ k0.T, (qq @ k1.T).masked_fill(hide, -math.inf)], -1) * s["scale"]
                z = torch.logsumexp(sc, -1)
                w = torch.exp(sc - z[:, None])
                o[m, i, h * g:(h + 1) * g] = w[:, :P] @ v0 + w[:, P:] @ v1
                lse[m, i, h * g:(h + 1) * g] = z
    return None, None, o, lse


def exact(case, seed):
    if case["op"] in ("settle", "branch"):  # whole numbers and copies: nothing is computed
        return None
    s = prepare(case, seed)
    return {"logp": _exact_logp, "logp_bwd": _exact_logp_bwd, "tree": _exact_tree}[case["op"]](s)
