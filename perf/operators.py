"""The operators around the attention calls, as they are measured.

A layer's stage between its projections and the attention (per-head norms of queries and
keys with the rotary positions, forward, backward, and fused with the write into pages)
and the decode step of a group whose members share one captured prompt (pages and slots
from the members' lengths; attention over the prompt and each member's own pages).

Every case is run in its plain form (elementary torch operations in 32 bits) or, with
``own`` set, through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

D = 128          # head dimension
EPS = 1e-6       # of the norms
BASE = 1.0e7     # rotary base of long-context models
DEV = "cuda"


def listed():
    return [
        # One short response of the smallest workload (8 / 2 heads, 256 tokens), every
        # value rotated: latency counts.
        {"name": "norm_rotary_fwd short response", "op": "fwd", "T": 256, "hq": 8, "hkv": 2,
         "rot": 128, "axes": 1, "interleaved": False, "offset": 0.0},
        # A whole group's responses (8 x 4,096 tokens, 24 / 4 heads) before the replay
        # forward, half of each head rotated, zero-centred weights.
        {"name": "norm_rotary_fwd group", "op": "fwd", "T": 32768, "hq": 24, "hkv": 4, "rot": 64,
         "axes": 1, "interleaved": False, "offset": 1.0},
        # An odd number of image and video tokens: three axes (time, height, width),
        # neighbouring values as pairs.
        {"name": "norm_rotary_fwd three axes", "op": "fwd", "T": 8191, "hq": 16, "hkv": 8,
         "rot": 128, "axes": 3, "interleaved": True, "offset": 0.0},
        # The backward of one 4,096-token response, fed by the replay backward's fp32.
        {"name": "norm_rotary_bwd response", "op": "bwd", "T": 4096, "hq": 24, "hkv": 4, "rot": 128,
         "axes": 1, "interleaved": False, "offset": 0.0, "grads": "fp32"},
        # A ragged group's tokens with three axes and bf16 gradients.
        {"name": "norm_rotary_bwd three axes", "op": "bwd", "T": 20011, "hq": 12, "hkv": 2,
         "rot": 64, "axes": 3, "interleaved": False, "offset": 1.0, "grads": "bf16"},
        # One decode step of an 8-member group: 8 tokens into their pages.
        {"name": "append decode step", "op": "append", "T": 8, "hq": 24, "hkv": 4, "rot": 128,
         "axes": 1, "interleaved": False, "offset": 0.0, "ps": 64, "pages": 64},
        # A chunk of the prompt on its way into the page pool.
        {"name": "append prompt chunk", "op": "append", "T": 65536, "hq": 24, "hkv": 4, "rot": 64,
         "axes": 1, "interleaved": False, "offset": 1.0, "ps": 64, "pages": 1100},
        # Pages and slots of one decode step of an 8-member group.
        {"name": "extend decode step", "op": "extend", "M": 8, "add": 1, "len": 4096, "ps": 64,
         "pos0": 2097152},
        # 64 ragged responses of 512 to 8,192 tokens entered at once.
        {"name": "extend ragged group", "op": "extend", "M": 64, "add": 8192, "len": 300, "ps": 256,
         "pos0": 4194304},
        # The first steps of a two-member group over a short prompt: latency.
        {"name": "decode short prompt", "op": "decode", "P": 4096, "M": 2, "n": 1, "hq": 8, "hkv": 2,
         "ps": 64, "len": 100},
        # An 8-member group over the 2,097,152-token prompt, responses up to 4,096 tokens.
        {"name": "decode 2M prompt", "op": "decode", "P": 2097152, "M": 8, "n": 1, "hq": 24, "hkv": 4,
         "ps": 64, "len": 4096},
        # 64 members with long ragged responses over an odd 262,139-token prompt: more
        # rows than one tile, and as much response as prompt.
        {"name": "decode 64 members", "op": "decode", "P": 262139, "M": 64, "n": 1, "hq": 24, "hkv": 4,
         "ps": 256, "len": 8192},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "bwd", "append", "extend", "decode", "decode"])
    hkv, g = rng.choice([(1, 8), (2, 4), (4, 6), (8, 2), (5, 1), (2, 7), (4, 8), (3, 5)])
    if op == "extend":
        c = {"op": op, "M": _log(rng, 1, 1000), "add": 1, "len": _log(rng, 1, 8192),
             "ps": rng.choice([16, 64, 256]), "pos0": rng.choice([0, 131072, 2097152])}
        c["add"] = _log(rng, 1, max(2, min(8192, 300000 // c["M"])))
        return c
    if op == "decode":
        c = {"op": op, "P": _log(rng, 1, 1000000), "M": _log(rng, 1, 64), "n": rng.choice([1, 1, 1, 2, 5]),
             "hq": hkv * g, "hkv": hkv, "ps": rng.choice([16, 64, 256]), "len": _log(rng, 5, 8192)}
        if c["P"] * c["M"] * c["n"] * c["hq"] > 2097152 * 8 * 24:
            c["P"] = 2097152 * 8 * 24 // (c["M"] * c["n"] * c["hq"]) - rng.randrange(1000)
        return c
    c = {"op": op, "T": _log(rng, 1, 900000 // (hkv * (g + 2))), "hq": hkv * g, "hkv": hkv,
         "rot": rng.choice([32, 64, 96, 128]), "axes": rng.choice([1, 1, 2, 3, 4]),
         "interleaved": rng.random() < 0.4, "offset": float(rng.choice([0, 1]))}
    if op == "bwd":
        c["grads"] = rng.choice(["fp32", "bf16"])
    if op == "append":
        c["ps"] = rng.choice([16, 64, 256])
        c["pages"] = -(-c["T"] // c["ps"]) + rng.randrange(1, 40)
    return c


# ------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed) * 7919 + 11)
    return g


def _perm(n, g):
    return torch.randperm(n, generator=g, device=DEV).to(torch.int32)


def _inv_freq(rot):
    j = torch.arange(rot // 2, dtype=torch.float64, device=DEV)
    return torch.exp(-math.log(BASE) * 2.0 * j / rot)


def _pair_axis(rot, axes):
    # pairs dealt to the axes in contiguous sections, the first one the largest
    half = rot // 2
    per = half // (axes + 1)
    cuts = [half - per * (axes - 1 - a) for a in range(axes)]
    a = torch.zeros(half, dtype=torch.int32, device=DEV)
    for i in range(1, axes):
        a[cuts[i - 1]:] = i
    return a


def _prepare_norm(case, seed):
    g = _gen(seed)
    T, hq, hkv = case["T"], case["hq"], case["hkv"]
    # the packed projection of a layer: queries, keys and values of a token side by side
    x = torch.randn(T, (hq + 2 * hkv) * D, generator=g, device=DEV, dtype=torch.float32)
    x *= torch.rand(T, 1, generator=g, device=DEV) * 3 + 0.1
    x = x.to(torch.bfloat16)
    s = dict(case)
    s["q"] = x[:, :hq * D].unflatten(1, (hq, D))
    s["k"] = x[:, hq * D:(hq + hkv) * D].unflatten(1, (hkv, D))
    s["v"] = x[:, (hq + hkv) * D:].unflatten(1, (hkv, D))
    for n in ("wq", "wk"):
        s[n] = torch.rand(D, generator=g, device=DEV) + 0.5 - case["offset"]
    # positions behind a long prompt; image axes are small grids behind it
    p = torch.randint(0, 4194304 - T, (1,), generator=g, device=DEV) + torch.arange(T, device=DEV)
    rows = [p] + [p // (7 * a) % 977 + p[0] for a in range(1, case["axes"])]
    s["pos"] = torch.stack(rows).to(torch.int32).contiguous()
    s["freq"] = _inv_freq(case["rot"])
    s["axis"] = _pair_axis(case["rot"], case["axes"]) if case["axes"] > 1 else None
    if case["op"] == "bwd":
        dt = torch.float32 if case["grads"] == "fp32" else torch.bfloat16
        for n, h in (("dq", hq), ("dk", hkv), ("dv", hkv)):
            s[n] = torch.randn(T, h, D, generator=g, device=DEV).to(dt)
    if case["op"] == "append":
        ps, pages = case["ps"], case["pages"]
        if T <= pages:  # one token per member: each in a page of its own
            page, off = _perm(pages, g)[:T], torch.randint(0, ps, (T,), generator=g, device=DEV)
        else:
            t = torch.arange(T, device=DEV)
            page, off = _perm(pages, g)[t // ps], t % ps
        s["slots"] = (page * ps + off).to(torch.int32)
        s["k_pool"] = torch.zeros(pages, hkv, ps, D, dtype=torch.bfloat16, device=DEV)
        s["v_pool"] = torch.zeros_like(s["k_pool"])
    if own:
        from response_replay_gb300 import torch_api as api
        s["rotary"] = api.Rotary(s["freq"], pair_axis=s["axis"], axes=case["axes"],
                                 interleaved=case["interleaved"])
        if case["op"] == "append":
            s["pool"] = api.PagePool(s["k_pool"], s["v_pool"])
    return s


def _adds(case):
    lo, hi, M = max(1, case["add"] // 16), case["add"], case["M"]
    return [lo + (hi - lo) * (m + 1) // M for m in range(M)]


def _prepare_extend(case, seed):
    g = _gen(seed)
    M, ps = case["M"], case["ps"]
    lens = torch.randint(0, case["len"] + 1, (M,), generator=g, device=DEV)
    # ragged, and the same total for every seed: the user's buffers keep their size
    add = torch.tensor(_adds(case), device=DEV)[torch.randperm(M, generator=g, device=DEV)]
    have = (lens + ps - 1) // ps
    need = (lens + add + ps - 1) // ps
    max_blocks = (case["len"] + case["add"] + ps - 1) // ps + 3
    total = int(need.sum())
    free = _perm(total + 17, g)
    used = int(have.sum())
    table = torch.full((M, max_blocks), -1, dtype=torch.int32, device=DEV)
    first = torch.cumsum(have, 0) - have
    cols = torch.arange(max_blocks, device=DEV)[None]
    idx = (first[:, None] + cols).clamp(max=total)
    table = torch.where(cols < have[:, None], free[idx], table).contiguous()
    s = dict(case)
    cap = int(add.sum())
    cap += -cap % 64
    s.update(lens=lens.to(torch.int32), add=add.to(torch.int32), table=table, free=free,
             used=torch.tensor([used], dtype=torch.int32, device=DEV),
             slots=torch.empty(cap, dtype=torch.int32, device=DEV),
             pos=torch.empty(1, cap, dtype=torch.int32, device=DEV),
             lens_out=torch.empty(M, dtype=torch.int32, device=DEV),
             used_out=torch.empty(1, dtype=torch.int32, device=DEV))
    if own:
        from response_replay_gb300 import torch_api as api
        s["alloc"] = api.PageAllocator(s["table"], s["lens"], s["free"], s["used"], ps)
    return s


def _prepare_decode(case, seed):
    g = _gen(seed)
    P, M, n, hq, hkv, ps = (case[k] for k in ("P", "M", "n", "hq", "hkv", "ps"))
    lens = torch.randint(max(n, case["len"] // 16), max(n, case["len"]) + 1, (M,), generator=g, device=DEV)
    s = dict(case)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEV, dtype=torch.bfloat16)

    # queries and keys behind a norm with its weights: unit keys, queries somewhat larger,
    # so that some keys carry much of a row's weight
    npg = -(-P // ps) + 2
    s["k_prompt"], s["v_prompt"] = normal(npg, hkv, ps, D), normal(npg, hkv, ps, D)
    s["table"] = _perm(npg, g)[:-(-P // ps)].contiguous()
    nb = -(-max(n, case["len"]) // ps)
    s["k_resp"], s["v_resp"] = normal(M * nb, hkv, ps, D), normal(M * nb, hkv, ps, D)
    s["blocks"] = _perm(M * nb, g).view(M, nb).contiguous()
    s["lens"] = lens.to(torch.int32)
    s["q"] = (normal(M, n, hq, D) * 2).contiguous()
    s["scale"] = D ** -0.5
    s["o"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(M, n, hq, device=DEV)
    if own:
        from response_replay_gb300 import torch_api as api
        s["cache"] = api.PagedKVCache(npg, s["table"], ps, hkv, P, k_pool=s["k_prompt"],
                                      v_pool=s["v_prompt"])
        s["resp"] = api.ResponseCache(api.PagePool(s["k_resp"], s["v_resp"]), s["blocks"], s["lens"])
    return s


def prepare(case, seed):
    if case["op"] == "extend":
        return _prepare_extend(case, seed)
    if case["op"] == "decode":
        return _prepare_decode(case, seed)
    return _prepare_norm(case, seed)


# ------------------------------------------------------------------------- plain forms

def _angles(s):
    pos = s["pos"].double()
    p = pos[0][:, None] if s["axis"] is None else pos[s["axis"].long()].T
    a = p * s["freq"]
    return torch.cos(a).float(), torch.sin(a).float()


def _rotate(y, cos, sin, rot, interleaved, back=False):
    if back:
        sin = -sin
    c, n = cos[:, None], sin[:, None]
    out = y.clone()
    if interleaved:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        out[..., 0:rot:2] = a * c - b * n
        out[..., 1:rot:2] = b * c + a * n
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        out[..., :rot // 2] = a * c - b * n
        out[..., rot // 2:rot] = b * c + a * n
    return out


def _plain_fwd(s):
    cos, sin = _angles(s)
    outs = []
    for n in ("q", "k"):
        x = s[n].float()
        y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (s["w" + n] + s["offset"])
        outs.append(_rotate(y, cos, sin, s["rot"], s["interleaved"]).to(torch.bfloat16))
    return outs[0], outs[1], s["v"].contiguous()


def _plain_bwd(s):
    cos, sin = _angles(s)
    dx, dw = [], []
    for n in ("q", "k"):
        x = s[n].float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        xh = x * r
        gr = _rotate(s["d" + n].float(), cos, sin, s["rot"], s["interleaved"], back=True)
        dw.append((gr * xh).double().sum((0, 1)).float())
        h = gr * (s["w" + n] + s["offset"])
        dx.append((r * (h - xh * (h * xh).mean(-1, keepdim=True))).to(torch.bfloat16))
    return dx[0], dx[1], s["dv"].to(torch.bfloat16), dw[0], dw[1]


def _plain_append(s):
    q, k, v = _plain_fwd(s)
    page, off = (s["slots"] // s["ps"]).long(), (s["slots"] % s["ps"]).long()
    s["k_pool"][page, :, off] = k
    s["v_pool"][page, :, off] = v
    return q, s["k_pool"], s["v_pool"]


def _plain_extend(s):
    ps, cap = s["ps"], s["slots"].numel()
    lens, add = s["lens"].long(), s["add"].long()
    have, need = (lens + ps - 1) // ps, (lens + add + ps - 1) // ps
    new = need - have
    first = s["used"].long() + torch.cumsum(new, 0) - new
    cols = torch.arange(s["table"].shape[1], device=DEV)[None]
    fresh = (cols >= have[:, None]) & (cols < need[:, None])
    idx = (first[:, None] + cols - have[:, None]).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][idx], s["table"])
    end = torch.cumsum(add, 0)
    t = torch.arange(cap, device=DEV)
    m = torch.searchsorted(end, t, right=True)
    real = m < lens.numel()
    m = m.clamp(max=lens.numel() - 1)
    i = lens[m] + t - (end - add)[m]
    page = table[m, (i // ps).clamp(0, table.shape[1] - 1)]
    slots = torch.where(real, page * ps + i % ps, -1).to(torch.int32)
    pos = torch.where(real, s["pos0"] + i, 0).to(torch.int32)[None]
    used = (s["used"] + new.sum()).to(torch.int32)
    return slots, pos, table, (lens + add).to(torch.int32), used


def _plain_decode(s):
    P, M, n, hq, hkv, ps = (s[k] for k in ("P", "M", "n", "hq", "hkv", "ps"))
    g = hq // hkv
    table, blocks = s["table"].long(), s["blocks"].long()
    q = (s["q"].float() * s["scale"]).view(M, n, hkv, g, D)
    L = blocks.shape[1] * ps
    seen = s["lens"].long()[:, None] - n + 1 + torch.arange(n, device=DEV)[None]     # [M][n]
    hide = torch.arange(L, device=DEV)[None, None] >= seen[..., None]                 # [M][n][L]
    gone = torch.arange(L, device=DEV)[None] >= s["lens"].long()[:, None]
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
        b = b.masked_fill(hide[:, :, None], -math.inf).view(M * n * g, L)
        mx = torch.maximum(a.amax(-1), b.amax(-1))[:, None]
        a, b = torch.exp(a.sub_(mx)), torch.exp(b.sub_(mx))
        den = (a.sum(-1, dtype=torch.float64) + b.sum(-1, dtype=torch.float64)).float()[:, None]
        o = a @ vp + torch.einsum("mxl,mld->mxd", b.view(M, n * g, L), vr).reshape(M * n * g, D)
        os.append((o / den).view(M, n, g, D))
        ls.append((mx + torch.log(den)).view(M, n, g))
    return torch.cat(os, 2).to(torch.bfloat16), torch.cat(ls, 2)


def run(s):
    op = s["op"]
    if not own:
        return {"fwd": _plain_fwd, "bwd": _plain_bwd, "append": _plain_append,
                "extend": _plain_extend, "decode": _plain_decode}[op](s)
    from response_replay_gb300 import torch_api as api
    if op == "fwd":
        return api.qk_norm_rope_fwd(s["q"], s["k"], s["v"], s["pos"], s["rotary"], wq=s["wq"],
                                    wk=s["wk"], eps=EPS, weight_offset=s["offset"])
    if op == "bwd":
        return api.qk_norm_rope_bwd(s["q"], s["k"], s["pos"], s["rotary"], s["dq"], s["dk"], s["dv"],
                                    wq=s["wq"], wk=s["wk"], eps=EPS, weight_offset=s["offset"])
    if op == "append":
        q = api.qk_norm_rope_append(s["pool"], s["q"], s["k"], s["v"], s["slots"], s["pos"],
                                    s["rotary"], wq=s["wq"], wk=s["wk"], eps=EPS,
                                    weight_offset=s["offset"])
        return q, s["k_pool"], s["v_pool"]
    if op == "extend":
        api.extend_pages(s["alloc"], s["add"], s["pos0"], s["slots"], s["pos"],
                         lens_out=s["lens_out"], used_out=s["used_out"])
        return s["slots"], s["pos"], s["table"], s["lens_out"], s["used_out"]
    return api.decode_attn(s["cache"], s["resp"], s["q"], s["scale"], o=s["o"], lse=s["lse"])


# ------------------------------------------------------------------------------- work

def work(case):
    op = case["op"]
    if op == "extend":
        M, tok = case["M"], sum(_adds(case))
        pages = tok / case["ps"]
        # lengths in and out, one table entry and free-list entry per new page, a slot and
        # a position per token
        return {"bytes": 12 * M + 8 * pages + 8 * tok, "flops": 0}
    if op == "decode":
        P, M, n, hq, hkv = (case[k] for k in ("P", "M", "n", "hq", "hkv"))
        resp = M * (max(n, case["len"] // 16) + max(n, case["len"])) / 2
        rows = M * n * hq
        return {"bytes": (P + resp) * hkv * D * 4 + rows * (D * 4 + 4),
                "flops": 4.0 * D * hq * n * (M * P + resp)}
    T, hq, hkv = case["T"], case["hq"], case["hkv"]
    elems = T * (hq + 2 * hkv) * D
    if op == "bwd":
        gb = 4 if case["grads"] == "fp32" else 2
        # x of queries and keys, the three gradients in, the three gradients out
        return {"bytes": T * (hq + hkv) * D * 2 + elems * (gb + 2) + 4 * T * case["axes"],
                "flops": 20.0 * T * (hq + hkv) * D}
    return {"bytes": elems * 4 + 4 * T * case["axes"], "flops": 8.0 * T * (hq + hkv) * D}


# ------------------------------------------------------------------------------ exact

def _turn(s):
    """exp(i angle) of each token and pair, in 64 bits: [T][1][rot/2]."""
    T, half = s["pos"].shape[1], s["rot"] // 2
    ang = torch.empty(T, half, dtype=torch.float64, device=DEV)
    for j in range(half):
        a = 0 if s["axis"] is None else int(s["axis"][j])
        ang[:, j] = s["pos"][a].double() * BASE ** (-2.0 * j / s["rot"])
    return torch.polar(torch.ones_like(ang), ang)[:, None]


def _as_complex(x, s):
    r = s["rot"]
    if s["interleaved"]:
        return torch.complex(x[..., 0:r:2], x[..., 1:r:2])
    return torch.complex(x[..., :r // 2], x[..., r // 2:r])


def _from_complex(z, x, s):
    r = s["rot"]
    parts = (torch.stack([z.real, z.imag], -1).flatten(-2) if s["interleaved"]
             else torch.cat([z.real, z.imag], -1))
    return torch.cat([parts, x[..., r:]], -1)


def _exact_norm(s):
    turn = _turn(s)
    res = {}
    for n in ("q", "k"):
        x = s[n].double()
        w = s["w" + n].double() + s["offset"]
        rms = (x.square().sum(-1, keepdim=True) / D + EPS).sqrt()
        if s["op"] != "bwd":
            y = x / rms * w
            res[n] = _from_complex(_as_complex(y, s) * turn, y, s)
            continue
        up = s["d" + n].double()
        gr = _from_complex(_as_complex(up, s) * turn.conj(), up, s)
        res["w" + n] = (gr * x / rms).sum((0, 1))
        h = gr * w
        res[n] = h / rms - x * (h * x).sum(-1, keepdim=True) / (D * rms ** 3)
    return res


def _exact_decode(s):
    P, M, n, hq, hkv, ps = (s[k] for k in ("P", "M", "n", "hq", "hkv", "ps"))
    g = hq // hkv
    o = torch.empty(M, n, hq, D, dtype=torch.float64, device=DEV)
    lse = torch.empty(M, n, hq, dtype=torch.float64, device=DEV)
    lens = s["lens"].tolist()
    for h in range(hkv):
        k0 = s["k_prompt"][:, h][s["table"].long()].flatten(0, 1)[:P].double()
        v0 = s["v_prompt"][:, h][s["table"].long()].flatten(0, 1)[:P].double()
        for m in range(M):
            pg = s["blocks"][m].long()
            for i in range(n):
                end = lens[m] - n + 1 + i
                k1 = s["k_resp"][pg, h].flatten(0, 1)[:end].double()
                v1 = s["v_resp"][pg, h].flatten(0, 1)[:end].double()
                qq = s["q"][m, i, h * g:(h + 1) * g].double()
                sc = torch.cat([qq @ k0.T, qq @ k1.T], -1) * s["scale"]
                z = torch.logsumexp(sc, -1)
                w = torch.exp(sc - z[:, None])
                o[m, i, h * g:(h + 1) * g] = w[:, :P] @ v0 + w[:, P:] @ v1
                lse[m, i, h * g:(h + 1) * g] = z
    return o, lse


def _exact_extend(s):
    ps = s["ps"]
    table, free = s["table"].cpu().numpy().copy(), s["free"].cpu().numpy()
    lens, add = s["lens"].cpu().numpy().astype(np.int64), s["add"].cpu().numpy().astype(np.int64)
    used = int(s["used"])
    slots = np.full(s["slots"].numel(), -1, np.int32)
    pos = np.zeros((1, slots.size), np.int32)
    t = 0
    for m in range(len(lens)):
        for b in range(-(-lens[m] // ps), -(-(lens[m] + add[m]) // ps)):
            table[m, b] = free[used]
            used += 1
        i = np.arange(lens[m], lens[m] + add[m])
        slots[t:t + add[m]] = table[m, i // ps] * ps + i % ps
        pos[0, t:t + add[m]] = s["pos0"] + i
        t += add[m]
    return slots, pos, table, (lens + add).astype(np.int32), np.array([used], np.int32)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "extend":
        return _exact_extend(s)
    if case["op"] == "decode":
        return _exact_decode(s)
    r = _exact_norm(s)
    if case["op"] == "fwd":
        return r["q"], r["k"], s["v"].double()
    if case["op"] == "bwd":
        return r["q"], r["k"], s["dv"].double(), r["wq"], r["wk"]
    kp, vp = s["k_pool"].double(), s["v_pool"].double()
    for t, slot in enumerate(s["slots"].split(case["ps"])):  # a page's tokens together
        page, off = slot.long() // case["ps"], slot.long() % case["ps"]
        at = slice(t * case["ps"], t * case["ps"] + len(slot))
        kp.transpose(1, 2)[page, off] = r["k"][at]
        vp.transpose(1, 2)[page, off] = s["v"][at].double()
    return r["q"], kp, vp
