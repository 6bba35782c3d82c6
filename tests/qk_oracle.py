"""Plain 64-bit implementations of the query/key stage, page allocation and the decode
step (numpy, on the host), with the error bounds the GPU tests hold the kernels to."""
from __future__ import annotations

import numpy as np
import torch

D = 128
U32 = 2.0 ** -24   # half a step of fp32, relative
U16 = 2.0 ** -8    # half a step of bf16
SUB = 2.0 ** -134  # half a step of bf16 below its smallest normal number 2^-126: its
                   # values there are the multiples of 2^-133, so rounding to one is off by
                   # up to 2^-134 however small the value


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()


def bf16(x) -> torch.Tensor:
    return torch.from_numpy(np.asarray(x, np.float32)).to(torch.bfloat16)


def turn(y, positions, inv_freq, pair_axis, interleaved, back=False):
    """The rotation of y [T][H][128]; positions [axes][T], inv_freq [rot / 2]."""
    half = len(inv_freq)
    if half == 0:
        return y.copy()
    ax = np.zeros(half, int) if pair_axis is None else np.asarray(pair_axis)
    ang = np.asarray(positions, np.float64)[ax].T * np.asarray(inv_freq, np.float64)  # [T][half]
    c, s = np.cos(ang)[:, None], np.sin(ang)[:, None]
    if back:
        s = -s
    out = y.copy()
    if interleaved:
        ia, ib = np.arange(0, 2 * half, 2), np.arange(1, 2 * half, 2)
    else:
        ia, ib = np.arange(half), np.arange(half, 2 * half)
    a, b = y[..., ia], y[..., ib]
    out[..., ia] = a * c - b * s
    out[..., ib] = b * c + a * s
    return out


def pair_abs(y, half, interleaved):
    """|a| + |b| of each value's pair (the value itself behind the rotated ones)."""
    out = np.abs(y)
    if half == 0:
        return out
    if interleaved:
        s = np.abs(y[..., 0:2 * half:2]) + np.abs(y[..., 1:2 * half:2])
        out[..., 0:2 * half:2] = s
        out[..., 1:2 * half:2] = s
    else:
        s = np.abs(y[..., :half]) + np.abs(y[..., half:2 * half])
        out[..., :half] = s
        out[..., half:2 * half] = s
    return out


def norm(x, w, offset, eps):
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return x * r * (offset + w), r


def fwd(x, w, offset, eps, positions, inv_freq, pair_axis, interleaved, with_norm=True):
    """Returns (y, bound): bound is half a bf16 step of the result plus the fp32
    arithmetic's share of the pair it is made of (norm: about 8 roundings and rsqrt's 2
    steps; cos and sin: the angle to 2^-25 of a turn; two products and a sum)."""
    u = norm(x, w, offset, eps)[0] if with_norm else x
    y = turn(u, positions, inv_freq, pair_axis, interleaved)
    pa = pair_abs(u, len(inv_freq), interleaved)
    e = 32 * U32 * pa
    return y, U16 * (np.abs(y) + e) + e + SUB


def bwd(x, dy, w, offset, eps, positions, inv_freq, pair_axis, interleaved, with_norm=True):
    """Returns (dx, dx bound, dw, dw bound)."""
    g = turn(dy, positions, inv_freq, pair_axis, interleaved, back=True)
    ge = 16 * U32 * pair_abs(dy, len(inv_freq), interleaved)
    if not with_norm:
        return g, U16 * (np.abs(g) + ge) + ge + SUB, None, None
    _, r = norm(x, w, offset, eps)
    xh = x * r
    wt = offset + w
    h = g * wt
    mean = (h * xh).mean(-1, keepdims=True)
    dx = r * (h - xh * mean)
    # every term carries the relative error of its factors (about 32 roundings) and g's
    mag = np.abs(h) + np.abs(xh) * np.abs(h * xh).mean(-1, keepdims=True)
    gmag = ge * np.abs(wt) + np.abs(xh) * (ge * np.abs(wt * xh)).mean(-1, keepdims=True)
    e = r * (32 * U32 * mag + gmag)
    dw = (g * xh).sum((0, 1))
    # a lane adds one term per head and block of tokens it walks, then 16 lanes in turn
    T, H, _ = x.shape
    chain = H * (1 + T // 16) + 32
    dwe = U32 * chain * np.abs(g * xh).sum((0, 1)) + (ge * np.abs(xh)).sum((0, 1))
    return dx, U16 * (np.abs(dx) + e) + e + SUB, dw, dwe


def extend(table, lens, add, free, used, ps, pos0, axes, capacity):
    """Member by member; None when the call has to be refused."""
    table, lens = np.array(table), np.array(lens, np.int64)
    slots = np.full(capacity, -1, np.int32)
    pos = np.zeros((axes, capacity), np.int32)
    t = 0
    for m, n in enumerate(np.asarray(add, np.int64)):
        if n < 0 or (lens[m] < 0 and n > 0):
            return None
        if lens[m] < 0:
            continue
        if -(-(lens[m] + n) // ps) > table.shape[1] or t + n > capacity:
            return None
        for b in range(-(-lens[m] // ps), -(-(lens[m] + n) // ps)):
            if used >= len(free):
                return None
            table[m, b] = free[used]
            used += 1
        i = np.arange(lens[m], lens[m] + n)
        slots[t:t + n] = table[m, i // ps] * ps + i % ps
        pos[:, t:t + n] = pos0 + i
        lens[m] += n
        t += n
    return slots, pos, table, lens.astype(np.int32), used


def decode(q, k_prompt, v_prompt, k_resp, v_resp, lens, scale):
    """q [M][n][Hq][128]; k/v_prompt [P][Hkv][128]; k/v_resp: a list of [len][Hkv][128] per
    member.  Returns (o, o bound, lse, lse bound); members with lens < 0 are zero.

    Bounds: each weight enters the value product as bf16 (half a step of it) and o leaves
    as bf16; a score is a 128-term fp32 sum, off by at most 128 half steps of its terms'
    sizes, which changes a weight by as much relatively; the exponentials, row sums and
    merges add less than 2^-18."""
    M, n, hq, _ = q.shape
    hkv = k_prompt.shape[1]
    g = hq // hkv
    o, lse = np.zeros(q.shape), np.full(q.shape[:3], -np.inf)
    ob, lb = np.zeros(q.shape), np.zeros(q.shape[:3])
    for m in range(M):
        if lens[m] < 0:
            continue
        for i in range(n):
            end = max(0, lens[m] - n + 1 + i)
            for h in range(hkv):
                k = np.concatenate([k_prompt[:, h], k_resp[m][:end, h]])
                v = np.concatenate([v_prompt[:, h], v_resp[m][:end, h]])
                if len(k) == 0:
                    continue
                qq = q[m, i, h * g:(h + 1) * g]
                s = qq @ k.T * scale
                mag = np.abs(qq) @ np.abs(k).T * scale
                mx = s.max(-1, keepdims=True)
                p = np.exp(s - mx)
                den = p.sum(-1, keepdims=True)
                p /= den
                ds = (128 * U32 * (p * mag).sum(-1) + 2.0 ** -18)[:, None]
                a = p @ np.abs(v)
                sl = slice(h * g, (h + 1) * g)
                o[m, i, sl] = p @ v
                lse[m, i, sl] = (mx + np.log(den))[:, 0]
                e = (U16 + 2 * 128 * U32 * mag.max(-1, keepdims=True) + 2.0 ** -18) * a
                ob[m, i, sl] = e + U16 * (np.abs(o[m, i, sl]) + e)
                lb[m, i, sl] = ds[:, 0] + 2.0 ** -20 * np.abs(lse[m, i, sl])
    return o, ob, lse, lb
