"""The stage's weight gradients within a bound of the walk that sums them, close enough to see
any one row that is lost or taken twice; and the angles, which they show in 32 bits."""
import math

import numpy as np
import pytest
import torch

import qk_oracle as qo
from response_replay_gb300 import torch_api as api
from test_gpu_qk_norm_rope import EPS, Stage, gen, ok

pytestmark = pytest.mark.gpu


def additions(T, hq, hkv, with_v, sms):
    """Most additions that a term goes through.  The rows of all pairs of tokens are cut evenly
    over the warps of two blocks of eight an SM: a lane adds its warp's rows of one kind of a
    token, then adds those sums up as often as the kind or the token changes; then a block's 16
    half-warps; then 128 chains of blocks, four of which are added in two steps, and 32 in five."""
    rows = hq + (2 if with_v else 1) * hkv
    total = (T + 1) // 2 * rows
    blocks = min(-(-total // 8), 2 * sms)
    mine = -(-total // min(total, 8 * blocks))
    runs = 2 + 2 * -(-mine // rows) + 1
    return mine + runs + 16 + -(-blocks // 128) + 2 + 5


def reference(x, dy, rotary, T, hq, hkv, with_v, sms):
    """(dw, bound, terms): the 64-bit sum, and the sum of the terms' sizes times a term's own
    error and its additions'.  A term is g xh: g is off by 8 half steps of its pair's sizes (the
    angle's 2^-26 of a turn is 2^-23.3 in radians, cos and sin 2 steps each, two products and
    a sum), xh by 8 of its own (16 squares of a lane in a chain of 8, four shuffles, the mean,
    rsqrt's 2 steps, halved by the root, and the product)."""
    g = qo.turn(dy, *rotary, back=True)
    ge = 8 * qo.U32 * qo.pair_abs(dy, len(rotary[1]), rotary[3])
    xh = x / np.sqrt((x * x).mean(-1, keepdims=True) + EPS)
    terms = g * xh
    size = np.abs(terms).sum((0, 1))
    n = additions(T, hq, hkv, with_v, sms) + 12
    return terms.sum((0, 1)), n * qo.U32 * size + (ge * np.abs(xh)).sum((0, 1)), terms


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,hq,hkv,rot,axes,inter,with_v", [
    (10007, 2, 2, 48, 3, False, True),
    (5000, 3, 1, 128, 1, False, False),
    (20011, 12, 2, 64, 3, False, True),
    (4096, 24, 4, 128, 1, True, True),
    (301, 40, 8, 0, 1, False, True),
    (1, 5, 1, 32, 1, False, True),
])
def test_no_row_is_lost(cuda, T, hq, hkv, rot, axes, inter, with_v, dtype):
    s = Stage(cuda, T, hq, hkv, rot, axes, inter, seed=5 * T + hq)
    dy = [torch.randn(T, h, 128, generator=gen(T, cuda), device=cuda).to(dtype) for h in (hq, hkv, hkv)]
    out = api.qk_norm_rope_bwd(s.q, s.k, s.pos, s.rot, dy[0], dy[1], dy[2] if with_v else None, wq=s.wq,
                               wk=s.wk, eps=EPS)
    ok()
    sms = torch.cuda.get_device_properties(cuda).multi_processor_count
    for i, x in enumerate((s.q, s.k)):
        dw, bound, terms = reference(qo.f64(x), qo.f64(dy[i]), s.rotary(), T, hq, hkv, with_v, sms)
        # a row moves some weight by twice its bound and more: every row of up to 100,000 of
        # them (the bound grows with their number), nine in ten of 240,000
        seen = float(((np.abs(terms) / bound).max(-1) > 2).mean())
        assert seen == 1 or (terms.shape[0] * terms.shape[1] > 200000 and seen > 0.9), seen
        err = np.abs(qo.f64(out[3 + i]) - dw) / bound
        assert err.max() <= 1, (i, err.max())


@pytest.mark.parametrize("inter", [False, True])
def test_the_angle_in_32_bits(cuda, inter):
    """One token of one head, all ones, whose gradient is one in the first value of every pair:
    its weight gradient is (cos, -sin).  The angle is off by the fp32 rounding of its part of a
    turn, 2^-26, and 2^-54 a position; cosine and sine by 2 half steps each, the products, the
    sum and xh by another three."""
    half = 64
    freq = torch.tensor([1e7 ** (-j / half) for j in range(half)], dtype=torch.float64, device=cuda)
    rot = api.Rotary(freq, interleaved=inter)
    x = torch.ones(1, 1, 128, dtype=torch.bfloat16, device=cuda)
    first = np.arange(0, 128, 2) if inter else np.arange(half)
    second = first + (1 if inter else half)
    dy = torch.zeros(1, 1, 128, device=cuda)
    dy[0, 0, first] = 1.0
    w = torch.ones(128, device=cuda)
    for p in [0, 1, -1, 1000, 131071, 2097152, 4194304, *np.random.default_rng(1).integers(0, 4194304, 40)]:
        pos = torch.tensor([int(p)], dtype=torch.int32, device=cuda)
        dw = qo.f64(api.qk_norm_rope_bwd(x, x, pos, rot, dy, dy, wq=w, wk=w, eps=2e-38)[3])
        turns = [math.fmod(int(p) * f, 2 * math.pi) for f in freq.tolist()]
        # p f of a 64-bit product is off by 2^-53 of its size
        bound = 2 * math.pi * (2.0 ** -26 + abs(int(p)) * 2.0 ** -54) + abs(int(p)) * 2.0 ** -53 + 5 * qo.U32
        assert np.abs(dw[first] - np.cos(turns)).max() <= bound, p
        assert np.abs(dw[second] + np.sin(turns)).max() <= bound, p
    ok()
