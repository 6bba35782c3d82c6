"""GPU parity of the token statistics at the ends of their range: temperatures from 1e-6 to 1e6, rows
whose logits are all masks, rows without a finite logit, and gradients there."""
import math

import numpy as np
import pytest
import torch

import rollout_oracle as ro
from response_replay_gb300 import binding as B
from response_replay_gb300 import torch_api as api

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def stats(z, temp):
    """(log probabilities, lse, entropy, bound of what is counted from the row's maximum, bound of
    the entropy) in 64 bits.  Everything but lse is a difference of logits, so it is taken as one,
    whatever the logits' size; the bounds are rollout_oracle.stat_bounds' without lse's own
    rounding."""
    z = z.double()
    m = z.amax(-1, keepdim=True)
    d = (z - m) / temp
    log_sum = torch.log(torch.exp(d).sum(-1, keepdim=True))
    lp = d - log_sum
    p = torch.exp(lp)
    u = torch.where(p > 0, d, 0).abs()
    a1, a2 = (p * u).sum(-1), (p * u * u).sum(-1)
    V = z.shape[1]
    chain = 1.5 * max(V / 512, min(V / 64, 512)) + 80
    es = 2.0 ** -21 + chain * ro.U32 + 3 * ro.U32 * a1
    h = -torch.where(p > 0, p * lp, 0).sum(-1)
    e_h = es + 2.0 ** -21 + a1 * (2.0 ** -21 + es + (chain + 8) * ro.U32) + 3 * ro.U32 * a2 + 4 * ro.U32 * h
    return lp, (m / temp + log_sum)[:, 0], h, es + 2.0 ** -21, e_h


def check(z, y, temp, top):
    logp, lse, ent, tl, ti = api.token_logp_fwd(z, y, temperature=temp, top=top)
    assert B.ls_last_device_error(0) == B.LS_OK
    lp, l64, h64, e, e_h = stats(z, float(np.float32(temp)))
    want = lp.gather(1, y.long()[:, None])[:, 0]
    assert bool(((ent.double() - h64).abs() <= e_h).all()), float(((ent.double() - h64).abs() / e_h).max())
    off = (logp.double() - want).abs()
    assert bool((off <= e + ro.U32 * want.abs()).all()), float(off.max())
    # past fp32's largest by half a step: infinity
    l64 = torch.where(l64.abs() >= (2 - 2.0 ** -24) * 2.0 ** 127, torch.sign(l64) * math.inf, l64)
    off = (lse.double() - l64).abs()
    assert bool(((lse.double() == l64) | (off <= e + ro.U32 * l64.abs())).all()), float(off.max())
    if top:
        ids = z.double().sort(dim=-1, descending=True, stable=True).indices[:, :top]
        assert torch.equal(ti.long(), ids)
        w = lp.gather(1, ids)
        assert bool(((tl.double() - w).abs() <= e[:, None] + ro.U32 * w.abs()).all())
    return lse, ent


# a warp or a few a row, streamed, cut into parts; rows that begin inside a vector and end there
SHAPES = [(300, 1003, 20), (300, 1003, 0), (200, 90001, 0), (200, 90001, 5), (3, 150011, 20), (1, 20011, 1)]


def near_ties(dev, T, V, dt, level, steps, seed, offset):
    """Rows within a few of the type's steps of one level."""
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    step = abs(level) * torch.finfo(dt).eps
    z = level + step * torch.randint(0, steps, (T, V), generator=g, device=dev, dtype=torch.float64)
    flat = torch.zeros(T * V + offset, dtype=dt, device=dev)
    flat[offset:] = z.flatten().to(dt)
    y = torch.randint(0, V, (T,), generator=g, device=dev).to(torch.int32)
    return flat[offset:].view(T, V), y


@pytest.mark.parametrize("T,V,top", SHAPES)
@pytest.mark.parametrize("level,temp", [
    (20.0, 2.0 ** -19), (-20.0, 2.0 ** -19), (31.0, 1e-6), (30.0, 1e-3), (5000.0, 2.0 ** -10), (20.0, 1e6), (3e8, 1e6)])
def test_temperatures(cuda, T, V, top, level, temp):
    """Logits a few steps of fp32 apart, which a low temperature takes to distances of a few."""
    z, y = near_ties(cuda, T, V, F32, level, 9, V, 3)
    check(z, y, temp, top)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,V,top", SHAPES)
def test_broad_rows_at_the_ends(cuda, dt, T, V, top):
    """A model's logits at the lowest temperature (a few tokens at most are left) and at the highest
    (all are alike)."""
    g = torch.Generator(device=cuda)
    g.manual_seed(V)
    z = (torch.randn(T, V, generator=g, device=cuda) * 4).to(dt)
    z[0, 5:9] = z[0].max() + 1  # ties
    y = z.argmax(-1).to(torch.int32)
    for temp in (1e-6, 2.0 ** -14, 1e6):
        check(z, y, temp, top)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,V,top", SHAPES)
@pytest.mark.parametrize("level", [-1e4, -1e9, -1e10, -1e20, -1e29, -1e30, -3e38, 1e12])
def test_rows_of_masks(cuda, dt, T, V, top, level):
    """Every logit at a mask's value, or at one of three values a step apart near it: as probable as
    their distances say, whatever the type's step is there."""
    z, y = near_ties(cuda, T, V, dt, level, 1, 1, 5)
    check(z, y, 1.0, top)
    check(z, y, 0.37, top)
    step = abs(float(z[0, 0])) * torch.finfo(dt).eps
    z, y = near_ties(cuda, T, V, dt, float(z[0, 0]), 3, 1, 5)
    check(z, z.argmax(-1).to(torch.int32), min(max(step, 1e-6), 1e6), top)
    # some rows of masks among others
    z[1:] = torch.randn(T - 1, V, device=cuda).to(dt)
    check(z, z.argmax(-1).to(torch.int32), 1.0, top)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,V,top", [(300, 1003, 9), (200, 90001, 5), (200, 90001, 0), (3, 150011, 9)])
def test_rows_without_a_finite_logit(cuda, dt, T, V, top):
    """lse of a row of -inf is -inf, its other numbers are none; of one with NaN or +inf all are none.
    Their gradients are none either."""
    z = torch.randn(T, V, device=cuda).to(dt)
    z[0, 77], z[1, 78], z[2] = math.nan, math.inf, -math.inf
    y = torch.randint(0, V, (T,), device=cuda).to(torch.int32)
    logp, lse, ent, tl, ti = api.token_logp_fwd(z, y, top=top)
    assert B.ls_last_device_error(0) == B.LS_OK
    assert bool(torch.isnan(lse[:2]).all()) and float(lse[2]) == -math.inf
    assert bool(torch.isnan(logp[:3]).all()) and bool(torch.isnan(ent[:3]).all())
    if top:
        assert bool(torch.isnan(tl[:3]).all())
        assert bool(((ti >= -1) & (ti < V)).all())
    one = torch.ones(T, device=cuda)
    for de in (None, one):
        d = api.token_logp_bwd(z, y, lse, ent, one, de)
        assert B.ls_last_device_error(0) == B.LS_OK
        assert bool(torch.isnan(d[2]).all()) and bool(torch.isnan(d[:2]).all(-1).all())
        assert bool(torch.isfinite(d[3:]).all())


@pytest.mark.parametrize("dt", [BF, F32])
def test_gradients_of_rows_at_the_lowest_value(cuda, dt):
    """lse, in fp32, is the logit itself there: the formula gives every token a probability of 1."""
    T, V = 4, 5003
    z = torch.full((T, V), torch.finfo(dt).min, dtype=dt, device=cuda)
    y = torch.arange(T, dtype=torch.int32, device=cuda)
    _, lse, _, _, _ = api.token_logp_fwd(z, y)
    g = torch.tensor([1.0, -2.0, 0.5, 0.0], device=cuda)
    d = api.token_logp_bwd(z, y, lse, None, g)
    want = -g[:, None].expand(T, V).clone()
    want[torch.arange(T), y.long()] += g
    assert torch.equal(d.float(), want)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("temp", [1e-3, 2.0 ** -7, 100.0, 1e6])
@pytest.mark.parametrize("level", [20.0, -30.0])
def test_gradients_at_low_and_high_temperatures(cuda, dt, temp, level):
    """Against the formula with lse in 64 bits: off by what the header says besides the roundings that
    rollout_oracle counts."""
    T, V = 40, 3001
    z, y = near_ties(cuda, T, V, dt, level, 9, 4, 1)
    g = torch.randn(T, device=cuda)
    _, lse, _, _, _ = api.token_logp_fwd(z, y, temperature=temp)
    d = api.token_logp_bwd(z, y, lse, None, g, temperature=temp)
    assert B.ls_last_device_error(0) == B.LS_OK
    tau = float(np.float32(temp))
    lp, l64 = stats(z, tau)[:2]
    p, gg = lp.exp(), g.double()[:, None]
    want = -p * gg
    want.scatter_add_(1, y.long()[:, None], gg)
    # lse: the forward's own error (within 2^-20: a chain of V / 32 and less) and its rounding
    rel = torch.expm1(ro.U32 * l64.abs() + 2.0 ** -19)[:, None]
    # the exponent and, at the logits' size, 1 / tau's rounding
    rel = rel + 2.0 ** -21 + ro.U32 * (44 + 4 * lp.abs() + 4 * z.double().abs() / tau)
    err = (p * gg.abs() * rel).scatter_add_(1, y.long()[:, None], 40 * ro.U32 * gg.abs())
    # exponentials below 2^-126 are zero: p is off by as much, the product by |g| of that
    err = err + ro.TINY * gg.abs()
    half = ro.U16 if dt is BF else ro.U32
    off = (d.double() * tau - want).abs()
    assert bool((off <= err + half * (want.abs() + err)).all()), float(off.max())


@pytest.mark.parametrize("temp", [1e-6, 9e-4])
def test_no_gradient_where_lse_says_nothing(cuda, temp):
    z, y = near_ties(cuda, 3, 100, F32, 20.0, 9, 4, 0)
    _, lse, _, _, _ = api.token_logp_fwd(z, y, temperature=temp)
    with pytest.raises(B.LongstrawError) as e:
        api.token_logp_bwd(z, y, lse, None, torch.ones(3, device=cuda), temperature=temp)
    assert e.value.status == B.LS_ERR_UNSUPPORTED
