"""GPU parity of ls_token_logp_fwd / _bwd against the 64-bit implementation, within bounds that
count the roundings (rollout_oracle)."""
import math

import numpy as np
import pytest
import torch

import rollout_oracle as ro
from response_replay_gb300 import binding as B
from response_replay_gb300 import torch_api as api

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().double().cpu().numpy()


def rows(dev, T, V, dt, pad=0, seed=0, kind="model", offset=0):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    if kind == "coarse":  # many equal logits
        z = torch.randint(-3, 4, (T, V + pad), generator=g, device=dev).to(F32)
    else:
        z = torch.randn(T, V + pad, generator=g, device=dev) * 2
        hot = torch.randint(0, V, (T, 6), generator=g, device=dev)
        z.scatter_(1, hot, torch.rand(T, 6, generator=g, device=dev) * 8 + 4)
    z = z.to(dt)
    if offset:  # rows that begin anywhere
        flat = torch.full((z.numel() + offset,), 9.0, dtype=dt, device=dev)
        flat[offset:] = z.flatten()
        z = flat[offset:].view(T, V + pad)
    if pad:
        z[:, V:] = float("nan")  # not to be read
    y = torch.randint(0, V, (T,), generator=g, device=dev).to(torch.int32)
    return z[:, :V], y, g


def fp32_range(x):
    """Values past fp32's largest (2 - 2^-23) 2^127 by half a step or more round to infinity
    there: the lowest value of a type over a temperature below one is such a number."""
    return np.where(np.abs(x) >= (2 - 2.0 ** -24) * 2.0 ** 127, np.copysign(np.inf, x), x)


def check_fwd(z, y, temp, top):
    logp, lse, ent, tl, ti = api.token_logp_fwd(z, y, temperature=temp, top=top)
    assert B.ls_last_device_error(0) == B.LS_OK
    zz = f64(z)
    lp, l64, h64, e_lse, e_h = ro.stat_bounds(zz, temp)
    r = np.arange(len(zz))
    want = fp32_range(lp[r, y.cpu().numpy()])
    assert (np.abs(f64(lse) - l64) <= e_lse).all(), np.abs(f64(lse) - l64).max()
    assert (np.abs(f64(ent) - h64) <= e_h).all(), (np.abs(f64(ent) - h64) / e_h).max()
    fin = np.isfinite(want)
    assert (f64(logp)[~fin] == want[~fin]).all()
    assert (np.abs(f64(logp)[fin] - want[fin]) <= e_lse[fin] + ro.U32 * np.abs(want[fin])).all()
    if top:
        ids = ro.top(zz, top)
        np.testing.assert_array_equal(ti.cpu().numpy(), ids)
        w = fp32_range(np.take_along_axis(lp, ids, 1))
        fin = np.isfinite(w)
        assert (f64(tl)[~fin] == w[~fin]).all()
        bound = np.broadcast_to(e_lse[:, None], w.shape)[fin] + ro.U32 * np.abs(w[fin])
        assert (np.abs(f64(tl)[fin] - w[fin]) <= bound).all()
    else:
        assert tl is None and ti is None
    return lse, ent, ti


# Vocabularies from one token over odd ones to several parts a row; few rows (cut into parts) and
# many; every part of a 32-byte group at a row's beginning and end; padded rows.
CASES = [
    (1, 1, BF, 0, 1.0, 1, 0), (3, 2, F32, 0, 1.0, 2, 0), (5, 7, BF, 0, 0.5, 7, 1), (2, 33, BF, 0, 1.0, 32, 3),
    (7, 1000, BF, 24, 1.0, 5, 0), (9, 1001, F32, 0, 1.4, 20, 5), (1, 151936, BF, 0, 1.0, 20, 0),
    (8, 151936, BF, 0, 1.0, 20, 0), (3, 151936, F32, 0, 0.7, 32, 2), (200, 32003, BF, 0, 1.0, 8, 0),
    (170, 50257, F32, 47, 0.6, 0, 0), (1, 400003, F32, 0, 1.0, 32, 1), (161, 250002, BF, 0, 1.0, 3, 7),
    (400, 513, BF, 0, 2.0, 1, 0), (31, 4096, F32, 0, 1.0, 0, 0), (160, 100001, F32, 3, 1.0, 32, 0),
    # many rows of a warp or a few each
    (2500, 1000, BF, 24, 1.0, 32, 0), (3001, 333, F32, 1, 0.6, 12, 0), (1900, 63, BF, 0, 1.0, 13, 5),
    (1000, 8001, BF, 0, 1.0, 20, 3), (2000, 20011, BF, 0, 1.4, 32, 0), (700, 20011, F32, 0, 1.0, 17, 1),
    (1830, 33007, BF, 0, 1.0, 0, 1), (2000, 5, F32, 0, 1.0, 5, 0), (500, 70001, BF, 0, 1.0, 5, 0),
]


@pytest.mark.parametrize("T,V,dt,pad,temp,top,offset", CASES)
def test_forward(cuda, T, V, dt, pad, temp, top, offset):
    z, y, _ = rows(cuda, T, V, dt, pad, seed=V + T, offset=offset)
    check_fwd(z, y, temp, top)


@pytest.mark.parametrize("T,V,dt", [(2, 151936, BF), (200, 20000, BF), (200, 20000, F32), (3, 40, F32)])
@pytest.mark.parametrize("top", [1, 17, 32])
def test_equal_logits(cuda, T, V, dt, top):
    """Ties go to the lowest id, however many there are; both zeros are one."""
    z, y, _ = rows(cuda, T, V, dt, seed=top, kind="coarse")
    z[0] = 0.0
    z[0, ::2] = -0.0
    z[1] = 1.5
    check_fwd(z, y, 1.0, top)


@pytest.mark.parametrize("T,V,dt,temp", [(300, 50257, F32, 0.7), (300, 50257, F32, 1.0), (200, 100003, BF, 1.4)])
def test_entropies_of_likely_tokens(cuda, T, V, dt, temp):
    """Likely tokens far above the logits that a thread meets first.  Their exponents are taken
    against a number at most 2^8 below (half a step of 8: 2^-22) and moved to the row's maximum
    (16: 2^-21); a weight is off by as much, relatively, and moves the entropy by its share of
    |log p + H|.  Root mean square over the rows, so the roundings' largest sizes bound it with
    room for the sums' own."""
    z, y, _ = rows(cuda, T, V, dt, seed=3)
    _, _, ent, _, _ = api.token_logp_fwd(z, y, temperature=temp)
    x = z.double() / temp
    lp = x - torch.logsumexp(x, -1, keepdim=True)
    p = lp.exp()
    h = -(p * lp).sum(-1)
    spread = (p * (lp + h[:, None]).abs()).sum(-1)
    rms = lambda t: float((t ** 2).mean().sqrt())
    assert rms(ent.double() - h) <= 2.0 ** -21 * rms(1 + spread)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("rise", [2.0, 5.0, 5.5, 6.0, 30.0])
def test_rows_in_steps(cuda, dt, rise):
    """Rows that rise by steps about as high as the reference of a sum may lie below a logit, with
    many equal logits a step, and small rises between."""
    V = 150000
    at = torch.arange(V, device=cuda) // 25000
    z = torch.stack([at * rise, at * rise + (torch.arange(V, device=cuda) // 7000) % 3 * 0.25,
                     torch.where(torch.arange(V, device=cuda) % 5 == 0, at * rise, at * rise - 9)])
    z = z.repeat(60, 1).to(dt)
    y = torch.arange(180, device=cuda, dtype=torch.int32)
    check_fwd(z, y, 1.0, 0)
    check_fwd(z[:3], y[:3], 1.0, 4)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("V", [9600, 96000])
@pytest.mark.parametrize("order", ["up", "down", "columns", "threads"])
def test_orders_of_a_row(cuda, dt, V, order):
    """Rows whose largest logits all lie with one thread, or come last, or rise all along."""
    x = torch.linspace(-20, 20, V, device=cuda)
    if order == "down":
        x = x.flip(0)
    elif order == "columns":  # the largest a stride apart
        x = x.view(V // 64, 64).T.reshape(-1)
    elif order == "threads":  # whole groups of the largest, one thread's groups apart
        x = torch.where((torch.arange(V, device=cuda) // (16 if dt is BF else 8)) % 512 < 3, x + 60, x)
    z = torch.stack([x] * 170).to(dt).contiguous()
    y = torch.arange(170, device=cuda).to(torch.int32)
    check_fwd(z, y, 1.0, 32)
    check_fwd(z[:1].clone(), y[:1].clone(), 1.0, 20)


@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("T,V", [(3, 30011), (190, 30011), (3, 150011), (190, 100011)])
def test_masked_vocabulary(cuda, dt, T, V):
    """Logits of -inf and of the type's lowest value have no probability, and the alternatives
    that are left over take them in the order of their ids."""
    z, y, g = rows(cuda, T, V, dt, seed=T)
    low = torch.finfo(dt).min
    z[0, 5:] = -math.inf          # five tokens left
    z[1, :-3] = low
    z[2, torch.randperm(V, generator=g, device=cuda)[:V - 40]] = -math.inf
    y[0], y[1] = 2, V - 1
    for temp in (1.0, 0.3):
        lse, ent, _ = check_fwd(z, y, temp, 32)
        d = api.token_logp_bwd(z, y, lse, ent, torch.ones(T, device=cuda), torch.ones(T, device=cuda),
                               temperature=temp)
        assert bool(torch.isfinite(d).all()) and bool((d[0, 5:] == 0).all())
    y[0] = 9                      # a token of no probability
    logp = api.token_logp_fwd(z, y)[0]
    assert float(logp[0]) == -math.inf
    z[0] = low                    # all equal
    _, lse, ent, _, ids = api.token_logp_fwd(z, y, top=4)
    assert abs(float(ent[0]) - math.log(V)) < 1e-4 and ids[0].tolist() == [0, 1, 2, 3]


@pytest.mark.parametrize("T,V", [(4, 5000), (200, 5000), (4, 50000), (200, 50000)])
def test_rows_that_are_no_numbers(cuda, T, V):
    z, y, _ = rows(cuda, T, V, F32, seed=2)
    z[0, 77] = math.nan
    z[1, 78] = math.inf
    z[2] = -math.inf
    ref = api.token_logp_fwd(z[3:].clone(), y[3:].clone(), top=9)
    out = api.token_logp_fwd(z, y, top=9)
    # The others are what they are without these.  The copy's rows begin at other parts of a
    # 64-byte group, so their sums are taken in another order: each result is within its bound of
    # the formula's, and the two within twice that of one another.
    _, _, _, e_lse, e_h = ro.stat_bounds(f64(z[3:]), 1.0)
    for k, (a, b) in enumerate(zip(out, ref)):
        e = (e_h if k == 2 else e_lse).reshape(-1, *[1] * (b.dim() - 1)) + ro.U32 * np.abs(f64(b))
        assert torch.equal(a[3:], b) if k == 4 else (np.abs(f64(a[3:]) - f64(b)) <= 2 * e).all()
    assert torch.isnan(out[0][:3]).all() and torch.isnan(out[2][:3]).all()
    ids = out[4][:3]
    assert bool(((ids >= -1) & (ids < V)).all())
    assert B.ls_last_device_error(0) == B.LS_OK


@pytest.mark.parametrize("T", [5, 300])
def test_padding_rows_and_bad_targets(cuda, T):
    z, y, g = rows(cuda, T, 3001, BF, seed=4)
    y[1], y[3] = -1, -1
    z[1] = math.nan
    logp, lse, ent, tl, ti = api.token_logp_fwd(z, y, top=3)
    assert B.ls_last_device_error(0) == B.LS_OK
    for t in (logp, lse, ent, tl):
        assert bool((t[[1, 3]] == 0).all())
    assert bool((ti[[1, 3]] == -1).all())
    d = torch.full_like(z, 7.0)
    gt = torch.randn(T, 3, generator=g, device=cuda)
    api.token_logp_bwd(z, y, lse, ent, torch.ones(T, device=cuda), torch.ones(T, device=cuda),
                       top_ids=ti, d_top=gt, dlogits=d)
    assert B.ls_last_device_error(0) == B.LS_OK
    assert bool((d[[1, 3]] == 0).all()) and bool(torch.isfinite(d).all())
    y[0] = 3001
    logp, lse, ent, _, _ = api.token_logp_fwd(z, y)
    assert B.ls_last_device_error(0) == B.LS_ERR_DEVICE_CHECK
    assert math.isnan(float(logp[0])) and math.isfinite(float(lse[0]))
    d = api.token_logp_bwd(z, y, lse, ent, torch.ones(T, device=cuda))
    assert B.ls_last_device_error(0) == B.LS_ERR_DEVICE_CHECK
    assert bool(torch.isnan(d[0]).all()) and bool(torch.isfinite(d[2]).all())


def check_bwd(z, y, temp, top, g, with_logp=True, with_ent=True, dlogits=None):
    T, V = z.shape
    dev = z.device
    out = api.token_logp_fwd(z, y, temperature=temp, top=top)
    lse, ent, ids = out[1], out[2], out[4]
    dl = torch.randn(T, generator=g, device=dev) if with_logp else None
    de = torch.randn(T, generator=g, device=dev) if with_ent else None
    dt_ = torch.randn(T, top, generator=g, device=dev) if top else None
    zz = f64(z)
    d = api.token_logp_bwd(z, y if with_logp else None, lse, ent, dl, de, temperature=temp,
                           top_ids=ids, d_top=dt_, dlogits=dlogits)
    assert B.ls_last_device_error(0) == B.LS_OK
    ref, err = ro.token_logp_bwd(zz, y.cpu().numpy(), f64(lse), f64(ent),
                                 None if dl is None else f64(dl), None if de is None else f64(de), temp,
                                 None if ids is None else ids.cpu().numpy(), None if dt_ is None else f64(dt_))
    half = ro.U16 if z.dtype is BF else ro.U32
    # half a step of the result, and of bf16's (2^-134) below its normal numbers
    bound = err + half * (np.abs(ref) + err) + 2.0 ** -134
    off = np.abs(f64(d) - ref)
    assert (off <= bound).all(), (off / bound).max()
    return d


@pytest.mark.parametrize("T,V,dt,pad,temp,top,offset", CASES)
def test_backward(cuda, T, V, dt, pad, temp, top, offset):
    z, y, g = rows(cuda, T, V, dt, pad, seed=V + T, offset=offset)
    check_bwd(z, y, temp, top, g)


@pytest.mark.parametrize("with_logp,with_ent,top", [(True, False, 0), (False, True, 0), (False, False, 4)])
def test_backward_of_some_outputs(cuda, with_logp, with_ent, top):
    z, y, g = rows(cuda, 40, 2003, F32, seed=1)
    check_bwd(z, y, 0.8, top, g, with_logp, with_ent)


def test_backward_of_one_token_twice(cuda):
    """The target among the alternatives, and an alternative given twice: all of them count."""
    T, V = 6, 999
    z, y, g = rows(cuda, T, V, F32, seed=1)
    _, lse, ent, _, ids = api.token_logp_fwd(z, y, top=5)
    ids[:, 3] = ids[:, 1]
    y = ids[:, 0].contiguous()
    dl, dt_ = torch.randn(T, generator=g, device=cuda), torch.randn(T, 5, generator=g, device=cuda)
    d = api.token_logp_bwd(z, y, lse, None, dl, top_ids=ids, d_top=dt_)
    ref, err = ro.token_logp_bwd(f64(z), y.cpu().numpy(), f64(lse), None, f64(dl), None, 1.0,
                                 ids.cpu().numpy(), f64(dt_))
    assert (np.abs(f64(d) - ref) <= err + ro.U32 * (np.abs(ref) + err)).all()


@pytest.mark.parametrize("dt,V,T", [(BF, 4099, 37), (F32, 70001, 2)])
def test_backward_in_place_and_into_strided_rows(cuda, dt, V, T):
    z, y, g = rows(cuda, T, V, dt, pad=5, seed=8)
    wide = torch.full((T, V + 11), 3.0, dtype=dt, device=cuda)
    state = g.get_state()
    a = check_bwd(z, y, 1.0, 3, g, dlogits=wide[:, :V])
    assert bool((wide[:, V:] == 3.0).all())
    g.set_state(state)
    ref = a.clone()
    b = check_bwd(z, y, 1.0, 3, g, dlogits=z)
    assert b.data_ptr() == z.data_ptr() and torch.equal(b, ref)


def test_gradient_against_differences(cuda):
    """The whole call, from the logits to an objective's value, in a few directions: central
    differences of the 64-bit objective against the gradient's products with them."""
    T, V, top, temp = 3, 211, 4, 0.9
    z, y, g = rows(cuda, T, V, F32, seed=3)
    out = api.token_logp_fwd(z, y, temperature=temp, top=top)
    w = [torch.randn(T, generator=g, device=cuda) for _ in range(2)]
    wt = torch.randn(T, top, generator=g, device=cuda)
    d = f64(api.token_logp_bwd(z, y, out[1], out[2], w[0], w[1], temperature=temp, top_ids=out[4], d_top=wt))
    ids, yy, zz = out[4].cpu().numpy(), y.cpu().numpy(), f64(z)

    def value(x):
        lp, _ = ro.log_probs(x, temp)
        return ((lp[np.arange(T), yy] * f64(w[0])).sum() + (ro.entropy(lp) * f64(w[1])).sum()
                + (np.take_along_axis(lp, ids, 1) * f64(wt)).sum())

    rng = np.random.default_rng(0)
    for _ in range(10):
        v = rng.standard_normal((T, V))
        eps = 1e-5
        num = (value(zz + eps * v) - value(zz - eps * v)) / (2 * eps)
        # differences: eps^2 of a third derivative (below 1e-8 here); the gradient: fp32
        assert abs(num - (d * v).sum()) <= 1e-5 * np.abs(d * v).sum() + 1e-7


def test_same_bits_on_streams_and_in_graphs(cuda):
    T, V = 8, 151936
    z, y, g = rows(cuda, T, V, BF, seed=6)
    ref = [t.clone() for t in api.token_logp_fwd(z, y, top=20)]
    de = torch.randn(T, generator=g, device=cuda)
    dref = api.token_logp_bwd(z, y, ref[1], ref[2], de, de).clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        out = api.token_logp_fwd(z, y, top=20, stream=side)
        with torch.cuda.stream(side):
            assert all(torch.equal(a, b) for a, b in zip(out, ref))
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = api.token_logp_fwd(z, y, top=20)
        d = api.token_logp_bwd(z, y, out[1], out[2], de, de)
    z2 = z.flip(0).contiguous()
    z.copy_(z2)
    y.copy_(y.flip(0).clone())
    de.copy_(de.flip(0).clone())
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b.flip(0)) for a, b in zip(out, ref))
    assert torch.equal(d, dref.flip(0))


def test_calls_on_several_streams_at_once(cuda):
    """Rows dealt out while the call runs, parts of a row with a second launch, and rows of a warp
    each, under way together: the bits of each are what they are alone."""
    sets = [rows(cuda, T, V, dt, seed=T)[:2] for T, V, dt in
            [(900, 151936, BF), (9, 151936, F32), (2500, 5001, BF), (700, 60001, F32)]]
    ref = [api.token_logp_fwd(z, y, top=7) for z, y in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    outs = [[] for _ in sets]
    for _ in range(10):
        for (z, y), st, o in zip(sets, streams, outs):
            with torch.cuda.stream(st):
                o.append(api.token_logp_fwd(z, y, top=7))
    torch.cuda.synchronize()
    assert B.ls_last_device_error(0) == B.LS_OK
    for o, r in zip(outs, ref):
        for each in o:
            assert all(torch.equal(a, b) for a, b in zip(each, r))


@pytest.mark.parametrize("T,V", [(15000, 151936), (62000, 40000)])
def test_long_buffers(cuda, T, V):
    """Rows past 2^32 bytes and 2^31 values of the buffer."""
    z = torch.empty(T, V, dtype=BF, device=cuda)
    z.normal_()
    y = torch.randint(0, V, (T,), device=cuda).to(torch.int32)
    logp, lse, ent, tl, ti = api.token_logp_fwd(z, y, top=2)
    at = torch.tensor([0, 7000, 14134, T - 1], device=cuda)
    few = api.token_logp_fwd(z[at].contiguous(), y[at].contiguous(), top=2)
    assert torch.equal(ti[at], few[4])
    for a, b in zip((logp, lse, ent, tl), few):
        assert torch.allclose(a[at], b, rtol=1e-5, atol=1e-5)
    last = z[at].clone()
    one = torch.ones(T, device=cuda)
    api.token_logp_bwd(z, y, lse, ent, one, one, dlogits=z)
    ref = api.token_logp_bwd(last, y[at].contiguous(), lse[at].contiguous(), ent[at].contiguous(),
                             one[at].contiguous(), one[at].contiguous())
    assert torch.equal(z[at], ref)


def test_no_rows(cuda):
    z = torch.empty(0, 100, device=cuda)
    y = torch.empty(0, dtype=torch.int32, device=cuda)
    out = api.token_logp_fwd(z, y, top=3)
    assert out[0].shape == (0,) and out[3].shape == (0, 3)
    assert api.token_logp_bwd(z, y, out[1], out[2], out[0]).shape == (0, 100)
