"""GPU parity of the query/key stage (ls_qk_norm_rope_fwd / _append / _bwd) against the
64-bit implementation, within bounds that count the roundings (qk_oracle)."""
import numpy as np
import pytest
import torch

import qk_oracle as qo
from response_replay_gb300 import binding as B
from response_replay_gb300 import torch_api as api

pytestmark = pytest.mark.gpu
EPS = 1e-6


def gen(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


class Stage:
    """Inputs of one call: q, k, v as slices of a packed projection."""

    def __init__(self, dev, T, hq, hkv, rot, axes=1, interleaved=False, offset=0.0, seed=0,
                 w_dtype=torch.float32, pad=0, base=1e7, pos_max=4194304):
        g = gen(seed, dev)
        n = hq + 2 * hkv
        self.buf = torch.randn(T, n * 128 + pad, generator=g, device=dev)
        self.buf *= torch.rand(T, 1, generator=g, device=dev) * 4 + 0.01
        self.buf = self.buf.to(torch.bfloat16)
        x = self.buf[:, :n * 128]
        self.q = x[:, :hq * 128].unflatten(1, (hq, 128))
        self.k = x[:, hq * 128:(hq + hkv) * 128].unflatten(1, (hkv, 128))
        self.v = x[:, (hq + hkv) * 128:].unflatten(1, (hkv, 128))
        self.wq = (torch.rand(128, generator=g, device=dev) + 0.5 - offset).to(w_dtype)
        self.wk = (torch.rand(128, generator=g, device=dev) + 0.5 - offset).to(w_dtype)
        self.pos = torch.randint(-5, pos_max, (axes, T), generator=g, device=dev).to(torch.int32)
        self.freq = torch.tensor([base ** (-2.0 * j / max(rot, 1)) for j in range(rot // 2)],
                                 dtype=torch.float64, device=dev)
        self.axis = None
        if axes > 1:
            self.axis = torch.randint(0, axes, (rot // 2,), generator=g, device=dev).to(torch.int32)
        self.rot = (api.Rotary(self.freq, pair_axis=self.axis, axes=axes, interleaved=interleaved)
                    if rot else None)
        self.inter, self.offset, self.T, self.hq, self.hkv = interleaved, offset, T, hq, hkv

    def rotary(self):
        return (self.pos.cpu().numpy(), self.freq.cpu().numpy(),
                None if self.axis is None else self.axis.cpu().numpy(), self.inter)

    def ref(self, x, w, norm=True):
        return qo.fwd(qo.f64(x), qo.f64(w), self.offset, EPS, *self.rotary(), with_norm=norm)


def close(got, ref, bound, what=""):
    got = qo.f64(got)
    bad = ~(np.abs(got - ref) <= bound)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(),
                           float(np.nanmax(np.abs(got - ref) / np.maximum(bound, 1e-300))))


def ok():
    assert B.ls_last_device_error(0) == B.LS_OK


# One token to several blocks of 16; one and many heads (more rows than a round of a block);
# every rotated width class, both pair layouts, several axes, both weight types.
SHAPES = [
    (1, 1, 1, 128, 1, False, 0.0, torch.float32),
    (1, 24, 4, 64, 1, False, 1.0, torch.bfloat16),
    (7, 8, 2, 128, 3, True, 0.0, torch.float32),
    (33, 5, 5, 32, 2, False, 0.0, torch.bfloat16),
    (700, 6, 1, 96, 4, True, 1.0, torch.float32),
    (1300, 24, 4, 16, 1, True, 0.0, torch.float32),
    (5000, 3, 1, 128, 1, False, 0.0, torch.float32),
    (10007, 2, 2, 48, 3, False, 1.0, torch.bfloat16),
    (300, 40, 8, 0, 1, False, 0.0, torch.float32),
]


@pytest.mark.parametrize("T,hq,hkv,rot,axes,inter,offset,wd", SHAPES)
def test_forward(cuda, T, hq, hkv, rot, axes, inter, offset, wd):
    s = Stage(cuda, T, hq, hkv, rot, axes, inter, offset, T + hq, wd, pad=8)
    q, k, v = api.qk_norm_rope_fwd(s.q, s.k, s.v, s.pos, s.rot, s.wq, s.wk, eps=EPS,
                                   weight_offset=offset)
    ok()
    close(q, *s.ref(s.q, s.wq), "q")
    close(k, *s.ref(s.k, s.wk), "k")
    assert torch.equal(v, s.v) and v.is_contiguous()


@pytest.mark.parametrize("T,hq,hkv,rot,axes,inter,offset,wd", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_backward(cuda, T, hq, hkv, rot, axes, inter, offset, wd, dtype):
    s = Stage(cuda, T, hq, hkv, rot, axes, inter, offset, 3 * T + hq, wd)
    g = gen(T, cuda)
    dy = [torch.randn(T, h, 128, generator=g, device=cuda).to(dtype) for h in (hq, hkv, hkv)]
    out = api.qk_norm_rope_bwd(s.q, s.k, s.pos, s.rot, *dy, wq=s.wq, wk=s.wk, eps=EPS,
                               weight_offset=offset)
    ok()
    for i, (x, w) in enumerate(((s.q, s.wq), (s.k, s.wk))):
        dx, dxb, dw, dwb = qo.bwd(qo.f64(x), qo.f64(dy[i]), qo.f64(w), offset, EPS, *s.rotary())
        close(out[i], dx, dxb, f"dx {i}")
        close(out[3 + i], dw, dwb, f"dw {i}")
    assert torch.equal(out[2], dy[2].to(torch.bfloat16))


def test_rotation_alone_norm_alone_and_no_weights(cuda):
    s = Stage(cuda, 50, 6, 2, 64, 2, seed=5)
    q, k, _ = api.qk_norm_rope_fwd(s.q, s.k, None, s.pos, s.rot, norm=False)
    close(q, *s.ref(s.q, s.wq, norm=False))
    close(k, *s.ref(s.k, s.wk, norm=False))
    dy = torch.randn(50, 6, 128, device=cuda), torch.randn(50, 2, 128, device=cuda)
    out = api.qk_norm_rope_bwd(s.q, s.k, s.pos, s.rot, *dy, norm=False)
    dx, dxb, _, _ = qo.bwd(qo.f64(s.q), qo.f64(dy[0]), None, 0, EPS, *s.rotary(), with_norm=False)
    close(out[0], dx, dxb)
    assert out[2:] == (None, None, None)
    one = torch.ones(128, device=cuda)
    q, k, _ = api.qk_norm_rope_fwd(s.q, s.k, None, None, None, eps=EPS)
    ref = qo.fwd(qo.f64(s.q), qo.f64(one), 0.0, EPS, s.pos.cpu().numpy(), np.zeros(0), None, False)
    close(q, *ref)
    # without weights the norm's scale is one whatever the offset
    q2, _, _ = api.qk_norm_rope_fwd(s.q, s.k, None, None, None, eps=EPS, weight_offset=1.0)
    assert torch.equal(q, q2)
    ok()


def test_far_positions(cuda):
    """Angles of positions up to the int32 range, the fastest pair among them."""
    s = Stage(cuda, 64, 2, 1, 128, seed=9)
    p = torch.tensor([2 ** 31 - 1, -2 ** 31, 4456448, 2 ** 24 + 1, 0, 1, -1, 10 ** 9], device=cuda)
    s.pos = p.repeat(8).to(torch.int32)[None].contiguous()
    q, k, _ = api.qk_norm_rope_fwd(s.q, s.k, None, s.pos, s.rot, s.wq, s.wk, eps=EPS)
    y, bound = s.ref(s.q, s.wq)
    # at 2^31 the fraction's 2^-54 of a turn has grown to 2^-23: 2^-20 in radians
    u = qo.norm(qo.f64(s.q), qo.f64(s.wq), 0.0, EPS)[0]
    close(q, y, bound + 2.0 ** -20 * qo.pair_abs(u, 64, False))
    ok()


def test_in_place_strided_outputs_and_neighbours_untouched(cuda):
    s = Stage(cuda, 37, 4, 2, 128, seed=2, pad=16)
    before = s.buf.clone()
    q, k, v = api.qk_norm_rope_fwd(s.q, s.k, s.v, s.pos, s.rot, s.wq, s.wk, eps=EPS)
    api.qk_norm_rope_fwd(s.q, s.k, None, s.pos, s.rot, s.wq, s.wk, eps=EPS, q_out=s.q, k_out=s.k)
    assert torch.equal(s.q, q) and torch.equal(s.k, k)
    assert torch.equal(s.v, v) and torch.equal(s.buf[:, 8 * 128:], before[:, 8 * 128:])
    # head-major output: [H][T][128] seen as [T][H][128]
    qh = torch.full((4, 37, 128), float("nan"), dtype=torch.bfloat16, device=cuda).transpose(0, 1)
    s.buf.copy_(before)
    api.qk_norm_rope_fwd(s.q, s.k, None, s.pos, s.rot, s.wq, s.wk, eps=EPS, q_out=qh)
    assert torch.equal(qh, q)
    # the gradient straight into the packed projection's gradient
    dy = [torch.randn(37, h, 128, device=cuda) for h in (4, 2, 2)]
    dense = api.qk_norm_rope_bwd(s.q, s.k, s.pos, s.rot, *dy, wq=s.wq, wk=s.wk, eps=EPS)
    d = torch.full_like(s.buf, 7.0)
    args = dict(dx_q=d[:, :512].unflatten(1, (4, 128)), dx_k=d[:, 512:768].unflatten(1, (2, 128)),
                dx_v=d[:, 768:1024].unflatten(1, (2, 128)))
    api.qk_norm_rope_bwd(s.q, s.k, s.pos, s.rot, *dy, wq=s.wq, wk=s.wk, eps=EPS, **args)
    assert torch.equal(d[:, :1024], torch.cat([t.flatten(1) for t in dense[:3]], 1))
    assert bool((d[:, 1024:] == 7.0).all())
    # and over the inputs themselves
    api.qk_norm_rope_bwd(s.q, s.k, s.pos, s.rot, *dy, wq=s.wq, wk=s.wk, eps=EPS, dx_q=s.q, dx_k=s.k)
    assert torch.equal(s.q, dense[0]) and torch.equal(s.k, dense[1])
    ok()


def test_weight_gradients_accumulate_and_single(cuda):
    s = Stage(cuda, 200, 6, 2, 64, seed=4)
    dy = [torch.randn(200, h, 128, device=cuda) for h in (6, 2)]
    a = api.qk_norm_rope_bwd(s.q, s.k, s.pos, s.rot, *dy, wq=s.wq, wk=s.wk, eps=EPS)
    again = api.qk_norm_rope_bwd(s.q, s.k, s.pos, s.rot, *dy, wq=s.wq, wk=s.wk, eps=EPS)
    for x, y in zip(a[:2] + a[3:], again[:2] + again[3:]):
        assert torch.equal(x, y)  # the order of every sum is fixed
    dwq, dwk = a[3].clone(), a[4].clone()
    api.qk_norm_rope_bwd(s.q, s.k, s.pos, s.rot, *dy, wq=s.wq, wk=s.wk, eps=EPS, dwq=dwq, dwk=dwk,
                         accumulate=True)
    assert (dwq - 2 * a[3]).abs().max() <= 2 * qo.U32 * 2 * a[3].abs().max()
    assert (dwk - 2 * a[4]).abs().max() <= 2 * qo.U32 * 2 * a[4].abs().max()
    # no tokens: nothing but zero weight gradients
    e = api.qk_norm_rope_bwd(s.q[:0], s.k[:0], s.pos[:, :0].contiguous(), s.rot, dy[0][:0], dy[1][:0],
                             wq=s.wq, wk=s.wk)
    assert not e[3].any() and not e[4].any()
    q, k, _ = api.qk_norm_rope_fwd(s.q[:0], s.k[:0], None, s.pos[:, :0].contiguous(), s.rot, s.wq,
                                   s.wk)
    assert q.shape == (0, 6, 128)
    ok()


def test_rows_at_the_ends_of_the_range(cuda):
    """Zero rows, rows whose squares pass fp32, subnormal rows, and non-finite rows, which
    stay in their own."""
    s = Stage(cuda, 16, 2, 1, 64, seed=8)
    s.buf[1] = 0
    s.buf[2] *= 1e30
    s.buf[3] = 3e38
    s.buf[4] = 1e-40
    q, k, _ = api.qk_norm_rope_fwd(s.q, s.k, None, s.pos, s.rot, s.wq, s.wk, eps=EPS)
    close(q, *s.ref(s.q, s.wq))
    close(k, *s.ref(s.k, s.wk))
    dy = [torch.randn(16, h, 128, device=cuda) for h in (2, 1)]
    out = api.qk_norm_rope_bwd(s.q, s.k, s.pos, s.rot, *dy, wq=s.wq, wk=s.wk, eps=EPS)
    dx, dxb, dw, dwb = qo.bwd(qo.f64(s.q), qo.f64(dy[0]), qo.f64(s.wq), 0.0, EPS, *s.rotary())
    close(out[0], dx, dxb)
    close(out[3], dw, dwb)
    s.q[5, 0, 3] = float("inf")
    s.q[6, 1, 100] = float("nan")
    s.k[7, 0, 127] = float("-inf")
    q2, k2, _ = api.qk_norm_rope_fwd(s.q, s.k, None, s.pos, s.rot, s.wq, s.wk, eps=EPS)
    keep_q = torch.ones(16, 2, dtype=torch.bool, device=cuda)
    keep_q[5, 0] = keep_q[6, 1] = False
    assert torch.equal(q[keep_q], q2[keep_q])
    assert not torch.isfinite(q2[5, 0, 3]) and torch.isnan(q2[6, 1]).all()
    assert torch.equal(k[:7], k2[:7]) and torch.equal(k[8:], k2[8:])
    # the rotation alone keeps a non-finite value within its pair
    s.q[5, 0, 70] = float("inf")
    q3, _, _ = api.qk_norm_rope_fwd(s.q, s.k, None, s.pos, s.rot, norm=False)
    bad = ~torch.isfinite(q3[5, 0])
    assert bad.nonzero().flatten().tolist() == [3, 35, 70]
    ok()


@pytest.mark.parametrize("T,ps", [(1, 16), (8, 64), (333, 32), (5000, 256)])
def test_append(cuda, T, ps):
    hq, hkv = 6, 2
    s = Stage(cuda, T, hq, hkv, 64, seed=T)
    pages = -(-T // ps) + 3
    g = gen(T + 1, cuda)
    slots = torch.randperm(pages * ps, generator=g, device=cuda)[:T].to(torch.int32)
    if T > 4:
        slots[3] = -1
    pool = api.PagePool.empty(pages, hkv, ps, cuda)
    pool.k_pool.fill_(3.0)
    pool.v_pool.fill_(4.0)
    q_out = torch.full((T, hq, 128), 9.0, dtype=torch.bfloat16, device=cuda)
    api.qk_norm_rope_append(pool, s.q, s.k, s.v, slots, s.pos, s.rot, s.wq, s.wk, eps=EPS,
                            q_out=q_out)
    ok()
    q, k, v = api.qk_norm_rope_fwd(s.q, s.k, s.v, s.pos, s.rot, s.wq, s.wk, eps=EPS)
    kp, vp = torch.full_like(pool.k_pool, 3.0), torch.full_like(pool.v_pool, 4.0)
    live = slots >= 0
    page, off = slots[live].long() // ps, slots[live].long() % ps
    kp[page, :, off], vp[page, :, off] = k[live], v[live]
    assert torch.equal(kp, pool.k_pool) and torch.equal(vp, pool.v_pool)
    assert torch.equal(q_out[live], q[live])
    assert bool((q_out[~live] == 9.0).all())


def test_append_to_a_prompt_cache_is_the_capture(cuda):
    """Chunks of a prompt appended by slot give the pages that capture writes from the
    forward's output."""
    P, ps, hkv, n = 300, 64, 2, 5
    table = torch.tensor([4, 1, 6, 0, 2], dtype=torch.int32, device=cuda)
    a = api.PagedKVCache(7, table, ps, hkv, P, fill=0.0)
    b = api.PagedKVCache(7, table, ps, hkv, P, fill=0.0)
    s = Stage(cuda, P, 4, hkv, 128, seed=77)
    _, k, v = api.qk_norm_rope_fwd(s.q, s.k, s.v, s.pos, s.rot, s.wq, s.wk)
    a.capture(k, v)
    p = torch.arange(P, device=cuda)
    slots = (table[p // ps] * ps + p % ps).to(torch.int32)
    for lo, hi in ((0, 100), (100, 101), (101, P)):
        api.qk_norm_rope_append(api.PagePool.of(b), s.q[lo:hi], s.k[lo:hi], s.v[lo:hi], slots[lo:hi],
                                s.pos[:, lo:hi].contiguous(), s.rot, s.wq, s.wk)
    assert torch.equal(a.k_pool, b.k_pool) and torch.equal(a.v_pool, b.v_pool)
    ok()


def test_bad_slots_and_axes_are_reported(cuda):
    s = Stage(cuda, 4, 2, 1, 32, seed=3)
    pool = api.PagePool.empty(2, 1, 16, cuda)
    pool.k_pool.fill_(1.0)
    pool.v_pool.fill_(1.0)
    slots = torch.tensor([0, 32, 2 ** 31 - 1, 5], dtype=torch.int32, device=cuda)
    q = api.qk_norm_rope_append(pool, s.q, s.k, s.v, slots, s.pos, s.rot, s.wq, s.wk)
    assert B.ls_last_device_error(0) == B.LS_ERR_DEVICE_CHECK
    close(q, *s.ref(s.q, s.wq))
    assert int((pool.v_pool != 1.0).any(-1).sum()) == 2
    axis = torch.tensor([0, 1, 2, 0, 1, -1, 0, 1, 0, 1, 0, 1, 0, 1, 0, 1], dtype=torch.int32,
                        device=cuda)
    pos = torch.arange(8, device=cuda, dtype=torch.int32).view(2, 4)
    rot = api.Rotary(s.freq, pair_axis=axis, axes=2)
    q, _, _ = api.qk_norm_rope_fwd(s.q, s.k, None, pos, rot, s.wq, s.wk, eps=EPS)
    assert B.ls_last_device_error(0) == B.LS_ERR_DEVICE_CHECK
    good = np.where((axis.cpu().numpy() < 0) | (axis.cpu().numpy() > 1), 0, axis.cpu().numpy())
    close(q, *qo.fwd(qo.f64(s.q), qo.f64(s.wq), 0.0, EPS, pos.cpu().numpy(), s.freq.cpu().numpy(),
                     good, False))
    ok()


def test_other_stream_and_graph(cuda):
    """On a side stream, and captured: replays follow inputs changed in place."""
    s = Stage(cuda, 100, 6, 2, 128, seed=12)
    dy = [torch.randn(100, h, 128, device=cuda) for h in (6, 2, 2)]
    q = torch.empty(100, 6, 128, dtype=torch.bfloat16, device=cuda)
    k = torch.empty(100, 2, 128, dtype=torch.bfloat16, device=cuda)
    dwq, dwk = torch.empty(128, device=cuda), torch.empty(128, device=cuda)
    dxq, dxk = torch.empty_like(q), torch.empty_like(k)

    def step():
        api.qk_norm_rope_fwd(s.q, s.k, None, s.pos, s.rot, s.wq, s.wk, q_out=q, k_out=k)
        api.qk_norm_rope_bwd(s.q, s.k, s.pos, s.rot, dy[0], dy[1], wq=s.wq, wk=s.wk, dx_q=dxq,
                             dx_k=dxk, dwq=dwq, dwk=dwk)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    st.synchronize()
    want = [t.clone() for t in (q, k, dxq, dxk, dwq, dwk)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        step()
    for t in (q, k, dxq, dxk, dwq, dwk):
        t.zero_()
    graph.replay()
    for t, w in zip((q, k, dxq, dxk, dwq, dwk), want):
        assert torch.equal(t, w)
    s.pos += 17
    s.buf.mul_(0.5)
    graph.replay()
    got = [t.clone() for t in (q, k, dxq, dxk, dwq, dwk)]
    step()
    for t, w in zip((q, k, dxq, dxk, dwq, dwk), got):
        assert torch.equal(t, w)
    ok()


def test_two_graphs_of_one_stream_at_once(cuda):
    """Backward passes captured on one stream and replayed on two: each has its workspace."""
    st, other = torch.cuda.Stream(), torch.cuda.Stream()
    runs = []
    for seed in (3, 4):
        s = Stage(cuda, 9000, 8, 2, 128, seed=seed)
        dy = [torch.randn(9000, h, 128, device=cuda, generator=gen(seed, cuda)) for h in (8, 2)]
        args = (s.q, s.k, s.pos, s.rot, dy[0], dy[1])
        want = api.qk_norm_rope_bwd(*args, wq=s.wq, wk=s.wk)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            got = api.qk_norm_rope_bwd(*args, wq=s.wq, wk=s.wk)
        runs.append((g, got, want, (s, dy)))  # a graph needs its inputs alive
    for _ in range(20):
        for (g, got, _, _), on in zip(runs, (st, other)):
            with torch.cuda.stream(on):
                g.replay()
    torch.cuda.synchronize()
    for _, got, want, _ in runs:
        for i in (0, 1, 3, 4):
            assert torch.equal(got[i], want[i])
    ok()


def test_a_given_stream_owns_what_the_call_allocates(cuda):
    """Memory that the current stream has freed but still uses is not handed to a call on
    another stream."""
    s = Stage(cuda, 300, 8, 2, 128, seed=5)
    want = api.qk_norm_rope_fwd(s.q, s.k, s.v, s.pos, s.rot, s.wq, s.wk)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    for given in (st, st.cuda_stream):
        freed = torch.empty_like(want[0])
        at = freed.data_ptr()
        del freed
        got = api.qk_norm_rope_fwd(s.q, s.k, s.v, s.pos, s.rot, s.wq, s.wk, stream=given)
        assert got[0].data_ptr() != at
        st.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)
    ok()


def test_offsets_past_32_bits(cuda):
    """Rows further than 2^32 elements into their tensors and pages."""
    T, far = 3, 2 ** 31 + 2 ** 20
    s = Stage(cuda, T, 2, 1, 128, seed=6)
    big = torch.empty(2 * far + 1024, dtype=torch.bfloat16, device=cuda)
    q = big.as_strided((T, 2, 128), (far, 128, 1))
    k = big.as_strided((T, 1, 128), (far, 128, 1), 256)
    q.copy_(s.q)
    k.copy_(s.k)
    want = api.qk_norm_rope_fwd(s.q, s.k, None, s.pos, s.rot, s.wq, s.wk)
    got = api.qk_norm_rope_fwd(q, k, None, s.pos, s.rot, s.wq, s.wk)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    dy = [torch.randn(T, h, 128, device=cuda) for h in (2, 1)]
    want_b = api.qk_norm_rope_bwd(s.q, s.k, s.pos, s.rot, dy[0], dy[1], wq=s.wq, wk=s.wk)
    got_b = api.qk_norm_rope_bwd(q, k, s.pos, s.rot, dy[0], dy[1], wq=s.wq, wk=s.wk, dx_q=q, dx_k=k)
    for x, y in zip(got_b, want_b):
        assert (x is None and y is None) or torch.equal(x, y)
    del big, q, k, got_b
    n = 2 ** 21 + 8  # pages of 16 rows of one head: 2^32 elements and some
    pool = api.PagePool.empty(n, 1, 16, cuda)
    slots = torch.tensor([n * 16 - 1, 5, n * 16 - 100], dtype=torch.int32, device=cuda)
    api.qk_norm_rope_append(pool, s.q, s.k, s.v, slots, s.pos, s.rot, s.wq, s.wk)
    at = slots.long()
    assert torch.equal(pool.k_pool[at // 16, 0, at % 16], want[1][:, 0])
    assert torch.equal(pool.v_pool[at // 16, 0, at % 16], s.v[:, 0])
    ok()
