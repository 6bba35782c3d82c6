"""GPU parity of ls_decode_attn against the 64-bit implementation, within bounds that
count the roundings (qk_oracle.decode), and a decode loop of the whole set."""
import numpy as np
import pytest
import torch

import qk_oracle as qo
from response_replay_gb300 import binding as B
from response_replay_gb300 import torch_api as api

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


class Group:
    """A captured prompt and the responses of a group in pages; whatever lies behind a
    sequence's end is NaN."""

    def __init__(self, dev, P, lens, hq, hkv, n=1, ps=64, rps=64, seed=0, sharp=2.0):
        g = torch.Generator(device=dev)
        g.manual_seed(seed)

        def normal(*s):
            return torch.randn(*s, generator=g, device=dev).to(torch.bfloat16)

        self.kp, self.vp = normal(P, hkv, 128), normal(P, hkv, 128)
        npg = -(-P // ps)
        table = torch.randperm(npg + 2, generator=g, device=dev)[:npg].to(torch.int32)
        self.cache = api.PagedKVCache(npg + 2, table, ps, hkv, P, fill=float("nan"))
        if P:
            self.cache.capture(self.kp, self.vp)
        M, top = len(lens), max([*lens, 1])
        nb = -(-top // rps) + 1
        self.kr = [normal(max(x, 0), hkv, 128) for x in lens]
        self.vr = [normal(max(x, 0), hkv, 128) for x in lens]
        pool = api.PagePool.empty(M * nb + 1, hkv, rps, dev)
        pool.k_pool.fill_(float("nan"))
        pool.v_pool.fill_(float("nan"))
        blocks = torch.randperm(M * nb, generator=g, device=dev).view(M, nb).to(torch.int32)
        for m, x in enumerate(lens):
            t = torch.arange(max(x, 0), device=dev)
            page = blocks[m, t // rps].long()
            pool.k_pool[page, :, t % rps] = self.kr[m]
            pool.v_pool[page, :, t % rps] = self.vr[m]
            used = -(-max(x, 0) // rps)
            blocks[m, used:] = 2 ** 30  # not read
        self.lens = torch.tensor(lens, dtype=torch.int32, device=dev)
        self.resp = api.ResponseCache(pool, blocks.contiguous(), self.lens)
        self.q = (normal(M, n, hq, 128) * sharp).contiguous()

    def run(self, **kw):
        out = api.decode_attn(self.cache, self.resp, self.q, SCALE, **kw)
        assert B.ls_last_device_error(0) == B.LS_OK
        return out

    def check(self, o, lse):
        ref, ob, lref, lb = qo.decode(qo.f64(self.q), qo.f64(self.kp), qo.f64(self.vp),
                                      [qo.f64(x) for x in self.kr], [qo.f64(x) for x in self.vr],
                                      self.lens.tolist(), SCALE)
        live = np.array(self.lens.tolist()) >= 0
        o, lse = qo.f64(o)[live], qo.f64(lse)[live]
        assert (np.abs(o - ref[live]) <= ob[live]).all(), np.nanmax(np.abs(o - ref[live]) / ob[live].clip(1e-30))
        lref, lb = lref[live], lb[live]
        none = np.isinf(lref)
        assert (lse[none] == -np.inf).all()
        assert (np.abs(lse[~none] - lref[~none]) <= lb[~none]).all(), np.abs(lse[~none] - lref[~none]).max()


# Prompts from none over a ragged last page to many tiles; lengths around tile and page
# edges, empty responses; one row tile and several; members straddling row tiles; several
# new tokens; head groups that do not divide a tile; every page size class.
CASES = [
    (1000, [1], 1, 1, 1, 64, 64),
    (0, [5, 0, 300], 6, 2, 1, 64, 16),
    (0, [0], 4, 4, 1, 64, 64),
    (1, [1, 2], 8, 2, 1, 16, 16),
    (128, [128, 129, 127, 64, 65], 12, 2, 1, 128, 64),
    (5000, [7, 250, 63, 64, 1000, 1, 33, 500], 24, 4, 1, 64, 64),
    (3001, [40, 41], 5, 1, 3, 256, 256),
    (700, [10, 2, 600], 14, 2, 5, 32, 16),
    (2500, [100 + 7 * i for i in range(30)], 24, 4, 1, 64, 64),
    (2049, [3 * i for i in range(70)], 6, 1, 2, 64, 32),
    (640, [20 + i for i in range(9)], 16, 1, 8, 64, 64),
    (4096, [1, 4096], 40, 8, 1, 4096, 4096),
    (300, [9, 130], 128, 1, 1, 64, 64),
]


# Many tiles to a CTA: long segments, in which the ring of tiles goes round many times and
# loads land out of order; several segments of several tiles each.
LONG = [
    (200003, [5000, 37, 1, 2600], 6, 1, 1, 64, 64),
    (0, [40000, 129, 30001], 6, 2, 1, 64, 16),
    (70000, [300 + 100 * i for i in range(44)], 12, 2, 1, 16, 256),
    (128000, [513, 30000], 8, 8, 2, 256, 32),
]


@pytest.mark.parametrize("P,lens,hq,hkv,n,ps,rps", LONG)
def test_long_segments(cuda, P, lens, hq, hkv, n, ps, rps):
    g = Group(cuda, P, lens, hq, hkv, n, ps, rps, seed=P + hq)
    o, lse = g.run()
    g.check(o, lse)
    for _ in range(50):  # the same bits whatever order the loads land in
        o2, lse2 = api.decode_attn(g.cache, g.resp, g.q, SCALE)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    assert B.ls_last_device_error(0) == B.LS_OK


@pytest.mark.parametrize("P,lens,hq,hkv,n,ps,rps", CASES)
def test_decode(cuda, P, lens, hq, hkv, n, ps, rps):
    g = Group(cuda, P, lens, hq, hkv, n, ps, rps, seed=P + hq)
    g.check(*g.run())


def test_members_out_of_use_and_short_rows(cuda):
    """Rows of a member out of use are not written; tokens before a response's start see
    the prompt only."""
    g = Group(cuda, 500, [-1, 30, -9, 1, 0], 12, 2, n=3, seed=3)
    o = torch.full_like(g.q, 5.0)
    lse = torch.full(g.q.shape[:3], 6.0, device=cuda)
    g.run(o=o, lse=lse)
    g.check(o, lse)
    for m in (0, 2):
        assert bool((o[m] == 5.0).all()) and bool((lse[m] == 6.0).all())
    g = Group(cuda, 0, [1, 0], 4, 2, n=2, seed=4)
    o, lse = g.run()
    g.check(o, lse)
    assert bool((o[1] == 0).all()) and bool((o[0, 0] == 0).all())


def test_many_members(cuda):
    """As many members as the call takes (more row tiles than columns could hold twice),
    their lengths summed over several rounds of threads."""
    lens = [(i * 37) % 90 for i in range(1024)]
    g = Group(cuda, 900, lens, 8, 2, seed=8, rps=16)
    g.check(*g.run())


def test_large_scores_and_rising_maxima(cuda):
    """Keys that grow along the prompt: the running maximum keeps moving, past the
    threshold at which the accumulator is rescaled; huge scores stay finite."""
    g = Group(cuda, 3000, [700, 20], 8, 2, seed=6, sharp=6.0)
    ramp = torch.linspace(0.1, 8.0, 3000, device=cuda)[:, None, None]
    g.kp = (g.kp.float() * ramp).to(torch.bfloat16)
    g.cache.capture(g.kp, g.vp)
    o, lse = g.run()
    assert torch.isfinite(o.float()).all()
    g.check(o, lse)


def test_agrees_with_the_replay_forward(cuda):
    """The last row of a replay over the same prompt and response."""
    g = Group(cuda, 2000, [150], 24, 4, seed=10)
    q = torch.randn(150, 24, 128, device=cuda).to(torch.bfloat16)
    q[149] = g.q[0, 0]
    o, lse = api.replay_fwd(g.cache, q, g.kr[0], g.vr[0], SCALE, 4)
    od, ld = g.run()
    assert (o[149].float() - od[0, 0].float()).abs().max() <= 2 ** -7
    assert (lse[149] - ld[0, 0]).abs().max() <= 1e-5


def test_bad_pages_and_lengths_are_reported(cuda):
    g = Group(cuda, 500, [100, 20], 8, 2, seed=11)
    ref, _ = g.run()
    blocks = g.resp.block_table
    keep = int(blocks[0, 1])
    blocks[0, 1] = 10 ** 6
    o, _ = api.decode_attn(g.cache, g.resp, g.q, SCALE)
    assert B.ls_last_device_error(0) == B.LS_ERR_DEVICE_CHECK
    assert torch.equal(o[1], ref[1]) and torch.isfinite(o.float()).all()
    blocks[0, 1] = keep
    g.lens[1] = 10 ** 9   # past the table: cut, and its unset entries reported
    o, _ = api.decode_attn(g.cache, g.resp, g.q, SCALE)
    assert B.ls_last_device_error(0) == B.LS_ERR_DEVICE_CHECK
    assert torch.equal(o[0], ref[0])


def test_repeatable_and_streams(cuda):
    g = Group(cuda, 9000, [300, 2000, 5], 12, 2, seed=12)
    o, lse = g.run()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        o2, lse2 = api.decode_attn(g.cache, g.resp, g.q, SCALE)
    st.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_prompt_in_host_memory(cuda):
    g = Group(cuda, 700, [50, 3], 8, 2, seed=13)
    ref = g.run()
    host = api.PagedKVCache(g.cache.k_pool.shape[0], g.cache.page_table, 64, 2, 700, host_pools=True)
    host.k_pool.copy_(g.cache.k_pool)
    host.v_pool.copy_(g.cache.v_pool)
    torch.cuda.synchronize()
    g.cache = host
    out = g.run()
    assert torch.equal(ref[0], out[0]) and torch.equal(ref[1], out[1])


@pytest.mark.parametrize("graph", [False, True])
def test_decode_loop(cuda, graph):
    """The set as it is used: a group generates token by token over a captured prompt
    (pages and slots, norm + rotation into the pages, attention), eager and as one
    captured graph; every step's output is that of the whole response's replay."""
    P, M, hq, hkv, ps, steps = 333, 3, 6, 2, 16, 40
    gen = torch.Generator(device=cuda)
    gen.manual_seed(21)

    def normal(*s):
        return torch.randn(*s, generator=gen, device=cuda).to(torch.bfloat16)

    rot = api.Rotary.from_base(1e6, 64, cuda)
    wq, wk = torch.rand(128, device=cuda) + 0.5, torch.rand(128, device=cuda) + 0.5
    table = torch.randperm(8, generator=gen, device=cuda)[:6].to(torch.int32)
    cache = api.PagedKVCache(8, table, 64, hkv, P, fill=float("nan"))
    pos = torch.arange(P, device=cuda, dtype=torch.int32)
    px = normal(P, (hq + 2 * hkv), 128)
    _, k, v = api.qk_norm_rope_fwd(px[:, :hq], px[:, hq:hq + hkv], px[:, hq + hkv:], pos, rot, wq, wk)
    cache.capture(k, v)
    alloc = api.PageAllocator.empty(M, 4, M * 4, ps, cuda)
    pool = api.PagePool.empty(M * 4, hkv, ps, cuda)
    pool.k_pool.fill_(float("nan"))
    pool.v_pool.fill_(float("nan"))
    resp = api.ResponseCache.of(pool, alloc)
    x = normal(steps, M, hq + 2 * hkv, 128)
    cur = torch.empty_like(x[0])
    add = torch.ones(M, dtype=torch.int32, device=cuda)
    slots = torch.empty(M, dtype=torch.int32, device=cuda)
    rpos = torch.empty((1, M), dtype=torch.int32, device=cuda)
    o = torch.empty(M, 1, hq, 128, dtype=torch.bfloat16, device=cuda)
    lse = torch.empty(M, 1, hq, device=cuda)

    def step():
        api.extend_pages(alloc, add, P, slots, rpos)
        q = api.qk_norm_rope_append(pool, cur[:, :hq], cur[:, hq:hq + hkv], cur[:, hq + hkv:], slots,
                                    rpos, rot, wq, wk)
        api.decode_attn(cache, resp, q.view(M, 1, hq, 128), SCALE, o=o, lse=lse)

    outs, lses, first = [], [], 0
    if graph:
        cur.copy_(x[0])
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            step()
        st.synchronize()
        outs, lses, first = [o.clone()], [lse.clone()], 1
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            step()
    for t in range(first, steps):
        cur.copy_(x[t])
        gr.replay() if graph else step()
        outs.append(o.clone())
        lses.append(lse.clone())
    assert B.ls_last_device_error(0) == B.LS_OK and alloc.lens.tolist() == [steps] * M
    got, gl = torch.cat(outs, 1), torch.cat(lses, 1)                  # [M][steps][hq]..
    rp = torch.arange(P, P + steps, device=cuda, dtype=torch.int32)
    for m in range(M):
        xm = x[:, m]
        q, k, v = api.qk_norm_rope_fwd(xm[:, :hq], xm[:, hq:hq + hkv], xm[:, hq + hkv:], rp, rot, wq, wk)
        ro, rl = api.replay_fwd(cache, q, k, v, SCALE, 2)
        assert (ro.float() - got[m].float()).abs().max() <= 2 ** -7 * got[m].float().abs().max()
        assert (rl - gl[m]).abs().max() <= 1e-5


def test_layered_responses(cuda):
    """Two layers under one allocator, ragged first tokens, then decode steps: every layer's
    output of a member's newest token is that of the replay of its whole response."""
    from response_replay_gb300 import layers as L
    P, M, hq, hkv, ps, nl = 200, 3, 6, 2, 16, 2
    gen = torch.Generator(device=cuda)
    gen.manual_seed(5)

    def normal(*s):
        return torch.randn(*s, generator=gen, device=cuda).to(torch.bfloat16)

    table = torch.tensor([3, 0, 2, 1], dtype=torch.int32, device=cuda)
    prompt = L.LayeredKVCache(nl, 5, table, 64, hkv, P, fill=float("nan"))
    for l in range(nl):
        prompt.capture(l, normal(P, hkv, 128), normal(P, hkv, 128))
    r = L.LayeredResponses(prompt, hkv, M, 64, 12, ps, cuda, capacity=60)
    r.k_pools.fill_(float("nan"))
    r.v_pools.fill_(float("nan"))
    rot = api.Rotary.from_base(1e6, 128, cuda)
    w = torch.rand(128, generator=gen, device=cuda) + 0.5
    adds = [[17, 0, 33], [1, 1, 1], [1, 1, 1]]
    xs = [[normal(sum(a[m] for a in adds), hq + 2 * hkv, 128) for m in range(M)] for _ in range(nl)]
    done = [0] * M
    for add in adds:
        r.extend(torch.tensor(add, dtype=torch.int32, device=cuda))
        n = sum(add)
        for l in range(nl):
            x = torch.zeros(60, hq + 2 * hkv, 128, dtype=torch.bfloat16, device=cuda)
            x[:n] = torch.cat([xs[l][m][done[m]:done[m] + add[m]] for m in range(M)])
            q = r.append(l, x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], rot, w, w)
            last = torch.tensor([sum(add[:m + 1]) - 1 for m in range(M)], device=cuda).clamp(min=0)
            o, lse = r.attend(l, q[last].view(M, 1, hq, 128), SCALE)
            for m in range(M):
                R = done[m] + add[m]
                if add[m] == 0:
                    continue
                pos = torch.arange(P, P + R, dtype=torch.int32, device=cuda)
                xm = xs[l][m][:R]
                rq, rk, rv = api.qk_norm_rope_fwd(xm[:, :hq], xm[:, hq:hq + hkv], xm[:, hq + hkv:],
                                                  pos, rot, w, w)
                ro, rl = api.replay_fwd(prompt[l], rq, rk, rv, SCALE, 2)
                assert (ro[R - 1].float() - o[m, 0].float()).abs().max() <= 2 ** -7 * ro.float().abs().max()
                assert (rl[R - 1] - lse[m, 0]).abs().max() <= 1e-5
        done = [d + a for d, a in zip(done, add)]
    assert r.alloc.lens.tolist() == done and B.ls_last_device_error(0) == B.LS_OK


def test_two_graphs_of_one_stream_at_once(cuda):
    """Decode steps captured on one stream and replayed on two: each has its workspace."""
    st, other = torch.cuda.Stream(), torch.cuda.Stream()
    runs = []
    for seed in (30, 31):
        g = Group(cuda, 60000, [500, 90, 1], 12, 2, seed=seed)
        want = g.run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            got = api.decode_attn(g.cache, g.resp, g.q, SCALE)
        runs.append((graph, got, want, g))
    for _ in range(30):
        for (graph, *_), on in zip(runs, (st, other)):
            with torch.cuda.stream(on):
                graph.replay()
    torch.cuda.synchronize()
    for _, got, want, _ in runs:
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert B.ls_last_device_error(0) == B.LS_OK


def test_shared_pages_and_responses_in_host_memory(cuda):
    """Two members over the same response pages; pages appended to and read in pinned host
    memory; pages further than 2^32 elements into a pool."""
    g = Group(cuda, 300, [70, 70, 5], 8, 2, rps=16, seed=32)
    g.resp.block_table[1] = g.resp.block_table[0]
    g.kr[1], g.vr[1], g.q[1] = g.kr[0], g.vr[0], g.q[0]
    o, lse = g.run()
    g.check(o, lse)
    assert torch.equal(o[0], o[1]) and torch.equal(lse[0], lse[1])

    n = 5
    slots = torch.tensor([3, 2, 17, 40, -1], dtype=torch.int32, device=cuda)
    x = torch.randn(n, 3, 128, device=cuda).to(torch.bfloat16)
    args = (x[:, :1].expand(n, 4, 128), x[:, 1:2], x[:, 2:], slots, None, None)
    dev = api.PagePool.empty(3, 1, 16, cuda)
    dev.k_pool.zero_(), dev.v_pool.zero_()
    host = api.PagePool(*(torch.zeros(3, 1, 16, 128, dtype=torch.bfloat16, pin_memory=True) for _ in "kv"))
    for pool in (dev, host):
        q = api.qk_norm_rope_append(pool, *args)
    torch.cuda.synchronize()
    assert torch.equal(host.k_pool, dev.k_pool.cpu()) and torch.equal(host.v_pool, dev.v_pool.cpu())
    cache = api.PagedKVCache(1, torch.zeros(1, dtype=torch.int32, device=cuda), 16, 1, 0)
    table = torch.tensor([[0, 1, 2], [2, 0, 1]], dtype=torch.int32, device=cuda)
    lens = torch.tensor([48, 20], dtype=torch.int32, device=cuda)
    out = [api.decode_attn(cache, api.ResponseCache(pool, table, lens), q[:2].view(2, 1, 4, 128), SCALE)
           for pool in (dev, host)]
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])

    far = 2 ** 21
    big = api.PagePool.empty(far + 3, 1, 16, cuda)
    big.k_pool[far:], big.v_pool[far:] = dev.k_pool, dev.v_pool
    got = api.decode_attn(cache, api.ResponseCache(big, table + far, lens), q[:2].view(2, 1, 4, 128), SCALE)
    assert torch.equal(out[0][0], got[0]) and torch.equal(out[0][1], got[1])
    assert B.ls_last_device_error(0) == B.LS_OK
