"""GPU tests of decode calls as a group's life brings them: every member out of use, calls
from several host threads, captures that torch does not make, members that end at different
times; and of every V tile's way into the output."""
import ctypes as C
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import qk_oracle as qo
from response_replay_gb300 import binding as B
from response_replay_gb300 import layers as L
from response_replay_gb300 import torch_api as api
from test_gpu_decode import SCALE, Group
from test_stage_calls import run_threads

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("P,members", [(300000, 8), (5000, 70)])
def test_every_member_out_of_use(cuda, P, members):
    """A finished group's call writes nothing, and what follows it on the stream (lengths
    written anew, a live call with the same workspace) finds it done."""
    g = Group(cuda, P, [40 + 3 * i for i in range(members)], 12, 2, seed=50)
    live = g.lens.clone()
    want = [x.clone() for x in g.run()]
    gone = torch.full_like(live, -1)
    o, lse = torch.full_like(want[0], 5.0), torch.full_like(want[1], 6.0)
    got = [torch.empty_like(x) for x in want]
    for _ in range(20):
        g.lens.copy_(gone)
        api.decode_attn(g.cache, g.resp, g.q, SCALE, o=o, lse=lse)
        g.lens.copy_(live)
        api.decode_attn(g.cache, g.resp, g.q, SCALE, o=got[0], lse=got[1])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert bool((o == 5.0).all()) and bool((lse == 6.0).all())
    assert B.ls_last_device_error(0) == B.LS_OK


def test_two_host_threads_on_one_stream(cuda):
    """Decode calls and backward calls from two threads, each with inputs of its own: every
    call gives the bits that it gives alone."""
    runs = []
    for seed, (P, lens) in enumerate([(30000, [500, 90, 1]), (9000, [7, 1300, 64])]):
        g = Group(cuda, P, lens, 12, 2, seed=60 + seed)
        gen = torch.Generator(device=cuda)
        gen.manual_seed(seed)
        x = torch.randn(300 + 100 * seed, 8, 128, generator=gen, device=cuda).to(torch.bfloat16)
        dy = torch.randn(x.shape, generator=gen, device=cuda)
        w = torch.rand(128, generator=gen, device=cuda) + 0.5

        def work(g=g, x=x, dy=dy, w=w):
            o, lse = api.decode_attn(g.cache, g.resp, g.q, SCALE)
            return [o, lse, *api.qk_norm_rope_bwd(x[:, :6], x[:, 6:], None, None, dy[:, :6], dy[:, 6:],
                                                  wq=w, wk=w)]

        runs.append((work, [t.clone() for t in work() if t is not None]))
    torch.cuda.synchronize()

    def body(i):
        work, want = runs[i]
        for _ in range(100):
            got = [t for t in work() if t is not None]
            assert all(torch.equal(a, b) for a, b in zip(got, want, strict=True))

    run_threads(2, body)
    assert B.ls_last_device_error(0) == B.LS_OK


def test_capture_through_the_runtime(cuda):
    """A capture that torch does not make: its replays write into no other tensor."""
    rt = C.CDLL(f"libcudart.so.{torch.version.cuda.split('.')[0]}")

    def ok(status):
        assert status == 0, status

    g = Group(cuda, 60000, [500, 90, 1], 12, 2, seed=70)
    x = torch.randn(700, 8, 128, device=cuda).to(torch.bfloat16)
    dy = torch.randn(x.shape, device=cuda)
    w = torch.ones(128, device=cuda)
    grads = [torch.empty_like(t) for t in (x[:, :6], x[:, 6:])] + [torch.empty_like(w) for _ in "qk"]
    o, lse = torch.empty_like(g.q), torch.empty(g.q.shape[:3], device=cuda)

    def work():
        api.decode_attn(g.cache, g.resp, g.q, SCALE, o=o, lse=lse)
        api.qk_norm_rope_bwd(x[:, :6], x[:, 6:], None, None, dy[:, :6], dy[:, 6:], wq=w, wk=w,
                             dx_q=grads[0], dx_k=grads[1], dwq=grads[2], dwk=grads[3])

    work()
    outs = [o, lse, *grads]
    want = [t.clone() for t in outs]
    sizes = (B.ls_decode_attn_workspace(g.cache.struct, g.resp.struct, 1, 12),
             B.ls_qk_norm_rope_bwd_workspace(700))
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph, run = C.c_void_p(), C.c_void_p()
    handle = C.c_void_p(st.cuda_stream)
    with torch.cuda.stream(st):
        spare = [torch.empty(n, dtype=torch.uint8, device=cuda) for n in sizes]  # blocks to be taken
        del spare
        ok(rt.cudaStreamBeginCapture(handle, C.c_int(2)))  # relaxed
        work()
        ok(rt.cudaStreamEndCapture(handle, C.byref(graph)))
        ok(rt.cudaGraphInstantiate(C.byref(run), graph, C.c_ulonglong(0)))
        later = [torch.full((n,), 77, dtype=torch.uint8, device=cuda) for n in sizes for _ in range(8)]
        for t in outs:
            t.zero_()
        for _ in range(3):
            ok(rt.cudaGraphLaunch(run, handle))
    st.synchronize()
    assert all(bool((t == 77).all()) for t in later)
    assert all(torch.equal(a, b) for a, b in zip(outs, want, strict=True))
    ok(rt.cudaGraphExecDestroy(run))
    ok(rt.cudaGraphDestroy(graph))
    assert B.ls_last_device_error(0) == B.LS_OK


def test_workspaces_of_torch_graphs_stay_in_their_pools(cuda):
    """Captures of torch's own take nothing from the memory that all tensors share."""
    g = Group(cuda, 3000, [50, 9], 12, 2, seed=71)
    want = [t.clone() for t in g.run()]
    kept = len(api._captured_workspaces)
    pool = torch.cuda.graph_pool_handle()
    graphs = [torch.cuda.CUDAGraph() for _ in range(3)]  # a pool lives as long as its graphs
    for graph, p in zip(graphs, (None, pool, pool)):
        with torch.cuda.graph(graph, pool=p):
            got = api.decode_attn(g.cache, g.resp, g.q, SCALE)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want, strict=True))
    assert len(api._captured_workspaces) == kept


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("lens,add,rows,ps", [
    ([15, 16, 0, 31, -1], [1, 0, 1, 1, 0], 1, 16),
    ([15, 16, 0, 31, -1, 7], [3, 0, 1, 2, 0, 5], 5, 16),
    ([i % 50 for i in range(1024)], [i % 8 for i in range(1024)], 7, 16),       # several blocks
    ([0, 300, 5], [4001, 0, 6000], 6000, 256),
    ([3, 4], [1, 3], 2, 16),                                                    # more than its rows
    ([3, -1], [1, 1], 2, 16),                                                   # out of use
])
def test_extend_by_member(cuda, lens, add, rows, ps, in_place):
    """Pages, lengths and slots are those of the packed call, every member's in its rows."""
    M, spare = len(lens), 3
    have = [-(-x // ps) if x > 0 else 0 for x in lens]
    blocks = max(-(-(max(x, 0) + a) // ps) for x, a in zip(lens, add)) + 1
    free = np.random.default_rng(M).permutation(M * blocks + spare)
    table, used = np.full((M, blocks), -7), 0
    for m, h in enumerate(have):
        table[m, :h] = free[used:used + h]
        used += h

    def i32(x):
        return torch.tensor(np.asarray(x), dtype=torch.int32, device=cuda)

    a = api.PageAllocator(i32(table), i32(lens), i32(free), i32([used]), ps)
    slots = torch.full((M * rows,), 99, dtype=torch.int32, device=cuda)
    pos = torch.full((2, M * rows), 99, dtype=torch.int32, device=cuda)
    lo, uo = (None, None) if in_place else (torch.empty_like(a.lens), torch.empty_like(a.used))
    api.extend_pages(a, i32(add), 1000, slots, pos, lens_out=lo, used_out=uo, member_rows=rows)
    lo, uo = (a.lens, a.used) if in_place else (lo, uo)
    ref = qo.extend(table, lens, add, free, used, ps, 1000, 2, sum(add))
    if ref is None or max(add) > rows:
        assert B.ls_last_device_error(0) == B.LS_ERR_DEVICE_CHECK
        assert bool((slots == -1).all()) and bool((pos == 0).all())
        assert lo.tolist() == lens and int(uo) == used and a.block_table.tolist() == table.tolist()
        return
    assert B.ls_last_device_error(0) == B.LS_OK
    want_slots, want_pos, t = np.full((M, rows), -1), np.zeros((2, M, rows), int), 0
    for m, n in enumerate(add):
        want_slots[m, rows - n:] = ref[0][t:t + n]
        want_pos[:, m, rows - n:] = ref[1][:, t:t + n]
        t += n
    np.testing.assert_array_equal(slots.cpu().numpy(), want_slots.ravel())
    np.testing.assert_array_equal(pos.cpu().numpy(), want_pos.reshape(2, -1))
    np.testing.assert_array_equal(a.block_table.cpu().numpy(), ref[2])
    np.testing.assert_array_equal(lo.cpu().numpy(), ref[3])
    assert int(uo) == ref[4]


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("rows", [1, 3])
def test_loop_whose_members_end_at_different_times(cuda, graph, rows):
    """Steps of fixed rows, eager and as one captured graph, in which members end, pause and
    add up to `rows` tokens: every token's output is that of its response's replay."""
    P, M, hq, hkv, ps = 200, 4, 6, 2, 16
    gen = torch.Generator(device=cuda)
    gen.manual_seed(80 + rows)

    def normal(*s):
        return torch.randn(*s, generator=gen, device=cuda).to(torch.bfloat16)

    table = torch.tensor([3, 0, 2, 1], dtype=torch.int32, device=cuda)
    prompt = L.LayeredKVCache(1, 5, table, 64, hkv, P, fill=float("nan"))
    prompt.capture(0, normal(P, hkv, 128), normal(P, hkv, 128))
    r = L.LayeredResponses(prompt, hkv, M, 64, 16, ps, cuda, member_rows=rows)
    r.k_pools.fill_(float("nan"))
    r.v_pools.fill_(float("nan"))
    rot = api.Rotary.from_base(1e6, 128, cuda)
    w = torch.rand(128, generator=gen, device=cuda) + 0.5
    rng = np.random.default_rng(rows)
    last = [20, 5, 0, 13]  # step after which a member adds nothing
    adds = [[int(rng.integers(0 if rows > 1 else 1, rows + 1)) if t < last[m] else 0 for m in range(M)]
            for t in range(20)]
    total = [sum(a[m] for a in adds) for m in range(M)]
    x = [normal(max(n, 1), hq + 2 * hkv, 128) for n in total]
    cur = torch.empty(M, rows, hq + 2 * hkv, 128, dtype=torch.bfloat16, device=cuda)
    add = torch.zeros(M, dtype=torch.int32, device=cuda)
    o = torch.empty(M, rows, hq, 128, dtype=torch.bfloat16, device=cuda)
    lse = torch.empty(M, rows, hq, device=cuda)

    def step():
        r.extend(add)
        f = cur.view(M * rows, hq + 2 * hkv, 128)
        q = r.append(0, f[:, :hq], f[:, hq:hq + hkv], f[:, hq + hkv:], rot, w, w)
        r.attend(0, q.view(M, rows, hq, 128), SCALE, o=o, lse=lse)

    run = step
    if graph:
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            step()  # adds nothing yet
        st.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured, stream=st):
            step()
        run = captured.replay
    got, got_lse, done = [[] for _ in x], [[] for _ in x], [0] * M
    for a in adds:
        cur.fill_(float("nan"))  # rows without a token hold anything
        for m, n in enumerate(a):
            cur[m, rows - n:] = x[m][done[m]:done[m] + n]
            done[m] += n
        add.copy_(torch.tensor(a, dtype=torch.int32))
        run()
        for m, n in enumerate(a):
            got[m].append(o[m, rows - n:].clone())
            got_lse[m].append(lse[m, rows - n:].clone())
    assert r.alloc.lens.tolist() == total and B.ls_last_device_error(0) == B.LS_OK
    for m, n in enumerate(total):
        if n == 0:
            continue
        pos = torch.arange(P, P + n, dtype=torch.int32, device=cuda)
        q, k, v = api.qk_norm_rope_fwd(x[m][:, :hq], x[m][:, hq:hq + hkv], x[m][:, hq + hkv:], pos, rot, w, w)
        ro, rl = api.replay_fwd(prompt[0], q, k, v, SCALE, 2)
        od, ld = torch.cat(got[m]), torch.cat(got_lse[m])
        assert (ro.float() - od.float()).abs().max() <= 2 ** -7 * ro.float().abs().max()
        assert (rl - ld).abs().max() <= 1e-5


def test_member_rows_refused(cuda):
    a = api.PageAllocator.empty(3, 4, 12, 16, cuda)
    add = torch.ones(3, dtype=torch.int32, device=cuda)
    for n, rows in ((4, 1), (3, 2), (0, 0), (3, -1)):
        with pytest.raises(ValueError, match="member_rows"):
            api.extend_pages(a, add, 0, torch.empty(n, dtype=torch.int32, device=cuda), member_rows=rows)
    with pytest.raises(ValueError, match="member_rows"):
        L.LayeredResponses([None], 2, 3, 64, 12, 16, cuda, capacity=5, member_rows=2)
    assert a.lens.tolist() == [0, 0, 0]


# long segments of one and several row tiles, one and several KV heads; small and large pages
TILES = [
    (200003, [5000, 37, 1, 2600], 6, 1, 1, 64, 64),
    (0, [40000, 129, 30001], 6, 2, 1, 64, 16),
    (70000, [300 + 100 * i for i in range(44)], 12, 2, 1, 16, 256),
    (128000, [513, 30000], 8, 8, 2, 256, 32),
    (16389, [700, 2000], 16, 8, 2, 16, 16),
]


@pytest.mark.parametrize("mod", [128, 101])
@pytest.mark.parametrize("P,lens,hq,hkv,n,ps,rps", TILES)
def test_every_v_tile_shows(cuda, P, lens, hq, hkv, n, ps, rps, mod):
    """Nearly even weights, and values that are one in a single dimension, another for every
    tile of 128 keys until `mod` of them have gone by: a tile that is left out, taken twice or
    taken from another place of the ring moves o by more than its bound allows, twice over."""
    g = Group(cuda, P, lens, hq, hkv, n, ps, rps, seed=P + mod, sharp=0.03)

    def coded(keys, first):
        d = (first + torch.arange(keys, device=cuda) // 128)[:, None] + 17 * torch.arange(hkv, device=cuda)
        return torch.nn.functional.one_hot(d % mod, 128).to(torch.bfloat16)

    before = -(-P // 128)  # a response's tiles are numbered behind the prompt's
    g.vp = coded(P, 0)
    if P:
        g.cache.capture(g.kp, g.vp)
    for m, x in enumerate(lens):
        g.vr[m] = coded(x, before + 3 * m)
        t = torch.arange(x, device=cuda)
        g.resp.pool.v_pool[g.resp.block_table[m, t // rps].long(), :, t % rps] = g.vr[m]
    o, lse = g.run()
    # what half a tile brings into its dimension at the least, against that dimension's bound
    _, ob, _, _ = qo.decode(qo.f64(g.q), qo.f64(g.kp), qo.f64(g.vp), [qo.f64(x) for x in g.kr],
                            [qo.f64(x) for x in g.vr], lens, SCALE)
    for m, x in enumerate(lens):
        qh = g.q[m].double().view(n, hkv, hq // hkv, 128).permute(1, 0, 2, 3).flatten(1, 2)
        s = SCALE * max(float((qh @ k.double().permute(1, 2, 0)).abs().max())
                        for k in (g.kp, g.kr[m]) if len(k))
        assert 64 / (P + x) * np.exp(-2 * s) > 2 * ob[m].max(), m
    g.check(o, lse)


ASYNC = """
import sys
sys.path[:0] = {paths!r}
import torch
from response_replay_gb300 import binding as B, torch_api as api
from test_gpu_decode import SCALE, Group
assert torch.cuda.get_allocator_backend() == "cudaMallocAsync"
g = Group(torch.device("cuda:0"), 3000, [50, 9], 12, 2, seed=71)
want = [t.clone() for t in g.run()]
graph = torch.cuda.CUDAGraph()
outs = [torch.empty_like(t) for t in want]
with torch.cuda.graph(graph):
    for _ in range(3):
        api.decode_attn(g.cache, g.resp, g.q, SCALE, o=outs[0], lse=outs[1])
for _ in range(3):
    for t in outs:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want, strict=True))
assert B.ls_last_device_error(0) == B.LS_OK and not api._captured_workspaces
"""


def test_captured_with_the_stream_ordered_allocator(cuda):
    """A process whose allocator is cudaMallocAsync: captured calls and their replays."""
    tests = os.path.dirname(os.path.abspath(__file__))
    env = {**os.environ, "PYTORCH_CUDA_ALLOC_CONF": "backend:cudaMallocAsync",
           "PYTORCH_ALLOC_CONF": "backend:cudaMallocAsync"}
    r = subprocess.run([sys.executable, "-c", ASYNC.format(paths=[os.path.dirname(tests), tests])], env=env,
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
