"""GPU tests of decode calls as a group's life brings them: every member out of use, calls
from several host threads, captures that torch does not make, members that end at different
times; and of every V tile's way into the output."""
import ctypes as C

import pytest
import torch

from response_replay_gb300 import binding as B
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
