"""CPU tests of what surrounds the kernels of the query/key stage and the decode step: the
order of dependent launches, workspaces, and the values that the smoke run compares with."""
import os
import re
import threading
import weakref

import pytest
import torch

import __graft_entry__ as entry
import qk_oracle as qo
from response_replay_gb300 import binding as B
from response_replay_gb300 import torch_api as api

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "response_replay_gb300", "csrc")
WAIT = 'griddepcontrol.wait;'


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith(".cu")))
def test_dependent_grids_wait_before_every_exit(name):
    """A grid that is launched while the one before it still runs may end only after that
    one: whatever comes next on the stream waits for the dependent grid alone.  So no block
    leaves such a kernel ahead of its wait."""
    with open(os.path.join(CSRC, name)) as f:
        kernels = re.split(r"(?m)^(?=.*__global__)", re.sub(r"//[^\n]*", "", f.read()))[1:]
    for k in kernels:
        if WAIT not in k:
            continue
        before = k[:k.rindex(WAIT)]
        for m in re.finditer(r"\breturn;", before):
            assert WAIT in before[before.rindex("{", 0, m.start()):m.start()], before[m.start() - 80:m.end()]


@pytest.fixture
def host_calls(monkeypatch):
    """_with_workspace on host tensors: run(call, bytes, stream) for a fake of a C call."""
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(api, "_stream_workspaces", {}, raising=False)
    monkeypatch.setattr(api, "_workspaces", {})
    like = torch.empty(0)

    def run(call, nbytes, stream=1):
        def checked(ws, have, st):
            if have < nbytes:
                raise B.LongstrawError("call", B.LS_ERR_WORKSPACE)
            call(ws)
        return api._with_workspace(checked, (), lambda: nbytes, like, "kind", stream)

    return run


def run_threads(n, body):
    errors = []

    def guarded(i):
        try:
            body(i)
        except BaseException as e:  # noqa: BLE001 - reported by the test's thread
            errors.append(e)

    threads = [threading.Thread(target=guarded, args=(i,)) for i in range(n)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


def test_one_workspace_serves_one_call_at_a_time(host_calls):
    """Two threads on one stream: a call's launches are not mixed with another's, whether
    they find the workspace, make it or outgrow it."""
    inside, clash, seen = [], [], []

    def body(i):
        def call(ws):
            seen.append(ws)
            if ws in inside:
                clash.append(ws)
            inside.append(ws)
            pause.wait(0.002)
            inside.remove(ws)

        for step in range(20):
            host_calls(call, 256 * (1 + (step * 7 + i) % (step + 1)))

    pause = threading.Event()
    run_threads(4, body)
    assert len(seen) == 80 and not clash


def test_calls_on_two_streams_do_not_wait_for_each_other(host_calls):
    both = threading.Barrier(2)
    run_threads(2, lambda i: host_calls(lambda ws: both.wait(10), 1000, stream=7 + i))


@pytest.mark.parametrize("pool,kept", [((0, 0), True), ((3, 0), False), ((0, 9), False)])
def test_a_captured_workspace_lives_as_long_as_its_graph(monkeypatch, pool, kept):
    """Within torch's capture the graph's own memory pool holds on to the workspace; in a
    capture of another library the memory would go to the next tensor, under every replay's
    writes, so it stays taken."""
    made, empty = [], torch.empty

    def recorded(*a, **kw):
        t = empty(*a, **kw)
        made.append(weakref.ref(t))
        return t

    segments = [{"address": 0, "total_size": 16, "segment_pool_id": (5, 0)},
                {"address": 16, "total_size": 2 ** 63, "segment_pool_id": pool}]
    like = empty(0)
    monkeypatch.setattr(torch, "empty", recorded)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    monkeypatch.setattr(torch.cuda, "get_allocator_backend", lambda: "native")
    monkeypatch.setattr(torch.cuda, "memory_snapshot", lambda *a: segments)
    monkeypatch.setattr(api, "_captured_workspaces", [], raising=False)
    for _ in range(2):
        api._with_workspace(lambda *a: None, (), lambda: 1000, like, "kind", 1)
    assert [r() is not None for r in made] == [kept, kept]


def test_an_outgrown_workspace_is_given_back(monkeypatch, host_calls):
    made, empty = [], torch.empty

    def recorded(*a, **kw):
        t = empty(*a, **kw)
        made.append(weakref.ref(t))
        return t

    monkeypatch.setattr(torch, "empty", recorded)
    for nbytes in (1000, 2000, 1500, 3000):
        host_calls(lambda ws: None, nbytes)
    assert [r() is not None for r in made] == [False, False, True]


def test_smoke_weight_gradient():
    """The smoke run's value is that of the tests' 64-bit backward, and its limit takes what
    fp32 gives for any inputs and refuses a gradient that lacks a row."""
    T, H, lim = 40, 4, 2.0 ** -16
    f = 1e6 ** (-torch.arange(32, dtype=torch.float64) / 32)
    pos = torch.arange(700, 700 + T, dtype=torch.int32)
    for seed in range(50):
        gen = torch.Generator().manual_seed(seed)
        x = torch.randn(T, H, 128, generator=gen).to(torch.bfloat16)
        dy = torch.randn(T, H, 128, generator=gen)
        want, size = entry.norm_weight_gradient(x, dy, pos, f, 1e-6)
        ref = qo.bwd(qo.f64(x), qo.f64(dy), 1.0, 0.0, 1e-6, pos[None].numpy(), f.numpy(), None, False)[2]
        assert abs(want.numpy() - ref).max() <= 1e-12 * float(size.max())

        def error(dw):
            return float(((dw.double() - want).abs() / size).max())

        r = torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)
        a = (pos.double()[:, None] * f)[:, None]
        c, s = a.cos().float(), a.sin().float()
        g = torch.cat([dy[..., :32] * c + dy[..., 32:64] * s, dy[..., 32:64] * c - dy[..., :32] * s,
                       dy[..., 64:]], -1)
        terms = g * (x.float() * r)
        assert error(terms.sum((0, 1))) <= lim
        terms[seed % T, seed % H] = 0
        assert error(terms.sum((0, 1))) > lim


def test_extend_by_member_refuses():
    if not os.path.exists(B.LIB_PATH):
        from response_replay_gb300 import build
        build.build()
    lib, A = B.lib(), 1 << 20
    base = dict(table=A, members=4, max_blocks=8, ps=64, pages=100, lens=A, add=A, free=A, nfree=50,
                used=A, pos0=0, axes=1, rows=2, slots=A, pos=A, lo=A, uo=A)
    for kw, want in [
        (dict(rows=0), B.LS_ERR_INVALID_ARG), (dict(rows=-3), B.LS_ERR_INVALID_ARG),
        (dict(members=-1), B.LS_ERR_INVALID_ARG), (dict(members=1025), B.LS_ERR_UNSUPPORTED),
        (dict(rows=2 ** 29), B.LS_ERR_UNSUPPORTED), (dict(members=1024, rows=2 ** 30), B.LS_ERR_UNSUPPORTED),
        (dict(ps=8), B.LS_ERR_UNSUPPORTED), (dict(slots=None), B.LS_ERR_INVALID_ARG),
        (dict(slots=A + 4), B.LS_ERR_INVALID_ARG), (dict(pos=A + 8), B.LS_ERR_INVALID_ARG),
        (dict(lens=None), B.LS_ERR_INVALID_ARG), (dict(axes=0), B.LS_ERR_INVALID_ARG),
    ]:
        assert lib.ls_extend_pages_by_member(*{**base, **kw}.values(), None) == want, kw
    assert lib.ls_extend_pages_by_member(*{**base, "members": 0}.values(), None) == B.LS_OK


@pytest.mark.parametrize("eps", [3.1e38, float("inf"), float("nan"), 0.0, 1e-39, -1.0])
def test_eps_refused(eps):
    """3e38 and the largest mean of squares that fit fp32 have a sum in fp32."""
    lib, A = B.lib(), 1 << 20
    view = B.ls_qkv_view(A, A, A, *(4096, 128) * 3)
    norm = B.ls_qk_norm(A, A, B.LS_FP32, 0.0, eps)
    assert lib.ls_qk_norm_rope_fwd(view, 4, 8, 4, norm, None, None, view, None) == B.LS_ERR_INVALID_ARG


@pytest.mark.parametrize("backend,graph", [("cudaMallocAsync", True), ("pluggable", False)])
def test_captured_workspaces_of_other_allocators(monkeypatch, backend, graph):
    """The stream-ordered allocator's memory is the graph's; one that keeps no record of its
    segments is taken not to have pools."""
    def none(*a):
        raise RuntimeError("no snapshot")

    monkeypatch.setattr(torch.cuda, "get_allocator_backend", lambda: backend)
    monkeypatch.setattr(torch.cuda, "memory_snapshot", none)
    assert api._graph_memory(torch.empty(1)) is graph


@pytest.mark.parametrize("pos0", [-2 ** 31 - 1, 2 ** 31, 2 ** 32 + 7])
def test_positions_past_an_int_are_refused(pos0):
    with pytest.raises(ValueError, match="pos0"):
        api.extend_pages(None, None, pos0, None)


def test_a_call_within_a_call_does_not_wait_for_itself(host_calls):
    """A finalizer or a signal handler that calls while the same thread is between a call's
    lookup and its launch."""
    done = []

    def body(i):
        host_calls(lambda ws: host_calls(lambda inner: done.append(inner), 5000), 1000)

    t = threading.Thread(target=body, args=(0,), daemon=True)
    t.start()
    t.join(10)
    assert not t.is_alive() and len(done) == 1
