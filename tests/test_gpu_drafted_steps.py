"""Steps over drafted trees as LayeredResponses runs them: members that have ended, extensions that
are refused, and steps in CUDA graphs."""
import numpy as np
import pytest
import torch

import rollout_oracle as ro
from response_replay_gb300 import binding as B
from response_replay_gb300 import layers
from response_replay_gb300 import torch_api as api

pytestmark = pytest.mark.gpu
L, HKV, HQ, PS, P = 2, 2, 4, 16, 40
SCALE = 128 ** -0.5


def i32(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


def normal(dev, seed, *s):
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    return torch.randn(*s, generator=g, device=dev).to(torch.bfloat16)


def chains(M, n, drafted=None):
    """Drafts without branches, of the last drafted[m] rows (default: all)."""
    p = np.tile(np.arange(n) - 1, (M, 1))
    if drafted is not None:
        p[p < n - np.minimum(drafted, n)[:, None]] = -1
    return p


class Group:
    """A captured prompt and a group that holds `lens` tokens (negative: out of use), their keys and
    values random."""

    def __init__(self, dev, n, lens, num_pages=40, max_tokens=200, sharing=False):
        self.dev, self.n, self.M = dev, n, len(lens)
        table = torch.arange(-(-P // PS), dtype=torch.int32, device=dev)
        self.prompt = layers.LayeredKVCache(L, table.numel(), table, PS, HKV, P)
        for l in range(L):
            self.prompt.capture(l, normal(dev, l, P, HKV, 128), normal(dev, 9 + l, P, HKV, 128))
        self.rs = rs = layers.LayeredResponses(self.prompt, HKV, self.M, max_tokens, num_pages, PS, dev,
                                               member_rows=n, sharing=sharing)
        rs.k_pools.copy_(normal(dev, 20, *rs.k_pools.shape))
        rs.v_pools.copy_(normal(dev, 21, *rs.v_pools.shape))
        left = np.maximum(lens, 0)
        while left.any():
            step = np.minimum(left, n)
            rs.extend(i32(step, dev))
            left = left - step
        rs.alloc.lens.copy_(i32(lens, dev))
        assert B.ls_last_device_error(0) == B.LS_OK

    def state(self):
        a = self.rs.alloc
        return [t.clone() for t in (a.block_table, a.lens, a.free_list, a.used, self.rs.k_pools, self.rs.v_pools)]

    def lens(self):
        return self.rs.alloc.lens.cpu().numpy()


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_first_draft_in_a_capture(cuda):
    """A step that is captured before any was run: the next one runs eagerly, before a replay."""
    n, lens = 5, np.array([17, 30, 4])
    g = Group(cuda, n, lens)
    parents = i32(chains(3, n), cuda)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = g.rs.draft(parents)
    np.testing.assert_array_equal(g.lens(), lens)
    for step in range(2):
        visible = g.rs.draft(parents) if step == 0 else captured
        if step == 1:
            graph.replay()
        assert B.ls_last_device_error(0) == B.LS_OK
        lens = lens + n
        np.testing.assert_array_equal(g.lens(), lens)
        _, words, pos = ro.draft_tree(chains(3, n), lens, None, P)
        np.testing.assert_array_equal(visible.cpu().numpy(), words)
        np.testing.assert_array_equal(g.rs.positions.view(3, n).cpu().numpy(), pos)
        assert bool((g.rs.slots >= 0).all())


def test_draft_of_every_row_with_ended_members(cuda):
    """Without counts the members in use draft every row, and those that have ended nothing."""
    n, lens = 4, np.array([9, -1, 33, -1, 0])
    g = Group(cuda, n, lens)
    parents = chains(5, n)
    visible = g.rs.draft(i32(parents, cuda))
    assert B.ls_last_device_error(0) == B.LS_OK
    new = np.where(lens < 0, lens, lens + n)
    np.testing.assert_array_equal(g.lens(), new)
    np.testing.assert_array_equal(g.rs.drafted.cpu().numpy(), np.where(lens < 0, 0, n))
    _, words, _ = ro.draft_tree(parents, new, None, P)
    np.testing.assert_array_equal(visible.cpu().numpy(), words)
    slots = g.rs.slots.view(5, n).cpu().numpy()
    assert (slots[lens < 0] == -1).all() and (slots[lens >= 0] >= 0).all()
    q = normal(cuda, 3, 5, n, HQ, 128)
    o = torch.full_like(q, 7.0)
    g.rs.attend(0, q, SCALE, o=o, visible=visible)
    assert bool((o[[1, 3]] == 7.0).all()) and not bool((o[[0, 2, 4]] == 7.0).any())
    tokens = i32(np.tile(np.arange(n), (5, 1)), cuda)
    rows, count, _ = g.rs.settle(i32(parents, cuda), tokens, tokens + 1)
    assert B.ls_last_device_error(0) == B.LS_OK
    np.testing.assert_array_equal(count.cpu().numpy(), np.where(lens < 0, 0, n))
    np.testing.assert_array_equal(g.lens(), new)


@pytest.mark.parametrize("why,counts", [("pages", True), ("pages", False), ("table", True), ("table", False),
                                        ("ended", True), ("rows", True)])
def test_refused_draft_leaves_the_responses_alone(cuda, why, counts):
    """No room for the drafts, a count that no member can have: the error is recorded, and nothing
    of the step, its acceptance included, touches a response."""
    n, lens = 6, np.array([30, 47, 16])
    if why == "ended":
        lens[1] = -1
    g = Group(cuda, n, lens, num_pages={"pages": 6}.get(why, 40), max_tokens={"table": 48}.get(why, 200))
    drafted = np.array([3, 6, n + 1 if why == "rows" else 6])
    d = i32(drafted, cuda) if counts else None
    was = g.state()
    parents = i32(chains(3, n, drafted if counts else None), cuda)
    visible = g.rs.draft(parents, d)
    assert B.ls_last_device_error(0) == B.LS_ERR_DEVICE_CHECK
    assert same(g.state(), was)
    assert bool((visible == 0).all()) and bool((g.rs.drafted == 0).all())
    x = normal(cuda, 5, 3 * n, HQ, 128)
    rot = api.Rotary.from_base(1e6, 128, cuda)
    o = torch.full((3, n, HQ, 128), 7.0, dtype=torch.bfloat16, device=cuda)
    for l in range(L):
        q = g.rs.append(l, x, x[:, :HKV].contiguous(), x[:, HKV:].contiguous(), rot)
        g.rs.attend(l, q.view(3, n, HQ, 128), SCALE, o=o, visible=visible, drafted=d)
    assert bool((o == 7.0).all())
    # choices that would take some rows and leave others
    tokens = np.tile(np.arange(n), (3, 1))
    chosen = tokens + 1
    chosen[:, 3] = 99
    rows, count, follow = g.rs.settle(parents, i32(tokens, cuda), i32(chosen, cuda), d)
    assert B.ls_last_device_error(0) == B.LS_OK
    assert bool((rows == -1).all()) and bool((count == 0).all()) and bool((follow == -1).all())
    assert same(g.state(), was)
    # and with room again the next step goes on
    out = np.full(3, -1)
    out[0] = lens[0]
    g.rs.trim(i32(out, cuda))
    add = np.array([2, 0, 0])
    g.rs.draft(i32(chains(3, n, add), cuda), i32(add, cuda))
    assert B.ls_last_device_error(0) == B.LS_OK
    np.testing.assert_array_equal(g.lens(), [32, -1, -1])


@pytest.mark.parametrize("counts", [True, False])
def test_steps_in_a_graph_are_the_eager_ones(cuda, counts):
    """A whole step (room, plan, both layers' keys and attention, acceptance) captured once, replayed
    with other trees, counts and choices, members ending between: state and outputs of the same
    steps run eagerly."""
    n, lens, dev = 6, np.array([20, 3, 0, 41]), cuda
    M, vocab = 4, 6
    rng = np.random.default_rng(3)
    groups = [Group(dev, n, lens, sharing=True) for _ in range(2)]
    rot = api.Rotary.from_base(1e6, 128, dev)
    emb = [[normal(dev, 50 + 3 * l + i, vocab, h, 128) for i, h in enumerate((HQ, HKV, HKV))] for l in range(L)]
    parents, tokens, chosen = (torch.zeros(M, n, dtype=torch.int32, device=dev) for _ in range(3))
    drafted = torch.zeros(M, dtype=torch.int32, device=dev)
    d = drafted if counts else None

    def step(rs, o):
        visible = rs.draft(parents, d)
        for l in range(L):
            q, k, v = (e[tokens.view(-1).long()] for e in emb[l])
            q = rs.append(l, q, k, v, rot)
            rs.attend(l, q.view(M, n, HQ, 128), SCALE, o=o[l], visible=visible)
        return rs.settle(parents, tokens, chosen)

    outs = [torch.zeros(L, M, n, HQ, 128, dtype=torch.bfloat16, device=dev) for _ in range(2)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(groups[0].rs, outs[0])
    for s in range(5):
        live = groups[1].lens() >= 0
        c = np.where(live, rng.integers(0, n + 1, M), 0) if counts else np.full(M, n)
        p = np.full((M, n), -1)
        for m in range(M):
            for r in range(n - c[m] + 1, n):
                p[m, r] = rng.integers(n - c[m], r)
        for t, x in ((parents, p), (drafted, c), (tokens, rng.integers(0, vocab, (M, n))),
                     (chosen, rng.integers(0, vocab, (M, n)))):
            t.copy_(i32(x, dev))
        for o in outs:
            o.zero_()
        graph.replay()
        want = step(groups[1].rs, outs[1])
        assert B.ls_last_device_error(0) == B.LS_OK
        assert same(got, want) and torch.equal(*outs)
        assert same(groups[0].state(), groups[1].state())
        if s == 2:
            for g in groups:
                end = g.rs.alloc.lens.clone()
                end[1] = -1
                g.rs.trim(end)
