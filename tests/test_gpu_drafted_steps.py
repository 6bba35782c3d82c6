"""Steps over drafted trees as LayeredResponses runs them: members that have ended, and steps in CUDA
graphs."""
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


def chains(M, n):
    return np.broadcast_to(np.arange(n) - 1, (M, n))


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

    def lens(self):
        return self.rs.alloc.lens.cpu().numpy()


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
