"""GPU parity of ls_extend_pages: pages, slots and positions of growing responses."""
import numpy as np
import pytest
import torch

import qk_oracle as qo
from response_replay_gb300 import binding as B
from response_replay_gb300 import torch_api as api

pytestmark = pytest.mark.gpu


def i32(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


class Case:
    def __init__(self, dev, lens, add, ps, max_blocks=None, spare=5, capacity=None, axes=1, pos0=100,
                 seed=0):
        rng = np.random.default_rng(seed)
        lens, add = np.asarray(lens, np.int64), np.asarray(add, np.int64)
        have = np.where(lens > 0, -(-lens // ps), 0)
        need = np.where(lens >= 0, -(-np.maximum(lens + add, 0) // ps), 0)
        mb = int(max(need.max(initial=0), have.max(initial=0), 1)) + 1 if max_blocks is None else max_blocks
        n = int(have.sum() + np.maximum(need - have, 0).sum()) + spare
        free = rng.permutation(max(n, 1))[:n]
        used, table = 0, np.full((len(lens), mb), -7, np.int64)
        for m, h in enumerate(have):
            for b in range(min(h, mb)):
                table[m, b] = free[used]
                used += 1
        self.np = (table.astype(np.int32), lens.astype(np.int32), add.astype(np.int32),
                   free.astype(np.int32), used)
        self.ps, self.pos0, self.axes = ps, pos0, axes
        self.cap = int(add.clip(0).sum()) + 3 if capacity is None else capacity
        self.alloc = api.PageAllocator(i32(table, dev), i32(lens, dev), i32(free, dev),
                                       i32([used], dev), ps)
        self.add = i32(add, dev)
        self.slots = torch.full((self.cap,), 99, dtype=torch.int32, device=dev)
        self.pos = torch.full((axes, self.cap), 99, dtype=torch.int32, device=dev)

    def ref(self):
        t, lens, add, free, used = self.np
        return qo.extend(t, lens, add, free, used, self.ps, self.pos0, self.axes, self.cap)

    def check(self, in_place):
        a = self.alloc
        lo, uo = (None, None) if in_place else (torch.empty_like(a.lens), torch.empty_like(a.used))
        api.extend_pages(a, self.add, self.pos0, self.slots, self.pos, lens_out=lo, used_out=uo)
        err = B.ls_last_device_error(0)
        lo, uo = (a.lens, a.used) if in_place else (lo, uo)
        ref = self.ref()
        got = [x.cpu().numpy() for x in (self.slots, self.pos, a.block_table, lo, uo)]
        if ref is None:
            assert err == B.LS_ERR_DEVICE_CHECK
            assert (got[0] == -1).all() and (got[1] == 0).all()
            for x, y in zip(got[2:], (self.np[0], self.np[1], [self.np[4]])):
                np.testing.assert_array_equal(x, y)
            return
        assert err == B.LS_OK
        for x, y in zip(got, (*ref[:4], [ref[4]])):
            np.testing.assert_array_equal(x, y)
        if not in_place:
            np.testing.assert_array_equal(a.lens.cpu().numpy(), self.np[1])
            assert int(a.used) == self.np[4]


R = np.random.default_rng(5)
CASES = {
    "one token": ([0], [1], 16),
    "nothing": ([5, 0, 16], [0, 0, 0], 16),
    "page edges": ([15, 16, 17, 0, 31, 32], [1, 1, 1, 16, 2, 0], 16),
    "decode step": (list(R.integers(0, 5000, 8)), [1] * 8, 64),
    "out of use": ([-1, 20, -5, 0], [0, 3, 0, 40], 32),
    "empty members": ([0, 0, 0, 0], [0, 70, 0, 1], 64),
    "several blocks": (list(R.integers(0, 300, 64)), list(R.integers(0, 2000, 64)), 64),
    "all threads": (list(R.integers(0, 40, 1024)), list(R.integers(0, 40, 1024)), 16),
    "large pages": (list(R.integers(0, 9000, 3)), [20000, 1, 4096], 4096),
}


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("name", CASES)
def test_extend(cuda, name, in_place):
    lens, add, ps = CASES[name]
    Case(cuda, lens, add, ps, axes=1 + len(name) % 3).check(in_place)


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("kw", [
    dict(lens=[3, 4], add=[1, -1], ps=16),                          # a negative count
    dict(lens=[3, -1], add=[1, 2], ps=16),                          # a member out of use grows
    dict(lens=[3, 60], add=[1, 10], ps=16, max_blocks=4),           # a full row of the table
    dict(lens=[30, 60], add=[40, 10], ps=16, spare=-1),             # the free list ends
    dict(lens=[30, 60], add=[40, 10], ps=16, capacity=49),          # more tokens than slots
    dict(lens=[3, 4], add=[2 ** 31 - 1, 2 ** 31 - 1], ps=16, max_blocks=4, capacity=64),
    dict(lens=[0] * 9, add=[4000] * 9, ps=16, spare=-1),            # as above, several blocks
])
def test_refused_whole(cuda, kw, in_place):
    if kw["add"][0] == 2 ** 31 - 1:
        c = Case(cuda, kw["lens"], [0, 0], kw["ps"], max_blocks=4, capacity=64)
        c.add.fill_(2 ** 31 - 1)
        c.np = (*c.np[:2], np.full(2, 2 ** 31 - 1, np.int32), *c.np[3:])
    else:
        c = Case(cuda, **kw)
    assert c.ref() is None
    c.check(in_place)


def test_exact_fit(cuda):
    Case(cuda, [16, 3], [16, 13], 16, max_blocks=2, spare=0, capacity=29).check(True)
    Case(cuda, [1] * 300, [40] * 300, 16, spare=0, capacity=12000).check(True)


def test_bad_page_ids_give_no_slot(cuda):
    c = Case(cuda, [10, 0], [10, 5], 16)
    c.alloc.block_table[0, 0] = 1000
    c.alloc.free_list[c.np[4]] = -4
    api.extend_pages(c.alloc, c.add, 0, c.slots, c.pos)
    assert B.ls_last_device_error(0) == B.LS_ERR_DEVICE_CHECK
    s = c.slots.cpu().numpy()
    assert (s[:10] == -1).all() and (s[10:15] >= 0).all() and (s[15:] == -1).all()


def test_steps_in_a_graph(cuda):
    """A captured step in place: every replay grows the responses by one token."""
    a = api.PageAllocator.empty(3, 8, 24, 16, cuda)
    add = torch.ones(3, dtype=torch.int32, device=cuda)
    slots = torch.empty(4, dtype=torch.int32, device=cuda)
    pos = torch.empty((1, 4), dtype=torch.int32, device=cuda)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(st):
        api.extend_pages(a, add, 7, slots, pos)
    st.synchronize()
    with torch.cuda.graph(g, stream=st):
        api.extend_pages(a, add, 7, slots, pos)
    seen = [slots.tolist()]
    for _ in range(39):
        g.replay()
        seen.append(slots.tolist())
    assert a.lens.tolist() == [40, 40, 40] and int(a.used) == 9
    assert pos.tolist() == [[46, 46, 46, 0]] and all(s[3] == -1 for s in seen)
    flat = [x for s in seen for x in s[:3]]
    assert len(set(flat)) == 120 and B.ls_last_device_error(0) == B.LS_OK


def test_no_members_and_lengths_over_the_counts(cuda):
    """Nothing to extend still fills the outputs; lens_out may lie over add."""
    Case(cuda, [], [], 16, capacity=0).check(False)
    Case(cuda, [], [], 16, capacity=9).check(False)
    lens, add = list(range(64)), [90 + i for i in range(64)]  # several blocks
    c, ref = Case(cuda, lens, add, 16), Case(cuda, lens, add, 16)
    api.extend_pages(ref.alloc, ref.add, 3, ref.slots, ref.pos)
    used = torch.empty_like(c.alloc.used)
    api.extend_pages(c.alloc, c.add, 3, c.slots, c.pos, lens_out=c.add, used_out=used)
    assert torch.equal(c.slots, ref.slots) and torch.equal(c.pos, ref.pos)
    assert torch.equal(c.add, ref.alloc.lens) and torch.equal(used, ref.alloc.used)
    assert c.alloc.lens.tolist() == lens and B.ls_last_device_error(0) == B.LS_OK
