"""GPU parity of ls_extend_drafts with ls_extend_pages_by_member, and what it says each member got."""
import numpy as np
import pytest
import torch

from response_replay_gb300 import binding as B
from response_replay_gb300 import torch_api as api

pytestmark = pytest.mark.gpu


def i32(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


def group(dev, rng, M, ps, top, spare, rows):
    lens = rng.integers(0, top + 1, M)
    lens[rng.random(M) < 0.25] = -1
    have = -(-np.maximum(lens, 0) // ps)
    nb = -(-(top + rows) // ps)
    free = rng.permutation(int(have.sum()) + spare)
    table = np.full((M, nb), -7)
    at = 0
    for m in range(M):
        table[m, :have[m]] = free[at:at + have[m]]
        at += have[m]
    return lens, lambda: api.PageAllocator(i32(table, dev), i32(lens, dev), i32(free, dev), i32([at], dev), ps)


# one block and several, a member and the most, no page to spare, in place and apart
@pytest.mark.parametrize("M,rows,ps,top,spare", [(1, 1, 16, 20, 4), (8, 16, 64, 300, 20), (64, 40, 16, 100, 400),
                                                 (64, 128, 16, 100, 700), (1024, 5, 16, 60, 3000), (12, 7, 32, 90, 0)])
@pytest.mark.parametrize("counts", [True, False])
@pytest.mark.parametrize("apart", [True, False])
def test_drafts_get_what_members_do(cuda, M, rows, ps, top, spare, counts, apart):
    rng = np.random.default_rng(M * rows + spare)
    lens, make = group(cuda, rng, M, ps, top, spare, rows)
    add = np.where(lens < 0, 0, rng.integers(0, rows + 1, M) if counts else rows)
    res = []
    for drafts in (False, True):
        alloc = make()
        slots = torch.full((M * rows,), 5, dtype=torch.int32, device=cuda)
        pos = torch.full((2, M * rows), 5, dtype=torch.int32, device=cuda)
        added = torch.full((M,), 77, dtype=torch.int32, device=cuda)
        lo, uo = (torch.zeros_like(alloc.lens), torch.zeros_like(alloc.used)) if apart else (None, None)
        kw = dict(member_rows=rows, lens_out=lo, used_out=uo)
        if drafts:
            api.extend_pages(alloc, i32(add, cuda) if counts else None, 1000, slots, pos, added=added, **kw)
        else:
            api.extend_pages(alloc, i32(add, cuda), 1000, slots, pos, **kw)
        err = B.ls_last_device_error(0)
        res.append((err, added, [alloc.block_table, alloc.lens, alloc.used, slots, pos] + ([lo, uo] if apart else [])))
    assert res[0][0] == res[1][0] == (B.LS_OK if spare else B.LS_ERR_DEVICE_CHECK)
    assert all(torch.equal(a, b) for a, b in zip(res[0][2], res[1][2]))
    np.testing.assert_array_equal(res[1][1].cpu().numpy(), add if spare else 0 * add)


def test_refusals(cuda):
    rng = np.random.default_rng(1)
    lens, make = group(cuda, rng, 4, 16, 50, 9, 3)
    alloc = make()
    slots = torch.zeros(12, dtype=torch.int32, device=cuda)
    added = torch.zeros(4, dtype=torch.int32, device=cuda)
    add = torch.zeros(4, dtype=torch.int32, device=cuda)
    for bad in (dict(add=None), dict(add=add, added=added), dict(add=None, member_rows=3, added=added[:3]),
                dict(add=None, member_rows=3, added=added.long())):
        with pytest.raises(ValueError):
            api.extend_pages(alloc, bad.pop("add"), 0, slots, **bad)
    # counts that no member can have: nobody gets anything
    for bad in ([4, 0, 0, 0], [-1, 0, 0, 0]):
        added.fill_(77)
        api.extend_pages(alloc, i32(bad, cuda), 0, slots, member_rows=3, added=added)
        assert B.ls_last_device_error(0) == B.LS_ERR_DEVICE_CHECK
        assert bool((added == 0).all()) and bool((slots == -1).all())
        np.testing.assert_array_equal(alloc.lens.cpu().numpy(), lens)
