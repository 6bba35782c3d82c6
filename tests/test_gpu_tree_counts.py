"""Drafts that are longer than their member or its rows: cut, in every call in the same way, and
reported by each."""
import numpy as np
import pytest
import torch

from response_replay_gb300 import binding as B
from response_replay_gb300 import torch_api as api
from test_gpu_tree import SCALE, Tree, i32

pytestmark = pytest.mark.gpu

# rows a tile and more; counts and none; a member shorter than its rows, an empty one
CASES = [
    ([3, 60, 0], None, 8, 8, 2), ([3, 60, 0], [8, 8, 8], 8, 8, 2), ([3, 60, 2], [5, 9, -2], 8, 8, 2),
    ([3, 60, 0] * 4, None, 16, 24, 2), ([3, 60, 5] * 4, [16, 20, 7] * 4, 16, 24, 2),
]


@pytest.mark.parametrize("lens,drafted,n,hq,hkv", CASES)
def test_attention_cuts_drafts(cuda, lens, drafted, n, hq, hkv):
    counts = [n] * len(lens) if drafted is None else drafted
    cut = [min(max(c, 0), n, x) for c, x in zip(counts, lens)]
    t = Tree(cuda, 100, lens, cut, n, hq, hkv, seed=n)
    if drafted is None:
        given = None
    else:
        given = i32(drafted, cuda)
    o = torch.full_like(t.q, 5.0)
    lse = torch.full(t.q.shape[:3], 6.0, device=cuda)
    api.decode_attn_tree(t.cache, t.resp, t.q, t.visible, SCALE, drafted=given, o=o, lse=lse)
    assert B.ls_last_device_error(0) == B.LS_ERR_DEVICE_CHECK
    t.check(o, lse)
    for m, c in enumerate(cut):
        assert bool((o[m, :n - c] == 5.0).all()) and bool((lse[m, :n - c] == 6.0).all()), m


@pytest.mark.parametrize("lens,drafted,n,hq,hkv", CASES)
def test_moves_report_cut_drafts(cuda, lens, drafted, n, hq, hkv):
    M, ps = len(lens), 16
    k = torch.randn(1, M * 4, 1, ps, 128, device=cuda).to(torch.bfloat16)
    v = torch.randn_like(k)
    k0, v0 = k.clone(), v.clone()
    alloc = api.PageAllocator(i32(np.arange(M * 4).reshape(M, 4), cuda), i32(lens, cuda), i32([0], cuda),
                              i32([0], cuda), ps, num_pages=M * 4)
    rows = torch.full((M, n), -1, dtype=torch.int32, device=cuda)
    api.compact_rows(alloc, api.LayerPools(k, v), rows, torch.zeros(M, dtype=torch.int32, device=cuda),
                     drafted=None if drafted is None else i32(drafted, cuda))
    assert B.ls_last_device_error(0) == B.LS_ERR_DEVICE_CHECK
    assert torch.equal(k, k0) and torch.equal(v, v0)
