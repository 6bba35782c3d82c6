"""GPU parity of pages given back and shared: trim_pages, fork_pages, copy_pages, alone and as a
rollout with branches runs them."""
import numpy as np
import pytest
import torch

import rollout_oracle as ro
from response_replay_gb300 import binding as B
from response_replay_gb300 import layers
from response_replay_gb300 import torch_api as api

pytestmark = pytest.mark.gpu


def i32(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


class Pages:
    """Members' pages, some of them branches of earlier members, on the host and on the GPU."""

    def __init__(self, rng, M, ps, top, branches=0.0, spare=6, empty=0.2):
        self.ps, self.M = ps, M
        nb = -(-top // ps) + 1
        lens = rng.integers(0, top + 1, M)
        lens[rng.random(M) < empty] = -1
        num = M * nb + spare
        free = rng.permutation(num)
        table = np.full((M, nb), -9)
        shared = np.zeros(num, int)
        used = 0
        for m in range(M):
            olds = [s for s in range(m) if lens[s] > 0]
            if lens[m] > 0 and olds and rng.random() < branches:
                s = int(rng.choice(olds))
                lens[m] = rng.integers(1, lens[s] + 1)
                whole = lens[m] // ps
                table[m, :whole] = table[s, :whole]
                for p in table[s, :whole]:
                    shared[p] += 1
            else:
                whole = 0
            for b in range(whole, ro.pages_of(lens[m], ps)):
                table[m, b] = free[used]
                used += 1
        self.table, self.lens, self.free, self.used, self.shared, self.num = table, lens, free, used, shared, num

    def on(self, dev, sharing=True):
        return api.PageAllocator(i32(self.table, dev), i32(self.lens, dev), i32(self.free, dev),
                                 i32([self.used], dev), self.ps, shared=i32(self.shared, dev) if sharing else None)

    def same(self, alloc):
        for t, x in ((alloc.block_table, self.table), (alloc.lens, self.lens), (alloc.free_list, self.free),
                     (alloc.used, [self.used])):
            np.testing.assert_array_equal(t.cpu().numpy(), x)
        if alloc.shared is not None:
            np.testing.assert_array_equal(alloc.shared.cpu().numpy(), self.shared)

    def trim(self, new, sharing=True):
        r = ro.trim(self.table, self.lens, new, self.free, self.used, self.shared if sharing else None,
                    self.ps, self.num)
        if r is not None:
            self.lens, self.free, self.used = r[:3]
            if sharing:
                self.shared = r[3]
        return r is not None

    def fork(self, src, keep):
        r = ro.fork(self.table, self.lens, src, keep, self.free, self.used, self.shared, self.ps, self.num)
        if r is not None:
            self.table, self.lens, self.used, self.shared = r[:4]
        return None if r is None else r[4]


def shorter(rng, pages, p_out=0.3):
    """New lengths that do not end inside a shared page."""
    new = np.array([x if x < 0 else rng.integers(0, x + 1) for x in pages.lens])
    for m, (x, y) in enumerate(zip(pages.lens, new)):
        if 0 < y < x and y % pages.ps and pages.shared[pages.table[m, y // pages.ps]]:
            new[m] = y // pages.ps * pages.ps
    new[(rng.random(len(new)) < p_out) & (new >= 0)] = -1
    return new


@pytest.mark.parametrize("M,ps,top,branches,sharing", [
    (1, 16, 100, 0, False), (8, 16, 300, 0, False), (8, 16, 300, 0.6, True), (64, 64, 4096, 0.7, True),
    (1024, 16, 40, 0.8, True), (30, 16, 3000, 0.9, True), (200, 32, 700, 0, False), (5, 4096, 9000, 0.5, True)])
def test_trim(cuda, M, ps, top, branches, sharing):
    rng = np.random.default_rng(M + top)
    pages = Pages(rng, M, ps, top, branches)
    alloc = pages.on(cuda, sharing)
    for step in range(3):
        new = shorter(rng, pages)
        if step == 0:  # outputs apart
            lo, uo = torch.zeros_like(alloc.lens), torch.zeros_like(alloc.used)
            was = [alloc.lens.clone(), alloc.used.clone()]
            api.trim_pages(alloc, i32(new, cuda), lens_out=lo, used_out=uo)
            assert torch.equal(alloc.lens, was[0]) and torch.equal(alloc.used, was[1])
            alloc.lens.copy_(lo)
            alloc.used.copy_(uo)
        else:
            api.trim_pages(alloc, i32(new, cuda))
        assert B.ls_last_device_error(0) == B.LS_OK
        assert pages.trim(new, sharing)
        pages.same(alloc)


def test_trim_refuses(cuda):
    """Nothing changes when any member's new length, page or owner count is not what it can be."""
    rng = np.random.default_rng(3)
    for case in range(7):
        pages = Pages(rng, 12, 16, 200, 0.7, empty=0.0)
        new = np.maximum(shorter(rng, pages, p_out=0.5), -1)
        shared = np.flatnonzero(pages.shared)
        holders = [(m, b) for p in shared for m, b in zip(*np.nonzero(pages.table == p))
                   if b * 16 < pages.lens[m]]
        if case == 0:
            new[4] = pages.lens[4] + 1
        elif case == 1:
            pages.lens[5] = -1
            new[5] = 0
        elif case == 2:
            new[:] = -1
            pages.table[7, 0] = pages.num
        elif case == 3:  # a page with more owners than are counted
            new[:] = -1
            pages.shared[shared[0]] -= 1
        elif case == 4:
            new[:] = -1
            pages.used = 2
        elif case == 5:  # inside a page that another member holds
            m, b = holders[-1]
            new = pages.lens.copy()
            new[m] = b * 16 + 5
        else:
            new[:] = pages.lens
            pages.lens[2] = 16 * pages.table.shape[1] + 1
        alloc = pages.on(cuda)
        api.trim_pages(alloc, i32(new, cuda))
        assert B.ls_last_device_error(0) == B.LS_ERR_DEVICE_CHECK, case
        assert not pages.trim(new), case
        pages.same(alloc)


@pytest.mark.parametrize("M,ps,top", [(2, 16, 50), (8, 16, 300), (64, 64, 4096), (1024, 16, 60), (7, 4096, 20000)])
def test_fork(cuda, M, ps, top):
    rng = np.random.default_rng(M + ps)
    pages = Pages(rng, M, ps, top, 0.3, spare=M + 4, empty=0.6)
    pages.lens[0] = max(pages.lens[0], -1)
    alloc = pages.on(cuda)
    for step in range(3):
        live, out = np.flatnonzero(pages.lens > 0), np.flatnonzero(pages.lens <= 0)
        if len(live) == 0:
            pages = Pages(rng, M, ps, top, 0, spare=M + 4, empty=0)
            pages.lens[1:][rng.random(M - 1) < 0.5] = -1
            alloc = pages.on(cuda)
            continue
        src, keep = np.full(M, -1), np.zeros(M, int)
        for m in out[rng.random(len(out)) < 0.5]:
            src[m] = rng.choice(live)
            n = pages.lens[src[m]]
            keep[m] = [n, 0, n // ps * ps, rng.integers(0, n + 1)][rng.integers(0, 4)]
        copies = api.fork_pages(alloc, i32(src, cuda), i32(keep, cuda) if step else None)
        err = B.ls_last_device_error(0)
        want = pages.fork(src, keep if step else None)
        if want is None:
            assert err == B.LS_ERR_DEVICE_CHECK
            assert copies.tolist() == [[-1] * M, [-1] * M, [0] * M]
        else:
            assert err == B.LS_OK
            np.testing.assert_array_equal(copies.cpu().numpy(), want)
        pages.same(alloc)


def test_fork_refuses(cuda):
    rng = np.random.default_rng(8)
    for case in range(7):
        pages = Pages(rng, 6, 16, 100, 0, empty=0)
        pages.lens[:] = [90, 50, -1, -1, 0, 33]
        for m in (0, 1, 5):
            pages.table[m, :ro.pages_of(pages.lens[m], 16)] = pages.free[10 * m:10 * m + ro.pages_of(pages.lens[m], 16)]
        pages.used = 20
        src, keep = np.array([-1, -1, 0, 1, 0, -1]), np.array([0, 0, 40, 50, 7, 0])
        good = case == 6
        if case == 0:
            keep[3] = 51
        elif case == 1:
            src[3] = 2          # a branch of this call
        elif case == 2:
            src[5] = 0          # in use
        elif case == 3:
            src[2] = 6
        elif case == 4:
            pages.used = len(pages.free) - 2
        elif case == 5:
            pages.table[0, 1] = -1
        alloc = pages.on(cuda)
        api.fork_pages(alloc, i32(src, cuda), i32(keep, cuda))
        assert (B.ls_last_device_error(0) == B.LS_OK) == good, case
        assert (pages.fork(src, keep) is not None) == good, case
        pages.same(alloc)


@pytest.mark.parametrize("L,hkv,ps,count", [(1, 1, 16, 1), (3, 2, 64, 5), (2, 4, 256, 3), (1, 1, 4096, 2), (5, 3, 32, 60)])
def test_copy(cuda, L, hkv, ps, count):
    rng = np.random.default_rng(ps)
    pages = 2 * count + 3
    k = torch.randn(L, pages, hkv, ps, 128, device=cuda).to(torch.bfloat16)
    v = torch.randn_like(k)
    ids = rng.permutation(pages)
    pairs = np.stack([ids[:count], ids[count:2 * count], rng.integers(0, ps + 1, count)])
    pairs[2, 0] = ps
    if count > 2:
        pairs[:, 1] = -1, -1, 0
        pairs[2, 2] = 0
    want = []
    for x in (k, v):
        y = x.clone()
        for f, t, n in pairs.T:
            if f >= 0:
                y[:, t, :, :n] = x[:, f, :, :n]
        want.append(y)
    api.copy_pages(api.LayerPools(k, v), i32(pairs, cuda))
    assert B.ls_last_device_error(0) == B.LS_OK
    assert torch.equal(k, want[0]) and torch.equal(v, want[1])
    for bad in ([0, pages, 1], [-1, 2, 1], [0, 1, ps + 1], [pages, 0, 0], [0, 1, -1]):
        api.copy_pages(api.LayerPools(k, v), i32(np.array(bad)[:, None], cuda))
        assert B.ls_last_device_error(0) == B.LS_ERR_DEVICE_CHECK
        assert torch.equal(k, want[0])


def test_pools_past_32_bits(cuda):
    """A copy and a move in a pool of more than 2^32 bytes a layer, and two layers."""
    hkv, ps, pages, L = 8, 64, 33000, 2
    k = torch.zeros(L, pages, hkv, ps, 128, dtype=torch.bfloat16, device=cuda)
    v = torch.zeros_like(k)
    assert k[0].numel() * 2 > 2 ** 32
    k[:, pages - 1] = torch.randn(L, hkv, ps, 128, device=cuda).to(torch.bfloat16)
    pools = api.LayerPools(k, v)
    api.copy_pages(pools, i32([[pages - 1], [pages - 2], [ps]], cuda))
    assert torch.equal(k[:, pages - 1], k[:, pages - 2])
    alloc = api.PageAllocator(i32([[pages - 1]], cuda), i32([40], cuda), i32([0], cuda), i32([0], cuda), ps,
                              num_pages=pages)
    was = k[:, pages - 1].clone()
    api.compact_rows(alloc, pools, i32([[0, 3, 6, -1, -1, -1, -1, -1]], cuda), i32([3], cuda))
    assert B.ls_last_device_error(0) == B.LS_OK
    assert torch.equal(k[:, pages - 1, :, 33], was[:, :, 35]) and torch.equal(k[:, pages - 1, :, 34], was[:, :, 38])
    assert torch.equal(k[:, pages - 2], was)


def test_branches_grow_apart(cuda):
    """A response branched at three places and pruned again, in two layers: every member reads
    its own tokens, whatever the others write, and in the end every page is free."""
    dev, L, M, hkv, hq, ps = cuda, 2, 5, 2, 4, 16
    table = torch.zeros(0, dtype=torch.int32, device=dev)
    prompt = layers.LayeredKVCache(L, 1, table, ps, hkv, 0)
    resp = layers.LayeredResponses(prompt, hkv, M, 200, 40, ps, dev, capacity=300, sharing=True)
    resp.alloc.lens.copy_(i32([0, 0, -1, -1, -1], dev))
    resp.k_pools.fill_(float("nan"))
    resp.v_pools.fill_(float("nan"))
    rng = np.random.default_rng(2)
    kept = [[np.zeros((0, hkv, 128)) for _ in range(L)] for _ in range(M)]

    def grow(add):
        resp.extend(i32(add, dev))
        for l in range(L):
            rows = torch.randn(300, hkv, 128, device=dev).to(torch.bfloat16)
            resp.append(l, torch.zeros(300, hq, 128, dtype=torch.bfloat16, device=dev), rows, rows, None,
                        norm=False)
            at = 0
            for m, n in enumerate(add):
                kept[m][l] = np.concatenate([kept[m][l], rows[at:at + n].double().cpu().numpy()])
                at += n

    def check():
        assert B.ls_last_device_error(0) == B.LS_OK
        lens = resp.alloc.lens.tolist()
        for m in range(M):
            if lens[m] < 0:
                continue
            for l in range(L):
                assert len(kept[m][l]) == lens[m]
                t = torch.arange(lens[m], device=dev)
                page = resp.alloc.block_table[m, t // ps].long()
                for pools in (resp.k_pools, resp.v_pools):
                    np.testing.assert_array_equal(pools[l][page, :, t % ps].double().cpu().numpy(), kept[m][l])

    grow([100, 37, 0, 0, 0])
    check()
    resp.fork(i32([-1, -1, 0, 0, 1], dev), i32([0, 0, 100, 53, 16], dev))
    for m, (s, n) in {2: (0, 100), 3: (0, 53), 4: (1, 16)}.items():
        kept[m] = [x[:n] for x in kept[s]]
    check()
    for _ in range(3):
        grow(list(rng.integers(0, 20, M)))
        check()
    resp.trim(i32([-1, len(kept[1][0]), 100, 60, 16], dev))  # the first one's branches live on
    kept[2], kept[3], kept[4] = ([x[:n] for x in kept[m]] for m, n in ((2, 100), (3, 60), (4, 16)))
    check()
    grow([0, 5, 9, 30, 40])
    check()
    resp.trim(i32([-1] * M, dev))
    assert B.ls_last_device_error(0) == B.LS_OK
    assert int(resp.alloc.used) == 0 and bool((resp.alloc.shared == 0).all())
    assert sorted(resp.alloc.free_list.tolist()) == list(range(40))


def test_graph_of_a_step(cuda):
    """Prune and branch as one captured graph, replayed as the lengths change."""
    rng = np.random.default_rng(5)
    pages = Pages(rng, 8, 16, 200, 0, spare=40, empty=0)
    pages.lens[4:] = -1
    alloc = pages.on(cuda)
    k = torch.randn(2, pages.num, 1, 16, 128, device=cuda).to(torch.bfloat16)
    v = torch.randn_like(k)
    pools = api.LayerPools(k, v)
    new, src, keep = i32(pages.lens, cuda), i32(np.full(8, -1), cuda), i32(np.zeros(8), cuda)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            api.trim_pages(alloc, new)
            copies = api.fork_pages(alloc, src, keep)
            api.copy_pages(pools, copies)
    torch.cuda.current_stream().wait_stream(side)
    pages.same(alloc)
    for step in range(4):
        n = pages.lens.copy()
        n[4:] = -1
        s, c = np.full(8, -1), np.zeros(8, int)
        for m in range(4, 8):
            s[m] = rng.integers(0, 4)
            c[m] = rng.integers(0, max(pages.lens[s[m]], 0) + 1)
        new.copy_(i32(n, cuda))
        src.copy_(i32(s, cuda))
        keep.copy_(i32(c, cuda))
        was = k.clone()
        graph.replay()
        assert B.ls_last_device_error(0) == B.LS_OK
        assert pages.trim(n)
        want = pages.fork(s, c)
        np.testing.assert_array_equal(copies.cpu().numpy(), want)
        pages.same(alloc)
        for f, t, r in want.T:
            if f >= 0:
                was[:, t, :, :r] = was[:, f, :, :r]
        assert torch.equal(k, was)
