"""GPU parity of drafted trees: the plan, the attention over prompt, context and tree, the
accepted path and the moves of its rows; and the whole of them as a rollout uses it."""
import numpy as np
import pytest
import torch

import qk_oracle as qo
import rollout_oracle as ro
from response_replay_gb300 import binding as B
from response_replay_gb300 import layers
from response_replay_gb300 import torch_api as api

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def i32(x, dev):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device=dev)


def trees(rng, M, n, drafted, kind="random"):
    """Parents [M][n] of drafts that are the last drafted[m] rows."""
    p = np.full((M, n), -1)
    for m in range(M):
        first = n - drafted[m]
        for r in range(first + 1, n):
            p[m, r] = {"chain": r - 1, "star": first, "roots": -1,
                       "random": rng.integers(max(first, r - 5), r)}[kind]
    return p


@pytest.mark.parametrize("M,n,kind,ragged", [
    (1, 1, "chain", False), (3, 8, "random", False), (5, 31, "random", True), (4, 32, "chain", False),
    (7, 33, "star", True), (2, 128, "chain", False), (9, 100, "random", True), (1024, 5, "random", True),
    (6, 64, "roots", True)])
def test_plan(cuda, M, n, kind, ragged):
    rng = np.random.default_rng(M * n)
    drafted = rng.integers(0, n + 1, M) if ragged else np.full(M, n)
    lens = drafted + rng.integers(0, 5000, M)
    lens[::3][1:] = -1
    p = trees(rng, M, n, drafted, kind)
    vis, pos = api.draft_tree(i32(p, cuda), i32(lens, cuda), 2000000,
                              drafted=i32(drafted, cuda) if ragged else None, axes=3)
    assert B.ls_last_device_error(0) == B.LS_OK
    _, words, want = ro.draft_tree(p, lens, drafted, 2000000)
    np.testing.assert_array_equal(vis.cpu().numpy(), words)
    for a in range(3):
        np.testing.assert_array_equal(pos[a].cpu().numpy(), want)


def test_plan_reports_bad_trees(cuda):
    """A parent that is no earlier row of the draft is taken as none; a draft longer than its
    rows or its member is cut."""
    p = np.array([[-1, 0, 2, 1], [-1, -1, 0, 2], [-1, 0, 5, -7]])
    lens, drafted = [10, 10, 10], [4, 2, 4]
    fixed = np.array([[-1, 0, -1, 1], [-1, -1, -1, 2], [-1, 0, -1, -1]])
    vis, pos = api.draft_tree(i32(p, cuda), i32(lens, cuda), 0, drafted=i32(drafted, cuda))
    assert B.ls_last_device_error(0) == B.LS_ERR_DEVICE_CHECK
    _, words, want = ro.draft_tree(fixed, lens, drafted, 0)
    np.testing.assert_array_equal(vis.cpu().numpy(), words)
    np.testing.assert_array_equal(pos[0].cpu().numpy(), want)
    p = trees(np.random.default_rng(0), 2, 4, [4, 4])
    vis, _ = api.draft_tree(i32(p, cuda), i32([9, 2], cuda), 0, drafted=i32([7, 4], cuda))
    assert B.ls_last_device_error(0) == B.LS_ERR_DEVICE_CHECK
    assert bool((vis[1, :2] == 0).all())


# ------------------------------------------------------------------------------- attention

class Tree:
    """A captured prompt and a group's responses in pages with their drafts; whatever lies behind
    a sequence's end is NaN."""

    def __init__(self, dev, P, lens, drafted, n, hq, hkv, ps=64, rps=64, seed=0, sees=None, sharp=2.0):
        g = torch.Generator(device=dev)
        g.manual_seed(seed)
        rng = np.random.default_rng(seed)

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
            blocks[m, -(-max(x, 0) // rps):] = 2 ** 30  # not read
        self.n, self.scale_lens, self.drafted = n, list(lens), drafted
        self.lens = i32(lens, dev)
        self.resp = api.ResponseCache(pool, blocks.contiguous(), self.lens)
        self.q = (normal(M, n, hq, 128) * sharp).contiguous()
        self.count = i32(drafted, dev) if drafted is not None else None
        d = [n] * M if drafted is None else drafted
        if sees is None:
            self.sees, words, _ = ro.draft_tree(trees(rng, M, n, d), lens, d, 0)
        else:  # any bits
            self.sees = sees(rng, M, n)
            W = (n + 31) // 32
            bits = np.zeros((M, n, W * 32), np.uint64)
            bits[..., :n] = self.sees
            words = (bits.reshape(M, n, W, 32) << np.arange(32, dtype=np.uint64)).sum(-1)
            words = words.astype(np.uint32).view(np.int32)
        self.visible = i32(words, dev)

    def run(self, **kw):
        out = api.decode_attn_tree(self.cache, self.resp, self.q, self.visible, SCALE,
                                   drafted=self.count, **kw)
        assert B.ls_last_device_error(0) == B.LS_OK
        return out

    def check(self, o, lse):
        """Row by row: the oracle's decode of one token over the keys that the row sees."""
        M, n = len(self.scale_lens), self.n
        kp, vp = qo.f64(self.kp), qo.f64(self.vp)
        q, o, lse = qo.f64(self.q), qo.f64(o), qo.f64(lse)
        for m in range(M):
            x = self.scale_lens[m]
            if x < 0:
                continue
            c = n if self.drafted is None else self.drafted[m]
            kr, vr = qo.f64(self.kr[m]), qo.f64(self.vr[m])
            for r in range(n - c, n):
                keys = [*range(x - c), *(x - n + j for j in range(n - c, n) if self.sees[m, r, j])]
                ref, ob, lref, lb = qo.decode(q[m:m + 1, r:r + 1], kp, vp, [kr[keys]], [vr[keys]],
                                              [len(keys)], SCALE)
                assert (np.abs(o[m, r] - ref[0, 0]) <= ob[0, 0]).all(), (m, r)
                none = np.isinf(lref[0, 0])
                assert (lse[m, r][none] == -np.inf).all()
                assert (np.abs(lse[m, r][~none] - lref[0, 0][~none]) <= lb[0, 0][~none]).all(), (m, r)


# Drafts of one token and of many; a member's rows in less than a row tile, in one, in several;
# drafts that lie in one tile of keys, across two, and alone; prompts of none and of many tiles;
# row groups that are padding altogether.
CASES = [
    (1000, [1], None, 1, 4, 2, 64, 64),
    (500, [8, 100], None, 8, 8, 2, 64, 64),
    (0, [20, 300, 129], None, 13, 6, 2, 64, 16),
    (777, [30, 127, 128, 140, 500], [5, 16, 1, 12, 16], 16, 24, 4, 128, 64),
    (300, [64, 70, 256], [64, 3, 33], 64, 24, 4, 64, 32),
    (0, [5, 9, 0], [5, 0, 0], 9, 8, 8, 64, 64),
    (130, [128, 1000], None, 128, 8, 8, 256, 256),
    (2049, [40 + 30 * i for i in range(20)], [1 + i for i in range(20)], 20, 14, 2, 64, 16),
    (64, [200], None, 48, 40, 8, 16, 4096),
    (100, [70, 3], [60, 3], 60, 7, 1, 32, 64),
    (33, [10], None, 3, 128, 1, 64, 64),
    (5000, [300] * 6, None, 32, 15, 3, 64, 64),
]


@pytest.mark.parametrize("P,lens,drafted,n,hq,hkv,ps,rps", CASES)
def test_attention(cuda, P, lens, drafted, n, hq, hkv, ps, rps):
    t = Tree(cuda, P, lens, drafted, n, hq, hkv, ps, rps, seed=P + n)
    t.check(*t.run())


@pytest.mark.parametrize("P,M,top,n,hq,hkv,ps,rps", [
    (5003, 40, 3000, 24, 24, 4, 16, 256), (257, 58, 460, 48, 16, 8, 256, 16), (40000, 9, 200, 29, 35, 5, 64, 64),
    (3, 22, 2900, 64, 24, 4, 64, 64)])
def test_groups(cuda, P, M, top, n, hq, hkv, ps, rps):
    """Ragged drafts of many members, a CTA's share of several prompt strips and responses, of one row
    tile and of two; member by member against 64 bits on the GPU, with qk_oracle.decode's bounds."""
    rng = np.random.default_rng(P)
    drafted = rng.integers(0, n + 1, M)
    lens = drafted + rng.integers(0, top, M)
    lens[::7] = -1
    t = Tree(cuda, P, lens.tolist(), drafted.tolist(), n, hq, hkv, ps, rps, seed=P)
    o, lse = t.run(o=torch.zeros_like(t.q), lse=torch.zeros(M, n, hq, device=cuda))
    g = hq // hkv
    kp, vp = t.kp.double(), t.vp.double()
    for m in range(M):
        x, c = int(lens[m]), int(drafted[m])
        if x < 0 or c == 0:
            continue
        see = torch.ones(c, P + x, dtype=torch.bool, device=cuda)
        see[:, P + x - c:] = torch.as_tensor(t.sees[m, n - c:, n - c:], device=cuda)
        for h in range(hkv):
            k, v = torch.cat([kp[:, h], t.kr[m][:, h].double()]), torch.cat([vp[:, h], t.vr[m][:, h].double()])
            q = t.q[m, n - c:, h * g:(h + 1) * g].double()
            s = (q @ k.T * SCALE).masked_fill(~see[:, None], -torch.inf)
            mag = (q.abs() @ k.abs().T * SCALE).masked_fill(~see[:, None], 0)
            z = torch.logsumexp(s, -1, keepdim=True)
            p = torch.exp(s - z)
            want = p @ v
            e = (qo.U16 + 2 * 128 * qo.U32 * mag.amax(-1, keepdim=True) + 2.0 ** -18) * (p @ v.abs())
            e = e + qo.U16 * (want.abs() + e)
            ez = 128 * qo.U32 * (p * mag).sum(-1) + 2.0 ** -18 + 2.0 ** -20 * z[..., 0].abs()
            got = o[m, n - c:, h * g:(h + 1) * g].double()
            assert bool(((got - want).abs() <= e).all()), (m, h)
            assert bool(((lse[m, n - c:, h * g:(h + 1) * g].double() - z[..., 0]).abs() <= ez).all()), (m, h)


def test_any_bits(cuda):
    """Rows may see any rows of the draft, also later ones, or none of it."""
    def some(rng, M, n):
        s = rng.random((M, n, n)) < 0.4
        s[:, 3] = False
        s[0, :, :] = False
        return s

    for P, lens, drafted in [(90, [40, 60, 45], None), (0, [40, 60, 45], [40, 38, 40]), (0, [40, 40, 50], None)]:
        t = Tree(cuda, P, lens, drafted, 40, 12, 2, seed=P, sees=some)
        o, lse = t.run()
        t.check(o, lse)
        if P == 0 and lens[0] == 40:  # the first member's rows see nothing at all
            assert bool((o[0] == 0).all()) and bool((lse[0] == -float("inf")).all())


def test_rows_that_are_not_written(cuda):
    t = Tree(cuda, 200, [-1, 30, 50, 9], [4, 2, 12, 0], 12, 24, 4, seed=5)
    o = torch.full_like(t.q, 5.0)
    lse = torch.full(t.q.shape[:3], 6.0, device=cuda)
    t.run(o=o, lse=lse)
    t.check(o, lse)
    for m, first in enumerate([12, 10, 0, 12]):
        assert bool((o[m, :first] == 5.0).all()) and bool((lse[m, :first] == 6.0).all())


def test_a_line_is_the_plain_decode(cuda):
    """A draft without branches sees what decode_attn's tokens see.  The two calls cut the keys
    differently, so both are held to the one oracle, each within the bound of its roundings."""
    t = Tree(cuda, 3000, [70, 300, 21], None, 8, 24, 4, seed=9,
             sees=lambda rng, M, n: np.tril(np.ones((n, n), bool))[None].repeat(M, 0))
    o, lse = t.run()
    o2, lse2 = api.decode_attn(t.cache, t.resp, t.q, SCALE)
    t.check(o, lse)
    t.check(o2, lse2)


def test_many_row_groups(cuda):
    """As many rows as the call takes."""
    M = 90
    t = Tree(cuda, 300, [40 + 3 * m for m in range(M)], [1 + m % 36 for m in range(M)], 36, 6, 1, seed=2)
    assert -(-M * 36 * 6 // 128) == 152
    t.check(*t.run())
    over = torch.zeros(M, 37, 6, 128, dtype=torch.bfloat16, device=cuda)
    with pytest.raises(B.LongstrawError) as e:
        api.decode_attn_tree(t.cache, t.resp, over, torch.zeros(M, 37, 2, dtype=torch.int32, device=cuda), SCALE)
    assert e.value.status == B.LS_ERR_UNSUPPORTED


def test_streams_graphs_and_changing_drafts(cuda):
    t = Tree(cuda, 4000, [100, 260, 30], [16, 9, 3], 16, 24, 4, seed=11)
    o, lse = (x.clone() for x in t.run(o=torch.zeros_like(t.q), lse=torch.zeros(3, 16, 24, device=cuda)))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(20):
        o2, lse2 = torch.zeros_like(o), torch.zeros_like(lse)
        side.wait_stream(torch.cuda.current_stream())
        t.run(o=o2, lse=lse2, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        api.decode_attn_tree(t.cache, t.resp, t.q, t.visible, SCALE, drafted=t.count, o=o2, lse=lse2)
    # shorter drafts of the same members
    t.count.copy_(i32([2, 9, 1], cuda))
    t.drafted = [2, 9, 1]
    t.scale_lens = [100, 255, 30]
    t.lens.copy_(i32(t.scale_lens, cuda))
    t.kr, t.vr = [k[:x] for k, x in zip(t.kr, t.scale_lens)], [v[:x] for v, x in zip(t.vr, t.scale_lens)]
    graph.replay()
    torch.cuda.synchronize()
    assert B.ls_last_device_error(0) == B.LS_OK
    t.check(o2, lse2)


def test_bad_counts_and_pages(cuda):
    """A count outside its rows is cut; a bad page's keys count as zeros; both are reported."""
    t = Tree(cuda, 100, [50, 60], [3, 4], 8, 8, 2, seed=1)
    t.count.copy_(i32([9, 4], cuda))
    o, lse = api.decode_attn_tree(t.cache, t.resp, t.q, t.visible, SCALE, drafted=t.count)
    assert B.ls_last_device_error(0) == B.LS_ERR_DEVICE_CHECK
    assert bool(torch.isfinite(o[1, 4:]).all())
    t.count.copy_(i32([3, 4], cuda))
    t.resp.block_table[0, 0] = 10 ** 6
    api.decode_attn_tree(t.cache, t.resp, t.q, t.visible, SCALE, drafted=t.count, o=o, lse=lse)
    assert B.ls_last_device_error(0) == B.LS_ERR_DEVICE_CHECK
    assert bool(torch.isfinite(o[1, 4:]).all())


# ------------------------------------------------------------------------------- acceptance

def drafts(rng, M, n, ragged, chain):
    """Trees with tokens and the policy's choices, many of which follow the draft."""
    drafted = rng.integers(0, n + 1, M) if ragged else np.full(M, n)
    p = trees(rng, M, n, drafted, "chain" if chain else "random")
    tokens = rng.integers(0, 3, (M, n))  # few tokens: siblings share them
    chosen = rng.integers(0, 3, (M, n))
    for m in range(M):
        for r in range(n):
            kids = [c for c in range(n) if p[m, c] == r]
            if kids and rng.random() < (0.98 if chain else 0.8):
                chosen[m, r] = tokens[m, rng.choice(kids)]
    return drafted, p, tokens, chosen


@pytest.mark.parametrize("M,n,ragged,chain", [
    (1, 1, False, False), (6, 8, False, False), (40, 16, True, False), (9, 128, True, True),
    (300, 33, True, False), (1024, 12, False, False), (5, 64, False, True)])
def test_acceptance_and_moves(cuda, M, n, ragged, chain):
    rng = np.random.default_rng(M + n)
    drafted, p, tokens, chosen = drafts(rng, M, n, ragged, chain)
    tokens[rng.random((M, n)) < 0.05] = -1  # rows without a token
    chosen[rng.random((M, n)) < 0.02] = -1
    lens = drafted + rng.integers(0, 100, M)
    lens[2::5] = -3
    dd = i32(drafted, cuda) if ragged else None
    rows, count, follow, ends = api.accept_draft(i32(p, cuda), i32(tokens, cuda), i32(chosen, cuda),
                                                 i32(lens, cuda), drafted=dd)
    assert B.ls_last_device_error(0) == B.LS_OK
    want = ro.accept(p, tokens, chosen, lens, drafted)
    for got, ref in zip((rows, count, follow, ends), want):
        np.testing.assert_array_equal(got.cpu().numpy(), ref)
    # the moves, in two layers of small pages
    ps, hkv, L = 16, 2, 2
    nb = -(-max(int(lens.max()), 1) // ps) + 1
    table = rng.permutation(M * nb).reshape(M, nb)
    k = torch.randn(L, M * nb, hkv, ps, 128, device=cuda).to(torch.bfloat16)
    v = torch.randn_like(k)
    k0, v0 = (x.view(torch.int16).cpu().numpy() for x in (k, v))
    alloc = api.PageAllocator(i32(table, cuda), i32(lens, cuda), i32(np.zeros(1), cuda), i32([0], cuda), ps,
                              num_pages=M * nb)
    api.compact_rows(alloc, api.LayerPools(k, v), rows, count, drafted=dd)
    assert B.ls_last_device_error(0) == B.LS_OK
    for got, was in ((k, k0), (v, v0)):
        for layer in range(L):
            ref = ro.compact(was[layer], table, lens, drafted, want[0], want[1], ps)
            np.testing.assert_array_equal(got[layer].view(torch.int16).cpu().numpy(), ref)


def test_moves_refuse_what_is_no_path(cuda):
    """Rows that do not ascend, lie outside the draft or are more than it, a length past the
    table: nothing of the member is moved; others are."""
    M, n, ps, nb = 6, 8, 16, 2
    k = torch.randn(1, M * nb, 1, ps, 128, device=cuda).to(torch.bfloat16)
    v = torch.randn_like(k)
    k0 = k.clone()
    table = np.arange(M * nb).reshape(M, nb)
    lens, drafted = [20, 20, 20, 20, 40, 20], [6, 6, 6, 6, 6, 6]
    rows = np.full((M, n), -1)
    rows[0, :3] = [2, 5, 4]
    rows[1, :2] = [1, 5]
    rows[2, :2] = [4, 8]
    rows[3, :8] = np.arange(8)
    rows[4, :2] = [2, 4]
    rows[5, :2] = [3, 7]
    alloc = api.PageAllocator(i32(table, cuda), i32(lens, cuda), i32(np.zeros(1), cuda), i32([0], cuda), ps,
                              num_pages=M * nb)
    api.compact_rows(alloc, api.LayerPools(k, v), i32(rows, cuda), i32([3, 2, 2, 8, 2, 2], cuda),
                     drafted=i32(drafted, cuda))
    assert B.ls_last_device_error(0) == B.LS_ERR_DEVICE_CHECK
    assert torch.equal(k[:, :10], k0[:, :10])
    ref = ro.compact(k0[0].view(torch.int16).cpu().numpy(), table, lens, drafted, rows, [0] * 5 + [2], ps)
    np.testing.assert_array_equal(k[0].view(torch.int16).cpu().numpy(), ref)


# ------------------------------------------------------------------------------- together

@pytest.mark.parametrize("hq", [8, 40])  # drafts of a row tile, and of several
def test_drafted_rollout_equals_the_plain_one(cuda, hq):
    """A rollout with drafts over two layers: extend, plan, append, attend, accept, settle.  Its
    accepted tokens, lengths, pages and keys are those of a rollout one token at a time, whose
    tokens the drafts partly foresee."""
    dev, L, M, n, hkv, ps, P = cuda, 2, 3, 7, 2, 16, 200
    g = torch.Generator(device=dev)
    g.manual_seed(4)
    rng = np.random.default_rng(4)

    def normal(*s):
        return torch.randn(*s, generator=g, device=dev).to(torch.bfloat16)

    table = torch.arange(-(-P // ps), dtype=torch.int32, device=dev)
    prompt = layers.LayeredKVCache(L, table.numel(), table, ps, hkv, P)
    for l in range(L):
        prompt.capture(l, normal(P, hkv, 128), normal(P, hkv, 128))
    # a "model": a token's projections in every layer come from tables
    vocab = 50
    emb = [[normal(vocab, h, 128) for h in (hq, hkv, hkv)] for _ in range(L)]
    rot = api.Rotary.from_base(1e6, 128, dev)
    stream = rng.integers(0, vocab, (M, 60))  # the tokens that the policy chooses, by length

    plain = layers.LayeredResponses(prompt, hkv, M, 80, 40, ps, dev)
    drafty = layers.LayeredResponses(prompt, hkv, M, 80, 40, ps, dev, member_rows=n, sharing=True)

    def outputs(resp, tokens, step_rows, **kw):
        outs = []
        for l in range(L):
            t = torch.as_tensor(tokens, device=dev).reshape(-1)
            q, k, v = (e[t] for e in emb[l])
            q = resp.append(l, q, k, v, rot)
            outs.append(resp.attend(l, q.view(M, step_rows, hq, 128), SCALE, **kw)[0])
        return outs

    plain_out = []
    one = torch.ones(M, dtype=torch.int32, device=dev)
    for step in range(40):
        plain.extend(one)
        plain_out.append(outputs(plain, stream[:, step], 1))
    done = np.zeros(M, int)
    while done.min() < 40:
        # the next token, then guesses: right ones, wrong ones, in branches
        drafted = rng.integers(1, n + 1, M)
        drafted[done >= 40] = 0
        p = trees(rng, M, n, drafted)
        tokens = np.full((M, n), 0)
        depth = np.zeros((M, n), int)
        for m in range(M):
            for r in range(n - drafted[m], n):
                if p[m, r] >= 0:
                    depth[m, r] = depth[m, p[m, r]] + 1
                right = stream[m, done[m] + depth[m, r]]
                tokens[m, r] = right if r == n - drafted[m] or rng.random() < 0.7 else (right + 1) % vocab
        visible = drafty.draft(i32(p, dev), i32(drafted, dev))
        outs = outputs(drafty, tokens, n, visible=visible, drafted=i32(drafted, dev))
        chosen = stream[np.arange(M)[:, None], done[:, None] + depth + 1]
        rows, count, follow = drafty.settle(i32(p, dev), i32(tokens, dev), i32(chosen, dev),
                                            i32(drafted, dev))
        assert B.ls_last_device_error(0) == B.LS_OK
        rows, count = rows.cpu().numpy(), count.cpu().numpy()
        for m in range(M):
            for i in range(count[m]):
                at = done[m] + i
                if at < 40:
                    for l in range(L):
                        a, b = outs[l][m, rows[m, i]].float(), plain_out[at][l][m, 0].float()
                        # two results of the same numbers by other tiles: two times the bound of
                        # each, roundings of weights (2^-8 of |values| <= 5) and of the output
                        assert float((a - b).abs().max()) <= 2 * 2 * 2.0 ** -8 * 5
            if count[m]:
                assert int(follow[m]) == stream[m, done[m] + count[m]]
            done[m] += count[m]
        np.testing.assert_array_equal(drafty.alloc.lens.cpu().numpy(), done)
        assert int(drafty.alloc.used) == sum(-(-d // ps) for d in done)
    # the kept keys are the plain rollout's
    for l in range(L):
        for m in range(M):
            for pools in ("k_pools", "v_pools"):
                got = []
                for resp in (plain, drafty):
                    t = torch.arange(40, device=dev)
                    page = resp.alloc.block_table[m, t // ps].long()
                    got.append(getattr(resp, pools)[l][page, :, t % ps])
                assert torch.equal(*got)
