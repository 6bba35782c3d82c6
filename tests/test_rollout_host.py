"""CPU tests of token statistics, drafted trees and branching pages: what the calls refuse (every
rejected call returns before any launch), and the 64-bit implementations that the GPU tests
compare with, against differences and walks of their own."""
import os

import numpy as np
import pytest
import torch

import rollout_oracle as ro
from response_replay_gb300 import binding as B
from response_replay_gb300 import torch_api as api

A = 1 << 20  # an aligned address that nothing reads: every call below is refused
INV, UNS, WS = B.LS_ERR_INVALID_ARG, B.LS_ERR_UNSUPPORTED, B.LS_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from response_replay_gb300 import build
        build.build()
    return B.lib()


def pool(**kw):
    return B.ls_page_pool(**{**dict(k_pool=A, v_pool=A, num_pages=8, page_size=64, num_kv_heads=4,
                                    head_dim=128), **kw})


def refused(call, base, cases):
    for kw, want in cases:
        assert set(kw) <= set(base), kw
        assert call(*{**base, **kw}.values(), None) == want, kw


def test_token_logp_refuses(lib):
    base = dict(logits=A, dtype=B.LS_BF16, T=4, V=100, ld=100, y=A, temp=1.0, top=5, logp=A, lse=A, ent=A,
                tl=A, ti=A, ws=A, nbytes=0)
    common = [(dict(dtype=2), INV), (dict(T=-1), INV), (dict(V=0), INV), (dict(ld=99), INV),
              (dict(top=-1), INV), (dict(V=4, ld=4), INV), (dict(top=33), UNS), (dict(T=2 ** 31), UNS),
              (dict(V=2 ** 30 + 1, ld=2 ** 31), UNS), (dict(temp=0.0), INV), (dict(temp=-1.0), INV),
              (dict(temp=float("nan")), INV), (dict(temp=float("inf")), INV), (dict(temp=1e-7), INV),
              (dict(logits=None), INV), (dict(logits=A + 1), INV), (dict(dtype=B.LS_FP32, logits=A + 2), INV),
              (dict(y=A + 2), INV), (dict(lse=A + 1), INV)]
    refused(lib.ls_token_logp_fwd, base, common + [
        (dict(y=None), INV), (dict(tl=None), INV), (dict(ti=None), INV), (dict(ti=A + 2), INV),
        (dict(logp=A + 3), INV)])
    base = dict(logits=A, dtype=B.LS_BF16, T=4, V=100, ld=100, y=A, temp=1.0, lse=A, ent=A, top=5, ti=A, dl=A,
                de=A, dt=A, d=A + 65536, dld=100)
    refused(lib.ls_token_logp_bwd, base, common + [
        (dict(dld=99), INV), (dict(d=None), INV), (dict(d=A + 1), INV), (dict(lse=None), INV),
        (dict(ent=None), INV), (dict(y=None), INV), (dict(ti=None), INV), (dict(dt=None), INV),
        (dict(d=A, dld=104), INV), (dict(de=A + 2), INV)])
    assert lib.ls_token_logp_fwd_workspace(B.LS_BF16, 4, 100, 5, None) == INV
    assert lib.ls_token_logp_fwd(None, B.LS_BF16, 0, 100, 100, None, 1.0, 5, None, None, None, None, None,
                                 None, 0, None) == B.LS_OK
    assert lib.ls_token_logp_bwd(None, B.LS_BF16, 0, 100, 100, None, 1.0, None, None, 0, None, None, None,
                                 None, None, 100, None) == B.LS_OK


def test_drafts_refuse(lib):
    base = dict(p=A, lens=A, drafted=A, M=4, n=8, pos0=0, axes=1, vis=A, pos=A)
    size = [(dict(M=-1), INV), (dict(n=0), INV), (dict(M=1025), UNS), (dict(n=129), UNS), (dict(lens=None), INV),
            (dict(lens=A + 2), INV), (dict(drafted=A + 1), INV)]
    refused(lib.ls_draft_tree, base, size + [
        (dict(p=None), INV), (dict(p=A + 2), INV), (dict(vis=None), INV), (dict(vis=A + 1), INV),
        (dict(pos=A + 3), INV), (dict(pos0=-1), INV), (dict(axes=0), INV), (dict(axes=9), UNS)])
    base = dict(p=A, tok=A, cho=A, lens=A, drafted=A, M=4, n=8, rows=A, count=A, follow=A, ends=A)
    refused(lib.ls_accept_draft, base, size + [({k: x}, INV) for k in ("p", "tok", "cho", "rows", "count",
                                                                      "follow", "ends") for x in (None, A + 2)])
    base = dict(pool=pool(), L=3, stride=8 * 4 * 64 * 128, table=A, blocks=10, lens=A, drafted=A, M=4, n=8,
                rows=A, count=A)
    pools = [(dict(pool=pool(page_size=8)), UNS), (dict(pool=pool(head_dim=64)), UNS),
             (dict(pool=pool(k_pool=None)), INV), (dict(pool=pool(v_pool=A + 8)), INV), (dict(L=0), INV),
             (dict(stride=8 * 4 * 64 * 128 - 8), INV), (dict(stride=8 * 4 * 64 * 128 + 4), INV),
             (dict(L=1, stride=-8), INV), (dict(L=70000), UNS)]
    refused(lib.ls_compact_rows, base, size + pools + [
        (dict(table=None), INV), (dict(table=A + 2), INV), (dict(rows=None), INV), (dict(count=A + 1), INV),
        (dict(blocks=-1), INV), (dict(blocks=2 ** 30), UNS)])
    base = dict(pool=pool(), L=3, stride=8 * 4 * 64 * 128, count=5, f=A, t=A, rows=A)
    refused(lib.ls_copy_pages, base, pools + [
        (dict(count=-1), INV), (dict(f=None), INV), (dict(t=A + 2), INV), (dict(rows=A + 1), INV),
        (dict(count=2 ** 30), UNS)])
    for call, args in ((lib.ls_draft_tree, (None, None, None, 0, 8, 0, 1, None, None)),
                       (lib.ls_accept_draft, (None,) * 5 + (0, 8) + (None,) * 4),
                       (lib.ls_compact_rows, (pool(), 1, 0, None, 4, None, None, 0, 8, None, None)),
                       (lib.ls_copy_pages, (pool(), 1, 0, 0, None, None, None))):
        assert call(*args, None) == B.LS_OK


def test_tree_attention_refuses(lib):
    def cache(**kw):
        return B.ls_kv_cache(**{**dict(k_pool=A, v_pool=A, page_table=A, num_pages=8, num_logical_pages=8,
                                       page_size=64, num_kv_heads=4, head_dim=128, num_tokens=500), **kw})

    def resp(**kw):
        return B.ls_resp_cache(**{**dict(pool=pool(), block_table=A, lens=A, members=2, max_blocks=4), **kw})

    base = dict(c=cache(), r=resp(), q=A, n=8, hq=24, vis=A, drafted=A, scale=0.1, o=A, lse=A, ws=A, nbytes=1)
    refused(lib.ls_decode_attn_tree, base, [
        (dict(scale=0.0), INV), (dict(scale=float("nan")), INV), (dict(n=0), INV), (dict(n=129), UNS),
        (dict(hq=26), INV), (dict(hq=4 * 129), UNS), (dict(c=cache(head_dim=64)), UNS),
        (dict(r=resp(pool=pool(num_kv_heads=2))), INV), (dict(r=resp(members=1025)), UNS),
        (dict(r=resp(lens=None)), INV)])


def test_pages_refuse(lib):
    base = dict(table=A, M=4, blocks=8, ps=64, pages=100, lens=A, new=A, free=A, nfree=50, used=A, shared=A, lo=A,
                uo=A)
    common = [(dict(M=-1), INV), (dict(M=1025), UNS), (dict(blocks=-1), INV), (dict(blocks=2 ** 29), UNS),
              (dict(ps=8), UNS), (dict(ps=100), UNS), (dict(pages=-1), INV), (dict(pages=2 ** 26), UNS),
              (dict(lens=None), INV), (dict(lo=None), INV), (dict(used=None), INV), (dict(uo=A + 2), INV),
              (dict(table=None), INV), (dict(free=None), INV), (dict(nfree=-1), INV), (dict(shared=A + 1), INV)]
    refused(lib.ls_trim_pages, base, common + [(dict(new=None), INV), (dict(new=A + 2), INV)])
    base = dict(table=A, M=4, blocks=8, ps=64, pages=100, lens=A, src=A, keep=A, free=A, nfree=50, used=A,
                shared=A, copies=A, lo=A, uo=A)
    refused(lib.ls_fork_pages, base, common + [
        (dict(src=None), INV), (dict(src=A + 1), INV), (dict(keep=A + 2), INV), (dict(shared=None), INV),
        (dict(copies=None), INV), (dict(copies=A + 2), INV)])


def test_torch_calls_refuse():
    z = torch.zeros(4, 10)
    i = torch.zeros(4, dtype=torch.int32)
    for bad in (z.double(), z[0], z.T, torch.zeros(1, 10).expand(4, 10)):
        with pytest.raises(ValueError):
            api.token_logp_fwd(bad, i)
    with pytest.raises(ValueError):
        api.token_logp_fwd(z, i)  # not on a GPU
    with pytest.raises(ValueError):
        api.token_logp_bwd(z, i, z[:, 0], None, z[:, 0], top_ids=None, d_top=z)
    for bad in (i, torch.zeros(4, 3)):
        with pytest.raises(ValueError):
            api.draft_tree(bad, i, 0)
    k = torch.zeros(2, 3, 1, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.LayerPools(k, k)  # neither on a GPU nor pinned
    with pytest.raises(ValueError):
        api.LayerPools(k[0], k[0])


# ------------------------------------------------------------------------------- the oracle

@pytest.mark.parametrize("temp", [1.0, 0.6])
def test_the_gradient_is_that_of_the_formula(temp):
    """Central differences of the 64-bit objective against the 64-bit gradient."""
    rng = np.random.default_rng(1)
    T, V, k = 3, 40, 5
    z = rng.standard_normal((T, V)) * 3
    z[1, 7:12] = -np.inf
    y = np.array([3, 0, 39])
    ids = ro.top(z, k)
    ids[:, 2] = ids[:, 0]
    w, wh, wt = rng.standard_normal(T), rng.standard_normal(T), rng.standard_normal((T, k))

    def value(x):
        lp, _ = ro.log_probs(x, temp)
        return ((lp[np.arange(T), y] * w).sum() + (ro.entropy(lp) * wh).sum()
                + (np.take_along_axis(lp, ids, 1) * wt).sum())

    lp, lse = ro.log_probs(z, temp)
    d, err = ro.token_logp_bwd(z, y, lse, ro.entropy(lp), w, wh, temp, ids, wt)
    assert (d[1, 7:12] == 0).all() and np.isfinite(err).all()
    for t in range(T):
        for v in range(V):
            if not np.isfinite(z[t, v]):
                continue
            e = np.zeros_like(z)
            e[t, v] = 1e-5
            assert abs((value(z + e) - value(z - e)) / 2e-5 - d[t, v]) < 1e-8


def test_fp32_stays_within_the_bounds():
    """A plain fp32 computation is within the bounds, and one with a wrong logit is not."""
    rng = np.random.default_rng(2)
    z = (rng.standard_normal((6, 5000)) * 3).astype(np.float32)
    lp, lse, h, e_lse, e_h = ro.stat_bounds(z, 1.0)
    m = z.max(-1, keepdims=True)
    e = np.exp(z - m)
    s = e.sum(-1)
    got = m[:, 0] + np.log(s)
    ent = np.log(s) - (e * (z - m)).sum(-1) / s
    assert (np.abs(got - lse) <= e_lse).all() and (np.abs(ent - h) <= e_h).all()
    # e_lse is below what one logit of a thousandth of the weight changes
    assert (e_lse < 1e-4).all() and (e_h < 1e-3).all()


def test_a_draft_walks_its_parents():
    p = [[-1, 0, 0, 1, 3, 2, -1]]
    see, words, pos = ro.draft_tree(p, [17], [7], 100)
    assert [np.flatnonzero(r).tolist() for r in see[0]] == [[0], [0, 1], [0, 2], [0, 1, 3], [0, 1, 3, 4],
                                                            [0, 2, 5], [6]]
    assert words[0, :, 0].tolist() == [1, 3, 5, 11, 27, 37, 64]
    assert pos[0].tolist() == [110, 111, 111, 112, 113, 112, 110]
    tokens, chosen = [[9, 4, 5, 6, 7, 8, 9]], [[5, 6, 8, 0, 0, 3, 0]]
    rows, count, follow, ends = ro.accept(p, tokens, chosen, [17], [7])
    assert rows[0].tolist() == [0, 2, 5, -1, -1, -1, -1] and count[0] == 3 and follow[0] == 3 and ends[0] == 13


def test_pages_go_back_once():
    """Two branches of one response: a page goes back with its last owner, in member order."""
    table = np.array([[5, 6, 7], [5, 6, 2], [5, 1, 0]])
    free, shared = np.array([5, 6, 7, 2, 1, 9, 8, 3]), np.zeros(10, int)
    shared[5], shared[6] = 2, 1
    lens = np.array([40, 35, 20])
    new, f, used, s = ro.trim(table, lens, [-1, 35, 20], free, 5, shared, 16, 10)
    assert used == 4 and f[4] == 7 and s[5] == 1 and s[6] == 0 and new.tolist() == [-1, 35, 20]
    new, f, used, s = ro.trim(table, lens, [-1, -1, -1], free, 5, shared, 16, 10)
    assert used == 0 and f[:5].tolist() == [5, 6, 7, 2, 1] and not s.any()
    assert ro.trim(table, lens, [40, 20, 20], free, 5, shared, 16, 10) is None  # inside page 6
    assert ro.trim(table, lens, [20, 16, 20], free, 5, shared, 16, 10)[3][6] == 0
