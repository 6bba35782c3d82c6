"""CPU tests of the query/key stage, page allocation and decode calls: what they refuse
(every rejected call returns before any launch), and the 64-bit backward that the GPU
tests compare with, against differences."""
import ctypes as C
import os

import numpy as np
import pytest
import torch

import qk_oracle as qo
from response_replay_gb300 import binding as B
from response_replay_gb300 import torch_api as api

A = 1 << 20  # an aligned address that nothing reads: every call below is refused


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from response_replay_gb300 import build
        build.build()
    return B.lib()


def view(**kw):
    s = {f"{n}_{d}": x for n in "qkv" for d, x in zip(("ts", "hs"), kw.pop(f"{n}_stride", (4096, 128)))}
    return B.ls_qkv_view(**{**dict(q=A, k=A, v=A), **s, **kw})


def norm(**kw):
    return B.ls_qk_norm(**{**dict(wq=A, wk=A, w_dtype=B.LS_FP32, w_offset=0.0, eps=1e-6), **kw})


def rotary(**kw):
    return B.ls_rotary(**{**dict(inv_freq=A, pair_axis=None, rot_dim=64, axes=1, interleaved=0), **kw})


def pool(**kw):
    return B.ls_page_pool(**{**dict(k_pool=A, v_pool=A, num_pages=8, page_size=64, num_kv_heads=4,
                                    head_dim=128), **kw})


BAD_COMMON = [
    (dict(T=-1), B.LS_ERR_INVALID_ARG),
    (dict(T=2 ** 31), B.LS_ERR_UNSUPPORTED),
    (dict(Hq=0), B.LS_ERR_INVALID_ARG),
    (dict(norm=norm(eps=0.0)), B.LS_ERR_INVALID_ARG),
    (dict(norm=norm(eps=1e-39)), B.LS_ERR_INVALID_ARG),
    (dict(norm=norm(eps=float("nan"))), B.LS_ERR_INVALID_ARG),
    (dict(norm=norm(w_offset=float("inf"))), B.LS_ERR_INVALID_ARG),
    (dict(norm=norm(w_dtype=7)), B.LS_ERR_INVALID_ARG),
    (dict(norm=norm(wk=A + 4)), B.LS_ERR_INVALID_ARG),
    (dict(rotary=rotary(rot_dim=-16)), B.LS_ERR_INVALID_ARG),
    (dict(rotary=rotary(rot_dim=144)), B.LS_ERR_INVALID_ARG),
    (dict(rotary=rotary(rot_dim=24)), B.LS_ERR_UNSUPPORTED),
    (dict(rotary=rotary(axes=0)), B.LS_ERR_INVALID_ARG),
    (dict(rotary=rotary(axes=2)), B.LS_ERR_INVALID_ARG),
    (dict(rotary=rotary(axes=9, pair_axis=A)), B.LS_ERR_UNSUPPORTED),
    (dict(rotary=rotary(inv_freq=None)), B.LS_ERR_INVALID_ARG),
    (dict(rotary=rotary(inv_freq=A + 4)), B.LS_ERR_INVALID_ARG),
    (dict(rotary=rotary(pair_axis=A + 2)), B.LS_ERR_INVALID_ARG),
    (dict(positions=None), B.LS_ERR_INVALID_ARG),
    (dict(positions=A + 1), B.LS_ERR_INVALID_ARG),
    (dict(x=view(q=None)), B.LS_ERR_INVALID_ARG),
    (dict(x=view(q=A + 8)), B.LS_ERR_INVALID_ARG),
    (dict(x=view(k_stride=(4096, 124))), B.LS_ERR_INVALID_ARG),
    (dict(x=view(q_stride=(-4096, 128))), B.LS_ERR_INVALID_ARG),
    (dict(x=view(q_stride=(4100, 128))), B.LS_ERR_INVALID_ARG),
]
BASE = dict(x=None, T=10, Hq=8, Hkv=4, norm=None, rotary=None, positions=A, out=None)


def args(kw):
    d = {**BASE, "x": view(), "out": view(), "norm": norm(), "rotary": rotary(), **kw}
    return d


def test_forward_and_append_refuse(lib):
    more = [(dict(x=view(k=None)), B.LS_ERR_INVALID_ARG),
            (dict(out=view(q=None)), B.LS_ERR_INVALID_ARG),
            (dict(out=view(k=None)), B.LS_ERR_INVALID_ARG),
            (dict(out=view(v=None)), B.LS_ERR_INVALID_ARG),
            (dict(Hkv=0), B.LS_ERR_INVALID_ARG)]
    for kw, want in BAD_COMMON + more:
        d = args(kw)
        got = lib.ls_qk_norm_rope_fwd(d["x"], d["T"], d["Hq"], d["Hkv"], d["norm"], d["rotary"],
                                      d["positions"], d["out"], None)
        assert got == want, kw
    more = [(dict(x=view(v=None)), B.LS_ERR_INVALID_ARG), (dict(slots=None), B.LS_ERR_INVALID_ARG),
            (dict(slots=A + 2), B.LS_ERR_INVALID_ARG), (dict(out=view(q=None)), B.LS_ERR_INVALID_ARG),
            (dict(pool=pool(page_size=48)), B.LS_ERR_UNSUPPORTED),
            (dict(pool=pool(page_size=8192)), B.LS_ERR_UNSUPPORTED),
            (dict(pool=pool(head_dim=64)), B.LS_ERR_UNSUPPORTED),
            (dict(pool=pool(num_pages=0)), B.LS_ERR_INVALID_ARG),
            (dict(pool=pool(num_pages=2 ** 30)), B.LS_ERR_UNSUPPORTED),
            (dict(pool=pool(v_pool=None)), B.LS_ERR_INVALID_ARG),
            (dict(pool=None), B.LS_ERR_INVALID_ARG)]
    for kw, want in BAD_COMMON + more:
        d = {"slots": A, "pool": pool(), **args(kw)}
        got = lib.ls_qk_norm_rope_append(d["pool"], d["x"], d["T"], d["Hq"], d["norm"], d["rotary"],
                                         d["positions"], d["slots"], d["out"], None)
        assert got == want, kw
    # no tokens: nothing to do, whatever the tensors
    assert lib.ls_qk_norm_rope_fwd(None, 0, 8, 4, norm(), rotary(), None, None, None) == B.LS_OK


def test_backward_refuses(lib):
    more = [(dict(x=None), B.LS_ERR_INVALID_ARG), (dict(dtype=5), B.LS_ERR_INVALID_ARG),
            (dict(norm=None), B.LS_ERR_INVALID_ARG),        # weight gradients without a norm
            (dict(dwq=A + 4), B.LS_ERR_INVALID_ARG),
            (dict(dy=view(q=None)), B.LS_ERR_INVALID_ARG), (dict(dy=view(k=None)), B.LS_ERR_INVALID_ARG),
            (dict(out=view(v=None)), B.LS_ERR_INVALID_ARG)]
    for kw, want in BAD_COMMON + more:
        d = {"dy": view(), "dtype": B.LS_FP32, "dwq": A, **args(kw)}
        got = lib.ls_qk_norm_rope_bwd(d["x"], d["T"], d["Hq"], d["Hkv"], d["norm"], d["rotary"],
                                      d["positions"], d["dy"], d["dtype"], 0, d["out"], d["dwq"], None,
                                      A, 1 << 30, None)
        assert got == want, kw
    n = C.c_size_t(0)
    assert lib.ls_qk_norm_rope_bwd_workspace(-1, C.byref(n)) == B.LS_ERR_INVALID_ARG
    assert lib.ls_qk_norm_rope_bwd_workspace(2 ** 31, C.byref(n)) == B.LS_ERR_UNSUPPORTED
    assert lib.ls_qk_norm_rope_bwd_workspace(1, None) == B.LS_ERR_INVALID_ARG


def test_extend_refuses(lib):
    base = dict(table=A, members=4, max_blocks=8, ps=64, pages=100, lens=A, add=A, free=A, nfree=50,
                used=A, pos0=0, axes=1, cap=16, slots=A, pos=A, lo=A, uo=A)
    for kw, want in [
        (dict(members=-1), B.LS_ERR_INVALID_ARG), (dict(members=1025), B.LS_ERR_UNSUPPORTED),
        (dict(max_blocks=-1), B.LS_ERR_INVALID_ARG), (dict(ps=8), B.LS_ERR_UNSUPPORTED),
        (dict(ps=100), B.LS_ERR_UNSUPPORTED), (dict(nfree=-1), B.LS_ERR_INVALID_ARG),
        (dict(pages=-1), B.LS_ERR_INVALID_ARG), (dict(pages=2 ** 30), B.LS_ERR_UNSUPPORTED),
        (dict(max_blocks=2 ** 30), B.LS_ERR_UNSUPPORTED), (dict(pos0=-1), B.LS_ERR_INVALID_ARG),
        (dict(pos0=2 ** 31 - 100), B.LS_ERR_UNSUPPORTED), (dict(axes=0), B.LS_ERR_INVALID_ARG),
        (dict(axes=9), B.LS_ERR_UNSUPPORTED), (dict(cap=-1), B.LS_ERR_INVALID_ARG),
        (dict(cap=2 ** 31), B.LS_ERR_UNSUPPORTED), (dict(table=None), B.LS_ERR_INVALID_ARG),
        (dict(lens=None), B.LS_ERR_INVALID_ARG), (dict(add=A + 1), B.LS_ERR_INVALID_ARG),
        (dict(free=None), B.LS_ERR_INVALID_ARG), (dict(used=None), B.LS_ERR_INVALID_ARG),
        (dict(slots=A + 4), B.LS_ERR_INVALID_ARG), (dict(slots=None), B.LS_ERR_INVALID_ARG),
        (dict(pos=A + 8), B.LS_ERR_INVALID_ARG), (dict(lo=None), B.LS_ERR_INVALID_ARG),
        (dict(uo=A + 2), B.LS_ERR_INVALID_ARG),
    ]:
        d = {**base, **kw}
        assert lib.ls_extend_pages(*d.values(), None) == want, kw
    assert lib.ls_extend_pages(*{**base, "members": 0, "cap": 0}.values(), None) == B.LS_OK


def test_decode_refuses(lib):
    def cache(**kw):
        return B.ls_kv_cache(**{**dict(k_pool=A, v_pool=A, page_table=A, num_pages=8,
                                       num_logical_pages=8, page_size=64, num_kv_heads=4,
                                       head_dim=128, num_tokens=512), **kw})

    def resp(**kw):
        return B.ls_resp_cache(**{**dict(pool=pool(), block_table=A, lens=A, members=4, max_blocks=2),
                                  **kw})

    base = dict(cache=cache(), resp=resp(), q=A, n=1, hq=24, scale=0.1, o=A, lse=A, ws=A, nws=1 << 40)
    IA, UN = B.LS_ERR_INVALID_ARG, B.LS_ERR_UNSUPPORTED
    n = C.c_size_t(0)
    for kw, want in [
        (dict(cache=cache(head_dim=64)), UN), (dict(cache=cache(num_tokens=600)), IA),
        (dict(cache=cache(k_pool=None)), IA), (dict(cache=cache(num_kv_heads=2)), IA),
        (dict(cache=cache(num_tokens=2 ** 31, num_logical_pages=2 ** 26)), UN),
        (dict(resp=resp(pool=pool(page_size=7))), UN), (dict(resp=resp(pool=pool(k_pool=A + 8))), IA),
        (dict(resp=resp(members=-1)), IA), (dict(resp=resp(members=1025)), UN),
        (dict(resp=resp(max_blocks=-1)), IA), (dict(resp=resp(max_blocks=2 ** 25)), UN),
        (dict(resp=resp(max_blocks=2 ** 24, members=1024)), UN),
        (dict(resp=resp(block_table=None)), IA), (dict(resp=resp(lens=None)), IA),
        (dict(resp=resp(lens=A + 2)), IA), (dict(resp=None), IA), (dict(cache=None), IA),
        (dict(n=0), IA), (dict(hq=23), IA), (dict(hq=0), IA), (dict(n=22), UN), (dict(hq=516), UN),
    ]:
        d = {**base, **kw}
        assert lib.ls_decode_attn(*d.values(), None) == want, kw
        assert lib.ls_decode_attn_workspace(d["cache"], d["resp"], d["n"], d["hq"],
                                            C.byref(n)) == want, kw
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert lib.ls_decode_attn(*{**base, "scale": scale}.values(), None) == IA
    assert lib.ls_decode_attn_workspace(base["cache"], base["resp"], 1, 24, None) == IA


def test_torch_calls_refuse_host_tensors_and_shapes():
    q, k = torch.zeros(3, 4, 128, dtype=torch.bfloat16), torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        api.qk_norm_rope_fwd(q, k, None, None, None)
    with pytest.raises(ValueError, match="inv_freq"):
        api.Rotary(torch.ones(4, dtype=torch.float64))
    with pytest.raises(ValueError, match="k_pool"):
        api.PagePool(torch.zeros(2, 3), torch.zeros(2, 3))
    with pytest.raises(ValueError, match="block_table"):
        api.PageAllocator(*(torch.zeros(1, dtype=torch.int32) for _ in range(4)), 64)
    m = torch.zeros(5, 6, 128, dtype=torch.bfloat16)
    api._no_overlap(m, "m")
    api._no_overlap(m.transpose(0, 1), "m")
    for bad in (m[:1].expand(5, 6, 128), m.as_strided((5, 6, 128), (128, 128, 1)),
                m.as_strided((5, 6, 128), (640, 128, 1)), m.as_strided((5, 6, 128), (768, 64, 1))):
        with pytest.raises(ValueError, match="overlap"):
            api._no_overlap(bad, "m")


@pytest.mark.parametrize("inter", [False, True])
def test_the_backward_formula_matches_differences(inter):
    rng = np.random.default_rng(1)
    x, w, dy = rng.standard_normal((3, 2, 128)), rng.standard_normal(128), rng.standard_normal((3, 2, 128))
    rot = (rng.integers(0, 1000, (2, 3)), 1e4 ** (-np.arange(24) / 24.0), rng.integers(0, 2, 24), inter)

    def loss(x, w):
        return (qo.fwd(x, w, 1.0, 1e-6, *rot)[0] * dy).sum()

    dx, _, dw, _ = qo.bwd(x, dy, w, 1.0, 1e-6, *rot)
    h = 1e-5   # the difference is off by h^2 of the third derivative, and 1e-16 / h in rounding
    for _ in range(3):
        d = rng.standard_normal(x.shape)
        assert abs((loss(x + h * d, w) - loss(x - h * d, w)) / (2 * h) - (dx * d).sum()) <= 1e-6
        d = rng.standard_normal(128)
        assert abs((loss(x, w + h * d) - loss(x, w - h * d)) / (2 * h) - (dw * d).sum()) <= 1e-6
