"""CPU test of what ls_extend_drafts refuses (before any launch)."""
import os

import pytest

from response_replay_gb300 import binding as B

A = 1 << 20  # an aligned address that nothing reads: every call below is refused
BASE = dict(table=A, M=4, blocks=8, ps=64, pages=100, lens=A, add=A, free=A, nfree=50, used=A, pos0=0, axes=1, rows=8,
            slots=A, pos=A, lo=A, uo=A, added=A)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(B.LIB_PATH):
        from response_replay_gb300 import build
        build.build()
    return B.lib()


@pytest.mark.parametrize("kw,want", [
    (dict(added=None), B.LS_ERR_INVALID_ARG), (dict(added=A + 2), B.LS_ERR_INVALID_ARG),
    (dict(rows=0), B.LS_ERR_INVALID_ARG), (dict(M=-1), B.LS_ERR_INVALID_ARG), (dict(M=1025), B.LS_ERR_UNSUPPORTED),
    (dict(add=A + 1), B.LS_ERR_INVALID_ARG), (dict(lens=None), B.LS_ERR_INVALID_ARG),
    (dict(lens=None, add=None), B.LS_ERR_INVALID_ARG), (dict(lo=None), B.LS_ERR_INVALID_ARG),
    (dict(used=None), B.LS_ERR_INVALID_ARG), (dict(slots=A + 4), B.LS_ERR_INVALID_ARG),
    (dict(pos=A + 4), B.LS_ERR_INVALID_ARG), (dict(table=None), B.LS_ERR_INVALID_ARG),
    (dict(ps=8), B.LS_ERR_UNSUPPORTED), (dict(axes=9), B.LS_ERR_UNSUPPORTED), (dict(pos0=-1), B.LS_ERR_INVALID_ARG)])
def test_refuses(lib, kw, want):
    assert lib.ls_extend_drafts(*{**BASE, **kw}.values(), None) == want


def test_calls_by_member_still_need_counts(lib):
    base = {k: v for k, v in BASE.items() if k != "added"}
    assert lib.ls_extend_pages_by_member(*{**base, "add": None}.values(), None) == B.LS_ERR_INVALID_ARG


def test_no_members(lib):
    assert lib.ls_extend_drafts(None, 0, 8, 64, 100, None, None, None, 0, A, 0, 1, 8, None, None, None, A, None,
                                None) == B.LS_OK
