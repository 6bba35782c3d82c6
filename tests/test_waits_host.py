"""CPU test of a hand-over between warps that may give up: a model of the named barriers, and that the
kernel goes by it."""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "response_replay_gb300", "csrc")
WARPS, ITEMS = 5, 6


def consumer(s, w, leaves_at, arrives):
    """Steps of a consumer warp: a hand-over an item, until there is none or it gives up."""
    q = 0
    while q < ITEMS:
        yield lambda: True
        if q == leaves_at or (s["abort"] and s["rng"].random() < 0.5):
            s["abort"] = True
            break
        # the buffers of the item two before (a wait with a limit: it goes on all the same)
        yield lambda q=q: s["taken"] >= q - 1 or s["abort"]
        s["count"][q & 1] += 1
        q += 1
    if s["abort"] and arrives:
        s["count"][q & 1] += 1


def last(s, looks):
    for q in range(ITEMS):
        yield lambda: True
        if s["abort"] and looks:
            return
        yield lambda q=q: s["count"][q & 1] >= WARPS
        s["count"][q & 1] -= WARPS
        s["taken"] = q + 1


def ends(seed, arrives=True, looks=True):
    """Whether all warps end, in a random order of their steps, when up to two give up."""
    rng = random.Random(seed)
    s = {"abort": False, "count": [0, 0], "taken": 0, "rng": rng}
    give_up = {w: rng.randrange(ITEMS) for w in rng.sample(range(WARPS), rng.randint(0, 2))}
    live = [consumer(s, w, give_up.get(w), arrives) for w in range(WARPS)] + [last(s, looks)]
    wait = [next(g) for g in live]
    while live:
        ready = [i for i, c in enumerate(wait) if c()]
        if not ready:
            return False
        i = rng.choice(ready)
        try:
            wait[i] = next(live[i])
        except StopIteration:
            del live[i], wait[i]
    return True


def test_every_warp_ends():
    assert all(ends(seed) for seed in range(4000))


@pytest.mark.parametrize("mistake", [dict(arrives=False), dict(looks=False)])
def test_the_model_sees_a_missing_part(mistake):
    assert not all(ends(seed, **mistake) for seed in range(4000))


def test_the_kernel_has_both_parts():
    with open(os.path.join(CSRC, "token_logp.cu")) as f:
        src = f.read()
    kernel = src[src.index("logp_fwd(const FwdArgs a)"):]
    kernel = kernel[:kernel.index("\n}\n")]
    look = r"if \(__any_sync\(0xffffffffu, \*abort\)\) "
    assert len(re.findall(r"take_over\(", kernel)) == 1
    assert re.search(look + r"break;\s*take_over\(par\);", kernel)
    assert len(re.findall(r"hand_over\(", kernel)) == 2
    assert re.search(r"hand_over\(par\);\s*\}\s*" + look + r"hand_over\(q & 1\);$", kernel)
