"""CPU tests of what surrounds the kernels of the query/key stage and the decode step: the
order of dependent launches, workspaces, and the values that the smoke run compares with."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "response_replay_gb300", "csrc")
WAIT = 'griddepcontrol.wait;'


@pytest.mark.parametrize("name", sorted(f for f in os.listdir(CSRC) if f.endswith(".cu")))
def test_dependent_grids_wait_before_every_exit(name):
    """A grid that is launched while the one before it still runs may end only after that
    one: whatever comes next on the stream waits for the dependent grid alone.  So no block
    leaves such a kernel ahead of its wait."""
    with open(os.path.join(CSRC, name)) as f:
        kernels = re.split(r"(?m)^(?=.*__global__)", re.sub(r"//[^\n]*", "", f.read()))[1:]
    for k in kernels:
        if WAIT not in k:
            continue
        before = k[:k.rindex(WAIT)]
        for m in re.finditer(r"\breturn;", before):
            assert WAIT in before[before.rindex("{", 0, m.start()):m.start()], before[m.start() - 80:m.end()]
