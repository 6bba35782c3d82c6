"""GPU parity of the token statistics on the longest rows, past 2^31 bytes each."""
import pytest
import torch

import rollout_oracle as ro
from response_replay_gb300 import binding as B
from response_replay_gb300 import torch_api as api

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,V,offset", [(torch.bfloat16, 2 ** 30, 0), (torch.bfloat16, 2 ** 30 - 7, 3),
                                         (torch.float32, 2 ** 29 + 5, 1)])
def test_rows_past_2_to_31_bytes(cuda, dt, V, offset):
    """A row in one piece (with many rows in the call, of which the others are padding, whose logits
    are not read) and cut into parts, with alternatives."""
    z = torch.empty(V + offset, dtype=dt, device=cuda).normal_()[offset:]
    at = torch.tensor([V - 1, 5, V // 2, V - 2], device=cuda)
    z[at] = torch.tensor([24.0, 23.0, 22.0, 21.0], device=cuda).to(dt)  # half and more of the weight
    # in 64 bits, piece by piece
    s = e = a1 = a2 = 0.0
    for piece in z.split(2 ** 26):
        x = piece.double() - 24
        p = x.exp()
        s, e, a2 = s + float(p.sum()), e + float((p * x).sum()), a2 + float((p * x * x).sum())
    lse = 24 + torch.log(torch.tensor(s, dtype=torch.float64)).item()
    h, a1, a2 = (lse - 24) - e / s, -e / s, a2 / s
    # rollout_oracle.stat_bounds' bounds; a streamed thread's chain of V / (values of 64 bytes x 384),
    # with the rescales
    chain = V / (64 // dt.itemsize * 384) + 80
    es = 2.0 ** -21 + chain * ro.U32 + 3 * ro.U32 * a1
    e_lse = es + 2.0 ** -21 + ro.U32 * lse
    e_h = es + 2.0 ** -21 + a1 * (2.0 ** -21 + es + (chain + 8) * ro.U32) + 3 * ro.U32 * a2 + 4 * ro.U32 * h
    T = 77  # rows enough that none is cut, on 152 SMs
    y = torch.full((T,), -1, dtype=torch.int32, device=cuda)
    y[0] = V - 1
    out = [torch.full((T,), 5.0, device=cuda) for _ in range(3)]
    st = torch.cuda.current_stream().cuda_stream
    code = B.LS_BF16 if dt is torch.bfloat16 else B.LS_FP32
    # the rows behind the first are padding: no memory stands behind them, none is read
    B.ls_token_logp_fwd(z.data_ptr(), code, T, V, V, y.data_ptr(), 1.0, 0, *(t.data_ptr() for t in out), None,
                        None, None, 0, st)
    logp, l32, ent = out
    one = api.token_logp_fwd(z[None], y[:1], top=4)
    assert B.ls_last_device_error(0) == B.LS_OK
    for got in ((logp[:1], l32[:1], ent[:1]), one[:3]):
        assert abs(float(got[1]) - lse) <= e_lse
        assert abs(float(got[0]) - (24 - lse)) <= e_lse + ro.U32 * abs(24 - lse)
        assert abs(float(got[2]) - h) <= e_h
    assert one[4].tolist() == [at.tolist()]
    for t in out:
        assert bool((t[1:] == 0).all())
