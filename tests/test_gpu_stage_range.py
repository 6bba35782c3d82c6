"""The query/key stage at the ends of what it takes: eps beside the largest rows."""
import pytest
import torch

import qk_oracle as qo
from response_replay_gb300 import torch_api as api
from test_gpu_qk_norm_rope import Stage, close, ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("eps", [1e30, 1e34, 2e36, 3e38])
def test_large_eps(cuda, eps, inter):
    """An eps of the size of a row's mean square, below and above where the squares pass fp32."""
    s = Stage(cuda, 24, 2, 1, 64, interleaved=inter, seed=18)
    s.buf[2] *= 1e15
    s.buf[3] *= 1e17
    s.buf[4] *= 1e18
    s.buf[5] *= 3e18
    s.buf[6] *= 1e19
    s.buf[7] *= 1e25
    s.buf[8] = 3e38
    q, k, _ = api.qk_norm_rope_fwd(s.q, s.k, None, s.pos, s.rot, s.wq, s.wk, eps=eps)
    close(q, *qo.fwd(qo.f64(s.q), qo.f64(s.wq), 0.0, eps, *s.rotary()))
    close(k, *qo.fwd(qo.f64(s.k), qo.f64(s.wk), 0.0, eps, *s.rotary()))
    dy = [torch.randn(24, h, 128, device=cuda) for h in (2, 1)]
    out = api.qk_norm_rope_bwd(s.q, s.k, s.pos, s.rot, *dy, wq=s.wq, wk=s.wk, eps=eps)
    for i, (x, w) in enumerate(((s.q, s.wq), (s.k, s.wk))):
        dx, dxb, dw, dwb = qo.bwd(qo.f64(x), qo.f64(dy[i]), qo.f64(w), 0.0, eps, *s.rotary())
        close(out[i], dx, dxb)
        close(out[3 + i], dw, dwb)
    ok()
