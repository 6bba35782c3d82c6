"""The query/key stage at the ends of what it takes: eps beside the largest rows, gradients
whose products with the rows pass fp32."""
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


@pytest.mark.parametrize("inter", [False, True])
def test_large_gradients_of_large_rows(cuda, inter):
    """Gradients and rows whose products pass fp32 where neither's own squares' sum does, and
    rows of gradients near fp32's end; the result fits bf16 in every one."""
    s = Stage(cuda, 24, 2, 1, 64, interleaved=inter, seed=19)
    dy = [torch.randn(24, h, 128, device=cuda) for h in (2, 1)]
    for t, (fx, fg) in enumerate([(1e17, 1e22), (1e18, 1e21), (1e10, 1e30), (1e25, 1e20), (1e30, 1e36),
                                  (3e17, 3e20)]):
        s.buf[t] *= fx
        for d in dy:
            d[t] *= fg
    out = api.qk_norm_rope_bwd(s.q, s.k, s.pos, s.rot, *dy)
    for i, x in enumerate((s.q, s.k)):
        dx, dxb, _, _ = qo.bwd(qo.f64(x), qo.f64(dy[i]), 1.0, 0.0, 1e-6, *s.rotary())
        assert torch.isfinite(out[i].float()).all()
        close(out[i], dx, dxb)
    # the other rows keep the bits that they have without them
    rest = api.qk_norm_rope_bwd(s.q[6:], s.k[6:], s.pos[:, 6:].contiguous(), s.rot, dy[0][6:], dy[1][6:])
    assert torch.equal(rest[0], out[0][6:]) and torch.equal(rest[1], out[1][6:])
    mixed = [d[5:7].contiguous() for d in dy]  # a pair of tokens, one of them such a row
    pair = api.qk_norm_rope_bwd(s.q[5:7], s.k[5:7], s.pos[:, 5:7].contiguous(), s.rot, *mixed)
    assert torch.equal(pair[0][1], rest[0][0]) and torch.equal(pair[1][1], rest[1][0])
    ok()
