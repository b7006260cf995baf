"""Operators of the attention layers on values that leave the range of 32-bit numbers: scores, and squares of heads."""
import math

import pytest
import torch

from test_gpu_attn_decode import Cache
from gateddeltanet_linear_attention_gb300 import gdn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act,Hq,Hkv,D,tokens", [("fp32", 2, 1, 64, 1), ("fp32", 4, 1, 128, 8), ("fp32", 16, 1, 256, 8), ("bf16", 2, 1, 64, 1), ("bf16", 4, 1, 256, 2),
                                                 ("bf16", 8, 1, 128, 8), ("bf16", 16, 1, 256, 8)])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_beyond_the_range(act, Hq, Hkv, D, tokens, sign):
    """Above the range a row is NaN, in a sequence of one tile as in longer ones and in parts; below it its tokens count as masked."""
    c = Cache([1, 20, 33, 200, 9000, 0], Hq, Hkv, D, 16, act, tokens, seed=1)
    c.q = sign * (c.q.abs() + 0.5)
    for r, K in enumerate(c.K):
        K.copy_(K.abs() + 0.5)
        for i in range(K.shape[1]):
            c.kp[c.table[r, i // 16], :, i % 16] = K[:, i]
    c.upload()
    out, lse = c.run(scale=1e38)                        # every score is 16 at least, of either sign
    sees = torch.tensor([length - tokens + 1 + j > 0 for length in c.lens for j in range(tokens)], device="cuda")
    if sign > 0:
        assert torch.isnan(out[sees]).all() and torch.isnan(lse[sees]).all()
        out, lse = out[~sees], lse[~sees]
    assert not out.any() and (lse == -math.inf).all()
    assert gdn.gdn_device_error() == 0


@pytest.mark.parametrize("D,R,interleaved", [(64, 64, False), (128, 20, False), (256, 64, True)])
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
def test_squares_beyond_the_range(act, D, R, interleaved):
    """Head vectors whose squares leave the range have norms and gradients of 0; their neighbours are as without them."""
    T, Hq, Hkv = 40, 6, 2
    cfg = gdn.make_attn_config(Hq, Hkv, D, act="bf16" if act == torch.bfloat16 else "fp32")
    g = torch.Generator(device="cuda").manual_seed(D)
    q, dq_out, k, dk_out = (torch.randn(T, h, D, generator=g, device="cuda").to(act) for h in (Hq, Hq, Hkv, Hkv))
    w = 1 + 0.1 * torch.randn(2, D, generator=g, device="cuda")
    f = (1000.0 ** (-torch.arange(0, R, 2, device="cuda").double() / R)).float()
    kw = dict(w_q=w[0], w_k=w[1], interleaved=interleaved)

    def run():
        q_out, dq, k_out, dk = (torch.full_like(x, 7.0) for x in (q, q, k, k))
        gdn.gdn_attn_prep(cfg, q, k, q_out, f, k_out=k_out, **kw)
        gdn.gdn_attn_prep_backward(cfg, q, k, dq_out, dk_out, f, dq=dq, dk=dk, **kw)
        return q_out, dq, k_out, dk
    clean = run()
    q[5, 3] *= 1e20
    k[17, 1, 9] = -1e20
    for x, want, at in zip(run(), clean, ((5, 3), (5, 3), (17, 1), (17, 1))):
        want[at] = 0
        assert torch.equal(x, want)
    assert gdn.gdn_device_error() == 0
