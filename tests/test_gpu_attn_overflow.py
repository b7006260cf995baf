"""Attention of new tokens whose scores leave the range of 32-bit numbers."""
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
