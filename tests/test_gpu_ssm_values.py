"""The scan at parameters and inputs of unusual values, against the plain 64-bit reference."""
import pytest
import torch

import ssm_ref as ref
from gateddeltanet_linear_attention_gb300 import gdn
from test_gpu_ssm import Batch

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("act", ["fp32", "bf16"])
@pytest.mark.parametrize("P", [64, 128])
@pytest.mark.parametrize("what,fill", [("A_log", NAN), ("dt_bias", NAN), ("D", NAN), ("D", INF), ("A_log", INF), ("A_log", -INF)])
def test_parameters_that_are_not_finite(act, P, what, fill):
    """One head's parameter: the other heads are right, and what it reaches is not finite.  (A_log of
    +inf forgets at once and of -inf never: both have values.)"""
    b = Batch([200, 600, 40], H=4, G=2, N=64, P=P, act=act, seed=70)
    getattr(b, what)[1] = fill
    y, out = b.run()
    for n, L in enumerate(b.lens):
        s, e = int(b.cu[n]), int(b.cu[n + 1])
        val, mag, S, M = b.reference(n)
        rel = (8 * L + b.N + 64) * ref.U32
        rel_y = rel + (2 * 2.0 ** -8 + 2 * 128 * 60 * ref.U32 if act == "bf16" else 0)
        for got, v, m, r, name in ((y[s:e].cpu(), val.reshape(L, -1), mag.reshape(L, -1), rel_y, "y"), (out[n].cpu(), S, M, rel, "state")):
            ok = v.isfinite()
            assert not got[~ok].isfinite().any(), "%s of sequence %d" % (name, n)
            ref.check(got[ok], v[ok], m[ok], r, name)
    assert gdn.gdn_device_error() == 0
