"""A process whose first call of an operator is a captured one: nothing has to be called before."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import sys
sys.path[:0] = [%r, %r]
import torch
from gateddeltanet_linear_attention_gb300 import gdn
from test_gpu_ssm import Batch

what = sys.argv[1]
gen = torch.Generator(device="cuda").manual_seed(1)
r = lambda *s, dtype=torch.bfloat16: torch.randn(s, generator=gen, device="cuda").to(dtype)
outs = []
if what in ("bf16", "fp32"):
    b = Batch([700, 31], H=2, G=1, act=what, seed=11)
    b.upload()
    outs = [torch.zeros(b.rows, b.H * b.P, dtype=b.act, device="cuda"), torch.zeros_like(b.d_state)]
    call = lambda: b.launch(*outs)
elif what in ("conv", "step"):
    cfg = gdn.make_ssm_config(1, 2, 64, 64, n_slots=3)
    CH, n = 256, 3
    x, w, u, A = r(n, CH), r(CH, 4), r(n, 2), torch.zeros(2, device="cuda")
    hist0, state0 = r(n, CH, 3), r(n, 2, 64, 64, dtype=torch.float32)
    hist, state, cu = hist0.clone(), state0.clone(), torch.tensor([0, 1, 1, 3], dtype=torch.int32, device="cuda")
    outs = [torch.zeros_like(x) if what == "conv" else r(n, 128), hist, state]
    ws = torch.empty(gdn.gdn_ssm_workspace_size(cfg, n, n), dtype=torch.uint8, device="cuda")
    def call():
        hist.copy_(hist0)
        state.copy_(state0)
        if what == "conv":
            gdn.gdn_ssm_conv_prefill(cfg, x, cu, w, None, hist, None, outs[0])
        else:
            gdn.gdn_ssm_decode(cfg, x, u, w, hist, A, state, outs[0], ws)
else:
    p, q, w = r(9, 520), r(9, 520), torch.ones(520, device="cuda")
    k = torch.ones(2, 9, device="cuda")
    outs = [torch.zeros_like(p), torch.zeros_like(p), torch.zeros(2, 520, device="cuda")]
    ws = torch.empty(gdn.gdn_block_norm_workspace_size(9, 520), dtype=torch.uint8, device="cuda")
    if what == "norm":
        call = lambda: gdn.gdn_block_norm(q, w, outs[0], block=p, res_out=outs[1], w_post=w)
    else:
        call = lambda: gdn.gdn_block_norm_backward(q, k[0], w, p, q, outs[0], outs[2][0], block=p, rstd_post=k[1], w_post=w, d_block=outs[1],
                                                   dw_post=outs[2][1], workspace=ws)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in outs]
assert any(float(t.float().abs().sum()) > 0 for t in got)
call()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, outs))
assert gdn.gdn_device_error() == 0
print("same")
"""


@pytest.mark.parametrize("what", ["bf16", "fp32", "conv", "step", "norm", "norm_bwd"])
def test_first_call_in_a_capture(what):
    r = subprocess.run([sys.executable, "-c", SCRIPT % (ROOT, os.path.join(ROOT, "tests")), what], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
