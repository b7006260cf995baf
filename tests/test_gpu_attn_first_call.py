"""A process whose first call of an operator of the attention layers is a captured one: nothing has to be called before, and the
eager call behind it gives the same."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import sys
sys.path[:0] = [%r]
import torch
from gateddeltanet_linear_attention_gb300 import gdn

what, act, tokens = sys.argv[1], sys.argv[2], int(sys.argv[3])
dt = torch.bfloat16 if act == "bf16" else torch.float32
gen = torch.Generator(device="cuda").manual_seed(1)
r = lambda *s: torch.randn(s, generator=gen, device="cuda").to(dt)
ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
Hq, Hkv, D, page, n_pages, n_rows, mp = 8, 1, 128, 16, 64, 5, 20
cfg = gdn.make_attn_config(Hq, Hkv, D, page_size=page, act=act, n_pages=n_pages, n_rows=n_rows, max_pages=mp)
kp0, vp0 = r(n_pages, Hkv, page, D), r(n_pages, Hkv, page, D)
kp, vp = kp0.clone(), vp0.clone()
lens0, table0, refs0 = [300, 17, 0, 40, 0], [[-1] * mp for _ in range(n_rows)], [0] * n_pages
free = iter(range(n_pages))
for row, L in enumerate(lens0):
    for p in range((L + page - 1) // page):
        table0[row][p] = next(free)
        refs0[table0[row][p]] = 1
start = [ints(table0), ints(lens0), ints(refs0)]
table, lens, refs = (t.clone() for t in start)
freq = torch.linspace(1.0, 0.01, 32, device="cuda")
w = torch.ones(D, device="cuda")
lanes = [ints([9] * n_pages) for _ in range(3)]
page_ws = torch.empty(gdn.gdn_page_workspace_size(cfg, n_pages), dtype=torch.uint8, device="cuda")
n = n_rows * tokens
if what == "prep":
    q, k, v = r(n, Hq, D), r(n, Hkv, D), r(n, Hkv, D)
    lens = start[1] = ints([300, 17, 16, 40, 20])
    start[0][2, 0], start[0][4, 0], start[0][4, 1] = 50, 51, 52
    outs = [torch.zeros_like(q), kp, vp]
    op = lambda: gdn.gdn_attn_prep(cfg, q, k, outs[0], freq, v=v, k_pages=kp, v_pages=vp, page_table=table, lens=lens, tokens=tokens, w_q=w, w_k=w)
elif what == "prep_bwd":
    q, k = r(n, Hq, D), r(n, Hkv, D)
    outs = [torch.zeros_like(q), torch.zeros_like(k), torch.zeros(D, device="cuda"), torch.zeros(D, device="cuda")]
    ws = torch.empty(gdn.gdn_attn_prep_workspace_size(cfg, n), dtype=torch.uint8, device="cuda")
    op = lambda: gdn.gdn_attn_prep_backward(cfg, q, k, q, k, freq, dq=outs[0], dk=outs[1], dw_q=outs[2], dw_k=outs[3], w_q=w, w_k=w, tokens=tokens,
                                            workspace=ws)
elif what == "decode":
    q = r(n, Hq, D)
    outs = [torch.zeros_like(q), torch.zeros(n, Hq, device="cuda")]
    ws = torch.empty(gdn.gdn_attn_workspace_size(cfg, n_rows, tokens), dtype=torch.uint8, device="cuda")
    op = lambda: gdn.gdn_attn_decode(cfg, q, kp, vp, table, lens, outs[0], ws, tokens=tokens, lse=outs[1])
else:
    outs = [table, lens, refs, *lanes, kp, vp]
    three = [t[:3] for t in lanes]
    op = {"resize": lambda: gdn.gdn_page_resize(cfg, table, lens, refs, ints3, new3, *three, page_ws),
          "fork": lambda: gdn.gdn_page_fork(cfg, table, lens, refs, src2, dst2),
          "compact": lambda: gdn.gdn_page_compact(cfg, table, lens, refs, table, refs, lanes[0], lanes[1], page_ws),
          "copy": lambda: gdn.gdn_page_copy(cfg, kp, vp, kp, vp, src2, dst2)}[what]
    ints3, new3, src2, dst2 = ints([0, 2, 3]), ints([280, 33, 0]), ints([0, 1]), ints([2, 4])
    if what == "compact":
        start[0][0, 0], start[2][0], start[2][60] = 60, 0, 1

def call():
    for t, t0 in ((table, start[0]), (lens, start[1]), (refs, start[2]), (kp, kp0), (vp, vp0)):
        t.copy_(t0)
    op()

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    call()
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in outs]
assert all(float(t.float().abs().sum()) > 0 for t in got)
call()
torch.cuda.synchronize()
assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, outs))
assert gdn.gdn_device_error() == 0
print("same")
"""


@pytest.mark.parametrize("what,act,tokens", [("prep", "bf16", 1), ("prep", "fp32", 3), ("prep_bwd", "bf16", 2), ("decode", "bf16", 1),
                                             ("decode", "bf16", 8), ("decode", "fp32", 2), ("resize", "bf16", 1), ("fork", "bf16", 1),
                                             ("compact", "bf16", 1), ("copy", "bf16", 1)])
def test_first_call_in_a_capture(what, act, tokens):
    r = subprocess.run([sys.executable, "-c", SCRIPT % ROOT, what, act, str(tokens)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]
