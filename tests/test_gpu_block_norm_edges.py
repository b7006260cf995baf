"""The block norms at edges of their arguments."""
import pytest
import torch

import ssm_ref as ref
from gateddeltanet_linear_attention_gb300 import gdn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dim", [72, 4096, 77])
def test_residuals_of_32_bits_have_gates_of_32_bits(dim):
    """r' of a zero residual and a plain block is res_scale sigmoid(gate) block: exponential (2 units in
    the last place, 4 half steps), sum, quotient, three products: 12 half steps at most, whatever the
    gate's size."""
    rows = 40
    g = torch.Generator().manual_seed(80)
    p = torch.randn(rows, dim, generator=g).to(BF)
    gate = (torch.rand(rows, dim, generator=g) * 100 - 70).to(BF)
    r = torch.zeros(rows, dim)
    out = torch.empty(rows, dim, device="cuda")
    gdn.gdn_block_norm(r.cuda(), block=p.cuda(), gate=gate.cuda(), res_scale=0.7, res_out=out)
    ref.check(out, *ref.norm(p, gate, r, None, None, 0.0, 0.0, 0.7)["res_out"], 12 * ref.U32, "r'")


@pytest.mark.parametrize("act,res", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("cols", [64, 1])
def test_gates_of_infinity(act, res, cols):
    """Open and shut for good: r + n and r; a NaN is the row's (or the element's) own."""
    g = torch.Generator().manual_seed(81)
    p, r = torch.randn(6, 64, generator=g).to(act), torch.randn(6, 64, generator=g).to(res)
    gate = torch.zeros(6, cols, dtype=act)
    gate[0], gate[1], gate[2, 0], gate[3], gate[4] = float("inf"), float("-inf"), float("nan"), 300.0, -300.0
    out = torch.empty(6, 64, dtype=res, device="cuda")
    gdn.gdn_block_norm(r.cuda(), block=p.cuda(), gate=gate.cuda(), res_out=out)
    want = ref.norm(p, gate, r, None, None, 0.0, 0.0, 1.0)["res_out"]
    ref.check(out, *want, 12 * ref.U32, "r'")
    assert torch.equal(out.cpu().isnan(), want[0].isnan())
    assert torch.equal(out[1].cpu(), r[1]) and torch.equal(out[4].cpu(), r[4])


@pytest.mark.parametrize("act,res", [(BF, BF), (BF, F32), (F32, F32)])
@pytest.mark.parametrize("cols", [64, 1])
def test_gradients_of_gates_that_are_shut(act, res, cols):
    """Gates below -80, of -inf and of +inf: what passes them is as small as the sigmoid, or nothing.  The
    bound is that of gates that are all but shut: a dozen roundings, two sums over 64 elements, and the fast exponential's
    2 + 1.2 |x| units in the last place."""
    x = torch.tensor([-70.0, -82.0, -87.0, -95.0, -200.0, float("-inf"), float("inf"), 90.0])
    g = torch.Generator().manual_seed(82)
    p, u, dro, = torch.randn(8, 64, generator=g).to(act), torch.randn(8, 64, generator=g).to(res), torch.randn(8, 64, generator=g).to(res)
    gate = x[:, None].expand(8, cols).contiguous().to(act)
    w, k = 1 + 0.2 * torch.randn(64, generator=g), 1 + torch.rand(8, generator=g)
    out = dict(d_block=torch.empty(8, 64, dtype=act, device="cuda"), d_gate=torch.empty(8, cols, dtype=act, device="cuda"),
               dw_post=torch.empty(64, device="cuda"))
    ws = torch.empty(gdn.gdn_block_norm_workspace_size(8, 64), dtype=torch.uint8, device="cuda")
    gdn.gdn_block_norm_backward(u.cuda(), d_res_out=dro.cuda(), block=p.cuda(), rstd_post=k.cuda(), w_post=w.cuda(), gate=gate.cuda(),
                                workspace=ws, **out)
    want = ref.norm_backward(p, gate, u, w, None, k, None, None, dro, 0.0, 1.0)
    for name, got in out.items():
        ref.check(got, *want[name], (2 * 64 + 64 + 2 * (2 + 1.2 * 88)) * ref.U32, name)


def test_no_rows_in_a_graph_behind_a_copy():
    """Zero weight gradients of a batch without rows, captured behind an operation that is no kernel."""
    e, w = torch.empty(0, 64, device="cuda"), torch.ones(64, device="cuda")
    a, dw = torch.ones(1 << 20, device="cuda"), torch.full((64,), 7.0, device="cuda")
    b = torch.zeros_like(a)
    k = torch.empty(0, device="cuda")
    ws = torch.empty(gdn.gdn_block_norm_workspace_size(0, 64), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.copy_(a)
        gdn.gdn_block_norm_backward(e, k, w, e, dw_pre=dw, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert (dw == 0).all() and (b == 1).all()
