"""The block norms over more rows than run at once: every form's walk over the rows (loads of the next
row ahead, alternating stages and sum buffers, weight gradients of several rows), with bounds that
do not grow with the width.

A sum over a row is at most 16 terms in a thread, 5 steps in a warp and 5 over warps: 26 roundings and a
square's, halved by the root, then products, quotients and exponentials: below 64 of them for what
needs the sums once, and 2 + 1.2 |gate| units in the last place for a 16-bit gate's sigmoid (|gate| < 6)."""
import pytest
import torch

import ssm_ref as ref
from gateddeltanet_linear_attention_gb300 import gdn
from test_gpu_block_norm import BF, F32, make, up

pytestmark = pytest.mark.gpu
REL = 96 * ref.U32
# Gradients need two sums one after the other; those of the weights also one over the rows (in a
# CTA at most rows / CTAs, then 32 at a time over the CTAs, then 5 steps).
REL_BWD = 256 * ref.U32


def rows_for(dim):
    """More than two rows for each CTA (or warp) of the widest grid: 8 of 128 threads an SM, a warp a row,
    up to 512 wide, then 1,024 threads an SM, 16 elements a thread."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return int(2.3 * sms * (32 if dim <= 512 else max(1, 1024 // ((dim + 15) // 16 + 31 & ~31))))


@pytest.mark.parametrize("act,res", [(F32, F32), (BF, F32), (BF, BF)])
@pytest.mark.parametrize("dim,pad", [(300, 0), (304, 0), (1111, 0), (1600, 6), (2000, 0), (3000, 0), (4096, 0), (5120, 0), (8192, 0), (8200, 0),
                                     (9001, 0)])
def test_more_rows_than_run_at_once(act, res, dim, pad):
    rows, scale, eps = rows_for(dim), 0.7, 1e-5
    d = make(rows, dim, act, res, pad=pad, seed=1)
    t = {k: up(v) for k, v in d.items()}
    ro, h = torch.full((rows, dim), 7.0, dtype=res, device="cuda"), torch.full((rows, dim), 7.0, dtype=act, device="cuda")
    k1, k2 = torch.zeros(2, rows, device="cuda")
    gdn.gdn_block_norm(t["residual"], t["w_pre"], h, block=t["block"], res_out=ro, w_post=t["w_post"], gate=t["gate"], res_scale=scale, eps=eps,
                       rstd_post=k1, rstd_pre=k2)
    want = ref.norm(d["block"], d["gate"], d["residual"], d["w_post"], d["w_pre"], eps, 0.0, scale)
    for name, got in (("res_out", ro), ("h", h), ("rstd_post", k1), ("rstd_pre", k2)):
        ref.check(got, *want[name], REL, name)
    out = dict(d_residual=torch.full_like(ro, 7.0), d_block=torch.full_like(h, 7.0), d_gate=torch.full_like(h, 7.0),
               dw_post=torch.full((dim,), 7.0, device="cuda"), dw_pre=torch.full((dim,), 7.0, device="cuda"))
    ws = torch.full((gdn.gdn_block_norm_workspace_size(rows, dim),), 0xFF, dtype=torch.uint8, device="cuda")
    gdn.gdn_block_norm_backward(ro, k2, t["w_pre"], t["dh"], t["d_res_out"], block=t["block"], rstd_post=k1, w_post=t["w_post"],
                                gate=t["gate"], res_scale=scale, workspace=ws, **out)
    want = ref.norm_backward(d["block"], d["gate"], ro.cpu(), d["w_post"], d["w_pre"], k1.cpu(), k2.cpu(), d["dh"], d["d_res_out"], 0.0, scale)
    for name, got in out.items():
        ref.check(got, *want[name], REL_BWD, name)
