"""Gradients of the norms and the rotation in the place of the gradients that they are computed from."""
import pytest
import torch

from gateddeltanet_linear_attention_gb300 import gdn

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,Hq,Hkv,D,R,interleaved", [(700, 6, 2, 64, 64, False), (333, 5, 1, 128, 20, False), (40, 4, 2, 256, 12, True), (1, 3, 1, 64, 64, False)])
@pytest.mark.parametrize("act", [torch.bfloat16, torch.float32])
def test_contiguous_gradients_in_place(T, Hq, Hkv, D, R, interleaved, act):
    """The bits of the call with outputs of its own; the same memory as a view with other distances is refused and left."""
    cfg = gdn.make_attn_config(Hq, Hkv, D, act="bf16" if act == torch.bfloat16 else "fp32")
    g = torch.Generator(device="cuda").manual_seed(T)
    q, dq_out = (torch.randn(T, Hq, D, generator=g, device="cuda").to(act) for _ in range(2))
    k, dk_out = (torch.randn(T, Hkv, D, generator=g, device="cuda").to(act) for _ in range(2))
    w = 1 + 0.1 * torch.randn(2, D, generator=g, device="cuda")
    f = (1000.0 ** (-torch.arange(0, R, 2, device="cuda").double() / R)).float()
    kw = dict(w_q=w[0], w_k=w[1], interleaved=interleaved)
    dq, dk = torch.empty_like(q), torch.empty_like(k)
    gdn.gdn_attn_prep_backward(cfg, q, k, dq_out, dk_out, f, dq=dq, dk=dk, **kw)
    wide = torch.zeros(T, 2 * Hq, D, dtype=act, device="cuda")
    start = wide.view(-1)[:T * Hq * D].view(T, Hq, D)
    start.copy_(dq_out)
    if T > 1:
        keep = wide.clone()
        with pytest.raises(gdn.GDNError):
            gdn.gdn_attn_prep_backward(cfg, q, k, start, dk_out, f, dq=wide[:, :Hq], dk=torch.empty_like(k), **kw)
        assert torch.equal(wide, keep)
    gdn.gdn_attn_prep_backward(cfg, q, k, start, dk_out, f, dq=start, dk=dk_out, **kw)
    assert torch.equal(start, dq) and torch.equal(dk_out, dk) and not wide.view(-1)[T * Hq * D:].any()
    assert gdn.gdn_device_error() == 0
