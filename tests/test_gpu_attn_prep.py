"""Query and key norms with the position rotation on the GPU against the 64-bit forms: types, head layouts, strides, packed
and uniform batches, padding, far positions, the cache's places, gradients."""
import pytest
import torch

import attn_ref as ref
from attn_ref import U, half_step
from gateddeltanet_linear_attention_gb300 import gdn

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}

# 32-bit roundings of one output: the sum of squares of a head runs over 8 terms a lane and at most 5 halvings, 13 U, halved
# by the root; reciprocal root 4 U; three products and a weight's sum 4 U; the pair's two terms 2 U; cos and sin 4 U beside the
# angle's 2 U.  Together below 24 U of the sum of magnitudes.
FORWARD = 24 * U
# Backward: the same norm and rotation, then the row's mean (13 U) times two products, the difference and the scale.
BACKWARD = 48 * U


def cu_of(lens):
    return torch.tensor([0] + lens, dtype=torch.int32).cumsum(0).to(torch.int32)


class Case:
    def __init__(self, lens, Hq=4, Hkv=2, D=64, act="bf16", rotary=None, seed=0, extra=0, scale=1.0):
        self.lens, self.Hq, self.Hkv, self.D, self.act = lens, Hq, Hkv, D, DT[act]
        self.T = sum(lens) + extra
        g = torch.Generator().manual_seed(seed)
        self.r = lambda *s: torch.randn(s, generator=g)
        R = D if rotary is None else rotary
        qkv = (self.r(self.T, (Hq + 2 * Hkv) * D) * scale).to(self.act)
        self.qkv, self.parts = qkv, [Hq * D, Hkv * D, Hkv * D]
        self.q, self.k, self.v = self.split(qkv)
        self.w_q, self.w_k = 1 + 0.1 * self.r(D), 1 + 0.1 * self.r(D)
        self.f = (10000.0 ** (-torch.arange(0, R, 2).double() / R)).float() if R else None
        self.cfg = gdn.make_attn_config(Hq, Hkv, D, act=act)

    def split(self, t):
        return [x.unflatten(1, (-1, self.D)) for x in t.split(self.parts, 1)]

    def index(self):
        return torch.cat([torch.arange(n) for n in self.lens]) if self.lens else torch.zeros(0, dtype=torch.long)


def near(got, want, mag, c, act):
    got = got.double().cpu()
    tol = half_step(act) * want.abs() + c * mag + 1e-37
    bad = (got - want).abs() > tol
    assert not bad.any(), "%d of %d, worst %.3g of its bound" % (bad.sum(), bad.numel(), float(((got - want).abs() / tol).max()))


def freq(c):
    return c.f if c.f is not None else torch.zeros(0)


def gpu(*ts):
    return [None if t is None else t.cuda() for t in ts]


@pytest.mark.parametrize("act", ["bf16", "fp32"])
@pytest.mark.parametrize("D,rotary,interleaved", [(64, 64, False), (64, 24, False), (64, 20, True), (64, 2, False), (128, 128, False),
                                                  (128, 32, True), (128, 0, False), (128, 128, True), (256, 64, False), (256, 256, False),
                                                  (256, 250, False)])
def test_forward(act, D, rotary, interleaved):
    c = Case([5, 0, 17, 1], Hq=6, Hkv=3, D=D, act=act, rotary=rotary, seed=D + rotary)
    qkv, f, w_q, w_k, cu = gpu(c.qkv, c.f, c.w_q, c.w_k, cu_of(c.lens))
    q, k, _ = c.split(qkv)
    q_out, k_out = torch.full(c.q.shape, 9.0, dtype=c.act, device="cuda"), torch.full(c.k.shape, 9.0, dtype=c.act, device="cuda")
    gdn.gdn_attn_prep(c.cfg, q, k, q_out, f, k_out=k_out, cu_seqlens=cu, w_q=w_q, w_k=w_k, weight_offset=0.5, interleaved=interleaved)
    for got, x, w in ((q_out, c.q, c.w_q), (k_out, c.k, c.w_k)):
        near(got, *ref.prep(x, w, c.index(), freq(c), 0.5, 1e-6, interleaved), FORWARD, c.act)
    assert gdn.gdn_device_error() == 0


@pytest.mark.parametrize("act", ["bf16", "fp32"])
@pytest.mark.parametrize("w_q,w_k,keys", [(False, False, True), (True, False, True), (False, True, True), (True, False, False), (False, False, False)])
def test_without_norms_or_keys(act, w_q, w_k, keys):
    c = Case([9, 4], Hq=5, Hkv=1, D=128, act=act, seed=3)
    qkv, f, wq, wk, cu = gpu(c.qkv, c.f, c.w_q, c.w_k, cu_of(c.lens))
    q, k, _ = c.split(qkv)
    q_out, k_out = torch.empty(c.q.shape, dtype=c.act, device="cuda"), torch.empty(c.k.shape, dtype=c.act, device="cuda")
    gdn.gdn_attn_prep(c.cfg, q, k if keys else None, q_out, f, k_out=k_out if keys else None, cu_seqlens=cu, w_q=wq if w_q else None,
                      w_k=wk if w_k else None)
    near(q_out, *ref.prep(c.q, c.w_q if w_q else None, c.index(), freq(c)), FORWARD, c.act)
    if keys:
        near(k_out, *ref.prep(c.k, c.w_k if w_k else None, c.index(), freq(c)), FORWARD, c.act)


@pytest.mark.parametrize("act", ["bf16", "fp32"])
def test_far_positions(act):
    """Angles of far positions are as exact as near ones: 16,777,215 turns of frequencies down to 1e-6."""
    pos = torch.tensor([0, 1, 4095, 65537, 1 << 20, 12345678, (1 << 24) - 1])
    c = Case([len(pos)], D=128, act=act, seed=5)
    c.f = torch.cat([torch.tensor([1.0, 0.99999994, 3.7, 0.5, 1e-6]), torch.rand(59, generator=torch.Generator().manual_seed(1))])
    qkv, f, p = gpu(c.qkv, c.f, pos.to(torch.int32))
    q, k, _ = c.split(qkv)
    q_out, k_out = torch.empty(c.q.shape, dtype=c.act, device="cuda"), torch.empty(c.k.shape, dtype=c.act, device="cuda")
    gdn.gdn_attn_prep(c.cfg, q, k, q_out, f, k_out=k_out, positions=p)
    near(q_out, *ref.prep(c.q, None, pos, c.f), FORWARD, c.act)
    near(k_out, *ref.prep(c.k, None, pos, c.f), FORWARD, c.act)
    assert gdn.gdn_device_error() == 0


def test_positions_given():
    """Positions out of order; negative ones are padding, too large ones too and reported."""
    pos = torch.tensor([7, 3, -1, 7, 1 << 24, 0, -5])
    c = Case([3, 4], D=64, act="fp32", seed=6)
    qkv, f, w, p, cu = gpu(c.qkv, c.f, c.w_q, pos.to(torch.int32), cu_of(c.lens))
    q, k, _ = c.split(qkv)
    q_out, k_out = torch.full(c.q.shape, 9.0, device="cuda"), torch.full(c.k.shape, 9.0, device="cuda")
    gdn.gdn_attn_prep(c.cfg, q, k, q_out, f, k_out=k_out, positions=p, cu_seqlens=cu, w_q=w, eps=0.0)
    want, mag = ref.prep(c.q, c.w_q, pos, c.f, eps=0.0)
    live = (pos >= 0) & (pos < 1 << 24)
    near(q_out.cpu()[live], want[live], mag[live], FORWARD, c.act)
    assert not q_out.cpu()[~live].any() and not k_out.cpu()[~live].any()
    assert gdn.gdn_device_error() == gdn.DEVERR_PAGE and gdn.gdn_device_error() == 0


def test_rows_behind_the_last_sequence():
    c = Case([4, 6], D=128, extra=7, seed=8)
    qkv, f, cu = gpu(c.qkv, c.f, cu_of(c.lens))
    q, k, _ = c.split(qkv)
    q_out, k_out = torch.full(c.q.shape, 9.0, dtype=c.act, device="cuda"), torch.full(c.k.shape, 9.0, dtype=c.act, device="cuda")
    gdn.gdn_attn_prep(c.cfg, q, k, q_out, f, k_out=k_out, cu_seqlens=cu)
    assert (q_out[10:] == 9).all() and (k_out[10:] == 9).all()
    near(q_out[:10], *ref.prep(c.q[:10], None, c.index(), c.f), FORWARD, c.act)
    dq, dw = torch.full_like(q_out, 9.0), torch.empty(2, c.D, device="cuda")
    ws = torch.empty(gdn.gdn_attn_prep_workspace_size(c.cfg, c.T), dtype=torch.uint8, device="cuda")
    w = c.w_q.cuda()
    gdn.gdn_attn_prep_backward(c.cfg, q, None, q_out, None, f, dq=dq, dw_q=dw[0], w_q=w, cu_seqlens=cu, workspace=ws)
    assert (dq[10:] == 9).all()
    cut = [t[:10].contiguous() for t in (q, q_out)]
    gdn.gdn_attn_prep_backward(c.cfg, cut[0], None, cut[1], None, f, dq=torch.empty_like(cut[1]), dw_q=dw[1], w_q=w, cu_seqlens=cu, workspace=ws)
    assert torch.equal(dw[0], dw[1]) or (dw[0] - dw[1]).abs().max() < 1e-5 * dw[0].abs().max()
    assert gdn.gdn_device_error() == 0


@pytest.mark.parametrize("cu,bit", [([1, 4, 8], 1), ([0, 9, 8], 1), ([0, 4, 20], 1), ([0, -3, 8], 1), ([0, 4, 8], 0)])
def test_malformed_bounds(cu, bit):
    c = Case([8], D=64, seed=9)
    qkv, f = gpu(c.qkv, c.f)
    q, k, _ = c.split(qkv)
    q_out = torch.zeros(c.q.shape, dtype=c.act, device="cuda")
    gdn.gdn_attn_prep(c.cfg, q, None, q_out, f, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    assert gdn.gdn_device_error() == bit and torch.isfinite(q_out.float()).all()


@pytest.mark.parametrize("act,D,page", [("bf16", 64, 16), ("bf16", 128, 64), ("bf16", 256, 32), ("fp32", 128, 16), ("fp32", 64, 128)])
@pytest.mark.parametrize("uniform", [False, True])
def test_into_the_cache(act, D, page, uniform):
    """New tokens behind cached ones, through rows and shuffled pages; a padding lane; places of no new token stay."""
    new = [3, 3, 3, 3] if uniform else [3, 40, 0, 2]
    total, rows = [3, 57, 9, 20], [4, 0, 2, -1]
    c = Case(new, Hq=4, Hkv=2, D=D, act=act, rotary=D // 2, seed=page)
    n_pages, mp = 24, -(-64 // page) + 1
    g = torch.Generator().manual_seed(1)
    table, lens = torch.full((5, mp), -1, dtype=torch.int32), torch.zeros(5, dtype=torch.int32)
    order = torch.randperm(n_pages, generator=g).int()
    at = 0
    for r, t in zip(rows, total):
        if r >= 0:
            n = -(-t // page)
            table[r, :n] = order[at:at + n]
            lens[r] = t
            at += n
    cfg = gdn.make_attn_config(4, 2, D, page_size=page, act=act, n_pages=n_pages, n_rows=5, max_pages=mp)
    before = [torch.randn(n_pages, 2, page, D, generator=g).to(c.act) for _ in range(2)]
    qkv, f, w_q, w_k, kp, vp, tab, ln, rw, cu = gpu(c.qkv, c.f, c.w_q, c.w_k, *before, table, lens, torch.tensor(rows, dtype=torch.int32), cu_of(new))
    q, k, v = c.split(qkv)
    q_out, k_out = torch.full(c.q.shape, 9.0, dtype=c.act, device="cuda"), torch.full(c.k.shape, 9.0, dtype=c.act, device="cuda")
    gdn.gdn_attn_prep(cfg, q, k, q_out, f, k_out=k_out, v=v, k_pages=kp, v_pages=vp, page_table=tab, lens=ln, rows=rw, w_q=w_q, w_k=w_k,
                      **(dict(tokens=3) if uniform else dict(cu_seqlens=cu)))
    idx = torch.cat([torch.arange(t - n, t) for t, n in zip(total, new)])
    live = torch.cat([torch.full((n,), r >= 0) for r, n in zip(rows, new)])
    row = torch.cat([torch.full((n,), r) for r, n in zip(rows, new)])
    for got, x, w in ((q_out, c.q, c.w_q), (k_out, c.k, c.w_k)):
        want, mag = ref.prep(x, w, idx, c.f)
        near(got.cpu()[live], want[live], mag[live], FORWARD, c.act)
        assert not got.cpu()[~live].any()
    want_k, want_v = before[0].clone(), before[1].clone()
    for t in range(c.T):
        if live[t]:
            p, o = table[row[t], idx[t] // page], idx[t] % page
            want_k[p, :, o], want_v[p, :, o] = k_out[t].cpu(), c.v[t]
    assert torch.equal(kp.cpu(), want_k) and torch.equal(vp.cpu(), want_v)
    assert gdn.gdn_device_error() == 0


def test_bad_places_are_reported():
    """A row beyond the table, a page beyond the pool, a length beyond the table and more new tokens than the row has."""
    D, page, mp = 64, 16, 2
    c = Case([2] * 5, Hq=2, Hkv=1, D=D, act="fp32", seed=2)
    table = torch.tensor([[0, 1], [99, -1], [2, -1], [3, -1]], dtype=torch.int32)
    cfg = gdn.make_attn_config(2, 1, D, page_size=page, act="fp32", n_pages=6, n_rows=4, max_pages=mp)
    for lens, rows, bits, live in (([20, 5, 5, 5], [0, 2, 3, 7, -1], gdn.DEVERR_SLOT, [1, 1, 1, 0, 0]),
                                   ([20, 5, 5, 5], [0, 1, 2, 3, -1], gdn.DEVERR_PAGE, [1, 1, 1, 1, 0]),     # q' of a lost token is as ever
                                   ([33, 5, 5, 5], [0, 2, 3, -1, -1], gdn.DEVERR_PAGE, [0, 1, 1, 0, 0]),
                                   ([20, 5, 1, 5], [0, 2, 3, -1, -1], gdn.DEVERR_PAGE, [1, 2, 1, 0, 0])):
        qkv, f, tab, ln, rw = gpu(c.qkv, c.f, table, torch.tensor(lens, dtype=torch.int32), torch.tensor(rows, dtype=torch.int32))
        kp, vp = torch.zeros(2, 6, 1, page, D, device="cuda")
        q, k, v = c.split(qkv)
        q_out = torch.full(c.q.shape, 9.0, device="cuda")
        gdn.gdn_attn_prep(cfg, q, k, q_out, f, v=v, k_pages=kp, v_pages=vp, page_table=tab, lens=ln, rows=rw, tokens=2)
        assert gdn.gdn_device_error() == bits
        got = [int((q_out[2 * i:2 * i + 2].abs().amax((1, 2)) > 0).sum()) for i in range(5)]
        assert got == [{0: 0, 1: 2, 2: 1}[v] for v in live]
        assert not kp[4:].any() and not vp[4:].any()


def test_views():
    """Heads apart from each other (a gate between them) and head-major tensors; outputs of gradients likewise."""
    T, H, D = 11, 3, 128
    g = torch.Generator(device="cuda").manual_seed(0)
    wide = torch.randn(T, H, 2, D, generator=g, device="cuda").bfloat16()
    major = torch.randn(H, T, D, generator=g, device="cuda").bfloat16()
    cfg = gdn.make_attn_config(H, H, D)
    f = (100.0 ** (-torch.arange(64) / 64)).cuda()
    w = torch.rand(D, generator=g, device="cuda")
    outs = []
    for q, k in ((wide[:, :, 0], major.transpose(0, 1)), (wide[:, :, 0].contiguous(), major.transpose(0, 1).contiguous())):
        q_out, k_out = torch.empty(2, T, H, D, dtype=torch.bfloat16, device="cuda")
        gdn.gdn_attn_prep(cfg, q, k, q_out, f, k_out=k_out, w_q=w, w_k=w)
        dq, dk = torch.zeros(T, H, 2, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(H, T, D, dtype=torch.bfloat16, device="cuda")
        gdn.gdn_attn_prep_backward(cfg, q, k, q_out, k_out, f, dq=dq[:, :, 1], dk=dk.transpose(0, 1), w_q=w, w_k=w)
        assert not dq[:, :, 0].any()
        outs.append((q_out, k_out, dq, dk))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    for bad in (wide[:, :, 0, ::2], wide.flatten()[4:4 + T * H * D].view(T, H, D), torch.empty(T, H, D + 4, device="cuda").bfloat16()[..., :D]):
        with pytest.raises((gdn.GDNError, ValueError)):
            gdn.gdn_attn_prep(cfg, bad, None, q_out, f)
    with pytest.raises(ValueError):
        gdn.gdn_attn_prep(cfg, wide[:, :, 0].float(), None, q_out, f)
    with pytest.raises(ValueError):
        gdn.gdn_attn_prep(cfg, wide[:, :, 0].cpu(), None, q_out, f)
    with pytest.raises(ValueError):
        gdn.gdn_attn_prep(cfg, wide[:, :, 0], None, q_out, f, tokens=2)
    with pytest.raises(ValueError):
        gdn.gdn_attn_prep(cfg, wide[:, :, 0], None, q_out[:5], f)


@pytest.mark.parametrize("act", ["bf16", "fp32"])
@pytest.mark.parametrize("D,rotary,interleaved,w", [(64, 64, False, "qk"), (64, 12, False, "qk"), (128, 128, False, "qk"), (128, 20, True, "q"),
                                                    (256, 64, False, "k"), (256, 256, True, ""), (128, 0, False, "qk"), (64, 36, False, "")])
def test_backward(act, D, rotary, interleaved, w):
    c = Case([13, 0, 1, 30], Hq=6, Hkv=2, D=D, act=act, rotary=rotary, seed=rotary + 1)
    w_q, w_k = c.w_q if "q" in w else None, c.w_k if "k" in w else None
    d = [c.r(c.T, H, D).to(c.act) for H in (6, 2)]
    qkv, f, gq, gk, dqo, dko, cu = gpu(c.qkv, c.f, w_q, w_k, *d, cu_of(c.lens))
    q, k, _ = c.split(qkv)
    ws = torch.full((gdn.gdn_attn_prep_workspace_size(c.cfg, c.T),), 255, dtype=torch.uint8, device="cuda")
    res = []
    for _ in range(2):
        dq, dk, dw = torch.empty_like(dqo), torch.empty_like(dko), torch.empty(2, D, device="cuda")
        gdn.gdn_attn_prep_backward(c.cfg, q, k, dqo, dko, f, dq=dq, dk=dk, dw_q=dw[0] if w_q is not None else None,
                                   dw_k=dw[1] if w_k is not None else None, w_q=gq, w_k=gk, weight_offset=0.25, interleaved=interleaved,
                                   cu_seqlens=cu, workspace=ws)
        res.append((dq, dk, dw))
    for i, (x, wt, dd) in enumerate(((c.q, w_q, d[0]), (c.k, w_k, d[1]))):
        (dx, mag), want_w = ref.prep_backward(x, wt, dd, c.index(), freq(c), 0.25, 1e-6, interleaved)
        near(res[0][i], dx, mag, BACKWARD, c.act)
        if wt is not None:
            # a term errs by 24 U; it passes fewer than 64 additions
            near(res[0][2][i], *want_w, (24 + 64) * U, torch.float32)
            assert torch.equal(res[0][2][i], res[1][2][i])
        assert torch.equal(res[0][i], res[1][i])
    # in the gradients' own place
    gdn.gdn_attn_prep_backward(c.cfg, q, k, dqo, dko, f, dq=dqo, dk=dko, w_q=gq, w_k=gk, weight_offset=0.25, interleaved=interleaved, cu_seqlens=cu)
    assert torch.equal(dqo, res[0][0]) and torch.equal(dko, res[0][1])
    assert gdn.gdn_device_error() == 0


def test_backward_without_tokens():
    cfg = gdn.make_attn_config(2, 1, 64, act="fp32")
    e = torch.empty(0, 2, 64, device="cuda")
    w, dw = torch.ones(64, device="cuda"), torch.full((64,), 9.0, device="cuda")
    ws = torch.empty(gdn.gdn_attn_prep_workspace_size(cfg, 0), dtype=torch.uint8, device="cuda")
    gdn.gdn_attn_prep_backward(cfg, e, None, e, None, None, dq=e, dw_q=dw, w_q=w, workspace=ws)
    assert not dw.any()
    gdn.gdn_attn_prep(cfg, e, None, e, None)


def test_gradients_are_differences():
    """The kernels' own gradients against central differences of the kernels' forward pass, summed in 64 bits."""
    c = Case([6], Hq=2, Hkv=1, D=64, act="fp32", rotary=40, seed=4)
    d = [c.r(6, 2, 64).cuda(), c.r(6, 1, 64).cuda()]
    q, k, f, w_q, w_k = gpu(c.q.contiguous(), c.k.contiguous(), c.f, c.w_q, c.w_k)

    def loss():
        q_out, k_out = torch.empty_like(q), torch.empty_like(k)
        gdn.gdn_attn_prep(c.cfg, q, k, q_out, f, k_out=k_out, w_q=w_q, w_k=w_k, eps=1e-3)
        return float((q_out.double() * d[0]).sum() + (k_out.double() * d[1]).sum())
    dq, dk, dw = torch.empty_like(q), torch.empty_like(k), torch.empty(2, 64, device="cuda")
    ws = torch.empty(gdn.gdn_attn_prep_workspace_size(c.cfg, 6), dtype=torch.uint8, device="cuda")
    gdn.gdn_attn_prep_backward(c.cfg, q, k, *d, f, dq=dq, dk=dk, dw_q=dw[0], dw_k=dw[1], w_q=w_q, w_k=w_k, eps=1e-3, workspace=ws)
    g = torch.Generator().manual_seed(9)
    step = 2.0 ** -7
    for leaf, grad in ((q, dq), (k, dk), (w_q, dw[0]), (w_k, dw[1])):
        for i in torch.randint(0, leaf.numel(), (12,), generator=g).tolist():
            keep = float(leaf.view(-1)[i])
            ends = []
            for e in (step, -step):
                leaf.view(-1)[i] = keep + e
                ends.append((float(leaf.view(-1)[i]), loss()))
            leaf.view(-1)[i] = keep
            slope = (ends[0][1] - ends[1][1]) / (ends[0][0] - ends[1][0])
            # 768 values of a size near 1 off by 24 U each at most, over 2 steps, walk to 5 sqrt(768) * 24 U / 2^-6 = 0.013; the
            # third derivative of a head's norm is below 20 / 64, times step^2 / 6 and |d| sums below 64: 2e-3
            assert abs(slope - float(grad.reshape(-1)[i])) < 0.015


def test_graph_and_streams():
    c = Case([5, 9], D=128, seed=12)
    qkv, f, w, cu, dqo = gpu(c.qkv, c.f, c.w_q, cu_of(c.lens), c.r(14, 4, 128).to(c.act))
    q, k, _ = c.split(qkv)
    outs = [torch.zeros(c.q.shape, dtype=c.act, device="cuda"), torch.zeros(c.k.shape, dtype=c.act, device="cuda"), torch.zeros_like(dqo),
            torch.zeros(128, device="cuda")]
    ws = torch.empty(gdn.gdn_attn_prep_workspace_size(c.cfg, 14), dtype=torch.uint8, device="cuda")

    def call():
        gdn.gdn_attn_prep(c.cfg, q, k, outs[0], f, k_out=outs[1], cu_seqlens=cu, w_q=w)
        gdn.gdn_attn_prep_backward(c.cfg, q, None, dqo, None, f, dq=outs[2], dw_q=outs[3], w_q=w, cu_seqlens=cu, workspace=ws)
    call()
    torch.cuda.synchronize()
    want = [t.clone() for t in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for t in outs:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    for t in outs:
        t.zero_()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_large_batch_uses_every_block():
    """More tokens than run at once: blocks of several tokens, backward blocks that walk."""
    c = Case([9000, 4001], Hq=3, Hkv=1, D=64, act="bf16", seed=13)
    qkv, f, w_q, w_k, cu = gpu(c.qkv, c.f, c.w_q, c.w_k, cu_of(c.lens))
    q, k, _ = c.split(qkv)
    q_out, k_out = torch.empty(c.q.shape, dtype=c.act, device="cuda"), torch.empty(c.k.shape, dtype=c.act, device="cuda")
    gdn.gdn_attn_prep(c.cfg, q, k, q_out, f, k_out=k_out, cu_seqlens=cu, w_q=w_q, w_k=w_k)
    near(q_out, *ref.prep(c.q, c.w_q, c.index(), c.f), FORWARD, c.act)
    near(k_out, *ref.prep(c.k, c.w_k, c.index(), c.f), FORWARD, c.act)
    d = [c.r(c.T, H, 64).to(c.act) for H in (3, 1)]
    dqo, dko = gpu(*d)
    dw = torch.empty(2, 64, device="cuda")
    ws = torch.empty(gdn.gdn_attn_prep_workspace_size(c.cfg, c.T), dtype=torch.uint8, device="cuda")
    dq, dk = torch.empty_like(dqo), torch.empty_like(dko)
    gdn.gdn_attn_prep_backward(c.cfg, q, k, dqo, dko, f, dq=dq, dk=dk, dw_q=dw[0], dw_k=dw[1], w_q=w_q, w_k=w_k, cu_seqlens=cu, workspace=ws)
    for got, got_w, x, w, dd in ((dq, dw[0], c.q, c.w_q, d[0]), (dk, dw[1], c.k, c.w_k, d[1])):
        (dx, mag), want_w = ref.prep_backward(x, w, dd, c.index(), c.f)
        near(got, dx, mag, BACKWARD, c.act)
        near(got_w, *want_w, (24 + 128) * U, torch.float32)    # fewer than 128 additions for each of the 39,003 terms
