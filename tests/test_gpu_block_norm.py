"""The gated block norms and their gradients on the GPU against the plain 64-bit reference."""
import pytest
import torch

import ssm_ref as ref
from gateddeltanet_linear_attention_gb300 import gdn

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
TYPES = [(BF, BF), (BF, F32), (F32, F32)]
DIMS = [1, 7, 8, 48, 255, 256, 520, 1000, 1024, 1032, 1111, 2048, 4096, 5120, 8192, 8200, 9001, 16384]


def make(rows, dim, act, res, gate="channel", post=True, pre=True, block=True, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed + rows * 31 + dim)

    def r(*shape, std=1.0, dtype=F32):
        return (torch.randn(shape, generator=g) * std).to(dtype)

    def wide(cols, dtype):
        return r(rows, cols + pad, dtype=dtype)[:, pad // 2:pad // 2 + cols] if pad else r(rows, cols, dtype=dtype)

    d = dict(block=wide(dim, act) if block else None, residual=wide(dim, res),
             gate=None if gate == "none" or not block else wide(dim if gate == "channel" else 1, act),
             w_post=1 + 0.2 * r(dim) if post and block else None, w_pre=1 + 0.2 * r(dim) if pre else None,
             dh=wide(dim, act) if pre else None, d_res_out=wide(dim, res))
    return d


def up(t):
    """To the GPU with its strides."""
    if t is None:
        return None
    if t.is_contiguous():
        return t.cuda()
    base = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda")
    base.copy_(t)
    return base


def rel_fwd(dim):
    """A sum of dim squares in 32 bits, then root, quotient, products, exp: 8 more roundings and 8 of exp's."""
    return (dim + 32) * ref.U32


def forward(d, act, res, offset=0.0, scale=0.7, eps=1e-5, in_place=False):
    rows, dim = d["residual"].shape
    t = {k: up(v) for k, v in d.items()}
    res_out = t["residual"] if in_place else torch.full((rows, dim), 7.0, dtype=res, device="cuda")
    h = torch.full((rows, dim), 7.0, dtype=act, device="cuda") if d["w_pre"] is not None else None
    k1 = torch.zeros(rows, device="cuda") if d["w_post"] is not None else None
    k2 = torch.zeros(rows, device="cuda") if d["w_pre"] is not None else None
    gdn.gdn_block_norm(t["residual"], t["w_pre"], h, block=t["block"], res_out=res_out if d["block"] is not None else None,
                       w_post=t["w_post"], gate=t["gate"], res_scale=scale, eps=eps, weight_offset=offset, rstd_post=k1, rstd_pre=k2)
    torch.cuda.synchronize()
    want = ref.norm(d["block"], d["gate"], d["residual"], d["w_post"], d["w_pre"], eps, offset, scale)
    got = dict(res_out=res_out if d["block"] is not None else None, h=h, rstd_post=k1, rstd_pre=k2)
    for k, v in got.items():
        if v is not None:
            ref.check(v, *want[k], rel_fwd(dim), k)
    return got


def backward(d, act, res, offset=0.0, scale=0.7, eps=1e-5):
    rows, dim = d["residual"].shape
    f = ref.norm(d["block"], d["gate"], d["residual"], d["w_post"], d["w_pre"], eps, offset, scale)
    kept = {k: f[k][0].to(F32) for k in ("rstd_post", "rstd_pre") if k in f}
    u = f["res_out"][0].to(res)
    t = {k: up(v) for k, v in d.items()}
    out = dict(d_residual=torch.full((rows, dim), 7.0, dtype=res, device="cuda"))
    if d["block"] is not None:
        out["d_block"] = torch.full((rows, dim), 7.0, dtype=act, device="cuda")
    if d["gate"] is not None:
        out["d_gate"] = torch.full(d["gate"].shape, 7.0, dtype=act, device="cuda")
    if d["w_post"] is not None:
        out["dw_post"] = torch.full((dim,), 7.0, device="cuda")
    if d["w_pre"] is not None:
        out["dw_pre"] = torch.full((dim,), 7.0, device="cuda")
    ws = torch.full((gdn.gdn_block_norm_workspace_size(rows, dim),), 0xFF, dtype=torch.uint8, device="cuda")
    gdn.gdn_block_norm_backward(u.cuda(), up(kept.get("rstd_pre")), t["w_pre"], t["dh"], t["d_res_out"], block=t["block"],
                                rstd_post=up(kept.get("rstd_post")), w_post=t["w_post"], gate=t["gate"], res_scale=scale,
                                weight_offset=offset, workspace=ws, **out)
    torch.cuda.synchronize()
    want = ref.norm_backward(d["block"], d["gate"], u, d["w_post"], d["w_pre"], kept.get("rstd_post"), kept.get("rstd_pre"),
                             d["dh"], d["d_res_out"], offset, scale)
    for k, v in out.items():
        # 32-bit sums over a row (twice) or over the rows, and some twenty roundings besides
        ref.check(v, *want[k], (2 * dim + rows + 64) * ref.U32, k)
    return out


@pytest.mark.parametrize("act,res", TYPES)
@pytest.mark.parametrize("dim", DIMS)
def test_forward_widths(act, res, dim):
    forward(make(5, dim, act, res), act, res)


@pytest.mark.parametrize("act,res", TYPES)
@pytest.mark.parametrize("dim", DIMS)
def test_backward_widths(act, res, dim):
    backward(make(5, dim, act, res), act, res)


@pytest.mark.parametrize("rows", [1, 2, 33, 700, 2500])
@pytest.mark.parametrize("dim", [96, 1200])
def test_row_counts(rows, dim):
    d = make(rows, dim, BF, F32, gate="row")
    forward(d, BF, F32)
    backward(d, BF, F32)


@pytest.mark.parametrize("gate", ["channel", "row", "none"])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("dim", [200, 1600, 1111])
def test_parts(gate, post, pre, dim):
    d = make(9, dim, BF, BF, gate=gate, post=post, pre=pre)
    forward(d, BF, BF, offset=1.0)
    backward(d, BF, BF, offset=1.0)


@pytest.mark.parametrize("dim", [64, 2000])
def test_plain_pre_norm(dim):
    d = make(6, dim, BF, F32, block=False)
    forward(d, BF, F32)
    backward(d, BF, F32)


@pytest.mark.parametrize("pad", [16, 6])
@pytest.mark.parametrize("dim", [64, 1600])
def test_row_strides(pad, dim):
    """Rows that start on 16 bytes, and rows that do not."""
    d = make(7, dim, BF, F32, pad=pad)
    forward(d, BF, F32)
    backward(d, BF, F32)


def test_in_place_residual():
    for dim in (96, 4096):
        forward(make(40, dim, BF, BF), BF, BF, in_place=True)


def test_in_place_gradient():
    d = make(300, 1500, BF, BF)
    want = backward(d, BF, BF)
    f = ref.norm(d["block"], d["gate"], d["residual"], d["w_post"], d["w_pre"], 1e-5, 0.0, 0.7)
    dro = d["d_res_out"].cuda()
    gdn.gdn_block_norm_backward(f["res_out"][0].to(BF).cuda(), f["rstd_pre"][0].float().cuda(), up(d["w_pre"]), up(d["dh"]), dro, dro,
                                block=up(d["block"]), rstd_post=f["rstd_post"][0].float().cuda(), w_post=up(d["w_post"]),
                                gate=up(d["gate"]), res_scale=0.7)
    assert torch.equal(dro, want["d_residual"])


def test_rows_of_zeros_and_large_values():
    d = make(8, 512, F32, F32)
    d["block"][0] = 0
    d["residual"][1] = 0
    d["block"][1] = 0
    d["block"][2] *= 1e15
    d["residual"][3] *= 1e-20
    d["block"][4] *= 1e-30
    forward(d, F32, F32)
    backward(d, F32, F32)


def test_no_rows():
    e = torch.empty(0, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    gdn.gdn_block_norm(e, w, e.clone())
    dw = torch.full((64,), 7.0, device="cuda")
    ws = torch.empty(gdn.gdn_block_norm_workspace_size(0, 64), dtype=torch.uint8, device="cuda")
    gdn.gdn_block_norm_backward(e, torch.empty(0, device="cuda"), w, e, dw_pre=dw, workspace=ws)
    assert (dw == 0).all()


def test_no_gradient_of_the_residual_stream():
    d = make(11, 300, BF, BF)
    d["d_res_out"] = None
    backward(d, BF, BF)


def test_same_bits_again_and_in_a_graph():
    d = make(600, 1300, BF, BF)
    one, two = backward(d, BF, BF), backward(d, BF, BF)
    assert all(torch.equal(one[k], two[k]) for k in one)
    r, p, w = d["residual"].cuda(), d["block"].cuda(), up(d["w_pre"])
    h, ro, h2, ro2 = (torch.empty_like(r) for _ in range(4))
    gdn.gdn_block_norm(r, w, h, block=p, res_out=ro, w_post=w)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            gdn.gdn_block_norm(r, w, h2, block=p, res_out=ro2, w_post=w)
        graph.replay()
    s.synchronize()
    assert torch.equal(h, h2) and torch.equal(ro, ro2)


def test_residual_not_kept():
    """A block without a place for the new residual: h alone."""
    d = make(9, 700, BF, BF)
    t = {k: up(v) for k, v in d.items()}
    h = torch.empty(9, 700, dtype=BF, device="cuda")
    gdn.gdn_block_norm(t["residual"], t["w_pre"], h, block=t["block"], w_post=t["w_post"], gate=t["gate"], res_scale=0.7, eps=1e-5)
    ref.check(h, *ref.norm(d["block"], d["gate"], d["residual"], d["w_post"], d["w_pre"], 1e-5, 0.0, 0.7)["h"], rel_fwd(700), "h")


def test_in_place_over_many_rows():
    """More rows than CTAs: rows loaded ahead, written in place."""
    d = make(3000, 520, BF, BF)
    forward(d, BF, BF, in_place=True)
    want = backward(d, BF, BF)
    f = ref.norm(d["block"], d["gate"], d["residual"], d["w_post"], d["w_pre"], 1e-5, 0.0, 0.7)
    dro = d["d_res_out"].cuda()
    gdn.gdn_block_norm_backward(f["res_out"][0].to(BF).cuda(), f["rstd_pre"][0].float().cuda(), up(d["w_pre"]), up(d["dh"]), dro, dro,
                                block=up(d["block"]), rstd_post=f["rstd_post"][0].float().cuda(), w_post=up(d["w_post"]),
                                gate=up(d["gate"]), res_scale=0.7)
    assert torch.equal(dro, want["d_residual"])


def test_offsets_past_32_bits():
    rows, dim = (1 << 31) // 4096 + 700, 4096
    g = torch.Generator(device="cuda").manual_seed(3)
    p, r = (torch.empty(rows, dim, dtype=BF, device="cuda").normal_(generator=g) for _ in range(2))
    w = 1 + 0.1 * torch.randn(dim, generator=g, device="cuda")
    ro, h = torch.empty_like(p), torch.empty_like(p)
    k1, k2 = torch.empty(2, rows, device="cuda")
    gdn.gdn_block_norm(r, w, h, block=p, res_out=ro, w_post=w, rstd_post=k1, rstd_pre=k2)
    s = slice(rows - 20, rows)
    want = ref.norm(p[s].cpu(), None, r[s].cpu(), w.cpu(), w.cpu(), 1e-6, 0.0, 1.0)
    ref.check(ro[s], *want["res_out"], rel_fwd(dim), "r'")
    ref.check(h[s], *want["h"], rel_fwd(dim), "h")
    dr, dp = r, torch.empty_like(p)               # the gradient in place of d_r'
    dro = r[s].cpu()
    gdn.gdn_block_norm_backward(ro, k2, w, h, r, dr, block=p, rstd_post=k1, w_post=w, d_block=dp)
    want = ref.norm_backward(p[s].cpu(), None, ro[s].cpu(), w.cpu(), w.cpu(), k1[s].cpu(), k2[s].cpu(), h[s].cpu(), dro, 0.0, 1.0)
    for k, v in (("d_residual", dr), ("d_block", dp)):
        ref.check(v[s], *want[k], (2 * dim + 64) * ref.U32, k)


@pytest.mark.parametrize("act", [BF, F32])
@pytest.mark.parametrize("kind", ["channel", "row"])
def test_gradient_of_gates_that_are_all_but_open_or_shut(act, kind):
    """1 - sigmoid is not taken as a difference.  With one column and d_r' alone the gradient is a product:
    a dozen roundings and the exponential's error, 2 + 1.2 |x| units in the last place where it is the fast one."""
    x = torch.tensor([-70.0, -30.0, -8.0, 0.0, 8.0, 17.0, 30.0, 70.0])
    rows, dim = (8, 1) if kind == "row" else (8, 8)
    g = torch.Generator().manual_seed(5)
    p, u, dro = (torch.randn(rows, dim, generator=g).to(act) for _ in range(3))
    gate = (x[:, None] if kind == "row" else x[None].expand(8, 8).contiguous()).to(act)
    w, k = 1 + 0.2 * torch.randn(dim, generator=g), 1 + torch.rand(rows, generator=g)
    dg = torch.empty(rows, dim, dtype=act, device="cuda")
    gdn.gdn_block_norm_backward(u.cuda(), d_res_out=dro.cuda(), block=p.cuda(), rstd_post=k.cuda(), w_post=w.cuda(),
                                gate=gate.cuda(), res_scale=0.7, d_gate=dg)
    want = ref.norm_backward(p, gate, u, w, None, k, None, None, dro, 0.0, 0.7)["d_gate"][0]
    ref.check(dg, want, want.abs(), (40 + (2 * (2 + 1.2 * 70) if act == BF else 0)) * ref.U32, "d_gate")


def test_binding_refuses_tensors_that_do_not_fit():
    d = {k: up(v) for k, v in make(6, 64, BF, BF).items()}
    h = torch.empty(6, 64, dtype=BF, device="cuda")

    def call(**kw):
        a = dict(residual=d["residual"], w_pre=d["w_pre"], h=h, block=d["block"], res_out=torch.empty_like(h), w_post=d["w_post"],
                 gate=d["gate"])
        a.update(kw)
        gdn.gdn_block_norm(**a)

    call()
    for bad in (dict(gate=d["gate"][:, :2]), dict(gate=d["gate"][:, 0]), dict(block=d["block"].float()), dict(w_pre=d["w_pre"].cpu()),
                dict(h=h[:5]), dict(residual=d["residual"][:, :32]), dict(res_out=torch.empty(6, 1, dtype=BF, device="cuda").expand(6, 64)),
                dict(residual=d["residual"][0]), dict(block=None), dict(w_pre=None)):
        with pytest.raises((ValueError, RuntimeError)):
            call(**bad)


def test_gradients_in_a_graph_and_on_another_stream():
    d = make(900, 1300, BF, BF)
    want = backward(d, BF, BF)
    f = ref.norm(d["block"], d["gate"], d["residual"], d["w_post"], d["w_pre"], 1e-5, 0.0, 0.7)
    t = {k: up(v) for k, v in d.items()}
    u, k1, k2 = f["res_out"][0].to(BF).cuda(), f["rstd_post"][0].float().cuda(), f["rstd_pre"][0].float().cuda()
    got = {k: torch.full_like(v, 7.0) for k, v in want.items()}
    ws = torch.empty(gdn.gdn_block_norm_workspace_size(900, 1300), dtype=torch.uint8, device="cuda")
    s, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        gdn.gdn_block_norm_backward(u, k2, t["w_pre"], t["dh"], t["d_res_out"], block=t["block"], rstd_post=k1, w_post=t["w_post"],
                                    gate=t["gate"], res_scale=0.7, workspace=ws, stream=s, **got)
    with torch.cuda.stream(s):
        graph.replay()
    s.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)


@pytest.mark.parametrize("one", ["dw_post", "dw_pre", "d_block", "d_gate", "d_residual"])
def test_one_gradient_alone(one):
    d = make(300, 200, BF, F32)
    want = backward(d, BF, F32)
    f = ref.norm(d["block"], d["gate"], d["residual"], d["w_post"], d["w_pre"], 1e-5, 0.0, 0.7)
    t = {k: up(v) for k, v in d.items()}
    got = torch.full_like(want[one], 7.0)
    ws = torch.empty(gdn.gdn_block_norm_workspace_size(300, 200), dtype=torch.uint8, device="cuda") if one[:2] == "dw" else None
    gdn.gdn_block_norm_backward(f["res_out"][0].float().cuda(), f["rstd_pre"][0].float().cuda(), t["w_pre"], t["dh"], t["d_res_out"],
                                block=t["block"], rstd_post=f["rstd_post"][0].float().cuda(), w_post=t["w_post"], gate=t["gate"],
                                res_scale=0.7, workspace=ws, **{one: got})
    assert torch.equal(got, want[one])
