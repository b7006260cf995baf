"""What needs no GPU of the state space mixer and the block norms: refusals before any launch
(fake pointers that are never read), structure layouts, workspace sizes, and the 64-bit
references themselves against differences and the recurrence's closed forms."""
import ctypes
import math
import shutil
import subprocess

import pytest
import torch

import ssm_ref as ref
from gateddeltanet_linear_attention_gb300 import build_lib, gdn

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A, B, MIS = 0x100000, 0x200000, 0x100008


@pytest.fixture(scope="module")
def lib():
    return gdn.load()


def cfg(**kw):
    base = dict(groups=2, heads=8, d_state=128, head_dim=64, act="bf16", n_slots=4)
    base.update(kw)
    return gdn.make_ssm_config(**base)


def scan_io(**kw):
    d = dict(x=A, ld_x=512, b=A, c=A, ld_bc=256, dt=A, ld_dt=8, z=A, ld_z=512, A_log=A, dt_bias=A, D=A, cu_seqlens=A, n_seqs=2,
             T=100, state_idx=None, state_in=A, state_out=B, y=B)
    d.update(kw)
    return gdn.SSMIO(**d)


def step_io(**kw):
    d = dict(x=A, ld_x=1024, dt=A, ld_dt=8, z=A, ld_z=512, A_log=A, dt_bias=A, D=A, conv_w=A, conv_bias=A, n_seqs=2, T=2, state_in=B,
             state_out=B, conv_state=B, y=B)
    d.update(kw)
    return gdn.SSMIO(**d)


@pytest.mark.parametrize("kw,want", [
    (dict(groups=0), INVALID), (dict(heads=7), INVALID), (dict(heads=0), INVALID), (dict(n_slots=-1), INVALID),
    (dict(d_state=48), UNSUPPORTED), (dict(d_state=256), UNSUPPORTED), (dict(head_dim=16), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED),
    (dict(dt_min=-1.0), INVALID), (dict(dt_min=0.2, dt_max=0.1), INVALID), (dict(dt_min=math.nan), INVALID),
    (dict(dt_max=math.nan), INVALID), (dict(dt_min=math.inf), INVALID), (dict(groups=1, heads=8192), UNSUPPORTED)])
def test_configurations(lib, kw, want):
    c = cfg(**kw)
    assert lib.gdn_ssm_prefill(ctypes.byref(c), ctypes.byref(scan_io()), A, 1 << 40, None) == want
    assert lib.gdn_ssm_decode(ctypes.byref(c), ctypes.byref(step_io()), A, 1 << 40, None) == want
    assert lib.gdn_ssm_conv_prefill(ctypes.byref(c), A, 1024, A, 1, 5, A, A, A, None, B, None) == want
    assert gdn.gdn_ssm_workspace_size(c, 100, 2) == 0


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=MIS), dict(ld_x=504), dict(ld_x=516), dict(b=None), dict(c=MIS), dict(ld_bc=128), dict(dt=None), dict(dt=A + 1),
    dict(ld_dt=7), dict(z=MIS), dict(ld_z=500), dict(A_log=None), dict(A_log=A + 2), dict(D=A + 1), dict(dt_bias=A + 2), dict(cu_seqlens=None),
    dict(cu_seqlens=A + 2), dict(n_seqs=-1), dict(n_seqs=0), dict(T=-1), dict(state_in=MIS), dict(state_out=MIS), dict(state_idx=A + 1),
    dict(y=None), dict(y=MIS)])
def test_scan_refusals(lib, kw):
    assert lib.gdn_ssm_prefill(ctypes.byref(cfg()), ctypes.byref(scan_io(**kw)), A, 1 << 40, None) == INVALID


def test_scan_limits(lib):
    c = ctypes.byref(cfg())
    assert lib.gdn_ssm_prefill(c, None, A, 1 << 40, None) == INVALID
    assert lib.gdn_ssm_prefill(c, ctypes.byref(scan_io(n_seqs=65536)), A, 1 << 40, None) == UNSUPPORTED
    assert lib.gdn_ssm_prefill(c, ctypes.byref(scan_io(T=1 << 31)), A, 1 << 40, None) == UNSUPPORTED
    assert lib.gdn_ssm_prefill(c, ctypes.byref(scan_io(n_seqs=0, T=0)), None, 0, None) == OK
    assert lib.gdn_ssm_prefill(ctypes.byref(cfg(n_slots=0)), ctypes.byref(scan_io()), A, 1 << 40, None) == INVALID
    # one long sequence is cut, and the states between its segments need the workspace
    for ws, size in ((None, 1 << 40), (MIS, 1 << 40), (A, 0), (A, 1000)):
        assert lib.gdn_ssm_prefill(c, ctypes.byref(scan_io(T=100000, n_seqs=1)), ws, size, None) == WORKSPACE


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(x=MIS), dict(ld_x=1016), dict(b=A), dict(c=A), dict(dt=None), dict(ld_dt=7), dict(z=MIS), dict(conv_w=None),
    dict(conv_w=MIS), dict(conv_bias=MIS), dict(A_log=None), dict(state_in=None), dict(state_in=A), dict(state_out=None),
    dict(conv_state=None), dict(conv_state=MIS), dict(y=None), dict(T=3), dict(n_seqs=-1, T=-1), dict(state_idx=A + 2)])
def test_step_refusals(lib, kw):
    assert lib.gdn_ssm_decode(ctypes.byref(cfg()), ctypes.byref(step_io(**kw)), A, 1 << 40, None) == INVALID


def test_step_limits(lib):
    c = ctypes.byref(cfg())
    assert lib.gdn_ssm_decode(c, ctypes.byref(step_io(n_seqs=0, T=0)), None, 0, None) == OK
    assert lib.gdn_ssm_decode(c, ctypes.byref(step_io(n_seqs=65536, T=65536)), A, 1 << 40, None) == UNSUPPORTED
    for ws, size in ((None, 1 << 40), (MIS, 1 << 40), (A, 8000)):
        assert lib.gdn_ssm_decode(c, ctypes.byref(step_io()), ws, size, None) == WORKSPACE
    assert lib.gdn_ssm_decode(ctypes.byref(cfg(n_slots=0)), ctypes.byref(step_io()), A, 1 << 40, None) == INVALID


def test_conv_refusals(lib):
    c = cfg()
    good = dict(x=A, ld=1024, cu=A, n=1, T=5, w=A, bias=A, hist=A, idx=None, out=B)

    def call(c=c, **kw):
        d = dict(good, **kw)
        return lib.gdn_ssm_conv_prefill(ctypes.byref(c), d["x"], d["ld"], d["cu"], d["n"], d["T"], d["w"], d["bias"], d["hist"], d["idx"],
                                        d["out"], None)
    for kw in (dict(x=None), dict(x=MIS), dict(ld=1016), dict(ld=1028), dict(cu=None), dict(n=-1), dict(n=0), dict(T=-1), dict(w=None),
               dict(w=MIS), dict(bias=MIS), dict(hist=MIS), dict(idx=A + 1), dict(out=None), dict(out=MIS)):
        assert call(**kw) == INVALID, kw
    assert call(n=65536) == UNSUPPORTED
    assert call(T=0, x=None, out=None) == OK
    assert call(c=cfg(n_slots=0)) == INVALID


def test_workspace_grows(lib):
    c, last = cfg(), 0
    for T in (1, 100, 256, 257, 1000, 5000, 70000, 1 << 20):
        size = gdn.gdn_ssm_workspace_size(c, T, 3)
        assert size >= last
        last = size
    assert gdn.gdn_ssm_workspace_size(c, 100, 5) >= 5 * (512 + 2 * 256) * 4
    assert gdn.gdn_ssm_workspace_size(c, -1, 1) == 0
    assert gdn.gdn_block_norm_workspace_size(10, 0) == gdn.gdn_block_norm_workspace_size(-1, 8) == 0
    assert gdn.gdn_block_norm_workspace_size(10, 16385) == 0


def norm_io(**kw):
    d = dict(rows=4, dim=64, act=0, res=0, eps=1e-6, res_scale=1.0, block=A, ld_block=64, gate=A, ld_gate=64, gate_cols=64, residual=A,
             ld_residual=64, w_post=A, w_pre=A, res_out=B, ld_res_out=64, h=B, ld_h=64)
    d.update(kw)
    return gdn.BlockNormIO(**d)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INVALID), (dict(dim=0), INVALID), (dict(dim=16385, gate_cols=1), UNSUPPORTED), (dict(act=1, res=0), UNSUPPORTED),
    (dict(act=2), INVALID), (dict(res=-1), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID),
    (dict(res_scale=math.inf), INVALID), (dict(weight_offset=math.nan), INVALID), (dict(gate_cols=2), INVALID), (dict(gate_cols=0), INVALID),
    (dict(ld_gate=63), INVALID), (dict(block=A + 1), INVALID), (dict(ld_block=63), INVALID), (dict(residual=None), INVALID),
    (dict(ld_residual=10), INVALID), (dict(block=None), INVALID), (dict(block=None, gate=None, w_post=None), INVALID),
    (dict(w_pre=None), INVALID), (dict(h=None), INVALID), (dict(h=None, w_pre=None, res_out=None), INVALID), (dict(w_pre=A + 2), INVALID),
    (dict(rstd_post=A + 1), INVALID), (dict(rstd_post=A, w_post=None), INVALID), (dict(ld_h=0), INVALID), (dict(res_out=A + 1), INVALID)])
def test_norm_refusals(lib, kw, want):
    assert lib.gdn_block_norm(ctypes.byref(norm_io(**kw)), None) == want


@pytest.mark.parametrize("kw", [
    dict(dh=None), dict(w_pre=None), dict(rstd_pre=None), dict(rstd_post=None), dict(residual=None), dict(d_gate=B, gate=None),
    dict(d_block=B, ld_d_block=3), dict(dw_pre=B, w_pre=None, dh=None), dict(dh=None, w_pre=None, d_res_out=None), dict(d_residual=B + 1),
    dict(dw_post=B + 2), dict(block=None)])
def test_norm_backward_refusals(lib, kw):
    d = dict(rstd_post=A, rstd_pre=A, dh=A, ld_dh=64, d_res_out=A, ld_d_res_out=64, d_residual=B, ld_d_residual=64, d_block=B, ld_d_block=64,
             d_gate=B, ld_d_gate=64, dw_post=B, dw_pre=B)
    io = norm_io(**dict(d, **kw))
    assert lib.gdn_block_norm_backward(ctypes.byref(io), A, 1 << 40, None) == INVALID
    for ws, size in ((None, 1 << 40), (MIS, 1 << 40), (A, 100)):
        assert lib.gdn_block_norm_backward(ctypes.byref(norm_io(**d)), ws, size, None) == WORKSPACE


def test_null_structures(lib):
    assert lib.gdn_block_norm(None, None) == INVALID
    assert lib.gdn_block_norm_backward(None, A, 1, None) == INVALID
    assert lib.gdn_ssm_decode(ctypes.byref(cfg()), None, A, 1, None) == INVALID


def test_structure_layouts(tmp_path):
    """The binding's structures have the header's field offsets."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = {"gdn_ssm_config": gdn.SSMConfig, "gdn_ssm_io": gdn.SSMIO, "gdn_block_norm_io": gdn.BlockNormIO}
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "gdn.h"', "int main(void) {"]
    for name, s in structs.items():
        lines += ['printf("%%zu\\n", offsetof(%s, %s));' % (name, f) for f, _ in s._fields_]
        lines.append('printf("%%zu\\n", sizeof(%s));' % name)
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["return 0; }"]))
    exe = str(tmp_path / "layout")
    subprocess.run([cc, "-I" + build_lib.INCLUDE, str(src), "-o", exe], check=True)
    got = [int(v) for v in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    want = []
    for s in structs.values():
        want += [getattr(s, f).offset for f, _ in s._fields_] + [ctypes.sizeof(s)]
    assert got == want


# ------------------------------------------------------------- the references

def test_reference_scan_is_its_closed_form():
    """y_t = sum_{i<=t} (C_t . B_i) exp(A sum_{i<j<=t} dt_j) dt_i x_i + C_t^T exp(...) S_0 + D x_t."""
    g = torch.Generator().manual_seed(0)
    L, H, G, N, P = 9, 4, 2, 5, 3
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    x, b, c, u, A_log, D, S0 = r(L, H, P), r(L, G, N), r(L, G, N), r(L, H), r(H), r(H), r(H, N, P)
    y, mag, S, M = ref.scan(x, b, c, u, A_log, D, None, None, S0, G)
    dt, rate = torch.log1p(torch.exp(u)), -torch.exp(A_log)
    for h in range(H):
        k = h // 2
        for t in range(L):
            want = D[h] * x[t, h] + math.exp(rate[h] * dt[:t + 1, h].sum()) * (c[t, k] @ S0[h])
            for i in range(t + 1):
                want = want + (c[t, k] @ b[i, k]) * math.exp(rate[h] * dt[i + 1:t + 1, h].sum()) * dt[i, h] * x[i, h]
            assert torch.allclose(y[t, h], want, rtol=0, atol=1e-11)
    assert (mag >= y.abs() - 1e-12).all() and (M >= S.abs() - 1e-12).all()


@pytest.mark.parametrize("gate", ["channel", "row", "none"])
@pytest.mark.parametrize("post", [True, False])
def test_reference_gradients_are_differences(gate, post):
    """The written-out gradients against central differences of the forward formula."""
    g = torch.Generator().manual_seed(1)
    rows, dim, eps, off, scale = 3, 5, 1e-3, 0.5, 0.7
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    leaves = dict(p=r(rows, dim), gate=None if gate == "none" else r(rows, dim if gate == "channel" else 1), r=r(rows, dim),
                  w1=r(dim) if post else None, w2=r(dim))
    dh, dro = r(rows, dim), r(rows, dim)

    def loss(v):
        o = ref.norm(v["p"], v["gate"], v["r"], v["w1"], v["w2"], eps, off, scale)
        return float((o["h"][0] * dh).sum() + (o["res_out"][0] * dro).sum())
    f = ref.norm(leaves["p"], leaves["gate"], leaves["r"], leaves["w1"], leaves["w2"], eps, off, scale)
    out = ref.norm_backward(leaves["p"], leaves["gate"], f["res_out"][0], leaves["w1"], leaves["w2"],
                            f["rstd_post"][0] if post else None, f["rstd_pre"][0], dh, dro, off, scale)
    for name, grad in (("p", "d_block"), ("gate", "d_gate"), ("r", "d_residual"), ("w1", "dw_post"), ("w2", "dw_pre")):
        if leaves[name] is None:
            continue
        want = torch.zeros_like(leaves[name])
        for i in range(want.numel()):
            vals = []
            for e in (1e-5, -1e-5):
                v = dict(leaves, **{name: leaves[name].clone()})
                v[name].view(-1)[i] += e
                vals.append(loss(v))
            want.view(-1)[i] = (vals[0] - vals[1]) / 2e-5
        assert torch.allclose(out[grad][0], want, rtol=1e-6, atol=1e-8), name
        assert (out[grad][1] >= out[grad][0].abs() - 1e-12).all()
