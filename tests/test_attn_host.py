"""What needs no GPU of the attention layers: refusals before any launch (fake pointers that are never read), structure
layouts, workspace sizes, and the 64-bit references against differences and closed forms."""
import ctypes
import math
import shutil
import subprocess

import pytest
import torch

import attn_ref as ref
from gateddeltanet_linear_attention_gb300 import build_lib, gdn

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
A, B, MIS = 0x100000, 0x200000, 0x100008


@pytest.fixture(scope="module")
def lib():
    return gdn.load()


def cfg(**kw):
    base = dict(q_heads=8, kv_heads=2, head_dim=128, page_size=64, act="bf16", n_pages=10, n_rows=4, max_pages=5)
    base.update(kw)
    return gdn.make_attn_config(**base)


def prep_io(**kw):
    d = dict(q=A, ld_q=1024, hs_q=128, k=A, ld_k=256, hs_k=128, v=A, ld_v=256, hs_v=128, T=6, w_q=A, w_k=A, weight_offset=0.0, eps=1e-6,
             rotary_dim=64, interleaved=0, inv_freq=A, positions=None, cu_seqlens=A, n_seqs=2, rows=None, lens=A, page_table=A, k_pages=B,
             v_pages=B, q_out=B, k_out=None)
    d.update(kw)
    return gdn.AttnPrepIO(**d)


def bwd_io(**kw):
    d = dict(q=A, ld_q=1024, hs_q=128, k=A, ld_k=256, hs_k=128, T=6, w_q=A, w_k=A, eps=1e-6, rotary_dim=64, inv_freq=A, cu_seqlens=A, n_seqs=2,
             dq_out=A, dk_out=A, dq=B, ld_dq=1024, hs_dq=128, dk=B, ld_dk=256, hs_dk=128, dw_q=B, dw_k=B)
    d.update(kw)
    return gdn.AttnPrepIO(**d)


def decode_io(**kw):
    d = dict(q=A, ld_q=1024, hs_q=128, k_pages=A, v_pages=A, page_table=A, lens=A, rows=None, n_seqs=3, tokens=2, window=0, scale=0.1, out=B, lse=B)
    d.update(kw)
    return gdn.AttnDecodeIO(**d)


def prep(lib, c=None, **kw):
    return lib.gdn_attn_prep(ctypes.byref(c or cfg()), ctypes.byref(prep_io(**kw)), None)


def backward(lib, c=None, ws=A, size=1 << 40, **kw):
    return lib.gdn_attn_prep_backward(ctypes.byref(c or cfg()), ctypes.byref(bwd_io(**kw)), ws, size, None)


def decode(lib, c=None, ws=A, size=1 << 40, **kw):
    return lib.gdn_attn_decode(ctypes.byref(c or cfg()), ctypes.byref(decode_io(**kw)), ws, size, None)


def resize(lib, c=None, n=3, ws=A, size=1 << 40, **kw):
    d = dict(table=A, lens=A, refs=A, rows=A, new=A, granted=B, src=B, dst=B)
    d.update(kw)
    return lib.gdn_page_resize(ctypes.byref(c or cfg()), d["table"], d["lens"], d["refs"], d["rows"], d["new"], n, d["granted"], d["src"],
                               d["dst"], ws, size, None)


def compact(lib, c=None, n=3, ws=A, size=1 << 40, **kw):
    d = dict(table=A, lens=A, refs=A, table_out=B, refs_out=B, src=B, dst=B)
    d.update(kw)
    return lib.gdn_page_compact(ctypes.byref(c or cfg()), d["table"], d["lens"], d["refs"], d["table_out"], d["refs_out"], d["src"], d["dst"], n,
                                ws, size, None)


def fork(lib, c=None, n=3, **kw):
    d = dict(table=A, lens=A, refs=A, src=A, dst=A)
    d.update(kw)
    return lib.gdn_page_fork(ctypes.byref(c or cfg()), d["table"], d["lens"], d["refs"], d["src"], d["dst"], n, None)


def copy(lib, c=None, n=3, n_src=4, n_dst=4, **kw):
    d = dict(sk=A, sv=A, dk=B, dv=B, src=A, dst=A)
    d.update(kw)
    return lib.gdn_page_copy(ctypes.byref(c or cfg()), d["sk"], d["sv"], n_src, d["dk"], d["dv"], n_dst, d["src"], d["dst"], n, None)


@pytest.mark.parametrize("kw,want", [
    (dict(q_heads=0), INVALID), (dict(kv_heads=0), INVALID), (dict(kv_heads=3), INVALID), (dict(head_dim=0), INVALID), (dict(page_size=0), INVALID),
    (dict(n_pages=-1), INVALID), (dict(n_rows=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(head_dim=96), UNSUPPORTED),
    (dict(head_dim=32), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED), (dict(page_size=256), UNSUPPORTED),
    (dict(q_heads=34), UNSUPPORTED), (dict(q_heads=8192, kv_heads=4096), UNSUPPORTED), (dict(n_rows=65536), UNSUPPORTED),
    (dict(n_pages=(1 << 24) + 1), UNSUPPORTED), (dict(max_pages=1 << 25), UNSUPPORTED), (dict(n_pages=1 << 24), UNSUPPORTED)])
def test_configurations(lib, kw, want):
    c = cfg(**kw)
    assert {prep(lib, c), backward(lib, c), decode(lib, c), resize(lib, c), fork(lib, c), compact(lib, c), copy(lib, c)} == {want}
    assert gdn.gdn_attn_workspace_size(c, 3, 1) == gdn.gdn_attn_prep_workspace_size(c, 3) == gdn.gdn_page_workspace_size(c, 3) == 0


def test_unknown_type(lib):
    c = cfg()
    c.act = 2
    assert {prep(lib, c), backward(lib, c), decode(lib, c), resize(lib, c), fork(lib, c), compact(lib, c), copy(lib, c)} == {INVALID}


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q=MIS), dict(ld_q=1020), dict(hs_q=100), dict(hs_q=64), dict(ld_q=64), dict(k=None), dict(k=MIS), dict(ld_k=4),
    dict(v=None), dict(v=MIS), dict(hs_v=4), dict(T=-1), dict(n_seqs=-1), dict(n_seqs=0), dict(cu_seqlens=None, n_seqs=4), dict(cu_seqlens=A + 2),
    dict(w_q=MIS), dict(w_k=A + 4), dict(weight_offset=math.nan), dict(eps=-1.0), dict(eps=math.inf), dict(rotary_dim=-2), dict(rotary_dim=63),
    dict(rotary_dim=130), dict(interleaved=2), dict(inv_freq=None), dict(inv_freq=A + 1), dict(positions=A + 2), dict(rows=A + 1), dict(lens=None),
    dict(lens=A + 2), dict(page_table=None), dict(page_table=A + 2), dict(k_pages=None), dict(v_pages=None), dict(k_pages=MIS), dict(q_out=None),
    dict(q_out=MIS), dict(k_out=MIS), dict(k_pages=None, v_pages=None), dict(k_pages=None, v_pages=None, v=None)])
def test_prep_refusals(lib, kw):
    assert prep(lib, **kw) == INVALID


def test_prep_limits(lib):
    assert lib.gdn_attn_prep(ctypes.byref(cfg()), None, None) == INVALID
    assert prep(lib, T=1 << 31) == UNSUPPORTED
    assert prep(lib, T=0, q=None, k=None, v=None, q_out=None) == OK
    for c in (cfg(n_pages=0), cfg(n_rows=0), cfg(max_pages=0)):
        assert prep(lib, c) == INVALID


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(dq_out=None), dict(dq_out=MIS), dict(dk_out=None), dict(k=None), dict(k=None, dk_out=None), dict(dq=MIS), dict(ld_dq=512),
    dict(hs_dq=64), dict(ld_dk=128), dict(dw_q=B + 2), dict(w_q=None), dict(w_k=None), dict(n_seqs=0), dict(rotary_dim=200), dict(eps=math.nan)])
def test_backward_refusals(lib, kw):
    assert backward(lib, **kw) == INVALID


def test_backward_limits(lib):
    need = gdn.gdn_attn_prep_workspace_size(cfg(), 6)
    assert need > 0
    for ws, size in ((None, 1 << 40), (MIS, 1 << 40), (A, 100)):
        assert backward(lib, ws=ws, size=size) == WORKSPACE
    assert backward(lib, T=0, dw_q=None, dw_k=None, ws=None, size=0) == OK
    assert lib.gdn_attn_prep_backward(ctypes.byref(cfg()), None, A, 1, None) == INVALID


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(q=MIS), dict(ld_q=1020), dict(hs_q=64), dict(k_pages=None), dict(k_pages=MIS), dict(v_pages=None), dict(v_pages=MIS),
    dict(page_table=None), dict(page_table=A + 2), dict(lens=None), dict(lens=A + 1), dict(rows=A + 2), dict(n_seqs=-1), dict(tokens=0),
    dict(tokens=-1), dict(window=-1), dict(scale=0.0), dict(scale=-1.0), dict(scale=math.nan), dict(scale=math.inf), dict(out=None), dict(out=MIS),
    dict(lse=B + 2)])
def test_decode_refusals(lib, kw):
    assert decode(lib, **kw) == INVALID


def test_decode_limits(lib):
    assert lib.gdn_attn_decode(ctypes.byref(cfg()), None, A, 1 << 40, None) == INVALID
    assert decode(lib, tokens=9) == UNSUPPORTED
    assert decode(lib, n_seqs=65536) == UNSUPPORTED
    assert decode(lib, n_seqs=0, ws=None, size=0) == OK
    for c in (cfg(n_pages=0), cfg(n_rows=0), cfg(max_pages=0)):
        assert decode(lib, c) == INVALID
    need = gdn.gdn_attn_workspace_size(cfg(), 3, 2)
    assert need > gdn.gdn_attn_workspace_size(cfg(), 3, 1) > 0
    for ws, size in ((None, 1 << 40), (MIS, 1 << 40), (A, 1000)):
        assert decode(lib, ws=ws, size=size) == WORKSPACE
    assert gdn.gdn_attn_workspace_size(cfg(), 3, 0) == gdn.gdn_attn_workspace_size(cfg(), 3, 9) == gdn.gdn_attn_workspace_size(cfg(), -1, 1) == 0


def test_longest_length(lib):
    """Lengths leave room for a tile in 32 bits."""
    assert gdn.gdn_attn_workspace_size(cfg(page_size=64, max_pages=1 << 24), 3, 1) > 0
    assert decode(lib, cfg(page_size=64, max_pages=(1 << 24) + 1)) == UNSUPPORTED


def test_scale_beyond_the_powers_of_two(lib):
    """A scale whose product with log2(e) is no 32-bit number."""
    assert decode(lib, scale=3e38) == INVALID


def test_page_refusals(lib):
    for kw in (dict(table=None), dict(lens=None), dict(refs=A + 2), dict(rows=None), dict(new=A + 1), dict(granted=None), dict(src=None),
               dict(dst=B + 2), dict(n=-1)):
        assert resize(lib, **kw) == INVALID, kw
    for kw in (dict(table=None), dict(lens=A + 1), dict(refs=None), dict(src=None), dict(dst=None), dict(n=-1)):
        assert fork(lib, **kw) == INVALID, kw
    for kw in (dict(table=None), dict(lens=None), dict(refs=None), dict(table_out=None), dict(refs_out=B + 1), dict(src=None), dict(dst=None),
               dict(n=-1)):
        assert compact(lib, **kw) == INVALID, kw
    for kw in (dict(sk=MIS), dict(dv=MIS), dict(dk=None, dv=None), dict(src=None), dict(dst=A + 2), dict(n=-1), dict(n_src=-1), dict(n_dst=-1)):
        assert copy(lib, **kw) == INVALID, kw
    for c in (cfg(n_pages=0), cfg(n_rows=0), cfg(max_pages=0)):
        assert {resize(lib, c), fork(lib, c), compact(lib, c)} == {INVALID}
    assert {resize(lib, n=0), fork(lib, n=0), copy(lib, n=0)} == {OK}
    assert {resize(lib, n=65536), fork(lib, n=65536)} == {UNSUPPORTED}
    for ws, size in ((None, 1 << 40), (MIS, 1 << 40), (A, 40)):
        assert {resize(lib, ws=ws, size=size), compact(lib, ws=ws, size=size)} == {WORKSPACE}
    assert gdn.gdn_page_workspace_size(cfg(), -1) == 0


def test_structure_layouts(tmp_path):
    """The binding's structures have the header's field offsets."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    structs = {"gdn_attn_config": gdn.AttnConfig, "gdn_attn_prep_io": gdn.AttnPrepIO, "gdn_attn_decode_io": gdn.AttnDecodeIO}
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

@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_rotation_is_a_rotation(interleaved):
    """Lengths of pairs stay, and a query's product with a key depends on the distance of their positions alone."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn(1, 2, 10, generator=g, dtype=torch.float64)
    f = torch.tensor([1.0, 0.3, 0.01], dtype=torch.float64)

    def at(p):
        return ref.rotate(x, x.abs(), torch.tensor([p]), f, interleaved)[0][0]
    assert torch.allclose(at(0), x[0])
    assert torch.allclose(at(5).square().sum(-1), x[0].square().sum(-1))
    assert torch.equal(at(7)[:, 6:], x[0, :, 6:])
    assert torch.allclose(at(9)[0] @ at(4)[1], at(105)[0] @ at(100)[1])
    # one pair by hand: (1, 0) at angle t is (cos t, sin t)
    e = torch.zeros(1, 1, 10, dtype=torch.float64)
    e[..., 0] = 1.0
    y = ref.rotate(e, e, torch.tensor([2]), f, interleaved)[0][0, 0]
    assert math.isclose(y[0], math.cos(2.0)) and math.isclose(y[1 if interleaved else 3], math.sin(2.0))


@pytest.mark.parametrize("weights", [True, False])
@pytest.mark.parametrize("interleaved", [False, True])
def test_reference_gradients_are_differences(weights, interleaved):
    g = torch.Generator().manual_seed(1)
    r = lambda *s: torch.randn(s, generator=g, dtype=torch.float64)  # noqa: E731
    x, w, d = r(3, 2, 8), r(8) if weights else None, r(3, 2, 8)
    pos, f = torch.tensor([0, 4, 11]), torch.tensor([1.0, 0.2], dtype=torch.float64)

    def loss(x, w):
        return float((ref.prep(x, w, pos, f, 0.5, 1e-3, interleaved)[0] * d).sum())
    (dx, mag), dw = ref.prep_backward(x, w, d, pos, f, 0.5, 1e-3, interleaved)
    assert (mag >= dx.abs() - 1e-12).all() and (dw is None) == (w is None)
    for leaf, grad in ((x, dx),) + (((w, dw[0]),) if weights else ()):
        for i in range(leaf.numel()):
            vals = []
            for e in (1e-5, -1e-5):
                keep = float(leaf.view(-1)[i])
                leaf.view(-1)[i] = keep + e
                vals.append(loss(x, w))
                leaf.view(-1)[i] = keep
            assert math.isclose(grad.reshape(-1)[i], (vals[0] - vals[1]) / 2e-5, rel_tol=1e-6, abs_tol=1e-8)


def test_reference_attention_closed_forms():
    """One visible token gives its value; equal scores the mean; masked tokens nothing; an empty row zero and -inf."""
    g = torch.Generator().manual_seed(2)
    q, K, V = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((2, 4, 8), (2, 6, 8), (2, 6, 8)))
    out, lse, mag, top = ref.attend(q, K, V, [1, 0], 0.5)
    assert torch.allclose(out[0, 3], V[1, 0]) and math.isclose(lse[0, 3], 0.5 * float(K[1, 0] @ q[0, 3]))
    assert not out[1].any() and (lse[1] == -math.inf).all()
    out, lse, _, _ = ref.attend(torch.zeros_like(q), K, V, [5, 6], 0.5, window=3)
    assert torch.allclose(out[0, 0], V[0, 2:5].mean(0)) and torch.allclose(out[1, 2], V[1, 3:6].mean(0)) and math.isclose(lse[1, 0], math.log(3))
    out, _, _, _ = ref.attend(q, K, V, [6, 6], 0.5, seen=[False] * 5 + [True])
    assert torch.allclose(out[0, 0], V[0, 5])


def test_reference_pages():
    """A worked example: fork, copy on write, exhaustion, truncation, compaction."""
    p = ref.Pages(n_pages=6, n_rows=3, max_pages=4, page=16)
    assert p.resize([0], [20]) == ([20], [-1], [-1], 0) and p.table[0] == [0, 1, -1, -1] and p.refs == [1, 1, 0, 0, 0, 0]
    assert p.fork([0, 0], [1, 2]) == 0 and p.refs == [3, 3, 0, 0, 0, 0] and p.lens == [20, 20, 20]
    assert p.resize([1, 2], [21, 33]) == ([21, 33], [1, 1], [2, 3], 0)
    assert p.table[1] == [0, 2, -1, -1] and p.table[2] == [0, 3, 4, -1] and p.refs == [3, 1, 1, 1, 1, 0]
    p.check()
    assert p.resize([0, 1, 2], [49, 22, 34]) == ([20, 22, 34], [-1, -1, -1], [-1, -1, -1], 0)      # two pages wanted, one free
    assert p.resize([1, 1, 5], [0, 0, 0]) == ([-1, -1, -1], [-1] * 3, [-1] * 3, 2)
    assert p.resize([0, 1], [0, 3]) == ([0, 3], [-1, -1], [-1, -1], 0) and p.refs == [2, 0, 0, 1, 1, 0]
    assert p.resize([1], [5]) == ([5], [0], [1], 0) and p.refs == [1, 1, 0, 1, 1, 0]
    assert p.compact(3) == ([4, -1, -1], [2, -1, -1]) and p.table[2] == [0, 3, 2, -1] and p.refs == [1, 1, 1, 1, 0, 0]
    p.check()
