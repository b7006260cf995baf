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
        for got, v, m, r, name in ((y[s:e].cpu(), val.reshape(L, b.H * b.P), mag.reshape(L, b.H * b.P), rel_y, "y"), (out[n].cpu(), S, M, rel, "state")):
            ok = v.isfinite()
            assert not got[~ok].isfinite().any(), "%s of sequence %d" % (name, n)
            ref.check(got[ok], v[ok], m[ok], r, name)
    assert gdn.gdn_device_error() == 0


@pytest.mark.parametrize("act", ["fp32", "bf16"])
@pytest.mark.parametrize("decay", [70.0, 80.0, 200.0])
def test_tokens_that_add_nothing_forget(act, decay):
    """Tokens of zeros with a log-decay below -60 each: what is left of the state is exp(-decay) of it,
    not a floor that stands above that."""
    b = Batch([100, 300, 600], H=2, G=1, N=64, P=64, act=act, seed=71, dt_min=1.0, dt_max=1.0)
    b.A_log = torch.full((2,), decay).log()
    b.D = None
    x, bb, _ = b.parts(b.xbc)
    for n, L in enumerate(b.lens):
        s = int(b.cu[n])
        for t in (3, 40, 41, L // 2, L - 1):
            x[s + t] = 0
    b.verify(*b.run())


@pytest.mark.parametrize("act", ["fp32", "bf16"])
def test_slow_tokens_behind_fast_ones(act):
    """Tokens that forget everything, then tokens that forget little: the latter's decays are differences
    of sums that the former made large."""
    b = Batch([110, 300, 520], H=2, G=1, N=64, P=64, act=act, seed=72, rate=(30.0, 40.0), dt_shift=0.0)
    for n, L in enumerate(b.lens):
        s = int(b.cu[n])
        b.u[s:s + L] = -7.0
        for t in range(0, L - 12, 128):
            b.u[s + t:s + min(t + 98, L - 12)] = 5.0
    b.dt_bias = None
    b.verify(*b.run())


@pytest.mark.parametrize("act", ["fp32", "bf16"])
@pytest.mark.parametrize("cu", [[0, 900, 900, 300, 900], [0, 500, 400, 900], [-5, 100, 200, 900], [0, 100, 200, 5000], [0, 900, 0, 900]])
def test_conv_reports_malformed_lengths(act, cu):
    """Wherever the pair that goes back stands, also behind the last token.  (Every bound is clamped to the
    batch before it is used.)"""
    dt = torch.bfloat16 if act == "bf16" else torch.float32
    n, CH = len(cu) - 1, 64 + 32
    cfg = gdn.make_ssm_config(1, 1, 16, 64, act=act, n_slots=n)
    x, w = torch.zeros(900, CH, dtype=dt, device="cuda"), torch.zeros(CH, 4, dtype=dt, device="cuda")
    hist, out = torch.zeros(n, CH, 3, dtype=dt, device="cuda"), torch.empty(900, CH, dtype=dt, device="cuda")
    assert gdn.gdn_device_error() == 0
    gdn.gdn_ssm_conv_prefill(cfg, x, torch.tensor(cu, dtype=torch.int32, device="cuda"), w, None, hist, None, out)
    assert gdn.gdn_device_error() & gdn.DEVERR_CU_SEQLENS
    gdn.gdn_ssm_conv_prefill(cfg, x, torch.tensor([0] * n + [900], dtype=torch.int32, device="cuda"), w, None, hist, None, out)
    assert gdn.gdn_device_error() == 0


@pytest.mark.parametrize("act", ["fp32", "bf16"])
@pytest.mark.parametrize("fill", [NAN, INF])
def test_states_that_are_not_finite(act, fill):
    """One value of a state that comes in: its column of its head, and nothing else."""
    b = Batch([200, 600, 0, 40], H=4, G=2, N=64, P=64, act=act, seed=73)
    b.state[1, 2, 5, 7] = fill
    b.state[2, 0, 1, 3] = fill
    y, out = b.run()
    for n, L in enumerate(b.lens):
        s, e = int(b.cu[n]), int(b.cu[n + 1])
        val, mag, S, M = b.reference(n)
        rel = (8 * L + b.N + 64) * ref.U32
        rel_y = rel + (2 * 2.0 ** -8 + 2 * 128 * 60 * ref.U32 if act == "bf16" else 0)
        for got, v, m, r, name in ((y[s:e].cpu(), val.reshape(L, b.H * b.P), mag.reshape(L, b.H * b.P), rel_y, "y"), (out[n].cpu(), S, M, rel, "state")):
            ok = v.isfinite()
            assert not got[~ok].isfinite().any(), "%s of sequence %d" % (name, n)
            ref.check(got[ok], v[ok], m[ok], r, name)
    assert gdn.gdn_device_error() == 0


@pytest.mark.parametrize("act", ["fp32", "bf16"])
def test_many_sequences_in_a_graph_with_other_lengths(act):
    """A captured call of more sequences than a warp lays out, some cut, replayed with other lengths, fewer
    tokens and nothing behind them written; into a pool of its own, then in place."""
    lens = [5, 0, 40] * 12 + [700, 300, 1, 900]
    b = Batch(lens, H=2, G=1, act=act, seed=74).upload()
    y, out = torch.full((b.rows, b.H * b.P), 7.0, dtype=b.act, device="cuda"), torch.full_like(b.d_state, 7.0)
    state = b.d_state.clone()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        b.launch(y, out)
    with torch.cuda.graph(graphs[1]):
        b.launch(y, state, state=state)
    graphs[0].replay()
    b.verify(y, out)
    assert (out == b.d_state)[[n for n, L in enumerate(lens) if L == 0]].all()
    b.lens = [300, 0, 3] + [0, 1, 30] * 12 + [513]
    b.cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
    b.cu[1:] = torch.tensor(b.lens).cumsum(0)
    b.d_cu.copy_(b.cu)
    for graph, to in zip(graphs, (out, state)):
        y.fill_(7.0)
        graph.replay()
        b.verify(y, to)
        assert (y[int(b.cu[-1]):] == 7).all()
    assert torch.equal(out, state)
    assert gdn.gdn_device_error() == 0
