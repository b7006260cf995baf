"""The selective state space mixer on the GPU against the plain 64-bit reference: types, head
layouts, lengths from nothing to several segments, slots, strides, clamps, streams, graphs."""
import pytest
import torch

import ssm_ref as ref
from gateddeltanet_linear_attention_gb300 import gdn

pytestmark = pytest.mark.gpu
INF = float("inf")


def randn(*shape, gen, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen) * std).to(dtype)


class Batch:
    """Inputs of one packed batch on the CPU, its call on the GPU and its reference."""

    def __init__(self, lens, H=4, G=2, N=64, P=64, act="bf16", seed=0, slots=None, state_idx=None, z=True, D=True,
                 bias=True, state=True, dt_min=0.0, dt_max=INF, tail=0, rate=(1.0, 16.0), dt_shift=-3.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.H, self.G, self.N, self.P = lens, H, G, N, P
        self.act = torch.bfloat16 if act == "bf16" else torch.float32
        T = self.T = sum(lens)
        R = self.rows = T + tail
        self.cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
        self.cu[1:] = torch.tensor(lens).cumsum(0)
        xbc = randn(R, H * P + 2 * G * N, gen=g)
        self.xbc = (xbc * torch.sigmoid(xbc)).to(self.act)
        self.u = randn(R, H, gen=g, dtype=self.act)
        self.z = randn(R, H * P, gen=g, dtype=self.act) if z else None
        self.A_log = torch.log(torch.rand(H, generator=g) * (rate[1] - rate[0]) + rate[0])
        self.D = 1 + 0.1 * randn(H, gen=g) if D else None
        self.dt_bias = dt_shift + randn(H, gen=g) if bias else None
        self.slots = slots or max(len(lens), 1)
        self.state_idx = None if state_idx is None else torch.tensor(state_idx, dtype=torch.int32)
        self.state = randn(self.slots, H, N, P, gen=g, std=0.5) if state else None
        self.dt_min, self.dt_max = dt_min, dt_max
        self.cfg = gdn.make_ssm_config(G, H, N, P, act=act, n_slots=self.slots, dt_min=dt_min, dt_max=dt_max)

    def parts(self, t):
        HP, GN = self.H * self.P, self.G * self.N
        return t[:, :HP], t[:, HP:HP + GN], t[:, HP + GN:]

    def upload(self):
        for k in ("xbc", "u", "z", "A_log", "D", "dt_bias", "cu", "state_idx", "state"):
            v = getattr(self, k)
            setattr(self, "d_" + k, None if v is None else v.cuda())
        need = gdn.gdn_ssm_workspace_size(self.cfg, self.rows, len(self.lens))
        self.ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
        return self

    def launch(self, y, out, state=None, stream=None):
        x, b, c = self.parts(self.d_xbc)
        gdn.gdn_ssm_prefill(self.cfg, x, b, c, self.d_u, self.d_A_log, self.d_cu, y, D=self.d_D, dt_bias=self.d_dt_bias,
                            z=self.d_z, state_in=self.d_state if state is None else state, state_out=out,
                            state_idx=self.d_state_idx, workspace=self.ws, stream=stream)

    def run(self, in_place=False):
        self.upload()
        y = torch.full((self.rows, self.H * self.P), 7.0, dtype=self.act, device="cuda")
        if in_place:
            out = self.d_state.clone()
            self.launch(y, out, state=out)
        else:
            out = torch.full((self.slots, self.H, self.N, self.P), 7.0, device="cuda")
            self.launch(y, out)
        torch.cuda.synchronize()
        return y, out

    def slot(self, n):
        return n if self.state_idx is None else int(self.state_idx[n])

    def reference(self, n):
        s, e = int(self.cu[n]), int(self.cu[n + 1])
        x, b, c = self.parts(self.xbc[s:e])
        L = e - s
        S = torch.zeros(self.H, self.N, self.P) if self.state is None else self.state[self.slot(n)]
        return ref.scan(x.reshape(L, self.H, self.P), b.reshape(L, self.G, self.N), c.reshape(L, self.G, self.N), self.u[s:e],
                        self.A_log, self.D, self.dt_bias, None if self.z is None else self.z[s:e], S, self.G,
                        self.dt_min, self.dt_max)

    def verify(self, y, out, seqs=None):
        """32-bit arithmetic: about 8 roundings a token in the recurrence and N in the sum over the
        state (the chunked form has fewer); exp of a log-decay summed in 32 bits over a chunk of 128
        tokens of at most 60 in size (the clamp): below 128 * 60 * 2^-24 of relative error, and the
        same again for its products.  Scores and states that enter 16-bit products: half a step."""
        for n in range(len(self.lens)) if seqs is None else seqs:
            s, e, slot = int(self.cu[n]), int(self.cu[n + 1]), self.slot(n)
            if slot < 0:
                assert (y[s:e] == 0).all()
                continue
            val, mag, S, M = self.reference(n)
            L = e - s
            rel = (8 * L + self.N + 64) * ref.U32
            rel_y = rel + (2 * 2.0 ** -8 + 2 * 128 * 60 * ref.U32 if self.act == torch.bfloat16 else 0)
            ref.check(y[s:e], val.reshape(L, self.H * self.P), mag.reshape(L, self.H * self.P), rel_y, "y of sequence %d" % n)
            if out is not None:
                ref.check(out[slot], S, M, rel, "state of sequence %d" % n)


@pytest.mark.parametrize("act", ["fp32", "bf16"])
@pytest.mark.parametrize("N,P", [(16, 32), (16, 64), (32, 32), (32, 128), (64, 32), (64, 64), (64, 128), (128, 32),
                                 (128, 64), (128, 128), (16, 128)])
def test_sizes(act, N, P):
    b = Batch([1, 130, 0, 64, 3, 257], N=N, P=P, act=act)
    b.verify(*b.run())


@pytest.mark.parametrize("act", ["fp32", "bf16"])
@pytest.mark.parametrize("H,G", [(1, 1), (3, 1), (6, 2), (5, 5), (8, 1), (12, 4)])
def test_head_layouts(act, H, G):
    b = Batch([37, 200], H=H, G=G, act=act, seed=1)
    b.verify(*b.run())


@pytest.mark.parametrize("act", ["fp32", "bf16"])
@pytest.mark.parametrize("N,P,H,G", [(64, 64, 2, 1), (128, 128, 1, 1), (128, 64, 3, 1)])
def test_long_sequences_are_cut(act, N, P, H, G):
    """Several segments, next to sequences of one; the workspace holds garbage before the call."""
    b = Batch([300, 1500, 0, 1, 256, 257, 770], H=H, G=G, N=N, P=P, act=act, seed=2)
    b.verify(*b.run())


@pytest.mark.parametrize("lens", [[1], [0], [127], [128], [129], [255], [512, 513]])
@pytest.mark.parametrize("act", ["fp32", "bf16"])
def test_lengths(act, lens):
    b = Batch(lens, H=2, G=1, N=128, P=64, act=act, seed=3)
    b.verify(*b.run())


@pytest.mark.parametrize("act", ["fp32", "bf16"])
@pytest.mark.parametrize("off", ["z", "D", "bias", "state"])
def test_optional_inputs(act, off):
    b = Batch([150, 20], act=act, seed=4, **{off: False})
    y, out = b.run()
    b.verify(y, out)


@pytest.mark.parametrize("act", ["fp32", "bf16"])
def test_clamped_steps(act):
    b = Batch([200], act=act, seed=5, dt_min=0.01, dt_max=0.05)
    b.verify(*b.run())
    x = Batch([200], act=act, seed=5)
    assert not torch.equal(x.run()[0], b.run()[0])


@pytest.mark.parametrize("act", ["fp32", "bf16"])
@pytest.mark.parametrize("rate,shift", [((1e-4, 1e-3), -3.0), ((50.0, 400.0), 2.0), ((1.0, 16.0), -40.0), ((1e30, 1e38), 30.0)])
def test_decays(act, rate, shift):
    """Nearly none, one that forgets within a token, step sizes of nothing, exponents past every range."""
    b = Batch([140, 300, 5], N=64, P=64, act=act, seed=6, rate=rate, dt_shift=shift)
    b.verify(*b.run())


@pytest.mark.parametrize("act", ["fp32", "bf16"])
@pytest.mark.parametrize("in_place", [False, True])
def test_slots_and_padding_lanes(act, in_place):
    b = Batch([300, 40, 0, 600, 17], H=2, G=1, act=act, seed=7, slots=9, state_idx=[4, -1, 8, 0, -3])
    y, out = b.run(in_place)
    b.verify(y, out)
    touched = {4, 8, 0}
    for s in range(9):
        if s not in touched:
            want = b.state[s] if in_place else torch.full_like(b.state[s], 7.0)
            assert torch.equal(out[s].cpu(), want)
    assert torch.equal(out[8].cpu(), b.state[8])           # an empty sequence's state as it was
    assert gdn.gdn_device_error() == 0


@pytest.mark.parametrize("act", ["fp32", "bf16"])
@pytest.mark.parametrize("fill", [float("nan"), INF, -INF])
def test_neighbours_and_rows_behind_do_not_leak(act, fill):
    """A sequence of infinities or NaN, and such rows behind the last sequence: the others are right
    and the rows behind keep what they held."""
    b = Batch([100, 30, 61, 300], H=2, G=1, act=act, seed=8, tail=70)
    s, e = int(b.cu[1]), int(b.cu[2])
    for t in (b.xbc, b.u, b.z):
        t[s:e] = fill
        t[b.T:] = fill
    y, out = b.run()
    b.verify(y, out, seqs=[0, 2, 3])
    assert (y[b.T:] == 7).all()
    assert gdn.gdn_device_error() == 0


def test_padding_lane_of_nan_is_zero():
    b = Batch([90, 30], H=2, G=1, seed=9, slots=2, state_idx=[0, -1])
    s = int(b.cu[1])
    for t in (b.xbc, b.u, b.z):
        t[s:] = float("nan")
    y, out = b.run()
    b.verify(y, out)


@pytest.mark.parametrize("act", ["fp32", "bf16"])
def test_row_strides_and_separate_views(act):
    b = Batch([70, 260], H=2, G=1, act=act, seed=10).upload()
    T, HP, GN = b.T, b.H * b.P, b.G * b.N
    x, bb, cc = b.parts(b.d_xbc)
    wide = torch.randn(T, HP + 24, device="cuda").to(b.act)
    wide[:, 8:8 + HP] = x
    bc = torch.randn(T, 3 * GN + 16, device="cuda").to(b.act)
    bc[:, 8:8 + GN], bc[:, 2 * GN:3 * GN] = bb, cc
    u = torch.randn(T, b.H + 3, device="cuda").to(b.act)
    u[:, 1:1 + b.H] = b.d_u
    z = torch.randn(T, HP + 8, device="cuda").to(b.act)
    z[:, :HP] = b.d_z
    y, y2 = (torch.empty(T, HP, dtype=b.act, device="cuda") for _ in range(2))
    o, o2 = (torch.empty_like(b.d_state) for _ in range(2))
    b.launch(y, o)
    gdn.gdn_ssm_prefill(b.cfg, wide[:, 8:8 + HP], bc[:, 8:8 + GN], bc[:, 2 * GN:3 * GN], u[:, 1:1 + b.H], b.d_A_log, b.d_cu, y2,
                        D=b.d_D, dt_bias=b.d_dt_bias, z=z[:, :HP], state_in=b.d_state, state_out=o2, workspace=b.ws)
    assert torch.equal(y, y2) and torch.equal(o, o2)


@pytest.mark.parametrize("act", ["fp32", "bf16"])
def test_same_bits_again_and_on_another_stream_and_in_a_graph(act):
    b = Batch([700, 31], H=2, G=1, act=act, seed=11)
    y, out = b.run()
    y2, out2 = torch.empty_like(y), torch.empty_like(out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.launch(y2, out2)
    s.synchronize()
    assert torch.equal(y, y2) and torch.equal(out, out2)
    y3, out3 = torch.empty_like(y), torch.empty_like(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.launch(y3, out3)
    y3.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, y3) and torch.equal(out, out3)
    # a smaller batch of other lengths through the same graph: the rows behind it stay
    b.d_cu.copy_(torch.tensor([0, 333, 340], dtype=torch.int32))
    y3.fill_(3.0)
    graph.replay()
    torch.cuda.synchronize()
    b.cu = torch.tensor([0, 333, 340], dtype=torch.int32)
    b.lens = [333, 7]
    b.verify(y3, out3)
    assert (y3[340:] == 3).all()


def test_two_calls_at_once():
    one, two = (Batch([500, 40], H=2, G=1, seed=s) for s in (12, 13))
    want = [b.run() for b in (one, two)]
    outs = [[torch.empty_like(t) for t in w] for w in want]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for b, o, s in zip((one, two), outs, streams):
            with torch.cuda.stream(s):
                b.launch(*o)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(p, q) for p, q in zip(w, o))


def test_cut_in_two_calls_is_one_call():
    """A prompt in two parts, the state carried in its slot: the reference's values to the same bounds."""
    b = Batch([400], H=2, G=1, act="fp32", seed=14)
    y, out = b.run()
    b2 = Batch([400], H=2, G=1, act="fp32", seed=14).upload()
    state = b2.d_state.clone()
    y2 = torch.empty_like(y)
    for lo, hi in ((0, 155), (155, 400)):
        x, bb, c = b2.parts(b2.d_xbc[lo:hi])
        gdn.gdn_ssm_prefill(b2.cfg, x, bb, c, b2.d_u[lo:hi], b2.d_A_log, torch.tensor([0, hi - lo], dtype=torch.int32, device="cuda"),
                            y2[lo:hi], D=b2.d_D, dt_bias=b2.d_dt_bias, z=b2.d_z[lo:hi], state_in=state, state_out=state, workspace=b2.ws)
    b.verify(y2, state)


@pytest.mark.parametrize("act", ["fp32", "bf16"])
@pytest.mark.parametrize("cu", [[0, 500, 400, 900], [0, 900, 0, 900], [-5, 100, 200, 900], [0, 100, 200, 5000],
                                [0, 900, -2000000000, 2000000000]])
def test_malformed_lengths_are_reported(act, cu):
    b = Batch([300, 300, 300], H=2, G=1, act=act, seed=15).upload()
    y = torch.zeros(900, 128, dtype=b.act, device="cuda")
    b.d_cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
    assert gdn.gdn_device_error() == 0
    b.launch(y, torch.zeros_like(b.d_state))
    assert gdn.gdn_device_error() & gdn.DEVERR_CU_SEQLENS
    b.d_cu = b.cu.cuda()
    out = torch.zeros_like(b.d_state)
    b.launch(y, out)
    assert gdn.gdn_device_error() == 0
    b.verify(y, out)


def test_slot_out_of_range_is_reported():
    b = Batch([60, 60], H=2, G=1, seed=16, slots=2, state_idx=[0, 2]).upload()
    y = torch.full((120, 128), 7.0, dtype=b.act, device="cuda")
    out = torch.full_like(b.d_state, 7.0)
    b.launch(y, out)
    assert gdn.gdn_device_error() & gdn.DEVERR_SLOT
    b.verify(y, out, seqs=[0])
    assert (out[1] == 7).all()


# ------------------------------------------------------------------- convolution

def conv_case(lens, H, G, N, P, act, seed, slots=None, state_idx=None, tail=0, ld_extra=0):
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if act == "bf16" else torch.float32
    CH, T = H * P + 2 * G * N, sum(lens)
    wide = randn(T + tail, CH + ld_extra, gen=g, dtype=dt)
    slots = slots or max(1, len(lens))
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(lens).cumsum(0)
    return dict(cfg=gdn.make_ssm_config(G, H, N, P, act=act, n_slots=slots), x=wide[:, ld_extra // 2:ld_extra // 2 + CH], wide=wide,
                w=randn(CH, 4, gen=g, dtype=dt), bias=randn(CH, gen=g, dtype=dt), hist=randn(slots, CH, 3, gen=g, dtype=dt), cu=cu,
                lens=lens, CH=CH, idx=None if state_idx is None else torch.tensor(state_idx, dtype=torch.int32), off=ld_extra // 2)


CONV_REL = 16 * ref.U32      # four products, four sums, exp, sum, quotient


@pytest.mark.parametrize("act", ["fp32", "bf16"])
@pytest.mark.parametrize("lens", [[1], [2, 1, 0, 3, 0, 0, 4], [15, 1, 1, 1, 16, 17], [33, 2, 14, 2, 100], [0, 0], [14, 3, 15, 2, 30]])
@pytest.mark.parametrize("hist,bias", [(True, True), (False, False)])
def test_conv(act, lens, hist, bias):
    c = conv_case(lens, 3, 1, 32, 64, act, 20, tail=9, ld_extra=16)
    d_hist = c["hist"].cuda() if hist else None
    wide = c["wide"].cuda()
    x = wide[:, c["off"]:c["off"] + c["CH"]]
    out = torch.full((x.shape[0], c["CH"]), 7.0, dtype=x.dtype, device="cuda")
    gdn.gdn_ssm_conv_prefill(c["cfg"], x, c["cu"].cuda(), c["w"].cuda(), c["bias"].cuda() if bias else None, d_hist, None, out)
    for n, L in enumerate(lens):
        s = int(c["cu"][n])
        val, mag, new = ref.conv(c["x"][s:s + L], c["w"], c["bias"] if bias else None, c["hist"][n] if hist else torch.zeros(c["CH"], 3))
        ref.check(out[s:s + L], val, mag, CONV_REL, "conv of sequence %d" % n)
        if hist:
            assert torch.equal(d_hist[n].cpu().double(), new)
    assert (out[sum(lens):] == 7).all()
    assert gdn.gdn_device_error() == 0


@pytest.mark.parametrize("act", ["fp32", "bf16"])
def test_conv_slots(act):
    c = conv_case([20, 5, 0, 2], 2, 1, 32, 64, act, 21, slots=6, state_idx=[5, -1, 3, 0])
    d_hist = c["hist"].cuda()
    out = torch.empty(27, c["CH"], dtype=d_hist.dtype, device="cuda")
    gdn.gdn_ssm_conv_prefill(c["cfg"], c["x"].cuda(), c["cu"].cuda(), c["w"].cuda(), c["bias"].cuda(), d_hist, c["idx"].cuda(), out)
    for n, slot in ((0, 5), (3, 0)):
        s, e = int(c["cu"][n]), int(c["cu"][n + 1])
        val, mag, new = ref.conv(c["x"][s:e], c["w"], c["bias"], c["hist"][slot])
        ref.check(out[s:e], val, mag, CONV_REL, "sequence %d" % n)
        assert torch.equal(d_hist[slot].cpu().double(), new)
    assert (out[20:25] == 0).all()
    for slot in (1, 2, 3, 4):
        assert torch.equal(d_hist[slot].cpu(), c["hist"][slot])
    assert gdn.gdn_device_error() == 0


# ------------------------------------------------------------------- single tokens

@pytest.mark.parametrize("act", ["fp32", "bf16"])
@pytest.mark.parametrize("n,H,G,N,P", [(1, 1, 1, 16, 32), (3, 4, 2, 64, 64), (5, 6, 1, 128, 64), (2, 4, 4, 128, 128), (70, 2, 1, 32, 128),
                                       (4, 3, 3, 64, 32), (2, 2, 1, 16, 64), (2, 2, 1, 16, 128), (300, 1, 1, 32, 32)])
@pytest.mark.parametrize("full", [True, False])
def test_step(act, n, H, G, N, P, full):
    g = torch.Generator().manual_seed(30 + n)
    dt = torch.bfloat16 if act == "bf16" else torch.float32
    CH, slots = H * P + 2 * G * N, n + 2
    order = torch.randperm(slots, generator=g)[:n].to(torch.int32)
    if n > 2:
        order[1] = -1
    x, u = randn(n, CH + 8, gen=g, dtype=dt), randn(n, H + 1, gen=g, dtype=dt)
    w, hist = randn(CH, 4, gen=g, std=0.5, dtype=dt), randn(slots, CH, 3, gen=g, dtype=dt)
    state = randn(slots, H, N, P, gen=g, std=0.5)
    A_log = torch.rand(H, generator=g)
    z, D, dt_bias, bias = (randn(n, H * P, gen=g, dtype=dt), randn(H, gen=g), randn(H, gen=g), randn(CH, gen=g, dtype=dt)) if full else [None] * 4
    cfg = gdn.make_ssm_config(G, H, N, P, act=act, n_slots=slots)

    def up(t):
        return None if t is None else t.cuda()

    dx, du, dh, ds = up(x), up(u), up(hist), up(state)
    y = torch.full((n, H * P), 7.0, dtype=dt, device="cuda")
    ws = torch.full((gdn.gdn_ssm_workspace_size(cfg, n, n),), 0xFF, dtype=torch.uint8, device="cuda")
    gdn.gdn_ssm_decode(cfg, dx[:, :CH], du[:, 1:], up(w), dh, up(A_log), ds, y, ws, conv_bias=up(bias), D=up(D), dt_bias=up(dt_bias),
                       z=up(z), state_idx=up(order))
    torch.cuda.synchronize()
    live = set()
    for i in range(n):
        slot = int(order[i])
        if slot < 0:
            assert (y[i] == 0).all()
            continue
        live.add(slot)
        xbc, xm, new = ref.conv(x[i:i + 1, :CH], w, bias, hist[slot])
        assert torch.equal(dh[slot].cpu().double(), new)
        HP, GN = H * P, G * N
        args = (u[i:i + 1, 1:], A_log, D, dt_bias, None if z is None else z[i:i + 1], state[slot], G)
        val, mag, S, M = ref.scan(xbc[:, :HP].view(1, H, P), xbc[:, HP:HP + GN].view(1, G, N), xbc[:, HP + GN:].view(1, G, N), *args)
        # the convolution's own error enters through its magnitude (each of two factors)
        _, mag, _, M = ref.scan(xm[:, :HP].view(1, H, P), xm[:, HP:HP + GN].view(1, G, N), xm[:, HP + GN:].view(1, G, N), *args[:5], state[slot].abs(), G)
        mag = mag.abs()
        rel = (N + 64) * ref.U32
        ref.check(y[i:i + 1], val.view(1, -1), mag.view(1, -1), rel, "y of %d" % i)
        ref.check(ds[slot], S, M, rel, "state of %d" % i)
    for slot in range(slots):
        if slot not in live:
            assert torch.equal(ds[slot].cpu(), state[slot]) and torch.equal(dh[slot].cpu(), hist[slot])
    assert gdn.gdn_device_error() == 0


@pytest.mark.parametrize("act", ["fp32", "bf16"])
def test_prompt_then_tokens_then_norm_as_a_model_runs_them(act):
    """A mixer layer of a hybrid model: norm, convolution, scan, norm; then the next tokens one by
    one, captured in a graph.  The whole against 64 bits over the uncut sequence."""
    H, G, N, P, n, L, steps = 4, 2, 64, 64, 2, 150, 4
    g = torch.Generator().manual_seed(40)
    dt = torch.bfloat16 if act == "bf16" else torch.float32
    CH, HP, GN, dim = H * P + 2 * G * N, H * P, G * N, H * P
    raw, u = randn(n, L + steps, CH, gen=g, dtype=dt), randn(n, L + steps, H, gen=g, dtype=dt)
    w, bias = randn(CH, 4, gen=g, std=0.5, dtype=dt), randn(CH, gen=g, std=0.1, dtype=dt)
    A_log, D, dt_bias = torch.rand(H, generator=g), randn(H, gen=g), randn(H, gen=g) - 3
    res, w_post = randn(n, L + steps, dim, gen=g), 1 + 0.1 * randn(dim, gen=g)
    cfg = gdn.make_ssm_config(G, H, N, P, act=act, n_slots=n)
    dev = [t.cuda() for t in (raw, u, w, bias, A_log, D, dt_bias, res, w_post)]
    draw, du, dw, dbias, dA, dD, ddt, dres, dwp = dev
    hist, state = torch.zeros(n, CH, 3, dtype=dt, device="cuda"), torch.zeros(n, H, N, P, device="cuda")
    cu = torch.tensor([0, L, 2 * L], dtype=torch.int32, device="cuda")
    x = draw[:, :L].reshape(n * L, CH).contiguous()
    xbc, y = torch.empty_like(x), torch.empty(n * L, HP, dtype=dt, device="cuda")
    ws = torch.empty(gdn.gdn_ssm_workspace_size(cfg, n * L, n), dtype=torch.uint8, device="cuda")
    gdn.gdn_ssm_conv_prefill(cfg, x, cu, dw, dbias, hist, None, xbc)
    gdn.gdn_ssm_prefill(cfg, xbc[:, :HP], xbc[:, HP:HP + GN], xbc[:, HP + GN:], du[:, :L].reshape(n * L, H).contiguous(), dA, cu, y,
                        D=dD, dt_bias=ddt, state_in=state, state_out=state, workspace=ws)
    r1 = torch.empty(n * L, dim, device="cuda")
    gdn.gdn_block_norm(dres[:, :L].reshape(n * L, dim).contiguous(), block=y, res_out=r1, w_post=dwp)
    sx, su, sr = (torch.empty(n, k, dtype=t, device="cuda") for k, t in ((CH, dt), (H, dt), (dim, torch.float32)))
    sy = torch.empty(n, HP, dtype=dt, device="cuda")

    def token():
        gdn.gdn_ssm_decode(cfg, sx, su, dw, hist, dA, state, sy, ws, conv_bias=dbias, D=dD, dt_bias=ddt)
        gdn.gdn_block_norm(sr, block=sy, res_out=sr, w_post=dwp)

    ys, rs = [], []
    graph = None
    for k in range(steps):
        sx.copy_(draw[:, L + k]); su.copy_(du[:, L + k]); sr.copy_(dres[:, L + k])
        if k == 0:
            token()
        else:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    token()
            graph.replay()
        ys.append(sy.clone()); rs.append(sr.clone())
    torch.cuda.synchronize()
    assert gdn.gdn_device_error() == 0
    for i in range(n):
        c, cm, new = ref.conv(raw[i], w, bias, torch.zeros(CH, 3))
        assert torch.equal(hist[i].cpu().double(), new)
        T = L + steps
        pick = lambda t: (t[:, :HP].reshape(T, H, P), t[:, HP:HP + GN].reshape(T, G, N), t[:, HP + GN:].reshape(T, G, N))  # noqa: E731
        val, _, S, _ = ref.scan(*pick(c), u[i], A_log, D, dt_bias, None, torch.zeros(H, N, P), G)
        _, mag, _, M = ref.scan(*pick(cm), u[i], A_log, D.abs(), dt_bias, None, torch.zeros(H, N, P), G)
        # what the convolution writes is rounded to the activations' type: three factors of it
        h = ref.HALF[dt]
        rel = 3 * h + (2 * h if act == "bf16" else 0) + (8 * T + N + 64) * ref.U32 + (2 * 128 * 60 * ref.U32 if act == "bf16" else 0)
        got = torch.cat([y[i * L:(i + 1) * L]] + [t[i:i + 1] for t in ys])
        ref.check(got, val.reshape(T, -1), mag.reshape(T, -1), rel, "y")
        ref.check(state[i], S, M, 3 * h + (8 * T + N + 64) * ref.U32, "state")
        # the residual stream from the y that the norm was given
        out = ref.norm(got.cpu(), None, res[i], w_post, None, 1e-6, 0.0, 1.0)["res_out"]
        ref.check(torch.cat([r1[i * L:(i + 1) * L]] + [t[i:i + 1] for t in rs]), *out, (dim + 32) * ref.U32, "residual")


def test_lost_copy_runs_out_then_recovers():
    """A tile that never arrives: the call returns by itself, reports the timeout and stores no state;
    the next call is right.  (Nothing faults or hangs: every wait has the 20 ms limit set here.)"""
    b = Batch([300, 40], H=2, G=1, N=128, P=64, seed=17).upload()
    y = torch.empty(340, 128, dtype=b.act, device="cuda")
    out = torch.full_like(b.d_state, 7.0)
    assert gdn.gdn_device_error() == 0
    gdn.gdn_debug_set_wait(20_000_000, 4)
    try:
        b.launch(y, out)
        code = gdn.gdn_device_error()
    finally:
        gdn.gdn_debug_set_wait()
    assert code & gdn.DEVERR_TIMEOUT
    assert (out == 7).all()
    b.launch(y, out)
    assert gdn.gdn_device_error() == 0
    b.verify(y, out)


@pytest.mark.parametrize("act", ["fp32", "bf16"])
def test_many_sequences_some_cut(act):
    """More sequences than a warp lays out by itself, long ones among them."""
    lens = [3, 0, 17] * 13 + [600, 1, 0, 1100, 256, 257]
    b = Batch(lens, H=2, G=1, N=64, P=64, act=act, seed=18)
    b.verify(*b.run())
    assert gdn.gdn_device_error() == 0


@pytest.mark.parametrize("act,heads", [("bf16", 64), ("fp32", 32)])
def test_offsets_past_32_bits(act, heads):
    """Rows behind 2^31 elements: the last sequences of a long batch are right."""
    H, G, N, P = heads, 1, 64, 128
    dt = torch.bfloat16 if act == "bf16" else torch.float32
    first = (1 << 31) // (H * P) + 1000
    lens = [first, 90, 1]
    T = sum(lens)
    gen = torch.Generator(device="cuda").manual_seed(50)
    x = torch.empty(T, H * P, dtype=dt, device="cuda").normal_(generator=gen)
    bc = torch.empty(T, 2 * G * N, dtype=dt, device="cuda").normal_(generator=gen)
    u = torch.empty(T, H, dtype=dt, device="cuda").normal_(generator=gen)
    A_log, D = torch.rand(H, generator=gen, device="cuda"), torch.ones(H, device="cuda")
    cu = torch.tensor([0] + lens, dtype=torch.int64).cumsum(0).to(torch.int32).cuda()
    cfg = gdn.make_ssm_config(G, H, N, P, act=act, n_slots=3)
    y, out = torch.empty_like(x), torch.empty(3, H, N, P, device="cuda")
    ws = torch.empty(gdn.gdn_ssm_workspace_size(cfg, T, 3), dtype=torch.uint8, device="cuda")
    gdn.gdn_ssm_prefill(cfg, x, bc[:, :G * N], bc[:, G * N:], u, A_log, cu, y, D=D, state_out=out, workspace=ws)
    h = heads // 2                                              # one head in the middle
    for n in (1, 2):
        s, e = int(cu[n]), int(cu[n + 1])
        L = e - s
        val, mag, S, M = ref.scan(x[s:e].view(L, H, P)[:, h:h + 1].cpu(), bc[s:e, :G * N].reshape(L, G, N).cpu(),
                                  bc[s:e, G * N:].reshape(L, G, N).cpu(), u[s:e, h:h + 1].cpu(), A_log[h:h + 1].cpu(), D[h:h + 1].cpu(),
                                  None, None, torch.zeros(1, N, P), 1)
        rel = (8 * L + N + 64) * ref.U32
        rel_y = rel + (2 * 2.0 ** -8 + 2 * 128 * 60 * ref.U32 if act == "bf16" else 0)
        ref.check(y[s:e].view(L, H, P)[:, h], val[:, 0], mag[:, 0], rel_y, "y")
        ref.check(out[n, h], S[0], M[0], rel, "state")
    conv = gdn.make_ssm_config(1, H, 16, P, act=act, n_slots=3)
    CH = H * P + 32
    del y, bc
    xc = torch.empty(T, CH, dtype=dt, device="cuda")
    xc[:, :H * P] = x
    xc[:, H * P:].normal_(generator=gen)
    del x
    w, hist = torch.empty(CH, 4, dtype=dt, device="cuda").normal_(generator=gen), torch.zeros(3, CH, 3, dtype=dt, device="cuda")
    oc = torch.empty_like(xc)
    gdn.gdn_ssm_conv_prefill(conv, xc, cu, w, None, hist, None, oc)
    for n in (1, 2):
        s, e = int(cu[n]), int(cu[n + 1])
        val, mag, new = ref.conv(xc[s:e].cpu(), w.cpu(), None, torch.zeros(CH, 3))
        ref.check(oc[s:e], val, mag, CONV_REL, "conv")
        assert torch.equal(hist[n].cpu().double(), new)
    assert gdn.gdn_device_error() == 0


@pytest.mark.parametrize("act", ["fp32", "bf16"])
@pytest.mark.parametrize("fill", [float("nan"), INF])
@pytest.mark.parametrize("what", ["x", "b", "c", "dt"])
def test_not_finite_stays_behind_its_token(act, fill, what):
    """One value that is not finite: tokens in front of it, and the columns, heads and groups that do
    not see it, are right; what it reaches is not finite either."""
    b = Batch([600, 90], H=4, G=2, N=64, P=64, act=act, seed=19)
    at = 341                                       # inside a chunk, of a segment with others on both sides
    x, bb, c = b.parts(b.xbc)
    {"x": x, "b": bb, "c": c, "dt": b.u}[what][at, 1] = fill
    y, out = b.run()
    for n in (0, 1):
        s, e = int(b.cu[n]), int(b.cu[n + 1])
        val, mag, S, M = b.reference(n)
        L = e - s
        rel = (8 * L + b.N + 64) * ref.U32
        rel_y = rel + (2 * 2.0 ** -8 + 2 * 128 * 60 * ref.U32 if act == "bf16" else 0)
        for got, v, m, r, name in ((y[s:e].cpu(), val.reshape(L, -1), mag.reshape(L, -1), rel_y, "y"), (out[n].cpu(), S, M, rel, "state")):
            ok = v.isfinite()
            assert n == 1 or not ok.all() or what == "c"
            assert not got[~ok].isfinite().any()
            ref.check(got[ok], v[ok], m[ok], r, name)
    assert gdn.gdn_device_error() == 0


@pytest.mark.parametrize("act", ["fp32", "bf16"])
def test_conv_and_step_on_another_stream_and_in_a_graph(act):
    b = Batch([37, 0, 5], act=act, seed=20).upload()
    CH, n = b.xbc.shape[1], 3
    g = torch.Generator().manual_seed(21)
    w, hist = randn(CH, 4, gen=g, dtype=b.act).cuda(), randn(3, CH, 3, gen=g, dtype=b.act).cuda()
    ws = torch.empty(gdn.gdn_ssm_workspace_size(b.cfg, n, n), dtype=torch.uint8, device="cuda")

    def run(h, state, out, y, stream=None):
        gdn.gdn_ssm_conv_prefill(b.cfg, b.d_xbc, b.d_cu, w, None, h, None, out, stream=stream)
        gdn.gdn_ssm_decode(b.cfg, b.d_xbc[:n], b.d_u[:n], w, h, b.d_A_log, state, y, ws, D=b.d_D, stream=stream)

    def fresh():
        return (hist.clone(), b.d_state.clone(), torch.empty_like(b.d_xbc),
                torch.empty(n, b.H * b.P, dtype=b.act, device="cuda"))

    want = fresh()
    run(*want)
    other, s = fresh(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    run(*other, stream=s)
    s.synchronize()
    captured, graph = fresh(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(*captured)
    assert torch.equal(captured[0], hist)          # capturing ran nothing
    graph.replay()
    torch.cuda.synchronize()
    for i in range(4):
        assert torch.equal(want[i], other[i]) and torch.equal(want[i], captured[i])


def test_binding_refuses_tensors_that_do_not_fit():
    b = Batch([40], H=2, G=1, seed=22).upload()
    y = torch.empty(40, 128, dtype=b.act, device="cuda")
    good = dict(y=y, out=b.d_state)
    b.launch(**good)
    for k, bad in (("d_xbc", b.d_xbc.float()), ("d_xbc", b.d_xbc[:, :-64]), ("d_u", b.d_u[:-1]), ("d_u", b.u),
                   ("d_A_log", b.d_A_log.double()), ("d_cu", b.d_cu.long()), ("d_z", b.d_z.T), ("d_D", b.d_D[:1])):
        kept = getattr(b, k)
        setattr(b, k, bad)
        with pytest.raises(ValueError):
            b.launch(**good)
        setattr(b, k, kept)
    for bad in (dict(good, y=y[:, ::2]), dict(good, y=y.expand(40, 128).T), dict(good, out=b.d_state[:0]), dict(good, state=b.state)):
        with pytest.raises(ValueError):
            b.launch(**bad)
    b.ws = b.ws[:0]
    b.launch(**good)                               # (not cut: no workspace is needed)


@pytest.mark.parametrize("act,long", [("fp32", 600), ("bf16", 600), ("bf16", 9000)])
def test_more_sequences_than_a_block_lays_out(act, long):
    """More than 1,024 of them, few tokens each but for some that are cut: in order, none left out."""
    lens = [1, 0, 2, 1] * 330
    for n in (3, 700, 1023, 1100, 1318):
        lens[n] = 300
    lens[1024] = long
    b = Batch(lens, H=2, G=1, N=64, P=64, act=act, seed=23)
    picked = [0, 1, 2, 3, 4, 699, 700, 701, 1022, 1023, 1024, 1025, 1100, 1317, 1318, 1319]
    y, out = b.run()
    b.verify(y, out, seqs=picked + list(range(30, 1000, 61)))
    assert y.isfinite().all() and not (y == 7).all(1).any()
    assert gdn.gdn_device_error() == 0


@pytest.mark.parametrize("lens", [[8] * 40, [33], [32], [9] * 40, [1] * 64])
def test_short_sequences_of_either_form(lens):
    b = Batch(lens, H=4, G=2, N=128, P=64, act="bf16", seed=24)
    b.verify(*b.run())


@pytest.mark.parametrize("act", ["fp32", "bf16"])
def test_outputs_and_states_on_16_bytes(act):
    b = Batch([300, 40], H=2, G=1, act=act, seed=25).upload()
    step = 16 // torch.empty(0, dtype=b.act).element_size()
    y = torch.full((b.T * 128 + 2 * step,), 7.0, dtype=b.act, device="cuda")
    out = torch.full((b.d_state.numel() + 8,), 7.0, device="cuda")
    b.launch(y[step:-step].view(b.T, 128), out[4:-4].view_as(b.d_state))
    b.verify(y[step:-step].view(b.T, 128), out[4:-4].view_as(b.d_state))
    for edge in (y[:step], y[-step:], out[:4], out[-4:]):
        assert (edge == 7).all()


def test_as_many_sequences_as_are_allowed():
    n, lens = 65535, [1] * 65534 + [900]
    b = Batch(lens, H=1, G=1, N=16, P=32, act="fp32", seed=26)
    y, out = b.run()
    seqs = [0, 1, 31, 32, 1023, 1024, 33333, 65533, 65534]
    b.verify(y, out, seqs=seqs)
    assert not (y == 7).all(1).any()
    # the next token of each
    g = torch.Generator().manual_seed(27)
    x, w, u = randn(n, 64, gen=g), randn(64, 4, gen=g), randn(n, 1, gen=g)
    hist, state, ys = torch.zeros(n, 64, 3, device="cuda"), out.clone(), torch.empty(n, 32, device="cuda")
    ws = torch.empty(gdn.gdn_ssm_workspace_size(b.cfg, n, n), dtype=torch.uint8, device="cuda")
    gdn.gdn_ssm_decode(b.cfg, x.cuda(), u.cuda(), w.cuda(), hist, b.d_A_log, state, ys, ws)
    for s in seqs:
        c, cm, new = ref.conv(x[s:s + 1], w, None, torch.zeros(64, 3))
        val, mag, S, M = ref.scan(c[:, :32].view(1, 1, 32), c[:, 32:48].view(1, 1, 16), c[:, 48:].view(1, 1, 16), u[s:s + 1], b.A_log, None,
                                  None, None, out[s].cpu(), 1)
        # the convolution's 32-bit error enters each factor once: 24 roundings a value, three factors
        grow = 1 + (cm / c.abs()).max()
        ref.check(ys[s], val[0, 0], mag[0, 0], 128 * grow * ref.U32, "y")
        ref.check(state[s], S, M, 128 * grow * ref.U32, "state")
        assert torch.equal(hist[s].cpu().double(), new)
    assert gdn.gdn_device_error() == 0
