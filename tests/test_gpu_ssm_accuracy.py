"""Accuracy of the tensor-core scan's states, closer than the general bounds: x, B and C positive and
decays slow, so that a state is a sum without cancellation and its relative error is bounded term by
term.

In units of 2^-24, U: the step size 12 (softplus: 2 + 1 units in the last place, and the rounding of
u + dt_bias, up to 6 in size); the weight 5 (exponential 2 units in the last place, one product); w x 1; the
24 products of a chunk (8 steps of 16 tokens in 3 parts), each with one truncation of its 24-bit sum,
48; per chunk the decay's exponential and one multiply-add, 5, and the same per segment.  Without the
third part of w x the sums lose 7e-6 of their size (118 U; the test without a GPU shows it)."""
import pytest
import torch

import ssm_ref as ref
from test_gpu_ssm import Batch


def batch(lens, H, N, P, seed=60):
    b = Batch(lens, H=H, G=1, N=N, P=P, seed=seed, z=False, D=False, state=False, rate=(1e-3, 2e-3))
    b.xbc = b.xbc.abs()
    return b


def bound(L, segments=1):
    return (66 + 5 * ((L + 127) // 128) + 5 * segments) * ref.U32


def test_two_parts_are_outside_the_bound():
    """The mistake planted in the 64-bit form: w x in two parts of 8 bits, cut off, where three hold all 24."""
    b = batch([128, 384], 2, 64, 64)
    for n, L in enumerate(b.lens):
        s = int(b.cu[n])
        x, bb, _ = b.parts(b.xbc[s:s + L])
        dt = ref.step_size(b.u[s:s + L], b.dt_bias, 0.0, float("inf"))
        g = dt * torch.exp(b.A_log.double())
        w = dt * torch.exp(g.cumsum(0) - g.sum(0))                     # [L, H]: decay from behind each token
        v = (w.float()[:, :, None] * x.float().view(L, 2, 64))
        cut = lambda t: (t.view(torch.int32) & -65536).view(torch.float32)  # noqa: E731
        p0 = cut(v)
        p1 = cut(v - p0)
        assert torch.equal(p0 + p1 + cut(v - p0 - p1), v)              # three parts: every bit
        whole, two = (torch.einsum("ln,lhp->hnp", bb.double(), t.double()) for t in (v, p0.double() + p1.double()))
        loss = (whole - two) / whole
        assert loss.max() > 1.1 * bound(L, 2) and loss.mean() > bound(L, 2)


@pytest.mark.gpu
@pytest.mark.parametrize("N,P", [(64, 64), (128, 64), (64, 128), (128, 128)])
def test_states_of_few_chunks(N, P):
    """One chunk, three in two segments, odd lengths beside them."""
    b = batch([128, 384, 77, 300], 2, N, P)
    _, out = b.run()
    for n, L in enumerate(b.lens):
        _, _, S, _ = b.reference(n)
        worst = float(((out[n].cpu().double() - S).abs() / S).max())
        print("N %d P %d, %d tokens: %.1f U" % (N, P, L, worst / ref.U32))
        assert worst <= bound(L, 2)


@pytest.mark.gpu
def test_states_of_many_chunks_uncut():
    """20 chunks in turn (heads fill the GPU, so nothing is cut)."""
    H, N, P, L = 160, 64, 128, 2560
    b = batch([L], H, N, P)
    _, out = b.run()
    x, bb, c = b.parts(b.xbc)
    for h in (0, 77, 159):
        _, _, S, _ = ref.scan(x.view(L, H, P)[:, h:h + 1], bb.view(L, 1, N), c.view(L, 1, N), b.u[:, h:h + 1], b.A_log[h:h + 1], None,
                              b.dt_bias[h:h + 1], None, torch.zeros(1, N, P), 1)
        worst = float(((out[0, h].cpu().double() - S[0]).abs() / S[0]).max())
        print("head %d: %.1f U" % (h, worst / ref.U32))
        assert worst <= bound(L)


@pytest.mark.gpu
@pytest.mark.parametrize("length", [9, 16, 24])
def test_many_short_sequences_take_the_form_of_single_tokens(length):
    """More than ten rounds of CTAs of mostly empty chunks: the form of single tokens, whose outputs have
    one rounding to 16 bits and 32-bit errors beside it (8 a token in the recurrence, N in a sum)."""
    b = Batch([length] * 100, H=32, G=2, N=64, P=128, seed=61)
    y, out = b.run()
    for n in (0, 31, 32, 99):
        s, e = int(b.cu[n]), int(b.cu[n + 1])
        val, mag, S, M = b.reference(n)
        rel = (8 * length + b.N + 64) * ref.U32
        ref.check(y[s:e], val.reshape(length, -1), mag.reshape(length, -1), rel, "y of sequence %d" % n)
        ref.check(out[n], S, M, rel, "state of sequence %d" % n)


@pytest.mark.gpu
def test_a_long_sequence_among_single_tokens():
    """Either form, and a long sequence that is cut in it."""
    for count in (30, 99):
        lens = [1] * count + [1200]
        b = Batch(lens, H=32, G=2, N=64, P=128, seed=62)
        y, out = b.run()
        b.verify(y, out, seqs=[0, 17, count - 1, count])
