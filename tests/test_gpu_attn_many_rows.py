"""Attention of new tokens where a key head has 17 to 128 query rows: values that are not finite in places that only some of
the new tokens see, in many units one after another, so that every unit finds the marks of the one before; faults and keys of
-inf in that kernel."""
import math
import random

import pytest
import torch

from test_gpu_attn_decode import Cache, compare
from gateddeltanet_linear_attention_gb300 import gdn

pytestmark = pytest.mark.gpu

# query heads, key heads, columns, tokens of a page, new tokens
ONE_GROUP = [(4, 1, 256, 16, 8), (16, 1, 256, 64, 8), (16, 2, 256, 128, 3)]      # of warps takes all tiles of a unit
TWO_GROUPS = [(8, 1, 64, 16, 8), (6, 2, 128, 32, 7), (16, 1, 64, 64, 8), (16, 1, 128, 128, 8), (10, 1, 128, 16, 2), (8, 2, 64, 128, 5)]  # take turns


def spoil(c, pool, window, seed, share):
    """Puts values that are not finite where the newest token alone or only some see them, in `share` of the units; which outputs
    [T, Hq, D] and sums [T, Hq] then are not finite."""
    rng, k, G = random.Random(seed), c.tokens, c.Hq // c.Hkv
    out = torch.zeros(c.q.shape, dtype=torch.bool)
    kp, vp = c.kp.clone(), c.vp.clone()
    for r, length in enumerate(c.lens):
        for h in range(c.Hkv):
            # of the tokens that some see: the newest ones, or those that the window leaves behind
            edge = rng.randrange(length - k + 1, length) if not window or rng.random() < 0.5 else rng.randrange(length - k + 1 - window, length - window)
            if rng.random() >= share or edge < 0:
                continue
            col, at = rng.randrange(c.D), (c.table[r, edge // c.page], h, edge % c.page)
            (kp if pool == "k" else vp)[at][col] = math.nan if pool == "k" else rng.choice([math.inf, -math.inf, math.nan])
            for j in range(k):
                end = length - k + 1 + j
                if edge < end and (not window or edge >= end - window):
                    out[r * k + j, h * G:(h + 1) * G, slice(None) if pool == "k" else col] = True
    c.d[1].copy_(kp)
    c.d[2].copy_(vp)
    return out.cuda()


def check(layout, pool, window, lens, share=0.6, turns=20):
    Hq, Hkv, D, page, tokens = layout
    assert 16 < Hq // Hkv * tokens <= 128
    c = Cache(lens, Hq, Hkv, D, page, "bf16", tokens, seed=D + tokens).upload()
    clean, clean_lse = c.run(window=window)
    assert torch.isfinite(clean).all()
    for turn in range(turns):
        bad = spoil(c, pool, window, turn, share) if turn % 5 == 0 else bad
        out, lse = c.run(window=window)
        assert torch.equal(torch.isfinite(out), ~bad)
        assert torch.equal(torch.where(bad, 0, out), torch.where(bad, 0, clean))
        if pool == "k":
            assert torch.equal(torch.isnan(lse), bad.any(-1))
            lse = torch.where(bad.any(-1), clean_lse, lse)
        assert torch.equal(lse, clean_lse)
    assert gdn.gdn_device_error() == 0


@pytest.mark.parametrize("pool", ["v", "k"])
@pytest.mark.parametrize("window", [0, 40])
@pytest.mark.parametrize("layout", ONE_GROUP + TWO_GROUPS)
def test_values_that_are_not_finite_in_unit_after_unit(layout, window, pool):
    """Units of one to a few tiles, several a CTA, most of them with such a value: the marks are set and cleared all the time."""
    g = torch.Generator().manual_seed(1)
    check(layout, pool, window, torch.randint(0, 200, (400,), generator=g).tolist())


@pytest.mark.parametrize("layout", ONE_GROUP + TWO_GROUPS)
def test_values_that_are_not_finite_in_parts(layout):
    """Units that several CTAs hold: the marks are those of the last tiles' CTA, and reach the sums through the join."""
    check(layout, "v", 0, [30000, 70, 64, 9001, 3, 12345], share=1.0, turns=6)


@pytest.mark.parametrize("layout", TWO_GROUPS)
@pytest.mark.parametrize("length", [60, 128])
def test_marks_of_one_unit_stay_out_of_the_next(layout, length):
    """Every second unit has such a value, all of one or two tiles: one group marks in a unit while the other writes the outputs
    of the unit before."""
    check(layout, "v", 0, [length - i % 2 * (i % 7) for i in range(2000)], share=0.5, turns=40)


LAYOUTS = [(8, 1, 64, 16, 8), (16, 1, 128, 16, 8), (4, 1, 256, 16, 8), (16, 1, 256, 16, 8)]


@pytest.mark.parametrize("Hq,Hkv,D,page,tokens", LAYOUTS)
def test_faults_are_reported(Hq, Hkv, D, page, tokens):
    """A row beyond the table and a length beyond it are padding lanes; tokens of bad pages are masked, whole tiles of them too."""
    k = tokens
    c = Cache([30, 250, 50], Hq, Hkv, D, page, "bf16", k, seed=7).upload()
    good, good_lse = c.run()
    out, lse = c.run(rows=torch.tensor([0, 3, 2], dtype=torch.int32, device="cuda"))
    assert gdn.gdn_device_error() == gdn.DEVERR_SLOT
    assert not out[k:2 * k].any() and torch.equal(out[:k], good[:k]) and torch.equal(out[2 * k:], good[2 * k:])
    assert (lse[k:2 * k] == -math.inf).all()
    c.d[4][1] = page * c.table.shape[1] + 1
    out, lse = c.run()
    assert gdn.gdn_device_error() == gdn.DEVERR_PAGE
    assert not out[k:2 * k].any() and torch.equal(out[:k], good[:k]) and (lse[k:2 * k] == -math.inf).all()
    c.d[4][1] = 250
    table = c.d[3].clone()
    # one page inside a tile; the first tile; the last pages, the newest tokens among them; all
    for bad, first, last in ((-1, 2, 3), (c.n_pages, 0, 4), (1 << 30, 13, 16), (-(1 << 31), 0, 16)):
        c.d[3].copy_(table)
        c.d[3][1, first:last] = bad
        out, lse = c.run()
        assert gdn.gdn_device_error() == gdn.DEVERR_PAGE
        compare(out[k:2 * k].double().cpu(), lse[k:2 * k].double().cpu(), c.want(1, seen=[not first * page <= i < last * page for i in range(250)]), 250, D,
                c.act)
        assert torch.equal(out[:k], good[:k]) and torch.equal(out[2 * k:], good[2 * k:]) and torch.equal(lse[:k], good_lse[:k])


@pytest.mark.parametrize("Hq,Hkv,D,page,tokens", LAYOUTS + [(2, 1, 64, 16, 2), (4, 1, 256, 16, 1)])
def test_scores_of_minus_infinity(Hq, Hkv, D, page, tokens):
    """Keys of -inf where the query is positive are masked by their own score, a first tile of them too; a row of them alone is
    empty."""
    k = tokens
    c = Cache([200, 40, 300], Hq, Hkv, D, page, "bf16", k, seed=9)
    c.q = c.q.abs() + 0.1
    gone = [[i < 70 or i == 150 for i in range(200)], [True] * 40, [i % 3 > 0 or i > 200 for i in range(300)]]
    for r, which in enumerate(gone):
        for i, x in enumerate(which):
            if x:
                c.K[r][:, i] = c.kp[c.table[r, i // page], :, i % page] = -math.inf
    c.upload()
    out, lse = c.run()
    for r, which in enumerate(gone):
        compare(out[r * k:(r + 1) * k].double().cpu(), lse[r * k:(r + 1) * k].double().cpu(), c.want(r, seen=[not x for x in which]), len(which), D, c.act)
    assert not out[k:2 * k].any() and (lse[k:2 * k] == -math.inf).all() and gdn.gdn_device_error() == 0


@pytest.mark.parametrize("act,Hq,Hkv,D,tokens", [("bf16", 4, 2, 64, 1), ("bf16", 4, 2, 128, 4), ("bf16", 4, 2, 256, 1)] + [("bf16", 16, 2, D, 8) for D in (64, 128, 256)] +
                         [("fp32", 4, 2, 64, 1), ("fp32", 16, 2, 128, 8)])
@pytest.mark.parametrize("value", [math.inf, -math.inf])
@pytest.mark.parametrize("length", [300, 5000])
def test_infinite_values_that_all_rows_see(act, Hq, Hkv, D, tokens, value, length):
    """The column of the value is not finite in the rows of its key head, and infinite in fp32; nothing else changes."""
    c = Cache([length, 90], Hq, Hkv, D, 16, act, tokens, seed=3).upload()
    clean, clean_lse = c.run()
    c.d[2][c.table[0, 2], 1, 7, 11] = value
    out, lse = c.run()
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[:tokens, Hq // 2:, 11] = True
    assert torch.equal(torch.isfinite(out), ~bad) and torch.equal(torch.where(bad, 0, out), torch.where(bad, 0, clean)) and torch.equal(lse, clean_lse)
    if act == "fp32":
        assert (out[bad] == value).all()
    assert gdn.gdn_device_error() == 0
