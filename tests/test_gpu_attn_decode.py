"""Attention of new tokens over a paged cache on the GPU against the 64-bit form: types, head layouts, page sizes, lengths
from none to several tiles, masks, what masked places may hold, splits, streams, graphs."""
import math

import pytest
import torch

import attn_ref as ref
from gateddeltanet_linear_attention_gb300 import gdn

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


class Cache:
    """Sequences of given lengths in shuffled pages; everything that no sequence holds is NaN."""

    def __init__(self, lens, Hq, Hkv, D, page, act="bf16", tokens=1, seed=0, spare=3, columns=0, std=1.5):
        self.lens, self.Hq, self.Hkv, self.D, self.page, self.act, self.tokens = lens, Hq, Hkv, D, page, DT[act], tokens
        g = torch.Generator().manual_seed(seed)
        held = [-(-v // page) for v in lens]
        self.n_pages = sum(held) + spare
        mp = max(max(held + [0]), columns, 1)
        order = torch.randperm(self.n_pages, generator=g).int()
        self.table = torch.full((len(lens), mp), 1 << 30, dtype=torch.int32)
        self.kp, self.vp = (torch.full((self.n_pages, Hkv, page, D), math.nan, dtype=self.act) for _ in range(2))
        self.K, self.V, at = [], [], 0
        for r, (length, n) in enumerate(zip(lens, held)):
            self.table[r, :n] = order[at:at + n]
            at += n
            for pool, keep in ((self.kp, self.K), (self.vp, self.V)):
                x = torch.randn(Hkv, length, D, generator=g).to(self.act)
                keep.append(x)
                for i in range(n):
                    part = x[:, i * page:(i + 1) * page]
                    pool[self.table[r, i], :, :part.shape[1]] = part
        self.q = (std * torch.randn(len(lens) * tokens, Hq, D, generator=g)).to(self.act)
        self.cfg = gdn.make_attn_config(Hq, Hkv, D, page_size=page, act=act, n_pages=self.n_pages, n_rows=len(lens), max_pages=mp)

    def upload(self):
        self.d = [t.cuda() for t in (self.q, self.kp, self.vp, self.table, torch.tensor(self.lens, dtype=torch.int32))]
        # a used workspace
        self.ws = torch.full((gdn.gdn_attn_workspace_size(self.cfg, len(self.lens), self.tokens),), 255, dtype=torch.uint8, device="cuda")
        return self

    def run(self, q=None, rows=None, lse=True, **kw):
        q = self.d[0] if q is None else q
        out = torch.full(q.shape, 9.0, dtype=self.act, device="cuda")
        lse = torch.full(q.shape[:2], 9.0, device="cuda") if lse else None
        gdn.gdn_attn_decode(self.cfg, q, *self.d[1:], out, self.ws, tokens=self.tokens, rows=rows, lse=lse, **kw)
        return out, lse

    def want(self, n, row=None, window=0, scale=None, seen=None, q=None):
        r = n if row is None else row
        k, L = self.tokens, self.lens[r]
        q = (self.q if q is None else q)[n * k:(n + 1) * k]
        return ref.attend(q, self.K[r], self.V[r], [L - k + 1 + j for j in range(k)], self.D ** -0.5 if scale is None else scale, window, seen)

    def check(self, out, lse, rows=None, window=0, scale=None, seqs=None):
        k = self.tokens
        for n in range(out.shape[0] // k) if seqs is None else seqs:
            row = n if rows is None else rows[n]
            o, s = out[n * k:(n + 1) * k].double().cpu(), lse[n * k:(n + 1) * k].double().cpu()
            if row < 0:
                assert not o.any() and (s == -math.inf).all()
                continue
            compare(o, s, self.want(n, row, window, scale), self.lens[row], self.D, self.act)


def compare(o, s, want, length, D, act):
    w, l, mag, top = want
    tol_o, tol_s = ref.attend_tolerance(w, mag, top, length, D, act)
    assert ((o - w).abs() <= tol_o).all(), "worst %.3g of its bound" % float(((o - w).abs() / tol_o.clamp(min=1e-300)).max())
    empty = l == -math.inf
    assert torch.equal(s == -math.inf, empty)
    assert ((s - l).abs()[~empty] <= ref.attend_lse_tolerance(l, tol_s)[~empty]).all()


LENS = [1, 0, 2, 17, 64, 65, 31, 200, 333]


@pytest.mark.parametrize("act", ["bf16", "fp32"])
@pytest.mark.parametrize("Hq,Hkv,D,page,tokens", [
    (1, 1, 64, 16, 1), (4, 4, 128, 64, 1), (8, 2, 128, 32, 1), (12, 3, 64, 128, 1), (16, 1, 256, 64, 1), (6, 2, 256, 16, 1), (8, 1, 128, 16, 2),
    (3, 1, 64, 64, 3), (16, 1, 128, 64, 8), (4, 2, 256, 128, 5), (10, 2, 64, 32, 7), (32, 2, 64, 64, 4)])
def test_layouts(act, Hq, Hkv, D, page, tokens):
    c = Cache(LENS, Hq, Hkv, D, page, act, tokens, seed=Hq + page).upload()
    out, lse = c.run()
    c.check(out, lse)
    assert gdn.gdn_device_error() == 0
    again, _ = c.run(lse=False)
    assert torch.equal(out, again)


@pytest.mark.parametrize("act", ["bf16", "fp32"])
@pytest.mark.parametrize("window,tokens", [(1, 1), (1, 4), (5, 3), (64, 1), (100, 8), (63, 2), (1000, 2)])
def test_windows(act, window, tokens):
    c = Cache(LENS + [400], 4, 2, 64, 16, act, tokens, seed=window).upload()
    out, lse = c.run(window=window)
    c.check(out, lse, window=window)
    # what lies in front of every window may be anything, missing pages too
    for r, length in enumerate(c.lens):
        first = max(0, length - tokens + 1 - window) // 16
        c.d[3][r, :first] = -7
    out2, lse2 = c.run(window=window)
    assert gdn.gdn_device_error() == 0
    assert torch.equal(out, out2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("act,Hq", [("bf16", 2), ("bf16", 8), ("fp32", 2)])
@pytest.mark.parametrize("window", [2**31 - 1, 2**31 - 7, 2**30])
def test_windows_without_end(act, Hq, window):
    """A window of any size that no length reaches changes nothing, in sequences shorter than the new tokens either."""
    c = Cache([0, 1, 3, 7, 8, 40, 130], Hq, 1, 64, 16, act, 8, seed=5).upload()
    out, lse = c.run(window=window)
    c.check(out, lse)
    plain, _ = c.run()
    assert torch.equal(out, plain)


@pytest.mark.parametrize("act", ["bf16", "fp32"])
def test_lengths_around_tiles(act):
    """Every length around the tiles' and pages' ends, in one batch."""
    lens = sorted({b + e for b in (16, 32, 64, 128, 192, 256) for e in (-2, -1, 0, 1, 2)})
    for tokens in (1, 4):
        c = Cache(lens, 2, 1, 64, 16, act, tokens, seed=tokens).upload()
        c.check(*c.run())


@pytest.mark.parametrize("act", ["bf16", "fp32"])
@pytest.mark.parametrize("n,Hkv", [(1, 1), (1, 2), (3, 1)])
def test_long_sequences_are_split(act, n, Hkv):
    """Few sequences: every one in parts of all CTAs."""
    lens = [9000, 33, 12345][:n]
    c = Cache(lens, 2 * Hkv, Hkv, 64, 64, act, 1, seed=n).upload()
    c.check(*c.run())


def test_many_sequences():
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 40, (2500,), generator=g).tolist()
    c = Cache(lens, 2, 1, 64, 16, "bf16", 1, seed=4).upload()
    out, lse = c.run()
    c.check(out, lse, seqs=list(range(0, 2500, 61)) + [2499])
    assert gdn.gdn_device_error() == 0


@pytest.mark.parametrize("act", ["bf16", "fp32"])
@pytest.mark.parametrize("scale", [1e-3, 1.0, 30.0])
def test_scales(act, scale):
    """Flat weights, and ones that single tokens win by far."""
    c = Cache([150, 70, 3], 4, 1, 64, 32, act, 2, seed=5).upload()
    c.check(*c.run(scale=scale), scale=scale)


def test_rows_and_padding_lanes():
    c = Cache([30, 100, 5, 0], 4, 2, 128, 32, "bf16", 2, seed=6).upload()
    rows = [2, -1, 1, 1, 3, 0, -9]
    g = torch.Generator().manual_seed(1)
    c.q = torch.randn(len(rows) * 2, 4, 128, generator=g).bfloat16()
    out, lse = c.run(q=c.q.cuda(), rows=torch.tensor(rows, dtype=torch.int32, device="cuda"))
    c.check(out, lse, rows=rows)
    assert gdn.gdn_device_error() == 0


def test_faults_are_reported():
    """A row beyond the table and a length beyond it are padding lanes; tokens of bad pages are masked."""
    c = Cache([30, 100, 50], 4, 2, 64, 16, "bf16", 2, seed=7).upload()
    good, good_lse = c.run()
    rows = torch.tensor([0, 3, 2], dtype=torch.int32, device="cuda")
    out, lse = c.run(rows=rows)
    assert gdn.gdn_device_error() == gdn.DEVERR_SLOT
    assert not out[2:4].any() and torch.equal(out[:2], good[:2]) and torch.equal(out[4:], good[4:]) and (lse[2:4] == -math.inf).all()
    c.d[4][1] = 16 * c.table.shape[1] + 1
    out, lse = c.run()
    assert gdn.gdn_device_error() == gdn.DEVERR_PAGE
    assert not out[2:4].any() and torch.equal(out[:2], good[:2]) and (lse[2:4] == -math.inf).all()
    c.d[4][1] = 100
    c.d[4][0] = -4
    assert not c.run()[0][:2].any() and gdn.gdn_device_error() == 0
    c.d[4][0] = 30
    for bad in (-1, c.n_pages, 1 << 30, -(1 << 31)):
        c.d[3][1, 2] = bad
        out, lse = c.run()
        assert gdn.gdn_device_error() == gdn.DEVERR_PAGE
        seen = [not 32 <= i < 48 for i in range(100)]
        compare(out[2:4].double().cpu(), lse[2:4].double().cpu(), c.want(1, seen=seen), 100, 64, c.act)
        assert torch.equal(out[:2], good[:2]) and torch.equal(out[4:], good[4:])
    c.d[3][1, :7] = -1                                          # nothing left to see
    out, lse = c.run()
    assert not out[2:4].any() and (lse[2:4] == -math.inf).all() and gdn.gdn_device_error() == gdn.DEVERR_PAGE


@pytest.mark.parametrize("act", ["bf16", "fp32"])
@pytest.mark.parametrize("pool", ["k", "v"])
@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan, 3e38])
def test_values_that_are_not_finite_stay_with_their_rows(act, pool, value):
    """The newest of four tokens holds such a value in key head 1: rows that see it show it, all others are as without it."""
    lens, tokens = [70, 20, 4, 130], 4
    c = Cache(lens, 4, 2, 64, 16, act, tokens, seed=8).upload()
    clean, clean_lse = c.run()
    for r, length in enumerate(lens):
        i = length - 1
        c.d[1 if pool == "k" else 2][c.table[r, i // 16], 1, i % 16, 5] = value
    out, lse = c.run()
    for r in range(len(lens)):
        for j in range(tokens):
            t = r * tokens + j
            assert torch.equal(out[t, :2], clean[t, :2])        # the other key head
            if j < tokens - 1:
                assert torch.equal(out[t], clean[t]) and torch.equal(lse[t], clean_lse[t])
            elif pool == "v" and not abs(value) < math.inf:
                assert not torch.isfinite(out[t, 2:, 5]).any() and torch.isfinite(out[t, 2:, :5]).all() and torch.equal(lse[t], clean_lse[t])
            elif pool == "k" and math.isnan(value):
                assert torch.isnan(out[t, 2:]).all() and torch.isnan(lse[t, 2:]).all()
    # outside a window: no row sees it
    c2 = Cache(lens, 4, 2, 64, 16, act, tokens, seed=8).upload()
    want, want_lse = c2.run(window=3)
    for r, length in enumerate(lens):
        i = length - 7
        if i >= 0:
            c2.d[1 if pool == "k" else 2][c2.table[r, i // 16], 1, i % 16, 5] = value
    out, lse = c2.run(window=3)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_scores_of_minus_infinity():
    """A key of -inf where the query is positive is masked by its own score; a row of such keys alone is empty."""
    c = Cache([20, 3], 1, 1, 64, 16, "fp32", 1, seed=9)
    c.q = c.q.abs() + 0.1
    c.K[0][0, 4] = c.kp[c.table[0, 0], 0, 4] = -math.inf
    c.K[1][0, :3] = c.kp[c.table[1, 0], 0, :3] = -math.inf
    c.upload()
    out, lse = c.run()
    seen = [i != 4 for i in range(20)]
    compare(out[:1].double().cpu(), lse[:1].double().cpu(), c.want(0, seen=seen), 20, 64, c.act)
    assert not out[1].any() and (lse[1] == -math.inf).all()


def test_query_views_and_refusals():
    c = Cache([40, 7, 90], 4, 2, 128, 16, "bf16", 2, seed=10).upload()
    want, _ = c.run()
    gated = torch.empty(6, 4, 2, 128, dtype=torch.bfloat16, device="cuda")
    gated[:, :, 0] = c.d[0]
    assert torch.equal(c.run(q=gated[:, :, 0])[0], want)
    assert torch.equal(c.run(q=c.d[0].transpose(0, 1).contiguous().transpose(0, 1))[0], want)
    with pytest.raises(ValueError):
        c.run(q=c.d[0].float())
    with pytest.raises(ValueError):
        c.run(q=c.d[0][:5])
    with pytest.raises(gdn.GDNError):
        c.run(scale=0.0)
    c.ws = c.ws[:1000]
    with pytest.raises(gdn.GDNError):
        c.run()


def test_offsets_beyond_32_bits():
    """Pages beyond 2^31 elements and 2^32 bytes of a pool."""
    Hkv, D, page = 8, 256, 128
    n_pages = (1 << 31) // (Hkv * D * page) + 40
    c = Cache([300, 129], 16, Hkv, D, page, "bf16", 1, seed=11)
    pools = [torch.empty(n_pages, Hkv, page, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for pool, small in zip(pools, (c.kp, c.vp)):
        pool[-c.n_pages:] = small.cuda()
        pool[:c.n_pages] = math.nan
    c.table[c.table < c.n_pages] += n_pages - c.n_pages
    c.cfg = gdn.make_attn_config(16, Hkv, D, page_size=page, n_pages=n_pages, n_rows=2, max_pages=c.table.shape[1])
    c.upload()
    c.d[1:3] = pools
    c.check(*c.run())
    # and the way there: the newest tokens are written once more
    qkv = torch.randn(2, (16 + 2 * Hkv) * D, device="cuda").bfloat16()
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([16 * D, Hkv * D, Hkv * D], 1))
    gdn.gdn_attn_prep(c.cfg, q, k, torch.empty(2, 16, D, dtype=torch.bfloat16, device="cuda"), None, v=v, k_pages=pools[0], v_pages=pools[1],
                      page_table=c.d[3], lens=c.d[4], tokens=1)
    for r, length in enumerate(c.lens):
        i = length - 1
        p = int(c.table[r, i // page])
        assert torch.equal(pools[0][p, :, i % page], k[r]) and torch.equal(pools[1][p, :, i % page], v[r])
    src = torch.tensor([n_pages - 1, 3], dtype=torch.int32, device="cuda")
    dst = torch.tensor([1, n_pages - 2], dtype=torch.int32, device="cuda")
    pools[0][3] = 4.0
    gdn.gdn_page_copy(c.cfg, *pools, *pools, src, dst)
    assert torch.equal(pools[0][1].nan_to_num(), pools[0][n_pages - 1].nan_to_num()) and (pools[0][n_pages - 2] == 4).all()
    assert gdn.gdn_device_error() == 0


def test_graph_replayed_with_other_lengths():
    """Lengths, tables and rows are read when the graph runs; two graphs share a workspace."""
    c = Cache([500, 90, 2000], 4, 1, 128, 64, "bf16", 1, seed=12).upload()
    out, lse = torch.zeros_like(c.d[0]), torch.zeros(3, 4, device="cuda")
    out2 = torch.zeros_like(c.d[0])
    gdn.gdn_attn_decode(c.cfg, *c.d, out, c.ws, lse=lse)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        gdn.gdn_attn_decode(c.cfg, *c.d, out, c.ws, lse=lse)
    with torch.cuda.graph(graphs[1]):
        gdn.gdn_attn_decode(c.cfg, *c.d, out2, c.ws, window=70)
    for lens in ([500, 90, 2000], [499, 0, 1], [64, 65, 1999]):
        c.d[4].copy_(torch.tensor(lens, dtype=torch.int32))
        keep, c.lens = c.lens, lens
        K, V = c.K, c.V
        c.K, c.V = [x[:, :n] for x, n in zip(K, lens)], [x[:, :n] for x, n in zip(V, lens)]
        for g in graphs + graphs:
            g.replay()
        torch.cuda.synchronize()
        c.check(out, lse)
        c.check(out2, c.run(window=70)[1], window=70)
        c.lens, c.K, c.V = keep, K, V


def test_other_stream():
    c = Cache([700, 9], 8, 2, 128, 64, "bf16", 1, seed=13).upload()
    want, want_lse = c.run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        out, lse = c.run()
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    out3 = torch.empty_like(want)
    gdn.gdn_attn_decode(c.cfg, *c.d, out3, c.ws, stream=side)
    side.synchronize()
    assert torch.equal(out3, want)


def test_calls_at_once():
    """Calls on two streams, each with a workspace of its own, while the other's kernels run."""
    pair = [Cache([900, 30, 2500, 0, 640], 8, 2, 128, 32, "bf16", tokens, seed=tokens).upload() for tokens in (8, 2)]
    want = [c.run()[0] for c in pair]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in pair], [[torch.empty_like(w) for _ in range(20)] for w in want]
    for i in range(20):
        for c, s, g in zip(pair, streams, got):
            gdn.gdn_attn_decode(c.cfg, *c.d, g[i], c.ws, tokens=c.tokens, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, w) for g, w in zip(got, want) for x in g)
    assert gdn.gdn_device_error() == 0


@pytest.mark.parametrize("D,tokens", [(64, 1), (128, 8), (256, 1)])
def test_a_lost_tile_times_out(D, tokens):
    """A copy that never comes: the call ends by itself within its limit, says so, and the next one is right."""
    c = Cache([3000, 40, 700], 8, 1, D, 16, "bf16", tokens, seed=14).upload()
    want, want_lse = c.run()
    torch.cuda.synchronize()
    gdn.gdn_debug_set_wait(20_000_000, 8)
    try:
        c.run()
        assert gdn.gdn_device_error() == gdn.DEVERR_TIMEOUT
    finally:
        gdn.gdn_debug_set_wait()
    out, lse = c.run()
    assert torch.equal(out, want) and torch.equal(lse, want_lse) and gdn.gdn_device_error() == 0


@pytest.mark.parametrize("Hq,Hkv,D,page,tokens", [(16, 2, 256, 128, 1), (4, 1, 256, 16, 8), (8, 1, 128, 64, 8), (6, 2, 128, 32, 3), (1, 1, 64, 64, 1),
                                                  (16, 1, 64, 128, 8)])
def test_every_layout_walks_its_ring(Hq, Hkv, D, page, tokens):
    """More tiles a CTA than it has places for, so that every place is filled again and again."""
    c = Cache([80000, 64, 60001], Hq, Hkv, D, page, "bf16", tokens, seed=15)
    c.upload()
    out, lse = c.run()
    k = tokens
    for n in range(3):
        for j in (0, k - 1):
            t = n * k + j
            L = c.lens[n] - k + 1 + j
            K, V = c.K[n][:, :L].double(), c.V[n][:, :L].double()
            q = c.q[t].double().view(Hkv, Hq // Hkv, D)
            s = torch.einsum("hgd,htd->hgt", q, K) * D ** -0.5
            top = (torch.einsum("hgd,htd->hgt", q.abs(), K.abs()) * D ** -0.5).amax(-1).view(1, Hq)
            p = torch.softmax(s, -1)
            want, mag = (torch.einsum("hgt,htd->hgd", p, x).reshape(1, Hq, D) for x in (V, V.abs()))
            compare(out[t:t + 1].double().cpu(), lse[t:t + 1].double().cpu(), (want, torch.logsumexp(s, -1).view(1, Hq), mag, top), L, D, c.act)
    assert gdn.gdn_device_error() == 0


@pytest.mark.parametrize("window", [0, 90])
@pytest.mark.parametrize("act,Hq,Hkv,D,tokens", [("bf16", 8, 1, 64, 8), ("bf16", 16, 1, 64, 8), ("bf16", 6, 2, 128, 7), ("bf16", 16, 1, 128, 8), ("bf16", 4, 1, 256, 8),
                                                 ("bf16", 16, 1, 256, 8), ("bf16", 16, 2, 256, 2), ("bf16", 4, 2, 64, 1), ("fp32", 6, 2, 64, 1),
                                                 ("fp32", 8, 1, 128, 3), ("fp32", 16, 1, 256, 8)])
def test_many_short_units(act, Hq, Hkv, D, tokens, window):
    """Every CTA has several units, of no to a few tiles, and some begin or end inside one."""
    g = torch.Generator().manual_seed(D + tokens)
    lens = torch.randint(0, 260, (600,), generator=g).tolist()
    lens[100], lens[101], lens[300] = 3000, 0, 1500
    c = Cache(lens, Hq, Hkv, D, 32, act, tokens, seed=16).upload()
    out, lse = c.run(window=window)
    c.check(out, lse, window=window, seqs=list(range(0, 600, 23)) + [99, 100, 101, 102, 299, 300, 301, 599])
    assert gdn.gdn_device_error() == 0
    again, _ = c.run(window=window)
    assert torch.equal(out, again)


@pytest.mark.parametrize("Hq,Hkv,D,page,tokens", [(16, 1, 256, 64, 8), (8, 1, 64, 16, 8), (16, 1, 128, 128, 8)])
def test_long_cache_of_many_rows(Hq, Hkv, D, page, tokens):
    """One long sequence of many query rows beside a short one, in more tiles a CTA than its rings hold."""
    c = Cache([150000, 5], Hq, Hkv, D, page, "bf16", tokens, seed=17).upload()
    out, lse = c.run()
    c.check(out, lse)
    assert gdn.gdn_device_error() == 0
