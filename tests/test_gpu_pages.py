"""The cache's pages on the GPU against the rules on lists, the copies bit for bit, and a serving run of all operators of
the attention layers together."""
import random

import pytest
import torch

import attn_ref as ref
from gateddeltanet_linear_attention_gb300 import gdn

pytestmark = pytest.mark.gpu


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


class Device:
    """The pages on the device beside the model."""

    def __init__(self, n_pages, n_rows, max_pages, page=16, lanes=64):
        self.m = ref.Pages(n_pages, n_rows, max_pages, page)
        self.cfg = gdn.make_attn_config(2, 1, 64, page_size=page, n_pages=n_pages, n_rows=n_rows, max_pages=max_pages)
        self.table, self.lens, self.refs = ints(self.m.table), ints(self.m.lens), ints(self.m.refs)
        self.ws = torch.full((gdn.gdn_page_workspace_size(self.cfg, lanes),), 255, dtype=torch.uint8, device="cuda")

    def same(self):
        assert self.lens.tolist() == self.m.lens
        assert self.refs.tolist() == self.m.refs
        assert self.table.tolist() == self.m.table

    def resize(self, rows, new):
        n = len(rows)
        granted, src, dst = (torch.full((n,), 77, dtype=torch.int32, device="cuda") for _ in range(3))
        gdn.gdn_page_resize(self.cfg, self.table, self.lens, self.refs, ints(rows), ints(new), granted, src, dst, self.ws)
        want = self.m.resize(rows, new)
        assert (granted.tolist(), src.tolist(), dst.tolist()) == want[:3]
        assert gdn.gdn_device_error() == want[3]
        self.same()
        return src, dst

    def fork(self, src, dst):
        gdn.gdn_page_fork(self.cfg, self.table, self.lens, self.refs, ints(src), ints(dst))
        assert gdn.gdn_device_error() == self.m.fork(src, dst)
        self.same()

    def compact(self, n, in_place):
        src, dst = (torch.full((n,), 77, dtype=torch.int32, device="cuda") for _ in range(2))
        table, refs = (self.table, self.refs) if in_place else (torch.zeros_like(self.table), torch.zeros_like(self.refs))
        gdn.gdn_page_compact(self.cfg, self.table, self.lens, self.refs, table, refs, src, dst, self.ws)
        assert (src.tolist(), dst.tolist()) == self.m.compact(n)
        self.table, self.refs = table, refs
        self.same()
        assert gdn.gdn_device_error() == 0
        return src, dst


def test_worked_example():
    d = Device(6, 3, 4)
    d.resize([0], [20])
    d.fork([0, 0], [1, 2])
    d.resize([1, 2], [21, 33])
    d.resize([0, 1, 2], [49, 22, 34])
    d.resize([1, 1, 5], [0, 0, 0])
    d.resize([0, 1], [0, 3])
    d.resize([1], [5])
    d.compact(3, True)
    d.m.check()


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("n_pages,n_rows,max_pages,page", [(40, 9, 12, 16), (3000, 70, 64, 64), (5, 4, 3, 128)])
def test_runs(seed, n_pages, n_rows, max_pages, page):
    """Random runs: growth, truncation, frees, forks, exhaustion, inactive lanes, rows named twice or out of range."""
    rng = random.Random(seed * 1000 + n_pages)
    d = Device(n_pages, n_rows, max_pages, page, lanes=max(n_rows + 5, n_pages))
    for step in range(25):
        kind = rng.random()
        if kind < 0.6:
            rows = rng.sample(range(n_rows), rng.randint(1, n_rows))
            if rng.random() < 0.3:
                rows += [rng.choice([-1, n_rows, rows[0], n_rows + 7]) for _ in range(rng.randint(1, 4))]
                rng.shuffle(rows)
            new = []
            for r in rows:
                old = d.m.lens[r] if 0 <= r < n_rows else 0
                new.append(rng.choice([old, old + 1, old + 1, old + rng.randint(0, 3 * page), max(0, old - rng.randint(0, 2 * page)), 0,
                                       rng.randint(0, max_pages * page), -1, max_pages * page + rng.randint(0, 1)]))
            d.resize(rows, new)
        elif kind < 0.85:
            live = [r for r in range(n_rows) if d.m.lens[r]] or [0]
            empty = [r for r in range(n_rows) if not d.m.lens[r]]
            dst = rng.sample(empty, rng.randint(0, len(empty)))
            src = [rng.choice(live) for _ in dst]
            if rng.random() < 0.4:
                dst += [rng.choice([-1, n_rows, rng.randrange(n_rows)]) for _ in range(3)]
                src += [rng.choice([-1, n_rows, rng.randrange(n_rows)]) for _ in range(3)]
            if dst:
                d.fork(src, dst)
        else:
            d.compact(rng.choice([0, 1, 3, n_pages]), rng.random() < 0.5)
        d.m.check()


def test_many_lanes_and_pages():
    """More lanes than a cluster's warps, more pages than its threads take at once, and a pool that runs out in the middle."""
    d = Device(100_000, 4000, 40, 16, lanes=100_000)
    rng = random.Random(5)
    rows = list(range(4000))
    rng.shuffle(rows)
    d.resize(rows, [rng.randint(0, 640) for _ in rows])
    d.resize(rows, [rng.randint(0, 640) for _ in rows])
    empty = [r for r in range(4000) if d.m.lens[r] == 0]
    d.resize(rows[:500], [0] * 500)
    d.fork([rows[500 + i % 100] for i in range(500)], rows[:500])
    d.resize(rows[:500], [d.m.lens[r] + 1 if d.m.lens[r] < 640 else 640 for r in rows[:500]])
    d.compact(100_000, False)
    d.m.check()
    assert len(empty) >= 0


@pytest.mark.parametrize("act,Hkv,D,page", [("bf16", 1, 64, 16), ("bf16", 3, 128, 64), ("fp32", 2, 256, 32), ("bf16", 8, 128, 128)])
def test_copies(act, Hkv, D, page):
    dt = torch.bfloat16 if act == "bf16" else torch.float32
    cfg = gdn.make_attn_config(Hkv, Hkv, D, page_size=page, act=act)
    g = torch.Generator(device="cuda").manual_seed(0)
    a = [torch.randn(9, Hkv, page, D, generator=g, device="cuda").to(dt) for _ in range(2)]
    b = [torch.randn(12, Hkv, page, D, generator=g, device="cuda").to(dt) for _ in range(2)]
    src, dst = [3, -1, 8, 0, 9, 2, 3], [5, 0, 11, -1, 1, 12, 6]
    keep = [t.clone() for t in b]
    gdn.gdn_page_copy(cfg, *a, *b, ints(src), ints(dst))
    assert gdn.gdn_device_error() == gdn.DEVERR_PAGE                 # 9 -> 1 and 2 -> 12 are skipped
    for x, y, k in zip(a, b, keep):
        k[5], k[11], k[6], k[0] = x[3], x[8], x[3], 0
        assert torch.equal(y.view(torch.uint8), k.view(torch.uint8))
    # one pool alone, within itself, NaN payloads and all
    raw = torch.randint(0, 256, a[0].view(torch.uint8).shape, dtype=torch.uint8, device="cuda", generator=g)
    a[0].view(torch.uint8).copy_(raw)
    gdn.gdn_page_copy(cfg, a[0], None, a[0], None, ints([0, 1]), ints([7, 8]))
    want = raw.clone()
    want[7], want[8] = raw[0], raw[1]
    assert torch.equal(a[0].view(torch.uint8), want)
    v = a[1].clone()
    gdn.gdn_page_copy(cfg, None, None, None, a[1], ints([4]), ints([2]))
    v[2] = 0
    assert torch.equal(a[1], v) and gdn.gdn_device_error() == 0
    gdn.gdn_page_copy(cfg, *a, *a, ints([]), ints([]))


def test_refusals():
    d = Device(8, 4, 4)
    lane = ints([0])
    with pytest.raises(ValueError):
        gdn.gdn_page_resize(d.cfg, d.table[:, :3], d.lens, d.refs, lane, lane, lane, lane, lane, d.ws)
    with pytest.raises(ValueError):
        gdn.gdn_page_resize(d.cfg, d.table, d.lens, d.refs, lane, ints([1, 2]), lane, lane, lane, d.ws)
    with pytest.raises(ValueError):
        gdn.gdn_page_fork(d.cfg, d.table, d.lens.long(), d.refs, lane, lane)
    with pytest.raises(gdn.GDNError):
        gdn.gdn_page_resize(d.cfg, d.table, d.lens, d.refs, lane, lane, lane, lane, lane, d.ws[:16])
    with pytest.raises(ValueError):
        gdn.gdn_page_copy(d.cfg, torch.zeros(3, 1, 16, 64, device="cuda"), None, torch.zeros(3, 1, 16, 64, device="cuda"), None, lane, lane)


class Layer:
    def __init__(self, g, Hq, Hkv, D, page, n_pages, act):
        self.pools = [torch.full((n_pages, Hkv, page, D), float("nan"), dtype=act, device="cuda") for _ in range(2)]
        self.w_q, self.w_k = 1 + 0.1 * torch.randn(2, D, generator=g, device="cuda")


@pytest.mark.parametrize("act,tokens", [("bf16", 1), ("bf16", 3), ("fp32", 2)])
@pytest.mark.parametrize("graph", [False, True])
def test_serving_run(act, tokens, graph):
    """Prompts into the cache, forks, then decode steps of two layers as they are used: resize, copy, norm and rotation into
    the pages, attention; rejected tokens are taken back by a shorter length; a compaction in between.  In the graph form a
    step is captured once, allocation included, and replayed."""
    dt = torch.bfloat16 if act == "bf16" else torch.float32
    Hq, Hkv, D, page, R = 4, 2, 64, 16, 32
    n_pages, n_rows, mp = 60, 6, 10
    cfg = gdn.make_attn_config(Hq, Hkv, D, page_size=page, act=act, n_pages=n_pages, n_rows=n_rows, max_pages=mp)
    g = torch.Generator(device="cuda").manual_seed(7)
    layers = [Layer(g, Hq, Hkv, D, page, n_pages, dt) for _ in range(2)]
    f = (1000.0 ** (-torch.arange(0, R, 2, device="cuda").double() / R)).float()
    table, lens, refs = torch.full((n_rows, mp), -1, dtype=torch.int32, device="cuda"), ints([0] * n_rows), ints([0] * n_pages)
    ws = torch.empty(gdn.gdn_page_workspace_size(cfg, n_pages), dtype=torch.uint8, device="cuda")
    attn_ws = torch.empty(gdn.gdn_attn_workspace_size(cfg, n_rows, tokens), dtype=torch.uint8, device="cuda")
    lanes = [torch.empty(n_rows, dtype=torch.int32, device="cuda") for _ in range(3)]
    # what the model of the test keeps: per layer and row the prepared keys and values, tokens first
    kept = [[(torch.zeros(0, Hkv, D), torch.zeros(0, Hkv, D)) for _ in range(n_rows)] for _ in layers]

    def qkv(T):
        x = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device="cuda").to(dt)
        return x, [t.unflatten(1, (-1, D)) for t in x.split([Hq * D, Hkv * D, Hkv * D], 1)]

    # prompts
    prompt = {0: 37, 3: 16, 4: 5}
    rows, new = list(prompt), list(prompt.values())
    out3 = [t[:3] for t in lanes]
    gdn.gdn_page_resize(cfg, table, lens, refs, ints(rows), ints(new), *out3, ws)
    cu = ints([0, 37, 53, 58])
    for li, layer in enumerate(layers):
        _, (q, k, v) = qkv(58)
        q_out, k_out = torch.empty(58, Hq, D, dtype=dt, device="cuda"), torch.empty(58, Hkv, D, dtype=dt, device="cuda")
        gdn.gdn_attn_prep(cfg, q, k, q_out, f, k_out=k_out, v=v, k_pages=layer.pools[0], v_pages=layer.pools[1], page_table=table, lens=lens,
                          rows=ints(rows), cu_seqlens=cu, w_q=layer.w_q, w_k=layer.w_k)
        for r, a, b in ((0, 0, 37), (3, 37, 53), (4, 53, 58)):
            kept[li][r] = (k_out[a:b].cpu(), v[a:b].cpu())
    # two samples of the first prompt
    gdn.gdn_page_fork(cfg, table, lens, refs, ints([0, 0]), ints([1, 5]))
    for li in range(2):
        kept[li][1] = kept[li][5] = kept[li][0]
    live = [0, 1, 3, 4, 5]
    n = len(live)
    rows_t = ints(live)
    x_in = [qkv(n * tokens)[0] for _ in layers]
    q_out, out = torch.empty(n * tokens, Hq, D, dtype=dt, device="cuda"), [torch.empty(n * tokens, Hq, D, dtype=dt, device="cuda") for _ in layers]
    k_out, lse = [torch.empty(n * tokens, Hkv, D, dtype=dt, device="cuda") for _ in layers], torch.empty(n * tokens, Hq, device="cuda")
    target = ints([0] * n)
    step_lanes = [t[:n] for t in lanes]
    q_seen = [torch.empty_like(q_out) for _ in layers]

    def step():
        gdn.gdn_page_resize(cfg, table, lens, refs, rows_t, target, *step_lanes, ws)
        for li, layer in enumerate(layers):
            gdn.gdn_page_copy(cfg, *layer.pools, *layer.pools, step_lanes[1], step_lanes[2])
            q, k, v = [t.unflatten(1, (-1, D)) for t in x_in[li].split([Hq * D, Hkv * D, Hkv * D], 1)]
            gdn.gdn_attn_prep(cfg, q, k, q_seen[li], f, k_out=k_out[li], v=v, k_pages=layer.pools[0], v_pages=layer.pools[1], page_table=table,
                              lens=lens, rows=rows_t, tokens=tokens, w_q=layer.w_q, w_k=layer.w_k)
            gdn.gdn_attn_decode(cfg, q_seen[li], *layer.pools, table, lens, out[li], attn_ws, tokens=tokens, rows=rows_t, lse=lse)

    cg = None
    if graph:
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            step()
    for turn in range(9):
        lengths = [len(kept[0][r][0]) + tokens for r in live]
        target.copy_(torch.tensor(lengths, dtype=torch.int32))
        for x in x_in:
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        cg.replay() if graph else step()
        torch.cuda.synchronize()
        assert step_lanes[0].tolist() == lengths and gdn.gdn_device_error() == 0
        for li in range(2):
            v = x_in[li].cpu().split([Hq * D, Hkv * D, Hkv * D], 1)[2].unflatten(1, (-1, D))
            for i, r in enumerate(live):
                part = slice(i * tokens, (i + 1) * tokens)
                kept[li][r] = (torch.cat([kept[li][r][0], k_out[li][part].cpu()]), torch.cat([kept[li][r][1], v[part]]))
                K, V = (t.transpose(0, 1) for t in kept[li][r])
                L = lengths[i]
                want, l, mag, top = ref.attend(q_seen[li][part].cpu(), K, V, [L - tokens + 1 + j for j in range(tokens)], D ** -0.5)
                tol, _ = ref.attend_tolerance(want, mag, top, L, D, dt)
                assert ((out[li][part].double().cpu() - want).abs() <= tol).all(), (turn, li, r)
        if tokens > 1:          # the last token of two rows is rejected
            back = [0, 4]
            for li in range(2):
                for r in back:
                    kept[li][r] = tuple(t[:-1] for t in kept[li][r])
            short = [t[:2] for t in lanes]
            gdn.gdn_page_resize(cfg, table, lens, refs, ints(back), ints([len(kept[0][r][0]) for r in back]), *short, ws)
        if turn == 4:           # one sample ends, and what it held is closed up
            moves = [torch.empty(n_pages, dtype=torch.int32, device="cuda") for _ in range(2)]
            one = [t[:1] for t in lanes]
            gdn.gdn_page_resize(cfg, table, lens, refs, ints([1]), ints([0]), *one, ws)
            gdn.gdn_page_compact(cfg, table, lens, refs, table, refs, *moves, ws)
            for layer in layers:
                gdn.gdn_page_copy(cfg, *layer.pools, *layer.pools, *moves)
            gdn.gdn_page_fork(cfg, table, lens, refs, ints([5]), ints([1]))
            for li in range(2):
                kept[li][1] = kept[li][5]
            assert (refs > 0).sum() == refs.nonzero().max() + 1
