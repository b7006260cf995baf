"""The attention layers' operators beside the recurrent mixers, as cases to measure: query and key
norms with the position rotation, attention of new tokens over a paged cache, and the cache's pages.

`run` computes one pass of an operator: in its plain form, elementary torch operations in 32 bits
(64 for the rotation's angles), or, where `own` is true, by the library's entry points.  `exact`
computes the same from the definition in 64 bits, sequence by sequence.

Operators (`case["op"]`):
  prep      norm of every query and key head, position rotation, new keys and values into the pages
            (`pages` true) or the keys into a tensor (training)
  prep_bwd  the gradients of the norm and the rotation
  decode    attention of 1 to 8 new tokens a sequence over a paged cache
  fork      a serving step's upkeep of the pages: finished rows are freed, prompts forked into samples
            that share their pages, every sample grown (new pages, copies of shared last pages), and
            the copies carried out
  compact   a used cache compacted: pages moved to the lowest places, tables rewritten, data copied
"""
import math

import torch

own = False

EPS = 1e-6


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # a serving step's prompts: six packed ones that continue cached prefixes, wide heads rotated in a quarter of their columns
        dict(name="prep_prompts", op="prep", lens="rand:6:500:2500", past=4096, q_heads=16, kv_heads=2, dim=256, rotary=64, page=64, act="bf16",
             pages=True, offset=1.0, interleaved=False),
        # one decode step of 64 sequences
        dict(name="prep_step_64", op="prep", lens="each:64:1", past=9000, q_heads=32, kv_heads=8, dim=128, rotary=128, page=64, act="bf16",
             pages=True, offset=0.0, interleaved=False),
        # the backward pass of a training batch of four documents
        dict(name="prep_bwd_8k", op="prep_bwd", lens="4096,2048,1500,548", q_heads=32, kv_heads=8, dim=128, rotary=128, act="bf16", offset=0.0,
             interleaved=False),
        # a small model's gradient check in 32 bits: odd lengths and heads, neighbouring pairs, part of the columns
        dict(name="prep_bwd_odd_fp32", op="prep_bwd", lens="333,1,444", q_heads=9, kv_heads=3, dim=64, rotary=24, act="fp32", offset=0.0,
             interleaved=True),
        # a full decode batch of mixed lengths
        dict(name="decode_64", op="decode", lens="rand:64:256:16384", tokens=1, q_heads=32, kv_heads=8, dim=128, page=64, act="bf16", window=0),
        # one user's next token behind a long document, few wide heads: the work has to be split along the cache
        dict(name="decode_1x128k", op="decode", lens="131072", tokens=1, q_heads=16, kv_heads=2, dim=256, page=128, act="bf16", window=0),
        # a verification round: eight tokens for each of 32 sequences
        dict(name="decode_verify_32", op="decode", lens="rand:32:64:8192", tokens=8, q_heads=32, kv_heads=4, dim=128, page=32, act="bf16", window=0),
        # one user's next token in a short chat: latency
        dict(name="decode_1", op="decode", lens="700", tokens=1, q_heads=24, kv_heads=8, dim=128, page=16, act="bf16", window=0),
        # ragged lengths in 32 bits with a sliding window, as a numerics check of a model runs them
        dict(name="decode_odd_fp32", op="decode", lens="1,37,300,1025,64,0,2047", tokens=2, q_heads=12, kv_heads=4, dim=64, page=16, act="fp32", window=500),
        # parallel sampling: 64 prompts of mixed lengths, eight samples each
        dict(name="fork_64x8", op="fork", lens="rand:64:200:3000", samples=8, grow=1, kv_heads=8, dim=128, page=64, act="bf16"),
        # a beam of five on one short prompt in a small model
        dict(name="fork_1x5_fp32", op="fork", lens="77", samples=5, grow=20, kv_heads=3, dim=64, page=16, act="fp32"),
        # a cache of 8,192 pages, three fifths in use, compacted before it is shrunk
        dict(name="compact_8k", op="compact", rows=96, n_pages=8192, live=0.6, kv_heads=8, dim=128, page=64, act="bf16"),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["prep", "prep", "prep_bwd", "decode", "decode", "decode", "fork", "compact"])
    act = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    kv, dim = rng.choice([1, 2, 3, 4, 8]), rng.choice([64, 128, 128, 256])
    case = dict(op=op, kv_heads=kv, dim=dim, act=act)
    if op != "prep_bwd":
        case["page"] = rng.choice([16, 32, 64, 128])
    if op in ("prep", "prep_bwd", "decode"):
        case["q_heads"] = kv * rng.choice([1, 2, 3, 4, 6, 8, 16] if kv <= 4 else [1, 2, 4, 6])
    row = kv * dim * (2 if act == "bf16" else 4)
    if op in ("prep", "prep_bwd"):
        tokens = max(1, min(spread(1, 16384), (1 << 28) // (row * (2 + case["q_heads"] // kv))))
        case.update(rotary=rng.choice([dim, dim // 2, dim // 4, 2 * rng.randint(1, dim // 2)]), offset=rng.choice([0.0, 1.0]),
                    interleaved=rng.random() < 0.3)
        n = min(tokens, spread(1, 64))
        mean = tokens // n
        if op == "prep_bwd":
            return dict(case, lens="rand:%d:%d:%d" % (n, max(1, mean // 2), mean + mean // 2))
        lens = "each:%d:%d" % (min(tokens, spread(1, 256)), rng.randint(1, 8)) if rng.random() < 0.4 else "rand:%d:%d:%d" % (n, max(1, mean // 2), mean + mean // 2)
        return dict(case, lens=lens, past=spread(1, 4096), pages=rng.random() < 0.7)
    if op == "decode":
        hi = spread(1, 131072)
        n = max(1, min(spread(1, 128), int(2.1e9 / (2 * row * hi))))
        hi = min(hi, int(2.1e9 / (2 * row * n)))
        return dict(case, lens="rand:%d:%d:%d" % (n, spread(1, hi), hi), tokens=rng.choice([1, 1, 1, 2, 3, 4, 5, 8]),
                    window=rng.choice([0, 0, 0, spread(1, 8192)]))
    page = 2 * row * case["page"]
    if op == "fork":
        samples = spread(1, 12)
        n = max(1, min(spread(1, 64), int(1.5e8 / (page * samples))))
        hi = max(1, min(spread(16, 4000), int(1e9 / (2 * row * n))))
        return dict(case, lens="rand:%d:%d:%d" % (n, spread(1, hi), hi), samples=samples, grow=spread(1, 64))
    pages = max(32, min(spread(64, 16384), int(2e9 / page)))
    return dict(case, rows=spread(1, 128), n_pages=pages, live=round(rng.uniform(0.1, 0.9), 2))


# --------------------------------------------------------------------------- inputs

def _lens(case):
    """Lengths of the sequences: given, or drawn the same for every seed of a case."""
    spec = case["lens"].split(":")
    if spec[0] == "each":
        return [int(spec[2])] * int(spec[1])
    if spec[0] != "rand":
        return [int(v) for v in case["lens"].split(",")]
    n, lo, hi = (int(v) for v in spec[1:])
    g = torch.Generator().manual_seed(n * 1000003 + lo * 1009 + hi)
    return torch.randint(lo, hi + 1, (n,), generator=g).tolist()


def _pasts(case):
    """Tokens that each sequence has in the cache before a `prep`."""
    g = torch.Generator().manual_seed(case["past"])
    return torch.randint(0, case["past"] + 1, (len(_lens(case)),), generator=g).tolist()


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _ceil(a, b):
    return -(-a // b)


def _table(lens, page, order, columns=None):
    """Page table of sequences of these lengths, pages taken from `order` in turn; -1: none."""
    count = [_ceil(v, page) for v in lens]
    table = torch.full((len(lens), max(1, columns or max(count))), -1, dtype=torch.int32)
    at = 0
    for row, c in enumerate(count):
        table[row, :c] = order[at:at + c]
        at += c
    return table


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    host = torch.Generator().manual_seed(seed)
    act = _dtype(case["act"])

    def normal(*shape, std=1.0, dtype=act):
        t = torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=gen)
        return t if std == 1.0 else t.mul_(std)

    def pools(n_pages):
        return {k: normal(n_pages, case["kv_heads"], case["page"], case["dim"]) for k in ("k_pages", "v_pages")}

    op, Hkv, D = case["op"], case["kv_heads"], case["dim"]
    s = dict(case=case, op=op)
    if op in ("prep", "prep_bwd"):
        Hq, R, lens = case["q_heads"], case["rotary"], _lens(case)
        T = sum(lens)
        cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
        cu[1:] = torch.tensor(lens).cumsum(0)
        # views into one projection's output
        qkv = normal(T, (Hq + 2 * Hkv) * D)
        q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
        around = 1.0 - case["offset"]
        s.update(T=T, cu=cu.cuda(), q=q, k=k, v=v, w_q=around + normal(D, std=0.1, dtype=torch.float32),
                 w_k=around + normal(D, std=0.1, dtype=torch.float32),
                 inv_freq=(1e6 ** (-torch.arange(0, R, 2, dtype=torch.float64) / R)).float().cuda())
        if op == "prep_bwd":
            s.update(dq_out=normal(T, Hq, D), dk_out=normal(T, Hkv, D))
        elif case["pages"]:
            total = [a + b for a, b in zip(_pasts(case), lens)]
            used = sum(_ceil(v, case["page"]) for v in total)
            n_pages = used + used // 8 + 4
            s.update(pools(n_pages), table=_table(total, case["page"], torch.randperm(n_pages, generator=host).int()).cuda(),
                     lens=torch.tensor(total, dtype=torch.int32, device="cuda"))
        else:
            s.update(k_out=torch.empty(T, Hkv, D, dtype=act, device="cuda"))
        return s
    if op == "decode":
        lens, Hq = _lens(case), case["q_heads"]
        used = sum(_ceil(v, case["page"]) for v in lens)
        n_pages = used + used // 16 + 2
        s.update(pools(n_pages), table=_table(lens, case["page"], torch.randperm(n_pages, generator=host).int()).cuda(),
                 lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), q=normal(len(lens) * case["tokens"], Hq, D, std=1.5))
        return s
    if op == "fork":
        lens, samples = _lens(case), case["samples"]
        rows = len(lens) * (1 + samples)
        pages = [_ceil(v, case["page"]) for v in lens]
        columns = _ceil(max(lens) + case["grow"], case["page"]) + 1
        n_pages = sum(pages) + len(lens) * samples * (1 + _ceil(case["grow"], case["page"])) + 3
        order = torch.randperm(n_pages, generator=host).int()
        table = torch.full((rows, columns), -1, dtype=torch.int32)
        table[:len(lens)] = _table(lens, case["page"], order, columns)
        refs = torch.zeros(n_pages, dtype=torch.int32)
        refs[order[:sum(pages)].long()] = 1
        all_lens = torch.zeros(rows, dtype=torch.int32)
        all_lens[:len(lens)] = torch.tensor(lens)
        parents = torch.arange(len(lens), dtype=torch.int32).repeat_interleave(samples)
        children = torch.arange(len(lens), rows, dtype=torch.int32)
        s.update(pools(n_pages), table=table.cuda(), refs=refs.cuda(), lens=all_lens.cuda(), parents=parents.cuda(), children=children.cuda(),
                 none=torch.zeros_like(children).cuda(), new_lens=(all_lens[parents.long()] + case["grow"]).cuda(),
                 granted=torch.empty_like(children).cuda(), src=torch.empty_like(children).cuda(), dst=torch.empty_like(children).cuda())
        return s
    # compact: pairs of rows, the second of which shares the first half of the first one's pages
    rows, n_pages, page = case["rows"], case["n_pages"], case["page"]
    target = max(1, int(n_pages * case["live"]))
    weight = torch.rand(rows, generator=torch.Generator().manual_seed(rows)) + 0.1         # the same for every seed of a case
    own_pages = (weight / weight.sum() * target).int().clamp(min=0)
    order = torch.randperm(n_pages, generator=host).int()
    shared = [0 if r % 2 == 0 else int(own_pages[r - 1]) // 2 for r in range(rows)]
    columns = max(1, max(int(own_pages[r]) + shared[r] for r in range(rows)))
    table, refs = torch.full((rows, columns), -1, dtype=torch.int32), torch.zeros(n_pages, dtype=torch.int32)
    lens, at = torch.zeros(rows, dtype=torch.int32), 0
    for r in range(rows):
        c = int(own_pages[r])
        if shared[r]:
            table[r, :shared[r]] = table[r - 1, :shared[r]]
        table[r, shared[r]:shared[r] + c] = order[at:at + c]
        at += c
        held = shared[r] + c
        lens[r] = max(0, held * page - int(torch.randint(0, page, (1,), generator=host)))
        refs.index_add_(0, table[r, :held].long(), torch.ones(held, dtype=torch.int32))
    moves = n_pages // 2 + 1
    s.update(pools(n_pages), table=table.cuda(), refs=refs.cuda(), lens=lens.cuda(), table_out=torch.empty_like(table).cuda(),
             refs_out=torch.empty_like(refs).cuda(), src=torch.empty(moves, dtype=torch.int32, device="cuda"),
             dst=torch.empty(moves, dtype=torch.int32, device="cuda"))
    return s


# --------------------------------------------------------------------------- the library's calls

def _handle(s):
    """The configuration that a program keeps."""
    if "cfg" not in s:
        from gateddeltanet_linear_attention_gb300 import gdn
        c = s["case"]
        table = s.get("table")
        s["gdn"], s["cfg"] = gdn, gdn.make_attn_config(c.get("q_heads", c["kv_heads"]), c["kv_heads"], c["dim"], page_size=c.get("page", 64), act=c["act"],
                                                       n_pages=s["k_pages"].shape[0] if "k_pages" in s else 0,
                                                       n_rows=0 if table is None else table.shape[0], max_pages=0 if table is None else table.shape[1])
    return s["gdn"], s["cfg"]


def _workspace(s, size):
    if "ws" not in s:
        s["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    return s["ws"]


def _own(s):
    op, c = s["op"], s["case"]
    gdn, cfg = _handle(s)
    if op == "prep":
        q_out = torch.empty(s["q"].shape, dtype=s["q"].dtype, device="cuda")
        norm = dict(w_q=s["w_q"], w_k=s["w_k"], weight_offset=c["offset"], eps=EPS, interleaved=c["interleaved"])
        if c["lens"].startswith("each:"):
            norm["tokens"] = s["T"] // (s["cu"].shape[0] - 1)
        else:
            norm["cu_seqlens"] = s["cu"]
        if not c["pages"]:
            gdn.gdn_attn_prep(cfg, s["q"], s["k"], q_out, s["inv_freq"], k_out=s["k_out"], **norm)
            return [q_out, s["k_out"]]
        gdn.gdn_attn_prep(cfg, s["q"], s["k"], q_out, s["inv_freq"], v=s["v"], k_pages=s["k_pages"], v_pages=s["v_pages"], page_table=s["table"],
                          lens=s["lens"], **norm)
        return [q_out, s["k_pages"], s["v_pages"]]
    if op == "prep_bwd":
        ws = _workspace(s, gdn.gdn_attn_prep_workspace_size(cfg, s["T"]))
        dq, dk = torch.empty_like(s["dq_out"]), torch.empty_like(s["dk_out"])
        dw_q, dw_k = torch.empty(2, c["dim"], device="cuda")
        gdn.gdn_attn_prep_backward(cfg, s["q"], s["k"], s["dq_out"], s["dk_out"], s["inv_freq"], dq=dq, dk=dk, dw_q=dw_q, dw_k=dw_k, w_q=s["w_q"],
                                   w_k=s["w_k"], weight_offset=c["offset"], eps=EPS, interleaved=c["interleaved"], cu_seqlens=s["cu"], workspace=ws)
        return [dq, dk, dw_q, dw_k]
    if op == "decode":
        n = s["lens"].shape[0]
        ws = _workspace(s, gdn.gdn_attn_workspace_size(cfg, n, c["tokens"]))
        out = torch.empty_like(s["q"])
        lse = torch.empty(s["q"].shape[:2], device="cuda")
        gdn.gdn_attn_decode(cfg, s["q"], s["k_pages"], s["v_pages"], s["table"], s["lens"], out, ws, tokens=c["tokens"], window=c["window"], lse=lse)
        return [out, lse]
    if op == "fork":
        ws = _workspace(s, gdn.gdn_page_workspace_size(cfg, s["children"].shape[0]))
        lanes = (s["granted"], s["src"], s["dst"], ws)
        gdn.gdn_page_resize(cfg, s["table"], s["lens"], s["refs"], s["children"], s["none"], *lanes)
        gdn.gdn_page_fork(cfg, s["table"], s["lens"], s["refs"], s["parents"], s["children"])
        gdn.gdn_page_resize(cfg, s["table"], s["lens"], s["refs"], s["children"], s["new_lens"], *lanes)
        gdn.gdn_page_copy(cfg, s["k_pages"], s["v_pages"], s["k_pages"], s["v_pages"], s["src"], s["dst"])
        return [s["table"], s["lens"], s["refs"], s["granted"], s["src"], s["dst"], s["k_pages"], s["v_pages"]]
    ws = _workspace(s, gdn.gdn_page_workspace_size(cfg, s["src"].shape[0]))
    gdn.gdn_page_compact(cfg, s["table"], s["lens"], s["refs"], s["table_out"], s["refs_out"], s["src"], s["dst"], ws)
    gdn.gdn_page_copy(cfg, s["k_pages"], s["v_pages"], s["k_pages"], s["v_pages"], s["src"], s["dst"])
    return [s["table_out"], s["refs_out"], s["src"], s["dst"], s["k_pages"], s["v_pages"]]


# --------------------------------------------------------------------------- the plain forms

def _places(s):
    """Sequence of every packed token and its index in that sequence."""
    cu = s["cu"].long()
    t = torch.arange(s["T"], device="cuda")
    seq = torch.searchsorted(cu, t, right=True) - 1
    at = t - cu[seq]
    if "lens" in s:
        at = at + s["lens"].long()[seq] - (cu[1:] - cu[:-1])[seq]
    return seq, at


def _angles(s, at):
    angle = at.double()[:, None] * s["inv_freq"].double()
    return torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]


def _halves(x, R, interleaved):
    return (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])


def _joined(a, b, rest, interleaved):
    pair = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([pair, rest], -1)


def _rotated(x, cos, sin, R, interleaved):
    a, b = _halves(x, R, interleaved)
    return _joined(a * cos - b * sin, b * cos + a * sin, x[..., R:], interleaved)


def _plain_prep(s):
    c, R = s["case"], s["case"]["rotary"]
    seq, at = _places(s)
    cos, sin = _angles(s, at)

    def prepared(x, w):
        x = x.float()
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * (c["offset"] + w)
        return _rotated(x, cos, sin, R, c["interleaved"]).to(s["q"].dtype)

    q, k = prepared(s["q"], s["w_q"]), prepared(s["k"], s["w_k"])
    if not c["pages"]:
        return [q, k]
    page, off = s["table"][seq, at // c["page"]].long(), at % c["page"]
    s["k_pages"][page, :, off] = k
    s["v_pages"][page, :, off] = s["v"]
    return [q, s["k_pages"], s["v_pages"]]


def _plain_prep_bwd(s):
    c, R = s["case"], s["case"]["rotary"]
    cos, sin = _angles(s, _places(s)[1])

    def back(x, w, d):
        x = x.float()
        g = _rotated(d.float(), cos, -sin, R, c["interleaved"])
        rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        x_hat = x * rstd
        gw = g * (c["offset"] + w)
        return (rstd * (gw - x_hat * (gw * x_hat).mean(-1, keepdim=True))).to(d.dtype), (g * x_hat).sum((0, 1))

    dq, dw_q = back(s["q"], s["w_q"], s["dq_out"])
    dk, dw_k = back(s["k"], s["w_k"], s["dk_out"])
    return [dq, dk, dw_q, dw_k]


def _plain_decode(s):
    c = s["case"]
    k, Hq, Hkv, D = c["tokens"], c["q_heads"], c["kv_heads"], c["dim"]
    n, G = s["lens"].shape[0], Hq // Hkv
    pages = s["table"].long().clamp(min=0)

    def whole(pool):        # [n, Hkv, tokens, D]
        return pool[pages].permute(0, 2, 1, 3, 4).reshape(n, Hkv, -1, D).float()

    q = s["q"].float().view(n, k, Hkv, G, D).transpose(1, 2).reshape(n, Hkv, k * G, D)
    score = q @ whole(s["k_pages"]).transpose(2, 3) * D ** -0.5                            # [n, Hkv, k * G, tokens]
    end = s["lens"].long()[:, None] - k + 1 + torch.arange(k, device="cuda")               # tokens that each new one sees
    end = end.repeat_interleave(G, 1)[:, None, :, None]
    at = torch.arange(score.shape[-1], device="cuda")
    seen = at < end
    if c["window"]:
        seen = seen & (at >= end - c["window"])
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-1e30)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = (p @ whole(s["v_pages"])) / total.clamp(min=1e-30)
    lse = torch.where(total > 0, top + torch.log(total), -math.inf)

    def rows(t):
        return t.view(n, Hkv, k, G, -1).transpose(1, 2).reshape(n * k, Hq, -1)

    return [rows(o).to(s["q"].dtype), rows(lse)[..., 0]]


def _plain_resize(s, rows, new):
    """Sets lengths: pages released behind a shorter one, and taken, lowest first, for a longer one."""
    page, table, lens, refs = s["case"]["page"], s["table"], s["lens"], s["refs"]
    rows, new = rows.long(), new.long()
    old = lens[rows].long()
    have, want = (old + page - 1) // page, (new + page - 1) // page
    last = table[rows, (have - 1).clamp(min=0)].long().clamp(min=0)
    copied = (new > old) & (old % page != 0) & (refs[last] > 1)
    need = (want - have).clamp(min=0) + copied.long()
    upto = torch.cumsum(need, 0)
    granted = (need == 0) | (upto <= (refs == 0).sum())
    copied = copied & granted
    free = torch.argsort((refs != 0).to(torch.int32), stable=True)                         # free pages first, ascending
    column = torch.arange(table.shape[1], device="cuda")
    mine = table[rows].long()
    first = upto - need                                                                    # a lane's first place among them
    at_copy = copied[:, None] & (column == have[:, None] - 1)
    added = granted[:, None] & (column >= have[:, None]) & (column < want[:, None])
    place = torch.where(at_copy, first[:, None], first[:, None] + copied.long()[:, None] + column - have[:, None])
    taken = at_copy | added
    fresh = free[place.clamp(0, free.shape[0] - 1)]
    dropped = granted[:, None] & (column >= want[:, None]) & (column < have[:, None])
    given = dropped | at_copy                                                              # references that end
    refs.index_add_(0, mine.clamp(min=0).flatten(), -given.flatten().to(refs.dtype))
    refs.index_add_(0, fresh.flatten(), taken.flatten().to(refs.dtype))
    table[rows] = torch.where(taken, fresh, torch.where(dropped, -1, mine)).to(table.dtype)
    lens[rows] = torch.where(granted, new, old).to(lens.dtype)
    s["granted"].copy_(torch.where(granted, new, old))
    s["src"].copy_(torch.where(copied, last, -1))
    s["dst"].copy_(torch.where(copied, free[first.clamp(max=free.shape[0] - 1)], -1))


def _plain_copy(s, stay):
    """Pages to pages; lanes without a copy write `stay`, which is nobody's destination, onto itself."""
    live = s["dst"] >= 0
    src, dst = torch.where(live, s["src"], stay).long(), torch.where(live, s["dst"], stay).long()
    s["k_pages"][dst] = s["k_pages"][src]
    s["v_pages"][dst] = s["v_pages"][src]


def _plain_fork(s):
    table, lens, refs = s["table"], s["lens"], s["refs"]
    _plain_resize(s, s["children"], s["none"])
    mine = table[s["parents"].long()]
    held = torch.arange(table.shape[1], device="cuda") < ((lens[s["parents"].long()] + s["case"]["page"] - 1) // s["case"]["page"])[:, None]
    refs.index_add_(0, mine.clamp(min=0).flatten().long(), held.flatten().to(refs.dtype))
    table[s["children"].long()] = torch.where(held, mine, -1)
    lens[s["children"].long()] = lens[s["parents"].long()]
    _plain_resize(s, s["children"], s["new_lens"])
    _plain_copy(s, table[0, 0])
    return [table, lens, refs, s["granted"], s["src"], s["dst"], s["k_pages"], s["v_pages"]]


def _plain_compact(s):
    table, refs, moves = s["table"], s["refs"], s["src"].shape[0]
    live = refs > 0
    page = torch.arange(refs.shape[0], device="cuda")
    kept = live.sum()
    hole, mover = ~live & (page < kept), live & (page >= kept)
    to = torch.argsort((~hole).to(torch.int32), stable=True)[:moves]
    frm = torch.argsort((~mover).to(torch.int32), stable=True)[:moves]
    active = torch.arange(moves, device="cuda") < hole.sum()
    s["src"].copy_(torch.where(active, frm, -1))
    s["dst"].copy_(torch.where(active, to, -1))
    goes = page.scatter(0, frm, torch.where(active, to, frm))
    used = torch.arange(table.shape[1], device="cuda") < ((s["lens"] + s["case"]["page"] - 1) // s["case"]["page"])[:, None]
    s["table_out"].copy_(torch.where(used, goes[table.long().clamp(min=0)], table))
    s["refs_out"].zero_().index_add_(0, goes, refs)
    _plain_copy(s, refs.shape[0] - 1)
    return [s["table_out"], s["refs_out"], s["src"], s["dst"], s["k_pages"], s["v_pages"]]


def run(state):
    if own:
        return _own(state)
    return {"prep": _plain_prep, "prep_bwd": _plain_prep_bwd, "decode": _plain_decode, "fork": _plain_fork, "compact": _plain_compact}[state["op"]](state)


# --------------------------------------------------------------------------- the work of a pass

def work(case):
    e = 2 if case["act"] == "bf16" else 4
    op, Hkv, D = case["op"], case["kv_heads"], case["dim"]
    if op in ("prep", "prep_bwd"):
        T, n, Hq = sum(_lens(case)), len(_lens(case)), case["q_heads"]
        heads = Hq + Hkv
        if op == "prep_bwd":
            return {"bytes": 3 * e * T * heads * D + 16 * D + 2 * case["rotary"] + 4 * n, "flops": 16 * T * heads * D}
        table = 4 * sum(_ceil(v, case["page"]) for v in _lens(case)) + 8 * n if case["pages"] else 0
        return {"bytes": 2 * e * T * (heads + (Hkv if case["pages"] else 0)) * D + 8 * D + 2 * case["rotary"] + table, "flops": 8 * T * heads * D}
    if op == "decode":
        k, Hq = case["tokens"], case["q_heads"]
        lens = _lens(case)
        kept = [min(v, case["window"] + k - 1) if case["window"] else v for v in lens]
        return {"bytes": 2 * e * Hkv * D * sum(kept) + len(lens) * (k * Hq * (2 * e * D + 4) + 4) + 4 * sum(_ceil(v, case["page"]) for v in kept),
                "flops": 4 * k * Hq * D * sum(kept)}
    page = 2 * e * Hkv * D * case["page"]
    if op == "fork":
        lens = _lens(case)
        held = sum(_ceil(v, case["page"]) for v in lens) * case["samples"]
        grown = sum(_ceil(v + case["grow"], case["page"]) - _ceil(v, case["page"]) + (v % case["page"] != 0) for v in lens) * case["samples"]
        copies = sum(v % case["page"] != 0 for v in lens) * case["samples"]
        # freeing: entries and counts read and written; forking: entries read and written, counts too; growing: entries and counts written
        return {"bytes": 2 * page * copies + 16 * (held + grown) + 16 * held + 8 * grown + 40 * len(lens) * case["samples"], "flops": held}
    # pages in random places: those in use beyond their own number are moved
    moved = case["n_pages"] * case["live"] * (1 - case["live"])
    return {"bytes": 2 * page * moved + 8 * case["n_pages"] + 8 * case["n_pages"] * case["live"] * 1.25 + 16 * moved, "flops": case["n_pages"]}


# --------------------------------------------------------------------------- the definition, in 64 bits

def _exact_index(s):
    """Index of every packed token in its sequence, and the sequence."""
    cu = s["cu"].tolist()
    seq, at = [], []
    for i in range(len(cu) - 1):
        L = cu[i + 1] - cu[i]
        start = int(s["lens"][i]) - L if "lens" in s else 0
        seq += [i] * L
        at += range(start, start + L)
    return torch.tensor(seq, device="cuda"), torch.tensor(at, dtype=torch.float64, device="cuda")


def _exact_turn(s, at):
    """The rotation as one complex factor per token and pair."""
    angle = torch.outer(at, s["inv_freq"].double())
    return torch.polar(torch.ones_like(angle), angle)[:, None]


def _exact_rotate(x, turn, R, interleaved):
    x = x.clone()
    first, second = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    z = torch.complex(x[..., first], x[..., second]) * turn
    x[..., first], x[..., second] = z.real, z.imag
    return x


def _exact_prep(s):
    c = s["case"]
    seq, at = _exact_index(s)
    turn = _exact_turn(s, at)
    out = []
    for x, w in ((s["q"], s["w_q"]), (s["k"], s["w_k"])):
        x = x.double()
        n = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["dim"] + EPS) * (c["offset"] + w.double())
        out.append(_exact_rotate(n, turn, c["rotary"], c["interleaved"]))
    if not c["pages"]:
        return out
    kp, vp = s["k_pages"].double(), s["v_pages"].double()
    at = at.long()
    page, off = s["table"][seq, at // c["page"]].long(), at % c["page"]
    for h in range(c["kv_heads"]):
        kp[page, h, off], vp[page, h, off] = out[1][:, h], s["v"][:, h].double()
    return [out[0], kp, vp]


def _exact_prep_bwd(s):
    """n = x a w with a = (mean x^2 + eps)^-1/2, so dn/dx = a w - a^3 (x w) x^T / dim."""
    c = s["case"]
    turn = _exact_turn(s, _exact_index(s)[1]).conj()
    grads, weights = [], []
    for x, w, d in ((s["q"], s["w_q"], s["dq_out"]), (s["k"], s["w_k"], s["dk_out"])):
        x, w = x.double(), c["offset"] + w.double()
        g = _exact_rotate(d.double(), turn, c["rotary"], c["interleaved"])
        a = 1 / torch.sqrt((x * x).sum(-1, keepdim=True) / c["dim"] + EPS)
        grads.append(a * w * g - a ** 3 / c["dim"] * (g * w * x).sum(-1, keepdim=True) * x)
        weights.append(torch.einsum("thd,thd->d", g, x * a))
    return grads + weights


def _exact_decode(s):
    """Every sequence and every new token by itself."""
    c = s["case"]
    k, Hq, Hkv, D = c["tokens"], c["q_heads"], c["kv_heads"], c["dim"]
    G, lens = Hq // Hkv, s["lens"].tolist()
    out = torch.zeros(len(lens) * k, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((len(lens) * k, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for n, L in enumerate(lens):
        if L == 0:
            continue
        pages = s["table"][n, :_ceil(L, c["page"])].long()
        K, V = (pool[pages].transpose(0, 1).reshape(Hkv, -1, D)[:, :L].double() for pool in (s["k_pages"], s["v_pages"]))
        for j in range(k):
            end = L - k + 1 + j
            start = max(0, end - c["window"]) if c["window"] else 0
            if end <= start:
                continue
            q = s["q"][n * k + j].double().view(Hkv, G, D)
            score = torch.einsum("hgd,htd->hgt", q, K[:, start:end]) / math.sqrt(D)
            lse[n * k + j] = torch.logsumexp(score, -1).flatten()
            out[n * k + j] = torch.einsum("hgt,htd->hgd", torch.softmax(score, -1), V[:, start:end]).reshape(Hq, D)
    return [out, lse]


def _exact_fork(s):
    """The pages' upkeep, lane after lane on lists."""
    page = s["case"]["page"]
    table, lens, refs = s["table"].tolist(), s["lens"].tolist(), s["refs"].tolist()
    granted, src, dst = [], [], []
    for p, child in zip(s["parents"].tolist(), s["children"].tolist()):
        for i in range(_ceil(lens[p], page)):
            table[child][i] = table[p][i]
            refs[table[p][i]] += 1
        lens[child] = lens[p]
    shared = list(refs)
    free = [i for i, r in enumerate(refs) if r == 0]
    for child, new in zip(s["children"].tolist(), s["new_lens"].tolist()):
        held = _ceil(lens[child], page)
        fork = lens[child] % page != 0 and shared[table[child][held - 1]] > 1
        need = _ceil(new, page) - held + fork
        assert need <= len(free)
        src.append(-1)
        dst.append(-1)
        if fork:
            src[-1], dst[-1] = table[child][held - 1], free.pop(0)
            refs[src[-1]] -= 1
            refs[dst[-1]] = 1
            table[child][held - 1] = dst[-1]
        for i in range(held, _ceil(new, page)):
            table[child][i] = free.pop(0)
            refs[table[child][i]] = 1
        lens[child] = new
        granted.append(new)
    return [torch.tensor(v, dtype=torch.int32, device="cuda") for v in (table, lens, refs, granted, src, dst)] + _exact_copies(s, src, dst)


def _exact_copies(s, src, dst):
    pools = []
    for name in ("k_pages", "v_pages"):
        pool = s[name].clone()
        for a, b in zip(src, dst):
            if b >= 0:
                pool[b] = s[name][a]
        pools.append(pool)
    return pools


def _exact_compact(s):
    page, table, refs, lens = s["case"]["page"], s["table"].tolist(), s["refs"].tolist(), s["lens"].tolist()
    kept = sum(r > 0 for r in refs)
    holes = [i for i in range(kept) if refs[i] == 0]
    movers = [i for i in range(kept, len(refs)) if refs[i] > 0]
    goes = dict(zip(movers, holes))
    for a, b in goes.items():
        refs[a], refs[b] = 0, refs[a]
    for row, L in zip(table, lens):
        for i in range(_ceil(L, page)):
            row[i] = goes.get(row[i], row[i])
    rest = [-1] * (s["src"].shape[0] - len(movers))
    src, dst = movers + rest, holes + rest
    return [torch.tensor(v, dtype=torch.int32, device="cuda") for v in (table, refs, src, dst)] + _exact_copies(s, src, dst)


def exact(case, seed):
    s = prepare(case, seed)
    return {"prep": _exact_prep, "prep_bwd": _exact_prep_bwd, "decode": _exact_decode, "fork": _exact_fork, "compact": _exact_compact}[s["op"]](s)
