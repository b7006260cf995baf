"""The state space mixer's operators and the block norms, as cases to measure.

`run` computes one pass of an operator: in its plain form, elementary torch operations in 32 bits
(64 for the running log-decays), or, where `own` is true, by the library's entry points.  `exact`
computes the same from the definition, token by token in 64 bits.

Operators (`case["op"]`):
  scan      selective state space scan over a packed batch of prompts
  conv      its short causal convolution (width 4, bias, SiLU) over a packed batch
  step      one token per sequence: convolution step and scan step, states in place
  norm      gated post-norm of a block's output, residual add, next block's pre-norm
  norm_bwd  the gradients of `norm`
"""
import math

import torch

own = False

PLAIN_CHUNK = 64
EPS = 1e-6


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # a prompt of 8,192 tokens at the mixer's own head layout (16 groups, 32 heads, 128 x 128 states)
        dict(name="scan_8k", op="scan", lens="8192", heads=32, groups=16, d_state=128, head_dim=128, act="bf16", state=False, z=True),
        # a serving batch: 16 packed prompts of ragged lengths continuing from their states, many narrow heads
        dict(name="scan_varlen", op="scan", lens="rand:16:256:4096", heads=64, groups=8, d_state=128, head_dim=64, act="bf16", state=True, z=True),
        # one long document in a small model: few heads, so the work has to be split along the sequence
        dict(name="scan_64k", op="scan", lens="65536", heads=8, groups=1, d_state=64, head_dim=64, act="bf16", state=False, z=False),
        # a few short prompts in 32 bits, as a numerics check of a model runs them
        dict(name="scan_short_fp32", op="scan", lens="1,7,0,33,100,256,129", heads=8, groups=2, d_state=64, head_dim=64, act="fp32", state=True, z=True),
        # the convolution in front of scan_8k
        dict(name="conv_8k", op="conv", lens="8192", heads=32, groups=16, d_state=128, head_dim=128, act="bf16", state=False),
        # ragged short prompts in 32 bits, some shorter than the window
        dict(name="conv_ragged_fp32", op="conv", lens="rand:33:1:200", heads=24, groups=1, d_state=64, head_dim=64, act="fp32", state=True),
        # a full decode batch: 64 sequences, 128 MiB of states read and written
        dict(name="step_64", op="step", n=64, heads=32, groups=16, d_state=128, head_dim=128, act="bf16", z=True),
        # one user's next token: latency
        dict(name="step_1", op="step", n=1, heads=24, groups=1, d_state=128, head_dim=64, act="bf16", z=True),
        # the norms around a block in training or a long prompt's prefill
        dict(name="norm_8k", op="norm", rows=8192, dim=4096, act="bf16", res="bf16", gate="channel"),
        # one decode step of 64 sequences with a 32-bit residual stream
        dict(name="norm_64", op="norm", rows=64, dim=5120, act="bf16", res="fp32", gate="row"),
        # the training step's backward of norm_8k
        dict(name="norm_bwd_8k", op="norm_bwd", rows=8192, dim=4096, act="bf16", res="bf16", gate="channel"),
        # an odd width in 32 bits: no vector loads
        dict(name="norm_bwd_odd_fp32", op="norm_bwd", rows=777, dim=1111, act="fp32", res="fp32", gate="row"),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["scan", "scan", "conv", "step", "norm", "norm_bwd"])
    act = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("norm", "norm_bwd"):
        dim = spread(48, 8192)
        dim = dim if rng.random() < 0.4 else max(8, dim // 8 * 8)
        rows = min(spread(1, 16384), (1 << 25) // dim)
        return dict(op=op, rows=rows, dim=dim, act=act, res=rng.choice(["bf16", "fp32"]) if act == "bf16" else "fp32",
                    gate=rng.choice(["channel", "row", "none"]))
    groups = rng.choice([1, 2, 4, 8])
    heads = groups * rng.choice([1, 2, 3, 4, 8])
    case = dict(op=op, heads=heads, groups=groups, d_state=rng.choice([32, 64, 128, 128]), head_dim=rng.choice([32, 64, 64, 128]), act=act)
    if op == "step":
        return dict(case, n=spread(1, 96), z=rng.random() < 0.7)
    lo = spread(1, 512)
    hi = max(lo, spread(8, 4096))
    n = max(1, min(spread(1, 48), 24000 // ((lo + hi) // 2 + 1)))
    case = dict(case, lens="rand:%d:%d:%d" % (n, lo, hi), state=rng.random() < 0.5)
    return dict(case, z=rng.random() < 0.7) if op == "scan" else case


# --------------------------------------------------------------------------- inputs

def _lens(case):
    """Lengths of the packed sequences: given, or drawn the same for every seed of a case."""
    spec = case["lens"]
    if not spec.startswith("rand:"):
        return [int(v) for v in spec.split(",")]
    n, lo, hi = (int(v) for v in spec.split(":")[1:])
    g = torch.Generator().manual_seed(n * 1000003 + lo * 1009 + hi)
    return torch.randint(lo, hi + 1, (n,), generator=g).tolist()


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    act = _dtype(case["act"])

    def normal(*shape, std=1.0, dtype=act):
        return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0):
        return torch.rand(shape, generator=gen, device="cuda") * (hi - lo) + lo

    s = dict(case=case, op=case["op"])
    if case["op"] in ("norm", "norm_bwd"):
        rows, dim, res = case["rows"], case["dim"], _dtype(case["res"])
        s.update(block=normal(rows, dim), residual=normal(rows, dim, std=2.0, dtype=res), scale=0.5,
                 w_post=1.0 + 0.1 * normal(dim, dtype=torch.float32), w_pre=1.0 + 0.1 * normal(dim, dtype=torch.float32),
                 gate=None if case["gate"] == "none" else normal(rows, dim if case["gate"] == "channel" else 1))
        if case["op"] == "norm_bwd":
            # what the forward pass left: the new residual and the rows' 1 / rms
            p = s["block"].float()
            s["rstd_post"] = torch.rsqrt(p.square().mean(1) + EPS)
            u = s["residual"].float() + s["scale"] * (1.0 if s["gate"] is None else torch.sigmoid(s["gate"].float())) * (
                p * s["rstd_post"][:, None] * s["w_post"])
            s["rstd_pre"] = torch.rsqrt(u.square().mean(1) + EPS)
            s["res_out"] = u.to(res)
            s["dh"] = normal(rows, dim)
            s["d_res_out"] = normal(rows, dim, dtype=res)
        return s

    H, G, N, P = case["heads"], case["groups"], case["d_state"], case["head_dim"]
    CH = H * P + 2 * G * N
    s.update(H=H, G=G, N=N, P=P, CH=CH)
    # step sizes log-uniform in [1e-3, 0.1] at a zero projection, decay rates in [1, 16]
    dt0 = torch.exp(uniform(H, lo=math.log(1e-3), hi=math.log(0.1)))
    s.update(dt_bias=dt0 + torch.log(-torch.expm1(-dt0)), A_log=torch.log(uniform(H, lo=1.0, hi=16.0)),
             D=1.0 + 0.1 * normal(H, dtype=torch.float32))
    if case["op"] == "step":
        n = case["n"]
        s.update(x=normal(n, CH), dt=normal(n, H), z=normal(n, H * P) if case["z"] else None,
                 conv_w=normal(CH, 4, std=0.5), conv_bias=normal(CH, std=0.1),
                 conv_state=normal(n, CH, 3), state=normal(n, H, N, P, std=0.2, dtype=torch.float32))
        return s
    lens = _lens(case)
    T = sum(lens)
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
    cu[1:] = torch.tensor(lens).cumsum(0)
    s.update(lens=lens, cu=cu.cuda(), T=T)
    if case["op"] == "conv":
        s.update(x=normal(T, CH), conv_w=normal(CH, 4, std=0.5), conv_bias=normal(CH, std=0.1),
                 conv_state=normal(len(lens), CH, 3) if case["state"] else torch.zeros(len(lens), CH, 3, device="cuda", dtype=act))
        return s
    xbc = normal(T, CH, dtype=torch.float32)
    xbc = (xbc * torch.sigmoid(xbc)).to(act)          # what the convolution's SiLU leaves
    s.update(x=xbc[:, :H * P], b=xbc[:, H * P:H * P + G * N], c=xbc[:, H * P + G * N:], dt=normal(T, H),
             z=normal(T, H * P) if case["z"] else None,
             state=normal(len(lens), H, N, P, std=0.2, dtype=torch.float32) if case["state"] else None)
    return s


# --------------------------------------------------------------------------- the library's calls

def _own_cfg(s, n_slots):
    from gateddeltanet_linear_attention_gb300 import gdn
    return gdn, gdn.make_ssm_config(s["G"], s["H"], s["N"], s["P"], act=s["case"]["act"], n_slots=n_slots)


def _own(s):
    op = s["op"]
    if op == "scan":
        n = len(s["lens"])
        if "cfg" not in s:      # the handle and the workspace that a program keeps
            gdn, s["cfg"] = _own_cfg(s, n)
            s["gdn"], s["ws"] = gdn, torch.empty(gdn.gdn_ssm_workspace_size(s["cfg"], s["T"], n), dtype=torch.uint8, device="cuda")
        y = torch.empty(s["T"], s["H"] * s["P"], dtype=s["x"].dtype, device="cuda")
        out = torch.empty(n, s["H"], s["N"], s["P"], device="cuda")
        s["gdn"].gdn_ssm_prefill(s["cfg"], s["x"], s["b"], s["c"], s["dt"], s["A_log"], s["cu"], y, D=s["D"], dt_bias=s["dt_bias"],
                                 z=s["z"], state_in=s["state"], state_out=out, workspace=s["ws"])
        return [y, out]
    if op == "conv":
        if "cfg" not in s:
            s["gdn"], s["cfg"] = _own_cfg(s, len(s["lens"]))
        out = torch.empty(s["T"], s["CH"], dtype=s["x"].dtype, device="cuda")
        s["gdn"].gdn_ssm_conv_prefill(s["cfg"], s["x"], s["cu"], s["conv_w"], s["conv_bias"], s["conv_state"], None, out)
        return [out, s["conv_state"]]
    if op == "step":
        n = s["case"]["n"]
        if "cfg" not in s:
            gdn, s["cfg"] = _own_cfg(s, n)
            s["gdn"], s["ws"] = gdn, torch.empty(gdn.gdn_ssm_workspace_size(s["cfg"], n, n), dtype=torch.uint8, device="cuda")
        y = torch.empty(n, s["H"] * s["P"], dtype=s["x"].dtype, device="cuda")
        s["gdn"].gdn_ssm_decode(s["cfg"], s["x"], s["dt"], s["conv_w"], s["conv_state"], s["A_log"], s["state"], y, s["ws"],
                                conv_bias=s["conv_bias"], D=s["D"], dt_bias=s["dt_bias"], z=s["z"])
        return [y, s["state"], s["conv_state"]]
    from gateddeltanet_linear_attention_gb300 import gdn
    rows = s["block"].shape[0]
    if op == "norm":
        res_out, h = torch.empty_like(s["residual"]), torch.empty_like(s["block"])
        rstd_post, rstd_pre = torch.empty(2, rows, device="cuda")
        gdn.gdn_block_norm(s["residual"], s["w_pre"], h, block=s["block"], res_out=res_out, w_post=s["w_post"], gate=s["gate"],
                           res_scale=s["scale"], eps=EPS, rstd_post=rstd_post, rstd_pre=rstd_pre)
        return [res_out, h, rstd_post, rstd_pre]
    if "ws" not in s:
        s["ws"] = torch.empty(gdn.gdn_block_norm_workspace_size(rows, s["block"].shape[1]), dtype=torch.uint8, device="cuda")
    d_res, d_block = torch.empty_like(s["res_out"]), torch.empty_like(s["block"])
    d_gate = None if s["gate"] is None else torch.empty_like(s["gate"])
    dw_post, dw_pre = torch.empty(2, s["block"].shape[1], device="cuda")
    gdn.gdn_block_norm_backward(s["res_out"], s["rstd_pre"], s["w_pre"], s["dh"], s["d_res_out"], d_res, dw_pre, block=s["block"],
                                rstd_post=s["rstd_post"], w_post=s["w_post"], gate=s["gate"], res_scale=s["scale"],
                                d_block=d_block, d_gate=d_gate, dw_post=dw_post, workspace=s["ws"])
    return [d_res, d_block, d_gate, dw_post, dw_pre]


# --------------------------------------------------------------------------- the plain forms

def _silu(v):
    return v * torch.sigmoid(v)


def _softplus(v):
    return torch.clamp(v, min=0) + torch.log1p(torch.exp(-v.abs()))


def _plain_scan(s):
    """Chunks of 64 tokens of one sequence each: products inside a chunk, then between the chunks of a sequence."""
    H, G, N, P, T, L = s["H"], s["G"], s["N"], s["P"], s["T"], PLAIN_CHUNK
    n, per = len(s["lens"]), H // G
    NC = sum((v + L - 1) // L for v in s["lens"])
    cu = s["cu"].long()
    lens = cu[1:] - cu[:-1]
    count = (lens + L - 1) // L
    first = torch.cumsum(count, 0) - count
    seq = torch.repeat_interleave(torch.arange(n, device="cuda"), count, output_size=NC)
    local = (torch.arange(NC, device="cuda") - first[seq])[:, None] * L + torch.arange(L, device="cuda")
    valid = (local < lens[seq][:, None])[..., None]
    pos = (cu[seq][:, None] + local).clamp(max=T - 1)
    x = (s["x"].float()[pos] * valid).view(NC, L, H, P).permute(0, 2, 1, 3)                # [NC, H, L, P]
    b = (s["b"].float()[pos] * valid).view(NC, L, G, N).permute(0, 2, 1, 3)                # [NC, G, L, N]
    c = (s["c"].float()[pos] * valid).view(NC, L, G, N).permute(0, 2, 1, 3)
    dt = (_softplus(s["dt"].float()[pos] + s["dt_bias"]) * valid).permute(0, 2, 1)         # [NC, H, L]
    cs = torch.cumsum((dt * -torch.exp(s["A_log"])[:, None]).double(), 2)
    causal = torch.ones(L, L, dtype=torch.bool, device="cuda").tril()
    decay = torch.exp((cs[..., :, None] - cs[..., None, :]).float().masked_fill(~causal, -math.inf))
    scores = (c @ b.transpose(2, 3)).repeat_interleave(per, 1) * decay * dt[:, :, None]
    y = scores @ x
    total = cs[..., -1]
    w = dt * torch.exp((total[..., None] - cs).float())
    part = b.transpose(2, 3).repeat_interleave(per, 1) @ (x * w[..., None])                # [NC, H, N, P]
    run_to = torch.cumsum(total, 0)
    before = run_to - total
    link = (seq[:, None] == seq[None]) & torch.ones(NC, NC, dtype=torch.bool, device="cuda").tril(-1)
    carry = torch.exp((before.T[:, :, None] - run_to.T[:, None]).float().masked_fill(~link, -math.inf))
    enter = (carry @ part.transpose(0, 1).reshape(H, NC, N * P)).view(H, NC, N, P).transpose(0, 1)
    if s["state"] is not None:
        enter = enter + torch.exp((before - before[first[seq].clamp(max=NC - 1)]).float())[..., None, None] * s["state"][seq]
    y = y + torch.exp(cs.float())[..., None] * (c.repeat_interleave(per, 1) @ enter) + s["D"][:, None, None] * x
    last = (first + count - 1).clamp(min=0)
    out = torch.exp(total.float())[last][..., None, None] * enter[last] + part[last]
    old = torch.zeros_like(out) if s["state"] is None else s["state"]
    out = torch.where((lens == 0)[:, None, None, None], old, out)
    t = torch.arange(T, device="cuda")
    mine = torch.searchsorted(cu, t, right=True) - 1
    row = first[mine] * L + t - cu[mine]
    y = y.permute(0, 2, 1, 3).reshape(NC * L, H * P)[row]
    y = y if s["z"] is None else y * _silu(s["z"].float())
    return [y.to(s["x"].dtype), out]


def _plain_conv(s):
    cu = s["cu"].long()
    t = torch.arange(s["T"], device="cuda")
    seq = torch.searchsorted(cu, t, right=True) - 1
    local = t - cu[seq]
    x, hist, w = s["x"].float(), s["conv_state"].float(), s["conv_w"].float()

    def back(d):        # the raw input d tokens before each token
        return torch.where((local >= d)[:, None], x[(t - d).clamp(min=0)], hist[seq, :, (3 + local - d).clamp(max=2)])

    out = s["conv_bias"].float() + x * w[:, 3] + back(1) * w[:, 2] + back(2) * w[:, 1] + back(3) * w[:, 0]
    lens = cu[1:] - cu[:-1]
    at = lens[:, None] - 3 + torch.arange(3, device="cuda")                                # positions of the last three inputs
    new = torch.where((at >= 0)[..., None], x[(cu[:-1, None] + at).clamp(0, max(s["T"] - 1, 0))],
                      hist.transpose(1, 2)[torch.arange(len(lens), device="cuda")[:, None], (3 + at).clamp(max=2)])
    s["conv_state"].copy_(new.transpose(1, 2))
    return [_silu(out).to(s["x"].dtype), s["conv_state"]]


def _plain_step(s):
    H, G, N, P = s["H"], s["G"], s["N"], s["P"]
    n = s["x"].shape[0]
    window = torch.cat([s["conv_state"].float(), s["x"].float()[..., None]], 2)
    xbc = _silu((window * s["conv_w"].float()).sum(2) + s["conv_bias"].float())
    s["conv_state"].copy_(window[..., 1:])
    x = xbc[:, :H * P].view(n, H, P)
    b = xbc[:, H * P:H * P + G * N].view(n, G, N).repeat_interleave(H // G, 1)
    c = xbc[:, H * P + G * N:].view(n, G, N).repeat_interleave(H // G, 1)
    dt = _softplus(s["dt"].float() + s["dt_bias"])
    a = torch.exp(-torch.exp(s["A_log"]) * dt)
    s["state"].copy_(a[..., None, None] * s["state"] + b[..., None] * (dt[..., None] * x)[:, :, None])
    y = (c[:, :, None] @ s["state"])[:, :, 0] + s["D"][:, None] * x
    y = y.reshape(n, H * P)
    y = y if s["z"] is None else y * _silu(s["z"].float())
    return [y.to(s["x"].dtype), s["state"], s["conv_state"]]


def _plain_norm(s):
    p, r = s["block"].float(), s["residual"].float()
    rstd_post = torch.rsqrt(p.square().mean(1) + EPS)
    v = p * rstd_post[:, None] * s["w_post"]
    u = r + s["scale"] * (v if s["gate"] is None else torch.sigmoid(s["gate"].float()) * v)
    rstd_pre = torch.rsqrt(u.square().mean(1) + EPS)
    h = u * rstd_pre[:, None] * s["w_pre"]
    return [u.to(s["residual"].dtype), h.to(s["block"].dtype), rstd_post, rstd_pre]


def _plain_norm_bwd(s):
    dh, u_hat = s["dh"].float(), s["res_out"].float() * s["rstd_pre"][:, None]
    g = dh * s["w_pre"]
    du = s["d_res_out"].float() + s["rstd_pre"][:, None] * (g - u_hat * (g * u_hat).mean(1, keepdim=True))
    p_hat = s["block"].float() * s["rstd_post"][:, None]
    sig = None if s["gate"] is None else torch.sigmoid(s["gate"].float())
    dv = s["scale"] * du if sig is None else s["scale"] * du * sig
    d_gate = None
    if sig is not None:
        d_gate = dv * (1 - sig) * p_hat * s["w_post"]
        d_gate = (d_gate if s["case"]["gate"] == "channel" else d_gate.sum(1, keepdim=True)).to(s["gate"].dtype)
    g1 = dv * s["w_post"]
    dp = s["rstd_post"][:, None] * (g1 - p_hat * (g1 * p_hat).mean(1, keepdim=True))
    return [du.to(s["res_out"].dtype), dp.to(s["block"].dtype), d_gate, (dv * p_hat).sum(0), (dh * u_hat).sum(0)]


def run(state):
    if own:
        return _own(state)
    return {"scan": _plain_scan, "conv": _plain_conv, "step": _plain_step, "norm": _plain_norm, "norm_bwd": _plain_norm_bwd}[state["op"]](state)


# --------------------------------------------------------------------------- the work of a pass

def work(case):
    e = 2 if case["act"] == "bf16" else 4
    if case["op"] in ("norm", "norm_bwd"):
        rows, dim, r = case["rows"], case["dim"], 2 if case["res"] == "bf16" else 4
        gate = {"channel": dim, "row": 1, "none": 0}[case["gate"]] * e
        if case["op"] == "norm":
            return {"bytes": rows * (dim * (2 * e + 2 * r) + gate + 8) + 8 * dim, "flops": 12 * rows * dim}
        return {"bytes": rows * (dim * (3 * e + 3 * r) + 2 * gate + 8) + 16 * dim, "flops": 24 * rows * dim}
    H, G, N, P = case["heads"], case["groups"], case["d_state"], case["head_dim"]
    CH = H * P + 2 * G * N
    if case["op"] == "step":
        n = case["n"]
        return {"bytes": n * (8 * H * N * P + (1 + 6) * CH * e + H * e + (2 if case["z"] else 1) * H * P * e) + 5 * CH * e + 12 * H,
                "flops": n * (5 * H * N * P + 10 * CH)}
    lens = _lens(case)
    T, n = sum(lens), len(lens)
    if case["op"] == "conv":
        return {"bytes": 2 * T * CH * e + 5 * CH * e + 6 * n * CH * e, "flops": 10 * T * CH}
    # x, B, C, dt and z once, y once, the states once; products of the recurrence
    states = (2 if case["state"] else 1) * n * H * N * P * 4
    return {"bytes": T * (CH + H + (2 if case["z"] else 1) * H * P) * e + states + 12 * H, "flops": 5 * T * H * N * P}


# --------------------------------------------------------------------------- the definition, in 64 bits

def _exact_dt(s):
    v = s["dt"].double() + s["dt_bias"].double()
    return torch.where(v > 0, v + torch.log1p(torch.exp(-v)), torch.log1p(torch.exp(v)))


def _exact_scan(s):
    H, G, N, P, T = s["H"], s["G"], s["N"], s["P"], s["T"]
    n, longest = len(s["lens"]), max(s["lens"])
    if longest * n * H * N * P > 60e9:      # beyond about 20 s of token steps
        return None
    S = torch.zeros(n, H, N, P, dtype=torch.float64, device="cuda") if s["state"] is None else s["state"].double()
    dt, rate = _exact_dt(s), torch.exp(s["A_log"].double())
    x, b, c = s["x"].double().view(T, H, P), s["b"].double().view(T, G, N), s["c"].double().view(T, G, N)
    y = torch.zeros(T, H, P, dtype=torch.float64, device="cuda")
    starts = s["cu"].tolist()
    for step in range(longest):
        live = [k for k in range(n) if s["lens"][k] > step]
        rows = torch.tensor([starts[k] + step for k in live], device="cuda")
        heads = dt[rows]                                                                   # [live, H]
        xs, bs, cs = x[rows], b[rows].repeat_interleave(H // G, 1), c[rows].repeat_interleave(H // G, 1)
        add = bs[..., None] * (heads[..., None] * xs)[:, :, None]
        every = len(live) == n
        here = S if every else S[live]
        here = here * torch.exp(-rate * heads)[..., None, None] + add
        y[rows] = (cs[..., None] * here).sum(2)
        if every:
            S = here
        else:
            S[live] = here
    y = (y + s["D"].double()[:, None] * x).reshape(T, H * P)
    if s["z"] is not None:
        z = s["z"].double()
        y = y * z / (1 + torch.exp(-z))
    return [y, S]


def _exact_conv_rows(s):
    """Each sequence by itself: its history, then its inputs."""
    outs, hists, starts = [], [], s["cu"].tolist()
    w, bias = s["conv_w"].double(), s["conv_bias"].double()
    for k, length in enumerate(s["lens"]):
        seen = torch.cat([s["conv_state"][k].double().T, s["x"][starts[k]:starts[k + 1]].double()], 0)
        acc = bias.expand(length, -1).clone()
        for j in range(4):
            acc += seen[j:j + length] * w[:, j]
        outs.append(acc / (1 + torch.exp(-acc)))
        hists.append(seen[-3:].T)
    return [torch.cat(outs), torch.stack(hists)]


def _exact_step(s):
    H, G, N, P = s["H"], s["G"], s["N"], s["P"]
    n = s["x"].shape[0]
    seen = torch.cat([s["conv_state"].double(), s["x"].double()[:, :, None]], 2)
    acc = torch.einsum("ncj,cj->nc", seen, s["conv_w"].double()) + s["conv_bias"].double()
    xbc = acc / (1 + torch.exp(-acc))
    x, b, c = torch.split(xbc, [H * P, G * N, G * N], 1)
    x = x.reshape(n, H, P)
    group = torch.arange(H, device="cuda") // (H // G)
    b, c = b.reshape(n, G, N)[:, group], c.reshape(n, G, N)[:, group]
    dt = _exact_dt(s)
    S = s["state"].double() * torch.exp(-torch.exp(s["A_log"].double()) * dt)[:, :, None, None] + torch.einsum("nhk,nhp,nh->nhkp", b, x, dt)
    y = (torch.einsum("nhk,nhkp->nhp", c, S) + s["D"].double()[:, None] * x).reshape(n, H * P)
    if s["z"] is not None:
        z = s["z"].double()
        y = y * z / (1 + torch.exp(-z))
    return [y, S, seen[:, :, 1:]]


def _exact_norm(s):
    p, r = s["block"].double(), s["residual"].double()
    a = 1 / torch.sqrt((p * p).mean(1, keepdim=True) + EPS)
    v = p * a * s["w_post"].double()
    if s["gate"] is not None:
        v = v / (1 + torch.exp(-s["gate"].double()))
    u = r + s["scale"] * v
    k = 1 / torch.sqrt((u * u).mean(1, keepdim=True) + EPS)
    return [u, u * k * s["w_pre"].double(), a[:, 0], k[:, 0]]


def _exact_norm_bwd(s):
    """Reverse-mode differentiation of the definition at the kept 1 / rms values."""
    dim = s["block"].shape[1]
    u, k = s["res_out"].double(), s["rstd_pre"].double()[:, None]
    p, a = s["block"].double(), s["rstd_post"].double()[:, None]
    dh, w2, w1 = s["dh"].double(), s["w_pre"].double(), s["w_post"].double()
    # h = u k w2 with k = (mean u^2 + eps)^-1/2: dk/du = -k^3 u / dim
    du = s["d_res_out"].double() + dh * w2 * k - (dh * w2 * u).sum(1, keepdim=True) * k ** 3 * u / dim
    gate = torch.ones_like(p) if s["gate"] is None else (1 / (1 + torch.exp(-s["gate"].double()))).expand_as(p)
    dn = s["scale"] * du * gate
    d_gate = None
    if s["gate"] is not None:
        d_gate = s["scale"] * du * (p * a * w1) * gate * (1 - gate)
        if s["gate"].shape[1] == 1 and dim > 1:
            d_gate = d_gate.sum(1, keepdim=True)
    dp = dn * w1 * a - (dn * w1 * p).sum(1, keepdim=True) * a ** 3 * p / dim
    return [du, dp, d_gate, (dn * p * a).sum(0), (dh * u * k).sum(0)]


def exact(case, seed):
    s = prepare(case, seed)
    return {"scan": _exact_scan, "conv": _exact_conv_rows, "step": _exact_step, "norm": _exact_norm, "norm_bwd": _exact_norm_bwd}[s["op"]](s)
