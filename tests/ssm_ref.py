"""Plain 64-bit references of the selective state space mixer and of the block norms, on the CPU.

Beside every value stands the magnitude that its rounding errors are measured by: the same
expression with every term's absolute value.  A tolerance is a number of half steps of the
output's type at the value, and of 2^-24 (or of an operand's rounding) at the magnitude."""
import torch

U32 = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def check(got, value, mag, rel, name):
    """|got - value| <= half a step of got's type at the value + rel * mag, element by element."""
    g = got.detach().double().cpu()
    tol = HALF[got.dtype] * value.abs() + rel * mag + 1e-37
    bad = ~((g - value).abs() <= tol)
    bad &= ~(g.isnan() & value.isnan())
    assert not bad.any(), "%s: %d of %d off, worst %.3g of the tolerance" % (
        name, int(bad.sum()), bad.numel(), float(((g - value).abs() / tol)[bad].max()))


def conv(x, w, bias, hist):
    """One sequence: x [L, CH], w [CH, 4], hist [CH, 3] -> out, its magnitude, new history."""
    seen = torch.cat([hist.double().T, x.double()], 0)
    L = x.shape[0]
    acc = torch.zeros(L, x.shape[1], dtype=torch.float64)
    mag = acc.clone()
    if bias is not None:
        acc += bias.double()
        mag += bias.double().abs()
    for j in range(4):
        acc += seen[j:j + L] * w.double()[:, j]
        mag += (seen[j:j + L] * w.double()[:, j]).abs()
    # |SiLU'| <= 1.1
    return acc * torch.sigmoid(acc), 1.1 * mag, seen[-3:].T.clone()


def step_size(u, dt_bias, dt_min, dt_max):
    v = u.double() + (0 if dt_bias is None else dt_bias.double())
    return torch.nn.functional.softplus(v, threshold=700).clamp(dt_min, dt_max)


def scan(x, b, c, u, A_log, D, dt_bias, z, S, groups, dt_min=0.0, dt_max=float("inf")):
    """One sequence: x [L, H, P], b, c [L, G, N], u [L, H], S [H, N, P] -> y [L, H, P], its
    magnitude, the final state, its magnitude."""
    L, H, P = x.shape
    of = torch.arange(H) // (H // groups)
    S = S.double().clone()
    M = S.abs()
    dt = step_size(u, dt_bias, dt_min, dt_max)
    x, b, c = x.double(), b.double()[:, of], c.double()[:, of]
    y, mag = torch.zeros(L, H, P, dtype=torch.float64), torch.zeros(L, H, P, dtype=torch.float64)
    for t in range(L):
        a = torch.exp(-torch.exp(A_log.double()) * dt[t])[:, None, None]
        add = b[t][:, :, None] * (dt[t][:, None] * x[t])[:, None]
        S = a * S + add
        M = a * M + add.abs()
        y[t] = torch.einsum("hn,hnp->hp", c[t], S)
        mag[t] = torch.einsum("hn,hnp->hp", c[t].abs(), M)
    if D is not None:
        y += D.double()[:, None] * x
        mag += (D.double()[:, None] * x).abs()
    if z is not None:
        g = z.double().view(L, H, P)
        g = g * torch.sigmoid(g)
        y, mag = y * g, mag * g.abs()
    return y, mag, S, M


def norm(p, gate, r, w1, w2, eps, offset, scale):
    """-> dict of (value, magnitude) of r', h, rstd_post, rstd_pre."""
    r = r.double()
    out = {}
    u, mag = r, r.abs()
    if p is not None:
        p = p.double()
        n = p
        if w1 is not None:
            k = 1 / torch.sqrt((p * p).mean(1, keepdim=True) + eps)
            out["rstd_post"] = (k[:, 0], k[:, 0])
            n = p * k * (offset + w1.double())
        s = scale * (1.0 if gate is None else torch.sigmoid(gate.double()))
        u, mag = r + s * n, r.abs() + (s * n).abs()
    out["res_out"] = (u, mag)
    if w2 is not None:
        k = 1 / torch.sqrt((u * u).mean(1, keepdim=True) + eps)
        out["rstd_pre"] = (k[:, 0], k[:, 0] * (1 + (mag * mag).mean(1) * k[:, 0] ** 2))
        grow = 1 + (mag * mag).mean(1, keepdim=True) * k ** 2       # of an error of the mean square
        out["h"] = (u * k * (offset + w2.double()), mag * k * (offset + w2.double()).abs() * grow)
    return out


def norm_backward(p, gate, u, w1, w2, k1, k2, dh, dro, offset, scale):
    """Gradients written out, each with its magnitude."""
    dim = u.shape[1]
    u = u.double()
    du = torch.zeros_like(u) if dro is None else dro.double()
    mag = du.abs()
    out = {}
    if dh is not None:
        k2 = k2.double()[:, None]
        uh, g = u * k2, dh.double() * (offset + w2.double())
        du = du + k2 * (g - uh * (g * uh).sum(1, keepdim=True) / dim)
        mag = mag + k2 * (g.abs() + uh.abs() * (g * uh).abs().sum(1, keepdim=True) / dim)
        out["dw_pre"] = ((dh.double() * uh).sum(0), (dh.double() * uh).abs().sum(0))
    out["d_residual"] = (du, mag)
    if p is not None:
        p = p.double()
        k1 = 1.0 if k1 is None else k1.double()[:, None]
        ph = p * k1
        w = 1.0 if w1 is None else offset + w1.double()
        sg = 1.0 if gate is None else torch.sigmoid(gate.double())
        dn, dnm = scale * sg * du, (scale * sg * mag if gate is not None else abs(scale) * mag)
        dnm = dnm.abs()
        if gate is not None:
            shut = torch.sigmoid(-gate.double())           # 1 - sg, without the difference
            dg, dgm = dn * shut * ph * w, (dnm * shut * ph * w).abs()
            if gate.shape[1] == 1 and dim > 1:
                dg, dgm = dg.sum(1, keepdim=True), dgm.sum(1, keepdim=True)
            out["d_gate"] = (dg, dgm)
        g1, g1m = dn * w, (dnm * w).abs()
        if w1 is not None:
            out["dw_post"] = ((dn * ph).sum(0), (dnm * ph).abs().sum(0))
            out["d_block"] = (k1 * (g1 - ph * (g1 * ph).sum(1, keepdim=True) / dim),
                              k1 * (g1m + ph.abs() * (g1m * ph.abs()).sum(1, keepdim=True) / dim))
        else:
            out["d_block"] = (g1, g1m)
    return out
