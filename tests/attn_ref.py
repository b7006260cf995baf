"""Plain 64-bit forms of the attention layers' operators on the CPU, each value with the sum of the magnitudes that it is a
sum of (what 32-bit roundings are relative to), and the pages' rules on Python lists."""
import math

import torch

U = 2.0 ** -24                      # half a step of a 32-bit float, relative


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def rotate(x, mag, pos, inv_freq, interleaved, sign=1.0):
    """x, mag [T, H, D] turned by sign * pos * inv_freq."""
    R = 2 * inv_freq.numel()
    if R == 0:
        return x, mag
    ang = pos.double()[:, None] * inv_freq.double()
    c, s = torch.cos(ang)[:, None], sign * torch.sin(ang)[:, None]
    ia = torch.arange(0, R, 2) if interleaved else torch.arange(R // 2)
    ib = ia + 1 if interleaved else ia + R // 2
    y, m = x.clone(), mag.clone()
    y[..., ia], y[..., ib] = x[..., ia] * c - x[..., ib] * s, x[..., ib] * c + x[..., ia] * s
    # the angle's own error is absolute, so each term counts in full
    m[..., ia] = m[..., ib] = mag[..., ia] + mag[..., ib]
    return y, m


def prep(x, w, pos, inv_freq, offset=0.0, eps=1e-6, interleaved=False):
    """(values, magnitudes) of the norm and rotation of x [T, H, D]."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * (offset + w.double())
    return rotate(x, x.abs(), pos, inv_freq, interleaved)


def prep_backward(x, w, d, pos, inv_freq, offset=0.0, eps=1e-6, interleaved=False):
    """((dx, magnitudes), (dw, magnitudes) or None)."""
    d = d.double()
    g, gm = rotate(d, d.abs(), pos, inv_freq, interleaved, -1.0)
    if w is None:
        return (g, gm), None
    x, wv = x.double(), offset + w.double()
    a = 1 / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
    h = x * a
    dx = a * (g * wv - h * (g * wv * h).mean(-1, keepdim=True))
    mag = a * (gm * wv.abs() + h.abs() * (gm * wv.abs() * h.abs()).mean(-1, keepdim=True))
    return (dx, mag), ((g * h).sum((0, 1)), (gm * h.abs()).sum((0, 1)))


def attend(q, K, V, ends, scale, window=0, seen=None):
    """q [k, Hq, D], K and V [Hkv, L, D], token j sees [ends[j] - window, ends[j]) and of it what `seen` [L] says.
    Returns out, lse, sum of softmax * |v|, and the largest sum of |q||k| * scale of a row (all 64 bits)."""
    k, Hq, D = q.shape
    Hkv, L = K.shape[0], K.shape[1]
    G = Hq // Hkv
    out, mag = torch.zeros(k, Hq, D, dtype=torch.float64), torch.zeros(k, Hq, D, dtype=torch.float64)
    lse, top = torch.full((k, Hq), -math.inf, dtype=torch.float64), torch.zeros(k, Hq, dtype=torch.float64)
    q, K, V = q.double(), K.double(), V.double()
    for j in range(k):
        at = [i for i in range(max(0, ends[j] - window) if window else 0, max(0, ends[j])) if seen is None or seen[i]]
        if not at:
            continue
        for h in range(Hq):
            kk, vv = K[h // G, at], V[h // G, at]
            s = (kk @ q[j, h]) * scale
            m = s.max()
            p = torch.exp(s - m)
            total = p.sum()
            out[j, h], mag[j, h] = (p @ vv) / total, (p @ vv.abs()) / total
            lse[j, h] = m + torch.log(total)
            top[j, h] = float((kk.abs() @ q[j, h].abs()).max()) * scale
    return out, lse, mag, top


def attend_tolerance(out, mag, top, n, D, act):
    """Bounds of out and lse.  A score sums D products: roundings of either sign walk, 8 standard deviations of them are
    8 sqrt(D) U, and sums that a tensor core cuts off lose up to 2 U in each of its D / 16 steps at most, all one way: of
    the largest sum of magnitudes `top`.  A score's error is a softmax weight's relative error, once in the sum over
    values and once in the normaliser; those sums run over n tokens and err in the same ways; the exponential and its
    argument's rounding are 4 U and U * top.  Weights split in two 16-bit parts keep 2^-16.  One rounding at the end."""
    score = (8 * math.sqrt(D) + D / 8 + 8) * U * top
    sums = (8 * math.sqrt(n) + n / 8 + 64) * U
    split = 2.0 ** -16 if act == torch.bfloat16 else 0.0
    o = half_step(act) * out.abs() + (2 * score + 2 * sums + split)[..., None] * mag
    return o, score + sums


def attend_lse_tolerance(lse, score_and_sums):
    return score_and_sums + 4 * U * lse.abs().nan_to_num(posinf=0.0, neginf=0.0)


class Pages:
    """The pages' rules, lane after lane."""

    def __init__(self, n_pages, n_rows, max_pages, page):
        self.page, self.max_pages, self.n_rows = page, max_pages, n_rows
        self.refs, self.lens = [0] * n_pages, [0] * n_rows
        self.table = [[-1] * max_pages for _ in range(n_rows)]

    def held(self, length):
        return -(-length // self.page)

    def resize(self, rows, new):
        """granted, src, dst, error bits."""
        err, granted, src, dst = 0, [], [], []
        named = [r for r, v in zip(rows, new) if v >= 0 and 0 <= r < self.n_rows]
        free = [p for p, c in enumerate(self.refs) if c == 0]
        at_start, used, out_of = list(self.refs), 0, False
        drop = []
        for r, v in zip(rows, new):
            granted.append(-1)
            src.append(-1)
            dst.append(-1)
            if r < 0 or v < 0:
                continue
            if r >= self.n_rows or named.count(r) > 1:
                err |= 2
                continue
            old = self.lens[r]
            granted[-1] = old
            if v > self.max_pages * self.page:
                err |= 8
                continue
            have, want = self.held(old), self.held(v)
            last = self.table[r][have - 1] if have else -1
            copy = v > old and old % self.page != 0 and at_start[last] > 1
            need = max(0, want - have) + copy
            if need and (out_of or used + need > len(free)):
                out_of = True
                continue
            mine = free[used:used + need]
            used += need
            if copy:
                src[-1], dst[-1] = last, mine[0]
                drop.append(last)
                self.table[r][have - 1] = mine.pop(0)
            for c in range(have, want):
                self.table[r][c] = mine.pop(0)
            for c in range(want, have):
                drop.append(self.table[r][c])
                self.table[r][c] = -1
            self.lens[r] = granted[-1] = v
        for p in free[:used]:
            self.refs[p] = 1
        for p in drop:
            self.refs[p] -= 1
        return granted, src, dst, err

    def fork(self, src, dst):
        err = 0
        named = [d for s, d in zip(src, dst) if s >= 0 and 0 <= d < self.n_rows]
        for s, d in zip(src, dst):
            if s < 0 or d < 0:
                continue
            if s >= self.n_rows or d >= self.n_rows or named.count(d) > 1 or s in named or self.lens[d]:
                err |= 2
                continue
            for c in range(self.held(self.lens[s])):
                self.table[d][c] = self.table[s][c]
                self.refs[self.table[s][c]] += 1
            self.lens[d] = self.lens[s]
        return err

    def compact(self, n):
        kept = sum(c > 0 for c in self.refs)
        holes = [p for p in range(kept) if self.refs[p] == 0][:n]
        movers = [p for p in range(kept, len(self.refs)) if self.refs[p] > 0][:n]
        goes = dict(zip(movers, holes))
        for a, b in goes.items():
            self.refs[b], self.refs[a] = self.refs[a], 0
        for row, length in zip(self.table, self.lens):
            for c in range(self.held(length)):
                row[c] = goes.get(row[c], row[c])
        pad = [-1] * (n - len(movers))
        return movers + pad, holes + pad

    def check(self):
        """Counts are what the rows hold."""
        count = [0] * len(self.refs)
        for row, length in zip(self.table, self.lens):
            assert all(p >= 0 for p in row[:self.held(length)]) and all(p == -1 for p in row[self.held(length):])
            for p in row[:self.held(length)]:
                count[p] += 1
        assert count == self.refs
