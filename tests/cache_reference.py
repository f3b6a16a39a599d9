"""Plain float64 forms of the key-value cache's operators, on the host, for
the GPU tests: loops over sequences and rows, from the definitions in
include/psi_verify.h."""
from __future__ import annotations

import math

import torch

EPS32 = 2.0 ** -24
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # half a step, relative


def chains(parents, R):
    """Per row: the rows it sees (root first), or None when its chain is invalid."""
    rows = [[0]]
    for r in range(1, R):
        p = r - 2 if parents is None else int(parents[r - 1])
        bad = p < -1 or p >= r - 1 or rows[p + 1] is None
        rows.append(None if bad else rows[p + 1] + [r])
    return rows


def gather(pool, table_row, S, count):
    """[count, H, D] float64 keys or values of a sequence; rows of bad pages are None."""
    out = []
    for t in range(count):
        p = int(table_row[t // S]) if t // S < len(table_row) else -1
        out.append(pool[p, t % S].double() if 0 <= p < pool.shape[0] else None)
    return out


def attend(q, k_pages, v_pages, table, lens, parents=None, scale=None):
    """(o, lse, tol): float64 results and, per output element, how far a
    float kernel's may be off.

    The bound counts, for an output o = sum_t p_t v_t: half a step of the
    output's type; for bf16 half a bf16 step of each weight p_t; and in float
    32 bits the score's sum of D products (D + 2 roundings of 2^-24 relative
    to scale * sum |q_d k_d|, which enter p_t's exponent, for numerator and
    denominator), ex2's error and a few products (16 roundings), and the sum
    over T positions (T roundings)."""
    q, k_pages, v_pages = q.cpu(), k_pages.cpu(), v_pages.cpu()
    N, R, Hq, D = q.shape
    S, H = k_pages.shape[1], k_pages.shape[2]
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    bf16 = q.dtype == torch.bfloat16
    o = torch.zeros(N, R, Hq, D, dtype=torch.float64)
    lse = torch.full((N, R, Hq), -math.inf, dtype=torch.float64)
    tol = torch.zeros_like(o)
    for n in range(N):
        length = int(lens[n])
        if length < 0:
            continue
        K = gather(k_pages, table[n], S, length + R)
        V = gather(v_pages, table[n], S, length + R)
        for r, rows in enumerate(chains(None if parents is None else parents[n], R)):
            if rows is None:
                continue
            at = [t for t in range(length) if K[t] is not None]
            at += [length + x for x in rows if K[length + x] is not None]
            if not at:
                continue
            k, v = torch.stack([K[t] for t in at]), torch.stack([V[t] for t in at])
            for h in range(Hq):
                x = q[n, r, h].double()
                kk, vv = k[:, h // G], v[:, h // G]
                s = scale * (kk @ x)
                top = s.max()
                w = torch.exp(s - top)
                total = w.sum()
                p = w / total
                o[n, r, h] = p @ vv
                lse[n, r, h] = top + total.log()
                delta = 2 * (D + 2) * EPS32 * abs(scale) * float((kk.abs() @ x.abs()).max())
                err = 2 * delta + (len(at) + 16) * EPS32 + (2.0 ** -8 if bf16 else 0.0)
                tol[n, r, h] = HALF_STEP[q.dtype] * o[n, r, h].abs() + err * (p @ vv.abs()) + 1e-30
    return o, lse, tol


def append(q, k, v, lens, q_weight, k_weight, eps, inv_freq, interleaved, rope_scale, parents):
    """(q, k, v, valid, tolq, tolk): float64 rows as they are to be stored;
    valid[n][r] False for rows that are not part of the block.

    The bound: half a step of the type, and 24 roundings of 2^-24 of the
    terms |a cos| + |b sin| (mean of squares and its root, the weight, the
    angle's functions, the turn)."""
    q, k, v = q.cpu(), k.cpu(), v.cpu()
    N, R, _, D = q.shape
    rot = 0 if inv_freq is None else 2 * len(inv_freq)
    depth = [[-1 if c is None else len(c) - 1
              for c in chains(None if parents is None else parents[n], R)] for n in range(N)]
    valid = torch.tensor([[d >= 0 for d in row] for row in depth])
    pos = torch.tensor([[int(lens[n]) + max(d, 0) for d in depth[n]] for n in range(N)],
                       dtype=torch.float64)
    out = []
    for x, w in ((q, q_weight), (k, k_weight)):
        y = x.double()
        if w is not None:
            y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.cpu().double()
        bound = y.abs()
        if rot:
            ang = pos[:, :, None, None] * inv_freq.cpu()
            c, s = rope_scale * torch.cos(ang), rope_scale * torch.sin(ang)
            first = list(range(0, rot, 2)) if interleaved else list(range(rot // 2))
            second = [i + 1 for i in first] if interleaved else [i + rot // 2 for i in first]
            a, b = y[..., first].clone(), y[..., second].clone()
            y, bound = y.clone(), bound.clone()
            y[..., first], y[..., second] = a * c - b * s, b * c + a * s
            bound[..., first] = (a * c).abs() + (b * s).abs() + EPS32 * (a.abs() + b.abs())
            bound[..., second] = (b * c).abs() + (a * s).abs() + EPS32 * (a.abs() + b.abs())
        out.append((y, HALF_STEP[q.dtype] * y.abs() + 24 * EPS32 * bound + 1e-30))
    return out[0][0], out[1][0], v, valid, out[0][1], out[1][1]


class Pages:
    """The page bookkeeping, sequence by sequence (``psi_page_state``)."""

    def __init__(self, table, counts, refs, free, n_free):
        self.table = [list(map(int, r)) for r in table]
        self.counts = list(map(int, counts))
        self.refs = list(map(int, refs))
        self.free = list(map(int, free))
        self.n_free = int(n_free)

    def pop(self):
        self.n_free -= 1
        p = self.free[self.n_free]
        self.refs[p] = 1
        return p

    def resize(self, lens, extra, S):
        need = [c if n < 0 else -(-(n + extra) // S) for n, c in zip(lens, self.counts)]
        gone = []
        for n, want in enumerate(need):
            for i in range(want, self.counts[n]):
                p = self.table[n][i]
                self.table[n][i] = -1
                self.refs[p] -= 1
                if self.refs[p] == 0:
                    gone.append(p)
            self.counts[n] = min(self.counts[n], want)
        for p in sorted(gone):
            self.free[self.n_free] = p
            self.n_free += 1
        starved = False
        for n, want in enumerate(need):
            missing = want - self.counts[n]
            if missing <= 0 or want > len(self.table[n]):
                continue
            starved |= missing > self.n_free
            if starved:
                continue
            for i in range(self.counts[n], want):
                self.table[n][i] = self.pop()
            self.counts[n] = want

    def fork(self, lens, src, dst, S):
        """[(from, to, count)] pages to copy; lens is changed in place."""
        before, table = list(self.counts), [list(r) for r in self.table]
        old, copies, starved = list(lens), [], False
        for k, (s, d) in enumerate(zip(src, dst)):
            N = len(old)
            if not (0 <= s < N and 0 <= d < N) or d in src or d in dst[:k] or before[d] or \
                    old[s] < 0:
                continue
            whole, part = divmod(old[s], S)
            if whole + (part > 0) > before[s]:
                continue
            if part:
                starved |= self.n_free == 0
                if starved:
                    continue
                p = self.pop()
                copies.append((table[s][whole], p, part))
                self.table[d][whole] = p
            for i in range(whole):
                self.table[d][i] = table[s][i]
                self.refs[table[s][i]] += 1
            self.counts[d] = whole + (part > 0)
            lens[d] = old[s]
        return copies
