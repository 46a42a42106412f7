"""Plain definitions of the operators for long contexts and several hypotheses: whole
numbers by Python loops, attention in 64 bits.  Test infrastructure only."""
from __future__ import annotations

import math
from fractions import Fraction

import torch


def _least_exponent(big: float) -> int:
    """Least e of [-100, 100] with big <= 127 * 2^e."""
    for e in range(-100, 100):
        if Fraction(big) <= 127 * Fraction(2) ** e:
            return e
    return 100


def row_values(codes, scale_bytes):
    """8-bit rows (codes uint8 [..., d], bytes [...]) as fp64."""
    x = codes.view(torch.float8_e4m3fn).double()
    return x * torch.pow(2.0, scale_bytes.double() - 127.0)[..., None]


def page_bounds(keys):
    """keys fp64 [n][d] of a page's committed tokens -> (hi codes, lo codes, byte)."""
    most = float(torch.finfo(torch.bfloat16).max)
    his, los = [], []
    for col in keys.t().tolist():
        some = [max(-most, min(most, x)) for x in col if not math.isnan(x)]
        his.append(max(some) if some else 0.0)
        los.append(min(some) if some else 0.0)
    e = _least_exponent(max(max(abs(x) for x in his), max(abs(x) for x in los)))
    unit = 2.0 ** e

    def held(x):
        return max(-127, min(127, x))
    return ([held(math.ceil(x / unit)) for x in his], [held(math.floor(x / unit)) for x in los],
            e + 127)


def query_codes(q):
    """q [G][d] -> whole numbers [G][d] of one group."""
    x = q.double()
    fine = x[torch.isfinite(x)].abs()
    e = _least_exponent(float(fine.max()) if fine.numel() else 0.0)
    y = torch.round(torch.nan_to_num(x, 0.0, math.inf, -math.inf) / 2.0 ** e).clamp(-127, 127)
    return y.long()


def choose(q, bounds, exps, k, n_first, n_last):
    """q [G][d], bounds int8 [nb][2][d], exps [nb] -> ascending list of at most k pages."""
    nb = bounds.shape[0]
    if nb == 0:
        return []
    c, hi, lo = query_codes(q), bounds[:, 0].long(), bounds[:, 1].long()
    dots = torch.maximum(c[:, None] * hi, c[:, None] * lo).sum(-1).amax(0)
    score = [int(d) * Fraction(2) ** (int(e) - 127) for d, e in zip(dots, exps)]
    forced = [j for j in range(nb) if j < n_first or j >= nb - n_last]
    rest = sorted(set(range(nb)) - set(forced), key=lambda j: (-score[j], j))
    return sorted((forced + rest)[:k])


def attend(q, keys, values, scale):
    """q [G][d], keys, values [n][d] fp64 -> (out [G][d], lse [G])."""
    if keys.shape[0] == 0:
        return torch.zeros_like(q, dtype=torch.float64), torch.full((q.shape[0],), -math.inf,
                                                                    dtype=torch.float64)
    x = (q.double() @ keys.t()) * scale
    lse = torch.logsumexp(x, 1)
    return torch.exp(x - lse[:, None]) @ values, lse


def fork(table, lens, refs, src, reserve, P):
    """Lists in, lists out: (table, lens, refs, [(from, to)])."""
    free = [p for p, c in enumerate(refs) if c == 0]
    width = len(table[0]) if table else 0
    out, out_lens, moves, seen = [], [], [], set()
    short = False
    for p, more in zip(src, reserve):
        row = [-1] * width
        L = lens[p] if p >= 0 else 0
        keep = L
        for j in range(min(width, -(-(L + max(more, 0)) // P)) if p != -1 else 0):
            has = table[p][j] if p >= 0 else -1
            if j < L // P or (p >= 0 and p not in seen and has >= 0 and refs[has] == 1):
                row[j] = has
                continue
            if free:
                row[j] = free.pop(0)
            else:
                short = True
                if j * P < L:
                    keep = j * P
            if j * P < L and row[j] >= 0:
                moves.append((has, row[j]))
        if p >= 0:
            seen.add(p)
        out.append(row)
        out_lens.append(keep)
    count = list(refs)
    for rows, sign in ((table, -1), (out, 1)):
        for row in rows:
            for p in row:
                if p >= 0:
                    count[p] += sign
    return out, out_lens, count, moves, short


def compact(table, refs):
    n = sum(c > 0 for c in refs)
    holes = [p for p in range(n) if refs[p] <= 0]
    to = {}
    for p, c in enumerate(refs):
        if c > 0:
            to[p] = p if p < n else holes.pop(0)
    counts = [0] * len(refs)
    for p, z in to.items():
        counts[z] = refs[p]
    moved = [[to[p] if p >= 0 else -1 for p in row] for row in table]
    return moved, counts, n, [(p, z) for p, z in to.items() if p != z]


def beams(logits, scores, finished, eos, k):
    """One sequence: logits [W][V], scores [W] -> [(score, beam, token)], best first."""
    some = []
    for w in range(logits.shape[0]):
        s = float(scores[w])
        if math.isnan(s) or s == -math.inf:
            continue
        if finished is not None and bool(finished[w]):
            some.append((-s, w, eos))
            continue
        x = logits[w].double()
        x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
        top = x.max()
        if top == -math.inf:
            continue
        if top == math.inf:
            x = torch.where(x == math.inf, 0.0, -math.inf).double()
            top = x.max()
        y = (x - top) - torch.log(torch.exp(x - top).sum()) + s
        for v in (x > -math.inf).nonzero()[:, 0].tolist():
            some.append((-float(y[v]), w, v))
    some.sort()
    return [(-a, w, v) for a, w, v in some[:k]]
