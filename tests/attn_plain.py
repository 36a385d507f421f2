"""Plain 64-bit attention of new tokens over a paged cache with window and sinks, inputs whose unseen
rows are NaN and whose unseen blocks are absent, and how far a call may be off."""
import math

import torch

SCALE = 1.0 / math.sqrt(128)


def seen(last, total, window, sinks):
    """[rows, total]: which keys the queries at positions `last` (a list) see."""
    at = torch.tensor(last, dtype=torch.int64)[:, None]
    p = torch.arange(total)[None]
    mask = p <= at
    if window:
        mask = mask & ((p > at - window) | (p < sinks))
    return mask


def attend(q, k, v, mask, scale=SCALE, rounded=False):
    """(out, lse, out's tolerance, lse's) of q [R, Hq, 128] over k, v [P, H, 128] with mask [R, P].

    A call rounds its output once, to bf16: 2^-8 of it. A logit is a sum of 128 exact products in fp32,
    off by 128 roundings of 2^-24 of its terms' sizes at most, d = 2^-17 scale sum|q k|, and the
    exponential and the sums add some 2^-19 more: each weight is off by 2 (d + 2^-19) of itself, the
    sum of up to 2^14 weights by 2^14 2^-24 in any order, 2^-10 at the very worst and the output alike;
    in pieces of a few hundred keys, as they are summed, 2^-15. `rounded`: the weights themselves are
    rounded to bf16, 2^-8 of each, and divided by the sum of the rounded: 2 2^-8."""
    G = q.shape[1] // k.shape[1]
    q, k, v = (x.double().cpu() for x in (q, k, v))
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float64)
    tol, ltol = torch.zeros_like(q), torch.zeros_like(lse)
    for h in range(q.shape[1]):
        kh, vh = k[:, h // G], v[:, h // G]
        z = (q[:, h] @ kh.T * scale).masked_fill(~mask, -math.inf)
        size = (q[:, h].abs() @ kh.abs().T * abs(scale)).masked_fill(~mask, 0.0).amax(1)
        lse[:, h] = torch.logsumexp(z, 1)
        w = torch.exp(z - lse[:, h, None])
        out[:, h] = w @ vh
        each = 2 * (2.0 ** -17 * size + 2.0 ** -19) + 2.0 ** -15 + (2.0 ** -7 if rounded else 0.0)
        tol[:, h] = 2.0 ** -8 * out[:, h].abs() + each[:, None] * (w @ vh.abs()) * (1 + 2.0 ** -7)
        ltol[:, h] = 2.0 ** -17 * size + 2.0 ** -15 + 2.0 ** -22 * lse[:, h].abs()
    return out, lse, tol, ltol


class Batch:
    """Sequences of `keys` keys of which the last new[s] are queries, over a cache that holds the rows that
    a query of the sequence sees and is NaN elsewhere; blocks that none of them is in are absent (-1)."""

    def __init__(self, keys, new, Hq, H, bs, window, sinks, seed, device="cuda", spare=2, extra_rows=0, scale=SCALE,
                 spread=1.0):
        g = torch.Generator().manual_seed(seed)
        S, width = len(keys), max(1, max(-(-n // bs) for n in keys))
        need = sum(-(-n // bs) for n in keys) + spare
        ids = torch.randperm(need, generator=g).tolist()
        nan = float("nan")
        kc, vc = (torch.full((need, bs, H, 128), nan, dtype=torch.bfloat16) for _ in range(2))
        bt = torch.full((S, width), -1, dtype=torch.int32)
        self.parts, at = [], 0
        rows = sum(new)
        self.q = torch.full((rows + extra_rows, Hq, 128), nan, dtype=torch.bfloat16)
        self.q[:rows] = (torch.randn(rows, Hq, 128, generator=g) * spread).to(torch.bfloat16)
        for s, (n, r) in enumerate(zip(keys, new)):
            k, v = ((torch.randn(n, H, 128, generator=g) * f).to(torch.bfloat16) for f in (spread, 1.0))
            mask = seen(list(range(n - r, n)), n, window, sinks)
            any_row = mask.any(0)
            k, v = (torch.where(any_row[:, None, None], x, torch.zeros_like(x)) for x in (k, v))
            for j in range(-(-n // bs)):
                b = ids.pop()
                here = any_row[j * bs:(j + 1) * bs]
                if not bool(here.any()):
                    continue
                bt[s, j] = b
                at_rows = torch.nonzero(here)[:, 0]
                kc[b, at_rows], vc[b, at_rows] = k[j * bs + at_rows], v[j * bs + at_rows]
            self.parts.append((slice(at, at + r), k, v, mask))
            at += r
        self.keys, self.new, self.Hq, self.H, self.bs, self.scale = keys, new, Hq, H, bs, scale
        self.window, self.sinks = window, sinks
        self.kc, self.vc, self.bt = kc.to(device), vc.to(device), bt.to(device)
        self.q_cpu, self.q = self.q, self.q.to(device)
        self.lens = torch.tensor(keys, dtype=torch.int32, device=device)
        self.cu = torch.tensor([0] + new).cumsum(0).to(torch.int32).to(device)
        self.rows = rows

    def check(self, out, lse, rounded=False, skip=()):
        out, lse = out.double().cpu(), lse.double().cpu()
        for s, (rows, k, v, mask) in enumerate(self.parts):
            if s in skip or rows.start == rows.stop:
                continue
            want, wl, tol, ltol = attend(self.q_cpu[rows], k, v, mask, self.scale, rounded)
            off, loff = (out[rows] - want).abs(), (lse[rows] - wl).abs()
            assert bool((off <= tol).all()), (s, float((off - tol).max()), float(off.max()))
            assert bool((loff <= ltol).all()), (s, float((loff - ltol).max()), float(loff.max()))
