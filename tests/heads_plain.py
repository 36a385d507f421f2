"""Plain 64-bit norm and position rotation of heads, and how far a call may be off it."""
import math

import torch


def frequencies(R, base, scaling=None, factor=1.0, original=0, fast=32.0, slow=1.0):
    """(radians a position of each pair, magnitude), from the formulas of pkv.h."""
    if scaling == "ntk" and R:
        base = base * factor ** (R / (R - 2))
    f = [base ** (-2 * i / R) for i in range(R // 2)]
    if scaling == "linear":
        f = [x / factor for x in f]
    if scaling != "yarn":
        return f, 1.0
    d = [R * math.log(original / (2 * math.pi * b)) / (2 * math.log(base)) for b in (fast, slow)]
    lo, hi = max(math.floor(d[0]), 0), min(math.ceil(d[1]), R - 1)
    ramp = [min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0) for i in range(R // 2)]
    return [x * (1 - r) + x / factor * r for x, r in zip(f, ramp)], 0.1 * math.log(factor) + 1.0


def turned(x, w, pos, R, freqs=(), magnitude=1.0, interleaved=False, eps=1e-6):
    """(rows, tolerance) of x [T, heads, 128] normed with w (None: not) and rotated, in 64 bits.

    A call rounds its result once, to bf16: 2^-8 of it. Before that it works in fp32: the sum of 128
    squares is off by 128 roundings of 2^-24 at most and its inverse root by half of that, 2^-18; the
    root, the products, the angle (2^-25 of half a turn) and its sine and cosine by some 2^-21 together:
    2^-17 of a pair's two values covers them. An angle here and there is off by 2^-53 of its size and
    by 2^-54 turns a position: pos 2^-50."""
    y = x.double().cpu()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double().cpu()
    size = y.abs()
    if R:
        t = pos.double().cpu()[:, None, None] * torch.tensor(list(freqs), dtype=torch.float64)
        c, s = torch.cos(t) * magnitude, torch.sin(t) * magnitude
        a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
        ya, yb = y[..., a].clone(), y[..., b].clone()
        y, size = y.clone(), size.clone()
        y[..., a], y[..., b] = ya * c - yb * s, yb * c + ya * s
        size[..., a] = size[..., b] = (ya.abs() + yb.abs()) * abs(magnitude)
    far = pos.double().cpu().abs()[:, None, None] * 2.0 ** -50 if R else 0.0
    return y, 2.0 ** -8 * y.abs() + size * (2.0 ** -17 + far) * (1 + 2.0 ** -8)
