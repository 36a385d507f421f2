"""Plain 64-bit implementations for the tests of the 4-bit cache and of eviction,
written from the definitions in include/pkv.h, and the tolerances that the
kernels' roundings allow. bf16 arrays are torch tensors on the CPU."""
import math

import torch

D = 128
U16 = torch.finfo(torch.bfloat16).eps / 2   # 2^-8: half a step of a bf16, relative
U32 = torch.finfo(torch.float32).eps / 2    # 2^-24


def quantise(x, group):
    """(codes [..., 64] uint8, params [..., 128 / group, 2] bf16) of rows x [..., 128] bf16."""
    f = x.float().reshape(*x.shape[:-1], D // group, group)
    lo, hi = f.amin(-1), f.amax(-1)          # NaN if the group holds one
    span = (hi - lo) * torch.tensor(1.0 / 15.0, dtype=torch.float32)
    scale = torch.where(span < 2.0 ** -100, torch.zeros_like(span), span).to(torch.bfloat16).float()
    offset = ((lo + 0.0) - 16.0 * scale).to(torch.bfloat16).float()
    bad = ~torch.isfinite(hi - lo) | ~torch.isfinite(offset)
    scale[bad], offset[bad] = 0.0, float("nan")
    t = (f - offset[..., None]).double()     # the definition's fp32 difference
    n = torch.floor(t / scale[..., None].double() + 0.5) - 16
    n = torch.where(scale[..., None] == 0, torch.zeros_like(n), n.clamp(0, 15)).to(torch.uint8)
    n = n.reshape(*x.shape)
    return n[..., 0::2] + 16 * n[..., 1::2], torch.stack([scale, offset], -1).to(torch.bfloat16)


def values(codes, params):
    """The bf16 values that rows stand for, as float64 [..., 128]."""
    n = torch.empty(*codes.shape[:-1], D, dtype=torch.float64)
    n[..., 0::2], n[..., 1::2] = (codes & 15).double(), (codes >> 4).double()
    group = D // params.shape[-2]
    s, b = (params[..., i].double().repeat_interleave(group, -1) for i in (0, 1))
    # 13 significant bits of s (16 + n) and 8 of b: float32 holds the sum exactly
    return (s * (16 + n) + b).float().to(torch.bfloat16).double()


def attend(q, k, v, scale, first, last):
    """Attention of one head's query rows q [R, 128] over k, v [P, 128] (float64),
    row r seeing keys first[r] .. last[r]. Returns (out, lse, weights [R, P],
    sum of weight |v|, largest sum |q k| scale)."""
    z = q @ k.T * scale
    p = torch.arange(k.shape[0])
    hidden = (p < torch.as_tensor(first)[:, None]) | (p > torch.as_tensor(last)[:, None])
    z = z.masked_fill(hidden, -math.inf)
    lse = torch.logsumexp(z, 1)
    w = torch.exp(z - lse[:, None])
    absq = (q.abs() @ k.abs().T * abs(scale)).masked_fill(hidden, 0.0)
    return w @ v, lse, w, w @ v.abs(), absq.amax(1)


def out_tolerance(out, weight_abs_v):
    """Each probability is rounded to bf16 (U16, relative) and the output divided
    by the sum of the rounded ones: a weight is off by at most 2 U16. The output
    is rounded once more. The fp32 arithmetic in between (exponentials good to
    2^-20, sums) stays below 2^-12 of the weighted magnitudes."""
    return (2 * U16 * (1 + U16) + 2.0 ** -12) * weight_abs_v + U16 * out.abs() + 1e-30


def lse_tolerance(lse, abs_qk, adds):
    """A logit sums 128 exact products in fp32 (128 steps of at most 2 U32 of their
    magnitudes: the tensor core may truncate); the sum of the exponentials has at
    most adds + 64 additions in a row; 2^-20 covers the exponential and the
    logarithm, relative to 1 + |lse|."""
    return 256 * U32 * abs_qk + (adds + 64) * U32 + 2.0 ** -20 * (1 + lse.abs())


class Cache:
    """A paged 4-bit cache whose unused rows hold poison (codes 255, parameters
    NaN), with sequences of the given lengths in blocks drawn at random."""

    def __init__(self, seed, lens, heads, block, group, spare=2, outliers=0.0, shared=0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.heads, self.block, self.group = list(lens), heads, block, group
        need = [-(-n // block) for n in self.lens]
        self.num_blocks = sum(need) + spare
        ids = torch.randperm(self.num_blocks, generator=g).tolist()
        width = max(max(need), 1)
        self.tables = torch.full((len(need), width), -1, dtype=torch.int32)
        for s, n in enumerate(need):
            for j in range(n):
                # the first `shared` blocks are sequence 0's in every table
                own = s > 0 and j < shared and j < need[0]
                self.tables[s, j] = self.tables[0, j] if own else ids.pop()
        shape = (self.num_blocks, heads, block)
        self.k = self._rows(g, shape, outliers)
        self.v = self._rows(g, shape, 0.0)
        used = torch.zeros(self.num_blocks, block, dtype=torch.bool)
        for s, n in enumerate(self.lens):
            for p in range(n):
                used[self.tables[s, p // block], p % block] = True
        for codes, params in (self.k, self.v):
            codes[~used[:, None].expand(shape)] = 255
            params[~used[:, None].expand(shape)] = float("nan")

    def _rows(self, g, shape, outliers):
        x = torch.randn(*shape, D, generator=g)
        if outliers:
            x *= 1 + 7 * (torch.rand(shape, generator=g) < outliers)[..., None]
        return quantise(x.to(torch.bfloat16), self.group)

    def logical(self, cache, s, n, head):
        """The values of the first n rows of sequence s, float64 [n, 128]."""
        p = torch.arange(n)
        blk = self.tables[s].long()[p // self.block]
        return values(cache[0][blk, head, p % self.block], cache[1][blk, head, p % self.block])

    def cuda(self):
        """(k_cache, v_cache, block_tables) on the GPU."""
        return (tuple(x.cuda() for x in self.k), tuple(x.cuda() for x in self.v), self.tables.cuda())
