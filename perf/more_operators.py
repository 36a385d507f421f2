"""The operators around and inside a serving engine's attention layer, as measured workloads: norms of
queries and keys for each head with the position rotation in the same pass, the same on the way into
the paged cache, decode attention under a sliding window with first tokens that stay visible (sinks),
and attention of chunks of new tokens over the paged cache.

``run`` takes either the plain form (elementary torch operations in 32 bits) or, with ``own`` set,
the calls of ``paged_kv_attention_22_gb300``; ``exact`` gives the same outputs in 64 bits.

A head's row x of 128 values, with weights w: y = w x / sqrt(mean(x^2) + eps). The first `rotary` dims
of y are rotated in pairs, (i, i + rotary / 2) or, interleaved, (2 i, 2 i + 1), by the token's position
times the pair's frequency base^(-2 i / rotary), which a scaling for long contexts changes.
"""
import math

import torch

own = False

D = 128  # head dim
DEV = "cuda"
BASE, EPS = 1.0e6, 1.0e-6
# YaRN: contexts four times as long as the 32,768 positions that the frequencies were made for
FACTOR, ORIGINAL, FAST, SLOW = 4.0, 32768, 32.0, 1.0


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the decode step of four sequences, queries and keys from one packed projection: latency
        dict(name="heads tiny", op="heads", tokens=4, heads=8, gqa=2, rotary=128, inter=False, norm=True, scaling="none"),
        # a prefill batch of 32,768 tokens, no norms, half of each head rotated in neighbouring pairs
        dict(name="heads prompts", op="heads", tokens=32768, heads=8, gqa=2, rotary=64, inter=True, norm=False, scaling="linear"),
        # a decode step of 64 sequences into the cache
        dict(name="append step", op="append", tokens=64, heads=8, gqa=2, rotary=128, inter=False, norm=True, scaling="none", block=256, pad=0),
        # a prefill batch of 32,768 tokens into the cache: bandwidth
        dict(name="append prompts", op="append", tokens=32768, heads=8, gqa=2, rotary=128, inter=False, norm=True, scaling="none", block=256, pad=0),
        # a padded batch for a long context, part of the head in neighbouring pairs, odd block size
        dict(name="append padded", op="append", tokens=5001, heads=2, gqa=4, rotary=96, inter=True, norm=True, scaling="yarn", block=48, pad=57),
        # four short sequences: the smallest decode call
        dict(name="sinks tiny", op="decode", seqs=4, lo=17, hi=128, heads=8, gqa=2, block=16, window=32, sinks=4, store=False),
        # 64 sequences at context 640 with the new token's rows stored by the call, window 256
        dict(name="sinks sweep", op="decode", seqs=64, lo=640, hi=640, heads=8, gqa=2, block=256, window=256, sinks=4, store=True),
        # 16 long streams: half of the context in the window, 128 first tokens
        dict(name="sinks long", op="decode", seqs=16, lo=16384, hi=16384, heads=8, gqa=2, block=256, window=8192, sinks=128, store=False),
        # five drafted tokens for each of 64 sequences at context 640
        dict(name="chunk drafts", op="chunk", seqs=64, lo=5, hi=5, clo=635, chi=635, heads=8, gqa=2, block=256, window=0, sinks=0),
        # sixteen new tokens on each of two long documents
        dict(name="chunk documents", op="chunk", seqs=2, lo=16, hi=16, clo=32752, chi=32752, heads=8, gqa=2, block=256, window=0, sinks=0),
        # a mixed batch, from single tokens to short prompts, over ragged contexts with window and sinks
        dict(name="chunk mixed", op="chunk", seqs=23, lo=1, hi=300, clo=0, chi=8193, heads=4, gqa=4, block=64, window=1000, sinks=20),
        # pieces of 2,048 tokens of four long prompts: bound by the products
        dict(name="chunk prompts", op="chunk", seqs=4, lo=2048, hi=2048, clo=8192, chi=8192, heads=8, gqa=2, block=256, window=0, sinks=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["heads", "append", "decode", "decode", "chunk", "chunk", "chunk"])
    c = dict(op=op, heads=rng.choice([1, 2, 3, 4, 8, 8]), gqa=rng.choice([1, 2, 4]))
    if op in ("heads", "append"):
        tokens = _log(rng, 1, 32768)
        c.update(tokens=tokens, rotary=rng.choice([0, 16, 32, 64, 80, 96, 128, 128]), inter=rng.choice([False, True]), norm=rng.choice([False, True, True]),
                 scaling=rng.choice(["none", "linear", "ntk", "yarn"]))
        if op == "append":
            c.update(block=rng.choice([16, 32, 48, 64, 256]), pad=rng.choice([0, 0, rng.randrange(0, tokens)]))
        return c
    c.update(block=rng.choice([16, 32, 48, 64, 256]), window=rng.choice([0, _log(rng, 1, 4096), _log(rng, 1, 4096)]), sinks=rng.choice([0, 1, 4, _log(rng, 1, 300)]))
    if op == "decode":
        seqs = _log(rng, 1, 64)
        hi = _log(rng, 2, min(16384, 262144 // seqs))
        return dict(c, seqs=seqs, lo=rng.choice([1, hi, rng.randrange(1, hi + 1)]), hi=hi, store=rng.choice([False, True]))
    seqs = _log(rng, 1, 32)
    hi = _log(rng, 1, min(2048, 8192 // seqs))
    chi = rng.choice([0, _log(rng, 1, min(16384, 131072 // seqs))])
    return dict(c, seqs=seqs, lo=rng.choice([1, hi, rng.randrange(1, hi + 1)]), hi=hi, clo=rng.choice([0, chi]), chi=chi)


def _lens(n, lo, hi, step=0.6180339887498949):
    """n lengths from lo to hi, spread in a fixed irregular order; the largest is hi."""
    return [hi if i == n - 1 else lo + int((hi - lo + 1) * ((i + 1) * step % 1.0)) for i in range(n)]


def _chunks(case):
    """(new tokens, keys) of every sequence of a chunk case."""
    new = _lens(case["seqs"], case["lo"], case["hi"])
    return new, [n + c for n, c in zip(new, _lens(case["seqs"], case["clo"], case["chi"], 0.4142135623730951))]


def _seen(at, window, sinks):
    """How many keys the query at position `at` sees."""
    first = max(0, at + 1 - window) if window else 0
    return at + 1 - first + min(sinks, first)


def work(case):
    H, Hq = case["heads"], case["heads"] * case["gqa"]
    if case["op"] == "heads":
        return {"bytes": case["tokens"] * (4 * D * (Hq + H) + 4), "flops": 8 * D * case["tokens"] * (Hq + H)}
    if case["op"] == "append":
        kept = case["tokens"] - case["pad"]
        return {"bytes": case["tokens"] * (4 * D * Hq + 8) + kept * 8 * D * H, "flops": 8 * D * (case["tokens"] * Hq + kept * H)}
    W, N = case["window"], case["sinks"]
    if case["op"] == "decode":
        lens = _lens(case["seqs"], case["lo"], case["hi"])
        keys = sum(_seen(n - 1, W, N) for n in lens)
        more = len(lens) * 8 * D * H if case["store"] else 0
        return {"bytes": keys * 4 * D * H + len(lens) * Hq * (4 * D + 4) + more, "flops": 4 * D * Hq * keys}
    keys, pairs, rows = 0, 0, 0
    for n, k in zip(*_chunks(case)):
        first = max(0, k - n + 1 - W) if W else 0  # of the earliest query
        keys += k - first + min(N, first)
        pairs += sum(_seen(p, W, N) for p in range(k - n, k))
        rows += n
    return {"bytes": keys * 4 * D * H + rows * Hq * (4 * D + 4), "flops": 4 * D * Hq * pairs}


# ------------------------------------------------------------------------------------------ inputs

def _rows(g, n, heads, outliers):
    """n token rows [n, heads, 128] bf16: normal, with channels of larger spread as keys have."""
    x = torch.randn(n, heads, D, generator=g, device=DEV)
    if outliers:
        x = x * (1.0 + 3.0 * (torch.rand(1, heads, D, generator=g, device=DEV) > 0.95))
    return x.to(torch.bfloat16)


def _tables(g, lens, bs, blocks):
    """Block tables of sequences of these lengths, ids drawn from the pool without repetition, -1 past the end."""
    width = -(-max(lens) // bs)
    ids = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    need = torch.tensor([-(-n // bs) for n in lens], device=DEV)
    start = need.cumsum(0) - need
    j = torch.arange(width, device=DEV)
    return torch.where(j < need[:, None], ids[(start[:, None] + j).clamp(max=blocks - 1)], -1).to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(int(seed))
    st = dict(case)
    H, Hq = case["heads"], case["heads"] * case["gqa"]
    st["scale"] = 1.0 / math.sqrt(D)
    if case["op"] in ("heads", "append"):
        T = case["tokens"]
        # one projection's output, of which queries, keys and values are views
        st["qkv"] = _rows(g, T, Hq + 2 * H, True)
        st["q"], st["k"], st["v"] = st["qkv"].split([Hq, H, H], 1)
        st["wq"], st["wk"] = ((1.0 + 0.3 * torch.randn(D, generator=g, device=DEV)).to(torch.bfloat16) if case["norm"] else None for _ in range(2))
        reach = 32768 if case["scaling"] == "none" else 131072
        first = torch.randint(0, reach, (1 + T // 512,), generator=g, device=DEV)  # sequences of 512 tokens or less
        i = torch.arange(T, device=DEV)
        st["pos"] = (first[i // 512] + i % 512).to(torch.int32)
        st["q_out"] = torch.empty(T, Hq, D, dtype=torch.bfloat16, device=DEV)
        if case["op"] == "heads":
            st["k_out"] = torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)
            return st
        bs = case["block"]
        blocks = -(-T // bs) + 2
        slots = torch.randperm(blocks * bs, generator=g, device=DEV)[:T]
        st["live"] = torch.randperm(T, generator=g, device=DEV)[: T - case["pad"]].sort().values  # the others are padding
        st["slots"] = torch.full((T,), -1, dtype=torch.int32, device=DEV)
        st["slots"][st["live"]] = slots[st["live"]].to(torch.int32)
        st["kc"], st["vc"] = (_rows(g, blocks * bs, H, False).view(blocks, bs, H, D) for _ in range(2))
        return st
    bs = case["block"]
    if case["op"] == "decode":
        keys = _lens(case["seqs"], case["lo"], case["hi"])
        rows = len(keys)
    else:
        new, keys = _chunks(case)
        rows = sum(new)
        st["max_q"] = max(new)
        st["cu_q"] = torch.tensor([0] + new, device=DEV).cumsum(0).to(torch.int32)
    blocks = sum(-(-n // bs) for n in keys) + 1
    st["kc"], st["vc"] = (_rows(g, blocks * bs, H, o).view(blocks, bs, H, D) for o in (True, False))
    st["bt"] = _tables(g, keys, bs, blocks)
    st["lens"] = torch.tensor(keys, dtype=torch.int32, device=DEV)
    st["max_k"] = max(keys)
    st["q"] = torch.randn(rows, Hq, D, generator=g, device=DEV).to(torch.bfloat16)
    if case.get("store"):
        st["k"], st["v"] = (_rows(g, rows, H, o) for o in (True, False))
        last = st["lens"].long() - 1
        st["slots"] = (st["bt"].long().gather(1, (last // bs)[:, None])[:, 0] * bs + last % bs).to(torch.int32)
    st["out"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty(rows, Hq, device=DEV)
    return st


# ------------------------------------------------------------------------------------------ plain forms

def _frequencies(st):
    """(frequency of each pair in radians a position, factor of the rotated dims), in 64 bits: far positions need them."""
    R = st["rotary"]
    i = torch.arange(R // 2, device=DEV, dtype=torch.float64)
    base = BASE * FACTOR ** (R / (R - 2)) if st["scaling"] == "ntk" else BASE
    f = base ** (-2.0 * i / R)
    if st["scaling"] == "linear":
        return f / FACTOR, 1.0
    if st["scaling"] != "yarn":
        return f, 1.0
    low, high = (R * math.log(ORIGINAL / (b * 2 * math.pi)) / (2 * math.log(BASE)) for b in (FAST, SLOW))
    low, high = max(math.floor(low), 0), min(math.ceil(high), R - 1)
    ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return f * (1 - ramp) + f / FACTOR * ramp, 0.1 * math.log(FACTOR) + 1.0


def _turned(x, w, st):
    """Rows x [T, heads, 128] normed with weights w (None: not normed) and rotated: bf16."""
    y = x.float()
    if w is not None:
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS) * w.float()
    R = st["rotary"]
    if R:
        f, factor = _frequencies(st)
        angle = st["pos"].double()[:, None] * f
        c, s = (t.float()[:, None] for t in (torch.cos(angle) * factor, torch.sin(angle) * factor))
        if st["inter"]:
            a, b = y[..., 0:R:2], y[..., 1:R:2]
            r = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
        else:
            a, b = y[..., : R // 2], y[..., R // 2: R]
            r = torch.cat([a * c - b * s, b * c + a * s], -1)
        y = torch.cat([r, y[..., R:]], -1)
    return y.to(torch.bfloat16)


def _plain_heads(st):
    return [_turned(st["q"], st["wq"], st), _turned(st["k"], st["wk"], st)]


def _plain_append(st):
    q, k = _plain_heads(st)
    at = st["slots"].long()[st["live"]]
    for cache, rows in ((st["kc"], k), (st["vc"], st["v"])):
        cache[at // st["block"], at % st["block"]] = rows[st["live"]]
    return [q, st["kc"], st["vc"]]


def _keys(st):
    """K and V of every sequence in logical order, padded to the longest: fp32 [S, P, heads, 128]."""
    p = torch.arange(st["max_k"], device=DEV)
    blk = st["bt"].long()[:, p // st["block"]].clamp(min=0)
    off = (p % st["block"]).expand_as(blk)
    return st["kc"][blk, off].float(), st["vc"][blk, off].float()


def _visible(at, n, st):
    """Whether the queries at positions `at` [S, R] see each key: [S, R, P]; n [S] keys."""
    p = torch.arange(st["max_k"], device=DEV)
    at = at[..., None]
    seen = (p <= at) & (p < n[:, None, None])
    if st["window"]:
        seen = seen & ((p > at - st["window"]) | (p < st["sinks"]))
    return seen


def _attend(q, k, v, seen, scale):
    """Softmax attention of q [S, H, G, R, 128] over k, v [S, P, H, 128] with the mask seen [S, R, P]: (out, lse)."""
    z = torch.matmul(q, k.permute(0, 2, 3, 1)[:, :, None]) * scale
    z = z.masked_fill(~seen[:, None, None], float("-inf"))
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e / total, v.permute(0, 2, 1, 3)[:, :, None])
    return out, (m + torch.log(total))[..., 0]


def _plain_decode(st):
    S, Hq = st["q"].shape[:2]
    H, G = st["heads"], st["gqa"]
    if st["store"]:
        at = st["slots"].long()
        for cache, rows in ((st["kc"], st["k"]), (st["vc"], st["v"])):
            cache[at // st["block"], at % st["block"]] = rows
    n = st["lens"].long()
    out, lse = _attend(st["q"].float().view(S, H, G, 1, D), *_keys(st), _visible(n[:, None] - 1, n, st), st["scale"])
    got = [out.reshape(S, Hq, D).to(torch.bfloat16), lse.reshape(S, Hq)]
    return got + ([st["kc"], st["vc"]] if st["store"] else [])


def _plain_chunk(st):
    Hq, H, G = st["q"].shape[1], st["heads"], st["gqa"]
    cu, n = st["cu_q"].long(), st["lens"].long()
    new = cu.diff()
    i = torch.arange(st["max_q"], device=DEV)
    rows = (cu[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][rows].float().view(*rows.shape, H, G, D).permute(0, 2, 3, 1, 4)
    at = (n - new)[:, None] + i.clamp(max=(new - 1)[:, None])  # rows past a segment's end repeat its last position
    out, lse = _attend(q, *_keys(st), _visible(at, n, st), st["scale"])
    # the row of `rows` that holds each token
    t = torch.arange(st["q"].shape[0], device=DEV)
    s = torch.searchsorted(cu[1:], t, right=True)
    j = t - cu[s]
    return [out.permute(0, 3, 1, 2, 4)[s, j].reshape(-1, Hq, D).to(torch.bfloat16), lse.permute(0, 3, 1, 2)[s, j].reshape(-1, Hq)]


# ------------------------------------------------------------------------------------------ the framework's calls

def _own(st):
    import paged_kv_attention_22_gb300 as pkv

    if st["op"] in ("heads", "append"):
        if "rope" not in st:  # made once, as for a model
            scaling = {"none": {}, "linear": dict(scaling="linear", factor=FACTOR), "ntk": dict(scaling="ntk", factor=FACTOR),
                       "yarn": dict(scaling="yarn", factor=FACTOR, original_positions=ORIGINAL, beta_fast=FAST, beta_slow=SLOW)}[st["scaling"]]
            st["rope"] = pkv.rope(st["rotary"], base=BASE, interleaved=st["inter"], **scaling)
        norms = dict(q_weight=st["wq"], k_weight=st["wk"], eps=EPS, q_out=st["q_out"])
        if st["op"] == "heads":
            return list(pkv.qk_norm_rope(st["q"], st["k"], st["rope"], st["pos"], k_out=st["k_out"], **norms))
        return [pkv.kv_append(st["q"], st["k"], st["v"], st["rope"], st["pos"], st["kc"], st["vc"], st["slots"], **norms), st["kc"], st["vc"]]
    sizes = (st["seqs"], st["q"].shape[1], st["heads"])
    rest = dict(out=st["out"], lse=st["lse"], sliding_window=st["window"], num_sinks=st["sinks"])
    if st["op"] == "chunk":
        if "ws" not in st:
            st["ws"] = pkv.new_chunk_workspace(*sizes)
        return list(pkv.paged_chunk_attn(st["q"], st["kc"], st["vc"], st["cu_q"], st["lens"], st["bt"], st["max_q"], st["max_k"], st["scale"], workspace=st["ws"], **rest))
    if "ws" not in st:
        st["ws"] = pkv.new_decode_workspace(*sizes, D, st["max_k"])
    if st["store"]:
        rest.update(k_new=st["k"], v_new=st["v"], slot_mapping=st["slots"])
    got = pkv.paged_decode_attn_sinks(st["q"], st["kc"], st["vc"], st["bt"], st["lens"], st["max_k"], st["scale"], workspace=st["ws"], **rest)
    return list(got) + ([st["kc"], st["vc"]] if st["store"] else [])


def run(st):
    if own:
        return _own(st)
    return {"heads": _plain_heads, "append": _plain_append, "decode": _plain_decode, "chunk": _plain_chunk}[st["op"]](st)


# ------------------------------------------------------------------------------------------ 64 bits

def _exact_turned(x, w, st):
    y = x.double()
    if w is not None:
        y = w.double() * y / (y.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt()
    R = st["rotary"]
    out = y.clone()
    low = high = 0.0
    if st["scaling"] == "yarn" and R:
        low = max(math.floor(R / 2 * math.log(ORIGINAL / (FAST * 2 * math.pi), BASE)), 0)
        high = min(math.ceil(R / 2 * math.log(ORIGINAL / (SLOW * 2 * math.pi), BASE)), R - 1)
    for i in range(R // 2):
        f = (BASE * FACTOR ** (R / (R - 2)) if st["scaling"] == "ntk" else BASE) ** (-2 * i / R)
        size = 1.0
        if st["scaling"] == "linear":
            f = f / FACTOR
        elif st["scaling"] == "yarn":
            keep = 1 - min(max((i - low) / max(high - low, 0.001), 0), 1)
            f, size = f * keep + f * (1 - keep) / FACTOR, 1 + 0.1 * math.log(FACTOR)
        a, b = (2 * i, 2 * i + 1) if st["inter"] else (i, i + R // 2)
        # the pair as a complex number, times the unit number of its angle
        z = torch.polar(torch.full_like(st["pos"], 1, dtype=torch.float64) * size, st["pos"].double() * f)[:, None] * torch.complex(y[..., a], y[..., b])
        out[..., a], out[..., b] = z.real, z.imag
    return out


def exact(case, seed):
    st = prepare(case, seed)
    H, G, W, N = case["heads"], case["gqa"], case.get("window", 0), case.get("sinks", 0)
    if case["op"] in ("heads", "append"):
        q, k = _exact_turned(st["q"], st["wq"], st), _exact_turned(st["k"], st["wk"], st)
        if case["op"] == "heads":
            return [q, k]
        kc, vc = st["kc"].double().flatten(0, 1), st["vc"].double().flatten(0, 1)
        there = st["slots"] >= 0
        kc[st["slots"][there].long()] = k[there]
        vc[st["slots"][there].long()] = st["v"][there].double()
        return [q, kc.view(st["kc"].shape), vc.view(st["vc"].shape)]
    kc, vc = st["kc"].double(), st["vc"].double()
    if case.get("store"):
        kc.flatten(0, 1)[st["slots"].long()] = st["k"].double()
        vc.flatten(0, 1)[st["slots"].long()] = st["v"].double()
    new, keys = _chunks(case) if case["op"] == "chunk" else ([1] * case["seqs"], _lens(case["seqs"], case["lo"], case["hi"]))
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(st["lse"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for s, (rows, total) in enumerate(zip(new, keys)):
        used = st["bt"][s, : -(-total // case["block"])].long()
        k, v = kc[used].flatten(0, 1)[:total], vc[used].flatten(0, 1)[:total]
        last = torch.arange(total - rows, total, device=DEV)[:, None]
        p = torch.arange(total, device=DEV)[None]
        hidden = p > last
        if W:
            hidden = hidden | ((p <= last - W) & (p >= N))
        for h in range(H * G):
            z = st["q"][at:at + rows, h].double() @ k[:, h // G].T * st["scale"]
            z[hidden] = float("-inf")
            lse[at:at + rows, h] = torch.logsumexp(z, 1)
            out[at:at + rows, h] = torch.exp(z - lse[at:at + rows, h, None]) @ v[:, h // G]
        at += rows
    return [out, lse] + ([kc, vc] if case.get("store") else [])
