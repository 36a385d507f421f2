"""The operators that make a KV cache smaller, as measured workloads: a paged cache held in 4 bits
(store, read back, decode, prefill) and eviction by accumulated attention weight (decode that
accumulates the weights, selection of the kept tokens, compaction of the cache).

``run`` takes either the plain form (elementary torch operations in 32 bits) or, with ``own`` set,
the calls of ``paged_kv_attention_22_gb300``; ``exact`` gives the same outputs in 64 bits.

The 4-bit cache: codes uint8 [blocks, kv heads, block size, 64], byte j of a row holding dims 2j
(low nibble) and 2j + 1 (high); params bf16 [blocks, kv heads, block size, 128 / group, 2], the
(scale, offset) of each group of dims. Code n stands for bf16(scale * (16 + n) + offset).
"""
import math

import torch

own = False

D = 128  # head dim
DEV = "cuda"


# ------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # a decode step's new tokens of 64 sequences, stored and read back: latency
        dict(name="store step", op="store", tokens=64, heads=8, block=256, group=32),
        # a prefill batch's K/V: 32,768 tokens, bandwidth
        dict(name="store prompts", op="store", tokens=32768, heads=8, block=256, group=32),
        # four short sequences: the smallest decode call
        dict(name="decode tiny", op="decode", seqs=4, lo=17, hi=128, heads=8, gqa=2, block=16, group=32, window=0),
        # 64 sequences at context 640: the batch of a decode sweep
        dict(name="decode sweep", op="decode", seqs=64, lo=640, hi=640, heads=8, gqa=2, block=256, group=32, window=0),
        # 16 long contexts: what a 4-bit cache is for
        dict(name="decode long", op="decode", seqs=16, lo=16384, hi=16384, heads=8, gqa=2, block=256, group=32, window=0),
        # ragged contexts under a sliding window, four query heads a KV head, one group a row
        dict(name="decode window", op="decode", seqs=23, lo=1, hi=8193, heads=8, gqa=4, block=64, group=128, window=1000),
        # short ragged prompts
        dict(name="prefill tiny", op="prefill", seqs=4, lo=9, hi=64, cached=0, heads=8, gqa=2, block=16, group=32, window=0),
        # 4,096 new tokens a sequence over a cached prefix of the same length
        dict(name="prefill cached", op="prefill", seqs=4, lo=4096, hi=4096, cached=4096, heads=8, gqa=2, block=256, group=32, window=0),
        # the sweep's decode step over a bf16 cache, accumulating each key's weight
        dict(name="weights sweep", op="weights", cache="bf16", seqs=64, lo=640, hi=640, heads=8, gqa=2, block=256, group=0, window=0),
        # the same over long contexts held in 4 bits
        dict(name="weights long q4", op="weights", cache="q4", seqs=8, lo=8193, hi=8193, heads=8, gqa=2, block=256, group=64, window=0),
        # a few short sequences cut to 48 tokens, 4-bit cache
        dict(name="evict tiny q4", op="evict", cache="q4", seqs=4, lo=40, hi=128, keep=48, recent=16, heads=8, block=16, group=32),
        # eight long sequences cut to a quarter, bf16 cache
        dict(name="evict long", op="evict", cache="bf16", seqs=8, lo=16384, hi=16384, keep=4096, recent=512, heads=8, block=256, group=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["store", "decode", "decode", "prefill", "weights", "evict"])
    c = dict(op=op, heads=rng.choice([1, 2, 3, 4, 8, 8]), block=rng.choice([16, 32, 48, 64, 256]), group=rng.choice([32, 64, 128]))
    if op == "store":
        return dict(c, tokens=_log(rng, 1, 32768))
    if op == "prefill":
        lo = _log(rng, 1, 1024)
        return dict(c, seqs=_log(rng, 1, 8), lo=lo, hi=min(2048, lo + rng.randrange(200)), cached=rng.choice([0, _log(rng, 1, 4096)]),
                    gqa=rng.choice([1, 2, 4]), window=rng.choice([0, 0, _log(rng, 1, 1024)]))
    seqs = _log(rng, 1, 64)
    hi = _log(rng, 2, min(16384, 262144 // seqs))
    lo = rng.choice([1, hi, rng.randrange(1, hi + 1)])
    if op == "evict":
        keep = rng.randrange(1, hi + 1)
        c = dict(c, seqs=seqs, lo=lo, hi=hi, keep=keep, recent=rng.randrange(0, keep + 1), cache=rng.choice(["q4", "bf16"]))
    else:
        c = dict(c, seqs=seqs, lo=lo, hi=hi, gqa=rng.choice([1, 2, 4]), window=rng.choice([0, 0, _log(rng, 1, 2048)]))
        if op == "weights":
            c["cache"] = rng.choice(["q4", "bf16"])
    if c.get("cache") == "bf16":
        c["group"] = 0
    return c


def _lens(n, lo, hi):
    """n lengths from lo to hi, spread in a fixed irregular order; the largest is hi."""
    return [hi if i == n - 1 else lo + int((hi - lo + 1) * ((i + 1) * 0.6180339887498949 % 1.0)) for i in range(n)]


def _row_bytes(group):
    """Bytes of one token's K (or V) row of one KV head."""
    return 2 * D if group == 0 else D // 2 + 4 * (D // group)


def work(case):
    H = case["heads"]
    row = _row_bytes(case["group"])
    if case["op"] == "store":
        T = case["tokens"]
        return {"bytes": 2 * T * H * (2 * 2 * D + 2 * row) + 8 * T, "flops": 2 * T * H * D * 8}
    n = _lens(case["seqs"], case["lo"], case["hi"])
    if case["op"] == "evict":
        kept = sum(min(x, case["keep"]) for x in n)
        back = kept * H * 2 * (row + 2 * D) if case["cache"] == "q4" else 0
        return {"bytes": 4 * sum(n) + kept * (4 + 8 + 4 * H * row) + back, "flops": sum(n)}
    W, Hq = case["window"], H * case["gqa"]
    if case["op"] == "prefill":
        k = [x + case["cached"] for x in n]
        seen = [min(c + i + 1, W) if W else c + i + 1 for x, c in zip(n, [case["cached"]] * len(n)) for i in range(x)]
        return {"bytes": sum(k) * 2 * H * row + sum(n) * Hq * (4 * D + 4), "flops": 4 * D * Hq * sum(seen)}
    keys = sum(min(x, W) if W else x for x in n)
    extra = 8 * keys if case["op"] == "weights" else 0
    return {"bytes": keys * 2 * H * row + len(n) * Hq * (4 * D + 4) + extra, "flops": 4 * D * Hq * keys}


# ------------------------------------------------------------------------------------------ inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _rows(g, n, heads, outliers):
    """n token rows [n, heads, 128] bf16: normal, with channels of larger spread as keys have."""
    x = torch.randn(n, heads, D, generator=g, device=DEV)
    if outliers:
        x = x * (1.0 + 3.0 * (torch.rand(1, heads, D, generator=g, device=DEV) > 0.95))
    return x.to(torch.bfloat16)


def _codes(x, group):
    """(codes, params) of rows x [..., 128]."""
    f = x.float().unflatten(-1, (D // group, group))
    lo, hi = f.amin(-1), f.amax(-1)
    span = (hi - lo) * (1.0 / 15.0)
    s = torch.where(span < 2.0 ** -100, 0.0, span).to(torch.bfloat16).float()
    b = (lo + 0.0 - 16.0 * s).to(torch.bfloat16).float()
    bad = ~torch.isfinite(hi - lo) | ~torch.isfinite(b)
    s, b = torch.where(bad, 0.0, s), torch.where(bad, float("nan"), b)
    t = (f - b[..., None]).double()
    n = torch.floor(t / s[..., None].double() + 0.5) - 16.0
    n = torch.where(s[..., None] == 0, 0.0, n.clamp(0, 15)).to(torch.uint8).flatten(-2)
    return n[..., 0::2] | (n[..., 1::2] << 4), torch.stack([s, b], -1).to(torch.bfloat16)


def _values(codes, params):
    """What rows of a 4-bit cache stand for, as fp32 (each value is a bf16)."""
    n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()
    group = D // params.shape[-2]
    s, b = params[..., 0].float(), params[..., 1].float()
    v = s.repeat_interleave(group, -1) * (n + 16.0) + b.repeat_interleave(group, -1)
    return v.to(torch.bfloat16).float()


def _pool(g, case, blocks):
    """K and V caches of `blocks` blocks filled with rows: two bf16 tensors [blocks, block, heads, 128], or two pairs (codes, params)."""
    H, bs = case["heads"], case["block"]
    made = []
    for outliers in (True, False):
        x = _rows(g, blocks * bs, H, outliers)
        if case["group"] == 0:
            made.append(x.view(blocks, bs, H, D))
            continue
        c, p = _codes(x, case["group"])
        made.append(tuple(y.unflatten(0, (blocks, bs)).transpose(1, 2).contiguous() for y in (c, p)))
    return made


def _tables(g, lens, bs, blocks):
    """Block tables of sequences of these lengths, ids drawn from the pool without repetition, -1 past the end."""
    width = -(-max(lens) // bs)
    ids = torch.randperm(blocks, generator=g, device=DEV).to(torch.int32)
    need = torch.tensor([-(-n // bs) for n in lens], device=DEV)
    start = need.cumsum(0) - need
    j = torch.arange(width, device=DEV)
    return torch.where(j < need[:, None], ids[(start[:, None] + j).clamp(max=blocks - 1)], -1).to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    H, bs = case["heads"], case["block"]
    st["scale"] = 1.0 / math.sqrt(D)
    if case["op"] == "store":
        T = case["tokens"]
        blocks = -(-T // bs) + 2
        st["k"], st["v"] = _rows(g, T, H, True), _rows(g, T, H, False)
        st["slots"] = torch.randperm(blocks * bs, generator=g, device=DEV)[:T].to(torch.int32)
        st["kc"], st["vc"] = [(torch.zeros(blocks, H, bs, D // 2, dtype=torch.uint8, device=DEV),
                               torch.zeros(blocks, H, bs, D // case["group"], 2, dtype=torch.bfloat16, device=DEV)) for _ in range(2)]
        return st
    lens = _lens(case["seqs"], case["lo"], case["hi"])
    keys = [n + case["cached"] for n in lens] if case["op"] == "prefill" else lens
    blocks = sum(-(-n // bs) for n in keys) + 1
    if case["op"] == "evict":
        # the kept rows go to fresh blocks of the same pool, as for sequences whose blocks are shared
        kept = [min(n, case["keep"]) for n in lens]
        more = sum(-(-n // bs) for n in kept)
        both = _tables(g, keys + [1] * more, bs, blocks + more)
        st["src"], fresh = both[: len(keys)].contiguous(), both[len(keys):, 0]
        width = -(-max(kept) // bs)
        need = torch.tensor([-(-n // bs) for n in kept], device=DEV)
        at = (need.cumsum(0) - need)[:, None] + torch.arange(width, device=DEV)
        st["dst"] = torch.where(torch.arange(width, device=DEV) < need[:, None], fresh[at.clamp(max=more - 1)], -1).to(torch.int32).contiguous()
        st["kc"], st["vc"] = _pool(g, case, blocks + more)
        # accumulated weights: a few keys hold most of the mass
        st["weights"] = torch.rand(len(keys), max(keys), generator=g, device=DEV) ** 8 * 50.0
        st["new_weights"] = torch.zeros(len(keys), case["keep"], device=DEV)
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        slots = st["dst"].long()[:, :, None] * bs + torch.arange(bs, device=DEV)
        slots = slots.flatten(1)[:, : case["keep"]]
        live = torch.arange(slots.shape[1], device=DEV) < torch.tensor(kept, device=DEV)[:, None]
        st["read"] = slots[live].to(torch.int32)
        return st
    st["kc"], st["vc"] = _pool(g, case, blocks)
    st["bt"] = _tables(g, keys, bs, blocks)
    rows = sum(lens) if case["op"] == "prefill" else len(lens)
    st["q"] = torch.randn(rows, H * case["gqa"], D, generator=g, device=DEV).to(torch.bfloat16)
    st["max_k"] = max(keys)
    if case["op"] == "prefill":
        st["max_q"], st["total_k"] = max(lens), sum(keys)
        st["cu_q"] = torch.tensor([0] + lens, device=DEV).cumsum(0).to(torch.int32)
        st["cu_k"] = torch.tensor([0] + keys, device=DEV).cumsum(0).to(torch.int32)
    else:
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    if case["op"] == "weights":
        st["weights"] = torch.zeros(len(keys), max(keys), device=DEV)
    st["out"] = torch.empty_like(st["q"])
    st["lse"] = torch.empty(rows, H * case["gqa"], device=DEV)
    return st


# ------------------------------------------------------------------------------------------ plain forms

def _slot_rows(cache, blk, off):
    """Rows at (block, offset) of a cache, as fp32 [..., heads, 128]."""
    if isinstance(cache, tuple):
        return _values(*(x.transpose(1, 2)[blk, off] for x in cache))
    return cache[blk, off].float()


def _keys(st):
    """K and V of every sequence in logical order, padded to the longest: fp32 [S, P, heads, 128]."""
    p = torch.arange(st["max_k"], device=DEV)
    blk = st["bt"].long()[:, p // st["block"]].clamp(min=0)
    off = (p % st["block"]).expand_as(blk)
    return _slot_rows(st["kc"], blk, off), _slot_rows(st["vc"], blk, off)


def _attend(q, k, v, seen, scale):
    """Softmax attention of q [S, H, G, R, 128] over k, v [S, P, H, 128] with the mask seen [S, R, P]: (out, lse, weights)."""
    kt = k.permute(0, 2, 3, 1)[:, :, None]
    z = torch.matmul(q, kt) * scale
    z = z.masked_fill(~seen[:, None, None], float("-inf"))
    m = z.amax(-1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(-1, keepdim=True)
    e = e / total
    v = torch.where(seen.any(1)[..., None, None], v, 0.0)
    out = torch.matmul(e, v.permute(0, 2, 1, 3)[:, :, None])
    return out, (m + torch.log(total))[..., 0], e


def _plain_store(st):
    blk, off = st["slots"].long() // st["block"], st["slots"].long() % st["block"]
    back = []
    for x, cache in ((st["k"], st["kc"]), (st["v"], st["vc"])):
        for to, new in zip(cache, _codes(x, st["group"])):
            to.transpose(1, 2)[blk, off] = new
        back.append(_slot_rows(cache, blk, off).to(torch.bfloat16))
    return back


def _plain_decode(st):
    S, Hq = st["q"].shape[:2]
    H, G = st["heads"], st["gqa"]
    k, v = _keys(st)
    p = torch.arange(st["max_k"], device=DEV)
    n = st["lens"][:, None]
    seen = p < n
    if st["window"]:
        seen = seen & (p >= n - st["window"])
    out, lse, e = _attend(st["q"].float().view(S, H, G, 1, D), k, v, seen[:, None], st["scale"])
    got = [out.reshape(S, Hq, D).to(torch.bfloat16), lse.reshape(S, Hq)]
    if st["op"] == "weights":
        st["weights"] += e.sum((1, 2, 3))
        got.append(st["weights"])
    return got


def _plain_prefill(st):
    Hq, H, G = st["q"].shape[1], st["heads"], st["gqa"]
    k, v = _keys(st)
    cu_q, n_k = st["cu_q"].long(), st["cu_k"].long().diff()
    n_q = cu_q.diff()
    i = torch.arange(st["max_q"], device=DEV)
    rows = (cu_q[:-1, None] + i).clamp(max=st["q"].shape[0] - 1)
    q = st["q"][rows].float().view(rows.shape[0], st["max_q"], H, G, D).permute(0, 2, 3, 1, 4)
    at = (n_k - n_q)[:, None] + i  # each query's position
    p = torch.arange(st["max_k"], device=DEV)
    seen = p <= at[..., None]
    if st["window"]:
        seen = seen & (p > at[..., None] - st["window"])
    seen = seen & (p < n_k[:, None, None])
    out, lse, _ = _attend(q, k, v, seen, st["scale"])
    live = i < n_q[:, None]
    return [out.permute(0, 3, 1, 2, 4).reshape(*rows.shape, Hq, D)[live].to(torch.bfloat16), lse.permute(0, 3, 1, 2).reshape(*rows.shape, Hq)[live]]


def _plain_evict(st):
    B, R, bs = st["keep"], st["recent"], st["block"]
    w, n = st["weights"], st["lens"].long()[:, None]
    p = torch.arange(w.shape[1], device=DEV)
    # the last R positions first, then by weight, ties by position
    rank = torch.where(p < n, torch.where(p >= n - R, float("inf"), w), float("-inf"))
    keep = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :B]
    j = torch.arange(keep.shape[1], device=DEV)
    new = n.clamp(max=B)
    keep = torch.where(j < new, keep, w.shape[1]).sort(1).values
    live = j < new
    keep_out = torch.full((keep.shape[0], B), -1, dtype=torch.int32, device=DEV)
    keep_out[:, : keep.shape[1]] = torch.where(live, keep, -1).to(torch.int32)
    s = torch.arange(keep.shape[0], device=DEV)[:, None].expand_as(keep)[live]
    src, to = keep[live], j.expand_as(keep)[live]
    a, b = st["src"].long()[s, src // bs], st["dst"].long()[s, to // bs]
    st["new_weights"][s, to] = w[s, src]
    for cache in (st["kc"], st["vc"]):
        for x in (y.transpose(1, 2) for y in cache) if isinstance(cache, tuple) else (cache,):
            x[b, to % bs] = x[a, src % bs]
    got = [keep_out, new[:, 0].to(torch.int32), st["new_weights"]]
    if not isinstance(st["kc"], tuple):
        return got + [st["kc"], st["vc"]]
    blk, off = st["read"].long() // bs, st["read"].long() % bs
    return got + [_slot_rows(c, blk, off).to(torch.bfloat16) for c in (st["kc"], st["vc"])]


# ------------------------------------------------------------------------------------------ the framework's calls

def _own(st):
    import paged_kv_attention_22_gb300 as pkv

    op = st["op"]
    if op == "store":
        pkv.kv_store_q4(st["k"], st["v"], st["kc"], st["vc"], st["slots"])
        return pkv.kv_load_q4(st["kc"], st["vc"], st["slots"])
    if op == "evict":
        q4 = isinstance(st["kc"], tuple)
        keep, new = pkv.evict_select(st["weights"], st["lens"], st["keep"], st["recent"])
        compact = pkv.evict_compact_q4 if q4 else pkv.evict_compact
        compact(st["kc"], st["vc"], st["src"], st["dst"], keep, new, key_scores=st["weights"], dst_key_scores=st["new_weights"])
        got = [keep, new, st["new_weights"]]
        return got + (list(pkv.kv_load_q4(st["kc"], st["vc"], st["read"])) if q4 else [st["kc"], st["vc"]])
    if op == "prefill":
        if "ws" not in st:
            st["ws"] = pkv.new_q4_prefill_workspace(st["seqs"], st["total_k"], st["max_k"], st["heads"])
        return list(pkv.paged_prefill_attn_q4(st["q"], st["kc"], st["vc"], st["cu_q"], st["cu_k"], st["bt"], st["max_q"], st["max_k"], st["total_k"],
                                              st["scale"], out=st["out"], lse=st["lse"], workspace=st["ws"], sliding_window=st["window"]))
    scores = st["weights"] if op == "weights" else None
    sizes = (st["seqs"], st["q"].shape[1], st["heads"], st["max_k"])
    rest = dict(out=st["out"], lse=st["lse"], sliding_window=st["window"])
    if isinstance(st["kc"], tuple):
        if "ws" not in st:
            st["ws"] = pkv.new_q4_decode_workspace(*sizes, with_scores=scores is not None)
        got = pkv.paged_decode_attn_q4(st["q"], st["kc"], st["vc"], st["bt"], st["lens"], st["max_k"], st["scale"], key_scores=scores, workspace=st["ws"], **rest)
    else:
        if "ws" not in st:
            st["ws"] = pkv.new_decode_scores_workspace(*sizes)
        got = pkv.paged_decode_attn_scores(st["q"], st["kc"], st["vc"], st["bt"], st["lens"], st["max_k"], st["scale"], scores, workspace=st["ws"], **rest)
    return list(got) + ([scores] if op == "weights" else [])


def run(st):
    if own:
        return _own(st)
    return {"store": _plain_store, "decode": _plain_decode, "weights": _plain_decode, "prefill": _plain_prefill, "evict": _plain_evict}[st["op"]](st)


# ------------------------------------------------------------------------------------------ 64 bits

def _exact_values(codes, params):
    """Rows of a 4-bit cache in 64 bits; each value is rounded to bf16, as its definition says."""
    out = torch.empty(*codes.shape[:-1], D, dtype=torch.float64, device=codes.device)
    out[..., 0::2], out[..., 1::2] = (codes % 16).double(), torch.div(codes, 16, rounding_mode="floor").double()
    size = D // params.shape[-2]
    for i in range(params.shape[-2]):
        s, b = params[..., i, 0:1].double(), params[..., i, 1:2].double()
        out[..., i * size:(i + 1) * size] = s * (16 + out[..., i * size:(i + 1) * size]) + b
    return out.to(torch.bfloat16).double()


def _exact_seq(st, cache, s, n):
    """The first n rows of sequence s [n, heads, 128] in 64 bits."""
    rows = []
    for j in range(-(-n // st["block"])):
        b = int(st["bt"][s, j])
        if isinstance(cache, tuple):
            rows.append(_exact_values(cache[0][b], cache[1][b]).transpose(0, 1))
        else:
            rows.append(cache[b].double())
    return torch.cat(rows)[:n]


def _exact_store(st):
    back = []
    for x in (st["k"], st["v"]):
        got = torch.empty(x.shape, dtype=torch.float64, device=x.device)
        for i in range(0, D, st["group"]):
            f = x[..., i:i + st["group"]].double()
            low, high = f.min(-1, keepdim=True).values, f.max(-1, keepdim=True).values
            s = ((high - low) / 15).to(torch.bfloat16).double()
            b = (low - 16 * s).to(torch.bfloat16).double()
            n = ((f - b) / s + 0.5).floor().clamp(16, 31)
            got[..., i:i + st["group"]] = (torch.where(s > 0, n, torch.full_like(n, 16)) * s + b).to(torch.bfloat16).double()
        back.append(got)
    return back


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "store":
        return _exact_store(st)
    if case["op"] == "evict":
        return _exact_evict(st, case)
    H, G, W = case["heads"], case["gqa"], case["window"]
    lens = _lens(case["seqs"], case["lo"], case["hi"])
    more = case["cached"] if case["op"] == "prefill" else 0
    out = torch.empty(st["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.empty(st["lse"].shape, dtype=torch.float64, device=DEV)
    weights = torch.zeros(len(lens), max(lens), dtype=torch.float64, device=DEV)
    at = 0
    for s, n in enumerate(lens):
        rows = n if case["op"] == "prefill" else 1
        total = n + more
        k, v = (_exact_seq(st, c, s, total) for c in (st["kc"], st["vc"]))
        last = torch.arange(total - rows, total, device=DEV)[:, None]
        p = torch.arange(total, device=DEV)[None]
        hidden = (p > last) | (p <= last - W) if W else p > last
        for h in range(H * G):
            z = st["q"][at:at + rows, h].double() @ k[:, h // G].T * st["scale"]
            z[hidden] = float("-inf")
            lse[at:at + rows, h] = torch.logsumexp(z, 1)
            a = torch.exp(z - lse[at:at + rows, h, None])
            out[at:at + rows, h] = a @ v[:, h // G]
            if case["op"] == "weights":
                weights[s, :n] += a[0]
        at += rows
    return [out, lse] + ([weights] if case["op"] == "weights" else [])


def _exact_evict(st, case):
    B, R, bs = case["keep"], case["recent"], case["block"]
    new_w = st["new_weights"].double()
    caches = [tuple(x.clone() for x in c) if isinstance(c, tuple) else c.clone() for c in (st["kc"], st["vc"])]
    for s, n in enumerate(_lens(case["seqs"], case["lo"], case["hi"])):
        w = st["weights"][s, :n].tolist()
        kept = sorted(sorted(range(n - min(R, n)), key=lambda p: (-w[p], p))[:max(0, min(B, n) - min(R, n))] + list(range(n - min(R, n), n)))
        i = torch.arange(len(kept), device=DEV)
        at = torch.tensor(kept, device=DEV)
        new_w[s, : len(kept)] = st["weights"][s][at].double()
        a, b = st["src"][s].long()[at // bs], st["dst"][s].long()[i // bs]
        for old, new in zip((st["kc"], st["vc"]), caches):
            if isinstance(old, tuple):
                for x, y in zip(old, new):
                    y[b, :, i % bs] = x[a, :, at % bs]
            else:
                new[b, i % bs] = old[a, at % bs]
    if case["cache"] == "q4":
        blk, off = st["read"].long() // bs, st["read"].long() % bs
        caches = [_exact_values(c[0][blk, :, off], c[1][blk, :, off]) for c in caches]
    return [None, None, new_w] + caches
