"""The 4-bit cache: quantising store, read-back, decode and prefill, against the
plain 64-bit implementation in q4_plain.py; and the refusals of each call."""
import ctypes
import math
import os
import subprocess
import threading

import pytest
import torch

import paged_kv_attention_22_gb300 as pkv
import q4_plain as Q
from paged_kv_attention_22_gb300 import build as pkv_build

SCALE = 1.0 / math.sqrt(128)


@pytest.fixture(scope="module")
def L():
    pkv_build.build()
    return pkv.lib()


# ------------------------------------------------------------------ CPU: the plain form and refusals

def test_plain_values_are_within_half_a_scale():
    g = torch.Generator().manual_seed(1)
    for group in (32, 64, 128):
        x = (torch.randn(500, 128, generator=g) * torch.exp(3 * torch.randn(500, 1, generator=g))
             + torch.randn(500, 1, generator=g)).to(torch.bfloat16)
        codes, params = Q.quantise(x, group)
        back = Q.values(codes, params)
        s = params[..., 0].double().repeat_interleave(group, -1)
        b = params[..., 1].double().repeat_interleave(group, -1)
        # half a scale; the scale's rounding moves the top code by 15 U16 s, the
        # offset's the whole grid by U16 |offset|, both only where codes clamp;
        # the result is rounded once
        tol = 0.5 * s + 15 * Q.U16 * s + Q.U16 * b.abs() + Q.U16 * back.abs()
        assert bool(((back - x.double()).abs() <= tol * (1 + 1e-6)).all())


FAKE = 0x10000


def _store(L, **kw):
    a = dict(k=FAKE, v=FAKE, kc=FAKE, kp=FAKE, vc=FAKE, vp=FAKE, sm=FAKE, T=4, H=8, D=128, gs=32, bs=16, NB=64)
    a.update(kw)
    return L.pkv_kv_store_q4(a["k"], a["v"], a["kc"], a["kp"], a["vc"], a["vp"], a["sm"], a["T"], a["H"], a["D"],
                             a["gs"], a["bs"], a["NB"], None)


def _load(L, **kw):
    a = dict(k=FAKE, v=FAKE, kc=FAKE, kp=FAKE, vc=FAKE, vp=FAKE, sm=FAKE, T=4, H=8, D=128, gs=32, bs=16, NB=64)
    a.update(kw)
    return L.pkv_kv_load_q4(a["kc"], a["kp"], a["vc"], a["vp"], a["sm"], a["k"], a["v"], a["T"], a["H"], a["D"],
                            a["gs"], a["bs"], a["NB"], None)


@pytest.mark.parametrize("call", [_store, _load])
def test_row_calls_refuse(L, call):
    for null in ("k", "v", "kc", "kp", "vc", "vp", "sm"):
        assert call(L, **{null: None}) == pkv.PKV_ERR_INVALID_ARG
    for odd in ("k", "v", "kc", "kp", "vc", "vp"):
        assert call(L, **{odd: FAKE + 8}) == pkv.PKV_ERR_INVALID_ARG
    assert call(L, T=-1) == pkv.PKV_ERR_INVALID_ARG
    assert call(L, NB=0) == pkv.PKV_ERR_INVALID_ARG
    assert call(L, D=64) == pkv.PKV_ERR_UNSUPPORTED
    assert call(L, gs=16) == pkv.PKV_ERR_UNSUPPORTED
    assert call(L, NB=1 << 40) == pkv.PKV_ERR_UNSUPPORTED
    assert call(L, T=0, k=None, v=None, sm=None) == pkv.PKV_OK


def _decode(L, **kw):
    a = dict(q=FAKE, kc=FAKE, kp=FAKE, vc=FAKE, vp=FAKE, bt=FAKE, mb=4, cl=FAKE, mcl=64, S=2, Hq=16, Hkv=8, D=128,
             gs=32, bs=16, NB=64, scale=0.088, win=0, out=FAKE, lse=None, ks=None, ld=0, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return L.pkv_paged_decode_attn_q4(a["q"], a["kc"], a["kp"], a["vc"], a["vp"], a["bt"], a["mb"], a["cl"], a["mcl"],
                                      a["S"], a["Hq"], a["Hkv"], a["D"], a["gs"], a["bs"], a["NB"], a["scale"],
                                      a["win"], a["out"], a["lse"], a["ks"], a["ld"], a["ws"], a["wsb"], None)


def test_decode_refuses(L):
    for null in ("q", "kc", "kp", "vc", "vp", "bt", "cl", "out"):
        assert _decode(L, **{null: None}) == pkv.PKV_ERR_INVALID_ARG
    for odd in ("q", "kc", "kp", "vc", "vp", "out", "ws"):
        assert _decode(L, **{odd: FAKE + 8}) == pkv.PKV_ERR_INVALID_ARG
    assert _decode(L, S=0) == pkv.PKV_ERR_INVALID_ARG
    assert _decode(L, mcl=0) == pkv.PKV_ERR_INVALID_ARG
    assert _decode(L, scale=float("inf")) == pkv.PKV_ERR_INVALID_ARG
    assert _decode(L, win=-1) == pkv.PKV_ERR_INVALID_ARG
    assert _decode(L, ks=FAKE, ld=63) == pkv.PKV_ERR_INVALID_ARG
    assert _decode(L, ws=None) == pkv.PKV_ERR_WORKSPACE_TOO_SMALL
    assert _decode(L, D=64) == pkv.PKV_ERR_UNSUPPORTED
    assert _decode(L, gs=48) == pkv.PKV_ERR_UNSUPPORTED
    assert _decode(L, bs=24) == pkv.PKV_ERR_UNSUPPORTED
    assert _decode(L, Hq=24) == pkv.PKV_ERR_UNSUPPORTED      # 3 query heads a KV head
    assert _decode(L, Hq=128) == pkv.PKV_ERR_UNSUPPORTED     # 16
    assert _decode(L, Hq=12) == pkv.PKV_ERR_UNSUPPORTED
    assert _decode(L, S=65536) == pkv.PKV_ERR_UNSUPPORTED
    assert _decode(L, NB=1 << 40) == pkv.PKV_ERR_UNSUPPORTED
    assert _decode(L, mcl=(1 << 30) + 1) == pkv.PKV_ERR_UNSUPPORTED
    assert _decode(L, S=65535, mcl=1 << 30, ks=FAKE, ld=1 << 30) == pkv.PKV_ERR_UNSUPPORTED
    assert L.pkv_decode_q4_workspace_size(65535, 16, 8, 128, 1 << 30, 1) == 0
    assert L.pkv_decode_q4_workspace_size(0, 16, 8, 128, 64, 0) == 0
    assert L.pkv_decode_q4_workspace_size(2, 12, 8, 128, 64, 0) == 0
    assert L.pkv_decode_q4_workspace_size(2, 16, 8, 64, 64, 0) == 0


def test_prefill_refuses(L):
    def call(**kw):
        a = dict(q=FAKE, kc=FAKE, kp=FAKE, vc=FAKE, vp=FAKE, cq=FAKE, ck=FAKE, bt=FAKE, mb=4, S=2, T=100, TK=128,
                 mq=64, mk=64, Hq=16, Hkv=8, D=128, gs=32, bs=16, NB=64, scale=0.088, win=0, out=FAKE, ws=FAKE,
                 wsb=1 << 30)
        a.update(kw)
        return L.pkv_paged_prefill_attn_q4(a["q"], a["kc"], a["kp"], a["vc"], a["vp"], a["cq"], a["ck"], a["bt"],
                                           a["mb"], a["S"], a["T"], a["TK"], a["mq"], a["mk"], a["Hq"], a["Hkv"],
                                           a["D"], a["gs"], a["bs"], a["NB"], a["scale"], a["win"], a["out"], None,
                                           a["ws"], a["wsb"], None)
    for null in ("q", "kc", "kp", "vc", "vp", "cq", "ck", "bt", "out"):
        assert call(**{null: None}) == pkv.PKV_ERR_INVALID_ARG
    for odd in ("q", "kc", "kp", "vc", "vp", "out", "ws"):
        assert call(**{odd: FAKE + 8}) == pkv.PKV_ERR_INVALID_ARG
    assert call(mq=65) == pkv.PKV_ERR_INVALID_ARG
    assert call(TK=-1) == pkv.PKV_ERR_INVALID_ARG
    assert call(win=-1) == pkv.PKV_ERR_INVALID_ARG
    assert call(Hq=64) == pkv.PKV_ERR_UNSUPPORTED            # 8 query heads a KV head
    assert call(S=65536) == pkv.PKV_ERR_UNSUPPORTED
    assert call(TK=2 ** 31 - 1, S=65535) == pkv.PKV_ERR_UNSUPPORTED
    assert call(wsb=1 << 10) == pkv.PKV_ERR_WORKSPACE_TOO_SMALL
    assert call(ws=None) == pkv.PKV_ERR_WORKSPACE_TOO_SMALL
    assert call(T=0, q=None, out=None) == pkv.PKV_OK
    assert call(S=0) == pkv.PKV_OK
    assert L.pkv_prefill_q4_workspace_size(2, 128, 64, 8, 64) == 0
    need = L.pkv_prefill_q4_workspace_size(2, 128, 64, 8, 128)   # depends on the device's SM count
    assert need >= 128 * 512 * 8 if torch.cuda.is_available() else need == 0


@pytest.mark.skipif(torch.cuda.is_available(), reason="only meaningful without a GPU")
def test_valid_calls_without_gpu_report_cuda_errors(L):
    assert _decode(L) == pkv.PKV_ERR_CUDA
    assert _store(L) == pkv.PKV_ERR_CUDA


def test_binding_refuses_shapes_and_types():
    k = torch.zeros(1, 1, 128, dtype=torch.bfloat16)
    sm = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(TypeError):
        pkv.kv_store_q4(k.tolist(), k, k, k, sm)                         # not a tensor
    with pytest.raises(TypeError):
        pkv.kv_store_q4(k.float(), k, k, k, sm)                          # not bf16
    with pytest.raises(TypeError):
        pkv.paged_decode_attn_q4(k, k, k, sm, sm, 1, 1.0, k, sm, sm)     # caches that are not pairs
    with pytest.raises(ValueError):
        pkv.kv_store_q4(k, k, pkv.new_q4_cache(1, 16, 1, device="cpu"),  # CPU tensors
                        pkv.new_q4_cache(1, 16, 1, device="cpu"), sm)
    with pytest.raises(ValueError):
        pkv.new_q4_cache(1, 16, 1, group_size=16, device="cpu")


# ------------------------------------------------------------------ GPU: rows

gpu = pytest.mark.gpu


def _special_rows(heads):
    """Rows where quantisation can go wrong."""
    g = torch.Generator().manual_seed(9)
    base = torch.randn(heads, 128, generator=g)
    rows = [base, torch.zeros(heads, 128), -torch.zeros(heads, 128), torch.full((heads, 128), 3.25),
            base * 1e-30, base * 2.0 ** -110, base * 1e30, base * 1e37, base + 1000.0,
            torch.linspace(-7.5, 7.5, 128).expand(heads, 128),     # many exact halves of a scale of 1
            torch.arange(128).float().expand(heads, 128) % 16 - 8,
            torch.where(torch.arange(128) == 5, 100.0, 1e-3).expand(heads, 128)]
    for bad in (float("nan"), float("inf"), -float("inf")):
        x = base.clone()
        x[:, 70] = bad
        rows.append(x)
    x = base.clone()
    x[:, 0], x[:, 1] = 3e38, -3e38
    rows.append(x)
    return torch.stack(rows).to(torch.bfloat16)


def _as_bits(t):
    return t.view(torch.uint8) if t.dtype == torch.uint8 else t.contiguous().view(torch.int16)


@gpu
@pytest.mark.parametrize("tokens,heads,block,group", [(1, 1, 16, 32), (16, 8, 16, 32), (333, 3, 48, 64), (1000, 8, 256, 128),
                                                      (77, 1, 7, 32), (129, 2, 16, 128)])
def test_store_and_load_are_exact(L, tokens, heads, block, group):
    g = torch.Generator().manual_seed(tokens)
    special = _special_rows(heads)
    k = torch.randn(tokens, heads, 128, generator=g).to(torch.bfloat16)
    k[:min(tokens, len(special))] = special[:tokens]
    v = (torch.randn(tokens, heads, 128, generator=g) * 4 + 1).to(torch.bfloat16)
    v[-min(tokens, len(special)):] = special[-tokens:]
    blocks = -(-tokens // block) + 2
    slots = torch.randperm(blocks * block, generator=g)[:tokens].to(torch.int32)
    skipped = torch.arange(tokens) % 5 == 3
    slots[skipped] = -1
    caches, plain = [], []
    for x in (k, v):
        codes = torch.full((blocks, heads, block, 64), 0xA5, dtype=torch.uint8)
        params = torch.full((blocks, heads, block, 128 // group, 2), 7.0, dtype=torch.bfloat16)
        caches.append(pkv.Q4Cache(codes.cuda(), params.cuda()))
        c, p = Q.quantise(x, group)
        for t in range(tokens):
            if slots[t] >= 0:
                b, o = divmod(int(slots[t]), block)
                codes[b, :, o], params[b, :, o] = c[t], p[t]
        plain.append((codes, params))
    pkv.kv_store_q4(k.cuda(), v.cuda(), *caches, slots.cuda())
    back = pkv.kv_load_q4(*caches, slots.cuda())
    assert pkv.check_device_errors() == 0
    for cache, (codes, params), x, got in zip(caches, plain, (k, v), back):
        assert torch.equal(cache.codes.cpu(), codes)
        nan = torch.isnan(params.float())
        assert torch.equal(torch.isnan(cache.params.cpu().float()), nan)
        assert torch.equal(_as_bits(cache.params.cpu())[~nan], _as_bits(params)[~nan])
        want = Q.values(*Q.quantise(x, group))
        want[skipped] = 0.0
        assert torch.equal(got.cpu().double().nan_to_num(nan=123.0), want.nan_to_num(nan=123.0))


@gpu
@pytest.mark.parametrize("group", [32, 64, 128])
def test_store_is_exact_to_the_ends_of_the_range(L, group):
    """Groups whose differences overflow fp32, and rows of any bits at all."""
    g = torch.Generator().manual_seed(group)
    x = torch.randint(-2 ** 15, 2 ** 15, (512, 2, 128), generator=g, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
    big = 3.3e38 * torch.rand(256, 2, 128, generator=g)          # from -x/8 to 7x/8 and the other way round
    x[:256] = torch.where(torch.rand(256, 2, 128, generator=g) < 0.3, -big / 8, big * 0.875).to(torch.bfloat16)
    x[128:256] = -x[128:256]
    y = x.flip(0).contiguous()
    kc, vc = (pkv.new_q4_cache(32, 16, 2, group) for _ in range(2))
    slots = torch.arange(512, dtype=torch.int32, device="cuda")
    pkv.kv_store_q4(x.cuda(), y.cuda(), kc, vc, slots)
    rk, rv = pkv.kv_load_q4(kc, vc, slots)
    assert pkv.check_device_errors() == 0
    for c, rows, back in ((kc, x, rk), (vc, y, rv)):
        codes, params = Q.quantise(rows, group)
        assert torch.equal(c.codes.permute(0, 2, 1, 3).reshape(512, 2, 64).cpu(), codes)
        got, nan = c.params.permute(0, 2, 1, 3, 4).reshape(params.shape).cpu(), torch.isnan(params.float())
        assert torch.equal(torch.isnan(got.float()), nan) and torch.equal(_as_bits(got)[~nan], _as_bits(params)[~nan])
        want = Q.values(codes, params)
        assert torch.equal(back.cpu().double().nan_to_num(nan=123.0, posinf=4e38, neginf=-4e38),
                           want.nan_to_num(nan=123.0, posinf=4e38, neginf=-4e38))


@gpu
def test_row_calls_report_bad_slots_and_touch_nothing_else(L):
    heads, block = 2, 16
    kc, vc = pkv.new_q4_cache(4, block, heads), pkv.new_q4_cache(4, block, heads)
    k = torch.randn(4, heads, 128).to(torch.bfloat16).cuda()
    slots = torch.tensor([64, 5, -2, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    pkv.kv_store_q4(k, k, kc, vc, slots)
    assert pkv.check_device_errors() == pkv.DEVERR_SLOT
    assert int((kc.codes != 0).any(-1).sum()) == heads      # slot 5 alone
    back, _ = pkv.kv_load_q4(kc, vc, slots)
    assert pkv.check_device_errors() == pkv.DEVERR_SLOT
    assert bool((back[[0, 2, 3]] == 0).all()) and bool((back[1] != 0).any())
    # the same slot any number of times; no tokens at all
    many, _ = pkv.kv_load_q4(kc, vc, torch.full((37,), 5, dtype=torch.int32, device="cuda"))
    assert torch.equal(many, back[1:2].expand(37, -1, -1))
    none, _ = pkv.kv_load_q4(kc, vc, slots[:0])
    assert none.shape == (0, heads, 128) and pkv.check_device_errors() == 0


# ------------------------------------------------------------------ GPU: decode

def _decode_plain(c, q, gqa, window, scale=SCALE):
    out, lse = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape[:2], dtype=torch.float64)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    weights = torch.zeros(len(c.lens), max(c.lens), dtype=torch.float64)
    tol_w = torch.zeros_like(weights)
    for s, n in enumerate(c.lens):
        first = max(0, n - window) if window else 0
        for h in range(c.heads):
            k, v = c.logical(c.k, s, n, h), c.logical(c.v, s, n, h)
            rows = slice(h * gqa, (h + 1) * gqa)
            o, l, w, wv, qk = Q.attend(q[s, rows].double(), k, v, scale, [first] * gqa, [n - 1] * gqa)
            out[s, rows], lse[s, rows] = o, l
            tol_o[s, rows] = Q.out_tolerance(o, wv)
            tol_l[s, rows] = Q.lse_tolerance(l, qk, n / 4)
            weights[s, :n] += w.sum(0)
            # a weight is exp(z - lse): both are off by at most the lse's tolerance
            tol_w[s, :n] += (w * 2 * tol_l[s, rows, None]).sum(0) + 2.0 ** -20 * w.sum(0)
    return out, lse, tol_o, tol_l, weights, tol_w


DECODE = [  # lens, heads, gqa, block, group, window
    ([1], 1, 1, 16, 32, 0),
    ([17, 64, 100, 128], 8, 2, 16, 32, 0),
    ([1, 2, 15, 16, 17, 31, 33, 255], 2, 4, 48, 64, 0),
    ([640] * 3, 8, 2, 256, 32, 0),
    ([700, 3, 129, 1024], 4, 8, 64, 128, 0),
    ([5000], 1, 2, 256, 32, 0),
    ([2500, 1, 4097], 2, 1, 32, 64, 0),
    ([9000, 40], 1, 4, 128, 128, 0),
    ([17, 64, 100, 128], 3, 2, 16, 32, 1),
    ([300, 5, 1000, 641], 2, 4, 64, 64, 100),
    ([3000, 10], 2, 2, 16, 128, 1025),
    ([500, 64], 1, 8, 32, 32, 4096),
    ([6000, 7, 300], 2, 8, 16, 64, 0),
    ([3300, 65], 3, 1, 32, 32, 0),
]


@gpu
@pytest.mark.parametrize("lens,heads,gqa,block,group,window", DECODE)
@pytest.mark.parametrize("scored", [False, True])
def test_decode(L, lens, heads, gqa, block, group, window, scored):
    c = Q.Cache(sum(lens) + group, lens, heads, block, group, outliers=0.05)
    g = torch.Generator().manual_seed(len(lens))
    q = torch.randn(len(lens), heads * gqa, 128, generator=g).to(torch.bfloat16)
    out, lse, tol_o, tol_l, weights, tol_w = _decode_plain(c, q, gqa, window)
    kc, vc, bt = c.cuda()
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    scores = None
    if scored:
        scores = torch.full((len(lens), max(lens) + 5), 0.5, device="cuda")
    o, l = pkv.paged_decode_attn_q4(q.cuda(), kc, vc, bt, cl, max(lens), SCALE, sliding_window=window, key_scores=scores)
    assert pkv.check_device_errors() == 0
    assert bool(((o.cpu().double() - out).abs() <= tol_o).all()), float(((o.cpu().double() - out).abs() / tol_o).max())
    assert bool(((l.cpu().double() - lse).abs() <= tol_l).all()), float(((l.cpu().double() - lse).abs() / tol_l).max())
    if scored:
        got = scores.cpu().double()
        assert bool((got[:, max(lens):] == 0.5).all())
        # untouched entries keep their bits; 0.5 + w rounds once
        untouched = weights == 0
        got = got[:, :max(lens)]
        for s, n in enumerate(lens):
            first = max(0, n - window) if window else 0
            assert bool((got[s, n:] == 0.5).all()) and bool((got[s, :first] == 0.5).all())
        tol = tol_w + Q.U32 * (0.5 + weights) + 1e-30
        assert bool(((got - 0.5 - weights).abs() <= tol).all()), float(((got - 0.5 - weights).abs() / tol).max())
        assert bool((got[untouched] == 0.5).all())


@gpu
def test_decode_long_and_short_sequences_of_many_pairs(L):
    """Many (sequence, KV head) pairs: one CTA each, the long one's warps with more
    than one batch of table entries."""
    lens = [4000] + [30] * 94
    c = Q.Cache(21, lens, 8, 256, 32)
    q = torch.randn(95, 16, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    out, lse, tol_o, tol_l, _, _ = _decode_plain(c, q, 2, 0)
    kc, vc, bt = c.cuda()
    o, l = pkv.paged_decode_attn_q4(q.cuda(), kc, vc, bt, torch.tensor(lens, dtype=torch.int32, device="cuda"), 4000, SCALE)
    assert pkv.check_device_errors() == 0
    assert bool(((o.cpu().double() - out).abs() <= tol_o).all()) and bool(((l.cpu().double() - lse).abs() <= tol_l).all())


@gpu
def test_decode_more_sequences_than_ranges_take(L):
    """Above 1,024 sequences every (sequence, KV head) has a CTA of its own."""
    lens = [5, 40, 17] * 350 + [900]
    c = Q.Cache(22, lens, 1, 16, 64)
    q = torch.randn(len(lens), 1, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    kc, vc, bt = c.cuda()
    scores = torch.zeros(len(lens), 900, device="cuda")
    o, none = pkv.paged_decode_attn_q4(q.cuda(), kc, vc, bt, torch.tensor(lens, dtype=torch.int32, device="cuda"), 900, SCALE,
                                       with_lse=False, key_scores=scores)
    assert none is None and pkv.check_device_errors() == 0
    for s in (0, 1, 2, 500, 1049, 1050):
        n = lens[s]
        want, lse, w, wv, qk = Q.attend(q[s].double(), c.logical(c.k, s, n, 0), c.logical(c.v, s, n, 0), SCALE, [0], [n - 1])
        assert bool(((o[s, 0].cpu().double() - want[0]).abs() <= Q.out_tolerance(want[0], wv[0])).all())
        tol = w[0] * (2 * Q.lse_tolerance(lse, qk, n / 4) + 2.0 ** -20) + 1e-30
        assert bool(((scores[s, :n].cpu().double() - w[0]).abs() <= tol).all()) and bool((scores[s, n:] == 0).all())


@gpu
def test_head_shards_of_a_4_bit_cache(L):
    """A rank of a KV-head shard (heads are dimension 1 of a 4-bit cache) computes
    its heads of the whole call."""
    from paged_kv_attention_22_gb300.shard import head_shard, take_heads
    lens = [700, 33, 64]
    c = Q.Cache(23, lens, 4, 64, 32)
    q = torch.randn(3, 8, 128, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    out, _, tol_o, _, _, _ = _decode_plain(c, q, 2, 0)
    kc, vc, bt = c.cuda()
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for rank in range(2):
        qs, ks = head_shard(rank, 2, 8, 4)
        kr, vr = (tuple(take_heads(x, ks, 1) for x in cache) for cache in (kc, vc))
        o, _ = pkv.paged_decode_attn_q4(take_heads(q, qs, 1).cuda(), kr, vr, bt, cl, 700, SCALE)
        assert bool(((o.cpu().double() - out[:, qs]).abs() <= tol_o[:, qs]).all())
    assert pkv.check_device_errors() == 0


def _random_cache(seqs, blocks_per_seq, heads, block, group):
    """A large random cache made on the GPU, tables of seqs sequences in shuffled blocks."""
    g = torch.Generator(device="cuda").manual_seed(3)
    n = seqs * blocks_per_seq
    caches = []
    for _ in range(2):
        codes = torch.randint(0, 256, (n, heads, block, 64), generator=g, device="cuda", dtype=torch.uint8)
        params = torch.rand(n, heads, block, 128 // group, 2, generator=g, device="cuda") * 0.2 + 0.1
        params[..., 1] = -23.5 * params[..., 0]
        caches.append((codes, params.to(torch.bfloat16)))
    return caches[0], caches[1], torch.randperm(n, generator=g, device="cuda").to(torch.int32).view(seqs, blocks_per_seq)


@gpu
@pytest.mark.parametrize("window", [0, 20000])
def test_decode_long_ranges(L, window):
    """Enough keys that every warp's range takes several batches of table entries;
    unequal lengths, one of them invalid; a few pairs compared."""
    seqs, heads, block = 12, 8, 256
    kc, vc, bt = _random_cache(seqs, 160, heads, block, 32)
    lens = [40960, 40959, 33000, 40960, 17, 0, 40960, 40000, 40960, 1, 40960, 40960]
    q = torch.randn(seqs, 16, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).cuda()
    o = torch.full_like(q, 9.0)
    o, l = pkv.paged_decode_attn_q4(q, kc, vc, bt, torch.tensor(lens, dtype=torch.int32, device="cuda"), 40960, SCALE, out=o,
                                    sliding_window=window)
    assert pkv.check_device_errors() == pkv.DEVERR_CONTEXT
    assert bool((o[5] == 9.0).all())
    for s, h in ((0, 0), (1, 3), (2, 7), (4, 5), (6, 2), (7, 7), (9, 0), (11, 7)):
        n = lens[s]
        first = max(0, n - window) if window else 0
        p = torch.arange(n, device="cuda")
        rows = (bt[s].long()[p // block], h, p % block)
        k, v = (Q.values(*(x[rows].cpu() for x in c)) for c in (kc, vc))
        want, lse, _, wv, qk = Q.attend(q[s, 2 * h:2 * h + 2].cpu().double(), k, v, SCALE, [first] * 2, [n - 1] * 2)
        err, tol = (o[s, 2 * h:2 * h + 2].cpu().double() - want).abs(), Q.out_tolerance(want, wv)
        assert bool((err <= tol).all()), (s, h, float((err / tol).max()))
        err, tol = (l[s, 2 * h:2 * h + 2].cpu().double() - lse).abs(), Q.lse_tolerance(lse, qk, n / 4)
        assert bool((err <= tol).all()), (s, h, float((err / tol).max()))


@gpu
def test_decode_scale_of_any_sign(L):
    lens = [100, 7]
    c = Q.Cache(31, lens, 2, 16, 32)
    q = torch.randn(2, 4, 128, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    kc, vc, bt = c.cuda()
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for scale in (-0.3, 0.0, 2.5):
        for s, n in enumerate(lens):
            o, l = pkv.paged_decode_attn_q4(q.cuda(), kc, vc, bt, cl, 100, scale)
            for h in range(4):
                k, v = c.logical(c.k, s, n, h // 2), c.logical(c.v, s, n, h // 2)
                want, lse, _, wv, qk = Q.attend(q[s, h:h + 1].double(), k, v, scale, [0], [n - 1])
                assert bool(((o[s, h].cpu().double() - want[0]).abs() <= Q.out_tolerance(want[0], wv[0])).all())
                assert abs(float(l[s, h]) - float(lse)) <= float(Q.lse_tolerance(lse, qk, n / 4))
    assert pkv.check_device_errors() == 0


@gpu
def test_decode_skips_invalid_rows_and_reports_them(L):
    lens = [40, 40, 40, 40]
    c = Q.Cache(5, lens, 2, 16, 32)
    q = torch.randn(4, 4, 128).to(torch.bfloat16)
    out, _, tol_o, _, _, _ = _decode_plain(c, q, 2, 0)
    kc, vc, bt = c.cuda()
    o = torch.full_like(q, 9.0).cuda()
    lse = torch.full((4, 4), 9.0, device="cuda")
    cl = torch.tensor([40, 0, 41, 40], dtype=torch.int32, device="cuda")
    scores = torch.zeros(4, 40, device="cuda")
    pkv.paged_decode_attn_q4(q.cuda(), kc, vc, bt, cl, 40, SCALE, out=o, lse=lse, key_scores=scores)
    assert pkv.check_device_errors() == pkv.DEVERR_CONTEXT
    assert bool((o[1:3] == 9.0).all()) and bool((lse[1:3] == 9.0).all()) and bool((scores[1:3] == 0).all())
    ok = [0, 3]
    assert bool(((o[ok].cpu().double() - out[ok]).abs() <= tol_o[ok]).all())
    # a bad table entry raises its bit and disturbs no other row
    for bad in (-1, c.num_blocks, 2 ** 31 - 1):
        bt2 = bt.clone()
        bt2[1, 1] = bad
        o, _ = pkv.paged_decode_attn_q4(q.cuda(), kc, vc, bt2, torch.full_like(cl, 40), 40, SCALE)
        assert pkv.check_device_errors() == pkv.DEVERR_BLOCK
        ok = [0, 2, 3]
        assert bool(((o[ok].cpu().double() - out[ok]).abs() <= tol_o[ok]).all())


@gpu
@pytest.mark.parametrize("ctx,block", [(40, 16), (20000, 64)])  # a CTA for each pair, ranges
def test_decode_leaves_keys_of_bad_table_entries_out(L, ctx, block):
    """Sequence 0 has one bad entry, sequence 1 nothing but bad ones, whatever an
    earlier call left in the workspace."""
    c = Q.Cache(11, [ctx, ctx], 1, block, 32)
    q = torch.randn(2, 2, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    kc, vc, bt = c.cuda()
    bt[0, 1] = c.num_blocks
    bt[1] = -1
    ws = pkv.new_q4_decode_workspace(2, 2, 1, ctx, True).fill_(255)    # NaNs
    scores = torch.full((2, ctx), 0.5, device="cuda")
    cl = torch.full((2,), ctx, dtype=torch.int32, device="cuda")
    out, lse = pkv.paged_decode_attn_q4(q.cuda(), kc, vc, bt, cl, ctx, SCALE, workspace=ws, key_scores=scores)
    assert pkv.check_device_errors() == pkv.DEVERR_BLOCK
    rest = torch.cat([torch.arange(block), torch.arange(2 * block, ctx)])
    ks, vs = c.logical(c.k, 0, ctx, 0)[rest], c.logical(c.v, 0, ctx, 0)[rest]
    o, l, w, wv, qk = Q.attend(q[0].double(), ks, vs, SCALE, [0, 0], [len(rest) - 1] * 2)
    assert bool(((out[0].cpu().double() - o).abs() <= Q.out_tolerance(o, wv)).all())
    tol_l = Q.lse_tolerance(l, qk, ctx / 4)
    assert bool(((lse[0].cpu().double() - l).abs() <= tol_l).all())
    got = scores.cpu().double()
    assert bool((got[0, block:2 * block] == 0.5).all()) and bool((got[1] == 0.5).all())
    # exp(z - lse): both within the lse's tolerance; the additions round
    tol = (w * (2 * tol_l[:, None] + 2.0 ** -20)).sum(0) + 2 * Q.U32 * (0.5 + w.sum(0))
    assert bool(((got[0, rest] - 0.5 - w.sum(0)).abs() <= tol).all())


@gpu
def test_decode_nan_group_reaches_its_sequence_only(L):
    c = Q.Cache(6, [33, 33], 1, 16, 32)
    b, o = int(c.tables[0, 1]), 4
    c.v[1][b, 0, o, 2] = float("nan")           # dims 64..95 of one V row of sequence 0
    kc, vc, bt = c.cuda()
    q = torch.randn(2, 2, 128).to(torch.bfloat16).cuda()
    out, lse = pkv.paged_decode_attn_q4(q, kc, vc, bt, torch.tensor([33, 33], dtype=torch.int32, device="cuda"), 33, SCALE)
    assert pkv.check_device_errors() == 0
    assert bool(torch.isnan(out[0, :, 64:96]).all()) and bool(torch.isfinite(out[0, :, :64]).all())
    assert bool(torch.isfinite(out[1]).all()) and bool(torch.isfinite(lse).all())


@gpu
def test_decode_workspace_serves_smaller_calls_and_refuses_larger(L):
    c = Q.Cache(7, [2000, 700, 30], 2, 32, 64)
    kc, vc, bt = c.cuda()
    q = torch.randn(3, 4, 128).to(torch.bfloat16)
    out, _, tol_o, _, _, _ = _decode_plain(c, q, 2, 0)
    ws = pkv.new_q4_decode_workspace(3, 4, 2, 2000, with_scores=True)
    for rows in ([0, 1, 2], [1, 2], [2], [0]):
        n = [c.lens[r] for r in rows]
        o, _ = pkv.paged_decode_attn_q4(q[rows].cuda(), kc, vc, bt[rows], torch.tensor(n, dtype=torch.int32, device="cuda"),
                                        max(n), SCALE, workspace=ws)
        assert bool(((o.cpu().double() - out[rows]).abs() <= tol_o[rows]).all())
    small = torch.empty(1024, dtype=torch.uint8, device="cuda")
    with pytest.raises(pkv.PkvError):
        pkv.paged_decode_attn_q4(q.cuda(), kc, vc, bt, torch.tensor(c.lens, dtype=torch.int32, device="cuda"), 2000, SCALE,
                                 workspace=small)
    assert pkv.check_device_errors() == 0


@gpu
def test_decode_in_a_graph_on_another_stream(L):
    """Captured on a side stream and replayed: the same bits as the eager call,
    with a context bound far above the lengths."""
    c = Q.Cache(8, [300, 1, 77], 4, 16, 32)
    kc, vc, bt = c.cuda()
    q = torch.randn(3, 8, 128).to(torch.bfloat16).cuda()
    cl = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    wide = torch.full((3, 1024), -1, dtype=torch.int32, device="cuda")
    wide[:, :bt.shape[1]] = bt
    eager, lse = pkv.paged_decode_attn_q4(q, kc, vc, wide, cl, 16384, SCALE)
    stream = torch.cuda.Stream()
    ws = pkv.new_q4_decode_workspace(3, 8, 4, 16384, with_scores=True)
    o, l = torch.zeros_like(eager), torch.zeros_like(lse)
    scores = torch.zeros(3, 16384, device="cuda")
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        pkv.paged_decode_attn_q4(q, kc, vc, wide, cl, 16384, SCALE, out=o, lse=l, workspace=ws, key_scores=scores)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, eager) and torch.equal(l, lse)
    once = torch.zeros_like(scores)
    pkv.paged_decode_attn_q4(q, kc, vc, wide, cl, 16384, SCALE, key_scores=once, stream=None)
    assert torch.equal(scores, once + once)
    assert pkv.check_device_errors() == 0


@gpu
def test_rows_past_32_bit_offsets(L):
    """A pool whose arrays pass 4 GiB: rows in its last blocks."""
    heads, block, group = 8, 256, 128
    NB = (1 << 32) // (heads * block * 64) + 40
    kc, vc = [(torch.empty(NB, heads, block, 64, dtype=torch.uint8, device="cuda"),
               torch.empty(NB, heads, block, 1, 2, dtype=torch.bfloat16, device="cuda")) for _ in range(2)]
    assert kc[0].numel() > 1 << 32
    n = 300
    tables = torch.tensor([[NB - 1, NB - 3]], dtype=torch.int32)
    g = torch.Generator().manual_seed(12)
    k, v = (torch.randn(n, heads, 128, generator=g).to(torch.bfloat16) for _ in range(2))
    p = torch.arange(n)
    slots = (tables[0].long()[p // block] * block + p % block).to(torch.int32).cuda()
    pkv.kv_store_q4(k.cuda(), v.cuda(), kc, vc, slots)
    kk, vv = (Q.values(*Q.quantise(x, group)) for x in (k, v))
    bk, bv = pkv.kv_load_q4(kc, vc, slots)
    assert torch.equal(bk.cpu().double(), kk) and torch.equal(bv.cpu().double(), vv)
    q = torch.randn(1, 8, 128, generator=g).to(torch.bfloat16)
    o, _ = pkv.paged_decode_attn_q4(q.cuda(), kc, vc, tables.cuda(), torch.tensor([n], dtype=torch.int32, device="cuda"), n, SCALE)
    po, _ = pkv.paged_prefill_attn_q4(q.cuda(), kc, vc, _cu([1]), _cu([n]), tables.cuda(), 1, n, n, SCALE)
    for h in range(8):
        want, _, _, wv, _ = Q.attend(q[0, h:h + 1].double(), kk[:, h], vv[:, h], SCALE, [0], [n - 1])
        for got in (o, po):
            assert bool(((got[0, h].cpu().double() - want[0]).abs() <= Q.out_tolerance(want[0], wv[0])).all())
    # compaction between far blocks
    keep = torch.arange(0, 300, 3, dtype=torch.int32, device="cuda")[None]
    dst = torch.tensor([[NB - 5]], dtype=torch.int32, device="cuda")
    pkv.evict_compact_q4(kc, vc, tables.cuda(), dst, keep, torch.tensor([100], dtype=torch.int32, device="cuda"))
    got, _ = pkv.kv_load_q4(kc, vc, (torch.arange(100) + (NB - 5) * block).to(torch.int32).cuda())
    assert torch.equal(got.cpu().double(), kk[::3])
    assert pkv.check_device_errors() == 0


@gpu
def test_two_streams_with_workspaces_of_their_own(L):
    """Calls that overlap on two streams: each gets the bits of the call alone."""
    c = Q.Cache(41, [3000, 50], 2, 16, 32)
    kc, vc, bt = c.cuda()
    cl = torch.tensor([3000, 50], dtype=torch.int32, device="cuda")
    g = torch.Generator().manual_seed(6)
    qs = [torch.randn(2, 4, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2)]
    alone = [pkv.paged_decode_attn_q4(q, kc, vc, bt, cl, 3000, SCALE) for q in qs]
    streams = [torch.cuda.Stream() for _ in qs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, st in enumerate(streams):
            got[i].append(pkv.paged_decode_attn_q4(qs[i], kc, vc, bt, cl, 3000, SCALE, stream=st))
    torch.cuda.synchronize()
    for i in range(2):
        for o, l in got[i]:
            assert torch.equal(o, alone[i][0]) and torch.equal(l, alone[i][1])
    assert pkv.check_device_errors() == 0


@gpu
@pytest.mark.parametrize("call", ["decode_q4", "prefill_q4", "store_q4", "decode", "scores", "prefill", "select"])
def test_first_call_of_a_host_thread(L, call):
    """A thread that has made no CUDA call yet: the same bits as from the main one."""
    c = Q.Cache(19, [40], 2, 16, 32)
    kc, vc, bt = c.cuda()
    g = torch.Generator().manual_seed(3)
    k16 = torch.randn(c.num_blocks, 16, 2, 128, generator=g).to(torch.bfloat16).cuda()
    q = torch.randn(1, 4, 128, generator=g).to(torch.bfloat16).cuda()
    out, lse, scores = torch.zeros_like(q), torch.zeros(1, 4, device="cuda"), torch.zeros(1, 40, device="cuda")
    cl, cu_q, cu_k = torch.tensor([40], dtype=torch.int32, device="cuda"), _cu([1]), _cu([40])
    keep, new = torch.zeros(1, 9, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    w4, wp = pkv.new_q4_decode_workspace(1, 4, 2, 40), pkv.new_q4_prefill_workspace(1, 40, 40, 2)
    w16, ws = pkv.new_decode_workspace(1, 4, 2, 128, 40), pkv.new_decode_scores_workspace(1, 4, 2, 40)
    stream = torch.cuda.current_stream()

    def run():
        if call == "decode_q4":
            pkv.paged_decode_attn_q4(q, kc, vc, bt, cl, 40, SCALE, out=out, lse=lse, workspace=w4, stream=stream)
        elif call == "prefill_q4":
            pkv.paged_prefill_attn_q4(q, kc, vc, cu_q, cu_k, bt, 1, 40, 40, SCALE, out=out, lse=lse, workspace=wp, stream=stream)
        elif call == "store_q4":
            pkv.kv_store_q4(k16[0, :1], k16[1, :1], kc, vc, cl * 0, stream=stream)
        elif call == "decode":
            pkv.paged_decode_attn(q, k16, k16, bt, cl, 40, SCALE, out=out, lse=lse, workspace=w16, stream=stream)
        elif call == "scores":
            pkv.paged_decode_attn_scores(q, k16, k16, bt, cl, 40, SCALE, scores, out=out, lse=lse, workspace=ws, stream=stream)
        elif call == "prefill":
            pkv.paged_prefill_attn(q, k16, k16, cu_q, cu_k, bt, 1, 40, SCALE, out=out, lse=lse, stream=stream)
        else:
            pkv.evict_select(scores, cl, 9, 2, keep=keep, new_lens=new, stream=stream)

    results = []
    for first in (False, True):
        for x in (out, lse, scores, keep, new):
            x.zero_()
        torch.cuda.synchronize()
        raised = []

        def body():
            try:
                run()
            except Exception as e:      # reported below: an exception would end in the thread
                raised.append(e)
        if first:
            t = threading.Thread(target=body)
            t.start()
            t.join()
        else:
            body()
        assert not raised, raised
        torch.cuda.synchronize()
        results.append([x.clone() for x in (out, lse, scores, keep, new, kc[0], vc[0])])
    assert all(torch.equal(a, b) for a, b in zip(*results))
    assert pkv.check_device_errors() == 0


# ------------------------------------------------------------------ GPU: prefill

PREFILL = [  # q lens, k lens, heads, gqa, block, group, window
    ([9, 33, 64, 64], [9, 33, 64, 64], 8, 2, 16, 32, 0),
    ([1], [1], 1, 1, 16, 128, 0),
    ([1, 0, 5], [300, 17, 5], 2, 4, 48, 64, 0),
    ([200, 37, 300], [330, 37, 429], 2, 2, 64, 32, 0),
    ([130, 1], [513, 2], 1, 4, 256, 128, 0),
    ([200, 37, 300], [330, 37, 700], 2, 2, 16, 64, 100),
    ([1, 3], [600, 129], 1, 2, 32, 32, 1),
    # few query tokens over many keys: by rows
    ([4, 1, 0, 2], [3000, 17, 40, 1025], 2, 2, 16, 32, 0),
    ([1], [9000], 1, 4, 64, 128, 0),
    ([16], [5000], 2, 1, 256, 64, 0),
    ([3, 8], [2500, 700], 2, 4, 32, 32, 300),
    ([1] * 20, [40] * 20, 8, 2, 16, 64, 0),
]


def _prefill_plain(c, q, q_lens, gqa, window):
    out, lse = torch.zeros(q.shape, dtype=torch.float64), torch.zeros(q.shape[:2], dtype=torch.float64)
    tol_o, tol_l = torch.zeros_like(out), torch.zeros_like(lse)
    at = 0
    for s, (n, m) in enumerate(zip(c.lens, q_lens)):
        last = torch.arange(n - m, n)
        first = (last - window + 1).clamp(min=0) if window else torch.zeros_like(last)
        for h in range(c.heads * gqa):
            if m == 0:
                continue
            k, v = c.logical(c.k, s, n, h // gqa), c.logical(c.v, s, n, h // gqa)
            o, l, _, wv, qk = Q.attend(q[at:at + m, h].double(), k, v, SCALE, first, last)
            out[at:at + m, h], lse[at:at + m, h] = o, l
            tol_o[at:at + m, h], tol_l[at:at + m, h] = Q.out_tolerance(o, wv), Q.lse_tolerance(l, qk, n)
        at += m
    return out, lse, tol_o, tol_l


def _cu(lens):
    return torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32).cuda()


@gpu
@pytest.mark.parametrize("q_lens,k_lens,heads,gqa,block,group,window", PREFILL)
def test_prefill(L, q_lens, k_lens, heads, gqa, block, group, window):
    c = Q.Cache(sum(k_lens), k_lens, heads, block, group)
    g = torch.Generator().manual_seed(len(k_lens))
    q = torch.randn(sum(q_lens), heads * gqa, 128, generator=g).to(torch.bfloat16)
    out, lse, tol_o, tol_l = _prefill_plain(c, q, q_lens, gqa, window)
    kc, vc, bt = c.cuda()
    if window:  # an engine may drop the blocks that lie wholly before every window
        for s, (n, m) in enumerate(zip(k_lens, q_lens)):
            bt[s, :max(0, n - m - window + 1) // block] = -1
    # a workspace of NaN: nothing may be read there that the call did not write
    ws = pkv.new_q4_prefill_workspace(len(k_lens), sum(k_lens) + 3, max(k_lens), heads)
    ws.fill_(0xFF)
    o, l = pkv.paged_prefill_attn_q4(q.cuda(), kc, vc, _cu(q_lens), _cu(k_lens), bt, max(q_lens), max(k_lens),
                                     sum(k_lens) + 3, SCALE, sliding_window=window, workspace=ws)
    assert pkv.check_device_errors() == 0
    assert bool(((o.cpu().double() - out).abs() <= tol_o).all()), float(((o.cpu().double() - out).abs() / tol_o).max())
    assert bool(((l.cpu().double() - lse).abs() <= tol_l).all()), float(((l.cpu().double() - lse).abs() / tol_l).max())


@gpu
def test_prefill_refuses_a_segment_past_total_k_alone(L):
    q_lens = k_lens = [20, 30]
    c = Q.Cache(11, k_lens, 2, 16, 32)
    q = torch.randn(50, 4, 128).to(torch.bfloat16)
    out, _, tol_o, _ = _prefill_plain(c, q, q_lens, 2, 0)
    kc, vc, bt = c.cuda()
    o, _ = pkv.paged_prefill_attn_q4(q.cuda(), kc, vc, _cu(q_lens), _cu(k_lens), bt, 30, 30, 49, SCALE)
    assert pkv.check_device_errors() & pkv.DEVERR_SEQLENS
    assert bool(((o[:20].cpu().double() - out[:20]).abs() <= tol_o[:20]).all())


@gpu
def test_prefill_by_rows_leaves_refused_segments_alone(L):
    """Few tokens over many keys, one segment past total_k, one longer than the stated
    maximum, and rows behind the last segment."""
    q_lens, k_lens = [2, 1, 3], [2000, 1500, 1000]
    c = Q.Cache(13, k_lens, 2, 16, 32)
    q = torch.randn(8, 4, 128, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    out, lse, tol_o, tol_l = _prefill_plain(c, q, q_lens, 2, 0)
    kc, vc, bt = c.cuda()
    for total_k, max_k, good in ((4500, 2000, [0, 1, 2, 3, 4, 5]), (4499, 2000, [0, 1, 2]), (4500, 1999, [2, 3, 4, 5])):
        o = torch.full_like(q, 9.0).cuda()
        l = torch.full((8, 4), 9.0, device="cuda")
        pkv.paged_prefill_attn_q4(q.cuda(), kc, vc, _cu(q_lens), _cu(k_lens), bt, 3, max_k, total_k, SCALE, out=o, lse=l)
        assert pkv.check_device_errors() == (0 if len(good) == 6 else pkv.DEVERR_SEQLENS)
        rest = [r for r in range(8) if r not in good]
        assert bool((o[rest] == 9.0).all()) and bool((l[rest] == 9.0).all())
        assert bool(((o[good].cpu().double() - out[good]).abs() <= tol_o[good]).all())
        assert bool(((l[good].cpu().double() - lse[good]).abs() <= tol_l[good]).all())


REFUSED = {  # what is wrong: the segments that are left alone (None: not looked at)
    "total_k": [2], "max_k": [0], "max_q": [0], "table": [0], "total_q": [2], "cu_k": [0], "decreasing": None, "empty": []}


@gpu
@pytest.mark.parametrize("what", list(REFUSED))
@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("q_lens,k_lens", [([3, 2, 1], [2000, 1500, 1000]), ([100, 80, 90], [300, 200, 150])])  # by rows, widened
def test_prefill_refuses_segments_alike_on_both_ways(L, q_lens, k_lens, window, what):
    """A segment that the call refuses raises the bit and keeps its rows; the others
    are attended. Sequence 0 is the longest in queries and in keys."""
    alone, heads, gqa, block = REFUSED[what], 2, 2, 16
    if what == "empty":                         # nothing to write, but keys past the maximum
        q_lens = [0] + q_lens[1:]
    c = Q.Cache(15, k_lens, heads, block, 32)
    rows = sum(q_lens) + (-1 if what == "total_q" else 3)
    q = torch.randn(rows + 1, heads * gqa, 128, generator=torch.Generator().manual_seed(4)).to(torch.bfloat16)
    out, lse, tol_o, tol_l = _prefill_plain(c, q, q_lens, gqa, window)
    q = q[:rows]
    kc, vc, bt = c.cuda()
    cu_q, cu_k = _cu(q_lens), _cu(k_lens)
    max_q, max_k, total_k = max(q_lens), max(k_lens), sum(k_lens)
    if what == "total_k":
        total_k -= 1
    elif what in ("max_k", "empty"):
        max_k -= 1
    elif what == "max_q":
        max_q -= 1
    elif what == "table":
        bt = bt[:, :-1].contiguous()            # sequence 0 alone needs the last column
    elif what == "cu_k":
        cu_k[0], max_k = -8, max_k + 8
    elif what == "decreasing":
        cu_q[1], max_q = cu_q[2] + 1, 64 if max_q < 64 else max_k
    o = torch.full_like(q, 9.0).cuda()
    l = torch.full((rows, heads * gqa), 9.0, device="cuda")
    pkv.paged_prefill_attn_q4(q.cuda(), kc, vc, cu_q, cu_k, bt, max_q, max_k, total_k, SCALE, out=o, lse=l,
                              sliding_window=window)
    assert pkv.check_device_errors() == pkv.DEVERR_SEQLENS
    if alone is None:
        return
    at = [0, q_lens[0], q_lens[0] + q_lens[1], sum(q_lens)]
    written = torch.zeros(rows, dtype=torch.bool)
    for s in range(3):
        if s not in alone:
            written[at[s]:at[s + 1]] = True
    o, l = o.cpu(), l.cpu()
    assert bool((o[~written] == 9.0).all()) and bool((l[~written] == 9.0).all())
    out, lse, tol_o, tol_l = (x[:rows][written] for x in (out, lse, tol_o, tol_l))
    assert bool(((o[written].double() - out).abs() <= tol_o).all()) and bool(((l[written].double() - lse).abs() <= tol_l).all())


@gpu
@pytest.mark.parametrize("segments", [32, 33, 129, 300])
def test_widened_prefill_of_many_segments(L, segments):
    """Lengths from 1 on, empty segments among them, and every 17th longer than the
    tables: those are left alone, the others attended."""
    g = torch.Generator().manual_seed(segments)
    q_lens = torch.randint(0, 12, (segments,), generator=g).tolist()
    q_lens[5] = 70                                      # more than the way by rows takes
    k_lens = [max(1, n + int(torch.randint(0, 40, (), generator=g))) for n in q_lens]
    for s in range(16, segments, 17):
        q_lens[s], k_lens[s] = 3, 113 + s % 8
    c = Q.Cache(20, k_lens, 1, 16, 32)
    rows = sum(q_lens)
    q = torch.randn(rows, 2, 128, generator=g).to(torch.bfloat16)
    out, lse, tol_o, tol_l = _prefill_plain(c, q, q_lens, 2, 0)
    kc, vc, bt = c.cuda()
    bt = bt[:, :7].contiguous()                         # 112 keys
    o, l = torch.full_like(q, 9.0).cuda(), torch.full((rows, 2), 9.0, device="cuda")
    pkv.paged_prefill_attn_q4(q.cuda(), kc, vc, _cu(q_lens), _cu(k_lens), bt, 70, 128, sum(k_lens), SCALE, out=o, lse=l)
    alone = torch.cat([torch.full((n,), s % 17 == 16) for s, n in enumerate(q_lens)])
    assert pkv.check_device_errors() == (pkv.DEVERR_SEQLENS if bool(alone.any()) else 0)
    o, l, ok = o.cpu(), l.cpu(), ~alone
    assert bool((o[alone] == 9.0).all()) and bool((l[alone] == 9.0).all())
    assert bool(((o[ok].double() - out[ok]).abs() <= tol_o[ok]).all()) and bool(((l[ok].double() - lse[ok]).abs() <= tol_l[ok]).all())


@gpu
@pytest.mark.parametrize("q_lens,k_lens", [([3, 2, 1], [2000, 1500, 1000]), ([100, 80, 90], [300, 200, 150])])  # by rows, widened
def test_prefill_reports_bad_table_entries_and_attends_the_other_segments(L, q_lens, k_lens):
    c = Q.Cache(16, k_lens, 2, 16, 32)
    q = torch.randn(sum(q_lens), 4, 128, generator=torch.Generator().manual_seed(5)).to(torch.bfloat16)
    out, lse, tol_o, tol_l = _prefill_plain(c, q, q_lens, 2, 0)
    kc, vc, bt = c.cuda()
    for bad in (-1, -7, c.num_blocks, 2 ** 31 - 1):
        bt[1, 1] = bad
        o, l = pkv.paged_prefill_attn_q4(q.cuda(), kc, vc, _cu(q_lens), _cu(k_lens), bt, max(q_lens), max(k_lens), sum(k_lens),
                                         SCALE)
        assert pkv.check_device_errors() == pkv.DEVERR_BLOCK
        good = list(range(q_lens[0])) + list(range(q_lens[0] + q_lens[1], sum(q_lens)))
        assert bool(((o[good].cpu().double() - out[good]).abs() <= tol_o[good]).all())
        assert bool(((l[good].cpu().double() - lse[good]).abs() <= tol_l[good]).all())


@gpu
@pytest.mark.parametrize("window", [0, 50])
def test_prefill_by_rows_of_more_rows_than_ranges_take(L, window):
    """1,280 query rows in 256 short segments: more sequences than a decode by ranges
    takes, fewer microseconds than widening."""
    g = torch.Generator().manual_seed(6)
    q_lens = [8, 0, 5, 4, 1, 16, 2, 4] * 32
    k_lens = [n + int(torch.randint(1, 200, (), generator=g)) for n in q_lens]
    c = Q.Cache(17, k_lens, 1, 16, 64)
    q = torch.randn(sum(q_lens), 2, 128, generator=g).to(torch.bfloat16)
    out, lse, tol_o, tol_l = _prefill_plain(c, q, q_lens, 2, window)
    kc, vc, bt = c.cuda()
    o, l = pkv.paged_prefill_attn_q4(q.cuda(), kc, vc, _cu(q_lens), _cu(k_lens), bt, max(q_lens), max(k_lens), sum(k_lens), SCALE,
                                     sliding_window=window)
    assert pkv.check_device_errors() == 0
    assert bool(((o.cpu().double() - out).abs() <= tol_o).all()) and bool(((l.cpu().double() - lse).abs() <= tol_l).all())


THREADS = r"""
#include <thread>
#include "pkv.h"
struct Call {
  const void *q, *kc, *kp, *vc, *vp;
  const int32_t *bt, *lens;
  int32_t max_blocks, bound, seqs, block;
  int64_t num_blocks;
  void *out, *ws;
  size_t ws_bytes;
  void *stream;
};
static pkv_status one(const Call &c) {
  if (c.kp != nullptr)
    return pkv_paged_decode_attn_q4(c.q, c.kc, c.kp, c.vc, c.vp, c.bt, c.max_blocks, c.lens, c.bound, c.seqs, 2, 1, 128, 32,
                                    c.block, c.num_blocks, 0.088f, 0, c.out, nullptr, nullptr, 0, c.ws, c.ws_bytes, c.stream);
  return pkv_paged_decode_attn(c.q, c.kc, c.vc, c.bt, c.max_blocks, c.lens, c.bound, c.seqs, 2, 1, 128, c.block, c.num_blocks,
                               0.088f, 0, c.out, nullptr, c.ws, c.ws_bytes, c.stream);
}
// n calls of each of two threads; how many failed
extern "C" void two_threads(const Call *calls, int n, int *failed) {
  auto run = [&](int i) {
    for (int k = 0; k < n; ++k) failed[i] += one(calls[i]) != PKV_OK;
  };
  std::thread other(run, 1);
  run(0);
  other.join();
}
"""


@gpu
@pytest.mark.parametrize("q4", [False, True])
def test_host_threads_with_calls_of_their_own_sizes(L, q4, tmp_path):
    """Two host threads, each with its stream, buffers and number of sequences: every
    call is launched."""
    (tmp_path / "threads.cpp").write_text(THREADS)
    here = os.path.dirname(pkv.LIBRARY_PATH)
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-pthread", str(tmp_path / "threads.cpp"), "-I",
                    os.path.join(os.path.dirname(here), "include"), "-L", here, "-Wl,-rpath," + here, "-l:libpkv.so", "-o",
                    str(tmp_path / "threads.so")], check=True)
    block, ctx, bound = 16, 16, 20000
    P, i32 = ctypes.c_void_p, ctypes.c_int32

    class Call(ctypes.Structure):
        _fields_ = ([(n, P) for n in ("q", "kc", "kp", "vc", "vp", "bt", "lens")] +
                    [(n, i32) for n in ("max_blocks", "bound", "seqs", "block")] +
                    [("num_blocks", ctypes.c_int64), ("out", P), ("ws", P), ("ws_bytes", ctypes.c_size_t), ("stream", P)])

    c = Q.Cache(18, [ctx], 1, block, 32)
    kc, vc, _ = c.cuda()
    k16 = torch.randn(c.num_blocks, block, 1, 128).to(torch.bfloat16).cuda()
    caches = [x.data_ptr() for x in (*kc, *vc)] if q4 else [k16.data_ptr(), None, k16.data_ptr(), None]
    calls, keep = (Call * 2)(), []
    for i, S in enumerate((1, 1000)):
        q = torch.randn(S, 2, 128).to(torch.bfloat16).cuda()
        bt = torch.full((S, bound // block), -1, dtype=torch.int32, device="cuda")
        bt[:, 0] = int(c.tables[0, 0])
        lens = torch.full((S,), ctx, dtype=torch.int32, device="cuda")
        out, stream = torch.full_like(q, float("nan")), torch.cuda.Stream()
        ws = pkv.new_q4_decode_workspace(S, 2, 1, bound) if q4 else pkv.new_decode_workspace(S, 2, 1, 128, bound)
        calls[i] = Call(q.data_ptr(), *caches, bt.data_ptr(), lens.data_ptr(), bt.shape[1], bound, S, block, c.num_blocks,
                        out.data_ptr(), ws.data_ptr(), ws.numel(), stream.cuda_stream)
        keep.append((q, bt, lens, out, stream, ws))
    torch.cuda.synchronize()
    failed = (ctypes.c_int * 2)()
    ctypes.CDLL(str(tmp_path / "threads.so")).two_threads(calls, 20000, failed)
    torch.cuda.synchronize()
    assert list(failed) == [0, 0]
    assert all(bool(torch.isfinite(k[3]).all()) for k in keep)
    assert pkv.check_device_errors() == 0


@gpu
@pytest.mark.parametrize("total,bound", [(12, 3000), (600, 400)])  # by rows, widened
def test_prefill_in_a_graph_replayed_for_other_segments(L, total, bound):
    """Captured with bounds; replayed for batches cut up differently, with padding
    rows and empty segments, on a stream of its own: the eager call's bits."""
    batches = {12: [([4, 4, 4], [3000, 100, 700]), ([1, 0, 11], [1, 0, 2500]), ([0, 0, 5], [0, 9, 5])],
               600: [([200, 200, 200], [400, 300, 200]), ([400, 0, 150], [400, 0, 151]), ([1, 2, 3], [400, 2, 400])]}[total]
    heads, gqa, block = 2, 2, 32
    c = Q.Cache(12, [bound] * 3, heads, block, 64)
    kc, vc, bt = c.cuda()
    q = torch.randn(total, heads * gqa, 128, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16).cuda()
    cu_q, cu_k = _cu(batches[0][0]), _cu(batches[0][1])
    total_k = 3 * bound
    ws = pkv.new_q4_prefill_workspace(3, total_k, bound, heads)
    out, lse = torch.zeros_like(q), torch.zeros(total, heads * gqa, device="cuda")

    def call(stream=None, o=out, l=lse):
        pkv.paged_prefill_attn_q4(q, kc, vc, cu_q, cu_k, bt, min(total, bound), bound, total_k, SCALE, out=o, lse=l, workspace=ws,
                                  stream=stream)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        call(side)
        with torch.cuda.graph(graph, stream=side):
            call(side)
    torch.cuda.synchronize()
    for q_lens, k_lens in batches:
        cu_q.copy_(_cu(q_lens))
        cu_k.copy_(_cu(k_lens))
        out.fill_(7)
        lse.fill_(7)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        got, got_l, n = out.clone(), lse.clone(), sum(q_lens)
        c.lens = k_lens
        want, want_l, tol_o, tol_l = _prefill_plain(c, q.cpu()[:n], q_lens, gqa, 0)
        assert bool(((got[:n].cpu().double() - want).abs() <= tol_o).all())
        assert bool(((got_l[:n].cpu().double() - want_l).abs() <= tol_l).all())
        assert bool((got[n:] == 7).all()) and bool((got_l[n:] == 7).all())     # rows behind the last segment
        eager, eager_l = torch.full_like(out, 7), torch.full_like(lse, 7)
        call(None, eager, eager_l)
        assert torch.equal(eager, got) and torch.equal(eager_l, got_l)
    assert pkv.check_device_errors() == 0


@gpu
def test_prefill_equals_the_bf16_call_on_the_same_values(L):
    """The values are bf16 by definition: widening the cache by hand and calling
    the bf16 prefill gives the same bits."""
    q_lens, k_lens = [100, 260], [400, 260]
    c = Q.Cache(12, k_lens, 4, 128, 32)
    q = torch.randn(360, 8, 128).to(torch.bfloat16).cuda()
    kc, vc, bt = c.cuda()
    o, l = pkv.paged_prefill_attn_q4(q, kc, vc, _cu(q_lens), _cu(k_lens), bt, 260, 400, 660, SCALE)
    slots = torch.arange(c.num_blocks * 128, dtype=torch.int32, device="cuda")
    k16, v16 = (x.view(c.num_blocks, 128, 4, 128) for x in pkv.kv_load_q4(kc, vc, slots))
    o16, l16 = pkv.paged_prefill_attn(q, k16, v16, _cu(q_lens), _cu(k_lens), bt, 260, 400, SCALE)
    assert pkv.check_device_errors() == 0
    assert torch.equal(o, o16) and torch.equal(l, l16)
