"""Norms and position rotation of queries and keys, alone and on the way into the cache, against the
plain 64-bit form in heads_plain.py; and the refusals of each call."""
import ctypes
import struct

import pytest
import torch

import heads_plain as P
import paged_kv_attention_22_gb300 as pkv
from paged_kv_attention_22_gb300 import build as pkv_build


@pytest.fixture(scope="module")
def L():
    pkv_build.build()
    return pkv.lib()


# ------------------------------------------------------------------ CPU: rotations and refusals

def _turns(rope):
    return struct.unpack("<iifi64Q", rope.data)[4:]


@pytest.mark.parametrize("R", [0, 8, 64, 96, 128])
@pytest.mark.parametrize("scaling", [None, "linear", "ntk", "yarn"])
def test_frequencies(L, R, scaling):
    how = dict(factor=4.0, original=4096) if scaling else {}
    want, magnitude = P.frequencies(R, 1e4, scaling, **how)
    if "original" in how:
        how["original_positions"] = how.pop("original")
    rope = pkv.rope(R, base=1e4, scaling=scaling, interleaved=True, **how)
    assert (rope.rotary_dim, rope.interleaved) == (R, True)
    assert abs(rope.magnitude - magnitude) <= 2.0 ** -23 * magnitude
    got = _turns(rope)
    for w, f in zip(got, want):
        # a power, a product or two and the division by 2 pi: a few roundings of 2^-53
        assert abs(w / 2.0 ** 64 - f / (2 * 3.141592653589793)) <= 2.0 ** -49 * f
    assert all(w == 0 for w in got[R // 2:])


def test_given_frequencies(L):
    rope = pkv.rope(16, frequencies=[0.0, 1.0, -1.0, 2 * 3.141592653589793 * 3.25, -1e-300, 1e3, 0.5, 2.0], magnitude=-0.5)
    w = _turns(rope)
    assert rope.magnitude == -0.5 and w[0] == 0 and w[4] == 0
    assert abs(w[1] + w[2] - 2 ** 64) <= 2 ** 12          # opposite angles
    assert abs(w[3] / 2.0 ** 64 - 0.25) <= 2.0 ** -49     # whole turns vanish


def test_rope_refuses(L):
    for bad in (4, 12, 129, 136):
        with pytest.raises(pkv.PkvError, match="UNSUPPORTED"):
            pkv.rope(bad)
    for bad in (dict(base=1.0), dict(base=float("inf")), dict(base=float("nan")), dict(rotary_dim=-8),
                dict(scaling="linear", factor=0.0), dict(scaling="ntk", factor=float("nan")),
                dict(scaling="ntk", base=1e300, factor=1e300),
                dict(scaling="yarn", factor=4.0), dict(scaling="yarn", factor=0.5, original_positions=4096),
                dict(scaling="yarn", factor=4.0, original_positions=4096, beta_fast=1.0, beta_slow=2.0),
                dict(scaling="yarn", factor=4.0, original_positions=4096, beta_slow=0.0),
                dict(scaling="yarn", factor=4.0, original_positions=4096, beta_fast=float("inf")),
                dict(rotary_dim=8, frequencies=[1.0, 2.0, float("nan"), 3.0]),
                dict(rotary_dim=8, frequencies=[1.0] * 4, magnitude=float("inf"))):
        with pytest.raises(pkv.PkvError, match="INVALID_ARG"):
            pkv.rope(**bad)
    for bad in (dict(scaling="cubic"), dict(magnitude=2.0), dict(rotary_dim=8, frequencies=[1.0]),
                dict(rotary_dim=8, frequencies=[1.0] * 4, scaling="linear")):
        with pytest.raises(ValueError):
            pkv.rope(**bad)
    assert L.pkv_rope_init(None, 128, 0, 1e4, 0, 1.0, 0, 0.0, 0.0) == pkv.PKV_ERR_INVALID_ARG
    made = pkv._RopeStruct()
    assert L.pkv_rope_init_frequencies(ctypes.byref(made), 8, 0, None, 1.0) == pkv.PKV_ERR_INVALID_ARG
    assert L.pkv_rope_init(ctypes.byref(made), 128, 0, 1e4, 4, 1.0, 0, 0.0, 0.0) == pkv.PKV_ERR_INVALID_ARG


FAKE = 0x10000


def _rope_struct(R=128, magnitude=1.0):
    made = pkv._RopeStruct()
    made.rotary_dim, made.magnitude = R, magnitude
    return ctypes.byref(made)


def _heads(L, **kw):
    a = dict(q=FAKE, qs=2048, k=FAKE, ks=1024, qw=None, kw=None, eps=1e-6, rope=_rope_struct(), pos=FAKE, T=4, Hq=16,
             Hkv=8, D=128, qo=FAKE, qos=2048, ko=FAKE, kos=1024)
    a.update(kw)
    return L.pkv_qk_norm_rope(a["q"], a["qs"], a["k"], a["ks"], a["qw"], a["kw"], a["eps"], a["rope"], a["pos"], a["T"],
                              a["Hq"], a["Hkv"], a["D"], a["qo"], a["qos"], a["ko"], a["kos"], None)


def _append(L, **kw):
    a = dict(q=FAKE, qs=2048, k=FAKE, ks=1024, v=FAKE, vs=1024, qw=None, kw=None, eps=1e-6, rope=_rope_struct(),
             pos=FAKE, sm=FAKE, T=4, Hq=16, Hkv=8, D=128, bs=16, NB=64, qo=FAKE, qos=2048, ko=FAKE, vo=FAKE)
    a.update(kw)
    return L.pkv_kv_append(a["q"], a["qs"], a["k"], a["ks"], a["v"], a["vs"], a["qw"], a["kw"], a["eps"], a["rope"],
                           a["pos"], a["sm"], a["T"], a["Hq"], a["Hkv"], a["D"], a["bs"], a["NB"], a["qo"], a["qos"],
                           a["ko"], a["vo"], None)


@pytest.mark.parametrize("call", [_heads, _append])
def test_calls_refuse(L, call):
    own = ("v", "sm", "vo") if call is _append else ()
    for null in ("q", "k", "qo", "ko", "pos") + own:
        assert call(L, **{null: None}) == pkv.PKV_ERR_INVALID_ARG, null
    for odd in ("q", "k", "qo", "ko", "qw", "kw") + (("v", "vo") if own else ()):
        assert call(L, **{odd: FAKE + 8}) == pkv.PKV_ERR_INVALID_ARG, odd
    for strides in ("qs", "ks", "qos") + (("vs",) if own else ("kos",)):
        assert call(L, **{strides: -1024}) == pkv.PKV_ERR_INVALID_ARG
        assert call(L, **{strides: 2052}) == pkv.PKV_ERR_INVALID_ARG
        assert call(L, **{strides: 1 << 50}) == pkv.PKV_ERR_INVALID_ARG
    assert call(L, qos=1024) == pkv.PKV_ERR_INVALID_ARG     # output rows that overlap
    for kw in (dict(T=-1), dict(Hq=-1), dict(Hkv=-1), dict(eps=-1.0), dict(eps=float("nan")), dict(D=0),
               dict(rope=_rope_struct(magnitude=float("nan")))):
        assert call(L, **kw) == pkv.PKV_ERR_INVALID_ARG, kw
    for kw in (dict(D=64), dict(rope=_rope_struct(12)), dict(rope=_rope_struct(136)), dict(T=1 << 30),
               dict(T=1, Hq=65536, qos=1 << 23), dict(T=1, Hkv=65536)):
        assert call(L, **kw) == pkv.PKV_ERR_UNSUPPORTED, kw
    assert call(L, T=0, q=None, k=None, pos=None, qo=None) == pkv.PKV_OK


def test_calls_refuse_what_is_theirs(L):
    assert _heads(L, kos=512) == pkv.PKV_ERR_INVALID_ARG
    assert _heads(L, Hq=0, Hkv=0, q=None, k=None, qo=None, ko=None) == pkv.PKV_OK
    assert _append(L, Hkv=0) == pkv.PKV_ERR_INVALID_ARG
    assert _append(L, bs=0) == pkv.PKV_ERR_INVALID_ARG
    assert _append(L, NB=0) == pkv.PKV_ERR_INVALID_ARG
    assert _append(L, NB=1 << 40) == pkv.PKV_ERR_UNSUPPORTED
    assert _append(L, NB=1 << 30, bs=16) == pkv.PKV_ERR_UNSUPPORTED


# ------------------------------------------------------------------ GPU

DEV = "cuda"
NAN_BITS = 0x7FC0


def _bits(t):
    return t.contiguous().view(torch.int16)


def _packed(T, Hq, Hkv, seed, spare=0):
    """q, k, v as parts of one projection [T, (Hq + 2 Hkv) * 128 + spare], and the whole."""
    g = torch.Generator().manual_seed(seed)
    whole = (torch.randn(T, (Hq + 2 * Hkv) * 128 + spare, generator=g) * 1.7).to(torch.bfloat16).to(DEV)
    parts, at = [], 0
    for H in (Hq, Hkv, Hkv):
        parts.append(whole[:, at:at + H * 128].unflatten(1, (H, 128)) if H else None)
        at += H * 128
    return parts, whole


def _weights(seed):
    g = torch.Generator().manual_seed(seed)
    return [(1 + 0.3 * torch.randn(128, generator=g)).to(torch.bfloat16).to(DEV) for _ in range(2)]


def _within(got, want_and_tol):
    want, tol = want_and_tol
    off = (got.double().cpu() - want).abs()
    assert bool((off <= tol).all()), float((off - tol).max())


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hkv", [(1, 1, 1), (1, 16, 8), (2, 3, 1), (7, 16, 8), (33, 5, 5), (301, 8, 2),
                                      (2000, 4, 2), (3001, 1, 1)])
@pytest.mark.parametrize("R,interleaved,norm,scaling", [(128, False, True, None), (128, True, False, "linear"),
                                                        (64, False, True, "yarn"), (96, True, True, "ntk"),
                                                        (8, False, False, None), (8, True, True, "yarn"),
                                                        (40, False, True, "linear"), (104, False, False, None),
                                                        (0, False, True, None)])
def test_norm_and_rotation(L, T, Hq, Hkv, R, interleaved, norm, scaling):
    (q, k, _), _ = _packed(T, Hq, Hkv, T + R)
    wq, wk = _weights(R) if norm else (None, None)
    pos = torch.randint(0, 200000, (T,), generator=torch.Generator().manual_seed(T)).to(torch.int32).to(DEV)
    how = dict(factor=8.0) if scaling else {}
    f, m = P.frequencies(R, 1e6, scaling, original=16384, **how)
    rope = pkv.rope(R, base=1e6, interleaved=interleaved, scaling=scaling, original_positions=16384, **how)
    got = pkv.qk_norm_rope(q, k, rope, pos, wq, wk, eps=1e-5)
    for x, w, y in ((q, wq, got[0]), (k, wk, got[1])):
        assert y.shape == x.shape and y.is_contiguous()
        _within(y, P.turned(x, w, pos, R, f, m, interleaved, eps=1e-5))
    assert pkv.check_device_errors() == 0


@pytest.mark.gpu
def test_far_and_negative_positions(L):
    (q, k, _), _ = _packed(6, 2, 2, 5)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, -1, 0, 1, 2 ** 24 + 1], dtype=torch.int32, device=DEV)
    f, m = P.frequencies(128, 1e4)
    for y, x in zip(pkv.qk_norm_rope(q, k, pkv.rope(128), pos), (q, k)):
        _within(y, P.turned(x, None, pos, 128, f, m))
    assert torch.equal(_bits(pkv.qk_norm_rope(q, k, pkv.rope(128), pos)[0][3]), _bits(q[3]))  # position 0 turns nothing


@pytest.mark.gpu
def test_without_a_rotation_positions_may_be_left_out(L):
    (q, k, _), _ = _packed(9, 4, 2, 6)
    wq, wk = _weights(3)
    for rope in (None, pkv.rope(0)):
        got = pkv.qk_norm_rope(q, k, rope, None, wq, wk)
        _within(got[0], P.turned(q, wq, torch.zeros(9), 0))
        _within(got[1], P.turned(k, wk, torch.zeros(9), 0))
    same = pkv.qk_norm_rope(q, k, None, None)
    assert torch.equal(_bits(same[0]), _bits(q)) and torch.equal(_bits(same[1]), _bits(k))


@pytest.mark.gpu
def test_weight_of_one_only(L):
    (q, k, _), _ = _packed(5, 3, 2, 7)
    wq, _ = _weights(4)
    pos = torch.arange(5, dtype=torch.int32, device=DEV)
    f, m = P.frequencies(128, 1e4)
    got = pkv.qk_norm_rope(q, k, pkv.rope(128), pos, q_weight=wq)
    _within(got[0], P.turned(q, wq, pos, 128, f, m))
    _within(got[1], P.turned(k, None, pos, 128, f, m))


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 500])
def test_in_place_within_a_packed_projection(L, T):
    (q, k, v), whole = _packed(T, 6, 3, 8, spare=64)
    wq, wk = _weights(5)
    pos = torch.arange(T, dtype=torch.int32, device=DEV) * 31
    want = pkv.qk_norm_rope(q, k, pkv.rope(128), pos, wq, wk)
    rest = _bits(whole[:, 9 * 128:])
    got = pkv.qk_norm_rope(q, k, pkv.rope(128), pos, wq, wk, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(_bits(q), _bits(want[0])) and torch.equal(_bits(k), _bits(want[1]))
    assert torch.equal(_bits(whole[:, 9 * 128:]), rest)


@pytest.mark.gpu
def test_queries_or_keys_alone(L):
    (q, k, _), _ = _packed(11, 4, 2, 9)
    pos = torch.arange(11, dtype=torch.int32, device=DEV)
    both = pkv.qk_norm_rope(q, k, pkv.rope(128), pos)
    a, none = pkv.qk_norm_rope(q, None, pkv.rope(128), pos)
    assert none is None and torch.equal(_bits(a), _bits(both[0]))
    none, b = pkv.qk_norm_rope(None, k, pkv.rope(128), pos)
    assert none is None and torch.equal(_bits(b), _bits(both[1]))


@pytest.mark.gpu
def test_a_broadcast_token_as_input(L):
    (q, k, _), _ = _packed(1, 2, 1, 10)
    pos = torch.arange(40, dtype=torch.int32, device=DEV)
    f, m = P.frequencies(128, 1e4)
    got = pkv.qk_norm_rope(q.expand(40, 2, 128), k.expand(40, 1, 128), pkv.rope(128), pos)
    _within(got[0], P.turned(q.expand(40, 2, 128), None, pos, 128, f, m))


@pytest.mark.gpu
def test_rows_of_zeros_nan_and_infinity_stay_their_own(L):
    (q, k, _), _ = _packed(8, 2, 2, 11)
    q, k = q.clone(), k.clone()
    q[1], q[2, 0, 5], q[3, 1, 7] = 0, float("nan"), float("inf")
    wq, wk = _weights(6)
    pos = torch.arange(8, dtype=torch.int32, device=DEV)
    got, _ = pkv.qk_norm_rope(q, k, pkv.rope(128), pos, wq, wk)
    assert bool((got[1] == 0).all())
    assert bool(torch.isnan(got[2, 0]).all()) and not bool(torch.isnan(got[2, 1]).any())
    f, m = P.frequencies(128, 1e4)
    want, tol = P.turned(q, wq, pos, 128, f, m)
    fine = torch.isfinite(want)
    assert bool(((got.double().cpu() - want).abs()[fine] <= tol[fine]).all())
    assert not bool(torch.isfinite(got[3, 1, 7]))


@pytest.mark.gpu
@pytest.mark.parametrize("R,interleaved", [(64, False), (40, False), (48, True), (72, True), (0, False)])
def test_what_is_not_rotated_passes_as_it_is(L, R, interleaved):
    (q, k, _), _ = _packed(5, 3, 1, 21)
    q = q.clone()
    q[..., R + (128 - R) // 2] = float("-inf")
    q[1, 1, 127], q[2, 2, R] = float("nan"), -0.0
    pos = torch.tensor([0, 1, 77, 4096, 100000], dtype=torch.int32, device=DEV)
    got, _ = pkv.qk_norm_rope(q, k, pkv.rope(R, interleaved=interleaved), pos)
    fine = torch.isnan(q[..., R:])
    assert torch.equal(torch.isnan(got[..., R:]), fine)
    assert torch.equal(_bits(got[..., R:])[~fine], _bits(q[..., R:])[~fine])


def _cache(NB, bs, H):
    return [torch.full((NB, bs, H, 128), NAN_BITS, dtype=torch.int16, device=DEV).view(torch.bfloat16) for _ in range(2)]


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hkv,bs", [(1, 2, 1, 16), (1, 16, 8, 256), (5, 3, 3, 48), (64, 16, 8, 256),
                                         (333, 8, 2, 16), (4000, 4, 2, 64)])
@pytest.mark.parametrize("R,interleaved", [(128, False), (64, True), (0, False)])
def test_append_is_rotation_then_store(L, T, Hq, Hkv, bs, R, interleaved):
    (q, k, v), _ = _packed(T, Hq, Hkv, T * 3 + R)
    wq, wk = _weights(7)
    NB = -(-T // bs) + 2
    g = torch.Generator().manual_seed(T)
    slots = torch.randperm(NB * bs, generator=g)[:T].to(torch.int32)
    slots[::5] = -1
    slots = slots.to(DEV)
    pos = torch.randint(0, 40960, (T,), generator=g).to(torch.int32).to(DEV)
    rope = pkv.rope(R, base=1e6, interleaved=interleaved)
    kc, vc = _cache(NB, bs, Hkv)
    want_kc, want_vc = _cache(NB, bs, Hkv)
    want_q, want_k = pkv.qk_norm_rope(q, k, rope, pos, wq, wk)
    pkv.kv_store(want_k, v.contiguous(), want_kc, want_vc, slots)
    got = pkv.kv_append(q, k, v, rope, pos, kc, vc, slots, wq, wk)
    assert torch.equal(_bits(got), _bits(want_q))
    assert torch.equal(_bits(kc), _bits(want_kc)) and torch.equal(_bits(vc), _bits(want_vc))
    assert pkv.check_device_errors() == 0


@pytest.mark.gpu
def test_append_keys_and_values_alone(L):
    (_, k, v), _ = _packed(6, 2, 2, 12)
    kc, vc = _cache(2, 16, 2)
    slots = torch.tensor([3, 7, -1, 0, 31, 16], dtype=torch.int32, device=DEV)
    assert pkv.kv_append(None, k, v, None, None, kc, vc, slots) is None
    want_kc, want_vc = _cache(2, 16, 2)
    pkv.kv_store(k.contiguous(), v.contiguous(), want_kc, want_vc, slots)
    assert torch.equal(_bits(kc), _bits(want_kc)) and torch.equal(_bits(vc), _bits(want_vc))


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [-2, 32, 2 ** 31 - 1, -2 ** 31])
def test_append_reports_slots_outside_the_pool(L, bad):
    (q, k, v), _ = _packed(3, 4, 2, 13)
    kc, vc = _cache(2, 16, 2)
    pos = torch.arange(3, dtype=torch.int32, device=DEV)
    slots = torch.tensor([5, bad, 9], dtype=torch.int32, device=DEV)
    got = pkv.kv_append(q, k, v, pkv.rope(128), pos, kc, vc, slots)
    assert pkv.check_device_errors() == pkv.DEVERR_SLOT
    assert pkv.check_device_errors() == 0
    want_kc, want_vc = _cache(2, 16, 2)
    want_q = pkv.kv_append(q, k, v, pkv.rope(128), pos, want_kc, want_vc,
                           torch.tensor([5, -1, 9], dtype=torch.int32, device=DEV))
    assert torch.equal(_bits(got), _bits(want_q))  # the queries are there all the same
    assert torch.equal(_bits(kc), _bits(want_kc)) and torch.equal(_bits(vc), _bits(want_vc))


@pytest.mark.gpu
def test_no_tokens(L):
    (q, k, v), _ = _packed(0, 4, 2, 14)
    pos = torch.empty(0, dtype=torch.int32, device=DEV)
    got = pkv.qk_norm_rope(q, k, pkv.rope(128), pos)
    assert got[0].shape == (0, 4, 128)
    kc, vc = _cache(1, 16, 2)
    assert pkv.kv_append(q, k, v, pkv.rope(128), pos, kc, vc, pos).shape == (0, 4, 128)
    assert bool((_bits(kc) == NAN_BITS).all())


@pytest.mark.gpu
def test_binding_refuses(L):
    (q, k, v), _ = _packed(3, 4, 2, 15)
    pos = torch.arange(3, dtype=torch.int32, device=DEV)
    kc, vc = _cache(1, 16, 2)
    r = pkv.rope(128)
    for bad in (lambda: pkv.qk_norm_rope(q.float(), k, r, pos), lambda: pkv.qk_norm_rope(q, k, r, pos.long()),
                lambda: pkv.qk_norm_rope(q.cpu(), k, r, pos), lambda: pkv.qk_norm_rope(q, k[:2], r, pos),
                lambda: pkv.qk_norm_rope(q, k, r, pos[:2]), lambda: pkv.qk_norm_rope(q, k, r, pos, q_weight=kc[0, 0, 0, :64]),
                lambda: pkv.qk_norm_rope(q.transpose(0, 1).contiguous().transpose(0, 1), k, r, pos),
                lambda: pkv.qk_norm_rope(q[..., :64], k, r, pos), lambda: pkv.qk_norm_rope(q, k, r, pos, q_out=k),
                lambda: pkv.kv_append(q, k, None, r, pos, kc, vc, pos), lambda: pkv.kv_append(q, k, v[:, :1], r, pos, kc, vc, pos),
                lambda: pkv.kv_append(q, k, v, r, pos, kc, vc[:, :8], pos), lambda: pkv.kv_append(q, q, q, r, pos, kc, vc, pos),
                lambda: pkv.kv_append(q, k, v, r, pos, kc, vc, pos[:1])):
        with pytest.raises((TypeError, ValueError)):
            bad()
    with pytest.raises(pkv.PkvError):
        pkv.qk_norm_rope(q, k, r, None)
    with pytest.raises(pkv.PkvError):  # every row of the output would be the same memory
        pkv.qk_norm_rope(q, k, r, pos, q_out=torch.empty_like(q)[:1].expand(3, 4, 128))


@pytest.mark.gpu
@pytest.mark.parametrize("programmatic", [True, False])
def test_captured_and_replayed_on_another_stream(L, programmatic):
    (q, k, v), whole = _packed(20, 4, 2, 16)
    wq, wk = _weights(8)
    pos = torch.arange(20, dtype=torch.int32, device=DEV)
    slots = torch.arange(20, dtype=torch.int32, device=DEV)
    kc, vc = _cache(2, 16, 2)
    rope = pkv.rope(128)
    q_out = torch.empty(20, 4, 128, dtype=torch.bfloat16, device=DEV)
    pkv.set_programmatic_launch(programmatic)
    try:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            pkv.qk_norm_rope(q, k, rope, pos, wq, wk, q_out=q, k_out=k)
            pkv.kv_append(q, k, v, rope, pos, kc, vc, slots, wq, wk, q_out=q_out)
        _, new = _packed(20, 4, 2, 17)
        whole.copy_(new)
        pos.add_(1000)
        slots.copy_(torch.arange(31, 11, -1, dtype=torch.int32))
        want_kc, want_vc = _cache(2, 16, 2)
        a, b = pkv.qk_norm_rope(q, k, rope, pos, wq, wk)
        want_q = pkv.kv_append(a, b, v, rope, pos, want_kc, want_vc, slots, wq, wk)
        graph.replay()
        torch.cuda.synchronize()
    finally:
        pkv.set_programmatic_launch(True)
    assert torch.equal(_bits(q_out), _bits(want_q))
    assert torch.equal(_bits(kc), _bits(want_kc)) and torch.equal(_bits(vc), _bits(want_vc))
    with torch.cuda.stream(side):
        again = pkv.qk_norm_rope(a, b, rope, pos, wq, wk, stream=side)
    side.synchronize()
    assert torch.equal(_bits(again[0]), _bits(want_q))
