"""Decode under a window with sinks, against the plain 64-bit form in attn_plain.py, over caches that
hold NaN wherever no query looks; and the refusals of the call."""
import pytest
import torch

import paged_kv_attention_22_gb300 as pkv
from attn_plain import SCALE, Batch
from paged_kv_attention_22_gb300 import build as pkv_build

DEV = "cuda"


@pytest.fixture(scope="module")
def L():
    pkv_build.build()
    return pkv.lib()


FAKE = 0x10000


def _call(L, **kw):
    a = dict(kn=None, vn=None, sm=None, q=FAKE, kc=FAKE, vc=FAKE, bt=FAKE, mb=4, cl=FAKE, mcl=64, S=2, Hq=16, Hkv=8,
             D=128, bs=16, NB=64, scale=0.088, win=16, sinks=4, out=FAKE, lse=None, ws=FAKE, wsb=1 << 30, flags=0)
    a.update(kw)
    return L.pkv_paged_decode_attn_sinks(a["kn"], a["vn"], a["sm"], a["q"], a["kc"], a["vc"], a["bt"], a["mb"], a["cl"],
                                         a["mcl"], a["S"], a["Hq"], a["Hkv"], a["D"], a["bs"], a["NB"], a["scale"],
                                         a["win"], a["sinks"], a["out"], a["lse"], a["ws"], a["wsb"], a["flags"], None)


def test_refuses(L):
    for null in ("q", "kc", "vc", "bt", "cl", "out"):
        assert _call(L, **{null: None}) == pkv.PKV_ERR_INVALID_ARG
    for odd in ("q", "kc", "vc", "out", "ws"):
        assert _call(L, **{odd: FAKE + 8}) == pkv.PKV_ERR_INVALID_ARG
    some = dict(kn=FAKE, vn=FAKE, sm=FAKE)
    for null in some:  # the new rows all or none
        assert _call(L, **{**some, null: None}) == pkv.PKV_ERR_INVALID_ARG
        assert _call(L, **{null: FAKE}) == pkv.PKV_ERR_INVALID_ARG
    assert _call(L, **{**some, "kn": FAKE + 8}) == pkv.PKV_ERR_INVALID_ARG
    assert _call(L, sinks=-1) == pkv.PKV_ERR_INVALID_ARG
    assert _call(L, win=-1) == pkv.PKV_ERR_INVALID_ARG
    assert _call(L, flags=1) == pkv.PKV_ERR_INVALID_ARG       # stable inputs go with new rows
    assert _call(L, **some, flags=2) == pkv.PKV_ERR_INVALID_ARG
    assert _call(L, S=0) == pkv.PKV_ERR_INVALID_ARG
    assert _call(L, scale=float("nan")) == pkv.PKV_ERR_INVALID_ARG
    assert _call(L, D=64) == pkv.PKV_ERR_UNSUPPORTED
    assert _call(L, Hq=24) == pkv.PKV_ERR_UNSUPPORTED
    assert _call(L, bs=24) == pkv.PKV_ERR_UNSUPPORTED
    assert _call(L, S=2000) == pkv.PKV_ERR_UNSUPPORTED
    assert _call(L, ws=None) == pkv.PKV_ERR_WORKSPACE_TOO_SMALL


def _run(b, **kw):
    kw = dict(dict(sliding_window=b.window, num_sinks=b.sinks), **kw)
    return pkv.paged_decode_attn_sinks(b.q, b.kc, b.vc, b.bt, b.lens, max(b.keys), b.scale, **kw)


# lengths around units, blocks, the window and the sinks
LENGTHS = [1, 2, 15, 16, 17, 31, 33, 48, 63, 64, 65, 100, 129, 300]


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,H", [(1, 1), (2, 1), (16, 8), (8, 8), (12, 3), (16, 4)])
@pytest.mark.parametrize("bs", [16, 48])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (17, 16), (33, 17), (40, 64), (100, 1000),
                                          (500, 4), (0, 4)])
def test_masks(L, Hq, H, bs, window, sinks):
    b = Batch(LENGTHS, [1] * len(LENGTHS), Hq, H, bs, window, sinks, seed=bs + window)
    b.check(*_run(b))
    assert pkv.check_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("ctas,variant", [(1, 0), (7, 1), (1000, 2), (0, 2), (0, 1)])
def test_launch_shapes(L, ctas, variant):
    b = Batch([700, 1, 90, 260, 1025], [1] * 5, 16, 8, 64, 200, 70, seed=3)
    pkv.decode_set_config(ctas, variant)
    try:
        b.check(*_run(b))
    finally:
        pkv.decode_set_config()
    assert pkv.check_device_errors() == 0


@pytest.mark.gpu
def test_long_streams(L):
    b = Batch([9000, 20000, 4097], [1] * 3, 16, 8, 256, 4096, 130, seed=4)
    b.check(*_run(b))
    b = Batch([30000], [1], 4, 1, 256, 20000, 300, seed=5)
    b.check(*_run(b))
    assert pkv.check_device_errors() == 0


@pytest.mark.gpu
def test_the_plain_call_where_nothing_is_hidden(L):
    b = Batch([40, 100, 7], [1] * 3, 16, 8, 16, 0, 0, seed=6)
    want = pkv.paged_decode_attn(b.q, b.kc, b.vc, b.bt, b.lens, 100, SCALE)
    got = _run(b, num_sinks=5)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    got = _run(b, sliding_window=2 ** 31 - 1, num_sinks=2 ** 31 - 1)
    b.check(*got)


@pytest.mark.gpu
@pytest.mark.parametrize("stable", [False, True])
def test_with_the_new_rows_stored(L, stable):
    keys = [1, 16, 17, 130, 300]
    b = Batch(keys, [1] * 5, 16, 8, 16, 40, 4, seed=7)
    new = [torch.stack([p[i][-1] for p in b.parts]).to(DEV) for i in (1, 2)]
    slots = torch.tensor([int(b.bt[s, (n - 1) // 16]) * 16 + (n - 1) % 16 for s, n in enumerate(keys)],
                         dtype=torch.int32, device=DEV)
    want = [c.clone() for c in (b.kc, b.vc)]
    for c in (b.kc, b.vc):  # the call has to put them there
        c.flatten(0, 1)[slots.long()] = float("nan")
    slots[2] = -1           # used as a key, not stored
    got = _run(b, k_new=new[0], v_new=new[1], slot_mapping=slots, stable_inputs=stable)
    b.check(*got)
    at = int(b.bt[2, 1]) * 16
    for c, w in zip((b.kc, b.vc), want):
        w.flatten(0, 1)[at] = float("nan")
        assert torch.equal(c.view(torch.int16), w.view(torch.int16))
    assert pkv.check_device_errors() == 0


@pytest.mark.gpu
def test_invalid_lengths_and_entries(L):
    b = Batch([100, 50, 80, 90], [1] * 4, 4, 2, 16, 30, 4, seed=8)
    b.lens[1] = 0
    b.bt[2, 0] = 10 ** 6
    out = torch.full_like(b.q, 7.0)
    got = _run(b, out=out)
    assert pkv.check_device_errors() == pkv.DEVERR_CONTEXT | pkv.DEVERR_BLOCK
    assert bool((got[0][1] == 7.0).all())
    b.check(*got, skip=(1, 2))


@pytest.mark.gpu
def test_replayed_for_grown_sequences(L):
    b = Batch([33, 47, 64], [1] * 3, 8, 4, 16, 20, 3, seed=9)
    grown = Batch([34, 48, 65], [1] * 3, 8, 4, 16, 20, 3, seed=10)
    q, kc, vc, lens = b.q.clone(), grown.kc.clone(), grown.vc.clone(), b.lens.clone()
    bt = torch.full_like(grown.bt, -1)
    bt[:, : b.bt.shape[1]] = b.bt
    kc[: b.kc.shape[0]], vc[: b.vc.shape[0]] = b.kc, b.vc
    out, lse = torch.empty_like(q), torch.empty(3, 8, device=DEV)
    ws = pkv.new_decode_workspace(3, 8, 4, 128, 128)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        pkv.paged_decode_attn_sinks(q, kc, vc, bt, lens, 128, SCALE, 20, 3, out=out, lse=lse, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    b.check(out, lse)
    for to, new in ((q, grown.q), (kc, grown.kc), (vc, grown.vc), (lens, grown.lens), (bt, grown.bt)):
        to.copy_(new)
    graph.replay()
    torch.cuda.synchronize()
    grown.check(out, lse)


@pytest.mark.gpu
def test_binding_refuses(L):
    b = Batch([40, 20], [1] * 2, 4, 2, 16, 10, 2, seed=11)
    for bad in (dict(num_sinks=-1), dict(sliding_window=-1)):
        with pytest.raises(pkv.PkvError):
            _run(b, **bad)
    rows = b.kc[0, :2].contiguous()
    slots = torch.zeros(2, dtype=torch.int32, device=DEV)
    for bad in (dict(k_new=rows), dict(k_new=rows, v_new=rows, slot_mapping=slots[:1]),
                dict(k_new=rows[:, :1].contiguous(), v_new=rows, slot_mapping=slots)):
        with pytest.raises(ValueError):
            _run(b, **bad)
    with pytest.raises(pkv.PkvError):
        _run(b, stable_inputs=True)
    with pytest.raises(ValueError):
        pkv.paged_decode_attn_sinks(b.q, b.kc, b.vc[:, :8], b.bt, b.lens, 40, SCALE, 10, 2)
