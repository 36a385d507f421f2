"""Attention of chunks of new tokens over the paged cache, against the plain 64-bit form in
attn_plain.py, over caches that hold NaN wherever no query looks; and the refusals of the call."""
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
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, cq=FAKE, cl=FAKE, bt=FAKE, mb=4, S=2, T=8, mq=4, mcl=64, Hq=16, Hkv=8, D=128,
             bs=16, NB=64, scale=0.088, win=0, sinks=0, out=FAKE, lse=None, ws=FAKE, wsb=1 << 30)
    a.update(kw)
    return L.pkv_paged_chunk_attn(a["q"], a["kc"], a["vc"], a["cq"], a["cl"], a["bt"], a["mb"], a["S"], a["T"], a["mq"],
                                  a["mcl"], a["Hq"], a["Hkv"], a["D"], a["bs"], a["NB"], a["scale"], a["win"],
                                  a["sinks"], a["out"], a["lse"], a["ws"], a["wsb"], None)


def test_refuses(L):
    for null in ("q", "kc", "vc", "cq", "cl", "bt", "out"):
        assert _call(L, **{null: None}) == pkv.PKV_ERR_INVALID_ARG
    for odd in ("q", "kc", "vc", "out", "ws"):
        assert _call(L, **{odd: FAKE + 8}) == pkv.PKV_ERR_INVALID_ARG
    for kw in (dict(S=-1), dict(T=-1), dict(mq=-1), dict(mcl=-1), dict(mq=65), dict(scale=float("inf")),
               dict(win=-1), dict(sinks=-1), dict(Hq=0), dict(bs=0), dict(mb=0)):
        assert _call(L, **kw) == pkv.PKV_ERR_INVALID_ARG, kw
    for kw in (dict(D=64), dict(Hq=24), dict(Hq=64), dict(Hq=12), dict(bs=24), dict(S=1025), dict(NB=1 << 40),
               dict(mcl=(1 << 30) + 1, mb=1 << 27)):
        assert _call(L, **kw) == pkv.PKV_ERR_UNSUPPORTED, kw
    assert _call(L, ws=None) == pkv.PKV_ERR_WORKSPACE_TOO_SMALL
    for kw in (dict(S=0), dict(T=0, q=None, out=None), dict(mq=0, ws=None)):
        assert _call(L, **kw) == pkv.PKV_OK, kw
    assert L.pkv_chunk_workspace_size(0, 16, 8, 128) == 0
    assert L.pkv_chunk_workspace_size(1, 12, 8, 128) == 0
    assert L.pkv_chunk_workspace_size(1, 16, 8, 64) == 0
    if torch.cuda.is_available():
        n = L.pkv_chunk_workspace_size(1, 16, 8, 128)
        assert n > 0 and n == L.pkv_chunk_workspace_size(1024, 16, 4, 128)
        assert _call(L, wsb=n - 1) == pkv.PKV_ERR_WORKSPACE_TOO_SMALL


def _run(b, **kw):
    kw = dict(dict(sliding_window=b.window, num_sinks=b.sinks), **kw)
    return pkv.paged_chunk_attn(b.q, b.kc, b.vc, b.cu, b.lens, b.bt, max(b.new), max(b.keys), b.scale, **kw)


# (keys, new tokens): around tiles, blocks and steps; empty segments among them
TINY = [(1, 1), (2, 1), (2, 2), (17, 3), (64, 64), (100, 0), (127, 5), (128, 1), (129, 2), (130, 130), (300, 65)]
LONG = [(1000, 1), (1, 1), (0, 0), (640, 5), (513, 300), (257, 257), (2500, 16)]


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,H", [(1, 1), (2, 1), (16, 8), (12, 3), (3, 3), (16, 4)])
@pytest.mark.parametrize("bs", [16, 48, 256])
@pytest.mark.parametrize("segments", [TINY, LONG], ids=["tiny", "long"])
def test_causal(L, Hq, H, bs, segments):
    keys, new = map(list, zip(*segments))
    b = Batch(keys, new, Hq, H, bs, 0, 0, seed=bs + Hq)
    b.check(*_run(b), rounded=True)
    assert pkv.check_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,H", [(2, 2), (16, 8), (8, 2)])
@pytest.mark.parametrize("bs", [16, 48, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (40, 0), (100, 17), (128, 128), (129, 200),
                                          (300, 300), (1000, 5), (0, 9)])
@pytest.mark.parametrize("segments", [TINY, LONG], ids=["tiny", "long"])
def test_window_and_sinks(L, Hq, H, bs, window, sinks, segments):
    keys, new = map(list, zip(*segments))
    b = Batch(keys, new, Hq, H, bs, window, sinks, seed=bs + window)
    b.check(*_run(b), rounded=True)
    assert pkv.check_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("segments,Hq,H,window,sinks", [
    ([(20000, 3)], 2, 1, 0, 0),                     # one tile over every SM
    ([(20000, 9), (9000, 20)], 16, 8, 0, 0),
    ([(30000, 2)], 4, 1, 20000, 300),
    ([(6000, 2500)], 4, 2, 0, 0),                   # many tiles of one head, 40 a head
    ([(9000, 5000)], 1, 1, 700, 130),
    ([(5, 1)] * 900 + [(3000, 40)] + [(1, 1)] * 100, 2, 1, 0, 0),
    ([(130, 130)] * 200, 4, 2, 0, 0),
])
def test_shares_of_the_work(L, segments, Hq, H, window, sinks):
    keys, new = map(list, zip(*segments))
    b = Batch(keys, new, Hq, H, 64, window, sinks, seed=len(segments))
    b.check(*_run(b), rounded=True)
    assert pkv.check_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,H", [(16, 8), (16, 16), (16, 4)])
@pytest.mark.parametrize("bs", [16, 256])
def test_long_chunks(L, Hq, H, bs):
    # long enough that two row tiles pass a K/V tile; one segment is empty, its length nothing
    keys, new = [1250, 1300, 0, 1501, 1280], [1250, 1153, 0, 1201, 1280]
    b = Batch(keys, new, Hq, H, bs, 0, 0, seed=bs + H, extra_rows=40)
    b.lens[2] = -7
    out, lse = torch.full_like(b.q, 7.0), torch.full((b.q.shape[0], Hq), 7.0, device=DEV)
    _run(b, out=out, lse=lse)
    b.check(out, lse, rounded=True)
    assert bool((out[b.rows:] == 7).all()) and bool((lse[b.rows:] == 7).all())
    assert torch.equal(_run(b, with_lse=False)[0][:b.rows], out[:b.rows])
    assert pkv.check_device_errors() == 0
    # a length that is too short: refused by itself, its rows left as they were
    b.lens[3] = 1200
    out, lse = torch.full_like(out, 7.0), torch.full_like(lse, 7.0)
    _run(b, out=out, lse=lse)
    assert pkv.check_device_errors() == pkv.DEVERR_SEQLENS
    b.check(out, lse, rounded=True, skip=(3,))
    rows = b.parts[3][0]
    assert bool((out[rows] == 7).all()) and bool((lse[rows] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [-0.1, 0.0, 1e-3, 2.0])
def test_scales(L, scale):
    b = Batch([300, 90], [70, 4], 4, 2, 16, 100, 5, seed=2, scale=scale)
    b.check(*_run(b), rounded=True)


@pytest.mark.gpu
def test_large_logits(L):
    # maxima that grow along the keys, some by far more than the lazy bound
    b = Batch([700, 300], [5, 140], 8, 4, 16, 0, 0, seed=3, spread=6.0)
    b.check(*_run(b), rounded=True)


@pytest.mark.gpu
def test_single_tokens_are_decode(L):
    keys = [1, 60, 700, 1500]
    b = Batch(keys, [1] * 4, 16, 8, 64, 0, 0, seed=4)
    out, lse = _run(b)
    want, want_lse = pkv.paged_decode_attn(b.q, b.kc, b.vc, b.bt, b.lens, 1500, SCALE)
    # each within its rounding of the same numbers; the chunk's weights are rounded as well
    assert float((out.float() - want.float()).abs().max()) <= 2.0 ** -6 * float(want.float().abs().max())
    assert float((lse - want_lse).abs().max()) <= 1e-4


@pytest.mark.gpu
def test_prefill_gives_the_same(L):
    keys, new = [900, 64, 300], [500, 64, 7]
    b = Batch(keys, new, 16, 8, 64, 0, 0, seed=5)
    out, lse = _run(b)
    cu_k = torch.tensor([0] + keys).cumsum(0).to(torch.int32).to(DEV)
    want, want_lse = pkv.paged_prefill_attn(b.q, b.kc, b.vc, b.cu, cu_k, b.bt, 500, 900, SCALE)
    assert float((out.float() - want.float()).abs().max()) <= 2.0 ** -6 * float(want.float().abs().max())
    assert float((lse - want_lse).abs().max()) <= 1e-4


@pytest.mark.gpu
def test_rows_behind_the_last_sequence_are_left(L):
    b = Batch([300, 20], [9, 3], 8, 4, 16, 0, 0, seed=6, extra_rows=150)
    out, lse = torch.full_like(b.q, 7.0), torch.full((b.q.shape[0], 8), 7.0, device=DEV)
    _run(b, out=out, lse=lse)
    b.check(out, lse, rounded=True)
    assert bool((out[12:] == 7.0).all()) and bool((lse[12:] == 7.0).all())


@pytest.mark.gpu
def test_without_lse(L):
    b = Batch([300, 2000], [9, 3], 8, 4, 16, 0, 0, seed=7)
    out, none = _run(b, with_lse=False)
    assert none is None
    assert torch.equal(out, _run(b)[0])


@pytest.mark.gpu
def test_the_same_bits_again(L):
    b = Batch([5000, 640, 3000], [12, 5, 300], 16, 8, 64, 0, 0, seed=8)
    first = _run(b)
    for _ in range(3):
        again = _run(b)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


@pytest.mark.gpu
@pytest.mark.parametrize("what", ["short", "long", "past", "over", "table", "rows", "decreasing"])
def test_refused_segments(L, what):
    keys, new = [200, 150, 1200, 90], [5, 6, 40, 8]
    b = Batch(keys, new, 4, 2, 16, 0, 0, seed=9)
    lens, cu, kw = b.lens, b.cu, {}
    max_q, max_k, skip = 40, 1200, (1,)
    if what == "short":
        lens[1] = 5                       # fewer keys than queries
    elif what == "long":
        max_q, skip = 39, (2,)
    elif what == "past":
        lens[1] = 1201                    # above the bound
    elif what == "over":
        lens[1], max_k = 1201, 2000       # past the table (75 blocks of 16)
    elif what == "table":
        b.bt[1, 3] = 10 ** 6
    elif what == "rows":
        cu[4], skip = 60, (3,)            # rows past q's
    else:
        cu[2], skip = 4, (1, 2)           # 5 -> 4; the next segment is then too long
    out, lse = torch.full_like(b.q, 7.0), torch.full((b.q.shape[0], 4), 7.0, device=DEV)
    pkv.paged_chunk_attn(b.q, b.kc, b.vc, cu, lens, b.bt, max_q, max_k, SCALE, out=out, lse=lse)
    assert pkv.check_device_errors() == (pkv.DEVERR_BLOCK if what == "table" else pkv.DEVERR_SEQLENS)
    b.check(out, lse, rounded=True, skip=skip)
    if what != "table":
        for s in skip:
            assert bool((out[b.parts[s][0]] == 7.0).all()) and bool((lse[b.parts[s][0]] == 7.0).all())


@pytest.mark.gpu
def test_no_work(L):
    b = Batch([20, 30], [0, 0], 4, 2, 16, 0, 0, seed=10, extra_rows=3)
    out = torch.full_like(b.q, 7.0)
    pkv.paged_chunk_attn(b.q, b.kc, b.vc, b.cu, b.lens, b.bt, 1, 30, SCALE, out=out)
    assert pkv.check_device_errors() == 0 and bool((out == 7.0).all())
    empty = b.q[:0]
    assert pkv.paged_chunk_attn(empty, b.kc, b.vc, b.cu, b.lens, b.bt, 0, 30, SCALE)[0].shape == (0, 4, 128)


@pytest.mark.gpu
@pytest.mark.parametrize("programmatic", [True, False])
def test_replayed_for_other_segments(L, programmatic):
    first = Batch([900, 64, 1, 300], [3, 64, 1, 7], 8, 4, 16, 200, 4, seed=11)
    then = Batch([33, 640, 800, 129], [33, 1, 21, 20], 8, 4, 16, 200, 4, seed=12)
    assert first.rows == then.rows
    blocks, width = max(first.kc.shape[0], then.kc.shape[0]), max(first.bt.shape[1], then.bt.shape[1])
    kc, vc = (torch.zeros(blocks, 16, 4, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    bt = torch.full((4, width), -1, dtype=torch.int32, device=DEV)
    q, cu, lens = first.q.clone(), first.cu.clone(), first.lens.clone()

    def put(b):
        kc[: b.kc.shape[0]], vc[: b.vc.shape[0]] = b.kc, b.vc
        bt.fill_(-1)
        bt[:, : b.bt.shape[1]] = b.bt
        for to, new in ((q, b.q), (cu, b.cu), (lens, b.lens)):
            to.copy_(new)

    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=DEV)
    ws = pkv.new_chunk_workspace(4, 8, 4)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    pkv.set_programmatic_launch(programmatic)
    try:
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=side):
            for _ in range(2):  # two calls one behind the other in one workspace
                pkv.paged_chunk_attn(q, kc, vc, cu, lens, bt, 64, 1024, SCALE, sliding_window=200, num_sinks=4,
                                     out=out, lse=lse, workspace=ws)
    finally:
        pkv.set_programmatic_launch(True)
    for b in (first, then, first):
        put(b)
        graph.replay()
        torch.cuda.synchronize()
        b.check(out, lse, rounded=True)
    assert pkv.check_device_errors() == 0


@pytest.mark.gpu
def test_a_timeout_skips_the_call(L):
    b = Batch([3000, 100], [4, 70], 8, 4, 16, 0, 0, seed=13)
    out, lse = torch.full_like(b.q, 7.0), torch.full((b.rows, 8), 7.0, device=DEV)
    pkv.raise_device_errors(pkv.DEVERR_TIMEOUT)
    _run(b, out=out, lse=lse)
    assert pkv.check_device_errors() & pkv.DEVERR_TIMEOUT
    assert bool((out == 7.0).all()) and bool((lse == 7.0).all())
    b.check(*_run(b, out=out, lse=lse), rounded=True)
    assert pkv.check_device_errors() == 0


@pytest.mark.gpu
def test_binding_refuses(L):
    b = Batch([40, 20], [3, 2], 4, 2, 16, 0, 0, seed=14)
    ok = dict(q=b.q, k_cache=b.kc, v_cache=b.vc, cu_seqlens_q=b.cu, context_lens=b.lens, block_tables=b.bt,
              max_seqlen_q=3, max_context_len=40, scale=SCALE)
    pkv.paged_chunk_attn(**ok)
    for bad in (dict(q=b.q.float()), dict(q=b.q[:, :, :64]), dict(context_lens=b.lens[:1]), dict(block_tables=b.bt[:1]),
                dict(v_cache=b.vc[:1]), dict(out=b.q[:2]), dict(lse=torch.zeros(5, 3, device=DEV)),
                dict(cu_seqlens_q=b.cu.long()), dict(q=b.q.cpu()), dict(out=b.q.transpose(0, 1))):
        with pytest.raises((TypeError, ValueError)):
            pkv.paged_chunk_attn(**{**ok, **bad})
    for bad in (dict(sliding_window=-1), dict(num_sinks=-1), dict(max_seqlen_q=41),
                dict(workspace=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(pkv.PkvError):
            pkv.paged_chunk_attn(**{**ok, **bad})
