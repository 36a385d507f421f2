"""Eviction by accumulated attention weight: decode that accumulates the weights
(bf16 cache), selection, compaction and the block manager's part, against plain
implementations; and the whole chain as an engine runs it."""
import math

import numpy as np
import pytest
import torch

import paged_kv_attention_22_gb300 as pkv
import q4_plain as Q
from paged_kv_attention_22_gb300 import build as pkv_build

SCALE = 1.0 / math.sqrt(128)
gpu = pytest.mark.gpu
FAKE = 0x10000


@pytest.fixture(scope="module")
def L():
    pkv_build.build()
    return pkv.lib()


def select_plain(scores, lens, budget, recent):
    """Kept positions of every sequence, as lists."""
    kept = []
    for row, n in zip(scores.tolist(), lens):
        r = min(recent, n)
        want = min(n, budget) - r
        # NaN behind every number
        rank = sorted(range(n - r), key=lambda p: (row[p] != row[p], -row[p] if row[p] == row[p] else 0.0, p))
        kept.append(sorted(rank[:want]) + list(range(n - r, n)))
    return kept


# ------------------------------------------------------------------ CPU

def test_select_refuses(L):
    def call(ks=FAKE, ld=64, cl=FAKE, mcl=64, S=2, B=16, R=4, keep=FAKE, nl=FAKE):
        return L.pkv_evict_select(ks, ld, cl, mcl, S, B, R, keep, nl, None)
    for null in ("ks", "cl", "keep", "nl"):
        assert call(**{null: None}) == pkv.PKV_ERR_INVALID_ARG
    for bad in (dict(S=-1), dict(B=0), dict(R=-1), dict(R=17), dict(mcl=0), dict(ld=63)):
        assert call(**bad) == pkv.PKV_ERR_INVALID_ARG
    assert call(B=(1 << 29) + 1) == pkv.PKV_ERR_UNSUPPORTED
    assert call(mcl=(1 << 30) + 1, ld=1 << 31) == pkv.PKV_ERR_UNSUPPORTED
    assert call(S=0) == pkv.PKV_OK


def test_select_into_new_arrays_refuses(L):
    def call(ks=FAKE, ld=64, S=2, B=16, R=4, keep=FAKE, nl=FAKE):
        return L.pkv_evict_select_new(ks, ld, FAKE, 64, S, B, R, keep, nl, None)
    for bad in (dict(ks=None), dict(keep=None), dict(nl=None), dict(S=-1), dict(B=0), dict(R=17), dict(ld=63)):
        assert call(**bad) == pkv.PKV_ERR_INVALID_ARG
    assert call(B=(1 << 29) + 1) == pkv.PKV_ERR_UNSUPPORTED
    assert call(S=0) == pkv.PKV_OK


def test_no_sequences(L):
    """An empty tensor has no address."""
    for call in (L.pkv_evict_select, L.pkv_evict_select_new):
        assert call(None, 64, None, 64, 0, 16, 4, None, None, None) == pkv.PKV_OK
        assert call(None, 64, None, 64, 0, 16, 17, None, None, None) == pkv.PKV_ERR_INVALID_ARG
    assert L.pkv_evict_compact(FAKE, FAKE, None, 4, None, 4, None, 16, None, 0, 8, 128, 16, 64, None, 0, None, 0,
                               None) == pkv.PKV_OK
    assert L.pkv_evict_compact(None, FAKE, None, 4, None, 4, None, 16, None, 0, 8, 128, 16, 64, None, 0, None, 0,
                               None) == pkv.PKV_ERR_INVALID_ARG


def test_compact_refuses(L):
    def call(k=FAKE, v=FAKE, src=FAKE, sb=4, dst=FAKE, db=4, keep=FAKE, B=16, nl=FAKE, S=2, H=8, D=128, bs=16, NB=64,
             ks=None, ld=0, dks=None, dld=0):
        return L.pkv_evict_compact(k, v, src, sb, dst, db, keep, B, nl, S, H, D, bs, NB, ks, ld, dks, dld, None)
    for null in ("k", "v", "src", "dst", "keep", "nl"):
        assert call(**{null: None}) == pkv.PKV_ERR_INVALID_ARG
    for bad in (dict(k=FAKE + 8), dict(S=-1), dict(B=0), dict(sb=0), dict(db=0), dict(H=0), dict(bs=0), dict(NB=0),
                dict(ks=FAKE, ld=64), dict(dks=FAKE, dld=64), dict(ks=FAKE, ld=0, dks=FAKE, dld=64),
                dict(ks=FAKE, ld=64, dks=FAKE, dld=32)):
        assert call(**bad) == pkv.PKV_ERR_INVALID_ARG
    assert call(D=64) == pkv.PKV_ERR_UNSUPPORTED
    assert call(S=65536) == pkv.PKV_ERR_UNSUPPORTED
    assert call(B=(1 << 29) + 1) == pkv.PKV_ERR_UNSUPPORTED
    assert call(NB=1 << 40) == pkv.PKV_ERR_UNSUPPORTED
    assert call(S=0) == pkv.PKV_OK

    def q4(gs=32, kc=FAKE, S=2):
        return L.pkv_evict_compact_q4(kc, FAKE, FAKE, FAKE, FAKE, 4, FAKE, 4, FAKE, 16, FAKE, S, 8, 128, gs, 16, 64,
                                      None, 0, None, 0, None)
    assert q4(gs=16) == pkv.PKV_ERR_UNSUPPORTED
    assert q4(kc=None) == pkv.PKV_ERR_INVALID_ARG
    assert q4(S=0) == pkv.PKV_OK


def test_scored_decode_refuses(L):
    def call(**kw):
        a = dict(q=FAKE, kc=FAKE, bt=FAKE, cl=FAKE, out=FAKE, ks=FAKE, ld=64, ws=FAKE, wsb=1 << 30, Hq=16)
        a.update(kw)
        return L.pkv_paged_decode_attn_scores(a["q"], a["kc"], a["kc"], a["bt"], 4, a["cl"], 64, 2, a["Hq"], 8, 128, 16, 64,
                                              0.088, 0, a["out"], None, a["ks"], a["ld"], a["ws"], a["wsb"], None)
    for null in ("q", "kc", "bt", "cl", "out", "ks"):
        assert call(**{null: None}) == pkv.PKV_ERR_INVALID_ARG
    assert call(ld=63) == pkv.PKV_ERR_INVALID_ARG
    assert call(Hq=64) == pkv.PKV_ERR_UNSUPPORTED
    assert call(ws=None) == pkv.PKV_ERR_WORKSPACE_TOO_SMALL
    assert L.pkv_decode_scores_workspace_size(0, 16, 8, 128, 64) == 0
    assert L.pkv_decode_scores_workspace_size(2, 16, 8, 128, 0) == 0
    assert L.pkv_decode_scores_workspace_size(1 << 30, 1 << 14, 1, 128, 1 << 30) == 0


def _manager(num_blocks):
    """Two sequences of 5 blocks of 8 tokens that share the first 2."""
    rng = np.random.default_rng(1)
    bm = pkv.BlockManager(num_blocks, 8)
    base = rng.integers(0, 50000, 40).astype(np.int32)
    other = np.concatenate([base[:16], rng.integers(0, 50000, 20).astype(np.int32)])
    assert bm.add_sequence(0, base) == 0 and bm.add_sequence(1, other) == 16
    return bm, base, other


@pytest.mark.parametrize("spare", [2, 12])
def test_manager_eviction(L, spare):
    """With 3 fresh blocks at hand the kept rows go there; with 2, only the shared
    blocks are replaced and the third is compacted in place."""
    bm, base, other = _manager(8 + spare)
    src, free = bm.block_table(1), bm.num_free_blocks
    assert free == spare
    bm.evict_sequences([1], [19])                           # 3 blocks stay
    dst = bm.block_table(1)
    assert len(dst) == 3 and bm.num_tokens(1) == 19
    fresh = 3 if spare == 12 else 2
    assert not set(dst[:fresh]) & set(src) and not set(dst[:fresh]) & set(bm.block_table(0))
    assert fresh == 3 or dst[2] == src[2]
    assert [bm.ref_count(b) for b in src] == [1, 1, 3 - fresh, 0, 0]
    assert bm.num_free_blocks == spare + 3 - 3              # three released or replaced, three in use
    if spare == 12:
        # sequence 0 is as it was, and still findable; the evicted rows are not
        assert bm.add_sequence(2, base) == 32
        # tokens appended to the evicted sequence fill blocks that nobody finds
        for t in range(21):
            bm.append_token(1, t)
        assert bm.num_tokens(1) == 40 and len(bm.block_table(1)) == 5
        assert np.array_equal(bm.slots(1, 0, 40), np.repeat(bm.block_table(1), 8) * 8 + np.tile(np.arange(8), 5))
        bm.free_sequence(2)
    bm.free_sequence(0)
    bm.free_sequence(1)
    assert bm.num_free_blocks == 8 + spare


def test_manager_eviction_of_several_hands_out_no_block_that_is_still_read(L):
    bm, _, _ = _manager(14)                                 # 6 free: exactly the kept blocks
    old = set(bm.block_table(0)) | set(bm.block_table(1))
    bm.evict_sequences([1, 0], [24, 20])
    new = list(bm.block_table(0)) + list(bm.block_table(1))
    assert len(set(new)) == 6 and not set(new) & old
    assert bm.num_free_blocks == 8 and all(bm.ref_count(b) == 0 for b in old)
    bm, _, _ = _manager(13)                                 # 5 free: in place but the shared blocks
    src = [bm.block_table(s) for s in range(2)]
    bm.evict_sequences([0, 1], [40, 20])
    assert all(b not in set(src[0]) | set(src[1]) for s in range(2) for b in bm.block_table(s)[:2])
    assert list(bm.block_table(0)[2:]) == list(src[0][2:]) and bm.block_table(1)[2] == src[1][2]
    assert bm.ref_count(src[0][0]) == 0                     # shared by nobody any more


def test_manager_eviction_refuses(L):
    bm, _, _ = _manager(9)                                  # 1 free, 2 shared
    state = [list(bm.block_table(s)) for s in range(2)]
    with pytest.raises(pkv.PkvError) as e:
        bm.evict_sequences([0], [20])
    assert e.value.status == pkv.PKV_ERR_OUT_OF_BLOCKS
    for seqs, kept in (([7], [1]), ([0], [0]), ([0], [41]), ([0, 0], [9, 9]), ([0, 7], [1, 1])):
        with pytest.raises(pkv.PkvError) as e:
            bm.evict_sequences(seqs, kept)
        assert e.value.status == pkv.PKV_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        bm.evict_sequences([0, 1], [1])
    bm.evict_sequences([], [])
    assert state == [list(bm.block_table(s)) for s in range(2)] and bm.num_free_blocks == 1


# ------------------------------------------------------------------ GPU: selection

def _scores(kind, S, width, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.rand(S, width, generator=g) ** 4
    if kind == "ties":
        x = (x * 3).round()
    elif kind == "equal":
        x = torch.full_like(x, 0.25)
    elif kind == "signed":
        x = (x - 0.2) * torch.tensor([1e-40, 1.0, 1e38])[torch.randint(0, 3, x.shape, generator=g)]
        x[x.abs() < 1e-42] = -0.0
    elif kind == "special":
        pick = torch.randint(0, 8, x.shape, generator=g)
        for i, v in enumerate((float("nan"), float("inf"), -float("inf"), 0.0, -0.0)):
            x[pick == i] = v
    return x


@gpu
@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "signed", "special"])
@pytest.mark.parametrize("lens,budget,recent", [
    ([1, 0, 5, 40], 16, 4), ([40, 41, 39, 1000], 40, 40), ([33, 64, 65], 32, 0), ([1, 2, 3], 1, 1), ([7, 100], 1, 0),
    ([1023, 1024, 1025, 4097], 1000, 17), ([20000, 5], 4096, 100), ([2049], 2048, 2047), ([60000, 51201, 100], 30000, 64)])
def test_select(L, kind, lens, budget, recent):
    S, width = len(lens), max(lens) + 3
    x = _scores(kind, S, width, sum(lens))
    keep, new = pkv.evict_select(x.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), budget, recent)
    assert pkv.check_device_errors() == 0
    for s, want in enumerate(select_plain(x, lens, budget, recent)):
        assert int(new[s]) == len(want) == min(lens[s], budget)
        assert keep[s].tolist() == want + [-1] * (budget - len(want))


@gpu
def test_select_reports_invalid_lengths(L):
    x = torch.rand(4, 10, device="cuda")
    keep = torch.full((4, 3), 77, dtype=torch.int32, device="cuda")
    new = torch.full((4,), 77, dtype=torch.int32, device="cuda")
    pkv.evict_select(x, torch.tensor([10, -1, 11, 2], dtype=torch.int32, device="cuda"), 3, 1, keep=keep, new_lens=new)
    assert pkv.check_device_errors() == pkv.DEVERR_CONTEXT
    assert new.tolist() == [3, 77, 77, 2] and bool((keep[1:3] == 77).all()) and keep[3].tolist() == [0, 1, -1]


@gpu
def test_invalid_length_moves_nothing_where_the_call_makes_the_arrays(L):
    """The arrays that a call without keep and new_lens makes may be memory of an
    earlier step's: a sequence of invalid length has no row of it in them, and the
    compaction behind the call refuses it."""
    S, block, heads, budget = 3, 16, 1, 20
    bf = torch.randn(2, S * 3, block, heads, 128, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16)
    k, v = bf.cuda()
    bt = torch.arange(S * 3, dtype=torch.int32, device="cuda").view(S, 3)
    scores = torch.rand(S, 48, device="cuda")
    for lens in ([48, 48, 48], [48, 49, -1]):
        before = [x.clone() for x in (k, v, scores)]
        keep, new = pkv.evict_select(scores, torch.tensor(lens, dtype=torch.int32, device="cuda"), budget, 4)
        pkv.evict_compact(k, v, bt, bt, keep, new, scores, scores)
        flags = pkv.check_device_errors()
        bad = [s for s in range(S) if not 0 <= lens[s] <= 48]
        assert flags == (pkv.DEVERR_CONTEXT if bad else 0)
        assert new.tolist() == [-1 if s in bad else budget for s in range(S)]
        for s in bad:
            assert bool((keep[s] == -1).all())
            for x, y in zip(before[:2], (k, v)):
                assert torch.equal(x[bt[s].long()], y[bt[s].long()])
            assert torch.equal(before[2][s], scores[s])
        del keep, new               # the next call's arrays are these again


@gpu
@pytest.mark.parametrize("given", ["keep", "new_lens"])
def test_invalid_length_where_one_array_is_given(L, given):
    """The call makes the other one: the sequence gets -1 in both."""
    lens = torch.tensor([10, -1, 11, 2], dtype=torch.int32, device="cuda")
    keep = torch.full((4, 3), 7, dtype=torch.int32, device="cuda") if given == "keep" else None
    new = torch.full((4,), 7, dtype=torch.int32, device="cuda") if given == "new_lens" else None
    keep, new = pkv.evict_select(torch.rand(4, 10, device="cuda"), lens, 3, 1, keep=keep, new_lens=new)
    assert pkv.check_device_errors() == pkv.DEVERR_CONTEXT
    assert new.tolist() == [3, -1, -1, 2] and bool((keep[1:3] == -1).all()) and keep[3].tolist() == [0, 1, -1]


def _select_sorted(row, n, budget, recent):
    """select_plain of one long sequence: a stable sort, NaN behind every number."""
    r = min(recent, n)
    order = torch.sort(-row[:n - r].double(), stable=True).indices
    return torch.cat([order[:min(n, budget) - r].sort().values, torch.arange(n - r, n)])


def test_sorted_selection_is_the_plain_one():
    for kind in ("plain", "ties", "equal", "signed", "special"):
        x = _scores(kind, 1, 700, 3)
        for n, budget, recent in ((700, 300, 20), (699, 1, 0), (700, 699, 5), (3, 9, 1)):
            assert _select_sorted(x[0], n, budget, recent).tolist() == select_plain(x, [n], budget, recent)[0]


@gpu
@pytest.mark.parametrize("kind", ["plain", "ties", "equal", "signed", "special"])
@pytest.mark.parametrize("lens,budget,recent", [
    ([65537, 65536, 70000, 1], 30000, 64), ([131073], 131072, 0), ([409600, 409599], 200000, 1000),   # keys in shared memory
    ([409601, 5, 300000], 1000, 100), ([450000], 449999, 64)])                                         # read again each pass
def test_select_of_very_long_sequences(L, kind, lens, budget, recent):
    S, width = len(lens), max(lens)
    x = _scores(kind, S, width, sum(lens))
    keep, new = pkv.evict_select(x.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), budget, recent)
    assert pkv.check_device_errors() == 0
    for s, n in enumerate(lens):
        want = _select_sorted(x[s], n, budget, recent)
        assert int(new[s]) == len(want) == min(n, budget)
        got = keep[s].cpu()
        assert torch.equal(got[:len(want)].long(), want) and bool((got[len(want):] == -1).all())


# ------------------------------------------------------------------ GPU: compaction

def _fresh_tables(lens, block, first):
    width = max(1, -(-max(lens) // block))
    t = torch.full((len(lens), width), -1, dtype=torch.int32)
    for s, n in enumerate(lens):
        for j in range(-(-n // block)):
            t[s, j], first = first, first + 1
    return t


def _compact_plain(arrays, src, dst, kept, block, planes_first):
    """Moved copies of the arrays [NB, block, ...] or, planes_first, [NB, planes, block, ...]."""
    moved = [a.clone() for a in arrays]
    for s, rows in enumerate(kept):
        for i, p in enumerate(rows):
            a, b = int(src[s, p // block]), int(dst[s, i // block])
            for old, new in zip(arrays, moved):
                if planes_first:
                    new[b, :, i % block] = old[a, :, p % block]
                else:
                    new[b, i % block] = old[a, p % block]
    return moved


COMPACT = [  # lens, budget, recent, heads, block
    ([40, 17, 100, 3], 16, 4, 2, 16),
    ([5, 1], 1, 1, 1, 16),
    ([1000, 700], 333, 50, 3, 7),
    ([2600], 2500, 100, 1, 256),
    ([300] * 3, 299, 0, 8, 64),
]


@gpu
@pytest.mark.parametrize("lens,budget,recent,heads,block", COMPACT)
@pytest.mark.parametrize("group", [0, 32, 64, 128])
@pytest.mark.parametrize("in_place", [True, False])
def test_compact(L, lens, budget, recent, heads, block, group, in_place):
    g = torch.Generator().manual_seed(sum(lens))
    kept_lens = [min(n, budget) for n in lens]
    used = sum(-(-n // block) for n in lens)
    NB = used + sum(-(-n // block) for n in kept_lens) + 1
    order = torch.randperm(NB, generator=g).to(torch.int32)
    src = _fresh_tables(lens, block, 0)
    dst = src if in_place else _fresh_tables(kept_lens, block, used)
    src, dst = (torch.where(t >= 0, order[t.clamp(min=0).long()], t) for t in (src, dst))
    if group == 0:
        arrays = [torch.randint(-2 ** 15, 2 ** 15, (NB, block, heads, 128), generator=g, dtype=torch.int32).to(torch.int16)
                  for _ in range(2)]
    else:
        arrays = [torch.randint(0, 256, (NB, heads, block, n), generator=g, dtype=torch.int32).to(torch.uint8)
                  for n in (64, 64, 512 // group, 512 // group)]
    scores = torch.rand(len(lens), max(lens) + 2, generator=g)
    kept = select_plain(scores, lens, budget, recent)
    want = _compact_plain(arrays, src, dst, kept, block, group > 0)
    cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    sc = scores.cuda()
    keep, new = pkv.evict_select(sc, cl, budget, recent)
    new_scores = sc if in_place else torch.full((len(lens), budget + 9), 5.0, device="cuda")
    dev = [a.cuda() for a in arrays]
    rest = (src.cuda(), dst.cuda(), keep, new)
    if group == 0:
        pkv.evict_compact(*(a.view(torch.bfloat16) for a in dev), *rest, key_scores=sc, dst_key_scores=new_scores)
    else:
        params = [a.view(torch.bfloat16).view(NB, heads, block, 128 // group, 2) for a in dev[2:]]
        pkv.evict_compact_q4((dev[0], params[0]), (dev[1], params[1]), *rest, key_scores=sc, dst_key_scores=new_scores)
    assert pkv.check_device_errors() == 0
    for got, w in zip(dev, want):
        assert torch.equal(got.cpu(), w)
    for s, rows in enumerate(kept):
        assert torch.equal(new_scores[s, :len(rows)].cpu(), scores[s][rows])
        assert bool((new_scores[s, len(rows):] == 0).all())


@gpu
def test_calls_of_no_sequences(L):
    kc, vc = (pkv.new_q4_cache(4, 16, 2) for _ in range(2))
    empty = torch.empty(0, 3, dtype=torch.int32, device="cuda")
    scores = torch.empty(0, 48, device="cuda")
    keep, new = pkv.evict_select(scores, torch.empty(0, dtype=torch.int32, device="cuda"), 9, 2)
    assert keep.shape == (0, 9) and new.shape == (0,)
    pkv.evict_compact_q4(kc, vc, empty, empty, keep, new, scores, scores)
    k16 = torch.zeros(4, 16, 2, 128, dtype=torch.bfloat16, device="cuda")
    pkv.evict_compact(k16, k16.clone(), empty, empty, keep, new)
    assert pkv.check_device_errors() == 0


@gpu
def test_compact_into_fresh_blocks_reports_bad_values(L):
    NB, block, heads = 8, 16, 2
    g = torch.Generator().manual_seed(4)
    codes = torch.randint(0, 256, (NB, heads, block, 64), generator=g, dtype=torch.int32).to(torch.uint8)
    params = torch.randn(NB, heads, block, 1, 2, generator=g).to(torch.bfloat16)
    src = torch.tensor([[0, 1], [2, -1], [3, 3]], dtype=torch.int32)
    dst = torch.tensor([[4], [5], [NB]], dtype=torch.int32)
    keep = torch.tensor([[3, 20, 31], [1, 17, 40], [0, 1, 2]], dtype=torch.int32)
    new = torch.tensor([3, 3, 1], dtype=torch.int32)
    kc, vc = [(codes.cuda(), params.cuda()) for _ in range(2)]
    pkv.evict_compact_q4(kc, vc, src.cuda(), dst.cuda(), keep.cuda(), new.cuda())
    assert pkv.check_device_errors() == pkv.DEVERR_CONTEXT | pkv.DEVERR_BLOCK
    for old, got in ((codes, kc[0]), (codes, vc[0]), (params, kc[1]), (params, vc[1])):
        want = old.clone()
        want[4, :, 0], want[4, :, 1], want[4, :, 2] = old[0, :, 3], old[1, :, 4], old[1, :, 15]
        want[5, :, 0] = old[2, :, 1]
        assert torch.equal(got.cpu().view(torch.uint8), want.view(torch.uint8))


@gpu
def test_compact_reports_bad_values_and_moves_the_rest(L):
    NB, block, heads = 8, 16, 1
    g = torch.Generator().manual_seed(3)
    k = torch.randint(-2 ** 15, 2 ** 15, (NB, block, heads, 128), generator=g, dtype=torch.int32).to(torch.int16)
    tables = torch.tensor([[0, 1], [2, 3], [4, 5], [6, NB]], dtype=torch.int32)
    keep = torch.tensor([[3, 20], [1, 32], [2, 5], [1, 17]], dtype=torch.int32)
    new = torch.tensor([2, 2, 3, 2], dtype=torch.int32)          # sequence 2: past the budget
    kc, vc = k.view(torch.bfloat16).cuda(), k.view(torch.bfloat16).cuda()
    pkv.evict_compact(kc, vc, tables.cuda(), tables.cuda(), keep.cuda(), new.cuda())
    assert pkv.check_device_errors() == pkv.DEVERR_CONTEXT | pkv.DEVERR_BLOCK
    want = k.clone()
    want[0, 0], want[0, 1] = k[0, 3], k[1, 4]
    want[2, 0] = k[2, 1]
    want[6, 0] = k[6, 1]
    assert torch.equal(kc.view(torch.int16).cpu(), want) and torch.equal(vc.view(torch.int16).cpu(), want)


# ------------------------------------------------------------------ GPU: accumulated weights over a bf16 cache

def _bf16_case(seed, lens, heads, block):
    """A bf16 cache whose unused rows hold NaN: (k, v, tables, k rows, v rows) with rows [P, H, 128] per sequence."""
    g = torch.Generator().manual_seed(seed)
    tables = _fresh_tables(lens, block, 0)
    NB = int(tables.max()) + 2
    order = torch.randperm(NB, generator=g).to(torch.int32)
    tables = torch.where(tables >= 0, order[tables.clamp(min=0).long()], tables)
    caches, rows = [], []
    for _ in range(2):
        c = torch.full((NB, block, heads, 128), float("nan"), dtype=torch.bfloat16)
        mine = []
        for s, n in enumerate(lens):
            x = torch.randn(n, heads, 128, generator=g).to(torch.bfloat16)
            p = torch.arange(n)
            c[tables[s].long()[p // block], p % block] = x
            mine.append(x)
        caches.append(c)
        rows.append(mine)
    return caches[0], caches[1], tables, rows[0], rows[1]


@gpu
@pytest.mark.parametrize("lens,heads,gqa,block,window", [
    ([1], 1, 1, 16, 0), ([17, 64, 100, 128], 8, 2, 16, 0), ([640] * 3, 8, 2, 256, 0), ([5, 900, 33], 2, 4, 48, 0),
    ([4000], 4, 2, 64, 0), ([300, 7, 1000], 8, 1, 32, 100), ([2000, 3], 2, 2, 16, 1)])
def test_scored_decode(L, lens, heads, gqa, block, window):
    pkv.decode_set_config(0, 0)
    k, v, tables, kr, vr = _bf16_case(sum(lens), lens, heads, block)
    g = torch.Generator().manual_seed(5)
    q = torch.randn(len(lens), heads * gqa, 128, generator=g).to(torch.bfloat16)
    width = max(lens) + 4
    scores = torch.full((len(lens), width), 0.25, device="cuda")
    args = (q.cuda(), k.cuda(), v.cuda(), tables.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), max(lens), SCALE)
    o, l = pkv.paged_decode_attn_scores(*args, scores, sliding_window=window)
    o0, l0 = pkv.paged_decode_attn(*args, sliding_window=window)
    pkv.paged_decode_attn_scores(*args, scores, sliding_window=window, with_lse=False)
    assert pkv.check_device_errors() == 0
    assert torch.equal(o, o0) and torch.equal(l, l0)        # the attention itself is the plain call's
    got = scores.cpu().double()
    for s, n in enumerate(lens):
        first = max(0, n - window) if window else 0
        want, tol = torch.zeros(n, dtype=torch.float64), torch.zeros(n, dtype=torch.float64)
        for h in range(heads * gqa):
            ks = kr[s][:, h // gqa].double()
            _, lse, w, _, qk = Q.attend(q[s, h:h + 1].double(), ks, vr[s][:, h // gqa].double(), SCALE, [first], [n - 1])
            want += w[0]
            # exp(z - lse): both within the lse's tolerance
            tol += w[0] * 2 * Q.lse_tolerance(lse, qk, n) + 2.0 ** -20 * w[0]
        # two calls add the weight twice; each addition rounds once
        err = (got[s, :n] - 0.25 - 2 * want).abs()
        assert bool((err <= 2 * tol + 2 * Q.U32 * (0.25 + 2 * want)).all()), float(err.max())
        assert bool((got[s, n:] == 0.25).all()) and bool((got[s, :first] == 0.25).all())


@gpu
@pytest.mark.parametrize("ctx,block,heads,gqa,window,variant", [
    (40, 16, 1, 2, 0, 0), (20000, 64, 2, 1, 0, 0), (3000, 32, 8, 2, 0, 2), (1000, 16, 4, 4, 0, 0), (700, 16, 8, 2, 300, 0)])
def test_scored_decode_leaves_keys_of_bad_table_entries_out(L, ctx, block, heads, gqa, window, variant):
    """Sequence 0 has one bad entry, sequence 1 nothing but bad ones, sequence 2 none:
    the weights of sequence 0 are those over its other keys, sequence 1's stay, and
    sequence 2 has the plain call's bits, whatever the workspace held."""
    k, v, tables, kr, vr = _bf16_case(ctx, [ctx] * 3, heads, block)
    q = torch.randn(3, heads * gqa, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    first = max(0, ctx - window) if window else 0
    bad = first // block + 1
    tables[0, bad] = int(tables.max()) + 9
    tables[1] = -1
    args = (q.cuda(), k.cuda(), v.cuda(), tables.cuda(), torch.full((3,), ctx, dtype=torch.int32, device="cuda"), ctx, SCALE)
    scores = torch.full((3, ctx), 0.5, device="cuda")
    pkv.decode_set_config(0, variant)
    try:
        ws = pkv.new_decode_scores_workspace(3, heads * gqa, heads, ctx).fill_(255)      # NaNs
        out, lse = pkv.paged_decode_attn_scores(*args, scores, workspace=ws, sliding_window=window)
        assert pkv.check_device_errors() == pkv.DEVERR_BLOCK
        o0, l0 = pkv.paged_decode_attn(*args, sliding_window=window)
        assert pkv.check_device_errors() == pkv.DEVERR_BLOCK
    finally:
        pkv.decode_set_config(0, 0)
    assert torch.equal(out[2], o0[2]) and torch.equal(lse[2], l0[2])
    got = scores.cpu().double()
    rest = torch.cat([torch.arange(first, bad * block), torch.arange((bad + 1) * block, ctx)])
    want, tol = torch.zeros(len(rest), dtype=torch.float64), torch.zeros(len(rest), dtype=torch.float64)
    for h in range(heads * gqa):
        ks, vs = kr[0][rest, h // gqa].double(), vr[0][rest, h // gqa].double()
        o, l, w, wv, qk = Q.attend(q[0, h:h + 1].double(), ks, vs, SCALE, [0], [len(rest) - 1])
        assert bool(((out[0, h].cpu().double() - o[0]).abs() <= Q.out_tolerance(o[0], wv[0])).all())
        tol_l = Q.lse_tolerance(l, qk, ctx)
        assert abs(float(lse[0, h]) - float(l)) <= float(tol_l)
        want += w[0]
        tol += w[0] * (2 * tol_l + 2.0 ** -20)          # exp(z - lse): both within the lse's tolerance
    # the heads' additions and the last one round
    tol += (heads * gqa + 2) * Q.U32 * (0.5 + want)
    assert bool(((got[0, rest] - 0.5 - want).abs() <= tol).all())
    others = torch.ones(ctx, dtype=torch.bool)
    others[rest] = False
    assert bool((got[0, others] == 0.5).all()) and bool((got[1] == 0.5).all())
    assert bool(torch.isfinite(got[2]).all())


@gpu
def test_scored_decode_adds_nothing_after_a_timeout(L):
    k, v, tables, _, _ = _bf16_case(1, [50, 20], 2, 16)
    args = (torch.randn(2, 4, 128).to(torch.bfloat16).cuda(), k.cuda(), v.cuda(), tables.cuda(),
            torch.tensor([50, 20], dtype=torch.int32, device="cuda"), 50, SCALE)
    scores = torch.zeros(2, 50, device="cuda")
    pkv.raise_device_errors(pkv.DEVERR_TIMEOUT)
    pkv.paged_decode_attn_scores(*args, scores)
    assert pkv.check_device_errors() == pkv.DEVERR_TIMEOUT
    assert bool((scores == 0).all())
    pkv.paged_decode_attn_scores(*args, scores)
    assert pkv.check_device_errors() == 0
    assert bool((scores[0] > 0).all())


@gpu
@pytest.mark.parametrize("q4", [False, True])
def test_scored_decode_of_very_many_heads(L, q4):
    """More query heads than a scoring CTA holds: the same as two calls of half the
    heads. The sums run over the heads in order, in fp32: n terms are off by at most
    n U32 of their sum, the logits and the lse are the same numbers in both."""
    heads, block, ctx = 8192, 16, 4200 if q4 else 100
    g = torch.Generator().manual_seed(4)
    bt = (torch.arange(-(-ctx // block)) % 2).to(torch.int32)[None].cuda()   # two blocks, again and again
    q = torch.randn(1, heads, 128, generator=g).to(torch.bfloat16).cuda()
    cl = torch.tensor([ctx], dtype=torch.int32, device="cuda")
    if q4:
        rows = torch.randn(2, 2, heads, block, 128, generator=g).to(torch.bfloat16)
        caches = [tuple(x.cuda() for x in Q.quantise(rows[i], 32)) for i in range(2)]
        call, cut = pkv.paged_decode_attn_q4, lambda c, a, b: tuple(x[:, a:b].contiguous() for x in c)
    else:
        caches = list(torch.randn(2, 2, block, heads, 128, generator=g).to(torch.bfloat16).cuda())
        call, cut = pkv.paged_decode_attn_scores, lambda c, a, b: c[:, :, a:b].contiguous()
    whole, halves = (torch.zeros(1, ctx, device="cuda") for _ in range(2))
    out, lse = call(q, *caches, bt, cl, ctx, SCALE, key_scores=whole)
    for a in (0, heads // 2):
        b = a + heads // 2
        o, l = call(q[:, a:b].contiguous(), *(cut(c, a, b) for c in caches), bt, cl, ctx, SCALE, key_scores=halves)
        # another plan may cut the keys elsewhere. out, below 4: 3 U16 of it, twice. lse:
        # its tolerance with sums |q k| scale below 16, twice: 2^-11
        assert bool(((o - out[:, a:b]).abs() <= 6 * Q.U16 * 4).all()) and bool(((l - lse[:, a:b]).abs() <= 2.0 ** -11).all())
    assert pkv.check_device_errors() == 0
    tol = (2 * heads * Q.U32 + 2.0 ** -10) * halves.double()                 # the lse's difference, too
    assert bool(((whole.double() - halves.double()).abs() <= tol).all())
    total = float(whole.double().sum())
    assert abs(total - heads) <= (heads * Q.U32 + 2.0 ** -11) * heads


# ------------------------------------------------------------------ GPU: the chain

@gpu
@pytest.mark.parametrize("q4", [False, True])
@pytest.mark.parametrize("pool", [13, 40])
def test_engine_steps_with_eviction(L, q4, pool):
    """Two sequences that share a prefix, driven by the block manager: prefill,
    decode steps that accumulate weights, eviction of the longer one (into fresh
    blocks, or with a small pool into fresh and own ones), and decode on. The attention after it equals plain attention over
    exactly the kept rows, and the other sequence sees nothing of it."""
    heads, gqa, block, group, budget, recent = 2, 2, 16, 32, 50, 12
    g = torch.Generator().manual_seed(8)
    bm = pkv.BlockManager(pool, block)
    prompts = [np.arange(100, dtype=np.int32), np.concatenate([np.arange(48), 900 + np.arange(30)]).astype(np.int32)]
    if q4:
        kc, vc = (pkv.new_q4_cache(pool, block, heads, group) for _ in range(2))
    else:
        kc, vc = (torch.full((pool, block, heads, 128), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    rows = [[], []]                      # each sequence's (k, v) rows in logical order, as the cache holds them

    def kept_value(x):
        return Q.values(*Q.quantise(x, group)) if q4 else x.double()

    def store(k, v, slots):
        put = pkv.kv_store_q4 if q4 else pkv.kv_store
        put(k.cuda(), v.cuda(), kc, vc, torch.from_numpy(slots).cuda())

    shared = torch.randn(2, 48, heads, 128, generator=g).to(torch.bfloat16)
    for s, prompt in enumerate(prompts):
        cached = bm.add_sequence(s, prompt)
        assert cached == (0, 48)[s]
        n = len(prompt) - (48 if s else 0)
        new = torch.randn(2, n, heads, 128, generator=g).to(torch.bfloat16)
        if s == 0:
            new[:, :48] = shared
            rows[s] = [new[0], new[1]]
        else:
            rows[s] = [torch.cat([shared[i], new[i]]) for i in range(2)]
        store(new[0], new[1], bm.slots(s, cached, n))

    def decode(scores):
        for s in range(2):
            bm.append_token(s, 7)
            x = torch.randn(2, 1, heads, 128, generator=g).to(torch.bfloat16)
            rows[s] = [torch.cat([rows[s][i], x[i]]) for i in range(2)]
            store(x[0], x[1], bm.slots(s, bm.num_tokens(s) - 1, 1))
        lens = [bm.num_tokens(s) for s in range(2)]
        tables = torch.from_numpy(bm.block_tables([0, 1], 8)).cuda()
        q = torch.randn(2, heads * gqa, 128, generator=g).to(torch.bfloat16)
        cl = torch.tensor(lens, dtype=torch.int32, device="cuda")
        if q4:
            o, _ = pkv.paged_decode_attn_q4(q.cuda(), kc, vc, tables, cl, 128, SCALE, key_scores=scores)
        else:
            o, _ = pkv.paged_decode_attn_scores(q.cuda(), kc, vc, tables, cl, 128, SCALE, scores)
        for s in range(2):
            assert lens[s] == rows[s][0].shape[0]
            for h in range(heads * gqa):
                k, v = (kept_value(rows[s][i][:, h // gqa]) for i in range(2))
                want, _, _, wv, _ = Q.attend(q[s, h:h + 1].double(), k, v, SCALE, [0], [lens[s] - 1])
                err = (o[s, h].cpu().double() - want[0]).abs()
                assert bool((err <= Q.out_tolerance(want[0], wv[0])).all()), (s, h, float(err.max()))
        return lens

    scores = torch.zeros(2, 128, device="cuda")
    for _ in range(3):
        lens = decode(scores)
    # evict sequence 0, in a call of its own
    src = torch.from_numpy(bm.block_table(0, 8)[None]).cuda()
    row = scores[:1].clone()
    before = row.cpu()
    keep, new = pkv.evict_select(row, torch.tensor(lens[:1], dtype=torch.int32, device="cuda"), budget, recent)
    bm.evict_sequences([0], [budget])
    dst = torch.from_numpy(bm.block_table(0, 8)[None]).cuda()
    assert bool((dst[0, :3] != src[0, :3]).all()) and (int(dst[0, 3]) == int(src[0, 3])) == (pool == 13)
    (pkv.evict_compact_q4 if q4 else pkv.evict_compact)(kc, vc, src, dst, keep, new, key_scores=row, dst_key_scores=row)
    scores[0] = row[0]
    assert new.tolist() == [budget]
    kept = keep[0].long().cpu()
    assert kept.tolist() == select_plain(before, lens[:1], budget, recent)[0]
    rows[0] = [x[kept] for x in rows[0]]
    for _ in range(15):                 # past the end of a block
        decode(scores)
    assert pkv.check_device_errors() == 0


@gpu
@pytest.mark.parametrize("pdl", [True, False])
def test_captured_step_with_eviction(L, pdl):
    """Store, decode with weights, selection, compaction into fresh blocks, decode over
    the kept rows and prefill, captured in one graph and replayed on new inputs: the
    bits of the eager calls; with programmatic launches and without."""
    heads, gqa, block, S, ctx, budget = 4, 2, 32, 3, 500, 128
    g = torch.Generator(device="cuda").manual_seed(17)
    per, kept_blocks = 16, budget // block
    NB = S * (per + kept_blocks)
    ids = torch.randperm(NB, generator=g, device="cuda").to(torch.int32)
    src, dst = ids[:S * per].view(S, per).contiguous(), ids[S * per:].view(S, kept_blocks).contiguous()
    lens = torch.tensor([ctx, ctx - 77, 129], dtype=torch.int32, device="cuda")
    p = torch.arange(ctx, device="cuda")
    slots = (src.long()[:, p // block] * block + p % block).to(torch.int32).flatten()
    slots[(p >= lens[:, None]).flatten()] = -1
    cu = torch.tensor([0, 8, 16, 24], dtype=torch.int32, device="cuda")
    cu_k = torch.tensor([0, budget, 2 * budget, 3 * budget], dtype=torch.int32, device="cuda")
    cache = [pkv.new_q4_cache(NB, block, heads) for _ in range(2)]
    k, v = (torch.zeros(S * ctx, heads, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(S, heads * gqa, 128, dtype=torch.bfloat16, device="cuda")
    qp = torch.zeros(24, heads * gqa, 128, dtype=torch.bfloat16, device="cuda")
    scores, new_scores = torch.zeros(S, ctx, device="cuda"), torch.zeros(S, budget, device="cuda")
    ws = pkv.new_q4_decode_workspace(S, heads * gqa, heads, ctx, with_scores=True)

    def step():
        scores.zero_()
        pkv.kv_store_q4(k, v, *cache, slots)
        a = pkv.paged_decode_attn_q4(q, *cache, src, lens, ctx, SCALE, workspace=ws, key_scores=scores)
        keep, new = pkv.evict_select(scores, lens, budget, 20)
        pkv.evict_compact_q4(*cache, src, dst, keep, new, key_scores=scores, dst_key_scores=new_scores)
        b = pkv.paged_decode_attn_q4(q, *cache, dst, new, budget, SCALE, workspace=ws)
        c = pkv.paged_prefill_attn_q4(qp, *cache, cu, cu_k, dst, 8, budget, 3 * budget, SCALE)
        return [*a, keep, new, new_scores, *b, *c, scores]

    def fill(seed):
        g.manual_seed(seed)
        for x in (k, v, q, qp):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda").to(torch.bfloat16))

    pkv.set_programmatic_launch(pdl)
    try:
        fill(1)
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            captured = step()
        for seed in (2, 3):
            fill(seed)
            want = [x.clone() for x in step()]
            graph.replay()
            torch.cuda.synchronize()
            for i, (x, y) in enumerate(zip(captured, want)):
                assert torch.equal(x, y), (seed, i)
            assert want[3].tolist() == [budget, budget, budget] and bool(torch.isfinite(want[7].float()).all())
        assert pkv.check_device_errors() == 0
    finally:
        pkv.set_programmatic_launch(True)
