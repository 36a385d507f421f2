"""Orders that the chunk kernel (csrc/chunk.cu) owes to copies and MMAs that overwrite what its
warps read. A missing order shows in results only when a warp is late, so it is read from the
source here, on the CPU; on the GPU the calls that pass these places give the same bits again
and again."""
import os
import re

import pytest
import torch

import paged_kv_attention_22_gb300 as pkv
from attn_plain import Batch
from paged_kv_attention_22_gb300 import build as pkv_build

# what lies in the place of the V tiles until the first copies, and what reads it
LIST = r"\b(steps|tiles|seqs|starts|ranks)\[|\b(find|scan|locate)\("
IN_BUILD = LIST + r"|\b(sums|totals)\["


@pytest.fixture(scope="module")
def L():
    pkv_build.build()
    return pkv.lib()


def _source():
    with open(os.path.join(pkv_build.CSRC, "chunk.cu")) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _block(text, head):
    """(start, end) of `head` and the braces behind it."""
    start = text.index(head)
    at = text.index("{", start)
    depth = 0
    for end in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        if depth == 0:
            return start, end + 1
    raise AssertionError(head)


def _without(text, head):
    start, end = _block(text, head)
    return text[:start] + text[end:]


@pytest.mark.parametrize("loop", [True, False], ids=["whole tiles tried", "no whole tiles"])
def test_the_lists_last_reads_are_behind_a_barrier(loop):
    # On every way out of build() the whole CTA has met behind the last read of the list: the
    # producer's copies of V overwrite it and wait for no other warp.
    text = _source()
    body = text[slice(*_block(text, "Shares build("))]
    body = _without(body, "auto locate = [&]")
    if not loop:
        body = _without(body, "for (r.waves = ")
    ways = [m.start() for m in re.finditer(r"\breturn\b", body)]
    assert len(ways) == 4
    for way in ways[1:]:  # the first is that of a call that does nothing
        last = [m.end() for m in re.finditer(r"__syncthreads(?:_or)?\(", body[:way])][-1]
        assert re.search(IN_BUILD, body[last:way]) is None, body[last:way]


def test_behind_the_list_only_the_producer_reads_it():
    text = _source()
    kernel = text[slice(*_block(text, "chunk_kernel(const __grid_constant__"))]
    build = kernel.index("build<kWindowed>(")
    start, end = _block(kernel, "if (warp == 0 && works)")
    between, behind = kernel[build:start], kernel[end:]
    assert re.search(LIST, behind) is None
    assert not any(name in behind for name in ("kStepsOff", "kTilesOff", "kSeqOff", "kShareOff", "kRankOff"))
    reads = [m.start() for m in re.finditer(LIST, between)]
    assert reads and "tid == 0 && cta >=" in between[:reads[0]]  # of the producer's warp


def test_what_was_read_from_tmem_is_ordered_before_the_next_product():
    # A softmax warp's arrival on kBarP lets the MMA warp issue the P.V that overwrites O, and the S
    # that overwrites the logits: between the warp's last access to TMEM (finish() reads O) and the
    # arrival stands tcgen05.fence::before_thread_sync.
    text = _source()
    kernel = text[slice(*_block(text, "chunk_kernel(const __grid_constant__"))]
    softmax = kernel[slice(*_block(kernel, "else if (warp >= kSoftmaxWarp0 && works)"))]
    arrivals = [m.start() for m in re.finditer(r"mbar_arrive\(bar\(kBarP ", softmax)]
    assert len(arrivals) == 2
    for at in arrivals:
        last = [m.end() for m in re.finditer(r"\b(tmem_\w+|finish|logits)\(", softmax[:at])][-1]
        assert "tc_fence_before();" in softmax[last:at], softmax[last:at]


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,H", [(1, 1), (4, 2)])
def test_few_tokens_behind_a_full_tile(L, Hq, H):
    # a CTA's softmax warps that have no row of the next tile still write the last one's output
    segments = [(200, 128 * H // Hq), (40, 2), (300, 1)] * 150
    keys, new = map(list, zip(*segments))
    b = Batch(keys, new, Hq, H, 16, 0, 0, seed=23)
    out, lse = pkv.paged_chunk_attn(b.q, b.kc, b.vc, b.cu, b.lens, b.bt, max(new), max(keys), b.scale)
    b.check(out, lse, rounded=True)
    assert pkv.check_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("segments,Hq,H,window,sinks", [
    ([(640, 5)] * 64, 16, 8, 0, 0),                         # one tile a sequence: no list of tiles
    ([(1, 1)], 2, 1, 0, 0),                                 # one CTA with one step
    ([(1000, 1), (7, 7), (0, 0), (300, 30)] * 5, 8, 2, 100, 5),
    ([(700, 300)] * 6, 4, 2, 0, 0),                         # several tiles, none of them whole to a CTA
    ([(1200, 512)] * 16, 16, 8, 256, 4),                    # whole tiles in front
    ([(260, 130)] * 300, 8, 4, 0, 0),
])
def test_the_same_bits_whatever_was_there_before(L, segments, Hq, H, window, sinks):
    keys, new = map(list, zip(*segments))
    b = Batch(keys, new, Hq, H, 32, window, sinks, seed=21)
    other = Batch([90, 2000], [90, 3], Hq, H, 32, 0, 0, seed=22)  # leaves other lists and keys on the SMs
    call = lambda b: pkv.paged_chunk_attn(b.q, b.kc, b.vc, b.cu, b.lens, b.bt, max(b.new), max(b.keys), b.scale,
                                          sliding_window=b.window, num_sinks=b.sinks)
    first = call(b)
    b.check(*first, rounded=True)
    for i in range(60):
        if i % 3 == 0:
            call(other)
        again = call(b)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    assert pkv.check_device_errors() == 0
