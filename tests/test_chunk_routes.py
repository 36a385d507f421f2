"""Chunks without a window that are long enough to run on the prefill kernel, whose running maximum
takes the scale for positive and normal: other scales stay on the chunk kernel, whatever the
lengths. Against the plain 64-bit form, over caches that hold NaN wherever no query looks."""
import pytest
import torch

import paged_kv_attention_22_gb300 as pkv
from attn_plain import Batch
from paged_kv_attention_22_gb300 import build as pkv_build


@pytest.fixture(scope="module")
def L():
    pkv_build.build()
    return pkv.lib()


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [-0.1, 0.0, -0.0, 6e-39, -6e-39, 2e-38, 0.3], ids=str)
def test_scales_of_long_chunks(L, scale):
    # 11 and 10 row tiles of 16 heads in each segment: more than half of the SMs have one. 6e-39 is
    # subnormal and stays so times log2 e, 2e-38 is normal: a weight for every key alike, and lse ln n.
    b = Batch([1500, 1281], [1290, 1270], 16, 8, 64, 0, 0, seed=31, scale=scale)
    out, lse = pkv.paged_chunk_attn(b.q, b.kc, b.vc, b.cu, b.lens, b.bt, 1290, 1500, scale)
    b.check(out, lse, rounded=True)
    assert pkv.check_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 3), (2 ** 31 - 1, 2 ** 31 - 1)])
@pytest.mark.parametrize("max_q,max_k", [(1290, 1 << 30), (1 << 30, 1 << 30)])
def test_bounds_far_above_the_segments(L, window, sinks, max_q, max_k):
    # as a graph that was captured for long chunks replays them: q has rows for three of some 1,000 tokens, which
    # without a window chooses the prefill kernel, and the segments have 3 and 130
    b = Batch([1500, 400, 0], [3, 130, 0], 16, 8, 48, min(window, 2000), min(sinks, 2000), seed=32, extra_rows=3000)
    out, lse = torch.full_like(b.q, 7.0), torch.full(b.q.shape[:2], 7.0, device="cuda")
    pkv.paged_chunk_attn(b.q, b.kc, b.vc, b.cu, b.lens, b.bt, max_q, max_k, b.scale, sliding_window=window,
                         num_sinks=sinks, out=out, lse=lse)
    b.check(out, lse, rounded=True)
    assert bool((out[b.rows:] == 7).all()) and bool((lse[b.rows:] == 7).all())
    assert pkv.check_device_errors() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,H", [(256, 64), (20, 5), (7, 7)])
@pytest.mark.parametrize("bs", [80, 1024])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 33)])
def test_many_and_odd_heads_and_blocks(L, Hq, H, bs, window, sinks):
    b = Batch([333, 1, 129], [5, 1, 129], Hq, H, bs, window, sinks, seed=33)
    out, lse = pkv.paged_chunk_attn(b.q, b.kc, b.vc, b.cu, b.lens, b.bt, 129, 333, b.scale, sliding_window=window,
                                    num_sinks=sinks)
    b.check(out, lse, rounded=True)
    assert pkv.check_device_errors() == 0
