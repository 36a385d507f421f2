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
