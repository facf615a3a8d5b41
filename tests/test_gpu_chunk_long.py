"""Chunk attention over long caches, paged and not, with two-part operands at every head_dim and biases by far distances, against
the oracle.  Bars: test_gpu_chunk.py's.  Its 1e-4 of the largest output for fp16 and fp32 holds for sums of any length here: a
running sum of n weights in fp32 is off by at most n / 2 half steps of its total, 20,000 * 2^-25 = 6e-4 if all steps erred one way,
while the tiles' partial sums (64 terms) and the pieces' (a few hundred tiles) each begin anew: (64 + 313) * 2^-24 = 2.2e-5."""

import numpy as np
import pytest

from kvq_testlib import require_gpu
from test_gpu_chunk import _cache, _check, _starts

pytestmark = pytest.mark.gpu

LENS, NEW = [20000, 5000, 70], [3, 21, 70]


@pytest.mark.parametrize("od", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("d,kt,vt,T,page", [(64, "q5_1", "q4_0", 300, 64), (128, "q4_0", "q5_0", 0, 256), (192, "q8_0", "q4_1", 77, 128),
                                            (256, "q4_1", "q8_0", 100, 64), (320, "q5_0", "q5_1", 0, 64), (320, "q8_0", "q8_0", 512, 0)])
def test_long_caches(d, kt, vt, T, page, od):
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(d + T)
    gc, oc = _cache(torch, kvq, rng, 3, 1, d, 20224, T, kt, vt, LENS, page)
    start = _starts(NEW)
    q = 0.7 * rng.standard_normal((start[-1], 2, d)).astype(np.float32)
    for mod in ({}, dict(slopes=np.array([2.0 ** -12, 0.01], np.float32)),
                dict(softcap=8.0, slopes=np.array([3e-4, 0.0], np.float32), prefix_len=[18000, 100, 70])):
        _check(torch, kvq, gc, oc, q, start, od, mod)
