"""Capped scores of chunk attention from tight caps to such as change nothing, against the oracle.

Bars: test_gpu_chunk.py's.  Its 1e-4 for fp16 and fp32 outputs has 5e-5 for the products of a score, at most 64 in size here (asserted),
doubled.  The cap adds at most 2^-20.8 of the capped score (a fit off by 2^-21.8 and its roundings, or a reciprocal and an
exponential): 3.5e-5 of 64, so that both stay below it.  For bf16 outputs the oracle's bound of the operands' rounding is 2^-10
of a score's terms, beside which 2^-20.8 of their sum is lost: a 2^-10th part of the bound is added for it."""

import numpy as np
import pytest

from kvq_testlib import require_gpu
from oracle import kvq_oracle as ko
from test_gpu_chunk import _cache, _close, _ref, _run

pytestmark = pytest.mark.gpu

CAPS = [1e-42, 1e-38, 1e-3, 0.1, 1.0, 5.0, 50.0, 300.0, 1e3, 1e4, 1e6, 1e8, 1e20, 1e30]


@pytest.mark.parametrize("od", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("d,T,page", [(64, 0, 0), (128, 33, 64), (256, 0, 64), (320, 20, 0)])
def test_caps(d, T, page, od):
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(d)
    gc, oc = _cache(torch, kvq, rng, 2, 1, d, 512, T, "q8_0", "q5_0", [300, 77], page)
    q = 0.7 * rng.standard_normal((80, 3, d)).astype(np.float32)
    for cap in CAPS:
        got, qr = _run(torch, kvq, gc, q, [0, 70, 80], od, dict(softcap=cap))
        assert kvq.kvq_sync_status(gc.desc) == (0, 0)
        size = max((np.abs(ko.rotate(qr.astype(np.float64))).reshape(-1, d) @ np.abs(oc.stored("k", b, 0)).T).max() for b in (0, 1))
        assert size * ko.default_scale(d) < 64
        ref, off = _ref(oc, qr, [0, 70, 80], softcap=cap)
        _close(got, (ref, off * (1 + 2.0 ** -10)), od)


@pytest.mark.parametrize("od", ["bf16", "f16", "f32"])
def test_a_cap_that_changes_nothing(od):
    """Large scores under a cap far above them: those of no cap, to the cap's own rounding."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(3)
    gc, oc = _cache(torch, kvq, rng, 1, 1, 64, 512, 0, "q8_0", "q8_0", [400])
    q = 0.7 * rng.standard_normal((50, 2, 64)).astype(np.float32)
    plain, _ = _run(torch, kvq, gc, q, [0, 50], od, {})
    for cap in (1e7, 1e30):
        got, qr = _run(torch, kvq, gc, q, [0, 50], od, dict(softcap=cap))
        _close(got, _ref(oc, qr, [0, 50]), od)
        assert np.abs(got - plain).max() <= 2.0 ** -7 * np.abs(plain).max()


@pytest.mark.parametrize("od", ["bf16", "f16", "f32"])
def test_scores_that_are_not_finite(od):
    """A query with NaN or an infinity makes NaN of its own row, capped or not; the others keep their bits."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(4)
    gc, oc = _cache(torch, kvq, rng, 1, 1, 64, 256, 0, "q8_0", "q4_0", [200])
    q = rng.standard_normal((30, 2, 64)).astype(np.float32)
    for cap in (1e-3, 20.0, 1e8):
        clean, _ = _run(torch, kvq, gc, q, [0, 30], od, dict(softcap=cap))
        for bad in (np.nan, np.inf):
            p = q.copy()
            p[7, 1, 3] = bad
            got, _ = _run(torch, kvq, gc, p, [0, 30], od, dict(softcap=cap))
            assert np.isnan(got[7, 1]).all()
            got[7, 1] = clean[7, 1]
            assert np.array_equal(got, clean)
