"""Chunk attention where tokens differ in size, against the oracle: every row is as exact as its own keys and values are, not as
the largest beside them.

Bars.  bf16 outputs: operands rounded to fp16 once, so that each is off by at most 2^-11 of itself; the oracle derives from
that how far an element may be off.  fp16 and fp32 outputs: operands of 22 bits, and sums of up to 320 terms in fp32 of which
each step loses at most 2^-23, 2^-14.7 in all: operands off by 2^-14 cover both.  The type's half step comes to either.  What
a format loses below its normal numbers comes besides (`_least`): fp16's steps end at 2^-24, and half a step is at most
2^-12 of the largest of a block's 32 values in bf16's quick conversion, 2^-34 of the tile's largest elsewhere (a power of two brings
that above 2^9)."""

import numpy as np
import pytest

from kvq_testlib import require_gpu
from oracle import kvq_oracle as ko
from oracle import share_oracle as sh
from test_gpu_chunk import STEP, _cache, _run

pytestmark = pytest.mark.gpu

FORMATS = ["q4_0", "q5_0", "q8_0", "q4_1", "q5_1"]


def _least(oc, od, head_top=None):
    """Functions of how far a stored key's and value's channels may be off for fp16's smallest step."""
    def of(w):
        def at(b, h):
            x = oc.stored(w, b, h)
            top = np.abs(x).max() if head_top is None else head_top
            off = np.full(x.shape, 2.0 ** -34 * top)
            body = max(0, len(x) - oc.T)
            if od == "bf16":
                off[:body] += 2.0 ** -12 * np.repeat(np.abs(x[:body]).reshape(body, -1, 32).max(-1), 32, -1)
            return off
        return at
    return of("k"), of("v")


def _compare(torch, kvq, gc, oc, q, od, what=None, **mod):
    """Every element within its bar; `what`: the rows looked at."""
    rows = np.arange(len(q)) if what is None else what
    got, qr = _run(torch, kvq, gc, q, [0, len(q)], od, mod, qd="f32")
    assert kvq.kvq_sync_status(gc.desc) == (0, 0)
    ref, off = sh.chunk(lambda b, h: oc.stored("k", b, h), lambda b, h: oc.stored("v", b, h), oc.rot["k"], oc.rot["v"], qr,
                        [0, len(q)], oc.seq_len, oc.H, ko.default_scale(oc.d), rounding=2.0 ** (-11 if od == "bf16" else -14),
                        least=_least(oc, od), **mod)
    got, ref, off = got[rows], ref[rows], off[rows]
    assert np.isfinite(off).all()
    bar = off + STEP[od] * (np.abs(ref) + off) + (2.0 ** -25 if od == "f16" else 0.0)
    bad = np.abs(got - ref) / bar
    assert (bad <= 1).all(), (bad.max(), np.argwhere(bad > 1)[:3].tolist(), (bad > 1).mean())


def _sized(torch, kvq, rng, d, T, fmt, n, keys, values, page=0):
    """A sequence of n tokens with keys and values of the given sizes."""
    factor = np.stack([keys, values]).reshape(2, 1, n, 1, 1)
    return _cache(torch, kvq, rng, 1, 1, d, -(-n // 64) * 64, T, fmt, fmt, [n], page=page, factor=factor)


@pytest.mark.parametrize("od", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("d,T", [(64, 0), (128, 70), (256, 0), (320, 40)])
def test_documents_of_different_size(d, T, fmt, od):
    """Documents of 16 tokens, 1, 2^-6, 2^-10 and 2^-14 of the largest, four to a tile: a row sees its own document alone.  Queries are
    as much larger as their keys are smaller, so that scores are alike."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(d + T)
    n = 200
    size = 2.0 ** np.array([0, -6, -10, -14])[np.arange(n) // 16 % 4]
    gc, oc = _sized(torch, kvq, rng, d, T, fmt, n, 16 * size, 32 * size, page=64)
    q = (0.7 / 16 * rng.standard_normal((n, 2, d)) / size[:, None, None]).astype(np.float32)
    _compare(torch, kvq, gc, oc, q, od, first_key=np.arange(n) // 16 * 16)


@pytest.mark.parametrize("od", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("fmt", FORMATS)
def test_large_tokens_far_behind(fmt, od):
    """Values of different size in view, the large ones with weights that a steep bias makes small."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(7)
    n = 300
    size = 2.0 ** np.array([0, -6, -10, -14])[np.arange(n) // 37 % 4]
    gc, oc = _sized(torch, kvq, rng, 64, 0, fmt, n, np.ones(n), 32 * size)
    q = 0.7 * rng.standard_normal((n, 2, 64)).astype(np.float32)
    _compare(torch, kvq, gc, oc, q, od, slopes=np.array([2.0, 0.7], np.float32))


@pytest.mark.parametrize("od", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T", [0, 200])
@pytest.mark.parametrize("at", [3, 150, 470])
def test_one_large_token(at, T, od):
    """One token 2^10 or 2^13 times as large as the others, early, in the middle and late: rows before it, rows that mask it and rows
    that see it."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    for fmt, up in (("q4_0", 2.0 ** 10), ("q5_1", 2.0 ** 10), ("q8_0", 2.0 ** 10), ("q5_0", 2.0 ** 13)):
        rng = np.random.default_rng(at)
        n = 500
        big = np.full(n, 0.125)
        big[at] *= up
        gc, oc = _sized(torch, kvq, rng, 128, T, fmt, n, 0.25 * np.ones(n), big)
        q = 2.0 * rng.standard_normal((n, 1, 128)).astype(np.float32)
        _compare(torch, kvq, gc, oc, q, od, first_key=np.where((np.arange(n) > at) & (np.arange(n) % 2 == 1), at + 1, 0))


@pytest.mark.parametrize("od", ["bf16", "f32"])
@pytest.mark.parametrize("d,n", [(64, 640), (128, 640), (256, 640), (64, 3008)])
def test_segments_that_fall_and_rise(d, n, od):
    """Values of 2^12 and 2^-10 by turns of 64 tokens, each a document: the scale of an item's values goes down and up."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(d)
    size = 2.0 ** np.array([-10, 12])[np.arange(n) // 64 % 2]
    gc, oc = _sized(torch, kvq, rng, d, 0, "q8_0", n, np.ones(n), size)
    q = 0.7 * rng.standard_normal((n, 2, d)).astype(np.float32)
    first = np.arange(n) // 64 * 64
    _compare(torch, kvq, gc, oc, q, od, first_key=first)
    _compare(torch, kvq, gc, oc, q[-70:], od)  # every kind in view
    if n < 1000:
        _compare(torch, kvq, gc, oc, q, od, first_key=first, prefix_len=[n])


@pytest.mark.parametrize("od", ["bf16", "f32"])
@pytest.mark.parametrize("fmt", FORMATS)
def test_the_largest_header(fmt, od):
    """A token with headers of 65504 in the middle of ordinary ones (a block's scale of them 2^-21 of it): rows that do not see it are
    as exact as ever."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(5)
    n, at, d = 300, 140, 64
    gc, oc = _sized(torch, kvq, rng, d, 0, fmt, n, 16 * np.ones(n), 16 * np.ones(n))
    halves = 2 if fmt.endswith("_1") else 1
    for w in "kv":
        gc.planes[w + "_d"].view(torch.float16).view(-1, d // 32, halves)[at] = 65504.0
    q = (0.7 / 16 * rng.standard_normal((n, 2, d))).astype(np.float32)
    rows = np.arange(n)
    first = np.where(rows > at, at + 1, 0)
    got, qr = _run(torch, kvq, gc, q, [0, n], od, dict(first_key=first), qd="f32")
    top = {"q4_0": 8, "q5_0": 16, "q8_0": 128, "q4_1": 16, "q5_1": 32}[fmt] * 65504.0
    ref, off = sh.chunk(lambda b, h: oc.stored("k", b, h), lambda b, h: oc.stored("v", b, h), True, True, qr, [0, n], oc.seq_len, 1,
                        ko.default_scale(d), first_key=first, rounding=2.0 ** (-11 if od == "bf16" else -14), least=_least(oc, od, top))
    keep = rows != at
    bar = off + STEP[od] * (np.abs(ref) + off)
    bad = (np.abs(got - ref) / bar)[keep]
    assert (bad <= 1).all(), (bad.max(), (bad > 1).mean())
