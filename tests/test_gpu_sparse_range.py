"""Sparse decode over the whole range of stored values, against the float64 oracle, on the GPU:
the relative L2 error alone, as an absolute bar says nothing about small values.

Bound.  The scores below are sums of products whose magnitudes add up to at most 2^4 in base 2
(order-1 scores of normal data); the query in two 11-bit parts and the sums on the tensor cores
hold them to 2^-20 of that, so the weights to 2^-16 of themselves, the exponential's 2^-22 beside it;
the weights' parts, their products with the scales and the sums of the output add 2^-20 of the
largest terms.  Outputs of a few dozen tokens' average: together below 2^-15 of the output's norm."""

import numpy as np
import pytest

from kvq_testlib import append_both, require_gpu, to_dev
from oracle import kvq_oracle as ko
from oracle import step_oracle as so

pytestmark = pytest.mark.gpu

TYPES = ["q4_0", "q5_0", "q8_0", "q4_1", "q5_1"]
BOUND = 2.0 ** -15


def _caches(kvq, d, ctx, T, kt, vt, k, v, torch, flags=None):
    flags = kvq.KVQ_ROT_AUTO if flags is None else flags
    gc = kvq.KVCache(1, k.shape[2], d, ctx, T, kt, vt, flags=flags)
    oc = ko.OracleCache(1, k.shape[2], d, ctx, T, kt, vt, not flags & kvq.KVQ_ROT_K_OFF, not flags & kvq.KVQ_ROT_V_OFF)
    append_both(gc, oc, k, v, torch=torch)
    return gc, oc


def _sparse(kvq, torch, gc, q, sel, bt=64):
    out = torch.full(q.shape, 9.0, device="cuda")
    kvq.kvq_sparse_decode_attention(gc.desc, to_dev(q, "f32", torch), torch.tensor(sel, dtype=torch.int32, device="cuda"), out, bt)
    assert kvq.kvq_sync_status(gc.desc)[0] == 0
    return out.cpu().numpy().astype(np.float64)


def _rel(got, ref):
    assert np.all(np.isfinite(got))
    return np.linalg.norm(got - ref) / np.linalg.norm(ref)


@pytest.mark.parametrize("d", [64, 128, 192, 256, 320])
@pytest.mark.parametrize("ks,vs", [(1.0, 1e-2), (1.0, 1e-3), (1.0, 1e-4), (1.0, 1e-5), (1e-2, 1.0), (1e-4, 1.0), (1e-5, 1e-5),
                                   (1.0, 1e-30), (1e-12, 1.0), (1e6, 1e7), (1e10, 1e20)])
def test_tail_values_of_every_size(d, ks, vs):
    """A sequence no longer than the tail: keys and values are the stored bf16 numbers, whatever their size."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(41)
    k, v = rng.standard_normal((2, 1, 61, 2, d))
    gc, oc = _caches(kvq, d, 128, 64, "q8_0", "q4_0", (ks * k).astype(np.float32), (vs * v).astype(np.float32), torch)
    q = (rng.standard_normal((1, 6, d)) / ks).astype(np.float32)
    got = _sparse(kvq, torch, gc, q, [[[0], [0]]])
    assert _rel(got, so.sparse_decode(oc, q, np.array([[[0], [0]]]), 64)) <= BOUND


@pytest.mark.parametrize("T", [0, 40])
@pytest.mark.parametrize("vt,d,lo,hi", [("q5_1", 128, -64000, 64000), ("q4_1", 128, -64000, 64000), ("q4_1", 64, 5e4, 9e4),
                                        ("q5_1", 320, 5e4, 9e4), ("q5_1", 192, -65000, -60000), ("q4_1", 256, -1e3, 2e5)])
def test_large_minima_and_scales(vt, d, lo, hi, T):
    """A block's minimum plus a multiple of its scale passes fp16's largest number; its values are finite all the same."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(42)
    n = 500
    k = rng.standard_normal((1, n, 2, d)).astype(np.float32)
    v = rng.uniform(lo, hi, (1, n, 2, d)).astype(np.float32)
    gc, oc = _caches(kvq, d, 512, T, "q8_0", vt, k, v, torch, flags=kvq.KVQ_ROT_AUTO | kvq.KVQ_ROT_V_OFF)
    q = rng.standard_normal((1, 6, d)).astype(np.float32)
    sel = [[[0, 7, 3, 4, 1], [6, 5, -1, 2, 7]]]
    got = _sparse(kvq, torch, gc, q, sel)
    assert _rel(got, so.sparse_decode(oc, q, np.array(sel), 64)) <= BOUND


@pytest.mark.parametrize("page", [0, 64])
@pytest.mark.parametrize("vt", TYPES)
def test_bits_do_not_depend_on_rows_past_the_end(vt, page):
    """Rows at or past a sequence's end, and body rows that the tail replaces, hold anything: the result is the same bits."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(43)
    H, d, ctx, T, n = 2, 128, 256, 20, 149
    table = torch.tensor([2, 0, 3, 1], dtype=torch.int32)
    paged = dict(page_tokens=page, n_pages=4, page_table=table) if page else {}
    gc = kvq.KVCache(1, H, d, ctx, T, vt, vt, **paged)
    k, v = (to_dev(rng.standard_normal((1, n, H, d)), "f32", torch) for _ in range(2))
    kvq.kvq_rotate_quantize_append(gc.desc, k, v)
    q = rng.standard_normal((1, 2 * H, d)).astype(np.float32)
    sel = [[[0, 1, 2], [2, 1, 0]]]
    want = _sparse(kvq, torch, gc, q, sel)
    dead = [gc.desc.max_ctx * h + p if not page else (table[p // page].item() * H + h) * page + p % page
            for h in range(H) for p in range(n - T, ctx)]
    dead = torch.tensor(dead, device="cuda")
    for word in (0x7FFF, 0x7BFF, -1):  # NaN, fp16's largest number, NaN with the sign
        for name in ("k_qs", "v_qs", "k_d", "v_d"):
            gc.plane(name).view(torch.int16).view(H * ctx, -1)[dead] = word
        assert np.array_equal(_sparse(kvq, torch, gc, q, sel), want), (vt, word)


@pytest.mark.parametrize("vt,d,T,scales", [(t, d, T, s) for t, d in zip(TYPES, (64, 128, 192, 256, 320)) for T in (0, 30)
                                           for s in ((1e-3,) * 8, (1e-4,) * 8, (1e-5,) * 8, (1e-4, 1e-3, 1e-2, 0.1, 1, 10, 1e2, 1e3),
                                                     (1e5,) * 8, (1e4, 1, 1e-2, 1e-4, 1e-5, 1e-5, 1e-5, 1e-5))])
def test_body_values_of_every_size(vt, d, T, scales):
    """Values from fp16's smallest scales to its largest, the same in all blocks, growing and falling along them."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(44)
    k, v = rng.standard_normal((2, 1, 512, 2, d)).astype(np.float32)
    v *= np.repeat(np.float32(scales), 64)[None, :, None, None]
    gc, oc = _caches(kvq, d, 512, T, "q8_0", vt, k, v, torch)
    q = rng.standard_normal((1, 6, d)).astype(np.float32)
    sel = [[[0, 1, 2, 3, 4, 5, 6, 7], [7, 5, 3, -1, 2, 0, -1, 1]]]
    got, ref = _sparse(kvq, torch, gc, q, sel), so.sparse_decode(oc, q, np.array(sel), 64)
    if scales[0] == 1e5 and vt in ("q4_1", "q5_1"):
        # a block's minimum is stored in fp16, down to -65504: of 32 normal values of spread 1e5 one lies below in
        # all but 0.744^32 of the blocks, so the cache holds -inf and every output is a sum with it
        assert not np.isfinite(ref).any() and not np.isfinite(got).any()
        return
    assert _rel(got, ref) <= BOUND
