"""Block index, block selection and sparse decode against the oracle, on the GPU.

The index's codes and scales and the selected blocks are compared exactly: their definition
fixes the order of every sum.  The attention is held to the decode's bars (max-abs 2e-3, rel-L2
1e-3 in fp32), plus half an eps of the output's type."""

import numpy as np
import pytest

from kvq_testlib import ATOL, RTOL, append_both, require_gpu, to_dev
from oracle import kvq_oracle as ko
from oracle import step_oracle as so

pytestmark = pytest.mark.gpu

TYPES = ["q4_0", "q5_0", "q8_0", "q4_1", "q5_1"]


def _pair(torch, kvq, rng, B, H, d, ctx, T, kt, vt, lens, page=0, flags=None):
    kw = {}
    if page:
        n = B * (ctx // page) + 3
        kw = dict(page_tokens=page, n_pages=n, page_table=torch.tensor(rng.permutation(n)[:B * (ctx // page)].astype(np.int32)))
    flags = kvq.KVQ_ROT_AUTO if flags is None else flags
    gc = kvq.KVCache(B, H, d, ctx, T, kt, vt, flags=flags, **kw)
    oc = ko.OracleCache(B, H, d, ctx, T, kt, vt, not flags & kvq.KVQ_ROT_K_OFF, not flags & kvq.KVQ_ROT_V_OFF)
    k, v = rng.standard_normal((2, B, max(max(lens), 1), H, d)).astype(np.float32)
    k[..., 5] *= 20
    v[..., 9] *= 20
    append_both(gc, oc, k, v, n_new_per_seq=lens, torch=torch)
    return gc, oc


def _sparse(torch, kvq, gc, q, qd, sel, bt, od="f32", scale=0.0):
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
    qt = to_dev(q, qd, torch)
    out = torch.full(q.shape, 9.0, dtype=dt[od], device="cuda")
    kvq.kvq_sparse_decode_attention(gc.desc, qt, torch.tensor(sel, dtype=torch.int32, device="cuda"), out, bt, scale=scale)
    torch.cuda.synchronize()
    return out.float().cpu().numpy().astype(np.float64), qt.float().cpu().numpy()


def _close(got, ref, eps=0.0):
    assert np.all(np.isfinite(got))
    err = np.abs(got - ref)
    assert np.all(err <= ATOL + eps * np.abs(ref)), err.max()
    assert np.linalg.norm(err) <= (RTOL + eps) * max(np.linalg.norm(ref), 1e-30)


@pytest.mark.parametrize("kt,d,bt,page", [("q4_0", 64, 64, 0), ("q5_0", 128, 64, 64), ("q8_0", 256, 128, 0), ("q4_1", 192, 192, 64),
                                          ("q5_1", 320, 64, 0), ("q8_0", 64, 64, 128), ("q4_0", 128, 1024, 0)])
def test_index_codes(kt, d, bt, page):
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(21)
    lens = [0, 1, 64, 200, 512]
    gc, oc = _pair(torch, kvq, rng, 5, 2, d, 512, 24, kt, "q4_0", lens, page)
    x = kvq.BlockIndex(gc.desc, bt)
    x.codes.fill_(3)
    x.scales.fill_(3)
    kvq.kvq_block_index_update(gc.desc, x)
    codes, scales = so.block_index(oc, bt)
    got = x.codes.cpu().numpy(), x.scales.cpu().numpy()
    for b, n in enumerate(lens):
        have = -(-n // bt)
        assert np.array_equal(got[0][b, :, :have], codes[b, :, :have]) and np.array_equal(got[1][b, :, :have], scales[b, :, :have])
        assert (got[0][b, :, have:] == 3).all() and (got[1][b, :, have:] == 3).all()
    # the last tokens' blocks alone
    for last in (1, 65, 130, 1 << 30):
        x.codes.fill_(3)
        kvq.kvq_block_index_update(gc.desc, x, n_last=last)
        got = x.codes.cpu().numpy()
        for b, n in enumerate(lens):
            first, have = max(0, n - last) // bt, -(-n // bt)
            assert np.array_equal(got[b, :, first:have], codes[b, :, first:have])
            assert (got[b, :, :first] == 3).all() and (got[b, :, have:] == 3).all()
    assert kvq.kvq_sync_status(gc.desc)[0] == 0


def test_index_of_many_blocks():
    """More blocks than CTAs run at once: a CTA takes several, one of them in a page outside the pool."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(29)
    lens = [0, 1, 64, 200, 4096, 4095, 65, 1000, 2049, 4000]
    gc, oc = _pair(torch, kvq, rng, 10, 8, 64, 4096, 24, "q5_1", "q4_0", lens, 64)
    x = kvq.BlockIndex(gc.desc, 64)
    x.codes.fill_(3)
    x.scales.fill_(3)
    kvq.kvq_block_index_update(gc.desc, x)
    assert kvq.kvq_sync_status(gc.desc)[0] == 0
    codes, scales = so.block_index(oc, 64)

    def check():
        got = x.codes.cpu().numpy(), x.scales.cpu().numpy()
        for b, n in enumerate(lens):
            have = -(-n // 64)
            assert np.array_equal(got[0][b, :, :have], codes[b, :, :have]) and np.array_equal(got[1][b, :, :have], scales[b, :, :have])
            assert (got[0][b, :, have:] == 3).all() and (got[1][b, :, have:] == 3).all()
    check()
    gc.page_table.view(10, 64)[4, 20] = 1 << 20
    x.codes.fill_(3)
    x.scales.fill_(3)
    kvq.kvq_block_index_update(gc.desc, x)
    assert kvq.kvq_sync_status(gc.desc) == (kvq.KVQ_ERR_DEVICE_RANGE, kvq.KVQ_DEV_ERR_PAGE)
    codes[4, :, 20] = 0
    scales[4, :, 20] = 0
    check()


def test_index_of_zero_keys_and_of_a_bad_page():
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    table = torch.tensor([0, 99, 1, 2], dtype=torch.int32)
    gc = kvq.KVCache(1, 1, 64, 256, 0, "q8_0", "q8_0", page_tokens=64, n_pages=4, page_table=table)
    gc.seq_len.fill_(200)
    gc.plane("k_qs").fill_(128)  # offset binary: zeros
    x = kvq.BlockIndex(gc.desc, 64)
    x.codes.fill_(3)
    kvq.kvq_block_index_update(gc.desc, x)
    assert kvq.kvq_sync_status(gc.desc) == (kvq.KVQ_ERR_DEVICE_RANGE, kvq.KVQ_DEV_ERR_PAGE)
    assert not x.codes.any() and not x.scales.any()


@pytest.mark.parametrize("d,g,nblk,nsel,first,last,dt,rot", [
    (64, 1, 1, 1, 0, 0, "f32", True), (64, 1, 9, 1, 1, 0, "f32", True), (64, 3, 40, 7, 1, 1, "bf16", True),
    (128, 4, 128, 32, 1, 1, "bf16", True), (128, 8, 100, 99, 2, 3, "f16", True), (192, 9, 77, 20, 0, 5, "f32", True),
    (256, 6, 1000, 64, 1, 1, "bf16", True), (320, 12, 33, 16, 1, 1, "bf16", True), (128, 16, 3000, 500, 4, 4, "f32", False),
    (64, 128, 50, 10, 1, 1, "bf16", True), (128, 1, 49152, 700, 1, 1, "bf16", True), (64, 2, 20000, 19999, 1, 1, "f32", True),
    (128, 5, 400, 30, 1, 1, "bf16", True), (64, 8, 2100, 1049, 600, 449, "f32", True), (320, 7, 4097, 33, 0, 0, "f16", True)])
def test_selection(d, g, nblk, nsel, first, last, dt, rot):
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(22)
    B, H, bt = (1, 1, 64) if nblk > 5000 else (3, 2, 64)
    lens = [nblk * bt] if B == 1 else [nblk * bt, max(1, nblk * bt // 2 - 5), 0]
    gc = kvq.KVCache(B, H, d, nblk * bt, 0, "q4_0", "q4_0", flags=kvq.KVQ_ROT_AUTO | (0 if rot else kvq.KVQ_ROT_K_OFF))
    gc.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
    x = kvq.BlockIndex(gc.desc, bt)
    codes = np.clip(np.rint(40 * rng.standard_normal((B, H, nblk, d))), -127, 127).astype(np.int8)
    scales = (0.01 * (1 + rng.random((B, H, nblk)))).astype(np.float32)
    x.codes.copy_(torch.from_numpy(codes))
    x.scales.copy_(torch.from_numpy(scales))
    q = to_dev(rng.standard_normal((B, H * g, d)), dt, torch)
    sel = torch.full((B, H, nsel), 77, dtype=torch.int32, device="cuda")
    kvq.kvq_select_blocks(gc.desc, x, q, sel, n_first=first, n_last=last)
    want = so.select_blocks(q.float().cpu().numpy(), codes, scales, lens, bt, first, last, nsel, rot)
    assert np.array_equal(sel.cpu().numpy(), want)


@pytest.mark.parametrize("kind", ["equal", "zero query", "zero scales", "two values", "inf scale", "nan query"])
def test_selection_of_equal_and_special_scores(kind):
    """Equal scores take the lowest blocks; scores that are not numbers rank last; nothing out of range is written."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    d, nblk, nsel = 64, 300, 21
    gc = kvq.KVCache(1, 1, d, nblk * 64, 0, "q4_0", "q4_0")
    gc.seq_len.fill_(nblk * 64)
    x = kvq.BlockIndex(gc.desc, 64)
    codes, scales = np.ones((1, 1, nblk, d), np.int8), np.ones((1, 1, nblk), np.float32)
    q = np.ones((1, 2, d), np.float32)
    if kind == "zero query":
        q[:] = 0
    elif kind == "zero scales":
        scales[:] = 0
        codes[:] = np.random.default_rng(3).integers(-9, 9, codes.shape)
    elif kind == "two values":
        codes[0, 0, ::7] = 2
    elif kind == "inf scale":
        scales[0, 0, 100:110] = np.inf
    elif kind == "nan query":
        q[0, 0, 3] = np.nan
        q[0, 1] = np.nan
    x.codes.copy_(torch.from_numpy(codes))
    x.scales.copy_(torch.from_numpy(scales))
    sel = torch.full((1, 1, nsel + 2), 77, dtype=torch.int32, device="cuda")[:, :, :nsel].contiguous()
    kvq.kvq_select_blocks(gc.desc, x, torch.from_numpy(q).cuda(), sel)
    got = sel[0, 0].tolist()
    assert got[0] == 0 and got[-1] == nblk - 1 and got == sorted(set(got)) and len(got) == nsel
    if kind != "nan query":
        with np.errstate(invalid="ignore"):
            assert got == so.select_blocks(q, codes, scales, [nblk * 64], 64, 1, 1, nsel, True)[0, 0].tolist()


@pytest.mark.parametrize("kt,vt", [(a, b) for a in TYPES for b in TYPES])
def test_sparse_decode_formats(kt, vt):
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(23)
    gc, oc = _pair(torch, kvq, rng, 3, 2, 128, 640, 40, kt, vt, [600, 77, 640], page=64)
    q = rng.standard_normal((3, 8, 128)).astype(np.float32)
    sel = np.array([[[9, 0, 4, 5], [1, -1, 9, 2]], [[1, 0, -1, 5], [0, -1, -1, -1]], [[9, 8, 7, 6], [2, 2, 0, 99]]])
    got, qn = _sparse(torch, kvq, gc, q, "f32", sel, 64)
    ref = so.sparse_decode(oc, qn, sel, 64)
    _close(got, ref)
    # fp32's precision: a weight times a V scale is held to 2^-25, the weights within 2^6 of the largest
    # (2^5 .. 2^7) times scales from 2^-6 on to 2^-18 of themselves and less; scores and weights add 2^-21
    assert np.linalg.norm(got - ref) <= 2.0 ** -18 * np.linalg.norm(ref)
    assert kvq.kvq_sync_status(gc.desc)[0] == 0


@pytest.mark.parametrize("vt,T", [(t, T) for t in TYPES for T in (0, 40)])
def test_sparse_decode_of_large_values(vt, T):
    """V scales past what the weights leave room for in fp16, in some blocks of some tokens only."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(33)
    gc, oc = (kvq.KVCache(1, 1, 128, 512, T, "q8_0", vt, flags=kvq.KVQ_ROT_AUTO | kvq.KVQ_ROT_V_OFF),
              ko.OracleCache(1, 1, 128, 512, T, "q8_0", vt, True, False))
    k, v = rng.standard_normal((2, 1, 500, 1, 128)).astype(np.float32)
    v[:, 200:210, :, 40:50] *= 1e4
    v[:, 490, :, 3] *= 3e4
    append_both(gc, oc, k, v, torch=torch)
    q = rng.standard_normal((1, 5, 128)).astype(np.float32)
    sel = np.array([[[0, 1, 2, 3, 4, 6, 7]]])
    got, qn = _sparse(torch, kvq, gc, q, "f32", sel, 64)
    ref = so.sparse_decode(oc, qn, sel, 64)
    assert np.all(np.isfinite(got))
    assert np.linalg.norm(got - ref) <= RTOL * np.linalg.norm(ref)
    # the channels without large values on their own
    calm = [c for c in range(128) if not 32 <= c < 64 and c >= 32]
    assert np.abs(got[..., calm] - ref[..., calm]).max() <= ATOL


@pytest.mark.parametrize("d,g,T,bt,qd,od,page", [
    (64, 1, 0, 64, "f32", "f32", 0), (64, 5, 512, 64, "bf16", "bf16", 0), (64, 8, 30, 128, "f16", "f32", 64),
    (128, 4, 100, 64, "bf16", "f16", 0), (128, 9, 17, 192, "f32", "f32", 64), (128, 20, 0, 64, "bf16", "bf16", 0),
    (192, 3, 64, 64, "f32", "f32", 0), (256, 6, 130, 64, "bf16", "bf16", 256), (256, 7, 7, 128, "f32", "bf16", 0),
    (320, 2, 33, 64, "f32", "f32", 64), (320, 12, 512, 64, "bf16", "f32", 0)])
def test_sparse_decode_shapes(d, g, T, bt, qd, od, page):
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(24)
    B, H, ctx = 4, 2, 768
    lens = [0, 1, 413, 768]
    gc, oc = _pair(torch, kvq, rng, B, H, d, ctx, T, "q8_0", "q5_1", lens, page)
    nblk = -(-ctx // bt)
    for nsel in (1, 3, nblk):
        sel = np.stack([[rng.permutation(nblk)[:nsel] for _ in range(H)] for _ in range(B)])
        q = rng.standard_normal((B, H * g, d)).astype(np.float32)
        got, qn = _sparse(torch, kvq, gc, q, qd, sel, bt, od)
        _close(got, so.sparse_decode(oc, qn, sel, bt), 0.0 if od == "f32" else torch.finfo(getattr(torch, {"bf16": "bfloat16", "f16": "float16"}[od])).eps / 2)
        assert not got[0].any()
    assert kvq.kvq_sync_status(gc.desc)[0] == 0


@pytest.mark.parametrize("off", [2, 4, 6])
def test_sparse_decode_rotation_switches_and_scale(off):
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(25)
    gc, oc = _pair(torch, kvq, rng, 1, 1, 64, 256, 20, "q8_0", "q8_0", [250], flags=1 | off)
    q = rng.standard_normal((1, 4, 64)).astype(np.float32)
    sel = np.array([[[3, 1]]])
    got, qn = _sparse(torch, kvq, gc, q, "f32", sel, 64, scale=0.02)
    _close(got, so.sparse_decode(oc, qn, sel, 64, scale=float(np.float32(0.02))))


def test_sparse_decode_of_nothing_and_of_far_entries():
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(26)
    gc, oc = _pair(torch, kvq, rng, 2, 1, 128, 512, 16, "q4_0", "q4_0", [512, 100])
    q = rng.standard_normal((2, 4, 128)).astype(np.float32)
    empty = np.zeros((2, 1, 0), np.int64)
    assert not _sparse(torch, kvq, gc, q, "f32", empty, 64)[0].any()
    far = np.array([[[-1, -2 ** 31, 8, 2 ** 31 - 1]], [[2, 1 << 25, -7, 3]]])
    assert not _sparse(torch, kvq, gc, q, "f32", far, 64)[0].any()
    # a page outside the pool is left out
    table = torch.tensor([0, 99, 1, 2], dtype=torch.int32)
    pc, po = _pair(torch, kvq, rng, 1, 1, 128, 256, 0, "q8_0", "q8_0", [256], page=64)
    keep = pc.page_table.clone()
    pc.page_table[1] = 99
    q = rng.standard_normal((1, 4, 128)).astype(np.float32)
    got, qn = _sparse(torch, kvq, pc, q, "f32", np.array([[[0, 1, 3]]]), 64)
    assert kvq.kvq_sync_status(pc.desc) == (kvq.KVQ_ERR_DEVICE_RANGE, kvq.KVQ_DEV_ERR_PAGE)
    _close(got, so.sparse_decode(po, qn, np.array([[[0, 3]]]), 64))
    pc.page_table.copy_(keep)


def test_every_block_listed_equals_dense_decode():
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(27)
    gc, oc = _pair(torch, kvq, rng, 2, 2, 128, 1024, 100, "q5_0", "q4_1", [1000, 333])
    q = rng.standard_normal((2, 8, 128)).astype(np.float32)
    sel = np.broadcast_to(np.arange(16), (2, 2, 16))
    got, qn = _sparse(torch, kvq, gc, q, "f32", sel, 64)
    _close(got, ko.decode_attention(oc, qn))


def test_sparse_binding_refuses_tensors():
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    gc = kvq.KVCache(2, 2, 64, 256, 0, "q4_0", "q4_0")
    x = kvq.BlockIndex(gc.desc, 64)
    q = torch.zeros(2, 4, 64, device="cuda")
    sel = torch.zeros(2, 2, 3, dtype=torch.int32, device="cuda")
    for kw in (dict(q=q[:1]), dict(q=q.double()), dict(sel=sel.long()), dict(sel=sel[:, :1]), dict(sel=sel.cpu()), dict(q=q.transpose(0, 1))):
        with pytest.raises((ValueError, kvq.KvqError)):
            kvq.kvq_select_blocks(gc.desc, x, **{**dict(q=q, sel=sel), **kw})
        with pytest.raises((ValueError, kvq.KvqError)):
            kvq.kvq_sparse_decode_attention(gc.desc, **{**dict(q=q, sel=sel, out=torch.empty_like(q), block_tokens=64), **kw})
    with pytest.raises(kvq.KvqError):
        kvq.kvq_select_blocks(gc.desc, x, q, sel, n_first=2, n_last=2)


def test_index_of_another_cache_is_refused():
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    small, large = (kvq.KVCache(1, 1, 64, n, 0, "q4_0", "q4_0") for n in (256, 512))
    x = kvq.BlockIndex(small.desc, 64)
    q = torch.zeros(1, 1, 64, device="cuda")
    with pytest.raises(ValueError):
        kvq.kvq_block_index_update(large.desc, x)
    with pytest.raises(ValueError):
        kvq.kvq_select_blocks(large.desc, x, q, torch.zeros(1, 1, 4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        kvq.BlockIndex(small.desc, 96)


@pytest.mark.parametrize("d,hkv,kt,vt,T", [(128, 8, "q8_0", "q4_0", 0), (64, 16, "q5_1", "q8_0", 40)])
def test_the_end_of_a_long_cache(d, hkv, kt, vt, T):
    """Planes past 2^32 bytes: the last tokens of four million, against the same tokens in a small cache."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(28)
    ctx, n = 1 << 22, 300
    start = ctx - 320                    # five blocks of 64 from the end
    long, short = (kvq.KVCache(1, hkv, d, c, T, kt, vt) for c in (ctx, 320))
    k, v = (to_dev(rng.standard_normal((1, n, hkv, d)), "bf16", torch) for _ in range(2))
    long.seq_len.fill_(start)
    for c in (long, short):
        kvq.kvq_rotate_quantize_append(c.desc, k, v)
    q = to_dev(rng.standard_normal((1, 2 * hkv, d)), "f32", torch)
    out = []
    for c, first in ((long, start // 64), (short, 0)):
        x = kvq.BlockIndex(c.desc, 64)
        kvq.kvq_block_index_update(c.desc, x, n_last=n)
        sel = torch.tensor([4, 2, 0, 1], dtype=torch.int32, device="cuda").expand(1, hkv, 4).add(first).contiguous()
        o = torch.empty_like(q)
        kvq.kvq_sparse_decode_attention(c.desc, q, sel, o, 64)
        out.append((o, x.codes[:, :, first:first + 5], x.scales[:, :, first:first + 5]))
        assert kvq.kvq_sync_status(c.desc)[0] == 0
    assert torch.equal(out[0][1], out[1][1]) and torch.equal(out[0][2], out[1][2])
    # (the tail's slots differ, the sums may be split elsewhere: a few fp32 roundings)
    assert torch.allclose(out[0][0], out[1][0], atol=1e-5, rtol=1e-5)


def test_calls_on_a_stream_of_their_own_and_at_once():
    """Two selections and sparse decodes of one cache on two streams at once give what they give alone."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(29)
    gc, oc = _pair(torch, kvq, rng, 2, 2, 128, 4096, 64, "q8_0", "q4_0", [4000, 3000])
    x = kvq.BlockIndex(gc.desc, 64)
    kvq.kvq_block_index_update(gc.desc, x)
    qs = [to_dev(rng.standard_normal((2, 8, 128)), "bf16", torch) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    res = [(torch.empty(2, 2, 9, dtype=torch.int32, device="cuda"), torch.empty(2, 8, 128, device="cuda")) for _ in range(2)]

    def one(i, stream):
        kvq.kvq_select_blocks(gc.desc, x, qs[i], res[i][0], stream=stream)
        kvq.kvq_sparse_decode_attention(gc.desc, qs[i], res[i][0], res[i][1], 64, stream=stream)

    alone = []
    for i in range(2):
        one(i, None)
        torch.cuda.synchronize()
        alone.append([t.clone() for t in res[i]])
        for t in res[i]:
            t.fill_(0)
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(2):
            one(i, streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(res[i][0], alone[i][0]) and torch.equal(res[i][1], alone[i][1])
        codes, scales = x.codes.cpu().numpy(), x.scales.cpu().numpy()
        assert np.array_equal(alone[i][0].cpu().numpy(), so.select_blocks(qs[i].float().cpu().numpy(), codes, scales, oc.seq_len, 64, 1, 1, 9, True))
        _close(alone[i][1].cpu().numpy().astype(np.float64), so.sparse_decode(oc, qs[i].float().cpu().numpy(), alone[i][0].cpu().numpy(), 64))


@pytest.mark.parametrize("B,hkv,g,nsel", [(300, 3, 2, 3), (1, 1, 8, 16), (2, 1, 100, 5)])
def test_sparse_decode_many_rows_and_many_heads(B, hkv, g, nsel):
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(30)
    lens = [int(n) for n in rng.integers(0, 257, B)]
    gc, oc = _pair(torch, kvq, rng, B, hkv, 64, 256, 10, "q4_0", "q5_0", lens)
    sel = rng.integers(-1, 4, (B, hkv, nsel))
    q = rng.standard_normal((B, hkv * g, 64)).astype(np.float32)
    got, qn = _sparse(torch, kvq, gc, q, "f16", sel, 64)
    _close(got, so.sparse_decode(oc, qn, sel, 64))
