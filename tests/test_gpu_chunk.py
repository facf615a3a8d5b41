"""Attention of packed rows of new tokens against the oracle, on the GPU.

Bars.  fp32 and fp16 outputs: operands as two parts of 11 bits each, so a score of size s is off by 3 * 2^-22 of the sum of
its terms' sizes, at most |q| |k| scale < 64 here: 5e-5, which is the relative error of a weight; doubled for the sums: 1e-4
of the largest output, plus half a step of the type.  bf16 outputs: operands rounded to fp16, by at most 2^-11 of
themselves; the oracle derives from that how far each element may be off, to which half a step of bf16 comes.  (The decode's
max-abs bar of 2e-3 is one for operands of 22 bits: a weight of 1 on a value of 8 is 4e-3 off by the value's rounding alone.)
Over all elements these roundings are independent: rel-L2 stays within the decode's 1e-3, plus half a step."""

import numpy as np
import pytest

from kvq_testlib import RTOL, append_both, require_gpu, to_dev
from oracle import kvq_oracle as ko
from oracle import share_oracle as sh

pytestmark = pytest.mark.gpu

STEP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def _cache(torch, kvq, rng, B, H, d, ctx, T, kt, vt, lens, page=0, flags=None, factor=1.0):
    kw = {}
    if page:
        n = B * (ctx // page) + 3
        kw = dict(page_tokens=page, n_pages=n, page_table=torch.tensor(rng.permutation(n)[:B * (ctx // page)].astype(np.int32)))
    flags = kvq.KVQ_ROT_AUTO if flags is None else flags
    gc = kvq.KVCache(B, H, d, ctx, T, kt, vt, flags=flags, **kw)
    oc = ko.OracleCache(B, H, d, ctx, T, kt, vt, not flags & kvq.KVQ_ROT_K_OFF, not flags & kvq.KVQ_ROT_V_OFF)
    k, v = factor * rng.standard_normal((2, B, max(max(lens), 1), H, d)).astype(np.float32)
    k[..., 5] *= 8
    v[..., 9] *= 8
    append_both(gc, oc, k, v, n_new_per_seq=lens, torch=torch)
    return gc, oc


def _starts(new):
    return np.concatenate([[0], np.cumsum(new)]).astype(np.int64)


def _run(torch, kvq, gc, q, start, od, mod, scale=0.0, qd=None, ws=None):
    dt = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
    qt = to_dev(q, qd or od, torch)
    out = torch.full(q.shape, 9.0, dtype=dt[od], device="cuda")
    i32 = lambda x: None if x is None else torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    f32 = lambda x: None if x is None else torch.tensor(np.asarray(x), dtype=torch.float32, device="cuda")  # noqa: E731
    m = kvq.ScoreMod(mod.get("softcap", 0.0), f32(mod.get("slopes")), i32(mod.get("first_key")), i32(mod.get("prefix_len"))) if mod else None
    if ws is None:
        ws = torch.full((kvq.kvq_chunk_workspace_bytes(gc.desc, q.shape[1], q.shape[0]),), 0xFF, dtype=torch.uint8, device="cuda")
    kvq.kvq_chunk_attention(gc.desc, qt, i32(start), out, ws, mod=m, scale=scale)
    torch.cuda.synchronize()
    return out.float().cpu().numpy().astype(np.float64), qt.float().cpu().numpy()


def _ref(oc, q, start, scale=0.0, lens=None, **mod):
    """The oracle's result, and how far operands rounded to fp16 may be off."""
    return sh.chunk(lambda b, h: oc.stored("k", b, h), lambda b, h: oc.stored("v", b, h), oc.rot["k"], oc.rot["v"], q, start,
                    oc.seq_len, oc.H, scale or ko.default_scale(oc.d), rounding=2.0 ** -11, **mod)


def _close(got, ref, od):
    ref, off = ref if isinstance(ref, tuple) else (ref, np.zeros(ref.shape))
    rest = np.isnan(ref)
    assert (got[rest] == 9.0).all(), "rows of no sequence were written"
    got, ref, off = got[~rest], ref[~rest], off[~rest]
    assert np.all(np.isfinite(got))
    if not ref.size:
        return
    err, step = np.abs(got - ref), STEP[od]
    top = np.abs(ref).max()
    if od == "bf16":
        assert np.all(err <= off + step * (np.abs(ref) + off)), err.max()
        assert np.linalg.norm(err) <= (RTOL + step) * max(np.linalg.norm(ref), 1e-30), np.linalg.norm(err) / np.linalg.norm(ref)
    else:
        tiny = 2.0 ** -25 if od == "f16" else 0.0  # half of fp16's smallest step
        assert np.all(err <= 1e-4 * top + step * np.abs(ref) + tiny), (err.max(), top)


def _check(torch, kvq, gc, oc, q, start, od, mod, scale=0.0, qd=None):
    got, qr = _run(torch, kvq, gc, q, start, od, mod, scale, qd)
    assert kvq.kvq_sync_status(gc.desc) == (0, 0)
    _close(got, _ref(oc, qr, start, scale, **mod), od)
    return got


SHAPES = [  # d, H, G, kt, vt, tail, page, lengths, new tokens
    (64, 1, 1, "q4_0", "q4_0", 0, 0, [100], [1]),
    (64, 2, 3, "q8_0", "q5_1", 30, 64, [0, 1, 64, 65, 300, 511], [0, 1, 64, 3, 7, 0]),
    (128, 2, 4, "q5_0", "q5_0", 128, 128, [129, 512, 1, 300, 127], [129, 70, 0, 1, 5]),
    (128, 1, 5, "q4_1", "q8_0", 33, 0, [1000, 64], [333, 64]),
    (192, 2, 1, "q5_1", "q4_1", 0, 64, [257, 2], [1, 2]),
    (256, 1, 6, "q8_0", "q4_0", 24, 64, [300, 63, 512], [41, 1, 1]),
    (320, 1, 12, "q4_0", "q5_0", 7, 0, [200, 0, 130], [9, 0, 130]),
    (64, 1, 128, "q4_0", "q8_0", 16, 0, [150], [2]),
    (128, 1, 130, "q5_1", "q5_1", 0, 64, [70], [3]),
]
MODS = [dict(), dict(softcap=20.0), dict(slopes=True), dict(first_key=True), dict(prefix_len=True),
        dict(softcap=5.0, slopes=True, first_key=True, prefix_len=True)]


@pytest.mark.parametrize("shape", range(len(SHAPES)))
@pytest.mark.parametrize("od", ["f32", "f16", "bf16"])
def test_shapes_and_scores(shape, od):
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    d, H, G, kt, vt, T, page, lens, new = SHAPES[shape]
    rng = np.random.default_rng(shape)
    ctx = max(512, -(-max(lens) // 64) * 64) if max(lens) <= 512 else 1024
    gc, oc = _cache(torch, kvq, rng, len(lens), H, d, ctx, T, kt, vt, lens, page)
    start = _starts(new)
    q = 0.7 * rng.standard_normal((start[-1], H * G, d)).astype(np.float32)
    pos = np.concatenate([np.arange(n - m, n) for n, m in zip(lens, new)] + [np.zeros(0, int)])
    for mod in MODS:
        mod = dict(mod)
        if mod.get("slopes"):
            mod["slopes"] = rng.uniform(0.0, 0.5, H * G).astype(np.float32)
        if mod.get("first_key"):  # documents; some rows see nothing, or only what lies ahead of them
            mod["first_key"] = np.where(rng.random(len(pos)) < 0.2, pos + 1, pos // 50 * 50)
        if mod.get("prefix_len"):
            mod["prefix_len"] = [int(rng.integers(-3, n + 10)) for n in lens]
        _check(torch, kvq, gc, oc, q, start, od, mod)


@pytest.mark.parametrize("kt", ["q4_0", "q5_0", "q8_0", "q4_1", "q5_1"])
@pytest.mark.parametrize("vt", ["q4_0", "q5_0", "q8_0", "q4_1", "q5_1"])
def test_format_pairs(kt, vt):
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(50)
    gc, oc = _cache(torch, kvq, rng, 2, 2, 64, 512, 20, kt, vt, [300, 77], 64)
    q = rng.standard_normal((36, 4, 64)).astype(np.float32)
    for od in ("bf16", "f16"):
        _check(torch, kvq, gc, oc, q, [0, 35, 36], od, {})


@pytest.mark.parametrize("d,od", [(64, "bf16"), (128, "bf16"), (128, "f16"), (256, "bf16"), (192, "bf16"), (320, "bf16")])
def test_long_context_in_many_pieces(d, od):
    """A sequence in more pieces than there are CTAs, and one token beside a chunk."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(60 + d)
    lens, new = [20000, 5000, 40], [1, 33, 2]
    gc, oc = _cache(torch, kvq, rng, 3, 1, d, 20032, 100, "q8_0", "q5_0", lens)
    q = rng.standard_normal((36, 3, d)).astype(np.float32)
    for mod in ({}, dict(first_key=np.concatenate([[7003], np.arange(33) * 90 + 700, [0, 0]]), softcap=30.0)):
        _check(torch, kvq, gc, oc, q, _starts(new), od, mod)


@pytest.mark.parametrize("od", ["bf16", "f16"])
def test_more_sequences_than_the_plan_keeps(od):
    """2,500 sequences of up to 64 tokens, from none to three rows each: the plan's loops, and its search past shared memory."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(77)
    lens = rng.integers(0, 65, 2500).tolist()
    new = [int(min(n, rng.integers(0, 4))) for n in lens]
    new[:2200] = [min(n, 1 + m) for n, m in zip(lens[:2200], new[:2200])]
    gc, oc = _cache(torch, kvq, rng, 2500, 2, 64, 64, 16, "q8_0", "q5_0", lens)
    start = _starts(new)
    assert sum(m > 0 for m in new) > 2048
    q = 0.7 * rng.standard_normal((start[-1], 4, 64)).astype(np.float32)
    _check(torch, kvq, gc, oc, q, start, od, dict(softcap=10.0))


@pytest.mark.parametrize("flags", [2, 4, 6])
@pytest.mark.parametrize("od", ["bf16", "f16"])
def test_rotation_off(flags, od):
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(70)
    gc, oc = _cache(torch, kvq, rng, 2, 1, 128, 512, 20, "q8_0", "q8_0", [200, 90], flags=kvq.KVQ_ROT_AUTO | flags)
    q = rng.standard_normal((60, 2, 128)).astype(np.float32)
    _check(torch, kvq, gc, oc, q, [0, 10, 60], od, {}, scale=0.05)


@pytest.mark.parametrize("qd", ["f32", "f16", "bf16"])
def test_query_types_and_packing(qd):
    """Rows before and behind the sequences' keep what they held."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(71)
    gc, oc = _cache(torch, kvq, rng, 3, 2, 64, 512, 0, "q8_0", "q8_0", [100, 100, 100])
    q = rng.standard_normal((50, 4, 64)).astype(np.float32)
    for od in ("bf16", "f32"):
        _check(torch, kvq, gc, oc, q, [5, 20, 20, 43], od, {}, qd=qd)


@pytest.mark.parametrize("od", ["bf16", "f16"])
@pytest.mark.parametrize("factor", [1e-5, 1e-3, 300.0])
def test_small_and_large_values(factor, od):
    """Keys and values far from 1: the result is as exact, relative to them (queries the other way round)."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(72)
    for T in (0, 64):
        gc, oc = _cache(torch, kvq, rng, 1, 1, 128, 512, T, "q8_0", "q8_0", [400], factor=factor)
        q = (rng.standard_normal((70, 2, 128)) / factor).astype(np.float32)
        got, qr = _run(torch, kvq, gc, q, [0, 70], od, {}, qd="f32")
        ref, off = _ref(oc, qr, [0, 70])
        if od == "f16" and factor < 1e-4:
            _close(got, ref, od)
        else:
            _close(got / factor, (ref / factor, off / factor), od)


@pytest.mark.parametrize("od", ["bf16", "f16", "f32"])
def test_infinities_stay_with_the_rows_that_see_them(od):
    """A value or key that is not finite makes NaN of the rows that see it; masked, it touches nobody."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(73)
    for plane, at, T in (("v_d", 150, 0), ("k_d", 150, 0), ("v_d", 150, 100), ("v_tail", 150, 100), ("k_tail", 199, 100)):
        gc, oc = _cache(torch, kvq, rng, 1, 1, 64, 256, T, "q8_0", "q4_0", [200])
        q = rng.standard_normal((100, 2, 64)).astype(np.float32)
        ref, off = _ref(oc, to_dev(q, od, torch).float().cpu().numpy(), [0, 100])
        if plane.endswith("_d"):
            gc.planes[plane].view(torch.float16).view(256, 2)[at, 1] = float("nan") if plane == "k_d" else float("inf")
            hit = T == 0
        else:
            gc.planes[plane].view(torch.bfloat16).view(T, 64)[at % T, 3] = float("inf")
            hit = True
        got, _ = _run(torch, kvq, gc, q, [0, 100], od, {})
        seen = np.arange(100) + 100 >= at
        if hit:
            assert np.isnan(got[seen]).all()
            got[seen], ref[seen] = 0, 0
        _close(got, (ref, off), od)
        # masked for everybody
        got, _ = _run(torch, kvq, gc, q[:1], [0, 1], od, dict(first_key=[at + 1]))
        if at + 1 < 200:
            assert np.isfinite(got).all()
        else:
            assert (got == 0).all()
    # a query that is not finite touches its own head's row alone
    gc, oc = _cache(torch, kvq, rng, 1, 1, 64, 256, 0, "q8_0", "q4_0", [200])
    clean, _ = _run(torch, kvq, gc, q, [0, 100], od, {})
    q[40, 1, 3] = np.inf
    got, _ = _run(torch, kvq, gc, q, [0, 100], od, {})
    assert np.isnan(got[40, 1]).all()
    got[40, 1] = clean[40, 1]
    assert np.array_equal(got, clean)


def test_errors_on_the_device():
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(74)
    gc, oc = _cache(torch, kvq, rng, 3, 1, 64, 512, 0, "q8_0", "q8_0", [100, 3, 200], 64)
    q = rng.standard_normal((20, 2, 64)).astype(np.float32)
    for od in ("bf16", "f16"):
        for start in ([0, 5, 4, 20], [-1, 5, 6, 7], [0, 5, 6, 21]):
            got, _ = _run(torch, kvq, gc, q, start, od, {})
            assert (got == 9.0).all()
            assert kvq.kvq_sync_status(gc.desc) == (kvq.KVQ_ERR_DEVICE_RANGE, kvq.KVQ_DEV_ERR_ROW)
        # more rows than tokens
        got, qr = _run(torch, kvq, gc, q, [0, 5, 15, 20], od, {})
        assert kvq.kvq_sync_status(gc.desc) == (kvq.KVQ_ERR_DEVICE_RANGE, kvq.KVQ_DEV_ERR_PREFILL_RANGE)
        _close(got, _ref(oc, qr, [0, 5, 15, 20]), od)
        assert (got[5:12] == 0).all() and (got[12:15] != 0).any()
    # a page outside the pool: its keys are left out
    gc.page_table.view(3, 8)[2, 1] = 1000
    for od in ("bf16", "f16"):
        got, qr = _run(torch, kvq, gc, q, [0, 0, 0, 20], od, dict(first_key=[64] * 10 + [0] * 10))
        assert kvq.kvq_sync_status(gc.desc) == (kvq.KVQ_ERR_DEVICE_RANGE, kvq.KVQ_DEV_ERR_PAGE)
        whole = _ref(oc, qr, [0, 0, 0, 20], first_key=[64] * 10 + [0] * 10)
        keep = np.r_[0:64, 128:200]
        K, V = oc.stored("k", 2, 0), oc.stored("v", 2, 0)
        ref = np.zeros(q.shape)
        for r in range(20):
            t = keep[(keep <= 180 + r) & (keep >= (64 if r < 10 else 0))]
            for h in range(2):
                s = ko.rotate(qr[r, h].astype(np.float64)) @ K[t].T * 0.125
                w = np.exp(s - s.max())
                ref[r, h] = ko.rotate((w / w.sum()) @ V[t])
        # (The whole's bound is a sum over all keys of weight times |value| terms.  Without the page's keys each weight is the whole's over
        # the rest's share of it, at least a quarter here: asserted below.  So is the bound, its sum only losing terms.)
        for r in range(20):
            t = np.arange(64 if r < 10 else 0, 181 + r)
            for h in range(2):
                s = ko.rotate(qr[r, h].astype(np.float64)) @ K[t].T * 0.125
                w = np.exp(s - s.max())
                assert w[(t < 64) | (t >= 128)].sum() >= 0.25 * w.sum()
        _close(got, (ref, 4 * whole[1]), od)


def test_two_streams_and_a_graph():
    """Calls with workspaces of their own on two streams at once, and a captured call, give the eager call's bits."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(75)
    gc, oc = _cache(torch, kvq, rng, 4, 2, 128, 2048, 64, "q5_0", "q8_0", [2000, 1500, 77, 900], 64)
    start = torch.tensor([0, 40, 41, 60, 100], dtype=torch.int32, device="cuda")
    for dt in (torch.bfloat16, torch.float16):
        q = torch.randn(100, 8, 128, device="cuda").to(dt)
        nb = kvq.kvq_chunk_workspace_bytes(gc.desc, 8, 100)
        ws = [torch.empty(nb, dtype=torch.uint8, device="cuda") for _ in range(3)]
        outs = [torch.zeros_like(q) for _ in range(4)]
        kvq.kvq_chunk_attention(gc.desc, q, start, outs[0], ws[0])
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream(), torch.cuda.Stream()]
        for _ in range(3):
            for i, st in enumerate(streams):
                kvq.kvq_chunk_attention(gc.desc, q, start, outs[1 + i], ws[1 + i], stream=st)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            kvq.kvq_chunk_attention(gc.desc, q, start, outs[3], ws[0])
        g.replay()
        g.replay()
        torch.cuda.synchronize()
        for o in outs[1:]:
            assert torch.equal(o, outs[0])


def test_a_life_of_shared_sequences():
    """Prompts, forks of them, new tokens of each appended and attended to, some freed, the pool compacted, on again: every
    step against an oracle that keeps every sequence by itself."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(76)
    B, H, G, d, ctx, P, T = 6, 2, 3, 64, 512, 64, 48
    gc = kvq.KVCache(B, H, d, ctx, T, "q8_0", "q5_0", page_tokens=P, n_pages=40,
                     page_table=torch.full((B, ctx // P), -1, dtype=torch.int32))
    oc = ko.OracleCache(B, H, d, ctx, T, "q8_0", "q5_0", True, True)
    pool, share = kvq.PagePool(gc.desc, free=[int(p) for p in rng.permutation(40)]), kvq.PageShare(gc.desc)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def step(new):
        granted = i32([0] * B)
        kvq.kvq_page_update(gc.desc, pool, i32(new), max(max(new), 1), granted)
        assert granted.tolist() == [max(n, 0) for n in new]
        k, v = rng.standard_normal((2, B, max(max(new), 1), H, d)).astype(np.float32)
        append_both(gc, oc, k, v, n_new_per_seq=np.maximum(new, 0), torch=torch)
        start = _starts(np.maximum(new, 0))
        q = rng.standard_normal((start[-1], H * G, d)).astype(np.float32)
        for od in ("bf16", "f16"):
            _check(torch, kvq, gc, oc, q, start, od, dict(softcap=30.0))

    def fork(src, dst, n):
        granted = i32([0] * len(src))
        kvq.kvq_page_fork(gc.desc, pool, share, i32(src), i32(dst), granted, n_tokens=i32(n))
        assert granted.tolist() == n
        for a, b, m in zip(src, dst, n):
            for w in "kv":
                oc.tail[w][b] = sh.forked_tail(oc, w, a, b, m)
                oc.codes[w][b], oc.dbits[w][b] = oc.codes[w][a], oc.dbits[w][a]
            oc.seq_len[b] = m

    ws = torch.empty(kvq.kvq_page_compact_workspace_bytes(gc.desc), dtype=torch.uint8, device="cuda")
    step([200, 100, 0, 0, 0, 0])
    fork([0, 0, 1], [2, 3, 4], [200, 150, 100])
    step([1, 5, 60, 1, 0, 0])
    kvq.kvq_page_free(gc.desc, pool, share, i32([1, 0, 0, 0, 1, 0]))
    oc.seq_len[[0, 4]] = 0
    kvq.kvq_page_compact(gc.desc, pool, share, None, None, ws)
    used = {int(p) for b in range(B) for p in gc.page_table.view(B, -1)[b, :-(-int(oc.seq_len[b]) // P)].tolist()}
    assert used == set(range(len(used)))
    step([0, 1, 1, 100, 0, 0])
    fork([3], [0], [251])
    step([3, 1, 1, 1, 64, 0])
    kvq.kvq_page_free(gc.desc, pool, share, i32([1] * B))
    assert kvq.kvq_sync_status(gc.desc) == (0, 0)
    assert pool.state.tolist()[1] == 40 and not share.count.any()
