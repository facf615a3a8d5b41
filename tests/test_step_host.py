"""Host checks of the step operators (norms with rotation, page maps, block index, block
selection, sparse decode): what the C ABI refuses before any launch, and the oracle against
closed forms.  No GPU."""

import ctypes

import numpy as np
import pytest

from oracle import kvq_oracle as ko
from oracle import step_oracle as so
from rotated_bit_kv_kvq_gb300 import kvq
from test_abi_host import FAKE, _full_desc

INVALID, UNSUPPORTED = kvq.KVQ_ERR_INVALID_ARG, kvq.KVQ_ERR_UNSUPPORTED


def _rope(**kw):
    r = kvq.kvq_rope_norm(128, 0, 1e-6, kvq.KVQ_F32, FAKE, FAKE, FAKE)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def _norm_rope(c=None, r=None, **kw):
    a = dict(dtype=kvq.KVQ_BF16, n_q_heads=8, q=FAKE, q_stride=1024, k=FAKE, k_stride=512, v=FAKE, v_stride=512, pos=FAKE,
             dst_row=None, n_rows=4, n_dst_rows=4, q_out=FAKE, k_out=FAKE, v_out=FAKE, stream=None)
    a.update(kw)
    c = _full_desc() if c is None else c
    return kvq.lib().kvq_qk_norm_rope(ctypes.byref(c), ctypes.byref(_rope() if r is None else r), *a.values())


@pytest.mark.parametrize("kw", [
    dict(dtype=3), dict(n_q_heads=0), dict(q=None), dict(k=None), dict(q_out=None), dict(v=None), dict(v_out=None),
    dict(q=FAKE + 8), dict(v_out=FAKE + 2), dict(q_stride=1023), dict(q_stride=512), dict(k_stride=508),
    dict(k_stride=513), dict(pos=None), dict(pos=FAKE + 2), dict(dst_row=FAKE + 1), dict(n_rows=-1),
    dict(n_dst_rows=3), dict(n_dst_rows=-1), dict(v_stride=1 << 61), dict(q_stride=1 << 59),
])
def test_norm_rope_refuses(built_lib_path, kw):
    assert _norm_rope(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(rot_dim=8), dict(rot_dim=-16), dict(rot_dim=144), dict(inv_freq=None),
                                dict(inv_freq=FAKE + 2), dict(eps=-1.0), dict(eps=float("nan")), dict(weight_dtype=4),
                                dict(q_weight=FAKE + 4)])
def test_norm_rope_refuses_the_plan(built_lib_path, kw):
    assert _norm_rope(r=_rope(**kw)) == INVALID


def test_norm_rope_without_rows_is_a_no_op(built_lib_path):
    assert _norm_rope(n_rows=0, n_dst_rows=0, q=None, k=None, v=None, q_out=None, k_out=None, v_out=None, pos=None) == 0
    assert kvq.lib().kvq_qk_norm_rope(None, ctypes.byref(_rope()), *([0] * 16)) == INVALID


def _paged():
    c = _full_desc()
    c.page_tokens, c.n_pages, c.page_table = 64, 8, FAKE
    return c


def _pages(c=None, pool=None, **kw):
    a = dict(n_new=FAKE, n_new_max=4, granted=FAKE, max_rows=8, row_pos=None, row_dst=None, row_slot=None,
             seq_len_out=None, stream=None)
    a.update(kw)
    pool = kvq.kvq_page_pool(FAKE, FAKE, FAKE) if pool is None else pool
    return kvq.lib().kvq_page_update(ctypes.byref(_paged() if c is None else c), ctypes.byref(pool), *a.values())


def test_page_update_refuses(built_lib_path):
    assert _pages(c=_full_desc()) == INVALID                       # not paged
    for kw in (dict(n_new=None), dict(granted=None), dict(n_new_max=-1), dict(max_rows=-1), dict(row_dst=FAKE + 2),
               dict(n_new_max=1 << 30), dict(seq_len_out=FAKE + 1)):
        assert _pages(**kw) == INVALID, kw
    for pool in ((None, FAKE, FAKE), (FAKE, None, FAKE), (FAKE, FAKE, None), (FAKE + 2, FAKE, FAKE)):
        assert _pages(pool=kvq.kvq_page_pool(*pool)) == INVALID
    c = _paged()
    c.n_pages = 1 << 26                                            # pool slots past int32
    assert _pages(c=c) == INVALID
    c = _paged()
    c.seq_len = None
    assert _pages(c=c) == INVALID


def _index(**kw):
    x = kvq.kvq_block_index(64, FAKE, FAKE)
    for k, v in kw.items():
        setattr(x, k, v)
    return ctypes.byref(x)


def test_block_index_and_selection_refuse(built_lib_path):
    L = kvq.lib()
    c = _full_desc()
    ref = ctypes.byref(c)
    for x in (_index(block_tokens=0), _index(block_tokens=96), _index(block_tokens=1 << 17), _index(codes=None),
              _index(codes=FAKE + 8), _index(scales=None), _index(scales=FAKE + 2)):
        assert L.kvq_block_index_update(ref, x, 0, None) == INVALID
    assert L.kvq_block_index_update(ref, _index(), -1, None) == INVALID
    assert L.kvq_block_index_update(ref, None, 0, None) == INVALID

    def select(c=c, x=None, q=FAKE, dt=0, hq=8, first=1, last=1, n=4, sel=FAKE):
        return L.kvq_select_blocks(ctypes.byref(c), x or _index(), q, dt, hq, first, last, n, sel, None)

    for kw in (dict(q=None), dict(q=FAKE + 4), dict(dt=3), dict(hq=6), dict(hq=0), dict(first=-1), dict(last=-1),
               dict(first=3, last=2), dict(n=0, first=0, last=0), dict(sel=None), dict(sel=FAKE + 2)):
        assert select(**kw) == INVALID, kw
    assert select(hq=4 * 129) == UNSUPPORTED
    assert select(n=49153) == UNSUPPORTED
    long = _full_desc(max_ctx=64 * 49153)
    assert select(c=long) == UNSUPPORTED                           # too many blocks of 64
    for bad in (dict(head_dim=96), dict(head_dim=512)):
        cc = _full_desc(**bad)
        assert select(c=cc) == UNSUPPORTED
        assert L.kvq_block_index_update(ctypes.byref(cc), _index(), 0, None) == UNSUPPORTED


def test_sparse_decode_refuses(built_lib_path):
    L = kvq.lib()

    def sparse(c=None, q=FAKE, qd=0, hq=8, scale=0.0, bt=64, sel=FAKE, n=4, out=FAKE, od=0):
        c = _full_desc() if c is None else c
        return L.kvq_sparse_decode_attention(ctypes.byref(c), q, qd, hq, scale, bt, sel, n, out, od, None)

    for kw in (dict(q=None), dict(out=None), dict(q=FAKE + 4), dict(qd=9), dict(od=-1), dict(hq=7), dict(scale=-1.0),
               dict(scale=float("nan")), dict(bt=32), dict(bt=0), dict(sel=None), dict(sel=FAKE + 1), dict(n=-1)):
        assert sparse(**kw) == INVALID, kw
    assert sparse(c=_full_desc(head_dim=160)) == UNSUPPORTED
    out = _full_desc()
    out.n_outlier, out.outlier_idx, out.outl = 32, FAKE, FAKE
    assert sparse(c=out) == UNSUPPORTED


# ---- the oracle --------------------------------------------------------------------------

def test_oracle_norm_rope_closed_forms():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((3, 2, 64))
    # position 0: the norm alone; pairs keep their length; a quarter turn swaps them
    y = so.norm_rope(x, np.ones(64), 0.0, [0, 0, 0], np.ones(32), False)
    assert np.allclose((y * y).mean(-1), 1.0)
    z = so.norm_rope(x, None, 0.0, [7, 8, 9], np.linspace(0.1, 1, 16), True)
    assert np.allclose((x[..., 0:32:2] ** 2 + x[..., 1:32:2] ** 2), z[..., 0:32:2] ** 2 + z[..., 1:32:2] ** 2)
    assert np.array_equal(x[..., 32:], z[..., 32:])
    t = so.norm_rope(x, None, 0.0, [1, 1, 1], [np.pi / 2], False)
    assert np.allclose(t[..., 0], -x[..., 1]) and np.allclose(t[..., 1], x[..., 0])
    # scores of rotated queries and keys depend on the distance alone
    q, k = rng.standard_normal((1, 1, 32)), rng.standard_normal((1, 1, 32))
    f = 10.0 ** -np.linspace(0, 3, 16)
    dot = [float((so.norm_rope(q, None, 0, [a + 5], f, False) * so.norm_rope(k, None, 0, [a], f, False)).sum())
           for a in (0, 3, 1000)]
    assert np.allclose(dot, dot[0])


def test_oracle_page_update_hands_out_each_page_once():
    rng = np.random.default_rng(6)
    P, ctx, B, n_pages = 64, 512, 6, 30
    table = np.full((B, ctx // P), -1)
    ring, state, lens = rng.permutation(n_pages), np.array([0, n_pages]), np.zeros(B, np.int64)
    for step in range(40):
        new = rng.integers(-1, 90, B)
        o = so.page_update(lens, new, 89, ctx, P, table, ring, state, 1000)
        lens, table, ring, state = o["after"] + o["granted"], o["table"], o["ring"], o["state"]
        held = [table[b, j] for b in range(B) for j in range(-(-int(lens[b]) // P))]
        free = [ring[(state[0] + i) % n_pages] for i in range(state[1])]
        assert sorted(held + free) == list(range(n_pages))
        got = [s for s in o["row_slot"] if s >= 0]
        assert len(set(got)) == len(got) == o["granted"].sum()


def test_oracle_selection_and_means():
    assert so.block_mean(np.full((5, 64), 0.5, np.float32))[0].tolist() == [127] * 64
    codes, scale = so.block_mean(np.zeros((64, 32), np.float32))
    assert scale == 0 and not codes.any()
    x = np.random.default_rng(7).standard_normal((64, 64)).astype(np.float32)
    codes, scale = so.block_mean(x)
    assert np.abs(codes * scale - x.mean(0)).max() <= scale * 0.501
    # equal scores: the lowest blocks; the first and the last always
    same = np.ones((1, 1, 9, 64), np.int8)
    sel = so.select_blocks(np.ones((1, 1, 64)), same, np.ones((1, 1, 9), np.float32), [9 * 64], 64, 1, 1, 4, False)
    assert sel[0, 0].tolist() == [0, 1, 2, 8]
    # all blocks listed: dense decode
    rng = np.random.default_rng(8)
    oc = ko.OracleCache(1, 1, 64, 256, 16, "q8_0", "q4_0", True, True)
    oc.append(rng.standard_normal((1, 150, 1, 64)), rng.standard_normal((1, 150, 1, 64)))
    q = rng.standard_normal((1, 2, 64))
    assert np.allclose(so.sparse_decode(oc, q, np.array([[[2, 0, 1, -1]]]), 64), ko.decode_attention(oc, q), atol=1e-12)


def test_binding_module_builds_and_refuses_descriptors():
    """The extension module loads without a GPU and tells descriptors apart before it looks at a tensor."""
    torch = pytest.importorskip("torch")
    n = kvq.native()
    c, x = kvq.descriptor(1, 1, 64, 64, 0, "q4_0", "q4_0"), kvq.kvq_block_index(64, FAKE, FAKE)
    t = torch.zeros(1, 1, 64)
    for args in ((c, c, 0, 0), (x, x, 0, 0), (None, x, 0, 0), (c, x, 1 << 40, 0), (c, x, "1", 0), (c, x, 0, "s"), (c, x)):
        with pytest.raises(ValueError):
            n.block_index_update(*args)
    assert n.block_index_update(_full_desc(), x, -1, 0) == INVALID           # through to the C ABI's own checks
    with pytest.raises(ValueError):
        n.select_blocks(c, x, [1.0], t, 1, 1, None)
    with pytest.raises(ValueError):
        n.sparse_decode_attention(c, t, None, t, 64, 0.0, None)
    with pytest.raises(ValueError):
        n.page_update(c, kvq.kvq_page_pool(FAKE, FAKE, FAKE), 0, None, 1, t, None, None, None, None, None)
