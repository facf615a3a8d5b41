"""Host checks of the operators for shared and continued sequences: what the C ABI and the binding refuse before any
launch, and the oracle against closed forms.  No GPU."""

import ctypes

import numpy as np
import pytest

from oracle import share_oracle as sh
from rotated_bit_kv_kvq_gb300 import kvq
from test_abi_host import FAKE, _full_desc

INVALID, UNSUPPORTED, WORKSPACE = kvq.KVQ_ERR_INVALID_ARG, kvq.KVQ_ERR_UNSUPPORTED, kvq.KVQ_ERR_WORKSPACE
POOL, SHARE = kvq.kvq_page_pool(FAKE, FAKE, FAKE), kvq.kvq_page_share(FAKE, FAKE)


def _paged(**kw):
    c = _full_desc()
    c.page_tokens, c.n_pages, c.page_table = 64, 8, FAKE
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def _ref(x):
    return None if x is None else ctypes.byref(x)


def _fork(c=None, pool=POOL, share=SHARE, **kw):
    a = dict(src=FAKE, dst=FAKE, n_tokens=None, n_forks=2, granted=FAKE, seq_len_out=FAKE, stream=None)
    a.update(kw)
    return kvq.lib().kvq_page_fork(_ref(_paged() if c is None else c), _ref(pool), _ref(share), *a.values())


def _free(c=None, pool=POOL, share=SHARE, **kw):
    a = dict(release=FAKE, seq_len_out=None, stream=None)
    a.update(kw)
    return kvq.lib().kvq_page_free(_ref(_paged() if c is None else c), _ref(pool), _ref(share), *a.values())


def _compact(c=None, pool=POOL, share=SHARE, **kw):
    a = dict(table_out=FAKE, ring_out=FAKE, page_map=None, workspace=FAKE, ws_bytes=1 << 20, stream=None)
    a.update(kw)
    return kvq.lib().kvq_page_compact(_ref(_paged() if c is None else c), _ref(pool), _ref(share), *a.values())


def _chunk(c=None, mod=None, **kw):
    a = dict(q=FAKE, q_dtype=kvq.KVQ_BF16, n_q_heads=8, n_rows=4, row_start=FAKE, scale=0.0, out=FAKE, out_dtype=kvq.KVQ_BF16,
             workspace=FAKE, ws_bytes=1 << 40, stream=None)
    a.update(kw)
    return kvq.lib().kvq_chunk_attention(_ref(_full_desc() if c is None else c), _ref(mod), *a.values())


@pytest.mark.parametrize("call", [_fork, _free, _compact])
def test_page_calls_refuse(built_lib_path, call):
    assert call(c=_full_desc()) == INVALID  # not paged
    for f in ("seq_len", "status", "page_table"):
        assert call(c=_paged(**{f: None})) == INVALID
        assert call(c=_paged(**{f: FAKE + 2})) == INVALID
    for bad in (dict(page_tokens=96), dict(n_pages=0), dict(batch=0), dict(max_ctx=100)):
        assert call(c=_paged(**bad)) == INVALID
    assert call(pool=None) == INVALID
    for i in range(3):
        for p in (None, FAKE + 1):
            assert call(pool=kvq.kvq_page_pool(*[p if j == i else FAKE for j in range(3)])) == INVALID
    assert call(share=kvq.kvq_page_share(None, FAKE)) == INVALID
    assert call(share=kvq.kvq_page_share(FAKE, FAKE + 2)) == INVALID


@pytest.mark.parametrize("kw", [dict(src=None), dict(dst=None), dict(granted=None), dict(seq_len_out=None), dict(src=FAKE + 1),
                                dict(n_tokens=FAKE + 2), dict(granted=FAKE + 3), dict(n_forks=-1), dict(share=None)])
def test_fork_refuses(built_lib_path, kw):
    assert _fork(**kw) == INVALID


def test_fork_of_nothing_and_outliers(built_lib_path):
    assert _fork(n_forks=0, src=None, dst=None, granted=None) == 0
    assert _fork(n_forks=0, seq_len_out=FAKE + 64) == INVALID
    assert _fork(n_forks=0, share=kvq.kvq_page_share(FAKE, FAKE + 64)) == INVALID
    assert _fork(c=_paged(k_qs=None)) == INVALID  # its pages are copied
    c = _paged(n_outlier=32, outlier_idx=FAKE, outl=FAKE)
    assert _fork(c=c) == (UNSUPPORTED if c.tail_len else kvq.KVQ_ERR_CUDA)


def test_free_refuses(built_lib_path):
    for kw in (dict(release=None), dict(release=FAKE + 1), dict(seq_len_out=FAKE + 2), dict(share=None)):
        assert _free(**kw) == INVALID


def test_compact_refuses(built_lib_path):
    for kw in (dict(table_out=None), dict(ring_out=None), dict(table_out=FAKE + 1), dict(ring_out=FAKE + 2), dict(page_map=FAKE + 3),
               dict(c=_paged(v_qs=None))):
        assert _compact(**kw) == INVALID
    need = kvq.kvq_page_compact_workspace_bytes(_paged())
    assert need >= 8 * 16 and kvq.kvq_page_compact_workspace_bytes(_full_desc()) == 0
    for kw in (dict(workspace=None), dict(workspace=FAKE + 8), dict(ws_bytes=need - 1)):
        assert _compact(**kw) == WORKSPACE


@pytest.mark.parametrize("kw", [dict(q=None), dict(out=None), dict(row_start=None), dict(q=FAKE + 8), dict(out=FAKE + 4),
                                dict(row_start=FAKE + 2), dict(q_dtype=3), dict(out_dtype=-1), dict(n_q_heads=0), dict(n_q_heads=7),
                                dict(n_rows=-1), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=1e31)])
def test_chunk_refuses(built_lib_path, kw):
    assert _chunk(**kw) == INVALID


@pytest.mark.parametrize("mod", [dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=1e31), dict(slopes=FAKE + 2),
                                 dict(first_key=FAKE + 1), dict(prefix_len=FAKE + 3)])
def test_chunk_refuses_the_scores(built_lib_path, mod):
    m = kvq.kvq_score_mod()
    for k, v in mod.items():
        setattr(m, k, v)
    assert _chunk(mod=m) == INVALID


def test_chunk_sizes(built_lib_path):
    c = _full_desc()
    need = kvq.kvq_chunk_workspace_bytes(c, 8, 4)
    assert need > 0 and kvq.kvq_chunk_workspace_bytes(c, 7, 4) == 0 and kvq.kvq_chunk_workspace_bytes(c, 8, -1) == 0
    for kw in (dict(workspace=None), dict(workspace=FAKE + 4), dict(ws_bytes=need - 1)):
        assert _chunk(**kw) == WORKSPACE
    assert _chunk(n_rows=0, q=None, out=None, row_start=None, workspace=None, ws_bytes=0) == 0
    for bad in (dict(head_dim=96), dict(n_outlier=32, outlier_idx=FAKE, outl=FAKE)):
        c = _full_desc()
        for k, v in bad.items():
            setattr(c, k, v)
        assert _chunk(c=c) == UNSUPPORTED and kvq.kvq_chunk_workspace_bytes(c, 8, 4) == 0
    assert _chunk(n_rows=1 << 28) == UNSUPPORTED  # 2^31 rows of work
    # the workspace holds the items of any division into sequences
    assert kvq.kvq_chunk_workspace_bytes(_full_desc(), 8, 100000) > need


def test_binding_refuses(built_lib_path):
    """What the Python calls refuse without a GPU: kinds of plans, and where they were made."""
    torch = pytest.importorskip("torch")
    c = _paged()
    t = torch.zeros(8, dtype=torch.int32)
    for f in (lambda p, s: kvq.kvq_page_fork(c, p, s, t, t, t), lambda p, s: kvq.kvq_page_free(c, p, s, t),
              lambda p, s: kvq.kvq_page_compact(c, p, s, None, None, t)):
        with pytest.raises(ValueError):
            f(3, SHARE)
        with pytest.raises(ValueError):
            f(POOL, "x")
        with pytest.raises(ValueError):
            f(POOL, kvq.PageShare(c, device="cpu"))
    with pytest.raises(ValueError):
        kvq.kvq_chunk_attention(c, t, t, t, t, mod=3)


def test_oracle_chunk_against_closed_forms():
    """Equal scores: the mean of the values seen; a steep bias: the nearest key's value; a tight cap: nearly the mean."""
    rng = np.random.default_rng(0)
    V, K = rng.standard_normal((10, 64)), np.zeros((10, 64))
    q = rng.standard_normal((4, 2, 64))
    one = lambda **kw: sh.chunk(lambda b, h: kw.pop("K", K), lambda b, h: V, False, False, q, [0, 4], [10], 1, 0.125, **kw)  # noqa: E731
    y = one()
    for i in range(4):
        assert np.allclose(y[i], V[:7 + i].mean(0))
    y = one(first_key=[7, 3, 0, 10], prefix_len=[9])
    assert np.allclose(y[0], V[7:9].mean(0)) and np.allclose(y[1], V[3:9].mean(0)) and np.allclose(y[2], V[:9].mean(0))
    assert (y[3] == 0).all()
    y = one(slopes=[1e4, 0.0])
    assert np.allclose(y[2, 0], V[8]) and np.allclose(y[2, 1], V[:9].mean(0))
    K2 = 50 * rng.standard_normal((10, 64))
    y = sh.chunk(lambda b, h: K2, lambda b, h: V, False, False, q, [0, 4], [10], 1, 0.125, softcap=1e-6)
    assert np.allclose(y[1], V[:8].mean(0), atol=1e-5)


def test_oracle_pages_by_hand():
    table = np.array([[4, 2, 7], [-1, -1, -1], [-1, -1, -1]])
    w = sh.fork([130, 0, 0], table, [1, 3, 0, 5, 6, -1, -1, -1], [0, 5], np.zeros(8, int), [0, 0], [1, 2], [130, 64], 192, 64)
    assert w["table"].tolist() == [[4, 2, 7], [4, 2, 1], [4, -1, -1]] and w["count"].tolist() == [0, 0, 1, 0, 2, 0, 0, 0]
    assert w["copies"] == [(7, 1)] and w["state"].tolist() == [1, 4] and w["after"].tolist() == [130, 130, 64] and w["bits"] == 0
    ring = np.array([1, 3, 0, 5, 6, -1, -1, -1])
    f = sh.free(w["after"], w["table"], ring, w["state"], w["count"], [1, 1, 0], 192, 64)
    assert f["count"].tolist() == [0] * 8 and f["ring"].tolist() == [1, 3, 0, 5, 6, 1, 2, 7] and f["state"].tolist() == [1, 7]
    c = sh.compact(f["after"], w["table"], f["ring"], f["state"], f["count"], 192, 64)
    assert c["moves"] == [(4, 0)] and c["table"][2].tolist() == [0, -1, -1] and c["ring"].tolist() == [1, 2, 3, 4, 5, 6, 7, -1]
