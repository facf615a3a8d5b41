"""Host checks of the step operators that came later: calls without rows, objects of another kind or place.  No GPU."""

import pytest

from rotated_bit_kv_kvq_gb300 import kvq
from test_abi_host import FAKE
from test_step_host import INVALID, _norm_rope


def test_norm_rope_without_rows_into_rows_of_a_padded_layout(built_lib_path):
    """No new tokens this step: inputs without rows have no address, the outputs have theirs."""
    empty = dict(q=None, k=None, v=None, pos=None, n_rows=0)
    assert _norm_rope(**empty, n_dst_rows=8) == 0
    assert _norm_rope(**empty, n_dst_rows=8, dst_row=FAKE, q_out=FAKE, k_out=FAKE, v_out=FAKE) == 0
    assert _norm_rope(**empty, n_dst_rows=0, q_out=None, k_out=None, v_out=None) == 0
    assert _norm_rope(v=None, n_dst_rows=8) == INVALID and _norm_rope(v_out=None, n_dst_rows=8) == INVALID
    assert kvq.KVQ_OK == 0


@pytest.fixture
def native(monkeypatch):
    """The calls that get as far as the compiled binding."""
    calls = []

    class Native:
        def __getattr__(self, name):
            return lambda *a: calls.append(name) or kvq.KVQ_OK
    monkeypatch.setattr(kvq, "_native", Native())
    return calls


def _objects(torch):
    c = kvq.descriptor(1, 1, 64, 64, 0, "q4_0", "q4_0", page_tokens=64, n_pages=2)
    return c, kvq.BlockIndex(c, 64, device="cpu"), kvq.PagePool(c, device="cpu")


def test_objects_of_another_kind_are_refused(native):
    """A pool and an index are descriptors of the same size: neither passes for the other."""
    torch = pytest.importorskip("torch")
    c, x, pool = _objects(torch)
    for index in (pool, pool.desc, c, None):
        with pytest.raises(ValueError):
            kvq.kvq_block_index_update(c, index)
        with pytest.raises(ValueError):
            kvq.kvq_select_blocks(c, index, None, None)
    for p in (x, x.desc, c, None):
        with pytest.raises(ValueError):
            kvq.kvq_page_update(c, p, None, 1, None)
    assert not native


@pytest.mark.parametrize("current", [0, 1])
def test_objects_of_another_device_are_refused(native, monkeypatch, current):
    torch = pytest.importorskip("torch")
    c, x, pool = _objects(torch)
    calls = [lambda: kvq.kvq_block_index_update(c, x), lambda: kvq.kvq_select_blocks(c, x, None, None),
             lambda: kvq.kvq_page_update(c, pool, None, 1, None)]
    for call in calls:  # host memory
        with pytest.raises(ValueError):
            call()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: current)
    plan = kvq.RopeNorm()
    calls.append(lambda: kvq.kvq_qk_norm_rope(c, plan, *[None] * 7))
    x.device = pool.device = plan.device = 1 - current  # as if made there
    for call in calls:
        with pytest.raises(ValueError):
            call()
    assert not native
    x.device = pool.device = plan.device = current
    for call in calls:
        call()
    assert native == ["block_index_update", "select_blocks", "page_update", "qk_norm_rope"]
    plan.device = None  # nothing in it
    calls[-1]()
