"""Host checks of the step operators that came later: calls without rows.  No GPU."""

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
