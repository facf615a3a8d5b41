"""Norms with rotation: calls without rows, on the GPU."""

import pytest

from kvq_testlib import require_gpu
from test_gpu_rope import _desc, _inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,values", [(0, True), (0, False), (6, True)])
def test_norm_rope_without_input_rows(rows, values):
    """A step without new tokens: nothing is written, with values or without, to padded rows or to none."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    hq, hkv, d = 4, 2, 64
    c, status = _desc(kvq, torch, hkv, d)
    (q, k, v), freq, pos = _inputs(torch, 3, hq, hkv, d, 64, torch.bfloat16, 500, 17)
    out = [torch.full((rows, h, d), 7.0, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv)]
    for dst in (None, pos[:0]):
        kvq.kvq_qk_norm_rope(c, kvq.RopeNorm(freq), q[:0], k[:0], v[:0] if values else None, pos[:0], out[0], out[1],
                             out[2] if values else None, dst_row=dst)
    torch.cuda.synchronize()
    assert all(bool((o == 7).all()) for o in out) and int(status[0]) == 0
