"""Block selection with queries and scales that are not numbers, and what it leaves alone, on the GPU."""

import numpy as np
import pytest

from kvq_testlib import require_gpu
from oracle import step_oracle as so

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("nblk", [300, 5000])
@pytest.mark.parametrize("rot", [True, False])
@pytest.mark.parametrize("kind", ["nan head", "inf head", "nan heads", "inf value", "nan scales", "inf scales of zero codes",
                                  "nan head and zero scales"])
def test_scores_that_are_not_numbers(kind, rot, nblk):
    """A head with a NaN score has no say; a block without a number ranks last, such blocks among themselves by place."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(51)
    d, nsel, G = 64, 40, 3
    gc = kvq.KVCache(1, 1, d, nblk * 64, 0, "q4_0", "q4_0", flags=kvq.KVQ_ROT_AUTO | (0 if rot else kvq.KVQ_ROT_K_OFF))
    gc.seq_len.fill_(nblk * 64)
    x = kvq.BlockIndex(gc.desc, 64)
    q = rng.standard_normal((1, G, d)).astype(np.float32)
    # codes along -q: the number-valued heads' scores are negative but for a few blocks
    way = so.ko.rotate(q[0].sum(0)) if rot else q[0].sum(0)
    codes = np.clip(np.rint(rng.normal(-20, 10, (nblk, 1)) * way / np.abs(way).max()), -127, 127).astype(np.int8)[None, None]
    scales = (0.01 + rng.random((1, 1, nblk))).astype(np.float32)
    if kind == "nan head":
        q[0, 1] = np.nan
    elif kind == "inf head":
        q[0, 2] = np.inf
    elif kind == "nan heads":
        q[:] = np.nan
    elif kind == "inf value":
        q[0, 0, 5] = -np.inf
    elif kind == "nan scales":
        scales[0, 0, 1:nblk - 20] = np.nan
    elif kind == "inf scales of zero codes":
        scales[0, 0, 1:nblk - 20] = np.inf
        codes[0, 0, 1:nblk - 20] = 0
    else:
        q[0, 1] = np.nan
        scales[0, 0, ::2] = 0
    x.codes.copy_(torch.from_numpy(codes))
    x.scales.copy_(torch.from_numpy(scales))
    sel = torch.full((1, 1, nsel), 77, dtype=torch.int32, device="cuda")
    kvq.kvq_select_blocks(gc.desc, x, torch.from_numpy(q).cuda(), sel)
    got = sel[0, 0].tolist()
    with np.errstate(invalid="ignore"):
        assert got == so.select_blocks(q, codes, scales, [nblk * 64], 64, 1, 1, nsel, rot)[0, 0].tolist()
    if kind in ("nan head", "inf head", "inf value"):  # what the other heads select alone
        bad = {"nan head": 1, "inf head": 2, "inf value": 0}[kind]
        alone = so.select_blocks(np.delete(q, bad, 1), codes, scales, [nblk * 64], 64, 1, 1, nsel, rot)
        assert got == alone[0, 0].tolist()
    elif kind == "nan heads":
        assert got == list(range(nsel - 1)) + [nblk - 1]
    elif kind in ("nan scales", "inf scales of zero codes"):
        assert got[-20:] == list(range(nblk - 20, nblk))


@pytest.mark.parametrize("kt", ["q4_0", "q5_0", "q8_0", "q4_1", "q5_1"])
def test_blocks_of_keys_that_are_not_numbers(kt):
    """A key scale that is infinite or NaN: its block's codes are zeros, its scale is no finite number, it ranks last."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    d, nblk = 64, 12
    gc = kvq.KVCache(1, 1, d, nblk * 64, 0, kt, "q4_0")
    gen = torch.Generator(device="cuda").manual_seed(52)
    k = torch.randn(1, nblk * 64, 1, d, device="cuda", generator=gen)
    kvq.kvq_rotate_quantize_append(gc.desc, k, k)
    x = kvq.BlockIndex(gc.desc, 64)
    kvq.kvq_block_index_update(gc.desc, x)
    before = x.codes.clone(), x.scales.clone()
    heads = gc.plane("k_d").view(torch.int16).view(nblk * 64, -1)
    heads[3 * 64 + 5, 0] = 0x7C00   # infinity
    heads[7 * 64 + 60, 0] = 0x7E00  # NaN
    kvq.kvq_block_index_update(gc.desc, x)
    bad = torch.tensor([3, 7], device="cuda")
    good = torch.tensor([j for j in range(nblk) if j not in (3, 7)], device="cuda")
    assert not x.codes[0, 0, bad].any() and not torch.isfinite(x.scales[0, 0, bad]).any()
    assert torch.equal(x.codes[0, 0, good], before[0][0, 0, good]) and torch.equal(x.scales[0, 0, good], before[1][0, 0, good])
    sel = torch.empty(1, 1, nblk - 2, dtype=torch.int32, device="cuda")
    kvq.kvq_select_blocks(gc.desc, x, torch.randn(1, 2, d, device="cuda", generator=gen), sel, n_first=0, n_last=0)
    assert sel[0, 0].tolist() == good.tolist()
