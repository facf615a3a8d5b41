"""The step operators write their outputs and nothing beside them: every output lies between guards, on the GPU."""

import numpy as np
import pytest

from kvq_testlib import require_gpu, to_dev

pytestmark = pytest.mark.gpu

GUARD = 64  # elements on both sides: whole 16-byte units of every type


class _Guarded:
    """Outputs inside larger buffers of one fill value."""

    def __init__(self, torch):
        self.torch, self.all = torch, []

    def __call__(self, shape, dtype, fill=77):
        n = int(np.prod(shape))
        base = self.torch.full((n + 2 * GUARD,), fill, dtype=dtype, device="cuda")
        self.all.append((base, n, fill))
        return base[GUARD:GUARD + n].view(shape)

    def check(self):
        self.torch.cuda.synchronize()
        for base, n, fill in self.all:
            assert bool((base[:GUARD] == fill).all()) and bool((base[GUARD + n:] == fill).all())


@pytest.mark.parametrize("d,g,nblk,nsel,first,last", [
    (64, 1, 1, 1, 0, 0), (64, 2, 3, 40, 1, 1), (128, 4, 128, 32, 1, 1), (128, 4, 256, 255, 1, 1), (64, 3, 257, 9, 1, 1),
    (128, 8, 2048, 333, 2, 1), (64, 2, 2049, 2048, 1, 1), (192, 3, 5000, 1, 0, 0), (128, 1, 5000, 49152, 1, 1),
    (64, 2, 20000, 700, 1, 1), (320, 12, 33, 16, 8, 8)])
@pytest.mark.parametrize("equal", [False, True])
def test_selection(d, g, nblk, nsel, first, last, equal):
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(61)
    lens = [nblk * 64, max(1, nblk * 64 // 3), 0]
    gc = kvq.KVCache(3, 1, d, nblk * 64, 0, "q4_0", "q4_0")
    gc.seq_len.copy_(torch.tensor(lens, dtype=torch.int32))
    x = kvq.BlockIndex(gc.desc, 64)
    x.codes.copy_(torch.from_numpy(rng.integers(-99, 99, x.codes.shape).astype(np.int8)) if not equal else torch.ones_like(x.codes))
    x.scales.fill_(1)
    out = _Guarded(torch)
    sel = out((3, 1, nsel), torch.int32)
    kvq.kvq_select_blocks(gc.desc, x, to_dev(rng.standard_normal((3, g, d)), "bf16", torch), sel, n_first=first, n_last=last)
    out.check()
    for row, n in zip(sel[:, 0].cpu().numpy(), lens):
        have = -(-n // 64)
        m = min(have, nsel)
        assert (row[m:] == -1).all() and (np.diff(row[:m]) > 0).all() and (row[:m] >= 0).all() and (row[:m] < have).all()
        assert list(row[:min(first, m)]) == list(range(min(first, m)))


@pytest.mark.parametrize("kt,d", [("q8_0", 64), ("q4_0", 128), ("q5_1", 320)])
def test_index_writes_codes_and_scales_of_zero_keys(kt, d):
    """Codes and scales of what holds tokens, zeros among them; what lies behind and beside keeps its fill."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    lens = [256, 70, 0]
    gc = kvq.KVCache(3, 2, d, 256, 0, kt, "q8_0")
    k = torch.zeros(3, 256, 2, d, device="cuda")
    kvq.kvq_rotate_quantize_append(gc.desc, k, k, n_new_per_seq=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    out = _Guarded(torch)
    codes, scales = out((3, 2, 4, d), torch.int8, 3), out((3, 2, 4), torch.float32, 3)
    kvq.kvq_block_index_update(gc.desc, kvq.kvq_block_index(64, codes.data_ptr(), scales.data_ptr()))
    out.check()
    for b, n in enumerate(lens):
        have = -(-n // 64)
        assert not codes[b, :, :have].any() and not scales[b, :, :have].any()
        assert bool((codes[b, :, have:] == 3).all()) and bool((scales[b, :, have:] == 3).all())


@pytest.mark.parametrize("d,g,hkv,od", [(64, 1, 1, "bfloat16"), (128, 5, 2, "float32"), (192, 9, 1, "float16"), (320, 12, 3, "float32")])
def test_sparse_decode(d, g, hkv, od):
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(62)
    gc = kvq.KVCache(2, hkv, d, 256, 20, "q5_0", "q4_1")
    k, v = (to_dev(rng.standard_normal((2, 200, hkv, d)), "bf16", torch) for _ in range(2))
    kvq.kvq_rotate_quantize_append(gc.desc, k, v, n_new_per_seq=torch.tensor([200, 0], dtype=torch.int32, device="cuda"))
    out = _Guarded(torch)
    o = out((2, hkv * g, d), getattr(torch, od))
    sel = torch.tensor([[[0, 3, 2]] * hkv] * 2, dtype=torch.int32, device="cuda")
    kvq.kvq_sparse_decode_attention(gc.desc, to_dev(rng.standard_normal((2, hkv * g, d)), "bf16", torch), sel, o, 64)
    out.check()
    assert bool(torch.isfinite(o.float()).all()) and not bool((o[0] == 77).any()) and not o[1].any()


@pytest.mark.parametrize("n,hq,hkv,d,dt", [(1, 1, 1, 32, "float32"), (5, 3, 2, 96, "bfloat16"), (500, 5, 3, 160, "float16"),
                                           (3000, 2, 1, 64, "bfloat16")])
def test_norm_rope(n, hq, hkv, d, dt):
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    c = kvq.descriptor(1, hkv, d, 64, 0, "q4_0", "q4_0")
    out, dtype = _Guarded(torch), getattr(torch, dt)
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    c.status = c.seq_len = status.data_ptr()
    q, k, v = (torch.randn(n, h * d, device="cuda").to(dtype) for h in (hq, hkv, hkv))
    to = [out((n, h, d), dtype) for h in (hq, hkv, hkv)]
    plan = kvq.RopeNorm(torch.ones(16, device="cuda"), q_weight=torch.ones(d, device="cuda"))
    kvq.kvq_qk_norm_rope(c, plan, q, k, v, torch.arange(n, dtype=torch.int32, device="cuda"), *to)
    out.check()
    assert not any(bool((t == 77).any()) for t in to) and torch.equal(to[2].view(n, -1), v)


@pytest.mark.parametrize("batch,rows", [(1, 1), (3, 130), (40, 5), (1500, 4000)])
def test_page_update(batch, rows):
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    rng = np.random.default_rng(63)
    out = _Guarded(torch)
    table = out((batch, 4), torch.int32)
    c = kvq.descriptor(batch, 1, 64, 256, 0, "q4_0", "q4_0", page_tokens=64, n_pages=2 * batch)
    lens = torch.tensor(rng.integers(0, 100, batch), dtype=torch.int32, device="cuda")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    c.status, c.seq_len, c.page_table = status.data_ptr(), lens.data_ptr(), table.data_ptr()
    ring, state = out((2 * batch,), torch.int32), out((2,), torch.int32)
    ring.copy_(torch.arange(2 * batch))
    state.copy_(torch.tensor([batch, batch]))
    table[:, :2] = 0
    new = torch.tensor(rng.integers(-1, 60, batch), dtype=torch.int32, device="cuda")
    granted, after = out((batch,), torch.int32), out((batch,), torch.int32)
    maps = [out((rows,), torch.int32, 99999) for _ in range(3)]
    kvq.kvq_page_update(c, kvq.kvq_page_pool(ring.data_ptr(), state.data_ptr(), state.data_ptr()), new, 60, granted, *maps,
                        seq_len_out=after)
    out.check()
    assert not any(bool((m == 99999).any()) for m in maps) and bool((granted >= 0).all()) and bool((after >= 0).all())
