"""A serving step as it is used: pages for the step's tokens, projection rows normed and rotated into
the padded layout, append, block index, selection and sparse decode, over several steps of a paged
cache, eager and as one replayed CUDA graph.  The oracle follows along in float64."""

import numpy as np
import pytest

from kvq_testlib import ATOL, RTOL, require_gpu
from oracle import kvq_oracle as ko
from oracle import step_oracle as so

pytestmark = pytest.mark.gpu

B, HQ, HKV, D, CTX, T, P, WIDE, BT, NSEL = 3, 8, 2, 128, 1024, 20, 64, 70, 64, 4
ROWS = 2 * WIDE


class _Step:
    def __init__(self, torch, kvq):
        i32 = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
        bf = lambda *n: torch.zeros(*n, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.torch, self.kvq = torch, kvq
        self.cache = kvq.KVCache(B, HKV, D, CTX, T, "q8_0", "q5_0", page_tokens=P, n_pages=40, page_table=i32(B * (CTX // P)))
        self.pool = kvq.PagePool(self.cache.desc, free=np.random.default_rng(1).permutation(40))
        self.index = kvq.BlockIndex(self.cache.desc, BT)
        freq = 1e-4 ** (torch.arange(D // 2, dtype=torch.float64) * 2 / D)
        self.plan = kvq.RopeNorm(freq.float().cuda(), q_weight=torch.full((D,), 1.5, device="cuda"), k_weight=torch.ones(D, device="cuda"))
        self.qkv, self.new = bf(ROWS, (HQ + 2 * HKV) * D), i32(B)
        self.granted, self.pos, self.dst, self.slot = i32(B), i32(ROWS), i32(ROWS), i32(ROWS)
        self.q, self.k, self.v = bf(B, WIDE, HQ, D), bf(B, WIDE, HKV, D), bf(B, WIDE, HKV, D)
        self.last, self.sel, self.out = bf(B, HQ, D), i32(B, HKV, NSEL), torch.zeros(B, HQ, D, device="cuda")
        self.rows = torch.arange(B, device="cuda")

    def __call__(self):
        kvq, c = self.kvq, self.cache.desc
        kvq.kvq_page_update(c, self.pool, self.new, WIDE, self.granted, self.pos, self.dst, self.slot, seq_len_out=self.cache.seq_len)
        x = self.qkv
        kvq.kvq_qk_norm_rope(c, self.plan, x[:, :HQ * D], x[:, HQ * D:(HQ + HKV) * D], x[:, (HQ + HKV) * D:], self.pos,
                             self.q, self.k, self.v, dst_row=self.dst)
        kvq.kvq_rotate_quantize_append(c, self.k, self.v, n_new_per_seq=self.granted)
        self.last.copy_(self.q[self.rows, (self.granted - 1).clamp(min=0).long()])  # the last token's query
        kvq.kvq_block_index_update(c, self.index, n_last=WIDE)
        kvq.kvq_select_blocks(c, self.index, self.last, self.sel)
        kvq.kvq_sparse_decode_attention(c, self.last, self.sel, self.out, BT)


@pytest.mark.parametrize("graph", [False, True])
def test_serving_steps(graph):
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    step = _Step(torch, kvq)
    run = step
    side = torch.cuda.Stream()
    if graph:
        with torch.cuda.stream(side):
            step()  # nothing asked for: a no-op that loads the kernels
        side.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            step()
        run = g.replay
    oc = ko.OracleCache(B, HKV, D, CTX, T, "q8_0", "q5_0", True, True)
    rng = np.random.default_rng(31)
    # prompts, decode steps, a chunk, a release and a new sequence in its place
    asks = [[70, 3, 0], [70, 1, 64], [1, 1, 1], [70, -1, 1], [70, 5, 1], [1, 1, 1], [60, 1, 1]]
    for new in asks:
        step.qkv.copy_(torch.from_numpy(rng.standard_normal(step.qkv.shape).astype(np.float32)))
        step.new.copy_(torch.tensor(new, dtype=torch.int32))
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            run()
        side.synchronize()
        assert kvq.kvq_sync_status(step.cache.desc) == (0, 0)
        granted = [max(n, 0) for n in new]
        assert step.granted.tolist() == granted
        for b, n in enumerate(new):
            if n == -1:
                oc.seq_len[b] = 0
        # the keys and values that the append saw, from the oracle's rows within a bf16 rounding of the GPU's
        x = step.qkv.float().cpu().numpy().astype(np.float64).reshape(ROWS, HQ + 2 * HKV, D)
        freq = step.plan.inv_freq.double().cpu().numpy()
        r = 0
        kn, vn = np.zeros((B, WIDE, HKV, D)), np.zeros((B, WIDE, HKV, D))
        for b, n in enumerate(granted):
            pos = int(oc.seq_len[b]) + np.arange(n)
            want = so.norm_rope(x[r:r + n, HQ:HQ + HKV], np.ones(D), float(np.float32(1e-6)), pos, freq, False)
            kn[b, :n] = step.k[b, :n].float().cpu().numpy()
            vn[b, :n] = step.v[b, :n].float().cpu().numpy()
            # one rounding to bf16, eps / 2 = 2^-8 of the value; the rest covers the fp32 error ahead of it
            # (2^-19 of the pair's size, here below 10)
            far = np.abs(kn[b, :n] - want) / (torch.finfo(torch.bfloat16).eps / 2 * np.abs(want) + 1e-4)
            assert not n or far.max() <= 1
            assert np.array_equal(vn[b, :n], x[r:r + n, HQ + HKV:])
            r += n
        oc.append(kn, vn, n_new_per_seq=granted)
        assert step.cache.seq_len.tolist() == oc.seq_len.tolist()
        q = step.last.float().cpu().numpy()
        have = [-(-int(n) // BT) for n in oc.seq_len]
        sel = step.sel.cpu().numpy()
        codes, scales = step.index.codes.cpu().numpy(), step.index.scales.cpu().numpy()
        assert np.array_equal(sel, so.select_blocks(q, codes, scales, oc.seq_len, BT, 1, 1, NSEL, True))
        assert all((sel[b] >= 0).sum() == HKV * min(have[b], NSEL) for b in range(B))
        got = step.out.cpu().numpy().astype(np.float64)
        ref = so.sparse_decode(oc, q, sel, BT)
        assert np.abs(got - ref).max() <= ATOL, np.abs(got - ref).max()
        assert np.linalg.norm(got - ref) <= RTOL * np.linalg.norm(ref)
