"""Page table and row maps built on the GPU against the oracle's one-by-one bookkeeping (exact)."""

import numpy as np
import pytest

from kvq_testlib import require_gpu
from oracle import step_oracle as so

pytestmark = pytest.mark.gpu


class _Pool:
    """A paged cache's descriptor with the arrays that the call touches, and their oracle twins."""

    def __init__(self, torch, kvq, B, ctx, P, n_pages, seed=0, head=0):
        rng = np.random.default_rng(seed)
        self.torch, self.kvq, self.B, self.ctx, self.P = torch, kvq, B, ctx, P
        self.status = torch.zeros(4, dtype=torch.int32, device="cuda")
        self.lens, self.table = np.zeros(B, np.int64), np.full((B, ctx // P), -1, np.int64)
        self.ring, self.state = rng.permutation(n_pages), np.array([head, n_pages])
        self.desc = kvq.descriptor(B, 1, 64, ctx, 0, "q4_0", "q4_0", page_tokens=P, n_pages=n_pages)

    def dev(self, x):
        return self.torch.tensor(np.asarray(x), dtype=self.torch.int32, device="cuda")

    def step(self, new, n_new_max, max_rows, in_place=True, maps=True):
        """One call on the GPU and in the oracle; their results compared; the state advanced."""
        torch, kvq = self.torch, self.kvq
        max_rows = max_rows if maps else self.B * n_new_max  # without maps the binding sets no limit
        want = so.page_update(self.lens, new, n_new_max, self.ctx, self.P, self.table, self.ring, self.state, max_rows)
        seq, table, ring, state = (self.dev(x) for x in (self.lens, self.table, self.ring, self.state))
        nxt, after = (state, seq) if in_place else (torch.full_like(state, 99), torch.full_like(seq, 99))
        granted = torch.full((self.B,), 99, dtype=torch.int32, device="cuda")
        rows = [torch.full((max_rows,), 99, dtype=torch.int32, device="cuda") for _ in range(3)] if maps else [None] * 3
        for f, t in (("seq_len", seq), ("status", self.status), ("page_table", table)):
            setattr(self.desc, f, t.data_ptr())
        pool = kvq.kvq_page_pool(ring.data_ptr(), state.data_ptr(), nxt.data_ptr())
        kvq.kvq_page_update(self.desc, pool, self.dev(new), n_new_max, granted, *rows, seq_len_out=after)
        torch.cuda.synchronize()
        got = dict(granted=granted, after=after, table=table, ring=ring, state=nxt)
        if maps:
            got.update(row_pos=rows[0], row_dst=rows[1], row_slot=rows[2])
        for name, t in got.items():
            assert np.array_equal(t.cpu().numpy(), want[name]), (name, t.cpu().numpy(), want[name])
        st = self.status.cpu().numpy()
        assert st[0] == want["bits"] and not st[1:].any(), (st, want["bits"])
        self.status.zero_()
        if not in_place:
            assert np.array_equal(state.cpu().numpy(), self.state) and np.array_equal(seq.cpu().numpy(), self.lens)
        self.lens, self.table, self.ring, self.state = want["after"] + want["granted"], want["table"], want["ring"], want["state"]
        return want


@pytest.mark.parametrize("B,P,ctx,pages,widest,seed", [(1, 64, 64, 1, 64, 1), (3, 64, 512, 20, 70, 2), (32, 64, 1024, 300, 200, 3),
                                                       (33, 256, 4096, 200, 1000, 4), (1025, 64, 256, 2000, 9, 5),
                                                       (2500, 128, 512, 9000, 130, 6)])
def test_serving_steps(B, P, ctx, pages, widest, seed):
    """Random steps: requests, releases, values out of range, a pool and a row space that run out."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    p = _Pool(torch, kvq, B, ctx, P, pages, seed, head=pages // 2)
    rng = np.random.default_rng(seed)
    for step in range(12):
        new = rng.integers(0, widest + 1, B)
        kind = rng.random(B)
        new = np.where(kind < 0.1, -1, np.where(kind < 0.3, 0, np.where(kind < 0.33, rng.choice([-2, widest + 1, 1 << 30], B), new)))
        total = int(np.clip(new, 0, widest).sum())
        p.step(new, widest, max(0, [total + 5, total // 2, total, 1][step % 4]), in_place=bool(step % 2), maps=step % 5 != 4)


def test_nothing_asked_everything_released():
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    p = _Pool(torch, kvq, 4, 512, 64, 32, 7, head=31)
    p.step(np.array([100, 64, 0, 512]), 512, 700)
    p.step(np.zeros(4, np.int64), 512, 0)
    want = p.step(np.full(4, -1), 512, 3)
    assert want["state"][1] == 32 and not want["after"].any()
    p.step(np.full(4, -1), 0, 0)                      # empty sequences hold nothing
    p.step(np.array([512, 512, 512, 512]), 512, 2048)  # the whole pool
    want = p.step(np.array([0, 0, 0, 1]), 1, 4)        # past max_ctx
    assert want["bits"] == kvq.KVQ_DEV_ERR_APPEND_RANGE


@pytest.mark.parametrize("state", [(-1, 4), (8, 4), (0, 9), (0, -1)])
def test_a_state_out_of_range_is_reported(state):
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    p = _Pool(torch, kvq, 2, 128, 64, 8)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    seq, table, ring, st, nxt = i32(64, 64), i32(0, -1, 1, -1), i32(*range(8)), i32(*state), i32(5, 5)
    granted, after, dst = i32(9, 9), i32(9, 9), i32(*[9] * 4)
    for f, t in (("seq_len", seq), ("status", p.status), ("page_table", table)):
        setattr(p.desc, f, t.data_ptr())
    kvq.kvq_page_update(p.desc, kvq.kvq_page_pool(ring.data_ptr(), st.data_ptr(), nxt.data_ptr()), i32(1, -1), 1, granted,
                        row_dst=dst, seq_len_out=after)
    torch.cuda.synchronize()
    assert p.status[0].item() & kvq.KVQ_DEV_ERR_PAGE
    assert granted.tolist() == [0, 0] and after.tolist() == [64, 64] and nxt.tolist() == list(state)
    assert table.tolist() == [0, -1, 1, -1] and ring.tolist() == list(range(8)) and dst.tolist() == [-1] * 4


def test_pool_class_refusals():
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    c = kvq.descriptor(2, 1, 64, 256, 0, "q4_0", "q4_0", page_tokens=64, n_pages=3)
    pool = kvq.PagePool(c, free=[2, 0])
    assert pool.state.tolist() == [0, 2] and pool.ring.tolist() == [2, 0, -1]
    for free in (range(4), [0, 0], [-1], [3]):
        with pytest.raises(ValueError):
            kvq.PagePool(c, free=free)
    i = torch.zeros(2, dtype=torch.int32, device="cuda")
    for bad in (i.long(), i[:1], i.cpu()):
        with pytest.raises(ValueError):
            kvq.kvq_page_update(c, pool, bad, 1, i)
    with pytest.raises(ValueError):
        kvq.kvq_page_update(c, pool, i, 1, i, row_pos=i, row_dst=i[:1])
