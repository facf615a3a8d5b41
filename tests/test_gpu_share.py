"""Forks, releases and compaction of pages on the GPU against the oracle's one-by-one bookkeeping (exact)."""

import numpy as np
import pytest

from kvq_testlib import append_both, require_gpu
from oracle import kvq_oracle as ko
from oracle import share_oracle as sh

pytestmark = pytest.mark.gpu

PLANES = ("k_qs", "k_qh", "k_d", "v_qs", "v_qh", "v_d", "outl")


class _Shared:
    """A paged cache with a pool and counts, their arrays on the GPU and in numpy."""

    def __init__(self, B, H, d, ctx, P, n_pages, T=0, kt="q4_0", vt="q4_0", seed=0, head=0, outliers=None, contents=True):
        self.contents = contents
        self.torch = torch = require_gpu()
        from rotated_bit_kv_kvq_gb300 import kvq
        self.kvq, self.rng = kvq, np.random.default_rng(seed)
        self.B, self.ctx, self.P, self.n_pages, self.per = B, ctx, P, n_pages, ctx // P
        self.gc = kvq.KVCache(B, H, d, ctx, T, kt, vt, page_tokens=P, n_pages=n_pages, outliers=outliers,
                              page_table=torch.full((B, self.per), -1, dtype=torch.int32))
        self.lens, self.table = np.zeros(B, np.int64), np.full((B, self.per), -1, np.int64)
        order = self.rng.permutation(n_pages)
        self.ring, self.state, self.count = np.roll(order, head), np.array([head, n_pages]), np.zeros(n_pages, np.int64)
        for name in PLANES:  # every page has contents of its own (finite headers)
            if contents and name in self.gc.planes:
                raw = self.rng.integers(0, 256, self.gc.planes[name].numel()).astype(np.uint8)
                if name in ("k_d", "v_d"):
                    raw = (self.rng.standard_normal(len(raw) // 2) * 0.1).astype(np.float16).view(np.uint8)
                self.gc.planes[name].copy_(torch.from_numpy(raw))

    def dev(self, x):
        return self.torch.tensor(np.asarray(x), dtype=self.torch.int32, device="cuda")

    def give(self, b, tokens):
        """Sequence b holds that many tokens (oracle side), its pages off the ring."""
        need = -(-tokens // self.P)
        head, have = self.state
        for j in range(need):
            self.table[b][j] = self.ring[(head + j) % self.n_pages]
        self.state = np.array([(head + need) % self.n_pages, have - need])
        self.lens[b] = tokens

    def upload(self, in_place):
        self.gc.seq_len.copy_(self.dev(self.lens))
        self.gc.page_table.copy_(self.dev(self.table).reshape(self.gc.page_table.shape))
        self.t = dict(ring=self.dev(self.ring), state=self.dev(self.state), count=self.dev(self.count), after=self.gc.seq_len)
        if not in_place:
            self.t.update({k + "_out": self.torch.full_like(self.t[k], 99) for k in ("ring", "state", "count", "after")})
        else:
            self.t.update({k + "_out": self.t[k] for k in ("ring", "state", "count", "after")})
        p = lambda k: self.t[k].data_ptr()  # noqa: E731
        self.pool = self.kvq.kvq_page_pool(p("ring"), p("state"), p("state_out"))
        self.share = self.kvq.kvq_page_share(p("count"), p("count_out"))
        self.before = {k: self.pages(k) for k in PLANES if self.contents and k in self.gc.planes}

    def pages(self, name):
        return self.gc.planes[name].cpu().numpy().reshape(self.n_pages, -1).copy()

    def check(self, want, got, copies, bits):
        self.torch.cuda.synchronize()
        for k, t in got.items():
            assert np.array_equal(t.cpu().numpy().reshape(np.shape(want[k])), want[k]), (k, t.cpu().numpy(), want[k])
        for k, old in self.before.items():
            now = old.copy()
            for f, t in copies:
                now[t] = old[f]
            assert np.array_equal(self.pages(k), now), k
        st = self.gc.planes["status"].view(self.torch.int32).cpu().numpy()
        assert st[0] == bits and not st[1:].any(), (st, bits)
        self.gc.planes["status"].zero_()

    def fork(self, src, dst, n_tokens=None, in_place=True):
        want = sh.fork(self.lens, self.table, self.ring, self.state, self.count, src, dst, n_tokens, self.ctx, self.P)
        self.upload(in_place)
        granted = self.torch.full((len(src),), 99, dtype=self.torch.int32, device="cuda")
        self.kvq.kvq_page_fork(self.gc.desc, self.pool, self.share, self.dev(src), self.dev(dst), granted,
                               n_tokens=None if n_tokens is None else self.dev(n_tokens), seq_len_out=self.t["after_out"])
        self.check(want, dict(granted=granted, table=self.gc.page_table, count=self.t["count_out"], after=self.t["after_out"],
                              state=self.t["state_out"]), want["copies"], want["bits"])
        assert np.array_equal(self.t["ring"].cpu().numpy(), self.ring)
        self.table, self.count, self.lens, self.state = (want[k] for k in ("table", "count", "after", "state"))
        return want

    def free(self, release, in_place=True):
        want = sh.free(self.lens, self.table, self.ring, self.state, self.count, release, self.ctx, self.P)
        self.upload(in_place)
        self.kvq.kvq_page_free(self.gc.desc, self.pool, self.share, self.dev(release), seq_len_out=self.t["after_out"])
        self.check(want, dict(ring=self.t["ring"], count=self.t["count_out"], after=self.t["after_out"], state=self.t["state_out"]),
                   [], want["bits"])
        self.ring, self.count, self.lens, self.state = (want[k] for k in ("ring", "count", "after", "state"))
        return want

    def compact(self, in_place=True, counts=True, page_map=True):
        want = sh.compact(self.lens, self.table, self.ring, self.state, self.count, self.ctx, self.P)
        self.upload(in_place)
        ws = self.torch.full((self.kvq.kvq_page_compact_workspace_bytes(self.gc.desc),), 0x5A, dtype=self.torch.uint8, device="cuda")
        table = self.gc.page_table if in_place else self.torch.full_like(self.gc.page_table, 99)
        m = self.torch.full((self.n_pages,), 99, dtype=self.torch.int32, device="cuda") if page_map else None
        self.kvq.kvq_page_compact(self.gc.desc, self.pool, self.share if counts else None, table.view(self.B, self.per),
                                  self.t["ring_out"], ws, page_map=m)
        got = dict(table=table, ring=self.t["ring_out"], state=self.t["state_out"])
        got.update(dict(count=self.t["count_out"]) if counts else {}, **(dict(map=m) if page_map else {}))
        self.check(want, got, want["moves"], want["bits"])
        if counts:
            self.count = want["count"]
        self.table, self.ring, self.state = (want[k] for k in ("table", "ring", "state"))
        return want


@pytest.mark.parametrize("d,H,P,kt,vt,B,ctx,in_place", [
    (64, 1, 64, "q4_0", "q4_0", 3, 64, True), (128, 3, 64, "q5_0", "q5_1", 9, 512, False), (256, 2, 128, "q8_0", "q4_1", 20, 1024, True),
    (96, 1, 64, "q4_1", "q5_0", 130, 256, False), (320, 2, 256, "q5_1", "q8_0", 5, 512, True)])
def test_random_steps(d, H, P, kt, vt, B, ctx, in_place):
    """Sequences begin, fork, end; the pool is compacted; now and then something invalid is asked for."""
    s = _Shared(B, H, d, ctx, P, 2 * B * (ctx // P) // 3 + 3, kt=kt, vt=vt, seed=d + B, head=1)
    bits = 0
    for step in range(8):
        for b in s.rng.permutation(B)[:max(1, B // 3)]:
            tokens = int(s.rng.integers(0, ctx + 1))
            if s.lens[b] == 0 and -(-tokens // P) <= s.state[1]:
                s.give(b, tokens)
        f = int(s.rng.integers(1, B + 3))
        src, dst = s.rng.integers(0, B, f), s.rng.integers(-1 if step % 3 == 0 else 0, B + (step % 3 == 0), f)
        if step % 2:  # mostly valid ones
            empty = s.rng.permutation(np.flatnonzero(s.lens == 0))[:f]
            if len(empty):
                dst, src = empty, src[:1].repeat(len(empty))
        n = None if step % 2 == 0 else [int(s.rng.integers(0, s.lens[b] + 2 if step % 4 == 3 else s.lens[b] + 1)) for b in src]
        bits |= s.fork(src, dst, n, in_place)["bits"]
        s.free((s.rng.random(B) < 0.4).astype(int), in_place)
        bits |= s.compact(in_place, page_map=step % 2 == 0)["bits"]
    assert bits & sh.FORK and not bits & sh.PAGE


def test_one_prompt_many_holders():
    """Pages of one sequence in 40 others: given back one by one and all at once."""
    s = _Shared(41, 1, 64, 1024, 64, 70, seed=3, head=60)
    s.give(0, 900)
    s.fork([0] * 20, range(1, 21))
    s.fork([5] * 20, range(21, 41), [64 * (i % 14) for i in range(20)])
    assert s.count.max() == 38  # (two of the shorter forks have no page)
    s.compact()
    s.free([0] + [1, 0] * 20)
    s.compact()
    s.free([1] * 41)
    assert s.state[1] == 70 and not s.count.any() and sorted(s.ring) == list(range(70))
    s.compact(in_place=False)


def test_large_pool_and_batch():
    """More pages than one CTA's threads, more sequences than a chunk of the plan."""
    s = _Shared(1500, 1, 32, 1024, 64, 20000, seed=4, head=19990)
    for b in range(0, 1500, 3):
        s.give(b, int(s.rng.integers(1, 1025)))
    s.fork([b // 3 * 3 for b in range(1500) if b % 3 == 1], [b for b in range(1500) if b % 3 == 1])
    s.free([b % 2 for b in range(1500)], in_place=False)
    s.compact(in_place=False)
    s.fork([0, 2, 4, 4], [1499, 1497, 1495, 1495], in_place=False)


def test_a_pool_past_the_bits_in_shared_memory():
    """1.1 million pages (2.5 GB): more than a cluster's shared memory has bits for, so that a release takes two rounds and a
    compaction marks in its workspace.  What is in the pages is not compared: the copies are those of the other tests."""
    s = _Shared(300, 1, 32, 1024, 64, 1100000, seed=9, head=1099000, contents=False)
    for b in range(0, 300, 2):
        s.give(b, int(s.rng.integers(1, 1025)))
    s.fork(range(0, 100, 2), range(1, 100, 2))
    assert (s.table > 8 * 4096 * 32).any()
    s.free(s.rng.random(300) < 0.5, in_place=False)
    s.free(s.rng.random(300) < 0.3)
    assert s.compact(in_place=False)["moves"]
    s.table[2][0] = s.ring[3]  # in use and free: nothing moves
    s.lens[2] = max(s.lens[2], 1)
    assert s.compact()["bits"] == sh.PAGE


def test_nothing_left():
    s = _Shared(6, 1, 64, 256, 64, 6, seed=5)
    s.give(0, 200)
    s.give(1, 64)  # 5 pages: one free
    w = s.fork([0, 1, 0, 1], [2, 3, 4, 5])
    assert list(w["granted"]) == [200, 64, -1, 64] and w["bits"] == sh.NO_ROOM
    w = s.compact(counts=False)
    assert w["bits"] == 0


def test_states_gone_wrong():
    s = _Shared(4, 1, 64, 256, 64, 8, seed=6)
    s.give(0, 200)
    s.give(1, 100)
    good, ring = s.state, s.ring
    for bad in ([-1, 2], [8, 2], [0, 9], [0, -1]):
        for in_place in (True, False):
            s.state = np.array(bad)
            s.fork([0], [2], in_place=in_place)
            s.free([1, 0, 0, 0], in_place)
            s.compact(in_place)
    s.state = good
    s.ring = ring.copy()
    s.ring[(good[0] + 1) % 8] = s.table[0][1]  # a page both held and free
    assert s.compact()["bits"] == sh.PAGE
    s.ring = np.where(np.arange(8) == (good[0] + 1) % 8, ring[good[0]], ring)  # one twice in the ring
    assert s.compact(in_place=False)["bits"] == sh.PAGE
    s.ring = ring
    s.table[0][1] = 100  # a page outside the pool
    assert s.compact()["bits"] == sh.PAGE
    assert s.free([1, 0, 0, 0])["bits"] == sh.PAGE
    s.lens[1] = 300
    assert s.free([0, 1, 0, 0])["bits"] == sh.APPEND_RANGE
    # given back more often than held
    s = _Shared(2, 1, 64, 256, 64, 8, seed=7)
    s.give(0, 64)
    s.table[1], s.lens[1] = s.table[0], 64
    assert s.free([1, 1])["bits"] == sh.PAGE
    s.ring, s.state = np.arange(8), np.array([0, 8])  # a pool that has no room
    s.give(0, 64)
    s.state = np.array([1, 8])
    assert s.free([1, 0])["bits"] == sh.PAGE


def test_outlier_planes_go_along():
    s = _Shared(3, 2, 64, 256, 64, 9, seed=8, outliers=[list(range(32)), list(range(16, 48))])
    s.give(0, 250)
    s.fork([0], [1])
    s.free([1, 0, 0])
    s.compact()
    s2 = _Shared(3, 2, 64, 256, 64, 9, T=64, seed=8, outliers=[list(range(32)), list(range(16, 48))])
    s2.give(0, 250)
    s2.upload(True)
    with pytest.raises(s2.kvq.KvqError) as e:
        s2.kvq.kvq_page_fork(s2.gc.desc, s2.pool, s2.share, s2.dev([0]), s2.dev([1]), s2.dev([0]))
    assert e.value.status == s2.kvq.KVQ_ERR_UNSUPPORTED


@pytest.mark.parametrize("d,T,kt,vt", [(64, 24, "q4_0", "q5_1"), (128, 512, "q5_0", "q8_0"), (192, 40, "q8_0", "q4_1"),
                                       (256, 64, "q5_1", "q5_0"), (32, 100, "q4_1", "q4_0")])
def test_tails(d, T, kt, vt):
    """Tails of whole and of shorter forks: rows copied where the source's tail still has them, else the stored values."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    B, H, ctx, P = 9, 2, 512, 64
    rng = np.random.default_rng(d)
    table = rng.permutation(B * 8).astype(np.int32).reshape(B, 8)
    gc = kvq.KVCache(B, H, d, ctx, T, kt, vt, page_tokens=P, n_pages=B * 8, page_table=torch.from_numpy(table))
    rot = d >= 64
    oc = ko.OracleCache(B, H, d, ctx, T, kt, vt, rot, rot)
    lens = [300, 20, 512] + [0] * 6
    k, v = rng.standard_normal((2, B, 512, H, d)).astype(np.float32)
    append_both(gc, oc, k, v, n_new_per_seq=lens, torch=torch)
    free = [p for b in range(3, B) for p in table[b]]
    pool = kvq.PagePool(gc.desc, free=[int(p) for p in free])
    share = kvq.PageShare(gc.desc)
    src, dst, n = [0, 0, 1, 2, 2, 0], [3, 4, 5, 6, 7, 8], [300, 290, 20, 100, 0, 64]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    mark = {w: gc.planes[w + "_tail"].view(torch.int16) for w in "kv"}
    for w in "kv":
        mark[w].view(B, -1)[3:] = 0x1234
        oc.tail[w][3:] = 0x1234
    granted = i32([0] * 6)
    kvq.kvq_page_fork(gc.desc, pool, share, i32(src), i32(dst), granted, n_tokens=i32(n))
    assert kvq.kvq_sync_status(gc.desc) == (0, 0)
    assert granted.tolist() == n and gc.seq_len.tolist() == lens[:3] + n
    for w in "kv":
        want = oc.tail[w].copy()
        for a, b, m in zip(src, dst, n):
            want[b] = sh.forked_tail(oc, w, a, b, m)
        assert np.array_equal(mark[w].cpu().numpy().view(np.uint16).reshape(want.shape), want)


def test_captured_and_replayed():
    """A step's fork and free in one graph, replayed: the state goes round as in eager calls."""
    s = _Shared(8, 1, 64, 512, 64, 80, seed=9)
    s.give(0, 500)
    s.give(1, 70)
    s.upload(True)
    torch, kvq = s.torch, s.kvq
    src, dst, drop = s.dev([0, 1, 0]), s.dev([2, 3, 4]), s.dev([0, 0, 1, 1, 1, 0, 0, 0])
    granted = s.dev([0, 0, 0])
    call = lambda: (kvq.kvq_page_fork(s.gc.desc, s.pool, s.share, src, dst, granted),  # noqa: E731
                    kvq.kvq_page_free(s.gc.desc, s.pool, s.share, drop))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    lens, table, ring, state, count = s.lens, s.table, s.ring, s.state, s.count
    for i in range(4):
        w = sh.fork(lens, table, ring, state, count, [0, 1, 0], [2, 3, 4], None, 512, 64)
        lens, table, state, count = w["after"], w["table"], w["state"], w["count"]
        w = sh.free(lens, table, ring, state, count, [0, 0, 1, 1, 1, 0, 0, 0], 512, 64)
        lens, ring, state, count = w["after"], w["ring"], w["state"], w["count"]
        if i:
            g.replay()
        torch.cuda.synchronize()
        for name, t, x in (("ring", s.t["ring"], ring), ("state", s.t["state"], state), ("count", s.t["count"], count),
                           ("lens", s.gc.seq_len, lens)):
            assert np.array_equal(t.cpu().numpy(), x), (i, name)
