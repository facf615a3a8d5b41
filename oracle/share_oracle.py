"""Plain CPU oracle of the operators for shared and continued sequences: forks, releases and compaction of pages,
attention of packed rows with capped, biased and masked scores.

TEST INFRASTRUCTURE ONLY, as ``kvq_oracle``: whole numbers one by one, float64 elsewhere, loops over sequences, pages,
heads and rows, no code shared with the CUDA library.
"""

from __future__ import annotations

import numpy as np

from . import kvq_oracle as ko

PAGE, NO_ROOM, APPEND_RANGE, FORK = 8, 32, 1, 128


def _state_ok(state, n_pages):
    return 0 <= state[0] < n_pages and 0 <= state[1] <= n_pages


def fork(seq_len, table, ring, state, count, src, dst, n_tokens, max_ctx, page_tokens):
    """Copies of the arrays that the call writes, `copies` (from page, to page) and the status bits."""
    B, n_pages = len(seq_len), len(ring)
    table, count, after = np.array(table), np.array(count), np.array(seq_len)
    head, free = (int(v) for v in state)
    granted, copies, bits, taken = [], [], 0, 0
    ok_state = _state_ok((head, free), n_pages)
    bits |= 0 if ok_state else PAGE
    named = list(dst)
    for i, (s, d) in enumerate(zip(src, dst)):
        s, d = int(s), int(d)
        if not (0 <= s < B and 0 <= d < B) or s == d or named.count(d) > 1 or seq_len[d] != 0 or not 0 <= seq_len[s] <= max_ctx:
            bits |= FORK
            granted.append(-1)
            continue
        n = int(seq_len[s]) if n_tokens is None else int(n_tokens[i])
        if not 0 <= n <= seq_len[s]:
            bits |= FORK
            granted.append(-1)
            continue
        if not ok_state:
            granted.append(-1)
            continue
        if n % page_tokens:
            taken += 1
            if taken > free:
                bits |= NO_ROOM
                granted.append(-1)
                continue
            to = int(ring[(head + taken - 1) % n_pages])
            copies.append((int(table[s][n // page_tokens]), to))
            table[d][n // page_tokens] = to
        for j in range(n // page_tokens):
            table[d][j] = table[s][j]
            count[table[s][j]] += 1
        after[d] = n
        granted.append(n)
    popped = min(taken, free) if ok_state else 0
    state = np.array([(head + popped) % n_pages if ok_state else head, free - popped])
    return dict(granted=np.array(granted), table=table, count=count, after=after, state=state, copies=copies, bits=bits)


def free(seq_len, table, ring, state, count, release, max_ctx, page_tokens):
    n_pages = len(ring)
    ring, count, after = np.array(ring), np.array(count), np.array(seq_len)
    head, have = (int(v) for v in state)
    if not _state_ok((head, have), n_pages):
        return dict(ring=ring, state=np.array(state), count=count, after=after, bits=PAGE)
    bits, drops = 0, np.zeros(n_pages, np.int64)
    for b, r in enumerate(release):
        if not r:
            continue
        if not 0 <= seq_len[b] <= max_ctx:
            bits |= APPEND_RANGE
            continue
        for j in range(-(-int(seq_len[b]) // page_tokens)):
            if 0 <= table[b][j] < n_pages:
                drops[table[b][j]] += 1
            else:
                bits |= PAGE
        after[b] = 0
    put = 0
    for p in range(n_pages):
        count[p] -= drops[p]
        if count[p] < 0:
            bits |= PAGE if count[p] < -1 else 0
            count[p] = 0
            if have + put < n_pages:
                ring[(head + have + put) % n_pages] = p
                put += 1
            else:
                bits |= PAGE
    return dict(ring=ring, state=np.array([head, have + put]), count=count, after=after, bits=bits)


def compact(seq_len, table, ring, state, count, max_ctx, page_tokens):
    """Copies of the arrays, `moves` (from page, to page), the page map and the status bits."""
    n_pages = len(ring)
    table, count = np.array(table), np.array(count)
    head, have = (int(v) for v in state)
    same = dict(table=table, ring=np.array(ring), state=np.array(state), count=count, map=np.arange(n_pages), moves=[], bits=PAGE)
    if not _state_ok((head, have), n_pages) or any(not 0 <= n <= max_ctx for n in seq_len):
        return same
    held = [[int(p) for p in table[b][:-(-int(n) // page_tokens)]] for b, n in enumerate(seq_len)]
    live = {p for row in held for p in row}
    spare = [int(ring[(head + i) % n_pages]) for i in range(have)]
    if any(not 0 <= p < n_pages for p in list(live) + spare) or len(set(spare)) < len(spare) or live & set(spare):
        return same
    hand = sorted(live | set(spare))
    low = set(hand[:len(live)])
    moves = list(zip(sorted(live - low), sorted(set(spare) & low)))
    to = dict(moves)
    for b, row in enumerate(held):
        for j, p in enumerate(row):
            table[b][j] = to.get(p, p)
    for f, t in moves:
        count[t], count[f] = count[f], 0
    left = hand[len(live):]
    ring = np.array(left + [-1] * (n_pages - len(left)))
    return dict(table=table, ring=ring, state=np.array([0, len(left)]), count=count,
                map=np.array([to.get(p, p) for p in range(n_pages)]), moves=moves, bits=0)


def forked_tail(oc, which, src, dst, n):
    """bf16 bits [H][T][d] of sequence dst's tail after it began with n tokens of src."""
    tail, whole = np.array(oc.tail[which][dst]), int(oc.seq_len[src])
    for h in range(oc.H):
        body = oc.body_values(which, src, h)
        for p in range(max(0, n - oc.T), n):
            late = p >= whole - oc.T  # else the source's slot holds a later position: the stored value, in fp32, to bf16
            tail[h, p % oc.T] = oc.tail[which][src, h, p % oc.T] if late else ko.bf16_bits(body[p].astype(np.float32))
    return tail


def chunk(keys, values, rot_k, rot_v, q, row_start, seq_len, n_kv_heads, scale, softcap=0.0, slopes=None, first_key=None,
          prefix_len=None, rounding=None, least=None):
    """keys, values(b, h): rotated rows [n][d] in float64; q [rows][heads][d].  Zeros where no key is seen; rows that belong
    to no sequence are NaN here (nothing is written there).

    rounding e: also how far the result may be off where rotated queries, keys, values and weights are each rounded by at
    most e of themselves.  A score is off by at most D = ((1 + e)^2 - 1) scale sum |q_i k_i| (the cap has a slope of at most
    1, the bias is exact), its weight by a factor within exp(+-D), a normalised one within exp(+-2D); with the weight's and
    the value's rounding a channel of the rotated result is off by at most (exp(2D) (1 + e)^2 - 1) sum p |v|, and the
    rotation back sums these over 1 / sqrt(G) of a group's channels.  least: functions like keys and values of how
    far a channel may be off besides (numbers that a format does not hold in full): D has (1 + e) scale |q| . of the first
    more, a channel of the result exp(2D) (1 + e) sum p of the second."""
    q = np.asarray(q, dtype=np.float64)
    rows, heads, d = q.shape
    G = heads // n_kv_heads
    out, off = np.full(q.shape, np.nan), np.zeros(q.shape)
    qr = ko.rotate(q) if rot_k else q
    for b in range(len(seq_len)):
        n, r0, r1 = int(seq_len[b]), int(row_start[b]), int(row_start[b + 1])
        if r1 == r0:
            continue
        t = np.arange(n)
        for h in range(n_kv_heads):
            K, V = keys(b, h), values(b, h)
            for r in range(r0, r1):
                p = n - (r1 - r)
                seen = t <= p
                if prefix_len is not None:
                    seen |= t < prefix_len[b]
                if first_key is not None:
                    seen &= t >= first_key[r]
                if p < 0 or not seen.any():
                    out[r, h * G:(h + 1) * G] = 0
                    continue
                s = (qr[r, h * G:(h + 1) * G] @ K[seen].T) * scale
                if softcap:
                    s = softcap * np.tanh(s / softcap)
                if slopes is not None:
                    s = s - np.asarray(slopes, np.float64)[h * G:(h + 1) * G, None] * np.abs(p - t[seen])
                w = np.exp(s - s.max(-1, keepdims=True))
                y = (w / w.sum(-1, keepdims=True)) @ V[seen]
                out[r, h * G:(h + 1) * G] = ko.rotate(y) if rot_v else y
                if rounding:
                    e = rounding
                    size = np.abs(qr[r, h * G:(h + 1) * G])
                    D = ((1 + e) ** 2 - 1) * scale * (size @ np.abs(K[seen]).T).max(-1, keepdims=True)
                    z = 0.0
                    if least:
                        D = D + (1 + e) * scale * (size @ least[0](b, h)[seen].T).max(-1, keepdims=True)
                        z = np.exp(2 * D) * (1 + e) * ((w / w.sum(-1, keepdims=True)) @ least[1](b, h)[seen])
                    z = z + (np.exp(2 * D) * (1 + e) ** 2 - 1) * ((w / w.sum(-1, keepdims=True)) @ np.abs(V[seen]))
                    if rot_v:
                        g = ko.rotation_group(d)
                        z = np.repeat(z.reshape(G, d // g, g).sum(-1) / np.sqrt(g), g, -1).reshape(G, d)
                    off[r, h * G:(h + 1) * G] = z
    return (out, off) if rounding else out
