"""Plain CPU oracle of the operators around a decode step: norms with the position
rotation, page and row maps, block index, block selection, sparse decode.

TEST INFRASTRUCTURE ONLY, as ``kvq_oracle``: float64 (integers where the results are
integers, float32 one operation at a time where the definition states float32), loops over
sequences, heads and blocks, no code shared with the CUDA library.
"""

from __future__ import annotations

import math

import numpy as np

from . import kvq_oracle as ko


def norm_rope(x, weight, eps, pos, inv_freq, interleaved):
    """x [n][heads][d], pos [n], inv_freq [rot / 2]: the normed (weight not None) and rotated heads in float64."""
    x = np.asarray(x, dtype=np.float64)
    if weight is not None:
        x = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(weight, dtype=np.float64)
    y = x.copy()
    half = len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        t = np.asarray(pos, dtype=np.float64) * float(inv_freq[i])
        c, s = np.cos(t)[:, None], np.sin(t)[:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def page_update(seq_len, n_new, n_new_max, max_ctx, page_tokens, table, ring, state, max_rows):
    """One sequence after the other; returns copies of everything the call writes, and the status bits."""
    B, n_pages = len(seq_len), len(ring)
    table, ring = np.array(table), np.array(ring)
    head, count = (int(v) for v in state)
    out = dict(granted=np.zeros(B, np.int64), after=np.array(seq_len), row_pos=np.zeros(max_rows, np.int64),
               row_dst=np.full(max_rows, -1), row_slot=np.full(max_rows, -1))
    bits, row, popped, pushed = 0, 0, 0, 0
    no_page = no_row = False
    old_table = table.copy()
    for b in range(B):
        n, r = int(seq_len[b]), int(n_new[b])
        held = -(-n // page_tokens)
        if r == -1:
            for j in range(held):
                ring[(head + count + pushed + j) % n_pages] = old_table[b][j]
            pushed += held
            out["after"][b] = 0
            continue
        if r < 0 or r > n_new_max or n + r > max_ctx:
            bits |= 1
            continue
        need = -(-(n + r) // page_tokens) - held
        no_page = no_page or (need > 0 and popped + need > count)
        no_row = no_row or (r > 0 and row + r > max_rows)
        ok = not (need > 0 and no_page) and not (r > 0 and no_row)
        if not ok:
            bits |= 32
            no_page = no_page or need > 0  # nothing behind it that needs a page gets one
        if ok:
            for j in range(need):
                table[b][held + j] = ring[(head + popped + j) % n_pages]
            popped += need
            out["granted"][b] = r
        for i in range(r):
            if row + i < max_rows:
                p = n + i
                out["row_pos"][row + i] = p
                if ok:
                    out["row_dst"][row + i] = b * n_new_max + i
                    out["row_slot"][row + i] = table[b][p // page_tokens] * page_tokens + p % page_tokens
        row += r
    out.update(table=table, ring=ring, state=np.array([(head + popped) % n_pages, count - popped + pushed]), bits=bits)
    return out


def block_mean(x):
    """Codes and scale of one block: x [tokens][d] float32 values, summed in the definition's order."""
    x = np.asarray(x, dtype=np.float32)
    part = [np.zeros(x.shape[1], np.float32) for _ in range(8)]
    for t in range(len(x)):
        part[t % 8] = part[t % 8] + x[t]
    while len(part) > 1:
        part = [part[i] + part[i + 1] for i in range(0, len(part), 2)]
    mean = part[0] / np.float32(len(x))
    scale = np.abs(mean).max() / np.float32(127)
    if scale == 0:
        return np.zeros(x.shape[1], np.int8), np.float32(0)
    return np.rint(mean / scale).astype(np.int8), scale


def body_f32(oc, which, b, h, t0, t1):
    """Dequantized rotated body values as float32 (code * d exact, + minimum rounded once)."""
    return oc.body_values(which, b, h, t0, t1).astype(np.float32)


def block_index(oc, block_tokens):
    nblk = -(-oc.max_ctx // block_tokens)
    codes = np.zeros((oc.B, oc.H, nblk, oc.d), np.int8)
    scales = np.zeros((oc.B, oc.H, nblk), np.float32)
    for b in range(oc.B):
        n = int(oc.seq_len[b])
        for h in range(oc.H):
            for j in range(-(-n // block_tokens)):
                x = body_f32(oc, "k", b, h, j * block_tokens, min(n, (j + 1) * block_tokens))
                codes[b, h, j], scales[b, h, j] = block_mean(x)
    return codes, scales


def coded_query(q, rot):
    """One head's query: float32 butterflies at distance 1, 2, 4, ..., times fp32(1/sqrt(G)); int codes and scale."""
    x = np.asarray(q, dtype=np.float32)
    if rot:
        g = ko.rotation_group(len(x))
        step = 1
        while step < g:
            y = x.reshape(-1, 2, step)
            x = np.stack([y[:, 0] + y[:, 1], y[:, 0] - y[:, 1]], 1).reshape(-1)
            step *= 2
        x = x * np.float32(1 / math.sqrt(g))
    scale = np.abs(x).max() / np.float32(127)
    if scale == 0 or not np.isfinite(scale):
        return np.zeros(len(x), np.int64), scale
    return np.rint(x / scale).astype(np.int64), scale


def block_scores(q, codes, scales, rot):
    """q [group][d], codes [nblk][d] int8, scales [nblk]: one float32 score per block."""
    best = np.full(len(codes), np.nan, np.float32)
    for head in q:
        code, sq = coded_query(head, rot)
        dot = codes.astype(np.int64) @ code
        best = np.fmax(best, dot.astype(np.float32) * sq)  # (a NaN head is left out)
    return best * scales


def select_blocks(q, codes, scales, seq_len, block_tokens, n_first, n_last, n_select, rot):
    """q [B][Hq][d]; returns sel [B][Hkv][n_select]."""
    B, H, nblk, d = codes.shape
    G = q.shape[1] // H
    sel = np.full((B, H, n_select), -1, np.int64)
    for b in range(B):
        have = -(-int(seq_len[b]) // block_tokens)
        for h in range(H):
            s = block_scores(q[b, h * G:(h + 1) * G], codes[b, h, :have], scales[b, h, :have], rot).astype(np.float64)
            always = [j for j in range(have) if j < n_first or j >= have - n_last]
            s[always] = np.inf
            take = sorted(sorted(range(have), key=lambda j: (np.isnan(s[j]), -s[j], j))[:n_select])
            sel[b, h, :len(take)] = take
    return sel


def sparse_decode(oc, q, sel, block_tokens, scale=None):
    """q [B][Hq][d], sel [B][Hkv][m]: softmax attention over the listed blocks' tokens (a block listed twice twice)."""
    B, Hq, d = q.shape
    H = oc.H
    G = Hq // H
    scale = ko.default_scale(d) if scale is None else scale
    out = np.zeros((B, Hq, d))
    for b in range(B):
        n = int(oc.seq_len[b])
        for h in range(H):
            K, V = oc.stored("k", b, h), oc.stored("v", b, h)
            pos = [t for j in sel[b, h] if 0 <= j * block_tokens < n and j >= 0
                   for t in range(j * block_tokens, min(n, (j + 1) * block_tokens))]
            if not pos:
                continue
            for i in range(h * G, (h + 1) * G):
                x = np.asarray(q[b, i], dtype=np.float64)
                y = ko.softmax_attention((ko.rotate(x) if oc.rot["k"] else x)[None], K[pos], V[pos], scale)[0]
                out[b, i] = ko.rotate(y) if oc.rot["v"] else y
    return out
