"""Workloads of the decode-step operators around the quantized cache, in two forms each.

Five operators: norms of queries and keys per head with the position rotation in the same
pass (``rope``), the page table and row maps of a step built on the GPU (``pages``), the
int8 key means of the cache's blocks (``index``), the selection of blocks by those means
(``select``), and decode attention over the selected blocks (``sparse``).  ``run`` computes
them with elementary torch operations, or, where ``own`` is true, by the calls a user makes.

A block index holds integers: for every block the keys' mean as int8 codes with one fp32
scale.  The order of its sums is part of its definition (token t of a block is added to
partial sum t % 8 in token order, the eight partial sums are joined in pairs), and so is the
selection's score (integer dot products of int8 codes, then two fp32 products), so both
forms give the same codes and the same blocks.
"""

import math

import numpy as np
import torch

own = False

TYPES = ("q4_0", "q5_0", "q8_0", "q4_1", "q5_1")
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---- cases ------------------------------------------------------------------------------

def listed():
    return [
        # one decode step of four long sequences: one row each out of a fused projection
        dict(name="rope_step_b4", op="rope", rows=4, hq=24, hkv=4, d=256, dt="bf16", rot=256, inter=False, norm=True,
             far=65536, ragged=False),
        # a mixed batch of packed rows (prompt chunks and single tokens) to padded rows, half the channels rotated
        dict(name="rope_mixed_1001", op="rope", rows=1001, hq=32, hkv=8, d=128, dt="f16", rot=64, inter=True, norm=True,
             far=8192, ragged=True),
        # a prompt of 2 x 4096 tokens
        dict(name="rope_prompt_8k", op="rope", rows=8192, hq=32, hkv=8, d=128, dt="bf16", rot=128, inter=False,
             norm=True, far=4096, ragged=False),
        # a decode step of 32 sequences: one token each, a page now and then
        dict(name="pages_step_b32", op="pages", batch=32, ctx=8192, page=64, lo=1024, hi=8000, chunk=1, every=0),
        # continuous batching: 512 sequences, every eighth a prompt chunk, some released
        dict(name="pages_mixed_b512", op="pages", batch=512, ctx=16384, page=64, lo=0, hi=12000, chunk=2000, every=8),
        # after one appended token: the last block of 32 ragged sequences
        dict(name="index_step_b32", op="index", batch=32, hkv=8, d=128, ctx=8192, kt="q5_0", bt=64, lo=1024, hi=8192,
             last=1, page=0),
        # after a long prompt: every block of four sequences
        dict(name="index_prompt_b4", op="index", batch=4, hkv=4, d=256, ctx=65536, kt="q8_0", bt=64, lo=65536, hi=65536,
             last=0, page=0),
        # blocks of 32 ragged sequences, a quarter of the longest kept
        dict(name="select_b32_8k", op="select", batch=32, hq=32, hkv=8, d=128, ctx=8192, bt=64, nsel=32, lo=1024,
             hi=8192, dt="bf16"),
        # blocks of one document of a million tokens
        dict(name="select_b1_1m", op="select", batch=1, hq=16, hkv=4, d=128, ctx=1 << 20, bt=64, nsel=128, lo=1 << 20,
             hi=1 << 20, dt="bf16"),
        # the smallest: one head, a thousand tokens, no tail
        dict(name="sparse_d64_1k", op="sparse", batch=1, hq=1, hkv=1, d=64, ctx=1024, kt="q4_0", vt="q4_0", tail=0,
             bt=64, nsel=4, lo=1000, hi=1000, dt="f32", page=0),
        # the ragged batch: 2048 of up to 8192 tokens per head, tail blocks among them
        dict(name="sparse_b32_ragged", op="sparse", batch=32, hq=32, hkv=8, d=128, ctx=8192, kt="q5_0", vt="q5_0",
             tail=512, bt=64, nsel=32, lo=1024, hi=8192, dt="bf16", page=0),
        # the 64k decode: 8192 of 65536 tokens per head, paged
        dict(name="sparse_b4_64k", op="sparse", batch=4, hq=24, hkv=4, d=256, ctx=65536, kt="q8_0", vt="q4_0",
             tail=1024, bt=64, nsel=128, lo=65500, hi=65536, dt="bf16", page=256),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "pages", "index", "select", "select", "sparse", "sparse", "sparse"])
    dt = rng.choice(["bf16", "f16", "f32"])
    d = rng.choice([64, 128, 192, 256, 320])
    hkv = rng.choice([1, 2, 3, 4, 8])
    if op == "rope":
        d = rng.choice([32, 64, 96, 128, 192, 256, 320, 512])
        hq = hkv * rng.choice([1, 2, 3, 4, 8])
        rows = min(_spread(rng, 1, 8192), max(1, 25_000_000 // ((hq + 2 * hkv) * d)))
        return dict(op=op, rows=rows, hq=hq, hkv=hkv, d=d, dt=dt, rot=16 * rng.randint(0, d // 16), inter=rng.random() < 0.5,
                    norm=rng.random() < 0.8, far=_spread(rng, 1, 1_000_000), ragged=rng.random() < 0.5)
    if op == "pages":
        page = rng.choice([64, 128, 256])
        ctx = page * rng.randint(2, 64)
        return dict(op=op, batch=_spread(rng, 1, 2000), ctx=ctx, page=page, lo=0, hi=ctx - 1,
                    chunk=_spread(rng, 1, 300), every=rng.choice([0, 2, 5, 16]))
    bt = 64 * rng.choice([1, 1, 1, 2, 3])
    batch = _spread(rng, 1, 32)
    if op == "index":
        ctx = 64 * _spread(rng, 2, max(3, min(1024, 250_000_000 // (64 * batch * hkv * d))))
        return dict(op=op, batch=batch, hkv=hkv, d=d, ctx=ctx, kt=rng.choice(TYPES), bt=bt, lo=0, hi=ctx,
                    last=rng.choice([0, 0, 1, 7, 200]), page=rng.choice([0, 64]))
    nsel = _spread(rng, 2, 160)
    if op == "select":
        ctx = 64 * _spread(rng, 4, max(5, min(16384, 500_000_000 // (64 * batch * hkv * d))))
        return dict(op=op, batch=batch, hq=hkv * rng.randint(1, 12), hkv=hkv, d=d, ctx=ctx, bt=bt, nsel=nsel, lo=0, hi=ctx,
                    dt=dt)
    ctx = 64 * _spread(rng, 2, max(3, min(1024, 200_000_000 // (64 * batch * hkv * d))))
    nsel = min(nsel, max(2, 26_000_000 // (batch * hkv * d * bt)))
    return dict(op=op, batch=batch, hq=hkv * rng.randint(1, 12), hkv=hkv, d=d, ctx=ctx, kt=rng.choice(TYPES),
                vt=rng.choice(TYPES), tail=rng.choice([0, 30, 128, 512]), bt=bt, nsel=nsel, lo=0, hi=ctx, dt=dt,
                page=rng.choice([0, 0, 64]))


def _lengths(c):
    """Tokens of each sequence: spread over [lo, hi], the same for every seed."""
    n = c["batch"]
    return [int(round(c["lo"] + (c["hi"] - c["lo"]) * (((i + 1) * 0.6180339887498949) % 1.0))) for i in range(n)]


def _blocks(tokens, bt):
    return -(-tokens // bt)


def _new_tokens(c):
    """Per sequence: the tokens a step asks room for; -1 releases the sequence."""
    got = []
    for i, n in enumerate(_lengths(c)):
        r = 1
        if c["every"]:
            r = max(c["chunk"] - 3 * (i % 5), 0) if i % c["every"] == 1 else -1 if i % 16 == 5 else 1
        got.append(max(min(r, c["ctx"] - n), 0) if r >= 0 else r)
    return got


# ---- the work that no implementation does without ------------------------------------------

def _row_bytes(kind, d):
    return (d // 32) * {"q4_0": 18, "q5_0": 22, "q8_0": 34, "q4_1": 20, "q5_1": 24}[kind]


def work(case):
    c = case
    es = 4 if c.get("dt") == "f32" else 2
    if c["op"] == "rope":
        n = c["rows"] * (c["hq"] + 2 * c["hkv"]) * c["d"]
        return {"bytes": 2 * n * es + c["rows"] * 8 + 2 * c["d"] * es + 2 * c["rot"], "flops": 8 * n}
    if c["op"] == "pages":
        new, lens = _new_tokens(c), _lengths(c)
        rows = sum(r for r in new if r > 0)
        pages = sum(_blocks(n + r, c["page"]) - _blocks(n, c["page"]) if r >= 0 else _blocks(n, c["page"])
                    for n, r in zip(lens, new))
        return {"bytes": c["batch"] * 16 + rows * 12 + pages * 8 + 16, "flops": c["batch"] * 4}
    lens = _lengths(c)
    if c["op"] == "index":
        tok = blk = 0
        for n in lens:
            b0 = 0 if c["last"] == 0 else max(0, n - c["last"]) // c["bt"]
            tok += max(0, n - b0 * c["bt"])
            blk += max(0, _blocks(n, c["bt"]) - b0)
        return {"bytes": c["hkv"] * (tok * _row_bytes(c["kt"], c["d"]) + blk * (c["d"] + 4)) + 4 * c["batch"],
                "flops": 2 * c["hkv"] * tok * c["d"]}
    if c["op"] == "select":
        blk = sum(_blocks(n, c["bt"]) for n in lens)
        return {"bytes": c["hkv"] * (blk * (c["d"] + 4) + 4 * c["batch"] * c["nsel"]) + c["batch"] * (c["hq"] * c["d"] * es + 4),
                "flops": 2 * c["hq"] * blk * c["d"]}
    tok = tail = 0
    for n in lens:  # the listed and drawn lists always hold the last block
        t = min(n, c["nsel"] * c["bt"] - (-n % c["bt"])) if n else 0
        tok += t
        tail += min(t, c["tail"], n - (_blocks(n, c["bt"]) - 1) * c["bt"] if n else 0)
    per = _row_bytes(c["kt"], c["d"]) + _row_bytes(c["vt"], c["d"])
    return {"bytes": c["hkv"] * ((tok - tail) * per + tail * 4 * c["d"] + 4 * c["batch"] * c["nsel"]) +
            c["batch"] * (2 * c["hq"] * c["d"] * es + 4), "flops": 4 * c["hq"] * tok * c["d"]}


# ---- inputs -----------------------------------------------------------------------------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)


def _dev(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


def _k_bits():
    """Bit of channel c in a K high-bit word of the cache."""
    c = torch.arange(32, device="cuda")
    b = lambda i: (c >> i) & 1  # noqa: E731
    return 16 * b(1) + 8 * b(3) + 4 * b(4) + 2 * b(2) + b(0)


def _v_bits():
    """Part and bit of channel c in a V row's two 16-bit high-bit parts."""
    c = torch.arange(32, device="cuda")
    b = lambda i: (c >> i) & 1  # noqa: E731
    return b(3), 8 * b(2) + 4 * b(4) + 2 * b(1) + b(0)


def _quantized(y, kind, v_side):
    """Rows y [n][d] as the planes (qs, high bits or None, headers) of the cache."""
    n, d = y.shape
    nb = d // 32
    y = y.view(n, nb, 32)
    if kind == "q8_0":
        s = y.abs().amax(-1) / 127
        code = torch.where(s[..., None] > 0, torch.round(y / s[..., None]), 0).to(torch.int32)
        return (code + 128).to(torch.uint8).view(n, d), None, s.half()
    top = 31 if kind[1] == "5" else 15
    if kind.endswith("_1"):
        lo, hi = y.amin(-1), y.amax(-1)
        s = (hi - lo) / top
        code = torch.where(s[..., None] > 0, torch.floor((y - lo[..., None]) / s[..., None] + 0.5), 0)
        head = torch.stack([s.half(), lo.half()], -1)
    else:
        m = y.gather(-1, y.abs().argmax(-1, keepdim=True)).squeeze(-1)
        s = m / -((top + 1) // 2)
        code = torch.where(s[..., None] != 0, torch.floor(y / s[..., None] + (top + 1) // 2 + 0.5), 0)
        head = s.half()
    code = code.clamp(0, top).to(torch.int32)
    qs = ((code[..., :16] & 15) | ((code[..., 16:] & 15) << 4)).to(torch.uint8).view(n, d // 2)
    high = None
    if kind[1] == "5":
        bit = ((code >> 4) & 1).long()
        if not v_side:
            high = (bit << _k_bits()).sum(-1).to(torch.int32)
        else:
            part, at = _v_bits()
            two = torch.stack([((bit << at) * (part == p)).sum(-1) for p in (0, 1)], -1).to(torch.int16)  # [n][nb][2]
            high = two.view(n // 2, 2, nb, 2).permute(0, 2, 3, 1).contiguous()  # [row pair][block][part][row]
    return qs, high, head


def _rotates(d):
    return d >= 64 and d % 64 == 0


def _group(d):
    return (d if d & (d - 1) == 0 else 64) if _rotates(d) else 32


def _hadamard(d):
    """The block-diagonal normalized Walsh-Hadamard matrix of a head."""
    g = _group(d)
    i = np.arange(g)
    bits = i[:, None] & i[None, :]
    par = np.zeros_like(bits)
    while bits.any():
        par ^= bits & 1
        bits >>= 1
    return np.kron(np.eye(d // g), (1.0 - 2.0 * par) / math.sqrt(g))


def _cache(c, g, sides):
    """The planes of a cache whose rotated keys and values are drawn from g (empty planes for a side not in `sides`)."""
    B, H, C, d = c["batch"], c["hkv"], c["ctx"], c["d"]
    s = dict(seq=_dev(_lengths(c)), status=torch.zeros(4, dtype=torch.int32, device="cuda"))
    page = c.get("page", 0)
    if page:
        s["table"] = torch.randperm(B * (C // page), generator=g, device="cuda").to(torch.int32)
    T = c.get("tail", 0)
    for side in "kv":
        kind = c.get(side + "t", "q4_0")
        if side not in sides:
            nb, rb = d // 32, d if kind == "q8_0" else d // 2
            s[side + "q"] = torch.empty(B * H * C, rb, dtype=torch.uint8, device="cuda")
            s[side + "h"] = torch.empty(B * H * C, nb, dtype=torch.int32, device="cuda") if kind[1] == "5" else None
            s[side + "s"] = torch.empty(B * H * C, nb * (2 if kind.endswith("_1") else 1), dtype=torch.float16, device="cuda")
            continue
        # keys of a block share a direction, as neighbouring tokens do; values do not
        y = _randn(g, B, H, C, d)
        if side == "k":
            y += 0.5 * _randn(g, B, H, C // 64, 1, d).expand(B, H, C // 64, 64, d).reshape(B, H, C, d)
        if T:
            p = s["seq"].long()[:, None] - 1 - torch.arange(T, device="cuda")  # the last T positions
            ok = p >= 0
            rows = y[torch.arange(B, device="cuda")[:, None], :, p.clamp(min=0)].to(torch.bfloat16)  # [B][T][H][d]
            tail = torch.zeros(B, T, H, d, dtype=torch.bfloat16, device="cuda")
            slot = torch.where(ok, p % T, torch.arange(T, device="cuda")[None, :].expand(B, T))
            tail[torch.arange(B, device="cuda")[:, None].expand(B, T)[ok], slot[ok]] = rows[ok]
            s[side + "tail"] = tail.transpose(1, 2).contiguous()
        if page:
            pool = torch.empty_like(y).view(B * (C // page), H, page, d)
            pool[s["table"].long()] = y.view(B, H, C // page, page, d).transpose(1, 2).reshape(B * (C // page), H, page, d)
            y = pool
        planes = [_quantized(part, kind, side == "v") for part in y.reshape(-1, d).split(1 << 20)]
        del y
        for k, name in enumerate("qhs"):
            s[side + name] = None if planes[0][k] is None else torch.cat([p[k] for p in planes])
        del planes
    return s


def _handle(c, s):
    """The framework's descriptor of those planes."""
    from rotated_bit_kv_kvq_gb300 import kvq
    page = c.get("page", 0)
    h = kvq.descriptor(c["batch"], c["hkv"], c["d"], c["ctx"], c.get("tail", 0), c.get("kt", "q4_0"), c.get("vt", "q4_0"),
                       page_tokens=page, n_pages=c.get("n_pages", c["batch"] * (c["ctx"] // page)) if page else 0)
    for field, name in (("k_qs", "kq"), ("k_qh", "kh"), ("k_d", "ks"), ("v_qs", "vq"), ("v_qh", "vh"), ("v_d", "vs"),
                        ("k_tail", "ktail"), ("v_tail", "vtail"), ("seq_len", "seq"), ("status", "status"),
                        ("page_table", "table")):
        if s.get(name) is not None:
            setattr(h, field, s[name].data_ptr())
    return h


def _prepare_rope(c, g):
    n, hq, hkv, d, dt = c["rows"], c["hq"], c["hkv"], c["d"], DTYPES[c["dt"]]
    qkv = (2 * _randn(g, n, (hq + 2 * hkv) * d)).to(dt)  # one projection's rows: q heads, k heads, v heads
    s = dict(q=qkv[:, :hq * d], k=qkv[:, hq * d:(hq + hkv) * d], v=qkv[:, (hq + hkv) * d:])
    s["wq"], s["wk"] = ((1 + 0.1 * _randn(g, d)).to(dt) for _ in range(2)) if c["norm"] else (None, None)
    rot = c["rot"]
    s["freq"] = (1e-6 ** (torch.arange(rot // 2, device="cuda", dtype=torch.float64) * 2 / max(rot, 1))).float()
    s["pos"] = torch.randint(0, max(1, c["far"]), (n,), generator=g, device="cuda", dtype=torch.int32)
    s["dst"], out = None, n
    if c["ragged"]:  # rows of a padded batch in another order, a few without a place
        out = n + n // 4 + 1
        s["dst"] = torch.randperm(out, generator=g, device="cuda")[:n].to(torch.int32)
        s["dst"][torch.rand(n, generator=g, device="cuda") < 0.03] = -1
    s["out"] = [torch.zeros(out, h, d, dtype=dt, device="cuda") for h in (hq, hkv, hkv)]
    if own:
        from rotated_bit_kv_kvq_gb300 import kvq
        e = torch.zeros(64, dtype=torch.uint8, device="cuda")
        s["keep"] = e
        s["handle"] = kvq.descriptor(1, hkv, d, 64, 0, "q4_0", "q4_0")
        for field in ("k_qs", "k_d", "v_qs", "v_d", "seq_len", "status"):
            setattr(s["handle"], field, e.data_ptr())
        s["plan"] = kvq.RopeNorm(s["freq"], q_weight=s["wq"], k_weight=s["wk"], eps=1e-6, interleaved=c["inter"])
    return s


def _prepare_pages(c, g):
    B, per = c["batch"], c["ctx"] // c["page"]
    lens, new = _lengths(c), _new_tokens(c)
    held = [_blocks(n, c["page"]) for n in lens]
    need = sum(_blocks(n + r, c["page"]) - h for n, r, h in zip(lens, new, held) if r >= 0)
    pages = sum(held) + need + 5
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    h = _dev(held, torch.int64)
    start = torch.cumsum(h, 0) - h
    at = torch.arange(per, device="cuda")[None, :]
    table = torch.where(at < h[:, None], order[(start[:, None] + at).clamp(max=pages - 1)], -1).to(torch.int32)
    used = sum(held)
    head = int(torch.randint(0, pages, (1,), generator=g, device="cuda"))
    ring = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    ring[(head + torch.arange(pages - used, device="cuda")) % pages] = order[used:]
    rows = sum(r for r in new if r > 0) + 3  # room for a few more rows than there are
    i32 = lambda *n: torch.empty(*n, dtype=torch.int32, device="cuda")  # noqa: E731
    s = dict(seq=_dev(lens), new=_dev(new), widest=max(max(new), 1), table=table, ring=ring,
             state=_dev([head, pages - used]), next=i32(2), after=i32(B), granted=i32(B), pos=i32(rows), dst=i32(rows),
             slot=i32(rows), rows=rows, pages=pages)
    if own:
        from rotated_bit_kv_kvq_gb300 import kvq
        e = torch.zeros(64, dtype=torch.uint8, device="cuda")
        s["keep"] = e
        case = dict(batch=B, hkv=1, d=64, ctx=c["ctx"], page=c["page"], n_pages=pages)
        s["handle"] = _handle(case, dict(kq=e, ks=e, vq=e, vs=e, status=e, seq=s["seq"], table=table))
        s["plan"] = kvq.kvq_page_pool(ring.data_ptr(), s["state"].data_ptr(), s["next"].data_ptr())
    return s


def prepare(case, seed):
    c, g = case, _gen(seed)
    if c["op"] in ("rope", "pages"):
        s = (_prepare_rope if c["op"] == "rope" else _prepare_pages)(c, g)
        return dict(s, case=c)
    B, H, d = c["batch"], c["hkv"], c["d"]
    s = _cache(c, g, {"index": "k", "select": "", "sparse": "kv"}[c["op"]])
    nblk = _blocks(c["ctx"], c["bt"])
    lens = s["seq"].long()
    have = (lens + c["bt"] - 1) // c["bt"]
    if c["op"] == "index":
        s["codes"] = torch.zeros(B, H, nblk, d, dtype=torch.int8, device="cuda")
        s["scales"] = torch.zeros(B, H, nblk, dtype=torch.float32, device="cuda")
    else:
        s["q"] = _randn(g, B, c["hq"], d).to(DTYPES[c["dt"]])
    if c["op"] == "select":
        s["codes"] = (40 * _randn(g, B, H, nblk, d)).round().clamp(-127, 127).to(torch.int8)
        s["scales"] = 0.002 * (1 + torch.rand(B, H, nblk, generator=g, device="cuda"))
        s["sel"] = torch.empty(B, H, c["nsel"], dtype=torch.int32, device="cuda")
    if c["op"] == "sparse":  # the first, the last and random blocks, in order, -1 behind them
        like = torch.rand(B, H, nblk, generator=g, device="cuda")
        at = torch.arange(nblk, device="cuda")
        like = torch.where(at < have[:, None, None], like, -1.0)
        like = torch.where((at == 0) | (at == (have - 1)[:, None, None]), like + 2, like)
        top = like.topk(min(c["nsel"], nblk), -1)
        sel = torch.where(top.values >= 0, top.indices, nblk).sort(-1).values
        sel = torch.where(sel < have[:, None, None], sel, -1)
        s["sel"] = torch.nn.functional.pad(sel, (0, c["nsel"] - sel.shape[-1]), value=-1).to(torch.int32)
        s["out"] = torch.empty(B, c["hq"], d, dtype=DTYPES[c["dt"]], device="cuda")
    if c["op"] == "sparse":
        s["had"] = torch.from_numpy(_hadamard(d)).float().cuda()
    if own:
        from rotated_bit_kv_kvq_gb300 import kvq
        s["handle"] = _handle(c, s)
        if c["op"] != "sparse":
            s["plan"] = kvq.kvq_block_index(c["bt"], s["codes"].data_ptr(), s["scales"].data_ptr())
    return dict(s, case=c)


# ---- the plain forms -----------------------------------------------------------------------

def _plain_rope(c, s):
    n, d, rot = c["rows"], c["d"], c["rot"]
    angle = s["pos"].double()[:, None] * s["freq"].double()  # [n][rot / 2]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def norm(x, w):
        x = x.reshape(n, -1, d).float()
        return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()

    def turn(x):
        if not rot:
            return x
        a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if c["inter"] else (x[..., :rot // 2], x[..., rot // 2:rot])
        y = (a * cos - b * sin, a * sin + b * cos)
        y = torch.stack(y, -1).flatten(-2) if c["inter"] else torch.cat(y, -1)
        return torch.cat([y, x[..., rot:]], -1)

    def put(x, out):
        x = x.to(out.dtype)
        if s["dst"] is None:
            return x
        full = torch.zeros(out.shape[0] + 1, *out.shape[1:], dtype=out.dtype, device="cuda")
        full[torch.where(s["dst"] < 0, out.shape[0], s["dst"]).long()] = x
        return full[:-1]

    q, k, v = s["out"]
    return {"q": put(turn(norm(s["q"], s["wq"])), q), "k": put(turn(norm(s["k"], s["wk"])), k),
            "v": put(s["v"].reshape(n, -1, d), v)}


def _plain_pages(c, s):
    P, B, per = c["page"], c["batch"], c["ctx"] // c["page"]
    n, r, pages = s["seq"].long(), s["new"].long(), s["pages"]
    head, count = s["state"].long().unbind()
    free = r == -1
    fits = (r >= 0) & (r <= s["widest"]) & (n + r <= c["ctx"])
    r = torch.where(fits, r, 0)
    held, need = (n + P - 1) // P, (n + r + P - 1) // P - (n + P - 1) // P
    row1, new1 = torch.cumsum(r, 0), torch.cumsum(need, 0)
    ok = ((need == 0) | (new1 <= count)) & ((r == 0) | (row1 <= s["rows"]))
    popped = (need * ok).sum()
    gone = torch.where(free, held, 0)
    gone1 = torch.cumsum(gone, 0)
    at = torch.arange(per, device="cuda")[None, :]
    new0, gone0, row0 = (new1 - need)[:, None], (gone1 - gone)[:, None], row1 - r
    mine = ok[:, None] & (at >= held[:, None]) & (at < (held + need)[:, None])
    from_ring = s["ring"][(head + torch.where(mine, new0 + at - held[:, None], 0)) % pages]
    table = torch.where(mine, from_ring, s["table"])
    back = free[:, None] & (at < held[:, None])
    ring = torch.cat([s["ring"], s["ring"][:1]])
    ring = ring.index_put((torch.where(back, (head + count + gone0 + at) % pages, pages),), s["table"])[:-1]
    i = torch.arange(s["rows"], device="cuda")
    b = torch.searchsorted(row1, i, right=True)
    real = b < B
    b = b.clamp(max=B - 1)
    j = i - row0[b]
    pos = torch.where(real, n[b] + j, 0)
    real = real & ok[b]
    slot = table[b, (pos // P).clamp(max=per - 1)].long() * P + pos % P
    i32 = torch.int32
    return {"granted": torch.where(ok, r, 0).to(i32), "table": table, "ring": ring,
            "state": torch.stack([(head + popped) % pages, count - popped + gone1[-1]]).to(i32),
            "after": torch.where(free, 0, n).to(i32), "pos": pos.to(i32),
            "dst": torch.where(real, b * s["widest"] + j, -1).to(i32), "slot": torch.where(real, slot, -1).to(i32)}


def _values(s, side, kind, rows, d):
    """The dequantized rows [...][d] of a plane."""
    nb = d // 32
    qs, head = s[side + "q"][rows], s[side + "s"][rows].float()
    if kind == "q8_0":
        return ((qs.float() - 128).unflatten(-1, (nb, 32)) * head[..., None]).flatten(-2)
    qs = qs.unflatten(-1, (nb, 16))
    code = torch.cat([qs & 15, qs >> 4], -1).int()
    if kind[1] == "5" and side == "k":
        code += ((s["kh"][rows][..., None] >> _k_bits()) & 1) << 4
    elif kind[1] == "5":
        part, bit = _v_bits()
        word = ((rows // 2)[..., None, None] * nb + torch.arange(nb, device="cuda")[:, None]) * 2 + part
        half = s["vh"].flatten()[word * 2 + (rows % 2)[..., None, None]]
        code += ((half.int() >> bit) & 1) << 4
    if kind.endswith("_1"):
        return (code.float() * head[..., :1] + head[..., 1:]).flatten(-2)
    return ((code - (16 if kind[1] == "5" else 8)).float() * head[..., None]).flatten(-2)


def _rows(c, s, pos):
    """Plane rows of positions pos [B][H][...]."""
    B, H, P = c["batch"], c["hkv"], c.get("page", 0)
    one = (1,) * (pos.dim() - 2)
    b = torch.arange(B, device="cuda").view(B, 1, *one)
    h = torch.arange(H, device="cuda").view(1, H, *one)
    if not P:
        return (b * H + h) * c["ctx"] + pos
    return (s["table"].long().view(B, -1)[b, pos // P] * H + h) * P + pos % P


def _plain_index(c, s):
    B, H, d, bt, n = c["batch"], c["hkv"], c["d"], c["bt"], s["seq"].long()
    nblk = s["codes"].shape[2]
    count = nblk if c["last"] == 0 else min(nblk, (c["last"] + bt - 2) // bt + 1)
    first = torch.zeros_like(n) if c["last"] == 0 else (n - c["last"]).clamp(min=0) // bt
    blk = first[:, None] + torch.arange(count, device="cuda")  # [B][count]; past the end only where nothing is left
    live = (blk < nblk) & (blk * bt < n[:, None])
    blk = blk % nblk
    pos = (blk[..., None] * bt + torch.arange(bt, device="cuda"))[:, None].expand(B, H, count, bt)
    seen = (pos < n[:, None, None, None])[..., None]
    x = _values(s, "k", c["kt"], _rows(c, s, pos.clamp(max=c["ctx"] - 1)), d)
    x = torch.where(seen, x, 0).view(B, H, count, bt // 8, 8, d)
    acc = x[..., 0, :, :]
    for i in range(1, bt // 8):  # the order of the sums is the definition's
        acc = acc + x[..., i, :, :]
    acc = acc[..., 0::2, :] + acc[..., 1::2, :]
    acc = acc[..., 0::2, :] + acc[..., 1::2, :]
    acc = acc[..., 0, :] + acc[..., 1, :]
    mean = acc / seen.float().sum(-2).clamp(min=1)
    scale = mean.abs().amax(-1) / torch.full((), 127.0, device="cuda")  # a tensor: a true division
    code = torch.where(scale[..., None] > 0, torch.round(mean / scale[..., None]), 0).to(torch.int8)
    b, h = torch.arange(B, device="cuda").view(B, 1, 1), torch.arange(H, device="cuda").view(1, H, 1)
    at = (b.expand(B, H, count), h.expand(B, H, count), blk[:, None].expand(B, H, count))
    keep = live[:, None].expand(B, H, count)
    return {"codes": s["codes"].index_put(at, torch.where(keep[..., None], code, s["codes"][at])),
            "scales": s["scales"].index_put(at, torch.where(keep, scale, s["scales"][at]))}


def _plain_select(c, s):
    B, H, d, nsel, bt = c["batch"], c["hkv"], c["d"], c["nsel"], c["bt"]
    G, nblk = c["hq"] // c["hkv"], s["codes"].shape[2]
    x, g = s["q"].float().view(B, H, G, d), _group(d)
    step = 1
    while step < g:  # sums and differences of channels that are `step` apart, in this order
        y = x.reshape(B, H, G, d // (2 * step), 2, step)
        x = torch.stack([y[..., 0, :] + y[..., 1, :], y[..., 0, :] - y[..., 1, :]], -2).reshape(B, H, G, d)
        step *= 2
    x = x * (1 / math.sqrt(g))
    qs = x.abs().amax(-1) / torch.full((), 127.0, device="cuda")
    code = torch.where(qs[..., None] > 0, torch.round(x / qs[..., None]), 0)
    dots = code @ s["codes"].float().transpose(-1, -2)  # whole numbers below 2^24: exact in any order
    score = ((dots * qs[..., None]) * s["scales"][:, :, None]).amax(2)  # [B][H][nblk]
    have = ((s["seq"].long() + bt - 1) // bt)[:, None, None]
    at = torch.arange(nblk, device="cuda")
    score = torch.where((at == 0) | (at == have - 1), math.inf, score)
    score = torch.where(at < have, score, -math.inf)
    order = score.sort(dim=-1, descending=True, stable=True).indices[..., :nsel]
    order = torch.where(order < have, order, nblk).sort(-1).values
    order = torch.where(order < nblk, order, -1)
    return {"sel": torch.nn.functional.pad(order, (0, nsel - order.shape[-1]), value=-1).to(torch.int32)}


def _plain_sparse(c, s):
    B, H, d, bt, T, n = c["batch"], c["hkv"], c["d"], c["bt"], c["tail"], s["seq"].long()
    sel = s["sel"].long()
    pos = (sel[..., None] * bt + torch.arange(bt, device="cuda")).flatten(-2)  # [B][H][tokens]
    end = n[:, None, None]
    seen = (pos >= 0) & (pos < end)
    pos = torch.where(seen, pos, 0)
    rows = _rows(c, s, pos)

    def read(side):
        x = _values(s, side, c[side + "t"], rows, d)
        if T:
            b, h = torch.arange(B, device="cuda").view(B, 1, 1), torch.arange(H, device="cuda").view(1, H, 1)
            x = torch.where((pos >= end - T)[..., None], s[side + "tail"][b, h, pos % T].float(), x)
        return torch.where(seen[..., None], x, 0)

    q = s["q"].float().view(B, H, -1, d) @ s["had"]
    score = (q @ read("k").transpose(-1, -2)) * (1 / math.sqrt(d))
    score = torch.where(seen[:, :, None], score, -math.inf)
    top = score.amax(-1, keepdim=True).clamp(min=-3e38)
    p = (score - top).exp()
    out = (p @ read("v")) / p.sum(-1, keepdim=True).clamp(min=1e-30)
    return {"out": (out @ s["had"]).view(B, -1, d).to(s["q"].dtype)}


# ---- one pass -------------------------------------------------------------------------------

def _own(c, s):
    from rotated_bit_kv_kvq_gb300 import kvq
    if c["op"] == "rope":
        q, k, v = s["out"]
        kvq.kvq_qk_norm_rope(s["handle"], s["plan"], s["q"], s["k"], s["v"], s["pos"], q, k, v, dst_row=s["dst"])
        return {"q": q, "k": k, "v": v}
    if c["op"] == "pages":
        kvq.kvq_page_update(s["handle"], s["plan"], s["new"], s["widest"], s["granted"], row_pos=s["pos"],
                            row_dst=s["dst"], row_slot=s["slot"], seq_len_out=s["after"])
        return {"granted": s["granted"], "table": s["table"], "ring": s["ring"], "state": s["next"], "after": s["after"],
                "pos": s["pos"], "dst": s["dst"], "slot": s["slot"]}
    if c["op"] == "index":
        kvq.kvq_block_index_update(s["handle"], s["plan"], n_last=c["last"])
        return {"codes": s["codes"], "scales": s["scales"]}
    if c["op"] == "select":
        kvq.kvq_select_blocks(s["handle"], s["plan"], s["q"], s["sel"], n_first=1, n_last=1)
        return {"sel": s["sel"]}
    kvq.kvq_sparse_decode_attention(s["handle"], s["q"], s["sel"], s["out"], block_tokens=c["bt"])
    return {"out": s["out"]}


def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    return {"rope": _plain_rope, "pages": _plain_pages, "index": _plain_index, "select": _plain_select,
            "sparse": _plain_sparse}[c["op"]](c, state)


# ---- the definitions in 64 bits ----------------------------------------------------------------

def _host(t):
    return None if t is None else (t.float() if t.dtype in (torch.bfloat16, torch.float16) else t).cpu().numpy()


def _exact_rope(c, s):
    n, d, rot = c["rows"], c["d"], c["rot"]
    pos, freq = _host(s["pos"]).astype(np.float64), _host(s["freq"]).astype(np.float64)
    z = np.exp(1j * np.outer(pos, freq))[:, None]  # the pairs as complex numbers
    dst = None if s["dst"] is None else _host(s["dst"])

    def one(x, w, rotated, out):
        x = _host(x).reshape(n, -1, d).astype(np.float64)
        if w is not None:
            x = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + 1e-6) * _host(w).astype(np.float64)
        if rotated and rot:
            y = x.copy()
            first = slice(0, rot, 2) if c["inter"] else slice(0, rot // 2)
            second = slice(1, rot, 2) if c["inter"] else slice(rot // 2, rot)
            t = (x[..., first] + 1j * x[..., second]) * z
            y[..., first], y[..., second] = t.real, t.imag
            x = y
        if dst is None:
            return x
        full = np.zeros((out.shape[0],) + x.shape[1:])
        full[dst[dst >= 0]] = x[dst >= 0]
        return full

    q, k, v = s["out"]
    return {"q": one(s["q"], s["wq"], True, q), "k": one(s["k"], s["wk"], True, k), "v": one(s["v"], None, False, v)}


class _Plane:
    """One side of a cache on the host: rows of values in 64 bits, decoded channel by channel."""

    def __init__(self, s, side, kind, d):
        self.kind, self.d, self.v = kind, d, side == "v"
        self.qs, self.hd = _host(s[side + "q"]), _host(s[side + "s"])
        self.hi = None if s[side + "h"] is None else _host(s[side + "h"])

    def rows(self, r):
        kind, nb = self.kind, self.d // 32
        qs, hd = self.qs[r].reshape(len(r), nb, -1), self.hd[r].reshape(len(r), nb, -1).astype(np.float64)
        out = np.empty((len(r), nb, 32))
        for ch in range(32):
            if kind == "q8_0":
                code = qs[..., ch].astype(np.int64) - 128
            else:
                code = (qs[..., ch % 16].astype(np.int64) >> (4 if ch >= 16 else 0)) & 15
                b = [(ch >> i) & 1 for i in range(5)]
                if kind[1] == "5" and not self.v:
                    code = code + 16 * ((self.hi[r].astype(np.int64) >> (16 * b[1] + 8 * b[3] + 4 * b[4] + 2 * b[2] + b[0])) & 1)
                elif kind[1] == "5":
                    half = self.hi[r // 2, :, b[3], r % 2].astype(np.int64)
                    code = code + 16 * ((half >> (8 * b[2] + 4 * b[4] + 2 * b[1] + b[0])) & 1)
                if not kind.endswith("_1"):
                    code = code - (16 if kind[1] == "5" else 8)
            out[..., ch] = code * hd[..., 0] + (hd[..., 1] if kind.endswith("_1") else 0.0)
        return out.reshape(len(r), self.d)


def _exact_row(c, table, b, h, pos):
    P = c.get("page", 0)
    if not P:
        return (b * c["hkv"] + h) * c["ctx"] + pos
    return (table[b * (c["ctx"] // P) + pos // P].astype(np.int64) * c["hkv"] + h) * P + pos % P


def _exact_index(c, s):
    scales = _host(s["scales"]).astype(np.float64)
    plane, table = _Plane(s, "k", c["kt"], c["d"]), _host(s.get("table"))
    for b, n in enumerate(_lengths(c)):
        for j in range(0 if c["last"] == 0 else max(0, n - c["last"]) // c["bt"], _blocks(n, c["bt"])):
            pos = np.arange(j * c["bt"], min(n, (j + 1) * c["bt"]))
            for h in range(c["hkv"]):
                scales[b, h, j] = np.abs(plane.rows(_exact_row(c, table, b, h, pos)).mean(0)).max() / 127
    return {"codes": None, "scales": scales}


def _exact_sparse(c, s):
    B, H, d, bt, T = c["batch"], c["hkv"], c["d"], c["bt"], c["tail"]
    G = c["hq"] // H
    k, v = _Plane(s, "k", c["kt"], d), _Plane(s, "v", c["vt"], d)
    table, sel, q, had = _host(s.get("table")), _host(s["sel"]), _host(s["q"]).astype(np.float64), _hadamard(d)
    tails = [_host(s[x]) if T else None for x in ("ktail", "vtail")]
    out = np.zeros((B, H * G, d))
    for b, n in enumerate(_lengths(c)):
        for h in range(H):
            pos = np.concatenate([np.arange(j * bt, min(n, (j + 1) * bt)) for j in sel[b, h] if j >= 0] or [np.arange(0)])
            if not len(pos):
                continue
            r = _exact_row(c, table, b, h, pos)
            keys, vals = k.rows(r), v.rows(r)
            if T:
                late = pos >= n - T
                keys[late], vals[late] = (t[b, h, pos[late] % T] for t in tails)
            a = (q[b, h * G:(h + 1) * G] @ had) @ keys.T / math.sqrt(d)
            a = np.exp(a - a.max(-1, keepdims=True))
            out[b, h * G:(h + 1) * G] = (a / a.sum(-1, keepdims=True)) @ vals @ had
    return {"out": out}


def exact(case, seed):
    """In 64 bits; None where the outputs are whole numbers, or where it would take too long on the host."""
    if case["op"] in ("pages", "select") or work(case)["flops"] > 3e10 or (case["op"] == "index" and work(case)["bytes"] > 6e7):
        return None
    s = prepare(case, seed)
    return {"rope": _exact_rope, "index": _exact_index, "sparse": _exact_sparse}[case["op"]](case, s)
