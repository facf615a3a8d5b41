"""Workloads of the operators for shared and continued sequences, in two forms each.

Chunk attention (``attn``): packed rows of new tokens, a different number for every sequence, over the quantized cache and
its bf16 tail; the scores capped, biased by distance, or masked by documents and prefixes.  Page operators of the paged
cache: ``fork`` (a sequence begins with the tokens of another: pages shared, the last one copied), ``free`` (sequences give
their pages back) and ``compact`` (the live pages move to the lowest places).  ``run`` computes them with elementary torch
operations, or, where ``own`` is true, by the calls a user makes.
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
        # the smallest: a decode step of one short sequence, one head, no tail
        _attn("attn_one_token", batch=1, hq=1, hkv=1, d=64, ctx=1024, kt="q4_0", vt="q4_0", lo=1000, hi=1000, new=1, dt="f16"),
        # one token each of the ragged batch, scores capped
        _attn("attn_step_b32", batch=32, hq=32, hkv=8, d=128, ctx=8192, kt="q5_0", vt="q5_0", tail=512, lo=1024, hi=8192, new=1,
              cap=50.0, page=64),
        # guesses of five tokens each, to be verified in one pass
        _attn("attn_guess_b32", batch=32, hq=32, hkv=8, d=128, ctx=8192, kt="q8_0", vt="q4_0", tail=512, lo=1024, hi=8192, new=5,
              page=64),
        # a serving batch: prompt chunks beside single tokens and sequences that rest, documents packed in each
        _attn("attn_mixed_b16", batch=16, hq=32, hkv=8, d=128, ctx=8192, kt="q8_0", vt="q8_0", tail=128, lo=700, hi=8000, new=511,
              mix=True, docs=1500, page=128, dt="f16"),
        # the next 512 tokens of a 64k context, with a bias by distance
        _attn("attn_chunk_64k", batch=1, hq=24, hkv=4, d=256, ctx=65536, kt="q8_0", vt="q4_0", tail=1024, lo=65536, hi=65536,
              new=512, alibi=True, page=256),
        # two prompts of 4096 tokens that see their first half in both directions
        _attn("attn_prompt_2x4k", batch=2, hq=32, hkv=8, d=128, ctx=4096, kt="q4_0", vt="q4_0", lo=4096, hi=4096, new=4096,
              prefix=0.5),
        # a prompt becomes two sequences
        _fork("fork_one", batch=4, hkv=2, d=64, ctx=2048, kt="q4_0", vt="q4_0", tail=0, page=64, forks=1, lo=900, hi=1500),
        # eight prompts, eight samples of each
        _fork("fork_8x8", batch=72, hkv=8, d=128, ctx=8192, kt="q5_0", vt="q5_0", tail=512, page=64, forks=64, lo=1024, hi=8000),
        # a few sequences end
        _free("free_b32", batch=32, ctx=8192, page=64, lo=1024, hi=8000, every=4),
        # a search over 512 sequences drops half of them; prompts are shared by eight
        _free("free_b512", batch=512, ctx=16384, page=64, lo=2000, hi=16000, every=2),
        # a small pool with a few holes
        _compact("compact_small", batch=4, hkv=2, d=64, ctx=1024, kt="q4_0", vt="q4_0", page=64, pages=48, lo=200, hi=900),
        # a pool of half a gigabyte, half of it in use
        _compact("compact_half", batch=16, hkv=8, d=128, ctx=16384, kt="q8_0", vt="q5_0", page=64, pages=4096, lo=4000, hi=12000),
    ]


def _attn(name=None, **kw):
    return _case(name, dict(op="attn", tail=0, page=0, mix=False, cap=0.0, alibi=False, docs=0, prefix=0.0, dt="bf16"), kw)


def _fork(name=None, **kw):
    return _case(name, dict(op="fork", dt="bf16"), kw)


def _free(name=None, **kw):
    return _case(name, dict(op="free"), kw)


def _compact(name=None, **kw):
    return _case(name, dict(op="compact", tail=0), kw)


def _case(name, base, kw):
    return {**({} if name is None else {"name": name}), **base, **kw}


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "attn", "fork", "free", "compact"])
    d = rng.choice([64, 128, 192, 256, 320])
    hkv = rng.choice([1, 2, 3, 4, 8])
    kt, vt = rng.choice(TYPES), rng.choice(TYPES)
    page = rng.choice([64, 128, 256])
    batch = _spread(rng, 1, 32)
    if op == "attn":
        ctx = 256 * _spread(rng, 1, max(2, min(256, 300_000_000 // (256 * batch * hkv * d))))
        hq = hkv * rng.choice([1, 2, 3, 4, 5, 8, 12])
        new = _spread(rng, 1, max(1, min(ctx, 4096, int(3.5e11 / (4.0 * batch * hq * d * ctx)))))
        return _attn(batch=batch, hq=hq, hkv=hkv, d=d, ctx=ctx, kt=kt, vt=vt, tail=rng.choice([0, 30, 128, 512]),
                     page=rng.choice([0, page]), lo=rng.choice([0, ctx // 2]), hi=ctx, new=new, mix=rng.random() < 0.5,
                     cap=rng.choice([0.0, 0.0, 5.0, 30.0]), alibi=rng.random() < 0.3,
                     docs=rng.choice([0, 0, _spread(rng, 40, 3000)]), prefix=rng.choice([0.0, 0.0, 0.3, 0.9]),
                     dt=rng.choice(["bf16", "f16"]))
    if op == "free":
        ctx = page * rng.randint(2, 200)
        return _free(batch=_spread(rng, 1, 512), ctx=ctx, page=page, lo=0, hi=ctx, every=rng.choice([1, 2, 3, 16]))
    ctx = page * _spread(rng, 1, 64)
    if op == "fork":
        forks = _spread(rng, 1, 48)
        return _fork(batch=forks + rng.randint(1, 8), hkv=hkv, d=d, ctx=ctx, kt=kt, vt=vt, tail=rng.choice([0, 30, 128, 512]),
                     page=page, forks=forks, lo=0, hi=ctx)
    ctx *= 2
    held = max(1, min(batch, 300_000_000 // (ctx * hkv * d * 2)))
    return _compact(batch=held, hkv=hkv, d=d, ctx=ctx, kt=kt, vt=vt, page=page, pages=held * (ctx // page) + rng.randint(0, 100),
                    lo=0, hi=ctx)


def _golden(i):
    """The i-th of numbers spread over [0, 1)."""
    return ((i + 1) * 0.6180339887498949) % 1.0


def _lengths(c):
    """Tokens of each sequence: spread over [lo, hi], the same for every seed."""
    return [int(round(c["lo"] + (c["hi"] - c["lo"]) * _golden(i))) for i in range(c["batch"])]


def _blocks(tokens, size):
    return -(-tokens // size)


def _new_tokens(c):
    """Per sequence: the new tokens whose rows are in the chunk (mixed: prompt chunks, single tokens, none)."""
    got = []
    for i, n in enumerate(_lengths(c)):
        m = c["new"] if not c["mix"] else (c["new"], 1, max(1, c["new"] // 3), 0, 1)[i % 5]
        got.append(min(m, n))
    return got


def _visible(c):
    """Per sequence: (first, last + 1) of the keys that each of its rows sees, as integer arrays."""
    got = []
    for n, m in zip(_lengths(c), _new_tokens(c)):
        p = np.arange(n - m, n)
        end = np.minimum(n, np.maximum(p + 1, int(c["prefix"] * n)))
        got.append((p // c["docs"] * c["docs"] if c["docs"] else np.zeros_like(p), end))
    return got


def _forks(c):
    """(source, destination, tokens) of each fork: every third one takes a shorter beginning; the last sequences are empty."""
    n, srcs = _lengths(c), c["batch"] - c["forks"]
    return [(i % srcs, srcs + i, n[i % srcs] if i % 3 else n[i % srcs] * 7 // 8) for i in range(c["forks"])]


# ---- the work that no implementation does without ------------------------------------------

def _row_bytes(kind, d):
    return (d // 32) * {"q4_0": 18, "q5_0": 22, "q8_0": 34, "q4_1": 20, "q5_1": 24}[kind]


def _page_bytes(c):
    return c["hkv"] * c["page"] * (_row_bytes(c["kt"], c["d"]) + _row_bytes(c["vt"], c["d"]))


def work(case):
    c = case
    if c["op"] == "attn":
        pairs = body = tail = 0
        for n, (lo, hi) in zip(_lengths(c), _visible(c)):
            pairs += int((hi - lo).sum())
            if len(lo):
                a, b, cut = int(lo.min()), int(hi.max()), max(0, n - c["tail"])
                body += max(0, min(b, cut) - a)
                tail += max(0, b - max(a, cut))
        rows = sum(_new_tokens(c))
        per = _row_bytes(c["kt"], c["d"]) + _row_bytes(c["vt"], c["d"])
        return {"bytes": c["hkv"] * (body * per + tail * 4 * c["d"]) + rows * 4 * c["hq"] * c["d"] + 8 * c["batch"],
                "flops": 4 * c["hq"] * c["d"] * pairs}
    lens = _lengths(c)
    if c["op"] == "fork":
        entries = sum(n // c["page"] for _, _, n in _forks(c))
        copied = sum(n % c["page"] > 0 for _, _, n in _forks(c)) * _page_bytes(c)
        tails = sum(min(n, c["tail"]) for _, _, n in _forks(c)) * c["hkv"] * c["d"] * 4
        read = sum(min(lens[s], c["tail"]) for s in range(min(c["batch"] - c["forks"], c["forks"]))) * c["hkv"] * c["d"] * 4
        return {"bytes": entries * 12 + 2 * copied + tails + read + 20 * c["forks"], "flops": entries}
    if c["op"] == "free":
        gone = sum(_blocks(n, c["page"]) for i, n in enumerate(lens) if i % c["every"] == 0)
        return {"bytes": gone * 12 + 12 * c["batch"], "flops": gone}
    used = sum(_blocks(n, c["page"]) for n in lens)
    moved = used * (c["pages"] - used) // c["pages"]  # of randomly placed pages
    return {"bytes": 2 * moved * _page_bytes(c) + 8 * used + 16 * c["pages"], "flops": c["pages"]}


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


def _random_planes(g, n, d, kind):
    """Planes of n rows with random codes and scales (what page operators move is not looked at)."""
    nb = d // 32
    qs = torch.randint(0, 256, (n, d if kind == "q8_0" else d // 2), generator=g, device="cuda", dtype=torch.uint8)
    high = torch.randint(-2 ** 31, 2 ** 31, (n, nb), generator=g, device="cuda").to(torch.int32) if kind[1] == "5" else None
    return qs, high, (0.05 * _randn(g, n, nb * (2 if kind.endswith("_1") else 1))).half()


def _group(d):
    return (d if d & (d - 1) == 0 else 64) if d >= 64 and d % 64 == 0 else 32


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


def _cache(c, g):
    """The planes of a cache whose rotated keys and values are drawn from g."""
    B, H, C, d, T, page = c["batch"], c["hkv"], c["ctx"], c["d"], c["tail"], c["page"]
    s = dict(seq=_dev(_lengths(c)), status=torch.zeros(4, dtype=torch.int32, device="cuda"))
    if page:
        s["table"] = torch.randperm(B * (C // page), generator=g, device="cuda").to(torch.int32).view(B, C // page)
    for side in "kv":
        # keys of a block share a direction, as neighbouring tokens do; values do not
        y = _randn(g, B, H, C, d)
        if side == "k":
            y += 0.5 * _randn(g, B, H, C // 64, 1, d).expand(B, H, C // 64, 64, d).reshape(B, H, C, d)
        if T:
            s[side + "tail"] = _tail_of(y, s["seq"].long(), T)
        if page:
            pool = torch.empty_like(y).view(B * (C // page), H, page, d)
            pool[s["table"].flatten().long()] = y.view(B, H, C // page, page, d).transpose(1, 2).reshape(-1, H, page, d)
            y = pool
        planes = [_quantized(part, c[side + "t"], side == "v") for part in y.reshape(-1, d).split(1 << 20)]
        del y
        for k, name in enumerate("qhs"):
            s[side + name] = None if planes[0][k] is None else torch.cat([p[k] for p in planes])
        del planes
    return s


def _tail_of(y, n, T):
    """bf16 rows [B][H][T][d] of the last T positions of y [B][H][C][d]."""
    B, H, _, d = y.shape
    b = torch.arange(B, device="cuda")[:, None]
    p = n[:, None] - 1 - torch.arange(T, device="cuda")
    ok = p >= 0
    rows = y[b, :, p.clamp(min=0)].to(torch.bfloat16)  # [B][T][H][d]
    tail = torch.zeros(B, T, H, d, dtype=torch.bfloat16, device="cuda")
    slot = torch.where(ok, p % T, 0)
    tail[b.expand(B, T)[ok], slot[ok]] = rows[ok]
    return tail.transpose(1, 2).contiguous()


def _handle(c, s):
    """The framework's descriptor of those planes."""
    from rotated_bit_kv_kvq_gb300 import kvq
    page = c["page"]
    h = kvq.descriptor(c["batch"], c["hkv"], c["d"], c["ctx"], c["tail"], c["kt"], c["vt"], page_tokens=page,
                       n_pages=s["table"].numel() if page and "pages" not in s else s.get("pages", 0))
    for field, name in (("k_qs", "kq"), ("k_qh", "kh"), ("k_d", "ks"), ("v_qs", "vq"), ("v_qh", "vh"), ("v_d", "vs"),
                        ("k_tail", "ktail"), ("v_tail", "vtail"), ("seq_len", "seq"), ("status", "status"),
                        ("page_table", "table")):
        if s.get(name) is not None:
            setattr(h, field, s[name].data_ptr())
    return h


def _prepare_attn(c, g):
    s = _cache(c, g)
    new, lens, seen = _new_tokens(c), _lengths(c), _visible(c)
    rows = sum(new)
    s["start"] = _dev([0] + list(np.cumsum(new)))
    s["first"] = _dev(np.concatenate([a for a, _ in seen]).tolist()) if c["docs"] else None
    s["prefix"] = _dev([int(c["prefix"] * n) for n in lens]) if c["prefix"] else None
    s["slopes"] = 2.0 ** (-8.0 * (torch.arange(c["hq"], device="cuda", dtype=torch.float32) + 1) / c["hq"]) if c["alibi"] else None
    s["q"] = _randn(g, rows, c["hq"], c["d"]).to(DTYPES[c["dt"]])
    s["out"] = torch.zeros(rows, c["hq"], c["d"], dtype=DTYPES[c["dt"]], device="cuda")
    s["had"] = torch.from_numpy(_hadamard(c["d"])).float().cuda()
    if own:
        from rotated_bit_kv_kvq_gb300 import kvq
        s["handle"] = _handle(c, s)
        s["mod"] = kvq.ScoreMod(softcap=c["cap"], slopes=s["slopes"], first_key=s["first"], prefix_len=s["prefix"])
        s["work"] = torch.empty(kvq.kvq_chunk_workspace_bytes(s["handle"], c["hq"], rows), dtype=torch.uint8, device="cuda")
    return s


def _placed(c, g, lens, pages):
    """Page table of sequences with these lengths, their pages anywhere in the pool; the free pages in a ring."""
    per = c["ctx"] // c["page"]
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    held = _dev([_blocks(n, c["page"]) for n in lens], torch.int64)
    start = (torch.cumsum(held, 0) - held)[:, None]
    at = torch.arange(per, device="cuda")[None, :]
    table = torch.where(at < held[:, None], order[(start + at).clamp(max=pages - 1)], -1).to(torch.int32)
    used = sum(_blocks(n, c["page"]) for n in lens)
    head = int(torch.randint(0, pages, (1,), generator=g, device="cuda"))
    ring = torch.full((pages,), -1, dtype=torch.int32, device="cuda")
    ring[(head + torch.arange(pages - used, device="cuda")) % pages] = order[used:]
    return dict(table=table, ring=ring, state=_dev([head, pages - used]), pages=pages, extra=torch.zeros_like(ring))


def _prepare_pages(c, g):
    B, P = c["batch"], c["page"]
    lens = _lengths(c)
    i32 = lambda *n: torch.zeros(*n, dtype=torch.int32, device="cuda")  # noqa: E731
    if c["op"] == "fork":
        lens = lens[:B - c["forks"]] + [0] * c["forks"]
    if c["op"] == "free":  # the first half of a sequence is that of the first sequence of its eight, where both have it
        s = _placed(c, g, lens, sum(_blocks(n, P) for n in lens) + 7)
        both = [min(n, lens[i // 8 * 8]) // 2 // P if i % 8 else 0 for i, n in enumerate(lens)]
        at = torch.arange(s["table"].shape[1], device="cuda")
        mine = at < _dev(both)[:, None]
        s["table"] = torch.where(mine, s["table"][torch.arange(B, device="cuda") // 8 * 8], s["table"]).contiguous()
        shared = torch.zeros(s["pages"] + 1, dtype=torch.int32, device="cuda")
        shared.index_put_((torch.where(mine, s["table"], s["pages"]).long().flatten(),), _dev(1), accumulate=True)
        s["extra"] = shared[:-1].contiguous()
        s["gone"] = _dev([int(i % c["every"] == 0) for i in range(B)])
    else:
        s = _placed(c, g, lens, c["pages"] if c["op"] == "compact" else sum(_blocks(n, P) for n in lens) + c["forks"] + 5)
        rows = s["pages"] * c["hkv"] * P
        for side in "kv":
            s.update(zip((side + "q", side + "h", side + "s"), _random_planes(g, rows, c["d"], c[side + "t"])))
            if c["tail"]:
                s[side + "tail"] = _randn(g, B, c["hkv"], c["tail"], c["d"]).to(torch.bfloat16)
    if c["op"] == "fork":
        for k, name in enumerate(("src", "dst", "count")):
            s[name] = _dev([f[k] for f in _forks(c)])
        s["granted"] = i32(c["forks"])
    s.update(seq=_dev(lens), after=i32(B), next=i32(2), extra_next=torch.zeros_like(s["extra"]),
             status=torch.zeros(4, dtype=torch.int32, device="cuda"))
    if c["op"] == "compact":
        s.update(table_next=torch.zeros_like(s["table"]), ring_next=torch.zeros_like(s["ring"]), map=i32(s["pages"]))
    if own:
        from rotated_bit_kv_kvq_gb300 import kvq
        if c["op"] == "free":
            e = torch.zeros(64, dtype=torch.uint8, device="cuda")
            s.update(kq=e, ks=e, vq=e, vs=e, keep=e)
            s["handle"] = _handle(dict(c, hkv=1, d=64, tail=0, kt="q4_0", vt="q4_0"), s)
        else:
            s["handle"] = _handle(c, s)
        s["pool"] = kvq.kvq_page_pool(s["ring"].data_ptr(), s["state"].data_ptr(), s["next"].data_ptr())
        s["share"] = kvq.kvq_page_share(s["extra"].data_ptr(), s["extra_next"].data_ptr())
        if c["op"] == "compact":
            s["work"] = torch.empty(kvq.kvq_page_compact_workspace_bytes(s["handle"]), dtype=torch.uint8, device="cuda")
    return s


def prepare(case, seed):
    return dict((_prepare_attn if case["op"] == "attn" else _prepare_pages)(case, _gen(seed)), case=case)


# ---- the plain forms -----------------------------------------------------------------------

def _values(s, side, kind, rows, d):
    """The dequantized rows [...][d] of a plane."""
    nb = d // 32
    qs, head = s[side + "q"][rows], s[side + "s"].view(-1, nb, 2 if kind.endswith("_1") else 1)[rows].float()
    if kind == "q8_0":
        return ((qs.float() - 128).unflatten(-1, (nb, 32)) * head).flatten(-2)
    qs = qs.unflatten(-1, (nb, 16))
    code = torch.cat([qs & 15, qs >> 4], -1).int()
    if kind[1] == "5" and side == "k":
        code += ((s["kh"][rows][..., None] >> _k_bits()) & 1) << 4
    elif kind[1] == "5":
        part, bit = _v_bits()
        word = ((rows // 2)[..., None, None] * nb + torch.arange(nb, device="cuda")[:, None]) * 2 + part
        half = s["vh"].flatten().view(torch.int16)[word * 2 + (rows % 2)[..., None, None]]
        code += ((half.int() >> bit) & 1) << 4
    if kind.endswith("_1"):
        return (code.float() * head[..., :1] + head[..., 1:]).flatten(-2)
    return ((code - (16 if kind[1] == "5" else 8)).float() * head).flatten(-2)


def _rows(c, s, b, pos):
    """Plane rows [hkv][len(pos)] of positions of sequence b."""
    h = torch.arange(c["hkv"], device="cuda")[:, None]
    if not c["page"]:
        return (b * c["hkv"] + h) * c["ctx"] + pos
    return (s["table"][b].long()[pos // c["page"]] * c["hkv"] + h) * c["page"] + pos % c["page"]


def _plain_attn(c, s):
    H, d, T, G = c["hkv"], c["d"], c["tail"], c["hq"] // c["hkv"]
    out, r0 = torch.zeros_like(s["out"]), 0
    for b, (n, m) in enumerate(zip(_lengths(c), _new_tokens(c))):
        if m == 0:
            continue
        r = slice(r0, r0 + m)
        r0 += m
        pos = torch.arange(n, device="cuda")

        def read(side):
            x = _values(s, side, c[side + "t"], _rows(c, s, b, pos), d)
            if T:
                x[:, max(0, n - T):] = s[side + "tail"][b][:, pos[max(0, n - T):] % T].float()
            return x

        q = (s["q"][r].float() @ s["had"]).view(m, H, G, d).permute(1, 2, 0, 3).reshape(H, G * m, d)
        score = (q @ read("k").transpose(-1, -2) * (1 / math.sqrt(d))).view(H, G, m, n)
        if c["cap"]:
            score = c["cap"] * torch.tanh(score / c["cap"])
        at = pos[n - m:, None]
        if c["alibi"]:
            score = score - s["slopes"].view(H, G, 1, 1) * (at - pos).abs()
        seen = pos <= at
        if c["prefix"]:
            seen = seen | (pos < s["prefix"][b])
        if c["docs"]:
            seen = seen & (pos >= s["first"][r, None])
        score = torch.where(seen, score, -math.inf)
        p = (score - score.amax(-1, keepdim=True).clamp(min=-3e38)).exp()
        p = (p / p.sum(-1, keepdim=True).clamp(min=1e-30)).view(H, G * m, n)
        got = (p @ read("v")) @ s["had"]
        out[r] = got.view(H, G, m, d).permute(2, 0, 1, 3).reshape(m, c["hq"], d).to(out.dtype)
    return {"out": out}


def _planes(c, s):
    """The pool's pages as bytes: what is copied is not computed with."""
    return {k: s[k].view(s["pages"], -1).view(torch.uint8) for k in ("kq", "kh", "ks", "vq", "vh", "vs") if s[k] is not None}


def _plain_fork(c, s):
    P, T, per, d = c["page"], c["tail"], c["ctx"] // c["page"], c["d"]
    src, dst, n = s["src"].long(), s["dst"].long(), s["count"].long()
    need = (n % P > 0).long()
    take = torch.cumsum(need, 0) - need
    head, free = s["state"].long().unbind()
    new = s["ring"][(head + take) % s["pages"]].long()
    at = torch.arange(per, device="cuda")[None, :]
    full = (n // P)[:, None]
    old = s["table"][src]
    entry = torch.where(at < full, old, torch.where((at == full) & (need[:, None] > 0), new[:, None].int(), s["table"][dst]))
    table = s["table"].index_put((dst,), entry)
    one = torch.where(at < full, old, s["pages"]).long().flatten()
    extra = torch.cat([s["extra"], s["extra"][:1]]).index_put((one,), _dev(1), accumulate=True)[:-1]
    part = need > 0
    page, fresh = s["table"][src[part], n[part] // P].long(), new[part]
    planes = _planes(c, s)
    for x in planes.values():
        x[fresh] = x[page]
    out = dict(granted=s["count"].clone(), table=table, extra=extra, after=s["seq"].index_put((dst,), s["count"]),
               state=torch.stack([(head + need.sum()) % s["pages"], free - need.sum()]).int(), **planes)
    if T:
        for side in "kv":
            tail = s[side + "tail"]
            for a, b, m in _forks(c):
                whole = _lengths(c)[a]
                p = torch.arange(max(0, m - T), m, device="cuda")
                row = (s["table"][a].long()[p // P] * c["hkv"] + torch.arange(c["hkv"], device="cuda")[:, None]) * P + p % P
                late = (p >= whole - T)[None, :, None]
                tail[b][:, p % T] = torch.where(late, tail[a][:, p % T],
                                                _values(s, side, c[side + "t"], row, d).to(torch.bfloat16))
            out[side + "tail"] = tail
    return out


def _plain_free(c, s):
    pages, per = s["pages"], s["table"].shape[1]
    gone = s["gone"] != 0
    held = torch.where(gone, (s["seq"].long() + c["page"] - 1) // c["page"], 0)
    mine = torch.arange(per, device="cuda") < held[:, None]
    drops = torch.zeros(pages + 1, dtype=torch.int32, device="cuda")
    drops.index_put_((torch.where(mine, s["table"], pages).long().flatten(),), _dev(1), accumulate=True)
    drops = drops[:-1]
    freed = drops > s["extra"]
    rank = torch.cumsum(freed, 0) - 1
    head, count = s["state"].long().unbind()
    ring = torch.cat([s["ring"], s["ring"][:1]])
    ring = ring.index_put((torch.where(freed, (head + count + rank) % pages, pages),), torch.arange(pages, device="cuda").int())[:-1]
    return dict(ring=ring, state=torch.stack([head, count + freed.sum()]).int(), extra=torch.where(freed, 0, s["extra"] - drops),
                after=torch.where(gone, 0, s["seq"]))


def _plain_compact(c, s):
    pages, per = s["pages"], s["table"].shape[1]
    i = torch.arange(pages, device="cuda")
    held = (s["seq"].long() + c["page"] - 1) // c["page"]
    mine = torch.arange(per, device="cuda") < held[:, None]
    live = torch.zeros(pages + 1, dtype=torch.bool, device="cuda")
    live[torch.where(mine, s["table"], pages).long().flatten()] = True
    live = live[:-1]
    head, count = s["state"].long().unbind()
    free = torch.zeros(pages + 1, dtype=torch.bool, device="cuda")
    free[torch.where(i < count, s["ring"][(head + i) % pages], pages).long()] = True
    free = free[:-1]
    rank = torch.cumsum(live | free, 0) - 1  # place among the pages in hand: the lowest `used` places are kept
    used = live.sum()
    source = torch.nonzero(live & (rank >= used)).flatten()
    target = torch.nonzero(free & (rank < used)).flatten()
    move = torch.arange(pages, device="cuda").index_put((source,), target)
    planes = _planes(c, s)
    for x in planes.values():
        x[target] = x[source]
    extra = s["extra"].index_put((target,), s["extra"][source]).index_put((source,), _dev(0))
    left = (live | free) & (rank >= used)
    spot = torch.where(left, torch.cumsum(left, 0) - 1, pages)
    ring = torch.full((pages + 1,), -1, dtype=torch.int32, device="cuda").index_put((spot,), i.int())[:-1]
    table = torch.where(mine, move[s["table"].long().clamp(min=0)].int(), s["table"])
    return dict(table=table, ring=ring, state=torch.stack([0 * count, left.sum()]).int(), extra=extra, map=move.int(), **planes)


# ---- one pass -------------------------------------------------------------------------------

def _own(c, s):
    from rotated_bit_kv_kvq_gb300 import kvq
    if c["op"] == "attn":
        kvq.kvq_chunk_attention(s["handle"], s["q"], s["start"], s["out"], s["work"], mod=s["mod"])
        return {"out": s["out"]}
    if c["op"] == "fork":
        kvq.kvq_page_fork(s["handle"], s["pool"], s["share"], s["src"], s["dst"], s["granted"], n_tokens=s["count"],
                          seq_len_out=s["after"])
        out = dict(granted=s["granted"], table=s["table"], extra=s["extra_next"], after=s["after"], state=s["next"])
    elif c["op"] == "free":
        kvq.kvq_page_free(s["handle"], s["pool"], s["share"], s["gone"], seq_len_out=s["after"])
        return dict(ring=s["ring"], state=s["next"], extra=s["extra_next"], after=s["after"])
    else:
        kvq.kvq_page_compact(s["handle"], s["pool"], s["share"], s["table_next"], s["ring_next"], s["work"], page_map=s["map"])
        out = dict(table=s["table_next"], ring=s["ring_next"], state=s["next"], extra=s["extra_next"], map=s["map"])
    out.update(_planes(c, s))
    if c["op"] == "fork" and c["tail"]:
        out.update(ktail=s["ktail"], vtail=s["vtail"])
    return out


def run(state):
    c = state["case"]
    if own:
        return _own(c, state)
    return {"attn": _plain_attn, "fork": _plain_fork, "free": _plain_free, "compact": _plain_compact}[c["op"]](c, state)


# ---- the definitions in 64 bits ----------------------------------------------------------------

def _host(t):
    return None if t is None else (t.float() if t.dtype in (torch.bfloat16, torch.float16) else t).cpu().numpy()


class _Plane:
    """One side of a cache on the host: rows of values in 64 bits, decoded channel by channel."""

    def __init__(self, s, side, kind, d):
        self.kind, self.d, self.v = kind, d, side == "v"
        self.qs, self.hd = _host(s[side + "q"]), _host(s[side + "s"]).reshape(-1, d // 32, 2 if kind.endswith("_1") else 1)
        self.hi = None if s[side + "h"] is None else _host(s[side + "h"]).reshape(-1).view(np.int32 if side == "k" else np.int16)
        if self.hi is not None:  # K: [row][block]; V: [row pair][block][part][row]
            self.hi = self.hi.reshape(-1, d // 32) if side == "k" else self.hi.reshape(-1, d // 32, 2, 2)

    def rows(self, r):
        kind, nb = self.kind, self.d // 32
        qs, hd = self.qs[r].reshape(len(r), nb, self.qs.shape[1] // nb), self.hd[r].astype(np.float64)
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
    P = c["page"]
    if not P:
        return (b * c["hkv"] + h) * c["ctx"] + pos
    return (table[b][pos // P].astype(np.int64) * c["hkv"] + h) * P + pos % P


def _exact_attn(c, s):
    H, d, T, G = c["hkv"], c["d"], c["tail"], c["hq"] // c["hkv"]
    k, v = _Plane(s, "k", c["kt"], d), _Plane(s, "v", c["vt"], d)
    table, q, had = _host(s.get("table")), _host(s["q"]).astype(np.float64), _hadamard(d)
    tails = [_host(s[x]) if T else None for x in ("ktail", "vtail")]
    slopes, out, r0 = _host(s["slopes"]), np.zeros((len(q), c["hq"], d)), 0
    for b, (n, (lo, hi)) in enumerate(zip(_lengths(c), _visible(c))):
        m, pos = len(lo), np.arange(n)
        if m == 0:
            continue
        for h in range(H):
            r = _exact_row(c, table, b, h, pos)
            keys, vals = k.rows(r), v.rows(r)
            if T:
                late = pos >= n - T
                keys[late], vals[late] = (t[b, h, pos[late] % T] for t in tails)
            hidden = (pos[None] < lo[:, None]) | (pos[None] >= hi[:, None])
            for j in range(h * G, (h + 1) * G):
                a = (q[r0:r0 + m, j] @ had) @ keys.T / math.sqrt(d)
                if c["cap"]:
                    a = np.tanh(a / c["cap"]) * c["cap"]
                if c["alibi"]:
                    a = a - float(slopes[j]) * np.abs(np.arange(n - m, n)[:, None] - pos[None])
                a[hidden] = -np.inf
                a = np.exp(a - a.max(-1, keepdims=True))
                out[r0:r0 + m, j] = (a / a.sum(-1, keepdims=True)) @ vals @ had
        r0 += m
    return {"out": out}


def _exact_fork(c, s):
    """The tails (values); everything else is whole numbers or a copy of them."""
    out = dict.fromkeys(["granted", "table", "extra", "after", "state"] + list(_planes(c, s)))
    if c["tail"]:
        table, T = _host(s["table"]), c["tail"]
        for side in "kv":
            plane, tail = _Plane(s, side, c[side + "t"], c["d"]), _host(s[side + "tail"]).astype(np.float64)
            old, lens = tail.copy(), _lengths(c)
            for a, b, m in _forks(c):
                for h in range(c["hkv"]):
                    p = np.arange(max(0, m - T), m)
                    late = p >= lens[a] - T
                    tail[b, h, p[late] % T] = old[a, h, p[late] % T]
                    tail[b, h, p[~late] % T] = plane.rows(_exact_row(c, table, a, h, p[~late]))
            out[side + "tail"] = tail
    return out


def exact(case, seed):
    """In 64 bits; None where the outputs are whole numbers, or where it would take too long on the host."""
    if case["op"] in ("free", "compact") or (case["op"] == "fork" and not case["tail"]) or work(case)["flops"] > 3e10 or work(case)["bytes"] > 1.5e9:
        return None
    return {"attn": _exact_attn, "fork": _exact_fork}[case["op"]](case, prepare(case, seed))
