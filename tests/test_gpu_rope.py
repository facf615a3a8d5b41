"""Norms with the position rotation against the float64 oracle, on the GPU.

Bound per value, M = r (|x w| + |x' w'|) with r the norm's factor: the angle is exact to 2^-31
turns and rounds to fp32 once (2^-24 of at most half a turn: 2^-22.3 in sine or cosine), sincospi
is good to 2 ulp (2^-23), four products and sums round (2^-22), and the sum of squares (at most 16
in a lane, then 5 pairs: 21 roundings, halved by the root) with root and division rounds to 2^-20.2:
together below 2^-19 M.  Then one rounding to the output's type: half its eps, or half its smallest step."""

import numpy as np
import pytest

from kvq_testlib import require_gpu
from oracle import step_oracle as so

pytestmark = pytest.mark.gpu


def _dt(torch, name):
    return {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[name]


def _np(t):
    return t.float().cpu().numpy().astype(np.float64)


def _close(torch, got, x, weight, eps, pos, freq, inter, dtype):
    ref = so.norm_rope(x, weight, eps, pos, freq, inter)
    w = np.ones(x.shape[-1]) if weight is None else np.abs(weight)
    r = 1.0 if weight is None else 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    a = np.abs(x) * w * r
    m = a.copy()
    half = len(freq)
    for i in range(half):
        p, s = (2 * i, 2 * i + 1) if inter else (i, i + half)
        m[..., p] = m[..., s] = a[..., p] + a[..., s]
    fi = torch.finfo(dtype)
    bound = 2.0 ** -19 * m + (np.abs(ref) + 2.0 ** -19 * m) * fi.eps / 2 + fi.tiny * fi.eps / 2
    assert np.all(np.isfinite(got))
    assert np.all(np.abs(got - ref) <= bound), np.max(np.abs(got - ref) / bound)


def _desc(kvq, torch, hkv, d):
    c = kvq.descriptor(1, hkv, d, 64, 0, "q4_0", "q4_0")
    status = torch.zeros(4, dtype=torch.int32, device="cuda")
    c.status = c.seq_len = status.data_ptr()
    return c, status


def _inputs(torch, n, hq, hkv, d, rot, dtype, far, seed, pad=0):
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(n, (hq + 2 * hkv) * d + pad, generator=g).mul(3).to(dtype).cuda()
    parts = qkv[:, :hq * d], qkv[:, hq * d:(hq + hkv) * d], qkv[:, (hq + hkv) * d:(hq + 2 * hkv) * d]
    freq = 1e-6 ** (torch.arange(rot // 2, dtype=torch.float64) * 2 / max(rot, 1))
    pos = torch.randint(0, far, (n,), generator=g, dtype=torch.int32)
    return parts, freq.float().cuda(), pos.cuda()


CASES = [  # n, hq, hkv, d, rot, interleaved, dtype, weight dtype, far
    (1, 1, 1, 32, 32, False, "f32", "f32", 10), (1, 1, 1, 32, 16, True, "bf16", "bf16", 10),
    (3, 4, 2, 64, 64, False, "bf16", "bf16", 100000), (5, 6, 3, 96, 96, True, "f16", "f16", 5000),
    (7, 6, 2, 96, 32, False, "f32", "bf16", 5000), (33, 8, 4, 128, 128, False, "f32", "f32", 1 << 30),
    (9, 8, 1, 128, 64, True, "bf16", "f32", 1 << 20), (4, 3, 1, 160, 160, False, "bf16", None, 4096),
    (4, 5, 5, 192, 128, False, "f16", "f16", 4096), (17, 24, 4, 256, 256, False, "bf16", "bf16", 65536),
    (2, 4, 4, 288, 288, False, "f32", "f32", 1000), (3, 2, 1, 320, 320, True, "bf16", "bf16", 1000),
    (3, 2, 1, 320, 320, False, "f16", None, 1000), (3, 3, 1, 448, 400, False, "f32", "f32", 100000),
    (2, 2, 1, 512, 512, False, "bf16", "bf16", 100000), (2, 2, 1, 512, 512, True, "f32", "f16", 100000),
    (2, 2, 1, 512, 0, False, "f16", "f16", 10), (1, 70, 1, 64, 32, False, "bf16", "bf16", 10),
    (700, 16, 2, 64, 64, False, "bf16", "bf16", 100000), (400, 12, 2, 128, 128, False, "bf16", "bf16", 100000),
]


@pytest.mark.parametrize("n,hq,hkv,d,rot,inter,dt,wdt,far", CASES)
def test_norm_rope(n, hq, hkv, d, rot, inter, dt, wdt, far):
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    dtype = _dt(torch, dt)
    c, status = _desc(kvq, torch, hkv, d)
    (q, k, v), freq, pos = _inputs(torch, n, hq, hkv, d, rot, dtype, far, 11, pad=8)
    g = torch.Generator().manual_seed(12)
    wq, wk = (None, None) if wdt is None else ((1 + 0.3 * torch.randn(d, generator=g)).to(_dt(torch, wdt)).cuda() for _ in range(2))
    plan = kvq.RopeNorm(freq, q_weight=wq, k_weight=wk, eps=1e-5, interleaved=inter)
    out = [torch.full((n, h, d), 7.0, dtype=dtype, device="cuda") for h in (hq, hkv, hkv)]
    kvq.kvq_qk_norm_rope(c, plan, q, k, v, pos, *out)
    torch.cuda.synchronize()
    f = freq.double().cpu().numpy()
    for x, w, o, h in ((q, wq, out[0], hq), (k, wk, out[1], hkv)):
        _close(torch, _np(o), _np(x).reshape(n, h, d), None if w is None else _np(w), np.float64(np.float32(1e-5)),
               pos.cpu().numpy(), f, inter, dtype)
    assert torch.equal(out[2].view(n, -1), v)
    assert int(status[0]) == 0


def test_norm_rope_rows_to_places():
    """Rows to other rows, rows left out, rows past the end reported; what no row goes to is left as it was."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    n, hq, hkv, d = 6, 4, 2, 64
    c, status = _desc(kvq, torch, hkv, d)
    (q, k, v), freq, pos = _inputs(torch, n, hq, hkv, d, 64, torch.bfloat16, 500, 13)
    plan = kvq.RopeNorm(freq)
    want = [torch.empty(n, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv)]
    kvq.kvq_qk_norm_rope(c, plan, q, k, v, pos, *want)
    dst = torch.tensor([3, -1, 0, 8, 1 << 30, 5], dtype=torch.int32, device="cuda")
    out = [torch.full((8, h, d), 7.0, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv)]
    kvq.kvq_qk_norm_rope(c, plan, q, k, v, pos, *out, dst_row=dst)
    torch.cuda.synchronize()
    for o, w in zip(out, want):
        for row in range(8):
            src = {3: 0, 0: 2, 5: 5}.get(row)
            assert torch.equal(o[row], w[src] if src is not None else torch.full_like(o[row], 7.0)), row
    assert int(status[0]) == kvq.KVQ_DEV_ERR_ROW


def test_norm_rope_in_place_without_values_and_negative_positions():
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    n, hq, hkv, d = 5, 3, 3, 128
    c, _ = _desc(kvq, torch, hkv, d)
    (q, k, _), freq, pos = _inputs(torch, n, hq, hkv, d, 128, torch.float32, 1000, 14)
    pos = -pos - 1
    q, k = q.reshape(n, hq, d).contiguous(), k.reshape(n, hkv, d).contiguous()
    x = _np(q), _np(k)
    plan = kvq.RopeNorm(freq, k_weight=torch.ones(d, device="cuda"))
    kvq.kvq_qk_norm_rope(c, plan, q, k, None, pos, q, k, None)
    torch.cuda.synchronize()
    f = freq.double().cpu().numpy()
    _close(torch, _np(q), x[0], None, 0.0, pos.cpu().numpy(), f, False, torch.float32)
    _close(torch, _np(k), x[1], np.ones(d), np.float64(np.float32(1e-6)), pos.cpu().numpy(), f, False, torch.float32)


def test_norm_rope_special_values():
    """An all-zero head stays zero (eps > 0); Inf and NaN stay in their own head, and without a norm in their own pair."""
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    n, hq, hkv, d = 1, 4, 1, 128
    c, _ = _desc(kvq, torch, hkv, d)
    (q, k, v), freq, pos = _inputs(torch, n, hq, hkv, d, 64, torch.bfloat16, 1000, 15)
    q = q.clone()
    q[:, 0:128] = 0
    q[0, 128 + 3] = float("inf")
    q[0, 256 + 100] = float("nan")
    ones = torch.ones(d, device="cuda")
    for w in (None, ones):
        out = [torch.empty(n, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv)]
        kvq.kvq_qk_norm_rope(c, kvq.RopeNorm(freq, q_weight=w), q, k, v, pos, *out)
        torch.cuda.synchronize()
        o = out[0][0]
        assert not o[0].any() and bool(torch.isfinite(o[3]).all())
        if w is None:
            bad = ~torch.isfinite(o)
            assert bad[1].nonzero().flatten().tolist() == [3, 35] and bad[2].nonzero().flatten().tolist() == [100]


def test_norm_rope_refuses_tensors():
    torch = require_gpu()
    from rotated_bit_kv_kvq_gb300 import kvq
    n, hq, hkv, d = 2, 2, 1, 64
    c, _ = _desc(kvq, torch, hkv, d)
    (q, k, v), freq, pos = _inputs(torch, n, hq, hkv, d, 64, torch.bfloat16, 10, 16)
    out = [torch.empty(n, h, d, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv)]
    plan = kvq.RopeNorm(freq)
    call = lambda **kw: kvq.kvq_qk_norm_rope(c, plan, **{**dict(  # noqa: E731
        q=q, k=k, v=v, pos=pos, q_out=out[0], k_out=out[1], v_out=out[2]), **kw})
    for kw in (dict(q=q.float()), dict(pos=pos.long()), dict(pos=pos[:1]), dict(k=k[:, :32]), dict(q=q.t()), dict(v=v.cpu()),
               dict(k_out=out[1].float()), dict(v_out=out[2][:1]), dict(q_out=out[0].transpose(0, 1))):
        with pytest.raises((ValueError, kvq.KvqError)):
            call(**kw)
    with pytest.raises(ValueError):
        kvq.RopeNorm(freq.double())
