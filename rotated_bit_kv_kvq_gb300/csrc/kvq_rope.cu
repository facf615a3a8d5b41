// Norms of query and key heads and the position rotation, from projection rows to
// the rows that the append and the attention take (kvq_qk_norm_rope).
//
// y = x * 1/sqrt(mean(x^2) + eps) * w, then (a, b) -> (a cos t - b sin t, a sin t + b cos t)
// for the pairs of the first rot_dim channels, t = pos * inv_freq.  With A = w cos t and
// B = -+ w' sin t (w' the partner's weight) a channel is r * (x A + x' B): the norm's
// factor r is the only thing that differs between the heads of a row.
//
// The angle modulo one turn is taken in integers: F = inv_freq / 2pi as a 64-bit fraction
// of a turn, pos * F modulo 2^64 its position (the overflow is whole turns), of which the
// upper 32 bits feed sincospi, rounded to fp32 (2^-26 turns).  No fp64, and as exact at position 2^30 as at 1.
//
// Bound by memory with many rows: 8192 rows of 48 heads of 128 in bf16, 201 MB in 36.7 us,
// 5.5 TB/s (82% of the card's measured copy rate); by the chain position - angle - factors -
// store with few: 4 rows of 32 heads of 256 4.3 us.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kMaxPairs = 256;

// floor(2^64 / 2pi)
constexpr unsigned long long kInvTwoPi = 0x28BE60DB9391054AULL;

// f / 2pi as a fraction of a turn, modulo 1, in units of 2^-64.  The significand of f
// (24 bits) times 1/2pi (64 bits), moved by f's exponent; the rounding of 1/2pi leaves an
// error of at most 2 units for |f| <= 1 and 2^(k + 1) for |f| < 2^k.
__device__ __forceinline__ unsigned long long turns64(float f) {
  const uint32_t u = __float_as_uint(f);
  const int e = int((u >> 23) & 255u);
  const uint32_t m = (u & 0x7FFFFFu) | (e ? 0x800000u : 0u);
  const int s = 150 - (e ? e : 1);  // |f| = m * 2^-s
  const unsigned long long lo = m * kInvTwoPi, hi = __umul64hi((unsigned long long)m, kInvTwoPi);
  unsigned long long t;
  if (s <= 0) t = s > -64 ? lo << -s : 0ULL;
  else if (s < 64) t = (hi << (64 - s)) | (lo >> s);
  else t = s < 128 ? hi >> (s - 64) : 0ULL;
  return (u >> 31) ? 0ULL - t : t;
}

template <int DT> struct Elem { using T = uint16_t; };
template <> struct Elem<KVQ_F32> { using T = float; };

// eight values of row memory
template <int DT>
struct Raw8 {
  uint4 w[DT == KVQ_F32 ? 2 : 1];
};
template <int DT>
__device__ __forceinline__ Raw8<DT> load8(const void* p, long long elem) {
  Raw8<DT> r;
  const uint4* s = reinterpret_cast<const uint4*>(static_cast<const typename Elem<DT>::T*>(p) + elem);
  r.w[0] = s[0];
  if constexpr (DT == KVQ_F32) r.w[1] = s[1];
  return r;
}
template <int DT>
__device__ __forceinline__ void store8(void* p, long long elem, const Raw8<DT>& r) {
  uint4* d = reinterpret_cast<uint4*>(static_cast<typename Elem<DT>::T*>(p) + elem);
  d[0] = r.w[0];
  if constexpr (DT == KVQ_F32) d[1] = r.w[1];
}
template <int DT>
__device__ __forceinline__ void to_f32(const Raw8<DT>& r, float2 (&x)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (DT == KVQ_F32) {
      const uint4& q = r.w[i / 2];
      x[i] = i & 1 ? make_float2(__uint_as_float(q.z), __uint_as_float(q.w)) : make_float2(__uint_as_float(q.x), __uint_as_float(q.y));
    } else {
      const uint32_t v = i == 0 ? r.w[0].x : i == 1 ? r.w[0].y : i == 2 ? r.w[0].z : r.w[0].w;
      if constexpr (DT == KVQ_BF16) x[i] = make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
      else x[i] = __half22float2(u32_as_h2(v));
    }
  }
}
template <int DT>
__device__ __forceinline__ Raw8<DT> from_f32(const float2 (&x)[4]) {
  Raw8<DT> r;
  if constexpr (DT == KVQ_F32) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      r.w[i] = make_uint4(__float_as_uint(x[2 * i].x), __float_as_uint(x[2 * i].y), __float_as_uint(x[2 * i + 1].x),
                          __float_as_uint(x[2 * i + 1].y));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == KVQ_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[i].x, x[i].y);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        w[i] = pack_h2(x[i].x, x[i].y);
      }
    }
    r.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return r;
}

__device__ __forceinline__ void load_weights(const void* w, int dt, int ch, float2 (&x)[4]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = make_float2(1.0f, 1.0f);
  } else if (dt == KVQ_F32) {
    to_f32<KVQ_F32>(load8<KVQ_F32>(w, ch), x);
  } else if (dt == KVQ_BF16) {
    to_f32<KVQ_BF16>(load8<KVQ_BF16>(w, ch), x);
  } else {
    to_f32<KVQ_F16>(load8<KVQ_F16>(w, ch), x);
  }
}

// A row is shared by WPR warps of a CTA of W.  A head lies on L lanes, NC chunks of 8 channels
// each; a warp takes 32 / L heads at a time and has the loads of the next kAhead - 1 times in
// flight, the first ones issued before the row's angles are computed.
// The channels' factors (norm weight times cosine or sine) are worked out once per warp and row,
// so with many rows a warp takes a whole row, and with few a row's heads spread over 8 warps.
template <int DT, int L, int NC, int W, int WPR>
__global__ void __launch_bounds__(32 * W, W == 4 ? (NC == 1 ? (WPR == 4 ? 8 : 6) : 4) : 2) qk_norm_rope_kernel(RopeArgs a, kvq_rope_norm r) {
  pdl_begin();
  constexpr int RPC = W / WPR, HW = 32 / L;  // rows of a CTA, heads of a warp
  constexpr int kAhead = DT == KVQ_F32 || NC > 1 || WPR == 4 ? 2 : 4;
  __shared__ __align__(16) float s_cos[RPC][kMaxPairs], s_sin[RPC][kMaxPairs];
  const int lane = threadIdx.x & 31, sub = lane / L, l = lane % L;
  const int rc = (threadIdx.x >> 5) / WPR, warp = (threadIdx.x >> 5) % WPR, rt = warp * 32 + lane;  // row of the CTA, place in it
  const int row = blockIdx.x * RPC + rc, d = a.head_dim, half = r.rot_dim / 2;
  int dst = row < a.n_rows ? (a.dst_row ? a.dst_row[row] : row) : -1;
  if (dst >= a.n_dst_rows) {
    if (rt == 0) atomicOr(a.status, KVQ_DEV_ERR_ROW);
    dst = -1;
  }
  if (WPR == W && dst < 0) return;  // (the CTA's only row)
  const bool live = dst >= 0;
  // the warp's units, HW heads each: the queries' (filled up to whole rounds of kAhead), then the keys'
  const int nq = ((a.n_q_heads + HW - 1) / HW - warp + WPR - 1) / WPR, nk = ((a.n_kv_heads + HW - 1) / HW - warp + WPR - 1) / WPR;
  const int nqp = (max(nq, 0) + kAhead - 1) / kAhead * kAhead;
  const long long qbase = row * a.stride[0], kbase = row * a.stride[1];
  Raw8<DT> raw[kAhead][NC];
  auto load = [&](int u, int n) {  // unit n into raw[u]
    const bool key = n >= nqp;
    const int h = (warp + (key ? n - nqp : n) * WPR) * HW + sub, heads = key ? a.n_kv_heads : a.n_q_heads;
    const void* in = key ? a.in[1] : a.in[0];
    const long long base = key ? kbase : qbase;
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int ch = 8 * (l + 32 * j);  // (NC > 1 only with L = 32)
      if (live && h < heads && ch < d) {
        raw[u][j] = load8<DT>(in, base + h * d + ch);
      } else {
#pragma unroll
        for (auto& q : raw[u][j].w) q = make_uint4(0, 0, 0, 0);
      }
    }
  };
#pragma unroll
  for (int u = 0; u < kAhead; ++u) load(u, u);
  const int pos = live ? a.pos[row] : 0;
  if (a.in[2] && live) {  // values: one run of n_kv_heads * head_dim elements
    const int n8 = a.n_kv_heads * d / 8;
    const long long from = row * a.stride[2], to = (long long)dst * a.n_kv_heads * d;
    constexpr int kCopy = 4;  // loads in flight
    for (int i0 = rt; i0 < n8; i0 += 32 * WPR * kCopy) {
      Raw8<DT> x[kCopy];
#pragma unroll
      for (int u = 0; u < kCopy; ++u)
        if (i0 + 32 * WPR * u < n8) x[u] = load8<DT>(a.in[2], from + 8 * (i0 + 32 * WPR * u));
#pragma unroll
      for (int u = 0; u < kCopy; ++u)
        if (i0 + 32 * WPR * u < n8) store8<DT>(a.out[2], to + 8 * (i0 + 32 * WPR * u), x[u]);
    }
  }
  for (int i = rt; i < half; i += 32 * WPR) {
    const unsigned long long t = (unsigned long long)(long long)pos * turns64(r.inv_freq[i]);
    // the upper 32 bits as a signed fraction of a turn in half turns: [-1, 1)
    sincospif(float(int32_t(t >> 32)) * 4.656612873077393e-10f, &s_sin[rc][i], &s_cos[rc][i]);
  }
  if (WPR == 1) __syncwarp(); else __syncthreads();
  if (!live) return;
  const float inv_d = 1.0f / float(d);

#pragma unroll 1
  for (int part = 0; part < 2; ++part) {  // queries, keys
    const int heads = part ? a.n_kv_heads : a.n_q_heads;
    const void* w = part ? r.k_weight : r.q_weight;
    void* out = part ? a.out[1] : a.out[0];
    const int first = part ? nqp : 0, count = part ? nk : nqp;
    float2 A[NC][4], B[NC][4];
    int from[NC];     // chunk (of the head) the partner channels come from; -1: not rotated, -2: own chunk
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int ck = l + 32 * j, ch = 8 * ck;
      from[j] = -1;
#pragma unroll
      for (int i = 0; i < 4; ++i) A[j][i] = B[j][i] = make_float2(0.0f, 0.0f);
      if (ch < d) {
        load_weights(w, r.weight_dtype, ch, A[j]);
        if (ch < r.rot_dim && r.interleaved) {
          from[j] = -2;
          const float4 c = *reinterpret_cast<const float4*>(&s_cos[rc][ch / 2]), s = *reinterpret_cast<const float4*>(&s_sin[rc][ch / 2]);
          const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            B[j][i] = make_float2(-A[j][i].y * ss[i], A[j][i].x * ss[i]);
            A[j][i] = make_float2(A[j][i].x * cc[i], A[j][i].y * cc[i]);
          }
        } else if (ch < r.rot_dim) {
          const bool second = ch >= half;
          const int c0 = second ? ch - half : ch;
          from[j] = second ? ck - half / 8 : ck + half / 8;
          load_weights(w, r.weight_dtype, 8 * from[j], B[j]);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float2 c = *reinterpret_cast<const float2*>(&s_cos[rc][c0 + 2 * i]);
            float2 s = *reinterpret_cast<const float2*>(&s_sin[rc][c0 + 2 * i]);
            if (!second) s = make_float2(-s.x, -s.y);
            A[j][i] = __fmul2_rn(A[j][i], c);
            B[j][i] = __fmul2_rn(B[j][i], s);
          }
        }
      }
    }
#pragma unroll 1
    for (int n0 = 0; n0 < count; n0 += kAhead) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int h = (warp + (n0 + u) * WPR) * HW + sub;
        if (h - sub < heads) {  // (warp-uniform)
          float2 x[NC][4], sq = make_float2(0.0f, 0.0f);
#pragma unroll
          for (int j = 0; j < NC; ++j) {
            to_f32<DT>(raw[u][j], x[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) sq = __ffma2_rn(x[j][i], x[j][i], sq);
          }
          float scale = 1.0f;
          if (w) {
            float ss = sq.x + sq.y;
#pragma unroll
            for (int o = 1; o < L; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            scale = rsqrtf(fmaf(ss, inv_d, r.eps));
          }
          const float2 scale2 = make_float2(scale, scale);
#pragma unroll
          for (int j = 0; j < NC; ++j) {
            float2 xp[4], y[4];
            if (r.interleaved || half == 0) {
#pragma unroll
              for (int i = 0; i < 4; ++i) xp[i] = make_float2(x[j][i].y, x[j][i].x);
            } else {
              // the partner's eight values; lanes that do not rotate read their own
              Raw8<DT> rp;
              const int fl = from[j] >= 0 ? from[j] % 32 : l, fj = from[j] >= 0 ? from[j] / 32 : j;
              const int src = sub * L + fl;
#pragma unroll
              for (int q = 0; q < int(sizeof(rp.w) / 16); ++q) {
                uint4 t = make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int jj = 0; jj < NC; ++jj) {
                  const uint4 g = make_uint4(__shfl_sync(0xffffffffu, raw[u][jj].w[q].x, src),
                                             __shfl_sync(0xffffffffu, raw[u][jj].w[q].y, src),
                                             __shfl_sync(0xffffffffu, raw[u][jj].w[q].z, src),
                                             __shfl_sync(0xffffffffu, raw[u][jj].w[q].w, src));
                  if (NC == 1 || fj == jj) t = g;
                }
                rp.w[q] = t;
              }
              to_f32<DT>(rp, xp);
            }
            if (from[j] == -1) {  // (B is zero, but not where the partner is no number)
#pragma unroll
              for (int i = 0; i < 4; ++i) xp[i] = make_float2(0.0f, 0.0f);
            }
            const int ch = 8 * (l + 32 * j);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              y[i] = __fmul2_rn(scale2, __ffma2_rn(x[j][i], A[j][i], __fmul2_rn(xp[i], B[j][i])));
            if (h < heads && ch < d)
              store8<DT>(out, ((long long)dst * heads + h) * d + ch, from_f32<DT>(y));
          }
        }
        load(u, first + n0 + u + kAhead);
      }
    }
  }
}

template <int DT>
cudaError_t launch_dt(const RopeArgs& a, const kvq_rope_norm& r, cudaStream_t st) {
  const int n = a.head_dim / 8;
  const int sms = device_sm_count();
  // As many warps per row as one wave holds: the factors of a row are worked out in each of its
  // warps, and a second wave costs a whole one.  1001 rows of 48 heads of 128: 4 warps a row 7.3 us
  // (8 CTAs an SM; 9 us with 6 of them, two waves), 2 warps 9.1, 1 warp 10.0; 8192 rows: 4 warps
  // 52.6 us, 1 warp 36.7; 4 rows of 32 heads of 256: 4 warps 6.0 us, 8 warps 4.3.
  auto go = [&](auto w8, auto w4, auto w2, auto w1) {
    const long long n = a.n_rows, m = sms > 0 ? sms : 148;
    if (n <= 2 * m) return launch_dependent(w8, unsigned(n), 256, 0, st, 1, a, r);
    if (n <= 8 * m) return launch_dependent(w4, unsigned(n), 128, 0, st, 1, a, r);
    if (n <= 12 * m) return launch_dependent(w2, unsigned((n + 1) / 2), 128, 0, st, 1, a, r);
    return launch_dependent(w1, unsigned((n + 3) / 4), 128, 0, st, 1, a, r);
  };
#define KVQ_ROPE(L, NC) \
  go(qk_norm_rope_kernel<DT, L, NC, 8, 8>, qk_norm_rope_kernel<DT, L, NC, 4, 4>, \
     qk_norm_rope_kernel<DT, L, NC, 4, 2>, qk_norm_rope_kernel<DT, L, NC, 4, 1>)
  if (n <= 4) return KVQ_ROPE(4, 1);
  if (n <= 8) return KVQ_ROPE(8, 1);
  if (n <= 16) return KVQ_ROPE(16, 1);
  if (n <= 32) return KVQ_ROPE(32, 1);
  return KVQ_ROPE(32, 2);
#undef KVQ_ROPE
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, const kvq_rope_norm& r, int dtype, cudaStream_t st) {
  if (dtype == KVQ_F32) return launch_dt<KVQ_F32>(a, r, st);
  if (dtype == KVQ_BF16) return launch_dt<KVQ_BF16>(a, r, st);
  return launch_dt<KVQ_F16>(a, r, st);
}

}  // namespace kvq
