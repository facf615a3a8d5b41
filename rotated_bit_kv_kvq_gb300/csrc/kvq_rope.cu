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
// upper 32 bits feed sincospi.  No fp64, and as exact at position 2^30 as at 1.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kRopeThreads = 128;
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
__device__ __forceinline__ void to_f32(const Raw8<DT>& r, float (&x)[8]) {
  if constexpr (DT == KVQ_F32) {
    const uint32_t w[8] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w, r.w[1].x, r.w[1].y, r.w[1].z, r.w[1].w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  } else {
    const uint32_t w[4] = {r.w[0].x, r.w[0].y, r.w[0].z, r.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == KVQ_BF16) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      } else {
        const float2 f = __half22float2(u32_as_h2(w[i]));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
      }
    }
  }
}
template <int DT>
__device__ __forceinline__ Raw8<DT> from_f32(const float (&x)[8]) {
  Raw8<DT> r;
  if constexpr (DT == KVQ_F32) {
    r.w[0] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    r.w[1] = make_uint4(__float_as_uint(x[4]), __float_as_uint(x[5]), __float_as_uint(x[6]), __float_as_uint(x[7]));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (DT == KVQ_BF16) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        w[i] = pack_h2(x[2 * i], x[2 * i + 1]);
      }
    }
    r.w[0] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  return r;
}

__device__ __forceinline__ void load_weights(const void* w, int dt, int ch, float (&x)[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 1.0f;
  } else if (dt == KVQ_F32) {
    to_f32<KVQ_F32>(load8<KVQ_F32>(w, ch), x);
  } else if (dt == KVQ_BF16) {
    to_f32<KVQ_BF16>(load8<KVQ_BF16>(w, ch), x);
  } else {
    to_f32<KVQ_F16>(load8<KVQ_F16>(w, ch), x);
  }
}

// One CTA per row.  A head lies on L lanes, NC chunks of 8 channels each; a warp takes
// 32 / L heads at a time.
template <int DT, int L, int NC>
__global__ void __launch_bounds__(kRopeThreads) qk_norm_rope_kernel(RopeArgs a, kvq_rope_norm r) {
  __shared__ __align__(16) float s_cos[kMaxPairs], s_sin[kMaxPairs];
  constexpr int HW = 32 / L;  // heads per warp
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = blockIdx.x, d = a.head_dim, half = r.rot_dim / 2;
  const int dst = a.dst_row ? a.dst_row[row] : row;
  if (dst < 0 || dst >= a.n_dst_rows) {
    if (dst >= 0 && threadIdx.x == 0) atomicOr(a.status, KVQ_DEV_ERR_ROW);
    return;
  }
  const int pos = a.pos[row];
  for (int i = threadIdx.x; i < half; i += kRopeThreads) {
    const unsigned long long t = (unsigned long long)(long long)pos * turns64(r.inv_freq[i]);
    // the upper 32 bits as a signed fraction of a turn in half turns: [-1, 1)
    sincospif(float(int32_t(t >> 32)) * 4.656612873077393e-10f, &s_sin[i], &s_cos[i]);
  }
  __syncthreads();
  const int sub = lane / L, l = lane % L;

  for (int part = 0; part < 2; ++part) {  // queries, keys
    const int heads = part ? a.n_kv_heads : a.n_q_heads;
    const void* w = part ? r.k_weight : r.q_weight;
    const void* in = a.in[part];
    void* out = a.out[part];
    float A[NC][8], B[NC][8];
    int from[NC];     // lane (of L) and chunk the partner channels come from; -1: not rotated, -2: own chunk
#pragma unroll
    for (int j = 0; j < NC; ++j) {
      const int ck = l + 32 * j, ch = 8 * ck;  // (NC > 1 only with L = 32)
      from[j] = -1;
      if (ch < d) {
        load_weights(w, r.weight_dtype, ch, A[j]);
        if (ch < r.rot_dim) {
          if (r.interleaved) {
            from[j] = -2;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const float c = s_cos[ch / 2 + i / 2], s = s_sin[ch / 2 + i / 2];
              B[j][i] = -A[j][i + 1] * s;
              B[j][i + 1] = A[j][i] * s;
              A[j][i] *= c;
              A[j][i + 1] *= c;
            }
          } else {
            const bool second = ch >= half;
            const int c0 = second ? ch - half : ch;
            from[j] = second ? ck - half / 8 : ck + half / 8;
            float wp[8];
            load_weights(w, r.weight_dtype, 8 * from[j], wp);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float c = s_cos[c0 + i], s = s_sin[c0 + i];
              A[j][i] *= c;
              B[j][i] = second ? wp[i] * s : -wp[i] * s;
            }
          }
        }
      }
    }
    for (int h0 = warp * HW; h0 < heads; h0 += (kRopeThreads / 32) * HW) {
      const int h = h0 + sub;
      Raw8<DT> raw[NC];
      float x[NC][8], ss = 0.0f;
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        const int ch = 8 * (l + 32 * j);
        if (h < heads && ch < d) {
          raw[j] = load8<DT>(in, row * a.stride[part] + (long long)h * d + ch);
        } else {
#pragma unroll
          for (auto& q : raw[j].w) q = make_uint4(0, 0, 0, 0);
        }
        to_f32<DT>(raw[j], x[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[j][i], x[j][i], ss);
      }
      float scale = 1.0f;
      if (w) {
#pragma unroll
        for (int o = 1; o < L; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        scale = 1.0f / sqrtf(ss / float(d) + r.eps);
      }
#pragma unroll
      for (int j = 0; j < NC; ++j) {
        float xp[8], y[8];
        if (r.interleaved || half == 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) xp[i] = x[j][i ^ 1];
        } else {
          // the partner's eight values; lanes that do not rotate read their own
          Raw8<DT> rp;
          const int fl = from[j] >= 0 ? from[j] % 32 : l, fj = from[j] >= 0 ? from[j] / 32 : j;
          const int src = sub * L + fl;
#pragma unroll
          for (int q = 0; q < int(sizeof(rp.w) / 16); ++q) {
            uint32_t t[4] = {0, 0, 0, 0};
#pragma unroll
            for (int jj = 0; jj < NC; ++jj) {
              const uint32_t g[4] = {__shfl_sync(0xffffffffu, raw[jj].w[q].x, src),
                                     __shfl_sync(0xffffffffu, raw[jj].w[q].y, src),
                                     __shfl_sync(0xffffffffu, raw[jj].w[q].z, src),
                                     __shfl_sync(0xffffffffu, raw[jj].w[q].w, src)};
              if (fj == jj) { t[0] = g[0]; t[1] = g[1]; t[2] = g[2]; t[3] = g[3]; }
            }
            rp.w[q] = make_uint4(t[0], t[1], t[2], t[3]);
          }
          to_f32<DT>(rp, xp);
        }
        const int ch = 8 * (l + 32 * j);
        if (h < heads && ch < d) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            y[i] = scale * (from[j] == -1 ? x[j][i] * A[j][i] : fmaf(x[j][i], A[j][i], xp[i] * B[j][i]));
          store8<DT>(out, ((long long)dst * heads + h) * d + ch, from_f32<DT>(y));
        }
      }
    }
  }
  if (a.in[2]) {  // values: one run of n_kv_heads * head_dim elements
    const int n8 = a.n_kv_heads * d / 8;
    for (int i = threadIdx.x; i < n8; i += kRopeThreads)
      store8<DT>(a.out[2], (long long)dst * a.n_kv_heads * d + 8 * i, load8<DT>(a.in[2], row * a.stride[2] + 8 * i));
  }
}

template <int DT>
cudaError_t launch_dt(const RopeArgs& a, const kvq_rope_norm& r, cudaStream_t st) {
  const int n = a.head_dim / 8;
  auto go = [&](auto kern) {
    kern<<<unsigned(a.n_rows), kRopeThreads, 0, st>>>(a, r);
    return cudaGetLastError();
  };
  if (n <= 4) return go(qk_norm_rope_kernel<DT, 4, 1>);
  if (n <= 8) return go(qk_norm_rope_kernel<DT, 8, 1>);
  if (n <= 16) return go(qk_norm_rope_kernel<DT, 16, 1>);
  if (n <= 32) return go(qk_norm_rope_kernel<DT, 32, 1>);
  return go(qk_norm_rope_kernel<DT, 32, 2>);
}

}  // namespace

cudaError_t launch_qk_norm_rope(const RopeArgs& a, const kvq_rope_norm& r, int dtype, cudaStream_t st) {
  if (dtype == KVQ_F32) return launch_dt<KVQ_F32>(a, r, st);
  if (dtype == KVQ_BF16) return launch_dt<KVQ_BF16>(a, r, st);
  return launch_dt<KVQ_F16>(a, r, st);
}

}  // namespace kvq
