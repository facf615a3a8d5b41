// Decode attention over selected blocks (kvq_sparse_decode_attention).
//
// One CTA per (query head, sequence): a warp takes a token at a time, lane l its channels
// l, l + 32, ...; online softmax per warp, the warps merged at the end.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math.h>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_quant.cuh"

namespace kvq {
namespace {

constexpr int kSpWarps = 8;

struct SparseArgs {
  kvq_cache c;
  const void* q;
  const int32_t* sel;
  void* out;
  int q_dtype, out_dtype, n_q_heads, group, block_tokens, n_select, rot_k, rot_v;
  float scale_log2;
};

// channel 32 * blk + lane of a body row
__device__ __forceinline__ float body_value(const kvq_cache& c, bool v, long long row, int blk, int lane) {
  const int qt = v ? c.v_type : c.k_type, d = c.head_dim, nb = d / 32;
  const uint8_t* qs = static_cast<const uint8_t*>(v ? c.v_qs : c.k_qs);
  const __half* hd = static_cast<const __half*>(v ? c.v_d : c.k_d);
  const long long e = row * nb + blk;
  if (qt == KVQ_TYPE_Q8_0) return float(int(qs[row * d + 32 * blk + lane]) - 128) * __half2float(hd[e]);
  int code = (qs[row * (d / 2) + 16 * blk + (lane & 15)] >> (lane & 16 ? 4 : 0)) & 15;
  if (type_has_qh(qt)) code |= int((qh_get(v ? c.v_qh : c.k_qh, !v, size_t(row), nb, blk) >> lane) & 1u) << 4;
  if (type_has_min(qt)) return fmaf(float(code), __half2float(hd[2 * e]), __half2float(hd[2 * e + 1]));
  return float(code - type_code_offset(qt)) * __half2float(hd[e]);
}

template <int D>
__global__ void __launch_bounds__(kSpWarps * 32) sparse_kernel(SparseArgs a) {
  constexpr int G = (D & (D - 1)) == 0 ? D : 64, E = D / 32;
  __shared__ float s_x[D], s_acc[kSpWarps][D], s_m[kSpWarps], s_l[kSpWarps];
  const kvq_cache& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int hq = blockIdx.x, b = blockIdx.y, h = hq / a.group, T = c.tail_len;
  const int n = min(max(c.seq_len[b], 0), c.max_ctx);
  const long long bh = (long long)b * c.n_kv_heads + h;
  const int32_t* sel = a.sel + bh * a.n_select;
  if (warp == 0) {
    float v[E];
    const size_t row = ((size_t)b * a.n_q_heads + hq) * D;
#pragma unroll
    for (int gi = 0; gi < D / G; ++gi) load_vals<G / 32>(a.q, a.q_dtype, row + gi * G + lane * (G / 32), v + gi * (G / 32));
    if (a.rot_k) warp_fwht<D, G>(v, lane);
    const float s = a.scale_log2 * (a.rot_k ? inv_sqrt_group<G>() : 1.0f);
#pragma unroll
    for (int e = 0; e < E; ++e) s_x[fwht_channel<D, G>(lane, e)] = v[e] * s;
  }
  __syncthreads();
  float q[E], acc[E], m = -INFINITY, l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) { q[e] = s_x[32 * e + lane]; acc[e] = 0.0f; }
  __syncthreads();
  const RowMap rm = row_map(c);
  for (int i = 0; i < a.n_select; ++i) {
    const int blk = sel[i];
    if (blk < 0 || (long long)blk * a.block_tokens >= n) continue;
    const int t0 = blk * a.block_tokens, t1 = min(n, t0 + a.block_tokens);
    for (int t = t0 + warp; t < t1; t += kSpWarps) {
      const bool tail = t >= n - T;
      const long long row = tail ? bh * T + t % T : body_row(rm, b, h, t);
      if (row < 0) {
        if (lane == 0) atomicOr(c.status, KVQ_DEV_ERR_PAGE);
        continue;
      }
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float x = tail ? bf16_bits_to_f32(static_cast<const uint16_t*>(c.k_tail)[row * D + 32 * e + lane])
                             : body_value(c, false, row, e, lane);
        s = fmaf(q[e], x, s);
      }
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      const float nm = fmaxf(m, s);
      const float f = m == -INFINITY ? 0.0f : exp2f(m - nm), p = exp2f(s - nm);
      m = nm;
      l = l * f + p;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float x = tail ? bf16_bits_to_f32(static_cast<const uint16_t*>(c.v_tail)[row * D + 32 * e + lane])
                             : body_value(c, true, row, e, lane);
        acc[e] = fmaf(acc[e], f, p * x);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < E; ++e) s_acc[warp][32 * e + lane] = acc[e];
  if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
  __syncthreads();
  if (warp != 0) return;
  float M = -INFINITY, L = 0.0f;
  for (int w = 0; w < kSpWarps; ++w) M = fmaxf(M, s_m[w]);
  float f[kSpWarps];
  for (int w = 0; w < kSpWarps; ++w) {
    f[w] = s_m[w] == -INFINITY ? 0.0f : exp2f(s_m[w] - M);
    L += s_l[w] * f[w];
  }
  const float inv = L > 0.0f ? 1.0f / L : 0.0f;
  float x[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const int ch = fwht_channel<D, G>(lane, e);
    x[e] = 0.0f;
    for (int w = 0; w < kSpWarps; ++w) x[e] = fmaf(s_acc[w][ch], f[w], x[e]);
    x[e] *= inv;
  }
  if (a.rot_v) {
    warp_fwht<D, G>(x, lane);
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] *= inv_sqrt_group<G>();
  }
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const size_t o = ((size_t)b * a.n_q_heads + hq) * D + fwht_channel<D, G>(lane, e);
    if (a.out_dtype == KVQ_F32) static_cast<float*>(a.out)[o] = x[e];
    else if (a.out_dtype == KVQ_BF16) static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(x[e]);
    else static_cast<__half*>(a.out)[o] = __float2half_rn(x[e]);
  }
}

}  // namespace

cudaError_t launch_sparse_decode(const kvq_cache& c, Rot rot, const void* q, int q_dtype, int n_q_heads, float scale,
                                 int block_tokens, const int32_t* sel, int n_select, void* out, int out_dtype,
                                 cudaStream_t st) {
  SparseArgs a{c, q, sel, out, q_dtype, out_dtype, n_q_heads, n_q_heads / c.n_kv_heads, block_tokens, n_select,
               rot.k, rot.v, scale * 1.4426950408889634f};
  const dim3 grid(n_q_heads, c.batch);
  switch (c.head_dim) {
    case 64: sparse_kernel<64><<<grid, kSpWarps * 32, 0, st>>>(a); break;
    case 128: sparse_kernel<128><<<grid, kSpWarps * 32, 0, st>>>(a); break;
    case 192: sparse_kernel<192><<<grid, kSpWarps * 32, 0, st>>>(a); break;
    case 256: sparse_kernel<256><<<grid, kSpWarps * 32, 0, st>>>(a); break;
    case 320: sparse_kernel<320><<<grid, kSpWarps * 32, 0, st>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace kvq
