// Block index of a cache: mean keys of its blocks as int8 codes
// (kvq_block_index_update), and the selection of blocks by them (kvq_select_blocks).

#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_quant.cuh"

namespace kvq {
namespace {

// ---------------------------------------------------------------------------
// Index update: one CTA per (block, KV head, sequence), one warp per 32-channel
// quantization block.  Lane (j, s) of a warp adds the tokens j, j + 8, ... of its
// eight channels: q8_0 channels 8s .. 8s+7 (eight bytes of a row), the nibble formats
// 4s .. 4s+3 and 16+4s .. (four bytes).  Token order within a partial sum, then the
// eight partial sums in pairs by shuffles: the definition's order, so the codes do not
// depend on the launch.  Every product code * d is exact in fp32 (8 x 11 bits), so a
// fused multiply-add rounds as the sum of the two does.
// ---------------------------------------------------------------------------
template <int KT>
__device__ __forceinline__ void add_token(const kvq_cache& c, long long row, int blk, int s, float (&acc)[8]) {
  const int d = c.head_dim, nb = d / 32;
  if constexpr (KT == KVQ_TYPE_Q8_0) {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.k_qs) + row * d + 32 * blk + 8 * s);
    const float dk = __half2float(static_cast<const __half*>(c.k_d)[row * nb + blk]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int u = ((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 255;
      acc[i] = fmaf(float(u - 128), dk, acc[i]);
    }
  } else {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(c.k_qs) + row * (d / 2) +
                                                          16 * blk + 4 * s);
    uint32_t hb = 0;
    if constexpr (type_has_qh(KT)) hb = qh_k_to_gguf(static_cast<const uint32_t*>(c.k_qh)[row * nb + blk]);
    float dk, lo = 0.0f;
    if constexpr (type_has_min(KT)) {
      const float2 f = __half22float2(static_cast<const __half2*>(c.k_d)[row * nb + blk]);
      dk = f.x;
      lo = f.y;
    } else {
      dk = __half2float(static_cast<const __half*>(c.k_d)[row * nb + blk]);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int code = (w >> (8 * (i & 3) + (i < 4 ? 0 : 4))) & 15;
      if constexpr (type_has_qh(KT)) code |= ((hb >> (4 * s + (i & 3) + (i < 4 ? 0 : 16))) & 1) << 4;
      if constexpr (type_has_min(KT)) acc[i] = __fadd_rn(acc[i], fmaf(float(code), dk, lo));
      else acc[i] = fmaf(float(code - type_code_offset(KT)), dk, acc[i]);
    }
  }
}

template <int KT>
__global__ void __launch_bounds__(320) index_update_kernel(kvq_cache c, kvq_block_index x, int n_last, int nblk) {
  __shared__ float s_max[10];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  const int h = blockIdx.y, b = blockIdx.z, bt = x.block_tokens, d = c.head_dim;
  const int n = min(max(c.seq_len[b], 0), c.max_ctx);
  const long long j0 = n_last ? max(0, n - n_last) / bt : 0;
  const long long blk = j0 + blockIdx.x;
  if (blk * bt >= n) return;
  const RowMap rm = row_map(c);
  const int t0 = int(blk * bt), cnt = min(bt, n - t0);
  const int j = lane >> 2, s = lane & 3;
  float acc[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
  bool bad = false;
  for (int u = 0; u < cnt; u += 64) {  // 64 positions lie in one page
    const long long row = body_row(rm, b, h, t0 + u);
    if (row < 0) { bad = true; continue; }
    const int m = min(64, cnt - u);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (8 * i + j < m) add_token<KT>(c, row + 8 * i + j, warp, s, acc);
  }
  if (bad && threadIdx.x == 0) atomicOr(c.status, KVQ_DEV_ERR_PAGE);
  float mean[8], mx = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float v = acc[i];
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
    mean[i] = __fdiv_rn(v, float(cnt));
    mx = fmaxf(mx, fabsf(mean[i]));
  }
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
  mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
  if (lane == 0) s_max[warp] = mx;
  __syncthreads();
  for (int w = 0; w < nw; ++w) mx = fmaxf(mx, s_max[w]);
  const float scale = __fdiv_rn(mx, 127.0f);
  const long long e = ((long long)b * c.n_kv_heads + h) * nblk + blk;
  if (threadIdx.x == 0) x.scales[e] = scale;
  if (j == 0) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int code = scale > 0.0f ? __float2int_rn(__fdiv_rn(mean[i], scale)) : 0;
      w[i >> 2] |= (uint32_t(code) & 255u) << (8 * (i & 3));
    }
    uint8_t* dst = reinterpret_cast<uint8_t*>(x.codes) + e * d + 32 * warp;
    if constexpr (KT == KVQ_TYPE_Q8_0) {
      *reinterpret_cast<uint2*>(dst + 8 * s) = make_uint2(w[0], w[1]);
    } else {
      *reinterpret_cast<uint32_t*>(dst + 4 * s) = w[0];
      *reinterpret_cast<uint32_t*>(dst + 16 + 4 * s) = w[1];
    }
  }
}

// ---------------------------------------------------------------------------
// Selection: one CTA per (KV head, sequence).  The queries of the group are rotated
// and coded, 16 blocks x 8 heads at a time scored on the tensor cores (int8 mma:
// integers, so every order gives the same sum), the scores kept in shared memory as
// order-preserving integers; then the n_select-th largest is found by histograms of
// ever finer bins and the blocks at or above it are written in order.
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 512;
constexpr int kBins = 2048;

// D = A (16x32 int8, row) * B (32x8 int8, col) + C, int32
__device__ __forceinline__ void mma16832_s8(int (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

struct SelArgs {
  const int32_t* seq_len;
  const int8_t* codes;
  const float* scales;
  const void* q;
  int32_t* sel;
  int q_dtype, n_q_heads, n_kv_heads, group, block_tokens, nblk, max_ctx, n_first, n_last, n_select, rot_k;
};

// bytes of coded queries: groups of eight heads, rows padded by 16 so that the eight
// rows of a fragment load fall into different banks
template <int D>
constexpr int sel_pitch() { return D + 16; }
template <int D>
int sel_q_bytes(int group) { return (group + 7) / 8 * 8 * (sel_pitch<D>() + 4); }

template <int D>
__global__ void __launch_bounds__(kSelThreads) select_kernel(SelArgs a) {
  constexpr int G = (D & (D - 1)) == 0 ? D : 64;
  constexpr int E = D / 32, SEG = D / 64, QP = sel_pitch<D>();
  extern __shared__ __align__(16) uint8_t smem[];
  const int heads8 = (a.group + 7) / 8 * 8;
  uint8_t* s_q = smem;                                                  // [heads8][QP]
  float* s_qs = reinterpret_cast<float*>(smem + heads8 * QP);           // [heads8]
  uint32_t* s_key = reinterpret_cast<uint32_t*>(s_qs + heads8);         // [blocks of the sequence]
  __shared__ uint32_t s_hist[kBins];
  __shared__ int s_warp[2][kSelThreads / 32];
  __shared__ uint32_t s_lim[2];
  __shared__ int s_bin, s_above, s_in;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x, b = blockIdx.y;
  const long long bh = (long long)b * a.n_kv_heads + h;
  int32_t* sel = a.sel + bh * a.n_select;
  const int n = min(max(a.seq_len[b], 0), a.max_ctx);
  const int nb = int(((long long)n + a.block_tokens - 1) / a.block_tokens);
  if (nb <= a.n_select) {  // all of them
    for (int i = tid; i < a.n_select; i += kSelThreads) sel[i] = i < nb ? i : -1;
    return;
  }
  // ---- queries: rotate, code
  for (int i = warp; i < heads8; i += kSelThreads / 32) {
    float v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = 0.0f;
    if (i < a.group) {
      const size_t row = ((size_t)b * a.n_q_heads + (size_t)h * a.group + i) * D;
#pragma unroll
      for (int gi = 0; gi < D / G; ++gi) load_vals<G / 32>(a.q, a.q_dtype, row + gi * G + lane * (G / 32), v + gi * (G / 32));
    }
    if (a.rot_k) {
      warp_fwht<D, G>(v, lane);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = __fmul_rn(v[e], inv_sqrt_group<G>());
    }
    float mx = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) mx = fmaxf(mx, fabsf(v[e]));
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float sq = __fdiv_rn(mx, 127.0f);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int code = sq > 0.0f ? __float2int_rn(__fdiv_rn(v[e], sq)) : 0;
      s_q[i * QP + fwht_channel<D, G>(lane, e)] = uint8_t(code);
    }
    if (lane == 0) s_qs[i] = sq;
  }
  if (tid == 0) { s_lim[0] = 0xFFFFFFFFu; s_lim[1] = 0; }
  __syncthreads();
  // ---- scores: lane (g, tig) loads 16 channels of rows g and g + 8 at a time; two mma
  // take them as their 32-wide inner index in an order of their own, the query's too
  const int g = lane >> 2, tig = lane & 3;
  const int8_t* codes = a.codes + bh * a.nblk * D;
  const float* scales = a.scales + bh * a.nblk;
  uint32_t lo = 0xFFFFFFFFu, hi = 0;
  for (int r0 = 16 * warp; r0 < nb; r0 += 16 * (kSelThreads / 32)) {
    const int ra = min(r0 + g, nb - 1), rb = min(r0 + g + 8, nb - 1);
    uint4 xa[SEG], xb[SEG];
#pragma unroll
    for (int s = 0; s < SEG; ++s) {
      xa[s] = *reinterpret_cast<const uint4*>(codes + (long long)ra * D + 64 * s + 16 * tig);
      xb[s] = *reinterpret_cast<const uint4*>(codes + (long long)rb * D + 64 * s + 16 * tig);
    }
    float ma = -INFINITY, mb = -INFINITY;
    for (int h0 = 0; h0 < a.group; h0 += 8) {
      int acc[4] = {0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < SEG; ++s) {
        const uint4 q = *reinterpret_cast<const uint4*>(s_q + (h0 + g) * QP + 64 * s + 16 * tig);
        mma16832_s8(acc, xa[s].x, xb[s].x, xa[s].y, xb[s].y, q.x, q.y);
        mma16832_s8(acc, xa[s].z, xb[s].z, xa[s].w, xb[s].w, q.z, q.w);
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int hh = h0 + 2 * tig + e;
        if (hh < a.group) {
          ma = fmaxf(ma, __fmul_rn(float(acc[e]), s_qs[hh]));
          mb = fmaxf(mb, __fmul_rn(float(acc[2 + e]), s_qs[hh]));
        }
      }
    }
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) {
      ma = fmaxf(ma, __shfl_xor_sync(0xffffffffu, ma, o));
      mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, o));
    }
    if (tig < 2) {
      const int r = r0 + g + 8 * tig;
      if (r < nb) {
        // (scale >= 0, so the product keeps the order of the heads' maximum; + 0 makes -0 equal to 0)
        const float sc = __fadd_rn(__fmul_rn(tig ? mb : ma, scales[r]), 0.0f);
        const uint32_t u = __float_as_uint(sc);
        uint32_t key = (u >> 31) ? ~u : (u | 0x80000000u);
        if (sc != sc) key = 0;
        if (r < a.n_first || r >= nb - a.n_last) key = 0xFFFFFFFFu;
        s_key[r] = key;
        lo = min(lo, key);
        hi = max(hi, key);
      }
    }
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) { atomicMin(&s_lim[0], lo); atomicMax(&s_lim[1], hi); }
  __syncthreads();
  lo = s_lim[0];
  hi = s_lim[1];
  // ---- the n_select-th largest key: bins of 2^sh keys over [lo, hi], then the same in the
  // bin that holds it, until a bin is one key wide or taken whole
  int need = a.n_select;   // keys to take from [lo, hi]; all above hi are taken
  bool ties = false;
  for (;;) {
    const uint32_t range = hi - lo;
    const int sh = range < kBins ? 0 : 32 - __clz(range) - 11;
    for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < nb; i += kSelThreads) {
      const uint32_t k = s_key[i];
      if (k >= lo && k <= hi) atomicAdd(&s_hist[(k - lo) >> sh], 1u);
    }
    __syncthreads();
    constexpr int BPT = kBins / kSelThreads;  // bins per thread, from the top
    int cnt[BPT], sum = 0;
#pragma unroll
    for (int i = 0; i < BPT; ++i) {
      cnt[i] = int(s_hist[kBins - 1 - (tid * BPT + i)]);
      sum += cnt[i];
    }
    int inc = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    if (lane == 31) s_warp[0][warp] = inc;
    __syncthreads();
    int above = inc - sum;
    for (int w = 0; w < warp; ++w) above += s_warp[0][w];
#pragma unroll
    for (int i = 0; i < BPT; ++i) {
      if (above < need && above + cnt[i] >= need) { s_bin = kBins - 1 - (tid * BPT + i); s_above = above; s_in = cnt[i]; }
      above += cnt[i];
    }
    __syncthreads();
    lo += uint32_t(s_bin) << sh;
    need -= s_above;
    const bool whole = s_in == need;
    hi = min(hi, lo + ((1u << sh) - 1u));
    if (whole) break;
    if (sh == 0) { ties = true; break; }
  }
  // ---- the blocks above, and of those equal the first `need`, in order
  const int per = (nb + kSelThreads - 1) / kSelThreads;
  const int i0 = min(nb, tid * per), i1 = min(nb, i0 + per);
  int gt = 0, eq = 0;
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = s_key[i];
    if (ties && k == lo) ++eq;
    else if (k >= lo) ++gt;
  }
  int ig = gt, ie = eq;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int yg = __shfl_up_sync(0xffffffffu, ig, o), ye = __shfl_up_sync(0xffffffffu, ie, o);
    if (lane >= o) { ig += yg; ie += ye; }
  }
  if (lane == 31) { s_warp[0][warp] = ig; s_warp[1][warp] = ie; }
  __syncthreads();
  int bg = ig - gt, be = ie - eq;
  for (int w = 0; w < warp; ++w) { bg += s_warp[0][w]; be += s_warp[1][w]; }
  for (int i = i0; i < i1; ++i) {
    const uint32_t k = s_key[i];
    if (ties && k == lo) {
      if (be < need) sel[bg + be] = i;
      ++be;
    } else if (k >= lo) {
      sel[bg + min(be, need)] = i;
      ++bg;
    }
  }
}

template <int D>
cudaError_t select_d(const SelArgs& a, int batch, cudaStream_t st) {
  const int bytes = sel_q_bytes<D>(a.group) + 4 * a.nblk;
  auto kern = select_kernel<D>;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), bytes);
  if (e != cudaSuccess) return e;
  kern<<<dim3(a.n_kv_heads, batch), kSelThreads, bytes, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_index_update(const kvq_cache& c, const kvq_block_index& x, int n_last, cudaStream_t st) {
  const int bt = x.block_tokens;
  const int nblk = int((c.max_ctx + (long long)bt - 1) / bt);
  // blocks that can hold any of the last n_last tokens
  const int nx = n_last ? int(std::min<long long>(nblk, ((long long)n_last + bt - 2) / bt + 1)) : nblk;
  const dim3 grid(nx, c.n_kv_heads, c.batch);
  const int threads = c.head_dim;
  switch (c.k_type) {
    case KVQ_TYPE_Q4_0: index_update_kernel<KVQ_TYPE_Q4_0><<<grid, threads, 0, st>>>(c, x, n_last, nblk); break;
    case KVQ_TYPE_Q5_0: index_update_kernel<KVQ_TYPE_Q5_0><<<grid, threads, 0, st>>>(c, x, n_last, nblk); break;
    case KVQ_TYPE_Q8_0: index_update_kernel<KVQ_TYPE_Q8_0><<<grid, threads, 0, st>>>(c, x, n_last, nblk); break;
    case KVQ_TYPE_Q4_1: index_update_kernel<KVQ_TYPE_Q4_1><<<grid, threads, 0, st>>>(c, x, n_last, nblk); break;
    default: index_update_kernel<KVQ_TYPE_Q5_1><<<grid, threads, 0, st>>>(c, x, n_last, nblk); break;
  }
  return cudaGetLastError();
}

cudaError_t launch_select_blocks(const kvq_cache& c, Rot rot, const kvq_block_index& x, const void* q, int q_dtype,
                                 int n_q_heads, int n_first, int n_last, int n_select, int32_t* sel, cudaStream_t st) {
  SelArgs a{};
  a.seq_len = c.seq_len; a.codes = x.codes; a.scales = x.scales; a.q = q; a.sel = sel;
  a.q_dtype = q_dtype; a.n_q_heads = n_q_heads; a.n_kv_heads = c.n_kv_heads; a.group = n_q_heads / c.n_kv_heads;
  a.block_tokens = x.block_tokens;
  a.nblk = int((c.max_ctx + (long long)x.block_tokens - 1) / x.block_tokens);
  a.max_ctx = c.max_ctx;
  a.n_first = n_first; a.n_last = n_last; a.n_select = n_select; a.rot_k = rot.k;
  switch (c.head_dim) {
    case 64: return select_d<64>(a, c.batch, st);
    case 128: return select_d<128>(a, c.batch, st);
    case 192: return select_d<192>(a, c.batch, st);
    case 256: return select_d<256>(a, c.batch, st);
    case 320: return select_d<320>(a, c.batch, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
