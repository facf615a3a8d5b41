// Block index of a cache: mean keys of its blocks as int8 codes
// (kvq_block_index_update), and the selection of blocks by them (kvq_select_blocks).

#include <cooperative_groups.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_quant.cuh"

namespace kvq {
namespace {

namespace cg = cooperative_groups;

// ---------------------------------------------------------------------------
// Index update: a CTA per (block, KV head, sequence) or for several blocks, one warp per 32-channel
// quantization block.  Lane (j, s) of a warp adds the tokens j, j + 8, ... of its
// eight channels: q8_0 channels 8s .. 8s+7 (eight bytes of a row), the nibble formats
// 4s .. 4s+3 and 16+4s .. (four bytes).  Token order within a partial sum, then the
// eight partial sums in pairs by shuffles: the definition's order, so the codes do not
// depend on the launch.  Every product code * d is exact in fp32 (8 x 11 bits), so a
// fused multiply-add rounds as the sum of the two does.
//
// A byte becomes a float by a byte permute into 2^23's significand and one subtraction, two at a
// time; the loads of a warp's 64 tokens are all in flight at once, and those of the next tokens while
// a block is finished.  4 x 4 x 65536 tokens of head_dim 256 in q8_0, 289 MB in 51.9 us, 5.6 TB/s (84%
// of the card's measured copy rate); one block a launch and sequence 2.1 us.
// ---------------------------------------------------------------------------
// four bytes as exact floats, less `off`: a byte in the low bits of 2^23's significand
__device__ __forceinline__ void bytes_f32(uint32_t w, float off, float2& a, float2& b) {
  const float2 m = make_float2(-8388608.0f - off, -8388608.0f - off);
  a = __fadd2_rn(make_float2(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7440)),
                             __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7441))), m);
  b = __fadd2_rn(make_float2(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7442)),
                             __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7443))), m);
}

// what lane s reads of one token's quantization block
template <int KT>
struct Token {
  uint32_t w[KT == KVQ_TYPE_Q8_0 ? 2 : 1], hd, qh;
};
template <int KT, int D>
__device__ __forceinline__ Token<KT> load_token(const kvq_cache& c, long long row, int blk, int s) {
  constexpr int d = D, nb = D / 32;
  Token<KT> t;
  if constexpr (KT == KVQ_TYPE_Q8_0) {
    const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(c.k_qs) + row * d + 32 * blk + 8 * s);
    t.w[0] = w.x;
    t.w[1] = w.y;
  } else {
    t.w[0] = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(c.k_qs) + row * (d / 2) + 16 * blk + 4 * s);
  }
  if constexpr (type_has_qh(KT)) t.qh = static_cast<const uint32_t*>(c.k_qh)[row * nb + blk];
  if constexpr (type_has_min(KT)) t.hd = static_cast<const uint32_t*>(c.k_d)[row * nb + blk];
  else t.hd = static_cast<const uint16_t*>(c.k_d)[row * nb + blk];
  return t;
}
template <int KT>
__device__ __forceinline__ void add_token(const Token<KT>& t, int s, float2 (&acc)[4]) {
  float2 x[4];
  const float2 hd = __half22float2(u32_as_h2(t.hd)), dk = make_float2(hd.x, hd.x);
  if constexpr (KT == KVQ_TYPE_Q8_0) {
    bytes_f32(t.w[0], 128.0f, x[0], x[1]);
    bytes_f32(t.w[1], 128.0f, x[2], x[3]);
  } else {
    uint32_t lo = t.w[0] & 0x0F0F0F0Fu, hi = (t.w[0] >> 4) & 0x0F0F0F0Fu;
    if constexpr (type_has_qh(KT)) {
      // the K plane's order: channels 4s .. 4s+3 at bits 0, 1, 16, 17 of the word moved down by
      // 8 (s / 2) + 2 (s % 2), channels 16 further at 4 bits above; to bit 4 of their bytes
      const uint32_t h = t.qh >> (8 * (s >> 1) + 2 * (s & 1));
      lo |= ((h << 4) & 0x00100010u) | ((h << 11) & 0x10001000u);
      hi |= (h & 0x00100010u) | ((h << 7) & 0x10001000u);
    }
    const float off = type_has_min(KT) ? 0.0f : float(type_code_offset(KT));
    bytes_f32(lo, off, x[0], x[1]);
    bytes_f32(hi, off, x[2], x[3]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (type_has_min(KT)) acc[i] = __fadd2_rn(acc[i], __ffma2_rn(x[i], dk, make_float2(hd.y, hd.y)));
    else acc[i] = __ffma2_rn(x[i], dk, acc[i]);
  }
}

struct IndexArgs {
  kvq_cache c;
  kvq_block_index x;
  int n_last, nblk, pages_per_seq;
  DivU32 by_block, by_page;
};

template <int KT, int D>
__global__ void __launch_bounds__(D) index_update_kernel(IndexArgs a) {
  pdl_begin();
  __shared__ uint32_t s_max[2][10];
  constexpr int nw = D / 32;
  const kvq_cache& c = a.c;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int h = blockIdx.y, b = blockIdx.z, bt = a.x.block_tokens;
  const int n = min(max(c.seq_len[b], 0), c.max_ctx);
  const int nb = int(div_u32(uint32_t(n + bt - 1), a.by_block));
  const int bh = b * c.n_kv_heads + h;
  const int j = lane >> 2, s = lane & 3;
  int blk = (a.n_last ? int(div_u32(uint32_t(max(0, n - a.n_last)), a.by_block)) : 0) + int(blockIdx.x);
  if (blk >= nb) return;
  bool bad = false;
  // 64 positions (they lie in one page) from t0 of a block's m that are left
  Token<KT> t[8];
  bool have;
  auto load = [&](int t0, int m) {
    long long row = (long long)bh * c.max_ctx + t0;
    have = true;
    if (c.page_tokens) {
      const int i = int(div_u32(uint32_t(t0), a.by_page)), pg = c.page_table[(long long)b * a.pages_per_seq + i];
      have = pg >= 0 && pg < c.n_pages;
      row = ((long long)pg * c.n_kv_heads + h) * c.page_tokens + t0 - i * c.page_tokens;
      if (!have) { bad = true; return; }
    }
    row += j;
    if (m >= 64) {
#pragma unroll
      for (int i = 0; i < 8; ++i) t[i] = load_token<KT, D>(c, row + 8 * i, warp, s);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (8 * i + j < m) t[i] = load_token<KT, D>(c, row + 8 * i, warp, s);
    }
  };
  float2 acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = make_float2(0.0f, 0.0f);
  int u = 0, buf = 0;
  load(blk * bt, n - blk * bt);
  for (;;) {
    const int t0 = blk * bt, cnt = min(bt, n - t0), m = cnt - u;
    if (have) {
      if (m >= 64) {
#pragma unroll
        for (int i = 0; i < 8; ++i) add_token<KT>(t[i], s, acc);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (8 * i + j < m) add_token<KT>(t[i], s, acc);
      }
    }
    // the next 64 tokens are on their way while this block is finished
    const bool last = m <= 64;
    const int next = blk + (last ? int(gridDim.x) : 0);
    const bool more = next < nb;
    u = last ? 0 : u + 64;
    if (more) load(next * bt + u, min(bt, n - next * bt) - u);
    if (!last) continue;
    // the partial sums in pairs (j, j ^ 1), (j, j ^ 2), (j, j ^ 4), each lane keeping half of its
    // channels at every step: lane (j, s) ends with channel e of the eight
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i & 1 ? acc[i / 2].y : acc[i / 2].x;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int step = 0; step < 3; ++step) {
      const int half = 4 >> step;
      const bool up = (j >> step) & 1;
#pragma unroll
      for (int i = 0; i < half; ++i) {
        const float give = up ? v[i] : v[i + half], keep = up ? v[i + half] : v[i];
        v[i] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, give, 4 << step));
      }
    }
    const int e = 4 * (j & 1) + (j & 2) + (j >> 2);
    // (a product with the power of two 1 / count is the quotient)
    const float mean = (cnt & (cnt - 1)) == 0 ? __fmul_rn(v[0], __uint_as_float(uint32_t(127 - (31 - __clz(cnt))) << 23))
                                              : __fdiv_rn(v[0], float(cnt));
    uint32_t mx = __reduce_max_sync(0xffffffffu, __float_as_uint(fabsf(mean)));
    if (lane == 0) s_max[buf][warp] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < nw; ++w) mx = max(mx, s_max[buf][w]);
    buf ^= 1;
    const float scale = __fdiv_rn(__uint_as_float(mx), 127.0f);
    const long long at = (long long)bh * a.nblk + blk;
    if (threadIdx.x == 0) a.x.scales[at] = scale;
    const int ch = KT == KVQ_TYPE_Q8_0 ? 8 * s + e : e < 4 ? 4 * s + e : 12 + 4 * s + e;
    a.x.codes[at * D + 32 * warp + ch] = int8_t(scale > 0.0f ? __float2int_rn(__fdiv_rn(mean, scale)) : 0);
    if (!more) break;
    blk = next;
  }
  if (bad && threadIdx.x == 0) atomicOr(c.status, KVQ_DEV_ERR_PAGE);
}

// ---------------------------------------------------------------------------
// Selection: a cluster of CTAs per (KV head, sequence).  The queries of the group are
// rotated and coded, 16 blocks x 8 heads at a time scored on the tensor cores (int8 mma:
// integers, so every order gives the same sum), the scores collected in the first CTA's
// shared memory as order-preserving integers; there the n_select-th largest is found by
// histograms of ever finer bins and the blocks at or above it are written in order.
//
// Bound by latency: 32 x 8 rows of up to 128 blocks 5.5 us; 4 rows of 16384 blocks 15.4 us, of
// which scoring takes about 5 and the one CTA that selects 6.  Tried for those and not kept: every
// CTA of the cluster keeping its own keys and searching with all the others' histograms (20.4 us:
// five cluster barriers and reads of all histograms by all), fp16 mma over the codes as subnormals
// (1.5 us slower: int8 mma is slow here, but that wants more registers than 1024 threads have), a
// histogram over equal steps of the score with a list of the one bin's keys (0.5 slower), clusters of
// 16 (0.4 slower).
// ---------------------------------------------------------------------------
constexpr int kBins = 2048;
constexpr int kMaxSelCluster = 8;
constexpr int kFewBlocks = 256;  // up to these a thread ranks each block
constexpr int kSmallIndex = 2048;  // up to these CTAs of 256 threads

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
int sel_q_bytes(int group) { return (group + 7) / 8 * 8 * (sel_pitch<D>() + 4); }  // (the API checks the sum, see there)

template <int D, int kThreads>
__global__ void __launch_bounds__(kThreads) select_kernel(SelArgs a) {
  constexpr int G = (D & (D - 1)) == 0 ? D : 64;
  constexpr int E = D / 32, SEG = D / 64, QP = sel_pitch<D>(), kW = kThreads / 32;
  extern __shared__ __align__(16) uint8_t smem[];
  pdl_begin();
  cg::cluster_group cl = cg::this_cluster();
  const int S = int(cl.num_blocks()), rank = int(cl.block_rank());
  cl.barrier_arrive();  // (no CTA touches the first one's shared memory before it runs)
  const int heads8 = (a.group + 7) / 8 * 8;
  uint8_t* s_q = smem;                                                  // [heads8][QP]
  float* s_qs = reinterpret_cast<float*>(smem + heads8 * QP);           // [heads8]
  uint32_t* s_key = reinterpret_cast<uint32_t*>(s_qs + heads8);         // [blocks of the sequence] (first CTA's)
  __shared__ uint32_t s_hist[kBins];
  __shared__ int s_warp[2][32];
  __shared__ uint32_t s_lim[2][32];
  __shared__ uint32_t s_range[kMaxSelCluster][2];  // smallest and largest key of each CTA (first CTA's)
  __shared__ int s_bin, s_above, s_in;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row = blockIdx.x / S, h = row % a.n_kv_heads, b = row / a.n_kv_heads;
  const long long bh = (long long)b * a.n_kv_heads + h;
  int32_t* sel = a.sel + bh * a.n_select;
  const int n = min(max(a.seq_len[b], 0), a.max_ctx);
  const int nb = int(((long long)n + a.block_tokens - 1) / a.block_tokens);
  if (nb <= a.n_select) {  // all of them
    if (rank == 0)
      for (int i = tid; i < a.n_select; i += kThreads) sel[i] = i < nb ? i : -1;
    cl.barrier_wait();
    return;
  }
  // ---- the first 16 blocks' codes of a warp are on their way while the queries are coded: lane
  // (g, tig) loads 16 channels of rows g and g + 8 at a time
  const int g = lane >> 2, tig = lane & 3;
  const int8_t* codes = a.codes + bh * a.nblk * D;
  const float* scales = a.scales + bh * a.nblk;
  uint4 xa[SEG], xb[SEG];
  auto load = [&](int r0) {
    const int ra = min(r0 + g, nb - 1), rb = min(r0 + g + 8, nb - 1);
#pragma unroll
    for (int s = 0; s < SEG; ++s) {
      xa[s] = *reinterpret_cast<const uint4*>(codes + (long long)ra * D + 64 * s + 16 * tig);
      xb[s] = *reinterpret_cast<const uint4*>(codes + (long long)rb * D + 64 * s + 16 * tig);
    }
  };
  const int step = 16 * kW * S;
  int r0 = 16 * (rank * kW + warp);
  if (r0 < nb) load(r0);
  // ---- queries: rotate, code
  for (int i = warp; i < heads8; i += kW) {
    float v[E];
#pragma unroll
    for (int e = 0; e < E; ++e) v[e] = 0.0f;
    if (i < a.group) {
      const size_t qrow = ((size_t)b * a.n_q_heads + (size_t)h * a.group + i) * D;
#pragma unroll
      for (int gi = 0; gi < D / G; ++gi) load_vals<G / 32>(a.q, a.q_dtype, qrow + gi * G + lane * (G / 32), v + gi * (G / 32));
    }
    if (a.rot_k) {
      warp_fwht<D, G>(v, lane);
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = __fmul_rn(v[e], inv_sqrt_group<G>());
    }
    uint32_t mx = 0;  // (as integers: a NaN is above every number, and makes the head's scores NaN)
#pragma unroll
    for (int e = 0; e < E; ++e) mx = max(mx, __float_as_uint(fabsf(v[e])));
    mx = __reduce_max_sync(0xffffffffu, mx);
    const float sq = __fdiv_rn(__uint_as_float(mx), 127.0f);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int code = sq > 0.0f ? __float2int_rn(__fdiv_rn(v[e], sq)) : 0;
      s_q[i * QP + fwht_channel<D, G>(lane, e)] = uint8_t(code);
    }
    if (lane == 0) s_qs[i] = sq;
  }
  __syncthreads();
  cl.barrier_wait();
  uint32_t* keys = S > 1 ? cl.map_shared_rank(s_key, 0) : s_key;
  // ---- scores: two mma take the 16 channels of a lane as their 32-wide inner index, in an
  // order of their own that is the query's too
  uint32_t lo = 0xFFFFFFFFu, hi = 0;
  for (; r0 < nb; r0 += step) {
    float ma = __uint_as_float(0x7FFFFFFFu), mb = ma;  // NaN: fmaxf keeps it only where every head's score is NaN
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
    if (r0 + step < nb) load(r0 + step);
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
        // (blocks taken in any case lie above every score, outside the range that is searched)
        const bool forced = r < a.n_first || r >= nb - a.n_last;
        keys[r] = forced ? 0xFFFFFFFFu : key;
        if (!forced) {
          lo = min(lo, key);
          hi = max(hi, key);
        }
      }
    }
  }
  lo = __reduce_min_sync(0xffffffffu, lo);
  hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) { s_lim[0][warp] = lo; s_lim[1][warp] = hi; }
  __syncthreads();
  if (warp == 0) {
    lo = __reduce_min_sync(0xffffffffu, lane < kW ? s_lim[0][lane] : 0xFFFFFFFFu);
    hi = __reduce_max_sync(0xffffffffu, lane < kW ? s_lim[1][lane] : 0u);
    if (lane == 0) {
      uint32_t* o = S > 1 ? cl.map_shared_rank(&s_range[0][0], 0) : &s_range[0][0];
      o[2 * rank] = lo;
      o[2 * rank + 1] = hi;
    }
  }
  if (S > 1) cl.sync(); else __syncthreads();
  if (rank != 0) return;
  lo = 0xFFFFFFFFu;
  hi = 0;
  for (int r = 0; r < S; ++r) {
    lo = min(lo, s_range[r][0]);
    hi = max(hi, s_range[r][1]);
  }
  if constexpr (kThreads == kFewBlocks) {
    if (nb <= kFewBlocks) {
      // few blocks: a thread per block counts the keys above its own and those equal to it
      const uint32_t k = tid < nb ? s_key[tid] : 0u;
      int gt = 0, ge = 0, ties_before = 0;
      for (int i = 0; i < nb; ++i) {
        const uint32_t o = s_key[i];
        gt += o > k;
        ge += o >= k;
      }
      const bool tie = tid < nb && gt < a.n_select && ge > a.n_select;  // equal keys on both sides of the border
      if (tie)
        for (int i = 0; i < tid; ++i) ties_before += s_key[i] == k;
      const bool in = tid < nb && gt + ties_before < a.n_select && (tie || ge <= a.n_select);
      const unsigned m = __ballot_sync(0xffffffffu, in);
      if (lane == 0) s_warp[0][warp] = __popc(m);
      __syncthreads();
      const int at = int(__reduce_add_sync(0xffffffffu, lane < warp ? unsigned(s_warp[0][lane]) : 0u));
      if (in) sel[at + __popc(m & ((1u << lane) - 1u))] = tid;
      return;
    }
  }
  // ---- the n_select-th largest key: bins of 2^sh keys over [lo, hi], then the same in the
  // bin that holds it, until a bin is one key wide or taken whole
  int need = a.n_select - a.n_first - a.n_last;  // keys to take from [lo, hi]; all above hi are taken
  bool ties = false;
  if (need == 0) lo = 0xFFFFFFFFu;
  while (need) {
    const uint32_t range = hi - lo;
    const int sh = range < kBins ? 0 : 32 - __clz(range) - 11;
    for (int i = tid; i < kBins; i += kThreads) s_hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < nb; i += kThreads) {
      const uint32_t k = s_key[i];
      if (k >= lo && k <= hi) atomicAdd(&s_hist[(k - lo) >> sh], 1u);
    }
    __syncthreads();
    constexpr int BPT = kBins / kThreads;  // bins per thread, from the top
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
    int above = inc - sum + int(__reduce_add_sync(0xffffffffu, lane < warp ? unsigned(s_warp[0][lane]) : 0u));
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
  // ---- the blocks above, and of those equal the first `need`, in order: a warp takes a run of
  // blocks, 32 at a time, and its lane i keeps the i-th (and 32 + i-th) 32 blocks' bits
  constexpr int kWords = ((kThreads == 1024 ? kMaxIndexBlocks : kSmallIndex) / kW + 1023) / 1024;
  const int per = ((nb + kW - 1) / kW + 31) / 32 * 32, i0 = warp * per, i1 = min(nb, i0 + per);
  unsigned mg[kWords], mt[kWords];
#pragma unroll
  for (int w = 0; w < kWords; ++w) mg[w] = mt[w] = 0u;
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    const int j0 = i0 + 1024 * w;
#pragma unroll 4
    for (int it = 0; it < 32; ++it) {
      if (j0 + 32 * it >= i1) break;
      const int i = j0 + 32 * it + lane;
      const uint32_t k = i < i1 ? s_key[i] : 0u;
      const bool in = i < i1 && k >= lo;
      const unsigned m = __ballot_sync(0xffffffffu, in);
      if (lane == it) mg[w] = m;
      if (ties) {
        const unsigned t = __ballot_sync(0xffffffffu, in && k == lo);
        if (lane == it) mt[w] = t;
      }
    }
  }
  int bg[kWords], be[kWords], gt = 0, eq = 0;  // taken and equal blocks of the warp before lane's word w
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    mg[w] &= ~mt[w];
    int g1 = __popc(mg[w]), e1 = __popc(mt[w]);
    bg[w] = gt - g1;
    be[w] = eq - e1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, g1, o), z = __shfl_up_sync(0xffffffffu, e1, o);
      if (lane >= o) { g1 += y; e1 += z; }
    }
    bg[w] += g1;
    be[w] += e1;
    gt += __shfl_sync(0xffffffffu, g1, 31);
    eq += __shfl_sync(0xffffffffu, e1, 31);
  }
  if (lane == 0) { s_warp[0][warp] = gt; s_warp[1][warp] = eq; }
  __syncthreads();
  const int wg = int(__reduce_add_sync(0xffffffffu, lane < warp ? unsigned(s_warp[0][lane]) : 0u));
  const int we = int(__reduce_add_sync(0xffffffffu, lane < warp ? unsigned(s_warp[1][lane]) : 0u));
#pragma unroll
  for (int w = 0; w < kWords; ++w) {
    const int e0 = we + be[w];
    unsigned m = mt[w];
    for (int t = __popc(m) - max(need - e0, 0); t > 0; --t) m &= ~(0x80000000u >> __clz(m));  // the last ties stay out
    int at = wg + bg[w] + min(e0, need);
    for (m |= mg[w]; m; m &= m - 1) sel[at++] = i0 + 1024 * w + 32 * lane + __ffs(m) - 1;
  }
}

template <int D, int kThreads>
cudaError_t select_t(const SelArgs& a, int batch, cudaStream_t st) {
  const int bytes = sel_q_bytes<D>(a.group) + 4 * a.nblk;
  auto kern = select_kernel<D, kThreads>;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), bytes);
  if (e != cudaSuccess) return e;
  // CTAs per row while each has 16 blocks per warp to score and the GPU has SMs for them
  const long long rows = (long long)a.n_kv_heads * batch;
  const int sms = device_sm_count();
  const int S = int(std::max<long long>(1, std::min<long long>({kMaxSelCluster, (sms > 0 ? sms : 148) / rows,
                                                               a.nblk / (16 * kThreads / 32)})));
  return launch_dependent(kern, unsigned(rows * S), kThreads, bytes, st, S, a);
}
template <int D>
cudaError_t select_d(const SelArgs& a, int batch, cudaStream_t st) {
  // few blocks: barriers of few warps
  return a.nblk <= kSmallIndex ? select_t<D, kFewBlocks>(a, batch, st) : select_t<D, 1024>(a, batch, st);
}

}  // namespace

cudaError_t launch_block_index_update(const kvq_cache& c, const kvq_block_index& x, int n_last, cudaStream_t st) {
  const int bt = x.block_tokens;
  const int nblk = int((c.max_ctx + (long long)bt - 1) / bt);
  // blocks that can hold any of the last n_last tokens
  const int nx = n_last ? int(std::min<long long>(nblk, ((long long)n_last + bt - 2) / bt + 1)) : nblk;
  // Where the device is full many times over a CTA takes three blocks, so that the loads of one run
  // while another is finished: 16384 blocks of head_dim 256 51.9 us (2: 52.4, 4: 52.4, 8: 53.5, 16:
  // 55.8, 1: 56.4).  Few blocks have a CTA each.
  const long long all = (long long)nx * c.n_kv_heads * c.batch;
  const int sms = device_sm_count();
  const int per = all > 32LL * (sms > 0 ? sms : 148) ? 3 : 1;
  const dim3 grid((nx + per - 1) / per, c.n_kv_heads, c.batch);
  const IndexArgs a{c, x, n_last, nblk, c.page_tokens ? c.max_ctx / c.page_tokens : 0, make_divu32(uint32_t(bt)),
                    make_divu32(uint32_t(std::max(1, c.page_tokens)))};
#define KVQ_INDEX(KT, D) return launch_dependent(index_update_kernel<KT, D>, grid, D, 0, st, 1, a)
#define KVQ_INDEX_KT(KT)                        \
  case KT:                                      \
    if (c.head_dim == 64) KVQ_INDEX(KT, 64);    \
    else if (c.head_dim == 128) KVQ_INDEX(KT, 128); \
    else if (c.head_dim == 192) KVQ_INDEX(KT, 192); \
    else if (c.head_dim == 256) KVQ_INDEX(KT, 256); \
    else KVQ_INDEX(KT, 320);                    \
    break;
  switch (c.k_type) {
    KVQ_INDEX_KT(KVQ_TYPE_Q4_0)
    KVQ_INDEX_KT(KVQ_TYPE_Q5_0)
    KVQ_INDEX_KT(KVQ_TYPE_Q8_0)
    KVQ_INDEX_KT(KVQ_TYPE_Q4_1)
    KVQ_INDEX_KT(KVQ_TYPE_Q5_1)
  }
#undef KVQ_INDEX_KT
#undef KVQ_INDEX
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
