// Attention of packed rows of new tokens (kvq_chunk_attention): the plan of a call, and the merge of items in several pieces.
//
// Both are bound by latency: the plan (one CTA, 4 to 6 us) by its scans' barriers, the merge (7 us for 32 sequences of one token,
// 16 for 2 x 4096 rows, 40 MB) by a chain of five loads -- header, item, rows, parts.
#include "kvq_chunk.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>


namespace kvq {
namespace {

constexpr int kPlanThreads = 256;  // (1024: its barriers cost a call 0.5 to 1.5 us more)
constexpr int kPlanItems = 2048;  // whose beginnings are kept in shared memory: a search there, not in L2, once for all kernels (2 us each)

// ---- plan --------------------------------------------------------------------------------------

// Inclusive sums over a block of kPlanThreads; s: 32 values.
__device__ __forceinline__ long long block_sums(long long v, long long* s, long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();
  if (lane == 31) s[warp] = v;
  __syncthreads();
  long long w = lane < kPlanThreads / 32 ? s[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const long long before = __shfl_sync(0xffffffffu, w, warp == 0 ? 0 : warp - 1);
  return v + (warp == 0 ? 0 : before);
}

__global__ void __launch_bounds__(kPlanThreads, 1) chunk_plan_kernel(ChunkArgs a) {
  pdl_begin();
  __shared__ long long s_sum[32], s_at[kPlanItems];
  __shared__ int s_bad;
  const int tid = threadIdx.x, B = a.c.batch;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  bool bad = false;
  for (int b = tid; b < B; b += kPlanThreads) {
    const int r0 = a.row_start[b], r1 = a.row_start[b + 1];
    bad |= r0 < 0 || r1 < r0 || r1 > a.n_rows;
  }
  if (bad) s_bad = 1;
  __syncthreads();
  if (s_bad) {
    if (tid == 0) {
      atomicOr(a.c.status, KVQ_DEV_ERR_ROW);
      *a.head = ChunkHeader{0, 0, 0, 0, 0, 0};
    }
    return;
  }
  // items of each sequence
  long long items = 0, total;
  bool late = false;
  for (int b0 = 0; b0 < B; b0 += kPlanThreads) {
    const int b = b0 + tid;
    long long n = 0;
    if (b < B) {
      const int m = a.row_start[b + 1] - a.row_start[b];
      n = ((long long)m * a.group + a.m - 1) / a.m;
      late |= m > min(max(a.c.seq_len[b], 0), a.c.max_ctx);
    }
    const long long at = items + block_sums(n, s_sum, total) - n;
    if (b < B) a.tiles0[b] = int(at);
    items += total;
  }
  if (tid == 0) a.tiles0[B] = int(items);
  if (late) atomicOr(a.c.status, KVQ_DEV_ERR_PREFILL_RANGE);
  __syncthreads();
  // each item's keys and tiles
  long long length = 0;
  for (int i0 = 0; i0 < int(items); i0 += kPlanThreads) {
    const int i = i0 + tid;
    ChunkItem it{};
    long long cost = 0;
    if (i < int(items)) {
      int lo = 0, hi = B - 1;  // the last sequence whose items begin at or before i (the one with items among equals)
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.tiles0[mid] <= i) lo = mid; else hi = mid - 1;
      }
      it.b = lo;
      const int row0 = a.row_start[lo], m = a.row_start[lo + 1] - row0, n = min(max(a.c.seq_len[lo], 0), a.c.max_ctx);
      it.r0 = (i - a.tiles0[lo]) * a.m;
      it.rows = min(a.m, m * a.group - it.r0);
      const int t0 = int(div_u32(uint32_t(it.r0), a.by_group)), t1 = int(div_u32(uint32_t(it.r0 + it.rows - 1), a.by_group));
      int k0 = 0x7fffffff, k1 = 0;
      if (!a.mod.first_key) {
        const ChunkSpan s0 = chunk_span(a, lo, n, row0, m, max(t0, m - n)), s1 = chunk_span(a, lo, n, row0, m, t1);
        if (t1 >= m - n) { k0 = s0.lo; k1 = s1.hi; }
      } else {
        for (int t = t0; t <= t1; ++t) {
          const ChunkSpan s = chunk_span(a, lo, n, row0, m, t);
          if (s.hi > s.lo) { k0 = min(k0, s.lo); k1 = max(k1, s.hi); }
        }
      }
      if (k1 > k0) {
        it.lo = k0;
        it.hi = k1;
        const int T = a.c.tail_len, body_end = n - T;
        const int be = min(k1, body_end), ts = max(k0, body_end);
        if (be > k0) it.n_body = (be - k0 / a.tile * a.tile + a.tile - 1) / a.tile;
        if (T > 0 && k1 > ts) {
          const int slot = ts - int(div_u32(uint32_t(ts), a.by_tail)) * T, first = min(T - slot, k1 - ts);
          it.n_tail = (first + a.tail_tile - 1) / a.tail_tile + (k1 - ts - first + a.tail_tile - 1) / a.tail_tile;
        }
      }
      cost = it.n_body + it.n_tail + kChunkGap;
    }
    it.at = length + block_sums(cost, s_sum, total) - cost;
    if (i < int(items)) a.items[i] = it;
    if (i < min(int(items), kPlanItems)) s_at[i] = it.at;
    length += total;
  }
  const long long all = length * a.c.n_kv_heads;
  ChunkHeader h{length, max((long long)kChunkMinPiece, (all + a.ctas - 1) / a.ctas), int(items), 0, items > 0, 0};
  h.pieces = int((all + h.piece - 1) / h.piece);
  if (tid == 0) *a.head = h;
  __syncthreads();
  for (int c = tid; c < h.pieces; c += kPlanThreads) {
    const long long z = c * h.piece % length;
    int lo = 0, hi = int(items) - 1;  // the last item that begins at or before z
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if ((items <= kPlanItems ? s_at[mid] : a.items[mid].at) <= z) lo = mid; else hi = mid - 1;
    }
    a.first[c] = lo;
  }
}

// ---- merge -------------------------------------------------------------------------------------

__device__ __forceinline__ void store_out(const ChunkArgs& a, size_t at, float v) {
  if (a.out_dtype == KVQ_F32) static_cast<float*>(a.out)[at] = v;
  else if (a.out_dtype == KVQ_BF16) static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
  else static_cast<__half*>(a.out)[at] = __float2half_rn(v);
}

// A row's output from its values in the FWHT layout: rotated back and stored by a warp.
template <int D>
__device__ __forceinline__ void finish_row(const ChunkArgs& a, const ChunkItem& it, int row0, int kvh, int r, float (&x)[D / 32],
                                           int lane) {
  constexpr int G = (D & (D - 1)) == 0 ? D : 64;
  if (a.rot_v) {
    warp_fwht<D, G>(x, lane);
#pragma unroll
    for (int j = 0; j < D / 32; ++j) x[j] *= inv_sqrt_group<G>();
  }
  const int w = it.r0 + r, tok = int(div_u32(uint32_t(w), a.by_group)), hh = w - tok * a.group;
  const size_t base = ((size_t)(row0 + tok) * a.n_q_heads + kvh * a.group + hh) * D;
#pragma unroll
  for (int j = 0; j < D / 32; ++j) store_out(a, base + fwht_channel<D, G>(lane, j), x[j]);
}

constexpr int kMergeRows = 8;  // rows of a merge CTA, a warp each

// CTA (c, part): the item cut for the first time between the pieces c and c + 1, if one is.
template <int D>
__global__ void __launch_bounds__(32 * kMergeRows) chunk_merge_kernel(ChunkArgs a) {
  pdl_begin();
  constexpr int G = (D & (D - 1)) == 0 ? D : 64;
  const ChunkHeader h = *a.head;
  const int c = blockIdx.x;
  if (!h.ok || c + 1 >= h.pieces) return;
  const long long cut = (c + 1) * h.piece;  // where piece c + 1 begins: an item that begins there itself is not cut
  const int kvh = int(cut / h.total);
  const ChunkItem it = a.items[a.first[c + 1]];
  const int nk = it.n_body + it.n_tail;
  const long long first = kvh * h.total + it.at + kChunkGap, last = first + nk - 1;  // places of the first and last tile
  // cut for the first time here: the first tile lies in piece c, the last one behind it
  if (nk == 0 || first >= cut || first < c * h.piece || last < cut) return;
  const int pieces = int(last / h.piece) - c + 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = a.row_start[it.b];
  for (int r = blockIdx.y * kMergeRows + warp; r < it.rows; r += gridDim.y * kMergeRows) {
    // the first piece's part lies in slot 2c + 1, those that begin inside the item in slots 2 (c + i)
    auto slot = [&](int i) { return i == 0 ? 2 * c + 1 : 2 * (c + i); };
    float M = -INFINITY, L = 0.0f, x[D / 32];
#pragma unroll
    for (int j = 0; j < D / 32; ++j) x[j] = 0.0f;
    for (int i = 0; i < pieces; i += 2) {  // (two pieces' loads in flight together; most items are cut once)
      float2 ml[2];
      float y[2][D / 32];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        ml[k] = make_float2(-INFINITY, 0.0f);
        if (i + k >= pieces) continue;
        const size_t at = (size_t)slot(i + k) * a.m + r;
        ml[k] = a.part_ml[at];
        const float* p = a.part + at * D;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) y[k][j] = p[fwht_channel<D, G>(lane, j)];
      }
      float next = M;
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (!(ml[k].y == 0.0f)) next = fmaxf(next, ml[k].x);  // (0: saw no key, nothing was stored; NaN goes on)
      const float f = M == -INFINITY ? 0.0f : ex2_approx(M - next);
      M = next;
      L *= f;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) x[j] *= f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (ml[k].y == 0.0f) continue;
        const float w = ex2_approx(ml[k].x - M);
        L = fmaf(ml[k].y, w, L);
#pragma unroll
        for (int j = 0; j < D / 32; ++j) x[j] = fmaf(y[k][j], w, x[j]);
      }
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) x[j] *= inv;
    finish_row<D>(a, it, row0, kvh, r, x, lane);
  }
}

template <class F>
cudaError_t by_dim(int d, F&& f) {
  switch (d) {
    case 64: return f(std::integral_constant<int, 64>());
    case 128: return f(std::integral_constant<int, 128>());
    case 192: return f(std::integral_constant<int, 192>());
    case 256: return f(std::integral_constant<int, 256>());
    case 320: return f(std::integral_constant<int, 320>());
    default: return cudaErrorInvalidValue;
  }
}

ChunkTiles tc_tiles_of(int d, int parts) {
  switch (d) {
    case 64: return chunk_tc_tiles_d64(parts);
    case 128: return chunk_tc_tiles_d128(parts);
    case 192: return chunk_tc_tiles_d192(parts);
    case 256: return chunk_tc_tiles_d256(parts);
    case 320: return chunk_tc_tiles_d320(parts);
    default: return ChunkTiles{0, 0, 0};
  }
}
cudaError_t launch_tc_of(ChunkArgs& a, int parts, cudaStream_t st) {
  switch (a.c.head_dim) {
    case 64: return launch_chunk_tc_d64(a, parts, st);
    case 128: return launch_chunk_tc_d128(a, parts, st);
    case 192: return launch_chunk_tc_d192(a, parts, st);
    case 256: return launch_chunk_tc_d256(a, parts, st);
    case 320: return launch_chunk_tc_d320(a, parts, st);
    default: return cudaErrorInvalidValue;
  }
}
// fp16 parts of the operands.  One rounds them to 2^-11 of themselves, an eighth of a bf16 output's step: against 64 bits such outputs are
// 1.70e-3 off where their own rounding alone is 1.66e-3 (32 sequences of one token), and one in six differs by a step.  Two are
// below fp16's step and at fp32's, for three products and twice the conversion: 2 x 4096 prompt rows 1389 us for 513.  So who
// wants more than bf16 shows takes another output type.
int parts_of(int out_dtype) { return out_dtype == KVQ_BF16 ? 1 : 2; }

// Sizes of a call with `t`'s items, and where its parts lie in the workspace; returns the bytes.
size_t layout(ChunkArgs& a, const ChunkTiles& t, char* ws) {
  const kvq_cache& c = a.c;
  a.m = t.m; a.tile = t.tile; a.tail_tile = t.tail_tile;
  const int sms = device_sm_count();
  a.ctas = sms > 0 ? sms : 148;
  const long long items = chunk_max_items(c, (long long)a.n_rows * a.group, a.m);
  size_t at = 0;
  auto take = [&](size_t bytes) {
    char* p = ws + at;
    at += (bytes + 255) / 256 * 256;
    return p;
  };
  a.head = reinterpret_cast<ChunkHeader*>(take(sizeof(ChunkHeader)));
  a.tiles0 = reinterpret_cast<int32_t*>(take(size_t(c.batch + 1) * 4));
  a.items = reinterpret_cast<ChunkItem*>(take(size_t(items) * sizeof(ChunkItem)));
  a.first = reinterpret_cast<int32_t*>(take(size_t(a.ctas) * sizeof(int32_t)));
  a.part_ml = reinterpret_cast<float2*>(take(size_t(2 * a.ctas) * a.m * sizeof(float2)));
  a.part = reinterpret_cast<float*>(take(size_t(2 * a.ctas) * a.m * c.head_dim * sizeof(float)));
  return at;
}

ChunkArgs chunk_args(const kvq_cache& c, int n_q_heads, int n_rows) {
  ChunkArgs a{};
  a.c = c;
  a.n_q_heads = n_q_heads; a.n_rows = n_rows; a.group = n_q_heads / c.n_kv_heads;
  return a;
}

}  // namespace

size_t chunk_workspace_bytes(const kvq_cache& c, int n_q_heads, int n_rows) {
  ChunkArgs a = chunk_args(c, n_q_heads, n_rows);
  return std::max(layout(a, tc_tiles_of(c.head_dim, 1), nullptr), layout(a, tc_tiles_of(c.head_dim, 2), nullptr));  // (any output type)
}

cudaError_t launch_chunk(const kvq_cache& c, Rot rot, const ChunkCall& call, void* ws, cudaStream_t st) {
  ChunkArgs a = chunk_args(c, call.n_q_heads, call.n_rows);
  const int parts = parts_of(call.out_dtype);
  layout(a, tc_tiles_of(c.head_dim, parts), static_cast<char*>(ws));
  if (call.mod) a.mod = *call.mod;
  a.q = call.q; a.out = call.out; a.row_start = call.row_start;
  a.q_dtype = call.q_dtype; a.out_dtype = call.out_dtype; a.scale = call.scale;
  a.rot_k = rot.k; a.rot_v = rot.v;
  a.by_group = make_divu32(uint32_t(a.group));
  a.by_tail = make_divu32(uint32_t(std::max(1, c.tail_len)));
  a.by_page = make_divu32(uint32_t(std::max(1, c.page_tokens)));
  a.pages_per_seq = c.page_tokens ? c.max_ctx / c.page_tokens : 0;
  cudaError_t e = launch_dependent(chunk_plan_kernel, 1u, kPlanThreads, 0, st, 1, a);
  if (e != cudaSuccess) return e;
  e = launch_tc_of(a, parts, st);
  if (e != cudaSuccess) return e;
  return by_dim(c.head_dim, [&](auto d) {
    return launch_dependent(chunk_merge_kernel<decltype(d)::value>, dim3(unsigned(a.ctas), unsigned(a.m / (2 * kMergeRows))),
                            32 * kMergeRows, 0, st, 1, a);
  });
}

}  // namespace kvq
