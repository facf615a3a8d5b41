// Attention of packed rows of new tokens (kvq_chunk_attention): the plan of a call, the merge of items in several pieces, and
// the kernel for fp32 and fp16 outputs.
#include "kvq_chunk.cuh"

#include <type_traits>

#include "kvq_decode_impl.cuh"
#include "kvq_rows.cuh"

namespace kvq {
namespace {

constexpr int kPlanThreads = 1024;

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
  long long w = s[lane];
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
  __shared__ long long s_sum[32];
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
    length += total;
  }
  if (tid == 0) {
    const long long all = length * a.c.n_kv_heads;
    ChunkHeader h{length, max((long long)kChunkMinPiece, (all + a.ctas - 1) / a.ctas), int(items), 0, items > 0, 0};
    h.pieces = int((all + h.piece - 1) / h.piece);
    *a.head = h;
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
  const long long cut = (c + 1) * h.piece, y = cut - 1;  // the last place of piece c
  const int kvh = int(y / h.total);
  const long long z = y - kvh * h.total;
  int lo = 0, hi = h.items - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.items[mid].at <= z) lo = mid; else hi = mid - 1;
  }
  const ChunkItem it = a.items[lo];
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
    for (int i = lane; i < pieces; i += 32) {
      const float2 ml = a.part_ml[(size_t)slot(i) * a.m + r];
      if (!(ml.y == 0.0f)) M = fmaxf(M, ml.x);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
    for (int j = 0; j < D / 32; ++j) x[j] = 0.0f;
    for (int i = 0; i < pieces; ++i) {
      const float2 ml = a.part_ml[(size_t)slot(i) * a.m + r];
      if (ml.y == 0.0f) continue;  // (saw no key; NaN goes on)
      const float w = ex2_approx(ml.x - M);
      L = fmaf(ml.y, w, L);
      const float* p = a.part + ((size_t)slot(i) * a.m + r) * D;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) x[j] = fmaf(p[fwht_channel<D, G>(lane, j)], w, x[j]);
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
#pragma unroll
    for (int j = 0; j < D / 32; ++j) x[j] *= inv;
    finish_row<D>(a, it, row0, kvh, r, x, lane);
  }
}

// ---- the kernel in tf32 ------------------------------------------------------------------------

// Operands as two tf32 parts (22 bits, fp32's range), so that nothing has to be scaled and the result has fp32's
// precision.  A warp has 16 rows, a CTA the kSm<D> of an item; keys and values of a tile of 32 are dequantized into shared memory.
template <int D> constexpr int kSm = D <= 192 ? 128 : 64;   // rows of an item
constexpr int kSt = 32;                                     // keys of a tile, body or tail
template <int D> constexpr int kSthreads = kSm<D> * 2;

__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xFFFFE000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

template <int D>
__global__ void __launch_bounds__(kSthreads<D>, 1) chunk_simple_kernel(ChunkArgs a) {
  pdl_begin();
  constexpr int G = (D & (D - 1)) == 0 ? D : 64, M = kSm<D>, S = D + 4, NT = kSthreads<D>;
  extern __shared__ __align__(16) float smem[];
  float* sq = smem;                  // [M][S] rotated queries times the scale; the outputs at an item's end
  float* sk = sq + M * S;            // [32][S]
  float* sv = sk + kSt * S;
  uint32_t* s_bad = reinterpret_cast<uint32_t*>(sv + kSt * S);  // [2]: keys of the tile with an infinity or NaN, by tile parity
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, tig = lane & 3;
  const ChunkHeader h = *a.head;
  const int T = a.c.tail_len;
  ChunkWalk walk;
  walk.begin(a, h, blockIdx.x);
  ChunkItem it;
  int kvh, j0, j1;
  while (walk.next(a, h, it, kvh, j0, j1)) {
    const int row0 = a.row_start[it.b], m = a.row_start[it.b + 1] - row0, n = min(max(a.c.seq_len[it.b], 0), a.c.max_ctx);
    const int nk = it.n_body + it.n_tail;
    // queries: a warp its own 16 rows
    for (int i = 0; i < 16; ++i) {
      const int r = warp * 16 + i, w = it.r0 + r, tok = int(div_u32(uint32_t(w), a.by_group));
      float v[D / 32];
      load_q_fwht<D, G>(a.q, a.q_dtype, (size_t)(row0 + tok) * a.n_q_heads + kvh * a.group + w - tok * a.group, r < it.rows, lane, v);
      if (a.rot_k) warp_fwht<D, G>(v, lane);
      const float sc = a.scale * (a.rot_k ? inv_sqrt_group<G>() : 1.0f);
#pragma unroll
      for (int j = 0; j < D / 32; ++j) sq[r * S + fwht_channel<D, G>(lane, j)] = v[j] * sc;
    }
    __syncwarp();
    // the lane's rows 16 warp + g, + 8
    ChunkSpan span[2];
    float slope[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = warp * 16 + g + 8 * e, w = it.r0 + r, tok = int(div_u32(uint32_t(w), a.by_group));
      span[e] = r < it.rows ? chunk_span(a, it.b, n, row0, m, tok) : ChunkSpan{0, 0, 0};
      slope[e] = a.mod.slopes && r < it.rows ? a.mod.slopes[kvh * a.group + w - tok * a.group] : 0.0f;
    }
    float o[D / 8][4], mx[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < D / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;
    bool nan[2] = {false, false};
    for (int j = j0; j < j1; ++j) {
      const ChunkTile t = chunk_tile<kSt, kSt>(a, it, n, j);
      __syncthreads();  // the tile before is done with
      if (tid < 2) s_bad[tid] = 0;
      __syncthreads();
      constexpr int CH = D / 8;
      for (int i = tid; i < 2 * kSt * CH; i += NT) {
        const bool is_k = i < kSt * CH;
        const int e = is_k ? i : i - kSt * CH, key = e / CH, ch = e % CH, pos = t.t0 + key;
        float x[8];
        bool have = key < t.cnt;
        if (have && t.tail) {
          const int slot = pos - int(div_u32(uint32_t(pos), a.by_tail)) * T;
          const uint16_t* src = static_cast<const uint16_t*>(is_k ? a.c.k_tail : a.c.v_tail) +
                                (((size_t)it.b * a.c.n_kv_heads + kvh) * T + slot) * D + ch * 8;
          const uint4 w = *reinterpret_cast<const uint4*>(src);
          const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            x[2 * q] = __uint_as_float(ww[q] << 16);
            x[2 * q + 1] = __uint_as_float(ww[q] & 0xFFFF0000u);
          }
        } else if (have) {
          const long long row = body_row(row_map(a.c), it.b, kvh, pos);
          if (row >= 0) {
            body_values8(body_side(a.c, is_k), D, row, ch, x);
          } else {  // a page outside the pool: its keys are left out
            have = false;
            atomicOr(a.c.status, KVQ_DEV_ERR_PAGE);
            atomicOr(&s_bad[1], 1u << key);
          }
        }
        if (have) {
          bool fin = true;
#pragma unroll
          for (int q = 0; q < 8; ++q) fin &= isfinite(x[q]);
          if (!fin) atomicOr(&s_bad[0], 1u << key);
          have = fin;
        }
        float* dst = (is_k ? sk : sv) + key * S + ch * 8;
        *reinterpret_cast<float4*>(dst) = have ? make_float4(x[0], x[1], x[2], x[3]) : make_float4(0.f, 0.f, 0.f, 0.f);
        *reinterpret_cast<float4*>(dst + 4) = have ? make_float4(x[4], x[5], x[6], x[7]) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      __syncthreads();
      const uint32_t bad = s_bad[0], gone = s_bad[1];
      if (warp * 16 >= it.rows) continue;
      float s[kSt / 8][4];
#pragma unroll
      for (int i = 0; i < kSt / 8; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.0f;
#pragma unroll 2
      for (int k = 0; k < D; k += 8) {
        const float* qr = sq + (warp * 16 + g) * S + k + tig;
        uint32_t ah[4], al[4];
        split_tf32(qr[0], ah[0], al[0]);
        split_tf32(qr[8 * S], ah[1], al[1]);
        split_tf32(qr[4], ah[2], al[2]);
        split_tf32(qr[8 * S + 4], ah[3], al[3]);
#pragma unroll
        for (int i = 0; i < kSt / 8; ++i) {
          const float* kr = sk + (8 * i + g) * S + k + tig;
          uint32_t bh[2], bl[2];
          split_tf32(kr[0], bh[0], bl[0]);
          split_tf32(kr[4], bh[1], bl[1]);
          mma_tf32(s[i], ah, bh);
          mma_tf32(s[i], ah, bl);
          mma_tf32(s[i], al, bh);
        }
      }
      // s[i][e]: row g + 8 (e / 2), key 8i + 2tig + e % 2
      float top[2] = {-INFINITY, -INFINITY};
      const float cap = a.mod.softcap, c2 = cap > 0.0f ? 2.0f * kChunkLog2e / cap : 0.0f;
#pragma unroll
      for (int i = 0; i < kSt / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = 8 * i + 2 * tig + (e & 1), pos = t.t0 + key, rr = e >> 1;
          float x = s[i][e];
          if (cap > 0.0f) x = soft_cap(x, cap, c2);
          x -= slope[rr] * float(abs(span[rr].pos - pos));
          const bool seen = key < t.cnt && pos >= span[rr].lo && pos < span[rr].hi && !(gone >> key & 1u);
          nan[rr] |= seen && (bad >> key & 1u);
          x = seen ? x * kChunkLog2e : -INFINITY;
          s[i][e] = x;
          top[rr] = fmaxf(top[rr], x);
          if (isnan(x)) nan[rr] = true;
        }
      float f[2], ref[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 1));
        top[e] = fmaxf(top[e], __shfl_xor_sync(0xffffffffu, top[e], 2));
        const float nm = fmaxf(mx[e], top[e]);
        f[e] = mx[e] == -INFINITY ? 0.0f : ex2_approx(mx[e] - nm);
        mx[e] = nm;
        ref[e] = nm == -INFINITY ? 0.0f : nm;
        l[e] *= f[e];
      }
#pragma unroll
      for (int i = 0; i < kSt / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          s[i][e] = ex2_approx(s[i][e] - ref[e >> 1]);
          l[e >> 1] += s[i][e];
        }
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        o[i][0] *= f[0]; o[i][1] *= f[0]; o[i][2] *= f[1]; o[i][3] *= f[1];
      }
      // keys 8i + 2tig, + 1 of the weights are the inner indices tig, tig + 4: they stay where they are
#pragma unroll
      for (int i = 0; i < kSt / 8; ++i) {
        uint32_t ph[4], pl[4];
        split_tf32(s[i][0], ph[0], pl[0]);
        split_tf32(s[i][2], ph[1], pl[1]);
        split_tf32(s[i][1], ph[2], pl[2]);
        split_tf32(s[i][3], ph[3], pl[3]);
        const float* vr = sv + (8 * i + 2 * tig) * S + g;
#pragma unroll
        for (int c = 0; c < D / 8; ++c) {
          uint32_t bh[2], bl[2];
          split_tf32(vr[8 * c], bh[0], bl[0]);
          split_tf32(vr[8 * c + S], bh[1], bl[1]);
          mma_tf32(o[c], ph, bh);
          mma_tf32(o[c], ph, bl);
          mma_tf32(o[c], pl, bh);
        }
      }
    }
    // the item's part of the rows: normalised to the output, or as it is for the merge
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 1);
      l[e] += __shfl_xor_sync(0xffffffffu, l[e], 2);
      int any = nan[e];
      any |= __shfl_xor_sync(0xffffffffu, any, 1);
      any |= __shfl_xor_sync(0xffffffffu, any, 2);
      if (any) { l[e] = NAN; if (mx[e] == -INFINITY) mx[e] = 0.0f; }
    }
    const bool whole = j0 == 0 && j1 == nk;
    float* out = sq + warp * 16 * S;  // only this warp's rows
    __syncwarp();
    const float inv0 = !whole ? 1.0f : l[0] == 0.0f ? 0.0f : 1.0f / l[0], inv1 = !whole ? 1.0f : l[1] == 0.0f ? 0.0f : 1.0f / l[1];
#pragma unroll
    for (int c = 0; c < D / 8; ++c) {
      *reinterpret_cast<float2*>(out + g * S + 8 * c + 2 * tig) = make_float2(o[c][0] * inv0, o[c][1] * inv0);
      *reinterpret_cast<float2*>(out + (g + 8) * S + 8 * c + 2 * tig) = make_float2(o[c][2] * inv1, o[c][3] * inv1);
    }
    const size_t slot = (size_t)(2 * blockIdx.x + (j0 == 0 ? 1 : 0)) * a.m;
    if (!whole && tig == 0) {
      a.part_ml[slot + warp * 16 + g] = make_float2(mx[0], l[0]);
      a.part_ml[slot + warp * 16 + g + 8] = make_float2(mx[1], l[1]);
    }
    __syncwarp();
    for (int i = 0; i < 16 && warp * 16 + i < it.rows; ++i) {
      float x[D / 32];
#pragma unroll
      for (int j = 0; j < D / 32; ++j) x[j] = out[i * S + fwht_channel<D, G>(lane, j)];
      if (whole) {
        finish_row<D>(a, it, row0, kvh, warp * 16 + i, x, lane);
      } else {
#pragma unroll
        for (int j = 0; j < D / 32; ++j) a.part[(slot + warp * 16 + i) * D + fwht_channel<D, G>(lane, j)] = x[j];
      }
    }
    __syncwarp();
  }
}

template <int D>
cudaError_t run_simple(ChunkArgs& a, cudaStream_t st) {
  constexpr int bytes = (kSm<D> + 2 * kSt) * (D + 4) * 4 + 16;
  static_assert(bytes <= 232448, "shared memory");
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(chunk_simple_kernel<D>), bytes);
  if (e != cudaSuccess) return e;
  return launch_dependent(chunk_simple_kernel<D>, unsigned(a.ctas), kSthreads<D>, bytes, st, 1, a);
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
// fp16 parts of the operands: one is an eighth of a bf16 output's step, two are below fp16's and at fp32's
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
  a.part_ml = reinterpret_cast<float2*>(take(size_t(2 * a.ctas) * a.m * sizeof(float2)));
  a.part = reinterpret_cast<float*>(take(size_t(2 * a.ctas) * a.m * c.head_dim * sizeof(float)));
  return at;
}
ChunkTiles simple_tiles(int d) { return ChunkTiles{d <= 192 ? 128 : 64, kSt, kSt}; }

ChunkArgs chunk_args(const kvq_cache& c, int n_q_heads, int n_rows) {
  ChunkArgs a{};
  a.c = c;
  a.n_q_heads = n_q_heads; a.n_rows = n_rows; a.group = n_q_heads / c.n_kv_heads;
  return a;
}

}  // namespace

size_t chunk_workspace_bytes(const kvq_cache& c, int n_q_heads, int n_rows) {
  ChunkArgs a = chunk_args(c, n_q_heads, n_rows);
  size_t most = layout(a, simple_tiles(c.head_dim), nullptr);  // (any output type)
  for (int parts = 1; parts <= 2; ++parts) {
    const ChunkTiles t = tc_tiles_of(c.head_dim, parts);
    if (t.m) most = std::max(most, layout(a, t, nullptr));
  }
  return most;
}

cudaError_t launch_chunk(const kvq_cache& c, Rot rot, const ChunkCall& call, void* ws, cudaStream_t st) {
  ChunkArgs a = chunk_args(c, call.n_q_heads, call.n_rows);
  const int parts = parts_of(call.out_dtype);
  const ChunkTiles t = tc_tiles_of(c.head_dim, parts);
  layout(a, t.m ? t : simple_tiles(c.head_dim), static_cast<char*>(ws));
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
  e = t.m ? launch_tc_of(a, parts, st) : by_dim(c.head_dim, [&](auto d) { return run_simple<decltype(d)::value>(a, st); });
  if (e != cudaSuccess) return e;
  return by_dim(c.head_dim, [&](auto d) {
    return launch_dependent(chunk_merge_kernel<decltype(d)::value>, dim3(unsigned(a.ctas), unsigned(a.m / (2 * kMergeRows))),
                            32 * kMergeRows, 0, st, 1, a);
  });
}

}  // namespace kvq
