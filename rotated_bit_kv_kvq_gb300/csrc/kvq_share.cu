// Pages that several sequences hold (kvq_page_fork, kvq_page_free, kvq_page_compact).
//
// A page's count is the number of sequences that hold it beyond the first, so that pages handed out by kvq_page_update have
// a count of 0 without knowing of it.  Only full pages are shared: a sequence appends to pages that it holds alone.
//
// All three are bound by what they move (fork and compact: page and tail bytes, read and written once) or by the latency of
// their launches and scans (free).  Measured (GB300): 64 forks of 8 prompts, tails of 512 tokens, 162 MB: 50 us (3.3 TB/s;
// most of it the decoding of tail rows that the source no longer has); half of a pool of 4096 pages moved, 234 MB: 52 us, 35
// of them the copy (6.7 TB/s); 256 of 512 sequences freed: 19 us.
//
// Results do not depend on the order of atomics: counts are sums, and pages freed in one call go into the ring in ascending
// order, from a scan over the bits that mark them.

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "kvq_rows.cuh"

namespace kvq {
namespace {

namespace cg = cooperative_groups;

constexpr int kPlanThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kCopyCtas = 4;             // of an SM
constexpr int kCopyBytes = 16 * 1024;    // of a unit: four 16-byte loads a thread, in flight together
constexpr int kMaxForkBatch = 65536;     // bits of a sequence bitmap in shared memory

__device__ __forceinline__ bool pool_ok(int head, int count, int n_pages) {
  return head >= 0 && head < n_pages && count >= 0 && count <= n_pages;
}
__device__ __forceinline__ int held_pages(int len, const ShareArgs& a) {  // 0 for a length out of range
  return len >= 0 && len <= a.max_ctx ? int((uint32_t(len) + uint32_t(a.page_tokens) - 1) / uint32_t(a.page_tokens)) : 0;
}

// Inclusive sums over a block of kPlanThreads; s: 32 values.  Returns this thread's, and the block's in total.
template <class T>
__device__ __forceinline__ T block_sums(T v, T* s, T& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  __syncthreads();  // (the sums before are read)
  if (lane == 31) s[warp] = v;
  __syncthreads();
  T w = s[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const T before = __shfl_sync(0xffffffffu, w, warp == 0 ? 0 : warp - 1);
  return v + (warp == 0 ? T(0) : before);
}

// `bytes` (a multiple of 16) by the threads of a CTA, both sides 16-byte aligned
__device__ __forceinline__ void copy_unit(uint8_t* dst, const uint8_t* src, int bytes) {
  const uint4* s = reinterpret_cast<const uint4*>(src);
  uint4* d = reinterpret_cast<uint4*>(dst);
  const int n = bytes / 16;
  for (int i = threadIdx.x; i < n; i += 4 * kCopyThreads) {
    uint4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k * kCopyThreads < n) v[k] = s[i + k * kCopyThreads];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k * kCopyThreads < n) d[i + k * kCopyThreads] = v[k];
  }
}
// unit u of a page's copy: the planes' pieces one after another
__device__ __forceinline__ void copy_page_unit(const ShareArgs& a, int u, int to, int from) {
  for (int p = 0; p < a.n_planes; ++p) {
    if (u < a.units[p]) {
      const long long at = (long long)u * kCopyBytes;
      const int n = int(min((long long)kCopyBytes, a.page_bytes[p] - at));
      copy_unit(a.plane[p] + to * a.page_bytes[p] + at, a.plane[p] + from * a.page_bytes[p] + at, n);
      return;
    }
    u -= a.units[p];
  }
}

// ---- fork ------------------------------------------------------------------------------------------

// CTA 0: which forks are valid, the pages they get, the pool's state.  The others: counts and lengths where the results go
// elsewhere.
__global__ void __launch_bounds__(kPlanThreads, 1) fork_plan_kernel(ShareArgs a, ForkArgs f) {
  pdl_begin();
  const int tid = threadIdx.x;
  if (blockIdx.x > 0) {
    const long long i0 = (long long)(blockIdx.x - 1) * kPlanThreads + tid, step = (long long)(gridDim.x - 1) * kPlanThreads;
    if (a.share.next != a.share.count)
      for (long long i = i0; i < a.n_pages; i += step) a.share.next[i] = a.share.count[i];
    if (f.seq_len_out != a.seq_len)
      for (long long i = i0; i < a.batch; i += step) f.seq_len_out[i] = a.seq_len[i];
    return;
  }
  __shared__ int s_sum[32];
  __shared__ uint32_t s_once[kMaxForkBatch / 32], s_twice[kMaxForkBatch / 32];
  const int P = a.page_tokens, per_seq = a.max_ctx / P;
  const int head = a.pool.state[0], count = a.pool.state[1];
  const bool pool = pool_ok(head, count, a.n_pages);
  for (int i = tid; i < (a.batch + 31) / 32; i += kPlanThreads) s_once[i] = s_twice[i] = 0u;
  __syncthreads();
  for (int i = tid; i < f.n_forks; i += kPlanThreads) {
    const int d = f.dst[i];
    if (d < 0 || d >= a.batch) continue;
    const uint32_t bit = 1u << (d & 31);
    if (atomicOr(&s_once[d >> 5], bit) & bit) atomicOr(&s_twice[d >> 5], bit);
  }
  __syncthreads();
  uint32_t err = pool ? 0u : KVQ_DEV_ERR_PAGE;
  int taken = 0;
  for (int i0 = 0; i0 < f.n_forks; i0 += kPlanThreads) {
    const int i = i0 + tid;
    int n = -1, dst = 0;
    if (i < f.n_forks) {
      const int src = f.src[i];
      dst = f.dst[i];
      bool ok = src >= 0 && src < a.batch && dst >= 0 && dst < a.batch && src != dst;
      if (ok) {
        const int len = a.seq_len[src], want = f.n_tokens ? f.n_tokens[i] : len;
        ok = len >= 0 && len <= a.max_ctx && want >= 0 && want <= len && a.seq_len[dst] == 0 &&
             !(s_twice[dst >> 5] >> (dst & 31) & 1u);
        if (ok) n = want;
      }
      if (!ok) err |= KVQ_DEV_ERR_FORK;
    }
    const int need = n > 0 && n % P ? 1 : 0;
    int total;
    const int at = taken + block_sums(need, s_sum, total) - need;
    if (i < f.n_forks) {
      int got = pool ? n : -1;
      if (pool && need) {
        if (at < count) {
          int r = head + at;
          if (r >= a.n_pages) r -= a.n_pages;
          const int pg = a.pool.ring[r];
          if (pg >= 0 && pg < a.n_pages) {
            a.table[(long long)dst * per_seq + n / P] = pg;
          } else {  // a ring gone wrong
            err |= KVQ_DEV_ERR_PAGE;
            got = -1;
          }
        } else {
          err |= KVQ_DEV_ERR_NO_ROOM;
          got = -1;
        }
      }
      f.granted[i] = got;
    }
    taken += total;
  }
  if (err) atomicOr(a.status, err);
  if (tid == 0) {
    const int popped = pool ? min(taken, count) : 0;
    int h = head;
    if (pool && (h += popped) >= a.n_pages) h -= a.n_pages;
    a.pool.next[0] = h;
    a.pool.next[1] = count - popped;
  }
}

// Units of a fork: its table row and length, the pieces of the page that is copied, the pieces of its tail.  A CTA takes every
// parts-th unit of a fork: one look at the fork's numbers for many units (a look a unit: 95 us for 64 forks with tails of 512
// tokens, 2 MB each).
__global__ void __launch_bounds__(kCopyThreads, kCopyCtas) fork_copy_kernel(ShareArgs a, ForkArgs f) {
  pdl_begin();
  const int P = a.page_tokens, per_seq = a.max_ctx / P, tid = threadIdx.x;
  const kvq_cache& c = f.c;
  const int T = c.tail_len, D = c.head_dim, H = c.n_kv_heads;
  for (long long w = blockIdx.x; w < (long long)f.n_forks * f.parts; w += gridDim.x) {
    const int i = int(w / f.parts), part = int(w - (long long)i * f.parts);
    const int n = f.granted[i], src = f.src[i], dst = f.dst[i];
    if (n < 0) continue;
    const int32_t* from = a.table + (long long)src * per_seq;
    if (part == 0) {
      if (tid == 0) f.seq_len_out[dst] = n;
      for (int j = tid; j < n / P; j += kCopyThreads) {
        const int pg = from[j];
        a.table[(long long)dst * per_seq + j] = pg;
        if (pg >= 0 && pg < a.n_pages) atomicAdd(&a.share.next[pg], 1);
        else atomicOr(a.status, KVQ_DEV_ERR_PAGE);
      }
    }
    if (n == 0) continue;
    const int old = n % P ? from[n / P] : 0, fresh = n % P ? a.table[(long long)dst * per_seq + n / P] : 0;
    const int first = a.seq_len[src] - T, r0 = T > 0 ? n % T : 0;
    const bool page_ok = old >= 0 && old < a.n_pages;
    if (!page_ok && part == 0 && tid == 0) atomicOr(a.status, KVQ_DEV_ERR_PAGE);
    for (int u = part; u < f.units; u += f.parts) {
      if (u < a.page_units) {
        if (n % P && page_ok) copy_page_unit(a, u, fresh, old);
        continue;
      }
      // tail slots s0 .. of (side, KV head): slot s holds the position p = s (mod T) of the last T
      int v = u - a.page_units;
      const int piece = v % f.tail_pieces, h = (v /= f.tail_pieces) % H;
      const bool k = v / H == 0;
      const int s0 = piece * f.tail_rows, rows = min(f.tail_rows, T - s0);
      uint8_t* plane = static_cast<uint8_t*>(k ? c.k_tail : c.v_tail);
      const uint8_t* in = plane + ((long long)src * H + h) * T * (2 * D);
      uint8_t* out = plane + ((long long)dst * H + h) * T * (2 * D);
      auto position = [&](int s) { return n - r0 + s - (s < r0 ? 0 : T); };
      if (n >= T && n - T >= first) {  // every slot is copied as it is
        copy_unit(out + (long long)s0 * 2 * D, in + (long long)s0 * 2 * D, rows * 2 * D);
        continue;
      }
      const BodySide side = body_side(c, k);
      // 16 channels a thread, those of 8 bytes of a 4-bit block's codes (8 channels a thread: 70 us for 64 forks, tails of 512)
      const int per_row = D / 16, pieces = rows * per_row;
      for (int j = tid; j < pieces; j += kCopyThreads) {
        const int r = int(div_u32(uint32_t(j), f.by_row)), s = s0 + r, blk = (j - r * per_row) / 2, u = j - r * per_row - 2 * blk, p = position(s);
        if (p < 0) continue;
        const long long at = ((long long)s * (D / 8) + blk * 4 + u) * 16;
        uint4 x[2];
        if (p >= first) {
#pragma unroll
          for (int k = 0; k < 2; ++k) x[k] = *reinterpret_cast<const uint4*>(in + at + 32 * k);
        } else {  // the source's tail has moved on: the stored values, rounded to bf16
          const long long row = body_row(row_map(c), src, h, p);
          if (row < 0) {
            atomicOr(a.status, KVQ_DEV_ERR_PAGE);
            continue;
          }
          float y[2][8];
          body_values16(side, D, row, blk, u, y);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t wds[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(y[k][2 * e], y[k][2 * e + 1]);
              wds[e] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            x[k] = make_uint4(wds[0], wds[1], wds[2], wds[3]);
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) *reinterpret_cast<uint4*>(out + at + 32 * k) = x[k];
      }
    }
  }
}

// ---- free ------------------------------------------------------------------------------------------

// One cluster.  Every released table entry takes one from its page's count; the page of the entry that finds 0 there is free.
// Free pages are bits in shared memory, a range of pages per CTA, and go, in ascending order, behind the ring's: a scan over
// words of 32 pages instead of the pool's counts.  (A pool of more pages than there are bits: in several rounds over the tables.)
constexpr int kFreeWords = 4096;
__global__ void __launch_bounds__(kPlanThreads, 1) free_kernel(ShareArgs a, const int32_t* release, int32_t* seq_len_out) {
  pdl_begin();
  cg::cluster_group cl = cg::this_cluster();
  __shared__ int s_sum[32], s_before[kPlanThreads];
  __shared__ uint32_t s_bits[kFreeWords];
  __shared__ int s_total;
  const int S = int(cl.num_blocks()), rank = int(cl.block_rank()), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nt = S * kPlanThreads, gt = rank * kPlanThreads + tid, per_seq = a.max_ctx / a.page_tokens;
  const int head = a.pool.state[0], count = a.pool.state[1];
  const bool pool = pool_ok(head, count, a.n_pages);
  uint32_t err = pool ? 0u : KVQ_DEV_ERR_PAGE;
  const int words = min(kFreeWords, int(((long long)a.n_pages + 32 * S - 1) / (32 * S)));  // of a CTA
  if (a.share.next != a.share.count)
    for (long long i = gt; i < a.n_pages; i += nt) a.share.next[i] = a.share.count[i];
  const int room = a.n_pages - count;  // (a bad state: nothing is free below)
  int all = 0;
  for (long long base = 0; pool && base < a.n_pages; base += (long long)S * words * 32) {
    __syncthreads();  // (the round before has been read)
    for (int w = tid; w < words; w += kPlanThreads) s_bits[w] = 0u;
    cl.sync();  // (the counts are there, too)
    for (int b = gt >> 5; b < a.batch; b += nt >> 5) {  // a warp a sequence
      const int32_t* row = a.table + (long long)b * per_seq;
      const int gone = release[b], len = a.seq_len[b];
      int next = lane < per_seq ? row[lane] : 0;  // (loads that wait for nothing: each wait is most of a microsecond)
      if (gone == 0) continue;
      const int held = held_pages(len, a);
      if (len < 0 || len > a.max_ctx) err |= KVQ_DEV_ERR_APPEND_RANGE;
      for (int j = lane; j < held; j += 32) {
        const int pg = next;
        if (j + 32 < held) next = row[j + 32];
        if (pg < 0 || pg >= a.n_pages) {
          err |= KVQ_DEV_ERR_PAGE;
          continue;
        }
        const long long at = pg - base;
        if (at < 0 || at >= (long long)S * words * 32) continue;  // another round's
        const int was = atomicSub(&a.share.next[pg], 1);
        if (was > 0) continue;
        if (was < 0) err |= KVQ_DEV_ERR_PAGE;  // given back more often than it was held
        const int r = int(uint32_t(at >> 5) / uint32_t(words)), w = int(at >> 5) - r * words;
        atomicOr(cl.map_shared_rank(s_bits, r) + w, 1u << (at & 31));
      }
    }
    cl.sync();
    int mine = 0, total;
    for (int w = tid; w < words; w += kPlanThreads) mine += __popc(s_bits[w]);
    block_sums(mine, s_sum, total);
    if (tid == 0) s_total = total;
    cl.sync();
    int before = all;
    for (int r = 0; r < S; ++r) {
      const int t = *cl.map_shared_rank(&s_total, r);
      if (r < rank) before += t;
      all += t;
    }
    const long long p0 = base + (long long)rank * words * 32;
    for (int q = 0; q < words; q += kPlanThreads) {
      const int n = q + tid < words ? __popc(s_bits[q + tid]) : 0;
      s_before[tid] = before + block_sums(n, s_sum, total) - n;
      before += total;
      __syncthreads();
      for (int i = warp; i < kPlanThreads && q + i < words; i += 32) {  // a warp a word
        const uint32_t bits = s_bits[q + i];
        if (!(bits >> lane & 1u)) continue;
        const int p = int(p0 + (q + i) * 32 + lane), at = s_before[i] + __popc(bits & ((1u << lane) - 1u));
        a.share.next[p] = 0;
        if (at < room) {
          long long k = (long long)head + count + at;
          while (k >= a.n_pages) k -= a.n_pages;
          a.pool.ring[k] = p;
        }
      }
    }
  }
  if (pool && all > room) err |= KVQ_DEV_ERR_PAGE;
  if (err) atomicOr(a.status, err);
  cl.sync();  // every CTA has read the lengths, the state and the others' sums
  if (seq_len_out)
    for (int b = gt; b < a.batch; b += nt) {
      const int len = a.seq_len[b];
      seq_len_out[b] = pool && release[b] != 0 && len >= 0 && len <= a.max_ctx ? 0 : len;
    }
  if (rank == 0 && tid == 0) {
    a.pool.next[0] = head;
    a.pool.next[1] = pool ? count + min(all, room) : count;
  }
}

// ---- compact ---------------------------------------------------------------------------------------

// One cluster.  Pages that are live (in a sequence's table) or free (in the ring) are bits, a range of pages per CTA, in shared
// memory, or in the workspace where they do not fit; of the n live ones those that are not among the n lowest marked pages
// move, the i-th to the i-th free page among these.  moves: [0] their number, then the sources and the destinations.
constexpr int kMarkWords = 2048;
struct Marked {  // pages, live ones in the upper half, live and free ones in the lower
  long long n;
  __device__ __forceinline__ int live() const { return int(n >> 32); }
  __device__ __forceinline__ int all() const { return int(n & 0xffffffffLL); }
};
__global__ void __launch_bounds__(kPlanThreads, 1) compact_plan_kernel(ShareArgs a, CompactArgs m) {
  pdl_begin();
  cg::cluster_group cl = cg::this_cluster();
  __shared__ long long s_sum[32], s_before[kPlanThreads], s_total;
  __shared__ uint32_t s_bits[2][kMarkWords];
  __shared__ int s_low, s_bad;
  const int S = int(cl.num_blocks()), rank = int(cl.block_rank()), tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nt = S * kPlanThreads, gt = rank * kPlanThreads + tid, per_seq = a.max_ctx / a.page_tokens;
  const int head = a.pool.state[0], count = a.pool.state[1];
  const bool pool = pool_ok(head, count, a.n_pages);
  const int words = int(((long long)a.n_pages + 32 * S - 1) / (32 * S));  // of a CTA
  const bool here = words <= kMarkWords;
  auto bits = [&](int r, int k) -> uint32_t* {  // CTA r's; k 0: free, 1: live
    return here ? cl.map_shared_rank(&s_bits[k][0], r) : reinterpret_cast<uint32_t*>(m.mark) + ((long long)k * S + r) * words;
  };
  volatile uint32_t *fre = bits(rank, 0), *liv = bits(rank, 1);
  if (tid == 0) {
    s_bad = pool ? 0 : 1;
    s_low = 0;
  }
  for (int w = tid; w < words; w += kPlanThreads) fre[w] = liv[w] = 0u;
  for (long long i = gt; i < a.n_pages; i += nt) {
    m.map[i] = int(i);
    if (a.share.next && a.share.next != a.share.count) a.share.next[i] = a.share.count[i];
  }
  cl.sync();
  bool bad = false;
  auto mark = [&](int pg, int k) {  // false: outside the pool, or marked before
    if (pg < 0 || pg >= a.n_pages) return false;
    const int r = int(uint32_t(pg >> 5) / uint32_t(words));
    const uint32_t bit = 1u << (pg & 31);
    return !(atomicOr(bits(r, k) + ((pg >> 5) - r * words), bit) & bit);
  };
  if (pool) {
    for (int b = gt >> 5; b < a.batch; b += nt >> 5) {
      const int32_t* row = a.table + (long long)b * per_seq;
      const int len = a.seq_len[b];
      int next = lane < per_seq ? row[lane] : 0;  // (no wait for the length)
      const int held = held_pages(len, a);
      bad |= len < 0 || len > a.max_ctx;
      for (int j = lane; j < held; j += 32) {
        const int pg = next;
        if (j + 32 < held) next = row[j + 32];
        bad |= !mark(pg, 1) && (pg < 0 || pg >= a.n_pages);  // (several sequences may hold it)
      }
    }
    for (int i = gt; i < a.n_pages; i += nt) {  // (no wait for the state)
      const int pg = a.pool.ring[i], at = i - head;
      if ((at < 0 ? at + a.n_pages : at) < count) bad |= !mark(pg, 0);
    }
  }
  cl.sync();
  long long mine = 0, total;
  for (int w = tid; w < words; w += kPlanThreads) {
    const uint32_t l = liv[w], f = fre[w];
    bad |= (l & f) != 0u;
    mine += ((long long)__popc(l) << 32) + __popc(l | f);
  }
  if (bad) s_bad = 1;
  block_sums(mine, s_sum, total);
  if (tid == 0) s_total = total;
  cl.sync();
  Marked sum{0}, before{0};
  bool any_bad = false;
  for (int r = 0; r < S; ++r) {
    const long long t = *cl.map_shared_rank(&s_total, r);
    any_bad |= *cl.map_shared_rank(&s_bad, r) != 0;
    if (r < rank) before.n += t;
    sum.n += t;
  }
  const int n_live = sum.live(), n_hand = sum.all();
  // marked pages before each word of words q ..; returns those before this thread's
  auto scan = [&](int q, Marked& at) {
    const uint32_t l = q + tid < words ? liv[q + tid] : 0u, f = q + tid < words ? fre[q + tid] : 0u;
    const long long n = ((long long)__popc(l) << 32) + __popc(l | f);
    const Marked b{at.n + block_sums(n, s_sum, total) - n};
    s_before[tid] = b.n;
    at.n += total;
    const int k = n_live - b.all();
    if (k > 0 && k <= __popc(l | f)) {  // the n_live-th marked page is in this word: the live ones up to it
      uint32_t rest = l | f;
      for (int i = 0; i < k; ++i) rest &= rest - 1u;
      const int low = b.live() + __popc(l & ~rest);
      for (int r = 0; r < S; ++r) *cl.map_shared_rank(&s_low, r) = low;
    }
    __syncthreads();
  };
  Marked at = before;
  for (int q = 0; q < words; q += kPlanThreads) scan(q, at);
  cl.sync();
  const int n_low = s_low, n_moves = any_bad ? 0 : n_live - n_low;
  int32_t *from = m.moves + 1, *to = from + a.n_pages;
  if (!any_bad) {
    at = before;
    for (int q = 0; q < words; q += kPlanThreads) {
      if (words > kPlanThreads) scan(q, at);  // (else as it was left)
      for (int i = warp; i < kPlanThreads && q + i < words; i += 32) {  // a warp a word
        const uint32_t l = liv[q + i], k = l | fre[q + i], below = (1u << lane) - 1u;
        if (!(k >> lane & 1u)) continue;
        const Marked b{s_before[i]};
        const int p = int(((long long)rank * words + q + i) * 32 + lane), al = b.live() + __popc(l & below), ah = b.all() + __popc(k & below);
        const bool is_live = l >> lane & 1u;
        if (ah < n_live) {
          if (!is_live) to[ah - al] = p;
        } else {
          if (is_live) from[al - n_low] = p;
          m.ring_out[ah - n_live] = p;
        }
      }
    }
    for (int i = n_hand - n_live + gt; i < a.n_pages; i += nt) m.ring_out[i] = -1;
  } else if (m.ring_out != a.pool.ring) {
    for (int i = gt; i < a.n_pages; i += nt) m.ring_out[i] = a.pool.ring[i];
  }
  cl.sync();
  for (int i = gt; i < n_moves; i += nt) {
    const int f = __ldcg(&from[i]), t = __ldcg(&to[i]);
    m.map[f] = t;
    if (a.share.next) {
      a.share.next[t] = a.share.count[f];
      a.share.next[f] = 0;
    }
  }
  if (rank == 0 && tid == 0) {
    if (any_bad) atomicOr(a.status, KVQ_DEV_ERR_PAGE);
    m.moves[0] = n_moves;
    a.pool.next[0] = any_bad ? head : 0;
    a.pool.next[1] = any_bad ? count : n_hand - n_live;
  }
}

__global__ void __launch_bounds__(kCopyThreads, kCopyCtas) compact_copy_kernel(ShareArgs a, CompactArgs m) {
  pdl_begin();
  const int n = m.moves[0], per_seq = a.max_ctx / a.page_tokens;
  const int32_t *from = m.moves + 1, *to = from + a.n_pages;
  const long long work = (long long)n * a.page_units;
  int i = int(blockIdx.x / a.page_units);
  int t = i < a.n_pages ? to[i] : 0, f = i < a.n_pages ? from[i] : 0;  // (loaded beside their number; no move: not used)
  for (long long w = blockIdx.x; w < work; w += gridDim.x) {
    const long long next = w + gridDim.x;
    const int u = int(w - (long long)i * a.page_units), t0 = t, f0 = f;
    i = int(next / a.page_units);
    if (next < work) {  // (known when its turn comes)
      t = to[i];
      f = from[i];
    }
    copy_page_unit(a, u, t0, f0);
  }
  const long long entries = (long long)a.batch * per_seq;
  // the table, by the last CTAs first: a few moves leave them free
  for (long long e = (long long)(gridDim.x - 1 - blockIdx.x) * kCopyThreads + threadIdx.x; e < entries; e += (long long)gridDim.x * kCopyThreads) {
    const int b = int(e / per_seq), pg = a.table[e], len = a.seq_len[b];
    const bool used = int(e - (long long)b * per_seq) < held_pages(len, a);
    const int out = used && pg >= 0 && pg < a.n_pages ? m.map[pg] : pg;
    if (m.table_out != a.table || out != pg) m.table_out[e] = out;
  }
}

ShareArgs share_args(const kvq_cache& c, const kvq_page_pool& pool, const kvq_page_share* share) {
  ShareArgs a{};
  a.seq_len = c.seq_len; a.status = c.status;
  a.table = const_cast<int32_t*>(c.page_table);
  a.batch = c.batch; a.max_ctx = c.max_ctx; a.page_tokens = c.page_tokens; a.n_pages = c.n_pages;
  a.pool = pool;
  if (share) a.share = *share;
  const long long rows = (long long)c.n_kv_heads * c.page_tokens, nb = c.head_dim / 32;
  auto plane = [&](void* p, long long bytes) {
    if (!p) return;
    a.plane[a.n_planes] = static_cast<uint8_t*>(p);
    a.page_bytes[a.n_planes] = bytes;
    a.units[a.n_planes] = int((bytes + kCopyBytes - 1) / kCopyBytes);
    a.page_units += a.units[a.n_planes++];
  };
  plane(c.k_qs, rows * (long long)qs_row_bytes_host(c.k_type, c.head_dim));
  plane(c.v_qs, rows * (long long)qs_row_bytes_host(c.v_type, c.head_dim));
  plane(c.k_d, rows * nb * (type_has_min(c.k_type) ? 4 : 2));
  plane(c.v_d, rows * nb * (type_has_min(c.v_type) ? 4 : 2));
  plane(c.k_qh, rows * nb * 4);
  plane(c.v_qh, rows * nb * 4);
  plane(c.outl, rows / 16 * kOutlTile);
  return a;
}
int sms() {
  const int n = device_sm_count();
  return n > 0 ? n : 148;
}
// a cluster of eight where there is work for it: a page a thread, or a table's pages a warp
int plan_ctas(const kvq_cache& c) { return c.n_pages > 4 * kPlanThreads || c.batch > 64 ? 8 : 1; }

}  // namespace

cudaError_t launch_page_fork(const kvq_cache& c, const kvq_page_pool& pool, const kvq_page_share& share, ForkArgs f,
                             cudaStream_t st) {
  ShareArgs a = share_args(c, pool, &share);
  f.c = c;
  f.tail_rows = std::max(1, kCopyBytes / (2 * c.head_dim));
  f.tail_pieces = (c.tail_len + f.tail_rows - 1) / f.tail_rows;
  f.by_row = make_divu32(uint32_t(c.head_dim / 16));
  f.units = a.page_units + 2 * c.n_kv_heads * f.tail_pieces;
  f.parts = int(std::max<long long>(1, std::min<long long>(f.units, 2LL * sms() * kCopyCtas / f.n_forks)));
  const bool elsewhere = share.next != share.count || f.seq_len_out != c.seq_len;
  const int more = elsewhere ? int(std::min<long long>(sms(), ((long long)std::max(c.n_pages, c.batch) + kPlanThreads - 1) / kPlanThreads)) : 0;
  cudaError_t e = launch_dependent(fork_plan_kernel, unsigned(1 + more), kPlanThreads, 0, st, 1, a, f);
  if (e != cudaSuccess) return e;
  const long long work = (long long)f.n_forks * f.parts;
  return launch_dependent(fork_copy_kernel, unsigned(std::min<long long>(work, (long long)sms() * kCopyCtas)), kCopyThreads, 0, st, 1, a, f);
}

cudaError_t launch_page_free(const kvq_cache& c, const kvq_page_pool& pool, const kvq_page_share& share, const int32_t* release,
                             int32_t* seq_len_out, cudaStream_t st) {
  const int S = plan_ctas(c);
  return launch_dependent(free_kernel, unsigned(S), kPlanThreads, 0, st, S, share_args(c, pool, &share), release, seq_len_out);
}

cudaError_t launch_page_compact(const kvq_cache& c, const kvq_page_pool& pool, const kvq_page_share* share, CompactArgs m,
                                cudaStream_t st) {
  const ShareArgs a = share_args(c, pool, share);
  const int S = plan_ctas(c);
  cudaError_t e = launch_dependent(compact_plan_kernel, unsigned(S), kPlanThreads, 0, st, S, a, m);
  if (e != cudaSuccess) return e;
  const long long work = std::max((long long)c.n_pages * a.page_units, ((long long)c.batch * (c.max_ctx / c.page_tokens) + kCopyThreads - 1) / kCopyThreads);
  return launch_dependent(compact_copy_kernel, unsigned(std::min<long long>(work, (long long)sms() * kCopyCtas)), kCopyThreads, 0, st, 1, a, m);
}

}  // namespace kvq
