// Page table and row maps of a step from request lengths (kvq_page_update).
//
// Sequence b asks for r_b tokens behind its n_b: need_b = ceil((n_b + r_b) / P) -
// ceil(n_b / P) new pages.  Exclusive prefix sums over the sequences in order give
// where its pages start in the ring of free pages and where its rows start in the
// packed order; a released sequence's pages go behind the free ones, by a third sum.
//
// Every CTA computes all the sums (12 bytes a sequence, from L2) and writes its share of
// the pages and rows, so no CTA waits for another: a row's page comes from the table or,
// where this call hands it out, from the ring itself.  What other CTAs read -- lengths and
// pool state -- is advanced by the last CTA to finish.
//
// Bound by latency (loads, two scans, a binary search per row): 32 sequences of one token each
// 4.1 us, 512 sequences with 128 thousand rows 6.3 us (one CTA for everything: 160 us).

#include <cuda_runtime.h>

#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kMaxPageThreads = 1024;  // sequences scanned at a time

// Prefix sums of one sequence.  Rows stay below 2^31 (checked on the host), pages asked
// for too (at most rows / 64 + 1 a sequence); what sequences say they hold may not.
struct Sums {
  int rows, need;
  long long back;
};

// What sequence b asks for: r tokens (0 for a release or an invalid value).
struct Ask {
  int n, r, held, need, back;
  bool released, bad;
};
__device__ __forceinline__ Ask ask_of(const PageArgs& a, int b, bool pool_ok) {
  Ask k{0, 0, 0, 0, 0, false, false};
  if (b >= a.batch) return k;
  const int n = a.seq_len[b], r = a.n_new[b];
  const bool len_ok = n >= 0 && n <= a.max_ctx;
  k.n = len_ok ? n : 0;
  k.held = int(div_u32(uint32_t(k.n + a.page_tokens - 1), a.by_page));
  if (r == KVQ_PAGE_RELEASE && len_ok) {
    k.back = pool_ok ? k.held : 0;
    k.released = pool_ok;
  } else if (len_ok && r >= 0 && r <= a.n_new_max && n + (long long)r <= a.max_ctx) {
    k.r = r;
    k.need = int(div_u32(uint32_t(n + r + a.page_tokens - 1), a.by_page)) - k.held;
  } else {
    k.bad = true;
  }
  return k;
}

__device__ __forceinline__ Sums warp_scan(Sums v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int r = __shfl_up_sync(0xffffffffu, v.rows, o), n = __shfl_up_sync(0xffffffffu, v.need, o);
    const long long k = __shfl_up_sync(0xffffffffu, v.back, o);
    if (lane >= o) { v.rows += r; v.need += n; v.back += k; }
  }
  return v;
}

__global__ void __launch_bounds__(kMaxPageThreads) page_update_kernel(PageArgs a) {
  pdl_begin();
  __shared__ Sums s_warp[32];
  __shared__ int s_row[kMaxPageThreads], s_need[kMaxPageThreads], s_n[kMaxPageThreads], s_held[kMaxPageThreads];
  __shared__ int s_get[kMaxPageThreads], s_put[kMaxPageThreads];  // pages to hand out (-1: nothing granted) and to take back
  __shared__ long long s_back[kMaxPageThreads];
  __shared__ int s_popped;
  __shared__ unsigned s_last;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, nw = nt >> 5;
  const int P = a.page_tokens, per_seq = a.max_ctx / P;
  const bool first = blockIdx.x == 0;
  const int head = a.pool.state[0], count = a.pool.state[1];
  const bool pool_ok = head >= 0 && head < a.n_pages && count >= 0 && count <= a.n_pages;
  auto ring_at = [&](long long i) {  // i below 2 n_pages
    return a.pool.ring[i >= a.n_pages ? i - a.n_pages : i];
  };
  if (tid == 0) s_popped = 0;
  uint32_t err = pool_ok ? 0u : KVQ_DEV_ERR_PAGE;
  Sums base{0, 0, 0};
  for (int b0 = 0; b0 < a.batch; b0 += nt) {
    const int b = b0 + tid, nb = min(nt, a.batch - b0);
    const Ask k = ask_of(a, b, pool_ok);
    if (k.bad) err |= KVQ_DEV_ERR_APPEND_RANGE;
    const Sums inc = warp_scan(Sums{k.r, k.need, k.back}, lane);
    __syncthreads();  // (the chunk before is done with the arrays)
    if (lane == 31) s_warp[warp] = inc;
    __syncthreads();
    const Sums w = warp_scan(lane < nw ? s_warp[lane] : Sums{0, 0, 0}, lane);  // every warp scans the warps' sums
    const int src = warp == 0 ? 0 : warp - 1;
    const Sums total{__shfl_sync(0xffffffffu, w.rows, 31), __shfl_sync(0xffffffffu, w.need, 31),
                     __shfl_sync(0xffffffffu, w.back, 31)};
    Sums before{__shfl_sync(0xffffffffu, w.rows, src), __shfl_sync(0xffffffffu, w.need, src),
                __shfl_sync(0xffffffffu, w.back, src)};
    if (warp == 0) before = Sums{0, 0, 0};
    const int row = base.rows + before.rows + inc.rows - k.r, need = base.need + before.need + inc.need - k.need;
    const long long back = base.back + before.back + inc.back - k.back;
    const bool ok = pool_ok && (k.need == 0 || need + k.need <= count) && (k.r == 0 || row + (long long)k.r <= a.max_rows);
    s_row[tid] = row; s_need[tid] = need; s_back[tid] = back;
    s_n[tid] = k.n; s_held[tid] = k.held;
    s_get[tid] = ok ? k.need : -1;
    s_put[tid] = count + back + k.back <= a.n_pages ? k.back : 0;  // (more than the pool holds: a state gone wrong)
    if (b < a.batch) {
      if (first) a.granted[b] = ok ? k.r : 0;
      if (!ok && pool_ok) err |= KVQ_DEV_ERR_NO_ROOM;
      if (ok && k.need) atomicAdd(&s_popped, k.need);
    }
    __syncthreads();
    // pages: a warp per sequence
    for (int i = blockIdx.x * nw + warp; i < nb; i += gridDim.x * nw) {
      const int get = s_get[i], put = s_put[i];
      int32_t* trow = a.table + (long long)(b0 + i) * per_seq;
      for (int j = lane; j < get; j += 32) {
        const int pg = ring_at((long long)head + s_need[i] + j);
        if (pg < 0 || pg >= a.n_pages) err |= KVQ_DEV_ERR_PAGE;
        trow[s_held[i] + j] = pg;
      }
      for (int j = lane; j < put; j += 32) {
        long long at = (long long)head + count + s_back[i] + j;  // below 3 n_pages
        while (at >= a.n_pages) at -= a.n_pages;
        a.pool.ring[at] = trow[j];
      }
    }
    // rows: a thread each
    const int r1 = min(base.rows + total.rows, a.max_rows);
    for (long long r = base.rows + (long long)blockIdx.x * nt + tid; r < r1; r += (long long)gridDim.x * nt) {
      int lo = 0, hi = nb - 1;  // the last sequence that starts at or before row r, with rows
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_row[mid] <= r) lo = mid; else hi = mid - 1;
      }
      const int j = int(r) - s_row[lo], pos = s_n[lo] + j;
      const bool ok = s_get[lo] >= 0;
      if (a.row_pos) a.row_pos[r] = pos;
      if (a.row_dst) a.row_dst[r] = ok ? (b0 + lo) * a.n_new_max + j : -1;
      if (a.row_slot) {
        int slot = -1;
        if (ok) {
          const int i = int(div_u32(uint32_t(pos), a.by_page)), held = s_held[lo];
          const int pg = i < held ? a.table[(long long)(b0 + lo) * per_seq + i] : ring_at((long long)head + s_need[lo] + i - held);
          if (pg >= 0 && pg < a.n_pages) slot = pg * P + pos - i * P;
          else err |= KVQ_DEV_ERR_PAGE;
        }
        a.row_slot[r] = slot;
      }
    }
    base = Sums{base.rows + total.rows, base.need + total.need, base.back + total.back};
  }
  for (long long r = (long long)min(base.rows, a.max_rows) + (long long)blockIdx.x * nt + tid; r < a.max_rows;
       r += (long long)gridDim.x * nt) {
    if (a.row_pos) a.row_pos[r] = 0;
    if (a.row_dst) a.row_dst[r] = -1;
    if (a.row_slot) a.row_slot[r] = -1;
  }
  const bool push = count + base.back <= a.n_pages;
  if (pool_ok && !push) err |= KVQ_DEV_ERR_PAGE;
  if (err) atomicOr(a.status, err);
  // ---- the last CTA: every other has read the lengths and the state
  __syncthreads();
  if (tid == 0) {
    __threadfence();
    s_last = gridDim.x == 1 || atomicAdd(&a.status[2], 1u) == gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (!s_last) return;
  if (a.seq_len_out)
    for (int b = tid; b < a.batch; b += nt) {
      const int n = a.seq_len[b];
      a.seq_len_out[b] = pool_ok && a.n_new[b] == KVQ_PAGE_RELEASE && n >= 0 && n <= a.max_ctx ? 0 : n;
    }
  if (tid == 0) {
    long long h = (long long)head + s_popped;
    if (h >= a.n_pages) h -= a.n_pages;
    a.pool.next[0] = pool_ok ? int(h) : head;
    a.pool.next[1] = pool_ok ? int(count - s_popped + (push ? base.back : 0)) : count;
    if (gridDim.x > 1) a.status[2] = 0;
  }
}

}  // namespace

cudaError_t launch_page_update(PageArgs a, cudaStream_t st) {
  a.by_page = make_divu32(uint32_t(a.page_tokens));
  // a thread per sequence up to 1024; CTAs for a row per thread (the sums are computed again in each,
  // which costs nothing while they run side by side)
  const int threads = std::min(kMaxPageThreads, std::max(128, (a.batch + 31) / 32 * 32));
  const int sms = device_sm_count();
  const int ctas = int(std::min<long long>(sms > 0 ? sms : 148, std::max<long long>(1, ((long long)a.max_rows + threads - 1) / threads)));
  return launch_dependent(page_update_kernel, unsigned(ctas), threads, 0, st, 1, a);
}

}  // namespace kvq
