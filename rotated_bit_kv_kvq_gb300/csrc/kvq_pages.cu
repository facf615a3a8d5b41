// Page table and row maps of a step from request lengths (kvq_page_update).
//
// Sequence b asks for r_b tokens behind its n_b: need_b = ceil((n_b + r_b) / P) -
// ceil(n_b / P) new pages.  Exclusive prefix sums over the sequences in order give
// where its pages start in the ring of free pages and where its rows start in the
// packed order; a released sequence's pages go behind the free ones, by a third sum.

#include <cuda_runtime.h>

#include "kvq_internal.h"

namespace kvq {
namespace {

constexpr int kPageThreads = 1024;  // sequences scanned at a time

struct Sums {
  long long rows, need, back;
};

// What sequence b asks for: r tokens (0 for a release or an invalid value).
struct Ask {
  int n, r, need, back;
  bool released;
};
__device__ __forceinline__ Ask ask_of(const PageArgs& a, int b, bool pool_ok) {
  Ask k{0, 0, 0, 0, false};
  if (b >= a.batch) return k;
  const int n = a.seq_len[b], r = a.n_new[b];
  const bool len_ok = n >= 0 && n <= a.max_ctx;
  k.n = len_ok ? n : 0;
  const int held = (k.n + a.page_tokens - 1) / a.page_tokens;
  if (r == KVQ_PAGE_RELEASE && len_ok) {
    k.back = pool_ok ? held : 0;
    k.released = pool_ok;
  } else if (len_ok && r >= 0 && r <= a.n_new_max && (long long)n + r <= a.max_ctx) {
    k.r = r;
    k.need = int(((long long)n + r + a.page_tokens - 1) / a.page_tokens) - held;
  } else {
    atomicOr(a.status, KVQ_DEV_ERR_APPEND_RANGE);
  }
  return k;
}

// exclusive prefix sums over the CTA; `total` gets the sums of all
__device__ __forceinline__ Sums scan(Sums v, Sums& total, long long (*s)[32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x[3] = {v.rows, v.need, v.back};
#pragma unroll
  for (int o = 1; o < 32; o <<= 1)
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      const long long y = __shfl_up_sync(0xffffffffu, x[i], o);
      if (lane >= o) x[i] += y;
    }
  __syncthreads();
  if (lane == 31)
#pragma unroll
    for (int i = 0; i < 3; ++i) s[i][warp] = x[i];
  __syncthreads();
  long long before[3] = {0, 0, 0}, all[3] = {0, 0, 0};
#pragma unroll
  for (int i = 0; i < 3; ++i)
    for (int w = 0; w < kPageThreads / 32; ++w) {
      before[i] += w < warp ? s[i][w] : 0;
      all[i] += s[i][w];
    }
  total = Sums{all[0], all[1], all[2]};
  return Sums{before[0] + x[0] - v.rows, before[1] + x[1] - v.need, before[2] + x[2] - v.back};
}

__global__ void __launch_bounds__(kPageThreads) page_update_kernel(PageArgs a) {
  __shared__ long long s_scan[3][32];
  __shared__ long long s_row[kPageThreads], s_need[kPageThreads], s_back[kPageThreads];
  __shared__ int s_n[kPageThreads], s_ok[kPageThreads], s_get[kPageThreads], s_put[kPageThreads];
  __shared__ long long s_popped;
  const int tid = threadIdx.x, P = a.page_tokens, per_seq = a.max_ctx / a.page_tokens;
  const int head = a.pool.state[0], count = a.pool.state[1];
  const bool pool_ok = head >= 0 && head < a.n_pages && count >= 0 && count <= a.n_pages;
  if (!pool_ok && tid == 0) atomicOr(a.status, KVQ_DEV_ERR_PAGE);
  if (tid == 0) s_popped = 0;
  Sums base{0, 0, 0};
  for (int b0 = 0; b0 < a.batch; b0 += kPageThreads) {
    const int b = b0 + tid, nb = min(kPageThreads, a.batch - b0);
    const Ask k = ask_of(a, b, pool_ok);
    Sums total;
    const Sums e = scan(Sums{k.r, k.need, k.back}, total, s_scan);
    const long long row = base.rows + e.rows, need = base.need + e.need, back = base.back + e.back;
    const bool ok = pool_ok && (k.need == 0 || need + k.need <= count) && (k.r == 0 || row + k.r <= a.max_rows);
    s_row[tid] = row; s_need[tid] = need; s_back[tid] = back;
    s_n[tid] = k.n;
    s_ok[tid] = ok;
    s_get[tid] = ok ? k.need : 0;
    s_put[tid] = count + back + k.back <= a.n_pages ? k.back : 0;  // (more than the pool holds: a state gone wrong)
    if (b < a.batch) {
      a.granted[b] = ok ? k.r : 0;
      if (a.seq_len_out) a.seq_len_out[b] = k.released ? 0 : a.seq_len[b];
      if (!ok && pool_ok) atomicOr(a.status, KVQ_DEV_ERR_NO_ROOM);
      if (ok && k.need) atomicAdd(reinterpret_cast<unsigned long long*>(&s_popped), (unsigned long long)k.need);
    }
    __syncthreads();
    const int warp = tid >> 5, lane = tid & 31;
    for (int i = warp; i < nb; i += kPageThreads / 32) {  // pages: a warp per sequence
      const int held = (s_n[i] + P - 1) / P, get = s_get[i], put = s_put[i];
      int32_t* trow = a.table + (long long)(b0 + i) * per_seq;
      for (int j = lane; j < get; j += 32) {
        const int pg = a.pool.ring[(head + s_need[i] + j) % a.n_pages];
        if (pg < 0 || pg >= a.n_pages) atomicOr(a.status, KVQ_DEV_ERR_PAGE);
        trow[held + j] = pg;
      }
      for (int j = lane; j < put; j += 32) a.pool.ring[(head + count + s_back[i] + j) % a.n_pages] = trow[j];
    }
    __syncthreads();  // this chunk's table entries are visible to the rows below
    const long long r1 = min(base.rows + total.rows, (long long)a.max_rows);
    for (long long r = base.rows + tid; r < r1; r += kPageThreads) {
      int lo = 0, hi = nb - 1;  // the last sequence that starts at or before row r, with rows
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_row[mid] <= r) lo = mid; else hi = mid - 1;
      }
      const int j = int(r - s_row[lo]), pos = s_n[lo] + j;
      const bool ok = s_ok[lo];
      const int pg = ok && a.row_slot ? a.table[(long long)(b0 + lo) * per_seq + pos / P] : -1;
      const bool in_pool = pg >= 0 && pg < a.n_pages;
      if (a.row_pos) a.row_pos[r] = pos;
      if (a.row_dst) a.row_dst[r] = ok ? (b0 + lo) * a.n_new_max + j : -1;
      if (a.row_slot) {
        a.row_slot[r] = in_pool ? pg * P + pos % P : -1;
        if (ok && !in_pool) atomicOr(a.status, KVQ_DEV_ERR_PAGE);
      }
    }
    base = Sums{base.rows + total.rows, base.need + total.need, base.back + total.back};
    __syncthreads();
  }
  for (long long r = min(base.rows, (long long)a.max_rows) + tid; r < a.max_rows; r += kPageThreads) {
    if (a.row_pos) a.row_pos[r] = 0;
    if (a.row_dst) a.row_dst[r] = -1;
    if (a.row_slot) a.row_slot[r] = -1;
  }
  if (tid == 0) {
    const bool push = pool_ok && count + base.back <= a.n_pages;
    if (pool_ok && !push) atomicOr(a.status, KVQ_DEV_ERR_PAGE);
    a.pool.next[0] = pool_ok ? int((head + s_popped) % a.n_pages) : head;
    a.pool.next[1] = pool_ok ? int(count - s_popped + (push ? base.back : 0)) : count;
  }
}

}  // namespace

cudaError_t launch_page_update(const PageArgs& a, cudaStream_t st) {
  page_update_kernel<<<1, kPageThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
