// Host-side declarations shared by the kvq translation units.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <map>
#include <mutex>
#include <tuple>
#include <unordered_map>

#include "kvq.h"
#include "kvq_divu32.h"

namespace kvq {

struct Rot {
  int k;  // K (and query) rotation on
  int v;  // V rotation on (output rotated back)
};

// Hadamard group width used for a head: head_dim when it is a power of two,
// 64 for other multiples of 64, 32 when rotation is impossible (layout only).
inline int rotation_group(int d) {
  if (d >= 64 && d % 64 == 0) return (d & (d - 1)) == 0 ? d : 64;
  return 32;
}

size_t qs_row_bytes_host(int qt, int d);
// rows of the body planes
inline long long body_row_count(const kvq_cache& c) {
  return c.page_tokens ? (long long)c.n_pages * c.n_kv_heads * c.page_tokens
                       : (long long)c.batch * c.n_kv_heads * c.max_ctx;
}

// The tables below may throw (no memory for an entry), which a C entry point must not: their
// users return an error, or do without the table.

// Raises a kernel's dynamic shared-memory limit once per device (again only for
// a larger size), so that steady-state calls make no attribute call and can be
// captured into a CUDA graph.
inline cudaError_t ensure_dynamic_smem(const void* kernel, int bytes) try {
  constexpr int kMaxDevices = 64;
  static std::mutex mu;
  static std::unordered_map<const void*, int[kMaxDevices]> done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices) return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  std::lock_guard<std::mutex> lock(mu);
  int& have = done[kernel][dev];
  if (have >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) have = bytes;
  return e;
} catch (...) {
  return cudaErrorMemoryAllocation;
}

// Allows a kernel clusters of more than 8 CTAs, once per device.
inline cudaError_t allow_large_clusters(const void* kernel) try {
  constexpr int kMaxDevices = 64;
  static std::mutex mu;
  static std::unordered_map<const void*, bool[kMaxDevices]> done;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lock(mu);
  if (dev >= 0 && dev < kMaxDevices && done[kernel][dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && dev >= 0 && dev < kMaxDevices) done[kernel][dev] = true;
  return e;
} catch (...) {
  return cudaErrorMemoryAllocation;
}

// Launches a kernel as a programmatic dependent of what runs before it on the stream, in clusters
// of `cluster` CTAs.  Its CTAs may become resident before that has finished, so such a kernel begins
// with pdl_begin() (kvq_device.cuh), in every thread and ahead of every access to memory; what this
// saves is the launch latency between two calls.
template <class... P, class... A>
inline cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t st, int cluster,
                                    const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(unsigned(threads));
  cfg.dynamicSmemBytes = size_t(smem);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = unsigned(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// How many clusters of k CTAs of a kernel the device runs at once (a cluster stays within a
// group of SMs, and the groups differ in size), for k = 2 .. kMaxCluster; asked once per kernel,
// shared-memory size and device.  NULL when the query fails or there is no memory for the answer.
constexpr int kMaxCluster = 16;
struct ClusterLimits {
  int clusters[kMaxCluster + 1];
};
inline const ClusterLimits* cluster_limits(const void* kernel, int threads, int smem) try {
  static std::mutex mu;
  static std::map<std::tuple<const void*, int, int>, ClusterLimits> known;  // (a map's values never move)
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
  std::lock_guard<std::mutex> lock(mu);
  const auto key = std::make_tuple(kernel, smem, dev);
  const auto it = known.find(key);
  if (it != known.end()) return &it->second;
  ClusterLimits lim{};
  for (int k = 2; k <= kMaxCluster; ++k) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(k));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = size_t(smem);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = unsigned(k);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&lim.clusters[k], kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();  // (this size is not available)
      lim.clusters[k] = 0;
    }
  }
  return &known.emplace(key, lim).first->second;
} catch (...) {
  return nullptr;
}

// Launchers (arguments already validated by the API layer).
// SMs of the current device (0 when the query fails).
int device_sm_count();

cudaError_t launch_append(const kvq_cache& c, Rot rot, const void* k, const void* v, int in_dtype,
                          int n_new, const int32_t* n_new_per_seq, uint32_t flags, cudaStream_t st);
cudaError_t launch_debug(const kvq_cache& c, Rot rot, int seq, int kv_head, int which, int t0,
                         int count, int original_basis, float* out, void* blocks, cudaStream_t st);

// One CTA waiting (bounded) on a barrier that never completes: the failure path.
cudaError_t launch_wait_timeout(uint32_t* status, long long limit_cycles, cudaStream_t st);

// Decode: split plan shared by the workspace query and the launch.  The work is cut
// on the device, from seq_len, by cost: per plane (KV head x head group) every
// sequence's tail and body form one stream of bytes to read, cut into `pieces`
// equal pieces, one CTA each (with a fused step every tail gets a CTA of its own,
// which also writes the new tokens, and the bodies form the stream).
struct DecodePlan {
  int heads_per_cta;   // query heads handled by one CTA (<= 8)
  int head_groups;     // CTAs along the head axis per KV head
  int planes;          // n_kv_heads * head_groups
  int pieces;          // stream pieces per plane (one wave of CTAs)
  int pieces_fused;    // stream pieces per plane beside the batch's tail CTAs (fused step)
  int slots;           // partial slots per plane (pieces plus the cuts at segment ends)
  long long cost_body; // bytes of one body token of one (sequence, KV head)
  long long cost_tail; // bytes of one tail token
  long long cost_min;  // smallest piece
  long long cost_gap;  // virtual bytes before each segment: a CTA's cost of switching segments
  int sms;             // SMs the plan fills
  // With one full wave of three CTAs per SM the pieces are weighted by dispatch slot
  // (an SM's first, second, third CTA), so that the SM's CTAs end together.
  int slot_weight[3];
  bool weighted, weighted_fused;
  size_t hdr_bytes;    // fused-step partition header at the start of the workspace
  size_t ws_bytes;     // header, then acc [planes][slots][heads_per_cta][D], (m, l) [..][2],
                       // with outlier channels their acc [..][32]
};
// n_outlier > 0: the q4_0 / q5_0 / q8_0 pairs at head_dim 64, 128 and 256.
bool decode_supported(int d, int kt, int vt, int n_outlier);
DecodePlan plan_decode(const kvq_cache& c, int n_q_heads, int sm_count);
// Address of the fixed decode scratch array on the current device (looked up
// once per device); size in *bytes.
cudaError_t decode_noalloc_scratch(void** ptr, size_t* bytes);
// New tokens appended by the decode launch itself (the fused step): the one
// tail CTA of each (sequence, KV head) writes them before its tail attention,
// and the merge kernel advances seq_len.  Requires n_new <= tail_len, one head
// group and one tail split (fused_step_ok).
struct FusedAppend {
  const void* k;
  const void* v;
  int in_dtype;
  int n_new;
  const int32_t* n_new_per_seq;  // device, may be NULL
  int prerotated;
};
bool fused_step_ok(const kvq_cache& c, const DecodePlan& plan, int n_new);
// grid dimensions within the launch limits
bool decode_grid_ok(const kvq_cache& c, const DecodePlan& plan);
cudaError_t launch_decode(const kvq_cache& c, Rot rot, const DecodePlan& plan, const void* q,
                          int q_dtype, int n_q_heads, float scale, void* out, int out_dtype,
                          void* ws, cudaStream_t st, const FusedAppend* fa = nullptr);
// per-head_dim launchers (one translation unit each)
#define KVQ_DECODE_LAUNCHER(NAME)                                                                     \
  cudaError_t NAME(const kvq_cache& c, Rot rot, const DecodePlan& plan, const void* q, int q_dtype,  \
                   int n_q_heads, float scale, void* out, int out_dtype, void* ws, cudaStream_t st,  \
                   const FusedAppend* fa);
KVQ_DECODE_LAUNCHER(launch_decode_d64)
KVQ_DECODE_LAUNCHER(launch_decode_d128)
KVQ_DECODE_LAUNCHER(launch_decode_d192)
KVQ_DECODE_LAUNCHER(launch_decode_d256)
KVQ_DECODE_LAUNCHER(launch_decode_d320)
#undef KVQ_DECODE_LAUNCHER

// Prefill (tcgen05): head_dim 64 or 128, GQA group up to 128.  The workspace
// holds every 64-key tile of every (sequence, KV head) up to max_ctx, staged
// once as fp16 hi / lo operand tiles (512 * head_dim bytes per tile).
bool prefill_supported(int d, int group);
size_t prefill_workspace_bytes(const kvq_cache& c);
cudaError_t launch_prefill(const kvq_cache& c, Rot rot, const void* q, int q_dtype, int n_q_heads, int n_tokens,
                           const int32_t* q_pos0, int causal, float scale, void* out, int out_dtype,
                           void* ws, cudaStream_t st);

// Norms and position rotation of query / key rows (kvq_qk_norm_rope).
struct RopeArgs {
  const void* in[3];        // q, k, v rows (v may be NULL)
  long long stride[3];      // elements between rows
  void* out[3];
  const int32_t* pos;
  const int32_t* dst_row;   // may be NULL
  int n_rows, n_dst_rows, n_q_heads, n_kv_heads, head_dim;
  uint32_t* status;
};
cudaError_t launch_qk_norm_rope(const RopeArgs& a, const kvq_rope_norm& r, int dtype, cudaStream_t st);

struct PageArgs {
  const int32_t* seq_len;
  uint32_t* status;
  int32_t* table;
  int batch, max_ctx, page_tokens, n_pages;
  kvq_page_pool pool;
  const int32_t* n_new;
  int n_new_max, max_rows;
  int32_t* granted;
  int32_t* row_pos;
  int32_t* row_dst;
  int32_t* row_slot;
  int32_t* seq_len_out;
  DivU32 by_page;  // set at the launch
};
cudaError_t launch_page_update(PageArgs a, cudaStream_t st);

// Shared pages (kvq_page_fork, kvq_page_free, kvq_page_compact).
constexpr int kMaxPlanes = 7;
struct ShareArgs {
  const int32_t* seq_len;
  uint32_t* status;
  int32_t* table;
  int batch, max_ctx, page_tokens, n_pages;
  kvq_page_pool pool;
  kvq_page_share share;                // (NULL pointers: no counts)
  int n_planes, page_units;            // the planes of the body, and the units of a page's copy over all of them
  uint8_t* plane[kMaxPlanes];
  long long page_bytes[kMaxPlanes];
  int units[kMaxPlanes];
};
struct ForkArgs {
  kvq_cache c;                         // set at the launch, as what follows `seq_len_out`
  const int32_t *src, *dst, *n_tokens;  // n_tokens may be NULL
  int n_forks;
  int32_t *granted, *seq_len_out;
  int units, parts;                    // units of a fork's copy, and the CTAs that share them
  int tail_rows, tail_pieces;          // tail rows of a unit, units of a (side, KV head)
  DivU32 by_row;                       // pieces of 16 channels of a tail row
};
struct CompactArgs {
  int32_t *table_out, *ring_out, *map;
  int32_t *mark, *moves;               // [n_pages], [1 + 2 n_pages]
};
cudaError_t launch_page_fork(const kvq_cache& c, const kvq_page_pool& pool, const kvq_page_share& share, ForkArgs f,
                             cudaStream_t st);
cudaError_t launch_page_free(const kvq_cache& c, const kvq_page_pool& pool, const kvq_page_share& share, const int32_t* release,
                             int32_t* seq_len_out, cudaStream_t st);
cudaError_t launch_page_compact(const kvq_cache& c, const kvq_page_pool& pool, const kvq_page_share* share, CompactArgs m,
                                cudaStream_t st);

// Attention of packed rows of new tokens (kvq_chunk_attention).
struct ChunkCall {
  const kvq_score_mod* mod;            // may be NULL
  const void* q;
  int q_dtype, n_q_heads, n_rows;
  const int32_t* row_start;
  float scale;
  void* out;
  int out_dtype;
};
size_t chunk_workspace_bytes(const kvq_cache& c, int n_q_heads, int n_rows);
cudaError_t launch_chunk(const kvq_cache& c, Rot rot, const ChunkCall& a, void* ws, cudaStream_t st);

// Block index and sparse decode (the decode's head dims, no outlier channels).
constexpr int kMaxIndexBlocks = 49152;  // keys of a row in shared memory: 192 KB
cudaError_t launch_block_index_update(const kvq_cache& c, const kvq_block_index& x, int n_last, cudaStream_t st);
cudaError_t launch_select_blocks(const kvq_cache& c, Rot rot, const kvq_block_index& x, const void* q, int q_dtype,
                                 int n_q_heads, int n_first, int n_last, int n_select, int32_t* sel, cudaStream_t st);
cudaError_t launch_sparse_decode(const kvq_cache& c, Rot rot, const void* q, int q_dtype, int n_q_heads, float scale,
                                 int block_tokens, const int32_t* sel, int n_select, void* out, int out_dtype,
                                 cudaStream_t st);

}  // namespace kvq
