// What the kernels of kvq_chunk_attention share: the plan of a call.
//
// A row of work is a (token, query head of a KV head): the rows of a sequence, token by token and a token's heads together,
// are cut into items of `m` rows.  An item's keys lie between the smallest first key and the largest end of its rows; they
// are taken in tiles, of body keys first (from a multiple of the tile's size), then of tail rows (a tile ends where the ring
// wraps).  The items of all KV heads form one stream of tiles, with kChunkGap tiles' worth of nothing before each item (what a CTA
// needs to change items), cut into pieces of equal length, one CTA each.  An item in several pieces is merged by another
// kernel, in the order of the pieces, so that the result depends on nothing but the plan.
#pragma once

#include <math.h>

#include <algorithm>

#include "kvq_device.cuh"
#include "kvq_internal.h"

namespace kvq {

// (4: 530 us for 2 x 4096 prompt rows, 194 for 16 mixed sequences; 8: 513, 184; 14: 513, 184)
constexpr int kChunkGap = 8;       // tiles
constexpr int kChunkMinPiece = 2;  // tiles of the shortest piece (a call of 1,000 tokens: 1 16.4 us, 2 15.9, 4 18.4, 8 23.8)
constexpr float kChunkLog2e = 1.4426950408889634f;

struct ChunkItem {
  int b, r0, rows;        // sequence, first row of work (token * group + head) and their number
  int lo, hi;             // keys [lo, hi)
  int n_body, n_tail;     // tiles
  int pad;
  long long at;           // where the item begins in its KV head's stream
};
static_assert(sizeof(ChunkItem) == 40, "");

struct ChunkHeader {
  long long total;        // length of a KV head's stream
  long long piece;        // length of a piece
  int items, pieces, ok, pad;
};

struct ChunkArgs {
  kvq_cache c;
  kvq_score_mod mod;      // softcap in natural units, 0: none
  const void* q;
  void* out;
  const int32_t* row_start;
  int q_dtype, out_dtype, n_q_heads, n_rows, group, rot_k, rot_v;
  float scale;
  DivU32 by_group, by_tail, by_page;
  int pages_per_seq, ctas;
  int m, tile, tail_tile;     // rows of an item, keys of a body tile and of a tail tile
  // workspace
  ChunkHeader* head;
  int32_t* tiles0;        // [batch + 1]: items before sequence b
  ChunkItem* items;
  int32_t* first;         // [ctas]: the item in which a piece begins
  float* part;            // [2 * ctas][m][head_dim]: sums of weighted values, unnormalised
  float2* part_ml;        // [2 * ctas][m]: their reference (log2) and sum of weights
};

// What a kernel's items and tiles are: rows, keys, tail rows.
struct ChunkTiles {
  int m, tile, tail_tile;
};
// The kernels on tcgen05, with operands in one or two fp16 parts; one translation unit per head_dim.
#define KVQ_CHUNK_TC(D)                      \
  ChunkTiles chunk_tc_tiles_d##D(int parts); \
  cudaError_t launch_chunk_tc_d##D(ChunkArgs& a, int parts, cudaStream_t st);
KVQ_CHUNK_TC(64)
KVQ_CHUNK_TC(128)
KVQ_CHUNK_TC(192)
KVQ_CHUNK_TC(256)
KVQ_CHUNK_TC(320)
#undef KVQ_CHUNK_TC

inline long long chunk_max_items(const kvq_cache& c, long long work_rows, int m) { return work_rows / m + c.batch; }

// One tile of an item: first position, keys, body or tail.
struct ChunkTile {
  int t0, cnt;
  bool tail;
};
template <int TILE, int TAIL>  // (= a.tile, a.tail_tile)
__device__ __forceinline__ ChunkTile chunk_tile(const ChunkArgs& a, const ChunkItem& it, int n, int j) {
  const int T = a.c.tail_len, body_end = n - T;
  if (j < it.n_body) {
    const int t0 = (it.lo / TILE + j) * TILE;
    return ChunkTile{t0, min(TILE, min(it.hi, body_end) - t0), false};
  }
  j -= it.n_body;
  const int ts = max(it.lo, body_end), slot = ts - int(div_u32(uint32_t(ts), a.by_tail)) * T;
  const int first = min(T - slot, it.hi - ts), n1 = int(uint32_t(first + TAIL - 1) / TAIL);  // up to where the ring wraps
  const int t0 = ts + (j < n1 ? j * TAIL : first + (j - n1) * TAIL), end = j < n1 ? ts + first : it.hi;
  return ChunkTile{t0, min(TAIL, end - t0), true};
}

// The keys that a row sees: [lo, hi)
struct ChunkSpan {
  int lo, hi, pos;
};
__device__ __forceinline__ ChunkSpan chunk_span(const ChunkArgs& a, int b, int n, int row0, int m, int i) {  // token i of m
  const int pos = n - m + i;
  ChunkSpan s{0, 0, pos};
  if (pos < 0) return s;
  s.lo = a.mod.first_key ? max(0, a.mod.first_key[row0 + i]) : 0;
  s.hi = pos + 1;
  if (a.mod.prefix_len) s.hi = max(s.hi, min(a.mod.prefix_len[b], n));
  if (s.lo >= s.hi) s.lo = s.hi = 0;
  return s;
}

// A walk over a CTA's piece of the stream: its segments (item, KV head, tiles [j0, j1)), in order.
struct ChunkWalk {
  long long x, end;       // place in the stream
  int kvh, item;
  __device__ __forceinline__ void begin(const ChunkArgs& a, const ChunkHeader& h, int piece) {
    const long long all = h.total * a.c.n_kv_heads;
    x = min(all, piece * h.piece);
    end = min(all, x + h.piece);
    if (!h.ok || piece >= h.pieces) end = x;
    if (x >= end) return;
    kvh = int(x / h.total);
    item = a.first[piece];
  }
  // The next segment with tiles, or an item without any whose place is here; false: none left.
  __device__ __forceinline__ bool next(const ChunkArgs& a, const ChunkHeader& h, ChunkItem& it, int& head, int& j0, int& j1) {
    while (x < end) {
      if (item == h.items) { item = 0; ++kvh; }
      it = a.items[item];
      const long long at = kvh * h.total + it.at;
      const int nk = it.n_body + it.n_tail;
      const long long s0 = x - at - kChunkGap, s1 = end - at - kChunkGap;
      j0 = int(max(0LL, min((long long)nk, s0)));
      j1 = int(max(0LL, min((long long)nk, s1)));
      head = kvh;
      const bool begins = x <= at;
      x = at + kChunkGap + nk;
      ++item;
      if (j1 > j0 || (nk == 0 && begins)) return true;
    }
    return false;
  }
};

}  // namespace kvq
