// Attention of packed rows of new tokens on tcgen05 (kvq_chunk_attention), included by one translation unit per head_dim.
//
// A CTA walks its piece of the plan's stream (kvq_chunk.cuh).  An item's 128 rows are the lanes of TMEM.  Roles:
//   producer      a warp: tiles of packed codes, headers and high bits (or bf16 tail rows) by TMA into a ring
//   converters    eight warps: a tile to fp16 operands, keys and values in the same layout (rows of 64 channels, 128-byte
//                 swizzle), which is K-major for Q K^T and, read along N, V for P V: nothing is transposed
//   S issuer      a thread: S = Q K^T, Q in TMEM (shared memory at head_dim 320)
//   P V issuer    a thread: O += P V, P in TMEM
//   softmax       one or two groups of four warps, a row per thread.  Two groups (small heads) take every other tile, each
//                 with its own running maximum, sum and accumulator, and are joined at the item's end: two chains of
//                 score -> weight -> product in flight, without a word between them.
//
// PARTS 1 (bf16 outputs): queries, keys, values and weights rounded once to fp16, 2^-11, an eighth of the output's step;
// PARTS 2 (fp16 and fp32): two fp16 parts each and three products, 22 bits.  Sums and softmax statistics are fp32.
// fp16's range is no limit: a row's queries, a tile's keys and a segment's values are scaled by powers of two taken from
// their largest values (a quantized tile's from its headers), and a segment's values keep the smallest scale met so far, O
// being brought down with it.  Weights are times 2^8.
//
// Channels lie in the order 0 2 1 3 within each four, as the codes' conversion leaves them, in Q, K and V alike; the
// epilogue reads O in that order.  A key with a header or tail value that is not finite is zeroed and noted, and the rows
// that see it are NaN at the end: 0 * NaN in the products would reach rows that do not.
//
// Every wait is bounded: one that gives up sets the status word's timeout bit and a flag that ends the other waits; the
// roles then run through their loops without waiting, so that no barrier between warps is left alone.
#pragma once

#include <string.h>

#include <type_traits>

#include "kvq_chunk.cuh"
#include "kvq_decode_impl.cuh"
#include "kvq_tcgen05.cuh"

namespace kvq {
namespace {

constexpr long long kTcWait = 2000000000LL;  // ~1 s per wait
constexpr float kTcLazy = 7.0f;              // log2: weights stay below 2^(8 + 7)
constexpr int kTcMaxStages = 8;
constexpr int kTcMeta = 8;
constexpr int kTcConv = 8;                   // converter warps

template <int D, int PARTS>
struct TC {
  static constexpr int NG = D <= 64 * (3 - PARTS) ? 2 : 1;     // groups of softmax warps, each with an O of its own
  static constexpr int TK = D == 320 ? 32 : 64;                // keys of a tile
  static constexpr int TT = D <= 128 ? 32 : 16;                // tail rows of a tile
  static constexpr bool QSMEM = D == 320;                      // (TMEM: O takes 320 columns)
  static constexpr bool OVER = D == 256;                       // P over S (TMEM again)
  static constexpr int G = (D & (D - 1)) == 0 ? D : 64, GC = G / 32, NB = D / 32;
  static constexpr int kSoft = NG * 128, kThreads = kSoft + (kTcConv + 3) * 32;
  // TMEM columns
  static constexpr int qcol = 0, ocol = QSMEM ? 0 : PARTS * D / 2, scol = ocol + NG * D;
  static constexpr int pw = PARTS * TK / 2, pcol = OVER ? scol : scol + 2 * TK, pstep = OVER ? TK : pw;
  static_assert((OVER ? scol + 2 * TK : pcol + 2 * pw) <= 512, "TMEM columns");
  // shared memory
  static constexpr int part = D * TK * 2, slot = PARTS * part;  // a tile's operand
  static constexpr int off_q = 0, off_k = QSMEM ? PARTS * D * 256 : 0, off_v = off_k + 2 * slot, off_ring = off_v + 2 * slot;
  static constexpr int N1 = D > 256 ? 192 : D, N2 = D - N1;     // P V as one or two instructions
};

struct TcStage {  // offsets in a stage of the ring: K codes, V codes (1024-aligned), headers, high bits; or K and V tail rows
  int v, kd, vd, kqh, vqh, vt, bytes, stages;
  int kh, vh;     // header bytes of a row
  uint32_t tx;
};

struct TcMeta {
  int t0, cnt, ks, vs;  // position of column 0, its keys, the powers of two that keys and values were multiplied by
  uint32_t bad[2];      // keys that are not finite
};

struct TcSync {
  uint64_t rfull[kTcMaxStages], rempty[kTcMaxStages];
  uint64_t kfull[2], kempty[2], vfull[2], vempty[2], sfull[2], sfree[2], pfull[2], odone[2], qready, tmax, fin[2];
  int4 job[kTcMaxStages];  // first position, keys (-1: the end), tail slot or -1, first tile of a segment
  TcMeta meta[kTcMeta];
  uint32_t tail_max[2][kTcConv][2];
  float rowmax[2][128];
  float4 join[2][128];     // a group's (reference, sum, value scale, NaN) of each row
  uint32_t tmem;
  int abort;
};

// Bounded wait; false once any wait of the CTA has given up.
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity, TcSync* sy, uint32_t* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity, 20000u)) {
    if (*reinterpret_cast<volatile int*>(&sy->abort)) return false;
    if (clock64() - t0 > kTcWait) {
      *reinterpret_cast<volatile int*>(&sy->abort) = 1;
      atomicOr(status, KVQ_DEV_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}

__device__ __forceinline__ float tc_pow2(int e) {  // clamped to normal numbers
  return __uint_as_float(uint32_t(127 + max(-126, min(126, e))) << 23);
}
__device__ __forceinline__ int tc_exp(float x) { return int(__float_as_uint(x) >> 23) - 126; }  // x < 2^this (x > 0, finite)
__device__ __forceinline__ uint32_t tc_lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t tc_lds16(uint32_t a) {
  uint16_t r;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ uint4 tc_lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
  return r;
}
__device__ __forceinline__ uint32_t tc_pack_bf2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void tc_sts128(uint32_t a, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

// ---- conversion ------------------------------------------------------------------------------------

// The fp16 pair code * d + m (d, m pairs), as one or two parts
template <int PARTS, bool MIN>
__device__ __forceinline__ void tc_value(uint32_t code, uint32_t d, uint32_t m, uint32_t& hi, uint32_t& lo) {
  if constexpr (!MIN) {
    hi = hmul2_bits(code, d);
    if constexpr (PARTS == 2)  // what the rounding left: exact, or below fp16's smallest step
      asm("{\n\t.reg .b32 nh;\n\tneg.f16x2 nh, %3;\n\tfma.rn.f16x2 %0, %1, %2, nh;\n\t}" : "=r"(lo) : "r"(code), "r"(d), "r"(hi));
  } else if constexpr (PARTS == 1) {
    hi = hfma2_bits(code, d, m);
  } else {
    const float2 c = __half22float2(u32_as_h2(code)), x = __half22float2(u32_as_h2(d)), y = __half22float2(u32_as_h2(m));
    split_h2(fmaf(c.x, x.x, y.x), fmaf(c.y, x.y, y.y), hi, lo);
  }
}

// 32 keys x 32 channels (block blk) of a body tile: lane = key.  dst: the operand's tile.
template <int D, int PARTS, int QT, bool KSIDE>
__device__ __forceinline__ void tc_body_unit(uint32_t codes, uint32_t hdr, uint32_t qh, uint32_t dst, int key, int blk, bool ok,
                                             float scale) {
  using C = TC<D, PARTS>;
  constexpr int TK = C::TK, NB = C::NB, ROW = QT == KVQ_TYPE_Q8_0 ? D : D / 2, W = box_w(ROW);
  constexpr bool MIN = type_has_min(QT), HIGH = type_has_qh(QT);
  uint32_t d, m = 0;
  {
    float fd, fm = 0.0f;
    if constexpr (MIN) {
      const float2 f = __half22float2(u32_as_h2(tc_lds32(hdr + (key * NB + blk) * 4)));
      fd = f.x;
      fm = f.y;
    } else {
      fd = __half2float(__ushort_as_half(uint16_t(tc_lds16(hdr + (key * NB + blk) * 2))));
    }
    if (!ok || !(fabsf(fd) <= 65504.0f) || !(fabsf(fm) <= 65504.0f)) fd = fm = 0.0f;
    d = pack_h2(fd * scale, fd * scale);
    if constexpr (MIN) m = pack_h2(fm * scale, fm * scale);
  }
  uint32_t w[QT == KVQ_TYPE_Q8_0 ? 8 : 4];
#pragma unroll
  for (int i = 0; i < (QT == KVQ_TYPE_Q8_0 ? 2 : 1); ++i) {
    const uint4 v = tc_lds128(codes + swz_off<W>(key, QT == KVQ_TYPE_Q8_0 ? 32 * blk + 16 * i : 16 * blk, TK));
    w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
  }
  uint32_t hb = 0, hv[2] = {0, 0};
  if constexpr (HIGH && KSIDE) hb = tc_lds32(qh + (key * NB + blk) * 4);
  if constexpr (HIGH && !KSIDE) {
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const uint32_t x = tc_lds16(qh + ((((key >> 1) * NB + blk) * 2 + p) * 2 + (key & 1)) * 2);
      hv[p] = x | x << 14;  // bits b and b + 2 of the part 16 apart
    }
  }
  constexpr int OFFC = MIN ? 0 : type_code_offset(QT);
  constexpr uint32_t OFF = (0x6400u + uint32_t(OFFC)) * 0x10001u, OFF16 = neg_off_x16_bits(OFFC);
  const uint32_t row = dst + (blk / 2) * (TK * 128) + key * 128;
#pragma unroll
  for (int c = 0; c < 4; ++c) {  // channels 8c .. 8c + 7 of the block
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t code[2];
      if constexpr (QT == KVQ_TYPE_Q8_0) {
        code[0] = i8_pair<0, 2>(w[2 * c + i]);
        code[1] = i8_pair<1, 3>(w[2 * c + i]);
      } else {
        const uint32_t x = w[2 * (c & 1) + i];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t magic = 0x64006400u;
          if constexpr (HIGH) {
            // the pair's bits go to bits 4 and 20 (first half of the block) or 8 and 24
            const int to = c < 2 ? 4 : 8;
            const int from = KSIDE ? 8 * (c & 1) + 4 * (c >> 1) + 2 * i + e : 8 * i + 4 * (c >> 1) + e;
            const uint32_t src = KSIDE ? hb : hv[c & 1];
            uint32_t r;
            if constexpr (KSIDE) r = __funnelshift_r(src, src, (from - to) & 31);  // (the word is full: rotate)
            else r = from >= to ? src >> (from - to) : src << (to - from);
            magic |= r & (c < 2 ? 0x00100010u : 0x01000100u);
          }
          const uint32_t y = e ? x >> 8 : x;
          code[e] = c < 2 ? nib_pair(y, 0, magic, OFF) : nib_pair_x16(y, magic, OFF16);
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) tc_value<PARTS, MIN>(code[e], d, m, hi[2 * i + e], lo[2 * i + e]);
    }
    const uint32_t at = row + ((((blk & 1) * 4 + c) ^ (key & 7)) << 4);
    tc_sts128(at, hi);
    if constexpr (PARTS == 2) tc_sts128(at + C::part, lo);
  }
}

// The same of a tail tile (bf16 rows, 128-byte box columns of TT rows)
template <int D, int PARTS>
__device__ __forceinline__ void tc_tail_unit(uint32_t rows, uint32_t dst, int key, int blk, bool ok, float scale) {
  using C = TC<D, PARTS>;
  const uint32_t row = dst + (blk / 2) * (C::TK * 128) + key * 128;
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t hi[4] = {0u, 0u, 0u, 0u}, lo[4] = {0u, 0u, 0u, 0u};
    if (ok) {
      const uint4 v = tc_lds128(rows + swz_off<128>(key, 64 * blk + 16 * c, C::TT));
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x[4] = {__uint_as_float(w[2 * i] << 16), __uint_as_float(w[2 * i] & 0xFFFF0000u),
                      __uint_as_float(w[2 * i + 1] << 16), __uint_as_float(w[2 * i + 1] & 0xFFFF0000u)};
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = fabsf(x[e]) <= 3.4e38f ? x[e] * scale : 0.0f;
        if constexpr (PARTS == 1) {
          hi[2 * i] = pack_h2(x[0], x[2]);
          hi[2 * i + 1] = pack_h2(x[1], x[3]);
        } else {
          split_h2(x[0], x[2], hi[2 * i], lo[2 * i]);
          split_h2(x[1], x[3], hi[2 * i + 1], lo[2 * i + 1]);
        }
      }
    }
    const uint32_t at = row + ((((blk & 1) * 4 + c) ^ (key & 7)) << 4);
    tc_sts128(at, hi);
    if constexpr (PARTS == 2) tc_sts128(at + C::part, lo);
  }
}

// Largest magnitude that a body tile's values can have, from the headers of its cnt rows; finite ones alone with `only`.
// raw: the largest header bits (halves: scales, and minima of the types that have them).
template <int D>
__device__ __forceinline__ float tc_body_bound(uint32_t hdr, int qt, int words, bool only, int lane, uint32_t& raw) {
  uint32_t mx = 0;
  for (int i = lane; i < words; i += 32) {
    uint32_t w = tc_lds32(hdr + 4 * i) & 0x7FFF7FFFu;
    if (only) {
      if ((w & 0xFFFFu) >= 0x7C00u) w &= 0xFFFF0000u;
      if ((w >> 16) >= 0x7C00u) w &= 0xFFFFu;
    }
    mx = __vmaxu2(mx, w);
  }
  const uint32_t a = __reduce_max_sync(0xffffffffu, mx & 0xFFFFu), b = __reduce_max_sync(0xffffffffu, mx >> 16);
  raw = max(a, b);
  const float fa = __half2float(__ushort_as_half(uint16_t(a))), fb = __half2float(__ushort_as_half(uint16_t(b)));
  switch (qt) {
    case KVQ_TYPE_Q4_0: return 8.0f * fmaxf(fa, fb);
    case KVQ_TYPE_Q5_0: return 16.0f * fmaxf(fa, fb);
    case KVQ_TYPE_Q8_0: return 128.0f * fmaxf(fa, fb);
    case KVQ_TYPE_Q4_1: return fmaf(15.0f, fa, fb);
    default: return fmaf(31.0f, fa, fb);
  }
}

template <int D, int PARTS>
__device__ void tc_convert(const ChunkArgs& a, const TcStage& L, uint8_t* sm, TcSync* sy, int warp, int lane) {
  using C = TC<D, PARTS>;
  constexpr int TK = C::TK, NB = C::NB, U = (TK + 31) / 32 * NB;  // units of a side
  uint32_t* status = a.c.status;
  const uint32_t sb = smem_u32(sm), ring = sb + C::off_ring;
  int vs = 0;
  uint32_t tails = 0;
  for (int ct = 0;; ++ct) {
    const int r = ct % L.stages, b = ct & 1;
    const uint32_t u = uint32_t(ct) >> 1;
    if (!tc_wait(&sy->rfull[r], (ct / L.stages) & 1, sy, status)) break;
    const uint4 jw = tc_lds128(smem_u32(&sy->job[r]));
    const int4 job = make_int4(int(jw.x), int(jw.y), int(jw.z), int(jw.w));
    if (job.y < 0) break;
    const uint32_t st = ring + r * L.bytes;
    const int cnt = job.y;
    const bool tail = job.z >= 0;
    // ---- scales
    float kb = 0.0f, vb = 0.0f;
    bool odd = false;  // something is not finite
    if (!tail) {
      uint32_t kraw, vraw;
      kb = tc_body_bound<D>(st + L.kd, a.c.k_type, cnt * L.kh / 4, false, lane, kraw);
      vb = tc_body_bound<D>(st + L.vd, a.c.v_type, cnt * L.vh / 4, false, lane, vraw);
      odd = kraw >= 0x7C00u || vraw >= 0x7C00u;
      if (odd) {
        kb = tc_body_bound<D>(st + L.kd, a.c.k_type, cnt * L.kh / 4, true, lane, kraw);
        vb = tc_body_bound<D>(st + L.vd, a.c.v_type, cnt * L.vh / 4, true, lane, vraw);
      }
    } else {  // every warp some rows' largest values, finite ones and any
      uint32_t mx[2] = {0, 0}, any = 0;
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        const uint32_t base = st + (side ? L.vt : 0);
        for (int i = warp * 32 + lane; i < cnt * (D / 8); i += kTcConv * 32) {
          const uint4 v = tc_lds128(base + swz_off<128>(i / (D / 8), i % (D / 8) * 16, C::TT));
          const uint32_t w[4] = {v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu, v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t lo = w[e] & 0xFFFFu, hi = w[e] >> 16;
            any |= uint32_t(lo >= 0x7F80u || hi >= 0x7F80u);
            mx[side] = max(mx[side], max(lo >= 0x7F80u ? 0u : lo, hi >= 0x7F80u ? 0u : hi));
          }
        }
        mx[side] = __reduce_max_sync(0xffffffffu, mx[side]);
      }
      any = __reduce_or_sync(0xffffffffu, any);
      const int p = tails & 1;
      if (lane == 0) {
        sy->tail_max[p][warp][0] = mx[0] | any << 31;
        sy->tail_max[p][warp][1] = mx[1];
        mbar_arrive(&sy->tmax);
      }
      if (!tc_wait(&sy->tmax, p, sy, status)) break;
      ++tails;
      uint32_t k = 0, v = 0;
#pragma unroll
      for (int w = 0; w < kTcConv; ++w) {
        const uint32_t x = reinterpret_cast<volatile uint32_t*>(sy->tail_max[p][w])[0];
        odd |= (x >> 31) != 0;
        k = max(k, x & 0x7FFFu);
        v = max(v, reinterpret_cast<volatile uint32_t*>(sy->tail_max[p][w])[1]);
      }
      kb = bf16_bits_to_f32(k);
      vb = bf16_bits_to_f32(v);
    }
    const int ks = kb > 0.0f ? min(15 - tc_exp(kb), 120) : 0;
    if (job.w) vs = vb > 0.0f ? min(13 - tc_exp(vb), 120) : 120;
    else if (vb > 0.0f && vs > 15 - tc_exp(vb)) vs = 13 - tc_exp(vb);
    const float kscale = tc_pow2(ks), vscale = tc_pow2(vs);
    if (warp == 0) {
      uint32_t bad[2] = {0u, 0u};
      if (odd) {
#pragma unroll
        for (int h = 0; h < (TK + 31) / 32; ++h) {
          const int key = 32 * h + lane;
          bool is = false;
          if (key < cnt && !tail) {
            for (int i = 0; i < L.kh / 2; ++i) is |= (tc_lds16(st + L.kd + key * L.kh + 2 * i) & 0x7FFFu) >= 0x7C00u;
            for (int i = 0; i < L.vh / 2; ++i) is |= (tc_lds16(st + L.vd + key * L.vh + 2 * i) & 0x7FFFu) >= 0x7C00u;
          } else if (key < cnt) {
            for (int i = 0; i < 2 * D; ++i) {
              const uint32_t base = st + (i >= D ? L.vt : 0);
              is |= (tc_lds16(base + swz_off<128>(key, (i % D) * 2, C::TT)) & 0x7FFFu) >= 0x7F80u;
            }
          }
          bad[h] = __ballot_sync(0xffffffffu, is);
        }
      }
      if (lane == 0) {
        volatile TcMeta* m = &sy->meta[ct % kTcMeta];
        m->t0 = job.x; m->cnt = cnt; m->ks = ks; m->vs = vs;
        m->bad[0] = bad[0]; m->bad[1] = bad[1];
      }
    }
    // ---- keys, then values
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      uint64_t* empty = side ? &sy->vempty[b] : &sy->kempty[b];
      if (u > 0 && !tc_wait(empty, (u - 1) & 1, sy, status)) goto out;
      const uint32_t dst = sb + (side ? C::off_v : C::off_k) + b * C::slot;
      for (int i = (warp + (side ? U : 0)) % kTcConv; i < U; i += kTcConv) {  // (with few units the sides take other warps)
        const int h = i / NB, blk = i - h * NB, key = 32 * h + lane;
        const bool ok = key < cnt;
        if (tail) {
          if (side == 0 && h > 0) continue;  // (scores of keys past the end are masked)
          tc_tail_unit<D, PARTS>(st + (side ? L.vt : 0), dst, key, blk, ok, side ? vscale : kscale);
        } else {
#define KVQ_UNIT(QT)                                                                                                          \
  case QT:                                                                                                                    \
    if (side == 0) tc_body_unit<D, PARTS, QT, true>(st, st + L.kd, st + L.kqh, dst, key, blk, ok, kscale);                    \
    else tc_body_unit<D, PARTS, QT, false>(st + L.v, st + L.vd, st + L.vqh, dst, key, blk, ok, vscale);                       \
    break;
          switch (side ? a.c.v_type : a.c.k_type) {
            KVQ_UNIT(KVQ_TYPE_Q4_0)
            KVQ_UNIT(KVQ_TYPE_Q5_0)
            KVQ_UNIT(KVQ_TYPE_Q8_0)
            KVQ_UNIT(KVQ_TYPE_Q4_1)
            KVQ_UNIT(KVQ_TYPE_Q5_1)
          }
#undef KVQ_UNIT
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(side ? &sy->vfull[b] : &sy->kfull[b]);
        if (side) mbar_arrive(&sy->rempty[r]);
      }
    }
  }
out:;
}

// ---- producer --------------------------------------------------------------------------------------

template <int D, int PARTS>
__device__ void tc_produce(const ChunkArgs& a, const TcStage& L, const ChunkHeader& h, uint8_t* sm, TcSync* sy, int lane,
                           const CUtensorMap* tmK, const CUtensorMap* tmV, const CUtensorMap* tmKt, const CUtensorMap* tmVt) {
  using C = TC<D, PARTS>;
  constexpr int TK = C::TK, NB = C::NB;
  const kvq_cache& c = a.c;
  const int T = c.tail_len;
  int ct = 0;
  bool ok = true;
  auto put = [&](int4 job, int row) {  // one lane
    const int r = ct % L.stages;
    if (ct >= L.stages && !tc_wait(&sy->rempty[r], (ct / L.stages - 1) & 1, sy, c.status)) return false;
    volatile int4* j = reinterpret_cast<volatile int4*>(&sy->job[r]);
    j->x = job.x; j->y = job.y; j->z = job.z; j->w = job.w;
    uint8_t* st = sm + C::off_ring + r * L.bytes;
    if (job.y <= 0) {  // the end, or a page outside the pool
      mbar_arrive(&sy->rfull[r]);
    } else if (job.z >= 0) {
      mbar_arrive_expect_tx(&sy->rfull[r], 2 * C::TT * 2 * D);
      tma_3d_g2s(st, tmKt, row, &sy->rfull[r]);
      tma_3d_g2s(st + L.vt, tmVt, row, &sy->rfull[r]);
    } else {
      mbar_arrive_expect_tx(&sy->rfull[r], L.tx);
      tma_3d_g2s(st, tmK, row, &sy->rfull[r]);
      tma_3d_g2s(st + L.v, tmV, row, &sy->rfull[r]);
      bulk_g2s(st + L.kd, static_cast<const uint8_t*>(c.k_d) + size_t(row) * L.kh, TK * L.kh, &sy->rfull[r]);
      bulk_g2s(st + L.vd, static_cast<const uint8_t*>(c.v_d) + size_t(row) * L.vh, TK * L.vh, &sy->rfull[r]);
      if (c.k_qh) bulk_g2s(st + L.kqh, static_cast<const uint32_t*>(c.k_qh) + size_t(row) * NB, TK * NB * 4, &sy->rfull[r]);
      if (c.v_qh) bulk_g2s(st + L.vqh, static_cast<const uint32_t*>(c.v_qh) + size_t(row) * NB, TK * NB * 4, &sy->rfull[r]);
    }
    return true;
  };
  ChunkWalk walk;
  walk.begin(a, h, blockIdx.x);
  ChunkItem it;
  int kvh, j0, j1;
  while (ok && walk.next(a, h, it, kvh, j0, j1)) {
    const int n = min(max(c.seq_len[it.b], 0), c.max_ctx);
    const int bh = it.b * c.n_kv_heads + kvh;
    for (int jb = j0; ok && jb < j1; jb += 32) {
      // a lane a tile: its rows, so that the page table's loads overlap
      int4 job = make_int4(0, 0, -1, 0);
      int row = 0;
      if (jb + lane < j1) {
        const ChunkTile t = chunk_tile(a, it, n, jb + lane);
        job = make_int4(t.t0, t.cnt, -1, jb + lane == j0);
        if (t.tail) {
          job.z = t.t0 - int(div_u32(uint32_t(t.t0), a.by_tail)) * T;
          row = bh * T + job.z;
        } else if (!c.page_tokens) {
          row = bh * c.max_ctx + t.t0;
        } else {
          const int i = int(div_u32(uint32_t(t.t0), a.by_page)), pg = c.page_table[(long long)it.b * a.pages_per_seq + i];
          if (pg >= 0 && pg < c.n_pages) {
            row = (pg * c.n_kv_heads + kvh) * c.page_tokens + t.t0 - i * c.page_tokens;
          } else {
            atomicOr(c.status, KVQ_DEV_ERR_PAGE);
            job.y = 0;
          }
        }
      }
      for (int k = 0; k < 32 && jb + k < j1; ++k) {
        const int4 x = make_int4(__shfl_sync(0xffffffffu, job.x, k), __shfl_sync(0xffffffffu, job.y, k),
                                 __shfl_sync(0xffffffffu, job.z, k), __shfl_sync(0xffffffffu, job.w, k));
        const int rw = __shfl_sync(0xffffffffu, row, k);
        int fine = 1;
        if (lane == 0) fine = put(x, rw);
        if (!__shfl_sync(0xffffffffu, fine, 0)) { ok = false; break; }
        ++ct;
      }
    }
  }
  if (lane == 0) {
    if (ok) put(make_int4(0, -1, -1, 0), 0);
    // copies still landing when a wait gave up: they end before the CTA does
    if (!ok)
      for (int k = max(0, ct - L.stages); k < ct; ++k) mbar_wait_bounded(&sy->rfull[k % L.stages], (k / L.stages) & 1, kTcWait);
  }
}

// ---- issuers ---------------------------------------------------------------------------------------

template <int D, int PARTS>
__device__ void tc_issue_s(const ChunkArgs& a, const ChunkHeader& h, uint32_t sb, uint32_t tmem, TcSync* sy) {
  using C = TC<D, PARTS>;
  constexpr uint32_t idesc = tc::idesc_f16_f32(128, C::TK);
  const uint64_t dk = tc::sdesc_sw128(sb + C::off_k), dq = tc::sdesc_sw128(sb + C::off_q);
  ChunkWalk walk;
  walk.begin(a, h, blockIdx.x);
  ChunkItem it;
  int kvh, j0, j1, ct = 0, seg = 0;
  bool ok = true;
  while (ok && walk.next(a, h, it, kvh, j0, j1)) {
    if (j1 == j0) continue;
    ok = tc_wait(&sy->qready, seg++ & 1, sy, a.c.status);
    for (int j = j0; ok && j < j1; ++j, ++ct) {
      const int b = ct & 1;
      const uint32_t u = uint32_t(ct) >> 1;
      ok = tc_wait(&sy->kfull[b], u & 1, sy, a.c.status) &&
           (u == 0 || tc_wait(C::OVER ? &sy->odone[b] : &sy->sfree[b], (u - 1) & 1, sy, a.c.status));
      if (!ok) break;
      tc::fence_after_sync();
      const uint64_t kb = dk + ((b * C::slot) >> 4);
      const uint32_t d = tmem + C::scol + b * C::TK;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        const uint32_t ko = ((ks / 4) * (C::TK * 128) + (ks % 4) * 32) >> 4;
        const uint32_t qo = ((ks / 4) * (128 * 128) + (ks % 4) * 32) >> 4;
        auto mma = [&](int qp, int kp, uint32_t acc) {
          if constexpr (C::QSMEM) tc::mma_f16(d, dq + qo + ((qp * D * 256) >> 4), kb + ko + ((kp * C::part) >> 4), idesc, acc);
          else tc::mma_f16_ts(d, tmem + C::qcol + qp * (D / 2) + ks * 8, kb + ko + ((kp * C::part) >> 4), idesc, acc);
        };
        mma(0, 0, ks > 0 ? 1u : 0u);
        if constexpr (PARTS == 2) {
          mma(0, 1, 1u);
          mma(1, 0, 1u);
        }
      }
      tc::commit(&sy->sfull[b]);
      tc::commit(&sy->kempty[b]);
    }
  }
  tc::commit(&sy->fin[0]);
}

template <int D, int PARTS>
__device__ void tc_issue_pv(const ChunkArgs& a, const ChunkHeader& h, uint32_t sb, uint32_t tmem, TcSync* sy) {
  using C = TC<D, PARTS>;
  constexpr uint32_t idesc1 = tc::idesc_f16_f32(128, C::N1) | tc::kIdescBmn;
  constexpr uint32_t idesc2 = tc::idesc_f16_f32(128, C::N2 > 0 ? C::N2 : 16) | tc::kIdescBmn;
  const uint64_t dv = tc::sdesc_sw128_mn(sb + C::off_v, C::TK * 128);
  ChunkWalk walk;
  walk.begin(a, h, blockIdx.x);
  ChunkItem it;
  int kvh, j0, j1, ct = 0;
  bool ok = true;
  while (ok && walk.next(a, h, it, kvh, j0, j1)) {
    for (int j = j0; ok && j < j1; ++j, ++ct) {
      const int b = ct & 1;
      const uint32_t u = uint32_t(ct) >> 1;
      ok = tc_wait(&sy->pfull[b], u & 1, sy, a.c.status) && tc_wait(&sy->vfull[b], u & 1, sy, a.c.status);
      if (!ok) break;
      tc::fence_after_sync();
      const uint64_t vb = dv + ((b * C::slot) >> 4);
      const uint32_t o = tmem + C::ocol + (C::NG == 2 ? b * D : 0), p = tmem + C::pcol + b * C::pstep;
      const uint32_t first = j - j0 < C::NG ? 0u : 1u;  // the group's first tile of the segment begins a new sum
#pragma unroll
      for (int ks = 0; ks < C::TK / 16; ++ks) {
        auto mma = [&](int pp, int vp, uint32_t acc) {
          const uint64_t v = vb + ((vp * C::part + ks * 2048) >> 4);
          tc::mma_f16_ts(o, p + pp * (C::TK / 2) + ks * 8, v, idesc1, acc);
          if constexpr (C::N2 > 0)
            tc::mma_f16_ts(o + C::N1, p + pp * (C::TK / 2) + ks * 8, v + (((C::N1 / 64) * C::TK * 128) >> 4), idesc2, acc);
        };
        mma(0, 0, ks > 0 ? 1u : first);
        if constexpr (PARTS == 2) {
          mma(0, 1, 1u);
          mma(1, 0, 1u);
        }
      }
      tc::commit(&sy->odone[b]);
      tc::commit(&sy->vempty[b]);
    }
  }
  tc::commit(&sy->fin[1]);
}

// ---- softmax ---------------------------------------------------------------------------------------

// In-place Hadamard of 32 values in natural order
__device__ __forceinline__ void tc_fwht32(float (&v)[32]) {
#pragma unroll
  for (int h = 1; h < 32; h <<= 1)
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if ((j & h) == 0) {
        const float x = v[j], y = v[j + h];
        v[j] = x + y;
        v[j + h] = x - y;
      }
}
// ... of GC values 32 channels apart, for 8 channels at once
template <int GC>
__device__ __forceinline__ void tc_fwht_chunks(float (&v)[GC][8]) {
#pragma unroll
  for (int h = 1; h < GC; h <<= 1)
#pragma unroll
    for (int k = 0; k < GC; ++k)
      if ((k & h) == 0)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = v[k][e], y = v[k + h][e];
          v[k][e] = x + y;
          v[k + h][e] = x - y;
        }
}

template <int D, int PARTS>
__device__ void tc_softmax(const ChunkArgs& a, const ChunkHeader& h, uint8_t* sm, uint32_t tmem, TcSync* sy, int warp, int lane) {
  using C = TC<D, PARTS>;
  constexpr int TK = C::TK, NG = C::NG;
  uint32_t* status = a.c.status;
  const int grp = NG == 2 ? warp / 4 : 0, row = (warp & 3) * 32 + lane;
  const uint32_t lanes = tmem + (uint32_t((warp & 3) * 32) << 16);
  auto all = [&]() {  // the softmax warps, TMEM contents included
    tc::fence_before_sync();
    named_sync(1, C::kSoft);
    tc::fence_after_sync();
  };
  const float cap2 = a.mod.softcap * kChunkLog2e, icap = a.mod.softcap > 0.0f ? 2.0f / a.mod.softcap : 0.0f;
  ChunkWalk walk;
  walk.begin(a, h, blockIdx.x);
  ChunkItem it;
  int kvh, j0, j1, ct = 0;
  while (walk.next(a, h, it, kvh, j0, j1)) {
    const int row0 = a.row_start[it.b], m = a.row_start[it.b + 1] - row0, n = min(max(a.c.seq_len[it.b], 0), a.c.max_ctx);
    const int nk = it.n_body + it.n_tail, nt = j1 - j0;
    const bool whole = nt == nk, have = row < it.rows, busy = (warp & 3) * 32 < it.rows;  // busy: the warp has rows
    const int w = have ? it.r0 + row : it.r0, tok = int(div_u32(uint32_t(w), a.by_group)), hh = w - tok * a.group;
    const size_t base = ((size_t)(row0 + tok) * a.n_q_heads + kvh * a.group + hh) * D;
    ChunkSpan span{0, 0, 0};
    float slope2 = 0.0f;
    int qs = 0;
    if (nt > 0) {
      if (have) span = chunk_span(a, it.b, n, row0, m, tok);
      if (a.mod.slopes && have) slope2 = a.mod.slopes[kvh * a.group + hh] * kChunkLog2e;
      // ---- queries: 32 channels at a time to TMEM (where O will be), rotated there, scaled, to their operand's place
      const uint32_t tmp = lanes + C::ocol;
      float top = 0.0f;
      if (busy) {
#pragma unroll 1
        for (int c = grp; c < C::NB; c += NG) {
          float v[32];
          if (a.q_dtype == KVQ_F32) {
            const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(a.q) + base + c * 32);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 x = src[i];
              v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = x.z; v[4 * i + 3] = x.w;
            }
          } else {
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) + base + c * 32);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint4 x = src[i];
              const uint32_t ww[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint32_t b16 = (ww[e / 2] >> (16 * (e & 1))) & 0xFFFFu;
                v[8 * i + e] = a.q_dtype == KVQ_BF16 ? bf16_bits_to_f32(b16) : __half2float(__ushort_as_half(uint16_t(b16)));
              }
            }
          }
          if (!have) {
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = 0.0f;
          }
          if (a.rot_k) tc_fwht32(v);
          else {
#pragma unroll
            for (int e = 0; e < 32; ++e) top = fmaxf(top, fabsf(v[e]));
          }
          tc::st_x16(tmp + c * 32, *reinterpret_cast<float(*)[16]>(&v[0]));
          tc::st_x16(tmp + c * 32 + 16, *reinterpret_cast<float(*)[16]>(&v[16]));
        }
        tc::wait_st();
      }
      if (a.rot_k) {
        all();
        if (busy) {
#pragma unroll 1
          for (int s = grp; s < 4 * (D / C::G); s += NG) {  // 8 of the 32 channels, of all chunks of a rotation group
            const uint32_t at = tmp + (s / 4) * C::G + (s % 4) * 8;
            float v[C::GC][8];
#pragma unroll
            for (int k = 0; k < C::GC; ++k) tc::ld_x8(at + k * 32, v[k]);
            tc::wait_ld();
            tc_fwht_chunks<C::GC>(v);
#pragma unroll
            for (int k = 0; k < C::GC; ++k) {
#pragma unroll
              for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(v[k][e]));
              tc::st_x8(at + k * 32, v[k]);
            }
          }
          tc::wait_st();
        }
      }
      if constexpr (NG == 2) sy->rowmax[grp][row] = top;
      all();
      if constexpr (NG == 2) top = fmaxf(top, sy->rowmax[1 - grp][row]);
      const float sc = a.scale * kChunkLog2e * (a.rot_k ? inv_sqrt_group<C::G>() : 1.0f);
      qs = min(11 - tc_exp(top * sc), 126);  // the largest below 2^11
      const float qf = tc_pow2(qs);
      if (busy) {
#pragma unroll 1
        for (int c = grp; c < C::NB; c += NG) {
          float v[32];
          tc::ld_x16(tmp + c * 32, *reinterpret_cast<float(*)[16]>(&v[0]));
          tc::ld_x16(tmp + c * 32 + 16, *reinterpret_cast<float(*)[16]>(&v[16]));
          tc::wait_ld();
          uint32_t hi[16], lo[16];
#pragma unroll
          for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // channels 0 2, 1 3 of each four
              const float x = v[4 * i + e] * sc * qf, y = v[4 * i + e + 2] * sc * qf;
              if constexpr (PARTS == 2) split_h2(x, y, hi[2 * i + e], lo[2 * i + e]);
              else hi[2 * i + e] = pack_h2(x, y);
            }
          if constexpr (C::QSMEM) {
            const uint32_t at = smem_u32(sm) + C::off_q + (c / 2) * (128 * 128);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              tc_sts128(at + tc::sw128_chunk(row, (c & 1) * 4 + i), *reinterpret_cast<uint32_t(*)[4]>(&hi[4 * i]));
          } else {
            tc::st_x16(lanes + C::qcol + c * 16, *reinterpret_cast<float(*)[16]>(&hi[0]));
            if constexpr (PARTS == 2) tc::st_x16(lanes + C::qcol + D / 2 + c * 16, *reinterpret_cast<float(*)[16]>(&lo[0]));
          }
        }
        tc::wait_st();
      }
      if constexpr (C::QSMEM) fence_proxy_async_smem();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sy->qready);
    }

    // ---- tiles
    float m_used = -INFINITY, l = 0.0f;
    int vs = 0, mine = 0, last = -1;  // the group's tiles so far, the last one's number
    bool nan = false;
    for (int k = 0; k < nt; ++k, ++ct) {
      const int b = ct & 1;
      const uint32_t u = uint32_t(ct) >> 1;
      if (NG == 2 && b != grp) continue;
      bool ok = tc_wait(&sy->sfull[b], u & 1, sy, status);
      ok = __all_sync(0xffffffffu, ok);
      if (ok && busy) {
        tc::fence_after_sync();
        float sv[TK];
#pragma unroll
        for (int c = 0; c < TK; c += 16) tc::ld_x16(lanes + C::scol + b * TK + c, *reinterpret_cast<float(*)[16]>(&sv[c]));
        const volatile TcMeta* mt = &sy->meta[ct % kTcMeta];
        const int t0 = mt->t0, cnt = mt->cnt, nvs = mt->vs;
        float f = tc_pow2(-mt->ks - qs);
        const uint32_t bad0 = mt->bad[0], bad1 = mt->bad[1];
        tc::wait_ld();
        if (!C::OVER) {
          tc::fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sy->sfree[b]);
        }
        if (a.mod.softcap > 0.0f) {
#pragma unroll
          for (int c = 0; c < TK; ++c) {
            float r;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + ex2_approx(sv[c] * (f * icap))));
            sv[c] = fmaf(-2.0f * cap2, r, cap2);
          }
          f = 1.0f;
        }
        if (a.mod.slopes) {
          const float d0 = float(t0 - span.pos);
#pragma unroll
          for (int c = 0; c < TK; ++c) sv[c] = fmaf(sv[c], f, -slope2 * fabsf(d0 + float(c)));
          f = 1.0f;
        }
        const int lo = span.lo - t0, hi = min(span.hi - t0, cnt);
        if (__any_sync(0xffffffffu, lo > 0 || hi < TK)) {
#pragma unroll
          for (int c = 0; c < TK; ++c)
            if (c < lo || c >= hi) sv[c] = -INFINITY;
        }
        if (bad0 | bad1) {
          const uint32_t ml = hi <= 0 ? 0u : hi >= 32 ? 0xFFFFFFFFu : (1u << hi) - 1u;
          const uint32_t mh = hi <= 32 ? 0u : hi >= 64 ? 0xFFFFFFFFu : (1u << (hi - 32)) - 1u;
          const uint32_t kl = lo <= 0 ? 0xFFFFFFFFu : lo >= 32 ? 0u : ~((1u << lo) - 1u);
          const uint32_t kh = lo <= 32 ? 0xFFFFFFFFu : lo >= 64 ? 0u : ~((1u << (lo - 32)) - 1u);
          nan |= ((bad0 & ml & kl) | (bad1 & mh & kh)) != 0;
        }
        float mx[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
        for (int c = 4; c < TK; ++c) mx[c & 3] = fmaxf(mx[c & 3], sv[c]);
        const float mt2 = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * f;
        float alpha = 1.0f;
        bool move = mt2 > m_used + kTcLazy || (m_used == -INFINITY && mt2 > -INFINITY);
        if (move) {
          alpha = m_used == -INFINITY ? 0.0f : ex2_approx(m_used - mt2);
          l *= alpha;
          m_used = mt2;
        }
        if (mine > 0 && nvs != vs) {
          alpha *= tc_pow2(nvs - vs);
          move = true;
        }
        vs = nvs;
        const float mb = m_used == -INFINITY ? 0.0f : m_used - 8.0f;
        float ls[2] = {0.0f, 0.0f};
        uint32_t ph[TK / 2], pl[PARTS == 2 ? TK / 2 : 1];
#pragma unroll
        for (int c = 0; c < TK; c += 2) {
          const float e0 = ex2_approx(fmaf(sv[c], f, -mb)), e1 = ex2_approx(fmaf(sv[c + 1], f, -mb));
          ls[0] += e0;
          ls[1] += e1;
          if constexpr (PARTS == 2) split_h2(e0, e1, ph[c / 2], pl[c / 2]);
          else ph[c / 2] = pack_h2(e0, e1);
        }
        l += ls[0] + ls[1];
        // the weights' place is free once the product that read it is done; to rescale O, the group's last product has to be
        if (u > 0) ok = tc_wait(&sy->odone[b], (u - 1) & 1, sy, status);
        const bool resc = mine > 0 && __any_sync(0xffffffffu, move);
        if (NG == 1 && resc) ok = tc_wait(&sy->odone[b ^ 1], ((uint32_t(ct) - 1) >> 1) & 1, sy, status) && ok;
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
          tc::fence_after_sync();
          if (resc) {
            const uint32_t o = lanes + C::ocol + grp * D;
#pragma unroll 2
            for (int c = 0; c < D; c += 16) {
              float t[16];
              tc::ld_x16(o + c, t);
              tc::wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) t[e] *= alpha;
              tc::st_x16(o + c, t);
            }
          }
          const uint32_t p = lanes + C::pcol + b * C::pstep;
#pragma unroll
          for (int c = 0; c < TK / 2; c += 16) {
            tc::st_x16(p + c, *reinterpret_cast<float(*)[16]>(&ph[c]));
            if constexpr (PARTS == 2) tc::st_x16(p + TK / 2 + c, *reinterpret_cast<float(*)[16]>(&pl[c]));
          }
          tc::wait_st();
          tc::fence_before_sync();
        }
      } else {  // no rows: in step with the others all the same, or its arrivals would count for their next tile
        __syncwarp();
        if (!C::OVER && lane == 0) mbar_arrive(&sy->sfree[b]);
        if (u > 0) tc_wait(&sy->odone[b], (u - 1) & 1, sy, status);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sy->pfull[b]);
      ++mine;
      last = ct;
    }

    // ---- the rows' results
    bool ok = true;
    if (last >= 0) ok = tc_wait(&sy->odone[last & 1], (uint32_t(last) >> 1) & 1, sy, status);
    float M = m_used, f[2] = {1.0f, 0.0f};
    bool read[2] = {mine > 0, false};
    if constexpr (NG == 2) {
      sy->join[grp][row] = make_float4(mine > 0 ? m_used : -INFINITY, l, tc_pow2(-vs), nan || mine == 0 ? (nan ? 1.0f : 2.0f) : 0.0f);
      all();
      const float4 x0 = sy->join[0][row], x1 = sy->join[1][row];
      M = fmaxf(x0.x, x1.x);
      f[0] = x0.x == -INFINITY ? 0.0f : ex2_approx(x0.x - M);
      f[1] = x1.x == -INFINITY ? 0.0f : ex2_approx(x1.x - M);
      l = x0.y * f[0] + x1.y * f[1];
      f[0] *= x0.z;
      f[1] *= x1.z;
      nan = x0.w == 1.0f || x1.w == 1.0f;
      read[0] = x0.w != 2.0f;
      read[1] = x1.w != 2.0f;
    } else {
      tc::fence_after_sync();
      f[0] = tc_pow2(-vs);
    }
    if (nan) l = NAN;
    ok = __all_sync(0xffffffffu, ok);
    const size_t slot = (size_t)(2 * blockIdx.x + (j0 == 0 ? 1 : 0)) * 128 + row;
    if (whole) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      f[0] *= inv;
      f[1] *= inv;
    } else if (have && grp == 0) {
      a.part_ml[slot] = make_float2(M == -INFINITY && nan ? 0.0f : M, l);
    }
    const bool any0 = __any_sync(0xffffffffu, read[0]) && ok, any1 = NG == 2 && __any_sync(0xffffffffu, read[1]) && ok;
    // 32 channels of O, joined, in natural order
    auto chunk = [&](int c, float (&v)[32]) {
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = 0.0f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (!(g ? any1 : any0)) continue;
        float t[32];
        tc::ld_x16(lanes + C::ocol + g * D + c * 32, *reinterpret_cast<float(*)[16]>(&t[0]));
        tc::ld_x16(lanes + C::ocol + g * D + c * 32 + 16, *reinterpret_cast<float(*)[16]>(&t[16]));
        tc::wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[4 * i] = fmaf(t[4 * i], f[g], v[4 * i]);
          v[4 * i + 2] = fmaf(t[4 * i + 1], f[g], v[4 * i + 2]);
          v[4 * i + 1] = fmaf(t[4 * i + 2], f[g], v[4 * i + 1]);
          v[4 * i + 3] = fmaf(t[4 * i + 3], f[g], v[4 * i + 3]);
        }
      }
    };
    auto store8 = [&](int ch, const float* v) {  // channels ch .. ch + 7
      if (a.out_dtype == KVQ_F32) {
        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out) + base + ch);
        dst[0] = make_float4(v[0], v[1], v[2], v[3]);
        dst[1] = make_float4(v[4], v[5], v[6], v[7]);
      } else {
        uint32_t x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = a.out_dtype == KVQ_BF16 ? tc_pack_bf2(v[2 * e], v[2 * e + 1]) : pack_h2(v[2 * e], v[2 * e + 1]);
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + base + ch) = make_uint4(x[0], x[1], x[2], x[3]);
      }
    };
    const bool turn = whole && a.rot_v;
    if (busy) {
#pragma unroll 1
      for (int c = grp; c < C::NB; c += NG) {
        float v[32];
        chunk(c, v);
        if (turn) {
          tc_fwht32(v);
          tc::st_x16(lanes + C::ocol + c * 32, *reinterpret_cast<float(*)[16]>(&v[0]));
          tc::st_x16(lanes + C::ocol + c * 32 + 16, *reinterpret_cast<float(*)[16]>(&v[16]));
        } else if (have && whole) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) store8(c * 32 + e, v + e);
        } else if (have) {
          float4* dst = reinterpret_cast<float4*>(a.part + slot * D + c * 32);
#pragma unroll
          for (int e = 0; e < 8; ++e) dst[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        }
      }
      if (turn) tc::wait_st();
    }
    if (turn) {
      all();
      if (busy) {
#pragma unroll 1
        for (int s = grp; s < 4 * (D / C::G); s += NG) {
          const int at = (s / 4) * C::G + (s % 4) * 8;
          float v[C::GC][8];
#pragma unroll
          for (int k = 0; k < C::GC; ++k) tc::ld_x8(lanes + C::ocol + at + k * 32, v[k]);
          tc::wait_ld();
          tc_fwht_chunks<C::GC>(v);
#pragma unroll
          for (int k = 0; k < C::GC; ++k) {
#pragma unroll
            for (int e = 0; e < 8; ++e) v[k][e] *= inv_sqrt_group<C::G>();
            if (have) store8(at + k * 32, v[k]);
          }
        }
      }
    }
    all();  // O, the queries' place and the exchanged words are free
  }
}

template <int D, int PARTS>
__global__ void __launch_bounds__(TC<D, PARTS>::kThreads, 1)
chunk_tc_kernel(ChunkArgs a, TcStage L, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                const __grid_constant__ CUtensorMap tmKt, const __grid_constant__ CUtensorMap tmVt) {
  using C = TC<D, PARTS>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  pdl_begin();
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TcSync* sy = reinterpret_cast<TcSync*>(sm + C::off_ring + L.stages * L.bytes);
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const ChunkHeader h = *a.head;
  if (!h.ok || int(blockIdx.x) >= h.pieces) return;  // (the whole CTA)
  if (warp == 0) {
    tc::tmem_alloc(&sy->tmem, 512);
    tc::tmem_relinquish();
  }
  if (tid == 32) {
    for (int i = 0; i < L.stages; ++i) {
      mbar_init(&sy->rfull[i], 1);
      mbar_init(&sy->rempty[i], kTcConv);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sy->kfull[i], kTcConv); mbar_init(&sy->kempty[i], 1);
      mbar_init(&sy->vfull[i], kTcConv); mbar_init(&sy->vempty[i], 1);
      mbar_init(&sy->sfull[i], 1); mbar_init(&sy->sfree[i], 4);
      mbar_init(&sy->pfull[i], 4); mbar_init(&sy->odone[i], 1);
      mbar_init(&sy->fin[i], 1);
    }
    mbar_init(&sy->qready, C::kSoft / 32);
    mbar_init(&sy->tmax, kTcConv);
    sy->abort = 0;
    fence_barrier_init();
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = sy->tmem;
  constexpr int W0 = C::kSoft / 32;
  if (warp < W0) {
    tc_softmax<D, PARTS>(a, h, sm, tmem, sy, warp, lane);
  } else if (warp < W0 + kTcConv) {
    tc_convert<D, PARTS>(a, L, sm, sy, warp - W0, lane);
  } else if (warp == W0 + kTcConv) {
    tc_produce<D, PARTS>(a, L, h, sm, sy, lane, &tmK, &tmV, &tmKt, &tmVt);
  } else if (lane == 0) {
    if (warp == W0 + kTcConv + 1) tc_issue_s<D, PARTS>(a, h, smem_u32(sm), tmem, sy);
    else tc_issue_pv<D, PARTS>(a, h, smem_u32(sm), tmem, sy);
  }
  __syncwarp();
  tc::fence_before_sync();
  __syncthreads();
  if (warp == 0) {
    // every product has ended (after a wait that gave up as well)
    mbar_wait_bounded(&sy->fin[0], 0, kTcWait);
    mbar_wait_bounded(&sy->fin[1], 0, kTcWait);
    __syncwarp();
    tc::fence_after_sync();
    tc::tmem_dealloc(tmem, 512);
  }
}

template <int D, int PARTS>
cudaError_t run_chunk_tc(ChunkArgs& a, cudaStream_t st) {
  using C = TC<D, PARTS>;
  constexpr int NB = C::NB;
  const kvq_cache& c = a.c;
  const int rowK = int(qs_row_bytes_host(c.k_type, D)), rowV = int(qs_row_bytes_host(c.v_type, D));
  TcStage s{};
  s.kh = NB * (type_has_min(c.k_type) ? 4 : 2);
  s.vh = NB * (type_has_min(c.v_type) ? 4 : 2);
  const int kq = type_has_qh(c.k_type) ? C::TK * NB * 4 : 0, vq = type_has_qh(c.v_type) ? C::TK * NB * 4 : 0;
  s.v = align_up(C::TK * rowK, 1024);
  s.kd = s.v + C::TK * rowV;
  s.vd = s.kd + C::TK * s.kh;
  s.kqh = s.vd + C::TK * s.vh;
  s.vqh = s.kqh + kq;
  s.tx = uint32_t(C::TK * (rowK + rowV + s.kh + s.vh) + kq + vq);
  s.vt = align_up(C::TT * 2 * D, 1024);
  s.bytes = align_up(std::max(s.vqh + vq, c.tail_len > 0 ? s.vt + C::TT * 2 * D : 0), 1024);
  const int room = 232448 - 1024 - C::off_ring - int(sizeof(TcSync));
  s.stages = std::min(kTcMaxStages, room / s.bytes);
  if (s.stages < 1) return cudaErrorInvalidValue;
  // (more than half of an SM's, so that no two CTAs of one SM ask for all of TMEM)
  const int bytes = std::max(120 * 1024, C::off_ring + s.stages * s.bytes + int(sizeof(TcSync)) + 1024);

  alignas(64) CUtensorMap mk, mv, mkt, mvt;
  memset(&mkt, 0, sizeof(mkt));
  memset(&mvt, 0, sizeof(mvt));
  if (!make_map(&mk, c.k_qs, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, body_rows(c), rowK, box_w(rowK), C::TK) ||
      !make_map(&mv, c.v_qs, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, body_rows(c), rowV, box_w(rowV), C::TK))
    return cudaErrorInvalidValue;
  if (c.tail_len > 0) {
    const long long trows = (long long)c.batch * c.n_kv_heads * c.tail_len;
    if (!make_map(&mkt, c.k_tail, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, trows, 2 * D, 128, C::TT) ||
        !make_map(&mvt, c.v_tail, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, trows, 2 * D, 128, C::TT))
      return cudaErrorInvalidValue;
  }
  auto kern = chunk_tc_kernel<D, PARTS>;
  const cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), bytes);
  if (e != cudaSuccess) return e;
  return launch_dependent(kern, unsigned(a.ctas), C::kThreads, bytes, st, 1, a, s, mk, mv, mkt, mvt);
}

constexpr int tc_max_parts(int d) { return d <= 128 ? 2 : 1; }  // (two parts of wider operands do not fit)
template <int D>
ChunkTiles tc_tiles(int parts) {
  return parts <= tc_max_parts(D) ? ChunkTiles{128, TC<D, 1>::TK, TC<D, 1>::TT} : ChunkTiles{0, 0, 0};
}
template <int D>
cudaError_t launch_tc(ChunkArgs& a, int parts, cudaStream_t st) {
  if constexpr (tc_max_parts(D) == 2)
    if (parts == 2) return run_chunk_tc<D, 2>(a, st);
  return parts == 1 ? run_chunk_tc<D, 1>(a, st) : cudaErrorInvalidValue;
}

}  // namespace
}  // namespace kvq
