// Attention of packed rows of new tokens on tcgen05 (kvq_chunk_attention), included by one translation unit per head_dim.
//
// A CTA walks its piece of the plan's stream (kvq_chunk.cuh).  128 rows are the lanes of TMEM.  Roles:
//   producer      a warp: tiles of packed codes, headers and high bits (or bf16 tail rows) by TMA into a ring
//   scout         a warp: a landed tile's scales, and its keys that are not finite
//   converters    eight warps: a tile to fp16 operands, keys and values in the same layout (rows of 64 channels, 128-byte
//                 swizzle), which is K-major for Q K^T and, read along N, V for P V: nothing is transposed
//   S issuer      a warp: S = Q K^T, Q in TMEM (shared memory at head_dim 320)
//   P V issuer    a warp: O += P V, P in TMEM
//   softmax       one or two groups of four warps, a row per thread.  Two groups (small heads) each have a running maximum, sum
//                 and accumulator of their own: two chains of score -> weight -> product in flight, without a word between
//                 them.  Of an item of more than 128 rows they take 128 each, so that a tile is converted once for both; of
//                 a smaller one every other tile, and are joined at the item's end.
//
// PARTS 1 (bf16 outputs): queries, keys, values and weights rounded once to fp16, 2^-11 of themselves, an eighth of the output's
// step; PARTS 2 (fp16 and fp32): two fp16 parts each and three products, 22 bits.  Sums and softmax statistics are fp32.
// fp16's range: a row's queries, a tile's keys and a tile's values are scaled by powers of two taken from their largest (a
// quantized tile's from its headers), so that no more than 2^-12 of the largest of its block of 32 is lost of any number.  Where a
// tile's tokens differ too much in size for that, it is converted from fp32 over the format's whole range, and 2^-34 of the
// tile's largest is.  Values keep the scale of the tile before where it serves; O is brought along where it changes.
// Weights are times 2^8.
//
// Channels lie in the order 0 2 1 3 within each four, as the codes' conversion leaves them, in Q, K and V alike; the
// epilogue reads O in that order.  A key with a header or tail value that is not finite is zeroed and noted, and the rows
// that see it are NaN at the end: 0 * NaN in the products would reach rows that do not.
//
// Measured (GB300, us): 2 x 4096 rows, 32/8 heads of 128, half of each prompt a prefix: 513, 670 TFLOP/s (35% of what a large bf16
// product reaches); 512 rows over 65,536 tokens, 24/4 heads of 256, with a bias: 1005, 817 TFLOP/s (42%); 32 sequences of up to
// 8k tokens, one token each, 32/8 heads of 128, capped: 266, 0.96 TB/s.  No pipe is near its limit (prompts: tensor 30%, special
// functions 15%, issue slots 53%): the roles wait for one another, a tile's chain of load, conversion, score, weight and product
// being 1.4 to 2 us, and for instructions (a warp per issue).  With few rows 4 of 128 lanes have use of it.
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
constexpr int kTcSyncBytes = 7168;           // of TcSync, in front of everything else in shared memory
constexpr int kTcMaxSlots = 4;
constexpr int kTcMeta = 16;                  // (a tile's is read before the ring has come round and two more tiles are done)
constexpr int kTcRise = 60;                  // see the scout
constexpr int kTcConv = 8;                   // converter warps, the first half for keys, the others for values

template <int D, int PARTS>
struct TC {
  static constexpr int NG = D <= 64 * (3 - PARTS) ? 2 : 1;     // groups of softmax warps, each with an O of its own
  // keys of a tile, and tail rows of one (as many as shared memory has room for)
  static constexpr int TK = PARTS == 1 ? (D == 320 ? 32 : 64) : D <= 128 ? 64 : D <= 256 ? 32 : 16;
  static constexpr int TT = PARTS == 1 ? (D == 64 ? 64 : D <= 256 ? 32 : 16) : D == 64 ? 64 : D <= 192 ? 32 : D == 256 ? 16 : 8;
  static_assert(TT <= TK, "");
  static constexpr int SB = NG == 2 && PARTS == 2 ? 1 : 2;     // score buffers of a group: with two, S of the next tile is ready
  static constexpr bool QSMEM = D == 320 || (D == 128 && PARTS == 1) || (D == 256 && PARTS == 2);  // (TMEM has no room for the queries)
  static constexpr bool OVER = PARTS == 1 && (D == 256 || NG == 2);  // P over S (TMEM again)
  static constexpr int KH = (TK + 31) / 32;                    // keys of a converting lane
  static constexpr int M = NG * 128;                           // rows of an item
  static constexpr int G = (D & (D - 1)) == 0 ? D : 64, GC = G / 32, NB = D / 32;
  static constexpr int kSoft = NG * 128, kThreads = kSoft + (kTcConv + 4) * 32;
  // TMEM columns
  static constexpr int qw = QSMEM ? 0 : PARTS * D / 2, ocol = NG * qw, scol = ocol + NG * D;  // (queries from column 0 on)
  static constexpr int pw = PARTS * TK / 2, pcol = OVER ? scol : scol + NG * SB * TK, pstep = OVER ? TK : pw;
  static_assert(pcol + NG * SB * pstep <= 512, "TMEM columns");
  static_assert(!OVER || PARTS == 1, "a second part of P would lie over scores not read yet");
  // shared memory
  static constexpr int part = D * TK * 2, slot = PARTS * part;  // a tile's operand
  // slots of each side: conversion may run that far ahead of the products (as many as leave room for a ring of three stages)
  static constexpr int NS = slot <= 8192 ? 4 : D == 192 ? 3 : PARTS == 2 && D >= 256 ? 1 : 2;
  static constexpr int off_q = kTcSyncBytes, off_k = off_q + (QSMEM ? NG * PARTS * D * 256 : 0), off_v = off_k + NS * slot, off_ring = off_v + NS * slot;
  static constexpr int N1 = D > 256 ? 192 : D, N2 = D - N1;     // P V as one or two instructions
};

struct TcStage {  // offsets in a stage of the ring: K codes, V codes (1024-aligned), headers, high bits; or K and V tail rows
  int v, kd, vd, kqh, vqh, vt, bytes, stages;
  int kh, vh;     // header bytes of a row
  uint32_t tx;
};

struct __align__(16) TcMeta {
  uint4 a;  // position of column 0, its keys, the powers of two that keys and values were multiplied by
  uint4 b;  // keys that are not finite (two words); sides (1 keys, 2 values) that the quick conversion is not for, 4: a tail tile
};

struct TcSync {
  uint64_t rfull[kTcMaxStages], mfull[kTcMaxStages], rempty[kTcMaxStages];
  uint64_t kfull[kTcMaxSlots], kempty[kTcMaxSlots], vfull[kTcMaxSlots], vempty[kTcMaxSlots], sfull[4], sfree[4], pfull[4], odone[4], qready, fin[2];
  int4 job[kTcMaxStages];  // first position, keys (-1: the end), tail slot or -1, first tile of a segment
  TcMeta meta[kTcMeta];
  float rowmax[2][128];
  float4 join[2][128];     // a group's (reference, sum, value scale, NaN) of each row
  uint32_t* status;
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(TcSync) <= kTcSyncBytes && kTcSyncBytes % 1024 == 0, "shared memory");

// Where TcSync lies: the first 1024-byte boundary of the dynamic shared memory.
__device__ __forceinline__ TcSync* tc_sync() {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  return reinterpret_cast<TcSync*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
}

// Bounded wait; false once any wait of the CTA has given up.  (Code that seldom runs is kept out of line throughout: the loops of all
// roles together are more than an SM's instruction cache holds, and 86 requests a tile go to the cache behind it in the prompt
// case.  Taking out of the loops what does not belong there made that case 1.07 ms from 1.71.)
__device__ __forceinline__ bool tc_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;  // (without a time hint: one of 20 us made 366 us for 32 rows of one token 411, 942 us for prompts 971)
  asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __noinline__ bool tc_wait_long(uint32_t bar, uint32_t parity) {
  TcSync* sy = tc_sync();
  const long long t0 = clock64();
#pragma unroll 1
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)  // (an attempt returns after some hundred cycles)
      if (tc_try(bar, parity)) return true;
    if (*reinterpret_cast<volatile int*>(&sy->abort)) return false;
    if (clock64() - t0 > kTcWait) {
      *reinterpret_cast<volatile int*>(&sy->abort) = 1;
      atomicOr(sy->status, KVQ_DEV_ERR_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ bool tc_wait(uint64_t* bar, uint32_t parity) {
  const uint32_t at = smem_u32(bar);
  return tc_try(at, parity) || tc_wait_long(at, parity);
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
__device__ __forceinline__ uint2 tc_lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
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

// What a unit of conversion (a tile's keys of one block of 32 channels) is told: shared addresses of a side's codes,
// headers and high bits (or tail rows), where the operand goes, and the power of two that it is taken times.
struct TcSide {
  uint32_t codes, hdr, qh, dst;
  int type, scale;
  bool is_k;
};

// One fp16 part.  Codes enter as fp16 subnormals, code * 2^-24, a mask or byte permute away from what is stored, and one
// fused operation gives code * d + m: exact before its one rounding, with d * 2^24 and the minimum (or -offset * d) exact.
// That takes d below 2^-8, and not so small that fp16's smallest step counts; the scout sees to both (tc_below_normal).  A lane
// has the keys lane and lane + 32: two chains of loads, conversions and stores at once.  (Centred codes times d have fp16's whole
// range for one operation a pair more, and with them 32 sequences of one token took 277 us for 255, 2 x 4096 prompt rows 533 for 488.)
template <int D, bool Q8, bool HIGH>
__device__ __forceinline__ void tc_unit1(const TcSide& u, int lane, int blk, const uint32_t (&d)[TC<D, 1>::KH],
                                         const uint32_t (&m)[TC<D, 1>::KH]) {
  using C = TC<D, 1>;
  constexpr int TK = C::TK, NB = C::NB, KH = C::KH, ROW = Q8 ? D : D / 2, W = box_w(ROW);
  // (the swizzle looks at key bits 0-2 alone: the same for both keys)
  const uint32_t row = u.dst + (blk / 2) * (TK * 128) + lane * 128 + (((blk & 1) * 64) ^ ((lane & 4) << 4));
  const uint32_t x3 = (lane & 3) << 4;  // (the block's four 16-byte pieces lie in one half of the row)
  if constexpr (Q8) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 v[KH];
#pragma unroll
      for (int k = 0; k < KH; ++k) v[k] = tc_lds128(u.codes + swz_off<W>(lane, 32 * blk + 16 * h, TK) + k * 32 * W);
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int k = 0; k < KH; ++k) {
          const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
          uint32_t o[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)  // bytes 0 2, 1 3 of two words
            o[i] = hfma2_bits(__byte_perm(w[2 * c + i / 2], 0u, i & 1 ? 0x4341 : 0x4240), d[k], m[k]);
          tc_sts128(row + k * 4096 + (((2 * h + c) << 4) ^ x3), o);
        }
    }
  } else {
    uint4 v[KH];
#pragma unroll
    for (int k = 0; k < KH; ++k) v[k] = tc_lds128(u.codes + swz_off<W>(lane, 16 * blk, TK) + k * 32 * W);
    // the high bits of pair e of word i of chunk c, 16 apart, at bit 4 (c / 2) + i * hstep + e of hw[c & 1] less 4
    uint32_t hw[KH][2];
    int hstep = 0;
    if constexpr (HIGH) {
      hstep = u.is_k ? 2 : 8;
#pragma unroll
      for (int k = 0; k < KH; ++k) {
        const int key = lane + 32 * k;
        if (u.is_k) {
          const uint32_t x = tc_lds32(u.qh + (key * NB + blk) * 4);
          hw[k][0] = __funnelshift_l(x, x, 4);      // bit b at b + 4
          hw[k][1] = __funnelshift_r(x, x, 4);      // bit b + 8 at b + 4
        } else {
#pragma unroll
          for (int p = 0; p < 2; ++p) {
            const uint32_t x = tc_lds16(u.qh + ((((key >> 1) * NB + blk) * 2 + p) * 2 + (key & 1)) * 2);
            const uint32_t y = x | x << 14;          // bits b and b + 2 of the part 16 apart
            hw[k][p] = __funnelshift_l(y, y, 4);
          }
        }
      }
    }
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int k = 0; k < KH; ++k) {
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            uint32_t t = (w[2 * (c & 1) + i] >> (4 * (c >> 1) + 8 * e)) & 0x000F000Fu;
            if constexpr (HIGH) {
              const int sh = 4 * (c >> 1) + e + (i ? hstep : 0);
              t |= __funnelshift_r(hw[k][c & 1], hw[k][c & 1], sh) & 0x00100010u;
            }
            o[2 * i + e] = hfma2_bits(t, d[k], m[k]);
          }
        tc_sts128(row + k * 4096 + ((c << 4) ^ x3), o);
      }
  }
}

// Two fp16 parts: centred codes, exact; code * d rounded, and what that left, exact too where d is a normal number (the scout
// sees to it); with a minimum both from the sum in fp32.
template <int D, bool Q8, bool HIGH>
__device__ __forceinline__ void tc_unit2(const TcSide& u, int key, int blk, uint32_t d, uint32_t m, uint32_t off, bool min) {
  using C = TC<D, 2>;
  constexpr int TK = C::TK, NB = C::NB, ROW = Q8 ? D : D / 2, W = box_w(ROW);
  const uint32_t row = u.dst + (blk / 2) * (TK * 128) + key * 128;
  uint32_t hw[2] = {0u, 0u};
  int hstep = 0;
  if constexpr (HIGH) {
    if (u.is_k) {
      const uint32_t x = tc_lds32(u.qh + (key * NB + blk) * 4);
      hw[0] = __funnelshift_l(x, x, 4);
      hw[1] = __funnelshift_r(x, x, 4);
      hstep = 2;
    } else {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const uint32_t x = tc_lds16(u.qh + ((((key >> 1) * NB + blk) * 2 + p) * 2 + (key & 1)) * 2);
        const uint32_t y = x | x << 14;
        hw[p] = __funnelshift_l(y, y, 4);
      }
      hstep = 8;
    }
  }
  uint32_t w[Q8 ? 8 : 4];
#pragma unroll
  for (int h = 0; h < (Q8 ? 2 : 1); ++h) {
    const uint4 v = tc_lds128(u.codes + swz_off<W>(key, Q8 ? 32 * blk + 16 * h : 16 * blk, TK));
    w[4 * h] = v.x; w[4 * h + 1] = v.y; w[4 * h + 2] = v.z; w[4 * h + 3] = v.w;
  }
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t code;
        if constexpr (Q8) {
          code = e ? i8_pair<1, 3>(w[(2 * c + i) % (Q8 ? 8 : 4)]) : i8_pair<0, 2>(w[(2 * c + i) % (Q8 ? 8 : 4)]);
        } else {
          uint32_t t = (w[2 * (c & 1) + i] >> (4 * (c >> 1) + 8 * e)) & 0x000F000Fu;
          if constexpr (HIGH) t |= __funnelshift_r(hw[c & 1], hw[c & 1], 4 * (c >> 1) + e + (i ? hstep : 0)) & 0x00100010u;
          code = hsub2_bits(t | 0x64006400u, off);
        }
        uint32_t &h = hi[2 * i + e], &l = lo[2 * i + e];
        if (!min) {
          h = hmul2_bits(code, d);
          asm("{\n\t.reg .b32 nh;\n\tneg.f16x2 nh, %3;\n\tfma.rn.f16x2 %0, %1, %2, nh;\n\t}" : "=r"(l) : "r"(code), "r"(d), "r"(h));
        } else {
          const float2 cf = __half22float2(u32_as_h2(code)), x = __half22float2(u32_as_h2(d)), y = __half22float2(u32_as_h2(m));
          split_h2(fmaf(cf.x, x.x, y.x), fmaf(cf.y, x.y, y.y), h, l);
        }
      }
    const uint32_t at = row + ((((blk & 1) * 4 + c) ^ (key & 7)) << 4);
    tc_sts128(at, hi);
    tc_sts128(at + C::part, lo);
  }
}

// A key's block of any format from its sum in fp32: the whole range of headers, for tiles that mix far-off ones (a token a
// thousand times as large as the others).  Rounded like the rest, once or in two parts.
template <int D, int PARTS>
__device__ __noinline__ void tc_wide_unit(uint32_t codes, uint32_t hdr, uint32_t qh, uint32_t dst, int type, int scale, bool is_k, int key,
                                          int blk, bool ok) {
  using C = TC<D, PARTS>;
  constexpr int TK = C::TK, NB = C::NB;
  const bool q8 = type == KVQ_TYPE_Q8_0;
  const int off = q8 ? 128 : type_code_offset(type);
  float fd, fm = 0.0f;
  if (type_has_min(type)) {
    const float2 f = __half22float2(u32_as_h2(tc_lds32(hdr + (key * NB + blk) * 4)));
    fd = f.x;
    fm = f.y;
  } else {
    fd = __half2float(__ushort_as_half(uint16_t(tc_lds16(hdr + (key * NB + blk) * 2))));
  }
  if (!ok || !(fabsf(fd) <= 65504.0f) || !(fabsf(fm) <= 65504.0f)) fd = fm = 0.0f;  // past the end, or noted as not finite
  const float sc = tc_pow2(scale);
  fd *= sc;
  fm *= sc;
  const uint32_t row = dst + (blk / 2) * (TK * 128) + key * 128;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t high = 0u;  // bits of pair e of word i at 2 i + e, 16 apart
    if (type_has_qh(type)) {
      if (is_k) {
        const uint32_t x = tc_lds32(qh + (key * NB + blk) * 4);
        const int at = 8 * (c & 1) + 4 * (c >> 1);
        high = __funnelshift_r(x, x, at) & 0x000F000Fu;
      } else {
        const uint32_t x = tc_lds16(qh + ((((key >> 1) * NB + blk) * 2 + (c & 1)) * 2 + (key & 1)) * 2) >> (4 * (c >> 1));
        high = (x & 3u) | (x >> 8 & 3u) << 2 | (x >> 2 & 3u) << 16 | (x >> 10 & 3u) << 18;
      }
    }
    const uint2 v = tc_lds64(codes + (q8 ? swz_off<box_w(D)>(key, 32 * blk + 8 * c, TK)
                                         : swz_off<box_w(D / 2)>(key, 16 * blk + 8 * (c & 1), TK)));
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint32_t w = i ? v.y : v.x;
        uint32_t t = q8 ? w >> (8 * e) & 0x00FF00FFu : w >> (4 * (c >> 1) + 8 * e) & 0x000F000Fu;
        t |= (high >> (2 * i + e) & 0x00010001u) << 4;
        const float x = fmaf(float(int(t & 0xFFFFu) - off), fd, fm), y = fmaf(float(int(t >> 16) - off), fd, fm);
        if constexpr (PARTS == 2) split_h2(x, y, hi[2 * i + e], lo[2 * i + e]);
        else hi[2 * i + e] = pack_h2(x, y);
      }
    const uint32_t at = row + ((((blk & 1) * 4 + c) ^ (key & 7)) << 4);
    tc_sts128(at, hi);
    if constexpr (PARTS == 2) tc_sts128(at + C::part, lo);
  }
}

// A block of a body tile's keys: headers, then the codes
template <int D, int PARTS>
__device__ __forceinline__ void tc_body_unit(const TcSide& u, int lane, int blk, int cnt) {
  constexpr int NB = TC<D, PARTS>::NB, KH = TC<D, PARTS>::KH;
  const bool min = type_has_min(u.type);
  const int off = u.type == KVQ_TYPE_Q8_0 ? 128 : type_code_offset(u.type);
  const float sc = tc_pow2(u.scale);
  uint32_t d[KH], m[KH];
#pragma unroll
  for (int k = 0; k < KH; ++k) {
    const int key = lane + 32 * k;
    float fd, fm;
    if (min) {
      const float2 f = __half22float2(u32_as_h2(tc_lds32(u.hdr + (key * NB + blk) * 4)));
      fd = f.x;
      fm = f.y;
    } else {
      fd = __half2float(__ushort_as_half(uint16_t(tc_lds16(u.hdr + (key * NB + blk) * 2))));
      fm = 0.0f;
    }
    if (KH * 32 > TC<D, PARTS>::TK && key >= TC<D, PARTS>::TK) return;  // (half a warp's keys)
    if (key >= cnt || !(fabsf(fd) <= 65504.0f) || !(fabsf(fm) <= 65504.0f)) fd = fm = 0.0f;  // past the end, or noted as not finite
    fd *= sc;
    fm *= sc;
    if constexpr (PARTS == 1) {
      if (!min) fm = -float(off) * fd;
      fd *= 16777216.0f;
    }
    d[k] = pack_h2(fd, fd);
    m[k] = pack_h2(fm, fm);
  }
  if constexpr (PARTS == 1) {
    if (u.type == KVQ_TYPE_Q8_0) tc_unit1<D, true, false>(u, lane, blk, d, m);
    else if (type_has_qh(u.type)) tc_unit1<D, false, true>(u, lane, blk, d, m);
    else tc_unit1<D, false, false>(u, lane, blk, d, m);
  } else {
    const uint32_t o = (0x6400u + uint32_t(type_code_offset(u.type))) * 0x10001u;
#pragma unroll 1
    for (int k = 0; k < KH; ++k) {
      const uint32_t dk = k ? d[KH - 1] : d[0], mk = k ? m[KH - 1] : m[0];
      if (u.type == KVQ_TYPE_Q8_0) tc_unit2<D, true, false>(u, lane + 32 * k, blk, dk, mk, o, false);
      else if (type_has_qh(u.type)) tc_unit2<D, false, true>(u, lane + 32 * k, blk, dk, mk, o, min);
      else tc_unit2<D, false, false>(u, lane + 32 * k, blk, dk, mk, o, min);
    }
  }
}

// The same of a tail tile (bf16 rows, 128-byte box columns of TT rows)
template <int D, int PARTS>
__device__ __noinline__ void tc_tail_unit(uint32_t rows, uint32_t dst, int pow, int key, int blk, bool ok) {
  using C = TC<D, PARTS>;
  const uint32_t row = dst + (blk / 2) * (C::TK * 128) + key * 128;
  const float scale = tc_pow2(pow);
#pragma unroll 1
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

// A warp's share of a side of a tile that the quick conversion is not for: bf16 rows, or headers too far apart.
template <int D, int PARTS>
__device__ __noinline__ void tc_slow_blocks(TcSide u, int first, int step, int cnt, bool tail, int lane) {
  using C = TC<D, PARTS>;
#pragma unroll 1
  for (int blk = first; blk < C::NB; blk += step)
#pragma unroll 1
    for (int key = lane; key < C::TK; key += 32) {
      if (!tail) tc_wide_unit<D, PARTS>(u.codes, u.hdr, u.qh, u.dst, u.type, u.scale, u.is_k, key, blk, key < cnt);
      else if (!u.is_k || key - lane < cnt) tc_tail_unit<D, PARTS>(u.codes, u.dst, u.scale, key, blk, key < cnt);  // (scores past the end are masked)
    }
}

// Values are below 2^this times their header's scale (with a minimum: twice the larger of that and the minimum).
__device__ __forceinline__ int tc_code_bits(int qt) {
  return qt == KVQ_TYPE_Q8_0 ? 7 : qt == KVQ_TYPE_Q5_0 || qt == KVQ_TYPE_Q4_1 ? 4 : qt == KVQ_TYPE_Q4_0 ? 3 : 5;
}
// A lane's share of a tile's headers: the largest and the smallest halves (scales, minima) in size, infinities and NaN going on in
// the first.
struct TcHeads {
  uint32_t most, least;
};
__device__ __forceinline__ uint32_t tc_most(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("{\n\t.reg .b32 x;\n\tabs.f16x2 x, %2;\n\tmax.NaN.f16x2 %0, %1, x;\n\t}" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ TcHeads tc_heads(uint32_t hdr, int words, int sub) {
  TcHeads t{0u, 0x7C007C00u};
  auto look = [&](uint32_t w) {
    t.most = tc_most(t.most, w);
    asm("{\n\t.reg .b32 x;\n\tabs.f16x2 x, %1;\n\tmin.f16x2 %0, %0, x;\n\t}" : "+r"(t.least) : "r"(w));
  };
#pragma unroll 1
  for (int i = sub; i < words / 4; i += 16) {
    const uint4 q = tc_lds128(hdr + 16 * i);
    look(q.x);
    look(q.y);
    look(q.z);
    look(q.w);
  }
  if (sub < (words & 3)) look(tc_lds32(hdr + 4 * (words / 4 * 4 + sub)));
  return t;
}
__device__ __noinline__ uint32_t tc_most_finite(uint32_t hdr, int words, int sub) {
  uint32_t mx = 0;
#pragma unroll 1
  for (int i = sub; i < words; i += 16) {
    uint32_t w = tc_lds32(hdr + 4 * i) & 0x7FFF7FFFu;
    if ((w & 0xFFFFu) >= 0x7C00u) w &= 0xFFFF0000u;
    if ((w >> 16) >= 0x7C00u) w &= 0xFFFFu;
    mx = tc_most(mx, w);
  }
  return mx;
}
// The quick conversion takes scales down to 2^-14 less this: half of fp16's smallest step, 2^-25, is 2^-12 of the largest of such
// a block's values (with a minimum: of half their range).
template <int PARTS>
__device__ __forceinline__ int tc_below_normal(int qt) {
  return PARTS == 2 ? 0 : qt == KVQ_TYPE_Q8_0 ? 5 : qt == KVQ_TYPE_Q5_0 ? 3 : qt == KVQ_TYPE_Q4_1 ? 1 : 2;
}
// The scales of a tile of which a header is 0 or too small for a first choice, s (all of a half warp): of each side one that has
// all that are not 0, else one over fp16's whole range, for the conversion from fp32.  keep: the values' scale of the tile
// before, top: how high it may go.  Returns the scales plus 512, ten bits each, and the sides for the conversion from fp32.
template <int PARTS>
__device__ __noinline__ uint32_t tc_scales(uint32_t hdr, int words, uint32_t most, int type, int s, int hi, int keep, int top,
                                        int lane) {
  const int side = lane >> 4, g = tc_below_normal<PARTS>(type), bits = tc_code_bits(type), p = most >> 10 & 31u, q = most >> 26;
  const bool sum = type_has_min(type);
  int least = 0x7FFF, full = sum ? max(p + bits, q) + 1 : max(p, q) + bits;
#pragma unroll 1
  for (int i = lane & 15; i < words * (sum ? 1 : 2); i += 16) {
    const int x = tc_lds16(hdr + i * (sum ? 4 : 2)) & 0x7FFF;
    if (x) least = min(least, x);
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
    full = max(full, __shfl_xor_sync(0xffffffffu, full, o));
  }
  full = 29 - full;
  const int lo = (least < 0x400 ? 10 : 1 - (least >> 10)) - g;
  uint32_t wide = 0u;
  if (s < lo) {
    wide = lo > hi;
    s = !wide ? max(lo, hi - 2 * side) : keep <= full && keep >= full - 4 ? keep : full - 2 * side;
    if (s > top) {
      s = top;
      wide = 1u;
    }
  }
  const uint32_t x = uint32_t(s + 512), k = __shfl_sync(0xffffffffu, x, 0), v = __shfl_sync(0xffffffffu, x, 16);
  return k | v << 10 | __shfl_sync(0xffffffffu, wide, 0) << 20 | __shfl_sync(0xffffffffu, wide, 16) << 21;
}
template <int D, int TT>
__device__ __noinline__ uint32_t tc_tail_max(uint32_t rows, int cnt, int lane) {  // (bit 31: not all are finite)
  uint32_t mx = 0, odd = 0;
#pragma unroll 4
  for (int i = lane; i < cnt * (D / 8); i += 32) {
    const uint4 q = tc_lds128(rows + swz_off<128>(i / (D / 8), i % (D / 8) * 16, TT));
    mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(q.x & 0x7FFF7FFFu, q.y & 0x7FFF7FFFu), __vmaxu2(q.z & 0x7FFF7FFFu, q.w & 0x7FFF7FFFu)));
  }
  mx = __reduce_max_sync(0xffffffffu, max(mx & 0xFFFFu, mx >> 16));
  if (mx >= 0x7F80u) {
    odd = 1u << 31;
    mx = 0;
#pragma unroll 1
    for (int i = lane; i < cnt * D; i += 32) {
      const uint32_t x = tc_lds16(rows + swz_off<128>(i / D, i % D * 2, TT)) & 0x7FFFu;
      if (x < 0x7F80u) mx = max(mx, x);
    }
    mx = __reduce_max_sync(0xffffffffu, mx);
  }
  return mx | odd;
}
// The keys of a tile that are not finite
template <int D, int TK, int TT>
__device__ __noinline__ uint2 tc_not_finite(uint32_t k, uint32_t v, int kh, int vh, int cnt, bool tail, int lane) {
  uint2 bad = make_uint2(0u, 0u);
#pragma unroll 1
  for (int h = 0; h < (TK + 31) / 32; ++h) {
    const int key = 32 * h + lane;
    bool is = false;
    if (key < cnt && !tail) {
#pragma unroll 1
      for (int i = 0; i < kh / 2; ++i) is |= (tc_lds16(k + key * kh + 2 * i) & 0x7FFFu) >= 0x7C00u;
#pragma unroll 1
      for (int i = 0; i < vh / 2; ++i) is |= (tc_lds16(v + key * vh + 2 * i) & 0x7FFFu) >= 0x7C00u;
    } else if (key < cnt) {
#pragma unroll 1
      for (int i = 0; i < 2 * D; ++i) {
        const uint32_t base = i >= D ? v : k;
        is |= (tc_lds16(base + swz_off<128>(key, (i % D) * 2, TT)) & 0x7FFFu) >= 0x7F80u;
      }
    }
    const uint32_t m = __ballot_sync(0xffffffffu, is);
    if (h) bad.y = m; else bad.x = m;
  }
  return bad;
}

// The scout: looks a tile's raw contents over when they have landed and notes its scales and the keys that are not finite.  (Every
// tile waits for it: both sides at once, by half a warp each, and what seldom runs out of line.)
template <int D, int PARTS>
__device__ void tc_scout(const ChunkArgs& a, const TcStage& L, uint32_t ring, TcSync* sy, int lane) {
  using C = TC<D, PARTS>;
  // A header's exponents are raised by `up`, a minimum's by `upm`: 6 less the largest is the scale (PARTS 1:
  // scales below 2^-8, minima below 2^14; else all values below 2^15).
  const int side = lane >> 4, sub = lane & 15, type = side ? a.c.v_type : a.c.k_type;
  const bool sum = type_has_min(type);
  const int up = PARTS == 1 ? 0 : tc_code_bits(type) - (sum ? 22 : 23), upm = sum ? -22 : up;
  const int hoff = side ? L.vd : L.kd, hrow = side ? L.vh : L.kh, g = tc_below_normal<PARTS>(type);
  const uint32_t only = sum ? 0x7FFF0000u : 0u;
  int vs = 0, low = 0, r = 0;
  uint32_t phase = 0;
#pragma unroll 1
  for (int ct = 0;; ++ct) {
    if (!tc_wait(&sy->rfull[r], phase)) return;
    const uint4 job = tc_lds128(smem_u32(&sy->job[r]));
    const int cnt = int(job.y);
    const uint32_t st = ring + r * L.bytes;
    const bool tail = int(job.z) >= 0;
    int ks, hi;  // the largest scales
    bool odd;
    TcHeads t{0u, 0x7C007C00u};
    if (!tail) {
      const int words = cnt * hrow / 4;
      t = tc_heads(st + hoff, words, sub);
      odd = __any_sync(0xffffffffu, (t.most & 0x7C00u) == 0x7C00u || t.most >= 0x7C000000u);
      if (odd) t.most = tc_most_finite(st + hoff, words, sub);
      const int e = max(int(t.most >> 10 & 31u) + up, int(t.most >> 26) + upm);
      ks = 6 - __reduce_max_sync(0xffffffffu, side ? -64 : e);
      hi = 6 - __reduce_max_sync(0xffffffffu, side ? e : -64);
    } else {
      const uint32_t k = tc_tail_max<D, C::TT>(st, cnt, lane), v = tc_tail_max<D, C::TT>(st + L.vt, cnt, lane);
      odd = (k | v) >> 31;
      ks = min(141 - int(k >> 7 & 255u), 100);
      hi = min(141 - int(v >> 7 & 255u), 100);
    }
    // Values keep the scale of the tile before where it serves, since O is rescaled where it changes.  Else they take one with
    // some room for a larger tile.  It goes up as well as down, so that rows that see small values alone have their bits
    // whatever else the segment holds, but not above kTcRise over its lowest: a sum of 2^20 products below 2^30,
    // 2^kTcRise times that, is within fp32.
    const int keep = vs;
    if (job.w || vs > hi || vs < hi - 4) vs = job.w ? hi - 2 : min(hi - 2, low + kTcRise);
    uint32_t wide = tail ? 7u : 0u;  // (sides that the quick conversion is not for; 4: bf16 rows)
    const int scale = side ? vs : ks;
    if (__any_sync(0xffffffffu, int(min(t.least & 0xFFFFu, (t.least | only) >> 16)) < max(1 - g - scale, 1) << 10)) {
      const bool first = side == 0 || job.w;
      const uint32_t x = tc_scales<PARTS>(st + hoff, cnt * hrow / 4, t.most, type, scale, side ? hi : ks, first ? 1000 : keep,
                                          first ? 1000 : low + kTcRise, lane);
      ks = int(x & 1023u) - 512;
      vs = int(x >> 10 & 1023u) - 512;
      wide = x >> 20;
    }
    low = job.w ? vs : min(low, vs);
    uint2 bad = make_uint2(0u, 0u);
    if (odd) bad = tc_not_finite<D, C::TK, C::TT>(st + (tail ? 0 : L.kd), st + (tail ? L.vt : L.vd), L.kh, L.vh, cnt, tail, lane);
    if (lane == 0) {
      const uint32_t at = smem_u32(&sy->meta[ct % kTcMeta]);
      tc_sts128(at, {job.x, job.y, uint32_t(ks), uint32_t(vs)});
      tc_sts128(at + 16, {bad.x, bad.y, wide, 0u});
      mbar_arrive(&sy->mfull[r]);
    }
    if (cnt < 0) return;  // (the end)
    if (++r == L.stages) { r = 0; phase ^= 1; }
  }
}

template <int D, int PARTS>
__device__ void tc_convert(const ChunkArgs& a, const TcStage& L, uint32_t sb, TcSync* sy, int warp, int lane) {
  using C = TC<D, PARTS>;
  constexpr int NB = C::NB, W = kTcConv / 2;  // blocks of a key, warps of a side
  const int side = warp / W;
  uint64_t *empty = side ? sy->vempty : sy->kempty, *full = side ? sy->vfull : sy->kfull;
  TcSide x;
  x.is_k = side == 0;
  x.type = side ? a.c.v_type : a.c.k_type;
  int r = 0, b = 0;
  uint32_t phase = 0, turn = 1;  // parities of the ring's round and of the slots' round before
#pragma unroll 1
  for (int ct = 0;; ++ct) {
    if (!tc_wait(&sy->rfull[r], phase) || !tc_wait(&sy->mfull[r], phase)) return;
    const uint4 mt = tc_lds128(smem_u32(&sy->meta[ct % kTcMeta]));
    const int cnt = int(mt.y);
    if (cnt < 0) return;
    const uint32_t how = tc_lds32(smem_u32(&sy->meta[ct % kTcMeta].b.z));
    const bool tail = how & 4u;
    const uint32_t st = sb + C::off_ring + r * L.bytes;
    if (ct >= C::NS && !tc_wait(&empty[b], turn)) return;
    x.scale = int(side ? mt.w : mt.z);
    x.codes = st + (side ? (tail ? L.vt : L.v) : 0);
    x.hdr = st + (side ? L.vd : L.kd);
    x.qh = st + (side ? L.vqh : L.kqh);
    x.dst = sb + (side ? C::off_v : C::off_k) + b * C::slot;
    if (how >> side & 1u) {
      tc_slow_blocks<D, PARTS>(x, warp % W, W, cnt, tail, lane);
    } else {
#pragma unroll 1
      for (int blk = warp % W; blk < NB; blk += W) tc_body_unit<D, PARTS>(x, lane, blk, cnt);
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&full[b]);
      mbar_arrive(&sy->rempty[r]);
    }
    if (++r == L.stages) { r = 0; phase ^= 1; }
    if (++b == C::NS) { b = 0; turn ^= 1; }
  }
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
  int r = 0;
  uint32_t phase = 1;  // (a ring's first round waits for nothing)
  auto put = [&](int4 job, int row) {  // one lane
    if (ct >= L.stages && !tc_wait(&sy->rempty[r], phase)) return false;
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
  bool more = true;
  while (ok && more) {
    more = walk.next(a, h, it, kvh, j0, j1);
    if (!more) { j0 = 0; j1 = 1; it.b = 0; kvh = 0; }  // one more job: the end
    const int n = min(max(c.seq_len[it.b], 0), c.max_ctx);
    const int bh = it.b * c.n_kv_heads + kvh;
#pragma unroll 1
    for (int jb = j0; ok && jb < j1; jb += 32) {
      // a lane a tile: its rows, so that the page table's loads overlap
      int4 job = make_int4(0, 0, -1, 0);
      int row = 0;
      if (!more) {
        job.y = -1;
      } else if (jb + lane < j1) {
        // from the last keys to the first: with a bias by distance the largest score comes first, and O is not rescaled
        const ChunkTile t = chunk_tile<C::TK, C::TT>(a, it, n, j1 - 1 - (jb + lane - j0));
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
#pragma unroll 1
      for (int k = 0; k < 32 && jb + k < j1; ++k) {
        const int4 x = make_int4(__shfl_sync(0xffffffffu, job.x, k), __shfl_sync(0xffffffffu, job.y, k),
                                 __shfl_sync(0xffffffffu, job.z, k), __shfl_sync(0xffffffffu, job.w, k));
        const int rw = __shfl_sync(0xffffffffu, row, k);
        int fine = 1;
        if (lane == 0) fine = put(x, rw);
        if (!__shfl_sync(0xffffffffu, fine, 0)) { ok = false; break; }
        ++ct;
        if (++r == L.stages) { r = 0; phase ^= 1; }
      }
    }
  }
  if (lane == 0) {
    // copies still landing when a wait gave up: they end before the CTA does
    if (!ok)
      for (int k = max(0, ct - L.stages); k < ct; ++k) mbar_wait_bounded(&sy->rfull[k % L.stages], (k / L.stages) & 1, kTcWait);
  }
}

// ---- issuers ---------------------------------------------------------------------------------------

// Which of its score buffers (with their weights) a group's n-th tile uses, and the parity of that use.
template <class C>
__device__ __forceinline__ int tc_buffer(int g, uint32_t n) { return C::SB == 2 ? 2 * g + int(n & 1) : g; }
template <class C>
__device__ __forceinline__ uint32_t tc_turn(uint32_t n) { return (C::SB == 2 ? n >> 1 : n) & 1; }

// The next segment's number of tiles (-1: none left), and whether its rows are more than a group's (C2: there are two groups).
template <bool C2>
__device__ __forceinline__ int tc_next_tiles(ChunkWalk& walk, const ChunkArgs& a, const ChunkHeader& h, bool& both) {
  ChunkItem it;
  int kvh, j0 = 0, j1 = 0;
  const bool more = walk.next(a, h, it, kvh, j0, j1);
  both = C2 && more && it.rows > 128;
  return more ? j1 - j0 : -1;
}

template <int D, int PARTS>
__device__ void tc_issue_s(const ChunkArgs& a, const ChunkHeader& h, uint32_t sb, uint32_t tmem, TcSync* sy) {
  using C = TC<D, PARTS>;
  constexpr uint32_t idesc = tc::idesc_f16_f32(128, C::TK);
  const uint64_t dk = tc::sdesc_sw128(sb + C::off_k), dq = tc::sdesc_sw128(sb + C::off_q);
  ChunkWalk walk;
  walk.begin(a, h, blockIdx.x);
  bool both;
  int seg = 0, s = 0;
  uint32_t phase = 0, n0 = 0, n1 = 0;  // the groups' tiles
  // (no loop ends on what a wait returns: the compiler has to see that all lanes go the same way)
#pragma unroll 1
  for (int nt; (nt = tc_next_tiles<C::NG == 2>(walk, a, h, both)) >= 0;) {
    if (nt == 0) continue;
    tc_wait(&sy->qready, seg++ & 1);
#pragma unroll 1
    for (int k = 0; k < nt; ++k) {
      const bool have = tc_wait(&sy->kfull[s], phase);
      const uint64_t kb = dk + ((s * C::slot) >> 4);
#pragma unroll 1
      for (int i = 0; i < (both ? 2 : 1); ++i) {
        const int g = C::NG == 1 ? 0 : both ? i : k & 1;
        const uint32_t n = g ? n1++ : n0++;
        const int b = tc_buffer<C>(g, n);
        const bool ok = have && (n < C::SB || tc_wait(C::OVER ? &sy->odone[b] : &sy->sfree[b], tc_turn<C>(n) ^ 1));
        if (!__all_sync(0xffffffffu, ok)) continue;
        tc::fence_after_sync();
        const uint32_t d = tmem + C::scol + b * C::TK, q = tmem + (both ? g * C::qw : 0);
        const uint64_t qd = dq + (both ? (g * PARTS * D * 256) >> 4 : 0);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint32_t ko = ((ks / 4) * (C::TK * 128) + (ks % 4) * 32) >> 4;
          const uint32_t qo = ((ks / 4) * (128 * 128) + (ks % 4) * 32) >> 4;
          auto mma = [&](int qp, int kp, uint32_t acc) {
            if constexpr (C::QSMEM) tc::mma_f16_warp(d, qd + qo + ((qp * D * 256) >> 4), kb + ko + ((kp * C::part) >> 4), idesc, acc);
            else tc::mma_f16_ts_warp(d, q + qp * (D / 2) + ks * 8, kb + ko + ((kp * C::part) >> 4), idesc, acc);
          };
          mma(0, 0, ks > 0 ? 1u : 0u);
          if constexpr (PARTS == 2) {
            mma(0, 1, 1u);
            mma(1, 0, 1u);
          }
        }
        tc::commit_warp(&sy->sfull[b]);
      }
      tc::commit_warp(&sy->kempty[s]);
      phase ^= s == C::NS - 1;
      s = s == C::NS - 1 ? 0 : s + 1;
    }
  }
  tc::commit_warp(&sy->fin[0]);
}

template <int D, int PARTS>
__device__ void tc_issue_pv(const ChunkArgs& a, const ChunkHeader& h, uint32_t sb, uint32_t tmem, TcSync* sy) {
  using C = TC<D, PARTS>;
  constexpr uint32_t idesc1 = tc::idesc_f16_f32(128, C::N1) | tc::kIdescBmn;
  constexpr uint32_t idesc2 = tc::idesc_f16_f32(128, C::N2 > 0 ? C::N2 : 16) | tc::kIdescBmn;
  const uint64_t dv = tc::sdesc_sw128_mn(sb + C::off_v, C::TK * 128);
  ChunkWalk walk;
  walk.begin(a, h, blockIdx.x);
  bool both;
  int s = 0;
  uint32_t phase = 0, n0 = 0, n1 = 0;
#pragma unroll 1
  for (int nt; (nt = tc_next_tiles<C::NG == 2>(walk, a, h, both)) >= 0;) {
#pragma unroll 1
    for (int k = 0; k < nt; ++k) {
      const bool have = tc_wait(&sy->vfull[s], phase);
      const uint64_t vb = dv + ((s * C::slot) >> 4);
      const uint32_t first = k < (C::NG == 2 && !both ? 2 : 1) ? 0u : 1u;  // a group's first tile begins a new sum
#pragma unroll 1
      for (int i = 0; i < (both ? 2 : 1); ++i) {
        const int g = C::NG == 1 ? 0 : both ? i : k & 1;
        const uint32_t n = g ? n1++ : n0++;
        const int b = tc_buffer<C>(g, n);
        const bool ok = have && tc_wait(&sy->pfull[b], tc_turn<C>(n));
        if (!__all_sync(0xffffffffu, ok)) continue;
        tc::fence_after_sync();
        const uint32_t o = tmem + C::ocol + g * D, p = tmem + C::pcol + b * C::pstep;
#pragma unroll
        for (int ks = 0; ks < C::TK / 16; ++ks) {
          auto mma = [&](int pp, int vp, uint32_t acc) {
            const uint64_t v = vb + ((vp * C::part + ks * 2048) >> 4);
            tc::mma_f16_ts_warp(o, p + pp * (C::TK / 2) + ks * 8, v, idesc1, acc);
            if constexpr (C::N2 > 0)
              tc::mma_f16_ts_warp(o + C::N1, p + pp * (C::TK / 2) + ks * 8, v + (((C::N1 / 64) * C::TK * 128) >> 4), idesc2, acc);
          };
          mma(0, 0, ks > 0 ? 1u : first);
          if constexpr (PARTS == 2) {
            mma(0, 1, 1u);
            mma(1, 0, 1u);
          }
        }
        tc::commit_warp(&sy->odone[b]);
      }
      tc::commit_warp(&sy->vempty[s]);
      phase ^= s == C::NS - 1;
      s = s == C::NS - 1 ? 0 : s + 1;
    }
  }
  tc::commit_warp(&sy->fin[1]);
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

// Scores in TMEM times f, capped: s = c tanh(s / c), off by 2^-20.8 of itself at most.  With y = s / c it is s p(y^2) where |y| is below
// 0.447, p being 1 and a fit of the smallest largest error (2^-21.8) to tanh(y) / y - 1 on y^2 from 0 to 0.2: a cap far above
// the scores changes none.  Further on it is c - 2 c / (1 + e^(2 y)), which for small y would lose the digits of s in those of
// c; most tiles have no such score.  (Out of line, so that calls without a cap do not fetch it: mixed chunks in fp16 183 us
// for 199, 2 x 4096 prompt rows with a cap 753 for 821, without one 511 for 479.)
template <int TK>
__device__ __noinline__ void tc_cap(uint32_t at, float f, float cap) {
  at = __shfl_sync(0xffffffffu, at, 0);
  const float c = cap * kChunkLog2e, i = fminf(1.0f / c, 3.4e38f);  // (no infinity: times a score of 0)
  const float fi = fminf(f * i, 3.4e38f), c1 = -0.33330584f * f, c2 = 0.13248634f * f, c3 = -0.046406726f * f;
#pragma unroll 1
  for (int c0 = 0; c0 < TK; c0 += 16) {
    float v[16];
    tc::ld_x16(at + c0, v);
    tc::wait_ld();
    float top = 0.0f;
#pragma unroll
    for (int k = 0; k < 16; ++k) top = fmaxf(top, fabsf(v[k]));
    if (!__any_sync(0xffffffffu, top * fi > 0.447f)) {
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float y = v[k] * fi, u = y * y;
        v[k] *= fmaf(fmaf(fmaf(c3, u, c2), u, c1), u, f);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const float y = v[k] * fi, u = y * y;
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + ex2_approx(2.0f * kChunkLog2e * y)));
        const float low = v[k] * fmaf(fmaf(fmaf(c3, u, c2), u, c1), u, f);
        v[k] = u < 0.2f ? low : fmaf(-2.0f * c, r, c);
      }
    }
    tc::st_x16(at + c0, v);
  }
  tc::wait_st();
}

// Whether one of the keys in bad0, bad1 (columns 0-31, 32-63) lies in [lo, hi)
__device__ __noinline__ bool tc_sees(uint32_t bad0, uint32_t bad1, int lo, int hi) {
  for (int c = max(lo, 0); c < min(hi, 64); ++c)
    if ((c < 32 ? bad0 >> c : bad1 >> (c - 32)) & 1u) return true;
  return false;
}

template <int D, int PARTS>
__device__ void tc_softmax(const ChunkArgs& a, const ChunkHeader& h, uint8_t* sm, uint32_t tmem, TcSync* sy, int warp, int lane) {
  using C = TC<D, PARTS>;
  constexpr int TK = C::TK, NG = C::NG;
  const int grp = NG == 2 ? warp / 4 : 0, line = (warp & 3) * 32 + lane;
  uint32_t used = 0;  // the group's tiles
  const uint32_t lanes = tmem + (uint32_t((warp & 3) * 32) << 16);
  auto all = [&]() {  // the softmax warps, TMEM contents included
    tc::fence_before_sync();
    named_sync(1, C::kSoft);
    tc::fence_after_sync();
  };
  ChunkWalk walk;
  walk.begin(a, h, blockIdx.x);
  ChunkItem it;
  int kvh, j0, j1, ct = 0;
  while (walk.next(a, h, it, kvh, j0, j1)) {
    const int row0 = a.row_start[it.b], m = a.row_start[it.b + 1] - row0, n = min(max(a.c.seq_len[it.b], 0), a.c.max_ctx);
    const int nk = it.n_body + it.n_tail, nt = j1 - j0;
    const bool both = NG == 2 && it.rows > 128;  // the groups have different rows
    const int row = both ? grp * 128 + line : line, c0 = both ? 0 : grp, cstep = both ? 1 : NG;  // the row's item; its chunks
    const bool whole = nt == nk, have = row < it.rows, busy = (both ? grp * 128 : 0) + (warp & 3) * 32 < it.rows;  // busy: the warp has rows
    const int w = have ? it.r0 + row : it.r0, tok = int(div_u32(uint32_t(w), a.by_group)), hh = w - tok * a.group;
    const size_t base = ((size_t)(row0 + tok) * a.n_q_heads + kvh * a.group + hh) * D;
    ChunkSpan span{0, 0x7fffffff, 0x7fffffff};  // (lanes without a row mask nothing)
    float slope2 = 0.0f;
    int qs = 0;
    if (nt > 0) {
      if (have) span = chunk_span(a, it.b, n, row0, m, tok);
      if (a.mod.slopes && have) slope2 = a.mod.slopes[kvh * a.group + hh] * kChunkLog2e;
      // ---- queries: 32 channels at a time to TMEM (where O will be), rotated there, scaled, to their operand's place
      const uint32_t tmp = lanes + C::ocol + (both ? grp * D : 0);
      float top = 0.0f;
      if (busy) {
#pragma unroll 1
        for (int c = c0; c < C::NB; c += cstep) {
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
          for (int s = c0; s < 4 * (D / C::G); s += cstep) {  // 8 of the 32 channels, of all chunks of a rotation group
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
      if constexpr (NG == 2) sy->rowmax[grp][line] = top;
      all();
      if constexpr (NG == 2)
        if (!both) top = fmaxf(top, sy->rowmax[1 - grp][line]);
      const float sc = a.scale * kChunkLog2e * (a.rot_k ? inv_sqrt_group<C::G>() : 1.0f);
      qs = min(11 - tc_exp(top * sc), 126);  // the largest below 2^11
      const float qf = tc_pow2(qs);
      if (busy) {
#pragma unroll 1
        for (int c = c0; c < C::NB; c += cstep) {
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
            const uint32_t at = smem_u32(sm) + C::off_q + (both ? grp * PARTS * D * 256 : 0) + (c / 2) * (128 * 128);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              tc_sts128(at + tc::sw128_chunk(line, (c & 1) * 4 + i), *reinterpret_cast<uint32_t(*)[4]>(&hi[4 * i]));
              if constexpr (PARTS == 2)
                tc_sts128(at + D * 256 + tc::sw128_chunk(line, (c & 1) * 4 + i), *reinterpret_cast<uint32_t(*)[4]>(&lo[4 * i]));
            }
          } else {
            const uint32_t qc = lanes + (both ? grp * C::qw : 0) + c * 16;
            tc::st_x16(qc, *reinterpret_cast<float(*)[16]>(&hi[0]));
            if constexpr (PARTS == 2) tc::st_x16(qc + D / 2, *reinterpret_cast<float(*)[16]>(&lo[0]));
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
    int vs = 0, mine = 0;  // the group's tiles so far
    bool nan = false;
    for (int k = 0; k < nt; ++k, ++ct) {
      if (NG == 2 && !both && (k & 1) != grp) continue;
      const uint32_t n = used++;
      const int b = tc_buffer<C>(grp, n);
      bool ok = tc_wait(&sy->sfull[b], tc_turn<C>(n));
      ok = __all_sync(0xffffffffu, ok);
      if (ok && busy) {
        tc::fence_after_sync();
        const uint32_t meta = smem_u32(&sy->meta[ct % kTcMeta]);
        const uint4 mt = tc_lds128(meta);
        const uint2 bad = tc_lds64(meta + 16);
        const int t0 = int(mt.x), cnt = int(mt.y), nvs = int(mt.w);
        float f = tc_pow2(-int(mt.z) - qs);
        const int lo = span.lo - t0, hi = min(span.hi - t0, cnt);
        const bool edge = __any_sync(0xffffffffu, lo > 0 || hi < TK), changed = a.mod.slopes || edge;
        const bool ahead = __any_sync(0xffffffffu, t0 + TK - 1 > span.pos);  // keys behind a row's own position
        if (bad.x | bad.y) nan |= tc_sees(bad.x, bad.y, lo, hi);
        // scores that are biased or masked: 16 columns at a time, back to TMEM, times f
        const uint32_t sc0 = lanes + C::scol + b * TK;
        float mt2 = -INFINITY;
        if (a.mod.softcap > 0.0f) {
          tc_cap<TK>(sc0, f, a.mod.softcap);
          f = 1.0f;
        }
        if (changed) {
          mt2 = -INFINITY;
#pragma unroll 1
          for (int c0 = 0; c0 < TK; c0 += 16) {
            float sv[16];
            tc::ld_x16(sc0 + c0, sv);
            tc::wait_ld();
            const float d0 = float(t0 + c0 - span.pos);  // (exact up to 2^24; beyond, a step of it is 2^-24 of the bias)
            if (a.mod.slopes && !ahead) {  // -slope |position - t| is linear
              const float b0 = slope2 * d0;
#pragma unroll
              for (int c = 0; c < 16; ++c) sv[c] = fmaf(sv[c], f, fmaf(slope2, float(c), b0));
            } else if (a.mod.slopes) {
#pragma unroll
              for (int c = 0; c < 16; ++c) sv[c] = fmaf(sv[c], f, -slope2 * fabsf(d0 + float(c)));
            } else {
#pragma unroll
              for (int c = 0; c < 16; ++c) sv[c] *= f;
            }
            if (edge) {  // columns c0 + c from lo on, below hi
              const uint32_t room = uint32_t(max(hi - lo, 0)), from = uint32_t(c0 - lo);
#pragma unroll
              for (int c = 0; c < 16; ++c)
                if (from + c >= room) sv[c] = -INFINITY;
            }
            tc::st_x16(sc0 + c0, sv);
            float mx[2] = {sv[0], sv[1]};
#pragma unroll
            for (int c = 2; c < 16; ++c) mx[c & 1] = fmaxf(mx[c & 1], sv[c]);
            mt2 = fmaxf(mt2, fmaxf(mx[0], mx[1]));
          }
          tc::wait_st();
          f = 1.0f;
        } else {
          float sv[TK];
#pragma unroll
          for (int c = 0; c < TK; c += 16) tc::ld_x16(sc0 + c, *reinterpret_cast<float(*)[16]>(&sv[c]));
          tc::wait_ld();
          float mx[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
          for (int c = 4; c < TK; ++c) mx[c & 3] = fmaxf(mx[c & 3], sv[c]);
          mt2 = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * f;
        }
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
        // the weights' place is free once the product that read it is done; to rescale O, the group's last product has to be
        if (n >= C::SB) ok = tc_wait(&sy->odone[b], tc_turn<C>(n) ^ 1);
        const bool resc = mine > 0 && __any_sync(0xffffffffu, move);
        if (C::SB == 2 && resc) ok = tc_wait(&sy->odone[tc_buffer<C>(grp, n - 1)], tc_turn<C>(n - 1)) && ok;
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
          tc::fence_after_sync();
          if (resc) {
            const uint32_t o = lanes + C::ocol + grp * D;
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              float t[16];
              tc::ld_x16(o + c, t);
              tc::wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) t[e] *= alpha;
              tc::st_x16(o + c, t);
            }
          }
          // the weights, kW columns at a time (a loop of 16 is shorter code, but waits for TMEM four times: prompts take 10% longer
          // with it, two-part operands 12% less).  (P over S: it lies before the scores still to be read)
          const uint32_t p = lanes + C::pcol + b * C::pstep;
          float ls[2] = {0.0f, 0.0f};
          constexpr int kW = PARTS == 1 ? TK : 16;
#pragma unroll 1
          for (int c0 = 0; c0 < TK; c0 += kW) {
            float sv[kW], ph[kW / 2], pl[PARTS == 2 ? kW / 2 : 8];
#pragma unroll
            for (int c = 0; c < kW; c += 16) tc::ld_x16(sc0 + c0 + c, *reinterpret_cast<float(*)[16]>(&sv[c]));
            tc::wait_ld();
#pragma unroll
            for (int c = 0; c < kW; c += 2) {
              const float e0 = ex2_approx(fmaf(sv[c], f, -mb)), e1 = ex2_approx(fmaf(sv[c + 1], f, -mb));
              ls[0] += e0;
              ls[1] += e1;
              if constexpr (PARTS == 2) split_h2(e0, e1, reinterpret_cast<uint32_t&>(ph[c / 2]), reinterpret_cast<uint32_t&>(pl[c / 2]));
              else ph[c / 2] = __uint_as_float(pack_h2(e0, e1));
            }
#pragma unroll
            for (int c = 0; c < kW / 2; c += 8) {
              tc::st_x8(p + c0 / 2 + c, *reinterpret_cast<float(*)[8]>(&ph[c]));
              if constexpr (PARTS == 2) tc::st_x8(p + TK / 2 + c0 / 2 + c, *reinterpret_cast<float(*)[8]>(&pl[c]));
            }
          }
          l += ls[0] + ls[1];
          tc::wait_st();
          tc::fence_before_sync();
          if (!C::OVER) {
            __syncwarp();
            if (lane == 0) mbar_arrive(&sy->sfree[b]);
          }
        }
      } else {  // no rows: in step with the others all the same, or its arrivals would count for their next tile
        __syncwarp();
        if (!C::OVER && lane == 0) mbar_arrive(&sy->sfree[b]);
        if (n >= C::SB) tc_wait(&sy->odone[b], tc_turn<C>(n) ^ 1);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sy->pfull[b]);
      ++mine;
    }

    // ---- the rows' results
    bool ok = true;
    if (mine > 0) ok = tc_wait(&sy->odone[tc_buffer<C>(grp, used - 1)], tc_turn<C>(used - 1));  // the last product
    float M = m_used, f[2] = {1.0f, 0.0f};
    bool read[2] = {mine > 0, false};
    if (NG == 2 && !both) {
      sy->join[grp][line] = make_float4(mine > 0 ? m_used : -INFINITY, l, tc_pow2(-vs), nan || mine == 0 ? (nan ? 1.0f : 2.0f) : 0.0f);
      all();
      const float4 x0 = sy->join[0][line], x1 = sy->join[1][line];
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
    const size_t slot = (size_t)(2 * blockIdx.x + (j0 == 0 ? 1 : 0)) * C::M + row;
    if (whole) {
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      f[0] *= inv;
      f[1] *= inv;
    } else if (have && (both || grp == 0)) {
      a.part_ml[slot] = make_float2(M == -INFINITY && nan ? 0.0f : M, l);
    }
    const bool any0 = __any_sync(0xffffffffu, read[0]) && ok, any1 = NG == 2 && __any_sync(0xffffffffu, read[1]) && ok;
    const uint32_t own = lanes + C::ocol + (both ? grp * D : 0);
    // 32 channels of O, joined, in natural order
    auto chunk = [&](int c, float (&v)[32]) {
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = 0.0f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        if (!(g ? any1 : any0)) continue;
        float t[32];
        tc::ld_x16(own + g * D + c * 32, *reinterpret_cast<float(*)[16]>(&t[0]));
        tc::ld_x16(own + g * D + c * 32 + 16, *reinterpret_cast<float(*)[16]>(&t[16]));
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
      for (int c = c0; c < C::NB; c += cstep) {
        float v[32];
        chunk(c, v);
        if (turn) {
          tc_fwht32(v);
          tc::st_x16(own + c * 32, *reinterpret_cast<float(*)[16]>(&v[0]));
          tc::st_x16(own + c * 32 + 16, *reinterpret_cast<float(*)[16]>(&v[16]));
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
        for (int s = c0; s < 4 * (D / C::G); s += cstep) {
          const int at = (s / 4) * C::G + (s % 4) * 8;
          float v[C::GC][8];
#pragma unroll
          for (int k = 0; k < C::GC; ++k) tc::ld_x8(own + at + k * 32, v[k]);
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
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  TcSync* sy = tc_sync();
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  // while the plan is made: what needs none of it
  if (warp == 0) {
    tc::tmem_alloc(&sy->tmem, 512);
    tc::tmem_relinquish();
  }
  if (tid == 32) {
    for (int i = 0; i < L.stages; ++i) {
      mbar_init(&sy->rfull[i], 1);
      mbar_init(&sy->mfull[i], 1);
      mbar_init(&sy->rempty[i], kTcConv);
    }
    for (int i = 0; i < C::NS; ++i) {
      mbar_init(&sy->kfull[i], kTcConv / 2); mbar_init(&sy->kempty[i], 1);
      mbar_init(&sy->vfull[i], kTcConv / 2); mbar_init(&sy->vempty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sy->sfull[i], 1); mbar_init(&sy->sfree[i], 4);
      mbar_init(&sy->pfull[i], 4); mbar_init(&sy->odone[i], 1);
    }
    mbar_init(&sy->fin[0], 1);
    mbar_init(&sy->fin[1], 1);
    mbar_init(&sy->qready, C::kSoft / 32);
    sy->abort = 0;
    sy->status = a.c.status;
    fence_barrier_init();
    prefetch_tmap(&tmK);
    prefetch_tmap(&tmV);
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  // (The compiler has to see that addresses of TMEM, and the way to an instruction on it, are the same in every lane of a warp: so
  // the walks are inlined, not on the stack, and no loop around one ends on what a wait returns.)
  const uint32_t tmem = __shfl_sync(0xffffffffu, sy->tmem, 0);
  pdl_begin();
  const ChunkHeader h = *a.head;
  if (!h.ok || int(blockIdx.x) >= h.pieces) {  // (the whole CTA)
    if (warp == 0) tc::tmem_dealloc(tmem, 512);
    return;
  }
  constexpr int W0 = C::kSoft / 32;
  if (warp < W0) {
    tc_softmax<D, PARTS>(a, h, sm, tmem, sy, warp, lane);
  } else if (warp < W0 + kTcConv) {
    tc_convert<D, PARTS>(a, L, smem_u32(sm), sy, warp - W0, lane);
  } else if (warp == W0 + kTcConv + 3) {
    tc_scout<D, PARTS>(a, L, smem_u32(sm) + C::off_ring, sy, lane);
  } else if (warp == W0 + kTcConv) {
    tc_produce<D, PARTS>(a, L, h, sm, sy, lane, &tmK, &tmV, &tmKt, &tmVt);
  } else if (warp == W0 + kTcConv + 1) {
    tc_issue_s<D, PARTS>(a, h, smem_u32(sm), tmem, sy);
  } else {
    tc_issue_pv<D, PARTS>(a, h, smem_u32(sm), tmem, sy);
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
  const int room = 232448 - 1024 - C::off_ring;
  s.stages = std::min(kTcMaxStages, room / s.bytes);
  if (s.stages < 1) return cudaErrorInvalidValue;
  // (more than half of an SM's, so that no two CTAs of one SM ask for all of TMEM)
  const int bytes = std::max(120 * 1024, C::off_ring + s.stages * s.bytes + 1024);

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

template <int D>
ChunkTiles tc_tiles(int parts) {
  return parts == 1 ? ChunkTiles{TC<D, 1>::M, TC<D, 1>::TK, TC<D, 1>::TT} : ChunkTiles{TC<D, 2>::M, TC<D, 2>::TK, TC<D, 2>::TT};
}
template <int D>
cudaError_t launch_tc(ChunkArgs& a, int parts, cudaStream_t st) {
  return parts == 1 ? run_chunk_tc<D, 1>(a, st) : run_chunk_tc<D, 2>(a, st);
}

}  // namespace
}  // namespace kvq
