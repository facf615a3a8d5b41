// Decode attention over selected blocks (kvq_sparse_decode_attention).
//
// A row of work is one (sequence, KV head, group of up to eight query heads).  A cluster of
// CTAs shares a row: its warps take the listed blocks' tiles (kRows<D> tokens) in turn, each
// with its own ring of shared-memory stages filled by TMA and its own online softmax, and the
// partials of all its warps are merged through distributed shared memory -- one launch, no
// workspace.
//
// Scores of a tile, heads x tokens, on the tensor cores: A = the query (16 rows: fp16 high
// parts of eight heads, then the low parts; the two rows of a head are added, so one mma does
// both parts), B = the codes less their offset, exact in fp16, a block's result times its scale
// in fp32.  The query is scaled by a power of two (its largest value below 2^11) so that its low
// parts stay far above fp16's smallest step.  The mma's result has exactly the layout of P as
// the B operand of P.V, so P never moves between lanes.  P.V is the decode's: A = centred codes
// (channels x tokens), B = P times the block's scale as fp16 high and low parts.
//
// Codes are centred everywhere.  Uncentred they could go in as fp16 subnormals, a mask or byte
// permute each, with the offset as the mma's initial value: 3% faster, but the sums are then
// some times larger than their result, and fp32 outputs were 1.4e-6 off instead of 1.5e-7.  The
// scale + minimum formats are centred too: code - c with the minimum + c * scale.
//
// Bound by the instruction stream, about 630 warp instructions per 16 tokens of head_dim 128 in
// q5_0 (the 5-bit codes' conversion takes 250 of them), and with many rows by their division: a row
// is one CTA then, so that some SMs have two and others one, and short rows leave theirs early.  32
// sequences x 8 KV heads x up to 2048 tokens, q5_0 / q5_0: 52.0 us (92 MB: 13.8 us at the card's measured
// copy rate); 4 x 4 x 8192 tokens of head_dim 256, q8_0 / q4_0, paged: 37.5 us (55 MB, 8.2 us), where the
// chain of 8 warps an SM and a call's fixed part (first tiles 5 us, merge 4 us) weigh; the smallest call 6.1 us.

#include <cooperative_groups.h>
#include <string.h>

#include <algorithm>

#include "kvq_decode_impl.cuh"

namespace kvq {
namespace {

namespace cg = cooperative_groups;

constexpr int kTailRows = 8;   // tokens of a tail tile
constexpr int kMaxStages = 4;

// Weights p = 2^(score - lim), lim a reference kLazyMax above the largest score at its last move, are at most 1.
// p times a V scale goes in as two fp16 parts, with an absolute error of 2^-25 (fp16's smallest step), so it is
// taken times 2^top: top is what brings the product with the largest scale met so far to 2^14 .. 2^15, so that
// small values keep their bits and large ones stay finite.  A warp begins with kTopMax and lowers top, with its
// sums, where a tile's scale reaches 2^(16 - top).  p 2^top is at most 2^15 in fp16: where top is larger (scales
// below 2^-10 only, so that others go without) the missing power of two 2^up goes to the tile's scales, in place.
// q8_0 codes go in divided by 16, 2^4 of top (with their range the product would lose 4 bits).
constexpr int kTopMax = 30;
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(uint32_t(127 + e) << 23); }

template <int D> constexpr int kRows = D <= 128 ? 32 : 16;               // tokens of a body tile
template <int D> constexpr int kW = D <= 128 ? 8 : D <= 256 ? 6 : 8;      // warps of a CTA
template <int D> constexpr int kSpCtas = D <= 256 ? 2 : 1;                // CTAs of an SM

// a stage's layout: K codes, V codes (1024-aligned: TMA swizzle), headers, high bits; or K and V tail rows
struct SpStage {
  int v, kd, vd, kqh, vqh, vt, bytes, stages;
  int kh, vh;  // bytes of a row's K and V headers
  uint32_t tx;
};

struct SpArgs {
  kvq_cache c;
  SpStage s;
  const void* q;
  const int32_t* sel;
  void* out;
  int q_dtype, out_dtype, n_q_heads, group, head_groups, heads_per_cta, block_tokens, n_select, rot_k, rot_v;
  int tiles, pages_per_seq;                 // tiles of a list; page table entries of a sequence
  DivU32 by_block, by_page, by_tail, by_plane;  // tiles of a block, tokens of a page, tail slots, planes of a sequence
  float scale_log2;
};

// Shared-memory loads by 32-bit address: from generic pointers into the stages the compiler
// makes generic loads with 64-bit address arithmetic.
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t r;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(r) : "r"(a));
  return r;
}
__device__ __forceinline__ void sts32(uint32_t a, uint32_t v) { asm volatile("st.shared.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory"); }
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 r;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "r"(a));
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 r;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "r"(a));
  return r;
}
// BYTES as words, in the widest loads that rows of BYTES bytes from a 16-byte aligned base allow
template <int BYTES>
__device__ __forceinline__ void lds_row(uint32_t a, uint32_t (&w)[BYTES / 4]) {
  if constexpr (BYTES % 16 == 0) {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const uint4 v = lds128(a + 16 * i);
      w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
  } else if constexpr (BYTES % 8 == 0) {
#pragma unroll
    for (int i = 0; i < BYTES / 8; ++i) {
      const uint2 v = lds64(a + 8 * i);
      w[2 * i] = v.x; w[2 * i + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < BYTES / 4; ++i) w[i] = lds32(a + 4 * i);
  }
}

// What the codes of a type are centred by; q8_0's are offset binary, centred by their conversion.
__host__ __device__ constexpr int code_centre(int qt) {
  return qt == KVQ_TYPE_Q8_0 ? 0 : type_has_qh(qt) ? 16 : 8;
}

// ldmatrix rows of a 16-row tile in W-byte box columns (R rows each): the lane's row and its
// swizzle key, and the address of 16-byte chunk j + (lane's half), j even, may be a run-time value
template <int W>
struct LdRow {
  uint32_t row, key;
  __device__ explicit LdRow(uint32_t base, int lane) {
    const int r = (lane & 7) + 8 * ((lane >> 3) & 1);
    const int k = W == 128 ? (r & 7) : W == 64 ? ((r >> 1) & 3) : ((r >> 2) & 1);
    row = base + r * W;
    key = uint32_t((k ^ (lane >> 4)) << 4);
  }
  template <int R>
  __device__ uint32_t at(int j) const {
    return row + (uint32_t((j % (W / 16)) << 4) ^ key) + (j / (W / 16)) * (R * W);
  }
};

// D = A (16x8, row) * B (8x8, col) + C in tf32: 11 bits of an fp32 operand, its whole range
__device__ __forceinline__ void mma1688_tf32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                             uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Scores of a body tile (st, qf, qsum: shared addresses of its stage, the query fragments and block sums): S[hh][t][e] of tokens 16hh + 8t + 2tig + e and head g.
template <int D, int KT>
__device__ __forceinline__ void body_scores(uint32_t st, const SpStage& L, uint32_t qf, uint32_t qsum, int lane,
                                            float (&S)[kRows<D> / 16][2][2]) {
  constexpr int NB = D / 32, RB = kRows<D>, HB = RB / 16, ROW = KT == KVQ_TYPE_Q8_0 ? D : D / 2, W = box_w(ROW);
  constexpr bool K1 = type_has_min(KT), K5 = type_has_qh(KT);
  constexpr int KHH = K1 ? 2 : 1, HP = NB * 2 * KHH;  // halves of a block header, bytes of a row's
  const int g = lane >> 2, tig = lane & 3;
  const LdRow<W> ld(st, lane);
  constexpr uint32_t OFF = (0x6400u + uint32_t(code_centre(KT))) * 0x10001u, OFF16 = neg_off_x16_bits(code_centre(KT));
  const uint32_t k0 = uint32_t(8 * (tig >> 1) + 2 * (tig & 1) - 4) & 31u, k1 = (k0 + 1) & 31u;
  const uint32_t hd0 = st + L.kd + 2 * tig * HP, qh0 = st + L.kqh + g * NB * 4, qf0 = qf + lane * 16, qs0 = qsum + g * 4;
  // Two blocks at a time.  Large heads keep the loop rolled: a call lasts a few tiles per warp, and
  // straight-line code of 8 or 10 blocks is fetched once for each of them.
  constexpr int kUnroll = D <= 128 ? NB / 2 : 1;
#pragma unroll kUnroll
  for (int bp = 0; bp < NB; bp += 2) {
    uint32_t r[HB][KT == KVQ_TYPE_Q8_0 ? 2 : 1][4], hd[HB][4][KHH];
#pragma unroll
    for (int hh = 0; hh < HB; ++hh) {
      if constexpr (KT == KVQ_TYPE_Q8_0) {
#pragma unroll
        for (int e = 0; e < 2; ++e)
          ldsm_x4(ld.template at<RB>(2 * (bp + e)) + hh * 16 * W, r[hh][e][0], r[hh][e][1], r[hh][e][2], r[hh][e][3]);
      } else {
        ldsm_x4(ld.template at<RB>(bp) + hh * 16 * W, r[hh][0][0], r[hh][0][1], r[hh][0][2], r[hh][0][3]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)  // headers of tokens 16hh + 2tig, + 1, + 8, + 9
        lds_row<4 * KHH>(hd0 + (16 * hh + (i & 1) + 8 * (i >> 1)) * HP + bp * 2 * KHH, hd[hh][i]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int blk = bp + e;
      const uint4 qa = lds128(qf0 + blk * 1024), qb = lds128(qf0 + blk * 1024 + 512);
      const uint32_t a0[4] = {qa.x, qa.y, qa.z, qa.w}, a1[4] = {qb.x, qb.y, qb.z, qb.w};
      const float qs = K1 ? __uint_as_float(lds32(qs0 + blk * (kMaxHeads * 4))) : 0.0f;
#pragma unroll
      for (int hh = 0; hh < HB; ++hh) {
        uint32_t b[2][4];  // operands of the two k-steps for the 8-token tiles of half hh
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if constexpr (KT == KVQ_TYPE_Q8_0) {  // r[t]: channels 4tig .. of the first half block, r[2 + t] of the second
            b[t][0] = i8_pair<0, 2>(r[hh][e][t]);
            b[t][1] = i8_pair<1, 3>(r[hh][e][t]);
            b[t][2] = i8_pair<0, 2>(r[hh][e][2 + t]);
            b[t][3] = i8_pair<1, 3>(r[hh][e][2 + t]);
          } else {
            const uint32_t w = r[hh][0][2 * e + t], w8 = w >> 8;
            uint32_t m0 = 0x64006400u, m1 = m0, m2 = m0, m3 = m0;
            if constexpr (K5) {  // rotated: the pairs' bits at 4 / 20 (low nibbles) and 8 / 24
              const uint32_t h = lds32(qh0 + ((16 * hh + 8 * t) * NB + blk) * 4);
              const uint32_t h0 = __funnelshift_r(h, h, k0), h1 = __funnelshift_r(h, h, k1);
              m0 = khb(h0, 0x00100010u); m1 = khb(h1, 0x00100010u);
              m2 = khb(h0, 0x01000100u); m3 = khb(h1, 0x01000100u);
            }
            b[t][0] = nib_pair(w, 0, m0, OFF);
            b[t][1] = nib_pair(w8, 0, m1, OFF);
            b[t][2] = nib_pair_x16(w, m2, OFF16);
            b[t][3] = nib_pair_x16(w8, m3, OFF16);
          }
        }
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          float cc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma16816(cc, a0, b[t][0], b[t][1]);
          mma16816(cc, a1, b[t][2], b[t][3]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t (&w)[KHH] = hd[hh][2 * t + i];
            const float dk = KHH == 1 ? h2f(w[0], e) : h2f(w[e % KHH], 0);
            S[hh][t][i] = fmaf(dk, cc[i] + cc[2 + i], S[hh][t][i]);
            if constexpr (K1) S[hh][t][i] = fmaf(fmaf(dk, float(code_centre(KT)), h2f(w[e % KHH], 1)), qs, S[hh][t][i]);
          }
        }
      }
    }
  }
}

// x as tf32 parts: its upper 11 bits, and what they leave
__device__ __forceinline__ void split_tf32(float x, uint32_t& hi, uint32_t& lo) {
  hi = __float_as_uint(x) & 0xFFFFE000u;
  lo = __float_as_uint(x - __uint_as_float(hi));
}

// bytes I0, I1 of offset-binary codes as the fp16 pair code / 16 (exact: 1152 / 16 = 72)
template <int I0, int I1>
__device__ __forceinline__ uint32_t i8_sixteenth(uint32_t r) {
  return hfma2_bits(__byte_perm(r, 0x64646464u, I0 | (4 << 4) | (I1 << 8) | (4 << 12)), 0x2C002C00u, 0xD480D480u);
}

// acc += codes_V^T . (P * scale) of the 16 body rows from row0: rows 2g (acc .. [0], [1]) and 2g + 1 of each
// 16 channels, columns heads 2tig, 2tig + 1; dmin += the blocks' minima . P (rows blocks g, g + 8; see below).
// cnt: the tile's tokens; ph, pl: P for scales in units of `unit`; p, times ps: P of tokens 8t + 2tig + e.
template <int D, int VT>
__device__ __forceinline__ void body_values(uint32_t st, const SpStage& L, int row0, const uint32_t (&ph)[2],
                                            const uint32_t (&pl)[2], const float (&p)[2][2], float ps, float unit,
                                            int cnt, int lane, float (&acc)[D / 32][2][4], float (&dmin)[4]) {
  constexpr int NB = D / 32, RB = kRows<D>, ROW = VT == KVQ_TYPE_Q8_0 ? D : D / 2, W = box_w(ROW);
  constexpr bool V1 = type_has_min(VT), V5 = type_has_qh(VT);
  constexpr int VHH = V1 ? 2 : 1;
  constexpr int HP = NB * 2 * VHH;
  const int g = lane >> 2, tig = lane & 3;
  const LdRow<W> ld(st + L.v + row0 * W, lane);
  const uint32_t vd = st + L.vd + (row0 + 2 * tig) * HP;
  auto ok = [&](int i) { return row0 + (i & 1) + 8 * (i >> 1) < cnt - 2 * tig; };  // token i of the lane's four is one
  const bool partial = cnt < RB;
  // headers of the lane's four tokens for blocks bp, bp + 1; rows past the end hold anything: theirs become zero
  auto headers = [&](int bp, uint32_t (&w)[4][VHH]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) lds_row<4 * VHH>(vd + ((i & 1) + 8 * (i >> 1)) * HP + bp * 2 * VHH, w[i]);
    if (partial) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < VHH; ++j) w[i][j] = ok(i) ? w[i][j] : 0u;
    }
  };
  auto block = [&](int blk, const uint32_t (&w)[4][VHH], const uint32_t (&a0)[4], const uint32_t (&a1)[4]) {
    const int e = blk & 1;
    const uint32_t d0 = VHH == 1 ? __byte_perm(w[0][0], w[1][0], e ? 0x7632 : 0x5410) : __byte_perm(w[0][e % VHH], w[1][e % VHH], 0x5410);
    const uint32_t d1 = VHH == 1 ? __byte_perm(w[2][0], w[3][0], e ? 0x7632 : 0x5410) : __byte_perm(w[2][e % VHH], w[3][e % VHH], 0x5410);
    uint32_t h0, l0, h1, l1;
    hscale_split(ph[0], pl[0], d0, h0, l0);
    hscale_split(ph[1], pl[1], d1, h1, l1);
    mma16816(acc[blk][0], a0, h0, h1);
    mma16816(acc[blk][0], a0, l0, l1);
    mma16816(acc[blk][1], a1, h0, h1);
    mma16816(acc[blk][1], a1, l0, l1);
  };
  if constexpr (V1) {
    // minimum + centre * scale of block blk at token i of the lane's four, in fp32 (fp16 may overflow), as tf32 high and
    // low parts.  Up to 8 blocks their low parts take the rows g + 8; the merge adds them.  16 x 8 rows of 2048 tokens,
    // head_dim 128, q4_1: 29.6 us, 28.8 with the sum in fp16.
    const float centre = float(code_centre(VT)) * unit;
    auto minimum = [&](int blk, int i, uint32_t& hi, uint32_t& lo) {
      uint32_t w = lds32(vd + ((i & 1) + 8 * (i >> 1)) * HP + (NB % 8 == 0 || blk < NB ? blk : NB - 1) * 4);
      if (partial) w = ok(i) ? w : 0u;
      const float2 f = __half22float2(u32_as_h2(w));
      split_tf32(fmaf(f.x, centre, f.y), hi, lo);
    };
#pragma unroll
    for (int t = 0; t < 2; ++t) {  // tokens 8t + 2tig, + 1 as inner indices tig, tig + 4
      uint32_t a[4], c[4], bh[2], bl[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if constexpr (NB <= 8) {
          minimum(g, 2 * t + e, a[2 * e], a[2 * e + 1]);
        } else {
          minimum(g, 2 * t + e, a[2 * e], c[2 * e]);
          minimum(g + 8, 2 * t + e, a[2 * e + 1], c[2 * e + 1]);
        }
        split_tf32(p[t][e] * ps, bh[e], bl[e]);
      }
      mma1688_tf32(dmin, a[0], a[1], a[2], a[3], bh[0], bh[1]);
      mma1688_tf32(dmin, a[0], a[1], a[2], a[3], bl[0], bl[1]);
      if constexpr (NB > 8) mma1688_tf32(dmin, c[0], c[1], c[2], c[3], bh[0], bh[1]);
    }
  }
  constexpr uint32_t OFF = (0x6400u + uint32_t(code_centre(VT))) * 0x10001u, OFF16 = neg_off_x16_bits(code_centre(VT));
  const uint32_t v0 = uint32_t(8 * ((g & 3) >> 1) + 2 * (g & 1) - 4) & 31u, v1 = (v0 + 1) & 31u;
  const uint32_t qh0 = st + L.vqh + (tig * NB * 2 + (g >> 2)) * 4 + row0 * NB * 4;
#pragma unroll
  for (int bp = 0; bp < NB; bp += 2) {
    uint32_t w[4][VHH];
    headers(bp, w);
    if constexpr (VT == KVQ_TYPE_Q8_0) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint32_t r0, r1, r2, r3;
        ldsm_x4_t(ld.template at<RB>(2 * (bp + e)), r0, r1, r2, r3);
        const uint32_t a0[4] = {i8_sixteenth<0, 2>(r0), i8_sixteenth<1, 3>(r0), i8_sixteenth<0, 2>(r1), i8_sixteenth<1, 3>(r1)};
        const uint32_t a1[4] = {i8_sixteenth<0, 2>(r2), i8_sixteenth<1, 3>(r2), i8_sixteenth<0, 2>(r3), i8_sixteenth<1, 3>(r3)};
        block(bp + e, w, a0, a1);
      }
    } else {
      uint32_t r[4];
      ldsm_x4_t(ld.template at<RB>(bp), r[0], r[1], r[2], r[3]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int blk = bp + e;
        uint32_t a0[4], a1[4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {  // tokens 0-7, 8-15
          const uint32_t c = r[2 * e + t], c8 = c >> 8;
          uint32_t m0 = 0x64006400u, m1 = m0, m2 = m0, m3 = m0;
          if constexpr (V5) {  // the lane's part word of rows 8t + 2tig, + 1
            const uint32_t h = lds32(qh0 + (4 * t * NB + blk) * 8);
            const uint32_t h0 = __funnelshift_r(h, h, v0), h1 = __funnelshift_r(h, h, v1);
            m0 = vhb(h0, 0x00100010u); m1 = vhb(h1, 0x00100010u);
            m2 = vhb(h0, 0x01000100u); m3 = vhb(h1, 0x01000100u);
          }
          a0[2 * t] = nib_pair(c, 0, m0, OFF);
          a0[2 * t + 1] = nib_pair(c8, 0, m1, OFF);
          a1[2 * t] = nib_pair_x16(c, m2, OFF16);
          a1[2 * t + 1] = nib_pair_x16(c8, m3, OFF16);
        }
        block(blk, w, a0, a1);
      }
    }
  }
}

// Tail rows go into the mma as they are stored, exact at every size: keys in tf32 (fp16's 11 bits of a query
// part and bf16's 8 fit its significand), values in bf16, the weights as three bf16 parts (24 bits).
__device__ __forceinline__ void mma16816_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                              uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// a, b less their rounding to bf16, which is returned
__device__ __forceinline__ uint32_t take_bf2(float& a, float& b) {
  const uint32_t r = pack_bf2(a, b);
  a -= __uint_as_float(r << 16);
  b -= __uint_as_float(r & 0xFFFF0000u);
  return r;
}
// the halves of an fp16 pair as fp32 bits
__device__ __forceinline__ uint32_t h_lo_f32(uint32_t h) { return __float_as_uint(__low2float(u32_as_h2(h))); }
__device__ __forceinline__ uint32_t h_hi_f32(uint32_t h) { return __float_as_uint(__high2float(u32_as_h2(h))); }

template <int D>
__global__ void __launch_bounds__(32 * kW<D>, kSpCtas<D>)
sparse_kernel(SpArgs a, const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
              const __grid_constant__ CUtensorMap tmKt, const __grid_constant__ CUtensorMap tmVt) {
  constexpr int NB = D / 32, RB = kRows<D>, HB = RB / 16, G = (D & (D - 1)) == 0 ? D : 64;
  constexpr int WT = 128, kWarps = kW<D>;  // (tail rows of 2 D bytes are whole 128-byte columns)
  static_assert(box_w(2 * D) == WT && kTailRows == 8, "tail rows' swizzle");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  pdl_begin();
  const kvq_cache& c = a.c;
  const int S = int(cg::this_cluster().num_blocks()), rank = int(cg::this_cluster().block_rank());
  const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int g = lane >> 2, tig = lane & 3;
  const int row = (blockIdx.x - rank) / S, b = int(div_u32(uint32_t(row), a.by_plane));
  const int plane = row - b * c.n_kv_heads * a.head_groups, kvh = plane / a.head_groups, hg = plane % a.head_groups;
  const int head0 = kvh * a.group + hg * a.heads_per_cta, nheads = min(a.heads_per_cta, a.group - hg * a.heads_per_cta);
  const int T = c.tail_len, NS = a.s.stages;
  // shared memory: stages [kWarps][NS] (the partials of the merge afterwards), query fragments,
  // block sums of the query, partial (m, l), score factors, barriers, jobs
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* wst = smem + warp * NS * a.s.bytes;
  uint8_t* sp = smem + kWarps * NS * a.s.bytes;
  float* sq = reinterpret_cast<float*>(sp);                             // [8][D], then the fragments
  uint4* qf = reinterpret_cast<uint4*>(sp);
  sp += 32 * D;
  float* qsum = reinterpret_cast<float*>(sp);                           // [NB][8]
  float* s_m = qsum + NB * kMaxHeads;                                   // [kWarps][8]
  float* s_l = s_m + kWarps * kMaxHeads;
  float* s_f = s_l + kWarps * kMaxHeads;                                // [8]
  uint64_t* bars = reinterpret_cast<uint64_t*>(s_f + kMaxHeads);        // [kWarps][kMaxStages]
  int2* jobs = reinterpret_cast<int2*>(bars + kWarps * kMaxStages);     // [kWarps][kMaxStages]

  const int n = min(max(c.seq_len[b], 0), c.max_ctx);
  const long long bh = (long long)b * c.n_kv_heads + kvh;
  const int32_t* sel = a.sel + bh * a.n_select;
  uint64_t* wbar = bars + warp * kMaxStages;
  int2* wjob = jobs + warp * kMaxStages;
  if (lane == 0) {
    for (int i = 0; i < NS; ++i) mbar_init(&wbar[i], 1);
    fence_barrier_init();
    if (warp == 0) {
      prefetch_tmap(&tmK); prefetch_tmap(&tmV);
      if (T > 0) { prefetch_tmap(&tmKt); prefetch_tmap(&tmVt); }
    }
  }
  __syncwarp();

  // ---- producer: the warp's tiles, in order.  Tile ordinal k is tile wid + k * nw of the list;
  // lane l holds ordinal 32 * (chunk) + l: its first position (-1: not listed) and body row
  const int body_end = n - T, wid = rank * kWarps + warp, nw = S * kWarps;
  auto slot_of = [&](int p) { return p - int(div_u32(uint32_t(p), a.by_tail)) * T; };
  int chunk = 0;           // ordinal of lane 0's tile
  int my_t0 = -1, my_row = 0;
  auto fetch = [&]() {
    const uint32_t u = uint32_t(wid) + uint32_t(chunk + lane) * uint32_t(nw);  // (below 2^32: see the launch)
    my_t0 = -1;
    if (u < uint32_t(a.tiles)) {
      const uint32_t e = div_u32(u, a.by_block);
      const int blk = sel[e];
      if (blk >= 0 && (long long)blk * a.block_tokens < n) {
        const int t0 = blk * a.block_tokens + int(u - e * a.by_block.d) * RB;
        if (t0 < n) {
          my_t0 = t0;
          my_row = 0;
          if (!c.page_tokens) {
            my_row = int(bh) * c.max_ctx + t0;
          } else if (t0 < body_end) {  // (rows of a tile lie in one page)
            const int i = int(div_u32(uint32_t(t0), a.by_page));
            const int pg = c.page_table[(long long)b * a.pages_per_seq + i];
            my_row = pg >= 0 && pg < c.n_pages ? (pg * c.n_kv_heads + kvh) * c.page_tokens + t0 - i * c.page_tokens : -1;
            if (my_row < 0) atomicOr(c.status, KVQ_DEV_ERR_PAGE);
          }
        }
      }
    }
  };
  fetch();
  unsigned live = __ballot_sync(0xffffffffu, my_t0 >= 0);  // the chunk's tiles still to come
  int pos = -1;            // next position of the tile in hand (-1: none)
  int end = 0, trow = 0;   // its end and body row
  bool done = false;
  // the next job: y > 0 body rows, y < 0 tail rows from slot x, 0 none left; copies issued by one lane
  auto produce = [&](int s) {
    while (pos < 0 && !done) {
      if (!live) {
        chunk += 32;
        done = wid + chunk * nw >= a.tiles;
        if (!done) {
          fetch();
          live = __ballot_sync(0xffffffffu, my_t0 >= 0);
        }
        continue;
      }
      const int src = __ffs(live) - 1;
      live &= live - 1;
      pos = __shfl_sync(0xffffffffu, my_t0, src);
      trow = __shfl_sync(0xffffffffu, my_row, src);
      end = min(n, pos + RB);
      if (trow < 0 && pos < body_end) {  // a page outside the pool: its body rows are left out
        pos = min(end, body_end);
        if (pos >= end) pos = -1;
      }
    }
    int2 job = make_int2(0, 0);
    if (!done) {
      if (pos < body_end) {
        job = make_int2(pos, min(end, body_end) - pos);
      } else {
        job = make_int2(slot_of(pos), -min(kTailRows, end - pos));
        job.y = max(job.y, job.x - T);  // (a tail tile ends where the ring wraps)
      }
    }
    if (lane == 0) {
      wjob[s] = job;
      uint8_t* st = wst + s * a.s.bytes;
      if (job.y > 0) {
        const size_t r = size_t(trow);
        mbar_arrive_expect_tx(&wbar[s], a.s.tx);
        tma_3d_g2s(st, &tmK, trow, &wbar[s]);
        tma_3d_g2s(st + a.s.v, &tmV, trow, &wbar[s]);
        bulk_g2s(st + a.s.kd, static_cast<const uint8_t*>(c.k_d) + r * a.s.kh, RB * a.s.kh, &wbar[s]);
        bulk_g2s(st + a.s.vd, static_cast<const uint8_t*>(c.v_d) + r * a.s.vh, RB * a.s.vh, &wbar[s]);
        if (c.k_qh) bulk_g2s(st + a.s.kqh, static_cast<const uint32_t*>(c.k_qh) + r * NB, RB * NB * 4, &wbar[s]);
        if (c.v_qh) bulk_g2s(st + a.s.vqh, static_cast<const uint32_t*>(c.v_qh) + r * NB, RB * NB * 4, &wbar[s]);
      } else if (job.y < 0) {
        const int r = int(bh) * T + job.x;
        mbar_arrive_expect_tx(&wbar[s], 2 * kTailRows * 2 * D);
        tma_3d_g2s(st, &tmKt, r, &wbar[s]);
        tma_3d_g2s(st + a.s.vt, &tmVt, r, &wbar[s]);
      }
    }
    if (job.y != 0) {
      pos += abs(job.y);
      if (pos >= end) pos = -1;
    }
    return job.y != 0;
  };
  int issued = 0;
  for (int i = 0; i < NS; ++i) issued += produce(i) ? 1 : 0;

  // ---- queries: rotate, scale, fragments (a warp per head)
  for (int hh = warp; hh < kMaxHeads; hh += kWarps) {
    float v[NB];
    load_q_fwht<D, G>(a.q, a.q_dtype, (size_t)b * a.n_q_heads + head0 + hh, hh < nheads, lane, v);
    if (a.rot_k) warp_fwht<D, G>(v, lane);
    const float sc = a.scale_log2 * (a.rot_k ? inv_sqrt_group<G>() : 1.0f);
    float mx = 0.0f;
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      v[j] *= sc;
      mx = fmaxf(mx, fabsf(v[j]));
    }
    mx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
    // a power of two that brings the largest value into [2^10, 2^11)
    const int e = min(137 - int(__float_as_uint(mx) >> 23), 126);
    const float up = __uint_as_float(uint32_t(127 + e) << 23);
#pragma unroll
    for (int j = 0; j < NB; ++j) sq[hh * D + fwht_channel<D, G>(lane, j)] = v[j] * up;
    if (lane == 0) s_f[hh] = __uint_as_float(uint32_t(127 - e) << 23);
  }
  __syncthreads();
  {
    constexpr int BPW = (NB + kWarps - 1) / kWarps;
    uint4 fb[BPW][2];
    float qs[BPW];
#pragma unroll
    for (int u = 0; u < BPW; ++u) {
      const int blk = warp + kWarps * u;
      qs[u] = 0.0f;
      if (blk < NB) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const float4 x = *reinterpret_cast<const float4*>(sq + g * D + 32 * blk + 16 * hf + 4 * tig);
          qs[u] += (x.x + x.y) + (x.z + x.w);
          uint4 f;
          split_h2(x.x, x.z, f.x, f.y);  // channels 4tig, 4tig + 2: high parts (row g), low parts (row g + 8)
          split_h2(x.y, x.w, f.z, f.w);
          fb[u][hf] = f;
        }
        qs[u] += __shfl_xor_sync(0xffffffffu, qs[u], 1);
        qs[u] += __shfl_xor_sync(0xffffffffu, qs[u], 2);
      }
    }
    __syncthreads();  // every warp has read the staged queries
#pragma unroll
    for (int u = 0; u < BPW; ++u) {
      const int blk = warp + kWarps * u;
      if (blk < NB) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) qf[(blk * 2 + hf) * 32 + lane] = fb[u][hf];
        if (tig == 0) qsum[blk * kMaxHeads + g] = qs[u];
      }
    }
  }
  __syncthreads();
  const float f = s_f[g];

  // ---- main loop
  const uint32_t wst_s = smem_u32(wst), qf_s = smem_u32(qf), qsum_s = smem_u32(qsum);
  float acc[NB][2][4];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[i][j][r] = 0.0f;
  float dmin[4] = {0.f, 0.f, 0.f, 0.f};
  float lim = -INFINITY, l = 0.0f;
  const int cs = c.v_type == KVQ_TYPE_Q8_0 ? 4 : 0;  // what of top the codes take
  int top = kTopMax;
  const uint32_t hmask = type_has_min(c.v_type) ? 0x00007FFFu : 0x7FFF7FFFu;
  bool timed_out = false;
  int k = 0;
  for (; k < issued; ++k) {
    const int s = k % NS;
    const bool arrived = mbar_wait_bounded(&wbar[s], (k / NS) & 1, kWaitCycles);
    if (!__all_sync(0xffffffffu, arrived)) { timed_out = true; break; }
    const int2 job = wjob[s];
    const uint32_t st = wst_s + s * a.s.bytes;
    const int cnt = abs(job.y);
    float sc[HB][2][2];
#pragma unroll
    for (int hh = 0; hh < HB; ++hh) sc[hh][0][0] = sc[hh][0][1] = sc[hh][1][0] = sc[hh][1][1] = 0.0f;
    if (job.y > 0) {
#define KVQ_SCORES(KT) \
  case KT: body_scores<D, KT>(st, a.s, qf_s, qsum_s, lane, sc); break;
      switch (c.k_type) {
        KVQ_SCORES(KVQ_TYPE_Q4_0)
        KVQ_SCORES(KVQ_TYPE_Q5_0)
        KVQ_SCORES(KVQ_TYPE_Q8_0)
        KVQ_SCORES(KVQ_TYPE_Q4_1)
        KVQ_SCORES(KVQ_TYPE_Q5_1)
      }
#undef KVQ_SCORES
    } else {
      float cc[4] = {0.f, 0.f, 0.f, 0.f};
      // token g, bytes 8tig .. of half block 0; half block j lies 32 bytes further, its 16-byte chunks swizzled
      const uint32_t k0 = st + g * WT + (((tig >> 1) ^ g) << 4) + (tig & 1) * 8;
#pragma unroll
      for (int j = 0; j < 2 * NB; ++j) {
        const uint2 x = lds64((k0 ^ ((2 * (j & 3)) << 4)) + (j >> 2) * (kTailRows * WT));
        const uint4 q = lds128(qf_s + lane * 16 + j * 512);
        // channels 4tig, 4tig + 2 as inner indices tig, tig + 4, then 4tig + 1, 4tig + 3
        mma1688_tf32(cc, h_lo_f32(q.x), h_lo_f32(q.y), h_hi_f32(q.x), h_hi_f32(q.y), x.x << 16, x.y << 16);
        mma1688_tf32(cc, h_lo_f32(q.z), h_lo_f32(q.w), h_hi_f32(q.z), h_hi_f32(q.w), x.x & 0xFFFF0000u, x.y & 0xFFFF0000u);
      }
      sc[0][0][0] = cc[0] + cc[2];
      sc[0][0][1] = cc[1] + cc[3];
    }
    // ---- online softmax (base 2) of head g; the tokens are 16hh + 8t + 2tig + e
    const bool partial = cnt < RB;
    float mx = -INFINITY;
#pragma unroll
    for (int hh = 0; hh < HB; ++hh)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) sc[hh][t][e] *= f;
    if (partial) {
#pragma unroll
      for (int i = 0; i < 4 * HB; ++i)
        if (16 * (i >> 2) + 8 * ((i >> 1) & 1) + (i & 1) >= cnt - 2 * tig) sc[i >> 2][(i >> 1) & 1][i & 1] = -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < 4 * HB; ++i) mx = fmaxf(mx, sc[i >> 2][(i >> 1) & 1][i & 1]);
    // The rescale runs only when a score passes the reference, or when the scales of a tile's tokens ask for smaller
    // weights (rows past its end hold anything).
    bool down = false;
    uint32_t mxs = 0;  // largest scales of the lane's headers, fp16 bits in each half
    if (job.y > 0) {
#pragma unroll 1  // (a warp has few tiles: code that is fetched once counts; unrolled the call takes 5% longer)
      for (int i = lane; i < cnt * a.s.vh / 4; i += 32) mxs = __vmaxu2(mxs, lds32(st + a.s.vd + 4 * i) & hmask);
      const uint32_t big = uint32_t(31 - top) << 10;  // 2^(16 - top) in fp16; infinity with top 0
      down = __any_sync(0xffffffffu, (mxs & 0xFFFFu) >= big || (mxs >> 16) >= big);
    }
    if (__any_sync(0xffffffffu, mx > lim) || down) {
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      int nt = top;
      if (down) {  // the largest scale lies in [2^(e - 15), 2^(e - 14)): half of what has room
        const int e = int(__reduce_max_sync(0xffffffffu, max(mxs & 0xFFFFu, mxs >> 16)) >> 10);
        nt = max(29 - e, 0);
        if (e >= 5) nt = min(nt, 15);
      }
      const float nl = mx > lim ? mx + kLazyMax : lim;
      float r = lim == -INFINITY ? 0.0f : fast_exp2(lim - nl);
      l *= r;
      r *= pow2(nt - top);
      lim = nl;
      top = nt;
      const float r0 = __shfl_sync(0xffffffffu, r, 8 * tig), r1 = __shfl_sync(0xffffffffu, r, 8 * tig + 4);
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) { acc[i][j][0] *= r0; acc[i][j][1] *= r1; acc[i][j][2] *= r0; acc[i][j][3] *= r1; }
      dmin[0] *= r0; dmin[1] *= r1; dmin[2] *= r0; dmin[3] *= r1;
    }
    const float ms = lim == -INFINITY ? 0.0f : lim;
    float p[HB][2][2];
#pragma unroll
    for (int hh = 0; hh < HB; ++hh)
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          p[hh][t][e] = fast_exp2(sc[hh][t][e] - ms);
          l += p[hh][t][e];
        }
    // ---- P.V
    if (job.y > 0) {
      uint32_t ph[HB][2], pl[HB][2];
      const int up = max(top - 15, 0);
      const float vs = pow2(top - up);
      if (up) {  // (other lanes' headers are read after the warp's barrier)
        const uint32_t m = uint32_t(15 + up) << 10, m2 = type_has_min(c.v_type) ? 0x3C000000u | m : m * 0x10001u;
#pragma unroll 1
        for (int i = lane; i < cnt * a.s.vh / 4; i += 32) sts32(st + a.s.vd + 4 * i, hmul2_bits(lds32(st + a.s.vd + 4 * i), m2));
        __syncwarp();
      }
#pragma unroll
      for (int hh = 0; hh < HB; ++hh)
#pragma unroll
        for (int t = 0; t < 2; ++t) split_h2(p[hh][t][0] * vs, p[hh][t][1] * vs, ph[hh][t], pl[hh][t]);
#define KVQ_VALUES(VT)                                                                                               \
  case VT:                                                                                                           \
    _Pragma("unroll") for (int hh = 0; hh < HB; ++hh) body_values<D, VT>(st, a.s, 16 * hh, ph[hh], pl[hh], p[hh], pow2(top), pow2(-up), cnt, lane, \
                                                                          acc, dmin);                                    \
    break;
      switch (c.v_type) {
        KVQ_VALUES(KVQ_TYPE_Q4_0)
        KVQ_VALUES(KVQ_TYPE_Q5_0)
        KVQ_VALUES(KVQ_TYPE_Q8_0)
        KVQ_VALUES(KVQ_TYPE_Q4_1)
        KVQ_VALUES(KVQ_TYPE_Q5_1)
      }
#undef KVQ_VALUES
    } else {
      const float ps = pow2(top - cs);
      float r0 = p[0][0][0] * ps, r1 = p[0][0][1] * ps;
      const uint32_t p1 = take_bf2(r0, r1), p2 = take_bf2(r0, r1), p3 = pack_bf2(r0, r1);
      // tokens 2tig and 2tig + 1, channels 2g, 2g + 1; 16 channels further 32 bytes, swizzled.  Rows past the
      // end hold anything: masked
      const uint32_t m0 = 2 * tig < cnt ? 0xFFFFFFFFu : 0u, m1 = 2 * tig + 1 < cnt ? 0xFFFFFFFFu : 0u;
      const uint32_t v0 = st + a.s.vt + 2 * tig * WT + (((g >> 2) ^ (2 * tig)) << 4) + (g & 3) * 4;
      const uint32_t v1 = st + a.s.vt + (2 * tig + 1) * WT + (((g >> 2) ^ (2 * tig + 1)) << 4) + (g & 3) * 4;
#pragma unroll
      for (int j = 0; j < 2 * NB; ++j) {
        const uint32_t w0 = lds32((v0 ^ ((2 * (j & 3)) << 4)) + (j >> 2) * (kTailRows * WT)) & m0;
        const uint32_t w1 = lds32((v1 ^ ((2 * (j & 3)) << 4)) + (j >> 2) * (kTailRows * WT)) & m1;
        // the eight tokens stand twice in the inner index: with the first two parts, then with the third
        const uint32_t a0 = __byte_perm(w0, w1, 0x5410), a1 = __byte_perm(w0, w1, 0x7632);
        mma16816_bf16(acc[j / 2][j % 2], a0, a1, a0, a1, p1, p2);
        mma16816_bf16(acc[j / 2][j % 2], a0, a1, 0u, 0u, p3, 0u);
      }
    }
    __syncwarp();
    if (lane == 0) fence_proxy_async_smem();
    issued += produce(s) ? 1 : 0;
    __syncwarp();
  }
  if (timed_out) {
    if (lane == 0) atomicOr(c.status, KVQ_DEV_ERR_TIMEOUT);
    for (; k < issued; ++k) mbar_wait_bounded(&wbar[k % NS], (k / NS) & 1, kWaitCycles);  // copies still in flight
  }

  // ---- merge: every warp's partial to its CTA's shared memory, then each head by one warp of the cluster
  l += __shfl_xor_sync(0xffffffffu, l, 1);
  l += __shfl_xor_sync(0xffffffffu, l, 2);
  if (tig == 0) {
    s_m[warp * kMaxHeads + g] = lim;
    s_l[warp * kMaxHeads + g] = l;
  }
  const float unscale = pow2(cs - top);
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 4; ++r) acc[i][j][r] *= unscale;
#pragma unroll
  for (int r = 0; r < 4; ++r) dmin[r] *= unscale;
  __syncthreads();  // the stages are free
  float* macc = reinterpret_cast<float*>(smem);  // [kWarps][8][D]
#pragma unroll
  for (int blk = 0; blk < NB; ++blk)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float* o = macc + (size_t)(warp * kMaxHeads + 2 * tig) * D + 32 * blk + 16 * j + 2 * g;
      *reinterpret_cast<float2*>(o) = make_float2(acc[blk][j][0], acc[blk][j][2]);
      *reinterpret_cast<float2*>(o + D) = make_float2(acc[blk][j][1], acc[blk][j][3]);
    }
  if (type_has_min(c.v_type)) {
    if constexpr (NB <= 8) {  // high and low parts
      dmin[0] += dmin[2];
      dmin[1] += dmin[3];
    }
    __syncwarp();
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int blk = g + 8 * half;
      if (blk < NB) {
        float* o = macc + (size_t)(warp * kMaxHeads + 2 * tig) * D + 32 * blk;
#pragma unroll 8
        for (int i = 0; i < 32; ++i) {
          o[i] += dmin[2 * half];
          o[D + i] += dmin[2 * half + 1];
        }
      }
    }
  }
  // the CTA's warps: every thread sums its (head, channel) elements, in the frame of the CTA's maximum
  __syncthreads();
  float* s_cta = s_f;  // [8]: the CTA's maximum per head; its sum goes to s_l[head] (the factors are done with)
  for (int i = tid; i < kMaxHeads * D / 4; i += 32 * kWarps) {
    const int hh = i / (D / 4);
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w * kMaxHeads + hh]);
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float mw = s_m[w * kMaxHeads + hh];
      const float f = mw == -INFINITY ? 0.0f : fast_exp2(mw - M);  // (a warp without tokens: zeros)
      const float4 x = reinterpret_cast<const float4*>(macc)[w * (kMaxHeads * D / 4) + i];
      v.x = fmaf(x.x, f, v.x); v.y = fmaf(x.y, f, v.y); v.z = fmaf(x.z, f, v.z); v.w = fmaf(x.w, f, v.w);
    }
    reinterpret_cast<float4*>(macc)[i] = v;  // (only this thread reads element i of warp 0's partial)
  }
  float cm = -INFINITY, csum = 0.0f;
  if (tid < kMaxHeads) {
    for (int w = 0; w < kWarps; ++w) cm = fmaxf(cm, s_m[w * kMaxHeads + tid]);
    for (int w = 0; w < kWarps; ++w) {
      const float mw = s_m[w * kMaxHeads + tid];
      if (mw != -INFINITY) csum = fmaf(s_l[w * kMaxHeads + tid], fast_exp2(mw - cm), csum);
    }
  }
  __syncthreads();
  if (tid < kMaxHeads) {
    s_cta[tid] = cm;
    s_l[tid] = csum;
  }
  // the cluster's CTAs: head hh by warp hh / S of rank hh % S
  cg::cluster_group cl = cg::this_cluster();
  cl.sync();
  for (int hh = rank + S * warp; hh < nheads; hh += S * kWarps) {
    // lane r: the maximum and sum of rank r
    const float mr = lane < S ? cl.map_shared_rank(s_cta, lane)[hh] : -INFINITY;
    const float lr = lane < S ? cl.map_shared_rank(s_l, lane)[hh] : 0.0f;
    float M = mr, x[NB];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float fr = mr == -INFINITY ? 0.0f : fast_exp2(mr - M);
    float Lsum = lr * fr;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) Lsum += __shfl_xor_sync(0xffffffffu, Lsum, o);
#pragma unroll
    for (int j = 0; j < NB; ++j) x[j] = 0.0f;
#pragma unroll 4
    for (int r = 0; r < S; ++r) {
      const float* ra = cl.map_shared_rank(macc, r) + hh * D;
      const float f = __shfl_sync(0xffffffffu, fr, r);
#pragma unroll
      for (int j = 0; j < NB; ++j) x[j] = fmaf(ra[fwht_channel<D, G>(lane, j)], f, x[j]);
    }
    const float inv = Lsum > 0.0f ? 1.0f / Lsum : 0.0f;
#pragma unroll
    for (int j = 0; j < NB; ++j) x[j] *= inv;
    if (a.rot_v) {
      warp_fwht<D, G>(x, lane);
#pragma unroll
      for (int j = 0; j < NB; ++j) x[j] *= inv_sqrt_group<G>();
    }
#pragma unroll
    for (int j = 0; j < NB; ++j) {
      const size_t o = ((size_t)b * a.n_q_heads + head0 + hh) * D + fwht_channel<D, G>(lane, j);
      if (a.out_dtype == KVQ_F32) static_cast<float*>(a.out)[o] = x[j];
      else if (a.out_dtype == KVQ_BF16) static_cast<__nv_bfloat16*>(a.out)[o] = __float2bfloat16_rn(x[j]);
      else static_cast<__half*>(a.out)[o] = __float2half_rn(x[j]);
    }
  }
  cl.sync();  // no CTA leaves while another reads its partials
}

template <int D>
cudaError_t run_sparse(SpArgs& a, cudaStream_t st) {
  constexpr int NB = D / 32, RB = kRows<D>, kWarps = kW<D>;
  const kvq_cache& c = a.c;
  const int rowK = int(qs_row_bytes_host(c.k_type, D)), rowV = int(qs_row_bytes_host(c.v_type, D));
  const int kh = NB * (type_has_min(c.k_type) ? 4 : 2), vh = NB * (type_has_min(c.v_type) ? 4 : 2);
  SpStage& s = a.s;
  s.kh = kh;
  s.vh = vh;
  s.v = align_up(RB * rowK, 1024);
  s.kd = s.v + RB * rowV;
  s.vd = s.kd + RB * kh;
  s.kqh = s.vd + RB * vh;
  s.vqh = s.kqh + (type_has_qh(c.k_type) ? RB * NB * 4 : 0);
  const int body = s.vqh + (type_has_qh(c.v_type) ? RB * NB * 4 : 0);
  s.tx = uint32_t(RB * (rowK + rowV + kh + vh) + (type_has_qh(c.k_type) ? RB * NB * 4 : 0) +
                  (type_has_qh(c.v_type) ? RB * NB * 4 : 0));
  s.vt = align_up(kTailRows * 2 * D, 1024);
  const int tail = c.tail_len > 0 ? s.vt + kTailRows * 2 * D : 0;
  s.bytes = align_up(std::max(body, tail), 1024);
  const int rest = 32 * D + (NB + 2 * kWarps + 1) * kMaxHeads * 4 + kWarps * kMaxStages * 16 + 1024;
  // as many stages as leave room for kSpCtas<D> CTAs on an SM (228 KB, 1 KB of it reserved per CTA), two at
  // least (the merge's partials, 32 * D bytes per warp, fit two stages of any pair: 2 * RB * D)
  const int room = 228 * 1024 / kSpCtas<D> - 1024 - rest;
  s.stages = std::min(kMaxStages, std::max(2, room / (kWarps * s.bytes)));
  const int bytes = kWarps * s.stages * s.bytes + rest;

  alignas(64) CUtensorMap mk, mv, mkt, mvt;
  memset(&mkt, 0, sizeof(mkt));
  memset(&mvt, 0, sizeof(mvt));
  if (!make_map(&mk, c.k_qs, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, body_rows(c), rowK, box_w(rowK), RB) ||
      !make_map(&mv, c.v_qs, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, body_rows(c), rowV, box_w(rowV), RB))
    return cudaErrorInvalidValue;
  if (c.tail_len > 0) {
    const long long trows = (long long)c.batch * c.n_kv_heads * c.tail_len;
    if (!make_map(&mkt, c.k_tail, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, trows, 2 * D, box_w(2 * D), kTailRows) ||
        !make_map(&mvt, c.v_tail, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, trows, 2 * D, box_w(2 * D), kTailRows))
      return cudaErrorInvalidValue;
  }
  auto kern = sparse_kernel<D>;
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), bytes);
  if (e != cudaSuccess) return e;
  if ((e = allow_large_clusters(reinterpret_cast<const void*>(kern))) != cudaSuccess) return e;
  // CTAs per row: as many as let all rows' clusters run at once, a tile per warp at least
  const long long rows = (long long)c.batch * c.n_kv_heads * a.head_groups;
  const long long tiles = (long long)a.n_select * (a.block_tokens / RB);
  if (tiles > 0x3fffffffLL) return cudaErrorInvalidValue;  // (the API refuses such lists)
  a.tiles = int(tiles);
  a.by_block = make_divu32(uint32_t(a.block_tokens / RB));
  a.pages_per_seq = c.page_tokens ? c.max_ctx / c.page_tokens : 0;
  a.by_page = make_divu32(uint32_t(std::max(1, c.page_tokens)));
  a.by_tail = make_divu32(uint32_t(std::max(1, c.tail_len)));
  a.by_plane = make_divu32(uint32_t(c.n_kv_heads * a.head_groups));
  const ClusterLimits* lim = cluster_limits(reinterpret_cast<const void*>(kern), 32 * kWarps, bytes);
  int S = 1;
  if (lim)
    for (int k = 2; k <= kMaxCluster && (long long)k * kWarps <= tiles; ++k)
      if (lim->clusters[k] >= rows) S = k;
  return launch_dependent(kern, unsigned(rows * S), 32 * kWarps, bytes, st, S, a, mk, mv, mkt, mvt);
}

}  // namespace

cudaError_t launch_sparse_decode(const kvq_cache& c, Rot rot, const void* q, int q_dtype, int n_q_heads, float scale,
                                 int block_tokens, const int32_t* sel, int n_select, void* out, int out_dtype,
                                 cudaStream_t st) {
  SpArgs a{};
  a.c = c; a.q = q; a.sel = sel; a.out = out;
  a.q_dtype = q_dtype; a.out_dtype = out_dtype; a.n_q_heads = n_q_heads; a.group = n_q_heads / c.n_kv_heads;
  a.head_groups = (a.group + kMaxHeads - 1) / kMaxHeads;
  a.heads_per_cta = (a.group + a.head_groups - 1) / a.head_groups;
  a.block_tokens = block_tokens; a.n_select = n_select; a.rot_k = rot.k; a.rot_v = rot.v;
  a.scale_log2 = scale * kLog2e;
  switch (c.head_dim) {
    case 64: return run_sparse<64>(a, st);
    case 128: return run_sparse<128>(a, st);
    case 192: return run_sparse<192>(a, st);
    case 256: return run_sparse<256>(a, st);
    case 320: return run_sparse<320>(a, st);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
