// Stored values of the body, eight at a time.
#pragma once

#include "kvq_device.cuh"

namespace kvq {

// One side (keys or values) of the body planes.
struct BodySide {
  const uint8_t* qs;
  const uint8_t* hd;   // fp16 d per block, or (d, lo) pairs
  const uint32_t* qh;  // q5_0 / q5_1, else NULL
  int type;
  bool is_k;
};
__host__ __device__ inline BodySide body_side(const kvq_cache& c, bool k) {
  return BodySide{static_cast<const uint8_t*>(k ? c.k_qs : c.v_qs), static_cast<const uint8_t*>(k ? c.k_d : c.v_d),
                  static_cast<const uint32_t*>(k ? c.k_qh : c.v_qh), k ? c.k_type : c.v_type, k};
}

// Values of channels 8u .. 8u + 7 and, 16 further, of the same 8 bytes of a 4-bit block's codes (u 0 or 1 within block blk), in
// fp32: (code - offset) * d is exact, the minimum's sum rounded once.
__device__ __forceinline__ void body_values16(const BodySide& s, int head_dim, long long row, int blk, int u, float (&x)[2][8]) {
  const int nb = head_dim / 32;
  const bool has_min = type_has_min(s.type);
  const uint8_t* h = s.hd + (size_t(row) * nb + blk) * (has_min ? 4 : 2);
  const uint32_t hdr = has_min ? *reinterpret_cast<const uint32_t*>(h) : uint32_t(*reinterpret_cast<const uint16_t*>(h));
  const float d = __half2float(__ushort_as_half(uint16_t(hdr & 0xFFFFu)));
  if (s.type == KVQ_TYPE_Q8_0) {
    const uint2* src = reinterpret_cast<const uint2*>(s.qs + size_t(row) * head_dim + blk * 32 + u * 8);
    const uint2 q[2] = {src[0], src[2]};
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) x[k][e] = float(int(((e < 4 ? q[k].x : q[k].y) >> (8 * (e & 3))) & 0xFFu) - 128) * d;  // offset binary
    return;
  }
  const float lo = has_min ? __half2float(__ushort_as_half(uint16_t(hdr >> 16))) : 0.0f;
  const uint2 q = *reinterpret_cast<const uint2*>(s.qs + size_t(row) * (head_dim / 2) + blk * 16 + u * 8);
  const uint32_t high = type_has_qh(s.type) ? qh_get(s.qh, s.is_k, size_t(row), nb, blk) >> (u * 8) : 0u;
  const int off = type_code_offset(s.type);
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t byte = (e < 4 ? q.x : q.y) >> (8 * (e & 3));
      const int code = int((byte >> (4 * k)) & 15u) | int(((high >> (16 * k + e)) & 1u) << 4);
      const float v = __fmul_rn(float(code - off), d);
      x[k][e] = has_min ? __fadd_rn(v, lo) : v;
    }
}

}  // namespace kvq
