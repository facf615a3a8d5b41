#pragma once

#include <stdint.h>

namespace kvq {

// Unsigned 32-bit division by a run-time invariant divisor d >= 1 with one
// high multiply (Granlund and Montgomery, "Division by invariant integers
// using multiplication", 1994, section 4): l = ceil(log2 d),
// m = floor(2^32 (2^l - d) / d) + 1, q = (t + ((n - t) >> min(l, 1))) >>
// max(l - 1, 0) with t = mulhi(m, n); exact for every 32-bit n.
struct DivU32 {
  uint32_t d, m, s1, s2;
};
inline DivU32 make_divu32(uint32_t d) {
  uint32_t l = 0;
  while (l < 32 && (uint64_t(1) << l) < d) ++l;
  const uint32_t m = uint32_t(((uint64_t(1) << 32) * ((uint64_t(1) << l) - d)) / d + 1);
  return DivU32{d, m, l < 1 ? l : 1u, l > 1 ? l - 1 : 0u};
}
#ifdef __CUDACC__
__device__ __forceinline__ uint32_t div_u32(uint32_t n, const DivU32& v) {
  const uint32_t t = __umulhi(v.m, n);
  return (t + ((n - t) >> v.s1)) >> v.s2;
}
#endif

}  // namespace kvq
