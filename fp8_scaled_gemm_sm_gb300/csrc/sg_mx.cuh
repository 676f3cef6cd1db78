// sg_mx.cuh -- power-of-two (e8m0) scales: the exponent rule shared by the
// quantiser and the key/value cache.
#pragma once

#include <cstdint>

namespace sg {

// Least integer e with amax <= 448 * 2^e, for finite amax > 0, by exact integer
// comparison: amax = M * 2^q, 448 = 7 * 2^6, so e = t - 6 + q with t the least
// integer such that 7 * 2^t >= M.
__device__ __forceinline__ int mx_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const uint32_t ef = (u >> 23) & 0xFFu;
  const uint64_t M = ef ? ((u & 0x7FFFFFu) | 0x800000u) : (u & 0x7FFFFFu);
  const int q = ef ? static_cast<int>(ef) - 150 : -149;
  int t = 0;
  if (M > 7) {
    // M has b bits, so 7 * 2^(b-3) < 2^b and 7 * 2^(b-2) >= 2^b > M: t is b-3 or b-2
    const int b = 32 - __clz(static_cast<uint32_t>(M));
    t = (7ull << (b - 3)) >= M ? b - 3 : b - 2;
  } else {
    while ((M << (1 - t)) <= 7) --t;
  }
  return t - 6 + q;
}

__device__ __forceinline__ float exp2_code(int code) {  // 2^(code - 127), code in [0, 254]
  return code > 0 ? __uint_as_float(static_cast<uint32_t>(code) << 23) : __uint_as_float(0x00400000u);
}

}  // namespace sg
