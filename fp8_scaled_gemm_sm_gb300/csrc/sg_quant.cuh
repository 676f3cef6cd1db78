// sg_quant.cuh -- eight activations at a time: raw vectors, e4m3 codes of
// quotients (shared by the quantiser and the norm before it).
#pragma once

#include <cstdint>
#include <cuda_fp8.h>

#include "sg_ptx.cuh"

namespace sg {

// The raw 16 (bf16) or 32 (fp32) bytes of one 8-element vector.
template <bool BF16>
struct Raw8 {
  uint4 w[BF16 ? 1 : 2];
};

template <bool BF16>
__device__ __forceinline__ void load_raw8(const void* X, int64_t elem, Raw8<BF16>& raw) {
  if constexpr (BF16) {
    raw.w[0] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(X) + elem));
  } else {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const float*>(X) + elem);
    raw.w[0] = __ldg(p);
    raw.w[1] = __ldg(p + 1);
  }
}

template <bool BF16>
__device__ __forceinline__ void unpack8(const Raw8<BF16>& raw, float (&f)[8]) {
  if constexpr (BF16) {
    const uint32_t w[4] = {raw.w[0].x, raw.w[0].y, raw.w[0].z, raw.w[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      f[4 * h + 0] = __uint_as_float(raw.w[h].x);
      f[4 * h + 1] = __uint_as_float(raw.w[h].y);
      f[4 * h + 2] = __uint_as_float(raw.w[h].z);
      f[4 * h + 3] = __uint_as_float(raw.w[h].w);
    }
  }
}

__device__ __forceinline__ uint2 cvt8(const float (&y)[8]) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t pair = __nv_cvt_float2_to_fp8x2(make_float2(y[2 * i], y[2 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    w[i >> 1] |= (pair & 0xFFFFu) << (16 * (i & 1));
  }
  return make_uint2(w[0], w[1]);
}

// Eight codes of x / s (round to nearest even, saturated), s a power of two
// whose reciprocal inv_s is representable: x * inv_s is then the same correctly
// rounded value as x / s.
__device__ __forceinline__ uint2 quant8_pow2(const float (&f)[8], float inv_s) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = f[i] * inv_s;
  return cvt8(y);
}

// The correctly rounded quotient x / s without a division, by Markstein's method
// (P. Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", IBM J. Res. Dev. 34(1), 1990): with r = RN(1/s), q = RN(x r), and
// twice q <- RN(q + (x - q s) r), each remainder x - q s exact in one fma, the
// second correction is RN(x / s) once r is correctly rounded and q within an ulp,
// barring underflow.  Here it is taken only for 2^-60 <= s <= 2^60: every quotient
// that can round to a nonzero e4m3 code (|x / s| >= 2^-11) then keeps its
// remainders normal, and smaller quotients round to +-0 either way.  A zero x
// would come out +0 from the corrections, so the sign of x is copied back (the
// quotient's sign is x's: s > 0).  Two lanes per packed fp32x2 instruction.
struct Recip {
  uint64_t r2;    // (r, r)
  uint64_t ns2;   // (-s, -s)
  bool fast;      // s in [2^-60, 2^60]
};

__device__ __forceinline__ Recip make_recip(float s, float r) {  // r = RN(1/s)
  Recip q;
  q.r2 = pack_f32x2(__float_as_uint(r), __float_as_uint(r));
  q.ns2 = pack_f32x2(__float_as_uint(-s), __float_as_uint(-s));
  q.fast = s >= 0x1p-60f && s <= 0x1p+60f;
  return q;
}

__device__ __forceinline__ Recip make_recip(float s) { return make_recip(s, __frcp_rn(s)); }

// Eight codes of x / s: the quotient correctly rounded in fp32 (the IEEE division
// where the scale is outside Markstein's range), then e4m3.
__device__ __forceinline__ uint2 quant8(const float (&f)[8], float s, const Recip& rc) {
  float y[8];
  if (rc.fast) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = __float_as_uint(f[2 * i]), b = __float_as_uint(f[2 * i + 1]);
      const uint64_t x = pack_f32x2(a, b);
      uint64_t q = mul_f32x2(x, rc.r2);
      uint64_t e = fma_f32x2(q, rc.ns2, x);
      q = fma_f32x2(e, rc.r2, q);
      e = fma_f32x2(q, rc.ns2, x);
      q = fma_f32x2(e, rc.r2, q);
      float lo, hi;
      unpack_f32x2(q, lo, hi);
      y[2 * i] = __uint_as_float((__float_as_uint(lo) & 0x7FFFFFFFu) | (a & 0x80000000u));
      y[2 * i + 1] = __uint_as_float((__float_as_uint(hi) & 0x7FFFFFFFu) | (b & 0x80000000u));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(f[i], s);
  }
  return cvt8(y);
}

}  // namespace sg
