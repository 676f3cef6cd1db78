// sg_norm.cu -- a residual's addition, root-mean-square norm and quantisation in one
// pass (scaled_gemm_norm_quantize).
//
// For a row of C elements, t the type of x:
//     r = t(x + residual)                      kept: the residual stream
//     y = (r * g) * w,   g = 1 / sqrt(sum r^2 / C + eps)
// and y is quantised in fp32 as sg_quant.cu does, without a rounding to t in between.
// The norm is that of r as it is kept, so it can be formed again from what is kept.
//
// g is the fp32 nearest to its value but for about one row in 2^16: squares are added up with their
// rounding errors (D. E. Knuth's two-sum and T. J. Dekker's representation as a sum of two), and the root is corrected by one
// step of Newton's iteration on such pairs.  So g, every y (two fp32 products) and every
// scale and code after it do not depend on the order of the sum: an e8m0 scale goes
// by which side of a power of two a block's largest value lies, where any difference would show.
// It costs 3.5 instructions an element (5.5 for fp32 rows, whose squares are not exact in 24 bits).
//
// The bound is memory: x and the residual are read once, the sum is written once and the
// codes once; the row stays in registers in between.  A CTA a row, rows dealt out in turn;
// the next row's vectors are already loading while this one is summed up.
#include <cuda.h>
#include <cuda_runtime.h>

#include "sg_common.cuh"
#include "sg_internal.h"
#include "sg_mx.cuh"
#include "sg_quant.cuh"

namespace sg {

namespace {

constexpr int kMaxWarps = 32;
constexpr float kFar = 0x1p90f;     // row sums of squares past this are formed again from
constexpr float kDown = 0x1p-80f;   // elements scaled by this

struct NormParams {
  const void *x, *residual, *weight;
  void *residual_out, *out, *scale;
  int R, C;
  float eps_hi, eps_lo;  // eps as a sum of two
};

// A number as the sum of two, the second small beside the first.
struct Pair {
  float hi, lo;
};

__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = __fadd_rn(a, b), bb = __fsub_rn(s, a);
  return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, bb)), __fsub_rn(b, bb))};
}

__device__ __forceinline__ Pair add(const Pair& a, const Pair& b) {
  const Pair s = two_sum(a.hi, b.hi);
  return {s.hi, __fadd_rn(__fadd_rn(a.lo, b.lo), s.lo)};
}

// 1 / sqrt(sum / C + eps).
__device__ __forceinline__ float inverse_root(const Pair& sum, float C, float eps_hi, float eps_lo) {
  const float q = __fdiv_rn(sum.hi, C);
  const float q_lo = __fdiv_rn(__fadd_rn(__fmaf_rn(-q, C, sum.hi), sum.lo), C);
  const Pair v = two_sum(q, eps_hi);
  const float lo = __fadd_rn(__fadd_rn(v.lo, q_lo), eps_lo);
  const float h = __fadd_rn(v.hi, lo), l = __fsub_rn(lo, __fsub_rn(h, v.hi));
  // y + y (1 - v y^2) / 2, v y^2 with its rounding errors
  const float y = rsqrtf(h);
  const float t = __fmul_rn(y, y), t_lo = __fmaf_rn(y, y, -t);
  const float p = __fmul_rn(h, t), p_lo = __fmaf_rn(h, t, -p) + __fmaf_rn(h, t_lo, __fmul_rn(l, t));
  return __fmaf_rn(0.5f * y, __fsub_rn(__fsub_rn(1.f, p), p_lo), y);
}

__device__ __forceinline__ uint64_t pair_of(float a, float b) { return pack_f32x2(__float_as_uint(a), __float_as_uint(b)); }

template <bool BF16>
__device__ __forceinline__ void load_vec(const void* X, int64_t elem, Raw8<BF16>& raw) {
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(X) + elem * (BF16 ? 2 : 4));
#pragma unroll
  for (int i = 0; i < (BF16 ? 1 : 2); ++i) raw.w[i] = p[i];
}

// VPT: vectors of eight elements a thread; MOST: threads at most.
template <int MODE, bool BF16, int VPT, int MOST>
__global__ void __launch_bounds__(MOST) norm_kernel(const NormParams p) {
  __shared__ Pair red_sum[2][kMaxWarps];
  __shared__ float red_max[2][kMaxWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, T = blockDim.x, warps = T >> 5;
  const int nvec = p.C / 8;
  // Vector i of this thread: as in the quantiser, so that a block's vectors lie in consecutive lanes.
  constexpr int kVB = MODE == kModeBlockscale ? (VPT < 4 ? VPT : 4) : 1;
  auto vidx = [&](int i) { return (i / kVB) * (T * kVB) + tid * kVB + (i % kVB); };
  constexpr bool kAhead = VPT == 1;  // the next row's vectors load while this one is worked on, where they take few registers
  auto fetch = [&](Raw8<BF16>(&x)[VPT], Raw8<BF16>(&r)[VPT], int row) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = vidx(i);
      if (v >= nvec || row >= p.R) continue;
      const int64_t at = static_cast<int64_t>(row) * p.C + 8 * static_cast<int64_t>(v);
      load_vec<BF16>(p.x, at, x[i]);
      if (p.residual) load_vec<BF16>(p.residual, at, r[i]);
    }
  };
  grid_dep_launch();
  grid_dep_wait();
  Raw8<BF16> next_x[VPT], next_r[VPT];
  if constexpr (kAhead) fetch(next_x, next_r, blockIdx.x);
  int turn = 0;
  for (int r = blockIdx.x; r < p.R; r += gridDim.x, turn ^= 1) {
    const int64_t row = static_cast<int64_t>(r) * p.C;
    float f[VPT][8];
    if constexpr (!kAhead) fetch(next_x, next_r, r);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = vidx(i);
      if (v >= nvec) {  // past the row: zeros
#pragma unroll
        for (int e = 0; e < 8; ++e) f[i][e] = 0.f;
        continue;
      }
      unpack8<BF16>(next_x[i], f[i]);
      if (!p.residual) continue;
      float g[8];
      unpack8<BF16>(next_r[i], g);
      const int64_t at = row + 8 * static_cast<int64_t>(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[i][e] = __fadd_rn(f[i][e], g[e]);
      if constexpr (BF16) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          w[e] = pack_bf16x2(f[i][2 * e], f[i][2 * e + 1]);
          f[i][2 * e] = __uint_as_float(w[e] << 16);
          f[i][2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.residual_out) + at) = make_uint4(w[0], w[1], w[2], w[3]);
      } else {
        float4* to = reinterpret_cast<float4*>(static_cast<float*>(p.residual_out) + at);
        to[0] = make_float4(f[i][0], f[i][1], f[i][2], f[i][3]);
        to[1] = make_float4(f[i][4], f[i][5], f[i][6], f[i][7]);
      }
    }
    if constexpr (kAhead) fetch(next_x, next_r, r + gridDim.x);

    // the sum of squares, of elements scaled by `by`
    auto square_sum = [&](float by, int slot) {
      const uint64_t minus = pair_of(-1.f, -1.f), by2 = pair_of(by, by);
      uint64_t s = 0, e = 0;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          uint64_t v = pair_of(f[i][2 * k], f[i][2 * k + 1]);
          if (by != 1.f) v = mul_f32x2(v, by2);
          const uint64_t q = mul_f32x2(v, v);
          if constexpr (!BF16) e = add_f32x2(e, fma_f32x2(v, v, mul_f32x2(q, minus)));
          const uint64_t t = add_f32x2(s, q), b = fma_f32x2(s, minus, t);
          e = add_f32x2(e, add_f32x2(fma_f32x2(fma_f32x2(b, minus, t), minus, s), fma_f32x2(b, minus, q)));
          s = t;
        }
      float s0, s1, e0, e1;
      unpack_f32x2(s, s0, s1);
      unpack_f32x2(e, e0, e1);
      Pair sum = add(Pair{s0, e0}, Pair{s1, e1});
#pragma unroll
      for (int o = 1; o < 32; o <<= 1)
        sum = add(sum, Pair{__shfl_xor_sync(0xffffffffu, sum.hi, o), __shfl_xor_sync(0xffffffffu, sum.lo, o)});
      if (warps == 1) return sum;
      if (lane == 0) red_sum[slot][warp] = sum;
      __syncthreads();
      sum = lane < warps ? red_sum[slot][lane] : Pair{0.f, 0.f};
      for (int o = 1; o < warps; o <<= 1)
        sum = add(sum, Pair{__shfl_xor_sync(0xffffffffu, sum.hi, o), __shfl_xor_sync(0xffffffffu, sum.lo, o)});
      return Pair{__shfl_sync(0xffffffffu, sum.hi, 0), __shfl_sync(0xffffffffu, sum.lo, 0)};
    };
    Pair sum = square_sum(1.f, turn);
    float g;
    if (sum.hi <= kFar) {
      g = inverse_root(sum, static_cast<float>(p.C), p.eps_hi, p.eps_lo);
    } else {  // squares near fp32's largest
      __syncthreads();
      sum = square_sum(kDown, turn);
      __syncthreads();
      g = inverse_root(sum, static_cast<float>(p.C), p.eps_hi * kDown * kDown, p.eps_lo * kDown * kDown) * kDown;
    }
    const uint64_t g2 = pair_of(g, g);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = vidx(i);
      if (v >= nvec) continue;
      Raw8<BF16> raw;
      load_vec<BF16>(p.weight, 8 * static_cast<int64_t>(v), raw);
      float w[8];
      unpack8<BF16>(raw, w);
#pragma unroll
      for (int e = 0; e < 8; e += 2)
        unpack_f32x2(mul_f32x2(mul_f32x2(pair_of(f[i][e], f[i][e + 1]), g2), pair_of(w[e], w[e + 1])), f[i][e], f[i][e + 1]);
    }

    if constexpr (MODE == kModeBf16) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = vidx(i);
        if (v < nvec)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + row + 8 * static_cast<int64_t>(v)) =
              make_uint4(pack_bf16x2(f[i][0], f[i][1]), pack_bf16x2(f[i][2], f[i][3]), pack_bf16x2(f[i][4], f[i][5]),
                         pack_bf16x2(f[i][6], f[i][7]));
      }
    } else if constexpr (MODE == kModePtpc) {
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[i][e]));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      if (warps > 1) {
        if (lane == 0) red_max[turn][warp] = top;
        __syncthreads();
        top = lane < warps ? red_max[turn][lane] : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
      const float s = top > 0.f ? __fdiv_rn(top, 448.0f) : 1.0f;
      if (tid == 0) static_cast<float*>(p.scale)[r] = s;
      const Recip rc = make_recip(s);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v = vidx(i);
        if (v < nvec)
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.out) + row + 8 * static_cast<int64_t>(v)) = quant8(f[i], s, rc);
      }
    } else {
      constexpr int kBV = MODE == kModeBlockscale ? 16 : 4;  // vectors of a block
      constexpr int kLanes = kBV / kVB;
#pragma unroll
      for (int b = 0; b < VPT / kVB; ++b) {
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < kVB; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) top = fmaxf(top, fabsf(f[b * kVB + j][e]));
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const int v0 = vidx(b * kVB);
        if (v0 >= nvec) continue;
        const int64_t blk = v0 / kBV;
        const bool first = v0 % kBV == 0;
        uint2 codes[kVB];
        if constexpr (MODE == kModeBlockscale) {
          const float s = top > 0.f ? __fdiv_rn(top, 448.0f) : 1.0f;
          if (first) static_cast<float*>(p.scale)[blk * p.R + r] = s;
          const Recip rc = make_recip(s);
#pragma unroll
          for (int j = 0; j < kVB; ++j) codes[j] = quant8(f[b * kVB + j], s, rc);
        } else {
          const int code = top > 0.f ? min(max(mx_exponent(top) + 127, 0), 254) : 127;
          if (first) static_cast<uint8_t*>(p.scale)[blk * p.R + r] = static_cast<uint8_t>(code);
#pragma unroll
          for (int j = 0; j < kVB; ++j) codes[j] = quant8_pow2(f[b * kVB + j], exp2_code(254 - code));
        }
        uint8_t* to = static_cast<uint8_t*>(p.out) + row + 8 * static_cast<int64_t>(v0);
        if constexpr (kVB == 1) {
          *reinterpret_cast<uint2*>(to) = codes[0];
        } else {
#pragma unroll
          for (int j = 0; j < kVB; j += 2)
            *reinterpret_cast<uint4*>(to + 8 * j) = make_uint4(codes[j].x, codes[j].y, codes[j + 1].x, codes[j + 1].y);
        }
      }
    }
  }
}

template <int MODE, bool BF16, int VPT, int MOST>
sg_status_t launch(const NormParams& p, int num_sms, cudaStream_t stream) {
  const int threads = ((p.C / 8 + VPT - 1) / VPT + 31) / 32 * 32;
  const int64_t most = static_cast<int64_t>(num_sms) * (threads >= 256 ? 8 : 2048 / threads < 24 ? 2048 / threads : 24);
  GemmLaunch l(dim3(static_cast<unsigned>(p.R < most ? p.R : most)), dim3(threads), 0, stream, 1);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, norm_kernel<MODE, BF16, VPT, MOST>, p);
  if (e == cudaSuccess) return SG_OK;
  note_cuda_error(e);
  cudaGetLastError();
  return SG_ERR_CUDA;
}

template <int MODE, bool BF16>
sg_status_t launch_width(const NormParams& p, int num_sms, cudaStream_t stream) {
  const int vecs = p.C / 8;  // at most 4096
  if (vecs <= 1024 && (!BF16 || p.R <= 2 * num_sms)) return launch<MODE, BF16, 1, 1024>(p, num_sms, stream);
  if (vecs <= (BF16 ? 1024 : 2048)) return launch<MODE, BF16, 2, 1024>(p, num_sms, stream);
  if (vecs <= 2048) return launch<MODE, BF16, 4, 512>(p, num_sms, stream);
  return launch<MODE, BF16, 8, 512>(p, num_sms, stream);
}

template <int MODE>
sg_status_t launch_type(bool bf16, const NormParams& p, int num_sms, cudaStream_t stream) {
  return bf16 ? launch_width<MODE, true>(p, num_sms, stream) : launch_width<MODE, false>(p, num_sms, stream);
}

}  // namespace

sg_status_t norm_launch(int mode, bool bf16, const void* x, const void* residual, void* residual_out, const void* weight,
                        double eps, int64_t R, int64_t C, void* out, void* scale, int num_sms, cudaStream_t stream) {
  const float hi = static_cast<float>(eps);
  const NormParams p{x, residual, weight, residual_out, out, scale, static_cast<int>(R), static_cast<int>(C), hi,
                     static_cast<float>(eps - hi)};
  switch (mode) {
    case kModeBf16: return launch_type<kModeBf16>(bf16, p, num_sms, stream);
    case kModePtpc: return launch_type<kModePtpc>(bf16, p, num_sms, stream);
    case kModeBlockscale: return launch_type<kModeBlockscale>(bf16, p, num_sms, stream);
    case kModeMxfp8: return launch_type<kModeMxfp8>(bf16, p, num_sms, stream);
  }
  return SG_ERR_INVALID_ARG;
}

}  // namespace sg
