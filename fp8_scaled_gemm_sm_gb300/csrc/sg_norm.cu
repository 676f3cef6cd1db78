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
// It costs 4 instructions an element (5.5 for fp32 rows, whose squares are not exact in 24 bits).
//
// The bound is memory: x and the residual are read once, the sum is written once and the
// codes once; the row stays in registers in between.  A CTA a row, rows dealt out in turn.  Where there are many rows, what is close to that
// bound is instructions and the wait for a row's sum: so rows are on their way two ahead, a warp of its own forms the root
// while the others take the next row, and a block's scale is divided once.  32768 x 7168 bf16 with a residual: blockscale
// 295 us (82 % of the copy rate), mxfp8 281, ptpc 279, bf16 309.
#include <cuda.h>
#include <cuda_runtime.h>

#include "sg_common.cuh"
#include "sg_internal.h"
#include "sg_mx.cuh"
#include "sg_quant.cuh"

namespace sg {

namespace {

constexpr int kMaxWarps = 32;
constexpr int kAhead = 2;           // rows on their way to a CTA
constexpr int kSmem = 232448;       // shared memory of an SM that CTAs get
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

__device__ __forceinline__ uint4 ld_shared_16b(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

template <bool BF16>
__device__ __forceinline__ void load_vec(const void* X, int64_t elem, Raw8<BF16>& raw) {
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(X) + elem * (BF16 ? 2 : 4));
#pragma unroll
  for (int i = 0; i < (BF16 ? 1 : 2); ++i) raw.w[i] = p[i];
}

// The largest of a warp's values, none of them negative: their bits are in the same order.
__device__ __forceinline__ float warp_max(float x) { return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(x))); }

// The sum of squares of a thread's elements, scaled by `by`.
template <bool BF16, int VPT>
__device__ __forceinline__ Pair squares(const float (&f)[VPT][8], float by) {
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
  return add(Pair{s0, e0}, Pair{s1, e1});
}

// The sum over a warp's first `lanes` lanes (a power of two, or less than one), in each of them.
__device__ __forceinline__ Pair across(Pair sum, int lanes) {
  for (int o = 1; o < lanes; o <<= 1)
    sum = add(sum, Pair{__shfl_xor_sync(0xffffffffu, sum.hi, o), __shfl_xor_sync(0xffffffffu, sum.lo, o)});
  return sum;
}

__device__ __forceinline__ float near_root(const NormParams& p, const Pair& sum) {
  return inverse_root(sum, static_cast<float>(p.C), p.eps_hi, p.eps_lo);
}
// Of squares of elements scaled by kDown.
__device__ __forceinline__ float far_root(const NormParams& p, const Pair& sum) {
  return inverse_root(sum, static_cast<float>(p.C), p.eps_hi * kDown * kDown, p.eps_lo * kDown * kDown) * kDown;
}

// x + residual of one vector, as it is kept and in fp32.
__device__ __forceinline__ uint4 add_residual(const float (&x)[8], const float (&r)[8], float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float a, b;
    unpack_f32x2(add_f32x2(pair_of(x[2 * e], x[2 * e + 1]), pair_of(r[2 * e], r[2 * e + 1])), a, b);
    w[e] = pack_bf16x2(a, b);
    f[2 * e] = __uint_as_float(w[e] << 16);
    f[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ void weigh(float (&f)[8], uint64_t g2, const float (&w)[8]) {
#pragma unroll
  for (int e = 0; e < 8; e += 2)
    unpack_f32x2(mul_f32x2(mul_f32x2(pair_of(f[e], f[e + 1]), g2), pair_of(w[e], w[e + 1])), f[e], f[e + 1]);
}

// Where a thread's vectors tid, tid + T, ... of a row go: `out` and `scale` are the first one's, scale_step
// lies from one's scale to the next one's.
template <int MODE>
struct Places {
  static constexpr int kLanes = MODE == kModeBlockscale ? 16 : MODE == kModeMxfp8 ? 4 : 1;  // vectors of a block
  static constexpr int kOut = MODE == kModeBf16 ? 16 : 8, kScale = MODE == kModeMxfp8 ? 1 : 4;  // bytes
  uint8_t *out, *scale;
  int64_t scale_step;
  __device__ __forceinline__ Places(const NormParams& p, int row, int tid, int T)
      : out(static_cast<uint8_t*>(p.out) + static_cast<int64_t>(row) * p.C * (kOut / 8) + kOut * tid),
        scale(static_cast<uint8_t*>(p.scale) + kScale * (MODE == kModePtpc ? row : static_cast<int64_t>(tid / kLanes) * p.R + row)),
        scale_step(static_cast<int64_t>(kScale) * (T / kLanes) * p.R) {}
};

// A row of y as a mode has it; all: the row has every vector of the thread's; `row_max` makes a warp's maximum the row's.
template <int MODE, int VPT, bool ALL, typename RowMax>
__device__ __forceinline__ void put(const Places<MODE>& at, const float (&f)[VPT][8], int nvec, int tid, int T, RowMax&& row_max) {
  auto there = [&](int i) { return ALL || i * T + tid < nvec; };
  auto out = [&](int i) { return at.out + i * T * at.kOut; };
  const int lane = tid & 31;
  if constexpr (MODE == kModeBf16) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (there(i))
        *reinterpret_cast<uint4*>(out(i)) = make_uint4(pack_bf16x2(f[i][0], f[i][1]), pack_bf16x2(f[i][2], f[i][3]),
                                                       pack_bf16x2(f[i][4], f[i][5]), pack_bf16x2(f[i][6], f[i][7]));
  } else {
    float top[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      top[i] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; e += 2) top[i] = max3(top[i], fabsf(f[i][e]), fabsf(f[i][e + 1]));
    }
    if constexpr (MODE == kModePtpc) {
#pragma unroll
      for (int i = 1; i < VPT; ++i) top[0] = fmaxf(top[0], top[i]);
      const float most = row_max(warp_max(top[0])), s = most > 0.f ? __fdiv_rn(most, 448.0f) : 1.0f;
      if (tid == 0) *reinterpret_cast<float*>(at.scale) = s;
      const Recip rc = make_recip(s);
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (there(i)) *reinterpret_cast<uint2*>(out(i)) = quant8(f[i], s, rc);
    } else {
      const bool first = tid % at.kLanes == 0;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int o = at.kLanes / 2; o > 0; o >>= 1) top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
      if constexpr (MODE == kModeBlockscale) {
        // a block's scale and its reciprocal are formed by one lane: lane i of a half warp has those of vector i's
        float s_lane = top[0];
#pragma unroll
        for (int i = 1; i < VPT; ++i) s_lane = lane % 16 == i ? top[i] : s_lane;
        s_lane = s_lane > 0.f ? __fdiv_rn(s_lane, 448.0f) : 1.0f;
        const float r_lane = __frcp_rn(s_lane);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          const float s = __shfl_sync(0xffffffffu, s_lane, i, 16), r = __shfl_sync(0xffffffffu, r_lane, i, 16);
          if (!there(i)) continue;
          if (first) *reinterpret_cast<float*>(at.scale + i * at.scale_step) = s;
          *reinterpret_cast<uint2*>(out(i)) = quant8(f[i], s, make_recip(s, r));
        }
      } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
          if (!there(i)) continue;
          const int code = top[i] > 0.f ? min(max(mx_exponent(top[i]) + 127, 0), 254) : 127;
          if (first) at.scale[i * at.scale_step] = static_cast<uint8_t>(code);
          *reinterpret_cast<uint2*>(out(i)) = quant8_pow2(f[i], exp2_code(254 - code));
        }
      }
    }
  }
}

// Rows from global memory straight to registers.  VPT: vectors of eight elements a thread; MOST: threads at most.
template <int MODE, bool BF16, int VPT, int MOST>
__global__ void __launch_bounds__(MOST) norm_kernel(const NormParams p) {
  __shared__ Pair red_sum[2][kMaxWarps];
  __shared__ float red_max[2][kMaxWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, T = blockDim.x, warps = T >> 5;
  const int nvec = p.C / 8, R = p.R, step = gridDim.x;
  auto vidx = [&](int i) { return i * T + tid; };  // vector i of this thread: a block's lie in consecutive lanes
  constexpr bool kNext = VPT == 1;  // the next row's vectors load while this one is worked on, where they take few registers
  auto fetch = [&](Raw8<BF16>(&x)[VPT], Raw8<BF16>(&r)[VPT], int row) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = vidx(i);
      if (v >= nvec || row >= R) continue;
      const int64_t at = static_cast<int64_t>(row) * p.C + 8 * static_cast<int64_t>(v);
      load_vec<BF16>(p.x, at, x[i]);
      if (p.residual) load_vec<BF16>(p.residual, at, r[i]);
    }
  };
  grid_dep_launch();
  grid_dep_wait();
  Raw8<BF16> next_x[VPT], next_r[VPT];
  if constexpr (kNext) fetch(next_x, next_r, blockIdx.x);
  int turn = 0;
  for (int r = blockIdx.x; r < R; r += step, turn ^= 1) {
    const int64_t row = static_cast<int64_t>(r) * p.C;
    float f[VPT][8];
    if constexpr (!kNext) fetch(next_x, next_r, r);
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
      if constexpr (BF16) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.residual_out) + at) = add_residual(f[i], g, f[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[i][e] = __fadd_rn(f[i][e], g[e]);
        float4* to = reinterpret_cast<float4*>(static_cast<float*>(p.residual_out) + at);
        to[0] = make_float4(f[i][0], f[i][1], f[i][2], f[i][3]);
        to[1] = make_float4(f[i][4], f[i][5], f[i][6], f[i][7]);
      }
    }
    if constexpr (kNext) fetch(next_x, next_r, r + step);

    auto square_sum = [&](float by) {
      Pair sum = across(squares<BF16, VPT>(f, by), 32);
      if (warps == 1) return sum;
      if (lane == 0) red_sum[turn][warp] = sum;
      __syncthreads();
      sum = across(lane < warps ? red_sum[turn][lane] : Pair{0.f, 0.f}, warps);
      return Pair{__shfl_sync(0xffffffffu, sum.hi, 0), __shfl_sync(0xffffffffu, sum.lo, 0)};
    };
    Pair sum = square_sum(1.f);
    float g;
    if (sum.hi <= kFar) {
      g = near_root(p, sum);
    } else {  // squares near fp32's largest
      __syncthreads();
      sum = square_sum(kDown);
      __syncthreads();
      g = far_root(p, sum);
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
      weigh(f[i], g2, w);
    }
    put<MODE, VPT, false>(Places<MODE>(p, r, tid, T), f, nvec, tid, T, [&](float top) {
      if (warps == 1) return top;
      if (lane == 0) red_max[turn][warp] = top;
      __syncthreads();
      return warp_max(lane < warps ? red_max[turn][lane] : 0.f);
    });
  }
}

// Many bf16 rows with a residual: they come through shared memory, kAhead before their turn, and a row's root is formed by a
// warp of its own (the last) while the others add up the next row.  A thread's words of a row are its own in
// shared memory too, [stage][x, residual][VPT][T], so loads need no barrier; a stage is filled again one row after it was read.
// ALL: rows have VPT vectors for every thread.
template <int MODE, int VPT, int MOST, int CTAS, bool ALL>
__global__ void __launch_bounds__(MOST, CTAS) norm_rows_kernel(const NormParams p) {
  __shared__ Pair sums[2][MOST - 32];
  __shared__ float roots[2], red_max[kMaxWarps];
  extern __shared__ __align__(16) uint8_t rows_smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, T = blockDim.x - 32, warps = T >> 5;
  const int nvec = p.C / 8, R = p.R, step = gridDim.x;
  auto all_sync = [&]() { asm volatile("bar.sync 2, %0;" ::"r"(T + 32) : "memory"); };  // of both kinds of warps
  grid_dep_launch();
  grid_dep_wait();
  if (warp == warps) {
    auto root = [&](int turn, bool far) {
      Pair a = sums[turn][lane], b{0.f, 0.f};
      for (int w = 1; w < warps; w += 2) {
        b = add(b, sums[turn][32 * w + lane]);
        if (w + 1 < warps) a = add(a, sums[turn][32 * w + 32 + lane]);
      }
      const Pair sum = across(add(a, b), 32);
      if (lane == 0) roots[turn] = far ? far_root(p, sum) : sum.hi <= kFar ? near_root(p, sum) : -1.f;
    };
    all_sync();
    int turn = 0;
    for (int r = blockIdx.x; r < R; r += step, turn ^= 1) {
      root(turn, false);
      all_sync();
      if (roots[turn] < 0.f) {
        all_sync();
        root(turn, true);
        all_sync();
      }
    }
    return;
  }
  auto there = [&](int i) { return ALL || i * T + tid < nvec; };
  const uint32_t mine = smem_addr(rows_smem) + 16 * tid, part = VPT * 16 * T, vec = 16 * T;
  // this thread's first vector of the row that is read next, of the row that is kept next
  const int64_t row_bytes = static_cast<int64_t>(step) * p.C * 2, begin = (static_cast<int64_t>(blockIdx.x) * p.C + 8 * tid) * 2;
  const uint8_t *x = static_cast<const uint8_t*>(p.x) + begin, *residual = static_cast<const uint8_t*>(p.residual) + begin;
  uint8_t* kept_at = static_cast<uint8_t*>(p.residual_out) + begin;
  auto ahead = [&](int row, int stage) {
    if (row < R) {
      const uint32_t to = mine + 2 * part * stage;
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        if (!there(i)) continue;
        cp_async_16(to + i * vec, x + i * vec, 16);
        cp_async_16(to + part + i * vec, residual + i * vec, 16);
      }
    }
    x += row_bytes, residual += row_bytes;
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kAhead; ++s) ahead(blockIdx.x + s * step, s);
  // Weights stay in registers where there are 128 a thread (32768 x 7168 ptpc 278 us, read again for each row 310), not where there are
  // 96, which would spill (8192 x 16384 195 and 201, 16384 x 8192 183 and 184).
  constexpr bool kKept = MOST == 256;
  Raw8<true> weight[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i)
    if (kKept && there(i)) load_vec<true>(p.weight, 8 * static_cast<int64_t>(i * T + tid), weight[i]);
  int stage = 0;
  // Row r as it is kept, and its squares.
  auto take = [&](int r, int turn, uint4(&kept)[VPT]) {
    ahead(r + kAhead * step, stage >= 1 ? stage - 1 : kAhead);
    cp_async_wait<kAhead>();
    float f[VPT][8];
    const uint32_t from = mine + 2 * part * stage;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      Raw8<true> a, b;
      a.w[0] = b.w[0] = make_uint4(0, 0, 0, 0);  // past the row
      if (there(i)) a.w[0] = ld_shared_16b(from + i * vec), b.w[0] = ld_shared_16b(from + part + i * vec);
      float u[8], v[8];
      unpack8<true>(a, u);
      unpack8<true>(b, v);
      kept[i] = add_residual(u, v, f[i]);
      if (there(i)) *reinterpret_cast<uint4*>(kept_at + i * vec) = kept[i];
    }
    kept_at += row_bytes;
    stage = stage == kAhead ? 0 : stage + 1;
    sums[turn][tid] = squares<true, VPT>(f, 1.f);
  };
  uint4 now[VPT], next[VPT];
  take(blockIdx.x, 0, now);
  all_sync();
  int turn = 0;
  Places<MODE> at(p, blockIdx.x, tid, T);
  for (int r = blockIdx.x; r < R; r += step, turn ^= 1) {
    if (r + step < R) take(r + step, turn ^ 1, next);
    all_sync();
    float f[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) unpack8<true>(Raw8<true>{{now[i]}}, f[i]);
    float g = roots[turn];
    if (__builtin_expect(g < 0.f, 0)) {  // squares near fp32's largest
      sums[turn][tid] = squares<true, VPT>(f, kDown);
      all_sync();
      all_sync();
      g = roots[turn];
    }
    const uint64_t g2 = pair_of(g, g);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      if (!kKept && there(i)) load_vec<true>(p.weight, 8 * static_cast<int64_t>(i * T + tid), weight[i]);
      float w[8];
      unpack8<true>(weight[i], w);
      weigh(f[i], g2, w);
    }
    put<MODE, VPT, ALL>(at, f, nvec, tid, T, [&](float top) {
      if (lane == 0) red_max[warp] = top;
      asm volatile("bar.sync 1, %0;" ::"r"(T) : "memory");
      return warp_max(lane < warps ? red_max[lane] : 0.f);
    });
    at.out += static_cast<int64_t>(step) * p.C * (at.kOut / 8);
    at.scale += at.kScale * step;
#pragma unroll
    for (int i = 0; i < VPT; ++i) now[i] = next[i];
  }
}

sg_status_t launch_error(cudaError_t e) {
  if (e == cudaSuccess) return SG_OK;
  note_cuda_error(e);
  cudaGetLastError();
  return SG_ERR_CUDA;
}

int threads_of(int C, int vpt) { return ((C / 8 + vpt - 1) / vpt + 31) / 32 * 32; }

template <int MODE, bool BF16, int VPT, int MOST>
sg_status_t launch(const NormParams& p, int num_sms, cudaStream_t stream) {
  const int threads = threads_of(p.C, VPT);
  const int64_t most = static_cast<int64_t>(num_sms) * (threads >= 256 ? 8 : 2048 / threads < 24 ? 2048 / threads : 24);
  GemmLaunch l(dim3(static_cast<unsigned>(p.R < most ? p.R : most)), dim3(threads), 0, stream, 1);
  return launch_error(cudaLaunchKernelEx(&l.cfg, norm_kernel<MODE, BF16, VPT, MOST>, p));
}

template <int MODE, int MOST, int CTAS, bool ALL>
sg_status_t launch_rows(const NormParams& p, int num_sms, cudaStream_t stream) {
  constexpr int VPT = 4;
  constexpr int kRegs = 65536 / (MOST * CTAS) / 8 * 8 < 128 ? 65536 / (MOST * CTAS) / 8 * 8 : 128;  // of a thread, at most
  const int threads = threads_of(p.C, VPT) + 32, bytes = (kAhead + 1) * 2 * (threads - 32) * VPT * 16;
  const int by_smem = kSmem / (bytes + 16 * MOST + 2048), by_regs = 65536 / (kRegs * threads);
  const int64_t most = static_cast<int64_t>(num_sms) * (by_smem < by_regs ? by_smem : by_regs);
  auto* const kernel = norm_rows_kernel<MODE, VPT, MOST, CTAS, ALL>;
  if (bytes > 32768) {  // of the device that is current
    const sg_status_t r = launch_error(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    if (r != SG_OK) return r;
  }
  GemmLaunch l(dim3(static_cast<unsigned>(p.R < most ? p.R : most)), dim3(threads), bytes, stream, 1);
  return launch_error(cudaLaunchKernelEx(&l.cfg, kernel, p));
}

template <int MODE, bool BF16>
sg_status_t launch_width(const NormParams& p, int num_sms, cudaStream_t stream) {
  const int vecs = p.C / 8;  // at most 4096
  // From four rows an SM and 2048 columns on, bf16 rows with a residual come through shared memory: 32768 x 7168 for blockscale
  // 295 us, straight to registers 400; 16384 x 4096 for mxfp8 86 and 100; 20000 x 2048 57 and 60; but 20000 x 1024 for ptpc 42 and 34, where a
  // CTA's last warp is one of two.  Up to 7168 columns two CTAs have 8 warps each and 128 registers a thread, at 8192 9 warps
  // and 96 (16384 x 8192 for ptpc 183 and 214 us), above 8192 one CTA has an SM (8192 x 16384 195 and 225; 16384 x 8192 264).
  // More CTAs with fewer registers for narrower rows: 30000 x 4096 blockscale 155 (four), 197 (three), two 147.
  // Past 7168 columns rows come that way where every thread has four vectors, at multiples of 1024 columns.  With 96 registers the check of each vector
  // that other widths need spills 8 to 40 bytes: it gains there (16384 x 7680 for ptpc 184 us, straight to registers 211, mxfp8 203 and 203;
  // 8192 x 10752 151 and 186, 175 and 187), loses where no check is needed (16384 x 8192 for ptpc 193 and 185, bf16 221 and 178),
  // and would be eight kernels more; those widths go straight to registers.
  if constexpr (BF16) {
    if (p.R >= 4 * num_sms && p.residual && vecs >= 256) {
      const bool all = vecs % 128 == 0;  // every thread has four
      if (vecs <= 896) return all ? launch_rows<MODE, 256, 2, true>(p, num_sms, stream) : launch_rows<MODE, 256, 2, false>(p, num_sms, stream);
      if (vecs == 1024) return launch_rows<MODE, 288, 2, true>(p, num_sms, stream);
      if (all && vecs <= 2048) return launch_rows<MODE, 544, 1, true>(p, num_sms, stream);
    }
  }
  // Straight to registers: a vector a thread, two for bf16 rows of which a CTA has several and for wide fp32 rows, and four or eight in 512 threads past that.  Rows past
  // 16384 columns, and fp32 rows past 8192, do not fit the registers: up to 16384 fp32 spills 36 to 64 bytes a thread (8192 x 12288 for ptpc 283 us, floor 193),
  // past that bf16 248 to 280 (8192 x 20480 585, floor 174) and fp32 448 to 544 (4096 x 32768 for mxfp8 594, floor 258).
  if (vecs <= 1024 && (!BF16 || p.R <= 2 * num_sms)) return launch<MODE, BF16, 1, 1024>(p, num_sms, stream);
  if (vecs <= (BF16 ? 1024 : 2048)) return launch<MODE, BF16, 2, 1024>(p, num_sms, stream);
  if constexpr (BF16) {
    if (vecs <= 2048) return launch<MODE, BF16, 4, 512>(p, num_sms, stream);
  }
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
