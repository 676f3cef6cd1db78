// sg_attn_prompt.cu -- attention over whole packed prompts (scaled_attn_prompt).
//
// For query row i of a sequence with n queries and m keys, over the keys
// j <= i + m - n (causal) or all m,
//     s_j = scale q_i . k_j,   o_i = sum_j e^(s_j - mx) v_j / sum_j e^(s_j - mx),
// in one pass with a running maximum and sum.  One warp per row and head; a lane
// owns 4 dimensions.
#include <cuda.h>
#include <cuda_runtime.h>

#include "sg_attn.h"
#include "sg_ptx.cuh"

namespace sg {

namespace {

struct PromptParams {
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t *cu_q, *cu_k;
  int Tq, Tk, B, Hq, Hk, D, causal;
  float scale_log2;
  uint16_t* out;
  float* lse;
};

__device__ __forceinline__ void load4(const uint16_t* x, float (&f)[4]) {
  const uint2 w = *reinterpret_cast<const uint2*>(x);
  f[0] = __uint_as_float(w.x << 16);
  f[1] = __uint_as_float(w.x & 0xFFFF0000u);
  f[2] = __uint_as_float(w.y << 16);
  f[3] = __uint_as_float(w.y & 0xFFFF0000u);
}

__global__ void __launch_bounds__(128) prompt_rows_kernel(const PromptParams p) {
  grid_dep_launch();
  grid_dep_wait();
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (item >= static_cast<int64_t>(p.Tq) * p.Hq) return;
  const int row = static_cast<int>(item / p.Hq), h = static_cast<int>(item % p.Hq), hk = h / (p.Hq / p.Hk);
  int b = 0;
  for (int i = lane; i < p.B; i += 32) b += p.cu_q[i + 1] <= row;
  b = __reduce_add_sync(0xffffffffu, b);
  const bool live = 4 * lane < p.D;
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  if (b < p.B) {
    const int q0 = min(max(p.cu_q[b], 0), p.Tq), q1 = min(max(p.cu_q[b + 1], 0), p.Tq);
    const int k0 = min(max(p.cu_k[b], 0), p.Tk), k1 = min(max(p.cu_k[b + 1], k0), p.Tk);
    const int see = p.causal ? min(k1 - k0, row - q0 + 1 + (k1 - k0) - (q1 - q0)) : k1 - k0;
    float q[4] = {0.f, 0.f, 0.f, 0.f};
    if (live) load4(p.q + row * p.q_stride + h * p.D + 4 * lane, q);
    for (int j = 0; j < see; ++j) {
      float k[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
      if (live) {
        load4(p.k + (k0 + j) * p.k_stride + hk * p.D + 4 * lane, k);
        load4(p.v + (k0 + j) * p.v_stride + hk * p.D + 4 * lane, v);
      }
      float s = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
      for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      s *= p.scale_log2;
      const float mn = fmaxf(m, s);
      const float keep = mn == -INFINITY ? 1.f : exp2f(m - mn), w = mn == -INFINITY ? 0.f : exp2f(s - mn);
      l = l * keep + w;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = o[e] * keep + w * v[e];
      m = mn;
    }
  }
  if (live) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    *reinterpret_cast<uint2*>(p.out + item * p.D + 4 * lane) =
        make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
  }
  if (lane == 0 && p.lse) p.lse[item] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

cudaError_t prompt_prepare() { return cudaSuccess; }

sg_status_t prompt_launch(const AttnShape& s, const AttnArgs& a) {
  PromptParams p{};
  p.q = static_cast<const uint16_t*>(a.q);
  p.k = static_cast<const uint16_t*>(a.k);
  p.v = static_cast<const uint16_t*>(a.v);
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.cu_q = a.cu_q;
  p.cu_k = a.cu_k;
  p.Tq = static_cast<int>(a.Tq);
  p.Tk = static_cast<int>(a.Tk);
  p.B = static_cast<int>(a.B);
  p.Hq = s.Hq;
  p.Hk = s.Hk;
  p.D = s.D;
  p.causal = a.causal;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  const int64_t rows = a.Tq * s.Hq;
  GemmLaunch l(dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0, a.stream, 1);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, prompt_rows_kernel, p);
  if (e != cudaSuccess) {
    note_cuda_error(e);
    cudaGetLastError();
    return SG_ERR_CUDA;
  }
  return SG_OK;
}

}  // namespace sg
