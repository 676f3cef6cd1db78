// sg_attn_decode.cu -- attention of the newest tokens over the paged e4m3 cache
// (scaled_attn_decode).
//
// For a query row x of head h and the keys j it sees,
//     s_j = scale x . k_j,   o = sum_j e^(s_j - m) v_j / sum_j e^(s_j - m),   m = max_j s_j,
// in one pass: a running maximum, sum and output, the last two scaled by
// e^(m_old - m_new) when the maximum grows.  k and v are e4m3 codes times their
// block's power of two.  One warp per row and head; a lane owns 4 dimensions.
#include <cuda.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "sg_attn.h"
#include "sg_mx.cuh"
#include "sg_ptx.cuh"

namespace sg {

namespace {

struct DecodeParams {
  sg_kv_cache_t cache;
  const uint16_t* q;
  int64_t q_stride;
  const int32_t *table, *lens;
  int64_t table_stride;
  int B, qn, Hq, Hk, D, page;
  float scale_log2;
  uint16_t* out;
  float* lse;
};

__device__ __forceinline__ float e8m0(uint8_t c) {
  return c == 255 ? __uint_as_float(0x7FC00000u) : exp2_code(c);
}

__device__ __forceinline__ void decode4(uint32_t w, float (&f)[4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w >> (16 * h)), __NV_E4M3);
    const float2 v = __half22float2(__half2(r));
    f[2 * h] = v.x;
    f[2 * h + 1] = v.y;
  }
}

__global__ void __launch_bounds__(128) decode_rows_kernel(const DecodeParams p) {
  grid_dep_launch();
  grid_dep_wait();
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (item >= static_cast<int64_t>(p.B) * p.qn * p.Hq) return;
  const int64_t row = item / p.Hq;
  const int h = static_cast<int>(item % p.Hq), hk = h / (p.Hq / p.Hk);
  const int b = static_cast<int>(row / p.qn), i = static_cast<int>(row % p.qn);
  const bool live = 4 * lane < p.D;
  float q[4] = {0.f, 0.f, 0.f, 0.f};
  if (live)
    for (int e = 0; e < 4; ++e)
      q[e] = __uint_as_float(static_cast<uint32_t>(p.q[row * p.q_stride + h * p.D + 4 * lane + e]) << 16) * p.scale_log2;
  int64_t n = min(static_cast<int64_t>(max(p.lens[b], 0)), p.table_stride * p.page) - (p.qn - 1 - i);
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  const int nb = p.page / kKvBlock;
  for (int64_t j = 0; j < n; ++j) {
    const int32_t pg = p.table[b * p.table_stride + j / p.page];
    if (pg < 0 || pg >= p.cache.num_pages) continue;
    const int slot = static_cast<int>(j % p.page);
    const int64_t sc = (static_cast<int64_t>(pg) * p.Hk + hk) * nb + slot / kKvBlock;
    const int64_t in_page = (static_cast<int64_t>(hk) * p.page + slot) * p.D + 4 * lane;
    float k[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
    if (live) {
      decode4(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.cache.k) + pg * p.cache.k_page_stride + in_page), k);
      decode4(*reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.cache.v) + pg * p.cache.v_page_stride + in_page), v);
    }
    float s = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= e8m0(p.cache.k_scale[sc]);
    const float mn = fmaxf(m, s);
    const float keep = mn == -INFINITY ? 1.f : exp2f(m - mn), w = mn == -INFINITY ? 0.f : exp2f(s - mn);
    const float vs = e8m0(p.cache.v_scale[sc]);
    l = l * keep + w;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = o[e] * keep + w * (v[e] * vs);
    m = mn;
  }
  if (live) {
    const float inv = m == -INFINITY && l == 0.f ? 0.f : 1.f / l;
    uint2 w = make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    *reinterpret_cast<uint2*>(p.out + (row * p.Hq + h) * p.D + 4 * lane) = w;
  }
  if (lane == 0 && p.lse) p.lse[row * p.Hq + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

size_t decode_workspace_bytes(const AttnShape&) { return 0; }
cudaError_t decode_prepare() { return cudaSuccess; }

sg_status_t decode_launch(const AttnShape& s, const AttnArgs& a) {
  DecodeParams p{};
  p.cache = a.cache;
  p.q = static_cast<const uint16_t*>(a.q);
  p.q_stride = a.q_stride;
  p.table = a.table;
  p.lens = a.lens;
  p.table_stride = a.table_stride;
  p.B = static_cast<int>(a.B);
  p.qn = static_cast<int>(a.qn);
  p.Hq = s.Hq;
  p.Hk = s.Hk;
  p.D = s.D;
  p.page = s.page;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  const int64_t rows = a.B * a.qn * s.Hq;
  GemmLaunch l(dim3(static_cast<unsigned>((rows + 3) / 4)), dim3(128), 0, a.stream, 1);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, decode_rows_kernel, p);
  if (e != cudaSuccess) {
    note_cuda_error(e);
    cudaGetLastError();
    return SG_ERR_CUDA;
  }
  return SG_OK;
}

}  // namespace sg
