// sg_kv_append.cu -- rotate new queries and keys, append keys and values to the
// paged e4m3 cache (scaled_attn_append).
//
// For a pair (x, y) of a head at position p, with c = cos, s = sin of its angle:
//     x' = x c - y s,   y' = x s + y c        (fp32, each operation rounded, so the
// codes do not depend on which products a compiler contracts).  A block is 16
// positions of one head; its scale is 2^e, e the least integer with |x| <= 448 2^e
// over the block's new tokens, and at least the scale its older tokens have.
// Codes are e4m3(x 2^-e): the product is exact, so there is one rounding.  Where
// e grows the older codes are rounded again, which for a power of two is exact
// unless they fall among e4m3's subnormals.
//
// The bound is memory: 2 (Hq + 2 Hk) D bytes read and 2 Hq D + 2 Hk D (+ 2 Hk D)
// written per token, each once.  One CTA takes the new tokens of one block of
// positions of one sequence (so a block's scale has one owner: no atomics, no
// order), and its warps share out the heads: a warp takes all tokens of a K or V
// head, or a few tokens of a run of query heads, whose cosines stay in registers.
// Lanes own 16 elements of a row (a run of 8 pairs, two 16-byte loads).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cfloat>

#include "sg_attn.h"
#include "sg_mx.cuh"
#include "sg_ptx.cuh"

namespace sg {

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kHeadPasses = 8;  // passes over query heads that reuse one set of cosines

struct AppendParams {
  sg_kv_cache_t cache;
  const float* rot_table;
  int64_t max_pos;
  int rot, interleaved;
  const uint16_t *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  const int32_t *table, *ctx, *cu;
  int64_t table_stride;
  int T, B, Hq, Hk, D, page;
  uint16_t *q_out, *k_out;
};

// The 16 elements of one lane of a row: 8 pairs.
struct Run {
  int off_a, off_b;  // element offsets of its two 8-element halves
  bool live, rotated;
};

__device__ __forceinline__ Run make_run(int j, const AppendParams& p) {
  Run r;
  r.live = j < p.D / 16;
  r.rotated = j < p.rot / 16;
  if (r.rotated && !p.interleaved) {
    r.off_a = 8 * j;
    r.off_b = p.rot / 2 + 8 * j;
  } else {
    r.off_a = 16 * j;
    r.off_b = 16 * j + 8;
  }
  return r;
}

struct Raw {
  uint4 a, b;
};

__device__ __forceinline__ Raw load_raw(const uint16_t* row, const Run& r) {
  Raw x;
  x.a = *reinterpret_cast<const uint4*>(row + r.off_a);
  x.b = *reinterpret_cast<const uint4*>(row + r.off_b);
  return x;
}

__device__ __forceinline__ void widen(const uint4& w, float* f) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(u[i] << 16);
    f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 narrow(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

struct Angles {
  float c[8], s[8];
};

__device__ __forceinline__ void load_angles(const AppendParams& p, int64_t pos, int j, Angles& g) {
  const int64_t row = pos < p.max_pos ? pos : p.max_pos - 1;
  const float4* c = reinterpret_cast<const float4*>(p.rot_table + row * p.rot + 8 * j);
  const float4* s = reinterpret_cast<const float4*>(p.rot_table + row * p.rot + p.rot / 2 + 8 * j);
  *reinterpret_cast<float4*>(g.c) = __ldg(c);
  *reinterpret_cast<float4*>(g.c + 4) = __ldg(c + 1);
  *reinterpret_cast<float4*>(g.s) = __ldg(s);
  *reinterpret_cast<float4*>(g.s + 4) = __ldg(s + 1);
}

// f[0..7] and f[8..15]: the run's halves; rotated in place.
__device__ __forceinline__ void rotate(float (&f)[16], const Angles& g, bool interleaved) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float x = interleaved ? f[2 * i] : f[i];
    const float y = interleaved ? f[2 * i + 1] : f[8 + i];
    const float xr = __fsub_rn(__fmul_rn(x, g.c[i]), __fmul_rn(y, g.s[i]));
    const float yr = __fadd_rn(__fmul_rn(x, g.s[i]), __fmul_rn(y, g.c[i]));
    if (interleaved) {
      f[2 * i] = xr;
      f[2 * i + 1] = yr;
    } else {
      f[i] = xr;
      f[8 + i] = yr;
    }
  }
}

__device__ __forceinline__ uint2 codes8(const float* f, float inv) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t pair =
        __nv_cvt_float2_to_fp8x2(make_float2(f[2 * i] * inv, f[2 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    w[i >> 1] |= (pair & 0xFFFFu) << (16 * (i & 1));
  }
  return make_uint2(w[0], w[1]);
}

// Sixteen codes to a scale larger by 2^-x = `by`.
__device__ __forceinline__ uint4 rescale16(uint4 c, float by) {
  uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t o = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const __half2_raw r =
          __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[i] >> (16 * h)), __NV_E4M3);
      const float2 f = __half22float2(__half2(r));
      const uint32_t pair = __nv_cvt_float2_to_fp8x2(make_float2(f.x * by, f.y * by), __NV_SATFINITE, __NV_E4M3);
      o |= (pair & 0xFFFFu) << (16 * h);
    }
    w[i] = o;
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// What a CTA works on: new tokens [t0, t0 + n) at positions [pos, pos + n) of one
// block of 16, `held` older tokens before them.
struct Unit {
  int t0, n, held;
  int64_t pos;
  int page_id;  // -1: no page, nothing is written
  int slot0;    // the block's first slot in the page
};

// All tokens of one K or V head of the unit.
template <int LPR>
__device__ __forceinline__ void append_head(const AppendParams& p, const Unit& u, int head, bool is_k, int lane) {
  constexpr int kRows = 32 / LPR;               // tokens a pass
  constexpr int kPasses = kKvBlock / kRows;
  const int j = lane % LPR, row = lane / LPR;
  const Run run = make_run(j, p);
  const uint16_t* src = is_k ? p.k + static_cast<int64_t>(head) * p.D : p.v + static_cast<int64_t>(head) * p.D;
  const int64_t stride = is_k ? p.k_stride : p.v_stride;
  Run vr = run;
  if (!is_k) {
    vr.off_a = 16 * j;
    vr.off_b = 16 * j + 8;
  }
  uint8_t* scale = nullptr;
  uint8_t* codes = nullptr;
  int was = 0;
  if (u.page_id >= 0) {
    const int64_t nb = p.page / kKvBlock;
    scale = (is_k ? p.cache.k_scale : p.cache.v_scale) +
            (static_cast<int64_t>(u.page_id) * p.Hk + head) * nb + u.slot0 / kKvBlock;
    codes = static_cast<uint8_t*>(is_k ? p.cache.k : p.cache.v) +
            static_cast<int64_t>(u.page_id) * (is_k ? p.cache.k_page_stride : p.cache.v_page_stride) +
            (static_cast<int64_t>(head) * p.page + u.slot0) * p.D;
    if (u.held > 0) was = min(static_cast<int>(*scale), 254);
  }
  Raw raw[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int t = i * kRows + row;
    if (t < u.n && run.live) raw[i] = load_raw(src + (u.t0 + t) * stride, vr);
  }
  float f[kPasses][16];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int t = i * kRows + row;
    if (t < u.n && run.live) {
      widen(raw[i].a, f[i]);
      widen(raw[i].b, f[i] + 8);
      if (is_k && run.rotated) {
        Angles g;
        load_angles(p, u.pos + t, j, g);
        if (p.interleaved)
          rotate(f[i], g, true);
        else
          rotate(f[i], g, false);
      }
      if (is_k && p.k_out) {
        uint16_t* o = p.k_out + (static_cast<int64_t>(u.t0 + t) * p.Hk + head) * p.D;
        *reinterpret_cast<uint4*>(o + vr.off_a) = narrow(f[i]);
        *reinterpret_cast<uint4*>(o + vr.off_b) = narrow(f[i] + 8);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(f[i][e]));
    }
  }
  if (u.page_id < 0) return;
  // non-negative floats order as their bits
  amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
  amax = fminf(amax, FLT_MAX);
  int code = amax > 0.f ? min(max(mx_exponent(amax) + 127, 0), 254) : 0;
  if (u.held > 0) {
    code = max(code, was);
    if (code > was) {
      const float by = exp2_code(max(127 + was - code, 0));
      const int vecs = u.held * p.D / 16;  // a block's rows are contiguous
      for (int i = lane; i < vecs; i += 32) {
        uint4* c = reinterpret_cast<uint4*>(codes) + i;
        *c = rescale16(*c, by);
      }
    }
  }
  const float inv = exp2_code(254 - code);
  if (lane == 0) *scale = static_cast<uint8_t>(code);
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int t = i * kRows + row;
    if (t < u.n && run.live) {
      uint8_t* o = codes + static_cast<int64_t>(u.held + t) * p.D;
      *reinterpret_cast<uint2*>(o + vr.off_a) = codes8(f[i], inv);
      *reinterpret_cast<uint2*>(o + vr.off_b) = codes8(f[i] + 8, inv);
    }
  }
}

template <int LPR>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const AppendParams p) {
  __shared__ int found[kWarps];
  grid_dep_launch();
  grid_dep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // Blocks of positions are numbered from cu[b] / 16 + 2 b for sequence b: n new
  // tokens touch at most n / 16 + 2 blocks, so the ranges do not overlap and the
  // number of starts at or below a block's number gives its sequence.
  const int unit = blockIdx.x;
  auto cu = [&](int i) { return min(max(__ldg(p.cu + i), 0), p.T); };
  int below = 0;
  for (int i = tid; i < p.B; i += kThreads) below += (cu(i) / kKvBlock + 2 * i <= unit);
  below = __reduce_add_sync(0xffffffffu, below);
  if (lane == 0) found[warp] = below;
  __syncthreads();
  int b = -1;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) b += found[w];
  if (b < 0) return;
  const int first = cu(b), last = cu(b + 1);
  const int64_t ctx = max(__ldg(p.ctx + b), 0);
  const int64_t block = ctx / kKvBlock + (unit - (first / kKvBlock + 2 * b));
  Unit u;
  u.pos = max(ctx, block * kKvBlock);
  const int64_t end = min(ctx + (last - first), (block + 1) * kKvBlock);
  if (u.pos >= end) return;
  u.n = static_cast<int>(end - u.pos);
  u.t0 = first + static_cast<int>(u.pos - ctx);
  u.held = static_cast<int>(u.pos - block * kKvBlock);
  const int64_t at = block * kKvBlock / p.page;
  u.page_id = at < p.table_stride ? __ldg(p.table + b * p.table_stride + at) : -1;
  if (u.page_id >= p.cache.num_pages) u.page_id = -1;
  u.slot0 = static_cast<int>(block * kKvBlock % p.page);

  constexpr int kGroups = 32 / LPR;  // rows a warp takes at once
  const int tq = u.n >= kGroups ? kGroups : (u.n > 1 ? min(kGroups, u.n > 2 ? 4 : 2) : 1);  // tokens among them
  const int hp = kGroups / tq;                                                                // heads among them
  const int head_runs = (p.Hq + hp * kHeadPasses - 1) / (hp * kHeadPasses);
  const int q_items = (u.n + tq - 1) / tq * head_runs;
  const int items = 2 * p.Hk + q_items;
  const int j = lane % LPR, row = lane / LPR;
  const Run run = make_run(j, p);
  for (int it = blockIdx.y * kWarps + warp; it < items; it += gridDim.y * kWarps) {
    if (it < 2 * p.Hk) {
      append_head<LPR>(p, u, it >> 1, (it & 1) == 0, lane);
      continue;
    }
    const int qi = it - 2 * p.Hk;
    const int t = qi / head_runs * tq + row % tq;
    const int h0 = (qi % head_runs) * hp * kHeadPasses + row / tq;
    if (t >= u.n || !run.live) continue;
    Angles g;
    if (run.rotated) load_angles(p, u.pos + t, j, g);
    const uint16_t* src = p.q + (u.t0 + t) * p.q_stride;
    uint16_t* dst = p.q_out + static_cast<int64_t>(u.t0 + t) * p.Hq * p.D;
#pragma unroll 4
    for (int i = 0; i < kHeadPasses; ++i) {
      const int h = h0 + i * hp;
      if (h < p.Hq) {
        const Raw raw = load_raw(src + h * p.D, run);
        float f[16];
        widen(raw.a, f);
        widen(raw.b, f + 8);
        if (run.rotated) {
          if (p.interleaved)
            rotate(f, g, true);
          else
            rotate(f, g, false);
        }
        *reinterpret_cast<uint4*>(dst + h * p.D + run.off_a) = narrow(f);
        *reinterpret_cast<uint4*>(dst + h * p.D + run.off_b) = narrow(f + 8);
      }
    }
  }
}

}  // namespace

sg_status_t append_launch(const AttnShape& s, const AttnArgs& a) {
  AppendParams p{};
  p.cache = a.cache;
  p.rot_table = a.rotary.table;
  p.max_pos = a.rotary.max_pos;
  p.rot = a.rotary.rot;
  p.interleaved = a.rotary.interleaved != 0;
  p.q = static_cast<const uint16_t*>(a.q);
  p.k = static_cast<const uint16_t*>(a.k);
  p.v = static_cast<const uint16_t*>(a.v);
  p.q_stride = a.q_stride;
  p.k_stride = a.k_stride;
  p.v_stride = a.v_stride;
  p.table = a.table;
  p.table_stride = a.table_stride;
  p.ctx = a.lens;
  p.cu = a.cu_q;
  p.T = static_cast<int>(a.Tq);
  p.B = static_cast<int>(a.B);
  p.Hq = s.Hq;
  p.Hk = s.Hk;
  p.D = s.D;
  p.page = s.page;
  p.q_out = static_cast<uint16_t*>(a.out);
  p.k_out = static_cast<uint16_t*>(a.k_out);
  const unsigned units = static_cast<unsigned>(a.Tq / kKvBlock + 2 * a.B);
  GemmLaunch l(dim3(units, 1), dim3(kThreads), 0, a.stream, 1);
  const cudaError_t e = s.D > 64 ? cudaLaunchKernelEx(&l.cfg, kv_append_kernel<8>, p)
                                 : cudaLaunchKernelEx(&l.cfg, kv_append_kernel<4>, p);
  if (e != cudaSuccess) {
    note_cuda_error(e);
    cudaGetLastError();
    return SG_ERR_CUDA;
  }
  return SG_OK;
}

}  // namespace sg
