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
// order).  Lanes own 16 elements of a row (a run of 8 pairs, two 16-byte loads); the
// rows that a warp holds at once are up to 4 tokens times heads, so that one new token a sequence
// fills lanes as well as sixteen.  A warp's work comes in items of 4 KB (a block's tokens of a key or value head, 4
// tokens of query heads), loaded to shared memory asynchronously while the item before is worked on.  K and V rows
// are rotated twice from there, for the block's maximum and for its codes: in registers their fp32 values would take
// the room of half the warps.  The tokens' cosines and sines, which all heads use, wait in shared memory too: the
// items leave L1 too little room for them.  48k prompt tokens, 32 heads of 128 over 8: 230 us, 91% of the
// rate of a copy (249 without loading ahead and with cosines through L1, 281 with fp32 kept); 41 chunks of up to 1500
// tokens, 24 heads of 64 over 24: 43 us (50), half of the issue slots and of the memory; one token of 512 sequences 6.5 us, of 8
// sequences 3.4, most of it the launch and four dependent loads.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <cfloat>

#include "sg_attn.h"
#include "sg_attn_ptx.cuh"
#include "sg_mx.cuh"

namespace sg {

namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kPassBytes = 1024;  // shared memory of a warp's pass: 32 bytes a lane
constexpr int kHeadPasses = 4;  // passes over query heads that reuse one set of cosines
constexpr int kTokens = 4;      // tokens that a warp holds at once, where there are as many; its other lanes take heads
constexpr int kPasses = kKvBlock / kTokens;  // passes over a block's tokens
constexpr int kItemBytes = 4 * kPassBytes;   // shared memory of an item: 4 passes
constexpr int kCtas = 4;        // resident CTAs an SM
constexpr int kWaves = 4;       // CTAs wanted, in times what the GPU holds

struct AppendParams {
  sg_kv_cache_t cache;
  const float* rot_table;
  int64_t max_pos;
  int rot, by_token;
  float one;  // 1
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

template <bool INTER, bool ROTATE>
__device__ __forceinline__ Run make_run(int j, const AppendParams& p) {
  Run r;
  r.live = j < p.D / 16;
  r.rotated = ROTATE && j < p.rot / 16;
  if (r.rotated && !INTER) {
    r.off_a = 8 * j;
    r.off_b = p.rot / 2 + 8 * j;
  } else {
    r.off_a = 16 * j;
    r.off_b = 16 * j + 8;
  }
  return r;
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

__device__ __forceinline__ uint4 ld_shared_16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

// What a CTA works on: new tokens [t0, t0 + n) at positions [pos, pos + n) of one
// block of 16, `held` older tokens before them.
struct Unit {
  int t0, n, held;
  int64_t pos;
  int page_id;  // outside [0, num_pages): no page, nothing is written
  int slot0;    // the block's first slot in the page
};

struct Angles {
  float c[8], s[8];
};

// The cosines and sines of a unit's tokens in shared memory: of a token, the first four of every run, then the
// other four (a warp's 16-byte reads then lie side by side), cosines before sines.
constexpr int kAngleRow = (128 + 16) * 4;

__device__ __forceinline__ void stage_angles(const AppendParams& p, const Unit& u, uint32_t angles) {
  const int vecs = p.rot / 4, runs = p.rot / 16;  // 16-byte pieces of a token, runs
  for (int i = threadIdx.x; i < u.n * vecs; i += kThreads) {
    const int t = i / vecs, x = i - t * vecs, sine = x >= 2 * runs, y = x - sine * 2 * runs;
    const int64_t row = min(u.pos + t, p.max_pos - 1);
    cp_async_16(angles + t * kAngleRow + (sine * 2 * runs + (y & 1) * runs + (y >> 1)) * 16, p.rot_table + row * p.rot + 4 * x, 16);
  }
}

__device__ __forceinline__ Angles load_angles(const AppendParams& p, uint32_t angles, int t, int j) {
  Angles g;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 v = ld_shared_16(angles + t * kAngleRow + (i * (p.rot / 16) + j) * 16);
    float* f = (i < 2 ? g.c : g.s) + 4 * (i & 1);
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  }
  return g;
}

// f[0..7] and f[8..15]: the run's halves; rotated in place, two pairs an instruction.  The sum of two
// rounded products is formed as fma(product, one, product) with a `one` that the
// compiler does not know: it contracts a packed multiplication and addition otherwise.
template <bool INTER>
__device__ __forceinline__ void rotate(float (&f)[16], const Angles& g, float one) {
  const uint64_t one2 = pack_f32x2(one, one);
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const int x0 = INTER ? 2 * i : i, x1 = INTER ? 2 * i + 2 : i + 1, y = INTER ? 1 : 8;
    const uint64_t x = pack_f32x2(f[x0], f[x1]), z = pack_f32x2(f[x0 + y], f[x1 + y]);
    const uint64_t c = pack_f32x2(g.c[i], g.c[i + 1]), s = pack_f32x2(g.s[i], g.s[i + 1]);
    const uint64_t ns = pack_f32x2(-g.s[i], -g.s[i + 1]);  // x c - y s = x c + y (-s), rounded alike
    unpack_f32x2(fma_f32x2(mul_f32x2(x, c), one2, mul_f32x2(z, ns)), f[x0], f[x1]);
    unpack_f32x2(fma_f32x2(mul_f32x2(x, s), one2, mul_f32x2(z, c)), f[x0 + y], f[x1 + y]);
  }
}

__device__ __forceinline__ uint2 codes8(const float* f, float inv) {
  uint32_t w[2] = {0, 0};
  const uint64_t inv2 = pack_f32x2(inv, inv);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 y;
    unpack_f32x2(mul_f32x2(pack_f32x2(f[2 * i], f[2 * i + 1]), inv2), y.x, y.y);
    const uint32_t pair = __nv_cvt_float2_to_fp8x2(y, __NV_SATFINITE, __NV_E4M3);
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

// How a warp's rows are split into tokens and heads: row r is token r % tokens of
// head r / tokens.
struct Split {
  int tokens, heads, shift;  // tokens = 1 << shift
};

// Loads the unit's tokens of `split.heads` K (or V) heads from `head0`; `keep`: this lane's shared memory.
template <int LPR, bool INTER, bool IS_K>
__device__ __forceinline__ void load_heads(const AppendParams& p, const Unit& u, const Split& split, int head0, int lane, uint32_t keep) {
  const int j = lane % LPR, row = lane / LPR;
  const int t0 = row & (split.tokens - 1), head = head0 + (row >> split.shift);
  const Run run = make_run<INTER, IS_K>(j, p);
  const int64_t stride = IS_K ? p.k_stride : p.v_stride;
  const uint16_t* src = (IS_K ? p.k : p.v) + static_cast<int64_t>(u.t0) * stride + head * p.D;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int t = i * split.tokens + t0;
    if (t < u.n && run.live && head < p.Hk) {
      cp_async_16(keep + i * kPassBytes, src + t * stride + run.off_a, 16);
      cp_async_16(keep + i * kPassBytes + 512, src + t * stride + run.off_b, 16);
    }
  }
}

// Appends them.
template <int LPR, bool INTER, bool IS_K>
__device__ __forceinline__ void append_heads(const AppendParams& p, const Unit& u, const Split& split, int head0, int lane,
                                             uint32_t keep, uint32_t angles) {
  const int j = lane % LPR, row = lane / LPR;
  const int t0 = row & (split.tokens - 1), head = head0 + (row >> split.shift);
  Run run = make_run<INTER, IS_K>(j, p);
  run.live = run.live && head < p.Hk;
  uint8_t* scale = nullptr;
  uint8_t* codes = nullptr;
  int was = 0;
  if (u.page_id >= 0 && u.page_id < p.cache.num_pages && head < p.Hk) {
    scale = (IS_K ? p.cache.k_scale : p.cache.v_scale) +
            (static_cast<int64_t>(u.page_id) * p.Hk + head) * (p.page / kKvBlock) + u.slot0 / kKvBlock;
    codes = static_cast<uint8_t*>(IS_K ? p.cache.k : p.cache.v) +
            static_cast<int64_t>(u.page_id) * (IS_K ? p.cache.k_page_stride : p.cache.v_page_stride) +
            (static_cast<int64_t>(head) * p.page + u.slot0) * p.D;
    if (u.held > 0) was = min(static_cast<int>(*scale), 254);
  }
  auto value = [&](int i, float (&f)[16]) {
    widen(ld_shared_16(keep + i * kPassBytes), f);
    widen(ld_shared_16(keep + i * kPassBytes + 512), f + 8);
    if (IS_K && run.rotated) {
      const Angles g = load_angles(p, angles, i * split.tokens + t0, j);
      rotate<INTER>(f, g, p.one);
    }
  };
  float amax = 0.f;
#pragma unroll 1
  for (int i = 0; i < kPasses; ++i) {
    const int t = i * split.tokens + t0;
    if (t < u.n && run.live) {
      float f[16];
      value(i, f);
#pragma unroll
      for (int e = 0; e < 16; e += 2) amax = fmaxf(amax, fmaxf(fabsf(f[e]), fabsf(f[e + 1])));
    }
  }
  // over the lanes of a head
  const int span = LPR << split.shift;
#pragma unroll
  for (int x = 1; x < 32; x <<= 1)
    if (x < span) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, x));
  amax = fminf(amax, FLT_MAX);
  int code = amax > 0.f ? min(max(mx_exponent(amax) + 127, 0), 254) : 0;
  if (u.held > 0 && codes) {
    code = max(code, was);
    if (code > was) {
      const float by = exp2_code(max(127 + was - code, 0));
      const int vecs = u.held * p.D / 16;  // a block's rows are contiguous
      for (int i = lane & (span - 1); i < vecs; i += span) {
        uint4* c = reinterpret_cast<uint4*>(codes) + i;
        *c = rescale16(*c, by);
      }
    }
  }
  const float inv = exp2_code(254 - code);
  if (scale && (lane & (span - 1)) == 0) *scale = static_cast<uint8_t>(code);
#pragma unroll 1
  for (int i = 0; i < kPasses; ++i) {
    const int t = i * split.tokens + t0;
    if (t < u.n && run.live) {
      float f[16];
      value(i, f);
      if (IS_K && p.k_out) {
        uint16_t* o = p.k_out + (static_cast<int64_t>(u.t0 + t) * p.Hk + head) * p.D;
        *reinterpret_cast<uint4*>(o + run.off_a) = narrow(f);
        *reinterpret_cast<uint4*>(o + run.off_b) = narrow(f + 8);
      }
      if (codes) {
        uint8_t* o = codes + (u.held + t) * p.D;
        *reinterpret_cast<uint2*>(o + run.off_a) = codes8(f, inv);
        *reinterpret_cast<uint2*>(o + run.off_b) = codes8(f + 8, inv);
      }
    }
  }
}

template <int LPR, bool INTER>
__global__ void __launch_bounds__(kThreads, kCtas) kv_append_kernel(const AppendParams p) {
  __shared__ int4 found;  // sequence, its first row, the row past its last, its tokens in the cache
  __shared__ __align__(16) uint8_t kept[kWarps][2 * kItemBytes];
  __shared__ __align__(16) uint8_t turns[kKvBlock * kAngleRow];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) found.x = -1;
  __syncthreads();
  grid_dep_launch();
  grid_dep_wait();
  // The blocks of positions that new tokens touch, by number: by token, a block belongs to its
  // first one; otherwise sequence b's begin at cu[b] / 16 + 2 b (n tokens touch at
  // most n / 16 + 2 blocks).  Either way the last start at or below gives the sequence; the thread that
  // finds it has read all there is to know of it (one round of loads, not two).
  const int unit = blockIdx.x;
  auto clamp = [&](int c) { return min(max(c, 0), p.T); };
  auto start = [&](int c, int i) { return p.by_token ? c : c / kKvBlock + 2 * i; };
  for (int i = tid; i < p.B; i += kThreads) {
    const int c0 = clamp(__ldg(p.cu + i)), c1 = clamp(__ldg(p.cu + i + 1)), ctx = __ldg(p.ctx + i);
    if (start(c0, i) <= unit && (i + 1 == p.B || unit < start(c1, i + 1))) found = make_int4(i, c0, c1, max(ctx, 0));
  }
  __syncthreads();
  const int b = found.x;
  if (b < 0) return;
  const int first = found.y, last = found.z;
  const int64_t ctx = found.w;
  int64_t block;
  if (p.by_token) {
    if (unit >= last || (unit > first && (ctx + (unit - first)) % kKvBlock != 0)) return;
    block = (ctx + (unit - first)) / kKvBlock;
  } else {
    block = ctx / kKvBlock + (unit - (first / kKvBlock + 2 * b));
  }
  Unit u;
  u.pos = max(ctx, block * kKvBlock);
  const int64_t end = min(ctx + (last - first), (block + 1) * kKvBlock);
  if (u.pos >= end) return;
  u.n = static_cast<int>(end - u.pos);
  u.t0 = first + static_cast<int>(u.pos - ctx);
  u.held = static_cast<int>(u.pos - block * kKvBlock);
  const int64_t at = block * kKvBlock / p.page;
  u.page_id = at < p.table_stride ? __ldg(p.table + b * p.table_stride + at) : -1;
  u.slot0 = static_cast<int>(block * kKvBlock % p.page);

  Split split{kTokens, 32 / LPR / kTokens, 2};
  while (split.tokens > 1 && split.tokens / 2 >= u.n) {
    split.tokens /= 2;
    split.heads *= 2;
    --split.shift;
  }
  const int kv_runs = (p.Hk + split.heads - 1) / split.heads;
  const int head_runs = (p.Hq + split.heads * kHeadPasses - 1) / (split.heads * kHeadPasses);
  const int items = 2 * kv_runs + (u.n + split.tokens - 1) / split.tokens * head_runs;
  const int j = lane % LPR, row = lane / LPR;
  const Run run = make_run<INTER, true>(j, p);
  const uint32_t keep = smem_addr(kept[warp]) + lane * 16;
  // query item qi: this lane's token and first head
  auto query = [&](int qi, int& t, int& h0) {
    t = (qi / head_runs << split.shift) + (row & (split.tokens - 1));
    h0 = (qi % head_runs) * split.heads * kHeadPasses + (row >> split.shift);
    return t < u.n && run.live;
  };
  auto load = [&](int it, uint32_t to) {
    if (it < kv_runs) {
      load_heads<LPR, INTER, true>(p, u, split, it * split.heads, lane, to);
    } else if (it < 2 * kv_runs) {
      load_heads<LPR, INTER, false>(p, u, split, (it - kv_runs) * split.heads, lane, to);
    } else if (int t, h0; it < items && query(it - 2 * kv_runs, t, h0)) {
      const uint16_t* src = p.q + (u.t0 + t) * p.q_stride;
#pragma unroll
      for (int i = 0; i < kHeadPasses; ++i) {
        const int h = h0 + i * split.heads;
        if (h < p.Hq) {
          cp_async_16(to + i * kPassBytes, src + h * p.D + run.off_a, 16);
          cp_async_16(to + i * kPassBytes + 512, src + h * p.D + run.off_b, 16);
        }
      }
    }
    cp_async_commit();
  };
  const int step = gridDim.y * kWarps;
  int it = blockIdx.y * kWarps + warp;
  const uint32_t angles = smem_addr(turns);
  if (p.rot) stage_angles(p, u, angles);
  cp_async_commit();
  load(it, keep);
  cp_async_wait<1>();
  __syncthreads();
  for (uint32_t buf = 0; it < items; it += step, buf ^= kItemBytes) {
    load(it + step, keep + (buf ^ kItemBytes));
    cp_async_wait<1>();  // this lane's own: no other reads them
    if (it < kv_runs) {
      append_heads<LPR, INTER, true>(p, u, split, it * split.heads, lane, keep + buf, angles);
      continue;
    }
    if (it < 2 * kv_runs) {
      append_heads<LPR, INTER, false>(p, u, split, (it - kv_runs) * split.heads, lane, keep + buf, angles);
      continue;
    }
    int t, h0;
    if (!query(it - 2 * kv_runs, t, h0)) continue;
    Angles g;
    if (run.rotated) g = load_angles(p, angles, t, j);
    uint16_t* dst = p.q_out + static_cast<int64_t>(u.t0 + t) * p.Hq * p.D;
#pragma unroll 1
    for (int i = 0; i < kHeadPasses; ++i) {
      const int h = h0 + i * split.heads;
      if (h >= p.Hq) break;
      float f[16];
      widen(ld_shared_16(keep + buf + i * kPassBytes), f);
      widen(ld_shared_16(keep + buf + i * kPassBytes + 512), f + 8);
      if (run.rotated) rotate<INTER>(f, g, p.one);
      *reinterpret_cast<uint4*>(dst + h * p.D + run.off_a) = narrow(f);
      *reinterpret_cast<uint4*>(dst + h * p.D + run.off_b) = narrow(f + 8);
    }
  }
  cp_async_wait_all();  // none is left in flight: the last load is empty
}

template <int LPR>
cudaError_t launch(const cudaLaunchConfig_t* cfg, bool inter, const AppendParams& p) {
  return inter ? cudaLaunchKernelEx(cfg, kv_append_kernel<LPR, true>, p) : cudaLaunchKernelEx(cfg, kv_append_kernel<LPR, false>, p);
}

}  // namespace

sg_status_t append_launch(const AttnShape& s, const AttnArgs& a) {
  AppendParams p{};
  p.cache = a.cache;
  p.rot_table = a.rotary.table;
  p.max_pos = a.rotary.max_pos;
  p.rot = a.rotary.rot;
  p.one = 1.f;
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
  // Numbering by token launches a CTA a token, which is less where most sequences get one or two.
  const int64_t by_block = a.Tq / kKvBlock + 2 * a.B;
  p.by_token = a.Tq <= by_block;
  const unsigned units = static_cast<unsigned>(p.by_token ? a.Tq : by_block);
  // A CTA's warps take one or more items each: of 16 tokens, 2 Hk heads of K and V, and the
  // query heads 8 at a time for as many tokens as a warp holds.  Fewer units than some waves of
  // CTAs are split along the items, down to one a warp.
  const int64_t rows = s.D > 64 ? 4 : 8, heads = p.by_token ? rows : rows / kTokens;
  const int64_t items = 2 * ((s.Hk + heads - 1) / heads) +
                        (p.by_token ? 1 : kKvBlock / kTokens) * ((s.Hq + heads * kHeadPasses - 1) / (heads * kHeadPasses));
  const int64_t want = (p.by_token ? 1 : kWaves) * kCtas * s.num_sms / units, most = (items + kWarps - 1) / kWarps;
  const unsigned split = static_cast<unsigned>(want < 1 ? 1 : want < most ? want : most);
  GemmLaunch l(dim3(units, split), dim3(kThreads), 0, a.stream, 1);
  const bool inter = a.rotary.interleaved != 0;
  const cudaError_t e = s.D > 64 ? launch<8>(&l.cfg, inter, p) : launch<4>(&l.cfg, inter, p);
  if (e != cudaSuccess) {
    note_cuda_error(e);
    cudaGetLastError();
    return SG_ERR_CUDA;
  }
  return SG_OK;
}

}  // namespace sg
