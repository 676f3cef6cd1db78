// sg_attn_decode.cu -- attention of the newest tokens over the paged e4m3 cache
// (scaled_attn_decode).
//
// For a query row x and the keys j it sees, with k_j = 2^a_j K_j and v_j = 2^b_j V_j
// (K, V codes, a, b the exponents of their block),
//     s_j = c x . k_j   (c = scale log2 e),   o = sum_j 2^(s_j) v_j / sum_j 2^(s_j).
// In one pass over tiles of 32 keys, with two references that follow running
// maxima: m for s_j (the denominator's weights 2^(s_j - m)) and n for s_j + b_j (the
// output's weights 2^(s_j + b_j - n), the value scale inside, so that the
// tensor cores multiply codes): o = 2^(n - m) sum_j 2^(s_j + b_j - n) V_j / sum_j 2^(s_j - m).
//
// The bound is memory: every code is read once, 2 D bytes a token and head, and a
// code takes 4 G multiply-adds for G query rows of its head.  Codes become fp16
// exactly (two a instruction), queries are scaled per row by a power of two and
// are then exact in fp16, weights are rounded to fp16 (2^-11 of each), products
// add up in fp32 in mma.sync m16n8k16 with up to 16 query rows of a key/value head as M: bf16
// has no room for them to be the bound.  A warp keeps everything in registers:
//   * the contraction order over dimensions is free, so a lane takes K as it
//     lies: lane (n, c) holds 16-byte runs c (and c + 4) of key n's row, four dimensions a k-step;
//   * the order of keys is free too: the keys whose weights the score tile leaves in a
//     lane are the ones whose V rows it reads, 16 bytes each; interleaving pairs of rows by
//     bytes gives the operand of one output tile per dimension.
// Rows lie in shared memory with the TMA swizzle; which key and run a lane takes
// is chosen so that these reads have no bank conflicts.
//
// Work: all tiles of all (sequence, head) segments are numbered, every warp takes
// the same number of consecutive ones (lengths are on the device; each CTA sums them up),
// loaded into its own ring by TMA ahead of use, across segments.  A segment inside a warp's range is
// finished there; a segment cut by ranges leaves partial sums, which a second kernel
// joins in the order of the ranges, so results do not depend on timing.
#include <cuda.h>
#include <cuda_runtime.h>

#include "sg_attn.h"
#include "sg_attn_ptx.cuh"
#include "sg_mx.cuh"

namespace sg {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kKeys = 32;       // keys of a tile
constexpr int kRowTile = 16;    // query rows of an MMA
constexpr int kMinTiles = 2;    // least tiles of a warp's range
constexpr float kSlack = 8.f;   // log2 of the largest output weight

struct Segment {  // a segment cut by ranges: the range that starts it joins it
  int32_t b, hr;        // sequence; head * row tiles + row tile; b < 0: none
  int32_t last;         // the last range with a part of it
  int32_t pad;
};

struct DecodeParams {
  const uint16_t* q;
  int64_t q_stride;
  const int32_t *table, *lens;
  int64_t table_stride;
  const uint8_t *k_scale, *v_scale;
  int64_t num_pages;
  int B, qn, Hq, Hk, D, page, group, row_tiles;
  float scale_log2;
  uint16_t* out;
  float* lse;
  float* part_o;      // [2 ranges][16][HD]
  float4* part_ml;    // [2 ranges][16]: m, n, sum
  Segment* cut;       // [ranges]
  int* status;
  uint64_t timeout_ns;
};

template <int HD>
struct DecodeLayout {
  static constexpr int kTile = kKeys * HD;               // bytes of a K or V tile
  static constexpr int kStages = HD == 128 ? 3 : 6;
  static constexpr int kRing = 2 * kTile * kStages;      // a warp's ring
  static constexpr int kOffInfo = kWarps * kRing;        // uint2 per warp and stage
  static constexpr int kOffBar = kOffInfo + kWarps * kStages * 8;
  static constexpr int kOffSum = kOffBar + kWarps * kStages * 8;  // int64 per thread
  static constexpr int kOffMisc = kOffSum + (kThreads + 1) * 8;
  static constexpr int kBytes = kOffMisc + 16 + 8 * kWarps;
  static constexpr int kDynSmem = kBytes + 1024;
  static_assert(kDynSmem <= 232448, "shared memory");
};

// Key row (of 8) that lane group n takes in a score tile.
template <int HD>
__device__ __forceinline__ int key_row(int n) {
  return HD == 128 ? (n >> 1) | ((n & 1) << 2) : n ^ ((n >> 1) & 1);
}

// Address of 16-byte run `run` of row `row` of a swizzled tile.
template <int HD>
__device__ __forceinline__ uint32_t run_addr(uint32_t tile, int row, int run) {
  return HD == 128 ? tile + row * 128 + ((run ^ (row & 7)) << 4) : tile + row * 64 + ((run ^ ((row >> 1) & 3)) << 4);
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ uint2 ld_shared_v2(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

// Two e4m3 codes (low 16 bits) as fp16.
__device__ __forceinline__ uint32_t codes_f16x2(uint32_t two) {
  uint32_t d;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<uint16_t>(two)));
  return d;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void mma_16x8x16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A position in the numbered tiles: tile t of the segment (b, hr), which has `tiles`.
struct Cursor {
  int b, hr, t, tiles, len;
};

struct Walk {
  const DecodeParams& p;
  int segs;  // segments of a sequence
  __device__ __forceinline__ int len(int b) const {
    const int64_t cap = p.table_stride * p.page;  // below 2^31
    return static_cast<int>(min(static_cast<int64_t>(max(__ldg(p.lens + b), 0)), cap));
  }
  __device__ __forceinline__ int tiles(int len) const { return (len + kKeys - 1) / kKeys; }
  __device__ __forceinline__ void load(Cursor& c) const {  // skips empty sequences
    while (c.b < p.B) {
      c.len = len(c.b);
      c.tiles = tiles(c.len);
      if (c.tiles > 0) return;
      ++c.b;
    }
  }
  __device__ __forceinline__ void next(Cursor& c) const {
    if (++c.t < c.tiles) return;
    c.t = 0;
    if (++c.hr < segs) return;
    c.hr = 0;
    ++c.b;
    load(c);
  }
};

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const DecodeParams p) {
  using L = DecodeLayout<HD>;
  constexpr int S = L::kStages;
  constexpr int kRuns = HD / 64;        // 16-byte runs of a key row in a lane
  constexpr int kOut = HD / 8;          // output tiles
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = smem_addr(smem + warp * L::kRing);
  const uint32_t info = smem_addr(smem + L::kOffInfo) + warp * S * 8;
  const uint32_t bars = smem_addr(smem + L::kOffBar) + warp * S * 8;
  int64_t* sums = reinterpret_cast<int64_t*>(smem + L::kOffSum);
  int* misc = reinterpret_cast<int*>(smem + L::kOffMisc);
  int64_t* warp_sums = reinterpret_cast<int64_t*>(smem + L::kOffMisc + 16);
  if (tid == 0) misc[0] = 0;
  if (lane == 0)
    for (int s = 0; s < S; ++s) mbar_init(bars + 8 * s, 1);
  if (tid == 0) fence_mbarrier_init();
  grid_dep_launch();
  grid_dep_wait();

  // Tiles before each run of `per` sequences, and in all.
  const Walk walk{p, p.Hk * p.row_tiles};
  const int per = (p.B + kThreads - 1) / kThreads;
  int64_t mine = 0;
  for (int i = tid * per; i < min((tid + 1) * per, p.B); ++i) mine += walk.tiles(walk.len(i));
  int64_t scan = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += up;
  }
  if (lane == 31) warp_sums[warp] = scan;
  __syncthreads();
  int64_t base = 0;
  for (int w = 0; w < warp; ++w) base += warp_sums[w];
  sums[tid + 1] = (base + scan) * walk.segs;
  if (tid == 0) sums[0] = 0;
  __syncthreads();
  const int64_t total = sums[kThreads];

  // sequences with nothing to see
  for (int b = blockIdx.x; b < p.B; b += gridDim.x)
    if (walk.len(b) == 0) {
      const int64_t n = static_cast<int64_t>(p.qn) * p.Hq;
      for (int64_t i = tid; i < n * p.D / 8; i += kThreads)
        reinterpret_cast<uint4*>(p.out + b * n * p.D)[i] = make_uint4(0, 0, 0, 0);
      if (p.lse)
        for (int64_t i = tid; i < n; i += kThreads) p.lse[b * n + i] = -INFINITY;
    }

  // this warp's range of tiles; neighbouring ranges on different SMs
  const int ranges = gridDim.x * kWarps;
  const int range = warp * gridDim.x + blockIdx.x;
  const int64_t quota = max((total + ranges - 1) / ranges, static_cast<int64_t>(kMinTiles));
  const int64_t begin = min(range * quota, total), end = min(begin + quota, total);
  if (lane == 0) p.cut[range].b = -1;
  if (begin >= end) return;

  Cursor c{};  // the tile to compute
  int64_t seg_begin;  // number of its segment's first tile
  {
    int lo = 0, hi = kThreads;  // the run of sequences: sums[lo] <= begin < sums[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (sums[mid] <= begin) lo = mid; else hi = mid;
    }
    int64_t at = sums[lo];
    c.b = lo * per;
    for (;;) {
      c.len = walk.len(c.b);
      c.tiles = walk.tiles(c.len);
      const int64_t n = static_cast<int64_t>(c.tiles) * walk.segs;
      if (begin < at + n) break;
      at += n;
      ++c.b;
    }
    const int64_t in = begin - at;
    c.hr = static_cast<int>(in / c.tiles);
    c.t = static_cast<int>(in % c.tiles);
    seg_begin = begin - c.t;
  }
  Cursor ahead = c;  // the tile to load
  int64_t loaded = begin;
  const Watchdog wd{p.status, p.timeout_ns, reinterpret_cast<volatile int*>(&misc[0])};
  const uint64_t policy = l2_policy_evict_first();
  const int blocks_page = p.page / kKvBlock;

  // Pages and scales of 32 tiles of the segment being loaded, a tile a lane.
  int batch = -1;                    // its first tile; -1: none
  int page0 = -1, page1 = -1;
  uint32_t scales = 0;               // k block 0, k block 1, v block 0, v block 1
  auto refresh = [&]() {
    batch = ahead.t;
    const int h = ahead.hr / p.row_tiles;
    const int key = (ahead.t + lane) * kKeys;
    const int32_t* row = p.table + ahead.b * p.table_stride;
    auto page_of = [&](int k) {
      if (k >= ahead.len) return -1;
      const int pg = __ldg(row + k / p.page);
      return pg >= 0 && pg < p.num_pages ? pg : -1;
    };
    page0 = page_of(key);
    page1 = p.page == 16 ? page_of(key + 16) : page0;
    scales = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int pg = i ? page1 : page0;
      if (pg >= 0) {
        const int64_t at = (static_cast<int64_t>(pg) * p.Hk + h) * blocks_page + (key + 16 * i) % p.page / kKvBlock;
        scales |= static_cast<uint32_t>(__ldg(p.k_scale + at)) << (8 * i) | static_cast<uint32_t>(__ldg(p.v_scale + at)) << (16 + 8 * i);
      }
    }
  };
  auto load = [&](int stage) {  // the tile at `ahead` into `stage`
    if (batch < 0 || ahead.t >= batch + 32) refresh();
    const int from = ahead.t - batch;
    const int pg0 = __shfl_sync(0xffffffffu, page0, from), pg1 = __shfl_sync(0xffffffffu, page1, from);
    const uint32_t sc = __shfl_sync(0xffffffffu, scales, from);
    if (lane == 0) {
      const uint32_t gone = (pg0 < 0 ? 1u : 0u) | (pg1 < 0 ? 2u : 0u);
      asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(info + 8 * stage), "r"(sc), "r"(gone) : "memory");
      const uint32_t bar = bars + 8 * stage, k = ring + 2 * stage * L::kTile, v = k + L::kTile;
      const int row = ahead.hr / p.row_tiles * p.page + ahead.t * kKeys % p.page;
      mbar_arrive_expect_tx(bar, 2 * L::kTile);
      tma_load_3d_hint(k, &tmK, 0, row, pg0, bar, policy);
      tma_load_3d_hint(v, &tmV, 0, row, pg0, bar, policy);
      if (p.page == 16) {
        tma_load_3d_hint(k + L::kTile / 2, &tmK, 0, row, pg1, bar, policy);
        tma_load_3d_hint(v + L::kTile / 2, &tmV, 0, row, pg1, bar, policy);
      }
    }
    const int b = ahead.b, hr = ahead.hr;
    walk.next(ahead);
    if (ahead.b != b || ahead.hr != hr) batch = -1;
    ++loaded;
  };
  int in_flight = 0;  // stages loaded and not yet consumed
  for (int s = 0; s < S && loaded < end; ++s, ++in_flight) load(s);

  const int n8 = lane >> 2, c4 = lane & 3;
  const int kr = key_row<HD>(n8), kv0 = key_row<HD>(2 * c4), kv1 = key_row<HD>(2 * c4 + 1);
  int stage = 0;
  uint32_t phase = 0;
  bool ok = true;
  int64_t tile = begin;
  while (tile < end && ok) {
    // ---- a segment, or the part of it in this range
    const int h = c.hr / p.row_tiles, rt = c.hr % p.row_tiles;
    const int part_first = c.t;
    const int part_tiles = static_cast<int>(min(static_cast<int64_t>(c.tiles - c.t), end - tile));
    uint32_t qf[4 * kRuns][4];
    float q_scale[2];
    int lim[2];      // keys that rows n8 and n8 + 8 see
    int64_t row_at[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = rt * kRowTile + n8 + 8 * r;
      const bool live = row < p.qn * p.group;
      const int qi = live ? row / p.group : 0;
      row_at[r] = live ? (static_cast<int64_t>(c.b) * p.qn + qi) * p.Hq + h * p.group + row % p.group : -1;
      lim[r] = live ? c.len - (p.qn - 1 - qi) : 0;
      uint4 w[2 * kRuns];
      float top = 0.f;
#pragma unroll
      for (int u = 0; u < kRuns; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int d = 64 * u + 16 * c4 + 8 * i;
          w[2 * u + i] = make_uint4(0, 0, 0, 0);
          if (live && d < p.D)
            w[2 * u + i] = *reinterpret_cast<const uint4*>(p.q + (static_cast<int64_t>(c.b) * p.qn + qi) * p.q_stride +
                                                           (h * p.group + row % p.group) * p.D + d);
        }
      auto lo = [](uint32_t x) { return __uint_as_float(x << 16); };
      auto hi = [](uint32_t x) { return __uint_as_float(x & 0xFFFF0000u); };
#pragma unroll
      for (int i = 0; i < 2 * kRuns; ++i) {
        const uint32_t x[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = fmaxf(top, fmaxf(fabsf(lo(x[e])), fabsf(hi(x[e]))));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // the row's largest value to [2^14, 2^15): then its bf16 values are exact in
      // fp16 down to 2^-38 of it
      const int field = min(268 - static_cast<int>(__float_as_uint(top) >> 23), 253);
      const float up = __uint_as_float(static_cast<uint32_t>(field) << 23);
      q_scale[r] = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(254 - field) << 23);
      // k-step 4 u + i: this lane's dimensions 64 u + 16 c + 4 i ..+3
#pragma unroll
      for (int u = 0; u < kRuns; ++u)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4& q4 = w[2 * u + i / 2];
          const uint32_t x = (i & 1) ? q4.z : q4.x, y = (i & 1) ? q4.w : q4.y;
          qf[4 * u + i][r] = pack_f16x2(lo(x) * up, hi(x) * up);
          qf[4 * u + i][2 + r] = pack_f16x2(lo(y) * up, hi(y) * up);
        }
    }
    float o[kOut][4];
#pragma unroll
    for (int i = 0; i < kOut; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, n[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};

    for (int pt = 0; pt < part_tiles; ++pt) {
      ok = __all_sync(0xffffffffu, mbar_wait(bars + 8 * stage, phase, wd, kWhereMmaFull));
      if (!ok) break;
      const uint32_t sk = ring + 2 * stage * L::kTile, sv = sk + L::kTile;
      const uint2 about = ld_shared_v2(info + 8 * stage);
      const int key0 = (part_first + pt) * kKeys;
      // scores
      float s[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][e] = 0.f;
#pragma unroll
        for (int u = 0; u < kRuns; ++u) {
          const uint4 k = ld_shared_v4(run_addr<HD>(sk, 8 * i + kr, c4 + 4 * u));
          const uint32_t w[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
          for (int x = 0; x < 4; ++x) mma_16x8x16(s[i], qf[4 * u + x], codes_f16x2(w[x]), codes_f16x2(w[x] >> 16));
        }
      }
      float kx[2], vx[2];  // key scales, value exponents of the two blocks
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int kc = (about.x >> (8 * i)) & 255, vc = (about.x >> (16 + 8 * i)) & 255;
        kx[i] = kc == 255 ? __uint_as_float(0x7FC00000u) : exp2_code(kc);
        vx[i] = vc == 255 ? __uint_as_float(0x7FC00000u) : static_cast<float>(vc - 127);
      }
      const bool edge = key0 + kKeys > c.len - (p.qn - 1) || about.y != 0;
      float ms[2] = {-INFINITY, -INFINITY}, mn[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int r = e >> 1;
          float x = s[i][e] * (kx[i >> 1] * q_scale[r]);
          if (edge) {
            const int key = key0 + 8 * i + ((e & 1) ? kv1 : kv0);
            if (key >= lim[r] || ((about.y >> (i >> 1)) & 1)) x = -INFINITY;
          }
          s[i][e] = x;
          ms[r] = fmaxf(ms[r], x);
          mn[r] = fmaxf(mn[r], x + vx[i >> 1]);
        }
      }
      bool move = false;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        ms[r] = fmaxf(ms[r], __shfl_xor_sync(0xffffffffu, ms[r], 1));
        mn[r] = fmaxf(mn[r], __shfl_xor_sync(0xffffffffu, mn[r], 1));
        ms[r] = fmaxf(ms[r], __shfl_xor_sync(0xffffffffu, ms[r], 2));
        mn[r] = fmaxf(mn[r], __shfl_xor_sync(0xffffffffu, mn[r], 2));
        if (ms[r] > m[r]) {
          sum[r] *= ex2(m[r] - ms[r]);
          m[r] = ms[r];
        }
        move |= mn[r] > n[r] + kSlack;
      }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (mn[r] > n[r] + kSlack) {
            const float by = ex2(n[r] - mn[r]);
            n[r] = mn[r];
#pragma unroll
            for (int i = 0; i < kOut; ++i) {
              o[i][2 * r] *= by;
              o[i][2 * r + 1] *= by;
            }
          }
      }
      // weights
      float neg_m[2], neg_n[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        neg_m[r] = m[r] == -INFINITY ? 0.f : -m[r];
        neg_n[r] = n[r] == -INFINITY ? 0.f : -n[r];
      }
      uint32_t w[4][2];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float x = s[i][2 * r], y = s[i][2 * r + 1];
          sum[r] += ex2(x + neg_m[r]) + ex2(y + neg_m[r]);
          const float by = vx[i >> 1] + neg_n[r];
          w[i][r] = pack_f16x2(ex2(x + by), ex2(y + by));
        }
      // output += weights times codes, 16 keys at a time
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const uint32_t a[4] = {w[2 * g][0], w[2 * g][1], w[2 * g + 1][0], w[2 * g + 1][1]};
        uint32_t v[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 16 * g + 8 * (i >> 1) + ((i & 1) ? kv1 : kv0);
          if constexpr (HD == 128) {
            const uint4 x = ld_shared_v4(run_addr<HD>(sv, row, key_row<HD>(n8)));
            v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
          } else {
            const uint2 x = ld_shared_v2(run_addr<HD>(sv, row, n8 >> 1) + 8 * (n8 & 1));
            v[i][0] = x.x, v[i][1] = x.y;
          }
          if (edge && key0 + row >= c.len) {  // stale codes may be NaN
#pragma unroll
            for (int e = 0; e < HD / 32; ++e) v[i][e] = 0;
          }
        }
#pragma unroll
        for (int e = 0; e < HD / 32; ++e) {
          const uint32_t x0 = __byte_perm(v[0][e], v[1][e], 0x5140), x1 = __byte_perm(v[0][e], v[1][e], 0x7362);
          const uint32_t y0 = __byte_perm(v[2][e], v[3][e], 0x5140), y1 = __byte_perm(v[2][e], v[3][e], 0x7362);
          mma_16x8x16(o[4 * e], a, codes_f16x2(x0), codes_f16x2(y0));
          mma_16x8x16(o[4 * e + 1], a, codes_f16x2(x0 >> 16), codes_f16x2(y0 >> 16));
          mma_16x8x16(o[4 * e + 2], a, codes_f16x2(x1), codes_f16x2(y1));
          mma_16x8x16(o[4 * e + 3], a, codes_f16x2(x1 >> 16), codes_f16x2(y1 >> 16));
        }
      }
      __syncwarp();  // every lane has read the stage
      --in_flight;
      if (loaded < end) {
        load(stage);
        ++in_flight;
      }
      if (++stage == S) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (!ok) break;

    // ---- the segment's end, or the range's
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
      sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
    }
    const bool whole = part_tiles == c.tiles;
    const int slot = 2 * range + (part_first == 0);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      if (row_at[r] < 0) continue;
      if (whole) {
        const bool none = sum[r] == 0.f;
        const float by = none ? 0.f : ex2(n[r] - m[r]) / sum[r];
        uint16_t* dst = p.out + row_at[r] * p.D;
        // this lane's dimensions: two runs of kOut from output columns 2 c and 2 c + 1
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int d0 = HD == 128 ? 64 * half + 16 * c4 : 16 * c4 + 8 * half;
          if (d0 < p.D) {
#pragma unroll
            for (int i = 0; i < kOut; i += 8) {
              uint32_t u[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float x = o[i + 2 * e][2 * r + half], y = o[i + 2 * e + 1][2 * r + half];
                u[e] = none ? 0u : pack_bf16x2(x * by, y * by);
              }
              *reinterpret_cast<uint4*>(dst + d0 + i) = make_uint4(u[0], u[1], u[2], u[3]);
            }
          }
        }
        if (c4 == 0 && p.lse) p.lse[row_at[r]] = none ? -INFINITY : (m[r] + log2f(sum[r])) * 0.6931471805599453f;
      } else {
        const int64_t at = static_cast<int64_t>(slot) * kRowTile + n8 + 8 * r;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int d0 = HD == 128 ? 64 * half + 16 * c4 : 16 * c4 + 8 * half;
#pragma unroll
          for (int i = 0; i < kOut; i += 4)
            *reinterpret_cast<float4*>(p.part_o + at * HD + d0 + i) =
                make_float4(o[i][2 * r + half], o[i + 1][2 * r + half], o[i + 2][2 * r + half], o[i + 3][2 * r + half]);
        }
        if (c4 == 0) p.part_ml[at] = make_float4(m[r], n[r], sum[r], 0.f);
      }
    }
    if (!whole && part_first == 0 && lane == 0)
      p.cut[range] = Segment{c.b, c.hr, static_cast<int32_t>((seg_begin + c.tiles - 1) / quota), 0};
    tile += part_tiles;
    seg_begin = tile;
    c.t += part_tiles - 1;
    walk.next(c);
  }
  if (!ok) {  // loads in flight must land before the CTA can exit
    for (int i = 0; i < in_flight; ++i) {
      if (lane == 0) mbar_wait_drain(bars + 8 * stage, phase, 200000000ull);
      if (++stage == S) {
        stage = 0;
        phase ^= 1;
      }
    }
    __syncwarp();
  }
}

// Joins the parts of the segment that range blockIdx.x starts and later ones continue.
template <int HD>
__global__ void __launch_bounds__(256) decode_join_kernel(const DecodeParams p) {
  grid_dep_launch();
  grid_dep_wait();
  const int first = blockIdx.x;
  const Segment s = p.cut[first];
  if (s.b < 0) return;
  const int h = s.hr / p.row_tiles, rt = s.hr % p.row_tiles;
  const int rows = min(kRowTile, p.qn * p.group - rt * kRowTile);
  constexpr int kQuads = HD / 4;
  auto slot = [&](int i) { return static_cast<int64_t>(2 * i + (i == first)) * kRowTile; };
  for (int i = threadIdx.x; i < rows * kQuads; i += 256) {
    const int row = i / kQuads, d = i % kQuads * 4;
    float m = -INFINITY, n = -INFINITY;
#pragma unroll 4
    for (int k = first; k <= s.last; ++k) {
      const float4 ml = p.part_ml[slot(k) + row];
      m = fmaxf(m, ml.x);
      n = fmaxf(n, ml.y);
    }
    const float neg_m = m == -INFINITY ? 0.f : -m, neg_n = n == -INFINITY ? 0.f : -n;
    float sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int k = first; k <= s.last; ++k) {
      const float4 ml = p.part_ml[slot(k) + row];
      const float4 x = *reinterpret_cast<const float4*>(p.part_o + (slot(k) + row) * HD + d);
      sum += ml.z * ex2(ml.x + neg_m);
      const float by = ex2(ml.y + neg_n);
      o[0] += x.x * by;
      o[1] += x.y * by;
      o[2] += x.z * by;
      o[3] += x.w * by;
    }
    const bool none = sum == 0.f;
    const float by = none ? 0.f : ex2(-neg_n + neg_m) / sum;
    const int r = rt * kRowTile + row;
    const int64_t at = (static_cast<int64_t>(s.b) * p.qn + r / p.group) * p.Hq + h * p.group + r % p.group;
    if (d < p.D)
      *reinterpret_cast<uint2*>(p.out + at * p.D + d) =
          none ? make_uint2(0, 0) : make_uint2(pack_bf16x2(o[0] * by, o[1] * by), pack_bf16x2(o[2] * by, o[3] * by));
    if (d == 0 && p.lse) p.lse[at] = none ? -INFINITY : (-neg_m + log2f(sum)) * 0.6931471805599453f;
  }
}

sg_status_t launch_error(cudaError_t e) {
  if (e == cudaSuccess) return SG_OK;
  note_cuda_error(e);
  cudaGetLastError();  // clear the non-sticky launch error
  return SG_ERR_CUDA;
}

int num_ranges(const AttnShape& s) { return s.num_sms * kWarps; }

template <int HD>
sg_status_t launch(const AttnShape& s, const AttnArgs& a, DecodeParams& p) {
  const uint64_t D = s.D, rows = static_cast<uint64_t>(s.Hk) * s.page;
  const uint64_t dims[3] = {D, rows, static_cast<uint64_t>(a.cache.num_pages)};
  const uint64_t sk[2] = {D, static_cast<uint64_t>(a.cache.k_page_stride)}, sv[2] = {D, static_cast<uint64_t>(a.cache.v_page_stride)};
  const uint32_t box[3] = {HD, static_cast<uint32_t>(s.page < kKeys ? s.page : kKeys), 1};
  const CUtensorMapSwizzle sw = HD == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  CUtensorMap tmK, tmV;
  if (!encode_3d(&tmK, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.cache.k, dims, sk, box, sw) ||
      !encode_3d(&tmV, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.cache.v, dims, sv, box, sw))
    return SG_ERR_CUDA;
  p.part_o = static_cast<float*>(s.workspace);
  p.part_ml = reinterpret_cast<float4*>(p.part_o + static_cast<size_t>(2) * num_ranges(s) * kRowTile * 128);
  p.cut = reinterpret_cast<Segment*>(p.part_ml + static_cast<size_t>(2) * num_ranges(s) * kRowTile);
  GemmLaunch l(dim3(s.num_sms), dim3(kThreads), DecodeLayout<HD>::kDynSmem, a.stream, 1);
  const sg_status_t r = launch_error(cudaLaunchKernelEx(&l.cfg, decode_kernel<HD>, tmK, tmV, p));
  if (r != SG_OK) return r;
  GemmLaunch j(dim3(num_ranges(s)), dim3(256), 0, a.stream, 1);
  return launch_error(cudaLaunchKernelEx(&j.cfg, decode_join_kernel<HD>, p));
}

}  // namespace

size_t decode_workspace_bytes(const AttnShape& s) {
  return static_cast<size_t>(2) * num_ranges(s) * kRowTile * (128 * 4 + 16) + static_cast<size_t>(num_ranges(s)) * sizeof(Segment);
}

cudaError_t decode_prepare() {
  const cudaError_t e = cudaFuncSetAttribute(decode_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize, DecodeLayout<64>::kDynSmem);
  return e == cudaSuccess
             ? cudaFuncSetAttribute(decode_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize, DecodeLayout<128>::kDynSmem)
             : e;
}

sg_status_t decode_launch(const AttnShape& s, const AttnArgs& a) {
  DecodeParams p{};
  p.q = static_cast<const uint16_t*>(a.q);
  p.q_stride = a.q_stride;
  p.table = a.table;
  p.lens = a.lens;
  p.table_stride = a.cache.num_pages > 0 ? a.table_stride : 0;  // no page, no keys
  p.k_scale = a.cache.k_scale;
  p.v_scale = a.cache.v_scale;
  p.num_pages = a.cache.num_pages;
  p.B = static_cast<int>(a.B);
  p.qn = static_cast<int>(a.qn);
  p.Hq = s.Hq;
  p.Hk = s.Hk;
  p.D = s.D;
  p.page = s.page;
  p.group = s.Hq / s.Hk;
  p.row_tiles = (p.qn * p.group + kRowTile - 1) / kRowTile;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  p.status = s.status;
  p.timeout_ns = s.timeout_ns;
  AttnArgs args = a;
  if (args.cache.num_pages == 0) args.cache.num_pages = 1;  // a tensor map has no empty dimension; nothing reads it
  return s.D > 64 ? launch<128>(s, args, p) : launch<64>(s, args, p);
}

}  // namespace sg
