// sg_attn_decode.cu -- attention of the newest tokens over the paged e4m3 cache
// (scaled_attn_decode).
//
// For a query row x and the keys j it sees, with k_j = 2^a_j K_j and v_j = 2^b_j V_j
// (K, V codes, a, b the exponents of their block),
//     s_j = c x . k_j   (c = scale log2 e),   o = sum_j 2^(s_j) v_j / sum_j 2^(s_j).
// In one pass over tiles of 32 keys, with two references that follow running
// maxima: m for s_j (the denominator's weights 2^(s_j - m)) and m + n for s_j + b_j (the
// output's weights 2^((s_j - m) + b_j - n), the value scale inside, so that the
// tensor cores multiply codes): o = 2^n sum_j 2^((s_j - m) + b_j - n) V_j / sum_j 2^(s_j - m).
// n is held relative to m, and s_j - m is formed first: beside a score of 2^24 or more b_j would be lost.
//
// The bound is memory: every code is read once, 2 D bytes a token and head.  What
// competes with it is the arithmetic on codes, so a warp does as little of it as it can, in registers:
//   * Products add up in fp32 in mma.sync with keys (or dimensions) as its M and the query rows of
//     a key/value head, 8 a tile, as its N: groups of up to 8 rows leave nothing idle but unused columns.
//     Codes become fp16 exactly (two a conversion); queries are scaled per row by a power of two and are then exact in
//     fp16; weights are rounded to fp16 (2^-11 of each, 2^-32 of the largest for those below 2^-21 of it).  (mma.sync on e4m3 operands measured slower: it
//     converts them too, and a query takes two terms.)
//   * The contraction order over dimensions is free, so a lane takes K as it
//     lies: lane (g, c) holds 16-byte runs c (and c + 4) of keys g and g + 8, four dimensions a k-step.
//   * The order of keys is free too: an 8 x 8 transpose (movmatrix) leaves lane (g, c) the weights
//     of row g and keys 2 c, 2 c + 1; it reads those keys' V rows, 16 bytes each, and
//     interleaving pairs of rows by bytes gives the operand of two dimensions.
//   * References move only when a maximum has passed them by 2^8, found by one vote a tile.
// Rows lie in shared memory with the TMA swizzle; which key and run a lane takes
// is chosen so that these reads have no bank conflicts.
//
// Work: all tiles of all (sequence, head) segments are numbered, with an allowance for each
// segment's own cost, and every warp takes an equal range of the numbers (lengths are on
// the device; each CTA sums them up), loaded into its own ring by TMA ahead of use, across
// segments.  Segments that are short beside a range are not cut; the parts of a cut one are joined
// by a second kernel in the order of its ranges, so results do not depend on timing.
// Measured, main kernel and join: 64 sequences of up to 16k tokens, 32 heads of 128 over 8: 98 us (the join 4; the
// main kernel at 92% of a copy's rate); 2 long ones 90 (6); 200 sequences with 4 drafted tokens, 16 heads of 64 over 16:
// 60 (5; 62% of the issue slots, DRAM at 59%: 64-wide heads have as many weights to make for half the bytes); one of 777 tokens
// 8.7.  With 16 query rows a key/value head (128 heads over 8, or 4 drafted tokens of 32 over 8) the 64 sequences take 118:
// 255 registers leave two warps a scheduler, which wait for one another's results (issue 46%, DRAM 64%).
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cfloat>

#include "sg_attn.h"
#include "sg_attn_ptx.cuh"
#include "sg_mx.cuh"

namespace sg {

namespace {

constexpr int kKeys = 32;       // keys of a tile
constexpr int kSegCost = 3;     // what a segment costs beside its tiles, in tiles
constexpr int kUncut = 10;      // segments of up to 1 / kUncut of a range are not cut (250 sequences of 20 to 1500 tokens, 16
                                // heads of 128 over 2, two tokens each: 27.8 us, 31.7 with 4, 32.6 with 2)
constexpr int kMaxWarps = 16;
constexpr int kJoinWarps = 8;
constexpr int kFirst = 4;
constexpr float kSlack = 8.f;   // log2 of how far a maximum may pass its reference
constexpr float kUnset = -FLT_MAX;  // references before a row has seen a key: finite, so that differences with them are
constexpr float kLift = 7.f;    // the output's weights at its reference are 2^kLift, the largest 2^15: the room that
                                // fp16 has above 1 keeps light weights among its normal numbers, down to 2^-21

// What the join kernel does for a segment (or range): ranges first .. last have parts of
// segment (b, hr); last < 0: nothing.
struct Cut {
  int b, hr, first, last;
};

struct DecodeParams {
  const uint16_t* q;
  int64_t q_stride;
  const int32_t *table, *lens;
  int64_t table_stride;
  const uint8_t *k_scale, *v_scale;
  int64_t num_pages;
  int B, qn, Hq, Hk, D, page, page_shift, group, row_tiles;
  float scale_log2;
  uint16_t* out;
  float* lse;
  float* part_o;      // [2 ranges][rows][HD]: the part that begins a segment (odd), one that does not
  float4* part_ml;    // [2 ranges][rows]: m, n (relative to m), sum
  Cut* cuts;          // by segment, or by range where there are fewer of those
  int by_segment;
  int skip;           // number of a tile that is not loaded (scaled_attn_set_debug); -1: none
  int* status;
  uint64_t timeout_ns;
};

// NR: tiles of 8 query rows.
template <int HD, int NR>
struct DecodeLayout {
  static constexpr int kWarps = HD == 128 ? (NR == 1 ? 12 : 8) : (NR == 1 ? 16 : 12);
  static constexpr int kThreads = 32 * kWarps;
  static constexpr int kTile = kKeys * HD;               // bytes of a K or V tile
  static constexpr int kStages = 196608 / (2 * kTile * kWarps);
  static constexpr int kRing = 2 * kTile * kStages;      // a warp's ring
  static constexpr int kOffInfo = kWarps * kRing;        // uint2 per warp and stage
  static constexpr int kOffBar = kOffInfo + kWarps * kStages * 8;
  static constexpr int kOffSum = kOffBar + kWarps * kStages * 8;  // int64 per thread
  static constexpr int kOffMisc = kOffSum + (kThreads + 1) * 8;
  static constexpr int kBytes = kOffMisc + 16 + 8 * kWarps;
  static constexpr int kDynSmem = kBytes + 1024;
  static_assert(kDynSmem <= 232448 && kWarps <= kMaxWarps, "shared memory");
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

// Four e4m3 codes as two pairs of fp16.
__device__ __forceinline__ void codes_f16(uint32_t four, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}

// Transpose of an 8 x 8 matrix of 16-bit elements, two a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void mma_16x8x16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// a / b for a >= 0, b > 0, in 32 bits where they fit.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// Tiles [t, t1) of segment (b, hr), whose numbers start at `start`.
struct Part {
  int b, hr, t, t1, tiles, len;
  int64_t start;
};

// The parts of a range [begin, end) of numbers: segment after segment, kSegCost
// numbers and then one a tile; uncut segments belong to the range of their start.
struct Walk {
  const DecodeParams& p;
  int segs;  // segments of a sequence
  int64_t begin, end;
  int uncut;
  __device__ __forceinline__ int len(int b) const {
    const int64_t cap = p.table_stride * p.page;  // below 2^31
    return static_cast<int>(min(static_cast<int64_t>(max(__ldg(p.lens + b), 0)), cap));
  }
  __device__ __forceinline__ static int tiles(int len) { return static_cast<int>((static_cast<uint32_t>(len) + kKeys - 1) / kKeys); }
  __device__ __forceinline__ static int64_t numbers(int len) { return len > 0 ? tiles(len) + kSegCost : 0; }
  // The first part at or after segment c; false: none.
  __device__ __forceinline__ bool find(Part& c) const {
    while (c.start < end) {
      if (c.hr == segs) {
        c.hr = 0;
        do {
          if (++c.b >= p.B) return false;
          c.len = len(c.b);
        } while (c.len == 0);
        c.tiles = tiles(c.len);
      }
      if (c.tiles <= uncut) {
        c.t = 0;
        c.t1 = c.start >= begin ? c.tiles : 0;
      } else {
        const int64_t first = c.start + kSegCost;
        c.t = static_cast<int>(max(begin - first, static_cast<int64_t>(0)));
        c.t1 = static_cast<int>(min(end - first, static_cast<int64_t>(c.tiles)));
      }
      if (c.t < c.t1) return true;
      c.start += c.tiles + kSegCost;
      ++c.hr;
    }
    return false;
  }
  __device__ __forceinline__ bool next(Part& c) const {
    c.start += c.tiles + kSegCost;
    ++c.hr;
    return find(c);
  }
};

template <int HD, int NR>
__global__ void __launch_bounds__(DecodeLayout<HD, NR>::kThreads, 1)
    decode_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const DecodeParams p) {
  using L = DecodeLayout<HD, NR>;
  constexpr int S = L::kStages, kWarps = L::kWarps, kThreads = L::kThreads;
  constexpr int kRuns = HD / 64;        // 16-byte runs of a key row in a lane
  constexpr int kOut = HD / 16;         // output tiles of 16 dimensions
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t ring = smem_addr(smem + warp * L::kRing);
  const uint32_t info = smem_addr(smem + L::kOffInfo) + warp * S * 8;
  const uint32_t bars = smem_addr(smem + L::kOffBar) + warp * S * 8;
  int64_t* sums = reinterpret_cast<int64_t*>(smem + L::kOffSum);
  int* misc = reinterpret_cast<int*>(smem + L::kOffMisc);  // [0] abort
  int64_t* warp_sums = reinterpret_cast<int64_t*>(smem + L::kOffMisc + 16);
  if (tid == 0) misc[0] = 0;
  if (lane == 0) {
    for (int s = 0; s < S; ++s) mbar_init(bars + 8 * s, 1);
    fence_mbarrier_init();
  }
  __syncthreads();
  grid_dep_launch();
  grid_dep_wait();

  // Numbers in all, and before each run of `per` sequences: up to 32 sequences every warp sums up for
  // itself, one a lane; more are summed by the block.
  Walk walk{p, p.Hk * p.row_tiles, 0, 0, 0};
  const bool few = p.B <= 32;
  const int per = few ? 1 : (p.B + kThreads - 1) / kThreads;
  int64_t mine = 0;
  const int first = few ? lane : tid * per;
  for (int i = first; i < min(first + per, p.B); ++i) mine += walk.numbers(walk.len(i));
  int64_t scan = mine;  // up to and with this lane's
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t up = __shfl_up_sync(0xffffffffu, scan, o);
    if (lane >= o) scan += up;
  }
  int64_t total;
  if (few) {
    total = __shfl_sync(0xffffffffu, scan, 31) * walk.segs;
  } else {
    if (lane == 31) warp_sums[warp] = scan;
    __syncthreads();
    int64_t base = 0;
    for (int w = 0; w < warp; ++w) base += warp_sums[w];
    sums[tid + 1] = (base + scan) * walk.segs;
    if (tid == 0) sums[0] = 0;
    __syncthreads();
    total = sums[kThreads];
  }

  // Sequences with nothing to see; after the first loads are on their way.
  auto write_empty = [&]() {
    for (int b = blockIdx.x * kWarps + warp; b < p.B; b += gridDim.x * kWarps)
      if (walk.len(b) == 0) {
        const int64_t n = static_cast<int64_t>(p.qn) * p.Hq;
        for (int64_t i = lane; i < n * p.D / 8; i += 32)
          reinterpret_cast<uint4*>(p.out + b * n * p.D)[i] = make_uint4(0, 0, 0, 0);
        if (p.lse)
          for (int64_t i = lane; i < n; i += 32) p.lse[b * n + i] = -INFINITY;
        if (p.by_segment)
          for (int i = lane; i < walk.segs; i += 32) p.cuts[b * walk.segs + i].last = -1;
      }
  };

  // As many ranges as there are warps; fewer numbers than warps go to as many SMs as there are.
  const int64_t quota = max(quotient(total + gridDim.x * kWarps - 1, gridDim.x * kWarps), static_cast<int64_t>(1));
  const int warps = static_cast<int>(quotient(quotient(total + quota - 1, quota) + gridDim.x - 1, gridDim.x));
  const int range = blockIdx.x * warps + warp;
  walk.begin = warp < warps ? min(range * quota, total) : total;
  walk.end = min(walk.begin + quota, total);
  walk.uncut = static_cast<int>(min(quota / kUncut, static_cast<int64_t>(1 << 20)));
  if (!p.by_segment && lane == 0) p.cuts[blockIdx.x + gridDim.x * warp].last = -1;
  if (walk.begin >= walk.end) {
    write_empty();
    return;
  }

  Part c{};  // the part to compute
  if (few) {
    const uint32_t after = __ballot_sync(0xffffffffu, scan * walk.segs > walk.begin);  // not zero: begin < total
    c.b = __ffs(after) - 1;
    c.start = __shfl_sync(0xffffffffu, scan - mine, c.b) * walk.segs;
  } else {
    int lo = 0;  // the run of sequences: sums[lo] <= begin < sums[lo + 1]
#pragma unroll 4
    for (int i = lane; i < kThreads; i += 32) lo += sums[i + 1] <= walk.begin;
    lo = __reduce_add_sync(0xffffffffu, lo);
    c.start = sums[lo];
    c.b = lo * per;
  }
  for (;;) {
    c.len = walk.len(c.b);
    const int64_t n = walk.numbers(c.len);
    if (walk.begin < c.start + n * walk.segs) {
      c.hr = static_cast<int>(quotient(walk.begin - c.start, n));
      c.start += c.hr * n;
      break;
    }
    c.start += n * walk.segs;
    ++c.b;
  }
  c.tiles = walk.tiles(c.len);
  bool some = walk.find(c);
  Part ahead = c;  // the part to load, its tile `ahead.t`
  bool more = some;
  const Watchdog wd{p.status, p.timeout_ns, reinterpret_cast<volatile int*>(&misc[0])};
  const uint64_t policy = l2_policy_evict_first();
  const int in_page = p.page - 1, block_shift = p.page_shift - 4;
  int ahead_head = 0;  // key/value head of the part being loaded

  // Pages and scales of 32 tiles of the part being loaded, a tile a lane.
  int batch = -1;                    // its first tile; -1: none
  int page0 = -1, page1 = -1;
  uint32_t scales = 0;               // k block 0, k block 1, v block 0, v block 1
  auto refresh = [&]() {
    batch = ahead.t;
    ahead_head = ahead.hr / p.row_tiles;
    const uint32_t key = static_cast<uint32_t>(ahead.t + lane) * kKeys, len = ahead.len;  // past 2^31 for lanes past the last tile
    const int32_t* row = p.table + ahead.b * p.table_stride;
    auto page_of = [&](uint32_t k) {
      if (k >= len) return -1;
      const int pg = __ldg(row + (k >> p.page_shift));
      return pg >= 0 && pg < p.num_pages ? pg : -1;
    };
    page0 = page_of(key);
    page1 = p.page == 16 ? page_of(key + 16) : page0;
    scales = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int pg = i ? page1 : page0;
      if (pg >= 0 && key + 16 * i < len) {  // a block past the end may hold any byte, NaN's among them
        const int64_t at = ((static_cast<int64_t>(pg) * p.Hk + ahead_head) << block_shift) + (((key + 16 * i) & in_page) >> 4);
        scales |= static_cast<uint32_t>(__ldg(p.k_scale + at)) << (8 * i) | static_cast<uint32_t>(__ldg(p.v_scale + at)) << (16 + 8 * i);
      }
    }
  };
  auto load = [&](int stage) {  // the tile at `ahead` into `stage`
    if (batch < 0 || ahead.t >= batch + 32) refresh();
    const int from = ahead.t - batch;
    const int pg0 = __shfl_sync(0xffffffffu, page0, from), pg1 = __shfl_sync(0xffffffffu, page1, from);
    if (lane == 0 && ahead.t != p.skip) {
      const uint32_t bar = bars + 8 * stage, k = ring + 2 * stage * L::kTile, v = k + L::kTile;
      const int row = (ahead_head << p.page_shift) + (ahead.t * kKeys & in_page);
      mbar_arrive_expect_tx(bar, 2 * L::kTile);
      tma_load_3d_hint(k, &tmK, 0, row, pg0, bar, policy);
      tma_load_3d_hint(v, &tmV, 0, row, pg0, bar, policy);
      if (p.page == 16) {
        tma_load_3d_hint(k + L::kTile / 2, &tmK, 0, row, pg1, bar, policy);
        tma_load_3d_hint(v + L::kTile / 2, &tmV, 0, row, pg1, bar, policy);
      }
    }
    const uint32_t sc = __shfl_sync(0xffffffffu, scales, from);
    if (lane == 0) {
      const uint32_t gone = (pg0 < 0 ? 1u : 0u) | (pg1 < 0 ? 2u : 0u);
      asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(info + 8 * stage), "r"(sc), "r"(gone) : "memory");
    }
    __syncwarp();
    if (++ahead.t == ahead.t1) {
      batch = -1;
      more = walk.next(ahead);
    }
  };
  // This lane's share of the part's query rows: row g8, runs c4 (and c4 + 4).
  const int g8 = lane >> 2, c4 = lane & 3;
  uint4 q_raw[NR][2 * kRuns];
  auto load_q = [&]() {
    const int h = c.hr / p.row_tiles, rt = c.hr % p.row_tiles;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const int row = (rt * NR + r) * 8 + g8;
      const bool live = row < p.qn * p.group;
      const uint16_t* src = p.q + (static_cast<int64_t>(c.b) * p.qn + (live ? row / p.group : 0)) * p.q_stride +
                            (h * p.group + row % p.group) * p.D;
#pragma unroll
      for (int i = 0; i < 2 * kRuns; ++i) {
        const int d = 64 * (i / 2) + 16 * c4 + 8 * (i % 2);
        q_raw[r][i] = live && d < p.D ? *reinterpret_cast<const uint4*>(src + d) : make_uint4(0, 0, 0, 0);
      }
    }
  };
  bool q_loaded = some;
  if (some) load_q();  // before the pages are looked up
  int in_flight = 0;   // stages loaded and not yet consumed
  for (int s = 0; s < S && more; ++s, ++in_flight) load(s);
  write_empty();

  const int kr = key_row<HD>(g8), kv0 = key_row<HD>(2 * c4), kv1 = key_row<HD>(2 * c4 + 1);
  const int run_d = HD == 128 ? 16 * kr : 8 * g8;  // first dimension of this lane's outputs
  int stage = 0;
  uint32_t phase = 0;
  bool ok = true;
  while (some && ok) {
    // ---- a segment, or the part of it in this range.  Row r of N is column r:
    // operands take row g8, results rows 2 c4 and 2 c4 + 1.
    const int h = c.hr / p.row_tiles, rt = c.hr % p.row_tiles;
    uint32_t qf[NR][4 * kRuns][2];
    float q_scale[NR][2];
    int lim[NR][2];      // keys that rows 2 c4, 2 c4 + 1 see
    if (!q_loaded) load_q();
    q_loaded = false;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      float top = 0.f;
      const uint4 (&w)[2 * kRuns] = q_raw[r];
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
      const float down = top == INFINITY ? __uint_as_float(0x7FC00000u)  // such a row is NaN
                                         : p.scale_log2 * __uint_as_float(static_cast<uint32_t>(254 - field) << 23);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        q_scale[r][e] = __shfl_sync(0xffffffffu, down, (2 * c4 + e) * 4);
        const int mine_row = (rt * NR + r) * 8 + 2 * c4 + e;
        lim[r][e] = mine_row < p.qn * p.group ? c.len - (p.qn - 1 - mine_row / p.group) : 0;
      }
      // k-step 4 u + i: this lane's dimensions 64 u + 16 c + 4 i ..+3
#pragma unroll
      for (int i = 0; i < 4 * kRuns; ++i) {
        const uint4& q4 = w[i / 2];
        const uint32_t x = (i & 1) ? q4.z : q4.x, y = (i & 1) ? q4.w : q4.y;
        qf[r][i][0] = pack_f16x2(lo(x) * up, hi(x) * up);
        qf[r][i][1] = pack_f16x2(lo(y) * up, hi(y) * up);
      }
    }
    float o[NR][kOut][4];
    float m[NR][2], n[NR][2], sum[NR][2];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
#pragma unroll
      for (int i = 0; i < kOut; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[r][i][e] = 0.f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        m[r][e] = n[r][e] = kUnset;
        sum[r][e] = 0.f;
      }
    }

    for (int t = c.t; t < c.t1; ++t) {
      ok = __all_sync(0xffffffffu, mbar_wait(bars + 8 * stage, phase, wd, kWhereMmaFull));
      if (!ok) break;
      const uint32_t sk = ring + 2 * stage * L::kTile, sv = sk + L::kTile;
      const uint2 about = ld_shared_v2(info + 8 * stage);
      const int key0 = t * kKeys;
      // scores: s[r][j][2 i + e] of key 16 j + 8 i + kr, row 2 c4 + e
      float s[NR][2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[r][j][e] = 0.f;
#pragma unroll
        for (int u = 0; u < kRuns; ++u) {
          const uint4 x = ld_shared_v4(run_addr<HD>(sk, 16 * j + kr, c4 + 4 * u));
          const uint4 y = ld_shared_v4(run_addr<HD>(sk, 16 * j + 8 + kr, c4 + 4 * u));
          const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t a0, a1, a2, a3;
            codes_f16(xw[i], a0, a2);
            codes_f16(yw[i], a1, a3);
#pragma unroll
            for (int r = 0; r < NR; ++r) mma_16x8x16(s[r][j], a0, a1, a2, a3, qf[r][4 * u + i][0], qf[r][4 * u + i][1]);
          }
        }
      }
      float kx[2], vx[2];  // key scales, value exponents of the two blocks
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int kc = (about.x >> (8 * j)) & 255, vc = (about.x >> (16 + 8 * j)) & 255;
        kx[j] = kc == 255 ? __uint_as_float(0x7FC00000u) : exp2_code(kc);
        vx[j] = vc == 255 ? __uint_as_float(0x7FC00000u) : static_cast<float>(vc - 127);
      }
      const bool edge = key0 > c.len - (p.qn - 1) - kKeys || about.y != 0;
      bool move = false;
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = -INFINITY, vtop = -INFINITY;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float by = kx[j] * q_scale[r][e];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float x = __fmul_rn(s[r][j][2 * i + e], by);  // rounded, as m is, so that their difference is exact near m
              if (edge && (key0 + 16 * j + 8 * i + kr >= lim[r][e] || ((about.y >> j) & 1))) x = -INFINITY;
              s[r][j][2 * i + e] = x;
            }
            const float two = fmaxf(s[r][j][e], s[r][j][2 + e]);
            top = fmaxf(top, two);
            vtop = fmaxf(vtop, (two - m[r][e]) + vx[j]);
          }
          move |= top > m[r][e] + kSlack || vtop > n[r][e] + kLift + kSlack;
        }
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float a = fmaxf(s[r][0][e], s[r][0][2 + e]), b = fmaxf(s[r][1][e], s[r][1][2 + e]);
            float top = fmaxf(fmaxf(a, b), kUnset);
            float vtop = fmaxf((a - top) + vx[0], (b - top) + vx[1]);  // relative to top
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
              const float other = __shfl_xor_sync(0xffffffffu, top, x), vother = __shfl_xor_sync(0xffffffffu, vtop, x);
              const float both = fmaxf(top, other);
              vtop = fmaxf(vtop + (top - both), vother + (other - both));
              top = both;
            }
            if (top > m[r][e]) {
              sum[r][e] *= ex2(m[r][e] - top);
              n[r][e] += m[r][e] - top;
              m[r][e] = top;
            }
            vtop += top - m[r][e];
            if (vtop - kLift > n[r][e]) {
              const float by = ex2(n[r][e] - (vtop - kLift));
              n[r][e] = vtop - kLift;
#pragma unroll
              for (int i = 0; i < kOut; ++i) {
                o[r][i][e] *= by;
                o[r][i][2 + e] *= by;
              }
            }
          }
      }
      // weights; then of row g8 and keys 2 c4, 2 c4 + 1
      uint32_t w[NR][2][2];
#pragma unroll
      for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float by[2] = {vx[j] - n[r][0], vx[j] - n[r][1]};
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float x = s[r][j][2 * i] - m[r][0], y = s[r][j][2 * i + 1] - m[r][1];
            sum[r][0] += ex2(x);
            sum[r][1] += ex2(y);
            w[r][j][i] = transpose8(pack_f16x2(ex2(x + by[0]), ex2(y + by[1])));
          }
        }
      // output += codes times weights, 16 keys at a time
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t v[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 16 * j + 8 * (i >> 1) + ((i & 1) ? kv1 : kv0);
          if constexpr (HD == 128) {
            const uint4 x = ld_shared_v4(run_addr<HD>(sv, row, kr));
            v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
          } else {
            const uint2 x = ld_shared_v2(run_addr<HD>(sv, row, g8 >> 1) + 8 * (g8 & 1));
            v[i][0] = x.x, v[i][1] = x.y;
          }
          if (edge && key0 + row >= c.len) {  // stale codes may be NaN
#pragma unroll
            for (int e = 0; e < HD / 32; ++e) v[i][e] = 0;
          }
        }
#pragma unroll
        for (int e = 0; e < HD / 32; ++e)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            // dimensions 4 e + 2 half and the next of this lane's run
            uint32_t a0, a1, a2, a3;
            codes_f16(__byte_perm(v[0][e], v[1][e], half ? 0x7362 : 0x5140), a0, a1);
            codes_f16(__byte_perm(v[2][e], v[3][e], half ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
            for (int r = 0; r < NR; ++r) mma_16x8x16(o[r][2 * e + half], a0, a1, a2, a3, w[r][j][0], w[r][j][1]);
          }
      }
      __syncwarp();  // every lane has read the stage
      --in_flight;
      if (more) {
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
    const bool whole = c.t == 0 && c.t1 == c.tiles;
    const int64_t slot = 2 * static_cast<int64_t>(range) + (c.t == 0);
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) sum[r][e] += __shfl_xor_sync(0xffffffffu, sum[r][e], x);
        const int in_tile = 8 * r + 2 * c4 + e, row = rt * NR * 8 + in_tile;
        if (row >= p.qn * p.group) continue;
        if (whole) {
          const int64_t at = (static_cast<int64_t>(c.b) * p.qn + row / p.group) * p.Hq + h * p.group + row % p.group;
          const bool none = sum[r][e] == 0.f;
          const float half = ex2(0.5f * n[r][e]), by = half / sum[r][e];  // 2^n in two steps: by itself it may leave fp32's range
          if (run_d < p.D) {
#pragma unroll
            for (int i = 0; i < kOut; i += 4) {
              uint32_t u[4];
#pragma unroll
              for (int x = 0; x < 4; ++x)
                u[x] = none ? 0u : pack_bf16x2(o[r][i + x][e] * half * by, o[r][i + x][2 + e] * half * by);
              *reinterpret_cast<uint4*>(p.out + at * p.D + run_d + 2 * i) = make_uint4(u[0], u[1], u[2], u[3]);
            }
          }
          if (g8 == 0 && p.lse) p.lse[at] = none ? -INFINITY : (m[r][e] + log2f(sum[r][e])) * 0.6931471805599453f;
        } else {
          const int64_t at = slot * (8 * NR) + in_tile;
#pragma unroll
          for (int i = 0; i < kOut; i += 2)
            *reinterpret_cast<float4*>(p.part_o + at * HD + run_d + 2 * i) =
                make_float4(o[r][i][e], o[r][i][2 + e], o[r][i + 1][e], o[r][i + 1][2 + e]);
          if (g8 == 0) p.part_ml[at] = make_float4(m[r][e], n[r][e], sum[r][e], 0.f);
        }
      }
    if (c.t == 0 && lane == 0 && (p.by_segment || !whole)) {
      const int64_t first = c.start + kSegCost;
      p.cuts[p.by_segment ? c.b * walk.segs + c.hr : blockIdx.x + gridDim.x * warp] =
          whole ? Cut{0, 0, 0, -1} : Cut{c.b, c.hr, range, static_cast<int>(quotient(first + c.tiles - 1, quota))};
    }
    some = walk.next(c);
  }
  if (!ok) {
    // the join must not find what an earlier call left for the segments that begin here
    while (some) {
      if (c.t == 0 && lane == 0 && p.by_segment) p.cuts[c.b * walk.segs + c.hr].last = -1;
      some = walk.next(c);
    }
    // loads in flight must land before the CTA can exit
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

// Joins the parts of a cut segment; a lane owns 4 dimensions.  Few parts: a warp a row, in the first
// block of the segment.  Many: a block a row, whose warps share out the parts.
template <int HD, int NR, int WARPS>
__global__ void __launch_bounds__(32 * WARPS) decode_join_kernel(const DecodeParams p) {
  __shared__ float4 shared_o[WARPS][32];
  __shared__ float shared_sum[WARPS];
  grid_dep_launch();
  grid_dep_wait();
  const Cut cut = p.cuts[blockIdx.x];
  if (cut.last < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row0 = cut.hr % p.row_tiles * NR * 8, head = cut.hr / p.row_tiles * p.group;
  const int rows = min(8 * NR, p.qn * p.group - row0);
  const int count = cut.last - cut.first + 1;
  const bool many = count > 2 * WARPS;
  if (!many && blockIdx.y > 0) return;
  auto at = [&](int k, int row) { return (2 * (cut.first + k) + (k == 0)) * (8 * NR) + row; };
  const int d = 4 * lane < HD ? 4 * lane : 0;
  for (int row = many ? blockIdx.y : warp; row < rows; row += many ? gridDim.y : WARPS) {
    float m = kUnset, n = kUnset, sum = 0.f;
    // this warp's first parts are on their way while the references are looked up
    const int step = many ? WARPS : 1, k0 = many ? warp : 0;
    float4 mls[kFirst], xs[kFirst];
#pragma unroll
    for (int i = 0; i < kFirst; ++i) {
      const int k = min(k0 + i * step, count - 1);
      mls[i] = p.part_ml[at(k, row)];
      xs[i] = *reinterpret_cast<const float4*>(p.part_o + static_cast<int64_t>(at(k, row)) * HD + d);
    }
    for (int k = lane; k < count; k += 32) {
      const float4 ml = p.part_ml[at(k, row)];
      m = fmaxf(m, ml.x);
      n = fmaxf(n, ml.x + ml.y);
    }
#pragma unroll
    for (int x = 1; x < 32; x <<= 1) {
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
      n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, x));
    }
    n = fabsf(m) < 1048576.f ? n - m : 0.f;  // any reference does that keeps 2^n in range; beside a larger m it would be lost
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](const float4& ml, const float4& x) {
      const float below = ml.x - m;
      sum += ml.z * ex2(below);
      const float by = ex2(below + (ml.y - n));
      o.x += x.x * by;
      o.y += x.y * by;
      o.z += x.z * by;
      o.w += x.w * by;
    };
#pragma unroll
    for (int i = 0; i < kFirst; ++i)
      if (k0 + i * step < count) add(mls[i], xs[i]);
#pragma unroll 4
    for (int k = k0 + kFirst * step; k < count; k += step)
      add(p.part_ml[at(k, row)], *reinterpret_cast<const float4*>(p.part_o + static_cast<int64_t>(at(k, row)) * HD + d));
    if (many) {
      __syncthreads();  // the last row's have been read
      shared_o[warp][lane] = o;
      shared_sum[warp] = sum;
      __syncthreads();
      if (warp != 0) continue;
#pragma unroll
      for (int i = 1; i < WARPS; ++i) {
        const float4 x = shared_o[i][lane];
        o.x += x.x;
        o.y += x.y;
        o.z += x.z;
        o.w += x.w;
        sum += shared_sum[i];
      }
    }
    const int r = row0 + row;
    const int64_t to = (static_cast<int64_t>(cut.b) * p.qn + r / p.group) * p.Hq + head + r % p.group;
    const bool none = sum == 0.f;
    const float half = ex2(0.5f * n), by = half / sum;
    if (4 * lane < p.D)
      *reinterpret_cast<uint2*>(p.out + to * p.D + d) =
          none ? make_uint2(0, 0)
               : make_uint2(pack_bf16x2(o.x * half * by, o.y * half * by), pack_bf16x2(o.z * half * by, o.w * half * by));
    if (lane == 0 && p.lse) p.lse[to] = none ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
  }
}

sg_status_t launch_error(cudaError_t e) {
  if (e == cudaSuccess) return SG_OK;
  note_cuda_error(e);
  cudaGetLastError();  // clear the non-sticky launch error
  return SG_ERR_CUDA;
}

int64_t max_ranges(const AttnShape& s) { return static_cast<int64_t>(s.num_sms) * kMaxWarps; }

template <int HD, int NR>
sg_status_t launch(const AttnShape& s, const AttnArgs& a, DecodeParams& p) {
  using L = DecodeLayout<HD, NR>;
  const uint64_t D = s.D, rows = static_cast<uint64_t>(s.Hk) * s.page;
  const uint64_t dims[3] = {D, rows, static_cast<uint64_t>(a.cache.num_pages)};
  const uint64_t sk[2] = {D, static_cast<uint64_t>(a.cache.k_page_stride)}, sv[2] = {D, static_cast<uint64_t>(a.cache.v_page_stride)};
  const uint32_t box[3] = {HD, static_cast<uint32_t>(s.page < kKeys ? s.page : kKeys), 1};
  const CUtensorMapSwizzle sw = HD == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  CUtensorMap tmK, tmV;
  if (!encode_3d(&tmK, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.cache.k, dims, sk, box, sw) ||
      !encode_3d(&tmV, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.cache.v, dims, sv, box, sw))
    return SG_ERR_CUDA;
  p.row_tiles = (p.qn * p.group + 8 * NR - 1) / (8 * NR);
  const int64_t segments = a.B * s.Hk * p.row_tiles, ranges = static_cast<int64_t>(s.num_sms) * L::kWarps;
  p.by_segment = segments <= ranges;
  GemmLaunch l(dim3(s.num_sms), dim3(L::kThreads), L::kDynSmem, a.stream, 1);
  const sg_status_t r = launch_error(cudaLaunchKernelEx(&l.cfg, decode_kernel<HD, NR>, tmK, tmV, p));
  if (r != SG_OK) return r;
  // blocks for a row each where that many fit the GPU at once
  const int64_t joins = p.by_segment ? segments : ranges, fit = 8 * s.num_sms / joins;
  const unsigned per_row = static_cast<unsigned>(fit < 1 ? 1 : fit < 8 * NR ? fit : 8 * NR);
  // where not even a block a segment fits, up to 4 rows take half the warps (200 sequences, 4 drafted tokens: 61.4 us,
  // 63.0 with 8 warps)
  if constexpr (NR == 1) {
    if (fit < 1 && p.qn * p.group <= kJoinWarps / 2) {
      GemmLaunch j(dim3(static_cast<unsigned>(joins), per_row), dim3(16 * kJoinWarps), 0, a.stream, 1);
      return launch_error(cudaLaunchKernelEx(&j.cfg, decode_join_kernel<HD, NR, kJoinWarps / 2>, p));
    }
  }
  GemmLaunch j(dim3(static_cast<unsigned>(joins), per_row), dim3(32 * kJoinWarps), 0, a.stream, 1);
  return launch_error(cudaLaunchKernelEx(&j.cfg, decode_join_kernel<HD, NR, kJoinWarps>, p));
}

template <int HD, int NR>
cudaError_t prepare() {
  return cudaFuncSetAttribute(decode_kernel<HD, NR>, cudaFuncAttributeMaxDynamicSharedMemorySize, DecodeLayout<HD, NR>::kDynSmem);
}

}  // namespace

size_t decode_workspace_bytes(const AttnShape& s) {
  return static_cast<size_t>(max_ranges(s)) * (2 * 16 * (128 * 4 + 16) + sizeof(Cut));
}

cudaError_t decode_prepare() {
  cudaError_t e = prepare<64, 1>();
  if (e == cudaSuccess) e = prepare<64, 2>();
  if (e == cudaSuccess) e = prepare<128, 1>();
  return e == cudaSuccess ? prepare<128, 2>() : e;
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
  while ((1 << p.page_shift) < s.page) ++p.page_shift;
  p.group = s.Hq / s.Hk;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  p.part_o = static_cast<float*>(s.workspace);
  p.part_ml = reinterpret_cast<float4*>(p.part_o + max_ranges(s) * 2 * 16 * 128);
  p.cuts = reinterpret_cast<Cut*>(p.part_ml + max_ranges(s) * 2 * 16);
  p.skip = s.skip_tile;
  p.status = s.status;
  p.timeout_ns = s.timeout_ns;
  AttnArgs args = a;
  if (args.cache.num_pages == 0) {  // a tensor map has no empty dimension; nothing reads it
    args.cache.num_pages = 1;
    args.cache.k = args.cache.v = const_cast<void*>(a.q);
    args.cache.k_page_stride = args.cache.v_page_stride = static_cast<int64_t>(s.Hk) * s.page * s.D;
  }
  // Up to 8 query rows of a key/value head take half the registers, which
  // more warps use; more rows go 16 at a time, so that the cache is read half as often.
  if (p.qn * p.group <= 8) return s.D > 64 ? launch<128, 1>(s, args, p) : launch<64, 1>(s, args, p);
  return s.D > 64 ? launch<128, 2>(s, args, p) : launch<64, 2>(s, args, p);
}

}  // namespace sg
