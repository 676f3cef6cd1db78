// sg_attn_chunk.cu -- attention of chunks of new tokens over the paged e4m3 cache
// (scaled_attn_chunk).
//
// For query row i of a sequence's n and the keys j < m - (n - 1 - i) of its m, with k_j = 2^a_j K_j and
// v_j = 2^b_j V_j (K, V codes, a, b the exponents of their block of 16 keys),
//     s_j = c q_i . k_j   (c = scale log2 e),   o_i = sum_j 2^(s_j) v_j / sum_j 2^(s_j),
// in one pass over tiles of 128 keys, as sg_attn_prompt.cu goes, with the cache's codes as operands:
//   * Scores: K as it lies in the cache, through the fp8 tensor cores.  A query row, scaled by a power of two so that its largest
//     value lies in [2^7, 2^8), is the sum of two terms: e4m3 (4 significant bits), and what that leaves of bf16's 8 in
//     e5m2 (3 bits hold every remainder).  Elements down to 2^-13 of the row's largest are exact, smaller ones off by at most
//     2^-21 of it.  Two products at twice bf16's rate, and K needs no conversion and no copy in shared memory.
//   * K's block scales are part of the factor that every score takes on its way to the exponential.
//   * Values: codes to fp16, which holds them exactly, by two warps; their block scales go into the weights, 2^(s_j - m + b_j - n)
//     in fp16 (2^-11 of each), and out of the row sum again, a block's sum at a time.  m follows the maximum of s_j, m + n
//     that of s_j + b_j, as in sg_attn_decode.cu; both are whole numbers here, so that one fma a score forms the exponent
//     with a single rounding.  Rows whose scores pass 2^22, or whose value scales lie 2^96 apart, take a
//     slower way that forms score, difference and sum one by one.
// Rows are packed as in sg_attn_prompt.cu: a tile's 128 rows are tokens times query heads of one key/value head.  A CTA
// works on two row tiles, or, where a unit has but one (few tokens), on the even and the odd
// key blocks of that one, whose halves it joins at the end out of tensor memory:
//   warps 0-3, 4-7  softmax and output of tile 0 / 1, one thread a row; the next unit's queries to their two terms
//   warp 8          work, pages and scales, TMA: K_0, V_0, K_1, V_1, ... through two rings
//   warp 9          MMAs, one thread
//   warps 10, 11    values to fp16
//
// Work: units (two row tiles of a sequence and head) are numbered by what they cost, and every CTA takes
// an equal range of the numbers, so a few tokens over a long cache fill the GPU as well as many over a short one.
// Units that are short beside a range are not cut; the parts of a cut one are joined by a second
// kernel in the order of their ranges, so results do not depend on timing.
//
// What bounds it: the chain scores, softmax, weights, product of a tile, 1.9 us (2 long documents) to 2.1 (4 chunks) a block of both where the tensor cores need
// 1.1 and take 1.5 without the softmax.  Two things lengthen it.  Shared memory: operands of the MMAs, loads and the
// conversion take 2200 of a block's cycles, and every load and barrier of the other warps waits in between (hundreds of
// cycles: so scales are read before the scores are there).  Instructions: five kinds of warps, each in a loop of its own, do not
// fit the caches nearest to them, and the code's length shows in every time.  And a unit costs 8 to 15 us beside its blocks, with its queries,
// first and last softmax and output.  Measured, with the join: 4 chunks of 1000 to 2048 tokens behind up to 24000,
// 32 heads of 128 over 8: 1180 us, 1.15 PFLOP/s; 40 sequences of 1 to 300 tokens, 40 heads over 8: 308; 2 of 101 and 256 behind 120000
// and more, 64 heads over 8: 1163; 24 of 5 to 700, 16 heads of 64: 111; one of 24 behind 900: 25.
// Measured slower (4 chunks, and the form that each was tried on): the issuing thread's code for both tiles written out 1444 us, one copy 1364; loads of
// scales after the scores are there, two threads a row or not, 1530 to 1580; two issuing threads, whose tiles then run in step, 1535, or
// in turn 1530 (1325 with one); a unit's cost taken as a third of what it is, 1335 (1230); pages and scales loaded a group ahead of their
// blocks, in one loop over jobs and groups, 1268 (1222), with a second copy of that code 1364.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cfloat>

#include "sg_attn.h"
#include "sg_attn_ptx.cuh"
#include "sg_mx.cuh"

namespace sg {

namespace {

constexpr int kRows = 128;  // rows of a tile, keys of a block
constexpr int kThreads = 384;
constexpr int kSoftmaxWarps = 8;
constexpr int kSoftmaxRegs = 208, kIssueRegs = 88;  // 2 x 208 + 88 = 3 x 168, what the block is launched with
constexpr int kWhereJob = 0x41, kWhereMerge = 0x42, kWhereConvert = 0x43;  // waits beside those of sg_ptx.cuh
constexpr int kJobReaders = kSoftmaxWarps + 3;  // warps that take jobs
constexpr int kEarly = 4;        // 16-key steps of a block whose weights are handed over first
// What work costs, in quarters of what a key costs a unit of two row tiles: a key of a unit with one tile, whose blocks are loaded and
// converted for half as many scores (1.2 to 1.6 us a block, 1.9 for both tiles; as half of a pair's 40 mixed take 364 us and
// 2 long documents 1420, as three quarters 308 and 1163, as five sixths 317 and 1163), and what a unit costs beside its keys
// (40 mixed and 4 chunks with 3200: 308 and 1182 us; 2304: 354 and 1243).
constexpr int kPairKey = 4, kSingleKey = 3, kUnitCost = 3200;
constexpr int kUncut = 32;       // units of up to 1 / kUncut of a range are not cut (4 chunks: 1190 us; 16: 1206)
constexpr int kLeast = 768;      // of a range, so that every range of a cut unit has a block of it (one question: 24.6 us; 512: 26.6)
constexpr float kSlack = 8.f;    // log2 of how far a maximum may pass its reference
constexpr float kLift = 7.f;     // the output's weights at its reference are 2^kLift, the largest 2^15
constexpr float kUnset = -FLT_MAX;
constexpr float kExact = 4194304.f;  // references past this take the slow way
constexpr float kSpread = -96.f;     // so do value scales this far below their reference, in log2,
constexpr float kWide = 96.f;        // value scales whose exponent is past this,
constexpr float kLight = 0x1p-60f;   // key scales below this or NaN, and, in blocks with hidden keys, queries whose factor is

// A unit that was cut: its rows, and the ranges that have parts of it; last < 0: none begins in this range.
struct Cut {
  int q0, lq, first, head0, tiles, from, last, unused;
};

struct ChunkParams {
  const uint16_t* q;
  int64_t q_stride;
  const int32_t *table, *lens, *cu;
  int64_t table_stride;
  const uint8_t *k_scale, *v_scale;
  int64_t num_pages;
  int T, B, Hq, Hk, D, page, page_shift;
  int group;            // query heads of a key/value head
  int pack;             // query heads packed into a tile
  int pack_inverse;     // a row's token: row * pack_inverse >> 16
  int head_groups;      // Hq / pack
  int skip;             // number of a key block that is not loaded (scaled_attn_set_debug); -1: none
  float scale_log2;
  uint16_t* out;
  float* lse;
  float* part_o;        // [2 ranges][2 tiles][HD / 4][kRows][4]: the part that begins a unit (odd), one that does not
  float4* part_ml;      // [2 ranges][2 tiles][kRows]: m, n, sum
  Cut* cuts;            // [ranges]
  int* status;
  uint64_t timeout_ns;
};

template <int HD>
struct ChunkLayout {
  static constexpr int kTile = kRows * 128;          // a term of a query tile, a K block
  static constexpr int kKStages = 3, kVStages = 2, kHalfStages = 2;
  static constexpr int kRaw = kRows * HD;            // codes of a V block
  static constexpr int kBox = kRows * 128;           // 64 dimensions of it in fp16
  static constexpr int kHalf = HD / 64 * kBox;
  static constexpr int kOffK = 4 * kTile;            // after two terms of two query tiles
  static constexpr int kOffHalf = kOffK + kKStages * kTile;
  static constexpr int kOffRaw = kOffHalf + kHalfStages * kHalf;
  static constexpr int kOffStats = kOffRaw + kVStages * kRaw;  // a row's references and sum, by row tile
  static constexpr int kInfo = 8;                    // key blocks whose scales are held
  static constexpr int kOffInfo = kOffStats + 2 * kRows * 16;        // of its 16-key blocks: the scores' factors, the values' exponents
  static constexpr int kOffInverse = kOffInfo + kInfo * 64;  // 2^-exponent
  static constexpr int kOffMask = kOffInverse + kInfo * 32;  // pages that are not there, value scales that are NaN, odd ones; least and largest exponent
  static constexpr int kOffRow = kOffMask + kInfo * 16;      // a query row's factor, by job and row
  static constexpr int kOffBar = kOffRow + 2 * 2 * kRows * 4;
  static constexpr int kNumBars = 2 * (kKStages + kVStages + kHalfStages) + 10 + 8 + kInfo;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffJobs = kOffMisc + 16;
  static constexpr int kOffSums = kOffStats;         // while work is planned: int64 per thread
  static constexpr int kBytes = kOffJobs + 2 * 48;
  static constexpr int kDynSmem = kBytes + 1024;
  static_assert(kThreads * 8 <= 2 * kRows * 16 && kOffInfo % 16 == 0 && kOffBar % 8 == 0 && kOffJobs % 16 == 0 && kDynSmem <= 232448, "shared memory");
};

// Key blocks; sizes reach 2^31.
__device__ __forceinline__ int blocks_of(int keys) { return static_cast<int>((static_cast<uint32_t>(keys) + kRows - 1) / kRows); }

// Tokens of a sequence, its keys, and units: a unit has `span` tokens, a row tile half of that.
struct Sequence {
  int q0, lq, lk, units;
};

__device__ __forceinline__ Sequence sequence(const ChunkParams& p, int b, int span) {
  Sequence s;
  s.q0 = min(max(__ldg(p.cu + b), 0), p.T);
  s.lq = max(min(max(__ldg(p.cu + b + 1), 0), p.T) - s.q0, 0);
  const int64_t cap = p.table_stride * p.page;
  s.lk = static_cast<int>(min(static_cast<int64_t>(max(__ldg(p.lens + b), 0)), cap));
  s.units = (s.lq + span - 1) / span;
  return s;
}

// Keys that the unit's last token sees, and its row tiles.
__device__ __forceinline__ int unit_keys(const Sequence& s, int i, int span) {
  return max(s.lk - s.lq + min((i + 1) * span, s.lq), 0);
}
__device__ __forceinline__ int unit_tiles(const Sequence& s, int i, int span) { return s.lq - i * span > span / 2 ? 2 : 1; }

// What a key costs a unit: an expression without a choice, since this kernel feels every instruction (4 chunks: 1190 us, 1222 with one).
static_assert(kPairKey == kSingleKey + 1, "");
__device__ __forceinline__ int key_cost(int tiles) { return tiles + kSingleKey - 1; }

// What the units before unit i (at most the last) cost; all but the last have two tiles and see lk - lq + span (x + 1) keys.
__device__ __forceinline__ int64_t cost_before(const Sequence& s, int i, int span) {
  const int64_t a = static_cast<int64_t>(s.lk) - s.lq, n = i;
  const int64_t none = a >= 0 ? 0 : min(n, -a / span);
  return n * kUnitCost + kPairKey * ((n - none) * a + span * (n * (n + 1) / 2 - none * (none + 1) / 2));
}
__device__ __forceinline__ int64_t cost(const Sequence& s, int span) {  // of one head group
  if (s.units == 0) return 0;
  return cost_before(s, s.units - 1, span) + kUnitCost + static_cast<int64_t>(key_cost(unit_tiles(s, s.units - 1, span))) * s.lk;
}

// The first sequence after b that has tokens; B: none.  By a whole warp, 32 at a time: between two that have some there may be
// millions that are idle, and every other warp of the CTA waits meanwhile, for 4 seconds at most.
__device__ __forceinline__ int next_sequence(const ChunkParams& p, int b) {
  for (++b; b < p.B; b += 32) {
    const int at = b + static_cast<int>(threadIdx.x & 31);
    auto upto = [&](int i) { return min(max(__ldg(p.cu + i), 0), p.T); };
    const unsigned there = __ballot_sync(0xffffffffu, at < p.B && upto(at + 1) > upto(at));
    if (there) return b + __ffs(there) - 1;
  }
  return p.B;
}

// What a CTA works on: blocks [t0, t1) of a unit.  b: -2 no more.
struct Job {
  int b, q0, lq, lk;     // sequence, its first row, tokens, keys
  int first, tiles;      // the unit's first token, its row tiles
  int t0, t1;
  int head0, whole, slot, unused;
};

// The jobs of a range [begin, end) of the numbers.
struct Walk {
  const ChunkParams& p;
  int span;
  int64_t begin, end, quota;
  Sequence s;
  int b, hg, unit;
  int64_t start;  // the unit's number
  // The first job at or after the unit; false: none.  By a whole warp.
  __device__ __forceinline__ bool find(Job& job, Cut& cut) {
    for (;;) {
      if (start >= end) return false;
      const int keys = unit_keys(s, unit, span), tiles = unit_tiles(s, unit, span), blocks = blocks_of(keys);
      const int64_t each = kRows * key_cost(tiles), first = start + kUnitCost;
      int t0 = 0, t1 = blocks;
      bool mine;
      if (static_cast<int64_t>(key_cost(tiles)) * keys * kUncut <= quota) {
        mine = start >= begin;
      } else {
        if (begin > first) t0 = static_cast<int>(min((begin - first + each - 1) / each, static_cast<int64_t>(blocks)));
        t1 = static_cast<int>(max(min((end - first + each - 1) / each, static_cast<int64_t>(blocks)), static_cast<int64_t>(0)));
        mine = t0 < t1;
      }
      if (mine) {
        const bool whole = t0 == 0 && t1 == blocks;
        const int range = static_cast<int>(begin / quota);
        job = Job{b, s.q0, s.lq, s.lk, unit * span, tiles, t0, t1, hg * p.pack, whole, 2 * range + (t0 == 0), 0};
        if (t0 == 0 && !whole)
          cut = Cut{s.q0, s.lq, unit * span, hg * p.pack, tiles, range, static_cast<int>((first + each * (blocks - 1)) / quota), 0};
      }
      // the next unit
      start += kUnitCost + static_cast<int64_t>(key_cost(tiles)) * keys;
      if (++unit == s.units) {
        unit = 0;
        if (++hg == p.head_groups) {
          hg = 0;
          b = next_sequence(p, b);
          if (b >= p.B)
            start = end;
          else
            s = sequence(p, b, span);
        }
      }
      if (mine) return true;
    }
  }
};

// Two fp32 values to two e4m3 (e5m2) codes, to nearest even; two e4m3 codes to fp16.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t to_e5m2x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t from_e4m3x2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
  return r;
}
__device__ __forceinline__ void half2_floats(uint32_t x, float& lo, float& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}" : "=f"(lo), "=f"(hi) : "r"(x));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t a) {
  const uint4 v = ld_shared_v4(a);
  return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}
__device__ __forceinline__ uint32_t ld_shared(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared(uint32_t a, uint32_t v) { asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory"); }
__device__ __forceinline__ void st_shared_v2(uint32_t a, uint32_t x, uint32_t y) {
  asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(a), "r"(x), "r"(y) : "memory");
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const ChunkParams p) {
  using L = ChunkLayout<HD>;
  constexpr int KS = L::kKStages, VS = L::kVStages, HS = L::kHalfStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t base = smem_addr(smem), bar0 = base + L::kOffBar;
  auto q_tile = [&](int t, int term) { return base + (2 * t + term) * L::kTile; };
  auto k_full = [&](int s) { return bar0 + 8 * s; };
  auto k_empty = [&](int s) { return bar0 + 8 * (KS + s); };
  auto v_full = [&](int s) { return bar0 + 8 * (2 * KS + s); };
  auto v_empty = [&](int s) { return bar0 + 8 * (2 * KS + VS + s); };
  auto h_full = [&](int s) { return bar0 + 8 * (2 * KS + 2 * VS + s); };
  auto h_empty = [&](int s) { return bar0 + 8 * (2 * KS + 2 * VS + HS + s); };
  constexpr int kMore = 2 * (KS + VS + HS);
  auto s_full = [&](int t) { return bar0 + 8 * (kMore + t); };
  auto p_full = [&](int t) { return bar0 + 8 * (kMore + 2 + t); };
  auto o_full = [&](int t) { return bar0 + 8 * (kMore + 4 + t); };
  auto job_full = [&](int s) { return bar0 + 8 * (kMore + 6 + s); };
  auto job_empty = [&](int s) { return bar0 + 8 * (kMore + 8 + s); };
  const uint32_t drain_bar = bar0 + 8 * (kMore + 10);
  const uint32_t q_full = bar0 + 8 * (kMore + 12), q_empty = bar0 + 8 * (kMore + 13), merge_bar = bar0 + 8 * (kMore + 14);
  auto p_half = [&](int t) { return bar0 + 8 * (kMore + 15 + t); };
  auto info_full = [&](uint32_t slot) { return bar0 + 8 * (kMore + 17 + slot); };
  int* misc = reinterpret_cast<int*>(smem + L::kOffMisc);  // [0] TMEM base, [1] abort
  Job* jobs = reinterpret_cast<Job*>(smem + L::kOffJobs);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tile_tokens = kRows / p.pack, span = 2 * tile_tokens;

  grid_dep_wait();
  if (warp == kSoftmaxWarps + 1) {
    tmem_alloc(smem_addr(&misc[0]), 512);
    tmem_relinquish();
  }
  if (tid == 32) {
    for (int i = 0; i < L::kNumBars; ++i) mbar_init(bar0 + 8 * i, 1);
    for (int s = 0; s < VS; ++s) mbar_init(v_empty(s), 2);
    for (int s = 0; s < HS; ++s) mbar_init(h_full(s), 2);
    for (int t = 0; t < 2; ++t) {
      mbar_init(p_full(t), kRows);
      mbar_init(p_half(t), kRows);
      mbar_init(job_empty(t), kJobReaders);
    }
    mbar_init(q_full, kSoftmaxWarps);
    mbar_init(merge_bar, 2 * kRows);
    misc[1] = 0;
    fence_mbarrier_init();
  }
  // Numbers before each run of `per` sequences, by thread.
  int64_t* sums = reinterpret_cast<int64_t*>(smem + L::kOffSums);
  const int per = (p.B + kThreads - 1) / kThreads;
  {
    int64_t mine = 0;
    for (int b = tid * per; b < min((tid + 1) * per, p.B); ++b) mine += cost(sequence(p, b, span), span) * p.head_groups;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t up = __shfl_up_sync(0xffffffffu, mine, o);
      if (lane >= o) mine += up;
    }
    sums[tid] = mine;  // up to and with this thread's, within the warp
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_launch();  // not before tensor memory is there
  const uint32_t tmem = static_cast<uint32_t>(misc[0]);
  const Watchdog wd{p.status, p.timeout_ns, reinterpret_cast<volatile int*>(&misc[1])};
  auto read = [&](int i, Job& job) {
    const int4* from = reinterpret_cast<const int4*>(jobs + (i & 1));
    const int4 x = from[0], y = from[1], z = from[2];
    auto same = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    job.b = same(x.x), job.q0 = same(x.y), job.lq = same(x.z), job.lk = same(x.w);
    job.first = same(y.x), job.tiles = same(y.y), job.t0 = same(y.z), job.t1 = same(y.w);
    job.head0 = same(z.x), job.whole = same(z.y), job.slot = same(z.z);
  };
  auto done = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(job_empty(i & 1));
  };
  auto peek = [&](int i, Job& job) {  // false: no more, or the CTA gives up
    if (!__all_sync(0xffffffffu, mbar_wait(job_full(i & 1), (i >> 1) & 1, wd, kWhereJob))) return false;
    read(i, job);
    return job.b != -2;
  };
  // Keys that a token's row sees, a row tile's last row, and its blocks in the job.  A unit with one row tile has
  // two halves of the job's blocks instead, the even ones and the odd ones.
  auto visible = [&](const Job& j, int tok) { return max(min(j.lk, j.lk - j.lq + tok + 1), 0); };
  auto tile_keys = [&](const Job& j, int t) {
    const int first = j.first + (j.tiles == 2 ? t * tile_tokens : 0);
    return first < j.lq ? visible(j, min(first + tile_tokens, j.lq) - 1) : 0;
  };
  auto tile_blocks = [&](const Job& j, int t) {
    if (j.tiles == 1) return (j.t1 - j.t0 + 1 - t) / 2;
    return max(min(blocks_of(tile_keys(j, t)), j.t1) - j.t0, 0);
  };

  if (warp >= kSoftmaxWarps) {
    reg_dec<kIssueRegs>();
    if (warp == kSoftmaxWarps) {
      // ---------------- work and TMA ----------------
      int64_t run = 0, total = 0;  // numbers before this lane's warp, in all
      for (int w = 0; w < kThreads / 32; ++w) {
        const int64_t x = sums[32 * w + 31];
        total += x;
        if (w < lane) run += x;
      }
      __syncwarp();
      const int64_t quota = max((total + gridDim.x - 1) / gridDim.x, static_cast<int64_t>(kLeast));
      Walk walk{p, span, min(static_cast<int64_t>(blockIdx.x) * quota, total), 0, quota, Sequence{0, 0, 0, 0}, 0, 0, 0, 0};
      walk.end = min(walk.begin + quota, total);
      bool some = walk.begin < walk.end;
      if (some) {
        // the run of sequences, the sequence in it, the head group and the unit with number `begin`
        const int w = __popc(__ballot_sync(0xffffffffu, lane < kThreads / 32 && run <= walk.begin)) - 1;
        walk.start = __shfl_sync(0xffffffffu, run, w);
        const int64_t upto = sums[32 * w + lane] + walk.start;
        const unsigned after = __ballot_sync(0xffffffffu, upto > walk.begin);  // not zero: begin is in this warp's
        const int l = __ffs(after) - 1;
        const int64_t before = __shfl_up_sync(0xffffffffu, upto, 1);
        if (l > 0) walk.start = __shfl_sync(0xffffffffu, before, l);
        walk.b = (32 * w + l) * per;
        for (;;) {
          walk.s = sequence(p, walk.b, span);
          const int64_t each = cost(walk.s, span);
          if (walk.begin < walk.start + each * p.head_groups) {
            walk.hg = static_cast<int>((walk.begin - walk.start) / each);
            walk.start += walk.hg * each;
            break;
          }
          walk.start += each * p.head_groups;
          ++walk.b;
        }
        int64_t lo = 0, step = walk.s.units;  // the unit is in [lo, lo + step)
        while (step > 1) {
          const int64_t next = (step + 31) / 32, i = lo + lane * next;
          const bool below = i < min(lo + step, static_cast<int64_t>(walk.s.units)) &&
                             walk.start + cost_before(walk.s, static_cast<int>(i), span) <= walk.begin;
          lo += (__popc(__ballot_sync(0xffffffffu, below)) - 1) * next;
          step = next;
        }
        walk.unit = static_cast<int>(lo);
        walk.start += cost_before(walk.s, walk.unit, span);
      }
      Cut cut{};
      cut.last = -1;
      const uint64_t policy = l2_policy_evict_first();
      int k_stage = 0, v_stage = 0, count = 0;
      uint32_t k_phase = 0, v_phase = 0, k_issued = 0, v_issued = 0, k_par = 0, v_par = 0;
      const int block_shift = p.page_shift - 4, boxes = min(kRows / p.page, 8);
      const uint32_t k_box = kRows / boxes * 128, v_box = kRows / boxes * HD;
      const int c8 = lane & 7;
      bool ok = true;
      for (int it = 0; ok; ++it) {
        Job job{};
        if (some) some = walk.find(job, cut);
        if (!some) job.b = -2;
        if (it >= 2) ok = __all_sync(0xffffffffu, mbar_wait(job_empty(it & 1), ((it >> 1) - 1) & 1, wd, kWhereJob));
        if (!ok) break;
        if (lane == 0) {
          jobs[it & 1] = job;
          mbar_arrive(job_full(it & 1));
        }
        if (!some) break;
        const int head = job.head0 / p.group;
        const int32_t* row = p.table + job.b * p.table_stride;
        int page = -1;
        float2 about = make_float2(1.f, 0.f);
        uint32_t gone = 0, nan = 0, odd = 0;  // by lane
        for (int t = job.t0; t < job.t1; ++t) {
          const int in = (t - job.t0) & 3;
          if (in == 0) {  // pages and scales of four blocks, 16 keys a lane
            const int64_t key = static_cast<int64_t>(t) * kRows + 16 * lane;
            page = -1;
            about = make_float2(1.f, 0.f);
            bool v_nan = false;
            if (key < job.lk) {
              const int pg = __ldg(row + (key >> p.page_shift));
              if (pg >= 0 && pg < p.num_pages) {
                page = pg;
                const int64_t at = ((static_cast<int64_t>(pg) * p.Hk + head) << block_shift) + ((key & (p.page - 1)) >> 4);
                const int kc = __ldg(p.k_scale + at), vc = __ldg(p.v_scale + at);
                about = make_float2(kc == 255 ? __uint_as_float(0x7FC00000u) : p.scale_log2 * exp2_code(kc), vc == 255 ? 0.f : static_cast<float>(vc - 127));
                v_nan = vc == 255;
              }
            }
            gone = __ballot_sync(0xffffffffu, page < 0);
            nan = __ballot_sync(0xffffffffu, v_nan);
            odd = __ballot_sync(0xffffffffu, page >= 0 && !(about.x >= kLight && about.y >= -kWide && about.y <= kWide));
          }
          // K
          ok = __all_sync(0xffffffffu, mbar_wait(k_empty(k_stage), k_phase ^ 1, wd, kWhereProducerEmpty));
          if (!ok) break;
          const uint32_t slot = count++ & (L::kInfo - 1);
          if ((lane >> 3) == in) {
            const uint32_t x = __float_as_uint(about.x), y = __float_as_uint(about.y);
            st_shared(base + L::kOffInfo + slot * 64 + c8 * 4, x);
            st_shared(base + L::kOffInfo + slot * 64 + 32 + c8 * 4, y);
            st_shared(base + L::kOffInverse + slot * 32 + c8 * 4, __float_as_uint(ex2(-about.y)));
          }
          float least = about.y, most = about.y;
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) {
            least = fminf(least, __shfl_xor_sync(0xffffffffu, least, o));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
          }
          if (lane == 8 * in)
            st_shared_v4(base + L::kOffMask + slot * 16, ((gone >> (8 * in)) & 255) | ((nan >> (8 * in)) & 255) << 8 | ((odd >> (8 * in)) & 255) << 16,
                         __float_as_uint(least), __float_as_uint(most), 0);
          const bool mine = (lane >> 3) == in && c8 % (8 / boxes) == 0;
          const int y = (head << p.page_shift) + ((t * kRows + 16 * c8) & (p.page - 1)), part = c8 / (8 / boxes);
          __syncwarp();
          if (lane == 0) mbar_arrive(info_full(slot));
          if (t != p.skip) {
            if (lane == 0) mbar_arrive_expect_tx(k_full(k_stage), L::kTile);
            __syncwarp();
            if (mine) tma_load_3d_hint(base + L::kOffK + k_stage * L::kTile + part * k_box, &tmK, 0, y, page, k_full(k_stage), policy);
            k_issued |= 1u << k_stage;
            k_par = (k_par & ~(1u << k_stage)) | (k_phase << k_stage);
          }
          if (++k_stage == KS) {
            k_stage = 0;
            k_phase ^= 1;
          }
          // V
          ok = __all_sync(0xffffffffu, mbar_wait(v_empty(v_stage), v_phase ^ 1, wd, kWhereProducerEmpty));
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(v_full(v_stage), L::kRaw);
          __syncwarp();
          if (mine) tma_load_3d_hint(base + L::kOffRaw + v_stage * L::kRaw + part * v_box, &tmV, 0, y, page, v_full(v_stage), policy);
          v_issued |= 1u << v_stage;
          v_par = (v_par & ~(1u << v_stage)) | (v_phase << v_stage);
          if (++v_stage == VS) {
            v_stage = 0;
            v_phase ^= 1;
          }
        }
      }
      // a call that gives up leaves nothing for the join: its outputs are undefined, but no row outside them may be written
      if (lane == 0) {
        if (!ok) cut.last = -1;
        p.cuts[blockIdx.x] = cut;
        // loads in flight must land before the CTA can exit
        for (int s = 0; s < KS; ++s)
          if ((k_issued >> s) & 1) mbar_wait_drain(k_full(s), (k_par >> s) & 1, 200000000ull);
        for (int s = 0; s < VS; ++s)
          if ((v_issued >> s) & 1) mbar_wait_drain(v_full(s), (v_par >> s) & 1, 200000000ull);
      }
    } else if (warp >= kSoftmaxWarps + 2) {
      // ---------------- values to fp16 ----------------
      const int me = warp - kSoftmaxWarps - 2;
      int v_stage = 0, h_stage = 0, count = 0;
      uint32_t v_phase = 0, h_phase = 0;
      Job job;
      bool ok = true;
      for (int it = 0; ok && peek(it, job); ++it) {
        const int blocks = job.t1 - job.t0;
        for (int j = 0; j < blocks; ++j) {
          ok = __all_sync(0xffffffffu, mbar_wait(v_full(v_stage), v_phase, wd, kWhereConvert) &&
                                           mbar_wait(h_empty(h_stage), h_phase ^ 1, wd, kWhereConvert));
          if (!ok) break;
          const uint32_t from = base + L::kOffRaw + v_stage * L::kRaw, to = base + L::kOffHalf + h_stage * L::kHalf;
          const uint32_t nan = (ld_shared(base + L::kOffMask + (count++ & (L::kInfo - 1)) * 16) >> 8) & 255;
          const int past = job.lk - (job.t0 + j) * kRows;  // rows from here on are not this sequence's
          // A lane takes a run of 16 codes to two runs of 16 bytes of fp16.  Eight lanes take four runs of two rows, 5 apart
          // (1, where a row has four runs), so that they meet in no bank: neither reading, with the codes' swizzle, nor writing.
          const int q = lane >> 3, sub = (lane >> 2) & 1;
          const int r8 = HD == 128 ? (sub ? (2 * q + 5) & 7 : 2 * q) : lane >> 2;
          const bool odd = past < kRows || nan != 0;
#pragma unroll 1
          for (int h = 0; h < HD / 64; ++h) {  // four of a row's runs
            const int r0 = me * (kRows / 2) + r8, run = 4 * h + (lane & 3);
            const uint32_t src = from + r0 * HD + (HD == 128 ? (run ^ r8) << 4 : run << 4);
            const uint32_t dst = to + h * L::kBox + r0 * 128;
            const uint32_t to0 = dst + (((2 * (lane & 3)) ^ r8) << 4), to1 = dst + (((2 * (lane & 3) + 1) ^ r8) << 4);
            uint4 all[kRows / 16];  // on their way together
#pragma unroll
            for (int i = 0; i < kRows / 16; ++i) all[i] = ld_shared_v4(src + i * 8 * HD);
            if (__builtin_expect(odd, 0)) {
#pragma unroll
              for (int i = 0; i < kRows / 16; ++i) {
                const int r = 8 * i + r0;
                if ((nan >> (r >> 4)) & 1) all[i] = make_uint4(0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                if (r >= past) all[i] = make_uint4(0, 0, 0, 0);
              }
            }
#pragma unroll
            for (int i = 0; i < kRows / 16; ++i) {
              const uint4& x = all[i];
              st_shared_v4(to0 + i * 1024, from_e4m3x2(x.x), from_e4m3x2(x.x >> 16), from_e4m3x2(x.y), from_e4m3x2(x.y >> 16));
              st_shared_v4(to1 + i * 1024, from_e4m3x2(x.z), from_e4m3x2(x.z >> 16), from_e4m3x2(x.w), from_e4m3x2(x.w >> 16));
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(h_full(h_stage));
            mbar_arrive(v_empty(v_stage));
          }
          if (++v_stage == VS) {
            v_stage = 0;
            v_phase ^= 1;
          }
          if (++h_stage == HS) {
            h_stage = 0;
            h_phase ^= 1;
          }
        }
        if (!ok) break;
        done(it);
      }
    } else if (elect_one()) {
      // ---------------- MMA issuer: one thread for all of it ----------------
      int k_stage = 0, h_stage = 0, q_uses = 0;
      uint32_t k_phase = 0, h_phase = 0, turn = 0;  // turn: parities of the tiles' next weights, a bit each
      auto wait = [&](uint32_t bar, uint32_t parity, int where) {
        const bool got = mbar_wait<true>(bar, parity, wd, where);
        tc_fence_after();
        return got;
      };
      bool ok = true;
      Job job;
      for (int it = 0; ok; ++it) {
        ok = wait(job_full(it & 1), (it >> 1) & 1, kWhereJob);
        if (!ok) break;
        job = jobs[it & 1];
        mbar_arrive(job_empty(it & 1));
        if (job.b == -2) break;
        const int blocks = job.t1 - job.t0;
        if (blocks == 0) continue;
        const bool pair = job.tiles == 2;
        const int keys0 = tile_keys(job, 0) - job.t0 * kRows, keys1 = pair ? tile_keys(job, 1) - job.t0 * kRows : keys0;
        const int mine0 = tile_blocks(job, 0);
        ok = wait(q_full, q_uses & 1, kWhereMmaFull);
        ++q_uses;
        // Step s: O_t += P_t V_j, then the scores of the block that tile t has next; t = s & 1, and j goes up every
        // other step (two row tiles) or every step (one, whose even and odd blocks are two).  Steps -2 and -1 have scores alone.
        // One copy of the code: instructions that it takes twice as many of are not there when they are wanted, and this
        // thread's time is in every tile's way.
        const int steps = pair ? 2 * blocks : blocks;
#pragma unroll 1
        for (int step = -2; step < steps && ok; ++step) {
          const int t = step & 1, j = pair ? step >> 1 : step, next = j + (pair ? 1 : 2);
          const bool first_of = !pair || t == 0, last_of = !pair || t == 1;  // of the steps that share K and V
          // What is due early is waited for before the weights are: a wait takes 300 cycles where its phase has long passed (the
          // tensor cores have shared memory to themselves).
          if (first_of) {
            if (j >= 0) ok = wait(h_full(h_stage), h_phase, kWhereMmaFull);
            if (ok && next < blocks) ok = wait(k_full(k_stage), k_phase, kWhereMmaFull);
            if (!ok) break;
          }
          const int keys = t ? keys1 : keys0, mine = pair ? (t ? blocks : mine0) : blocks;
          const uint32_t s_col = tmem + t * 128, o_col = s_col + 256;
          if (j >= 0 && j < mine) {  // what is stored first, then the rest
            const uint64_t v = smem_desc(base + L::kOffHalf + h_stage * L::kHalf, L::kBox, 1024, 2);
            constexpr uint32_t idesc = instr_desc(0, 0, kRows, HD) | kIdescBMajorN;
            const int parts = (min(kRows, keys - j * kRows) + 15) / 16;
            const bool first = pair ? j == 0 : j < 2;
            ok = wait(p_half(t), (turn >> t) & 1, kWhereMmaTmemEmpty);
            if (!ok) break;
#pragma unroll
            for (int i = 0; i < kEarly; ++i)
              if (i < parts) mma_f16_ts(o_col, s_col + i * 8, desc_advance(v, i * 2048), idesc, !(first && i == 0));
            ok = wait(p_full(t), (turn >> t) & 1, kWhereMmaTmemEmpty);
            if (!ok) break;
#pragma unroll
            for (int i = kEarly; i < 8; ++i)
              if (i < parts) mma_f16_ts(o_col, s_col + i * 8, desc_advance(v, i * 2048), idesc, 1);
            turn ^= 1u << t;
            if (pair ? next == mine : next >= blocks) mma_commit(o_full(t));
          }
          if (next < mine) {  // S_t = Q K^T, in two terms
            const int n = (min(kRows, keys - next * kRows) + 15) & ~15;
            const uint64_t k = kmajor_sw128_desc(base + L::kOffK + k_stage * L::kTile), a = kmajor_sw128_desc(q_tile(pair ? t : 0, 0));
#pragma unroll
            for (int term = 0; term < 2; ++term) {
              const uint32_t idesc = instr_desc(term, 0, kRows, n);  // e4m3, then e5m2
#pragma unroll
              for (int i = 0; i < HD / 32; ++i)
                mma_f8f6f4(s_col, desc_advance(a, term * L::kTile + i * 32), desc_advance(k, i * 32), idesc, (term | i) != 0);
            }
            mma_commit(s_full(t));
          }
          if (last_of) {
            if (j >= 0) {
              mma_commit(h_empty(h_stage));
              if (++h_stage == HS) {
                h_stage = 0;
                h_phase ^= 1;
              }
            }
            if (next < blocks) {
              mma_commit(k_empty(k_stage));
              if (++k_stage == KS) {
                k_stage = 0;
                k_phase ^= 1;
              }
              if (next + 1 == blocks) mma_commit(q_empty);  // the job's last scores
            }
          }
        }
      }
      // every MMA has finished and every commit has landed before the CTA exits
      mma_commit(drain_bar);
      mbar_wait_drain(drain_bar, 0, 200000000ull);
    }
  } else {
    reg_inc<kSoftmaxRegs>();
    // ---------------- softmax and output ----------------
    const int t = warp >> 2, quarter = warp & 3;
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t s_addr = tmem + lanes + t * 128, o_addr = tmem + lanes + 256;
    const int row = quarter * 32 + lane;
    uint32_t turn = 0, outputs = 0, merges = 0;  // parities of the next scores, output, meeting of the halves
    int count = 0;                               // key blocks of the jobs before
    auto tile_wait = [&](uint32_t bar, uint32_t parity, int where) {
      const bool got = __all_sync(0xffffffffu, mbar_wait(bar, parity, wd, where));
      tc_fence_after();
      return got;
    };
    auto take_job = [&](int i, Job& job) {  // false: no more, or the CTA gives up
      if (!tile_wait(job_full(i & 1), (i >> 1) & 1, kWhereJob)) return false;
      read(i, job);
      return job.b != -2;
    };
    int q_fills = 0;
    // The query rows of a job that has key blocks, as two terms: a share of them a warp.  Past the job's scores that
    // came before; false: the CTA gives up.
    auto queries = [&](int i, const Job& job) {
      if (q_fills > 0 && !tile_wait(q_empty, (q_fills - 1) & 1, kWhereConvert)) return false;
      ++q_fills;
      // HD / 8 lanes a row, 8 dimensions each
      constexpr int kLanes = HD / 8, kAtOnce = 32 / kLanes, kFlight = 8;
      const int d = 8 * (lane % kLanes), share = job.tiles == 2 ? 32 : 16, tile = job.tiles == 2 ? t : 0;
      const int rows = min(job.lq - job.first - tile * tile_tokens, tile_tokens) * p.pack;  // those that have a query
      const uint32_t hi_tile = q_tile(tile, 0), factors = base + L::kOffRow + (((i & 1) * 2 + tile) * kRows) * 4;
      const int begin = (job.tiles == 2 ? quarter : warp) * share + lane / kLanes;
      const uint16_t* const from = p.q + static_cast<int64_t>(job.q0 + job.first + tile * tile_tokens) * p.q_stride + job.head0 * p.D + d;
      auto fetch = [&](int r) {  // rows without a query are zeros, so that what their threads find does not vary
        const int token = r * p.pack_inverse >> 16;
        return r < rows && d < p.D ? *reinterpret_cast<const uint4*>(from + token * p.q_stride + (r - token * p.pack) * p.D) : make_uint4(0, 0, 0, 0);
      };
      uint4 flight[kFlight];
#pragma unroll
      for (int k = 0; k < kFlight; ++k) flight[k] = fetch(begin + k * kAtOnce);
#pragma unroll 1
      for (int r = begin; r < begin + share; r += kAtOnce) {
        const uint32_t w[4] = {flight[0].x, flight[0].y, flight[0].z, flight[0].w};
#pragma unroll
        for (int k = 1; k < kFlight; ++k) flight[k - 1] = flight[k];
        flight[kFlight - 1] = fetch(r + kFlight * kAtOnce < begin + share ? r + kFlight * kAtOnce : kRows);
        float x[8];
        float top = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[2 * e] = __uint_as_float(w[e] << 16);
          x[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
          top = max3(top, fabsf(x[2 * e]), fabsf(x[2 * e + 1]));
        }
#pragma unroll
        for (int o = 1; o < kLanes; o <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        // The row's largest value to [2^7, 2^8).  A row with an infinity has NaN for all of its codes, as a row with NaN has for one: every
        // score is NaN then, and those of keys that the row does not see are put out like any other's, which a factor that is NaN would undo.
        const int field = min(261 - static_cast<int>(__float_as_uint(top) >> 23), 253);
        const float up = __uint_as_float(top == INFINITY ? 0x7FC00000u : static_cast<uint32_t>(field) << 23);
        uint32_t hi[2], lo[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          hi[e] = lo[e] = 0;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float a = x[4 * e + 2 * h] * up, b = x[4 * e + 2 * h + 1] * up;
            const uint32_t code = to_e4m3x2(a, b);
            float ha, hb;
            half2_floats(from_e4m3x2(code), ha, hb);
            hi[e] |= code << (16 * h);
            lo[e] |= to_e5m2x2(a - ha, b - hb) << (16 * h);
          }
        }
        const uint32_t at = hi_tile + r * 128 + (((d >> 4) ^ (r & 7)) << 4) + (d & 8);
        st_shared_v2(at, hi[0], hi[1]);
        st_shared_v2(at + L::kTile, lo[0], lo[1]);
        if (d == 0) st_shared(factors + r * 4, static_cast<uint32_t>(254 - field) << 23);  // 1 / up
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full);
      return true;
    };
    bool ok = true;
    {
      Job job;
      if (take_job(0, job) && job.t1 > job.t0) ok = queries(0, job);
    }
#pragma unroll 1
    for (int it = 0; ok; ++it) {
      int n, lim, t0, each, blocks;  // key blocks of this tile; keys that this row sees; the job's first block; blocks from one to the next
      bool halves, idle;
      {
        Job job;
        if (!take_job(it, job)) break;
        halves = job.tiles == 1;
        n = tile_blocks(job, t);
        blocks = job.t1 - job.t0;
        t0 = job.t0 + (halves ? t : 0);
        each = halves ? 2 : 1;
        const int tok = job.first + (halves ? 0 : t * tile_tokens) + (row * p.pack_inverse >> 16);
        idle = row >= tile_tokens * p.pack || tok >= job.lq;
        lim = idle ? tile_keys(job, halves ? 0 : t) : visible(job, tok);  // past a tile's keys its scores are not formed
      }
      float factor = 0.f;                 // of the query row's codes
      float m = kUnset, nn = kUnset;      // references, in log2 units: of scores, of the output's weights (relative to m)
      float sum = 0.f;
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        // What shared memory holds is read before the scores are there: operands that the tensor cores take from it
        // keep a load waiting for hundreds of cycles.
        const uint32_t block = count + (halves ? 2 * j + t : j), slot = block & (L::kInfo - 1);
        ok = tile_wait(info_full(slot), (block / L::kInfo) & 1, kWhereEpiTmemFull);
        if (!ok) break;
        // of the 16-key blocks: factors of their scores, exponents of their values and the inverses of those
        float g[8], b[8], inverse[8];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float4 x = ld_shared_f4(base + L::kOffInfo + slot * 64 + c * 16), y = ld_shared_f4(base + L::kOffInfo + slot * 64 + 32 + c * 16);
          const float4 z = ld_shared_f4(base + L::kOffInverse + slot * 32 + c * 16);
          g[4 * c] = x.x, g[4 * c + 1] = x.y, g[4 * c + 2] = x.z, g[4 * c + 3] = x.w;
          b[4 * c] = y.x, b[4 * c + 1] = y.y, b[4 * c + 2] = y.z, b[4 * c + 3] = y.w;
          inverse[4 * c] = z.x, inverse[4 * c + 1] = z.y, inverse[4 * c + 2] = z.z, inverse[4 * c + 3] = z.w;
        }
        const float4 more = ld_shared_f4(base + L::kOffMask + slot * 16);
        const uint32_t about = __float_as_uint(more.x), gone = about & 255;
        const float least = more.y, most = more.z;
        ok = tile_wait(s_full(t), turn, kWhereEpiTmemFull);
        turn ^= 1;
        if (!ok) break;
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(s_addr + 32 * c, s[c]);  // past the last key: hidden below
        if (j == 0) factor = idle ? 1.f : __uint_as_float(ld_shared(base + L::kOffRow + (((it & 1) * 2 + (halves ? 0 : t)) * kRows + row) * 4));
#pragma unroll
        for (int c = 0; c < 8; ++c) g[c] *= factor;
        const int room = lim - (t0 + each * j) * kRows;
        const bool edge = __any_sync(0xffffffffu, room < kRows) || gone;
        tmem_wait_ld();
        bool slow = (about >> 16) != 0;
        if (__builtin_expect(edge, 0)) {
          slow |= __any_sync(0xffffffffu, factor < kLight);
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const int left = (gone >> c) & 1 ? 0 : room - 16 * c;
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (i >= left) s[c / 2][c % 2 * 16 + i] = 0xFF800000u;
          }
        }
        float top[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          float x = -INFINITY, y = -INFINITY;
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            x = max3(x, __uint_as_float(s[c / 2][c % 2 * 16 + i]), __uint_as_float(s[c / 2][c % 2 * 16 + i + 1]));
            y = max3(y, __uint_as_float(s[c / 2][c % 2 * 16 + i + 2]), __uint_as_float(s[c / 2][c % 2 * 16 + i + 3]));
          }
          x = fmaxf(x, y);
          top[c] = __fmul_rn(x, g[c]);  // rounded, as m will be; a scale that is NaN leaves the maximum alone
        }
        const float mx = fmaxf(max3(max3(top[0], top[1], top[2]), top[3], top[4]), max3(top[5], top[6], top[7]));
        // may a reference have to move?  (the largest exponent stands for those of the largest scores)
        if (__builtin_expect(__any_sync(0xffffffffu, mx > m + kSlack || (mx - m) + most > nn + (kLift + kSlack)), 0)) {
          const float up = ceilf(mx);
          if (up > m) {
            sum *= ex2(m - up);
            nn += m - up;
            m = up;
          }
          float vx = -INFINITY;
#pragma unroll
          for (int c = 0; c < 8; ++c) vx = fmaxf(vx, (top[c] - m) + b[c]);
          vx = ceilf(vx) - kLift;
          const bool lift = vx > nn;
          const float by = lift ? ex2(nn - vx) : 1.f;
          if (lift) nn = vx;
          if (j > 0 && __any_sync(0xffffffffu, lift)) {
            const uint64_t by2 = pack_f32x2(by, by);
#pragma unroll 1
            for (int c = 0; c < HD / 16; ++c) {  // S fills the registers: a little of O at a time
              uint32_t o[16];
              tmem_ld_32x32b_x16(o_addr + t * 128 + 16 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                float x, y;
                unpack_f32x2(mul_f32x2(pack_f32x2(o[i], o[i + 1]), by2), x, y);
                o[i] = __float_as_uint(x), o[i + 1] = __float_as_uint(y);
              }
              tmem_st_32x32b_x16(o_addr + t * 128 + 16 * c, o);
            }
          }
        }
        // before a row has seen a key its references are unset: any do
        const float ref = m == kUnset ? 0.f : m, vref = m == kUnset ? 0.f : nn;
        slow |= __any_sync(0xffffffffu, fabsf(ref) > kExact || least - vref < kSpread);
        if (__builtin_expect(!slow, 1)) {
          const float off = -vref - ref;
          float sums[2] = {0.f, 0.f};  // of the weights without the values' scales, by 2^vref
          uint32_t w[16];              // two blocks' weights
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const uint64_t g2 = pack_f32x2(g[c], g[c]), b2 = pack_f32x2(b[c] + off, b[c] + off);
            uint64_t part = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float x, y;
              unpack_f32x2(fma_f32x2(pack_f32x2(s[c / 2][c % 2 * 16 + 2 * i], s[c / 2][c % 2 * 16 + 2 * i + 1]), g2, b2), x, y);
              x = ex2(x);
              y = ex2(y);
              part = i ? add_f32x2(part, pack_f32x2(x, y)) : pack_f32x2(x, y);
              w[c % 2 * 8 + i] = pack_f16x2(x, y);
            }
            float lo, hi;
            unpack_f32x2(part, lo, hi);
            sums[c & 1] = fmaf(lo + hi, inverse[c], sums[c & 1]);
            if (c & 1) {
              if (c / 2 == kEarly / 2) {  // by now what was stored before is there
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(p_half(t));
              }
              tmem_st_32x32b_x16(s_addr + 16 * (c / 2), w);
            }
          }
          sum = fmaf(sums[0] + sums[1], ex2(vref), sum);
        } else {
          // Score, difference and sum one by one, 16 keys at a time; scores are still in tensor memory, and
          // weights (half as wide) do not reach those that are yet to be read.  A row's sum takes a block's, and that 16 keys', as above: of
          // 130000 equal weights added one by one it is off by up to 2^-9.  (Even and odd keys: with one sum for both 4 chunks take 1203 us, 1182.)
          uint64_t total = 0;
#pragma unroll 1
          for (int c = 0; c < 8; ++c) {
            uint32_t x[16], w[8];
            tmem_ld_32x32b_x16(s_addr + 16 * c, x);
            const float by = __uint_as_float(ld_shared(base + L::kOffInfo + slot * 64 + c * 4)) * factor;
            const float lift = __uint_as_float(ld_shared(base + L::kOffInfo + slot * 64 + 32 + c * 4)) - vref;
            const int left = !edge ? 16 : (gone >> c) & 1 ? 0 : room - 16 * c;
            tmem_wait_ld();
            uint64_t part = 0;
            float plain[2];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float y = i < left ? __fsub_rn(__fmul_rn(__uint_as_float(x[i]), by), ref) : -INFINITY;
              x[i] = __float_as_uint(ex2(y + lift));
              plain[i & 1] = ex2(y);
              if (i & 1) part = add_f32x2(part, pack_f32x2(plain[0], plain[1]));
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) w[i] = pack_f16x2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
            tmem_st_32x32b_x8(s_addr + 8 * c, w);
            total = add_f32x2(total, part);
          }
          float even, odd;
          unpack_f32x2(total, even, odd);
          sum += even + odd;
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive(p_half(t));
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_full(t));
      }
      if (!ok) break;
      count += blocks;
      {  // the next job's queries, while the last product runs
        Job job;
        if (take_job(it + 1, job) && job.t1 > job.t0) ok = queries(it + 1, job);
      }
      if (n > 0 && ok) {
        ok = tile_wait(o_full(t), outputs, kWhereEpiTmemFull);
        outputs ^= 1;
      }
      if (!ok) break;
      // A tile's output is what its thread has; the even and odd blocks of a unit that has one tile have outputs of their own,
      // whose threads meet here: each then writes half of the dimensions of both.
      const uint32_t stats = base + L::kOffStats;
      auto meet = [&]() {
        mbar_arrive(merge_bar);
        return tile_wait(merge_bar, merges++ & 1, kWhereMerge);
      };
      float part0 = 1.f, part1 = 0.f;   // what the halves' outputs are multiplied by
      bool has0 = n > 0, has1 = false;  // of a tile of its own: has0
      if (halves) {
        st_shared_v4(stats + (t * kRows + row) * 16, __float_as_uint(m), __float_as_uint(nn), __float_as_uint(sum), n > 0);
        ok = meet();
        if (!ok) break;
        const uint4 x = ld_shared_v4(stats + ((t ^ 1) * kRows + row) * 16);
        const float m1 = __uint_as_float(x.x), n1 = __uint_as_float(x.y), sum1 = __uint_as_float(x.z);
        const float both = fmaxf(m, m1);
        const float d0 = m == kUnset ? kUnset : (m - both) + nn, d1 = m1 == kUnset ? kUnset : (m1 - both) + n1;
        const float most = fmaxf(d0, d1);
        const float a0 = sum * ex2(m - both), a1 = sum1 * ex2(m1 - both);
        sum = t == 0 ? a0 + a1 : a1 + a0;  // in the order of the halves, so that both form the same
        const float mine = ex2(d0 - most), other = ex2(d1 - most);
        part0 = t ? other : mine;
        part1 = t ? mine : other;
        has0 = t ? x.w != 0 : n > 0;
        has1 = t ? n > 0 : x.w != 0;
        m = both;
        nn = most;
      }
      Job job;
      read(it, job);  // again: scores left no room to keep it
      const int token = row * p.pack_inverse >> 16, tok = job.first + (halves ? 0 : t * tile_tokens) + token;
      const bool mine = row < tile_tokens * p.pack && tok < job.lq;
      // dimensions [from, from + width) of this row, 16 at a time
      const int width = halves ? HD / 2 : HD, from = halves ? t * (HD / 2) : 0;
      const uint32_t first_o = o_addr + (halves ? 0 : t * 128);
      auto load = [&](int c, uint32_t (&x)[16]) {
        if (has0) {
          tmem_ld_32x32b_x16(first_o + c, x);
          tmem_wait_ld();
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = 0;
        }
        if (halves) {
          uint32_t y[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] = 0;
          if (has1) {
            tmem_ld_32x32b_x16(o_addr + 128 + c, y);
            tmem_wait_ld();
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = __float_as_uint(fmaf(__uint_as_float(y[i]), part1, __uint_as_float(x[i]) * part0));
        }
      };
      const bool writes_row = t == 0 || !halves;  // what a row has once
      if (job.whole) {
        const bool none = sum == 0.f;
        const float root = ex2(0.5f * nn), by = root / sum;  // 2^n in two steps: by itself it may leave fp32's range
        const int64_t at = static_cast<int64_t>(job.q0 + tok) * p.Hq + job.head0 + row - token * p.pack;
        const uint64_t root2 = pack_f32x2(root, root), by2 = pack_f32x2(by, by);
#pragma unroll 1
        for (int c = from; c < from + width; c += 16) {
          uint32_t x[16];
          load(c, x);
          if (!mine) continue;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (c + 8 * i >= p.D) break;
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float a, b;
              unpack_f32x2(mul_f32x2(mul_f32x2(pack_f32x2(x[8 * i + 2 * e], x[8 * i + 2 * e + 1]), root2), by2), a, b);
              w[e] = none ? 0u : pack_bf16x2(a, b);
            }
            *reinterpret_cast<uint4*>(p.out + at * p.D + c + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
        if (mine && p.lse && writes_row) p.lse[at] = none ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
      } else {
        const int64_t tile = 2 * static_cast<int64_t>(job.slot) + (halves ? 0 : t);
        if (writes_row) p.part_ml[tile * kRows + row] = make_float4(m, nn, sum, 0.f);
        float* const out = p.part_o + tile * (kRows * HD);
        if (halves || has0) {
#pragma unroll 1
          for (int c = from; c < from + width; c += 16) {
            uint32_t x[16];
            load(c, x);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<uint4*>(out + ((c / 4 + i) * kRows + row) * 4) = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
          }
        }
      }
      tc_fence_before();  // the next job's weights are handed over after these loads
      if (halves && !(ok = meet())) break;  // and by neither half while the other reads its output or its numbers
      done(it);
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == kSoftmaxWarps + 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of a cut unit, a quarter of a row tile (32 rows, one a lane) a block; a warp has every eighth
// group of four dimensions.
constexpr int kJoinWarps = 8;

template <int HD>
__global__ void __launch_bounds__(32 * kJoinWarps) chunk_join_kernel(const ChunkParams p) {
  constexpr int kGroups = HD / 4 / kJoinWarps;
  __shared__ uint2 staged[32][HD / 4 + 1];
  // The next kernel starts when this one ends: started early, the next chunk call's CTAs go to SMs in the order in which they get free, and
  // neighbours in work, which read the same keys, lie on two dies (24 ungrouped in a row: 106 us, early 122; 40 mixed 296, 303; 4 chunks 1178, 1162).
  grid_dep_wait();
  const Cut cut = p.cuts[blockIdx.x];
  if (cut.last < 0) return;
  const int tile_tokens = kRows / p.pack, t = blockIdx.y >> 2;
  if (t >= cut.tiles) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = (blockIdx.y & 3) * 32 + lane;
  const int tok = cut.first + t * tile_tokens + row / p.pack;
  const bool mine = row < tile_tokens * p.pack && tok < cut.lq;
  if (!__syncthreads_or(mine)) return;
  const int parts = cut.last - cut.from + 1;
  auto tile_of = [&](int k) { return 2 * static_cast<int64_t>(2 * (cut.from + k) + (k == 0)) + t; };
  // the references: the largest of the parts'
  float m = kUnset;
#pragma unroll 4
  for (int k = 0; k < parts; ++k) m = fmaxf(m, p.part_ml[tile_of(k) * kRows + row].x);
  float n = kUnset;
#pragma unroll 4
  for (int k = 0; k < parts; ++k) {
    const float4 ml = p.part_ml[tile_of(k) * kRows + row];
    if (ml.x != kUnset) n = fmaxf(n, (ml.x - m) + ml.y);
  }
  float sum = 0.f;
  float4 o[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) o[g] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int k = 0; k < parts; ++k) {
    const int64_t tile = tile_of(k);
    const float4 ml = p.part_ml[tile * kRows + row];
    sum += ml.z * ex2(ml.x - m);
    if (ml.x == kUnset && ml.z == 0.f) continue;  // it saw nothing, and its output may not be there
    const float by = ex2((ml.x - m) + (ml.y - n));
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const float4 x = *reinterpret_cast<const float4*>(p.part_o + tile * (kRows * HD) + ((warp + kJoinWarps * g) * kRows + row) * 4);
      o[g].x = fmaf(x.x, by, o[g].x);
      o[g].y = fmaf(x.y, by, o[g].y);
      o[g].z = fmaf(x.z, by, o[g].z);
      o[g].w = fmaf(x.w, by, o[g].w);
    }
  }
  const bool none = sum == 0.f;
  const float half = ex2(0.5f * n), by = half / sum;
#pragma unroll
  for (int g = 0; g < kGroups; ++g)
    staged[lane][warp + kJoinWarps * g] =
        none ? make_uint2(0, 0)
             : make_uint2(pack_bf16x2(o[g].x * half * by, o[g].y * half * by), pack_bf16x2(o[g].z * half * by, o[g].w * half * by));
  const int64_t at = static_cast<int64_t>(cut.q0 + tok) * p.Hq + cut.head0 + row % p.pack;
  if (warp == 0 && mine && p.lse) p.lse[at] = none ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
  __syncthreads();
  const int64_t to = mine ? at * p.D : -1;
#pragma unroll
  for (int r = warp; r < 32; r += kJoinWarps) {
    const int64_t there = __shfl_sync(0xffffffffu, to, r);
    if (there >= 0 && 4 * lane < p.D) *reinterpret_cast<uint2*>(p.out + there + 4 * lane) = staged[r][lane];
  }
}

int heads_packed(int group) {
  int pack = 1;
  for (int g = 2; g <= group && g <= kRows; ++g)
    if (group % g == 0 && kRows % g <= kRows / 16) pack = g;
  return pack;
}

sg_status_t launch_error(cudaError_t e) {
  if (e == cudaSuccess) return SG_OK;
  note_cuda_error(e);
  cudaGetLastError();
  return SG_ERR_CUDA;
}

template <int HD>
sg_status_t launch(const AttnShape& s, const AttnArgs& a, const ChunkParams& p) {
  const uint64_t D = s.D, rows = static_cast<uint64_t>(s.Hk) * s.page;
  const uint64_t dims[3] = {D, rows, static_cast<uint64_t>(a.cache.num_pages)};
  const uint64_t sk[2] = {D, static_cast<uint64_t>(a.cache.k_page_stride)}, sv[2] = {D, static_cast<uint64_t>(a.cache.v_page_stride)};
  // K rows take 128 bytes whatever D is, the rest of them zeros: one layout for the tensor cores
  const uint32_t bk[3] = {128, static_cast<uint32_t>(s.page), 1}, bv[3] = {HD, static_cast<uint32_t>(s.page), 1};
  CUtensorMap tmK, tmV;
  if (!encode_3d(&tmK, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.cache.k, dims, sk, bk, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_3d(&tmV, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.cache.v, dims, sv, bv,
                 HD == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE))
    return SG_ERR_CUDA;
  GemmLaunch l(dim3(s.num_sms), dim3(kThreads), ChunkLayout<HD>::kDynSmem, a.stream, 1);
  const sg_status_t r = launch_error(cudaLaunchKernelEx(&l.cfg, chunk_kernel<HD>, tmK, tmV, p));
  if (r != SG_OK) return r;
  GemmLaunch j(dim3(s.num_sms, 8), dim3(32 * kJoinWarps), 0, a.stream, 1);
  return launch_error(cudaLaunchKernelEx(&j.cfg, chunk_join_kernel<HD>, p));
}

template <int HD>
cudaError_t prepare() {
  return cudaFuncSetAttribute(chunk_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, ChunkLayout<HD>::kDynSmem);
}

}  // namespace

size_t chunk_workspace_bytes(const AttnShape& s) {
  return static_cast<size_t>(s.num_sms) * (2 * 2 * kRows * (128 * sizeof(float) + sizeof(float4)) + sizeof(Cut));
}

cudaError_t chunk_prepare() {
  const cudaError_t e = prepare<64>();
  return e == cudaSuccess ? prepare<128>() : e;
}

sg_status_t chunk_launch(const AttnShape& s, const AttnArgs& a) {
  ChunkParams p{};
  p.q = static_cast<const uint16_t*>(a.q);
  p.q_stride = a.q_stride;
  p.table = a.table;
  p.lens = a.lens;
  p.cu = a.cu_q;
  p.table_stride = a.cache.num_pages > 0 ? a.table_stride : 0;  // no page, no keys
  p.k_scale = a.cache.k_scale;
  p.v_scale = a.cache.v_scale;
  p.num_pages = a.cache.num_pages;
  p.T = static_cast<int>(a.Tq);
  p.B = static_cast<int>(a.B);
  p.Hq = s.Hq;
  p.Hk = s.Hk;
  p.D = s.D;
  p.page = s.page;
  while ((1 << p.page_shift) < s.page) ++p.page_shift;
  p.group = s.Hq / s.Hk;
  p.pack = heads_packed(p.group);
  p.pack_inverse = 65536 / p.pack + 1;
  p.head_groups = s.Hq / p.pack;
  p.skip = s.skip_tile;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  p.part_o = static_cast<float*>(s.workspace);
  p.part_ml = reinterpret_cast<float4*>(p.part_o + static_cast<size_t>(s.num_sms) * 2 * 2 * kRows * 128);
  p.cuts = reinterpret_cast<Cut*>(p.part_ml + static_cast<size_t>(s.num_sms) * 2 * 2 * kRows);
  p.status = s.status;
  p.timeout_ns = s.timeout_ns;
  AttnArgs args = a;
  if (args.cache.num_pages == 0) {  // a tensor map has no empty dimension; nothing reads it
    args.cache.num_pages = 1;
    args.cache.k = args.cache.v = const_cast<void*>(a.q);
    args.cache.k_page_stride = args.cache.v_page_stride = static_cast<int64_t>(s.Hk) * s.page * s.D;
  }
  return s.D > 64 ? launch<128>(s, args, p) : launch<64>(s, args, p);
}

}  // namespace sg
