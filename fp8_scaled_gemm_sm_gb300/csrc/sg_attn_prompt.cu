// sg_attn_prompt.cu -- attention over whole packed prompts (scaled_attn_prompt).
//
// For query row i of a sequence with n queries and m keys, over the keys
// j <= i + m - n (causal) or all m,
//     s_j = scale q_i . k_j,   o_i = sum_j 2^(c s_j - r) v_j / sum_j 2^(c s_j - r),   c = log2 e,
// in one pass over tiles of 128 keys.  r is a reference that follows the running
// maximum: any r gives the same quotient, so it is moved only when the maximum has
// passed it by more than 2^8 (weights up to 2^8 lose nothing in fp32 or bf16), which
// makes rescaling the output rare.
//
// Rows are packed: a tile's 128 rows are 128 / G tokens times G query heads of one
// key/value head (G the largest divisor of the group that leaves at most 8 rows idle), so grouped heads share
// each K and V tile, the causal edge wastes less, and short prompts fill rows.
// A CTA owns two such row tiles and runs them in opposition: while the tensor
// cores work for one, the other's softmax runs.  Per CTA:
//   warps 0-3, 4-7  softmax of tile 0 / 1, one thread a row: S from tensor memory to
//                   registers, maximum, 2^x, row sum, P = bf16 back over S's columns; at the end
//                   the output rows, divided by the sums, through shared memory to whole lines.
//   warp 8          TMA producer: both Q tiles, then K_0, V_0, K_1, V_1, ... through a ring.
//   warp 9          MMA issuer, one elected thread: S_t = Q_t K_j^T (operands in shared memory), O_t +=
//                   P_t V_j (P in tensor memory, V as it lies in memory: N-major).
//   warp 10         V rows past a sequence's end (below).
//   warp 11         what to do: the unit that the CTA was launched for, then those of CTAs that have not
//                   been launched yet, which it takes over before their time (cluster launch control): the next unit's
//                   loads and first scores go with this one's last softmax and output.  Launched one by one, a CTA a
//                   unit, a unit costs 6.7 us beside its blocks, taken over 3.5.
// The tensor cores take the MMAs in order, so S_t of block j + 1, issued after
// O_t += P_t V_j, cannot overwrite P_t early, and a softmax thread that sees it
// complete may also touch O_t.
// P is rounded to bf16 (V is bf16, and an MMA has one operand type): an error of at most 2^-8 of each weight,
// as the output's own rounding; the row sums take the unrounded weights.
//
// What bounds it: the tensor pipe, but for a unit's first and last softmax and its output: a block of both tiles
// takes 1.33 us, 1.9 PFLOP/s.  16384 tokens, 32 heads of 128 over 8, causal: 1240 us a launch by itself, 1.77 PFLOP/s, 91% of
// what the library's bf16 GEMM reaches in a burst; launched on and on, under the power cap, 1376 us, 1.60 PFLOP/s, 92% of what that
// reaches for seconds.  6 chunks of 300 to 2048 tokens behind contexts, 40 heads over 8: 295 us, 316 in a loop.  Measured
// beside it, launches by themselves: a CTA a unit 1275 and 323 us; output a row a lane 1257 and 309; key columns past a block's last key
// skipped in the loads and exponentials (they are hidden, and only the last block has any; the branches cost every
// block) 1377 us for the 16384 tokens, and, of that form, one S buffer a tile with P elsewhere 1509 us, 64-key
// blocks with two S buffers 1612, MMAs issued by lane 0 under a plain branch instead of one elected thread 1520.
//
// V rows past a sequence's end belong to the next one: those that share a 16-key
// MMA step with valid ones are zeroed in shared memory, the rest are not multiplied.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cfloat>

#include "sg_attn.h"
#include "sg_attn_ptx.cuh"

namespace sg {

namespace {

constexpr int kRows = 128;   // rows of a tile, keys of a block
constexpr int kThreads = 384;
// Registers a thread of the softmax warpgroups and of the third: 2 x 208 + 88 = 3 x 168, what the block is
// launched with (192 and 120: 334 us instead of 309 for the chunks above).
constexpr int kSoftmaxRegs = 208, kIssueRegs = 88;
constexpr int kWhereJob = 0x41;  // a wait for a job, beside those of sg_ptx.cuh
constexpr int kJobReaders = 11;  // warps that take jobs
constexpr int kAhead = 8;  // loads before a job's end at which the next one is looked for (chunks: 294.7 us, 298 with 4)
constexpr int kEarly = 4;  // 16-key steps of a block whose weights are handed over first
constexpr int kTileKeys = 64, kTileThreads = 192;  // of the kernel with one row tile a CTA
constexpr float kSlack = 8.f;  // log2 of the largest weight
constexpr float kFar = 1073741824.f;  // references past this are not stood by (row_sum)

struct PromptParams {
  const int32_t *cu_q, *cu_k;
  int Tq, Tk, B, Hq, D, causal;
  int group;            // query heads of a key/value head
  int pack;             // query heads packed into a tile
  int head_groups;      // Hq / pack
  int units;
  int skip;             // number of a key block that is not loaded (scaled_attn_set_debug); -1: none
  float scale_log2;
  uint16_t* out;
  float* lse;
  int* status;
  uint64_t timeout_ns;
};

// What a CTA works on: `tokens` consecutive query tokens of a sequence.
struct Unit {
  int b;            // sequence; -1: nothing
  int q0, lq;       // its first query and their number
  int k0, lk;       // its keys
  int first;        // the unit's first token in the sequence
};

__device__ __forceinline__ Unit sequence(const PromptParams& p, int b) {
  Unit u;
  u.b = b;
  u.q0 = min(max(__ldg(p.cu_q + b), 0), p.Tq);
  u.lq = max(min(max(__ldg(p.cu_q + b + 1), 0), p.Tq) - u.q0, 0);
  u.k0 = min(max(__ldg(p.cu_k + b), 0), p.Tk);
  u.lk = min(max(__ldg(p.cu_k + b + 1), u.k0), p.Tk) - u.k0;
  u.first = 0;
  return u;
}

// Unit `x` of all sequences' units of `tokens` tokens, those that see most keys first, so
// that the GPU does not end on a few long ones.  A unit's level is the number of
// its keys in units of tokens; the number of units at or above a level is a sum over sequences, one a
// lane and round, so a search for x's level takes a dozen warp sums.
// More than kPickRounds * 32 sequences are numbered from cu_q[b] / tokens + b
// (at most n / tokens + 1 units each), the last rows first.
constexpr int kPickRounds = 4;

__device__ __forceinline__ Unit pick_unit(const PromptParams& p, int x, int tokens, int lane) {
  if (p.B > kPickRounds * 32) {
    const int unit = p.units - 1 - x;
    int b = -1;
    for (int i = lane; i < p.B; i += 32) b += min(max(__ldg(p.cu_q + i), 0), p.Tq) / tokens + i <= unit;
    b = __reduce_add_sync(0xffffffffu, b) + 31;  // every lane began at -1
    Unit u{};
    u.b = -1;
    if (b < 0) return u;
    u = sequence(p, b);
    u.first = (unit - (u.q0 / tokens + b)) * tokens;
    if (u.first < 0 || u.first >= u.lq) u.b = -1;
    return u;
  }
  if (p.B == 1) {
    Unit u = sequence(p, 0);
    u.first = ((u.lq + tokens - 1) / tokens - 1 - x) * tokens;
    if (u.first < 0) u.b = -1;
    return u;
  }
  int n[kPickRounds], off[kPickRounds];  // a sequence's units, and the level below its first
  int top = 0;
#pragma unroll
  for (int r = 0; r < kPickRounds; ++r) {
    n[r] = off[r] = 0;
    if (32 * r + lane < p.B) {
      const Unit u = sequence(p, 32 * r + lane);
      n[r] = (u.lq + tokens - 1) / tokens;
      off[r] = (p.causal ? max(u.lk - u.lq, 0) : u.lk) / tokens;
      top = max(top, off[r] + (p.causal ? n[r] : 1));
    }
  }
  top = __reduce_max_sync(0xffffffffu, top);
  // units of a sequence at levels from `level` on: unit i is at off + i, or all at off
  auto above = [&](int r, int level) {
    return p.causal ? min(n[r], max(off[r] + n[r] - level, 0)) : (off[r] >= level ? n[r] : 0);
  };
  auto count = [&](int level) {
    int c = 0;
#pragma unroll
    for (int r = 0; r < kPickRounds; ++r)
      if (32 * r < p.B) c += above(r, level);
    return __reduce_add_sync(0xffffffffu, c);
  };
  int lo = 0, hi = top + 1;  // count(lo) > x >= count(hi)
  Unit u{};
  u.b = -1;
  if (count(0) <= x) return u;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (count(mid) > x) lo = mid; else hi = mid;
  }
  int rest = x - count(lo + 1);
#pragma unroll
  for (int r = 0; r < kPickRounds; ++r) {
    if (32 * r >= p.B) break;
    const int here = above(r, lo) - above(r, lo + 1);
    int scan = here;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, scan, o);
      if (lane >= o) scan += up;
    }
    const int all = __shfl_sync(0xffffffffu, scan, 31);
    if (rest < all) {
      const int owner = __ffs(__ballot_sync(0xffffffffu, rest < scan)) - 1;
      const int before = __shfl_sync(0xffffffffu, scan - here, owner), base = __shfl_sync(0xffffffffu, off[r], owner);
      u = sequence(p, 32 * r + owner);
      u.first = (p.causal ? lo - base : rest - before) * tokens;
      return u;
    }
    rest -= all;
  }
  return u;
}

// A row's sum; NaN where its reference is too large.  The weights come of fma's exact product less the rounded reference,
// off by up to half a unit in the reference's last place: all of a row share that, but past 2^31 it is a factor of
// 2^128, and sums are infinite or, worse, zero.  (Subtracting from the rounded product, for all rows or by a branch to the
// rows that need it, costs every call 2 to 3%.)
__device__ __forceinline__ float row_sum(float sum, float ref) {
  return fabsf(ref) > kFar && fabsf(ref) <= FLT_MAX ? __uint_as_float(0x7FC00000u) : sum;
}

// Two elements of an output row over its sum, as bf16.
__device__ __forceinline__ uint32_t scaled_pair(uint32_t x, uint32_t y, uint64_t by2) {
  float a, b;
  unpack_f32x2(mul_f32x2(pack_f32x2(__uint_as_float(x), __uint_as_float(y)), by2), a, b);
  return pack_bf16x2(a, b);
}

// One thread's row of the output: HD dimensions out of tensor memory, over its sum.
template <int HD>
__device__ __forceinline__ void put_row(const PromptParams& p, uint32_t o_addr, bool some, float sum, float ref, int q0, int tok,
                                        int lq, int head) {
  const bool none = sum == 0.f;
  const float inv = none ? 0.f : 1.f / sum;
  const uint64_t inv2 = pack_f32x2(inv, inv);
  const int64_t at = static_cast<int64_t>(q0 + tok) * p.Hq + head;
#pragma unroll
  for (int c = 0; c < HD / 32; ++c) {
    uint32_t o[32];
    if (some) {
      tmem_ld_32x32b_x32(o_addr + 32 * c, o);
      tmem_wait_ld();
    }
    if (tok < lq) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (32 * c + 8 * i < p.D) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            w[e] = none ? 0u : scaled_pair(o[8 * i + 2 * e], o[8 * i + 2 * e + 1], inv2);
          *reinterpret_cast<uint4*>(p.out + at * p.D + 32 * c + 8 * i) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
  }
  if (tok < lq && p.lse) p.lse[at] = none ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
}

// A warp's 32 rows of the output, a row a lane: HD dimensions out of tensor memory, over their sums, 64 at a time
// through 4 KB of shared memory at `stage`, so that a store writes whole lines (eight lanes a row): a row a lane
// wrote 32 lines at once, which took 2 us of a two-tile CTA's 128 x 2 rows.
template <int HD>
__device__ __forceinline__ void put_rows(const PromptParams& p, uint32_t o_addr, uint32_t stage, int lane, bool some, float sum,
                                         float ref, int q0, int tok, int lq, int head) {
  const bool none = sum == 0.f;
  const float inv = none ? 0.f : 1.f / sum;
  const uint64_t inv2 = pack_f32x2(inv, inv);
  const int64_t at = static_cast<int64_t>(q0 + tok) * p.Hq + head;
  const int64_t mine = tok < lq ? at * p.D : -1;
#pragma unroll
  for (int h = 0; h < HD / 64; ++h) {
    __syncwarp();  // what was staged before has been read
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t o[32];
      if (some) {
        tmem_ld_32x32b_x32(o_addr + 64 * h + 32 * c, o);
        tmem_wait_ld();
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          w[e] = none ? 0u : scaled_pair(o[8 * i + 2 * e], o[8 * i + 2 * e + 1], inv2);
        st_shared_v4(stage + lane * 128 + (((4 * c + i) ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
      }
    }
    __syncwarp();
    const int piece = lane & 7, d = 64 * h + 8 * piece;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = 4 * i + (lane >> 3);
      const int64_t to = __shfl_sync(0xffffffffu, mine, r);
      uint4 v;
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                   : "r"(stage + r * 128 + ((piece ^ (r & 7)) << 4))
                   : "memory");
      if (to >= 0 && d < p.D) *reinterpret_cast<uint4*>(p.out + to + d) = v;
    }
  }
  if (tok < lq && p.lse) p.lse[at] = none ? -INFINITY : (ref + log2f(sum)) * 0.6931471805599453f;
}

struct PromptLayout {
  static constexpr int HD = 128;
  static constexpr int kBoxes = HD / 64;                  // 64-column (128-byte) boxes of a row
  static constexpr int kBox = kRows * 128;                // bytes of a box
  static constexpr int kTile = kBoxes * kBox;             // a Q, K or V tile
  static constexpr int kStages = 4;
  static constexpr int kOffKv = 2 * kTile;
  static constexpr int kOffOut = kOffKv + kStages * kTile;  // 4 KB a softmax warp
  static constexpr int kOffBar = kOffOut + 8 * 4096;
  static constexpr int kNumBars = 2 * kStages + 20;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kOffJobs = kOffMisc + 16;
  static constexpr int kOffAnswer = kOffJobs + 2 * 32;
  static constexpr int kBytes = kOffAnswer + 16;
  static constexpr int kDynSmem = kBytes + 1024;
  static_assert(kOffAnswer % 16 == 0 && kDynSmem <= 232448, "shared memory");
};

// A unit and the first query head of its rows.  u.b: -1 nothing, -2 no more.
struct Job {
  Unit u;
  int head0, unused;
};

__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const PromptParams p) {
  using L = PromptLayout;
  constexpr int HD = L::HD;
  constexpr int S = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sQ = smem_addr(smem), sKv = smem_addr(smem + L::kOffKv), bar0 = smem_addr(smem + L::kOffBar);
  auto kv_full = [&](int s) { return bar0 + 8 * s; };
  auto kv_empty = [&](int s) { return bar0 + 8 * (S + s); };
  auto s_full = [&](int t) { return bar0 + 8 * (2 * S + t); };
  auto p_full = [&](int t) { return bar0 + 8 * (2 * S + 2 + t); };
  auto p_half = [&](int t) { return bar0 + 8 * (2 * S + 4 + t); };
  auto o_full = [&](int t) { return bar0 + 8 * (2 * S + 6 + t); };
  auto job_full = [&](int s) { return bar0 + 8 * (2 * S + 8 + s); };
  auto job_empty = [&](int s) { return bar0 + 8 * (2 * S + 10 + s); };
  const uint32_t q_full = bar0 + 8 * (2 * S + 12), q_empty = bar0 + 8 * (2 * S + 13), drain_bar = bar0 + 8 * (2 * S + 14);
  const uint32_t v_last = bar0 + 8 * (2 * S + 15), v_clean = bar0 + 8 * (2 * S + 16);
  const uint32_t more_wanted = bar0 + 8 * (2 * S + 17), answered = bar0 + 8 * (2 * S + 18);
  int* misc = reinterpret_cast<int*>(smem + L::kOffMisc);  // [0] TMEM base, [1] abort
  Job* jobs = reinterpret_cast<Job*>(smem + L::kOffJobs);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  grid_dep_wait();
  const int tile_tokens = kRows / p.pack;
  if (warp == 9) {
    tmem_alloc(smem_addr(&misc[0]), 512);
    tmem_relinquish();
  }
  if (tid == 32) {
    for (int s = 0; s < S; ++s) {
      mbar_init(kv_full(s), 1);
      mbar_init(kv_empty(s), 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(s_full(t), 1);
      mbar_init(p_half(t), kRows);
      mbar_init(p_full(t), kRows);
      mbar_init(o_full(t), 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(job_full(s), 1);
      mbar_init(job_empty(s), kJobReaders);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(v_last, 1);
    mbar_init(v_clean, 1);
    mbar_init(drain_bar, 1);
    mbar_init(more_wanted, 1);
    mbar_init(answered, 1);
    misc[1] = 0;
    fence_mbarrier_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_launch();  // not before tensor memory is there: a kernel that starts early may take all of an SM's and wait for this one
  const uint32_t tmem = static_cast<uint32_t>(misc[0]);
  const Watchdog wd{p.status, p.timeout_ns, reinterpret_cast<volatile int*>(&misc[1])};
  // Job i of this CTA; false: no more, or the CTA gives up.  A warp that has what it needs of it says so.
  auto read = [&](int i, Job& job) {
    const int4* from = reinterpret_cast<const int4*>(jobs + (i & 1));
    const int4 x = from[0], y = from[1];
    auto same = [](int v) { return __shfl_sync(0xffffffffu, v, 0); };
    job.u.b = same(x.x), job.u.q0 = same(x.y), job.u.lq = same(x.z), job.u.k0 = same(x.w);
    job.u.lk = same(y.x), job.u.first = same(y.y), job.head0 = same(y.z);
  };
  auto done = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(job_empty(i & 1));
  };
  auto peek = [&](int i, Job& job) {
    if (!__all_sync(0xffffffffu, mbar_wait(job_full(i & 1), (i >> 1) & 1, wd, kWhereJob))) return false;
    read(i, job);
    return job.u.b != -2;
  };
  auto take = [&](int i, Job& job) {
    const bool got = peek(i, job);
    if (got) done(i);
    return got;
  };
  // What follows from a job.
  struct Plan {
    int kmax[2], blocks[2];  // keys that a tile's last row sees, its key blocks
    int num_blocks, past, tail_rows;
  };
  auto visible = [&](const Unit& u, int tok) { return p.causal ? min(u.lk, tok + 1 + u.lk - u.lq) : u.lk; };
  auto plan = [&](const Unit& u) {
    Plan x{};
    if (u.b < 0) return x;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int first = u.first + t * tile_tokens;
      x.kmax[t] = first < u.lq ? max(visible(u, min(first + tile_tokens, u.lq) - 1), 0) : 0;
      x.blocks[t] = (x.kmax[t] + kRows - 1) / kRows;
    }
    x.num_blocks = max(x.blocks[0], x.blocks[1]);
    // rows of the last V block that are not this sequence's but share a 16-key step with some that are
    x.past = u.lk - (x.num_blocks - 1) * kRows;
    x.tail_rows = x.num_blocks > 0 && x.past < kRows ? (16 - x.past) & 15 : 0;
    return x;
  };

  if (warp >= 8) {
    reg_dec<kIssueRegs>();
    Job job;
    if (warp == 8) {
      // ---------------- TMA producer ----------------
      const uint64_t once = l2_policy_evict_first(), keep = l2_policy_evict_last();
      int stage = 0, q_fills = 0;
      uint32_t phase = 0, issued = 0, last_par = 0;
      bool ok = true;
      for (int it = 0; ok && take(it, job); ++it) {
        const Plan x = plan(job.u);
        if (lane == 0) {
          if (x.num_blocks == 0) mbar_arrive(more_wanted);
          const int tiles = job.u.first + tile_tokens < job.u.lq ? 2 : 1;
          const int kv_head = job.head0 / p.group;
          for (int i = 0; i < 2 * x.num_blocks; ++i) {
            if (i == 0) {
              ok = q_fills == 0 || mbar_wait(q_empty, (q_fills - 1) & 1, wd, kWhereProducerEmpty);
              if (!ok) break;
              mbar_arrive_expect_tx(q_full, tiles * L::kBoxes * tile_tokens * p.pack * 128);
              for (int t = 0; t < tiles; ++t)
                for (int b = 0; b < L::kBoxes; ++b)
                  tma_load_3d_hint(sQ + t * L::kTile + b * L::kBox, &tmQ, b * 64, job.head0, job.u.q0 + job.u.first + t * tile_tokens,
                                   q_full, once);
              ++q_fills;
            }
            if (i == max(2 * x.num_blocks - kAhead, 0)) mbar_arrive(more_wanted);
            ok = mbar_wait(kv_empty(stage), phase ^ 1, wd, kWhereProducerEmpty);
            if (!ok) break;
            if (i != 2 * p.skip) {
              mbar_arrive_expect_tx(kv_full(stage), L::kTile);
              for (int b = 0; b < L::kBoxes; ++b)
                tma_load_3d_hint(sKv + stage * L::kTile + b * L::kBox, (i & 1) ? &tmV : &tmK, b * 64, kv_head,
                                 job.u.k0 + (i >> 1) * kRows, kv_full(stage), keep);
              issued |= 1u << stage;
              last_par = (last_par & ~(1u << stage)) | (phase << stage);
            }
            if (++stage == S) {
              stage = 0;
              phase ^= 1;
            }
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      if (lane == 0) {  // loads in flight must land before the CTA can exit (all have, unless it gave up)
        if (q_fills > 0) mbar_wait_drain(q_full, (q_fills - 1) & 1, 200000000ull);
        for (int s = 0; s < S; ++s)
          if ((issued >> s) & 1) mbar_wait_drain(kv_full(s), (last_par >> s) & 1, 200000000ull);
      }
    } else if (warp == 11) {
      // ---------------- jobs: this CTA's own, then those of CTAs not yet launched ----------------
      int next = static_cast<int>(blockIdx.x);
      for (int it = 0;; ++it) {
        if (it >= 2 && !__all_sync(0xffffffffu, mbar_wait(job_empty(it & 1), ((it >> 1) - 1) & 1, wd, kWhereJob))) break;
        Unit u{};
        u.b = -2;
        if (next >= 0) u = pick_unit(p, next / p.head_groups, 2 * tile_tokens, lane);
        if (lane == 0) {
          jobs[it & 1] = Job{u, max(next, 0) % p.head_groups * p.pack, 0};
          mbar_arrive(job_full(it & 1));
        }
        if (next < 0 || !__all_sync(0xffffffffu, mbar_wait(more_wanted, it & 1, wd, kWhereJob))) break;
        if (lane == 0) {
          fence_proxy_async_smem();  // the last answer has been read
          mbar_arrive_expect_tx(answered, 16);
          take_cta(smem_addr(smem + L::kOffAnswer), answered);
        }
        if (!__all_sync(0xffffffffu, mbar_wait(answered, it & 1, wd, kWhereJob))) {
          mbar_wait_drain(answered, it & 1, 200000000ull);  // before the CTA can exit
          break;
        }
        next = taken_cta(smem_addr(smem + L::kOffAnswer));
        __syncwarp();
      }
    } else if (warp == 10) {
      // ---------------- V rows past the sequence's end ----------------
      int loads = 0, tails = 0;  // before this job
      for (int it = 0; take(it, job); ++it) {
        const Plan x = plan(job.u);
        loads += 2 * x.num_blocks;
        if (x.tail_rows == 0) continue;
        const int st = (loads - 1) % S;  // the job's last V block
        if (!__all_sync(0xffffffffu, mbar_wait(v_last, tails++ & 1, wd, kWhereMmaFull))) break;
        for (int i = lane; i < x.tail_rows * 8 * L::kBoxes; i += 32)
          st_shared_v4(sKv + st * L::kTile + (i / (x.tail_rows * 8)) * L::kBox + x.past * 128 + (i % (x.tail_rows * 8)) * 16, 0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(v_clean);
      }
    } else if (elect_one()) {
      // ---------------- MMA issuer: one thread for all of it ----------------
      int stage = 0, q_uses = 0, tails = 0;
      uint32_t phase = 0, turn[2] = {0, 0};  // parity of a tile's next weights
      auto advance = [&]() {
        if (++stage == S) {
          stage = 0;
          phase ^= 1;
        }
      };
      auto wait = [&](uint32_t bar, uint32_t parity, int where) {
        const bool got = mbar_wait<true>(bar, parity, wd, where);
        tc_fence_after();
        return got;
      };
      bool ok = true;
      for (int it = 0; ok; ++it) {
        ok = wait(job_full(it & 1), (it >> 1) & 1, kWhereJob);
        if (!ok) break;
        job = jobs[it & 1];
        mbar_arrive(job_empty(it & 1));
        if (job.u.b == -2) break;
        const Plan x = plan(job.u);
        if (x.num_blocks == 0) continue;
        const int num_blocks = x.num_blocks;
        auto scores = [&](int t, int j) {  // S_t = Q_t K_j^T
          const int n = (min(kRows, x.kmax[t] - j * kRows) + 15) & ~15;
          const uint32_t idesc = instr_desc(1, 1, kRows, n);
          const uint64_t a = kmajor_sw128_desc(sQ + t * L::kTile), k = kmajor_sw128_desc(sKv + stage * L::kTile);
#pragma unroll
          for (int i = 0; i < HD / 16; ++i) {
            const uint32_t at = (i / 4) * L::kBox + (i % 4) * 32;
            mma_f16_ss(tmem + t * 128, desc_advance(a, at), desc_advance(k, at), idesc, i != 0);
          }
          mma_commit(s_full(t));
        };
        ok = wait(q_full, q_uses & 1, kWhereMmaFull) && wait(kv_full(stage), phase, kWhereMmaFull);
        if (ok) {
          if (x.blocks[0] > 0) scores(0, 0);
          if (x.blocks[1] > 0) scores(1, 0);
          mma_commit(kv_empty(stage));
          if (num_blocks == 1) mma_commit(q_empty);
          advance();
        }
        for (int j = 0; j < num_blocks && ok; ++j) {
          ok = wait(kv_full(stage), phase, kWhereMmaFull);  // V_j
          const int vs = stage;
          advance();
          if (ok && j + 1 == num_blocks && x.tail_rows > 0) {
            mbar_arrive(v_last);
            ok = wait(v_clean, tails & 1, kWhereMmaFull);
          }
          bool k_ready = false;
          const uint64_t v = smem_desc(sKv + vs * L::kTile, L::kBox, 1024, 2);
          constexpr uint32_t idesc = instr_desc(1, 1, kRows, HD) | kIdescBMajorN;
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            if (ok && j < x.blocks[t]) {
              const int steps = (min(kRows, x.kmax[t] - j * kRows) + 15) / 16;
              // O_t += P_t V_j: what is stored first, then the rest
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                ok = ok && wait(h ? p_full(t) : p_half(t), turn[t], kWhereMmaTmemEmpty);
                if (ok) {
#pragma unroll
                  for (int i = h ? kEarly : 0; i < (h ? 8 : kEarly); ++i)
                    if (i < steps)
                      mma_f16_ts(tmem + 256 + t * HD, tmem + t * 128 + i * 8, desc_advance(v, i * 2048), idesc, (j | i) != 0);
                  if (h && j + 1 == x.blocks[t]) mma_commit(o_full(t));
                }
              }
              turn[t] ^= 1;
              if (ok && j + 1 < x.blocks[t]) {
                if (!k_ready) ok = wait(kv_full(stage), phase, kWhereMmaFull);
                k_ready = true;
                if (ok) scores(t, j + 1);
              }
            }
          }
          mma_commit(kv_empty(vs));
          if (k_ready) {
            mma_commit(kv_empty(stage));
            advance();
            if (j + 2 == num_blocks) mma_commit(q_empty);  // the job's last scores
          }
        }
        ++q_uses;
        tails += x.tail_rows > 0;
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
    const uint32_t s_addr = tmem + lanes + t * 128, o_addr = tmem + lanes + 256 + t * HD;
    const int row = quarter * 32 + lane;
    const uint64_t scale2 = pack_f32x2(p.scale_log2, p.scale_log2);
    uint32_t turn = 0, outputs = 0;  // parities of the next scores, of the next output
    bool ok = true;
#pragma unroll 1
    for (int it = 0; ok; ++it) {
      int n, lim;  // key blocks; keys that this row sees
      bool nothing;
      {
        Job job;
        if (!peek(it, job)) break;
        nothing = job.u.b < 0;
        const Plan pl = plan(job.u);
        const int tok0 = job.u.first + t * tile_tokens;
        n = pl.blocks[t];
        lim = visible(job.u, row < tile_tokens * p.pack ? tok0 + row / p.pack : job.u.lq);
      }
      float ref = -INFINITY;      // r, in log2 units
      uint64_t sum2[2] = {0, 0};  // four partial row sums
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        ok = __all_sync(0xffffffffu, mbar_wait(s_full(t), turn, wd, kWhereEpiTmemFull));
        turn ^= 1;
        if (!ok) break;
        tc_fence_after();
        uint32_t s[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c)
          tmem_ld_32x32b_x32(s_addr + 32 * c, s[c]);  // past the last key: hidden below
        tmem_wait_ld();
        const int room = lim - j * kRows;
        if (__shfl_sync(0xffffffffu, room, 0) < kRows) {  // the first row sees least
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * c + i >= room) s[c][i] = 0xFF800000u;
        }
        float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};  // four chains: one would wait for itself
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; i += 2)
            tops[(i >> 1) & 3] = max3(tops[(i >> 1) & 3], __uint_as_float(s[c][i]), __uint_as_float(s[c][i + 1]));
        float mx = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]);
        mx *= p.scale_log2;
        if (j == 0) {
          ref = mx;
        } else {
          const bool move = mx > ref + kSlack;
          if (__any_sync(0xffffffffu, move)) {
            const float by = move ? ex2(ref - mx) : 1.f;
            if (move) ref = mx;
            const uint64_t by2 = pack_f32x2(by, by);
            sum2[0] = mul_f32x2(sum2[0], by2);
            sum2[1] = mul_f32x2(sum2[1], by2);
#pragma unroll 1
            for (int c = 0; c < HD / 16; ++c) {  // S fills the registers: a little of O at a time
              uint32_t o[16];
              tmem_ld_32x32b_x16(o_addr + 16 * c, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * by);
              tmem_st_32x32b_x16(o_addr + 16 * c, o);
            }
          }
        }
        const float neg = ref == -INFINITY ? 0.f : -ref;
        const uint64_t neg2 = pack_f32x2(neg, neg);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          {
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              float x, y;
              unpack_f32x2(fma_f32x2(pack_f32x2(s[c][2 * i], s[c][2 * i + 1]), scale2, neg2), x, y);
              x = ex2(x);
              y = ex2(y);
              sum2[i & 1] = add_f32x2(sum2[i & 1], pack_f32x2(x, y));
              w[i] = pack_bf16x2(x, y);
            }
            if (c == kEarly / 2) {  // by now what was stored before is there
              tmem_wait_st();
              tc_fence_before();
              mbar_arrive(p_half(t));
            }
            tmem_st_32x32b_x16(s_addr + 16 * c, w);
          }
      }
      tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_full(t));
      }
      if (n > 0 && ok) {
        ok = __all_sync(0xffffffffu, mbar_wait(o_full(t), outputs, wd, kWhereEpiTmemFull));
        outputs ^= 1;
      }
      if (ok && !nothing) {
        tc_fence_after();
        float lo, hi;
        unpack_f32x2(add_f32x2(sum2[0], sum2[1]), lo, hi);
        Job job;
        read(it, job);  // again: scores left no room to keep it
        put_rows<HD>(p, o_addr, smem_addr(smem + L::kOffOut) + warp * 4096, lane, n > 0, row_sum(lo + hi, ref), ref, job.u.q0,
                     row < tile_tokens * p.pack ? job.u.first + t * tile_tokens + row / p.pack : job.u.lq, job.u.lq,
                     job.head0 + row % p.pack);
        tc_fence_before();  // the next job's weights are handed over after these loads
      }
      done(it);
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---- one row tile a CTA --------------------------------------------------------
//
// Heads of up to 64 dimensions: an MMA is half as long and the softmax is not, so two tiles an SM leave
// the tensor cores waiting.  Here a CTA owns one row tile with 64 columns of tensor memory
// for scores of 64 keys (weights over them) and 64 for the output, and four
// CTAs share an SM: four softmaxes hide each other's waits, and the tiles are dealt out one by one, which
// ragged prompts need (29 of 1 to 2500 tokens, 16 heads of 64: 63.8 us, 94 with two tiles a CTA).  What bounds
// it is the softmax's instructions.  With heads of 128, two CTAs an SM, it is for short
// sequences (77 tokens, 32 heads over 8: 5.3 us).
//   warps 0-3  softmax and output, one thread a row
//   warp 4     TMA producer: Q, then K_0, V_0, K_1, V_1, ...; then V rows past the sequence's end
//   warp 5     MMA issuer, one elected thread

template <int HD>
struct TileLayout {
  static constexpr int kCtas = 256 / HD;                  // an SM
  static constexpr int kBoxes = HD / 64;
  static constexpr int kQBox = kRows * 128;
  static constexpr int kQTile = kBoxes * kQBox;
  static constexpr int kBox = kTileKeys * 128;
  static constexpr int kTile = kBoxes * kBox;             // a K or V block
  static constexpr int kStages = 4;
  static constexpr int kCols = 64 + HD <= 128 ? 128 : 256;  // tensor memory: S, then O
  static constexpr int kOffKv = kQTile;
  static constexpr int kOffBar = kOffKv + kStages * kTile;
  static constexpr int kNumBars = 2 * kStages + 7;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kBytes = kOffMisc + 48;
  static constexpr int kDynSmem = kBytes + 1024;
  static_assert(kCtas * (kDynSmem + 1024) <= 233472 && (kCtas + 1) * kDynSmem > 233472, "shared memory of kCtas CTAs, and no more");
};

template <int HD>
__global__ void __launch_bounds__(kTileThreads, TileLayout<HD>::kCtas)
    prompt_tile_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                       const __grid_constant__ CUtensorMap tmV, const PromptParams p) {
  using L = TileLayout<HD>;
  constexpr int S = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sQ = smem_addr(smem), sKv = smem_addr(smem + L::kOffKv), bar0 = smem_addr(smem + L::kOffBar);
  auto kv_full = [&](int s) { return bar0 + 8 * s; };
  auto kv_empty = [&](int s) { return bar0 + 8 * (S + s); };
  const uint32_t s_full = bar0 + 8 * (2 * S), p_full = s_full + 8, o_full = s_full + 16, q_full = s_full + 24;
  const uint32_t drain_bar = s_full + 32, v_last = s_full + 40, v_clean = s_full + 48;
  int* misc = reinterpret_cast<int*>(smem + L::kOffMisc);  // [0] TMEM base, [1] abort, [2..7] the unit
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  grid_dep_wait();
  const int tile_tokens = kRows / p.pack;
  const int head0 = static_cast<int>(blockIdx.x) % p.head_groups * p.pack;
  if (warp == 0) {
    const Unit u = pick_unit(p, static_cast<int>(blockIdx.x) / p.head_groups, tile_tokens, lane);
    if (lane == 0) *reinterpret_cast<Unit*>(misc + 2) = u;
  }
  if (warp == 5) {
    tmem_alloc(smem_addr(&misc[0]), L::kCols);
    tmem_relinquish();
  }
  if (tid == 32) {
    for (int i = 0; i < L::kNumBars; ++i) mbar_init(bar0 + 8 * i, bar0 + 8 * i == p_full ? kRows : 1);
    misc[1] = 0;
    fence_mbarrier_init();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_launch();  // not before tensor memory is there
  if (misc[2] < 0) {
    if (warp == 5) tmem_dealloc(static_cast<uint32_t>(misc[0]), L::kCols);
    return;
  }
  const int q0 = __shfl_sync(0xffffffffu, misc[3], 0), lq = __shfl_sync(0xffffffffu, misc[4], 0), k0 = __shfl_sync(0xffffffffu, misc[5], 0),
            lk = __shfl_sync(0xffffffffu, misc[6], 0), tok0 = __shfl_sync(0xffffffffu, misc[7], 0);
  auto visible = [&](int tok) { return p.causal ? min(lk, tok + 1 + lk - lq) : lk; };
  const int kmax = max(visible(min(tok0 + tile_tokens, lq) - 1), 0);  // keys that the last row sees
  const int n = (kmax + kTileKeys - 1) / kTileKeys;
  // rows of the last V block that are not this sequence's but share a 16-key step with some that are
  const int past = lk - (n - 1) * kTileKeys;
  const int tail_rows = n > 0 && past < kTileKeys ? (16 - past) & 15 : 0;
  const uint32_t tmem = static_cast<uint32_t>(misc[0]);
  const Watchdog wd{p.status, p.timeout_ns, reinterpret_cast<volatile int*>(&misc[1])};

  uint32_t issued = 0, last_par = 0;  // the producer's loads: stages, and the parities of their last
  if (warp == 4) {
    // ---------------- TMA producer ----------------
    if (lane == 0 && n > 0) {
      const uint64_t once = l2_policy_evict_first(), keep = l2_policy_evict_last();
      mbar_arrive_expect_tx(q_full, L::kBoxes * tile_tokens * p.pack * 128);
      for (int x = 0; x < L::kBoxes; ++x)
        tma_load_3d_hint(sQ + x * L::kQBox, &tmQ, x * 64, head0, q0 + tok0, q_full, once);
      const int kv_head = head0 / p.group;
      int stage = 0;
      uint32_t phase = 0;
      for (int i = 0; i < 2 * n; ++i) {
        if (!mbar_wait(kv_empty(stage), phase ^ 1, wd, kWhereProducerEmpty)) break;
        if (i != 2 * p.skip) {
          mbar_arrive_expect_tx(kv_full(stage), L::kTile);
          for (int x = 0; x < L::kBoxes; ++x)
            tma_load_3d_hint(sKv + stage * L::kTile + x * L::kBox, (i & 1) ? &tmV : &tmK, x * 64, kv_head,
                             k0 + (i >> 1) * kTileKeys, kv_full(stage), keep);
          issued |= 1u << stage;
          last_par = (last_par & ~(1u << stage)) | (phase << stage);
        }
        if (++stage == S) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    __syncwarp();
    if (tail_rows > 0 && __all_sync(0xffffffffu, mbar_wait(v_last, 0, wd, kWhereMmaFull))) {
      const int st = (2 * n - 1) % S;
      for (int i = lane; i < tail_rows * 8 * L::kBoxes; i += 32)
        st_shared_v4(sKv + st * L::kTile + (i / (tail_rows * 8)) * L::kBox + past * 128 + (i % (tail_rows * 8)) * 16, 0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(v_clean);
    }
  } else if (warp == 5) {
    // ---------------- MMA issuer ----------------
    if (n > 0 && elect_one()) {
      int stage = 0;
      uint32_t phase = 0;
      auto advance = [&]() {
        if (++stage == S) {
          stage = 0;
          phase ^= 1;
        }
      };
      auto wait = [&](uint32_t bar, uint32_t parity, int where) {
        const bool got = mbar_wait<true>(bar, parity, wd, where);
        tc_fence_after();
        return got;
      };
      auto scores = [&](int j) {  // S = Q K_j^T
        const int keys = (min(kTileKeys, kmax - j * kTileKeys) + 15) & ~15;
        const uint32_t idesc = instr_desc(1, 1, kRows, keys);
        const uint64_t a = kmajor_sw128_desc(sQ), k = kmajor_sw128_desc(sKv + stage * L::kTile);
#pragma unroll
        for (int i = 0; i < HD / 16; ++i)
          mma_f16_ss(tmem, desc_advance(a, (i / 4) * L::kQBox + (i % 4) * 32), desc_advance(k, (i / 4) * L::kBox + (i % 4) * 32),
                     idesc, i != 0);
        mma_commit(s_full);
        mma_commit(kv_empty(stage));
        advance();
      };
      bool ok = wait(q_full, 0, kWhereMmaFull) && wait(kv_full(0), 0, kWhereMmaFull);
      if (ok) scores(0);
      constexpr uint32_t idesc = instr_desc(1, 1, kRows, HD) | kIdescBMajorN;
      for (int j = 0; j < n && ok; ++j) {
        const int vs = stage;
        ok = wait(kv_full(vs), phase, kWhereMmaFull);
        advance();
        if (ok && j + 1 == n && tail_rows > 0) {
          mbar_arrive(v_last);
          ok = wait(v_clean, 0, kWhereMmaFull);
        }
        // K_j+1 as well, so that nothing is waited for between the two products
        if (ok && j + 1 < n) ok = wait(kv_full(stage), phase, kWhereMmaFull);
        ok = ok && wait(p_full, j & 1, kWhereMmaTmemEmpty);
        if (!ok) break;
        const uint64_t v = smem_desc(sKv + vs * L::kTile, L::kBox, 1024, 2);
        const int steps = (min(kTileKeys, kmax - j * kTileKeys) + 15) / 16;
#pragma unroll
        for (int i = 0; i < kTileKeys / 16; ++i)
          if (i < steps) mma_f16_ts(tmem + 64, tmem + i * 8, desc_advance(v, i * 2048), idesc, (j | i) != 0);
        if (j + 1 < n)
          scores(j + 1);
        else
          mma_commit(o_full);
        mma_commit(kv_empty(vs));
      }
      // every MMA has finished and every commit has landed before the CTA exits
      mma_commit(drain_bar);
      mbar_wait_drain(drain_bar, 0, 200000000ull);
    }
  } else {
    // ---------------- softmax and output ----------------
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    const uint32_t s_addr = tmem + lanes, o_addr = s_addr + 64;
    const int row = warp * 32 + lane;
    const int tok = row < tile_tokens * p.pack ? tok0 + row / p.pack : lq;  // lq: an idle row
    const int head = head0 + row % p.pack;
    const int lim = visible(tok);
    const int lim_warp = visible(tok0 + warp * 32 / p.pack);  // least of the warp's
    const uint64_t scale2 = pack_f32x2(p.scale_log2, p.scale_log2);
    float ref = -INFINITY;      // r, in log2 units
    uint64_t sum2[2] = {0, 0};  // four partial row sums
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      ok = __all_sync(0xffffffffu, mbar_wait(s_full, j & 1, wd, kWhereEpiTmemFull));
      if (!ok) break;
      tc_fence_after();
      const int room = lim - j * kTileKeys;
      const bool edge = lim_warp - j * kTileKeys < kTileKeys;
      // Where registers hold all 64 scores (two CTAs an SM) they are read once, else 32 at a time and twice,
      // for the maximum and for the weights.
      constexpr int kHeld = HD == 128 ? 2 : 1;  // times 32 scores
      const int chunks = kHeld == 2 ? 2 : (min(kTileKeys, kmax - j * kTileKeys) + 31) / 32;
      uint32_t s[kHeld][32];
      auto scores = [&](int c) {
#pragma unroll
        for (int k = 0; k < kHeld; ++k) tmem_ld_32x32b_x32(s_addr + 32 * (c + k), s[k]);
        tmem_wait_ld();
        if (edge) {
#pragma unroll
          for (int k = 0; k < kHeld; ++k)
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * (c + k) + i >= room) s[k][i] = 0xFF800000u;
        }
      };
      float tops[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
      for (int c = 0; c < chunks; c += kHeld) {
        scores(c);
#pragma unroll
        for (int i = 0; i < 32 * kHeld; i += 2)
          tops[(i >> 1) & 3] = max3(tops[(i >> 1) & 3], __uint_as_float(s[i / 32][i % 32]), __uint_as_float(s[i / 32][i % 32 + 1]));
      }
      const float mx = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]) * p.scale_log2;
      if (j == 0) {
        ref = mx;
      } else {
        const bool move = mx > ref + kSlack;
        if (__any_sync(0xffffffffu, move)) {
          const float by = move ? ex2(ref - mx) : 1.f;
          if (move) ref = mx;
          const uint64_t by2 = pack_f32x2(by, by);
          sum2[0] = mul_f32x2(sum2[0], by2);
          sum2[1] = mul_f32x2(sum2[1], by2);
#pragma unroll 1
          for (int c = 0; c < HD / 16; ++c) {  // S fills the registers: a little of O at a time
            uint32_t o[16];
            tmem_ld_32x32b_x16(o_addr + 16 * c, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * by);
            tmem_st_32x32b_x16(o_addr + 16 * c, o);
          }
        }
      }
      const float neg = ref == -INFINITY ? 0.f : -ref;
      const uint64_t neg2 = pack_f32x2(neg, neg);
#pragma unroll 1
      for (int c = 0; c < chunks; c += kHeld) {
        if (kHeld == 1) scores(c);
#pragma unroll
        for (int k = 0; k < kHeld; ++k) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float x, y;
            unpack_f32x2(fma_f32x2(pack_f32x2(s[k][2 * i], s[k][2 * i + 1]), scale2, neg2), x, y);
            x = ex2(x);
            y = ex2(y);
            sum2[i & 1] = add_f32x2(sum2[i & 1], pack_f32x2(x, y));
            w[i] = pack_bf16x2(x, y);
          }
          tmem_st_32x32b_x16(s_addr + 16 * (c + k), w);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(p_full);
    }
    if (n > 0 && ok) ok = __all_sync(0xffffffffu, mbar_wait(o_full, 0, wd, kWhereEpiTmemFull));
    if (ok) {
      tc_fence_after();
      float lo, hi;
      unpack_f32x2(add_f32x2(sum2[0], sum2[1]), lo, hi);
      put_row<HD>(p, o_addr, n > 0, row_sum(lo + hi, ref), ref, q0, tok, lq, head);
    }
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (misc[1] && warp == 4 && lane == 0 && n > 0) {  // somebody gave up: loads in flight must land before the CTA can exit
    mbar_wait_drain(q_full, 0, 200000000ull);
    for (int s = 0; s < S; ++s)
      if ((issued >> s) & 1) mbar_wait_drain(kv_full(s), (last_par >> s) & 1, 200000000ull);
  }
  if (warp == 5) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kCols);
  }
}

int heads_packed(int group) {
  int pack = 1;
  for (int g = 2; g <= group && g <= kRows; ++g)
    if (group % g == 0 && kRows % g <= kRows / 16) pack = g;
  return pack;
}

template <int HD, bool TILE>
sg_status_t launch(const AttnShape& s, const AttnArgs& a) {
  PromptParams p{};
  p.cu_q = a.cu_q;
  p.cu_k = a.cu_k;
  p.Tq = static_cast<int>(a.Tq);
  p.Tk = static_cast<int>(a.Tk);
  p.B = static_cast<int>(a.B);
  p.Hq = s.Hq;
  p.D = s.D;
  p.causal = a.causal;
  p.group = s.Hq / s.Hk;
  p.pack = heads_packed(p.group);
  p.head_groups = s.Hq / p.pack;
  const int64_t units = a.Tq / ((TILE ? 1 : 2) * (kRows / p.pack)) + a.B;
  if (units * p.head_groups >= (int64_t(1) << 31)) return SG_ERR_UNSUPPORTED_SHAPE;
  p.units = static_cast<int>(units);
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.out = static_cast<uint16_t*>(a.out);
  p.lse = a.lse;
  p.skip = s.skip_tile;
  p.status = s.status;
  p.timeout_ns = s.timeout_ns;
  // q as [tokens][heads][D]; without keys nothing reads the other two maps
  const bool keys = a.Tk > 0;
  const uint64_t el = 2, D = s.D;
  const uint64_t dq[3] = {D, static_cast<uint64_t>(s.Hq), static_cast<uint64_t>(a.Tq)};
  const uint64_t dk[3] = {D, static_cast<uint64_t>(s.Hk), static_cast<uint64_t>(keys ? a.Tk : a.Tq)};
  const uint64_t sq[2] = {D * el, static_cast<uint64_t>(a.q_stride) * el};
  const uint64_t sk[2] = {D * el, static_cast<uint64_t>(keys ? a.k_stride : a.q_stride) * el};
  const uint64_t sv[2] = {D * el, static_cast<uint64_t>(keys ? a.v_stride : a.q_stride) * el};
  const uint32_t bq[3] = {64, static_cast<uint32_t>(p.pack), static_cast<uint32_t>(kRows / p.pack)};
  const uint32_t bk[3] = {64, 1, TILE ? kTileKeys : kRows};
  CUtensorMap tmQ, tmK, tmV;
  if (!encode_3d(&tmQ, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, dq, sq, bq, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_3d(&tmK, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, keys ? a.k : a.q, dk, sk, bk, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_3d(&tmV, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, keys ? a.v : a.q, dk, sv, bk, CU_TENSOR_MAP_SWIZZLE_128B))
    return SG_ERR_CUDA;
  const dim3 grid(static_cast<unsigned>(units * p.head_groups));
  cudaError_t e;
  if constexpr (TILE) {
    GemmLaunch l(grid, dim3(kTileThreads), TileLayout<HD>::kDynSmem, a.stream, 1);
    e = cudaLaunchKernelEx(&l.cfg, prompt_tile_kernel<HD>, tmQ, tmK, tmV, p);
  } else {
    GemmLaunch l(grid, dim3(kThreads), PromptLayout::kDynSmem, a.stream, 1);
    e = cudaLaunchKernelEx(&l.cfg, prompt_kernel, tmQ, tmK, tmV, p);
  }
  if (e != cudaSuccess) {
    note_cuda_error(e);
    cudaGetLastError();
    return SG_ERR_CUDA;
  }
  return SG_OK;
}

}  // namespace

template <typename Kernel>
cudaError_t allow(Kernel* kernel, int smem) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
}

cudaError_t prompt_prepare() {
  cudaError_t e = allow(prompt_tile_kernel<64>, TileLayout<64>::kDynSmem);
  if (e == cudaSuccess) e = allow(prompt_tile_kernel<128>, TileLayout<128>::kDynSmem);
  return e == cudaSuccess ? allow(prompt_kernel, PromptLayout::kDynSmem) : e;
}

sg_status_t prompt_launch(const AttnShape& s, const AttnArgs& a) {
  if (s.D <= 64) return launch<64, true>(s, a);
  // Two tiles a CTA read K and V half as often and overlap better, one a CTA starts sooner and deals out finer.
  // By the mean sequence: where two-tile units fill the SMs three times over, they win unless an odd tile leaves
  // half of too many units empty (32 heads over 8, 32 sequences of 200 tokens: 51.3 us with two, 56.2 with one; 8 of
  // 512: 34.8, 44.0; 128 of 100: 94.8, 128.4; one of 8000 and 63 of 100: 363, 542; but 8 heads over 8, 128 of 100, one tile each:
  // 50.2, 40.3; 64 of 300, three: 66.3, 63.8); with fewer units it is the keys that decide (32 over 8, one of 512, 1024, 2048
  // tokens: 12.6, 19.1, 32.6 with two, 11.4, 18.8, 40.5 with one; 8 over 8, one of 1024, 2048: 17.9, 28.5 and 18.1, 31.4).
  const int pack = heads_packed(s.Hq / s.Hk);
  const int64_t tiles = (a.Tq * pack / a.B + kRows - 1) / kRows, units = (tiles + 1) / 2 * a.B * (s.Hq / pack);
  const bool two = units >= 3 * s.num_sms ? tiles % 2 == 0 || tiles > 4 : a.Tk > 512 * a.B;
  return two ? launch<128, false>(s, a) : launch<128, true>(s, a);
}

}  // namespace sg
