// sg_kv_pages.cu -- pages of the key/value cache among the rows of a block table
// (scaled_attn_pool_release, _grow, _fork, _compact).
//
// Two kinds of work.  The bookkeeping is small and ordered: which pages are free, which request gets which.
// One CTA does it, each thread a stretch of the pages: it counts the free ones, a scan over the CTA gives their
// numbers, and a second look at the stretch (in L1 or L2 by then) writes the list.  Pages are taken lowest first and
// requests are served in order, so results do not depend on timing.  Moving the pages' bytes is the rest: a second kernel over
// all SMs, in pieces of 16 KB (four 16-byte loads a thread, all in flight before the first store), that
// reads what the first has listed.  The bound of that is memory, 2 bytes moved a byte.
#include <cuda.h>
#include <cuda_runtime.h>

#include <climits>

#include "sg_attn.h"
#include "sg_ptx.cuh"

namespace sg {

namespace {

constexpr int kThreads = 1024;      // of the bookkeeping CTA
constexpr int kMoveThreads = 256;
constexpr int kPiece = kMoveThreads * 4 * 16;  // bytes of a page that a CTA moves at a time
constexpr int kLayers = 32;         // caches of a launch

// The pool's scratch, in 32-bit words: counters; per row the request that owns it; per request its length and first
// free page; pages (free ones in order, or each moved page's new number); moves (from, to).
struct Scratch {
  int* counts;  // [0] moves, [1] pages in use after a compaction
  int *owner, *length, *pages;
  int2* moves;
};

__host__ __device__ inline int64_t up4(int64_t n) { return (n + 3) & ~int64_t(3); }

__host__ __device__ inline Scratch scratch_of(void* at, int64_t rows, int64_t num_pages) {
  int* p = static_cast<int*>(at);
  Scratch s;
  s.counts = p;
  s.owner = p + 4;
  s.length = s.owner + up4(rows);
  s.pages = s.length + up4(rows);
  s.moves = reinterpret_cast<int2*>(s.pages + up4(num_pages));
  return s;
}

struct PoolParams {
  int *table, *lens, *refs;
  int rows, width, num_pages, page;
  Scratch scratch;
  const int *first, *second;  // the requests
  int n;
  int* answer;
};

// Sum over the CTA of one value a thread; each thread's sum of those before it.
__device__ __forceinline__ int scan_cta(int mine, int& before) {
  __shared__ int warps[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int up = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += x;
  }
  __syncthreads();  // the last scan's have been read
  if (lane == 31) warps[warp] = up;
  __syncthreads();
  int sum = warps[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, sum, o);
    if (lane >= o) sum += x;
  }
  const int base = __shfl_sync(0xffffffffu, sum, max(warp - 1, 0));
  before = (warp ? base : 0) + up - mine;
  return __shfl_sync(0xffffffffu, sum, 31);
}

// f(page, references) of this thread's stretch of the pages, in order.
template <typename F>
__device__ __forceinline__ void each_page(const PoolParams& p, F&& f) {
  const int stretch = ((p.num_pages + kThreads - 1) / kThreads + 3) & ~3;
  const int64_t begin = static_cast<int64_t>(threadIdx.x) * stretch;
  const int end = static_cast<int>(min(begin + stretch, static_cast<int64_t>(p.num_pages)));
#pragma unroll 4
  for (int64_t i = begin; i < end; i += 4) {
    if (i + 4 <= end) {
      const int4 r = *reinterpret_cast<const int4*>(p.refs + i);
      f(static_cast<int>(i), r.x), f(static_cast<int>(i) + 1, r.y), f(static_cast<int>(i) + 2, r.z), f(static_cast<int>(i) + 3, r.w);
    } else {
      for (int64_t j = i; j < end; ++j) f(static_cast<int>(j), p.refs[j]);
    }
  }
}

// The first `want` free pages into the scratch's list; their number.
__device__ __forceinline__ int list_free(const PoolParams& p, int want) {
  int mine = 0, at;
  each_page(p, [&](int, int refs) { mine += refs <= 0; });
  const int all = scan_cta(mine, at);
  if (at < want)
    each_page(p, [&](int page, int refs) {
      if (refs <= 0) {
        if (at < want) p.scratch.pages[at] = page;
        ++at;
      }
    });
  __syncthreads();
  return min(all, want);
}

// Each row belongs to the first request that names it.
__device__ __forceinline__ void claim_rows(const PoolParams& p, const int* rows) {
  for (int i = threadIdx.x; i < p.n; i += kThreads)
    if (rows[i] >= 0 && rows[i] < p.rows) p.scratch.owner[rows[i]] = INT_MAX;
  __syncthreads();
  for (int i = threadIdx.x; i < p.n; i += kThreads)
    if (rows[i] >= 0 && rows[i] < p.rows) atomicMin(p.scratch.owner + rows[i], i);
  __syncthreads();
}

__device__ __forceinline__ int length_of(const PoolParams& p, int row) {
  return static_cast<int>(min(static_cast<int64_t>(max(p.lens[row], 0)), static_cast<int64_t>(p.width) * p.page));
}

__global__ void __launch_bounds__(256) release_kernel(const PoolParams p) {
  grid_dep_launch();
  grid_dep_wait();
  for (int i = blockIdx.x; i < p.n; i += gridDim.x) {
    const int row = p.first[i];
    if (row < 0 || row >= p.rows) continue;
    int* entries = p.table + static_cast<int64_t>(row) * p.width;
    for (int e = threadIdx.x; e < p.width; e += blockDim.x) {
      if (entries[e] == -1) continue;
      const int page = atomicExch(entries + e, -1);  // a row named twice gives each page back once
      if (page >= 0 && page < p.num_pages) atomicSub(p.refs + page, 1);
    }
    if (threadIdx.x == 0) p.lens[row] = 0;
  }
}

__global__ void __launch_bounds__(kThreads) grow_kernel(const PoolParams p) {
  grid_dep_launch();
  grid_dep_wait();
  claim_rows(p, p.first);
  // pages that request i needs; -1: it cannot be
  auto need = [&](int i, int& len) {
    const int row = p.first[i], add = p.second[i];
    len = 0;
    if (row < 0 || row >= p.rows || add < 0 || p.scratch.owner[row] != i) return -1;
    len = length_of(p, row);
    const int64_t to = static_cast<int64_t>(len) + add;
    if (to > static_cast<int64_t>(p.width) * p.page) return -1;
    return static_cast<int>((to + p.page - 1) / p.page) - (len + p.page - 1) / p.page;
  };
  int total = 0;
  for (int base = 0; base < p.n; base += kThreads) {
    int before, len;
    const int i = base + threadIdx.x;
    total += scan_cta(i < p.n ? max(need(i, len), 0) : 0, before);
  }
  const int have = list_free(p, min(total, p.num_pages));
  const int lane = threadIdx.x & 31;
  int start = 0;
  for (int base = 0; base < p.n; base += kThreads) {
    const int i = base + threadIdx.x;
    int before, len = 0;
    const int mine = i < p.n ? need(i, len) : -1;
    const int sum = scan_cta(max(mine, 0), before);
    before += start;
    start += sum;
    const bool ok = mine == 0 || (mine > 0 && before + mine <= have);
    // a warp writes its requests' entries one request after another
    for (unsigned left = __ballot_sync(0xffffffffu, ok && mine > 0); left; left &= left - 1) {
      const int who = __ffs(left) - 1;
      const int count = __shfl_sync(0xffffffffu, mine, who), from = __shfl_sync(0xffffffffu, before, who);
      const int row = p.first[i - lane + who], entry = (__shfl_sync(0xffffffffu, len, who) + p.page - 1) / p.page;
      for (int e = lane; e < count; e += 32) {
        const int page = p.scratch.pages[from + e];
        p.table[static_cast<int64_t>(row) * p.width + entry + e] = page;
        p.refs[page] = 1;
      }
    }
    if (i < p.n) {
      p.answer[i] = ok;
      if (ok) p.lens[p.first[i]] = len + p.second[i];
    }
  }
}

__global__ void __launch_bounds__(kThreads) fork_plan_kernel(const PoolParams p) {
  grid_dep_launch();
  grid_dep_wait();
  claim_rows(p, p.second);
  // the last page that request i copies; -1: it copies none, -2: it cannot be
  auto last = [&](int i, int& len) {
    const int src = p.first[i], dst = p.second[i];
    len = 0;
    if (src < 0 || src >= p.rows || dst < 0 || dst >= p.rows || p.scratch.owner[dst] != i || p.lens[dst] > 0) return -2;
    len = length_of(p, src);
    if (len % p.page == 0) return -1;
    const int page = p.table[static_cast<int64_t>(src) * p.width + len / p.page];
    return page >= 0 && page < p.num_pages ? page : -1;
  };
  int total = 0;
  for (int base = 0; base < p.n; base += kThreads) {
    int before, len;
    const int i = base + threadIdx.x;
    total += scan_cta(i < p.n && last(i, len) >= 0, before);
  }
  const int have = list_free(p, min(total, p.num_pages));
  int start = 0;
  for (int base = 0; base < p.n; base += kThreads) {
    const int i = base + threadIdx.x;
    int before, len = 0;
    const int page = i < p.n ? last(i, len) : -2;
    const int sum = scan_cta(page >= 0, before);
    before += start;
    start += sum;
    const bool ok = page == -1 || (page >= 0 && before < have);
    if (i < p.n) {
      p.answer[i] = ok;
      p.scratch.length[i] = ok ? len : 0;
    }
    if (ok && page >= 0) {
      const int to = p.scratch.pages[before];
      p.scratch.moves[before] = make_int2(page, to);
      p.refs[to] = 1;
      // the copy's place in the row; the rest of the row is the second kernel's
      p.table[static_cast<int64_t>(p.second[i]) * p.width + len / p.page] = to;
    }
  }
  if (threadIdx.x == 0) p.scratch.counts[0] = have;
}

__global__ void __launch_bounds__(kThreads) compact_plan_kernel(const PoolParams p) {
  grid_dep_launch();
  grid_dep_wait();
  int mine = 0, used_before;
  each_page(p, [&](int, int refs) { mine += refs > 0; });
  const int used = scan_cta(mine, used_before);
  // holes below `used` in order, and pages to move from above it
  int holes = 0, tails = 0, hole, tail;
  each_page(p, [&](int page, int refs) {
    holes += page < used && refs <= 0;
    tails += page >= used && refs > 0;
  });
  const int moves = scan_cta(holes, hole);
  scan_cta(tails, tail);
  each_page(p, [&](int page, int refs) {
    if (page < used && refs <= 0) p.scratch.moves[hole++].y = page;
    if (page >= used && refs > 0) p.scratch.moves[tail++].x = page;
    if (page >= used && refs <= 0) p.scratch.pages[page] = page;  // an entry may name it all the same
  });
  __syncthreads();
  for (int i = threadIdx.x; i < moves; i += kThreads) {
    const int2 m = p.scratch.moves[i];
    p.scratch.pages[m.x] = m.y;
    p.refs[m.y] = p.refs[m.x];
    p.refs[m.x] = 0;
  }
  if (threadIdx.x == 0) {
    p.scratch.counts[0] = moves;
    p.scratch.counts[1] = used;
    *p.answer = used;
  }
}

struct Layers {
  sg_kv_cache_t at[kLayers];
  int count;
  int64_t page_bytes, scale_bytes;
};

// The moves' pages in all layers: piece after piece of K and V of each, scales with the first.
__device__ __forceinline__ void move_pages(const PoolParams& p, const Layers& c) {
  const int pieces = static_cast<int>((c.page_bytes + kPiece - 1) / kPiece);
  const int64_t items = static_cast<int64_t>(p.scratch.counts[0]) * c.count * 2 * pieces;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int piece = static_cast<int>(it % pieces);
    const int64_t rest = it / pieces;
    const bool v = rest & 1;
    const int64_t move = (rest >> 1) / c.count;
    const sg_kv_cache_t& l = c.at[(rest >> 1) % c.count];
    const int2 m = p.scratch.moves[move];
    const int64_t stride = v ? l.v_page_stride : l.k_page_stride;
    uint8_t* const codes = static_cast<uint8_t*>(v ? l.v : l.k);
    const uint8_t* from = codes + m.x * stride;
    uint8_t* to = codes + m.y * stride;
    const int64_t at = static_cast<int64_t>(piece) * kPiece + 16 * threadIdx.x;
    uint4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at + i * 16 * kMoveThreads < c.page_bytes) x[i] = *reinterpret_cast<const uint4*>(from + at + i * 16 * kMoveThreads);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at + i * 16 * kMoveThreads < c.page_bytes) *reinterpret_cast<uint4*>(to + at + i * 16 * kMoveThreads) = x[i];
    if (piece == 0) {
      uint8_t* const scale = v ? l.v_scale : l.k_scale;
      for (int64_t i = threadIdx.x; i < c.scale_bytes; i += kMoveThreads) scale[m.y * c.scale_bytes + i] = scale[m.x * c.scale_bytes + i];
    }
  }
}

// `rows`: this launch also writes the forked rows (the first launch of a call).
__global__ void __launch_bounds__(kMoveThreads) fork_kernel(const PoolParams p, const __grid_constant__ Layers c, int rows) {
  grid_dep_launch();
  grid_dep_wait();
  if (rows)
    for (int i = blockIdx.x; i < p.n; i += gridDim.x) {
      const int len = p.scratch.length[i];
      if (len == 0) continue;  // nothing to fork, or not to be
      const int *from = p.table + static_cast<int64_t>(p.first[i]) * p.width;
      int* to = p.table + static_cast<int64_t>(p.second[i]) * p.width;
      for (int e = threadIdx.x; e < len / p.page; e += kMoveThreads) {
        const int page = from[e];
        to[e] = page;
        if (page >= 0 && page < p.num_pages) atomicAdd(p.refs + page, 1);
      }
      if (threadIdx.x == 0) p.lens[p.second[i]] = len;
    }
  move_pages(p, c);
}

__global__ void __launch_bounds__(kMoveThreads) compact_kernel(const PoolParams p, const __grid_constant__ Layers c, int rows) {
  grid_dep_launch();
  grid_dep_wait();
  if (rows) {
    const int used = p.scratch.counts[1];
    const int64_t entries = static_cast<int64_t>(p.rows) * p.width;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kMoveThreads + threadIdx.x; i < entries; i += static_cast<int64_t>(gridDim.x) * kMoveThreads) {
      const int page = p.table[i];
      if (page >= used && page < p.num_pages) p.table[i] = p.scratch.pages[page];
    }
  }
  move_pages(p, c);
}

template <typename Kernel, typename... Args>
sg_status_t start(Kernel* kernel, unsigned grid, unsigned threads, cudaStream_t stream, const Args&... args) {
  GemmLaunch l(dim3(grid), dim3(threads), 0, stream, 1);
  const cudaError_t e = cudaLaunchKernelEx(&l.cfg, kernel, args...);
  if (e == cudaSuccess) return SG_OK;
  note_cuda_error(e);
  cudaGetLastError();
  return SG_ERR_CUDA;
}

PoolParams params(const AttnShape& s, const sg_page_pool_t& pool, const int32_t* first, const int32_t* second, int64_t n,
                  int32_t* answer) {
  PoolParams p{};
  p.table = pool.table;
  p.lens = pool.lens;
  p.refs = pool.refs;
  p.rows = static_cast<int>(pool.rows);
  p.width = static_cast<int>(pool.table_stride);
  p.num_pages = static_cast<int>(pool.num_pages);
  p.page = s.page;
  p.scratch = scratch_of(pool.scratch, pool.rows, pool.num_pages);
  p.first = first;
  p.second = second;
  p.n = static_cast<int>(n);
  p.answer = answer;
  return p;
}

// The second kernel of a call, over the caches in groups of kLayers.
template <typename Kernel>
sg_status_t over_layers(const AttnShape& s, const PoolParams& p, const sg_kv_cache_t* caches, int64_t layers, Kernel* kernel,
                        cudaStream_t stream) {
  for (int64_t first = 0; first == 0 || first < layers; first += kLayers) {
    Layers c{};
    c.count = static_cast<int>(layers - first < kLayers ? layers - first : kLayers);
    for (int i = 0; i < c.count; ++i) c.at[i] = caches[first + i];
    c.page_bytes = static_cast<int64_t>(s.Hk) * s.page * s.D;
    c.scale_bytes = static_cast<int64_t>(s.Hk) * (s.page / kKvBlock);
    const sg_status_t r = start(kernel, 8 * s.num_sms, kMoveThreads, stream, p, c, static_cast<int>(first == 0));
    if (r != SG_OK) return r;
  }
  return SG_OK;
}

}  // namespace

int64_t pool_scratch_bytes(int64_t rows, int64_t num_pages) {
  // moves: a fork has at most one a row, a compaction one for every other page
  return 4 * (4 + 2 * up4(rows) + up4(num_pages)) + 8 * (rows > num_pages ? rows : num_pages);
}

sg_status_t pool_release(const AttnShape& s, const sg_page_pool_t& pool, const int32_t* rows, int64_t n, cudaStream_t stream) {
  const int64_t most = 8 * s.num_sms;
  return start(release_kernel, static_cast<unsigned>(n < most ? n : most), 256, stream, params(s, pool, rows, nullptr, n, nullptr));
}

sg_status_t pool_grow(const AttnShape& s, const sg_page_pool_t& pool, const int32_t* rows, const int32_t* add, int64_t n, int32_t* ok,
                      cudaStream_t stream) {
  return start(grow_kernel, 1, kThreads, stream, params(s, pool, rows, add, n, ok));
}

sg_status_t pool_fork(const AttnShape& s, const sg_page_pool_t& pool, const sg_kv_cache_t* caches, int64_t layers, const int32_t* src,
                      const int32_t* dst, int64_t n, int32_t* ok, cudaStream_t stream) {
  const PoolParams p = params(s, pool, src, dst, n, ok);
  const sg_status_t r = start(fork_plan_kernel, 1, kThreads, stream, p);
  return r == SG_OK ? over_layers(s, p, caches, layers, fork_kernel, stream) : r;
}

sg_status_t pool_compact(const AttnShape& s, const sg_page_pool_t& pool, const sg_kv_cache_t* caches, int64_t layers, int32_t* in_use,
                         cudaStream_t stream) {
  const PoolParams p = params(s, pool, nullptr, nullptr, 0, in_use);
  const sg_status_t r = start(compact_plan_kernel, 1, kThreads, stream, p);
  return r == SG_OK ? over_layers(s, p, caches, layers, compact_kernel, stream) : r;
}

}  // namespace sg
