// sg_attn.h -- host-side interface between the attention entry points
// (scaled_attention.cu) and the kernels' launchers.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "scaled_attention.h"
#include "sg_internal.h"

namespace sg {

// Tokens of a key/value cache block (one e8m0 scale per block and head).
constexpr int kKvBlock = 16;

// What a plan fixes.
struct AttnShape {
  int Hq, Hk, D, page;
  int num_sms;
  int* status;          // device status word of the plan
  uint64_t timeout_ns;  // limit of every wait in a kernel
  int skip_tile;        // tests: a key tile that is not loaded; -1: none
  void* workspace;      // decode and chunk: partial results
};

// Validated arguments of one call; unused fields are zero.
struct AttnArgs {
  sg_kv_cache_t cache;
  sg_rotary_t rotary;
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // elements between rows
  const int32_t* table;
  int64_t table_stride;
  const int32_t *lens, *cu_q, *cu_k;
  int64_t Tq, Tk, B, qn;
  int causal;
  float scale;
  void *out, *k_out;
  float* lse;
  cudaStream_t stream;
};

sg_status_t append_launch(const AttnShape& s, const AttnArgs& a);

int64_t pool_scratch_bytes(int64_t rows, int64_t num_pages);
sg_status_t pool_release(const AttnShape& s, const sg_page_pool_t& pool, const int32_t* rows, int64_t n, cudaStream_t stream);
sg_status_t pool_grow(const AttnShape& s, const sg_page_pool_t& pool, const int32_t* rows, const int32_t* add, int64_t n, int32_t* ok,
                      cudaStream_t stream);
sg_status_t pool_fork(const AttnShape& s, const sg_page_pool_t& pool, const sg_kv_cache_t* caches, int64_t layers, const int32_t* src,
                      const int32_t* dst, int64_t n, int32_t* ok, cudaStream_t stream);
sg_status_t pool_compact(const AttnShape& s, const sg_page_pool_t& pool, const sg_kv_cache_t* caches, int64_t layers, int32_t* in_use,
                         cudaStream_t stream);

size_t decode_workspace_bytes(const AttnShape& s);
cudaError_t decode_prepare();
sg_status_t decode_launch(const AttnShape& s, const AttnArgs& a);

size_t chunk_workspace_bytes(const AttnShape& s);
cudaError_t chunk_prepare();
sg_status_t chunk_launch(const AttnShape& s, const AttnArgs& a);

cudaError_t prompt_prepare();
sg_status_t prompt_launch(const AttnShape& s, const AttnArgs& a);

}  // namespace sg
