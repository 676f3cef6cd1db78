// scaled_attention.cu -- the C ABI of the attention operators: plans, argument
// checks and dispatch (include/scaled_attention.h).
#include <cmath>
#include <new>

#include <cuda.h>
#include <cuda_runtime.h>

#include "sg_attn.h"

struct sg_attn {
  sg::AttnShape shape;
  int device;
};

namespace {

using sg::refuse;

constexpr uint64_t kTimeoutNs = 4000000000ull;
constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// The rows of a bf16 [rows][heads][D] operand.
sg_status_t check_rows(const void* p, int64_t stride, int64_t heads, int64_t D, const char* what) {
  if (!p) return refuse(SG_ERR_INVALID_ARG, what);
  if (!aligned(p, 16) || stride % 8 != 0) return refuse(SG_ERR_MISALIGNED, what);
  if (stride < heads * D) return refuse(SG_ERR_INVALID_ARG, what);
  if (stride > kMaxDim) return refuse(SG_ERR_UNSUPPORTED_SHAPE, what);
  return SG_OK;
}

sg_status_t check_cache(const sg_attn* h, const sg_kv_cache_t* c) {
  if (!c) return refuse(SG_ERR_INVALID_ARG, "attn: NULL cache");
  if (c->num_pages < 0) return refuse(SG_ERR_INVALID_ARG, "attn: negative num_pages");
  if (c->num_pages == 0) return SG_OK;  // nothing is read or written
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return refuse(SG_ERR_INVALID_ARG, "attn: NULL cache");
  if (c->num_pages > kMaxDim) return refuse(SG_ERR_UNSUPPORTED_SHAPE, "attn: num_pages >= 2^31");
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->k_page_stride % 16 != 0 || c->v_page_stride % 16 != 0)
    return refuse(SG_ERR_MISALIGNED, "attn: cache codes");
  const int64_t least = int64_t(h->shape.Hk) * h->shape.page * h->shape.D;
  if (c->k_page_stride < least || c->v_page_stride < least)
    return refuse(SG_ERR_INVALID_ARG, "attn: cache page stride");
  if (c->k_page_stride >= (int64_t(1) << 40) || c->v_page_stride >= (int64_t(1) << 40))
    return refuse(SG_ERR_UNSUPPORTED_SHAPE, "attn: cache page stride >= 2^40");
  return SG_OK;
}

sg_status_t check_table(const int32_t* table, int64_t stride, int page) {
  if (stride < 0) return refuse(SG_ERR_INVALID_ARG, "attn: negative table_stride");
  if (stride * page > kMaxDim) return refuse(SG_ERR_UNSUPPORTED_SHAPE, "attn: table_stride * page >= 2^31");
  if (!table && stride > 0) return refuse(SG_ERR_INVALID_ARG, "attn: NULL table");
  if (!aligned(table, 4)) return refuse(SG_ERR_MISALIGNED, "attn: table");
  return SG_OK;
}

sg_status_t check_ints(const int32_t* p, const char* what) {
  if (!p) return refuse(SG_ERR_INVALID_ARG, what);
  return aligned(p, 4) ? SG_OK : refuse(SG_ERR_MISALIGNED, what);
}

sg_status_t check_device(const sg_attn* h) {
  int cur = -1;
  if (cudaGetDevice(&cur) != cudaSuccess) return refuse(SG_ERR_CUDA, "attn: cudaGetDevice");
  return cur == h->device ? SG_OK : refuse(SG_ERR_INVALID_ARG, "attn: current device differs from the plan's");
}

// The bytes that rows of a strided operand cover.
int64_t row_bytes(int64_t rows, int64_t stride, int64_t width) {
  return rows > 0 ? 2 * ((rows - 1) * stride + width) : 0;
}

#define SG_TRY(expr)                        \
  do {                                      \
    const sg_status_t try_status = (expr);  \
    if (try_status != SG_OK) return try_status; \
  } while (0)

}  // namespace

extern "C" {

sg_status_t scaled_attn_create(sg_attn_t* out, int64_t Hq, int64_t Hk, int64_t D, int64_t page, int device) {
  if (!out) return refuse(SG_ERR_INVALID_ARG, "attn create: out is NULL");
  *out = nullptr;
  if (Hq < 1 || Hk < 1 || D < 1 || page < 1) return refuse(SG_ERR_INVALID_ARG, "attn create: size below 1");
  if (Hq > 1024 || Hq % Hk != 0) return refuse(SG_ERR_UNSUPPORTED_SHAPE, "attn create: heads");
  if (D % 16 != 0 || D > 128) return refuse(SG_ERR_UNSUPPORTED_SHAPE, "attn create: D");
  if (page != 16 && page != 32 && page != 64 && page != 128) return refuse(SG_ERR_UNSUPPORTED_SHAPE, "attn create: page");
  int dev = device;
  if (dev < 0 && cudaGetDevice(&dev) != cudaSuccess) return refuse(SG_ERR_CUDA, "attn create: cudaGetDevice");
  int major = 0, minor = 0, sms = 0;
  if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return refuse(SG_ERR_CUDA, "attn create: device query");
  if (major != 10 || minor != 3) return refuse(SG_ERR_UNSUPPORTED_DEVICE, "attn create: not compute capability 10.3");
  sg_attn* h = new (std::nothrow) sg_attn();
  if (!h) return refuse(SG_ERR_CUDA, "attn create: out of host memory");
  h->device = dev;
  h->shape.Hq = static_cast<int>(Hq);
  h->shape.Hk = static_cast<int>(Hk);
  h->shape.D = static_cast<int>(D);
  h->shape.page = static_cast<int>(page);
  h->shape.num_sms = sms;
  h->shape.timeout_ns = kTimeoutNs;
  h->shape.skip_tile = -1;
  int prev = -1;
  cudaGetDevice(&prev);
  if (prev != dev && cudaSetDevice(dev) != cudaSuccess) {
    delete h;
    return refuse(SG_ERR_CUDA, "attn create: cudaSetDevice");
  }
  const size_t ws = sg::decode_workspace_bytes(h->shape);
  cudaError_t e = sg::decode_prepare();
  if (e == cudaSuccess) e = sg::prompt_prepare();
  if (e == cudaSuccess) e = cudaMalloc(&h->shape.status, 16);
  if (e == cudaSuccess) e = cudaMemset(h->shape.status, 0, 16);
  if (e == cudaSuccess && ws > 0) e = cudaMalloc(&h->shape.workspace, ws);
  if (e == cudaSuccess && ws > 0) e = cudaMemset(h->shape.workspace, 0, ws);
  if (e != cudaSuccess) {
    sg::note_cuda_error(e);
    if (h->shape.status) cudaFree(h->shape.status);
    if (h->shape.workspace) cudaFree(h->shape.workspace);
    delete h;
    h = nullptr;
  }
  if (prev >= 0 && prev != dev) cudaSetDevice(prev);
  if (!h) return refuse(SG_ERR_CUDA, "attn create: kernel attributes / status word / workspace");
  *out = h;
  return SG_OK;
}

sg_status_t scaled_attn_destroy(sg_attn_t h) {
  if (!h) return SG_OK;
  int prev = -1;
  cudaGetDevice(&prev);
  if (prev != h->device) cudaSetDevice(h->device);
  cudaError_t e = cudaFree(h->shape.status);
  if (h->shape.workspace) {
    const cudaError_t e2 = cudaFree(h->shape.workspace);
    if (e == cudaSuccess) e = e2;
  }
  if (prev >= 0 && prev != h->device) cudaSetDevice(prev);
  delete h;
  return e == cudaSuccess ? SG_OK : SG_ERR_CUDA;
}

sg_status_t scaled_attn_set_debug(sg_attn_t h, int64_t timeout_ns, int64_t skip_tile) {
  if (!h) return refuse(SG_ERR_INVALID_ARG, "attn set_debug: NULL handle");
  if (timeout_ns < 0 || skip_tile < -1 || skip_tile > kMaxDim) return refuse(SG_ERR_INVALID_ARG, "attn set_debug: bad value");
  h->shape.timeout_ns = timeout_ns ? static_cast<uint64_t>(timeout_ns) : kTimeoutNs;
  h->shape.skip_tile = static_cast<int>(skip_tile);
  return SG_OK;
}

sg_status_t scaled_attn_debug_status(sg_attn_t h, sg_stream_t stream, int32_t* code, int32_t* where) {
  if (!h || !code) return refuse(SG_ERR_INVALID_ARG, "attn debug_status: NULL argument");
  int32_t host[4] = {0, 0, 0, 0};
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cudaMemcpyAsync(host, h->shape.status, 16, cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess || cudaMemsetAsync(h->shape.status, 0, 16, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return refuse(SG_ERR_CUDA, "attn debug_status: copy");
  *code = host[0];
  if (where) *where = host[0] ? host[1] : 0;
  return SG_OK;
}

sg_status_t scaled_attn_append(sg_attn_t h, const sg_kv_cache_t* cache, const sg_rotary_t* rotary,
                               const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                               const void* v, int64_t v_stride, const int32_t* table,
                               int64_t table_stride, const int32_t* ctx_lens,
                               const int32_t* cu_seqlens, int64_t T, int64_t B, void* q_out,
                               void* k_out, sg_stream_t stream) {
  if (!h) return refuse(SG_ERR_INVALID_ARG, "append: NULL handle");
  const sg::AttnShape& s = h->shape;
  if (T < 0 || B < 0) return refuse(SG_ERR_INVALID_ARG, "append: negative size");
  if (T > kMaxDim || B > (1 << 24)) return refuse(SG_ERR_UNSUPPORTED_SHAPE, "append: T >= 2^31 or B > 2^24");
  if (!rotary) return refuse(SG_ERR_INVALID_ARG, "append: NULL rotary");
  if (rotary->rot < 0 || rotary->rot > s.D || rotary->rot % 16 != 0)
    return refuse(SG_ERR_UNSUPPORTED_SHAPE, "append: rot");
  if (rotary->rot > 0) {
    if (!rotary->table || rotary->max_pos < 1) return refuse(SG_ERR_INVALID_ARG, "append: rotary table");
    if (rotary->max_pos > kMaxDim) return refuse(SG_ERR_UNSUPPORTED_SHAPE, "append: max_pos >= 2^31");
    if (!aligned(rotary->table, 16)) return refuse(SG_ERR_MISALIGNED, "append: rotary table");
  }
  if (T == 0 || B == 0) return SG_OK;
  SG_TRY(check_cache(h, cache));
  SG_TRY(check_rows(q, q_stride, s.Hq, s.D, "append: q"));
  SG_TRY(check_rows(k, k_stride, s.Hk, s.D, "append: k"));
  SG_TRY(check_rows(v, v_stride, s.Hk, s.D, "append: v"));
  SG_TRY(check_table(table, table_stride, s.page));
  SG_TRY(check_ints(ctx_lens, "append: ctx_lens"));
  SG_TRY(check_ints(cu_seqlens, "append: cu_seqlens"));
  if (!q_out) return refuse(SG_ERR_INVALID_ARG, "append: q_out is NULL");
  if (!aligned(q_out, 16) || !aligned(k_out, 16)) return refuse(SG_ERR_MISALIGNED, "append: outputs");
  // An output may be its own input (each row is read before it is written), where the rows
  // coincide; any other overlap with an input or the other output is refused.
  const struct { const void* p; int64_t n; const void* own; int64_t stride, width; } in[3] = {
      {q, row_bytes(T, q_stride, int64_t(s.Hq) * s.D), q_out, q_stride, int64_t(s.Hq) * s.D},
      {k, row_bytes(T, k_stride, int64_t(s.Hk) * s.D), k_out, k_stride, int64_t(s.Hk) * s.D},
      {v, row_bytes(T, v_stride, int64_t(s.Hk) * s.D), nullptr, v_stride, 0}};
  const struct { const void* p; int64_t n; } outs[2] = {{q_out, 2 * T * s.Hq * s.D}, {k_out, 2 * T * s.Hk * s.D}};
  for (const auto& o : outs)
    for (const auto& i : in) {
      const bool same = o.p == i.p && o.p == i.own && i.stride == i.width;
      if (!same && sg::ranges_overlap(o.p, o.n, i.p, i.n)) return refuse(SG_ERR_INVALID_ARG, "append: an output overlaps an input");
    }
  if (sg::ranges_overlap(outs[0].p, outs[0].n, outs[1].p, outs[1].n))
    return refuse(SG_ERR_INVALID_ARG, "append: q_out overlaps k_out");
  SG_TRY(check_device(h));
  sg::AttnArgs a{};
  a.cache = *cache;
  a.rotary = *rotary;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.table = table;
  a.table_stride = table_stride;
  a.lens = ctx_lens;
  a.cu_q = cu_seqlens;
  a.Tq = T;
  a.B = B;
  a.out = q_out;
  a.k_out = k_out;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  const sg_status_t r = sg::append_launch(s, a);
  return r == SG_OK ? SG_OK : refuse(r, "append: kernel launch");
}

sg_status_t scaled_attn_decode(sg_attn_t h, const sg_kv_cache_t* cache, const void* q, int64_t q_stride,
                               int64_t qn, const int32_t* table, int64_t table_stride,
                               const int32_t* kv_lens, int64_t B, float scale, void* out, float* lse,
                               sg_stream_t stream) {
  if (!h) return refuse(SG_ERR_INVALID_ARG, "decode: NULL handle");
  const sg::AttnShape& s = h->shape;
  if (B < 0 || qn < 0) return refuse(SG_ERR_INVALID_ARG, "decode: negative size");
  if (B > (1 << 24) || qn > 4096 || B * qn > kMaxDim) return refuse(SG_ERR_UNSUPPORTED_SHAPE, "decode: B > 2^24 or qn > 4096");
  if (!(scale > 0.f) || !std::isfinite(scale)) return refuse(SG_ERR_INVALID_ARG, "decode: scale");
  if (B == 0 || qn == 0) return SG_OK;
  SG_TRY(check_cache(h, cache));
  SG_TRY(check_rows(q, q_stride, s.Hq, s.D, "decode: q"));
  SG_TRY(check_table(table, table_stride, s.page));
  SG_TRY(check_ints(kv_lens, "decode: kv_lens"));
  if (!out) return refuse(SG_ERR_INVALID_ARG, "decode: out is NULL");
  if (!aligned(out, 16) || !aligned(lse, 4)) return refuse(SG_ERR_MISALIGNED, "decode: outputs");
  const int64_t ob = 2 * B * qn * s.Hq * s.D;
  if (sg::ranges_overlap(out, ob, q, row_bytes(B * qn, q_stride, int64_t(s.Hq) * s.D)))
    return refuse(SG_ERR_INVALID_ARG, "decode: out overlaps q");
  SG_TRY(check_device(h));
  sg::AttnArgs a{};
  a.cache = *cache;
  a.q = q;
  a.q_stride = q_stride;
  a.qn = qn;
  a.table = table;
  a.table_stride = table_stride;
  a.lens = kv_lens;
  a.Tq = B * qn;
  a.B = B;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  const sg_status_t r = sg::decode_launch(s, a);
  return r == SG_OK ? SG_OK : refuse(r, "decode: kernel launch");
}

sg_status_t scaled_attn_prompt(sg_attn_t h, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                               const void* v, int64_t v_stride, const int32_t* cu_q, const int32_t* cu_k,
                               int64_t Tq, int64_t Tk, int64_t B, int causal, float scale, void* out,
                               float* lse, sg_stream_t stream) {
  if (!h) return refuse(SG_ERR_INVALID_ARG, "prompt: NULL handle");
  const sg::AttnShape& s = h->shape;
  if (Tq < 0 || Tk < 0 || B < 0) return refuse(SG_ERR_INVALID_ARG, "prompt: negative size");
  if (Tq > kMaxDim || Tk > kMaxDim || B > (1 << 24)) return refuse(SG_ERR_UNSUPPORTED_SHAPE, "prompt: T >= 2^31 or B > 2^24");
  if (!(scale > 0.f) || !std::isfinite(scale)) return refuse(SG_ERR_INVALID_ARG, "prompt: scale");
  if (Tq == 0 || B == 0) return SG_OK;
  SG_TRY(check_rows(q, q_stride, s.Hq, s.D, "prompt: q"));
  if (Tk > 0) {
    SG_TRY(check_rows(k, k_stride, s.Hk, s.D, "prompt: k"));
    SG_TRY(check_rows(v, v_stride, s.Hk, s.D, "prompt: v"));
  }
  SG_TRY(check_ints(cu_q, "prompt: cu_q"));
  SG_TRY(check_ints(cu_k, "prompt: cu_k"));
  if (!out) return refuse(SG_ERR_INVALID_ARG, "prompt: out is NULL");
  if (!aligned(out, 16) || !aligned(lse, 4)) return refuse(SG_ERR_MISALIGNED, "prompt: outputs");
  const int64_t ob = 2 * Tq * s.Hq * s.D;
  if (sg::ranges_overlap(out, ob, q, row_bytes(Tq, q_stride, int64_t(s.Hq) * s.D)) ||
      sg::ranges_overlap(out, ob, k, row_bytes(Tk, k_stride, int64_t(s.Hk) * s.D)) ||
      sg::ranges_overlap(out, ob, v, row_bytes(Tk, v_stride, int64_t(s.Hk) * s.D)))
    return refuse(SG_ERR_INVALID_ARG, "prompt: out overlaps an input");
  SG_TRY(check_device(h));
  sg::AttnArgs a{};
  a.q = q;
  a.q_stride = q_stride;
  a.k = k;
  a.k_stride = k_stride;
  a.v = v;
  a.v_stride = v_stride;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.Tq = Tq;
  a.Tk = Tk;
  a.B = B;
  a.causal = causal != 0;
  a.scale = scale;
  a.out = out;
  a.lse = lse;
  a.stream = reinterpret_cast<cudaStream_t>(stream);
  const sg_status_t r = sg::prompt_launch(s, a);
  return r == SG_OK ? SG_OK : refuse(r, "prompt: kernel launch");
}

}  // extern "C"
