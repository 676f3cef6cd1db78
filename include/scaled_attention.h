/*
 * scaled_attention.h -- C ABI of the attention operators beside the scaled GEMMs
 * (libscaledgemm.so, GB300 / sm_103a).
 *
 * A decoder's attention lies between two of the library's GEMMs, the QKV projection
 * and the output projection.  The operators here are what happens in between
 * when a server keeps keys and values in a paged 8-bit cache:
 *
 *   scaled_attn_append   rotate queries and keys by their positions; append keys and
 *                        values to the cache
 *   scaled_attn_decode   attention of each sequence's newest tokens over the cache
 *   scaled_attn_chunk    attention of chunks of new tokens, as many for each sequence as there are, over the cache
 *   scaled_attn_prompt   attention over whole prompts, packed one after another
 *
 * and scaled_attn_pool_* share the cache's pages out among sequences: release, grow, fork, compact.
 *
 * Layouts (device pointers, owned by the caller, never retained after the call
 * returns; 16-byte aligned unless stated):
 *   q, k, v      bf16 [rows][heads][D]: heads D apart and rows `*_stride` elements apart
 *                (a multiple of 8, at least heads * D), so they can be views of the
 *                projection's output rows [rows][(Hq + 2 Hk) D].  Query head h reads
 *                key/value head h / (Hq / Hk).
 *   cache        k, v: e4m3 codes [num_pages][Hk][page][D], pages `*_page_stride` bytes
 *                apart (a multiple of 16, at least Hk * page * D); k_scale, v_scale: e8m0 codes
 *                [num_pages][Hk][page / 16] (any alignment), one scale for each block of
 *                16 tokens and head: value = e4m3(code) * 2^(scale - 127).  Scale code 255 is NaN.
 *                With num_pages 0 the pointers and strides are not looked at.
 *   table        int32 [B][table_stride] (4-byte aligned): the pages of each sequence in order.
 *                An entry outside [0, num_pages) has no page: nothing is written for its tokens
 *                and attention does not see them.
 *   cu_seqlens   int32 [B + 1] (4-byte aligned), non-decreasing, cu_seqlens[0] = 0: sequence b's rows are
 *                [cu_seqlens[b], cu_seqlens[b + 1]).  Values are clamped to the rows there are.  Output rows
 *                past cu_seqlens[B] (a batch padded for a graph) are not written.
 *   rotary       float [max_pos][2][rot / 2] (cos, then sin) by position; a position past
 *                the table uses its last row.
 *   lse          float [rows][Hq] (4-byte aligned): natural logarithm of the softmax's denominator; -infinity
 *                for a row that sees no key, whose output is zero.  NULL: not written.
 * Outputs of the attention calls overlap neither q, k, v nor each other (checked: SG_ERR_INVALID_ARG), nor anything else that a call reads.
 *
 * Rules: 1 <= Hq, Hk <= 1024, Hq a multiple of Hk; D a multiple of 16, 16 <= D <= 128; page 16, 32, 64
 * or 128; rot a multiple of 16, 0 <= rot <= D; scale positive and finite; in scaled_attn_prompt scores scale q.k of up to 2^29
 * in magnitude (a row whose largest is past 2^30 gets NaN).
 *
 * Precision: scores, softmax statistics and sums are held in fp32; bf16 outputs are rounded once, to nearest even.
 * The weights of the product with v are rounded to what the tensor cores take, each to nearest: in
 * scaled_attn_prompt to bf16 (by at most 2^-8 of itself), in scaled_attn_decode and scaled_attn_chunk to fp16 (2^-11; with its value block's
 * scale inside, and light ones by up to 2^-32, in scaled_attn_chunk 2^-31, of the row's largest such weight: where one visible block's value scale is 2^22 or
 * more above the others', their light weights lose bits in every dimension).  The denominator takes them unrounded.
 * scaled_attn_chunk takes a query row's elements to 2^-21 of its largest; those from 2^-13 of it on are exact.
 *
 * NaN and infinity: what a row does not see does not reach it, with one exception, a non-finite
 * VALUE (v) of the row's own sequence behind the causal edge: its weight is zero, but the matrix
 * product takes it with keys that other rows see, and zero times infinity is NaN.  In
 * scaled_attn_prompt the value of a key up to 142 past the last that a row sees (the rest of its
 * tile of 128 rows, rounded up to 16 keys) may make that dimension of the row NaN, and so may it in scaled_attn_chunk
 * (where a value scale that is NaN stands for its 16 keys); in scaled_attn_decode with several query tokens, one of them may do so to the rows before it.
 * Keys (k), bytes of the cache that no token has been written to, and other sequences never do.
 *
 * Errors, streams and programmatic launches: as in scaled_gemm.h.  A handle owns a
 * workspace that scaled_attn_decode and scaled_attn_chunk use, so those calls on one handle must be ordered (one
 * stream, ordered streams, or a handle per stream); append and prompt may run
 * concurrently with anything that does not touch their buffers.  No call synchronises,
 * allocates or reads device memory on the host, so all of them can be captured in a CUDA graph.
 */
#ifndef SCALED_ATTENTION_H
#define SCALED_ATTENTION_H

#include "scaled_gemm.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct sg_attn* sg_attn_t;

typedef struct sg_kv_cache {
  void* k;
  void* v;
  uint8_t* k_scale;
  uint8_t* v_scale;
  int64_t num_pages;
  int64_t k_page_stride; /* bytes */
  int64_t v_page_stride;
} sg_kv_cache_t;

typedef struct sg_rotary {
  const float* table;
  int64_t max_pos;
  int32_t rot;         /* rotated dimensions of a head; 0: none (table may be NULL) */
  int32_t interleaved; /* 0: pairs (i, i + rot/2); 1: pairs (2i, 2i + 1) */
} sg_rotary_t;

/* Create a plan for Hq query heads, Hk key/value heads of D dimensions and pages of
 * `page` tokens on `device` (-1: the current one). */
sg_status_t scaled_attn_create(sg_attn_t* out, int64_t Hq, int64_t Hk, int64_t D, int64_t page, int device);

/* Free the plan; NULL is allowed.  Must not race a launch on it. */
sg_status_t scaled_attn_destroy(sg_attn_t h);

/* Append T new tokens of B sequences.  Sequence b has ctx_lens[b] tokens in the cache
 * (int32, a negative one counts as 0); its new ones, rows [cu_seqlens[b], cu_seqlens[b+1]),
 * take the positions after them.  With (a, b) a rotated pair and (c, s) its position's cosine and
 * sine, in fp32, every operation rounded:
 *     a' = a c - b s,   b' = a s + b c.
 * q_out [T][Hq][D] and k_out [T][Hk][D] (or NULL) get the rotated q and k in bf16.  The cache
 * gets e4m3 codes of the fp32 rotated k and of v.  The scale of a block of 16 positions
 * of a head is the least power of two s with |x| <= 448 s over the block's new tokens (code 0 for zeros), and
 * not less than the scale the block's older tokens already have; where it grows, their
 * codes are rounded to the new scale.  Codes are rounded to nearest even; NaN stays NaN and infinity
 * saturates.  q_out may be q and k_out k where their layouts agree. */
sg_status_t scaled_attn_append(sg_attn_t h, const sg_kv_cache_t* cache, const sg_rotary_t* rotary,
                               const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                               const void* v, int64_t v_stride, const int32_t* table,
                               int64_t table_stride, const int32_t* ctx_lens,
                               const int32_t* cu_seqlens, int64_t T, int64_t B, void* q_out,
                               void* k_out, sg_stream_t stream);

/* out [B * qn][Hq][D] = softmax(scale q k^T) v over each sequence's first kv_lens[b] tokens
 * in the cache (int32; clamped to [0, table_stride * page]).  q has qn rows for each
 * sequence, its newest tokens in order: row i of them sees the first kv_lens[b] - (qn - 1 - i) tokens. */
sg_status_t scaled_attn_decode(sg_attn_t h, const sg_kv_cache_t* cache, const void* q, int64_t q_stride,
                               int64_t qn, const int32_t* table, int64_t table_stride,
                               const int32_t* kv_lens, int64_t B, float scale, void* out, float* lse,
                               sg_stream_t stream);

/* The same for chunks of new tokens, as many for each sequence as there are: q and out have the T rows of B packed
 * sequences, [cu_q[b], cu_q[b + 1]) the newest tokens of sequence b in order, whose first kv_lens[b] tokens (themselves
 * included) are in the cache.  Row i of n sees the first kv_lens[b] - (n - 1 - i). */
sg_status_t scaled_attn_chunk(sg_attn_t h, const sg_kv_cache_t* cache, const void* q, int64_t q_stride,
                              const int32_t* table, int64_t table_stride, const int32_t* kv_lens,
                              const int32_t* cu_q, int64_t T, int64_t B, float scale, void* out, float* lse,
                              sg_stream_t stream);

/* out [Tq][Hq][D] = softmax(scale q k^T) v within each of B packed sequences: queries
 * [cu_q[b], cu_q[b+1]) over keys [cu_k[b], cu_k[b+1]).  causal: with n queries and m keys, query
 * i sees the keys j <= i + m - n. */
sg_status_t scaled_attn_prompt(sg_attn_t h, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                               const void* v, int64_t v_stride, const int32_t* cu_q, const int32_t* cu_k,
                               int64_t Tq, int64_t Tk, int64_t B, int causal, float scale, void* out,
                               float* lse, sg_stream_t stream);

/* The pages of a cache and the sequences that hold them, all in device memory.  An array without elements may be NULL.  The caches of a
 * model's layers share one pool: a page number means that page of each. */
typedef struct sg_page_pool {
  int32_t* table;  /* [rows][table_stride]: the pages of each row's tokens in order, -1 past the last (4-byte aligned) */
  int32_t* lens;   /* [rows]: tokens of each row; a negative one counts as 0 (4-byte aligned).  These calls alone change it: the pages behind a
                      length that is lowered by hand stay in the table, and grow would write others over them. */
  int32_t* refs;   /* [num_pages]: table entries that name the page; free at 0 (16-byte aligned) */
  int64_t rows, table_stride, num_pages;
  void* scratch;   /* scaled_attn_pool_scratch_bytes(rows, num_pages) bytes, 16-byte aligned */
} sg_page_pool_t;

/* Pool calls change table, lens and refs, so calls on a pool (or on a scratch) must be ordered, as must attention over
 * rows that they change.  Requests are served in their order and pages taken lowest first: results do not depend on timing.
 * Entries outside [0, num_pages) name no page.  Row numbers outside [0, rows) name no row.  Where a call names a
 * row twice to be changed, the first request has it and the others are refused (release: it is released).  ok[i] (int32) is 1
 * where request i was carried out, 0 where it was refused, which leaves its row as it was.  Once the free
 * pages do not suffice for a request, later ones that need any are refused too.  rows, num_pages < 2^31 - 65536; rows * table_stride < 2^31;
 * n <= rows, or < 2^31 - 65536 for release.  Requests overlap neither the pool's memory nor the answer, nor the answer the pool's (checked:
 * SG_ERR_INVALID_ARG; two requests of a call may be the same). */

/* Bytes of a pool's scratch; 0 for sizes that no pool has. */
int64_t scaled_attn_pool_scratch_bytes(int64_t rows, int64_t num_pages);

/* Rows which[0 .. n) give their pages back: entries -1, length 0. */
sg_status_t scaled_attn_pool_release(sg_attn_t h, const sg_page_pool_t* pool, const int32_t* which, int64_t n,
                                     sg_stream_t stream);

/* Row which[i] gets the pages for add[i] >= 0 more tokens, and its length grows by them; refused where the
 * row's entries or the free pages do not suffice. */
sg_status_t scaled_attn_pool_grow(sg_attn_t h, const sg_page_pool_t* pool, const int32_t* which, const int32_t* add,
                                  int64_t n, int32_t* ok, sg_stream_t stream);

/* Row dst[i], which is empty (length 0), becomes a copy of row src[i] as it was before the call: pages that
 * src's tokens fill are shared, and of a last page that they do not fill, dst gets a copy in each of the
 * `layers` caches.  What src or dst append after that, the other does not see.  Refused where dst is not empty or
 * there is no page for the copy.  A src of length 0 leaves dst empty. */
sg_status_t scaled_attn_pool_fork(sg_attn_t h, const sg_page_pool_t* pool, const sg_kv_cache_t* caches, int64_t layers,
                                  const int32_t* src, const int32_t* dst, int64_t n, int32_t* ok, sg_stream_t stream);

/* The pages in use move to the numbers [0, *in_use), each by the table and in all caches: those past it, in order, to
 * the free ones below it, in order.  Entries that name a free page stay.  in_use: int32, device memory. */
sg_status_t scaled_attn_pool_compact(sg_attn_t h, const sg_page_pool_t* pool, const sg_kv_cache_t* caches, int64_t layers,
                                     int32_t* in_use, sg_stream_t stream);

/* Synchronise `stream` and report (and clear) the plan's status word, as
 * scaled_gemm_debug_status does. */
sg_status_t scaled_attn_debug_status(sg_attn_t h, sg_stream_t stream, int32_t* code, int32_t* where);

/* Set the time limit of every kernel-side wait of the plan (nanoseconds; 0 = the default, 4 s) and, for tests only,
 * leave out the load of key tile `skip_tile` (-1: none) of every sequence (scaled_attn_decode, scaled_attn_chunk) or of every few
 * query tokens (scaled_attn_prompt), so that the wait for it runs out.  After a timeout the call's outputs are undefined;
 * nothing else is written.
 * Not to be called while a launch on the plan is being made. */
sg_status_t scaled_attn_set_debug(sg_attn_t h, int64_t timeout_ns, int64_t skip_tile);

#ifdef __cplusplus
}
#endif
#endif
