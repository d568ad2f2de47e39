/*
 * smla.h -- C ABI of libsmla: the FP8 lightning indexer, per-token top-k and
 * MLA attention (sparse, dense, expanded; prefill and decode), with the rotary
 * positions and the cache writes and reads around them, for GB300 (sm_103a).
 *
 * Every entry point takes plain device pointers and sizes, validates them on
 * the host, enqueues its kernels asynchronously on `stream` and returns an
 * smla_status_t.  The caller owns every buffer; the library allocates no
 * device memory.  No C++ exception crosses this boundary.  A call that
 * returns anything but SMLA_OK has enqueued nothing (except SMLA_ERR_CUDA,
 * where a launch was attempted and failed); smla_last_error() then holds a
 * message for the calling thread.
 *
 * Errors found on the device (an index or page id outside the pool, a
 * pipeline wait that gave up) are recorded in a per-device error word
 * instead of faulting; the kernel that found them skips the offending
 * access and finishes.  smla_check_device_errors() reads and clears that
 * word.  Outputs of a call that recorded a device error are unspecified.
 *
 * Layouts are row-major and dense unless a stride is given.  "e4m3" is the
 * float8_e4m3fn byte format; "bf16" is bfloat16 bits.  Each call states the
 * alignment its pointers need; a misaligned pointer returns
 * SMLA_ERR_INVALID_ARG.
 */
#ifndef SMLA_H_
#define SMLA_H_

#include <stddef.h>
#include <stdint.h>
#include <cuda_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SMLA_OK = 0,
  SMLA_ERR_INVALID_ARG = 1,  /* null pointer, bad size, misaligned pointer */
  SMLA_ERR_UNSUPPORTED = 2,  /* valid but outside the shapes this build implements */
  SMLA_ERR_CUDA = 3,         /* a CUDA runtime/driver call failed */
  SMLA_ERR_TIMEOUT = 4,      /* a device pipeline wait gave up (device error word) */
  SMLA_ERR_DEVICE_CHECK = 5  /* an index / page id was out of range (device error word) */
} smla_status_t;

enum { SMLA_BF16 = 0, SMLA_E4M3 = 1, SMLA_F32 = 2 };

/* Ragged batch of B sequences over a paged cache (all pointers on the device).
 * Sequence b owns query tokens cu_q[b] .. cu_q[b+1]-1 and kv_len[b] cached
 * tokens; its q_len = cu_q[b+1]-cu_q[b] new tokens are the LAST q_len cached
 * positions, so its token i sits at pos = kv_len[b] - q_len + i and may
 * attend to logical keys 0..pos.  Logical key j of sequence b is physical
 * row page_table[b*max_pages + j/page_size]*page_size + j%page_size.
 * T = cu_q[B] (passed on the host so that no call reads device memory to
 * size its grid).  Requires q_len <= kv_len for every sequence.  The three
 * pointers must be 4-byte aligned. */
typedef struct {
  const int32_t* cu_q;        /* [B+1] */
  const int32_t* kv_len;      /* [B] */
  const int32_t* page_table;  /* [B, max_pages] physical page ids */
  int32_t B;
  int32_t max_pages;
  int32_t page_size;          /* power of two, 8..4096 */
  int32_t T;
} smla_seqs_t;

/* Stage 1 -- FP8 lightning-indexer scores.
 * "sparse_index_fp8_sm100" (Modular Mojo kernel page), module summary and
 * section "Layout (crux)":
 *   scores[t, key] = k_scale[phys(key)] * sum_h relu(q[t,h,:] . k_pool[phys(key),:]) * q_scale[t,h]
 * for every logical key 0..pos(t) of t's sequence; every other entry of row
 * t (key > pos(t), up to score_stride) is written as -inf (the causal tail
 * fill, fused).
 *   q        e4m3 [T, H_idx, 128]
 *   q_scale  f32  [T, H_idx]
 *   k_pool   e4m3 [phys_rows, 128]  paged indexer keys
 *   k_scale  f32  [phys_rows]       per physical row
 *   scores   f32  [T, score_stride] (output; score_stride >= max kv_len, multiple of 4)
 * H_idx must be 4, 8, 16, 32 or 64 (SMLA_ERR_UNSUPPORTED otherwise).
 * Alignment: q, k_pool and scores 16 bytes; q_scale and k_scale 4 bytes.
 * The dot products run on tcgen05 FP8 tensor cores with f32 accumulation. */
smla_status_t smla_indexer_scores(const uint8_t* q, const float* q_scale, const uint8_t* k_pool,
                                  const float* k_scale, int64_t phys_rows, smla_seqs_t seqs,
                                  int32_t H_idx, float* scores, int64_t score_stride,
                                  cudaStream_t stream);

/* Stage 2 -- per-token top-k over the causally valid keys.
 * "sparse_index_fp8_sm100" (the indexer's score buffer is this stage's
 * input; the page verifies the result as a top-k set match) and
 * "mla_sm100_prefill_sparse_fp8" (indices in physical-row space + per-query
 * topk_lengths):
 *   topk_lengths[t] = min(k, pos(t)+1)
 *   indices[t, 0..len) = physical rows of the len largest scores[t, 0..pos(t)],
 *                        ties broken toward the lower logical key, emitted in
 *                        ascending logical-key order
 *   indices[t, len..k) = 0xFFFFFFFF
 *   scores   f32 [T, score_stride] (entries past pos(t) do not affect the
 *            result; a row's last 16-byte load may read up to three of them)
 *   indices  u32 [T, k] (output), topk_lengths u32 [T] (output)
 * workspace: caller-owned device scratch of at least
 * smla_topk_workspace_size(T, score_stride, k) bytes (16-byte aligned; may
 * be NULL when that size is 0, which it is for every shape this build
 * selects in one pass per row); its contents on entry do not matter and are
 * unspecified on return.  A smaller workspace_bytes returns
 * SMLA_ERR_INVALID_ARG.
 * 1 <= k <= 65536. NaN scores are unsupported (their order is unspecified).
 * Alignment: scores 16 bytes; indices and topk_lengths 4 bytes. */
size_t smla_topk_workspace_size(int32_t T, int64_t score_stride, int32_t k);
smla_status_t smla_topk(const float* scores, int64_t score_stride, smla_seqs_t seqs, int32_t k,
                        uint32_t* indices, uint32_t* topk_lengths, void* workspace, size_t workspace_bytes,
                        cudaStream_t stream);

/* Stages 1 + 2 fused -- indexer scores and per-token top-k in one pass, the
 * score rows kept in the SM's shared memory instead of an HBM buffer.
 * "sparse_index_fp8_sm100" (module summary: the scorer is a drop-in for the
 * buffer the top-k stage reads, and the fusions that follow it are left to
 * later work).  Outputs exactly what smla_indexer_scores followed by
 * smla_topk produce: the same scores (same MMAs and epilogue arithmetic in
 * the same order), the same selection rule (ties to the lower logical key),
 * indices u32 [T, k] in ascending logical-key order with the 0xFFFFFFFF
 * tail, topk_lengths u32 [T].
 *   q, q_scale, k_pool, k_scale, phys_rows, seqs, H_idx: as smla_indexer_scores
 *   score_stride: a bound on every kv_len (>= max kv_len, multiple of 4), as
 *                 the unfused pair's score row stride
 *   k, indices, topk_lengths: as smla_topk
 * Rows of up to 128 * H_idx keys (8192 at H_idx 64) stay on chip and need no
 * workspace; for a larger score_stride the call runs the unfused pair with
 * the score buffer [T, score_stride] in `workspace`.  workspace: caller-owned
 * device scratch of at least smla_indexer_topk_workspace_size(T,
 * score_stride, H_idx, k) bytes (16-byte aligned; NULL when that is 0);
 * contents on entry do not matter, unspecified on return.  Errors and
 * alignment as for the two stages. */
size_t smla_indexer_topk_workspace_size(int32_t T, int64_t score_stride, int32_t H_idx, int32_t k);
smla_status_t smla_indexer_topk(const uint8_t* q, const float* q_scale, const uint8_t* k_pool,
                                const float* k_scale, int64_t phys_rows, smla_seqs_t seqs, int32_t H_idx,
                                int64_t score_stride, int32_t k, uint32_t* indices, uint32_t* topk_lengths,
                                void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Stage 3 -- sparse MLA prefill attention.
 * "mla_sm100_prefill_sparse_fp8" (Modular Mojo function page: arguments,
 * scale_block_size modes) and "mla_prefill_sparse_qkv_fp8" (K and V share
 * the latent rows; V = the first v_depth columns).  For each token t and
 * head h, with n = topk_lengths[t] and K_j = dequant(latent_pool[indices[t,j]]):
 *   s_j = softmax_scale * q[t,h,:] . K_j,
 *   p_j = exp(s_j) / (exp(sink_h) + sum_i exp(s_i))   (sink_h = attn_sink[h], or no term when NULL),
 *   out[t,h,:] = bf16_rne( sum_j p_j * K_j[0:v_depth] )     (zeros if n == 0)
 *   q            [T, H, 576], bf16 (q_dtype SMLA_BF16) or e4m3 (SMLA_E4M3)
 *   latent_pool  e4m3 [phys_rows, 576] (512 nope + 64 rope)
 *   scales       f32 [phys_rows, ceil(576/scale_block_size)]; NULL when
 *                scale_block_size == 0 (unit scale); scale_block_size >= 576
 *                means one scale per row; 32 means 18 block scales per row
 *   indices      u32 [T, indices_stride] physical rows; topk_lengths u32 [T]
 *                (each <= indices_stride)
 *   attn_sink    f32 [H] or NULL: one logit per head, in the units of the
 *                scaled logits s_j, that joins every softmax denominator and
 *                carries no value (the page names the argument without
 *                defining it; this is the reading taken)
 *   out          bf16 [T, H, v_depth] (output)
 * Supported: H in {16, 32, 48, 64} or any multiple of 64; v_depth == 512;
 * scale_block_size in {0, 32} or >= 576, where 32 (block scales) requires e4m3
 * q.  Alignment: q, latent_pool and out 16 bytes; indices, topk_lengths,
 * scales and attn_sink 4 bytes.  Other shapes return SMLA_ERR_UNSUPPORTED,
 * misaligned pointers SMLA_ERR_INVALID_ARG; nothing is launched then.
 * Runs on tcgen05 FP8 tensor cores with f32 TMEM accumulation: e4m3 q is
 * used natively; bf16 q and the softmax weights P (bf16-accuracy path) are
 * carried as two e4m3 terms (hi + lo) so that the products stay on the FP8
 * pipe; blockwise-scaled rows are dequantised to the same two-term form. */
smla_status_t smla_sparse_prefill(const void* q, int32_t q_dtype, const uint8_t* latent_pool,
                                  int64_t phys_rows, const float* scales, int32_t scale_block_size,
                                  const uint32_t* indices, int32_t indices_stride,
                                  const uint32_t* topk_lengths, int32_t T, int32_t H,
                                  int32_t v_depth, float softmax_scale, const float* attn_sink,
                                  uint16_t* out, cudaStream_t stream);

/* Sparse MLA prefill over a BF16 latent cache: "mla_sm100_prefill_sparse_fp8"
 * names itself the FP8 KV-cache variant of "mla_sm100_prefill_sparse"; this
 * is that BF16-cache form.  The same computation as smla_sparse_prefill with
 * K_j = latent_pool[indices[t,j]] read as bf16 (no scales):
 *   q            bf16 [T, H, 576]
 *   latent_pool  bf16 [phys_rows, 576] (512 nope + 64 rope)
 *   indices, topk_lengths, attn_sink, out, H, v_depth: as smla_sparse_prefill
 * Alignment: q, latent_pool and out 16 bytes; indices, topk_lengths and
 * attn_sink 4 bytes.  The products run as tcgen05 kind::f16 (bf16 x bf16)
 * MMAs with f32 TMEM accumulation; P is rounded to bf16. */
smla_status_t smla_sparse_prefill_bf16_cache(const uint16_t* q, const uint16_t* latent_pool, int64_t phys_rows,
                                             const uint32_t* indices, int32_t indices_stride,
                                             const uint32_t* topk_lengths, int32_t T, int32_t H,
                                             int32_t v_depth, float softmax_scale, const float* attn_sink,
                                             uint16_t* out, cudaStream_t stream);

/* Dense causal MLA prefill over the paged latent cache, for prompts short
 * enough that a top-k selection would keep every key.  "SM100MLA" (the
 * dense MLA prefill struct page) and "mla_sm100_prefill_blockscale" (dense
 * MLA prefill with a block-scaled FP8 cache): token t of sequence b attends
 * to every logical key 0..pos(t) of b (pos as in smla_seqs_t), reached
 * through the page table, so no indices are read:
 *   out[t,h,:] = sum_{j <= pos(t)} p_j * K_j[0:v_depth],
 *   K_j = dequant(latent_pool[phys(b, j)]), p and the sink as for
 *   smla_sparse_prefill.
 * This equals smla_sparse_prefill with indices[t] = phys(b, 0..pos(t)) and
 * topk_lengths[t] = pos(t)+1.  T = seqs.T; q [T, H, 576] and out
 * [T, H, 512] as there; the other arguments, supported shapes, alignment
 * and errors as for smla_sparse_prefill. */
smla_status_t smla_dense_prefill(const void* q, int32_t q_dtype, const uint8_t* latent_pool,
                                 int64_t phys_rows, const float* scales, int32_t scale_block_size,
                                 smla_seqs_t seqs, int32_t H, int32_t v_depth, float softmax_scale,
                                 const float* attn_sink, uint16_t* out, cudaStream_t stream);

/* Sparse MLA decode: the sparse attention of smla_sparse_prefill for few
 * query tokens (one or two per sequence), the other serving phase of the
 * same cache and indices ("mla_prefill_sparse_qkv_fp8", which names the
 * FP8 decode QK / PV machinery the prefill reuses).  Same arguments, result
 * and rules as smla_sparse_prefill.  When the (token, 64-head group) pairs
 * are too few to fill the GPU, each token's key blocks are divided among
 * several CTAs, whose partial outputs and log-sum-exps go to `workspace`
 * and are merged by a second kernel.  workspace: caller-owned device
 * scratch of at least smla_sparse_decode_workspace_size(T, H,
 * indices_stride) bytes on the current device (16-byte aligned; NULL when
 * that size is 0); contents on entry do not matter, unspecified on return;
 * too small returns SMLA_ERR_INVALID_ARG. */
size_t smla_sparse_decode_workspace_size(int32_t T, int32_t H, int32_t indices_stride);
smla_status_t smla_sparse_decode(const void* q, int32_t q_dtype, const uint8_t* latent_pool,
                                 int64_t phys_rows, const float* scales, int32_t scale_block_size,
                                 const uint32_t* indices, int32_t indices_stride,
                                 const uint32_t* topk_lengths, int32_t T, int32_t H,
                                 int32_t v_depth, float softmax_scale, const float* attn_sink,
                                 uint16_t* out, void* workspace, size_t workspace_bytes,
                                 cudaStream_t stream);

/* smla_sparse_decode without a workspace, for callers that cannot allocate
 * device memory at the point where they decode: code running inside another
 * runtime's enqueue step that forbids allocation (an inference-engine
 * plugin, say), or a serving loop whose device memory is all reserved by a
 * pool it may not go around, or where a cudaMalloc would stall the loop.
 * The papers have no counterpart of this call; it is an integration
 * convenience.
 * Same arguments, result and rules as smla_sparse_decode, minus workspace
 * and workspace_bytes: the split partials live in a fixed 32 MiB scratch
 * array that the library declares in device memory.  Every GPU that loads
 * the library holds those 32 MiB until the process exits.  The call
 * allocates nothing (no cudaMalloc, cudaFree or allocating library routine).
 * The first call on a device looks the array's device address up (once,
 * with that device current) and should come before any stream capture.
 * The split count is the one smla_sparse_decode uses; on a 152-SM GB300 it
 * never needs more than about 20 MB.  Sizes that would need more than 32 MiB
 * return SMLA_ERR_UNSUPPORTED with a message naming the need, and nothing
 * is launched.  All calls share the one array, which keeps the last call's
 * contents; every entry a call reads back is written first by that call, so
 * nothing has to start at zero.  Calls whose kernels overlap on the GPU
 * (different streams, or other host threads) race on the array: order them
 * on one stream. */
smla_status_t smla_sparse_decode_noalloc(const void* q, int32_t q_dtype, const uint8_t* latent_pool,
                                         int64_t phys_rows, const float* scales, int32_t scale_block_size,
                                         const uint32_t* indices, int32_t indices_stride,
                                         const uint32_t* topk_lengths, int32_t T, int32_t H,
                                         int32_t v_depth, float softmax_scale, const float* attn_sink,
                                         uint16_t* out, cudaStream_t stream);

/* ------------------------------------------------------------------------
 * Around the attention calls: rotary positions, the caches' write and read
 * side, attention in the expanded form, and dense decode.  In all of them a
 * token's position is the one smla_seqs_t gives it, and tokens behind the
 * last sequence (t >= cu_q[B], as in a batch padded to a fixed T) are
 * skipped: their outputs are left as they were.
 * ------------------------------------------------------------------------ */

enum { SMLA_ROPE_INTERLEAVED = 0, SMLA_ROPE_HALF = 1 };
enum { SMLA_ROPE_PLAIN = 0, SMLA_ROPE_LINEAR = 1, SMLA_ROPE_YARN = 2 };

/* A rotary embedding over columns [offset, offset + dim) of a row: pair i of
 * the dim / 2 pairs is turned by pos * inv_freq[i] radians and multiplied by
 * `amplitude`,
 *   (p, q) -> amplitude * (p cos - q sin, q cos + p sin),
 * where (p, q) are the part's columns (2i, 2i+1) (SMLA_ROPE_INTERLEAVED) or
 * (i, i + dim/2) (SMLA_ROPE_HALF).  The angle is formed in 64-bit fixed
 * point, so it is as exact at position 2^31 as at position 0.
 * offset and dim are multiples of 8 and 16; dim = 0 turns nothing. */
typedef struct {
  const double* inv_freq;  /* device, f64 [dim/2], finite, 8-byte aligned */
  int32_t offset;
  int32_t dim;
  int32_t layout;          /* SMLA_ROPE_INTERLEAVED or SMLA_ROPE_HALF */
  float amplitude;
} smla_rope_t;

/* Host helper (no device work): the frequencies f_i = base^(-2i/dim) of a
 * rotary embedding, scaled for contexts longer than the model was trained
 * on, into inv_freq (host, f64 [dim/2]) and *amplitude.
 *   SMLA_ROPE_PLAIN   as they are
 *   SMLA_ROPE_LINEAR  every f_i / factor (position interpolation)
 *   SMLA_ROPE_YARN    f_i kept where the pair makes more than beta_fast turns
 *                     over original_len positions, f_i / factor where fewer
 *                     than beta_slow, a linear ramp over i between;
 *                     amplitude = 0.1 ln(factor) + 1
 * dim: even, 2..1024; base > 1; factor >= 1; original_len >= 1 and
 * beta_fast > beta_slow > 0 for YARN (ignored otherwise). */
smla_status_t smla_rope_frequencies(int32_t dim, double base, int32_t scaling, double factor, int32_t original_len,
                                    double beta_fast, double beta_slow, double* inv_freq, float* amplitude);

/* Rotary positions of x [T, H, D] (T = seqs.T) into out [T, H, D]: the
 * columns outside the rotated part are copied; everything is converted to
 * out's type with one rounding (e4m3: to nearest even, values beyond +-448
 * become +-448).
 *   x    bf16 or f32, element (t, h, c) at x[t * x_token_stride + h * x_head_stride + c]
 *   out  bf16, f32 or e4m3, likewise; either x itself (same pointer, type and
 *        strides: rotated in place) or memory that x does not overlap
 * D: a multiple of 8, 16..1024.  H: 1..65535.  Strides: in elements,
 * multiples of 8; out's rows may not overlap (a stride of 0 is refused; x's
 * may be 0: one row for several heads).  Alignment: x and out 16 bytes (out
 * e4m3: 8).
 * Reads only cu_q and kv_len of seqs (page_table may be any valid pointer). */
smla_status_t smla_rope(const void* x, int32_t x_dtype, int64_t x_token_stride, int64_t x_head_stride,
                        smla_seqs_t seqs, int32_t H, int32_t D, smla_rope_t rope, void* out, int32_t out_dtype,
                        int64_t out_token_stride, int64_t out_head_stride, cudaStream_t stream);

/* Writes the batch's new rows into a paged cache (the MLA latents, D = 576,
 * or the indexer keys, D = 128): for each token t of seqs
 *   r = x[t];  r[0:norm_dim] = r[0:norm_dim] * rsqrt(mean(r[0:norm_dim]^2) + norm_eps) * norm_weight
 *   r = rope(r) at pos(t)
 *   pool[phys(pos(t))] = r in the cache's format, rows_out[t] = bf16(r)
 * Formats: bf16 (scale_block_size 0), or e4m3 with scale_block_size 0 (unit
 * scale, values beyond +-448 become +-448), >= D (one scale per row) or 32
 * (D / 32 block scales per row), where scale = largest finite magnitude /
 * 448 (1 when that is 0; at least the smallest normal f32), byte = e4m3(r /
 * scale), of the f32 quotient (below a scale of 2^-100, of one that may be off in
 * its last place).  NaN stays NaN and infinities saturate.
 *   x            bf16 [T, D], rows x_stride elements apart
 *   norm_weight  bf16 [norm_dim], or NULL for no norm (norm_dim is then ignored)
 *   rope         dim = 0 for none; its columns may overlap the normalised ones
 *   pool         [phys_rows, D] (output)
 *   scales       f32 [phys_rows, D / min(scale_block_size, D)] (output), NULL
 *                when scale_block_size == 0
 *   rows_out     bf16 [T, D], rows rows_stride elements apart, or NULL; not
 *                overlapping x
 * D: a multiple of 8 (of 32 for block scales), 16..1024; norm_dim a multiple
 * of 8 up to D; x_stride and rows_stride multiples of 8, >= D.  Alignment:
 * x, norm_weight, pool, rows_out 16 bytes; scales 4.  A token whose page lies
 * outside the pool is reported (SMLA_ERR_DEVICE_CHECK) and not written.  No
 * two tokens of a call may share a physical row. */
smla_status_t smla_cache_append(const uint16_t* x, int64_t x_stride, smla_seqs_t seqs, int32_t D,
                                const uint16_t* norm_weight, int32_t norm_dim, float norm_eps, smla_rope_t rope,
                                void* pool, int32_t pool_dtype, int64_t phys_rows, float* scales,
                                int32_t scale_block_size, uint16_t* rows_out, int64_t rows_stride,
                                cudaStream_t stream);

/* Reads cached rows back: rows[t] = bf16(pool[phys(pos(t))] * scale) for each
 * token t of seqs.  With cu_q the running sum of kv_len (every q_len =
 * kv_len) this is the whole cached context of the batch, sequence after
 * sequence, as the expansion of a chunk's context needs it.  pool, scales,
 * phys_rows, D, formats and alignment as smla_cache_append; rows bf16 [T, D],
 * rows_stride elements apart. */
smla_status_t smla_cache_gather(const void* pool, int32_t pool_dtype, int64_t phys_rows, const float* scales,
                                int32_t scale_block_size, smla_seqs_t seqs, int32_t D, uint16_t* rows,
                                int64_t rows_stride, cudaStream_t stream);

/* Latent attention in the expanded form, for prefill: every head has keys and
 * values of its own, up-projected from the latents, and all heads share the
 * rotary part of the keys.  For token t of sequence b and head h, over the
 * keys j = 0..pos(t) of b,
 *   z_j = softmax_scale * (q[t,h,0:128] . k_nope[j,h] + q[t,h,128:192] . k_rope[j])
 *   out[t,h] = bf16( sum_j p_j v[j,h] ),  p and the sink as for smla_sparse_prefill
 *   lse[t,h] = ln( sum_j exp(z_j) [+ exp(sink_h)] )
 * Sequence b owns query tokens cu_q[b] .. cu_q[b+1]-1 and key rows cu_kv[b]
 * .. cu_kv[b+1]-1; its new tokens are the last of its keys, so token i sits
 * at pos = kv_len - q_len + i.  A token that attends to nothing (no keys, or
 * pos < 0) gets zeros, and lse -inf (the sink's logit with a sink).
 *   q       bf16 [T, H, 192]; element (t, h, c) at q[t * q_token_stride + h * q_head_stride + c]
 *   k_nope  bf16 [S, H, 128], v bf16 [S, H, 128]: likewise strided, so that they may be
 *           the two halves of one up-projection's output
 *   k_rope  bf16 [S, 64], rows k_rope_stride apart, rotated
 *   out     bf16 [T, H, 128], dense;  lse f32 [T, H] or NULL
 *   S       key rows in all (cu_kv[B] <= S)
 * Key rows outside a sequence never reach its outputs, whatever they hold.
 * Inside a sequence, a NaN or infinity in v at key j may also reach tokens of
 * that sequence before j (within the 128-key block), which weigh it by 0.
 * Strides: in elements, multiples of 8, at least the row's width.
 * H: 1..65535.  softmax_scale: 1e-30 .. 1e30.  Alignment: q, k_nope, k_rope, v,
 * out 16 bytes; the others 4.  workspace: caller-owned device scratch of at
 * least smla_expanded_prefill_workspace_size(T, S, B, H) bytes on the
 * current device (16-byte aligned; NULL when that is 0), used when the
 * queries alone are too few to fill the GPU; contents on entry do not matter,
 * unspecified on return; not shared by calls that may overlap.  The products
 * run as tcgen05 kind::f16 (bf16) MMAs with f32 TMEM accumulation.  The weights P
 * are carried as one bf16 term (rounded by up to 2^-8 of themselves, as the output
 * is) or two (2^-16).  smla_expanded_prefill takes two in calls of up to 64 rows
 * (T * H), where they cost little, and one in others; smla_expanded_prefill_terms
 * takes the caller's p_terms, 1 or 2, so that a row's accuracy does not depend on
 * how many others share its call (0: as smla_expanded_prefill). */
size_t smla_expanded_prefill_workspace_size(int32_t T, int32_t S, int32_t B, int32_t H);
smla_status_t smla_expanded_prefill(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride,
                                    const uint16_t* k_nope, int64_t k_token_stride, int64_t k_head_stride,
                                    const uint16_t* k_rope, int64_t k_rope_stride, const uint16_t* v,
                                    int64_t v_token_stride, int64_t v_head_stride, const int32_t* cu_q,
                                    const int32_t* cu_kv, int32_t B, int32_t T, int32_t S, int32_t H,
                                    float softmax_scale, const float* attn_sink, uint16_t* out, float* lse,
                                    void* workspace, size_t workspace_bytes, cudaStream_t stream);
smla_status_t smla_expanded_prefill_terms(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride,
                                          const uint16_t* k_nope, int64_t k_token_stride, int64_t k_head_stride,
                                          const uint16_t* k_rope, int64_t k_rope_stride, const uint16_t* v,
                                          int64_t v_token_stride, int64_t v_head_stride, const int32_t* cu_q,
                                          const int32_t* cu_kv, int32_t B, int32_t T, int32_t S, int32_t H,
                                          float softmax_scale, int32_t p_terms, const float* attn_sink, uint16_t* out,
                                          float* lse, void* workspace, size_t workspace_bytes, cudaStream_t stream);

/* Dense MLA decode (latent attention, absorbed form) for few query tokens over
 * the whole cache of their sequence: out[t,h] as for smla_dense_prefill, with
 *   - the keys of a token divided among several CTAs when the tokens are too
 *     few to fill the GPU, and the partial results merged by a second kernel;
 *   - the weights P carried at bf16's accuracy whatever q's type: each is off by
 *     at most 2^-8 of itself, or by 2^-28 of its row's largest where that is more
 *     (of p_j s_j, s_j the row's scale), so that the many keys far below a
 *     dominant one keep their weight.  (smla_dense_prefill and the sparse calls
 *     round P to one e4m3 term for e4m3 q, and to two, which end 2^-14 below a
 *     row's largest, for bf16 q.)  bf16 q is exact down to 2^-14 of its row's
 *     largest element over an e4m3 cache, smaller elements are off by up to 2^-22
 *     of that, and exact over a bf16 cache;
 *   - e4m3 caches in every scale mode, or a bf16 cache.
 *   q            [T, H, 576], bf16 or e4m3 (q_dtype)
 *   latent_pool  [phys_rows, 576], e4m3 or bf16 (pool_dtype)
 *   scales, scale_block_size, H, v_depth, softmax_scale, attn_sink, out: as for
 *                smla_dense_prefill
 *   max_kv_len   a bound on every kv_len, for the choice of the split; larger
 *                lengths are served too, only less evenly
 * Block scales (32) take e4m3 q; a bf16 cache takes bf16 q and
 * scale_block_size 0 (SMLA_ERR_UNSUPPORTED otherwise).  A block-scaled row's
 * values are carried in f16, off by at most 2^-10 of themselves or, in blocks of
 * very small scale, by 2^-30 of the row's largest scale.  Tokens behind the
 * last sequence keep their outputs.  A token of a sequence without keys gets
 * zeros.  Cache rows outside a sequence's keys never reach its outputs,
 * whatever they hold; a NaN in the row (or its scale) of one of a sequence's
 * new tokens may also reach the new tokens before it, which weigh it by 0.  A
 * row of q with a NaN or an infinity gets NaN.  workspace: caller-owned device scratch of at least
 * smla_dense_decode_workspace_size(T, H, max_kv_len) bytes on the current
 * device (16-byte aligned; NULL when that is 0); contents on entry do not
 * matter, unspecified on return; not shared by calls that may overlap. */
size_t smla_dense_decode_workspace_size(int32_t T, int32_t H, int32_t max_kv_len);
smla_status_t smla_dense_decode(const void* q, int32_t q_dtype, const void* latent_pool, int32_t pool_dtype,
                                int64_t phys_rows, const float* scales, int32_t scale_block_size, smla_seqs_t seqs,
                                int32_t max_kv_len, int32_t H, int32_t v_depth, float softmax_scale,
                                const float* attn_sink, uint16_t* out, void* workspace, size_t workspace_bytes,
                                cudaStream_t stream);

/* Synchronises `stream`, then reads and clears the current device's error
 * word.  Returns SMLA_OK, SMLA_ERR_DEVICE_CHECK (out-of-range index or page
 * id), SMLA_ERR_TIMEOUT (a pipeline wait gave up) or SMLA_ERR_CUDA. */
smla_status_t smla_check_device_errors(cudaStream_t stream);

/* Self-test of the device timeout path: enqueues one kernel whose only
 * thread waits, with a limit of limit_us microseconds (1 .. 1000000), on a
 * pipeline barrier that nothing completes, exactly as the stage kernels
 * wait on theirs.  When the limit passes, the kernel records the timeout
 * in the device error word and returns, so the next
 * smla_check_device_errors() reports SMLA_ERR_TIMEOUT.  No library function
 * calls it; it exists so that the timeout path can be tested without a
 * hung kernel. */
smla_status_t smla_selftest_wait_timeout(uint32_t limit_us, cudaStream_t stream);

/* Copies the calling thread's last error message (NUL-terminated, truncated
 * to n bytes) and returns its full length. */
size_t smla_last_error(char* buf, size_t n);

/* Library version, "major.minor.patch". */
const char* smla_version(void);

#ifdef __cplusplus
}
#endif
#endif /* SMLA_H_ */
