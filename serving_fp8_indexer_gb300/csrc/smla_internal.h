// Host-side internals shared by the library's translation units.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "../../include/smla.h"

namespace smla {

// Records a message for smla_last_error() and returns `st`.
smla_status_t fail(smla_status_t st, const char* fmt, ...);
smla_status_t fail_cuda(cudaError_t e, const char* what);

// Host-side checks and lookups shared by the entry points.
void clear_last_error();
smla_status_t device_err_ptr(unsigned** out);
smla_status_t check_seqs(const smla_seqs_t& s);
smla_status_t check_attn(const void* q, int32_t q_dtype, const void* latent_pool, int64_t phys_rows,
                         const float* scales, int32_t scale_block_size, bool keyed, const uint32_t* indices,
                         int32_t indices_stride, const uint32_t* topk_lengths, int32_t T, int32_t H, int32_t v_depth,
                         float softmax_scale, const float* attn_sink, const void* out);
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// uint8 tensor map of the given rank: dims[0] innermost (elements = bytes),
// strides[i] = byte stride of dimension i + 1, box per dimension, 64- or
// 128-byte swizzle, zero fill out of bounds.  False when cuTensorMapEncodeTiled rejects it.
bool encode_tma_u8(CUtensorMap* map, const void* base, int rank, const uint64_t* dims, const uint64_t* strides,
                   const uint32_t* box, int swizzle_bytes);
// 2-D uint8 tensor map [rows][inner] (row pitch = inner bytes), box
// [box_rows][box_inner], 128- (default) or 64-byte swizzle, zero fill out of
// bounds.
bool encode_tma_2d_u8(CUtensorMap* map, const void* base, uint64_t inner, uint64_t rows, uint32_t box_inner,
                      uint32_t box_rows, int swizzle_bytes = 128);

// Number of SMs of the current device (cached per device).
int device_sm_count();

// What a kernel needs before its launches on a device, done on the first one:
// its dynamic shared memory granted, and its register count checked where its
// register split (setmaxnreg) draws on it (0: no split).  `done`: one bit per
// device, the caller's, per kernel.
smla_status_t prepare_kernel(const void* fn, size_t smem, int regs, std::atomic<unsigned long long>& done,
                             const char* what);

smla_status_t launch_indexer(const uint8_t* q, const float* q_scale, const uint8_t* k_pool, const float* k_scale,
                             int64_t phys_rows, const smla_seqs_t& seqs, int h_idx, float* scores,
                             int64_t score_stride, unsigned* err, cudaStream_t stream);

// Fused indexer + top-k (score rows in shared memory): the longest row it
// holds for this H_idx, and its launcher (kv_len <= that cap).
int indexer_topk_row_cap(int h_idx);
smla_status_t launch_indexer_topk(const uint8_t* q, const float* q_scale, const uint8_t* k_pool, const float* k_scale,
                                  int64_t phys_rows, const smla_seqs_t& seqs, int h_idx, int k, uint32_t* indices,
                                  uint32_t* topk_lengths, unsigned* err, cudaStream_t stream);

smla_status_t launch_topk(const float* scores, int64_t score_stride, const smla_seqs_t& seqs, int k,
                          uint32_t* indices, uint32_t* topk_lengths, unsigned* err, cudaStream_t stream);

// One launch of the attention kernel: sparse (indices + lengths) or dense
// causal (seqs non-null: every key 0..pos through the page table), with an
// optional per-head sink and, for nsplit > 1, split-K partials instead of
// the bf16 output.
struct AttnArgs {
  const void* q;
  int q_dtype;
  const uint8_t* latent;
  int64_t phys_rows;
  const float* scales;
  int sbs;
  const uint32_t* indices;
  int indices_stride;
  const uint32_t* topk_lengths;
  const smla_seqs_t* seqs;
  int T, H;
  float softmax_scale;
  const float* sink;
  uint16_t* out;
  int nsplit;
  float* part_o;    // [T, nsplit, H, 512]
  float* part_lse;  // [T, nsplit, H]
  int cache_bf16;   // latent_pool holds bf16 [phys_rows, 576] (q bf16, no scales)
};
smla_status_t launch_attention(const AttnArgs& a, unsigned* err, cudaStream_t stream);

// Split-K decode: the split count for these sizes, the workspace it needs,
// and the kernel that combines the partials into the bf16 output.
int decode_splits(int T, int H, int indices_stride);
size_t decode_workspace_bytes(int T, int H, int nsplit);
// Fixed scratch of smla_sparse_decode_noalloc (a static device array): its
// size, and its device address on the current device when `need` bytes fit
// (SMLA_ERR_UNSUPPORTED otherwise; nullptr when need is 0).
size_t noalloc_scratch_bytes();
smla_status_t noalloc_scratch_for(size_t need, void** out);
smla_status_t launch_decode_combine(const float* part_o, const float* part_lse, const float* sink, int T, int H,
                                    int nsplit, uint16_t* out, cudaStream_t stream);

// Rotary positions of x [T, H, D] into out.
struct RopeArgs {
  const void* x;
  int x_dtype;
  int64_t x_ts, x_hs;  // token and head strides, elements
  int H, D;
  smla_rope_t rope;
  void* out;
  int out_dtype;
  int64_t o_ts, o_hs;
};
smla_status_t launch_rope(const RopeArgs& a, const smla_seqs_t& seqs, unsigned* err, cudaStream_t stream);

// Writing (x -> pool, optionally rows) and reading (pool -> rows) the cached
// rows of a batch's tokens.
struct CacheArgs {
  const void* x;
  int64_t x_stride;
  int D;
  const void* norm_weight;  // null: no norm
  int norm_dim;
  float norm_eps;
  smla_rope_t rope;
  void* pool;
  int pool_dtype;
  int64_t phys_rows;
  float* scales;
  int sbs;
  void* rows;
  int64_t rows_stride;
};
smla_status_t launch_cache_append(const CacheArgs& a, const smla_seqs_t& seqs, unsigned* err, cudaStream_t stream);
smla_status_t launch_cache_gather(const CacheArgs& a, const smla_seqs_t& seqs, unsigned* err, cudaStream_t stream);

// Latent attention in the expanded form.  Strides in elements.
struct ExpandedArgs {
  const void* q;  // [T, H, 192]
  int64_t q_ts, q_hs;
  const void* k_nope;  // [S, H, 128]
  int64_t k_ts, k_hs;
  const void* k_rope;  // [S, 64]
  int64_t r_ts;
  const void* v;  // [S, H, 128]
  int64_t v_ts, v_hs;
  const int32_t* cu_q;
  const int32_t* cu_kv;
  int B, T, S, H;
  float softmax_scale;
  const float* sink;
  uint16_t* out;
  float* lse;
  int nsplit;
  void* workspace;
  int p_terms;  // of the weights: 1, 2 or 0 (by the call's size)
};
// Splits of the keys for these sizes, the workspace they need, the launch.
int expanded_splits(int T, int S, int B, int H);
size_t expanded_workspace_bytes(int T, int H, int nsplit);
smla_status_t launch_expanded(const ExpandedArgs& a, unsigned* err, cudaStream_t stream);

// Dense decode: over an e4m3 cache with unit or per-row scales, and (`wide`:
// 16-bit operands) over a bf16 cache or one with block scales.
struct DenseDecodeArgs {
  const void* q;
  int q_dtype;
  const void* latent;
  int64_t phys_rows;
  const float* scales;  // null: unit (wide: a bf16 cache)
  const smla_seqs_t* seqs;
  int T, H, max_kv_len;
  float softmax_scale;
  const float* sink;
  uint16_t* out;
  void* workspace;
};
size_t dense_decode_workspace_bytes(int T, int H, int max_kv_len);
smla_status_t launch_dense_decode(const DenseDecodeArgs& a, unsigned* err, cudaStream_t stream);
smla_status_t launch_dense_decode_wide(const DenseDecodeArgs& a, unsigned* err, cudaStream_t stream);

}  // namespace smla
