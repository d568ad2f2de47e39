// The C ABI of the operators around the attention calls (include/smla.h):
// host-side argument validation and dispatch to their launchers.
#include <cmath>

#include "smla_internal.h"

namespace smla {

static smla_status_t check_rope(const smla_rope_t& r, int32_t D) {
  if (r.dim == 0) return SMLA_OK;
  if (r.layout != SMLA_ROPE_INTERLEAVED && r.layout != SMLA_ROPE_HALF)
    return fail(SMLA_ERR_INVALID_ARG, "rope: layout=%d", r.layout);
  if (r.dim < 0 || r.offset < 0 || r.offset > D || r.dim > D - r.offset)
    return fail(SMLA_ERR_INVALID_ARG, "rope: columns [%d, +%d) outside a row of %d", r.offset, r.dim, D);
  if (r.dim % 16 || r.offset % 8)
    return fail(SMLA_ERR_UNSUPPORTED, "rope: dim=%d must be a multiple of 16, offset=%d of 8", r.dim, r.offset);
  if (!r.inv_freq || (reinterpret_cast<uintptr_t>(r.inv_freq) & 7u))
    return fail(SMLA_ERR_INVALID_ARG, "rope: inv_freq must be non-null and 8-byte aligned");
  if (!std::isfinite(r.amplitude)) return fail(SMLA_ERR_INVALID_ARG, "rope: amplitude must be finite");
  return SMLA_OK;
}

static smla_status_t check_row_width(int32_t D) {
  if (D < 16 || D > 1024 || D % 8)
    return fail(SMLA_ERR_UNSUPPORTED, "D=%d must be a multiple of 8 in [16, 1024]", D);
  return SMLA_OK;
}

static smla_status_t check_cache(const void* pool, int32_t pool_dtype, int64_t phys_rows, const float* scales,
                                 int32_t sbs, int32_t D, bool any) {
  const smla_status_t st = check_row_width(D);
  if (st != SMLA_OK) return st;
  if (pool_dtype != SMLA_BF16 && pool_dtype != SMLA_E4M3)
    return fail(SMLA_ERR_INVALID_ARG, "pool_dtype=%d must be bf16 or e4m3", pool_dtype);
  if (!(sbs == 0 || sbs == 32 || sbs >= D))
    return fail(SMLA_ERR_UNSUPPORTED, "scale_block_size=%d: supported 0, 32 or >= D", sbs);
  if (pool_dtype == SMLA_BF16 && sbs != 0)
    return fail(SMLA_ERR_INVALID_ARG, "a bf16 cache takes scale_block_size 0");
  if (sbs == 32 && D % 32) return fail(SMLA_ERR_UNSUPPORTED, "block scales need D=%d to be a multiple of 32", D);
  if (sbs != 0 && !scales) return fail(SMLA_ERR_INVALID_ARG, "scales is NULL with scale_block_size != 0");
  if (!any) return SMLA_OK;
  if (!pool) return fail(SMLA_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(pool) || (scales && !aligned4(scales)))
    return fail(SMLA_ERR_INVALID_ARG, "pool must be 16-byte aligned; scales 4-byte aligned");
  if (phys_rows < 1 || phys_rows >= (int64_t(1) << 31))
    return fail(SMLA_ERR_INVALID_ARG, "phys_rows=%lld out of range", static_cast<long long>(phys_rows));
  return SMLA_OK;
}

static bool stride8(int64_t s) { return (s & 7) == 0; }

// What both appends check of a row and its way into the cache.
static smla_status_t check_append(const uint16_t* x, int64_t x_stride, const smla_seqs_t& seqs, int32_t D,
                                  const uint16_t* norm_weight, int32_t norm_dim, float norm_eps, const smla_rope_t& rope,
                                  const uint16_t* rows_out, int64_t rows_stride) {
  const smla_status_t st = check_rope(rope, D);
  if (st != SMLA_OK) return st;
  if (norm_weight) {
    if (norm_dim < 8 || norm_dim > D || norm_dim % 8)
      return fail(SMLA_ERR_UNSUPPORTED, "norm_dim=%d must be a multiple of 8 in [8, D]", norm_dim);
    if (!(norm_eps >= 0.f) || !std::isfinite(norm_eps))
      return fail(SMLA_ERR_INVALID_ARG, "norm_eps must be finite and >= 0");
    if (!aligned16(norm_weight)) return fail(SMLA_ERR_INVALID_ARG, "norm_weight must be 16-byte aligned");
  }
  if (x_stride < D || !stride8(x_stride) || (rows_out && (rows_stride < D || !stride8(rows_stride))))
    return fail(SMLA_ERR_INVALID_ARG, "x_stride and rows_stride must be multiples of 8, >= D");
  if (seqs.T == 0) return SMLA_OK;
  if (!x) return fail(SMLA_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(x) || (rows_out && !aligned16(rows_out)))
    return fail(SMLA_ERR_INVALID_ARG, "x and rows_out must be 16-byte aligned");
  if (rows_out == x) return fail(SMLA_ERR_INVALID_ARG, "rows_out must not be x");
  return SMLA_OK;
}

}  // namespace smla

using namespace smla;

extern "C" {

smla_status_t smla_rope_frequencies(int32_t dim, double base, int32_t scaling, double factor, int32_t original_len,
                                    double beta_fast, double beta_slow, double* inv_freq, float* amplitude) {
  clear_last_error();
  if (dim < 2 || dim > 1024 || dim % 2) return fail(SMLA_ERR_INVALID_ARG, "dim=%d must be even, in [2, 1024]", dim);
  if (!(base > 1.0) || !std::isfinite(base)) return fail(SMLA_ERR_INVALID_ARG, "base must be finite and > 1");
  if (scaling != SMLA_ROPE_PLAIN && scaling != SMLA_ROPE_LINEAR && scaling != SMLA_ROPE_YARN)
    return fail(SMLA_ERR_INVALID_ARG, "scaling=%d", scaling);
  if (!inv_freq || !amplitude) return fail(SMLA_ERR_INVALID_ARG, "null pointer");
  if (scaling != SMLA_ROPE_PLAIN && (!(factor >= 1.0) || !std::isfinite(factor)))
    return fail(SMLA_ERR_INVALID_ARG, "factor must be finite and >= 1");
  double low = 0, high = 0;
  if (scaling == SMLA_ROPE_YARN) {
    if (original_len < 1) return fail(SMLA_ERR_INVALID_ARG, "original_len=%d must be >= 1", original_len);
    if (!(beta_slow > 0.0) || !(beta_fast > beta_slow) || !std::isfinite(beta_fast))
      return fail(SMLA_ERR_INVALID_ARG, "beta_fast > beta_slow > 0 is required");
    // pair i makes original_len * base^(-2i/dim) / (2 pi) turns over the
    // original length; solved for the i that makes `turns`
    const auto pair_at = [&](double turns) {
      return dim * std::log(original_len / (turns * 6.283185307179586)) / (2.0 * std::log(base));
    };
    low = std::fmax(std::floor(pair_at(beta_fast)), 0.0);
    high = std::fmin(std::ceil(pair_at(beta_slow)), dim - 1.0);
  }
  for (int i = 0; i < dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / dim);
    double ramp = 0.0;  // share of the interpolated frequency
    if (scaling == SMLA_ROPE_LINEAR) ramp = 1.0;
    if (scaling == SMLA_ROPE_YARN) ramp = std::fmin(1.0, std::fmax(0.0, (i - low) / std::fmax(high - low, 1e-3)));
    inv_freq[i] = scaling == SMLA_ROPE_PLAIN ? f : f / factor * ramp + f * (1.0 - ramp);
  }
  *amplitude = scaling == SMLA_ROPE_YARN ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return SMLA_OK;
}

smla_status_t smla_rope(const void* x, int32_t x_dtype, int64_t x_token_stride, int64_t x_head_stride,
                        smla_seqs_t seqs, int32_t H, int32_t D, smla_rope_t rope, void* out, int32_t out_dtype,
                        int64_t out_token_stride, int64_t out_head_stride, cudaStream_t stream) {
  clear_last_error();
  smla_status_t st = check_seqs(seqs);
  if (st != SMLA_OK) return st;
  st = check_row_width(D);
  if (st != SMLA_OK) return st;
  if (H < 1 || H > 65535) return fail(SMLA_ERR_UNSUPPORTED, "H=%d must be in [1, 65535]", H);
  if (x_dtype != SMLA_BF16 && x_dtype != SMLA_F32) return fail(SMLA_ERR_INVALID_ARG, "x_dtype=%d", x_dtype);
  if (out_dtype != SMLA_BF16 && out_dtype != SMLA_F32 && out_dtype != SMLA_E4M3)
    return fail(SMLA_ERR_INVALID_ARG, "out_dtype=%d", out_dtype);
  st = check_rope(rope, D);
  if (st != SMLA_OK) return st;
  if (!stride8(x_token_stride) || !stride8(x_head_stride) || !stride8(out_token_stride) || !stride8(out_head_stride))
    return fail(SMLA_ERR_INVALID_ARG, "strides must be multiples of 8 elements");
  if (out_token_stride == 0 || out_head_stride == 0)
    return fail(SMLA_ERR_INVALID_ARG, "out's strides must not be 0: its rows may not share memory");
  if (seqs.T == 0) return SMLA_OK;
  if (!x || !out) return fail(SMLA_ERR_INVALID_ARG, "null pointer");
  const uintptr_t out_mask = out_dtype == SMLA_E4M3 ? 7u : 15u;
  if (!aligned16(x) || (reinterpret_cast<uintptr_t>(out) & out_mask))
    return fail(SMLA_ERR_INVALID_ARG, "x and out must be 16-byte aligned (e4m3 out: 8)");
  if (x == out && (x_dtype != out_dtype || x_token_stride != out_token_stride || x_head_stride != out_head_stride))
    return fail(SMLA_ERR_INVALID_ARG, "in place, out must have x's type and strides");
  unsigned* err = nullptr;
  st = device_err_ptr(&err);
  if (st != SMLA_OK) return st;
  const RopeArgs a{x, x_dtype, x_token_stride, x_head_stride, H, D, rope, out, out_dtype, out_token_stride,
                   out_head_stride};
  return launch_rope(a, seqs, err, stream);
}

smla_status_t smla_cache_append(const uint16_t* x, int64_t x_stride, smla_seqs_t seqs, int32_t D,
                                const uint16_t* norm_weight, int32_t norm_dim, float norm_eps, smla_rope_t rope,
                                void* pool, int32_t pool_dtype, int64_t phys_rows, float* scales,
                                int32_t scale_block_size, uint16_t* rows_out, int64_t rows_stride,
                                cudaStream_t stream) {
  clear_last_error();
  smla_status_t st = check_seqs(seqs);
  if (st != SMLA_OK) return st;
  st = check_cache(pool, pool_dtype, phys_rows, scales, scale_block_size, D, seqs.T > 0);
  if (st != SMLA_OK) return st;
  st = check_append(x, x_stride, seqs, D, norm_weight, norm_dim, norm_eps, rope, rows_out, rows_stride);
  if (st != SMLA_OK || seqs.T == 0) return st;
  unsigned* err = nullptr;
  st = device_err_ptr(&err);
  if (st != SMLA_OK) return st;
  const CacheArgs a{x,         x_stride, D,    norm_weight, norm_dim, norm_eps, rope, pool, pool_dtype,
                    phys_rows, scales,   scale_block_size,  rows_out, rows_stride};
  return launch_cache_append(a, seqs, err, stream);
}

smla_status_t smla_cache_gather(const void* pool, int32_t pool_dtype, int64_t phys_rows, const float* scales,
                                int32_t scale_block_size, smla_seqs_t seqs, int32_t D, uint16_t* rows,
                                int64_t rows_stride, cudaStream_t stream) {
  clear_last_error();
  smla_status_t st = check_seqs(seqs);
  if (st != SMLA_OK) return st;
  st = check_cache(pool, pool_dtype, phys_rows, scales, scale_block_size, D, seqs.T > 0);
  if (st != SMLA_OK) return st;
  if (rows_stride < D || !stride8(rows_stride))
    return fail(SMLA_ERR_INVALID_ARG, "rows_stride must be a multiple of 8, >= D");
  if (seqs.T == 0) return SMLA_OK;
  if (!rows) return fail(SMLA_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(rows)) return fail(SMLA_ERR_INVALID_ARG, "rows must be 16-byte aligned");
  unsigned* err = nullptr;
  st = device_err_ptr(&err);
  if (st != SMLA_OK) return st;
  CacheArgs a{};
  a.D = D;
  a.pool = const_cast<void*>(pool);
  a.pool_dtype = pool_dtype;
  a.phys_rows = phys_rows;
  a.scales = const_cast<float*>(scales);
  a.sbs = scale_block_size;
  a.rows = rows;
  a.rows_stride = rows_stride;
  return launch_cache_gather(a, seqs, err, stream);
}

smla_status_t smla_cache_append_fp4(const uint16_t* x, int64_t x_stride, smla_seqs_t seqs, const uint16_t* norm_weight,
                                    int32_t norm_dim, float norm_eps, smla_rope_t rope, uint8_t* pool,
                                    int64_t phys_rows, uint16_t* rows_out, int64_t rows_stride, cudaStream_t stream) {
  clear_last_error();
  constexpr int32_t D = 576;
  smla_status_t st = check_seqs(seqs);
  if (st != SMLA_OK) return st;
  st = check_cache(pool, SMLA_E4M3, phys_rows, nullptr, 0, D, seqs.T > 0);
  if (st != SMLA_OK) return st;
  st = check_append(x, x_stride, seqs, D, norm_weight, norm_dim, norm_eps, rope, rows_out, rows_stride);
  if (st != SMLA_OK || seqs.T == 0) return st;
  unsigned* err = nullptr;
  st = device_err_ptr(&err);
  if (st != SMLA_OK) return st;
  CacheArgs a{x, x_stride, D, norm_weight, norm_dim, norm_eps, rope, pool, SMLA_E4M3, phys_rows, nullptr, 0, rows_out, rows_stride};
  a.fp4 = true;
  return launch_cache_append(a, seqs, err, stream);
}

smla_status_t smla_cache_gather_fp4(const uint8_t* pool, int64_t phys_rows, smla_seqs_t seqs, void* rows,
                                    int32_t rows_dtype, int64_t rows_stride, float* row_scales, cudaStream_t stream) {
  clear_last_error();
  constexpr int32_t D = 576;
  smla_status_t st = check_seqs(seqs);
  if (st != SMLA_OK) return st;
  if (rows_dtype != SMLA_BF16 && rows_dtype != SMLA_E4M3)
    return fail(SMLA_ERR_INVALID_ARG, "rows_dtype=%d must be bf16 or e4m3", rows_dtype);
  st = check_cache(pool, SMLA_E4M3, phys_rows, nullptr, 0, D, seqs.T > 0);
  if (st != SMLA_OK) return st;
  const bool e4m3 = rows_dtype == SMLA_E4M3;
  if (rows_stride < D || rows_stride % (e4m3 ? 16 : 8))
    return fail(SMLA_ERR_INVALID_ARG, "rows_stride must be a multiple of 8 (e4m3: 16), >= 576");
  if (seqs.T == 0) return SMLA_OK;
  if (!rows || e4m3 != (row_scales != nullptr))
    return fail(SMLA_ERR_INVALID_ARG, "rows must be non-null; row_scales non-null for e4m3 rows, and for them alone");
  if (!aligned16(rows) || !aligned4(row_scales))
    return fail(SMLA_ERR_INVALID_ARG, "rows must be 16-byte aligned; row_scales 4-byte aligned");
  unsigned* err = nullptr;
  st = device_err_ptr(&err);
  if (st != SMLA_OK) return st;
  CacheArgs a{};
  a.D = D;
  a.pool = const_cast<uint8_t*>(pool);
  a.phys_rows = phys_rows;
  a.rows = rows;
  a.rows_stride = rows_stride;
  a.fp4 = true;
  a.row_scales = row_scales;
  return launch_cache_gather(a, seqs, err, stream);
}

smla_status_t smla_quantize_blocks(const uint16_t* x, int64_t x_stride, int32_t M, int32_t K, const uint16_t* norm_weight,
                                   float norm_eps, uint8_t* out, float* scales, cudaStream_t stream) {
  clear_last_error();
  if (M < 0) return fail(SMLA_ERR_INVALID_ARG, "M=%d must be >= 0", M);
  if (K < 16 || K > (1 << 20) || K % 16)
    return fail(SMLA_ERR_UNSUPPORTED, "K=%d must be a multiple of 16 in [16, 2^20]", K);
  if (norm_weight) {
    if (K > 16384) return fail(SMLA_ERR_UNSUPPORTED, "K=%d: at most 16384 with a norm", K);
    if (!(norm_eps >= 0.f) || !std::isfinite(norm_eps))
      return fail(SMLA_ERR_INVALID_ARG, "norm_eps must be finite and >= 0");
    if (!aligned16(norm_weight)) return fail(SMLA_ERR_INVALID_ARG, "norm_weight must be 16-byte aligned");
  }
  if (x_stride < 0 || !stride8(x_stride)) return fail(SMLA_ERR_INVALID_ARG, "x_stride must be a multiple of 8, >= 0");
  if (M == 0) return SMLA_OK;
  if (!x || !out || !scales) return fail(SMLA_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(x) || !aligned16(out) || !aligned4(scales))
    return fail(SMLA_ERR_INVALID_ARG, "x and out must be 16-byte aligned; scales 4-byte aligned");
  if (static_cast<int64_t>(M) * ((K + 255) / 256) >= (int64_t(1) << 31))
    return fail(SMLA_ERR_UNSUPPORTED, "M=%d rows of K=%d columns are too much for one call", M, K);
  const QuantizeArgs a{x, x_stride, M, K, norm_weight, norm_eps, out, scales};
  return launch_quantize(a, stream);
}

smla_status_t smla_block_matmul(const uint8_t* a, int64_t a_group_stride, int64_t a_row_stride, const float* a_scales,
                                int64_t as_group_stride, int64_t as_row_stride, const uint8_t* b, const float* b_scales,
                                int32_t G, int32_t M, int32_t N, int32_t K, void* out, int32_t out_dtype,
                                int64_t out_group_stride, int64_t out_row_stride, cudaStream_t stream) {
  clear_last_error();
  if (G < 0 || M < 0 || N < 0) return fail(SMLA_ERR_INVALID_ARG, "G=%d M=%d N=%d must be >= 0", G, M, N);
  if (K < 16 || K > (1 << 20) || K % 16)
    return fail(SMLA_ERR_UNSUPPORTED, "K=%d must be a multiple of 16 in [16, 2^20]", K);
  if (N % 8) return fail(SMLA_ERR_UNSUPPORTED, "N=%d must be a multiple of 8", N);
  constexpr int32_t kMost = 1 << 30;
  if (M > kMost || N > kMost / 4 || G > kMost)
    return fail(SMLA_ERR_UNSUPPORTED, "G and M must be at most 2^30, N at most 2^28");
  // (a dimension of one element has no stride to speak of)
  if (M == 1) {
    a_row_stride = K;
    as_row_stride = 0;
    out_row_stride = N;
  }
  if (G == 1) {
    a_group_stride = K;
    as_group_stride = 0;
    out_group_stride = N;
  }
  if (out_dtype != SMLA_BF16 && out_dtype != SMLA_F32)
    return fail(SMLA_ERR_INVALID_ARG, "out_dtype=%d must be bf16 or f32", out_dtype);
  if (G == 0 || M == 0 || N == 0) return SMLA_OK;  // (nor have empty tensors)
  const auto wide_enough = [](int64_t n, int64_t s, int64_t width) { return n <= 1 || s >= width; };
  constexpr int64_t kFar = int64_t(1) << 38;
  if (!wide_enough(M, a_row_stride, K) || !wide_enough(G, a_group_stride, K) || a_row_stride % 16 || a_group_stride % 16 ||
      a_row_stride >= kFar || a_group_stride >= kFar)
    return fail(SMLA_ERR_INVALID_ARG, "a's strides must be multiples of 16 below 2^38, at least K");
  if (as_group_stride < 0 || as_row_stride < 0) return fail(SMLA_ERR_INVALID_ARG, "a_scales' strides must be >= 0");
  if (!wide_enough(M, out_row_stride, N) || !wide_enough(G, out_group_stride, N) || !stride8(out_row_stride) ||
      !stride8(out_group_stride) || out_row_stride >= kFar || out_group_stride >= kFar)
    return fail(SMLA_ERR_INVALID_ARG, "out's strides must be multiples of 8 below 2^38, at least N");
  // rows of different batches share no memory: one of the two strides spans the other's range
  const __int128 rows_span = static_cast<__int128>(M - 1) * out_row_stride + N;
  const __int128 groups_span = static_cast<__int128>(G - 1) * out_group_stride + N;
  if (G > 1 && M > 1 && out_group_stride < rows_span && out_row_stride < groups_span)
    return fail(SMLA_ERR_INVALID_ARG, "out's rows must not share memory");
  if (!a || !a_scales || !b || !b_scales || !out) return fail(SMLA_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(a) || !aligned16(b) || !aligned16(out) || !aligned4(a_scales) || !aligned4(b_scales))
    return fail(SMLA_ERR_INVALID_ARG, "a, b and out must be 16-byte aligned; a_scales and b_scales 4-byte aligned");
  if (static_cast<__int128>(N) * K >= kFar)
    return fail(SMLA_ERR_UNSUPPORTED, "N=%d K=%d: b's matrices must be smaller than 2^38 bytes", N, K);
  if (static_cast<__int128>(G) * ((M + 15) / 16) * ((N + 127) / 128) >= (1 << 28))
    return fail(SMLA_ERR_UNSUPPORTED, "G=%d M=%d N=%d are too much for one call", G, M, N);
  unsigned* err = nullptr;
  const smla_status_t st = device_err_ptr(&err);
  if (st != SMLA_OK) return st;
  const MatmulArgs args{a, a_group_stride, a_row_stride, a_scales, as_group_stride, as_row_stride, b, b_scales, G, M, N, K,
                        out, out_dtype, out_group_stride, out_row_stride};
  return launch_block_matmul(args, err, stream);
}

size_t smla_expanded_prefill_workspace_size(int32_t T, int32_t S, int32_t B, int32_t H) {
  if (T <= 0 || S <= 0 || B <= 0 || H <= 0) return 0;
  return expanded_workspace_bytes(T, H, expanded_splits(T, S, B, H));
}

smla_status_t smla_expanded_prefill(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride,
                                    const uint16_t* k_nope, int64_t k_token_stride, int64_t k_head_stride,
                                    const uint16_t* k_rope, int64_t k_rope_stride, const uint16_t* v,
                                    int64_t v_token_stride, int64_t v_head_stride, const int32_t* cu_q,
                                    const int32_t* cu_kv, int32_t B, int32_t T, int32_t S, int32_t H,
                                    float softmax_scale, const float* attn_sink, uint16_t* out, float* lse,
                                    void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  return smla_expanded_prefill_terms(q, q_token_stride, q_head_stride, k_nope, k_token_stride, k_head_stride, k_rope,
                                     k_rope_stride, v, v_token_stride, v_head_stride, cu_q, cu_kv, B, T, S, H,
                                     softmax_scale, 0, attn_sink, out, lse, workspace, workspace_bytes, stream);
}

smla_status_t smla_expanded_prefill_terms(const uint16_t* q, int64_t q_token_stride, int64_t q_head_stride,
                                          const uint16_t* k_nope, int64_t k_token_stride, int64_t k_head_stride,
                                          const uint16_t* k_rope, int64_t k_rope_stride, const uint16_t* v,
                                          int64_t v_token_stride, int64_t v_head_stride, const int32_t* cu_q,
                                          const int32_t* cu_kv, int32_t B, int32_t T, int32_t S, int32_t H,
                                          float softmax_scale, int32_t p_terms, const float* attn_sink, uint16_t* out,
                                          float* lse, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  clear_last_error();
  if (p_terms < 0 || p_terms > 2) return fail(SMLA_ERR_INVALID_ARG, "p_terms=%d must be 0, 1 or 2", p_terms);
  if (T < 0 || S < 0 || B < 0) return fail(SMLA_ERR_INVALID_ARG, "T=%d S=%d B=%d must be >= 0", T, S, B);
  if (H < 1 || H > 65535) return fail(SMLA_ERR_UNSUPPORTED, "H=%d must be in [1, 65535]", H);
  if (!(softmax_scale > 0.f) || softmax_scale < 1.0e-30f || softmax_scale > 1.0e30f)
    return fail(SMLA_ERR_INVALID_ARG, "softmax_scale must be in [1e-30, 1e30]");
  const auto stride_ok = [](int64_t s, int64_t width) { return s >= width && (s & 7) == 0 && s < (int64_t(1) << 38); };
  if (!stride_ok(q_token_stride, 192) || !stride_ok(q_head_stride, 192) || !stride_ok(k_token_stride, 128) ||
      !stride_ok(k_head_stride, 128) || !stride_ok(k_rope_stride, 64) || !stride_ok(v_token_stride, 128) ||
      !stride_ok(v_head_stride, 128))
    return fail(SMLA_ERR_INVALID_ARG, "strides must be multiples of 8 elements, at least the row's width");
  if (T == 0) return SMLA_OK;
  if (B < 1) return fail(SMLA_ERR_INVALID_ARG, "B must be >= 1 when T > 0");
  if (!q || !cu_q || !cu_kv || !out || (S > 0 && (!k_nope || !k_rope || !v)))
    return fail(SMLA_ERR_INVALID_ARG, "null pointer");
  if (!aligned16(q) || !aligned16(k_nope) || !aligned16(k_rope) || !aligned16(v) || !aligned16(out) ||
      !aligned4(cu_q) || !aligned4(cu_kv) || !aligned4(attn_sink) || !aligned4(lse))
    return fail(SMLA_ERR_INVALID_ARG,
                "q, k_nope, k_rope, v, out must be 16-byte aligned; cu_q, cu_kv, attn_sink, lse 4-byte aligned");
  if (static_cast<int64_t>(T) * H >= (int64_t(1) << 31)) return fail(SMLA_ERR_UNSUPPORTED, "T*H too large");
  const int nsplit = expanded_splits(T, S, B, H);
  const size_t need = expanded_workspace_bytes(T, H, nsplit);
  if (workspace_bytes < need || (need && !workspace))
    return fail(SMLA_ERR_INVALID_ARG, "workspace: %zu bytes given, %zu needed", workspace_bytes, need);
  if (workspace && !aligned16(workspace)) return fail(SMLA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  unsigned* err = nullptr;
  const smla_status_t st = device_err_ptr(&err);
  if (st != SMLA_OK) return st;
  const ExpandedArgs a{q,    q_token_stride, q_head_stride,  k_nope,        k_token_stride, k_head_stride, k_rope,
                       k_rope_stride,        v,              v_token_stride, v_head_stride, cu_q,          cu_kv,
                       B,    T,              S,              H,             softmax_scale,  attn_sink,     out,
                       lse,  nsplit,         workspace,     p_terms};
  return launch_expanded(a, err, stream);
}

size_t smla_dense_decode_workspace_size(int32_t T, int32_t H, int32_t max_kv_len) {
  if (T <= 0 || H <= 0 || max_kv_len <= 0) return 0;
  return dense_decode_workspace_bytes(T, H, max_kv_len);
}

static smla_status_t dense_decode(const void* q, int32_t q_dtype, const void* latent_pool, int32_t pool_dtype,
                                  int64_t phys_rows, const float* scales, int32_t scale_block_size, bool fp4,
                                  smla_seqs_t seqs, int32_t max_kv_len, int32_t H, int32_t v_depth, float softmax_scale,
                                  const float* attn_sink, uint16_t* out, void* workspace, size_t workspace_bytes,
                                  cudaStream_t stream) {
  smla_status_t st = check_seqs(seqs);
  if (st != SMLA_OK) return st;
  if (pool_dtype != SMLA_BF16 && pool_dtype != SMLA_E4M3)
    return fail(SMLA_ERR_INVALID_ARG, "pool_dtype=%d must be bf16 or e4m3", pool_dtype);
  if (pool_dtype == SMLA_BF16 && (q_dtype != SMLA_BF16 || scale_block_size != 0))
    return fail(SMLA_ERR_UNSUPPORTED, "a bf16 cache takes bf16 q and scale_block_size 0");
  if (max_kv_len < 1) return fail(SMLA_ERR_INVALID_ARG, "max_kv_len=%d must be >= 1", max_kv_len);
  st = check_attn(q, q_dtype, latent_pool, phys_rows, scales, scale_block_size, false, nullptr, 0, nullptr, seqs.T, H,
                  v_depth, softmax_scale, attn_sink, out);
  if (st != SMLA_OK) return st;
  const int T = seqs.T;
  const size_t need = smla_dense_decode_workspace_size(T, H, max_kv_len);
  if (workspace_bytes < need || (need && !workspace))
    return fail(SMLA_ERR_INVALID_ARG, "workspace: %zu bytes given, %zu needed", workspace_bytes, need);
  if (workspace && !aligned16(workspace)) return fail(SMLA_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
  if (T == 0) return SMLA_OK;
  unsigned* err = nullptr;
  st = device_err_ptr(&err);
  if (st != SMLA_OK) return st;
  const DenseDecodeArgs d{q,    q_dtype, latent_pool, phys_rows,     scale_block_size == 0 ? nullptr : scales,
                          &seqs, T,       H,           max_kv_len,    softmax_scale,
                          attn_sink, out, workspace, fp4};
  // scales by the row (or none) leave the bytes as MMA operands; the others
  // take 16-bit ones
  const bool wide = pool_dtype == SMLA_BF16 || scale_block_size == 32;
  return wide ? launch_dense_decode_wide(d, err, stream) : launch_dense_decode(d, err, stream);
}

smla_status_t smla_dense_decode(const void* q, int32_t q_dtype, const void* latent_pool, int32_t pool_dtype,
                                int64_t phys_rows, const float* scales, int32_t scale_block_size, smla_seqs_t seqs,
                                int32_t max_kv_len, int32_t H, int32_t v_depth, float softmax_scale,
                                const float* attn_sink, uint16_t* out, void* workspace, size_t workspace_bytes,
                                cudaStream_t stream) {
  clear_last_error();
  return dense_decode(q, q_dtype, latent_pool, pool_dtype, phys_rows, scales, scale_block_size, false, seqs, max_kv_len, H,
                      v_depth, softmax_scale, attn_sink, out, workspace, workspace_bytes, stream);
}

smla_status_t smla_dense_decode_fp4(const void* q, int32_t q_dtype, const uint8_t* latent_pool, int64_t phys_rows,
                                    smla_seqs_t seqs, int32_t max_kv_len, int32_t H, int32_t v_depth,
                                    float softmax_scale, const float* attn_sink, uint16_t* out, void* workspace,
                                    size_t workspace_bytes, cudaStream_t stream) {
  clear_last_error();
  return dense_decode(q, q_dtype, latent_pool, SMLA_E4M3, phys_rows, nullptr, 0, true, seqs, max_kv_len, H, v_depth,
                      softmax_scale, attn_sink, out, workspace, workspace_bytes, stream);
}

}  // extern "C"
