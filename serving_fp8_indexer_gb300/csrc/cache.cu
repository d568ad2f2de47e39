// The paged caches' write and read side.
//
// cache_append: one warp per new token.  The row x[t] [D] is optionally
// RMS-normalised over its first norm_dim columns (times a weight), its rotary
// part turned by the token's position, quantised in the cache's scale mode
// and stored at the token's physical row; optionally the finished row is kept
// in bf16 too.  Everything stays in 32 bits from the load to the one rounding
// of the store, so a row is read once and written once and nothing is
// rounded in between (the unfused chain rounds to bf16 after the norm and
// again after the rotation).
//
// cache_gather: the inverse, token t's cached row dequantised to bf16.
//
// A few rows (a decode step) cost a launch and the chain cu_q -> page -> row:
// 16 rows of 576 are written in 3.5 us, 257 read in 2.4.  For many rows the
// append takes 2.5 times its HBM time (12 117 rows of 576 with rows_out: block
// scales 13.8 us against 5.3, row scales 12.6, unit 10.7, bf16 12.0): 876 warp
// instructions a row in block mode keep the issue slots 65 % busy, and half the
// warps that fit wait for the row's loads and shuffles beside it.  The gather is
// bound by HBM (8 sequences, 49 K rows: 16.8 us,
// 5.0 TB/s).  Rows of a 4-bit cache are written as fast as block-scaled ones (13.4 K rows
// 12 us) and read in 13.3 us in bf16 (5.6 TB/s).  The angles come from integer phases: in float64 they were the
// append's bound (27 us).
#include <algorithm>
#include <type_traits>

#include "quantize.cuh"
#include "rope.cuh"

namespace smla {
namespace ca {

constexpr int kWarps = 4;

struct AppendParams {
  const __nv_bfloat16* x;
  int64_t x_stride;
  SeqsDev seqs;
  int T, chunks;
  const __nv_bfloat16* norm_weight;
  int norm_chunks;
  float norm_eps;
  int c0, c1, half;  // rotated chunks, layout
  const double* inv_freq;
  float amplitude;
  void* pool;
  int64_t phys_rows;
  float* scales;
  __nv_bfloat16* rows_out;
  int64_t rows_stride;
  unsigned* err;
};

enum Mode { kBf16 = 0, kUnit = 1, kRow = 2, kBlock = 3, kFp4 = 4 };

// kSlots: 8-element chunks a lane holds.  Ten CTAs an SM (48 registers instead
// of 64) hide more of the rows' latency, 13.5 -> 13.0 us; four slots would spill.
template <int MODE, int kSlots>
__global__ void __launch_bounds__(32 * kWarps, kSlots <= 3 ? 10 : 1) append_kernel(const AppendParams p) {
  // the rotary angles' cos and sin, for each warp its token's
  extern __shared__ float2 s_cs[];
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int pairs = (p.c1 - p.c0) * 4;
  float2* cs = s_cs + (threadIdx.x >> 5) * pairs;
  if (t >= p.T) return;
  const __nv_bfloat16* x = p.x + t * p.x_stride;
  // the row's loads go out before the chain of index loads
  uint4 raw[kSlots];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int c = lane + 32 * i;
    raw[i] = c < p.chunks ? *reinterpret_cast<const uint4*>(x + c * 8) : make_uint4(0, 0, 0, 0);
  }
  const int b = warp_seq_of(p.seqs.cu_q, p.seqs.B, t, lane);
  if (b < 0) return;  // behind the last sequence: nothing is written
  const int pos = token_pos(p.seqs, b, t);
  const int64_t row = key_phys_row(p.seqs, b, pos, p.phys_rows, p.err);
  for (int i = lane; i < pairs; i += 32) rope_cos_sin(p.inv_freq[i], pos, p.amplitude, cs[i].x, cs[i].y);
  __syncwarp();
  float v[kSlots][8];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) unpack_bf16x8(raw[i], v[i]);

  float rstd = 1.f;
  if (p.norm_chunks) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
      if (lane + 32 * i < p.norm_chunks)
#pragma unroll
        for (int k = 0; k < 8; ++k) ss = fmaf(v[i][k], v[i][k], ss);
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    rstd = 1.f / sqrtf(ss / static_cast<float>(p.norm_chunks * 8) + p.norm_eps);
  }
  // chunk c of the row, normalised where the norm covers it
  auto normed = [&](int c, float (&a)[8]) {
    if (c < p.norm_chunks) {
      float w[8];
      unpack_bf16x8(*reinterpret_cast<const uint4*>(p.norm_weight + c * 8), w);
#pragma unroll
      for (int k = 0; k < 8; ++k) a[k] = a[k] * rstd * w[k];
    }
  };
  const int hc = (p.c1 - p.c0) >> 1;
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int c = lane + 32 * i;
    if (c >= p.chunks) continue;
    normed(c, v[i]);
    if (c < p.c0 || c >= p.c1) continue;
    if (!p.half) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 r = cs[(c - p.c0) * 4 + k];
        const float a = v[i][2 * k], q = v[i][2 * k + 1];
        v[i][2 * k] = a * r.x - q * r.y;
        v[i][2 * k + 1] = q * r.x + a * r.y;
      }
    } else {
      // the other half's chunk is another lane's, perhaps in another slot:
      // it is read again (from L1) rather than exchanged
      const bool first = c - p.c0 < hc;
      const int pc = first ? c + hc : c - hc;
      float o[8];
      unpack_bf16x8(*reinterpret_cast<const uint4*>(x + pc * 8), o);
      normed(pc, o);
      const int f0 = ((first ? c : pc) - p.c0) * 8;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 r = cs[f0 + k];
        v[i][k] = first ? v[i][k] * r.x - o[k] * r.y : v[i][k] * r.x + o[k] * r.y;
      }
    }
  }
  if (p.rows_out) {
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const int c = lane + 32 * i;
      if (c < p.chunks) *reinterpret_cast<uint4*>(p.rows_out + t * p.rows_stride + c * 8) = pack_bf16x8(v[i]);
    }
  }
  if (row < 0) return;  // reported; the row has no place in the pool
  if (MODE == kBf16) {
    __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.pool) + row * (p.chunks * 8);
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const int c = lane + 32 * i;
      if (c < p.chunks) *reinterpret_cast<uint4*>(dst + c * 8) = pack_bf16x8(v[i]);
    }
    return;
  }
  float scale = 1.f, inv = 1.f;
  if constexpr (MODE == kFp4) {
    // (chunks past the row's 72 hold zeros)
    float top[kSlots], most = 0.f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      top[i] = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        top[i] = fmaxf(top[i], finite_abs(v[i][k]));
        nan |= v[i][k] != v[i][k];
      }
      top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));  // two lanes hold a block
      most = fmaxf(most, top[i]);
    }
#pragma unroll
    for (int o = 16; o > 1; o >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
    scale = scale_of(most, kFp4Top);
    inv = 1.f / scale;
    uint8_t* dst = static_cast<uint8_t*>(p.pool) + row * kFp4Row;
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      const int c = lane + 32 * i;
      const int k = fp4_shift(top[i], most);
      const float unit = __uint_as_float(static_cast<uint32_t>(127 + k - 6) << 23);
      float q[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) q[e] = quotient(v[i][e], scale, inv) * unit;
      const int odd = __shfl_down_sync(0xffffffffu, k, 2);  // the next block's
      if (c < p.chunks) {
        *reinterpret_cast<uint32_t*>(dst + c * 4) = pack_e2m1x8(q);
        if ((c & 3) == 0) dst[kFp4Shifts + (c >> 2)] = static_cast<uint8_t>(k | odd << 4);
      }
    }
    if (__any_sync(0xffffffffu, nan)) scale = NAN;  // e2m1 has none: the whole row's values are
    if (lane == 0) {
      *reinterpret_cast<uint16_t*>(dst + kFp4Scale - 2) = 0;
      *reinterpret_cast<float*>(dst + kFp4Scale) = scale;
      *reinterpret_cast<uint32_t*>(dst + kFp4Scale + 4) = 0;
      *reinterpret_cast<uint32_t*>(dst + kFp4Scale + 8) = 0;
    }
    return;
  }
  if (MODE == kRow) {
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < kSlots; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) amax = fmaxf(amax, finite_abs(v[i][k]));  // 0 in lanes past the row
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    scale = scale_of(amax);
    inv = 1.f / scale;
    if (lane == 0) p.scales[row] = scale;
  }
  uint8_t* dst = static_cast<uint8_t*>(p.pool) + row * (p.chunks * 8);
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    const int c = lane + 32 * i;
    if (MODE == kBlock) {
      // four neighbouring lanes hold a 32-column block
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < 8; ++k) amax = fmaxf(amax, finite_abs(v[i][k]));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      scale = scale_of(amax);
      inv = 1.f / scale;
      if (c < p.chunks && (c & 3) == 0) p.scales[row * (p.chunks >> 2) + (c >> 2)] = scale;
    }
    if (c < p.chunks) {
      float q[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) q[k] = MODE == kUnit ? v[i][k] : quotient(v[i][k], scale, inv);
      *reinterpret_cast<uint2*>(dst + c * 8) = pack_e4m3x8(q);
    }
  }
}

// ---------------------------------------------------------------- gather
constexpr int kGatherThreads = 256;

struct GatherParams {
  const void* pool;
  int64_t phys_rows;
  const float* scales;
  SeqsDev seqs;
  int T, chunks;
  uint32_t magic;  // ceil(2^32 / chunks)
  int rows_per_cta;
  __nv_bfloat16* rows;  // (4-bit cache: or e4m3 bytes)
  int64_t rows_stride;
  float* row_scales;  // of e4m3 rows
  unsigned* err;
};

constexpr int kMaxGatherRows = 32;

// Physical rows of the nr tokens from t0 on (-1: none), by one warp.
__device__ __forceinline__ void find_rows(const GatherParams& p, int t0, int nr, int64_t* s_row) {
  const int lane = threadIdx.x, t = t0 + lane;
  int b = warp_seq_of(p.seqs.cu_q, p.seqs.B, t0, lane);
  if (lane < nr) {
    if (b < 0) b = p.seqs.cu_q[0] > t0 ? 0 : p.seqs.B;  // before the first sequence, or behind the last
    while (b < p.seqs.B && p.seqs.cu_q[b + 1] <= t) ++b;
    s_row[lane] = b >= p.seqs.B || p.seqs.cu_q[b] > t
                      ? -1
                      : key_phys_row(p.seqs, b, token_pos(p.seqs, b, t), p.phys_rows, p.err);
  }
}

// A CTA takes up to 32 consecutive tokens: a warp finds the first one's
// sequence, then each lane steps to its own token's (few steps, mostly none)
// and reads its page, one chain of reads for all rows.  Then the rows' chunks
// are spread flat over the threads, so that a row width that is no multiple of
// 32 chunks leaves no lane idle; a thread's loads go out before its stores.
template <int MODE>
__global__ void __launch_bounds__(kGatherThreads) gather_kernel(const GatherParams p) {
  __shared__ int64_t s_row[kMaxGatherRows];
  const int t0 = blockIdx.x * p.rows_per_cta;
  const int nr = min(p.rows_per_cta, p.T - t0);
  if (threadIdx.x < 32) find_rows(p, t0, nr, s_row);
  __syncthreads();
  const int n = nr * p.chunks;
  constexpr int kBatch = 5;  // loads of a thread in flight (a full CTA of 576-wide rows has nine)
  for (int i0 = threadIdx.x; i0 < n; i0 += kBatch * kGatherThreads) {
    uint4 raw[kBatch];
    float sc[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kGatherThreads, r = __umulhi(i, p.magic), c = i - r * p.chunks;
      const int64_t row = i < n ? s_row[r] : -1;
      raw[k] = make_uint4(0, 0, 0, 0);
      sc[k] = 1.f;
      if (row < 0) continue;
      const int64_t at = row * (p.chunks * 8) + c * 8;
      if (MODE == kBf16) {
        raw[k] = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.pool) + at));
      } else {
        const uint2 u = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p.pool) + at));
        raw[k].x = u.x;
        raw[k].y = u.y;
        if (MODE != kUnit) sc[k] = MODE == kRow ? p.scales[row] : p.scales[row * (p.chunks >> 2) + (c >> 2)];
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kGatherThreads, r = __umulhi(i, p.magic), c = i - r * p.chunks;
      if (i >= n || s_row[r] < 0) continue;
      uint4 o = raw[k];
      if (MODE != kBf16) {
        float v[8];
        unpack_e4m3x8(make_uint2(raw[k].x, raw[k].y), v);
        if (MODE != kUnit)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] *= sc[k];
        o = pack_bf16x8(v);
      }
      *reinterpret_cast<uint4*>(p.rows + (t0 + r) * p.rows_stride + c * 8) = o;
    }
  }
}

// The same for a 4-bit cache, by blocks of 16 columns: 8 bytes of codes and a
// shift become 16 e4m3 bytes by a table, stored as they are (with the row's
// scale) or times the scale in bf16.
// WIDE: bf16 rows on 32-byte boundaries, whose blocks are one store each (49 K rows:
// 13.3 us, 5.6 TB/s; by two stores 20).
template <bool E4M3, bool WIDE>
__global__ void __launch_bounds__(kGatherThreads) gather_fp4_kernel(const GatherParams p) {
  __shared__ int64_t s_row[kMaxGatherRows];
  __shared__ uint2 s_table[16];
  const int t0 = blockIdx.x * p.rows_per_cta;
  const int nr = min(p.rows_per_cta, p.T - t0);
  if (threadIdx.x < 32) find_rows(p, t0, nr, s_row);
  if (threadIdx.x >= 32 && threadIdx.x < 48) s_table[threadIdx.x - 32] = fp4_table_entry(threadIdx.x - 32);
  __syncthreads();
  const int n = nr * kFp4Blocks;
  constexpr int kBatch = 3;  // (five 13.9 us)
  for (int i0 = threadIdx.x; i0 < n; i0 += kBatch * kGatherThreads) {
    uint2 raw[kBatch];
    float sc[kBatch];
    int sh[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kGatherThreads, r = i / kFp4Blocks, c = i - r * kFp4Blocks;
      const int64_t row = i < n ? s_row[r] : -1;
      raw[k] = make_uint2(0u, 0u);
      sc[k] = 1.f;
      sh[k] = 0;
      if (row < 0) continue;
      const uint8_t* at = static_cast<const uint8_t*>(p.pool) + row * kFp4Row;
      raw[k] = __ldcs(reinterpret_cast<const uint2*>(at + c * 8));
      sh[k] = at[kFp4Shifts + (c >> 1)] >> (4 * (c & 1)) & 15;
      sc[k] = *reinterpret_cast<const float*>(at + kFp4Scale);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kGatherThreads, r = i / kFp4Blocks, c = i - r * kFp4Blocks;
      if (i >= n || s_row[r] < 0) continue;
      const uint2 t = s_table[sh[k]];
      const uint2 a = fp4x8_to_e4m3x8(raw[k].x, t), b = fp4x8_to_e4m3x8(raw[k].y, t);
      if constexpr (E4M3) {
        uint8_t* dst = reinterpret_cast<uint8_t*>(p.rows) + (t0 + r) * p.rows_stride + c * 16;
        *reinterpret_cast<uint4*>(dst) = make_uint4(a.x, a.y, b.x, b.y);
        if (c == 0) p.row_scales[t0 + r] = sc[k];
      } else {
        uint4* dst = reinterpret_cast<uint4*>(p.rows + (t0 + r) * p.rows_stride + c * 16);
        float v[8], w[8];
        unpack_e4m3x8(a, v);
        unpack_e4m3x8(b, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          v[e] *= sc[k];
          w[e] *= sc[k];
        }
        const uint4 lo = pack_bf16x8(v), hi = pack_bf16x8(w);
        if constexpr (WIDE) {
          st_global32(dst, lo, hi);
        } else {
          dst[0] = lo;
          dst[1] = hi;
        }
      }
    }
  }
}

static Mode mode_of(const CacheArgs& a) {
  if (a.fp4) return kFp4;
  if (a.pool_dtype == SMLA_BF16) return kBf16;
  return a.sbs == 0 ? kUnit : a.sbs >= a.D ? kRow : kBlock;
}

}  // namespace ca

smla_status_t launch_cache_append(const CacheArgs& a, const smla_seqs_t& seqs, unsigned* err, cudaStream_t stream) {
  using namespace ca;
  AppendParams p{};
  p.x = static_cast<const __nv_bfloat16*>(a.x);
  p.x_stride = a.x_stride;
  p.seqs = seqs_dev(seqs);
  p.T = seqs.T;
  p.chunks = a.D / 8;
  p.norm_weight = static_cast<const __nv_bfloat16*>(a.norm_weight);
  p.norm_chunks = a.norm_weight ? a.norm_dim / 8 : 0;
  p.norm_eps = a.norm_eps;
  p.c0 = a.rope.offset / 8;
  p.c1 = p.c0 + a.rope.dim / 8;
  p.half = a.rope.layout == SMLA_ROPE_HALF;
  p.inv_freq = a.rope.inv_freq;
  p.amplitude = a.rope.amplitude;
  p.pool = a.pool;
  p.phys_rows = a.phys_rows;
  p.scales = a.scales;
  p.rows_out = static_cast<__nv_bfloat16*>(a.rows);
  p.rows_stride = a.rows_stride;
  p.err = err;
  const unsigned grid = (static_cast<unsigned>(seqs.T) + kWarps - 1) / kWarps;
  const size_t smem = sizeof(float2) * kWarps * (p.c1 - p.c0) * 4;  // at most 16 KB
  const Mode mode = mode_of(a);
  const auto go = [&](auto slots) {
    constexpr int N = decltype(slots)::value;
    switch (mode) {
      case kBf16: append_kernel<kBf16, N><<<grid, 32 * kWarps, smem, stream>>>(p); break;
      case kUnit: append_kernel<kUnit, N><<<grid, 32 * kWarps, smem, stream>>>(p); break;
      case kRow: append_kernel<kRow, N><<<grid, 32 * kWarps, smem, stream>>>(p); break;
      case kBlock: append_kernel<kBlock, N><<<grid, 32 * kWarps, smem, stream>>>(p); break;
      case kFp4:
        if constexpr (N == 3) append_kernel<kFp4, 3><<<grid, 32 * kWarps, smem, stream>>>(p);  // (its rows are 576 wide)
        break;
    }
  };
  switch ((p.chunks + 31) / 32) {
    case 1: go(std::integral_constant<int, 1>{}); break;
    case 2: go(std::integral_constant<int, 2>{}); break;
    case 3: go(std::integral_constant<int, 3>{}); break;
    default: go(std::integral_constant<int, 4>{}); break;
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail_cuda(e, "cache append launch");
  return SMLA_OK;
}

smla_status_t launch_cache_gather(const CacheArgs& a, const smla_seqs_t& seqs, unsigned* err, cudaStream_t stream) {
  using namespace ca;
  GatherParams p{};
  p.pool = a.pool;
  p.phys_rows = a.phys_rows;
  p.scales = a.scales;
  p.seqs = seqs_dev(seqs);
  p.T = seqs.T;
  p.chunks = a.D / 8;
  p.magic = static_cast<uint32_t>(((uint64_t(1) << 32) + p.chunks - 1) / p.chunks);
  // full CTAs once they fill the GPU twice over, else fewer rows on more SMs
  p.rows_per_cta = seqs.T >= 2 * device_sm_count() * kMaxGatherRows ? kMaxGatherRows : 8;
  p.rows = static_cast<__nv_bfloat16*>(a.rows);
  p.rows_stride = a.rows_stride;
  p.row_scales = a.row_scales;
  p.err = err;
  const unsigned grid = (static_cast<unsigned>(seqs.T) + p.rows_per_cta - 1) / p.rows_per_cta;
  switch (mode_of(a)) {
    case kBf16: gather_kernel<kBf16><<<grid, kGatherThreads, 0, stream>>>(p); break;
    case kUnit: gather_kernel<kUnit><<<grid, kGatherThreads, 0, stream>>>(p); break;
    case kRow: gather_kernel<kRow><<<grid, kGatherThreads, 0, stream>>>(p); break;
    case kBlock: gather_kernel<kBlock><<<grid, kGatherThreads, 0, stream>>>(p); break;
    case kFp4:
      if (a.row_scales)
        gather_fp4_kernel<true, false><<<grid, kGatherThreads, 0, stream>>>(p);
      else if (reinterpret_cast<uintptr_t>(a.rows) % 32 == 0 && a.rows_stride % 16 == 0)
        gather_fp4_kernel<false, true><<<grid, kGatherThreads, 0, stream>>>(p);
      else
        gather_fp4_kernel<false, false><<<grid, kGatherThreads, 0, stream>>>(p);
      break;
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail_cuda(e, "cache gather launch");
  return SMLA_OK;
}

}  // namespace smla
