// Rows of activations in e4m3 with a scale for each 128 columns, the left
// operand of the block-scaled matrix product; optionally RMS-normalised first,
// all in 32 bits with one rounding at the end.
//
// Bound: HBM (2 bytes read and 1 written an element).  Without the norm the
// blocks are independent: sixteen lanes hold a block's 128 columns (16 bytes a
// lane), find its largest magnitude with four shuffles and store 8 bytes a lane.
// With it a row is read once, kept in registers as bf16 and summed first.
#include <algorithm>

#include "quantize.cuh"
#include "rope.cuh"

namespace smla {
namespace qz {

constexpr int kThreads = 256;
constexpr int kBlock = 128;

struct Params {
  const __nv_bfloat16* x;
  int64_t x_stride;
  int M, K, chunks, nblk;  // chunks of 8 columns, blocks of 128
  const __nv_bfloat16* w;
  float eps;
  uint8_t* out;
  float* scales;
};

// Chunk c (8 columns) of a row, held by lanes in order: its block's scale and
// its bytes.  All lanes of the warp call; `in`: the chunk exists.
__device__ __forceinline__ void quantize_chunk(const Params& p, int64_t row, int c, bool in, float (&v)[8], int lane) {
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) amax = fmaxf(amax, finite_abs(v[k]));
#pragma unroll
  for (int o = 8; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float scale = scale_of(amax), inv = 1.f / scale;
  if (!in) return;
  float q[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) q[k] = quotient(v[k], scale, inv);
  *reinterpret_cast<uint2*>(p.out + row * p.K + c * 8) = pack_e4m3x8(q);
  if ((lane & 15) == 0) p.scales[row * p.nblk + (c >> 4)] = scale;
}

// A warp takes kLoads * 256 columns of a row.
template <int kLoads>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const Params p, int units_per_row, int64_t units) {
  const int lane = threadIdx.x & 31;
  const int64_t u = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  if (u >= units) return;
  const int64_t row = u / units_per_row;
  const int c0 = static_cast<int>(u - row * units_per_row) * (kLoads * 32) + lane;
  const __nv_bfloat16* x = p.x + row * p.x_stride;
  uint4 raw[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int c = c0 + 32 * i;
    raw[i] = c < p.chunks ? __ldcs(reinterpret_cast<const uint4*>(x + c * 8)) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    float v[8];
    unpack_bf16x8(raw[i], v);
    quantize_chunk(p, row, c0 + 32 * i, c0 + 32 * i < p.chunks, v, lane);
  }
}

// kRowThreads threads take a row: its chunks stay in registers between the sum
// and the rounding.
template <int kRowThreads, int kLoads>
__global__ void __launch_bounds__(kThreads) quantize_norm_kernel(const Params p) {
  constexpr int kWarps = kRowThreads / 32;
  __shared__ float s_sum[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rt = threadIdx.x % kRowThreads;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / kRowThreads) + threadIdx.x / kRowThreads;
  const bool live = row < p.M;  // (whole warps; the others only keep the barrier)
  const __nv_bfloat16* x = p.x + (live ? row : 0) * p.x_stride;
  uint4 raw[kLoads];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int c = rt + kRowThreads * i;
    raw[i] = live && c < p.chunks ? *reinterpret_cast<const uint4*>(x + c * 8) : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    float v[8];
    unpack_bf16x8(raw[i], v);
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = fmaf(v[k], v[k], ss);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if constexpr (kWarps > 1) {
    if (lane == 0) s_sum[warp] = ss;
    __syncthreads();
    ss = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) ss += s_sum[warp / kWarps * kWarps + w];
  }
  if (!live) return;
  const float rstd = 1.f / sqrtf(ss / static_cast<float>(p.K) + p.eps);
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int c = rt + kRowThreads * i;
    const bool in = c < p.chunks;
    float v[8], w[8];
    unpack_bf16x8(raw[i], v);
    unpack_bf16x8(in ? *reinterpret_cast<const uint4*>(p.w + c * 8) : make_uint4(0, 0, 0, 0), w);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = v[k] * rstd * w[k];
    quantize_chunk(p, row, c, in, v, lane);
  }
}

}  // namespace qz

smla_status_t launch_quantize(const QuantizeArgs& a, cudaStream_t stream) {
  using namespace qz;
  Params p{};
  p.x = static_cast<const __nv_bfloat16*>(a.x);
  p.x_stride = a.x_stride;
  p.M = a.M;
  p.K = a.K;
  p.chunks = a.K / 8;
  p.nblk = (a.K + kBlock - 1) / kBlock;
  p.w = static_cast<const __nv_bfloat16*>(a.norm_weight);
  p.eps = a.norm_eps;
  p.out = a.out;
  p.scales = a.scales;
  if (p.w) {
    if (a.K <= 1024)
      quantize_norm_kernel<32, 4><<<(a.M + 7) / 8, kThreads, 0, stream>>>(p);
    else if (a.K <= 4096)
      quantize_norm_kernel<256, 2><<<a.M, kThreads, 0, stream>>>(p);
    else
      quantize_norm_kernel<256, 8><<<a.M, kThreads, 0, stream>>>(p);
  } else {
    const auto go = [&](auto kernel, int loads) {
      const int per_row = (p.chunks + 32 * loads - 1) / (32 * loads);
      const int64_t units = static_cast<int64_t>(a.M) * per_row;
      kernel<<<static_cast<unsigned>((units + kThreads / 32 - 1) / (kThreads / 32)), kThreads, 0, stream>>>(p, per_row, units);
    };
    if (a.K >= 1024 && static_cast<int64_t>(a.M) * a.K >= (1 << 22))
      go(quantize_kernel<4>, 4);
    else
      go(quantize_kernel<1>, 1);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SMLA_OK : fail_cuda(e, "quantize launch");
}

}  // namespace smla
