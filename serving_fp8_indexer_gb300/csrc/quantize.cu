// Rows of activations in e4m3 with a scale for each 128 columns, the left
// operand of the block-scaled matrix product; optionally RMS-normalised first,
// all in 32 bits with one rounding at the end.
//
// Bound: HBM (2 bytes read and 1 written an element).  Without the norm the
// blocks are independent: eight lanes hold a block's 128 columns (32 bytes a
// lane), find its largest magnitude with three shuffles and store 16 bytes a lane.
// With it a row is read once, kept in registers as bf16 and summed first.
// Measured: 4096 x 16384 33.4 us (6.1 TB/s, 0.91 of the copy rate; by 8 columns a lane 43.4,
// two loads a lane in flight 35.6), 16 x 2048 with the norm 2.0 us (a launch).
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
  int M, K, chunks, nblk;  // chunks of 16 columns, blocks of 128
  const __nv_bfloat16* w;
  float eps;
  uint8_t* out;
  float* scales;
};

// Chunk c (16 columns) of a row, held by lanes in order: its block's scale and
// its bytes.  All lanes of the warp call; `in`: the chunk exists.
__device__ __forceinline__ void quantize_chunk(const Params& p, int64_t row, int c, bool in, float (&v)[2][8], int lane) {
  float amax = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) amax = max3(amax, finite_abs(v[0][k]), finite_abs(v[1][k]));
#pragma unroll
  for (int o = 4; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const float scale = scale_of(amax), inv = 1.f / scale;
  if (!in) return;
  uint2 q[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[h][k] = quotient(v[h][k], scale, inv);
    q[h] = pack_e4m3x8(v[h]);
  }
  __stcs(reinterpret_cast<uint4*>(p.out + row * p.K + c * 16), make_uint4(q[0].x, q[0].y, q[1].x, q[1].y));
  if ((lane & 7) == 0) p.scales[row * p.nblk + (c >> 3)] = scale;
}
struct Raw {
  uint4 a, b;
};
__device__ __forceinline__ void unpack(const Raw& r, float (&v)[2][8]) {
  unpack_bf16x8(r.a, v[0]);
  unpack_bf16x8(r.b, v[1]);
}

// A warp takes kLoads * 512 columns of a row.
template <int kLoads>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const Params p, int units_per_row, int64_t units) {
  const int lane = threadIdx.x & 31;
  const int64_t u = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  if (u >= units) return;
  const int64_t row = u / units_per_row;
  const int c0 = static_cast<int>(u - row * units_per_row) * (kLoads * 32) + lane;
  const uint4* x = reinterpret_cast<const uint4*>(p.x + row * p.x_stride);
  const uint4 none = make_uint4(0, 0, 0, 0);
  Raw raw[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int c = c0 + 32 * i;
    raw[i] = c < p.chunks ? Raw{__ldcs(x + 2 * c), __ldcs(x + 2 * c + 1)} : Raw{none, none};
  }
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    float v[2][8];
    unpack(raw[i], v);
    quantize_chunk(p, row, c0 + 32 * i, c0 + 32 * i < p.chunks, v, lane);
  }
}

// Rows of a few whole blocks, side by side: a thread's chunks are 256 apart in the
// run of all rows' chunks.
template <int kLoads>
__global__ void __launch_bounds__(kThreads) quantize_flat_kernel(const Params p, uint32_t magic) {
  const int lane = threadIdx.x & 31;
  const int64_t base = static_cast<int64_t>(blockIdx.x) * (kThreads * kLoads), row0 = base / p.chunks;
  const int rem = static_cast<int>(base - row0 * p.chunks);  // (a multiple of 8: blocks stay with their eight lanes)
  const uint4 none = make_uint4(0, 0, 0, 0);
  Raw raw[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int at = rem + threadIdx.x + kThreads * i, r = __umulhi(at, magic), c = at - r * p.chunks;
    const uint4* x = reinterpret_cast<const uint4*>(p.x + (row0 + r) * p.x_stride);
    raw[i] = row0 + r < p.M ? Raw{__ldcs(x + 2 * c), __ldcs(x + 2 * c + 1)} : Raw{none, none};
  }
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int at = rem + threadIdx.x + kThreads * i, r = __umulhi(at, magic), c = at - r * p.chunks;
    float v[2][8];
    unpack(raw[i], v);
    quantize_chunk(p, row0 + r, c, row0 + r < p.M, v, lane);
  }
}

// kRowThreads threads take a row: its chunks stay in registers between the sum
// and the rounding.
template <int kRowThreads, int kLoads>
__global__ void __launch_bounds__(kThreads) quantize_norm_kernel(const Params p) {
  constexpr int kWarps = kRowThreads <= 32 ? 1 : kRowThreads / 32;
  __shared__ float s_sum[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, rt = threadIdx.x % kRowThreads;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / kRowThreads) + threadIdx.x / kRowThreads;
  const bool live = row < p.M;  // (the others keep the barrier and the shuffles)
  const uint4* x = reinterpret_cast<const uint4*>(p.x + (live ? row : 0) * p.x_stride);
  const uint4* weight = reinterpret_cast<const uint4*>(p.w);
  const uint4 none = make_uint4(0, 0, 0, 0);
  Raw raw[kLoads], w0{none, none};
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int c = rt + kRowThreads * i;
    raw[i] = live && c < p.chunks ? Raw{x[2 * c], x[2 * c + 1]} : Raw{none, none};
  }
  if (rt < p.chunks) w0 = Raw{weight[2 * rt], weight[2 * rt + 1]};  // beside the row's, not behind its sum
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    float v[2][8];
    unpack(raw[i], v);
#pragma unroll
    for (int k = 0; k < 8; ++k) ss = fmaf(v[1][k], v[1][k], fmaf(v[0][k], v[0][k], ss));
  }
#pragma unroll
  for (int o = (kRowThreads < 32 ? kRowThreads : 32) / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  if constexpr (kWarps > 1) {
    if (lane == 0) s_sum[warp] = ss;
    __syncthreads();
    ss = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) ss += s_sum[warp / kWarps * kWarps + w];
  }
  const float rstd = 1.f / sqrtf(ss / static_cast<float>(p.K) + p.eps);
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int c = rt + kRowThreads * i;
    const bool in = live && c < p.chunks;
    if (i > 0) w0 = in ? Raw{weight[2 * c], weight[2 * c + 1]} : Raw{none, none};
    float v[2][8], w[2][8];
    unpack(raw[i], v);
    unpack(w0, w);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int k = 0; k < 8; ++k) v[h][k] = v[h][k] * rstd * w[h][k];
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
  p.chunks = a.K / 16;
  p.nblk = (a.K + kBlock - 1) / kBlock;
  p.w = static_cast<const __nv_bfloat16*>(a.norm_weight);
  p.eps = a.norm_eps;
  p.out = a.out;
  p.scales = a.scales;
  const auto grid = [](int64_t n, int64_t per) { return static_cast<unsigned>((n + per - 1) / per); };
  if (p.w) {
    // where rows are many, as few threads a row as hold it in one or two loads (30 000 x
    // 2048 45.0 us; 50.5 in four loads, 70 by a CTA a row); where they are few, a CTA
    if (a.K > 1024 && a.M < 8 * device_sm_count()) {
      if (a.K <= 4096)
        quantize_norm_kernel<256, 1><<<a.M, kThreads, 0, stream>>>(p);
      else
        quantize_norm_kernel<256, 4><<<a.M, kThreads, 0, stream>>>(p);
    } else if (a.K <= 128) {
      quantize_norm_kernel<8, 1><<<grid(a.M, 32), kThreads, 0, stream>>>(p);
    } else if (a.K <= 256) {
      quantize_norm_kernel<16, 1><<<grid(a.M, 16), kThreads, 0, stream>>>(p);
    } else if (a.K <= 512) {
      quantize_norm_kernel<32, 1><<<grid(a.M, 8), kThreads, 0, stream>>>(p);
    } else if (a.K <= 1024) {
      quantize_norm_kernel<32, 2><<<grid(a.M, 8), kThreads, 0, stream>>>(p);
    } else if (a.K <= 2048) {
      quantize_norm_kernel<64, 2><<<grid(a.M, 4), kThreads, 0, stream>>>(p);
    } else if (a.K <= 4096) {
      quantize_norm_kernel<128, 2><<<grid(a.M, 2), kThreads, 0, stream>>>(p);
    } else if (a.K <= 8192) {
      quantize_norm_kernel<256, 2><<<a.M, kThreads, 0, stream>>>(p);
    } else {
      quantize_norm_kernel<256, 4><<<a.M, kThreads, 0, stream>>>(p);
    }
  } else if (a.K <= 512 && a.K % kBlock == 0) {
    const uint32_t magic = static_cast<uint32_t>(((uint64_t(1) << 32) + p.chunks - 1) / p.chunks);
    const int64_t chunks = static_cast<int64_t>(a.M) * p.chunks;
    if (chunks >= (1 << 18))
      quantize_flat_kernel<4><<<grid(chunks, kThreads * 4), kThreads, 0, stream>>>(p, magic);
    else
      quantize_flat_kernel<1><<<grid(chunks, kThreads), kThreads, 0, stream>>>(p, magic);
  } else {
    const auto go = [&](auto kernel, int loads) {
      const int per_row = (p.chunks + 32 * loads - 1) / (32 * loads);
      const int64_t units = static_cast<int64_t>(a.M) * per_row;
      kernel<<<grid(units, kThreads / 32), kThreads, 0, stream>>>(p, per_row, units);
    };
    // four loads a lane, unless their 2048 columns leave half a warp's work or more
    // idle at a row's end (60 000 x 1024 33.5 us in two, 44.0 in four)
    if (a.K < 1024 || static_cast<int64_t>(a.M) * a.K < (1 << 22))
      go(quantize_kernel<1>, 1);
    else if ((a.K - 1) % 2048 < 1024)
      go(quantize_kernel<2>, 2);
    else
      go(quantize_kernel<4>, 4);
  }
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SMLA_OK : fail_cuda(e, "quantize launch");
}

}  // namespace smla
