// Rotary positions (forward): y = x with `dim` of each head's columns turned
// pairwise by the token's position,
//   (u, v) = a * (p cos - q sin, q cos + p sin),  angle = pos(t) * inv_freq[i],
// (p, q) = columns (2i, 2i+1) of the rotated part (interleaved) or (i,
// i + dim/2) (half), and the other columns copied, converted to the output's
// type.
//
// Bound by HBM: every element is read and written once.  A CTA takes one
// token and a group of its heads, so the token's dim/2 angles are computed
// once per CTA into shared memory and serve all of the group's heads.  The
// group is sized to give the CTA about kChunksPerCta 8-element chunks (nine
// 16-byte loads a thread), and fewer when the batch is too small to fill the
// GPU that way.
#include <algorithm>
#include <cmath>

#include "rope.cuh"

namespace smla {
namespace rp {

constexpr int kThreads = 256;
constexpr int kChunksPerCta = 9 * kThreads;
constexpr int kMaxDim = 1024;

struct Params {
  const void* x;
  void* out;
  int64_t x_ts, x_hs, o_ts, o_hs;  // token and head strides, elements
  SeqsDev seqs;
  int H, chunks;       // heads; 8-element chunks per head
  int heads_per_cta;
  uint32_t magic;      // ceil(2^32 / chunks): i / chunks = umulhi(i, magic) for i < 2^16
  int c0, c1;          // the rotated chunks [c0, c1)
  int half;            // layout
  int in_place;        // the copied columns are there already
  const double* inv_freq;
  float amplitude;
  unsigned* err;
};

template <typename X>
__device__ __forceinline__ void load8(const X* p, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, float (&v)[8]) {
  unpack_bf16x8(*reinterpret_cast<const uint4*>(p), v);
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
template <typename Y>
__device__ __forceinline__ void store8(Y* p, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = pack_bf16x8(v);
}
template <>
__device__ __forceinline__ void store8<float>(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
template <>
__device__ __forceinline__ void store8<uint8_t>(uint8_t* p, const float (&v)[8]) {
  *reinterpret_cast<uint2*>(p) = pack_e4m3x8(v);
}

template <typename X, typename Y>
__global__ void __launch_bounds__(kThreads) rope_kernel(const Params p) {
  __shared__ float2 cs[kMaxDim / 2];
  __shared__ int s_pos;
  const int t = blockIdx.x;
  if (threadIdx.x < 32) {
    const int b = warp_seq_of(p.seqs.cu_q, p.seqs.B, t, threadIdx.x);
    if (threadIdx.x == 0) {
      int pos = b < 0 ? -1 : token_pos(p.seqs, b, t);
      if (b >= 0 && pos < 0) atomicOr(p.err, kErrShape);
      s_pos = pos;
    }
  }
  __syncthreads();
  const int pos = s_pos;
  if (pos < 0) return;  // behind the last sequence: left as it is
  for (int i = threadIdx.x; i < (p.c1 - p.c0) * 4; i += kThreads)
    rope_cos_sin(p.inv_freq[i], pos, p.amplitude, cs[i].x, cs[i].y);
  __syncthreads();
  const int h0 = blockIdx.y * p.heads_per_cta;
  const X* x = static_cast<const X*>(p.x) + t * p.x_ts + h0 * p.x_hs;
  Y* out = static_cast<Y*>(p.out) + t * p.o_ts + h0 * p.o_hs;
  const int n = min(p.heads_per_cta, p.H - h0) * p.chunks;
  const int hc = (p.c1 - p.c0) >> 1;  // chunks in half of the rotated part
#pragma unroll 3
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const int h = __umulhi(i, p.magic);
    const int c = i - h * p.chunks;
    const X* xr = x + h * p.x_hs + c * 8;
    Y* yr = out + h * p.o_hs + c * 8;
    if (c < p.c0 || c >= p.c1) {
      if (!p.in_place) {
        float v[8];
        load8(xr, v);
        store8(yr, v);
      }
    } else if (!p.half) {
      float v[8];
      load8(xr, v);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 r = cs[(c - p.c0) * 4 + k];
        const float a = v[2 * k], b = v[2 * k + 1];
        v[2 * k] = a * r.x - b * r.y;
        v[2 * k + 1] = b * r.x + a * r.y;
      }
      store8(yr, v);
    } else if (c - p.c0 < hc) {
      // both chunks of the pair by one thread, read before they are written
      // (the output may be the input)
      float a[8], b[8];
      load8(xr, a);
      load8(xr + hc * 8, b);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float2 r = cs[(c - p.c0) * 8 + k];
        const float u = a[k] * r.x - b[k] * r.y;
        b[k] = b[k] * r.x + a[k] * r.y;
        a[k] = u;
      }
      store8(yr, a);
      store8(yr + hc * 8, b);
    }
  }
}

}  // namespace rp

smla_status_t launch_rope(const RopeArgs& a, const smla_seqs_t& seqs, unsigned* err, cudaStream_t stream) {
  using namespace rp;
  Params p{};
  p.x = a.x;
  p.out = a.out;
  p.x_ts = a.x_ts;
  p.x_hs = a.x_hs;
  p.o_ts = a.o_ts;
  p.o_hs = a.o_hs;
  p.seqs = seqs_dev(seqs);
  p.H = a.H;
  p.chunks = a.D / 8;
  p.magic = static_cast<uint32_t>(((uint64_t(1) << 32) + p.chunks - 1) / p.chunks);
  p.c0 = a.rope.offset / 8;
  p.c1 = p.c0 + a.rope.dim / 8;
  p.half = a.rope.layout == SMLA_ROPE_HALF;
  p.in_place = a.x == a.out && a.x_dtype == a.out_dtype && a.x_ts == a.o_ts && a.x_hs == a.o_hs;
  p.inv_freq = a.rope.inv_freq;
  p.amplitude = a.rope.amplitude;
  p.err = err;
  // two CTAs per SM at least, where there are heads enough to give them
  const int full = std::max(1, kChunksPerCta / p.chunks);
  const int64_t want = 2 * device_sm_count();
  const int groups = static_cast<int>(std::max<int64_t>((a.H + full - 1) / full, (want + seqs.T - 1) / seqs.T));
  p.heads_per_cta = std::max(1, (a.H + groups - 1) / groups);
  const dim3 grid(static_cast<unsigned>(seqs.T), static_cast<unsigned>((a.H + p.heads_per_cta - 1) / p.heads_per_cta));
  using bf = __nv_bfloat16;
  if (a.x_dtype == SMLA_BF16) {
    if (a.out_dtype == SMLA_BF16)
      rope_kernel<bf, bf><<<grid, kThreads, 0, stream>>>(p);
    else if (a.out_dtype == SMLA_F32)
      rope_kernel<bf, float><<<grid, kThreads, 0, stream>>>(p);
    else
      rope_kernel<bf, uint8_t><<<grid, kThreads, 0, stream>>>(p);
  } else {
    if (a.out_dtype == SMLA_BF16)
      rope_kernel<float, bf><<<grid, kThreads, 0, stream>>>(p);
    else if (a.out_dtype == SMLA_F32)
      rope_kernel<float, float><<<grid, kThreads, 0, stream>>>(p);
    else
      rope_kernel<float, uint8_t><<<grid, kThreads, 0, stream>>>(p);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail_cuda(e, "rope launch");
  return SMLA_OK;
}

}  // namespace smla
