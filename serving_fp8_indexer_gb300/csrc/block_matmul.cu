// Batched product of e4m3 operands with a scale for each block of 128: the left
// one's for each row and 128 columns, the right one's (weights) for each 128 rows
// and 128 columns,
//   out[m, n] = sum_kb as[m, kb] bs[n / 128, kb] sum_{k in kb} a[m, k] b[n, k].
//
// The scales vary along k, so the tensor core's sum over a block of 128 columns
// goes into TMEM by itself and the warps of the epilogue add it, times its
// scales, to f32 sums in registers: four MMAs of 32 columns a block, two
// accumulators in turn, so that one block is read while the next is multiplied.
//
// Two forms.
// * wide: rows of a are the MMA's M (128), rows of b its N (256 or 128).  A thread
//   of the epilogue owns half a tile's row, so a block's scale is one number for
//   it.  Persistent CTAs, one an SM, walk the tiles in groups of 16 row tiles.
// * narrow, for calls whose few rows leave the wide form's tiles too few to fill
//   the GPU: rows of b (the weights, which are what such a call reads) are the M,
//   rows of a the N (16..128).  The CTAs of a cluster divide the columns k of a
//   tile and add their sums through distributed shared memory in a fixed order, so
//   that a result does not depend on the run.
#include <algorithm>
#include <type_traits>

#include "ptx.cuh"
#include "smla_internal.h"

namespace smla {
namespace bm {

constexpr int kBK = 128;  // columns of a block

struct Params {
  const float* as;
  int64_t as_gs, as_ms;
  const float* bs;
  int nb, kb;  // blocks of 128 along N and K
  void* out;
  int64_t o_gs, o_ms;
  bool out_f32;
  bool a_flip;  // a's tensor map has the batch before the rows
  int G, M, N;
  int m_tiles, n_tiles;
  int64_t tiles;
  unsigned* err;
};

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// ------------------------------------------------------------------------ wide
// (the launch's 384 x 168 registers are 128 x (2 x 216 + 72))
constexpr int kWideThreads = 384, kWideRegs = 168, kWideSoft = 8, kGroupM = 16;

template <int BN>
struct WideSmem {
  static constexpr int kStages = BN == 256 ? 4 : 6;
  uint8_t a[kStages][128 * kBK];
  uint8_t b[kStages][BN * kBK];
  unsigned long long full[kStages], empty[kStages], sum_full[2], sum_empty[2], drain;
  uint32_t tmem_base;
};

struct Tile {
  int g, m0, n0;
};
// Tile t of the walk: batch after batch; in each, groups of kGroupM row tiles,
// column after column, so that the CTAs of a moment share few rows of a and b.
template <int BN>
__device__ __forceinline__ Tile tile_at(const Params& p, int64_t t) {
  const int64_t per = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
  const int g = static_cast<int>(t / per);
  const int64_t r = t - g * per;
  const int64_t group = static_cast<int64_t>(kGroupM) * p.n_tiles;
  const int gr = static_cast<int>(r / group), first = gr * kGroupM;
  const int rows = min(kGroupM, p.m_tiles - first);
  const int in = static_cast<int>(r - gr * group);
  const int n = in / rows, m = in - n * rows;
  return {g, (first + m) * 128, n * BN};
}

template <int BN>
__global__ void __launch_bounds__(kWideThreads, 1)
    wide_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb, const Params p) {
  using S = WideSmem<BN>;
  constexpr int kStages = S::kStages, kCols = BN / 2;  // columns of a thread
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrShape);
    return;
  }
  S& s = *reinterpret_cast<S*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.sum_full[i]), 1);
      mbar_init(smem_u32(&s.sum_empty[i]), kWideSoft);
    }
    mbar_init(smem_u32(&s.drain), 1);
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(&s.tmem_base), 2 * BN);
    tmem_relinquish();
  }
  if (threadIdx.x == 8 * 32) {
    tma_prefetch_desc(&ta);
    tma_prefetch_desc(&tb);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;

  if (warp < kWideSoft) {
    // ================================================================ epilogue
    setmaxnreg_inc<216>();
    const int half = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int i = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; ok && t < p.tiles; t += gridDim.x) {
      const Tile tile = tile_at<BN>(p, t);
      const int m = tile.m0 + (warp & 3) * 32 + lane, n0 = tile.n0 + half * kCols;
      const bool in_m = m < p.M;
      const float* as = p.as + tile.g * p.as_gs + (in_m ? m : 0) * p.as_ms;
      const float* bs = p.bs + (static_cast<int64_t>(tile.g) * p.nb + min(n0 / 128, p.nb - 1)) * p.kb;
      float acc[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) acc[c] = 0.f;
      float sa = as[0], sb = bs[0];
      for (int kb = 0; kb < p.kb; ++kb, ++i) {
        const float scale = sa * sb;
        if (kb + 1 < p.kb) {
          sa = as[kb + 1];
          sb = bs[kb + 1];
        }
        const int buf = i & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&s.sum_full[buf]), (i >> 1) & 1, p.err));
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = tmem + lanes + buf * BN + half * kCols;
#pragma unroll
        for (int c = 0; c < kCols; c += 32) {
          uint32_t v[32];
          tmem_ld32(a + c, v);
          tmem_wait_ld_regs(v);
          if (c + 32 == kCols) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&s.sum_empty[buf]));
          }
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            const float2 r = fma2(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])), make_float2(scale, scale),
                                  make_float2(acc[c + k], acc[c + k + 1]));
            acc[c + k] = r.x;
            acc[c + k + 1] = r.y;
          }
        }
      }
      if (ok && in_m) {
        const int64_t at = tile.g * p.o_gs + m * p.o_ms + n0;
        const int left = p.N - n0;
        if (p.out_f32) {
          float* o = static_cast<float*>(p.out) + at;
#pragma unroll
          for (int c = 0; c < kCols; c += 4)
            if (c < left) *reinterpret_cast<float4*>(o + c) = make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
        } else {
          uint16_t* o = static_cast<uint16_t*>(p.out) + at;
#pragma unroll
          for (int c = 0; c < kCols; c += 8)
            if (c < left)
              *reinterpret_cast<uint4*>(o + c) = make_uint4(pack2(acc[c], acc[c + 1]), pack2(acc[c + 2], acc[c + 3]),
                                                            pack2(acc[c + 4], acc[c + 5]), pack2(acc[c + 6], acc[c + 7]));
        }
      }
    }
  } else {
    setmaxnreg_dec<72>();
  if (warp == 8) {
    // ==================================================================== loads
    int i = 0;
    if (elect_one()) {
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < p.tiles; t += gridDim.x) {
        const Tile tile = tile_at<BN>(p, t);
        for (int kb = 0; kb < p.kb; ++kb, ++i) {
          const int st = i % kStages;
          ok = mbar_wait(smem_u32(&s.empty[st]), ((i / kStages) & 1) ^ 1, p.err);
          if (!ok) break;
          const uint32_t bar = smem_u32(&s.full[st]);
          mbar_arrive_expect_tx(bar, (128 + BN) * kBK);
          tma_load_3d(smem_u32(s.a[st]), &ta, kb * kBK, p.a_flip ? tile.g : tile.m0, p.a_flip ? tile.m0 : tile.g, bar);
          tma_load_3d(smem_u32(s.b[st]), &tb, kb * kBK, tile.n0, tile.g, bar);
        }
      }
      // nothing is still landing when the CTA ends
      for (int st = 0; st < kStages; ++st) {
        const int loads = (i + kStages - 1 - st) / kStages;
        if (loads > 0) mbar_wait(smem_u32(&s.full[st]), (loads - 1) & 1, p.err);
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // ===================================================================== MMAs
    if (elect_one()) {
      constexpr uint32_t IDESC = idesc_e4m3_f32(128, BN, 0, 0);
      const uint64_t da = make_sdesc(smem_u32(s.a[0]), 16, 1024, kSwizzle128B);
      const uint64_t db = make_sdesc(smem_u32(s.b[0]), 16, 1024, kSwizzle128B);
      int i = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; ok && t < p.tiles; t += gridDim.x) {
        for (int kb = 0; kb < p.kb; ++kb, ++i) {
          const int st = i % kStages, buf = i & 1;
          ok = mbar_wait(smem_u32(&s.sum_empty[buf]), ((i >> 1) & 1) ^ 1, p.err) &&
               mbar_wait(smem_u32(&s.full[st]), (i / kStages) & 1, p.err);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f8f6f4_ss(tmem + buf * BN, da + static_cast<uint64_t>((st * 128 * kBK + k * 32) >> 4),
                          db + static_cast<uint64_t>((st * BN * kBK + k * 32) >> 4), IDESC, k ? 1u : 0u);
          mma_commit(smem_u32(&s.empty[st]));
          mma_commit(smem_u32(&s.sum_full[buf]));
        }
      }
      mma_commit(smem_u32(&s.drain));
      mbar_wait(smem_u32(&s.drain), 0, p.err);
    }
    __syncwarp();
  }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_dealloc(tmem, 2 * BN);
}

// ---------------------------------------------------------------------- narrow
constexpr int kNarrowThreads = 192;

template <int MT>
struct NarrowSmem {
  static constexpr int kStages = MT <= 32 ? 5 : 4;  // two CTAs an SM up to MT = 64
  uint8_t b[kStages][128 * kBK];
  uint8_t a[kStages][MT * kBK];
  alignas(16) float scale[4][2][MT];  // of each epilogue warp
  unsigned long long full[kStages], empty[kStages], sum_full[2], sum_empty[2], drain;
  uint32_t tmem_base;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The word at this CTA's shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ float cluster_ld(uint32_t addr, uint32_t rank) {
  uint32_t r;
  float v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(r) : "memory");
  return v;
}

template <int MT, int CS>
__global__ void __launch_bounds__(kNarrowThreads)
    narrow_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb, const Params p) {
  using S = NarrowSmem<MT>;
  constexpr int kStages = S::kStages;
  constexpr int kTmemCols = 2 * MT < 32 ? 32 : 2 * MT;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  S& s = *reinterpret_cast<S*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CS > 1 ? static_cast<int>(blockIdx.x % CS) : 0;
  const int64_t t = blockIdx.x / CS;
  const int64_t per = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
  const int g = static_cast<int>(t / per), r = static_cast<int>(t - g * per);
  const int n0 = r / p.m_tiles * 128, m0 = r % p.m_tiles * MT;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.kb) * rank / CS);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.kb) * (rank + 1) / CS);
  // (an unaligned base would be the same for every CTA)
  const bool aligned = (smem_u32(smem_raw) & 1023u) == 0;
  if (!aligned) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrShape);
    return;
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.sum_full[i]), 1);
      mbar_init(smem_u32(&s.sum_empty[i]), 4);
    }
    mbar_init(smem_u32(&s.drain), 1);
    fence_mbar_init();
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(&s.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == 4 * 32) {
    tma_prefetch_desc(&ta);
    tma_prefetch_desc(&tb);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;
  float acc[MT];

  if (warp < 4) {
    // ================================================================ epilogue
#pragma unroll
    for (int c = 0; c < MT; ++c) acc[c] = 0.f;
    const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
    constexpr int kPer = (MT + 31) / 32;  // rows whose scales a lane fetches
    const float* as[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) as[j] = p.as + g * p.as_gs + min(m0 + lane + 32 * j, p.M - 1) * p.as_ms;
    const float* bs = p.bs + (static_cast<int64_t>(g) * p.nb + n0 / 128) * p.kb;
    float na[kPer], nbs = 0.f;
    const auto fetch = [&](int kb) {
      nbs = bs[kb];
#pragma unroll
      for (int j = 0; j < kPer; ++j) na[j] = as[j][kb];
    };
    if (kb0 < kb1) fetch(kb0);
    for (int kb = kb0, i = 0; kb < kb1; ++kb, ++i) {
      const int buf = i & 1;
      float* sc = s.scale[warp][buf];
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (lane + 32 * j < MT) sc[lane + 32 * j] = na[j] * nbs;
      if (kb + 1 < kb1) fetch(kb + 1);
      const bool ok = mbar_wait(smem_u32(&s.sum_full[buf]), (i >> 1) & 1, p.err);
      if (!__all_sync(0xffffffffu, ok)) break;
      __syncwarp();
      tc_fence_after();
      const uint32_t a = tmem + lanes + buf * MT;
#pragma unroll
      for (int c = 0; c < MT; c += 16) {
        uint32_t v[16];
        tmem_ld16(a + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k) asm volatile("" : "+r"(v[k]));
        if (c + 16 == MT) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s.sum_empty[buf]));
        }
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
          const float4 f = *reinterpret_cast<const float4*>(sc + c + k);
          acc[c + k] = fmaf(__uint_as_float(v[k]), f.x, acc[c + k]);
          acc[c + k + 1] = fmaf(__uint_as_float(v[k + 1]), f.y, acc[c + k + 1]);
          acc[c + k + 2] = fmaf(__uint_as_float(v[k + 2]), f.z, acc[c + k + 2]);
          acc[c + k + 3] = fmaf(__uint_as_float(v[k + 3]), f.w, acc[c + k + 3]);
        }
      }
    }
  } else if (warp == 4) {
    // ==================================================================== loads
    if (elect_one()) {
      int i = 0;
      for (int kb = kb0; kb < kb1; ++kb, ++i) {
        const int st = i % kStages;
        if (!mbar_wait(smem_u32(&s.empty[st]), ((i / kStages) & 1) ^ 1, p.err)) break;
        const uint32_t bar = smem_u32(&s.full[st]);
        mbar_arrive_expect_tx(bar, (128 + MT) * kBK);
        tma_load_3d(smem_u32(s.b[st]), &tb, kb * kBK, n0, g, bar);
        tma_load_3d(smem_u32(s.a[st]), &ta, kb * kBK, p.a_flip ? g : m0, p.a_flip ? m0 : g, bar);
      }
      for (int st = 0; st < kStages; ++st) {
        const int loads = (i + kStages - 1 - st) / kStages;
        if (loads > 0) mbar_wait(smem_u32(&s.full[st]), (loads - 1) & 1, p.err);
      }
    }
    __syncwarp();
  } else {
    // ===================================================================== MMAs
    if (elect_one()) {
      constexpr uint32_t IDESC = idesc_e4m3_f32(128, MT, 0, 0);
      const uint64_t da = make_sdesc(smem_u32(s.b[0]), 16, 1024, kSwizzle128B);
      const uint64_t db = make_sdesc(smem_u32(s.a[0]), 16, 1024, kSwizzle128B);
      for (int kb = kb0, i = 0; kb < kb1; ++kb, ++i) {
        const int st = i % kStages, buf = i & 1;
        if (!(mbar_wait(smem_u32(&s.sum_empty[buf]), ((i >> 1) & 1) ^ 1, p.err) &&
              mbar_wait(smem_u32(&s.full[st]), (i / kStages) & 1, p.err)))
          break;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f8f6f4_ss(tmem + buf * MT, da + static_cast<uint64_t>((st * 128 * kBK + k * 32) >> 4),
                        db + static_cast<uint64_t>((st * MT * kBK + k * 32) >> 4), IDESC, k ? 1u : 0u);
        mma_commit(smem_u32(&s.empty[st]));
        mma_commit(smem_u32(&s.sum_full[buf]));
      }
      mma_commit(smem_u32(&s.drain));
      mbar_wait(smem_u32(&s.drain), 0, p.err);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_dealloc(tmem, kTmemCols);

  // ---- the cluster's sums, and the output
  constexpr int kOwn = MT / CS;  // rows of a that this CTA finishes
  float sum[kOwn];
  if constexpr (CS > 1) {
    float* part = reinterpret_cast<float*>(s.b);  // [MT][128], in place of the stages (all read)
    static_assert(sizeof(s.b) >= MT * 128 * sizeof(float), "");
    if (warp < 4) {
#pragma unroll
      for (int c = 0; c < MT; ++c) part[c * 128 + threadIdx.x] = acc[c];
    }
    cluster_sync();
    if (warp < 4) {
#pragma unroll
      for (int c = 0; c < kOwn; ++c) {
        const uint32_t addr = smem_u32(part + (rank * kOwn + c) * 128 + threadIdx.x);
        float v[CS];
#pragma unroll
        for (int k = 0; k < CS; ++k) v[k] = cluster_ld(addr, k);
        sum[c] = 0.f;
#pragma unroll
        for (int k = 0; k < CS; ++k) sum[c] += v[k];
      }
    }
    cluster_sync();  // every CTA's sums have been read
  } else {
#pragma unroll
    for (int c = 0; c < kOwn; ++c) sum[c] = acc[c];
  }
  const int n = n0 + threadIdx.x;
  if (warp < 4 && n < p.N) {
#pragma unroll
    for (int c = 0; c < kOwn; ++c) {
      const int m = m0 + rank * kOwn + c;
      if (m >= p.M) break;
      const int64_t at = g * p.o_gs + m * p.o_ms + n;
      if (p.out_f32)
        static_cast<float*>(p.out)[at] = sum[c];
      else
        static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(sum[c]);
    }
  }
}

// A [G][rows][K] byte operand in boxes of 128 columns x box_rows, its dimensions in
// the order of their strides; *flip: the batch's comes before the rows'.
static bool operand_map(CUtensorMap* map, const uint8_t* x, int64_t gs, int64_t rs, int G, int rows, int K, int box_rows,
                        bool* flip) {
  if (G == 1) gs = rs * rows;
  if (rows == 1) rs = gs;
  *flip = gs < rs;
  const int r = *flip ? 2 : 1, b = 3 - r;
  uint64_t dims[3] = {static_cast<uint64_t>(K)}, strides[2];
  uint32_t box[3] = {kBK};
  dims[r] = static_cast<uint64_t>(rows);
  dims[b] = static_cast<uint64_t>(G);
  strides[r - 1] = static_cast<uint64_t>(rs);
  strides[b - 1] = static_cast<uint64_t>(gs);
  box[r] = static_cast<uint32_t>(box_rows);
  box[b] = 1;
  return encode_tma_u8(map, x, 3, dims, strides, box, 128);
}

static Params params(const MatmulArgs& a, int rows, int cols, unsigned* err) {
  Params p{};
  p.as = a.a_scales;
  p.as_gs = a.as_gs;
  p.as_ms = a.as_ms;
  p.bs = a.b_scales;
  p.nb = (a.N + 127) / 128;
  p.kb = (a.K + kBK - 1) / kBK;
  p.out = a.out;
  p.o_gs = a.o_gs;
  p.o_ms = a.o_ms;
  p.out_f32 = a.out_dtype == SMLA_F32;
  p.G = a.G;
  p.M = a.M;
  p.N = a.N;
  p.m_tiles = (a.M + rows - 1) / rows;
  p.n_tiles = (a.N + cols - 1) / cols;
  p.tiles = static_cast<int64_t>(a.G) * p.m_tiles * p.n_tiles;
  p.err = err;
  return p;
}

static smla_status_t maps(const MatmulArgs& a, int a_rows, int b_rows, CUtensorMap* ta, CUtensorMap* tb, Params* p) {
  bool b_flip;
  if (operand_map(ta, a.a, a.a_gs, a.a_ms, a.G, a.M, a.K, a_rows, &p->a_flip) &&
      operand_map(tb, a.b, static_cast<int64_t>(a.N) * a.K, a.K, a.G, a.N, a.K, b_rows, &b_flip))
    return SMLA_OK;
  return fail(SMLA_ERR_CUDA, "cuTensorMapEncodeTiled failed for the block matmul's tensor maps");
}

template <int BN>
static smla_status_t launch_wide(const MatmulArgs& a, unsigned* err, cudaStream_t stream) {
  Params p = params(a, 128, BN, err);
  CUtensorMap ta, tb;
  smla_status_t st = maps(a, 128, BN, &ta, &tb, &p);
  if (st != SMLA_OK) return st;
  constexpr size_t smem = sizeof(WideSmem<BN>);
  static_assert(smem <= 232448, "");
  static std::atomic<unsigned long long> ready{0};
  st = prepare_kernel(reinterpret_cast<const void*>(wide_kernel<BN>), smem, kWideRegs, ready, "block matmul kernel");
  if (st != SMLA_OK) return st;
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(p.tiles, device_sm_count()));
  wide_kernel<BN><<<grid, kWideThreads, smem, stream>>>(ta, tb, p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SMLA_OK : fail_cuda(e, "block matmul launch");
}

template <int MT, int CS>
static smla_status_t launch_narrow(const MatmulArgs& a, unsigned* err, cudaStream_t stream) {
  Params p = params(a, MT, 128, err);
  CUtensorMap ta, tb;
  smla_status_t st = maps(a, MT, 128, &ta, &tb, &p);
  if (st != SMLA_OK) return st;
  constexpr size_t smem = sizeof(NarrowSmem<MT>);
  static std::atomic<unsigned long long> ready{0};
  st = prepare_kernel(reinterpret_cast<const void*>(narrow_kernel<MT, CS>), smem, 0, ready, "block matmul kernel");
  if (st != SMLA_OK) return st;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(p.tiles * CS));
  cfg.blockDim = dim3(kNarrowThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = CS;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, narrow_kernel<MT, CS>, ta, tb, p);
  return e == cudaSuccess ? SMLA_OK : fail_cuda(e, "block matmul launch");
}

}  // namespace bm

smla_status_t launch_block_matmul(const MatmulArgs& a, unsigned* err, cudaStream_t stream) {
  using namespace bm;
  const int sms = device_sm_count();
  const auto tiles = [&](int rows, int cols) {
    return static_cast<int64_t>(a.G) * ((a.M + rows - 1) / rows) * ((a.N + cols - 1) / cols);
  };
  if (a.M > 64 && tiles(128, 128) >= sms) {
    // the tile that wastes less of its last wave
    const auto waves = [&](int64_t n) { return (n + sms - 1) / sms; };
    return 2 * waves(tiles(128, 256)) <= waves(tiles(128, 128)) ? launch_wide<256>(a, err, stream)
                                                                : launch_wide<128>(a, err, stream);
  }
  const int kb = (a.K + kBK - 1) / kBK;
  const auto go = [&](auto mt) {
    constexpr int MT = decltype(mt)::value;
    const int64_t n = tiles(MT, 128);
    int cs = 1;
    while (cs < 8 && n * cs < 2 * sms && kb >= 4 * cs) cs *= 2;
    switch (cs) {
      case 1: return launch_narrow<MT, 1>(a, err, stream);
      case 2: return launch_narrow<MT, 2>(a, err, stream);
      case 4: return launch_narrow<MT, 4>(a, err, stream);
      default: return launch_narrow<MT, 8>(a, err, stream);
    }
  };
  if (a.M <= 16) return go(std::integral_constant<int, 16>{});
  if (a.M <= 32) return go(std::integral_constant<int, 32>{});
  return go(std::integral_constant<int, 64>{});
}

}  // namespace smla
