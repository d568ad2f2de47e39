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
// * wide: rows of a are the MMA's M, rows of b its N, a pair of CTAs a tile of 256 x
//   256.  A thread of the epilogue owns half a tile's row, so a block's scale is one
//   number for it.  Persistent pairs walk the tiles in groups of eight row tiles.  A
//   last wave that would leave half of the pairs idle goes as halves of 256 x 128, with
//   four accumulators (4096 x 4096 x 16384 218 -> 202 us when they came, 512 rows of it
//   60 -> 42.7).
// * narrow, for calls whose few rows leave the wide form's tiles too few to fill
//   the GPU: rows of b (the weights, which are what such a call reads) are the M,
//   rows of a the N (16, 32 or 64).  The CTAs of a cluster divide the columns k of a
//   tile and add their sums through distributed shared memory in a fixed order, so
//   that a result does not depend on the run.
//
// Bound and measured.  Wide: the epilogue's warps, whose waits, TMEM loads and
// multiply-adds follow one another, 870 cycles a block of 256 x 256 (MMAs 512): 4096 x
// 4096 x 16384 196-198 us (2790 TFLOP/s), 512 rows of it 38.4, 8192^3 376 (2920); with
// four blocks a tile and 269 MB to store, 4101 x 32768 x 512 97 us (a fill of as much 72).
// The heads of 4096 tokens, 128 x (4096 x 512 x 128): 108 us, of which HBM takes 92.
// (Slower or the same: one CTA's MMAs with b by multicast 216 us for 217; 16 epilogue
// warps of 64 columns 228; each load one piece ahead, over the end of a block, 237.)
// Narrow: HBM behind 4 us of start and end, 16 x 4096 x 16384 14.5 us (4.6 TB/s),
// 128 x (16 x 512 x 128) 5.1 us.
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
  bool a_flip, o_flip;  // a's (out's) tensor map has the batch before the rows
  int G, M, N;
  int m_tiles, n_tiles;
  int64_t tiles;
  unsigned whole;  // (wide: tiles from this one on are halves)
  unsigned* err;
};

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// ------------------------------------------------------------------------ wide
// A pair of CTAs takes 256 rows of a and BN of b: each loads 128 rows of a and BN / 2
// of b a block, and the first one's MMAs (cta_group::2) read both shared memories,
// where a CTA by itself, which stages all of b, is bound by them (48 KB in and 48
// KB out a block of 512 MMA cycles: 712 cycles).  Each CTA's TMEM holds its own
// 128 rows' sums.
// Warps: 0-7 epilogue (32 rows x BN / 2 columns each), 8 TMA loads (the second CTA's
// count on the first one's barrier too, which its MMAs wait for), 9 MMAs (in the first
// CTA), 10-11 a's and b's scales.
// (The launch's 384 x 168 registers are 128 x (2 x 216 + 72).)
constexpr int kWideThreads = 384, kWideRegs = 168, kWideSoft = 8, kGroupM = 8;
static_assert(128 * (2 * 216 + 72) <= kWideThreads * kWideRegs, "the split draws on the launch's registers");
constexpr int kScaleBlocks = 8;  // blocks whose scales are fetched together
constexpr int kScaleRow = 132;   // padded: the fetching warps' transposed stores meet all banks

constexpr int BN = 256;

struct WideSmem {
  // a stage's way round takes 1.5 us: what is in flight sets a half tile's rate (512 x
  // 4096 x 16384: 50 us with four for 42.7, before the loads of the second CTA counted
  // on the first one's barrier; 38.4 since)
  static constexpr int kStages = 5;
  // places for 64 bytes of an epilogue warp's 32 rows on their way out (4101 x 32768 x
  // 512 with one, and a stage more: 106 us for 101)
  static constexpr int kPlaces = 2;
  uint8_t a[kStages][128 * kBK];
  uint8_t b[kStages][BN / 2 * kBK];
  uint8_t out[kWideSoft][kPlaces][32 * 64];
  float as[2][kScaleBlocks][kScaleRow], bs[2][2][kScaleBlocks];
  unsigned long long full[kStages], empty[kStages];
  // of the two accumulators of BN columns, then of the four of BN / 2
  unsigned long long sum_full[6], sum_empty[6], scale_full[2], scale_empty[2], drain;
  uint32_t tmem_base;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// An address of this CTA's shared memory in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t cluster_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// Word to the first CTA of finished TMEM reads, which are over before it is given
// and leave nothing in memory to be seen.  (No release beyond the CTA's: a
// cluster-wide one waits for the warp's every store, 765 us at 4096^2 x 16384.)
__device__ __forceinline__ void cluster_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// A 3-D tiled load into this CTA's shared memory whose bytes count on a barrier of
// either CTA of the pair (`bar`: an address in the cluster).  (Told of by a thread of
// the second CTA instead they took 199 us for 196 at 4096^2 x 16384, with a release of
// CTA scope, which promises nothing to another CTA, and 453 with one of the cluster's.)
__device__ __forceinline__ void pair_load_3d(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%3, %4, "
      "%5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// The tcgen05 operations of a pair of CTAs.
__device__ __forceinline__ void pair_tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem), "r"(ncols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void pair_tmem_dealloc(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
__device__ __forceinline__ void pair_mma_f8f6f4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrives on the barrier at this address in the CTAs of the mask (both) when the MMAs
// so far complete.
__device__ __forceinline__ void pair_commit(uint32_t bar, uint16_t ctas = 3) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
               "h"(ctas)
               : "memory");
}

struct Tile {
  int g, m0, n0;
};
// Tile t of the walk (below 2^31: the entry checks it): batch after batch; in
// each, groups of kGroupM row tiles, column after column, so that the CTAs of a
// moment share few rows of a and b.
__device__ __forceinline__ Tile tile_at(const Params& p, unsigned t) {
  const unsigned per = static_cast<unsigned>(p.m_tiles) * p.n_tiles;
  const unsigned g = p.G == 1 ? 0 : t / per, r = t - g * per;
  const unsigned group = static_cast<unsigned>(kGroupM) * p.n_tiles;
  const unsigned gr = r / group, in = r - gr * group, first = gr * kGroupM;
  const unsigned rows = min(static_cast<unsigned>(kGroupM), p.m_tiles - first);
  const unsigned n = in / rows, m = in - n * rows;
  return {static_cast<int>(g), static_cast<int>(first + m) * 256, static_cast<int>(n) * BN};
}

__global__ void __launch_bounds__(kWideThreads, 1)
    wide_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                const __grid_constant__ CUtensorMap tb_half, const __grid_constant__ CUtensorMap to, const Params p) {
  using S = WideSmem;
  constexpr int kStages = S::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023u) {  // (the same for every CTA)
    if (threadIdx.x == 0) atomicOr(p.err, kErrShape);
    return;
  }
  S& s = *reinterpret_cast<S*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(blockIdx.x & 1), m_of = rank * 128;  // this CTA's rows of a tile
  const unsigned tiles = static_cast<unsigned>(p.tiles), pairs = gridDim.x >> 1;
  // The pair's tiles: role(columns, tile) of each whole one, then of the half that may
  // follow.  (The half's code is its own: with its size a variable, the whole tiles'
  // loop took 5 to 8 % longer.)
  const auto walk = [&](auto&& role) {
    unsigned t = blockIdx.x >> 1;
    bool ok = true;
    for (; ok && t < p.whole; t += pairs) ok = role(std::integral_constant<int, BN>{}, tile_at(p, t));
    if (!ok || t >= tiles) return;
    const unsigned in = t - p.whole;
    Tile tile = tile_at(p, p.whole + (in >> 1));
    tile.n0 += static_cast<int>(in & 1) * (BN / 2);
    role(std::integral_constant<int, BN / 2>{}, tile);
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);  // (the first CTA's counts)
      mbar_init(smem_u32(&s.empty[i]), 1);
    }
    for (int i = 0; i < 6; ++i) {
      mbar_init(smem_u32(&s.sum_full[i]), 1);
      mbar_init(smem_u32(&s.sum_empty[i]), 2 * kWideSoft);  // (the first CTA's counts)
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.scale_full[i]), 2);
      mbar_init(smem_u32(&s.scale_empty[i]), kWideSoft);
    }
    mbar_init(smem_u32(&s.drain), 1);
    fence_mbar_init();
  }
  if (warp == 9) {
    pair_tmem_alloc(smem_u32(&s.tmem_base), 2 * BN);
  }
  if (threadIdx.x == 8 * 32) {
    tma_prefetch_desc(&ta);
    tma_prefetch_desc(p.whole ? &tb : &tb_half);
    tma_prefetch_desc(&to);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are there
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;

  if (warp < kWideSoft) {
    // ================================================================ epilogue
    setmaxnreg_inc<216>();
    const int half = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t full0 = smem_u32(s.sum_full), empty0 = cluster_addr(smem_u32(s.sum_empty), 0);
    int buf = 0, q = 0;            // accumulator, group of scales
    uint32_t phase = 0, q_phase = 0;
    walk([&](auto c, const Tile& tile) {
      constexpr int cols = decltype(c)::value;
      constexpr int kCols = cols / 2, kSums = 2 * BN / cols;  // columns of a thread, accumulators
      constexpr int kFirst = cols == BN ? 0 : 2;
      if (cols != BN) buf = phase = 0;
      const uint32_t from = tmem + lanes + half * kCols;
      bool ok = true;
      float acc[kCols];
#pragma unroll
      for (int c = 0; c < kCols; ++c) acc[c] = 0.f;
      for (int kb0 = 0; ok && kb0 < p.kb; kb0 += kScaleBlocks) {
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&s.scale_full[q]), q_phase, p.err));
        const float* sa = &s.as[q][0][(warp & 3) * 32 + lane];
        const float* sb = s.bs[q][cols == BN ? half : 0];
#pragma unroll 1
        for (int left = min(kScaleBlocks, p.kb - kb0); ok && left > 0; --left, sa += kScaleRow, ++sb) {
          const float scale = *sa * *sb;
          ok = __all_sync(0xffffffffu, mbar_wait(full0 + 8 * (kFirst + buf), phase, p.err));
          tc_fence_after();
          const uint32_t a = from + buf * cols;
          // 32 columns at a time, two loads in flight.  (Paired multiply-adds had a move
          // beside each, for their register pairs: 252 us for 213 at 4096^2 x 16384.)
          const auto add = [&](const uint32_t (&v)[32], int c) {
#pragma unroll
            for (int k = 0; k < 32; ++k) acc[c + k] = fmaf(__uint_as_float(v[k]), scale, acc[c + k]);
          };
          uint32_t v0[32], v1[32];
          tmem_ld32(a, v0);
          tmem_ld32(a + 32, v1);
          tmem_wait_ld_regs(v0);
          tmem_wait_ld_regs(v1);
          if constexpr (cols == BN) {
            add(v0, 0);
            tmem_ld32(a + 64, v0);
            add(v1, 32);
            tmem_ld32(a + 96, v1);
            tmem_wait_ld_regs(v0);
            tmem_wait_ld_regs(v1);
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) cluster_arrive(empty0 + 8 * (kFirst + buf));
          add(v0, kCols - 64);
          add(v1, kCols - 32);
          buf = (buf + 1) % kSums;
          phase ^= buf == 0;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.scale_empty[q]));
        q ^= 1;
        q_phase ^= q ^ 1;
      }
      const int row0 = tile.m0 + m_of + (warp & 3) * 32, n0 = tile.n0 + half * kCols;
      if (ok && row0 < p.M) {
        // 64 bytes of the warp's 32 rows at a time, through shared memory: stores of a
        // row by each thread took a sector of their own each (K = 512, 4101 x 32768:
        // 166 us).  The tensor's ends are the store's to mind.
        const int per = p.out_f32 ? 16 : 32;
        const auto put = [&](int c, int place, auto&& piece) {  // columns [c, c + per)
          if (n0 + c >= p.N) {  // (an empty group: the wait for a place counts them)
            if (lane == 0) tma_store_commit();
            return;
          }
          uint8_t* stage = s.out[warp][place];
          if (lane == 0) tma_store_wait_read<S::kPlaces - 1>();
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            *reinterpret_cast<uint4*>(stage + lane * 64 + ((k ^ ((lane >> 1) & 3)) << 4)) = piece(k);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            const int x = (n0 + c) * (64 / per);
            tma_store_3d(&to, smem_u32(stage), x, p.o_flip ? tile.g : row0, p.o_flip ? row0 : tile.g);
            tma_store_commit();
          }
        };
        if (p.out_f32) {
#pragma unroll
          for (int c = 0; c < kCols; c += 16)
            put(c, c / 16 % S::kPlaces, [&](int k) {
              const float* f = acc + c + 4 * k;
              return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
            });
        } else {
#pragma unroll
          for (int c = 0; c < kCols; c += 32)
            put(c, c / 32 % S::kPlaces, [&](int k) {
              const float* f = acc + c + 8 * k;
              return make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
            });
        }
      }
      return ok;
    });
    if (lane == 0) tma_store_wait_all();
    __syncwarp();
  } else {
    setmaxnreg_dec<72>();
    if (warp == 8) {
      // ================================================================== loads
      if (elect_one()) {
        int st = 0;
        uint32_t phase = 0, used = 0;
        bool ok = true;
        const uint32_t full0 = cluster_addr(smem_u32(s.full), 0);
        walk([&](auto c, const Tile& tile) {
          constexpr int cols = decltype(c)::value;
          const CUtensorMap* const map = cols == BN ? &tb : &tb_half;
          const int m = tile.m0 + m_of, n = tile.n0 + rank * (cols / 2);
          const int y = p.a_flip ? tile.g : m, z = p.a_flip ? m : tile.g;
          for (int kb = 0; kb < p.kb; ++kb) {
            ok = mbar_wait(smem_u32(&s.empty[st]), phase ^ 1, p.err);
            if (!ok) return false;
            // (the second CTA's bytes may land ahead of this: the phase is not over
            // without the arrival)
            if (rank == 0) mbar_arrive_expect_tx(smem_u32(&s.full[st]), 2 * (128 + cols / 2) * kBK);
            pair_load_3d(smem_u32(s.a[st]), &ta, kb * kBK, y, z, full0 + 8 * st);
            pair_load_3d(smem_u32(s.b[st]), map, kb * kBK, n, tile.g, full0 + 8 * st);
            used |= 1u << st;
            if (++st == kStages) {
              st = 0;
              phase ^= 1;
            }
          }
          return true;
        });
        // nothing is on its way into this CTA's memory when it ends: each stage's last
        // load, and the word that the MMAs have read it (which comes to both CTAs; its
        // parity is the load's).  Where a wait has given up, the second CTA's own loads
        // were issued before that wait began, and are waited for by the first.
        for (int k = 0; k < kStages; ++k) {
          if (!(used >> k & 1)) continue;
          const uint32_t last = k < st ? phase : phase ^ 1;
          if (rank == 0) ok = mbar_wait(smem_u32(&s.full[k]), last, p.err) && ok;
          ok = ok && mbar_wait(smem_u32(&s.empty[k]), last, p.err);
        }
      }
      __syncwarp();
    } else if (warp == 9) {
      // =================================================================== MMAs
      if (rank == 0 && elect_one()) {
        const uint64_t da = make_sdesc(smem_u32(s.a[0]), 16, 1024, kSwizzle128B);
        const uint64_t db = make_sdesc(smem_u32(s.b[0]), 16, 1024, kSwizzle128B);
        // (One thread, whose every instruction the MMAs wait for: nothing is computed
        // that can be carried along.)
        const uint32_t full0 = smem_u32(s.full), empty0 = smem_u32(s.empty);
        const uint32_t sum_full0 = smem_u32(s.sum_full), sum_empty0 = smem_u32(s.sum_empty);
        int st = 0, buf = 0;
        uint32_t phase = 0, buf_phase = 1;
        walk([&](auto c, const Tile&) {
          constexpr int cols = decltype(c)::value;
          constexpr uint32_t IDESC = idesc_e4m3_f32(256, cols, 0, 0);
          constexpr int kSums = 2 * BN / cols, kFirst = cols == BN ? 0 : 2;
          if (cols != BN) {
            for (int i = 0; i < 2; ++i) {  // the wider accumulators have been read
              if (!mbar_wait(sum_empty0 + 8 * buf, buf_phase, p.err)) return false;
              buf ^= 1;
              buf_phase ^= buf ^ 1;
            }
            buf = 0;
            buf_phase = 1;
          }
          for (int kb = 0; kb < p.kb; ++kb) {
            if (!mbar_wait(full0 + 8 * st, phase, p.err)) return false;
            if (!mbar_wait(sum_empty0 + 8 * (kFirst + buf), buf_phase, p.err)) return false;
            tc_fence_after();
            const uint64_t a = da + static_cast<uint64_t>(st * (128 * kBK >> 4));
            const uint64_t b = db + static_cast<uint64_t>(st * (BN / 2 * kBK >> 4));
#pragma unroll
            for (int k = 0; k < 4; ++k)
              pair_mma_f8f6f4(tmem + buf * cols, a + static_cast<uint64_t>(2 * k), b + static_cast<uint64_t>(2 * k), IDESC,
                              k ? 1u : 0u);
            pair_commit(sum_full0 + 8 * (kFirst + buf));
            pair_commit(empty0 + 8 * st);
            buf = (buf + 1) % kSums;
            buf_phase ^= buf == 0;
            if (++st == kStages) {
              st = 0;
              phase ^= 1;
            }
          }
          return true;
        });
        pair_commit(smem_u32(&s.drain), 1);  // (the second CTA ends by its loads' waits)
        mbar_wait(smem_u32(&s.drain), 0, p.err);
      }
      __syncwarp();
    } else {
      // ================================================================= scales
      // Eight blocks' at a time, turned round: a warp reads four rows' eight numbers
      // at once, and the epilogue 32 rows' of one block.  (Read by the epilogue's
      // threads, a row each, they took a third of the kernel: 297 us for 208 at 4096^2
      // x 16384.)
      const int rows0 = (warp - 10) * 64 + (lane >> 3), b = lane & 7;
      int q = 0;
      const auto tile_scales = [&](const Tile& tile) {
        const float* as = p.as + tile.g * p.as_gs;
        const float* bs = p.bs + static_cast<int64_t>(tile.g) * p.nb * p.kb;
        for (int kb0 = 0; kb0 < p.kb; kb0 += kScaleBlocks, ++q) {
          const int kb = min(kb0 + b, p.kb - 1);
          float v[16], w = 0.f;
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = as[min(tile.m0 + m_of + rows0 + 4 * k, p.M - 1) * p.as_ms + kb];
          const int n = lane >> 3;  // half of the tile's columns
          if (n < 2) w = bs[static_cast<int64_t>(min((tile.n0 + n * 128) / 128, p.nb - 1)) * p.kb + kb];
          if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&s.scale_empty[q & 1]), ((q >> 1) & 1) ^ 1, p.err))) return false;
#pragma unroll
          for (int k = 0; k < 16; ++k) s.as[q & 1][b][rows0 + 4 * k] = v[k];
          if (warp == 10 && n < 2) s.bs[q & 1][n][b] = w;
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&s.scale_full[q & 1]));
        }
        return true;
      };
      walk([&](auto, const Tile& tile) { return tile_scales(tile); });
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA's memory is touched any more
  tc_fence_after();
  if (warp == 9) pair_tmem_dealloc(tmem, 2 * BN);
}

// ---------------------------------------------------------------------- narrow
constexpr int kNarrowThreads = 192;

constexpr int kNarrowStages = 5, kNarrowChunk = 32;
// (two CTAs an SM)
constexpr int most_stages(int mt) { return mt == 64 ? 4 : kNarrowStages; }
// Behind the stages (weights, then rows of a, each 1024-byte aligned).
template <int MT>
struct NarrowSmem {
  alignas(16) float scale[kNarrowChunk][MT + 4];  // of a chunk of blocks: a's times b's
  unsigned long long full[kNarrowStages], empty[kNarrowStages], sum_full[2], sum_empty[2], drain;
  uint32_t tmem_base;
};
template <int MT>
constexpr int stage_bytes() {
  return (128 + MT) * kBK;
}

// The word at this CTA's shared-memory address in CTA `rank` of the cluster.
__device__ __forceinline__ float cluster_ld(uint32_t addr, uint32_t rank) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr(addr, rank)) : "memory");
  return v;
}

template <int MT, int CS>
__global__ void __launch_bounds__(kNarrowThreads, 2)
    narrow_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb, const Params p,
                  const int stages) {
  constexpr int kTmemCols = 2 * MT < 32 ? 32 : 2 * MT;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* const s_b = smem_raw;                        // [stages][128][kBK]
  uint8_t* const s_a = smem_raw + stages * 128 * kBK;   // [stages][MT][kBK]
  auto& s = *reinterpret_cast<NarrowSmem<MT>*>(smem_raw + stages * (128 + MT) * kBK);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CS > 1 ? static_cast<int>(blockIdx.x % CS) : 0;
  const int64_t t = blockIdx.x / CS;
  const int64_t per = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
  const int g = static_cast<int>(t / per), r = static_cast<int>(t - g * per);
  const int n0 = r / p.m_tiles * 128, m0 = r % p.m_tiles * MT;
  const int kb0 = static_cast<int>(static_cast<int64_t>(p.kb) * rank / CS);
  const int kb1 = static_cast<int>(static_cast<int64_t>(p.kb) * (rank + 1) / CS);
  if (smem_u32(smem_raw) & 1023u) {  // (the same for every CTA)
    if (threadIdx.x == 0) atomicOr(p.err, kErrShape);
    return;
  }
  const auto load = [&](int i) {  // block kb0 + i into its stage
    const int st = i % stages, kb = kb0 + i;
    const uint32_t bar = smem_u32(&s.full[st]);
    mbar_arrive_expect_tx(bar, (128 + MT) * kBK);
    tma_load_3d(smem_u32(s_b + st * 128 * kBK), &tb, kb * kBK, n0, g, bar);
    tma_load_3d(smem_u32(s_a + st * MT * kBK), &ta, kb * kBK, p.a_flip ? g : m0, p.a_flip ? m0 : g, bar);
  };
  // (the first loads go out ahead of the rest of the set-up)
  if (threadIdx.x == 4 * 32) {
    for (int i = 0; i < stages; ++i) {
      mbar_init(smem_u32(&s.full[i]), 1);
      mbar_init(smem_u32(&s.empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.sum_full[i]), 1);
      mbar_init(smem_u32(&s.sum_empty[i]), 4);
    }
    mbar_init(smem_u32(&s.drain), 1);
    fence_mbar_init();
    for (int i = 0; i < min(stages, kb1 - kb0); ++i) load(i);
  }
  if (warp == 5) {
    tmem_alloc(smem_u32(&s.tmem_base), kTmemCols);
    tmem_relinquish();
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
    // Scales come 32 blocks at a time, each warp reading a quarter of the rows with a
    // lane for each block, and wait in registers while the chunk before is used.
    // (Read a block at a time they were late: 14.7 us for 16 x 4096 x 16384.)
    constexpr int kPer = MT / 4;
    const float* as = p.as + g * p.as_gs;
    const float* bs = p.bs + (static_cast<int64_t>(g) * p.nb + n0 / 128) * p.kb;
    float next[kPer];
    const auto fetch = [&](int kb) {
      const int at = min(kb + lane, p.kb - 1);
      const float w = bs[at];
#pragma unroll
      for (int j = 0; j < kPer; ++j) next[j] = as[min(m0 + warp * kPer + j, p.M - 1) * p.as_ms + at] * w;
    };
    if (kb0 < kb1) fetch(kb0);
    int buf = 0;
    uint32_t phase = 0;
    bool ok = true;
    // (a warp whose wait gives up still keeps the chunks' barriers)
    for (int kc = kb0; kc < kb1; kc += kNarrowChunk) {
      if (kc > kb0) named_bar_sync(1, 128);  // the chunk before has been used
#pragma unroll
      for (int j = 0; j < kPer; ++j) s.scale[lane][warp * kPer + j] = next[j];
      named_bar_sync(1, 128);
      if (kc + kNarrowChunk < kb1) fetch(kc + kNarrowChunk);
      const int n = min(kNarrowChunk, kb1 - kc);
#pragma unroll 1
      for (int k = 0; ok && k < n; ++k) {
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&s.sum_full[buf]), phase, p.err));
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = tmem + lanes + buf * MT;
        const float* sc = s.scale[k];
        uint32_t v[MT];
        if constexpr (MT == 16) {
          tmem_ld16(a, v);
        } else {
#pragma unroll
          for (int c = 0; c < MT; c += 32) tmem_ld32(a + c, reinterpret_cast<uint32_t(&)[32]>(v[c]));
        }
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < MT; ++c) asm volatile("" : "+r"(v[c]));
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s.sum_empty[buf]));
#pragma unroll
        for (int c = 0; c < MT; c += 4) {
          const float4 f = *reinterpret_cast<const float4*>(sc + c);
          acc[c] = fmaf(__uint_as_float(v[c]), f.x, acc[c]);
          acc[c + 1] = fmaf(__uint_as_float(v[c + 1]), f.y, acc[c + 1]);
          acc[c + 2] = fmaf(__uint_as_float(v[c + 2]), f.z, acc[c + 2]);
          acc[c + 3] = fmaf(__uint_as_float(v[c + 3]), f.w, acc[c + 3]);
        }
        buf ^= 1;
        phase ^= buf ^ 1;
      }
    }
  } else if (warp == 4) {
    // ==================================================================== loads
    if (lane == 0) {
      int i = min(stages, kb1 - kb0);
      for (; i < kb1 - kb0; ++i) {
        if (!mbar_wait(smem_u32(&s.empty[i % stages]), ((i / stages) & 1) ^ 1, p.err)) break;
        load(i);
      }
      // nothing is still landing when the CTA ends
      for (int st = 0; st < stages; ++st) {
        const int loads = (i + stages - 1 - st) / stages;
        if (loads > 0) mbar_wait(smem_u32(&s.full[st]), (loads - 1) & 1, p.err);
      }
    }
    __syncwarp();
  } else {
    // ===================================================================== MMAs
    if (elect_one()) {
      constexpr uint32_t IDESC = idesc_e4m3_f32(128, MT, 0, 0);
      const uint64_t da = make_sdesc(smem_u32(s_b), 16, 1024, kSwizzle128B);
      const uint64_t db = make_sdesc(smem_u32(s_a), 16, 1024, kSwizzle128B);
      const uint32_t full0 = smem_u32(s.full), empty0 = smem_u32(s.empty);
      const uint32_t sum_full0 = smem_u32(s.sum_full), sum_empty0 = smem_u32(s.sum_empty);
      int st = 0, buf = 0;
      uint32_t phase = 0, buf_phase = 1;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!(mbar_wait(sum_empty0 + 8 * buf, buf_phase, p.err) && mbar_wait(full0 + 8 * st, phase, p.err))) break;
        tc_fence_after();
        const uint64_t a = da + static_cast<uint64_t>(st * (128 * kBK >> 4)), b = db + static_cast<uint64_t>(st * (MT * kBK >> 4));
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_f8f6f4_ss(tmem + buf * MT, a + static_cast<uint64_t>(2 * k), b + static_cast<uint64_t>(2 * k), IDESC, k ? 1u : 0u);
        mma_commit(sum_full0 + 8 * buf);
        mma_commit(empty0 + 8 * st);
        buf ^= 1;
        buf_phase ^= buf ^ 1;
        if (++st == stages) {
          st = 0;
          phase ^= 1;
        }
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
    float* part = reinterpret_cast<float*>(smem_raw);  // [MT][128], in place of the stages (all read)
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

// A [G][rows][width] byte tensor in boxes of box_bytes x box_rows, its dimensions in
// the order of their strides; *flip: the batch's comes before the rows'.
static bool byte_map(CUtensorMap* map, const void* x, int64_t gs, int64_t rs, int G, int rows, int64_t width, int box_rows,
                     bool* flip, int box_bytes = 128) {
  if (G == 1) gs = rs * rows;
  if (rows == 1) rs = gs;
  *flip = gs < rs;
  const int r = *flip ? 2 : 1, b = 3 - r;
  uint64_t dims[3] = {static_cast<uint64_t>(width)}, strides[2];
  uint32_t box[3] = {static_cast<uint32_t>(box_bytes)};
  dims[r] = static_cast<uint64_t>(rows);
  dims[b] = static_cast<uint64_t>(G);
  strides[r - 1] = static_cast<uint64_t>(rs);
  strides[b - 1] = static_cast<uint64_t>(gs);
  box[r] = static_cast<uint32_t>(box_rows);
  box[b] = 1;
  return encode_tma_u8(map, x, 3, dims, strides, box, box_bytes);
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
  if (byte_map(ta, a.a, a.a_gs, a.a_ms, a.G, a.M, a.K, a_rows, &p->a_flip) &&
      byte_map(tb, a.b, static_cast<int64_t>(a.N) * a.K, a.K, a.G, a.N, a.K, b_rows, &b_flip))
    return SMLA_OK;
  return fail(SMLA_ERR_CUDA, "cuTensorMapEncodeTiled failed for the block matmul's tensor maps");
}

template <typename... Args>
static smla_status_t launch_cluster(void (*kernel)(Args...), unsigned grid, int threads, size_t smem, int cluster,
                                    cudaStream_t stream, const Args&... args) {
  if (cluster == 1) {  // (the plain launch costs the host less)
    kernel<<<grid, threads, smem, stream>>>(args...);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? SMLA_OK : fail_cuda(e, "block matmul launch");
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = cluster;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e == cudaSuccess ? SMLA_OK : fail_cuda(e, "block matmul launch");
}

// How many of the wide form's tiles go as halves: a last wave that leaves half of
// the pairs idle.
static int64_t tail(int64_t tiles) {
  const int64_t pairs = device_sm_count() / 2, last = tiles % pairs;
  return 2 * last <= pairs ? last : 0;
}

static smla_status_t launch_wide(const MatmulArgs& a, unsigned* err, cudaStream_t stream) {
  Params p = params(a, 256, BN, err);
  CUtensorMap ta, tb, tb_half, to;
  smla_status_t st = maps(a, 128, BN / 2, &ta, &tb, &p);
  if (st != SMLA_OK) return st;
  const int es = p.out_f32 ? 4 : 2;
  if (!byte_map(&to, a.out, a.o_gs * es, a.o_ms * es, a.G, a.M, static_cast<int64_t>(a.N) * es, 32, &p.o_flip, 64))
    return fail(SMLA_ERR_CUDA, "cuTensorMapEncodeTiled failed for the block matmul's output");
  constexpr size_t smem = sizeof(WideSmem);
  static_assert(smem <= 232448, "");
  static std::atomic<unsigned long long> ready{0};
  st = prepare_kernel(reinterpret_cast<const void*>(wide_kernel), smem, kWideRegs, ready, "block matmul kernel");
  if (st != SMLA_OK) return st;
  const int64_t last = tail(p.tiles);
  p.whole = static_cast<unsigned>(p.tiles - last);
  p.tiles += last;
  tb_half = tb;
  bool flip;
  if (last && !byte_map(&tb_half, a.b, static_cast<int64_t>(a.N) * a.K, a.K, a.G, a.N, a.K, BN / 4, &flip))
    return fail(SMLA_ERR_CUDA, "cuTensorMapEncodeTiled failed for the block matmul's half tiles");
  const unsigned pairs = static_cast<unsigned>(std::min<int64_t>(p.tiles, device_sm_count() / 2));
  return launch_cluster(wide_kernel, 2 * pairs, kWideThreads, smem, 2, stream, ta, tb, tb_half, to, p);
}

template <int MT, int CS>
static smla_status_t launch_narrow(const MatmulArgs& a, unsigned* err, cudaStream_t stream) {
  Params p = params(a, MT, 128, err);
  CUtensorMap ta, tb;
  smla_status_t st = maps(a, MT, 128, &ta, &tb, &p);
  if (st != SMLA_OK) return st;
  // as many stages as a CTA has blocks: with few of them more CTAs fit an SM
  // (128 heads x 16 rows, K = 128: 6.5 us with five, 5.4)
  const int least = CS > 1 ? (MT * 128 * 4 + stage_bytes<MT>() - 1) / stage_bytes<MT>() : 1;
  const int stages = std::min(most_stages(MT), std::max((p.kb + CS - 1) / CS, least));
  const size_t smem = static_cast<size_t>(stages) * stage_bytes<MT>() + sizeof(NarrowSmem<MT>);
  static std::atomic<unsigned long long> ready{0};
  st = prepare_kernel(reinterpret_cast<const void*>(narrow_kernel<MT, CS>),
                      most_stages(MT) * stage_bytes<MT>() + sizeof(NarrowSmem<MT>), 0, ready, "block matmul kernel");
  if (st != SMLA_OK) return st;
  return launch_cluster(narrow_kernel<MT, CS>, static_cast<unsigned>(p.tiles * CS), kNarrowThreads, smem, CS, stream, ta, tb, p,
                        stages);
}

}  // namespace bm

smla_status_t launch_block_matmul(const MatmulArgs& a, unsigned* err, cudaStream_t stream) {
  using namespace bm;
  const int64_t sms = device_sm_count();
  const auto tiles = [&](int rows, int cols) {
    return static_cast<int64_t>(a.G) * ((a.M + rows - 1) / rows) * ((a.N + cols - 1) / cols);
  };
  const int kb = (a.K + kBK - 1) / kBK;
  // The wide form where it is the faster one: a wave of its tiles takes about 1.5 us
  // and 0.42 a block (0.27 of halves), a 64-row tile of the narrow form an SM 1.5 us
  // and 0.27 a block (narrow / wide: 256 x 4096 x 4096 14.2 / 13.7 us, 512 rows 19.2 /
  // 14.0; 256 x 4096 x 16384 35.6 / 38.1, 512 rows 62 / 38.1; 64 x 24576 x 2048 14.0 /
  // 18.2, 128 rows 20.5 / 19.2, 256 rows 31.7 / 19.8; 128 heads x 64 x 512 x 128 10.2 /
  // 12.1, 128 rows 16.9 / 12.4; where the choice costs most, of 33 sizes: 1000 x 1000 x
  // 992, narrow, 8.5 / 6.7).
  const int64_t wide = tiles(256, BN), last = tail(wide), waves = (wide - last + sms / 2 - 1) / (sms / 2);
  const int64_t wide_cost = (waves * (72 + 20 * kb) + (last ? 72 + 13 * kb : 0)) * sms;
  if (a.M > 32 && wide_cost < tiles(64, 128) * (72 + 13 * kb)) return launch_wide(a, err, stream);
  const auto go = [&](auto mt) {
    constexpr int MT = decltype(mt)::value;
    const int64_t n = tiles(MT, 128);
    // a tile's columns divided while all CTAs still run at once (a cluster of eight
    // leaves some of a GPC's SMs out: 38 tiles of 128 blocks 17.9 us in clusters of four,
    // 22.5 of eight)
    int cs = 1;
    while (cs < 8 && 2 * n * cs <= 2 * sms - sms / 4 && kb >= 4 * cs) cs *= 2;
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
