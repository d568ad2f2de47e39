// Dense MLA decode over a paged e4m3 latent cache (unit or per-row scales):
// attention of a few query tokens over every cached key of their sequence.
//
// Orientation and precision are those of the prefill attention kernel: keys
// are the MMA M dimension and query rows the N dimension,
//   S^T[128 keys x NR rows] = K . Q^T,   O^T[512 x NR] += V^T . P^T,
// all on the FP8 pipe, with bf16 q as two e4m3 terms (hi + lo / 32), so that the e4m3
// cache rows are used as they lie in memory.  What is different here:
//
// * Weights.  A cache is long: thousands of keys far below one that dominates
//   still hold much of the weight between them, and each has to be carried to
//   the same relative accuracy.  P is three e5m2 terms (3 bits each, 2^-9 of a
//   weight together), whose range of 32 binary places keeps eight bits down to
//   2^-19 of a row's largest weight (13 nats) and something down to 2^-28.  (Two
//   e4m3 terms, as in the prefill kernel, end 2^-14 below the largest: a key 10
//   nats above 32 K others left an eighth of their weight.  46.8 us at 64 rows
//   then, where the third term is a pass of its own; no difference at 16.)
// * Rows.  An item is up to NR rows (tokens x heads) of one sequence that
//   share every key: up to NR / H consecutive tokens of a sequence when H <
//   64, or 64 of one token's heads.  NR is 16, 32 or 64, so that a few heads
//   do not pay for 64.  Rows of earlier tokens mask the last keys.
// * Work.  The blocks of 128 keys of all items form one line, cut into equal
//   parts, one per CTA, wherever the cuts fall: no SM waits for the longest
//   sequence.  A part that is a whole item writes its output; the others
//   write f32 partial results (at most two per CTA), which a second kernel
//   joins per cut item.
// * Loads.  Pages are contiguous, so a block is 10 TMA boxes (64-key pages,
//   issued straight from one thread: 220 cycles a box out of a loop with
//   shuffles) instead of 4608 16-byte gathers; nothing but the page table is read to
//   address them.  Columns 0..511 lie in four 128-byte-swizzled chunks (each
//   the K-major QK operand and, read MN-major, one 128-column tile of V), the
//   rotary part in a 64-byte-swizzled one, which P^T reuses after QK.
// * For NR < 64, P's three terms are one operand of 3 NR columns with an
//   accumulator each (summed at the end): a third of the MMAs.  With NR = 64
//   there is no TMEM for that, and PV runs three times into one accumulator.
//   (Keeping a tile's V operand in the tensor core's buffer for its third product
//   took 54.2 us instead of 55.5, but nothing promises that it is still there: QK's
//   products come from another warp and may fall between the two.)
//
// Bound: HBM for few rows (a block of 73.7 KB is 3140 cycles of an SM's share
// of 6.8 TB/s; its MMAs about 1430 cycles at NR = 16, 1760 at 32), at NR = 64 the
// chain load -> QK -> softmax -> PV over two slots (tensor time about 3460 cycles
// a block, where the shared-memory reads of N = 64 operands set the rate: 48
// cycles an MMA).
//
// Measured: 16 heads over 4 x <= 120 K keys 49 us (4.6 TB/s; 6.2 while the line
// runs, then 6 us of start and 5.7 of join), 32 heads 54; 8 x 2 tokens x 128 heads
// over <= 8192 keys 55.6 us (566 TFLOP/s).
//
// Warps: 0-7 softmax and epilogue (thread = one key x NR/2 rows), 8 TMA, 9 QK,
// 10 PV.
#include <algorithm>
#include <cstddef>
#include <type_traits>

#include "decode_line.cuh"

namespace smla {
namespace dd {

constexpr int kChunk = kBK * 128;        // 128 columns of a block
constexpr int kRopeOff = 4 * kChunk;     // columns 512..575: [128][64 bytes]
constexpr int kSlot = kRopeOff + kBK * 64;
constexpr int kNST = 2;                  // block slots
constexpr int kHalf = kBK / 2;           // keys that one PV step of the pipeline takes
constexpr int kPRow = kBK * 64;          // a term of P^T, 64 bytes a key
// An item's first blocks cost their CTA more than the blocks themselves (its q
// is loaded and split, its result reduced and stored): the line counts that as
// this many blocks.
constexpr int kItemCost = 5;

template <int NR, int QP>
struct Smem {
  uint8_t q[QP * NR * kD];  // [4][QP * NR rows][128] then [QP * NR][64]: hi rows, then lo rows
  uint8_t kv[kNST][kSlot];
  // What P's first place (the rotary chunk of the block's slot) does not hold.
  // NR = 64: the second and third term of half a block's keys; 32: the third
  // term, a place for each slot.
  uint8_t pmore[NR == 64 ? kPRow : NR == 32 ? kNST * kPRow : 16];
  alignas(16) float cs[NR];    // softmax_scale * log2(e) / 2^e per row
  alignas(16) float negm[NR];  // minus the reference, log2 units
  float delta[NR], fac[NR];
  int mx[NR];
  float sums[4][NR];           // row sums of each quarter of the key lanes
  int nk[NR];                  // keys each row sees
  unsigned long long bar_qraw, bar_q, bar_full[kNST], bar_empty[kNST][2];
  unsigned long long bar_s[2], bar_s_free[2], bar_p[2][2], bar_more[2], bar_pv[2], bar_drain[2];
  uint32_t tmem_base;
};

// Two floats -> e4m3 hi and lo pairs, through f16 (|x| <= 256): hi = e4m3(x),
// lo = e4m3(32 (x - hi)), the difference exact in f16 and at most 8.  A bf16
// query's eight bits fit both, down to 2^-14 of its row's largest value (its lo
// products have accumulators of their own, which are divided by 32; with lo as it
// is they would fit to 2^-9 only, and a query with one very large element lost
// bits of all others).
constexpr uint32_t kLoF16x2 = 0x50005000u;  // 32
constexpr float kLoDown = 1.f / 32.f;
__device__ __forceinline__ void split2(float a, float b, uint16_t& hi, uint16_t& lo) {
  const uint32_t h = f32x2_to_f16x2(a, b);
  hi = f16x2_to_e4m3x2(h);
  lo = f16x2_to_e4m3x2(hmul2(hsub2(h, e4m3x2_to_f16x2(hi)), kLoF16x2));
}
// Two weights (0 .. 2^15) -> three e5m2 terms each, through f16, every difference
// exact there: off by 2^-3 of 2^-3 of 2^-3, and 2^-11 for the f16, of the weight,
// or by half of e5m2's smallest step, 2^-17.
__device__ __forceinline__ void split3(float a, float b, uint16_t& t1, uint16_t& t2, uint16_t& t3) {
  uint32_t h = f32x2_to_f16x2(a, b);
  t1 = f16x2_to_e5m2x2(h);
  h = hsub2(h, e5m2x2_to_f16x2(t1));
  t2 = f16x2_to_e5m2x2(h);
  t3 = f16x2_to_e5m2x2(hsub2(h, e5m2x2_to_f16x2(t2)));
}

template <int NR, int QP, bool ROWSCALE>
__global__ void __launch_bounds__(kThreads, 1)
    decode_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tqr,
                  const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tr, const Params p) {
  using S = Smem<NR, QP>;
  constexpr int kQN = QP * NR;                 // QK's N
  constexpr int kQChunk = kQN * 128;           // a 128-column chunk of Q
  constexpr int kParts = NR == 64 ? 1 : 3;     // accumulators of a V tile: one for each term, or one for all
  constexpr int kPN = kParts * NR;             // PV's N
  constexpr uint32_t kS = NR == 32 ? 384 : kTmemS;  // S's columns, behind O's
  constexpr int NC = NR / 2;                   // rows of a softmax thread
  static_assert(offsetof(S, kv) % 1024 == 0 && offsetof(S, pmore) % 1024 == 0, "swizzled tiles need 1024-byte alignment");
  static_assert(4 * kPN <= static_cast<int>(kS) && 2 * kQN <= static_cast<int>(kTmemCols - kS), "TMEM budget");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrShape);
    return;
  }
  S& s = *reinterpret_cast<S*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&s.bar_qraw), 1);
    mbar_init(smem_u32(&s.bar_q), kSoftThreads);
    for (int i = 0; i < kNST; ++i) {
      mbar_init(smem_u32(&s.bar_full[i]), 1);
      mbar_init(smem_u32(&s.bar_empty[i][0]), 1);
      mbar_init(smem_u32(&s.bar_empty[i][1]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.bar_s[i]), 1);
      mbar_init(smem_u32(&s.bar_s_free[i]), kSoftWarps);
      mbar_init(smem_u32(&s.bar_p[i][0]), kSoftWarps / 2);
      mbar_init(smem_u32(&s.bar_p[i][1]), kSoftWarps / 2);
      mbar_init(smem_u32(&s.bar_more[i]), kSoftWarps / 2);
      mbar_init(smem_u32(&s.bar_pv[i]), 1);
      mbar_init(smem_u32(&s.bar_drain[i]), 1);
    }
    fence_mbar_init();
  }
  if (threadIdx.x < NR) s.mx[threadIdx.x] = kOrdMin;
  if (warp == kQkWarp) {
    tmem_alloc(smem_u32(&s.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  // (the descriptors' and the line's cold reads overlap)
  if (threadIdx.x == kTmaWarp * 32) {
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tr);
    if (QP == 1) tma_prefetch_desc(&tqr);
  }
  const Cursor start = find_part(p, lane);  // this CTA's part of the line
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;

  // requests a segment's q rows (one thread)
  const auto load_q = [&](const Seg& g) {
    const int row = g.t0 * p.H + g.h0;
    const uint32_t bar = smem_u32(&s.bar_qraw), dst = smem_u32(s.q);
    mbar_arrive_expect_tx(bar, NR * kD * QP);
    if (QP == 2) {
#pragma unroll
      for (int c = 0; c < 9; ++c) tma_load_2d(dst + c * (NR * 128), &tq, c * 128, row, bar);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c) tma_load_2d(dst + c * kQChunk, &tq, c * 128, row, bar);
      tma_load_2d(dst + 4 * kQChunk, &tqr, 512, row, bar);
    }
  };
  if (start.b < 0) {
    // nothing left of the line for this CTA
  } else if (warp < 8) {
    // ===================================================== softmax, epilogue
    const int r = threadIdx.x & 127;    // key lane
    const int hb = (warp >> 2) * NC;    // rows [hb, hb + NC)
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    int q_in = 0;  // q loads waited for
    // PV of block i.  The block before the last one's PV is not always waited
    // for, and a wait that lags its barrier by two phases returns at once:
    // two barriers in turn, of which PV(i - 2) has completed wherever block i's
    // S has been seen (its keys lie in PV(i - 2)'s slot).
    auto wait_pv = [&](int i) { return mbar_wait(smem_u32(&s.bar_pv[i & 1]), (i >> 1) & 1, p.err); };
    // q of a segment: bf16 rows are split in place into e4m3 hi + lo (a
    // power of two per row puts the largest |q| in [128, 256)); rows past the
    // segment's are cleared
    auto convert_q = [&](const Seg& g) -> bool {
      if (!named_bar_and(1, kSoftThreads, mbar_wait(smem_u32(&s.bar_qraw), q_in++ & 1, p.err))) return false;
      if (QP == 2) {
        constexpr int kPer = NR / 32 > 0 ? NR / 32 : 1;  // rows an octet of lanes handles
        const int r8 = threadIdx.x & 7;
        uint4 v[kPer][9];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const int row = 32 * k + (threadIdx.x >> 3);
#pragma unroll
          for (int c = 0; c < 9; ++c)  // raw chunk c: 64 columns, [NR][128 bytes]
            v[k][c] = row < g.rows ? *reinterpret_cast<const uint4*>(s.q + c * (NR * 128) + sw128(row, r8))
                                   : make_uint4(0, 0, 0, 0);
        }
        named_bar_sync(1, kSoftThreads);  // every byte is read before any is overwritten
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
          const int row = 32 * k + (threadIdx.x >> 3);
          float amax = 0.f;
#pragma unroll
          for (int c = 0; c < 9; ++c) {
            const uint32_t w[4] = {v[k][c].x, v[k][c].y, v[k][c].z, v[k][c].w};
#pragma unroll
            for (int u = 0; u < 4; ++u)
              amax = max3(amax, fabsf(__uint_as_float(w[u] << 16)), fabsf(__uint_as_float(w[u] & 0xffff0000u)));
          }
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
          // 2^e that puts amax into [128, 256), from its exponent bits; capped
          // (an all-zero or subnormal row keeps a finite factor)
          const int e = min(7 + 127 - static_cast<int>(__float_as_uint(amax) >> 23), 120);
          // (an infinite q has no finite logits: its row becomes NaN, where e4m3
          // would have made it a large number)
          const float sigma = amax < INFINITY ? __uint_as_float(static_cast<uint32_t>(127 + e) << 23) : NAN;
          if (row < NR) {
#pragma unroll
            for (int c = 0; c < 9; ++c) {
              const uint32_t w[4] = {v[k][c].x, v[k][c].y, v[k][c].z, v[k][c].w};
              uint16_t hi[4], lo[4];
#pragma unroll
              for (int u = 0; u < 4; ++u)
                split2(__uint_as_float(w[u] << 16) * sigma, __uint_as_float(w[u] & 0xffff0000u) * sigma, hi[u], lo[u]);
              const uint2 h2 = make_uint2(hi[0] | static_cast<uint32_t>(hi[1]) << 16, hi[2] | static_cast<uint32_t>(hi[3]) << 16);
              const uint2 l2 = make_uint2(lo[0] | static_cast<uint32_t>(lo[1]) << 16, lo[2] | static_cast<uint32_t>(lo[3]) << 16);
              // columns 64 c + 8 r8 .. +7
              if (c < 8) {
                const int piece = (c & 1) * 4 + (r8 >> 1);
                uint8_t* dst = s.q + (c >> 1) * kQChunk + (r8 & 1) * 8;
                *reinterpret_cast<uint2*>(dst + sw128(row, piece)) = h2;
                *reinterpret_cast<uint2*>(dst + sw128(NR + row, piece)) = l2;
              } else {
                uint8_t* dst = s.q + 4 * kQChunk + (r8 & 1) * 8;
                *reinterpret_cast<uint2*>(dst + sw64(row, r8 >> 1)) = h2;
                *reinterpret_cast<uint2*>(dst + sw64(NR + row, r8 >> 1)) = l2;
              }
            }
            if (r8 == 0) s.cs[row] = p.softmax_scale * kLog2e / sigma;
          }
        }
      } else {
        for (int i = threadIdx.x; i < (NR - g.rows) * 36; i += kSoftThreads) {
          const int row = g.rows + i / 36, pc = i % 36;
          uint8_t* dst = pc < 32 ? s.q + (pc >> 3) * kQChunk + row * 128 + (pc & 7) * 16
                                 : s.q + 4 * kQChunk + row * 64 + (pc & 3) * 16;
          *reinterpret_cast<uint4*>(dst) = make_uint4(0, 0, 0, 0);
        }
        if (threadIdx.x < NR) s.cs[threadIdx.x] = p.softmax_scale * kLog2e;
      }
      fence_proxy_async_smem();
      mbar_arrive(smem_u32(&s.bar_q));
      return true;
    };
    // Page of the thread's key of block j (-1 outside the keys), and its scale
    // (1 there, and on a bad page, which the TMA warp reports).  The page is
    // read two blocks ahead and the scale one, so that neither read is waited
    // for inside a segment.
    auto key_page = [&](const Seg& g, int j) -> int {
      const int key = (g.j0 + j) * kBK + r;
      return ROWSCALE && key < seg_keys(g)
                 ? p.seqs.page_table[static_cast<int64_t>(g.b) * p.seqs.max_pages + (key >> p.seqs.page_shift)]
                 : -1;
    };
    auto key_scale = [&](const Seg& g, int j, int pid) -> float {
      const int key = (g.j0 + j) * kBK + r;
      const int64_t row = (static_cast<int64_t>(pid) << p.seqs.page_shift) | (key & ((1 << p.seqs.page_shift) - 1));
      return !ROWSCALE || pid < 0 || row >= p.phys_rows ? 1.f : p.scales[row];
    };
    Cursor cur = start;
    Seg g;
    bool ok = next_seg(p, cur, g);
    float sr_next = 1.f;
    int pid_next = -1;
    if (ok) {
      sr_next = key_scale(g, 0, key_page(g, 0));
      if (g.nb > 1) pid_next = key_page(g, 1);
      ok = convert_q(g);
    }
    int gb = 0;  // blocks of the segments before
    bool more = ok;
    while (ok && more) {
      const int n_item = seg_keys(g);
      if (threadIdx.x < NR) {
        s.negm[threadIdx.x] = 0.f;  // the first block sets the reference
        const int tok = p.groups > 1 ? 0 : threadIdx.x / p.H;
        s.nk[threadIdx.x] = threadIdx.x < g.rows ? g.pos1 + tok : 0;
      }
      named_bar_sync(1, kSoftThreads);
      float lv[NC];
#pragma unroll
      for (int h = 0; h < NC; ++h) lv[h] = 0.f;
      Cursor cn = cur;
      Seg gn;
      const bool has_next = next_seg(p, cn, gn);
      for (int j = 0; j < g.nb; ++j) {
        const int i = gb + j, slot = i % kNST, buf = i & 1;
        const float sr = sr_next;
        if (j + 1 < g.nb) {
          sr_next = key_scale(g, j + 1, pid_next);
          if (j + 2 < g.nb) pid_next = key_page(g, j + 2);
        } else if (has_next) {
          sr_next = key_scale(gn, 0, key_page(gn, 0));
          if (gn.nb > 1) pid_next = key_page(gn, 1);
        }
        // (a wait that gives up is told to the others at the vote below)
        const bool late = !mbar_wait(smem_u32(&s.bar_s[buf]), (i >> 1) & 1, p.err);
        __syncwarp();
        tc_fence_after();
        float y[NC];
        {
          const uint32_t a = tmem + lanes + kS + buf * kQN + hb;
          uint32_t v0[NC], v1[NC];
          tmem_issue_ld(a, v0);
          if (QP == 2) tmem_issue_ld(a + NR, v1);
          tmem_wait_ld();
          after_wait(v0);
          if (QP == 2) after_wait(v1);
#pragma unroll
          for (int h = 0; h < NC; ++h)
            y[h] = QP == 2 ? fmaf(__uint_as_float(v1[h]), kLoDown, __uint_as_float(v0[h])) : __uint_as_float(v0[h]);
        }
        tc_fence_before();
        warp_arrive(smem_u32(&s.bar_s_free[buf]), lane);
        const float lg = ROWSCALE ? __log2f(sr) : 0.f, lgc = ROWSCALE ? fmaxf(lg, kLeastLg) : 0.f;
        float ymax = -INFINITY;
#pragma unroll
        for (int h = 0; h < NC; ++h) y[h] = fmaf(y[h], ROWSCALE ? sr * s.cs[hb + h] : s.cs[hb + h], s.negm[hb + h]);
        const int key = (g.j0 + j) * kBK + r;
        const bool edge = (g.j0 + j + 1) * kBK > g.pos1;  // some row's keys end in this block (or before it)
        if (edge) {
#pragma unroll
          for (int h = 0; h < NC; ++h)
            if (key >= s.nk[hb + h]) y[h] = -INFINITY;
        }
#pragma unroll
        for (int h = 0; h < NC; ++h) ymax = fmaxf(ymax, y[h]);
        if (named_bar_or(1, kSoftThreads, late || j == 0 || ymax + lgc > kTau)) {
          if (named_bar_or(1, kSoftThreads, late)) { ok = false; break; }
          // Rows whose largest exceeds their reference by 2^15 (all of them in
          // the first block) get a new one, and their sums and O^T columns
          // are rescaled.
          int mine = kOrdMin;
#pragma unroll
          for (int h = 0; h < NC; ++h) {
            const int m = __reduce_max_sync(0xffffffffu, ord_int(y[h] + lgc));
            if (lane == h) mine = m;
          }
          if (lane < NC) atomicMax(&s.mx[hb + lane], mine);
          named_bar_sync(1, kSoftThreads);
          if ((warp & 3) == 0 && lane < NC) {
            const int hh = hb + lane;
            const float t = ord_float(s.mx[hh]);
            s.mx[hh] = kOrdMin;
            float d = 0.f, f = 1.f;
            if ((j == 0 || t > kTau) && t > -INFINITY) {  // (a row without keys here keeps 0)
              d = t - kPOffset;
              if (j > 0) f = exp2f(-d);
              s.negm[hh] -= d;
            }
            s.delta[hh] = d;
            s.fac[hh] = f;
          }
          named_bar_sync(1, kSoftThreads);
#pragma unroll
          for (int h = 0; h < NC; ++h) y[h] -= s.delta[hb + h];
          if (j > 0) {
#pragma unroll
            for (int h = 0; h < NC; ++h) lv[h] *= s.fac[hb + h];
            if (!named_bar_and(1, kSoftThreads, wait_pv(i - 1))) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int part = 0; part < 4 * kParts; ++part) {
              const uint32_t a = tmem + lanes + (part / kParts) * kPN + (part % kParts) * NR + hb;
#pragma unroll
              for (int c = 0; c < NC; c += 8) {
                uint32_t v[8];
                tmem_issue_ld(a + c, v);
                tmem_wait_ld();
                after_wait(v);
#pragma unroll
                for (int h = 0; h < 8; ++h) v[h] = __float_as_uint(__uint_as_float(v[h]) * s.fac[hb + c + h]);
                tmem_st8(a + c, v);
              }
            }
            tmem_wait_st();
            tc_fence_before();
            named_bar_sync(1, kSoftThreads);  // all lanes are rescaled before any P is published
          }
        }
        // ---- P^T row r, this thread's rows, in three terms; row sums
        // The sums take the weights themselves, P / scale; where the scale is 0
        // or so small that P may have underflowed (P = 2^(y + lg) has 122 binary
        // places), from the logits instead.
        float isr = ROWSCALE ? 1.f / sr : 1.f;
        if (ROWSCALE && !(sr > 1e-18f)) {
          isr = 0.f;
#pragma unroll
          for (int h = 0; h < NC; ++h) lv[h] += ex2_approx(y[h]);
        }
        uint8_t* p_row = s.kv[slot] + kRopeOff;
        uint16_t t1[NC / 2], t2[NC / 2], t3[NC / 2];
#pragma unroll
        for (int k = 0; k < NC / 2; ++k) {
          const float a = ex2_approx(ROWSCALE ? y[2 * k] + lg : y[2 * k]);
          const float b = ex2_approx(ROWSCALE ? y[2 * k + 1] + lg : y[2 * k + 1]);
          lv[2 * k] = ROWSCALE ? fmaf(a, isr, lv[2 * k]) : lv[2 * k] + a;
          lv[2 * k + 1] = ROWSCALE ? fmaf(b, isr, lv[2 * k + 1]) : lv[2 * k + 1] + b;
          split3(a, b, t1[k], t2[k], t3[k]);
        }
        auto pack = [](const uint16_t* h) { return static_cast<uint32_t>(h[0]) | static_cast<uint32_t>(h[1]) << 16; };
        auto pack4 = [&](const uint16_t* h) { return make_uint4(pack(h), pack(h + 2), pack(h + 4), pack(h + 6)); };
        if constexpr (NR == 64) {
          // the first term in the slot's rotary chunk (read by QK, now dead)
#pragma unroll
          for (int c = 0; c < 2; ++c) *reinterpret_cast<uint4*>(p_row + sw64(r, (hb >> 4) + c)) = pack4(t1 + 8 * c);
        } else if constexpr (NR == 32) {
          // (the third's place was last read by PV(i - 2), which has completed)
          *reinterpret_cast<uint4*>(p_row + sw64(r, hb >> 4)) = pack4(t1);
          *reinterpret_cast<uint4*>(p_row + sw64(r, 2 + (hb >> 4))) = pack4(t2);
          *reinterpret_cast<uint4*>(s.pmore + slot * kPRow + sw64(r, hb >> 4)) = pack4(t3);
        } else {
          *reinterpret_cast<uint2*>(p_row + sw64(r, 0) + hb) = make_uint2(pack(t1), pack(t1 + 2));
          *reinterpret_cast<uint2*>(p_row + sw64(r, 1) + hb) = make_uint2(pack(t2), pack(t2 + 2));
          *reinterpret_cast<uint2*>(p_row + sw64(r, 2) + hb) = make_uint2(pack(t3), pack(t3 + 2));
        }
        if (edge && key >= n_item) {
          // nobody's key: whatever lies there must not meet a weight of 0
          for (int c = (warp >> 2); c < 32; c += 2)
            *reinterpret_cast<uint4*>(s.kv[slot] + (c >> 3) * kChunk + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        const int half = (warp & 3) >> 1;  // of the block's keys
        warp_arrive(smem_u32(&s.bar_p[i & 1][half]), lane);
        if constexpr (NR == 64) {
          // The other two terms of 64 keys have one place, which each half takes in
          // its turn: the first once the block before has been read, the second
          // once the first half has (8 KB more for both do not fit).
          if (half == 0) {
            if (i > 0) wait_pv(i - 1);
          } else {
            mbar_wait(smem_u32(&s.bar_empty[slot][0]), (i / kNST) & 1, p.err);
          }
          const int kr = r & (kHalf - 1);
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            *reinterpret_cast<uint4*>(s.pmore + sw64(kr, (hb >> 4) + c)) = pack4(t2 + 8 * c);
            *reinterpret_cast<uint4*>(s.pmore + kPRow / 2 + sw64(kr, (hb >> 4) + c)) = pack4(t3 + 8 * c);
          }
          fence_proxy_async_smem();
          warp_arrive(smem_u32(&s.bar_more[half]), lane);
        }
      }
      if (!ok) break;
      gb += g.nb;
      // ---- row sums over the key lanes, in an order that never changes
      // halving exchanges: lane l ends with the sum of row hb + l % NC
#pragma unroll
      for (int step = NC / 2; step >= 1; step >>= 1) {
        const bool upper = (lane & step) != 0;
#pragma unroll
        for (int h = 0; h < step; ++h) {
          const float send = upper ? lv[h] : lv[h + step];
          const float keep = upper ? lv[h + step] : lv[h];
          lv[h] = keep + __shfl_xor_sync(0xffffffffu, send, step);
        }
      }
#pragma unroll
      for (int o = NC; o < 32; o <<= 1) lv[0] += __shfl_xor_sync(0xffffffffu, lv[0], o);
      if (lane < NC) s.sums[warp & 3][hb + lane] = lv[0];
      named_bar_sync(1, kSoftThreads);
      float* linv = s.fac;
      // the next segment's q while this one's last PV runs
      float l_row = 0.f, ref_row = 0.f;
      if (threadIdx.x < NR) {
        l_row = (s.sums[0][threadIdx.x] + s.sums[1][threadIdx.x]) + (s.sums[2][threadIdx.x] + s.sums[3][threadIdx.x]);
        ref_row = s.negm[threadIdx.x];
      }
      if (has_next && !convert_q(gn)) { ok = false; break; }
      const bool done = named_bar_and(1, kSoftThreads, wait_pv(gb - 1));
      const int part = static_cast<int>(blockIdx.x) * 2 + (g.j0 == 0 ? 1 : 0);
      if (threadIdx.x < NR) {
        float l = l_row;
        if (g.whole) {
          if (p.sink && threadIdx.x < g.rows) {
            const int head = p.groups > 1 ? g.h0 + threadIdx.x : threadIdx.x % p.H;
            l += exp2f(fmaf(p.sink[head], kLog2e, ref_row));
          }
        } else if (threadIdx.x < g.rows) {
          p.part_lse[static_cast<int64_t>(part) * NR + threadIdx.x] = l == 0.f ? -INFINITY : log2f(l) - ref_row;
        }
        linv[threadIdx.x] = l_row == 0.f ? 0.f : 1.f / l;
      }
      named_bar_sync(1, kSoftThreads);
      if (done) {
        tc_fence_after();
        const int64_t row0 = static_cast<int64_t>(g.t0) * p.H + g.h0;
        const bool odd = lane & 1;
#pragma unroll 1
        for (int tile = 0; tile < 4; ++tile) {
          float o[NC];
          const uint32_t a = tmem + lanes + tile * kPN + hb;
#pragma unroll
          for (int c = 0; c < NC; c += 8) {
            uint32_t v[kParts][8];
#pragma unroll
            for (int k = 0; k < kParts; ++k) tmem_issue_ld(a + k * NR + c, v[k]);
            tmem_wait_ld();
#pragma unroll
            for (int k = 0; k < kParts; ++k) after_wait(v[k]);
#pragma unroll
            for (int h = 0; h < 8; ++h) {
              o[c + h] = __uint_as_float(v[kParts - 1][h]);  // the small terms first
#pragma unroll
              for (int k = kParts - 2; k >= 0; --k) o[c + h] += __uint_as_float(v[k][h]);
            }
          }
          if (!g.whole) {
            float* po = p.part_o + (static_cast<int64_t>(part) * NR + hb) * kDV + tile * 128 + r;
#pragma unroll
            for (int h = 0; h < NC; ++h)
              if (hb + h < g.rows) po[h * kDV] = o[h] * linv[hb + h];
          } else {
            // lane pairs swap one value per two rows, so that each stores two
            // neighbouring columns of one row
            uint32_t* o2 = reinterpret_cast<uint32_t*>(p.out + row0 * kDV + tile * 128 + (r & ~1));
#pragma unroll
            for (int h = 0; h < NC; h += 2) {
              const float va = o[h] * linv[hb + h], vb = o[h + 1] * linv[hb + h + 1];
              const float got = __shfl_xor_sync(0xffffffffu, odd ? va : vb, 1);
              const __nv_bfloat162 pr = odd ? __floats2bfloat162_rn(got, vb) : __floats2bfloat162_rn(va, got);
              const int row = hb + h + (odd ? 1 : 0);
              if (row < g.rows) o2[static_cast<int64_t>(row) * (kDV / 2)] = *reinterpret_cast<const uint32_t*>(&pr);
            }
          }
        }
      } else {
        ok = false;
      }
      tc_fence_before();
      named_bar_sync(1, kSoftThreads);  // O^T and linv are read before the next segment writes them
      more = has_next;
      cur = cn;
      g = gn;
    }
  } else if (warp == kTmaWarp) {
    // ============================================================= key blocks
    // A block's keys come in parts of a page, up to 64 keys each: five boxes a
    // part (four 128-byte columns, one of 64), all issued by one lane with the
    // part's page handed to it (boxes spread over the lanes are issued one
    // lane at a time, at 200 cycles a box).  Lane k reads part k's page, one
    // block ahead.
    const bool leader = elect_one();
    const int box = min(1 << p.seqs.page_shift, kBK / 2);
    const int half_parts = (kBK / 2) / box;
    const auto parts_of = [&](const Seg& g, int j) {  // parts with keys in them
      return (min(kBK, max(0, seg_keys(g) - (g.j0 + j) * kBK)) + box - 1) / box;
    };
    // the first physical row of the lane's part of block j
    const auto read_row = [&](const Seg& g, int j) -> int {
      const int key = (g.j0 + j) * kBK + lane * box;
      if (lane >= parts_of(g, j)) return 0;
      const int pg = p.seqs.page_table[static_cast<int64_t>(g.b) * p.seqs.max_pages + (key >> p.seqs.page_shift)];
      const int64_t row = (static_cast<int64_t>(pg) << p.seqs.page_shift) | (key & ((1 << p.seqs.page_shift) - 1));
      // (rows past the pool's end, where a page hangs over it, arrive as zeros)
      if (pg < 0 || row + min(box, seg_keys(g) - key) > p.phys_rows) {
        atomicOr(p.err, kErrPage);
        if (pg < 0 || row >= p.phys_rows) return 0;
      }
      return static_cast<int>(row);
    };
    Cursor cur = start;
    Seg g, gn;
    int i = 0;
    bool ok = true, more = next_seg(p, cur, g);
    // the first segment's q ahead of the keys (behind the first two blocks of
    // every CTA it took 3 us); the QK warp requests the others
    if (leader && more) load_q(g);
    __syncwarp();
    int row = more ? read_row(g, 0) : 0, row_n = 0;
    while (ok && more) {
      more = next_seg(p, cur, gn);
      for (int j = 0; ok && j < g.nb; ++j) {
        if (j + 1 < g.nb)
          row_n = read_row(g, j + 1);
        else if (more)
          row_n = read_row(gn, 0);
        const int slot = i % kNST, parts = parts_of(g, j);
        const uint32_t bar = smem_u32(&s.bar_full[slot]);
        const uint32_t dst = smem_u32(s.kv[slot]);
        const uint32_t par = ((i / kNST) & 1) ^ 1;
        const auto load = [&](int k, int y) {  // part k's keys
          const uint32_t d = dst + k * box * 128;
          tma_load_2d(d, &tk, 0, y, bar);
          tma_load_2d(d + kChunk, &tk, 128, y, bar);
          tma_load_2d(d + 2 * kChunk, &tk, 256, y, bar);
          tma_load_2d(d + 3 * kChunk, &tk, 384, y, bar);
          tma_load_2d(dst + kRopeOff + k * box * 64, &tr, 512, y, bar);
        };
        const int y0 = __shfl_sync(0xffffffffu, row, 0), y1 = __shfl_sync(0xffffffffu, row, 1);
        if (parts == 2 && half_parts == 1) {
          // two pages (the usual case), straight from one thread
          int done = 0;
          if (leader) {
            ok = mbar_wait(smem_u32(&s.bar_empty[slot][0]), par, p.err);
            if (ok) {
              done = 1;
              mbar_arrive_expect_tx(bar, 2 * box * kD);
              load(0, y0);
              // the second half of the keys once PV has given it back
              ok = mbar_wait(smem_u32(&s.bar_empty[slot][1]), par, p.err);
              if (ok) load(1, y1);
            }
          }
          ok = __all_sync(0xffffffffu, ok);
          i += __any_sync(0xffffffffu, done) ? 1 : 0;
          row = row_n;
          continue;
        }
        if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&s.bar_empty[slot][0]), par, p.err))) { ok = false; break; }
        if (leader) {
          if (parts > 0)
            mbar_arrive_expect_tx(bar, parts * box * kD);
          else
            mbar_arrive(bar);
        }
        for (int k = 0; k < parts; ++k) {
          if (k == half_parts &&
              !__all_sync(0xffffffffu, mbar_wait(smem_u32(&s.bar_empty[slot][1]), par, p.err))) {
            ok = false;
            break;
          }
          const int y = __shfl_sync(0xffffffffu, row, k);
          if (leader) load(k, y);
          __syncwarp();
        }
        ++i;
        row = row_n;
      }
      g = gn;
    }
    // nothing is still landing when the CTA ends
    for (int sl = 0; sl < kNST; ++sl) {
      const int loads = (i + kNST - 1 - sl) / kNST;
      if (loads > 0) mbar_wait(smem_u32(&s.bar_full[sl]), (loads - 1) & 1, p.err);
    }
  } else if (warp == kQkWarp) {
    // ============================================================== q and QK
    Cursor cur = start;
    Seg g;
    const bool leader = elect_one();
    constexpr uint32_t IDESC = idesc_e4m3_f32(kBK, kQN, 0, 0);
    const uint64_t ka = make_sdesc(smem_u32(s.kv[0]), 16, 1024, kSwizzle128B);
    const uint64_t kr = make_sdesc(smem_u32(s.kv[0]) + kRopeOff, 16, 512, kSwizzle64B);
    const uint64_t qa = make_sdesc(smem_u32(s.q), 16, 1024, kSwizzle128B);
    const uint64_t qr = make_sdesc(smem_u32(s.q) + 4 * kQChunk, 16, 512, kSwizzle64B);
    int i = 0, nq = 0;
    bool ok = true;
    while (ok && next_seg(p, cur, g)) {
      // the segment's q rows: every QK before has completed (waited for below)
      if (leader && nq > 0) load_q(g);
      __syncwarp();
      ++nq;
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&s.bar_q), (nq - 1) & 1, p.err));
      for (int j = 0; ok && j < g.nb; ++j, ++i) {
        const int slot = i % kNST, buf = i & 1;
        const bool w = (i < 2 || mbar_wait(smem_u32(&s.bar_s_free[buf]), ((i >> 1) - 1) & 1, p.err)) &&
                       mbar_wait(smem_u32(&s.bar_full[slot]), (i / kNST) & 1, p.err);
        if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
        tc_fence_after();
        if (leader) {
          const uint64_t so = static_cast<uint64_t>(slot * (kSlot >> 4));
          const uint32_t d = tmem + kS + buf * kQN;
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              mma_f8f6f4_ss(d, ka + so + static_cast<uint64_t>((c * kChunk + kk * 32) >> 4),
                            qa + static_cast<uint64_t>((c * kQChunk + kk * 32) >> 4), IDESC, (c | kk) ? 1u : 0u);
#pragma unroll
          for (int kk = 0; kk < 2; ++kk)
            mma_f8f6f4_ss(d, kr + so + static_cast<uint64_t>((kk * 32) >> 4), qr + static_cast<uint64_t>((kk * 32) >> 4),
                          IDESC, 1u);
          mma_commit(smem_u32(&s.bar_s[buf]));
        }
        __syncwarp();
      }
      // q's place is free once the segment's last QK has completed
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&s.bar_s[(i - 1) & 1]), ((i - 1) >> 1) & 1, p.err));
    }
    if (leader) mma_commit(smem_u32(&s.bar_drain[0]));
    __syncwarp();
    mbar_wait(smem_u32(&s.bar_drain[0]), 0, p.err);
    if (nq > 0) mbar_wait(smem_u32(&s.bar_qraw), (nq - 1) & 1, p.err);
  } else if (warp == kPvWarp) {
    // ==================================================================== PV
    Cursor cur = start;
    Seg g;
    const bool leader = elect_one();
    constexpr uint32_t IDESC = idesc_e4m3_e5m2_f32(128, kPN, 1, 1);
    const uint64_t va = make_sdesc(smem_u32(s.kv[0]), kChunk, 1024, kSwizzle128B);
    // P^T of each slot.  NR = 32 is 96 columns wide: 64 in the rotary chunk, 32 in
    // the slot's further place.
    const auto p_desc = [&](int slot) {
      const uint32_t a = smem_u32(s.kv[slot]) + kRopeOff;
      return make_sdesc(a, NR == 32 ? smem_u32(s.pmore) + slot * kPRow - a : kPRow, 512, kSwizzle64B);
    };
    const uint64_t p0 = p_desc(0), p1 = p_desc(1);
    const uint64_t pm = make_sdesc(smem_u32(s.pmore), kPRow, 512, kSwizzle64B);
    int i = 0;
    bool ok = true;
    while (ok && next_seg(p, cur, g)) {
      for (int j = 0; ok && j < g.nb; ++j, ++i) {
        const int slot = i % kNST;
        const uint64_t vs = va + static_cast<uint64_t>(slot * (kSlot >> 4)), ps = slot ? p1 : p0;
        // 32 keys (of half h: the kk-th) against a term at pd; `add` to what is there
        const auto pv = [&](int h, int kk, uint64_t pd, bool add) {
#pragma unroll
          for (int tile = 0; tile < 4; ++tile)
            mma_f8f6f4_ss(tmem + tile * kPN,
                          vs + static_cast<uint64_t>((tile * kChunk + (h * kHalf + kk * 32) * 128) >> 4), pd, IDESC,
                          add ? 1u : 0u);
        };
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&s.bar_p[i & 1][h]), (i >> 1) & 1, p.err))) { ok = false; break; }
          tc_fence_after();
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
              pv(h, kk, ps + static_cast<uint64_t>(((h * kHalf + kk * 32) * 64) >> 4), j > 0 || (h | kk));
          }
          __syncwarp();
          if constexpr (NR == 64) {
            if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&s.bar_more[h]), i & 1, p.err))) { ok = false; break; }
            tc_fence_after();
            if (leader) {
#pragma unroll
              for (int term = 0; term < 2; ++term)
#pragma unroll
                for (int kk = 0; kk < 2; ++kk)
                  pv(h, kk, pm + static_cast<uint64_t>((term * (kPRow / 2) + kk * 32 * 64) >> 4), true);
            }
          }
          if (leader) {
            mma_commit(smem_u32(&s.bar_empty[slot][h]));
            if (h == 1) mma_commit(smem_u32(&s.bar_pv[i & 1]));
          }
          __syncwarp();
        }
      }
    }
    if (leader) mma_commit(smem_u32(&s.bar_drain[1]));
    __syncwarp();
    mbar_wait(smem_u32(&s.bar_drain[1]), 0, p.err);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kQkWarp) tmem_dealloc(tmem, kTmemCols);
}

template <int NR, int QP, bool ROWSCALE>
static smla_status_t launch(const DenseDecodeArgs& a, const Params& p, cudaStream_t stream) {
  CUtensorMap tq, tqr, tk, tr;
  const uint64_t q_rows = static_cast<uint64_t>(a.T) * a.H;
  const uint32_t box = std::min(a.seqs->page_size, kBK / 2);
  bool enc = encode_tma_2d_u8(&tk, a.latent, kD, a.phys_rows, 128, box, 128) &&
             encode_tma_2d_u8(&tr, a.latent, kD, a.phys_rows, 64, box, 64) &&
             encode_tma_2d_u8(&tq, a.q, kD * QP, q_rows, 128, NR, 128);
  tqr = tq;
  if (QP == 1) enc = enc && encode_tma_2d_u8(&tqr, a.q, kD, q_rows, 64, NR, 64);
  if (!enc) return fail(SMLA_ERR_CUDA, "cuTensorMapEncodeTiled failed for the dense-decode tensor maps");
  constexpr size_t smem = sizeof(Smem<NR, QP>);
  static_assert(smem <= 232448, "shared memory exceeds a CTA's 227 KB");
  static std::atomic<unsigned long long> ready{0};
  const smla_status_t st = prepare_kernel(reinterpret_cast<const void*>(decode_kernel<NR, QP, ROWSCALE>), smem, 0, ready,
                                          "dense decode kernel");
  if (st != SMLA_OK) return st;
  decode_kernel<NR, QP, ROWSCALE><<<p.grid, kThreads, smem, stream>>>(tq, tqr, tk, tr, p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail_cuda(e, "dense decode launch");
  return launch_join<NR>(p, stream);
}

// Rows of an item: several tokens' while they fit 64 (16 rows cost 1360 cycles
// of MMAs a block, 64 rows 2688).
static int rows_per_item(int T, int B, int H) { return H >= 48 ? 64 : tokens_per_item(T, B, H, 64) * H; }

}  // namespace dd

size_t dense_decode_workspace_bytes(int T, int H, int max_kv_len) {
  using namespace dd;
  const size_t grid = decode_grid(T, H, max_kv_len), nr = rows_per_item(T, 1, H);  // (the most rows any batch of T gives)
  if (grid <= 1) return 0;
  return 2 * grid * nr * (kDV + 1) * sizeof(float) + ((grid * sizeof(Cut) + 255) & ~size_t(255)) + 256;
}

smla_status_t launch_dense_decode(const DenseDecodeArgs& a, unsigned* err, cudaStream_t stream) {
  using namespace dd;
  const int B = a.seqs->B, nr = rows_per_item(a.T, B, a.H), groups = std::max(1, a.H / 64);
  const smla_status_t st = check_line(a, groups, kItemCost);
  if (st != SMLA_OK) return st;
  const Params p = decode_params(a, tokens_per_item(a.T, B, a.H, 64), groups, kItemCost, nr, err);
  const bool bf16 = a.q_dtype == SMLA_BF16, rows = a.scales != nullptr;
  const auto go = [&](auto nr_c) {
    constexpr int NR = decltype(nr_c)::value;
    if (bf16) return rows ? launch<NR, 2, true>(a, p, stream) : launch<NR, 2, false>(a, p, stream);
    return rows ? launch<NR, 1, true>(a, p, stream) : launch<NR, 1, false>(a, p, stream);
  };
  if (nr == 64) return go(std::integral_constant<int, 64>{});
  if (nr == 32) return go(std::integral_constant<int, 32>{});
  return go(std::integral_constant<int, 16>{});
}

}  // namespace smla
