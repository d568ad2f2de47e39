// Dense MLA decode with 16-bit operands: over a bf16 latent cache, and over an
// e4m3 one with block scales (a scale for each 32 columns of a row, so no MMA
// can take the bytes as they lie).
//
//   S^T[128 keys x NR rows] = K . Q^T,   O^T[512 x NR] += V^T . P^T
//
// as in the e4m3 kernel, with kind::f16 MMAs and one term for everything.  A
// bf16 cache: q, K and P in bf16 (P's rounding is up to 2^-8 of a weight).  Block
// scales: f16, a row carried as byte * scale_blk 2^-e with 2^e five binary places
// below its largest scale (the scale and the product are off by up to 2^-11 each;
// e4m3 q is exact); its logits and its weights take 2^e instead, as the e4m3
// kernel does with a row's scale.  The largest product is below 2^15, the upper
// end of f16, so that blocks of much smaller scales keep their bits: those below
// 2^-19 of the largest are multiplied in two steps (see convert), and end at half
// of f16's smallest step, 2^-30 of the largest scale.  The product is one f16x2
// multiply for two elements (through f32 to bf16 it was five instructions: 101 us
// against 85 at 16 heads x 4 x <= 120 K keys).  The line of work, the walk along
// it and the join are shared with the e4m3 kernel.
//
// A block's 128 rows take 147 KB in 16 bits, so there is room for one block and
// a little: eight 64-column chunks as four pairs (a pair is K's columns for QK
// and one 128-column tile of V) in a ring of pairs, and the rotary chunk, which
// P^T reuses after QK.  PV runs tile by tile and hands each pair back, so the
// next block streams in behind it:
//   bf16 cache   TMA loads the pairs; a fifth one ahead where q leaves room.
//   block scales TMA loads the bytes into raw chunks, and the softmax warps,
//                which have nothing else to do until S is there, multiply and
//                round them into the pairs: two groups of four warps, each with
//                the raw slot and the pairs that are its own, so that one
//                group's waits run beside the other's (one group of eight: 103
//                us against 88).  Eight more warps for this alone, beside the
//                softmax, were slower (96-109 us: the registers then spill).
//
// Bound: HBM for a bf16 cache and few rows (147 KB a block, 6260 cycles of an
// SM's share), its tensor and softmax chain for 64 rows; for block scales the
// chain of a block, about 6.5 k cycles, of which raw chunks awaited 1.5 k, read
// 0.6 k, converted and stored 1.7 k, fenced and handed on 1.2 k, softmax 1.4 k.
//
// Measured: 16 heads over 4 x <= 120 K keys, bf16 cache 83 us (5.4 TB/s), block
// scales 79 us (3.2 TB/s); 8 x 2 tokens x 128 heads over <= 8192 keys, bf16 60 us
// (528 TFLOP/s), block scales 94 us.  (The prefill kernel's form with one block
// in flight: 142, 179, 85 and 115 us.)
//
// Warps: 0-7 conversion, softmax and epilogue (thread = one key x NR/2 rows),
// 8 TMA, 9 QK, 10 PV.
#include <cstddef>
#include <type_traits>

#include "decode_line.cuh"

namespace smla {
namespace dw {

using namespace dd;

constexpr int kChunk = kBK * 128;  // 64 columns of a block in bf16 (128 in e4m3)
constexpr int kItemCost = 3;       // an item's fixed cost, in blocks
constexpr float kTinyLg = -60.f;   // rows of smaller scales take their sums from the logits

template <int NR, bool BLOCK>
struct Smem {
  static constexpr int kPairs = BLOCK || NR == 64 ? 4 : 5;
  static constexpr int kRaws = 2;  // one for each group of converting warps, which then keep to their own barriers
  uint8_t q[NR * kD * 2];  // nine chunks [NR][128 bytes]
  uint8_t pair[kPairs][2 * kChunk];
  uint8_t rope[kChunk];    // then P^T [128 keys][128 bytes]
  uint8_t raw[BLOCK ? kRaws * kChunk : 16];
  alignas(1024) uint8_t raw_rope[BLOCK ? kChunk / 2 : 16];
  alignas(16) float negm[NR];  // minus the reference, log2 units
  float delta[NR], fac[NR];
  int mx[NR], bad[NR];         // bad: the next segment's row has a query element that is not finite
  float sums[4][NR];
  int nk[NR];
  int part_row[kBK / 8];
  float smax[BLOCK ? 2 : 1][BLOCK ? kBK : 1];  // largest scale of each half of a row's blocks
  unsigned long long bar_q, bar_pair_full[kPairs], bar_pair_empty[kPairs], bar_rope_full, bar_rope_empty;
  unsigned long long bar_raw_full[kRaws], bar_raw_empty[kRaws], bar_raw_rope_full, bar_raw_rope_empty;
  unsigned long long bar_s[2], bar_s_free[2], bar_p, bar_pv, bar_drain[2];
  uint32_t tmem_base;
};

// 16 e4m3 bytes -> two 16-byte pieces of f16, times a scale.
__device__ __forceinline__ void scaled16(const uint4& u, uint32_t scale2, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = hmul2(e4m3x2_to_f16x2(static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1)))), scale2);
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}
constexpr uint32_t kOneF16x2 = 0x3c003c00u, kDownF16x2 = 0x01000100u;  // 1, 2^-16

template <int NR, bool BLOCK>
__global__ void __launch_bounds__(kThreads, 1)
    decode_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tr,
                  const void* __restrict__ q_rows, const Params p) {
  using S = Smem<NR, BLOCK>;
  constexpr int kPairs = S::kPairs, kRaws = S::kRaws;
  constexpr int kQChunk = NR * 128;
  constexpr int NC = NR / 2;  // rows of a softmax thread
  static_assert(offsetof(S, pair) % 1024 == 0 && offsetof(S, rope) % 1024 == 0 && offsetof(S, raw) % 1024 == 0,
                "swizzled tiles need 1024-byte alignment");
  static_assert(4 * NR <= static_cast<int>(kTmemS) && 2 * NR <= static_cast<int>(kTmemCols - kTmemS), "TMEM budget");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrShape);
    return;
  }
  S& s = *reinterpret_cast<S*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&s.bar_q), kSoftThreads);
    for (int i = 0; i < kPairs; ++i) {
      mbar_init(smem_u32(&s.bar_pair_full[i]), BLOCK ? kSoftWarps / 2 : 1);
      mbar_init(smem_u32(&s.bar_pair_empty[i]), 1);
    }
    mbar_init(smem_u32(&s.bar_rope_full), BLOCK ? kSoftWarps : 1);
    mbar_init(smem_u32(&s.bar_rope_empty), 1);
    for (int i = 0; i < kRaws; ++i) {
      mbar_init(smem_u32(&s.bar_raw_full[i]), 1);
      mbar_init(smem_u32(&s.bar_raw_empty[i]), kSoftWarps / 2);
    }
    mbar_init(smem_u32(&s.bar_raw_rope_full), 1);
    mbar_init(smem_u32(&s.bar_raw_rope_empty), kSoftWarps);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&s.bar_s[i]), 1);
      mbar_init(smem_u32(&s.bar_s_free[i]), kSoftWarps);
      mbar_init(smem_u32(&s.bar_drain[i]), 1);
    }
    mbar_init(smem_u32(&s.bar_p), kSoftWarps);
    mbar_init(smem_u32(&s.bar_pv), 1);
    fence_mbar_init();
  }
  if (threadIdx.x < NR) {
    s.mx[threadIdx.x] = kOrdMin;
    s.bad[threadIdx.x] = 0;
  }
  if (warp == kQkWarp) {
    tmem_alloc(smem_u32(&s.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  if (threadIdx.x == kTmaWarp * 32) {
    tma_prefetch_desc(&tk);
    if (BLOCK) tma_prefetch_desc(&tr);
  }
  const Cursor start = find_part(p, lane);  // this CTA's part of the line
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s.tmem_base;

  if (start.b < 0) {
    // nothing left of the line for this CTA
  } else if (warp < 8) {
    // ========================================= conversion, softmax, epilogue
    const int r = threadIdx.x & 127;    // key lane
    const int half = warp >> 2;
    const int hb = half * NC;           // rows [hb, hb + NC)
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const float cs = p.softmax_scale * kLog2e;
    // The q rows of a segment, those past it zeros.  A row with an infinity has no
    // finite logits; where they are all -inf it would look like one without keys,
    // so such rows are marked, and made NaN.
    auto load_q = [&](const Seg& g) {
      constexpr int kPieces = BLOCK ? kD / 16 : kD / 8;  // 16-byte pieces of a row in memory
      constexpr int kPer = (NR * kPieces + kSoftThreads - 1) / kSoftThreads, kBatch = 9;
      const uint4* src = static_cast<const uint4*>(q_rows) + (static_cast<int64_t>(g.t0) * p.H + g.h0) * kPieces;
#pragma unroll 1
      for (int k0 = 0; k0 < kPer; k0 += kBatch) {
        uint4 v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int i = threadIdx.x + (k0 + k) * kSoftThreads;
          v[k] = i < g.rows * kPieces ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int i = threadIdx.x + (k0 + k) * kSoftThreads, row = i / kPieces, pc = i - row * kPieces;
          if (row >= NR) continue;
          if (BLOCK) {
            uint4 a, b;
            scaled16(v[k], kOneF16x2, a, b);
            *reinterpret_cast<uint4*>(s.q + (pc >> 2) * kQChunk + sw128(row, (pc & 3) * 2)) = a;
            *reinterpret_cast<uint4*>(s.q + (pc >> 2) * kQChunk + sw128(row, (pc & 3) * 2 + 1)) = b;
          } else {
            *reinterpret_cast<uint4*>(s.q + (pc >> 3) * kQChunk + sw128(row, pc & 7)) = v[k];
            // exponents of all ones, of two elements a word
            const auto full = [](uint32_t w) { return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u; };
            if (full(v[k].x) | full(v[k].y) | full(v[k].z) | full(v[k].w)) s.bad[row] = 1;
          }
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(smem_u32(&s.bar_q));
    };
    // Page of the thread's key of block j (-1 outside the keys), and the nine of
    // its row's scales that this half of the warps converts with (1 there, and
    // on a bad page, which the TMA warp reports): those of pairs half and half
    // + 2, and 16 + half of the rotary chunk.  Read two blocks and one ahead.
    auto key_page = [&](const Seg& g, int j) -> int {
      const int key = (g.j0 + j) * kBK + r;
      return BLOCK && key < seg_keys(g)
                 ? p.seqs.page_table[static_cast<int64_t>(g.b) * p.seqs.max_pages + (key >> p.seqs.page_shift)]
                 : -1;
    };
    float sc[9];
    auto key_scales = [&](const Seg& g, int j, int pid) {
      if (!BLOCK) return;
      const int key = (g.j0 + j) * kBK + r;
      const int64_t row = (static_cast<int64_t>(pid) << p.seqs.page_shift) | (key & ((1 << p.seqs.page_shift) - 1));
      const bool bad = pid < 0 || row >= p.phys_rows;
      const float* src = p.scales + (bad ? 0 : row * 18);
#pragma unroll
      for (int k = 0; k < 9; ++k) sc[k] = bad ? 1.f : src[k < 8 ? (k >> 2) * 8 + 4 * half + (k & 3) : 16 + half];
    };
    const uint32_t nil = static_cast<uint32_t>(p.grid) >> 16;  // 0
    // Block i's bytes to f16; `ex` receives the row's exponent.  Pairs 0 and 2
    // are the first four warps' work, 1 and 3 the others', so that one group's
    // latencies run beside the other's; the rotary chunk is shared.
    auto convert = [&](int i, int& ex) -> bool {
      bool fine = true;
      float most = 0.f;
#pragma unroll
      for (int k = 0; k < 9; ++k) most = fmaxf(most, fabsf(sc[k]));
      s.smax[half][r] = most;
      named_bar_sync(2 + (warp & 3), 64);
      ex = min(max(static_cast<int>(__float_as_uint(fmaxf(most, s.smax[half ^ 1][r])) >> 23) - 5, 1), 253);
      const float down = __uint_as_float(static_cast<uint32_t>(254 - ex) << 23);  // 2^(127 - ex)
      // A scale that f16 would round as a subnormal is taken 2^16 larger, and the
      // products of its block are brought down again: then nothing but the
      // products themselves can be subnormal.  (The branch alone costs 32 rows 89
      // -> 94 us, 16 rows 78.5 -> 79.0; without it such blocks lose a bit for each
      // factor of two.)
      uint32_t s2[5], deep = 0;  // two scales a word
#pragma unroll
      for (int k = 0; k < 9; k += 2) {
        float f[2] = {sc[k] * down, k < 8 ? sc[k + 1] * down : 1.f};
#pragma unroll
        for (int u = 0; u < 2; ++u)
          if (fabsf(f[u]) < 0x1p-14f) {
            f[u] *= 0x1p16f;
            deep |= 1u << (k + u);
          }
        s2[k >> 1] = f32x2_to_f16x2(f[0], f[1]);
      }
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const bool nope = k < 2;
        const int n = 4 * i + half + 2 * k, rs = half, sl = n % kPairs;  // the pair (k < 2)
        const int par = nope ? (n / kRaws) & 1 : i & 1;
        fine = mbar_wait(nope ? smem_u32(&s.bar_raw_full[rs]) : smem_u32(&s.bar_raw_rope_full), par, p.err) && fine;
        uint4 u[8];
        uint32_t seen = 0;
#pragma unroll
        for (int c = 0; c < (nope ? 8 : 2); ++c) {
          u[c] = *reinterpret_cast<const uint4*>(nope ? s.raw + rs * kChunk + sw128(r, c) : s.raw_rope + sw64(r, half * 2 + c));
          seen |= u[c].x;
        }
        // The raw chunk goes back once the reads have returned.  The arrival takes
        // every lane's values (against a 0 that the compiler does not know): one
        // that only follows the reads in the program may overtake them while the
        // tensor cores keep shared memory busy, and TMA then writes what is still
        // to be read.
        const uint32_t none = __any_sync(0xffffffffu, (seen & nil) != 0) ? 8u : 0u;  // 0
        warp_arrive((nope ? smem_u32(&s.bar_raw_empty[rs]) : smem_u32(&s.bar_raw_rope_empty)) + none, lane);
        fine = (nope ? mbar_wait(smem_u32(&s.bar_pair_empty[sl]), ((n / kPairs) & 1) ^ 1, p.err)
                     : mbar_wait(smem_u32(&s.bar_rope_empty), (i & 1) ^ 1, p.err)) && fine;
#pragma unroll
        for (int c = 0; c < (nope ? 8 : 2); ++c) {
          uint4 a, b;
          const int blk = nope ? 4 * k + (c >> 1) : 8;
          scaled16(u[c], __byte_perm(s2[blk >> 1], 0, blk & 1 ? 0x3232 : 0x1010), a, b);
          uint8_t* dst = nope ? s.pair[sl] + (c >> 2) * kChunk : s.rope;
          const int piece = nope ? (c & 3) * 2 : half * 4 + 2 * c;
          *reinterpret_cast<uint4*>(dst + sw128(r, piece)) = a;
          *reinterpret_cast<uint4*>(dst + sw128(r, piece + 1)) = b;
        }
        if (__builtin_expect((deep & (nope ? 0xfu << (4 * k) : 0x100u)) != 0, 0)) {
#pragma unroll 1
          for (int c = 0; c < (nope ? 16 : 4); ++c) {  // 16-byte pieces, four a block
            if (!(deep >> (nope ? 4 * k + (c >> 2) : 8) & 1)) continue;
            uint8_t* dst = nope ? s.pair[sl] + (c >> 3) * kChunk : s.rope;
            uint4& v = *reinterpret_cast<uint4*>(dst + sw128(r, nope ? c & 7 : half * 4 + c));
            v = make_uint4(hmul2(v.x, kDownF16x2), hmul2(v.y, kDownF16x2), hmul2(v.z, kDownF16x2), hmul2(v.w, kDownF16x2));
          }
        }
        fence_proxy_async_smem();
        warp_arrive(nope ? smem_u32(&s.bar_pair_full[sl]) : smem_u32(&s.bar_rope_full), lane);
      }
      return fine;
    };
    Cursor cur = start;
    Seg g;
    bool ok = next_seg(p, cur, g);
    int pid_next = -1;
    if (ok) {
      key_scales(g, 0, key_page(g, 0));
      if (g.nb > 1) pid_next = key_page(g, 1);
      load_q(g);
      named_bar_sync(1, kSoftThreads);  // every row's mark is there
    }
    int gb = 0;  // blocks of the segments before
    bool more = ok;
    while (ok && more) {
      const int n_item = seg_keys(g);
      if (threadIdx.x < NR) {
        s.negm[threadIdx.x] = s.bad[threadIdx.x] ? NAN : 0.f;  // the first block sets the reference
        s.bad[threadIdx.x] = 0;
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
        const int i = gb + j, buf = i & 1;
        // (a wait that gives up is told to the others at the vote below)
        bool late = false;
        int ex = 127;
        if (BLOCK) {
          late = !convert(i, ex);
          if (j + 1 < g.nb) {
            key_scales(g, j + 1, pid_next);
            if (j + 2 < g.nb) pid_next = key_page(g, j + 2);
          } else if (has_next) {
            key_scales(gn, 0, key_page(gn, 0));
            if (gn.nb > 1) pid_next = key_page(gn, 1);
          }
        }
        late = !mbar_wait(smem_u32(&s.bar_s[buf]), (i >> 1) & 1, p.err) || late;
        __syncwarp();
        tc_fence_after();
        // the row was carried as K 2^-lg: its logits take 2^lg, and so do its weights
        const float lg = BLOCK ? static_cast<float>(ex - 127) : 0.f, lgc = fmaxf(lg, kLeastLg);
        const float csr = BLOCK ? cs * __uint_as_float(static_cast<uint32_t>(ex) << 23) : cs;
        float y[NC];
        {
          uint32_t v[NC];
          tmem_issue_ld(tmem + lanes + kTmemS + buf * NR + hb, v);
          tmem_wait_ld();
          after_wait(v);
#pragma unroll
          for (int h = 0; h < NC; ++h) y[h] = fmaf(__uint_as_float(v[h]), csr, s.negm[hb + h]);
        }
        tc_fence_before();
        warp_arrive(smem_u32(&s.bar_s_free[buf]), lane);
        float ymax = -INFINITY;
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
            // (P has one place, so PV(i - 1) has long completed)
            if (!named_bar_and(1, kSoftThreads, mbar_wait(smem_u32(&s.bar_pv), (i - 1) & 1, p.err))) { ok = false; break; }
            tc_fence_after();
#pragma unroll 1
            for (int tile = 0; tile < 4; ++tile) {
              const uint32_t a = tmem + lanes + tile * NR + hb;
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
        // ---- P^T row r, this thread's rows, in the rotary chunk's place; row
        // sums from the f32 weights
        float isr = BLOCK ? __uint_as_float(static_cast<uint32_t>(254 - ex) << 23) : 1.f;  // 2^-lg
        if (BLOCK && lg < kTinyLg) {  // P may have underflowed: the sums from the logits
          isr = 0.f;
#pragma unroll
          for (int h = 0; h < NC; ++h) lv[h] += ex2_approx(y[h]);
        }
#pragma unroll
        for (int c = 0; c < NC / 8; ++c) {
          uint32_t w[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float a = y[8 * c + 2 * k], b = y[8 * c + 2 * k + 1];
            a = ex2_approx(BLOCK ? a + lg : a);
            b = ex2_approx(BLOCK ? b + lg : b);
            lv[8 * c + 2 * k] = BLOCK ? fmaf(a, isr, lv[8 * c + 2 * k]) : lv[8 * c + 2 * k] + a;
            lv[8 * c + 2 * k + 1] = BLOCK ? fmaf(b, isr, lv[8 * c + 2 * k + 1]) : lv[8 * c + 2 * k + 1] + b;
            if (BLOCK) {
              w[k] = f32x2_to_f16x2(a, b);
            } else {
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(a, b);
              w[k] = *reinterpret_cast<const uint32_t*>(&b2);
            }
          }
          *reinterpret_cast<uint4*>(s.rope + sw128(r, hb / 8 + c)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        if (edge && key >= n_item) {
          // nobody's key: whatever lies there must not meet a weight of 0
          for (int c = half; c < 64; c += 2)
            *reinterpret_cast<uint4*>(s.pair[(4 * i + (c >> 4)) % kPairs] + ((c >> 3) & 1) * kChunk + r * 128 + (c & 7) * 16) =
                make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        warp_arrive(smem_u32(&s.bar_p), lane);
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
      float l_row = 0.f, ref_row = 0.f;
      if (threadIdx.x < NR) {
        l_row = (s.sums[0][threadIdx.x] + s.sums[1][threadIdx.x]) + (s.sums[2][threadIdx.x] + s.sums[3][threadIdx.x]);
        ref_row = s.negm[threadIdx.x];
      }
      // the next segment's q while this one's last PV runs (its QKs are done)
      if (has_next) load_q(gn);
      const bool done = named_bar_and(1, kSoftThreads, mbar_wait(smem_u32(&s.bar_pv), (gb - 1) & 1, p.err));
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
          const uint32_t a = tmem + lanes + tile * NR + hb;
#pragma unroll
          for (int c = 0; c < NC; c += 8) {
            uint32_t v[8];
            tmem_issue_ld(a + c, v);
            tmem_wait_ld();
            after_wait(v);
#pragma unroll
            for (int h = 0; h < 8; ++h) o[c + h] = __uint_as_float(v[h]);
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
    // A block's keys come in parts of a page, up to 64 keys each; lane k reads
    // part k's page, one block ahead; one lane issues every box.
    const bool leader = elect_one();
    const int box = min(1 << p.seqs.page_shift, kBK / 2);
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
    int n_pair = 0, n_rope = 0;
    bool ok = true, more = next_seg(p, cur, g);
    int row = more ? read_row(g, 0) : 0, row_n = 0;
    while (ok && more) {
      more = next_seg(p, cur, gn);
      for (int j = 0; ok && j < g.nb; ++j) {
        if (j + 1 < g.nb)
          row_n = read_row(g, j + 1);
        else if (more)
          row_n = read_row(gn, 0);
        const int parts = parts_of(g, j);
        // chunk t of the block: its barriers and place
        const auto place = [&](int t, uint32_t& empty, uint32_t& full, uint32_t& dst, uint32_t& par) {
          if (t < 4) {
            const int sl = n_pair % kPairs, rs = n_pair % kRaws;
            empty = BLOCK ? smem_u32(&s.bar_raw_empty[rs]) : smem_u32(&s.bar_pair_empty[sl]);
            full = BLOCK ? smem_u32(&s.bar_raw_full[rs]) : smem_u32(&s.bar_pair_full[sl]);
            dst = BLOCK ? smem_u32(s.raw) + rs * kChunk : smem_u32(s.pair[sl]);
            par = ((n_pair / (BLOCK ? kRaws : kPairs)) & 1) ^ 1;
          } else {
            empty = BLOCK ? smem_u32(&s.bar_raw_rope_empty) : smem_u32(&s.bar_rope_empty);
            full = BLOCK ? smem_u32(&s.bar_raw_rope_full) : smem_u32(&s.bar_rope_full);
            dst = BLOCK ? smem_u32(s.raw_rope) : smem_u32(s.rope);
            par = (n_rope & 1) ^ 1;
          }
        };
        const auto requested = [&](int t) {
          if (t < 4)
            ++n_pair;
          else
            ++n_rope;
        };
        const auto load = [&](int t, uint32_t dst, int y, uint32_t full) {  // one part's keys
          if (BLOCK) {
            if (t < 4)
              tma_load_2d(dst, &tk, t * 128, y, full);
            else
              tma_load_2d(dst, &tr, 512, y, full);
          } else {
            tma_load_2d(dst, &tk, t * 256, y, full);
            if (t < 4) tma_load_2d(dst + kChunk, &tk, t * 256 + 128, y, full);
          }
        };
        // bytes of a key in chunk t, and in a row of its place
        const auto width = [](int t) { return BLOCK ? (t < 4 ? 128 : 64) : (t < 4 ? 256 : 128); };
        const auto pitch = [](int t) { return BLOCK && t == 4 ? 64 : 128; };
        // straight from one thread (out of a loop with shuffles a box took 220
        // cycles), which finds the parts' rows in shared memory.  Not unrolled:
        // with block scales the roles' code together is more than the
        // instruction cache holds well (unrolled, 92 us against 84).
        if (lane < parts) s.part_row[lane] = row;
        __syncwarp();
        if (leader) {
          const int y0 = s.part_row[0], y1 = s.part_row[1];
#pragma unroll 1
          for (int t = 0; t < 5; ++t) {
            uint32_t empty, full, dst, par;
            place(t, empty, full, dst, par);
            ok = ok && mbar_wait(empty, par, p.err);
            if (!ok) break;
            requested(t);
            if (parts == 0) {
              mbar_arrive(full);
              continue;
            }
            mbar_arrive_expect_tx(full, parts * box * width(t));
            load(t, dst, y0, full);
            if (parts > 1) load(t, dst + box * pitch(t), y1, full);
#pragma unroll 1
            for (int k = 2; k < parts; ++k) load(t, dst + k * box * pitch(t), s.part_row[k], full);
          }
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!leader) {
#pragma unroll
          for (int t = 0; t < 5; ++t) requested(t);
        }
        row = row_n;
      }
      g = gn;
    }
    // nothing is still landing when the CTA ends
    if (leader) {
      constexpr int kRing = BLOCK ? kRaws : kPairs;
      for (int sl = 0; sl < kRing; ++sl) {
        const int loads = (n_pair + kRing - 1 - sl) / kRing;
        if (loads > 0)
          mbar_wait(BLOCK ? smem_u32(&s.bar_raw_full[sl]) : smem_u32(&s.bar_pair_full[sl]), (loads - 1) & 1, p.err);
      }
      if (n_rope > 0)
        mbar_wait(BLOCK ? smem_u32(&s.bar_raw_rope_full) : smem_u32(&s.bar_rope_full), (n_rope - 1) & 1, p.err);
    }
    __syncwarp();
  } else if (warp == kQkWarp) {
    // ==================================================================== QK
    Cursor cur = start;
    Seg g;
    const bool leader = elect_one();
    constexpr uint32_t IDESC = BLOCK ? idesc_f16_f32(kBK, NR, 0, 0) : idesc_bf16_f32(kBK, NR, 0, 0);
    const uint64_t ka = make_sdesc(smem_u32(s.pair[0]), 16, 1024, kSwizzle128B);
    const uint64_t kr = make_sdesc(smem_u32(s.rope), 16, 1024, kSwizzle128B);
    const uint64_t qa = make_sdesc(smem_u32(s.q), 16, 1024, kSwizzle128B);
    int i = 0, nq = 0;
    bool ok = true;
    while (ok && next_seg(p, cur, g)) {
      ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&s.bar_q), nq++ & 1, p.err));
      for (int j = 0; ok && j < g.nb; ++j, ++i) {
        const int buf = i & 1;
        const uint32_t d = tmem + kTmemS + buf * NR;
        ok = __all_sync(0xffffffffu, i < 2 || mbar_wait(smem_u32(&s.bar_s_free[buf]), ((i >> 1) - 1) & 1, p.err));
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int n = 4 * i + t, sl = n % kPairs;
          ok = ok && __all_sync(0xffffffffu, mbar_wait(smem_u32(&s.bar_pair_full[sl]), (n / kPairs) & 1, p.err));
          if (!ok) break;
          tc_fence_after();
          if (leader) {
            const uint64_t a = ka + static_cast<uint64_t>(sl * (2 * kChunk >> 4));
#pragma unroll
            for (int c = 0; c < 2; ++c)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_f16_ss(d, a + static_cast<uint64_t>((c * kChunk + kk * 32) >> 4),
                           qa + static_cast<uint64_t>(((2 * t + c) * kQChunk + kk * 32) >> 4), IDESC,
                           (t | c | kk) ? 1u : 0u);
          }
          __syncwarp();
        }
        ok = ok && __all_sync(0xffffffffu, mbar_wait(smem_u32(&s.bar_rope_full), i & 1, p.err));
        if (!ok) break;
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f16_ss(d, kr + static_cast<uint64_t>((kk * 32) >> 4), qa + static_cast<uint64_t>((8 * kQChunk + kk * 32) >> 4),
                       IDESC, 1u);
          mma_commit(smem_u32(&s.bar_s[buf]));
        }
        __syncwarp();
      }
    }
    if (leader) mma_commit(smem_u32(&s.bar_drain[0]));
    __syncwarp();
    mbar_wait(smem_u32(&s.bar_drain[0]), 0, p.err);
  } else if (warp == kPvWarp) {
    // ==================================================================== PV
    Cursor cur = start;
    Seg g;
    const bool leader = elect_one();
    constexpr uint32_t IDESC = BLOCK ? idesc_f16_f32(128, NR, 1, 1) : idesc_bf16_f32(128, NR, 1, 1);
    const uint64_t va = make_sdesc(smem_u32(s.pair[0]), kChunk, 1024, kSwizzle128B);
    const uint64_t pa = make_sdesc(smem_u32(s.rope), kChunk, 1024, kSwizzle128B);
    int i = 0;
    bool ok = true;
    while (ok && next_seg(p, cur, g)) {
      for (int j = 0; ok && j < g.nb; ++j, ++i) {
        ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&s.bar_p), i & 1, p.err));
        if (!ok) break;
        tc_fence_after();
        if (leader) {
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const int sl = (4 * i + t) % kPairs;
            const uint64_t a = va + static_cast<uint64_t>(sl * (2 * kChunk >> 4));
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)  // 16 keys
              mma_f16_ss(tmem + t * NR, a + static_cast<uint64_t>((kk * 16 * 128) >> 4),
                         pa + static_cast<uint64_t>((kk * 16 * 128) >> 4), IDESC, (j > 0 || kk > 0) ? 1u : 0u);
            mma_commit(smem_u32(&s.bar_pair_empty[sl]));  // the tile's columns are free
          }
          mma_commit(smem_u32(&s.bar_rope_empty));
          mma_commit(smem_u32(&s.bar_pv));
        }
        __syncwarp();
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

template <int NR, bool BLOCK>
static smla_status_t launch(const DenseDecodeArgs& a, const Params& p, cudaStream_t stream) {
  CUtensorMap tk, tr;
  const uint32_t box = std::min(a.seqs->page_size, kBK / 2);
  bool enc = encode_tma_2d_u8(&tk, a.latent, BLOCK ? kD : 2 * kD, a.phys_rows, 128, box, 128);
  tr = tk;
  if (BLOCK) enc = enc && encode_tma_2d_u8(&tr, a.latent, kD, a.phys_rows, 64, box, 64);
  if (!enc) return fail(SMLA_ERR_CUDA, "cuTensorMapEncodeTiled failed for the dense-decode tensor maps");
  constexpr size_t smem = sizeof(Smem<NR, BLOCK>);
  static_assert(smem <= 232448, "shared memory exceeds a CTA's 227 KB");
  static std::atomic<unsigned long long> ready{0};
  const smla_status_t st = prepare_kernel(reinterpret_cast<const void*>(decode_kernel<NR, BLOCK>), smem, 0, ready,
                                          "dense decode kernel (16-bit operands)");
  if (st != SMLA_OK) return st;
  decode_kernel<NR, BLOCK><<<p.grid, kThreads, smem, stream>>>(tk, tr, a.q, p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail_cuda(e, "dense decode launch");
  return launch_join<NR>(p, stream);
}

}  // namespace dw

smla_status_t launch_dense_decode_wide(const DenseDecodeArgs& a, unsigned* err, cudaStream_t stream) {
  using namespace dw;
  // Rows of an item: up to 64 over a bf16 cache; up to 32 with block scales,
  // whose raw chunks take 64 rows' place.
  const bool block = a.scales != nullptr;
  const int most = block ? 32 : 64;
  const int tokens = tokens_per_item(a.T, a.seqs->B, a.H, most), groups = (a.H + most - 1) / most;
  const int rows = groups > 1 ? a.H / groups : tokens * a.H, nr = rows > 32 ? 64 : rows > 16 ? 32 : 16;
  const smla_status_t st = check_line(a, groups, kItemCost);
  if (st != SMLA_OK) return st;
  const Params p = decode_params(a, tokens, groups, kItemCost, nr, err);
  if (block) return nr == 16 ? launch<16, true>(a, p, stream) : launch<32, true>(a, p, stream);
  if (nr == 64) return launch<64, false>(a, p, stream);
  return nr == 32 ? launch<32, false>(a, p, stream) : launch<16, false>(a, p, stream);
}

}  // namespace smla
