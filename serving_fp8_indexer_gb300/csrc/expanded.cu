// Latent attention in the expanded form (prefill): per-head keys and values
// up-projected from the latents, the rotary part of the keys shared by all
// heads,
//   z_j = scale * (q_nope[t,h] . k_nope[j,h] + q_rope[t,h] . k_rope[j]),
//   out[t,h] = sum_{j <= pos(t)} exp(z_j) v[j,h] / (sum_j exp(z_j) [+ exp(sink_h)]).
//
// One pass over the keys with a running maximum and sum.  A CTA takes one
// head and 256 consecutive query tokens of a sequence, as two tiles of 128
// rows that share every key block:
//   S_X [128 x 128] = Q_X . K^T      (12 MMAs of depth 16, f32 in TMEM)
//   P_X = exp2(S_X c - m), bf16, written over S_X in TMEM
//   O_X [128 x 128] += P_X . V       (8 MMAs, P read from TMEM)
// TMEM is exactly full (2 x (128 S + 128 O) columns).  A 128 x 128 block is
// 20 MMAs of 64 cycles (8192 dense bf16 flops a cycle and SM): 1280 cycles of tensor time against
// 16384 exponentials, so while one tile's softmax runs the tensor cores work
// on the other tile.  S and P may share columns because one thread issues
// every MMA and they execute in its order: PV_X(j) reads P_X before
// QK_X(j+1) writes S_X over it.
//
// The keys are never concatenated: a K tile's three 64-column chunks come
// from k_nope (two) and k_rope (one) by TMA, straight from the up-projection's
// output.  Beside Q (96 KB), 128 KB hold two V tiles and a ring of four K
// chunks (a K tile is three): every chunk and tile is loaded at least 1280
// cycles of tensor work before it is read.  (Two whole K tiles and one V tile
// left V a third less, and PV waited for it.)
//
// A row's reference m is raised only when a block exceeds it by more than
// 2^8 (P <= 256; bf16 P keeps its relative precision), so O is rescaled
// rarely.  l sums the f32 weights before their rounding to bf16; that
// rounding (2^-8 relative at most, random) is the only one beside the output's,
// and as large at every length.  P in two bf16 terms does without it, for 20
// -> 28 MMAs a block; the caller may ask for either (launch_expanded).
//
// Warps: 0-3 softmax of tile A, 4-7 of tile B (thread = row = TMEM lane, no
// exchange between threads), 8 TMA, 9 MMA issue and TMEM, 10 the V tail.  One
// thread issues both tiles' MMAs, so that a tile's run of PV and QK completes
// before the other's begins (a warp for each tile let the two runs share the
// tensor cores and end together, and both softmaxes then ran with the tensor
// cores idle: 12 % slower).
// When one wave of (tile, head) items leaves SMs idle, the keys are split
// over grid.z and a second kernel joins the partial results.
//
// Measured: 4096 tokens x 128 heads 440 us (1560 TFLOP/s, 0.81 of the measured
// bf16 rate), 8192 x 16 heads 201 us (0.89), 1025 tokens over 6100 keys in four
// sequences x 32 heads 230 us (0.71).  What bounds it: the shared-memory traffic
// of the operands (Q and K twelve times 8 KB a tile, V, and the TMA writes: 2700
// cycles a pair of blocks beside 2560 of tensor time), the issue of the MMAs
// (ring slots taken from a loop instead of unrolled: 500 us; the waits' polling
// loops unrolled, which filled the instruction cache: 467), then a CTA's start
// and epilogue, 8-10 k cycles.
#include <algorithm>
#include <cstddef>

#include "ptx.cuh"
#include "smla_internal.h"

namespace smla {
namespace ex {

constexpr int kBM = 128;  // rows of a tile
constexpr int kBN = 128;  // keys of a block
constexpr int kNope = 128, kRope = 64, kDV = 128;
constexpr int kChunk = kBM * 128;         // a 128-row x 64-column bf16 chunk, 128-byte swizzle
constexpr int kQTile = 3 * kChunk;        // 128 x 192
constexpr int kVTile = 2 * kChunk;
constexpr int kKSlots = 4, kVSlots = 2;
constexpr int kSoftThreads = 256;
constexpr int kThreads = 384;
constexpr int kTmaWarp = 8, kMmaWarp = 9, kTailWarp = 10;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 256;          // O_A, O_B after S_A, S_B
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kTau = 8.f;
constexpr int kTwoTermRows = 64;  // rows of a call that take two terms unasked
constexpr int kLaunchRegs = 168, kSoftRegs = 208, kOtherRegs = 80;
static_assert(kSoftThreads * kSoftRegs + (kThreads - kSoftThreads) * kOtherRegs <= kThreads * kLaunchRegs,
              "register split exceeds the launch allocation");

struct Params {
  const int32_t* cu_q;
  const int32_t* cu_kv;
  int B, T, S, H;
  float c;            // softmax_scale * log2(e) > 0
  const float* sink;  // [H] or null
  uint16_t* out;      // [T, H, 128]
  float* lse;         // [T, H] or null
  int slots, head_group;  // grid.x decomposition
  int nsplit;
  float* part_o;      // [nsplit, T, H, 128]
  float* part_lse;    // [nsplit, T, H], log2 units
  unsigned* err;
};

struct Smem {
  uint8_t q[2][kQTile];
  uint8_t k[kKSlots][kChunk];
  uint8_t v[kVSlots][kVTile];
  unsigned long long bar_q, bar_k_full[kKSlots], bar_k_empty[kKSlots], bar_v_full[kVSlots], bar_v_empty[kVSlots];
  unsigned long long bar_s[2], bar_p[2][2], bar_o[2];  // per tile (bar_p: and half of the keys)
  unsigned long long bar_tail_go, bar_tail, bar_drain;
  uint32_t tmem_base;
  int b, tile;  // the CTA's sequence and 256-row tile; b < 0: none
};

// The CTA's work: rows [t0, t0 + rows) of sequence b, key blocks [j0, j0 + n).
struct Work {
  int t0, rows;     // first token, tokens of this CTA (up to 256)
  int k0, kv;       // first key row, keys of the sequence
  int pos0;         // position of token t0
  int j0;           // first key block of this split
  int n[2];         // key blocks of each tile in this split
  int last;         // max(n[0], n[1])
};

__device__ __forceinline__ Work work_of(const Params& p, int b, int tile) {
  Work w;
  const int qb = p.cu_q[b], qe = p.cu_q[b + 1];
  w.k0 = p.cu_kv[b];
  w.kv = p.cu_kv[b + 1] - w.k0;
  w.t0 = qb + tile * 2 * kBM;
  w.rows = min(2 * kBM, qe - w.t0);
  w.pos0 = w.kv - (qe - qb) + tile * 2 * kBM;
  if (w.k0 < 0 || w.kv < 0 || w.kv > p.S - w.k0) {  // cu_kv does not describe the key rows
    if (threadIdx.x == 0) atomicOr(p.err, kErrShape);
    w.kv = 0;
  }
  // blocks each tile sees in all: its last row's pos + 1 keys, rounded up
  int nb[2];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    const int r = min(w.rows, (x + 1) * kBM) - x * kBM;  // rows of this tile
    const int keys = r > 0 ? min(w.pos0 + x * kBM + r, w.kv) : 0;
    nb[x] = keys > 0 ? (keys + kBN - 1) / kBN : 0;
  }
  const int all = max(nb[0], nb[1]);
  const int per = (all + p.nsplit - 1) / p.nsplit;
  w.j0 = min(all, static_cast<int>(blockIdx.z) * per);
  const int j1 = min(all, w.j0 + per);
#pragma unroll
  for (int x = 0; x < 2; ++x) w.n[x] = max(0, min(nb[x], j1) - w.j0);
  w.last = max(w.n[0], w.n[1]);
  return w;
}

// kTwo: P as two bf16 terms (hi + lo, side by side over S's columns).
template <bool kTwo>
__global__ void __launch_bounds__(kThreads, 1)
    expanded_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                    const __grid_constant__ CUtensorMap tr, const __grid_constant__ CUtensorMap tv, const Params p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  if (smem_u32(smem_raw) & 1023u) {  // the swizzled tiles need 1024-byte alignment
    if (threadIdx.x == 0) atomicOr(p.err, kErrShape);
    return;
  }
  Smem& s = *reinterpret_cast<Smem*>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // CTA -> (head group, slot, head of the group): a group's keys and values
  // stay in L2 while all its tiles read them, and within a group the longest
  // tiles start first.
  const int per_group = p.slots * p.head_group;
  const int group = blockIdx.x / per_group, rem = blockIdx.x - group * per_group;
  const int g_heads = min(p.head_group, p.H - group * p.head_group);
  const int slot = rem / g_heads, head = group * p.head_group + rem - slot * g_heads;
  if (warp == 0) {
    // slot -> (sequence, 256-row tile), each sequence's longest tile first
    int base = 0, fb = -1, ft = 0;
    for (int b0 = 0; b0 < p.B && fb < 0; b0 += 32) {
      const int b = b0 + lane;
      const int nt = b < p.B ? (max(0, p.cu_q[b + 1] - p.cu_q[b]) + 2 * kBM - 1) / (2 * kBM) : 0;
      int inc = nt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, inc, o);
        if (lane >= o) inc += up;
      }
      const int at = slot - base - (inc - nt);
      const unsigned hit = __ballot_sync(0xffffffffu, at >= 0 && at < nt);
      if (hit) {
        const int src = __ffs(hit) - 1;
        fb = b0 + src;
        ft = __shfl_sync(0xffffffffu, nt - 1 - at, src);
      }
      base += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) {
      s.b = fb;
      s.tile = ft;
    }
  }
  // beside the search: barriers, TMEM, descriptors
  if (threadIdx.x == 32) {
    mbar_init(smem_u32(&s.bar_q), 1);
    for (int i = 0; i < kKSlots; ++i) {
      mbar_init(smem_u32(&s.bar_k_full[i]), 1);
      mbar_init(smem_u32(&s.bar_k_empty[i]), 1);
    }
    for (int i = 0; i < kVSlots; ++i) {
      mbar_init(smem_u32(&s.bar_v_full[i]), 1);
      mbar_init(smem_u32(&s.bar_v_empty[i]), 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(smem_u32(&s.bar_s[x]), 1);
      mbar_init(smem_u32(&s.bar_p[x][0]), kBM);
      mbar_init(smem_u32(&s.bar_p[x][1]), kBM);
      mbar_init(smem_u32(&s.bar_o[x]), 1);
    }
    mbar_init(smem_u32(&s.bar_drain), 1);
    mbar_init(smem_u32(&s.bar_tail_go), 1);
    mbar_init(smem_u32(&s.bar_tail), 32);
    fence_mbar_init();
  }
  if (threadIdx.x == kTmaWarp * 32) {
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tr);
    tma_prefetch_desc(&tv);
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&s.tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (s.b < 0) {  // a slot past the batch's tiles
    if (warp == kMmaWarp) tmem_dealloc(s.tmem_base, kTmemCols);
    return;
  }
  const Work w = work_of(p, s.b, s.tile);
  const uint32_t tmem = s.tmem_base;
  // The sequence ends inside the last block: the rows behind it are another
  // sequence's (or nobody's), and a weight of 0 does not cancel an infinity
  // or NaN there, so the tail warp clears them in shared memory.
  const int tail = w.kv - (w.j0 + w.last - 1) * kBN;  // the sequence's keys in the last block
  const bool has_tail = w.last > 0 && tail < kBN;

  if (warp < 8) {
    // ===================================================== softmax, epilogue
    setmaxnreg_inc<kSoftRegs>();
    const int x = warp >> 2;
    const int row = threadIdx.x & 127;
    const int i = x * kBM + row;                 // row of the CTA
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t ts = tmem + lanes + x * kBN, to = tmem + lanes + kTmemO + x * kDV;
    const int nk = i < w.rows ? min(w.pos0 + i + 1, w.kv) : 0;  // keys the row sees
    const int n = x ? w.n[1] : w.n[0];
    float m = -INFINITY;
    float2 l2[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};  // even and odd column pairs
    bool ok = true;
    for (int j = 0; j < n; ++j) {
      if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&s.bar_s[x]), j & 1, p.err))) { ok = false; break; }
      tc_fence_after();
      uint32_t v[4][32];
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_ld32(ts + 32 * q, v[q]);
#pragma unroll
      for (int q = 0; q < 4; ++q) tmem_wait_ld_regs(v[q]);
      const int lim = nk - (w.j0 + j) * kBN;  // the row's keys in this block
      if (__any_sync(0xffffffffu, lim < kBN)) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (q * 32 + e >= lim) v[q][e] = 0xff800000u;  // -inf
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int e = 0; e < 32; e += 2)
#pragma unroll
        for (int q = 0; q < 4; ++q) mx[q] = max3(mx[q], __uint_as_float(v[q][e]), __uint_as_float(v[q][e + 1]));
      const float z = max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * p.c;
      const bool raise = z > m + kTau;
      if (__any_sync(0xffffffffu, raise)) {
        const float m_new = raise ? z : m;
        const float f = raise ? ex2_approx(m - m_new) : 1.f;  // 0 for the row's first keys
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          l2[k].x *= f;
          l2[k].y *= f;
        }
        m = m_new;
        if (j > 0) {
          // O holds blocks < j: wait for the last PV, scale the row
          if (!__all_sync(0xffffffffu, mbar_wait(smem_u32(&s.bar_o[x]), (j - 1) & 1, p.err))) { ok = false; break; }
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < 8; ++q) {
            uint32_t o[16];
            tmem_ld16(to + 16 * q, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            tmem_st16(to + 16 * q, o);
          }
        }
      }
      const float neg = m == -INFINITY ? 0.f : -m;
      const float2 c2 = make_float2(p.c, p.c), n2 = make_float2(neg, neg);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        uint32_t pk[32], pl[kTwo ? 32 : 1];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const int q = hf * 2 + (e >> 4), a = (e & 15) * 2;
          const float2 y = fma2(make_float2(__uint_as_float(v[q][a]), __uint_as_float(v[q][a + 1])), c2, n2);
          const float2 w2 = make_float2(ex2_approx(y.x), ex2_approx(y.y));
          l2[e & 1] = add2(l2[e & 1], w2);
          const __nv_bfloat162 b2 = __floats2bfloat162_rn(w2.x, w2.y);
          pk[e] = *reinterpret_cast<const uint32_t*>(&b2);
          if constexpr (kTwo) {
            const float2 r = __bfloat1622float2(b2);
            const __nv_bfloat162 lo = __floats2bfloat162_rn(w2.x - r.x, w2.y - r.y);
            pl[e] = *reinterpret_cast<const uint32_t*>(&lo);
          }
        }
        tmem_st32(ts + 32 * hf, pk);
        if constexpr (kTwo) tmem_st32(ts + kBN / 2 + 32 * hf, pl);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(smem_u32(&s.bar_p[x][hf]));  // PV starts on the first 64 keys
      }
    }
    if (ok && n > 0) ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&s.bar_o[x]), (n - 1) & 1, p.err));
    tc_fence_after();
    const int64_t t = w.t0 + i;
    const bool store = ok && i < w.rows && t >= 0 && t < p.T;
    const int64_t r = t * p.H + head;
    const float l = (l2[0].x + l2[0].y) + (l2[1].x + l2[1].y);
    const bool any = !(l == 0.f);  // without weights O's row is not read: zeros
    float inv = 0.f;
    float* po = nullptr;
    if (p.nsplit > 1) {
      const int64_t pr = static_cast<int64_t>(blockIdx.z) * p.T * p.H + r;
      if (store) p.part_lse[pr] = any ? m + log2f(l) : -INFINITY;
      if (any) inv = 1.f / l;
      po = p.part_o + pr * kDV;
    } else {
      // the sink joins the denominator against the larger of the two
      // references, so that neither weight overflows
      const float sk = p.sink ? p.sink[head] * kLog2e : -INFINITY;
      const float top = fmaxf(m, sk);
      const float f = sk > m ? ex2_approx(m - top) : 1.f;
      const float total = sk == -INFINITY ? l : fmaf(l, f, exp2f(sk - top));
      if (any) inv = f / total;
      if (store && p.lse) p.lse[r] = total == 0.f ? -INFINITY : kLn2 * (top + log2f(total));
    }
    if (n > 0) {
      // O / l.  Partial results go out as they are; bf16 rows are first put
      // into Q's place (every QK of the tile has been read by now), 16-byte
      // pieces swizzled over the banks, so that a warp stores whole rows
      // (stored from the registers, 32 rows 16 bytes at a time: 3300 cycles).
      uint8_t* stage = s.q[x] + (row & ~31) * (kDV * 2);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t o[32];
        tmem_ld32(to + 32 * q, o);
        tmem_wait_ld_regs(o);
        if (po) {
          if (store && any)
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<float4*>(po + 32 * q + e) =
                  make_float4(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv,
                              __uint_as_float(o[e + 2]) * inv, __uint_as_float(o[e + 3]) * inv);
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float a = any ? __uint_as_float(o[e + 2 * k]) * inv : 0.f;
              const float b = any ? __uint_as_float(o[e + 2 * k + 1]) * inv : 0.f;
              const __nv_bfloat162 b2 = __floats2bfloat162_rn(a, b);
              u[k] = *reinterpret_cast<const uint32_t*>(&b2);
            }
            const int piece = q * 4 + e / 8;
            *reinterpret_cast<uint4*>(stage + lane * (kDV * 2) + ((piece ^ (lane & 7)) << 4)) =
                make_uint4(u[0], u[1], u[2], u[3]);
          }
        }
      }
      if (!po) {
        __syncwarp();
        const unsigned keep = __ballot_sync(0xffffffffu, store);
        const int64_t t_warp = t - lane;  // the warp's first token
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int rr = 2 * k + (lane >> 4), piece = lane & 15;
          const uint4 u = *reinterpret_cast<const uint4*>(stage + rr * (kDV * 2) + ((piece ^ (rr & 7)) << 4));
          if (keep >> rr & 1)
            reinterpret_cast<uint4*>(p.out + ((t_warp + rr) * p.H + head) * kDV)[piece] = u;
        }
      }
    } else if (store && !po) {
      for (int q = 0; q < kDV / 8; ++q) reinterpret_cast<uint4*>(p.out + r * kDV)[q] = make_uint4(0, 0, 0, 0);
    }
  } else if (warp == kTmaWarp) {
    // ================================================================== TMA
    setmaxnreg_dec<kOtherRegs>();
    if (elect_one() && w.last > 0) {
      const int tiles = w.n[1] > 0 ? 2 : 1;
      mbar_arrive_expect_tx(smem_u32(&s.bar_q), tiles * kQTile);
      for (int x = 0; x < tiles; ++x)
        for (int c = 0; c < 3; ++c)
          tma_load_3d(smem_u32(s.q[x]) + c * kChunk, &tq, c * 128, head, w.t0 + x * kBM, smem_u32(&s.bar_q));
      int nk = 0, nv = 0;  // K chunks and V tiles requested
      bool ok = true;
      // chunks [c0, c1) of K block j
      auto load_k = [&](int j, int c0, int c1) {
        const int key = w.k0 + (w.j0 + j) * kBN;
        for (int c = c0; c < c1; ++c) {
          const int g = j * 3 + c, sl = g % kKSlots;
          if (g >= kKSlots) ok = ok && mbar_wait(smem_u32(&s.bar_k_empty[sl]), (g / kKSlots - 1) & 1, p.err);
          if (!ok) return;
          const uint32_t bar = smem_u32(&s.bar_k_full[sl]);
          mbar_arrive_expect_tx(bar, kChunk);
          if (c < 2)
            tma_load_3d(smem_u32(s.k[sl]), &tk, c * 128, head, key, bar);
          else
            tma_load_2d(smem_u32(s.k[sl]), &tr, 0, key, bar);
          ++nk;
        }
      };
      auto load_v = [&](int j) {
        const int sl = j % kVSlots;
        if (j >= kVSlots) ok = ok && mbar_wait(smem_u32(&s.bar_v_empty[sl]), (j / kVSlots - 1) & 1, p.err);
        if (!ok) return;
        const int key = w.k0 + (w.j0 + j) * kBN;
        const uint32_t bar = smem_u32(&s.bar_v_full[sl]);
        mbar_arrive_expect_tx(bar, kVTile);
        tma_load_3d(smem_u32(s.v[sl]), &tv, 0, head, key, bar);
        tma_load_3d(smem_u32(s.v[sl]) + kChunk, &tv, 128, head, key, bar);
        ++nv;
      };
      // in the order in which their places come free: the next block's first
      // chunk has a spare slot, V(j + 1) the other tile, the other chunks
      // follow QK(j)
      load_k(0, 0, 3);
      load_v(0);
      for (int j = 0; j < w.last && ok; ++j) {
        if (j + 1 < w.last) {
          load_k(j + 1, 0, 1);
          if (ok) load_v(j + 1);
          if (ok) load_k(j + 1, 1, 3);
        }
      }
      // the last V is requested: from here on its barriers are in their last
      // phase, which the tail warp waits for
      if (ok) mbar_arrive(smem_u32(&s.bar_tail_go));
      // nothing is still landing when the CTA ends (all have landed long ago
      // unless a wait gave up)
      mbar_wait(smem_u32(&s.bar_q), 0, p.err);
      for (int sl = 0; sl < kKSlots; ++sl) {
        const int loads = (nk + kKSlots - 1 - sl) / kKSlots;
        if (loads > 0) mbar_wait(smem_u32(&s.bar_k_full[sl]), (loads - 1) & 1, p.err);
      }
      for (int sl = 0; sl < kVSlots; ++sl) {
        const int loads = (nv + kVSlots - 1 - sl) / kVSlots;
        if (loads > 0) mbar_wait(smem_u32(&s.bar_v_full[sl]), (loads - 1) & 1, p.err);
      }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    // ================================================================== MMA
    setmaxnreg_dec<kOtherRegs>();
    if (elect_one() && w.last > 0) {
      constexpr uint32_t IDESC_QK = idesc_bf16_f32(kBM, kBN, 0, 0);
      constexpr uint32_t IDESC_PV = idesc_bf16_f32(kBM, kDV, 0, 1);
      const uint64_t dq = make_sdesc(smem_u32(s.q[0]), 16, 1024, kSwizzle128B);
      const uint64_t dk = make_sdesc(smem_u32(s.k[0]), 16, 1024, kSwizzle128B);
      const uint64_t dv = make_sdesc(smem_u32(s.v[0]), kChunk, 1024, kSwizzle128B);
      bool ok = mbar_wait(smem_u32(&s.bar_q), 0, p.err);
      // S_x = Q_x K^T of block j; `first`: its chunks are waited for, `done`:
      // they are handed back
      auto qk = [&](int x, int j, bool first, bool done) {
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          const int g = j * 3 + c, sl = g % kKSlots;
          if (first) ok = ok && mbar_wait(smem_u32(&s.bar_k_full[sl]), (g / kKSlots) & 1, p.err);
          if (!ok) return;
          const uint64_t a = dq + static_cast<uint64_t>((x * kQTile + c * kChunk) >> 4);
          const uint64_t b = dk + static_cast<uint64_t>(sl * (kChunk >> 4));
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_f16_ss(tmem + x * kBN, a + static_cast<uint64_t>(kk * 2), b + static_cast<uint64_t>(kk * 2), IDESC_QK,
                       (c | kk) ? 1u : 0u);
          if (done) mma_commit(smem_u32(&s.bar_k_empty[sl]));
        }
        mma_commit(smem_u32(&s.bar_s[x]));
      };
      // O_x += P_x V of block j
      auto pv = [&](int x, int j, bool first, bool done) {
        const int sl = j % kVSlots;
        if (first) {
          ok = ok && mbar_wait(smem_u32(&s.bar_v_full[sl]), (j / kVSlots) & 1, p.err);
          if (ok && has_tail && j == w.last - 1) ok = mbar_wait(smem_u32(&s.bar_tail), 0, p.err);
        }
        const uint64_t b = dv + static_cast<uint64_t>(sl * (kVTile >> 4));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          ok = ok && mbar_wait(smem_u32(&s.bar_p[x][h]), j & 1, p.err);
          if (!ok) return;
          tc_fence_after();
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            const int ks = h * 4 + kk;  // 16 keys: 8 columns of P, 16 rows of V
            mma_f16_ts(tmem + kTmemO + x * kDV, tmem + x * kBN + ks * 8,
                       b + static_cast<uint64_t>((ks * 16 * 128) >> 4), IDESC_PV, (j > 0 || ks > 0) ? 1u : 0u);
            if (kTwo)
              mma_f16_ts(tmem + kTmemO + x * kDV, tmem + x * kBN + kBN / 2 + ks * 8,
                         b + static_cast<uint64_t>((ks * 16 * 128) >> 4), IDESC_PV, 1u);
          }
        }
        if (done) mma_commit(smem_u32(&s.bar_v_empty[sl]));
        mma_commit(smem_u32(&s.bar_o[x]));
      };
      if (ok && w.n[0] > 0) qk(0, 0, true, w.n[1] <= 0);
      if (ok && w.n[1] > 0) qk(1, 0, w.n[0] <= 0, true);
      for (int j = 0; j < w.last && ok; ++j) {
        const bool a = j < w.n[0], b = j < w.n[1];
        const bool a1 = j + 1 < w.n[0], b1 = j + 1 < w.n[1];
        if (a) {
          pv(0, j, true, !b);
          if (ok && a1) qk(0, j + 1, true, !b1);
        }
        if (ok && b) {
          pv(1, j, !a, true);
          if (ok && b1) qk(1, j + 1, !a1, true);
        }
      }
      // every MMA has finished before TMEM is freed
      mma_commit(smem_u32(&s.bar_drain));
      mbar_wait(smem_u32(&s.bar_drain), 0, p.err);
    }
    __syncwarp();
  } else {
    setmaxnreg_dec<kOtherRegs>();
    if (warp == kTailWarp && has_tail) {
      const int sl = (w.last - 1) % kVSlots, ph = (w.last - 1) / kVSlots & 1;
      const bool ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&s.bar_tail_go), 0, p.err) &&
                                                  mbar_wait(smem_u32(&s.bar_v_full[sl]), ph, p.err));
      if (ok) {
        // rows [tail, 128) of both 64-column chunks, 128 bytes each
        for (int u = lane; u < (kBN - tail) * 16; u += 32) {
          const int r = tail + (u >> 4), pc = u & 15;
          *reinterpret_cast<uint4*>(s.v[sl] + (pc >> 3) * kChunk + r * 128 + (pc & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
        mbar_arrive(smem_u32(&s.bar_tail));
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

// Joins the splits of a (token, head) row: one warp, four columns a lane.
__global__ void __launch_bounds__(128) join_kernel(const Params p) {
  const int64_t r = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int64_t rows = static_cast<int64_t>(p.T) * p.H;
  // rows behind the last sequence were never written: left as they are
  if (r >= rows || r / p.H < p.cu_q[0] || r / p.H >= p.cu_q[p.B]) return;
  const float sk = p.sink ? p.sink[r % p.H] * kLog2e : -INFINITY;
  float top = sk;
  for (int i = 0; i < p.nsplit; ++i) top = fmaxf(top, p.part_lse[i * rows + r]);
  const float m = top == -INFINITY ? 0.f : top;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float l = exp2f(sk - m);  // 0 without a sink
  for (int i = 0; i < p.nsplit; ++i) {
    const float e = p.part_lse[i * rows + r];
    if (e == -INFINITY) continue;  // an empty split wrote no partial
    const float f = exp2f(e - m);
    const float4 o = reinterpret_cast<const float4*>(p.part_o + (i * rows + r) * kDV)[lane];
    l += f;
    acc.x = fmaf(f, o.x, acc.x);
    acc.y = fmaf(f, o.y, acc.y);
    acc.z = fmaf(f, o.z, acc.z);
    acc.w = fmaf(f, o.w, acc.w);
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
  const __nv_bfloat162 b = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  reinterpret_cast<uint2*>(p.out + r * kDV)[lane] =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  if (p.lse && lane == 0) p.lse[r] = l == 0.f ? -INFINITY : kLn2 * (m + log2f(l));
}

}  // namespace ex

// Tiles the grid provides for: sum_b ceil(q_len_b / 256) is at most this.
static int64_t expanded_slots(int T, int B) { return T / (2 * ex::kBM) + B; }

int expanded_splits(int T, int S, int B, int H) {
  if (T <= 0 || S <= 0 || B <= 0 || H <= 0) return 1;
  // tiles of a batch of equal sequences (a bound for the choice only)
  const int64_t each = (T + B - 1) / B;
  const int64_t items = static_cast<int64_t>(B) * ((each + 2 * ex::kBM - 1) / (2 * ex::kBM)) * H;
  const int sms = device_sm_count();
  const int blocks = (S / B + ex::kBN - 1) / ex::kBN;
  // one wave of CTAs, each with at least four key blocks
  const int64_t n = std::min<int64_t>(sms / std::max<int64_t>(items, 1), blocks / 4);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(n, 64)));
}

size_t expanded_workspace_bytes(int T, int H, int nsplit) {
  if (nsplit <= 1) return 0;
  const size_t rows = static_cast<size_t>(nsplit) * T * H;
  return (rows * ex::kDV * sizeof(float) + 255 + rows * sizeof(float) + 255) & ~size_t(255);
}

smla_status_t launch_expanded(const ExpandedArgs& a, unsigned* err, cudaStream_t stream) {
  using namespace ex;
  CUtensorMap tq, tk, tr, tv;
  const auto map3 = [&](CUtensorMap* m, const void* base, int width, int heads, int rows, int64_t hs, int64_t rs,
                        uint32_t box_rows) {
    const uint64_t dims[3] = {static_cast<uint64_t>(width) * 2, static_cast<uint64_t>(heads),
                              static_cast<uint64_t>(rows)};
    const uint64_t strides[2] = {static_cast<uint64_t>(hs) * 2, static_cast<uint64_t>(rs) * 2};
    const uint32_t box[3] = {128, 1, box_rows};
    return encode_tma_u8(m, base, 3, dims, strides, box, 128);
  };
  bool enc = map3(&tq, a.q, kNope + kRope, a.H, a.T, a.q_hs, a.q_ts, kBM);
  if (a.S > 0) {
    enc = enc && map3(&tk, a.k_nope, kNope, a.H, a.S, a.k_hs, a.k_ts, kBN) &&
          map3(&tv, a.v, kDV, a.H, a.S, a.v_hs, a.v_ts, kBN);
    const uint64_t dims[2] = {kRope * 2, static_cast<uint64_t>(a.S)};
    const uint64_t strides[1] = {static_cast<uint64_t>(a.r_ts) * 2};
    const uint32_t box[2] = {128, kBN};
    enc = enc && encode_tma_u8(&tr, a.k_rope, 2, dims, strides, box, 128);
  } else {
    tk = tr = tv = tq;  // no key rows: none is loaded
  }
  if (!enc) return fail(SMLA_ERR_CUDA, "cuTensorMapEncodeTiled failed for the expanded-prefill tensor maps");
  Params p{};
  p.cu_q = a.cu_q;
  p.cu_kv = a.cu_kv;
  p.B = a.B;
  p.T = a.T;
  p.S = a.S;
  p.H = a.H;
  p.c = a.softmax_scale * kLog2e;
  p.sink = a.sink;
  p.out = a.out;
  p.lse = a.lse;
  p.nsplit = a.nsplit;
  p.err = err;
  if (a.nsplit > 1) {
    const size_t rows = static_cast<size_t>(a.nsplit) * a.T * a.H;
    p.part_o = static_cast<float*>(a.workspace);
    p.part_lse = p.part_o + ((rows * kDV + 63) & ~size_t(63));
  }
  const size_t smem = sizeof(Smem);
  static_assert(sizeof(Smem) <= 232448, "shared memory exceeds a CTA's 227 KB");
  static_assert(offsetof(Smem, k) % 1024 == 0 && offsetof(Smem, v) % 1024 == 0, "swizzled tiles need 1024-byte alignment");
  // One term or two: the error against 64 bits is 1.4 or 1.0 times that of the
  // output's own rounding, in every row and at every size.  Two cost little where
  // a call is mostly its launch (1 row of 4000 keys 14 -> 17 us) and 40 % where it
  // is not (4096 tokens x 128 heads 441 -> 614 us, 32 tokens x 128 heads over 4 x
  // 8000 keys 333 -> 467).  So, where the caller does not say: two for a call of
  // up to kTwoTermRows rows, one for others.
  const bool two = a.p_terms ? a.p_terms == 2 : static_cast<int64_t>(a.T) * a.H <= kTwoTermRows;
  const auto kernel = two ? expanded_kernel<true> : expanded_kernel<false>;
  static std::atomic<unsigned long long> ready[2];
  const smla_status_t st = prepare_kernel(reinterpret_cast<const void*>(kernel), smem, kLaunchRegs, ready[two],
                                          "expanded kernel");
  if (st != SMLA_OK) return st;
  p.slots = static_cast<int>(expanded_slots(a.T, a.B));
  // Groups of heads of even size whose keys and values (512 bytes a row) take
  // at most kGroupBytes, two thirds of L2: larger groups order more tiles by
  // their length, smaller ones read less again from HBM (4096 tokens, 128
  // heads: 12 MB 511 us, 48 MB 486, 80 MB 471, 112 MB 478, all heads 535).
  constexpr int64_t kGroupBytes = int64_t(80) << 20;
  const int most = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(a.H, kGroupBytes / (int64_t(512) * std::max(a.S, 1)))));
  const int n_groups = (a.H + most - 1) / most;
  p.head_group = (a.H + n_groups - 1) / n_groups;
  const int64_t ctas = static_cast<int64_t>(p.slots) * a.H;
  if (ctas > 0x7fffffff || static_cast<int64_t>(p.slots) * p.head_group > 0x7fffffff)
    return fail(SMLA_ERR_UNSUPPORTED, "expanded prefill: too many tiles (T=%d, B=%d, H=%d)", a.T, a.B, a.H);
  const dim3 grid(static_cast<unsigned>(ctas), 1, static_cast<unsigned>(a.nsplit));
  kernel<<<grid, kThreads, smem, stream>>>(tq, tk, tr, tv, p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail_cuda(e, "expanded launch");
  if (a.nsplit > 1) {
    const int64_t rows = static_cast<int64_t>(a.T) * a.H;
    join_kernel<<<static_cast<unsigned>((rows + 3) / 4), 128, 0, stream>>>(p);
    e = cudaGetLastError();
    if (e != cudaSuccess) return fail_cuda(e, "expanded join launch");
  }
  return SMLA_OK;
}

}  // namespace smla
