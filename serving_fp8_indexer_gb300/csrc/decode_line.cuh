// What the dense-decode kernels share: the line of work that is cut evenly over
// the CTAs, a CTA's walk along its part, and the join of the items that were
// cut.
#pragma once
#include <algorithm>

#include "rope.cuh"

namespace smla {
namespace dd {

constexpr int kD = 576, kDV = 512;
constexpr int kBK = 128;                 // keys of a block
constexpr int kSoftThreads = 256, kSoftWarps = 8, kThreads = 384;
constexpr int kTmaWarp = 8, kQkWarp = 9, kPvWarp = 10;
constexpr uint32_t kTmemCols = 512, kTmemS = 256;
constexpr float kLog2e = 1.4426950408889634f;
// The reference of a row's weights P = p * scale counts no scale as smaller than
// 2^kLeastLg: the sums of p itself stay finite where a block's rows all have
// scale 0 or almost (values below 2^-88 are then not told from 0).
constexpr float kLeastLg = -88.f;
// A row's largest weight is kept at 2^11 .. 2^15: a block's largest sets the
// reference to 2^kPOffset below it, and the reference is raised when a later
// block's exceeds it by more than 2^kTau.  That is the upper end of e5m2 and f16
// (57344, 65504): what they have below is left to the small weights.
constexpr float kPOffset = 11.f, kTau = 15.f;
constexpr int kOrdMin = static_cast<int>(0x80000000u);

struct Cut;
struct Params {
  SeqsDev seqs;
  int64_t phys_rows;
  const float* scales;  // [phys_rows] or null
  int T, H;
  int tok_per_item;     // tokens of an item, 1 where a token's heads fill one
  int groups, group_rows;  // head groups of a token, and their heads
  int item_cost;        // of the line, in blocks
  float softmax_scale;
  const float* sink;
  uint16_t* out;
  // Partial results: CTA c's slot 2c holds the item its part continues, slot
  // 2c + 1 the one that begins in it and goes on.
  float* part_o;        // [2 * grid][NR][512], each normalised by its own sum
  float* part_lse;      // [2 * grid][NR], log2 units
  Cut* cuts;            // [grid]
  int grid;
  unsigned* err;
};
// What CTA c's part begins with: an item cut at its first block, and whether
// that is the item's first cut (whose CTA the join goes by).
struct Cut {
  int first_cta;  // CTA where the item begins; -1: not an item's first cut
  int last_cta;
  int row0, rows, h0;  // output rows [row0, row0 + rows), head of the first
};


// ------------------------------------------------------------- the work line
// Items in order: sequence after sequence, its token groups, their head
// groups; each p.item_cost units without keys, then a unit for each of its
// `nblk` blocks of 128 keys (at least one, so that tokens without keys are
// visited and get their zeros).
struct SeqWork {
  int q0, q_len, kv, nblk, items, cost;
  __device__ __forceinline__ int item_units() const { return cost + nblk; }
  __device__ __forceinline__ int units() const { return items * item_units(); }
};
__device__ __forceinline__ SeqWork seq_work(const Params& p, int b) {
  SeqWork w;
  w.q0 = max(0, p.seqs.cu_q[b]);
  w.q_len = max(0, min(p.T, p.seqs.cu_q[b + 1]) - w.q0);
  w.kv = max(0, p.seqs.kv_len[b]);
  const int64_t most = static_cast<int64_t>(p.seqs.max_pages) << p.seqs.page_shift;
  if (w.kv > most) {
    atomicOr(p.err, kErrShape);
    w.kv = static_cast<int>(most);
  }
  w.nblk = max(1, (w.kv + kBK - 1) / kBK);
  w.cost = p.item_cost;
  w.items = (w.q_len + p.tok_per_item - 1) / p.tok_per_item * p.groups;
  return w;
}

// All units (below 2^31: the launcher checks the bound), by the whole warp.
__device__ __forceinline__ int warp_sum(int n) { return __reduce_add_sync(0xffffffffu, n); }

// Sequence that holds unit x of the line, and the line's position of its
// first unit; by the whole warp, lane l holding sequence b0 + l's units n.
// -1 when x lies behind these; `base` then moves past them.
__device__ __forceinline__ int find_among(int x, int n, int lane, int& base) {
  int inc = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += up;
  }
  const unsigned hit = __ballot_sync(0xffffffffu, x >= base + inc - n && x < base + inc);
  if (hit) {
    const int src = __ffs(hit) - 1;
    base += __shfl_sync(0xffffffffu, inc - n, src);
    return src;
  }
  base += __shfl_sync(0xffffffffu, inc, 31);
  return -1;
}

// A CTA's walk along its part of the line.
struct Cursor {
  int b, item, at;  // next: sequence, item of the sequence, unit of the item
  int left;         // units left
};
// One item's blocks within the part.
struct Seg {
  int t0, ntok, h0, rows;  // first token, tokens, first head, rows
  int b, pos1;             // sequence; keys that token t0 sees
  int j0, nb;              // blocks [j0, j0 + nb)
  bool whole;              // all of the item's blocks
};
__device__ __forceinline__ bool next_seg(const Params& p, Cursor& c, Seg& s) {
  for (;;) {
    if (c.left <= 0) return false;
    SeqWork w = seq_work(p, c.b);
    while (c.item >= w.items) {  // past the sequence's items
      if (++c.b >= p.seqs.B) return false;
      c.item = 0;
      w = seq_work(p, c.b);
    }
    const int tg = c.item / p.groups, hg = c.item - tg * p.groups;
    const int take = min(w.item_units() - c.at, c.left), end = c.at + take - p.item_cost;  // first block not taken
    s.b = c.b;
    s.t0 = w.q0 + tg * p.tok_per_item;
    s.ntok = min(p.tok_per_item, w.q_len - tg * p.tok_per_item);
    s.h0 = hg * p.group_rows;
    s.rows = p.groups > 1 ? p.group_rows : s.ntok * p.H;
    s.pos1 = w.kv - w.q_len + tg * p.tok_per_item + 1;
    s.j0 = max(0, c.at - p.item_cost);
    s.nb = end - s.j0;
    s.whole = s.nb == w.nblk;
    c.left -= take;
    c.at += take;
    if (c.at >= w.item_units()) {
      c.at = 0;
      ++c.item;
    }
    if (s.nb > 0) return true;  // (a part that ends before the item's blocks has nothing of it)
  }
}
__device__ __forceinline__ int seg_keys(const Seg& s) { return max(0, s.pos1 + s.ntok - 1); }  // the last token's keys

// The CTA's part of the line, by every warp (b < 0: none); records the cut that
// the part begins with for the join.
__device__ __forceinline__ Cursor find_part(const Params& p, int lane) {
  Cursor start{-1, 0, 0, 0};
  const int B = p.seqs.B;
  int n0 = 0, total = 0;  // n0: the lane's units among the first 32 sequences
  for (int b0 = 0; b0 < B; b0 += 32) {
    int n = 0;
    if (b0 + lane < B) {
      const SeqWork w = seq_work(p, b0 + lane);
      n = w.units();
    }
    if (b0 == 0) n0 = n;
    total += warp_sum(n);
  }
  const int grid = gridDim.x, cta = blockIdx.x;
  const int per = (total + grid - 1) / grid;
  const int x0 = total - per * cta > 0 ? per * cta : total;  // (per * cta stays below 2^31: cta < grid)
  Cut cut{-1, 0, 0, 0, 0};
  if (x0 < total) {
    int base = 0;
    start.b = find_among(x0, n0, lane, base);
    for (int b0 = 32; start.b < 0 && b0 < B; b0 += 32) {
      int n = 0;
      if (b0 + lane < B) {
        const SeqWork w = seq_work(p, b0 + lane);
        n = w.units();
      }
      const int at = find_among(x0, n, lane, base);
      if (at >= 0) start.b = b0 + at;
    }
    const SeqWork w = seq_work(p, max(start.b, 0));
    start.item = (x0 - base) / w.item_units();
    start.at = x0 - base - start.item * w.item_units();
    start.left = min(per, total - x0);
    if (start.b >= 0 && start.at > p.item_cost) {
      const int w0 = x0 - start.at + p.item_cost;  // the item's first block
      if (w0 / per + 1 == cta) {
        Cursor c = start;
        Seg g;
        next_seg(p, c, g);
        cut = {w0 / per, min((w0 + w.nblk - 1) / per, grid - 1), g.t0 * p.H + g.h0, g.rows, g.h0};
      }
    }
  }
  if (threadIdx.x == 0 && p.cuts) p.cuts[cta] = cut;
  return start;
}

__device__ __forceinline__ int ord_int(float f) {
  const int b = __float_as_int(f);
  return b >= 0 ? b : b ^ 0x7fffffff;
}
__device__ __forceinline__ float ord_float(int o) { return __int_as_float(o >= 0 ? o : o ^ 0x7fffffff); }
// byte offset of 16-byte piece c of row r in a 128- (64-) byte-swizzled chunk
__device__ __forceinline__ uint32_t sw128(int r, int c) { return static_cast<uint32_t>(r * 128 + ((c ^ (r & 7)) << 4)); }
__device__ __forceinline__ uint32_t sw64(int r, int c) { return static_cast<uint32_t>(r * 64 + ((c ^ ((r >> 1) & 3)) << 4)); }

// One arrival for the warp, behind what every lane did (an arrival from each
// lane is 32 in a row on one word).
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// N (8, 16 or 32) TMEM columns of the thread's lane, waited for.
template <int N>
__device__ __forceinline__ void tmem_issue_ld(uint32_t a, uint32_t (&v)[N]) {
  static_assert(N == 8 || N == 16 || N == 32, "");
  if constexpr (N == 32) {
    tmem_ld32(a, v);
  } else if constexpr (N == 16) {
    tmem_ld16(a, v);
  } else {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                 : "r"(a));
  }
}
// Ties v's uses to after the wait before it.
template <int N>
__device__ __forceinline__ void after_wait(uint32_t (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+r"(v[i]));
}
__device__ __forceinline__ void tmem_st8(uint32_t a, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(a), "r"(v[0]), "r"(v[1]),
               "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// Joins the parts of the cut items, row (token, head) by row:
//   out = sum_c 2^(L_c - M) O_c / (sum_c 2^(L_c - M) + 2^(sink - M)).
// Two CTAs an SM; each lists the cut items in shared memory and takes its
// share of their rows (a CTA for every possible row spent more on CTAs without
// work than on the sums: 13 us against 4).  A row of few parts is taken by a
// group of 128 threads, a float4 each; one of more than kManyParts by the four
// groups of a CTA together, every fourth part each.
constexpr int kJoinGroups = 4, kManyParts = 16, kMaxGrid = 256;

struct RowSum {
  float4 acc;
  float l;
};
// Parts first, first + step, ... of a row against the reference m.
template <int NR>
__device__ __forceinline__ RowSum sum_parts(const Params& p, const Cut& cut, int row, int parts, int first, int step,
                                            float m, int col) {
  const auto slot = [&](int c) { return static_cast<int64_t>(2 * (cut.first_cta + c) + (c == 0 ? 1 : 0)) * NR + row; };
  RowSum s{make_float4(0.f, 0.f, 0.f, 0.f), 0.f};
  for (int c0 = first; c0 < parts; c0 += 8 * step) {
    float w[8];
    float4 o[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int c = c0 + u * step;
      w[u] = c < parts ? p.part_lse[slot(c)] : -INFINITY;
      o[u] = c < parts ? __ldcs(reinterpret_cast<const float4*>(p.part_o + slot(c) * kDV) + col)
                       : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const float f = exp2f(w[u] - m);  // 0 for a part without keys, whose O is 0
      s.l += f;
      s.acc.x = fmaf(f, o[u].x, s.acc.x);
      s.acc.y = fmaf(f, o[u].y, s.acc.y);
      s.acc.z = fmaf(f, o[u].z, s.acc.z);
      s.acc.w = fmaf(f, o[u].w, s.acc.w);
    }
  }
  return s;
}

template <int NR>
__global__ void __launch_bounds__(128 * kJoinGroups, 2) join_kernel(const Params p) {
  __shared__ Cut s_cut[kMaxGrid];
  __shared__ int s_warp[kMaxGrid / 32];
  __shared__ float4 s_acc[kJoinGroups - 1][128];
  __shared__ float s_l[kJoinGroups - 1];
  const int grp = threadIdx.x / 128, col = threadIdx.x % 128, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // the cut items, in the order of their cuts
  Cut mine{-1, 0, 0, 0, 0};
  if (threadIdx.x > 0 && threadIdx.x < p.grid) mine = p.cuts[threadIdx.x];
  const unsigned cuts = __ballot_sync(0xffffffffu, mine.first_cta >= 0);
  if (warp < kMaxGrid / 32 && lane == 0) s_warp[warp] = __popc(cuts);
  __syncthreads();
  int n = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kMaxGrid / 32; ++w) {
    if (w < warp) before += s_warp[w];
    n += s_warp[w];
  }
  if (mine.first_cta >= 0) s_cut[before + __popc(cuts & ((1u << lane) - 1))] = mine;
  __syncthreads();

  // the row's reference: the largest of its parts' (and the sink's)
  const auto reference = [&](const Cut& cut, int row, int parts, float& sk) {
    const int head = p.groups > 1 ? cut.h0 + row : row % p.H;
    sk = p.sink ? p.sink[head] * kLog2e : -INFINITY;
    float top = sk;
    for (int c = lane; c < parts; c += 32)
      top = fmaxf(top, p.part_lse[static_cast<int64_t>(2 * (cut.first_cta + c) + (c == 0 ? 1 : 0)) * NR + row]);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    return top == -INFINITY ? 0.f : top;
  };
  const auto store = [&](const Cut& cut, int row, const RowSum& s) {
    const float inv = s.l == 0.f ? 0.f : 1.f / s.l;
    const __nv_bfloat162 a = __floats2bfloat162_rn(s.acc.x * inv, s.acc.y * inv);
    const __nv_bfloat162 b = __floats2bfloat162_rn(s.acc.z * inv, s.acc.w * inv);
    reinterpret_cast<uint2*>(p.out + static_cast<int64_t>(cut.row0 + row) * kDV)[col] =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  };
  for (int u = blockIdx.x * kJoinGroups + grp; u < n * NR; u += gridDim.x * kJoinGroups) {
    const Cut cut = s_cut[u / NR];
    const int row = u % NR, parts = cut.last_cta - cut.first_cta + 1;
    if (row >= cut.rows || parts > kManyParts) continue;
    float sk;
    const float m = reference(cut, row, parts, sk);
    RowSum s = sum_parts<NR>(p, cut, row, parts, 0, 1, m, col);
    s.l += exp2f(sk - m);
    store(cut, row, s);
  }
  for (int u = blockIdx.x; u < n * NR; u += gridDim.x) {
    const Cut cut = s_cut[u / NR];
    const int row = u % NR, parts = cut.last_cta - cut.first_cta + 1;
    if (row >= cut.rows || parts <= kManyParts) continue;  // (the same for the whole CTA)
    float sk;
    const float m = reference(cut, row, parts, sk);
    RowSum s = sum_parts<NR>(p, cut, row, parts, grp, kJoinGroups, m, col);
    __syncthreads();  // the sums of the row before have been read
    if (grp > 0) {
      s_acc[grp - 1][col] = s.acc;
      if (col == 0) s_l[grp - 1] = s.l;
    }
    __syncthreads();
    if (grp == 0) {
#pragma unroll
      for (int g = 0; g < kJoinGroups - 1; ++g) {
        const float4 o = s_acc[g][col];
        s.l += s_l[g];
        s.acc.x += o.x;
        s.acc.y += o.y;
        s.acc.z += o.z;
        s.acc.w += o.w;
      }
      s.l += exp2f(sk - m);
      store(cut, row, s);
    }
  }
}

// The CTAs of a call, and the tokens that share an item of `rows` rows: as many
// as a sequence has on average.
inline int tokens_per_item(int T, int B, int H, int rows) {
  int n = 1;
  while (2 * n * H <= rows && n * B < T) n *= 2;
  return n;
}
inline int decode_grid(int T, int H, int max_kv_len) {
  const int64_t blocks = static_cast<int64_t>(T) * std::max(1, H / 64) * ((max_kv_len + kBK - 1) / kBK);
  return static_cast<int>(std::min<int64_t>(std::min(device_sm_count(), kMaxGrid), std::max<int64_t>(blocks, 1)));
}
// A call's parameters, for items of up to `rows` rows (a multiple of H, or
// H's parts).
inline Params decode_params(const DenseDecodeArgs& a, int tok_per_item, int groups, int item_cost, int nr, unsigned* err) {
  Params p{};
  p.seqs = seqs_dev(*a.seqs);
  p.phys_rows = a.phys_rows;
  p.scales = a.scales;
  p.T = a.T;
  p.H = a.H;
  p.tok_per_item = tok_per_item;
  p.groups = groups;
  p.group_rows = a.H / groups;
  p.item_cost = item_cost;
  p.softmax_scale = a.softmax_scale;
  p.sink = a.sink;
  p.out = a.out;
  p.err = err;
  p.grid = decode_grid(a.T, a.H, a.max_kv_len);
  if (p.grid > 1) {
    p.part_o = static_cast<float*>(a.workspace);
    p.part_lse = p.part_o + static_cast<size_t>(2) * p.grid * nr * kDV;
    p.cuts = reinterpret_cast<Cut*>(p.part_lse + static_cast<size_t>(2) * p.grid * nr);
  }
  return p;
}
// The line's units stay below 2^31 when this many head groups walk it.
inline smla_status_t check_line(const DenseDecodeArgs& a, int groups, int item_cost) {
  const int64_t line = static_cast<int64_t>(a.T) * groups *
                       ((static_cast<int64_t>(a.seqs->max_pages) * a.seqs->page_size + kBK - 1) / kBK + 1 + item_cost);
  if (line >= (int64_t(1) << 30))
    return fail(SMLA_ERR_UNSUPPORTED, "dense decode: T=%d tokens of up to %d pages of %d keys are too much for one call",
                a.T, a.seqs->max_pages, a.seqs->page_size);
  return SMLA_OK;
}
template <int NR>
smla_status_t launch_join(const Params& p, cudaStream_t stream) {
  if (p.grid <= 1) return SMLA_OK;
  join_kernel<NR><<<2 * device_sm_count(), 128 * kJoinGroups, 0, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? SMLA_OK : fail_cuda(e, "dense decode join launch");
}

}  // namespace dd
}  // namespace smla
