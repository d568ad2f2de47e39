// Device helpers shared by the operators that work token by token on a
// ragged batch: the token's sequence and position, and rotary angles.
#pragma once
#include "ptx.cuh"
#include "smla_internal.h"

namespace smla {

// A smla_seqs_t in the form the kernels take.
struct SeqsDev {
  const int32_t* cu_q;
  const int32_t* kv_len;
  const int32_t* page_table;
  int B, max_pages, page_shift;
};
inline SeqsDev seqs_dev(const smla_seqs_t& s) {
  return {s.cu_q, s.kv_len, s.page_table, s.B, s.max_pages, __builtin_ctz(static_cast<unsigned>(s.page_size))};
}

// Sequence of token t, found by the whole warp: the number of cu_q[0..B]
// entries that are <= t, less one.  One strided pass (a warp covers 32
// sequences a load, the loads independent) instead of a binary search's
// chain of dependent loads.  -1 for a token outside every sequence.
SMLA_DEVICE_INLINE int warp_seq_of(const int32_t* cu_q, int B, int t, int lane) {
  int n = 0;
  for (int i = lane; i <= B; i += 32) n += cu_q[i] <= t ? 1 : 0;
  n = __reduce_add_sync(0xffffffffu, n);
  return n > B ? -1 : n - 1;
}

// Position of token t of sequence b (negative where its sequence has more
// new tokens than cached ones).
SMLA_DEVICE_INLINE int token_pos(const SeqsDev& s, int b, int t) {
  return s.kv_len[b] - s.cu_q[b + 1] + t;
}

// Physical row of logical key `key` of sequence b; -1 (and the error
// recorded) when it lies outside the page table or its page outside the pool.
SMLA_DEVICE_INLINE int64_t key_phys_row(const SeqsDev& s, int b, int key, int64_t phys_rows, unsigned* err) {
  if (key < 0 || (key >> s.page_shift) >= s.max_pages) {
    atomicOr(err, kErrShape);
    return -1;
  }
  const int pid = s.page_table[static_cast<int64_t>(b) * s.max_pages + (key >> s.page_shift)];
  const int64_t row = (static_cast<int64_t>(pid) << s.page_shift) | (key & ((1 << s.page_shift) - 1));
  if (pid < 0 || row >= phys_rows) {
    atomicOr(err, kErrPage);
    return -1;
  }
  return row;
}

// frac(f / 2 pi) * 2^64, the turns of one position as a 64-bit fraction, in
// integer arithmetic: f = m 2^e with a 53-bit m, and m times 2^66 / (2 pi) is a
// 117-bit product that is shifted into place; whole turns fall off the top.
// (In float64 arithmetic, of which this GPU does two operations a cycle and
// SM, the angles took most of an append's time.)
SMLA_DEVICE_INLINE unsigned long long rope_step(double f) {
  const unsigned long long bits = static_cast<unsigned long long>(__double_as_longlong(f));
  const int ex = static_cast<int>(bits >> 52) & 0x7ff;
  const unsigned long long m = (bits & 0xfffffffffffffull) | (ex ? 0x10000000000000ull : 0);
  constexpr unsigned long long kC = 11743562013128004906ull;  // round(2^66 / (2 pi))
  const unsigned long long hi = __umul64hi(m, kC), lo = m * kC;
  const int s = 2 + 1075 - (ex ? ex : 1);  // shift right
  unsigned long long r;
  if (s >= 64)
    r = s < 128 ? hi >> (s - 64) : 0ull;
  else if (s > 0)
    r = (hi << (64 - s)) | (lo >> s);
  else
    r = s > -64 ? lo << -s : 0ull;
  return bits >> 63 ? 0ull - r : r;
}

// cos and sin of pos * inv_freq, times `amplitude`: the integer product step *
// pos wraps modulo one turn exactly, so far positions lose nothing to the
// reduction (a 32-bit product pos * inv_freq is off by 2^-24 of the whole
// angle: 0.008 radians at position 130 000).  What is left is the rounding of the
// reduced angle to a float, 2^-24 of itself (of all 64 bits: its upper 32 alone
// are off by 2^-32 of a turn, a thousandth of the slowest pairs' first steps).
SMLA_DEVICE_INLINE void rope_cos_sin(double inv_freq, int pos, float amplitude, float& c, float& s) {
  const unsigned long long phase = rope_step(inv_freq) * static_cast<unsigned long long>(static_cast<long long>(pos));
  const float half_turns = __ll2float_rn(static_cast<long long>(phase)) * 0x1p-63f;
  sincospif(half_turns, &s, &c);
  c *= amplitude;
  s *= amplitude;
}

// Eight consecutive elements as floats.
SMLA_DEVICE_INLINE void unpack_bf16x8(const uint4& v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
SMLA_DEVICE_INLINE uint4 pack_bf16x8(const float (&x)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// (e4m3, nearest even, values past +-448 become +-448)
SMLA_DEVICE_INLINE uint2 pack_e4m3x8(const float (&x)[8]) {
  return make_uint2(static_cast<uint32_t>(f32x2_to_e4m3x2(x[0], x[1])) |
                        (static_cast<uint32_t>(f32x2_to_e4m3x2(x[2], x[3])) << 16),
                    static_cast<uint32_t>(f32x2_to_e4m3x2(x[4], x[5])) |
                        (static_cast<uint32_t>(f32x2_to_e4m3x2(x[6], x[7])) << 16));
}
SMLA_DEVICE_INLINE void unpack_e4m3x8(const uint2& v, float (&x)[8]) {
  const uint32_t w[2] = {v.x, v.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = e4m3x2_to_f16x2(static_cast<uint16_t>(w[i >> 1] >> (16 * (i & 1))));
    const __half2 h2 = *reinterpret_cast<const __half2*>(&h);
    const float2 f = __half22float2(h2);
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

}  // namespace smla
