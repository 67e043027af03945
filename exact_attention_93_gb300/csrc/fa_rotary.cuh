// fa_rotary.cuh -- what the kernels that turn pairs by position share: angles
// (along one axis of positions or several), and rows of 8 elements as fp32.
//
// A warp works on one token; D / 16 lanes cover a head.  With several axes each pair
// has its own position, read by the lane that computes its angle: one load more a
// lane, beside which nothing changes.
#pragma once

#include <type_traits>

#include "fa_serve.h"
#include "sm103_primitives.cuh"

namespace fa {

// Sine and cosine of turn32 * 2^-32 turns (Taylor series about the nearest
// quarter turn; the remainder is at most pi/4, where the first terms left
// out, r^11/11! and r^12/12!, are below 2e-9).
__device__ __forceinline__ void sincos_turns(uint32_t turn32, float& s, float& c) {
  const uint32_t quarter = (turn32 + 0x20000000u) >> 30;
  const int32_t rest = static_cast<int32_t>(turn32 - (quarter << 30));
  const float r = static_cast<float>(rest) * 1.4629180792671596e-9f;  // 2 pi / 2^32
  const float r2 = r * r;
  float ps = fmaf(r2, 2.7557319223985893e-6f, -1.984126984126984e-4f);
  ps = fmaf(r2, ps, 8.333333333333333e-3f);
  ps = fmaf(r2, ps, -1.6666666666666666e-1f);
  const float sn = fmaf(r * r2, ps, r);
  float pc = fmaf(r2, -2.755731922398589e-7f, 2.48015873015873e-5f);
  pc = fmaf(r2, pc, -1.388888888888889e-3f);
  pc = fmaf(r2, pc, 4.1666666666666664e-2f);
  pc = fmaf(r2, pc, -0.5f);
  const float cs = fmaf(r2, pc, 1.f);
  const float a = (quarter & 1u) ? cs : sn, b = (quarter & 1u) ? sn : cs;
  s = (quarter & 2u) ? -a : a;
  c = ((quarter + 1u) & 2u) ? -b : b;
}

// Eight elements as fp32.
template <int kElem>
struct Vec8;

template <>
struct Vec8<kElemFp32> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void load(const uint4* p, const uint4* q) {  // the words apart
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(q);
  }
  __device__ __forceinline__ void store(float* p) const {
    *reinterpret_cast<float4*>(p) = a;
    *reinterpret_cast<float4*>(p + 4) = b;
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
};

template <int kElem>
struct Vec8 {
  uint4 a;
  __device__ __forceinline__ void load(const uint16_t* p) {
    a = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void load(const uint4* p, const uint4*) { a = *p; }
  __device__ __forceinline__ void store(uint16_t* p) const { *reinterpret_cast<uint4*>(p) = a; }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 u = unpack2<kElem == kElemBf16>(w[i]);
      f[2 * i] = u.x;
      f[2 * i + 1] = u.y;
    }
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
    a = make_uint4(pack2<kElem == kElemBf16>(f[0], f[1]), pack2<kElem == kElemBf16>(f[2], f[3]),
                   pack2<kElem == kElemBf16>(f[4], f[5]), pack2<kElem == kElemBf16>(f[6], f[7]));
  }
};

// a / b for a >= 0, b > 0; a 64-bit division is a long instruction sequence.
__device__ __forceinline__ long long quotient(long long a, int b) {
  if ((a >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// A warp's items, `stride` apart: item i is heads of group i % groups of token i /
// groups, which is token n of batch b.  Stepping on takes additions alone; two
// divisions an item were a tenth of the kernels' instructions.
struct ItemWalk {
  int b, n, group;
  __device__ __forceinline__ ItemWalk(long long first, long long items, int stride, int groups, int N)
      : at_(first), items_(items), stride_(stride), groups_(groups), N_(N) {
    const long long token = groups > 1 ? quotient(first, groups) : first;
    group = static_cast<int>(first - token * groups);
    b = static_cast<int>(quotient(token, N));
    n = static_cast<int>(token - static_cast<long long>(b) * N);
    step_group_ = step_b_ = step_n_ = 0;
    if (first + stride < items) {  // (calls of few tokens have one item a warp)
      const int step = stride / groups;
      step_group_ = stride - step * groups;
      step_b_ = step / N;
      step_n_ = step - step_b_ * N;
    }
  }
  __device__ __forceinline__ bool valid() const { return at_ < items_; }
  __device__ __forceinline__ void next() {
    at_ += stride_;
    group += step_group_;
    n += step_n_;
    b += step_b_;
    if (group >= groups_) {
      group -= groups_;
      ++n;
    }
    if (n >= N_) {  // (n was below N, step_n_ is, and 1 was added at most: below 2 N)
      n -= N_;
      ++b;
    }
  }

 private:
  long long at_, items_;
  int stride_, groups_, N_, step_group_, step_n_, step_b_;
};

// The same where a warp keeps to one group of heads: tokens `stride` apart.
struct TokenWalk {
  int b, n;
  __device__ __forceinline__ TokenWalk(int first, long long tokens, int stride, int N)
      : at_(first), tokens_(tokens), stride_(stride), N_(N) {
    b = first / N;
    n = first - b * N;
    step_b_ = stride / N;
    step_n_ = stride - step_b_ * N;
  }
  __device__ __forceinline__ bool valid() const { return at_ < tokens_; }
  // Whether it went into another batch beyond the stride's own.
  __device__ __forceinline__ bool next() {
    at_ += stride_;
    n += step_n_;
    b += step_b_;
    const bool wraps = n >= N_;
    if (wraps) {
      n -= N_;
      ++b;
    }
    return wraps;
  }
  // What an operand's address grows by: with every token, and more when one wraps.
  __device__ __forceinline__ long long step(const RowStrides& s) const {
    return step_b_ * s.batch + step_n_ * s.seq;
  }
  __device__ __forceinline__ long long wrap(const RowStrides& s) const {
    return s.batch - N_ * s.seq;
  }

 private:
  long long at_, tokens_;
  int stride_, N_, step_n_, step_b_;
};

// The rows of one token in up to two operands, heads counted through both: what their
// addresses have in common, once per token.  (The operands' own fields are read where
// every lane reads the same: indexed by a lane's operand they cost a constant load each.)
template <typename T>
struct TokenRows {
  T *q, *k;
  long long q_head, k_head;
  __device__ __forceinline__ TokenRows(T* x0, const RowStrides& s0, T* x1, const RowStrides& s1,
                                       int heads0, int b, int n)
      : q_head(s0.head), k_head(s1.head) {
    q = x0 + b * s0.batch + n * s0.seq;
    k = x1 + b * s1.batch + n * s1.seq - heads0 * s1.head;
  }
  __device__ __forceinline__ T* row(int h, bool second) const {
    return (second ? k : q) + static_cast<unsigned long long>(second ? k_head : q_head) *
                                  static_cast<unsigned>(h);
  }
};

// How the heads of a token are dealt out: to `groups` items of a warp, in each of
// which every lane group takes up to `per` heads, `slots` apart.  As few items as
// kUnroll allows, since the angles are every item's own, and equally large ones.
struct HeadSplit {
  int groups, per;
  HeadSplit(int heads, int slots, int unroll) {
    const int each = (heads + slots - 1) / slots;
    groups = (each + unroll - 1) / unroll;
    per = groups ? (each + groups - 1) / groups : 0;
  }
};

// What a block keeps of its pairs: the 64-bit fraction of a turn per position, and
// where in `positions` a pair's axis begins.
template <int D, bool kAxes>
struct PairTable {
  unsigned long long turns[D / 2];
  long long axis[kAxes ? D / 2 : 1];
  // By every thread of the block, then a barrier.
  __device__ __forceinline__ void fill(const RotaryLaunch& p) {
    const int i = threadIdx.x;
    if (i < p.rotary >> 1) {
      // radians per position -> 64-bit fraction of a turn per position
      const double t = p.inv_freq[i] * 0.15915494309189535;
      const double frac = t - floor(t);
      const unsigned long long u = static_cast<unsigned long long>(frac * 18446744073709551616.0);
      turns[i] = p.inverse ? 0ull - u : u;
      if constexpr (kAxes) axis[i] = p.axis[i] * p.position_astride;
    }
  }
};

// Sines and cosines of a lane's 8 pairs, times the magnitude, token by token.  The
// angles depend on the token alone, so the lane groups of a warp compute a share of
// them each and exchange them by shuffles.
template <int D, bool kAxes>
struct PairAngles {
  static constexpr int kLanes = D / 16;       // lanes of one head
  static constexpr int kSlots = 32 / kLanes;  // heads a warp covers at once
  static constexpr int kShare = 8 / kSlots > 0 ? 8 / kSlots : 1;  // angles of a lane group
  unsigned long long mine[kShare];
  long long axis[kAxes ? kShare : 1];
  __device__ __forceinline__ void load(const PairTable<D, kAxes>& t, int sub, int slot,
                                       bool rotates) {
#pragma unroll
    for (int i = 0; i < kShare; ++i) {
      const int pair = sub * 8 + (slot * kShare + i) % 8;
      mine[i] = rotates ? t.turns[pair] : 0ull;
      if constexpr (kAxes) axis[i] = rotates ? t.axis[pair] : 0;
    }
  }
  // A token's positions, one for all pairs or one for each of the lane's share.
  struct Place {
    long long pos[kAxes ? kShare : 1];
  };
  __device__ __forceinline__ Place place(const RotaryLaunch& p, long long b, long long n) const {
    const long long first = b * p.position_bstride + n;
    Place at;
#pragma unroll
    for (int i = 0; i < (kAxes ? kShare : 1); ++i) {
      const long long o = kAxes ? first + axis[i] : first;
      at.pos[i] = p.position_bits == 32   ? static_cast<const int*>(p.positions)[o]
                  : p.position_bits == 64 ? static_cast<const long long*>(p.positions)[o]
                                          : n;
    }
    return at;
  }
  // (the whole warp)
  __device__ __forceinline__ void at(const Place& place, float magnitude, int sub, float (&sn)[8],
                                     float (&cs)[8]) const {
    float ms[kShare], mc[kShare];
#pragma unroll
    for (int i = 0; i < kShare; ++i) {
      // round the fraction to 32 bits; whole turns wrap away
      const unsigned long long a =
          mine[i] * static_cast<unsigned long long>(place.pos[kAxes ? i : 0]) + 0x80000000ull;
      sincos_turns(static_cast<uint32_t>(a >> 32), ms[i], mc[i]);
      ms[i] *= magnitude;
      mc[i] *= magnitude;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int from = (j / kShare) * kLanes + sub;
      sn[j] = __shfl_sync(0xffffffffu, ms[j % kShare], from);
      cs[j] = __shfl_sync(0xffffffffu, mc[j % kShare], from);
    }
  }
};

// The pairs of a lane's elements a (at e0) and c (at e1).
template <bool kInterleaved>
__device__ __forceinline__ void turn_pairs(float (&a)[8], float (&c)[8], const float (&sn)[8],
                                           const float (&cs)[8]) {
  if constexpr (kInterleaved) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float x1 = a[2 * j], x2 = a[2 * j + 1], z1 = c[2 * j], z2 = c[2 * j + 1];
      a[2 * j] = x1 * cs[j] - x2 * sn[j];
      a[2 * j + 1] = x1 * sn[j] + x2 * cs[j];
      c[2 * j] = z1 * cs[4 + j] - z2 * sn[4 + j];
      c[2 * j + 1] = z1 * sn[4 + j] + z2 * cs[4 + j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float x1 = a[j], x2 = c[j];
      a[j] = x1 * cs[j] - x2 * sn[j];
      c[j] = x1 * sn[j] + x2 * cs[j];
    }
  }
}

}  // namespace fa
