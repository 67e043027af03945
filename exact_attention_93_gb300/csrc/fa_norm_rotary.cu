// fa_norm_rotary.cu -- the root-mean-square norm of each head's row with the
// rotation by position in the same pass, forward and backward.
//
//   r = 1 / sqrt(mean x^2 + eps),  y = magnitude * R(a) (w r x)
//
// R(a) turns pairs as fa_rotary.cu does.  Its transpose is R(-a), so with
// g = magnitude * R(-a) dy
//
//   dw = sum over rows of g r x,   dx = r (w g - x r^2 mean(w g x)).
//
// r is taken from x again in the backward pass, which reads x anyway: nothing but
// the caller's inputs is kept between the two.  HBM is the bound: the forward reads
// and writes each element once, the backward reads x and dy and writes dx.  Norm and
// rotation apart would move the data twice each way.
//
// Work split.  As in fa_rotary.cu: a warp takes a token and D / 16 lanes a head, so a
// row's sums are three shuffles (two for D = 64) among neighbours.  Sums, statistics
// and products are fp32, two at a time (f32x2); values are rounded once, when stored.
// Few registers are left beside a row's values, weights, sines and sums for warps to
// hide the loads behind, so loads are always ahead: forward, the next token's row is
// loaded into the registers that a row has just been read from; backward, where x and
// dy and the running sums leave none, through a ring of asynchronous copies in shared
// memory, in which each lane reads what it copied itself.  A warp keeps to one group of
// heads, so that addresses step from token to token by additions.
//
// dw.  Each lane adds up its 16 columns over all rows that its warp takes; blocks
// work on queries or keys alone, so that one set of sums serves.  A block's lanes
// are added in shared memory and its sums go to the workspace, which a second small
// kernel adds up in a fixed order: the same inputs give the same bits.
//
// Measured, bf16, D = 128: 65536 tokens of 8 + 8 heads forward 87 us, 6.2 TB/s (92 % of the
// measured copy rate), backward 129 us, 6.2 TB/s; 5003 tokens of 32 + 8 heads forward 22 us,
// 32 tokens 3.5.  Steps of the way, forward and backward of the first: one token after
// the other with two divisions each 106 and 189; weights ordered for their readers 102;
// additions for divisions, operands' fields read where all lanes agree 92 and 158;
// a warp's heads fixed 87; the ring 129 (with two heads a lane, three blocks per SM and
// three stages; four blocks spill: 174; four stages 140; one head a lane 150).
#include "fa_norm.h"
#include "fa_rotary.cuh"

namespace fa {
namespace {

constexpr int kNormThreads = 128, kNormWarps = kNormThreads / 32;
// Heads in flight per lane group, and blocks per SM, as many as the registers allow at
// once: all blocks run from beginning to end.
// Forward, 16-bit: four, or five where that makes fewer items of a token's heads (us, four and
// five: 20000 tokens of 16 + 4 heads of 128 41.4 and 38.5, 65536 of 8 + 8 87 and 95).
template <int kElem>
constexpr int kFwdUnroll = kElem == kElemFp32 ? 3 : 4;
template <int kElem>
constexpr int kFwdMost = kElem == kElemFp32 ? 3 : 5;
constexpr int fwd_blocks(int unroll) { return unroll == 4 ? 4 : 3; }
template <int kElem>
constexpr int kBwdUnroll = kElem == kElemFp32 ? 1 : 2;
constexpr int kStages = 3;  // of the backward's ring

// A lane's 16 elements of a row as packed fp32: element i of x1 and x2 holds the first
// and the second elements of pairs 2 i and 2 i + 1.
struct Pairs {
  uint64_t x1[4], x2[4];
  template <bool kInterleaved>
  __device__ __forceinline__ void set(const float (&a)[8], const float (&c)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kInterleaved) {
        const float* v = i < 2 ? a + 4 * i : c + 4 * (i - 2);
        x1[i] = f32x2(v[0], v[2]);
        x2[i] = f32x2(v[1], v[3]);
      } else {
        x1[i] = f32x2(a[2 * i], a[2 * i + 1]);
        x2[i] = f32x2(c[2 * i], c[2 * i + 1]);
      }
    }
  }
  template <bool kInterleaved>
  __device__ __forceinline__ void get(float (&a)[8], float (&c)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 u = split_f32x2(x1[i]), v = split_f32x2(x2[i]);
      if constexpr (kInterleaved) {
        float* to = i < 2 ? a + 4 * i : c + 4 * (i - 2);
        to[0] = u.x; to[1] = v.x; to[2] = u.y; to[3] = v.y;
      } else {
        a[2 * i] = u.x; a[2 * i + 1] = u.y;
        c[2 * i] = v.x; c[2 * i + 1] = v.y;
      }
    }
  }
  template <bool kInterleaved, int kElem>
  __device__ __forceinline__ void from(const Vec8<kElem>& v0, const Vec8<kElem>& v1) {
    float a[8], c[8];
    v0.get(a);
    v1.get(c);
    set<kInterleaved>(a, c);
  }
  template <bool kInterleaved, int kElem>
  __device__ __forceinline__ void to(Vec8<kElem>& v0, Vec8<kElem>& v1) const {
    float a[8], c[8];
    get<kInterleaved>(a, c);
    v0.set(a);
    v1.set(c);
  }
  __device__ __forceinline__ void from(const ulonglong2* w, int step) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const ulonglong2 v = w[i * step];
      x1[i] = v.x;
      x2[i] = v.y;
    }
  }
  __device__ __forceinline__ void times(const Pairs& w) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x1[i] = mul_f32x2(x1[i], w.x1[i]);
      x2[i] = mul_f32x2(x2[i], w.x2[i]);
    }
  }
  __device__ __forceinline__ void times(float f) {
    const uint64_t ff = f32x2(f, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x1[i] = mul_f32x2(x1[i], ff);
      x2[i] = mul_f32x2(x2[i], ff);
    }
  }
  __device__ __forceinline__ float dot(const Pairs& w) const {
    uint64_t s1 = mul_f32x2(x1[0], w.x1[0]), s2 = mul_f32x2(x2[0], w.x2[0]);
#pragma unroll
    for (int i = 1; i < 4; ++i) {
      s1 = fma_f32x2(x1[i], w.x1[i], s1);
      s2 = fma_f32x2(x2[i], w.x2[i], s2);
    }
    const float2 s = split_f32x2(add_f32x2(s1, s2));
    return s.x + s.y;
  }
};

// Packed sines and cosines of a lane's pairs, of one token.
struct Turn {
  uint64_t cs[4], sn[4], neg[4];
  __device__ __forceinline__ Turn(const float (&s)[8], const float (&c)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cs[i] = f32x2(c[2 * i], c[2 * i + 1]);
      sn[i] = f32x2(s[2 * i], s[2 * i + 1]);
      neg[i] = f32x2(-s[2 * i], -s[2 * i + 1]);
    }
  }
  __device__ __forceinline__ void apply(Pairs& p) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t a = p.x1[i], b = p.x2[i];
      p.x1[i] = fma_f32x2(a, cs[i], mul_f32x2(b, neg[i]));
      p.x2[i] = fma_f32x2(a, sn[i], mul_f32x2(b, cs[i]));
    }
  }
};

// Weights as fp32 in shared memory (ones where there are none), in the order in which
// the lanes of a head read them: entry [i][sub] is x1[i], x2[i] of lane sub's Pairs.  Read
// row by row as they lie, lanes 64 bytes apart meet in the same banks (65536 tokens of
// 16 heads: 106 us, interleaved 136).
template <int D, int kElem, bool kInterleaved>
__device__ __forceinline__ void fill_weights(const NormLaunch& p, float4 (*w)[4][D / 16]) {
  constexpr int kLanes = D / 16;
  for (int t = threadIdx.x; t < 2 * 4 * kLanes; t += kNormThreads) {
    const int op = t / (4 * kLanes), i = t / kLanes % 4, sub = t % kLanes;
    const bool halves = sub * 16 < p.rot.rotary && !kInterleaved;
    const int a = halves ? sub * 8 + 2 * i : sub * 16 + (kInterleaved ? 4 * i : 2 * i);
    const int step = kInterleaved ? 2 : 1;  // from a pair's first element to the next pair's
    const int c = kInterleaved ? a + 1 : halves ? (p.rot.rotary >> 1) + a : a + 8;
    const int at[4] = {a, a + step, c, c + step};
    float v[4];
    const void* src = p.weight[op];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (!src) v[e] = 1.f;
      else if (p.weight_elem == kElemFp32) v[e] = static_cast<const float*>(src)[at[e]];
      else
        v[e] = unpack2<kElem == kElemBf16>(static_cast<const uint16_t*>(src)[at[e]]).x;
    }
    w[op][i][sub] = make_float4(v[0], v[1], v[2], v[3]);
  }
}

// Over the lanes of a head.
template <int kLanes>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int m = 1; m < kLanes; m <<= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

template <int kElem>
using ElemOf = typename std::conditional<kElem == kElemFp32, float, uint16_t>::type;

template <int D, int kElem, bool kInterleaved, bool kAxes, int kUnroll>
__global__ void __launch_bounds__(kNormThreads, fwd_blocks(kUnroll))
    norm_rotary_kernel(const __grid_constant__ NormLaunch p, int head_groups, int per) {
  using T = ElemOf<kElem>;
  using Angles = PairAngles<D, kAxes>;
  constexpr int kLanes = Angles::kLanes, kSlots = Angles::kSlots;
  __shared__ PairTable<D, kAxes> table;
  __shared__ float4 weight[2][4][D / 16];
  const RotaryLaunch& r = p.rot;
  table.fill(r);
  fill_weights<D, kElem, kInterleaved>(p, weight);
  __syncthreads();
  const int half = r.rotary >> 1;
  const int lane = threadIdx.x & 31, sub = lane % kLanes, slot = lane / kLanes;
  const bool rotates = sub * 16 < r.rotary;
  const int e0 = rotates && !kInterleaved ? sub * 8 : sub * 16;
  const int e1 = rotates && !kInterleaved ? half + sub * 8 : sub * 16 + 8;
  const int all = r.heads[0] + r.heads[1];
  Angles angles;
  angles.load(table, sub, slot, rotates);
  const T* const x0 = static_cast<const T*>(r.x[0]);
  const T* const x1 = static_cast<const T*>(r.x[1]);
  T* const y0 = static_cast<T*>(r.y[0]);
  T* const y1 = static_cast<T*>(r.y[1]);
  // A warp keeps to one group of heads: where they lie in a token does not change.
  const int id = blockIdx.x * kNormWarps + (threadIdx.x >> 5);
  // (The host launches a warp for every group at least.)
  const int lots = static_cast<int>(gridDim.x) * kNormWarps / head_groups, lot = id / head_groups;
  const int h_first = (id - lot * head_groups) * kSlots * per + slot;
  TokenWalk at(lot, lot < lots ? static_cast<long long>(r.B) * r.N : 0, lots, r.N);
  if (!at.valid()) return;
  Vec8<kElem> v0[kUnroll], v1[kUnroll];
  const auto load = [&](const TokenRows<const T>& rows, int u) {
    const int h = min(h_first + u * kSlots, all - 1);  // (the sums take the whole warp)
    const T* src = rows.row(h, h >= r.heads[0]);
    v0[u].load(src + e0);
    v1[u].load(src + e1);
  };
  const auto rows_at = [&]() {
    return TokenRows<const T>(x0, r.xs[0], x1, r.xs[1], r.heads[0], at.b, at.n);
  };
  {
    const TokenRows<const T> rows = rows_at();
#pragma unroll
    for (int u = 0; u < kUnroll; ++u)
      if (u < per) load(rows, u);
  }
  typename Angles::Place place = angles.place(r, at.b, at.n);
  while (true) {
    float sn[8], cs[8];
    angles.at(place, r.magnitude, sub, sn, cs);
    const Turn turn(sn, cs);
    const TokenRows<T> ys(y0, r.ys[0], y1, r.ys[1], r.heads[0], at.b, at.n);
    at.next();
    const bool more = at.valid();
    const TokenRows<const T> rows = rows_at();
    if (more) place = angles.place(r, at.b, at.n);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (u >= per) break;
      const int h = h_first + u * kSlots;
      const bool second = h >= r.heads[0];
      Pairs x, weights;
      x.from<kInterleaved>(v0[u], v1[u]);
      if (more) load(rows, u);  // into the registers just read: always on its way
      weights.from(reinterpret_cast<const ulonglong2*>(&weight[second][0][sub]), kLanes);
      weights.times(rsqrtf(fmaf(row_sum<kLanes>(x.dot(x)), 1.f / D, p.eps)));
      x.times(weights);
      if (rotates) turn.apply(x);
      if (h >= all) continue;
      Vec8<kElem> o0, o1;
      x.to<kInterleaved>(o0, o1);
      T* y = ys.row(h, second);
      o0.store(y + e0);
      o1.store(y + e1);
    }
    if (!more) break;
  }
}

// 16 bytes from global to shared memory, past the registers.
__device__ __forceinline__ void copy16(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int kPending>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

// What the backward kernel keeps in shared memory.  A lane reads what it copied itself.
template <int D, int kElem, bool kAxes>
struct BwdSmem {
  static constexpr int kWords = kElem == kElemFp32 ? 2 : 1;           // 16-byte words of 8 elements
  static constexpr int kWarpWords = kBwdUnroll<kElem> * 4 * kWords;  // of a lane and stage
  static constexpr int kParts = kNormWarps * 512 / D;  // sums of a block for each column
  union {
    uint4 ring[kNormWarps][kStages][kWarpWords][32];
    float part[kParts][D];  // when the ring has been read
  };
  float4 weight[2][4][D / 16];
  PairTable<D, kAxes> table;
};

// r.x: x, r.y: dx, p.dy: the incoming gradient; r.inverse turns it back.
template <int D, int kElem, bool kInterleaved, bool kAxes>
__global__ void __launch_bounds__(kNormThreads, kNormBlocks)
    norm_rotary_bwd_kernel(const __grid_constant__ NormLaunch p) {
  using T = ElemOf<kElem>;
  using Angles = PairAngles<D, kAxes>;
  using Smem = BwdSmem<D, kElem, kAxes>;
  constexpr int kLanes = Angles::kLanes, kSlots = Angles::kSlots, kUnroll = kBwdUnroll<kElem>;
  constexpr int kWords = Smem::kWords, kVec = 8 / kWords;  // elements of a 16-byte word
  extern __shared__ uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>(smem_raw);
  const RotaryLaunch& r = p.rot;
  s.table.fill(r);
  fill_weights<D, kElem, kInterleaved>(p, s.weight);
  __syncthreads();
  const int half = r.rotary >> 1;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int sub = lane % kLanes, slot = lane / kLanes;
  const bool rotates = sub * 16 < r.rotary;
  const int e0 = rotates && !kInterleaved ? sub * 8 : sub * 16;
  const int e1 = rotates && !kInterleaved ? half + sub * 8 : sub * 16 + 8;
  // this block's operand, and its place among the operand's blocks
  const int w = static_cast<int>(blockIdx.x) >= p.blocks[0];
  const int block = blockIdx.x - (w ? p.blocks[0] : 0);
  const int heads = r.heads[w], groups = p.groups[w], per = p.per[w];
  Angles angles;
  angles.load(s.table, sub, slot, rotates);
  Pairs sums;
#pragma unroll
  for (int i = 0; i < 4; ++i) sums.x1[i] = sums.x2[i] = 0ull;
  // A warp keeps to one group of heads, so that its pointers only step from token to token.
  // (With more groups than warps it takes several, one after the other.)
  const int warps = p.blocks[w] * kNormWarps, lots = max(1, warps / groups);
  const int id = block * kNormWarps + warp, lot = id / groups;
  const auto weights = reinterpret_cast<const ulonglong2*>(&s.weight[w][0][sub]);
  for (int group = id - lot * groups; group < groups; group += warps) {
    const int h_first = group * kSlots * per + slot;
    const long long tokens = lot < lots ? static_cast<long long>(r.B) * r.N : 0;
    TokenWalk at(lot, tokens, lots, r.N), ahead = at;
    const auto first = [&](auto* base, const RowStrides& st) {
      return base + at.b * st.batch + at.n * st.seq + h_first * st.head + e0;
    };
    const T* px = first(static_cast<const T*>(r.x[w]), r.xs[w]);
    const T* pg = first(static_cast<const T*>(p.dy[w]), p.dys[w]);
    T* py = first(static_cast<T*>(r.y[w]), r.ys[w]);
    const long long head_x = kSlots * r.xs[w].head, head_g = kSlots * p.dys[w].head;
    const long long head_y = kSlots * r.ys[w].head;
    const long long step_x = at.step(r.xs[w]), step_g = at.step(p.dys[w]), step_y = at.step(r.ys[w]);
    const long long wrap_x = at.wrap(r.xs[w]), wrap_g = at.wrap(p.dys[w]), wrap_y = at.wrap(r.ys[w]);
    const int second = e1 - e0;
    uint4(*const ring)[Smem::kWarpWords][32] = s.ring[warp];
    // this lane's elements of the token `ahead`, and on to the next
    const auto fetch = [&](int stage) {
      if (ahead.valid()) {
#pragma unroll
        for (int u = 0; u < kUnroll; ++u)
          if (u < per && h_first + u * kSlots < heads) {
#pragma unroll
            for (int j = 0; j < kWords; ++j) {
              uint4(*const to)[32] = ring[stage] + u * 4 * kWords + j;
              const T *x = px + u * head_x + j * kVec, *g = pg + u * head_g + j * kVec;
              copy16(&to[0][lane], x);
              copy16(&to[kWords][lane], x + second);
              copy16(&to[2 * kWords][lane], g);
              copy16(&to[3 * kWords][lane], g + second);
            }
          }
        const bool wraps = ahead.next();
        px += step_x + (wraps ? wrap_x : 0);
        pg += step_g + (wraps ? wrap_g : 0);
      }
      copies_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);
    int stage = 0;
    typename Angles::Place place{};
    if (at.valid()) place = angles.place(r, at.b, at.n);
    while (at.valid()) {
      fetch(stage == 0 ? kStages - 1 : stage - 1);  // (the stage before has been read)
      float sn[8], cs[8];
      angles.at(place, r.magnitude, sub, sn, cs);
      const Turn turn(sn, cs);
      const bool wraps = at.next();
      if (at.valid()) place = angles.place(r, at.b, at.n);
      copies_wait<kStages - 1>();
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        if (u >= per) break;
        Vec8<kElem> v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[i].load(&ring[stage][(u * 4 + i) * kWords][lane], &ring[stage][(u * 4 + i) * kWords + kWords - 1][lane]);
        Pairs x, g, gw;
        x.from<kInterleaved>(v[0], v[1]);
        g.from<kInterleaved>(v[2], v[3]);
        if (rotates) turn.apply(g);
        gw.from(weights, kLanes);
        gw.times(g);
        const float square = row_sum<kLanes>(x.dot(x)), mixed = row_sum<kLanes>(x.dot(gw));
        if (h_first + u * kSlots < heads) {
          const float rs = rsqrtf(fmaf(square, 1.f / D, p.eps));
          const float k = -mixed * (1.f / D) * rs * rs;
          const uint64_t kk = f32x2(k, k), rr = f32x2(rs, rs);
          x.times(rs);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            sums.x1[j] = fma_f32x2(g.x1[j], x.x1[j], sums.x1[j]);
            sums.x2[j] = fma_f32x2(g.x2[j], x.x2[j], sums.x2[j]);
            x.x1[j] = fma_f32x2(gw.x1[j], rr, mul_f32x2(x.x1[j], kk));
            x.x2[j] = fma_f32x2(gw.x2[j], rr, mul_f32x2(x.x2[j], kk));
          }
          Vec8<kElem> o0, o1;
          x.to<kInterleaved>(o0, o1);
          o0.store(py + u * head_y);
          o1.store(py + u * head_y + second);
        }
      }
      py += step_y + (wraps ? wrap_y : 0);
      stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    copies_wait<0>();
  }
  if (!p.dweight[w]) return;
  __syncthreads();  // the ring has been read
  float* mine = s.part[warp * kSlots + slot];
  float sa[8], sc[8];
  sums.get<kInterleaved>(sa, sc);
#pragma unroll
  for (int j = 0; j < 8; j += 4) {
    *reinterpret_cast<float4*>(mine + e0 + j) = make_float4(sa[j], sa[j + 1], sa[j + 2], sa[j + 3]);
    *reinterpret_cast<float4*>(mine + e1 + j) = make_float4(sc[j], sc[j + 1], sc[j + 2], sc[j + 3]);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += kNormThreads) {
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < Smem::kParts; ++i) sum += s.part[i][d];
    p.partial[static_cast<long long>(blockIdx.x) * D + d] = sum;
  }
}

// Adds up the blocks' sums: a block takes 8 columns of one operand, 32 threads each.
constexpr int kSumColumns = 8, kSumThreads = 256;

__global__ void __launch_bounds__(kSumThreads)
    norm_weight_kernel(const __grid_constant__ NormLaunch p) {
  pdl_wait_and_release();
  __shared__ float part[kSumThreads / kSumColumns][kSumColumns];
  const int w = blockIdx.y;
  if (!p.dweight[w]) return;
  const int col = threadIdx.x % kSumColumns, row = threadIdx.x / kSumColumns;
  constexpr int kRows = kSumThreads / kSumColumns;
  const int d = blockIdx.x * kSumColumns + col;
  const float* src = p.partial + static_cast<long long>(w ? p.blocks[0] : 0) * p.rot.D + d;
  float s = 0.f;
#pragma unroll 8
  for (int i = row; i < p.blocks[w]; i += kRows) s += src[static_cast<long long>(i) * p.rot.D];
  part[row][col] = s;
  __syncthreads();
  if (row == 0) {
    for (int i = 1; i < kRows; ++i) s += part[i][col];
    if (p.weight_elem == kElemFp32) static_cast<float*>(p.dweight[w])[d] = s;
    else
      static_cast<uint16_t*>(p.dweight[w])[d] = static_cast<uint16_t>(
          p.weight_elem == kElemBf16 ? pack2<true>(s, 0.f) : pack2<false>(s, 0.f));
  }
}

template <int D, int kElem, bool kInterleaved, bool kAxes, int kUnroll>
cudaError_t launch_fwd_u(const NormLaunch& a, const HeadSplit& split, cudaStream_t s) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const long long items = static_cast<long long>(a.rot.B) * a.rot.N * split.groups;
  // (warps for every group of heads, however few tokens there are)
  const long long most = std::max(static_cast<long long>(fwd_blocks(kUnroll)) * sms,
                                  (split.groups + kNormWarps - 1LL) / kNormWarps);
  const long long blocks = (items + kNormWarps - 1) / kNormWarps;
  norm_rotary_kernel<D, kElem, kInterleaved, kAxes, kUnroll>
      <<<static_cast<unsigned>(blocks < most ? blocks : most), kNormThreads, 0, s>>>(
          a, split.groups, split.per);
  return cudaGetLastError();
}

template <int D, int kElem, bool kInterleaved, bool kAxes>
cudaError_t launch_fwd_t(const NormLaunch& a, cudaStream_t s) {
  const int heads = a.rot.heads[0] + a.rot.heads[1], slots = 32 / (D / 16);
  const HeadSplit split(heads, slots, kFwdUnroll<kElem>), wide(heads, slots, kFwdMost<kElem>);
  if (wide.groups < split.groups)
    return launch_fwd_u<D, kElem, kInterleaved, kAxes, kFwdMost<kElem>>(a, wide, s);
  return launch_fwd_u<D, kElem, kInterleaved, kAxes, kFwdUnroll<kElem>>(a, split, s);
}

template <int D, int kElem, bool kInterleaved, bool kAxes>
cudaError_t launch_bwd_t(const NormLaunch& a, cudaStream_t s) {
  NormLaunch p = a;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  // the operands' shares of the blocks, by the rows they have
  const long long tokens = static_cast<long long>(a.rot.B) * a.rot.N;
  const long long most = static_cast<long long>(kNormBlocks) * sms;
  long long need[2], all = 0;
  for (int w = 0; w < 2; ++w) {
    const HeadSplit split(a.rot.heads[w], 32 / (D / 16), kBwdUnroll<kElem>);
    p.groups[w] = split.groups;
    p.per[w] = split.per;
    need[w] = (tokens * split.groups + kNormWarps - 1) / kNormWarps;
    all += need[w];
  }
  p.blocks[0] = static_cast<int>(need[0]);
  p.blocks[1] = static_cast<int>(need[1]);
  if (all > most) {
    p.blocks[1] = need[1] ? static_cast<int>(std::max(1LL, most * need[1] / all)) : 0;
    p.blocks[0] = static_cast<int>(most) - p.blocks[1];
  }
  auto kern = norm_rotary_bwd_kernel<D, kElem, kInterleaved, kAxes>;
  constexpr int kBytes = static_cast<int>(sizeof(BwdSmem<D, kElem, kAxes>));
  static AttrCache configured;
  if ((e = ensure_dynamic_smem(kern, kBytes, configured)) != cudaSuccess) return e;
  kern<<<static_cast<unsigned>(p.blocks[0] + p.blocks[1]), kNormThreads, kBytes, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess || (!p.dweight[0] && !p.dweight[1])) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(D / kSumColumns, 2);
  cfg.blockDim = dim3(kSumThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, norm_weight_kernel, p);
}

template <int D, int kElem>
cudaError_t launch_norm_t(const NormLaunch& a, bool backward, cudaStream_t s) {
  const bool axes = a.rot.position_axes > 1;
  if (a.rot.interleaved) {
    if (axes)
      return backward ? launch_bwd_t<D, kElem, true, true>(a, s)
                      : launch_fwd_t<D, kElem, true, true>(a, s);
    return backward ? launch_bwd_t<D, kElem, true, false>(a, s)
                    : launch_fwd_t<D, kElem, true, false>(a, s);
  }
  if (axes)
    return backward ? launch_bwd_t<D, kElem, false, true>(a, s)
                    : launch_fwd_t<D, kElem, false, true>(a, s);
  return backward ? launch_bwd_t<D, kElem, false, false>(a, s)
                  : launch_fwd_t<D, kElem, false, false>(a, s);
}

template <int D>
cudaError_t launch_norm_d(const NormLaunch& a, bool backward, cudaStream_t s) {
  switch (a.rot.elem) {
    case kElemBf16: return launch_norm_t<D, kElemBf16>(a, backward, s);
    case kElemFp16: return launch_norm_t<D, kElemFp16>(a, backward, s);
    default: return launch_norm_t<D, kElemFp32>(a, backward, s);
  }
}

}  // namespace

cudaError_t launch_norm_rotary(const NormLaunch& a, bool backward, cudaStream_t s) {
  return a.rot.D == 64 ? launch_norm_d<64>(a, backward, s) : launch_norm_d<128>(a, backward, s);
}

}  // namespace fa
