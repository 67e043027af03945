// fa_rotary.cu -- rotary positions, forward and (inverse) backward.
//
// Pair (x1, x2) at position p is the complex number x1 + i x2 times
// magnitude * e^(i a), a = p * inv_freq.  One pass over the data: each
// element is read and written once, so the bound is HBM (a bf16 element
// costs 4 bytes; the arithmetic, 3 fp32 operations, is free beside them).
//
// Angles.  p * inv_freq in fp32 loses a whole turn's worth of accuracy for
// far positions, and fp64 arithmetic is slow on this chip.  Instead
// inv_freq / 2 pi is held as a 64-bit fraction of a turn; multiplying by the
// integer position modulo 2^64 then drops whole turns exactly and leaves the
// angle good to p * 2^-53 turns (the fp64 rounding of inv_freq itself).  The
// top 32 bits split into the nearest quarter turn and a remainder within an
// eighth, for which Taylor polynomials of sine and cosine reach fp32 rounding.
//
// Work split.  A warp takes one token and up to kUnroll heads per lane group:
// D / 16 lanes cover a head, two 16-byte loads each (elements i and
// i + rotary/2, or 16 neighbours when interleaved), so a warp covers
// 512 / D heads at a time; the first loads of 16-bit rows are on their way while the pairs' table
// is filled.  The angles of a lane's 8 pairs depend on the
// token alone and serve all of its heads; the lane groups of a warp compute
// a share of them each and exchange them by shuffles.
//
// Measured: 65536 tokens of 16 heads of 128, bf16, 80.4 us, 6.7 TB/s, the measured
// copy rate; 20000 tokens of 20 heads 34 us; 5003 tokens of 40 heads 18.5 us; 32 tokens of
// 40 heads 2.6 us.  Along three axes, 32768 tokens of 20 heads 53 us, 6.3 TB/s.  (With four
// heads in flight instead of five, and the last item of a token's heads left with the
// rest, 20 heads took 66 us: one head in four of the second item's was there.)
#include "fa_rotary.cuh"

namespace fa {
namespace {

constexpr int kRotThreads = 128;
// Heads in flight per lane group: as many in each of a token's items, and few items, as
// each works its angles out anew; two where there are no more, for more warps then.  (us, five
// and two: 30000 tokens of 8 heads of 64 20.9 and 16.3, 100000 of 2 of 128 57.9 and 43.4.
// fp32, three and two: 1860 tokens of 72 heads of 128 22.9 and 23.1, 20000 of 16 57.1 and 54.1.)
// Two also where these make no more than kFewItems items per SM: a call then costs what one
// warp takes.  (Five and two, of 40 heads of 128: 32 tokens 3.0 and 2.6, 250 tokens, 8 items per
// SM, 3.13 and 3.06, 500 3.6 and 3.8.)
template <int kElem>
constexpr int kMostHeads = kElem == kElemFp32 ? 2 : 5;
constexpr int kFewHeads = 2;
constexpr long long kFewItems = 8;
// fp32 rows take twice the registers, and loaded across the filling of the pairs' table they
// leave room for fewer blocks: there they are loaded behind it.  (us, ahead and behind: 500 tokens
// of 40 heads of 128 6.7 and 6.3, 1860 of 72 23.3 and 23.1.)
template <int kElem>
constexpr bool kLoadsAhead = kElem != kElemFp32;

template <int D, int kElem, bool kInterleaved, bool kAxes, int kUnroll>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const __grid_constant__ RotaryLaunch p,
                                                             int head_groups, int per,
                                                             long long n_items) {
  using T = typename std::conditional<kElem == kElemFp32, float, uint16_t>::type;
  using Angles = PairAngles<D, kAxes>;
  constexpr int kLanes = Angles::kLanes, kSlots = Angles::kSlots;
  __shared__ PairTable<D, kAxes> table;
  const int half = p.rotary >> 1;
  const int lane = threadIdx.x & 31, sub = lane % kLanes, slot = lane / kLanes;
  const bool rotates = sub * 16 < p.rotary;
  // the lane's two groups of eight elements, and its pairs in inv_freq
  const int e0 = rotates && !kInterleaved ? sub * 8 : sub * 16;
  const int e1 = rotates && !kInterleaved ? half + sub * 8 : sub * 16 + 8;
  const int all = p.heads[0] + p.heads[1];
  const T* const x0 = static_cast<const T*>(p.x[0]);
  const T* const x1 = static_cast<const T*>(p.x[1]);
  T* const y0 = static_cast<T*>(p.y[0]);
  T* const y1 = static_cast<T*>(p.y[1]);
  ItemWalk at(blockIdx.x * (kRotThreads / 32LL) + (threadIdx.x >> 5), n_items,
              static_cast<int>(gridDim.x) * (kRotThreads / 32), head_groups, p.N);
  Vec8<kElem> v0[kUnroll], v1[kUnroll];
  const auto load = [&]() {
    const TokenRows<const T> xs(x0, p.xs[0], x1, p.xs[1], p.heads[0], at.b, at.n);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = (at.group * per + u) * kSlots + slot;
      if (u < per && h < all) {
        const T* x = xs.row(h, h >= p.heads[0]);
        v0[u].load(x + e0);
        v1[u].load(x + e1);
      }
    }
  };
  if (kLoadsAhead<kElem> && at.valid()) load();  // on its way while the table is filled
  table.fill(p);
  __syncthreads();
  if (!kLoadsAhead<kElem> && at.valid()) load();
  Angles angles;
  angles.load(table, sub, slot, rotates);
  while (at.valid()) {
    const int h_first = at.group * kSlots * per + slot;
    float sn[8], cs[8];
    angles.at(angles.place(p, at.b, at.n), p.magnitude, sub, sn, cs);
    const TokenRows<T> ys(y0, p.ys[0], y1, p.ys[1], p.heads[0], at.b, at.n);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h_first + u * kSlots;
      if (u >= per || h >= all) continue;
      if (rotates) {
        float a[8], c[8];
        v0[u].get(a);
        v1[u].get(c);
        turn_pairs<kInterleaved>(a, c, sn, cs);
        v0[u].set(a);
        v1[u].set(c);
      }
      T* y = ys.row(h, h >= p.heads[0]);
      v0[u].store(y + e0);
      v1[u].store(y + e1);
    }
    at.next();
    if (at.valid()) load();
  }
}

template <int D, int kElem, bool kInterleaved, bool kAxes, int kUnroll>
cudaError_t launch_rotary_u(const RotaryLaunch& a, cudaStream_t s) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const HeadSplit split(a.heads[0] + a.heads[1], 32 / (D / 16), kUnroll);
  const long long items = static_cast<long long>(a.B) * a.N * split.groups;
  const long long per_block = kRotThreads / 32;
  const long long blocks = (items + per_block - 1) / per_block;
  // Blocks stay for several items, as each first turns inv_freq into fractions of
  // a turn in fp64; but few enough items that they end together (65536 tokens of
  // 16 heads: 86.5 us with 16 blocks per SM, 80.5 with 64, 83.6 with one item each).
  const long long most = 64LL * sms;
  rotary_kernel<D, kElem, kInterleaved, kAxes, kUnroll>
      <<<static_cast<unsigned>(blocks < most ? blocks : most), kRotThreads, 0, s>>>(
          a, split.groups, split.per, items);
  return cudaGetLastError();
}

template <int D, int kElem, bool kInterleaved, bool kAxes>
cudaError_t launch_rotary_t(const RotaryLaunch& a, cudaStream_t s) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const HeadSplit split(a.heads[0] + a.heads[1], 32 / (D / 16), kFewHeads);
  if (split.groups <= 1 || static_cast<long long>(a.B) * a.N * split.groups <= kFewItems * sms)
    return launch_rotary_u<D, kElem, kInterleaved, kAxes, kFewHeads>(a, s);
  return launch_rotary_u<D, kElem, kInterleaved, kAxes, kMostHeads<kElem>>(a, s);
}

template <int D, int kElem>
cudaError_t launch_rotary_d(const RotaryLaunch& a, cudaStream_t s) {
  if (a.position_axes > 1)
    return a.interleaved ? launch_rotary_t<D, kElem, true, true>(a, s)
                         : launch_rotary_t<D, kElem, false, true>(a, s);
  return a.interleaved ? launch_rotary_t<D, kElem, true, false>(a, s)
                       : launch_rotary_t<D, kElem, false, false>(a, s);
}

template <int D>
cudaError_t launch_rotary_e(const RotaryLaunch& a, cudaStream_t s) {
  switch (a.elem) {
    case kElemBf16: return launch_rotary_d<D, kElemBf16>(a, s);
    case kElemFp16: return launch_rotary_d<D, kElemFp16>(a, s);
    default: return launch_rotary_d<D, kElemFp32>(a, s);
  }
}

}  // namespace

cudaError_t launch_rotary(const RotaryLaunch& a, cudaStream_t s) {
  return a.D == 64 ? launch_rotary_e<64>(a, s) : launch_rotary_e<128>(a, s);
}

}  // namespace fa
