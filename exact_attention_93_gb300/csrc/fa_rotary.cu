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
// 512 / D heads at a time.  The angles of a lane's 8 pairs depend on the
// token alone and serve all of its heads; the lane groups of a warp compute
// a share of them each and exchange them by shuffles.
//
// Measured: 65536 tokens of 16 heads of 128, bf16, 80.7 us, 6.65 TB/s, 98 % of
// the measured copy rate; 5003 tokens of 40 heads 18 us; 32 tokens of 40 heads
// 3.2 us.
#include <type_traits>

#include "fa_serve.h"
#include "sm103_primitives.cuh"

namespace fa {
namespace {

constexpr int kRotThreads = 128;
// Heads in flight per lane group: 128 bytes a lane.  (fp32: 28.0 us with four,
// 26.2 with two, 1860 tokens of 72 heads of 128.)
template <int kElem>
constexpr int kUnroll = kElem == kElemFp32 ? 2 : 4;

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

template <int D, int kElem, bool kInterleaved>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(const __grid_constant__ RotaryLaunch p,
                                                             int head_groups, long long n_items) {
  using T = typename std::conditional<kElem == kElemFp32, float, uint16_t>::type;
  constexpr int kLanes = D / 16;         // lanes of one head
  constexpr int kSlots = 32 / kLanes;    // heads a warp covers at once
  constexpr int kShare = 8 / kSlots > 0 ? 8 / kSlots : 1;  // angles each lane group computes
  __shared__ unsigned long long turns[D / 2];
  const int half = p.rotary >> 1;
  if (threadIdx.x < half) {
    // radians per position -> 64-bit fraction of a turn per position
    const double t = p.inv_freq[threadIdx.x] * 0.15915494309189535;
    const double frac = t - floor(t);
    const unsigned long long u = static_cast<unsigned long long>(frac * 18446744073709551616.0);
    turns[threadIdx.x] = p.inverse ? 0ull - u : u;
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, sub = lane % kLanes, slot = lane / kLanes;
  const bool rotates = sub * 16 < p.rotary;
  // the lane's two groups of eight elements, and its pairs in inv_freq
  const int e0 = rotates && !kInterleaved ? sub * 8 : sub * 16;
  const int e1 = rotates && !kInterleaved ? half + sub * 8 : sub * 16 + 8;
  const int all = p.heads[0] + p.heads[1];
  unsigned long long mine[kShare];  // this lane group's share of the pairs' turns
#pragma unroll
  for (int i = 0; i < kShare; ++i) {
    const int pair = sub * 8 + (slot * kShare + i) % 8;
    mine[i] = rotates ? turns[pair] : 0ull;
  }
  for (long long item = blockIdx.x * (kRotThreads / 32) + (threadIdx.x >> 5); item < n_items;
       item += static_cast<long long>(gridDim.x) * (kRotThreads / 32)) {
    const long long token = item / head_groups;
    const int hg = static_cast<int>(item - token * head_groups);
    const long long b = token / p.N, n = token - b * p.N;
    const int h_first = hg * (kSlots * kUnroll<kElem>) + slot;
    Vec8<kElem> v0[kUnroll<kElem>], v1[kUnroll<kElem>];
#pragma unroll
    for (int u = 0; u < kUnroll<kElem>; ++u) {
      const int h = h_first + u * kSlots;
      if (h < all) {
        const int w = h >= p.heads[0];
        const T* x = static_cast<const T*>(p.x[w]) + b * p.xs[w].batch + n * p.xs[w].seq +
                     (h - (w ? p.heads[0] : 0)) * p.xs[w].head;
        v0[u].load(x + e0);
        v1[u].load(x + e1);
      }
    }
    long long pos = n;
    if (p.position_bits == 32)
      pos = static_cast<const int*>(p.positions)[b * p.position_bstride + n];
    else if (p.position_bits == 64)
      pos = static_cast<const long long*>(p.positions)[b * p.position_bstride + n];
    float ms[kShare], mc[kShare];
#pragma unroll
    for (int i = 0; i < kShare; ++i) {
      // round the fraction to 32 bits; whole turns wrap away
      const unsigned long long a = mine[i] * static_cast<unsigned long long>(pos) + 0x80000000ull;
      sincos_turns(static_cast<uint32_t>(a >> 32), ms[i], mc[i]);
      ms[i] *= p.magnitude;
      mc[i] *= p.magnitude;
    }
    float sn[8], cs[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int from = (j / kShare) * kLanes + sub;
      sn[j] = __shfl_sync(0xffffffffu, ms[j % kShare], from);
      cs[j] = __shfl_sync(0xffffffffu, mc[j % kShare], from);
    }
#pragma unroll
    for (int u = 0; u < kUnroll<kElem>; ++u) {
      const int h = h_first + u * kSlots;
      if (h >= all) continue;
      if (rotates) {
        float a[8], c[8];
        v0[u].get(a);
        v1[u].get(c);
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
        v0[u].set(a);
        v1[u].set(c);
      }
      const int w = h >= p.heads[0];
      T* y = static_cast<T*>(p.y[w]) + b * p.ys[w].batch + n * p.ys[w].seq +
             (h - (w ? p.heads[0] : 0)) * p.ys[w].head;
      v0[u].store(y + e0);
      v1[u].store(y + e1);
    }
  }
}

template <int D, int kElem, bool kInterleaved>
cudaError_t launch_rotary_t(const RotaryLaunch& a, cudaStream_t s) {
  constexpr int kHeads = 32 / (D / 16) * kUnroll<kElem>;  // heads of one work item
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int groups = (a.heads[0] + a.heads[1] + kHeads - 1) / kHeads;
  const long long items = static_cast<long long>(a.B) * a.N * groups;
  const long long per_block = kRotThreads / 32;
  const long long blocks = (items + per_block - 1) / per_block;
  // Blocks stay for several items, as each first turns inv_freq into fractions of
  // a turn in fp64; but few enough items that they end together (65536 tokens of
  // 16 heads: 86.5 us with 16 blocks per SM, 80.5 with 64, 83.6 with one item each).
  const long long most = 64LL * sms;
  rotary_kernel<D, kElem, kInterleaved>
      <<<static_cast<unsigned>(blocks < most ? blocks : most), kRotThreads, 0, s>>>(a, groups, items);
  return cudaGetLastError();
}

template <int D, int kElem>
cudaError_t launch_rotary_d(const RotaryLaunch& a, cudaStream_t s) {
  return a.interleaved ? launch_rotary_t<D, kElem, true>(a, s)
                       : launch_rotary_t<D, kElem, false>(a, s);
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
