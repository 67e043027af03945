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
// and products are fp32; values are rounded once, when stored.
//
// dw.  Each lane adds up its 16 columns over all rows that its warp takes; blocks
// work on queries or keys alone, so that one set of sums serves.  A block's lanes
// are added in shared memory and its sums go to the workspace, which a second small
// kernel adds up in a fixed order: the same inputs give the same bits.
#include "fa_norm.h"
#include "fa_rotary.cuh"

namespace fa {
namespace {

constexpr int kNormThreads = 128, kNormWarps = kNormThreads / 32;
template <int kElem>
constexpr int kFwdUnroll = kElem == kElemFp32 ? 2 : 4;  // heads in flight per lane group
template <int kElem>
constexpr int kBwdUnroll = kElem == kElemFp32 ? 1 : 2;

// Weights as fp32 in shared memory; ones where there are none.
template <int D, int kElem>
__device__ __forceinline__ void fill_weights(const NormLaunch& p, float (*w)[D]) {
  for (int i = threadIdx.x; i < 2 * D; i += kNormThreads) {
    const void* src = p.weight[i / D];
    const int d = i % D;
    float v = 1.f;
    if (src) {
      if (p.weight_elem == kElemFp32) v = static_cast<const float*>(src)[d];
      else if (kElem == kElemBf16) v = unpack2<true>(static_cast<const uint16_t*>(src)[d]).x;
      else v = unpack2<false>(static_cast<const uint16_t*>(src)[d]).x;
    }
    w[i / D][d] = v;
  }
}

__device__ __forceinline__ void load8(float (&f)[8], const float* p) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
  f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

__device__ __forceinline__ float dot8(const float (&a)[8], const float (&b)[8]) {
  float s = a[0] * b[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) s = fmaf(a[i], b[i], s);
  return s;
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

template <int kElem>
__device__ __forceinline__ long long row_offset(const RowStrides& st, long long b, long long n,
                                                int h) {
  return b * st.batch + n * st.seq + h * st.head;
}

template <int D, int kElem, bool kInterleaved, bool kAxes>
__global__ void __launch_bounds__(kNormThreads)
    norm_rotary_kernel(const __grid_constant__ NormLaunch p, int head_groups, long long n_items) {
  using T = ElemOf<kElem>;
  using Angles = PairAngles<D, kAxes>;
  constexpr int kLanes = Angles::kLanes, kSlots = Angles::kSlots, kUnroll = kFwdUnroll<kElem>;
  __shared__ PairTable<D, kAxes> table;
  __shared__ alignas(16) float weight[2][D];
  const RotaryLaunch& r = p.rot;
  table.fill(r);
  fill_weights<D, kElem>(p, weight);
  __syncthreads();
  const int half = r.rotary >> 1;
  const int lane = threadIdx.x & 31, sub = lane % kLanes, slot = lane / kLanes;
  const bool rotates = sub * 16 < r.rotary;
  const int e0 = rotates && !kInterleaved ? sub * 8 : sub * 16;
  const int e1 = rotates && !kInterleaved ? half + sub * 8 : sub * 16 + 8;
  const int all = r.heads[0] + r.heads[1];
  Angles angles;
  angles.load(table, sub, slot, rotates);
  for (long long item = blockIdx.x * static_cast<long long>(kNormWarps) + (threadIdx.x >> 5);
       item < n_items; item += static_cast<long long>(gridDim.x) * kNormWarps) {
    const long long token = item / head_groups;
    const int hg = static_cast<int>(item - token * head_groups);
    const long long b = token / r.N, n = token - b * r.N;
    const int h_first = hg * (kSlots * kUnroll) + slot;
    Vec8<kElem> v0[kUnroll], v1[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = min(h_first + u * kSlots, all - 1);  // (the sums take the whole warp)
      const int w = h >= r.heads[0];
      const T* x = static_cast<const T*>(r.x[w]) +
                   row_offset<kElem>(r.xs[w], b, n, h - (w ? r.heads[0] : 0));
      v0[u].load(x + e0);
      v1[u].load(x + e1);
    }
    float sn[8], cs[8];
    angles.at(r, b, n, sub, sn, cs);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h_first + u * kSlots, w = h >= r.heads[0];
      float a[8], c[8], wa[8], wc[8];
      v0[u].get(a);
      v1[u].get(c);
      const float sum = row_sum<kLanes>(dot8(a, a) + dot8(c, c));
      const float rs = __frsqrt_rn(fmaf(sum, 1.f / D, p.eps));
      load8(wa, weight[w] + e0);
      load8(wc, weight[w] + e1);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        a[j] *= rs * wa[j];
        c[j] *= rs * wc[j];
      }
      if (rotates) turn_pairs<kInterleaved>(a, c, sn, cs);
      if (h >= all) continue;
      v0[u].set(a);
      v1[u].set(c);
      T* y = static_cast<T*>(r.y[w]) + row_offset<kElem>(r.ys[w], b, n, h - (w ? r.heads[0] : 0));
      v0[u].store(y + e0);
      v1[u].store(y + e1);
    }
  }
}

// r.x: x, r.y: dx, p.dy: the incoming gradient; r.inverse turns it back.
template <int D, int kElem, bool kInterleaved, bool kAxes>
__global__ void __launch_bounds__(kNormThreads)
    norm_rotary_bwd_kernel(const __grid_constant__ NormLaunch p) {
  using T = ElemOf<kElem>;
  using Angles = PairAngles<D, kAxes>;
  constexpr int kLanes = Angles::kLanes, kSlots = Angles::kSlots, kUnroll = kBwdUnroll<kElem>;
  constexpr int kParts = kNormWarps * kSlots;  // sums of a block for each column
  __shared__ PairTable<D, kAxes> table;
  __shared__ alignas(16) float weight[2][D];
  __shared__ alignas(16) float part[kParts][D];
  const RotaryLaunch& r = p.rot;
  table.fill(r);
  fill_weights<D, kElem>(p, weight);
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
  const int heads = r.heads[w], groups = (heads + kSlots * kUnroll - 1) / (kSlots * kUnroll);
  const long long n_items = static_cast<long long>(r.B) * r.N * groups;
  Angles angles;
  angles.load(table, sub, slot, rotates);
  float wa[8], wc[8], sa[8] = {}, sc[8] = {};
  load8(wa, weight[w] + e0);
  load8(wc, weight[w] + e1);
  const T* const xs = static_cast<const T*>(r.x[w]);
  const T* const gs = static_cast<const T*>(p.dy[w]);
  for (long long item = static_cast<long long>(block) * kNormWarps + warp; item < n_items;
       item += static_cast<long long>(p.blocks[w]) * kNormWarps) {
    const long long token = item / groups;
    const int hg = static_cast<int>(item - token * groups);
    const long long b = token / r.N, n = token - b * r.N;
    const int h_first = hg * (kSlots * kUnroll) + slot;
    Vec8<kElem> x0[kUnroll], x1[kUnroll], g0[kUnroll], g1[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = min(h_first + u * kSlots, heads - 1);
      const T* x = xs + row_offset<kElem>(r.xs[w], b, n, h);
      const T* g = gs + row_offset<kElem>(p.dys[w], b, n, h);
      x0[u].load(x + e0);
      x1[u].load(x + e1);
      g0[u].load(g + e0);
      g1[u].load(g + e1);
    }
    float sn[8], cs[8];
    angles.at(r, b, n, sub, sn, cs);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h_first + u * kSlots;
      float a[8], c[8], ga[8], gc[8];
      x0[u].get(a);
      x1[u].get(c);
      g0[u].get(ga);
      g1[u].get(gc);
      if (rotates) turn_pairs<kInterleaved>(ga, gc, sn, cs);
      float square = dot8(a, a) + dot8(c, c), mixed = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        mixed = fmaf(ga[j] * wa[j], a[j], mixed);
        mixed = fmaf(gc[j] * wc[j], c[j], mixed);
      }
      square = row_sum<kLanes>(square);
      mixed = row_sum<kLanes>(mixed);
      if (h >= heads) continue;
      const float rs = __frsqrt_rn(fmaf(square, 1.f / D, p.eps));
      const float k = mixed * (1.f / D) * rs * rs;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sa[j] = fmaf(ga[j], a[j] * rs, sa[j]);
        sc[j] = fmaf(gc[j], c[j] * rs, sc[j]);
        a[j] = rs * fmaf(ga[j], wa[j], -a[j] * k);
        c[j] = rs * fmaf(gc[j], wc[j], -c[j] * k);
      }
      x0[u].set(a);
      x1[u].set(c);
      T* dx = static_cast<T*>(r.y[w]) + row_offset<kElem>(r.ys[w], b, n, h);
      x0[u].store(dx + e0);
      x1[u].store(dx + e1);
    }
  }
  if (!p.dweight[w]) return;
  float* mine = part[warp * kSlots + slot];
#pragma unroll
  for (int j = 0; j < 8; j += 4) {
    *reinterpret_cast<float4*>(mine + e0 + j) = make_float4(sa[j], sa[j + 1], sa[j + 2], sa[j + 3]);
    *reinterpret_cast<float4*>(mine + e1 + j) = make_float4(sc[j], sc[j + 1], sc[j + 2], sc[j + 3]);
  }
  __syncthreads();
  for (int d = threadIdx.x; d < D; d += kNormThreads) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kParts; ++i) s += part[i][d];
    p.partial[static_cast<long long>(blockIdx.x) * D + d] = s;
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

template <int D, int kElem, bool kInterleaved, bool kAxes>
cudaError_t launch_fwd_t(const NormLaunch& a, cudaStream_t s) {
  constexpr int kHeads = 32 / (D / 16) * kFwdUnroll<kElem>;  // heads of one work item
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const int groups = (a.rot.heads[0] + a.rot.heads[1] + kHeads - 1) / kHeads;
  const long long items = static_cast<long long>(a.rot.B) * a.rot.N * groups;
  const long long blocks = (items + kNormWarps - 1) / kNormWarps, most = 64LL * sms;
  norm_rotary_kernel<D, kElem, kInterleaved, kAxes>
      <<<static_cast<unsigned>(blocks < most ? blocks : most), kNormThreads, 0, s>>>(a, groups,
                                                                                   items);
  return cudaGetLastError();
}

template <int D, int kElem, bool kInterleaved, bool kAxes>
cudaError_t launch_bwd_t(const NormLaunch& a, cudaStream_t s) {
  NormLaunch p = a;
  constexpr int kHeads = 32 / (D / 16) * kBwdUnroll<kElem>;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  // the operands' shares of the blocks, by the rows they have
  const long long tokens = static_cast<long long>(a.rot.B) * a.rot.N;
  const long long most = static_cast<long long>(kNormBlocks) * sms;
  long long need[2], all = 0;
  for (int w = 0; w < 2; ++w) {
    need[w] = (tokens * ((a.rot.heads[w] + kHeads - 1) / kHeads) + kNormWarps - 1) / kNormWarps;
    all += need[w];
  }
  p.blocks[0] = static_cast<int>(need[0]);
  p.blocks[1] = static_cast<int>(need[1]);
  if (all > most) {
    p.blocks[1] = need[1] ? static_cast<int>(std::max(1LL, most * need[1] / all)) : 0;
    p.blocks[0] = static_cast<int>(most) - p.blocks[1];
  }
  norm_rotary_bwd_kernel<D, kElem, kInterleaved, kAxes>
      <<<static_cast<unsigned>(p.blocks[0] + p.blocks[1]), kNormThreads, 0, s>>>(p);
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
