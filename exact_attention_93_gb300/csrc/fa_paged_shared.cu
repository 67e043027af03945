// fa_paged_shared.cu -- attention over prefixes that sequences share: groups of
// sequences made to look like sequences, and the joining of the two parts.
//
// The softmax of a row over shared and own keys is joined from its parts' results, each of
// them o_i divided by its sum l_i of 2^(score - m_i):
//
//   m = max(m1, m2),   w_i = l_i 2^(m_i - m),   o = (w1 o1 + w2 o2) / (w1 + w2)
//
// The shared part of a group is attention of all its rows over one sequence of keys,
// none of them masked: every shared key lies before every new token.  So the kernels
// of fa_paged_few.cu and fa_paged_many.cu do either part, once for the groups and once
// for the sequences behind their shared pages, with the first part's O in fp32.  Where the
// second takes the few-row kernel, that one and its joining kernel add the first part to
// their rows before they store them; else a kernel here reads both.
//
// Measured (32 query and 8 key heads of 128, in a graph): 64 single tokens under 16000 shared
// keys, 16 to 2000 of their own, 77 us (each walking all of its keys 209): groups 3, shared
// part 30 and 8 to join, own part 32 and 5; what bounds each is said in their files, and five
// starts.
#include <climits>

#include "fa_ragged.cuh"
#include "fa_serve.h"
#include "sm103_primitives.cuh"

namespace fa {
namespace {

constexpr int kSetupThreads = 128;

// Block g: group g.  The first and the last block also take the sequences before and
// behind all groups.
__global__ void __launch_bounds__(kSetupThreads)
    shared_setup_kernel(const __grid_constant__ SharedSetup p) {
  pdl_wait_and_release();
  __shared__ int least[kSetupThreads / 32], leader[kSetupThreads / 32];
  const int g = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = p.cu_groups[g], c1 = p.cu_groups[g + 1];
  const int lo = min(max(c0, 0), p.r.batch), hi = min(max(c1, lo), p.r.batch);
  int pages = p.shared_pages[g], row = INT_MAX;
  if (threadIdx.x == 0 && (c0 < 0 || c1 < c0 || c1 > p.r.batch || pages < 0 ||
                           pages > p.r.max_pages))
    atomicExch(p.err, kDevErrBadIndex);
  pages = min(max(pages, 0), p.r.max_pages);
  // no more than lies before every new token
  for (int b = lo + threadIdx.x; b < hi; b += kSetupThreads) {
    const Seq s = load_seq(p.r, p.page_log2, b, p.err);
    if (s.rows > 0) {
      pages = min(pages, max(s.pos0, 0) >> p.page_log2);
      row = min(row, b);
    }
  }
  pages = __reduce_min_sync(0xffffffffu, pages);
  row = __reduce_min_sync(0xffffffffu, row);
  if (lane == 0) {
    least[warp] = pages;
    leader[warp] = row;
  }
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSetupThreads / 32; ++w) {
    pages = min(pages, least[w]);
    row = min(row, leader[w]);
  }
  const auto packed = [&](int b) { return min(max(p.r.cu[b], 0), p.r.total); };
  if (threadIdx.x == 0) {
    p.lens[g] = row == INT_MAX ? 0 : pages << p.page_log2;
    p.rows[g] = row == INT_MAX ? 0 : row;
    p.cu[g] = packed(lo);
    if (g == p.groups - 1) p.cu[p.groups] = packed(hi);
  }
  for (int b = lo + threadIdx.x; b < hi; b += kSetupThreads)
    p.skip[b] = load_seq(p.r, p.page_log2, b, nullptr).rows > 0 ? pages : 0;
  if (g == 0)
    for (int b = threadIdx.x; b < lo; b += kSetupThreads) p.skip[b] = 0;
  if (g == p.groups - 1)
    for (int b = hi + threadIdx.x; b < p.r.batch; b += kSetupThreads) p.skip[b] = 0;
}

constexpr int kSharedThreads = 128;

// A warp joins one head's row.
template <int D, bool kBf16>
__global__ void __launch_bounds__(kSharedThreads)
    shared_join_kernel(const __grid_constant__ SharedJoin p) {
  pdl_wait_and_release();
  constexpr int kN = D / 32;
  const int lane = threadIdx.x & 31;
  const int first = max(p.cu[0], 0), last = min(p.cu[p.batch], p.total);
  const int first1 = *p.first, last1 = *p.end;
  const long long n = static_cast<long long>(last - first) * p.heads;
  for (long long i = blockIdx.x * (kSharedThreads / 32LL) + (threadIdx.x >> 5); i < n;
       i += gridDim.x * (kSharedThreads / 32LL)) {
    const int row = first + static_cast<int>(i / p.heads);
    const int head = static_cast<int>(i % p.heads);
    const long long stat = static_cast<long long>(head) * p.total + row;
    const long long at = (static_cast<long long>(row) * p.heads + head) * D + lane * kN;
    const float2 own = p.ml2[stat];
    float2 other = p.ml1[stat];
    if (row < first1 || row >= last1) other = make_float2(-INFINITY, 0.f);
    const bool both = other.y != 0.f;
    float x[kN], y[kN];
#pragma unroll
    for (int e = 0; e < kN; ++e) {
      x[e] = both ? p.o1[at + e] : 0.f;
      y[e] = p.o2[at + e];
    }
    const float top = fmaxf(other.x, own.x), ref = top == -INFINITY ? 0.f : top;
    const float wa = other.y * ex2_approx(other.x - ref), wb = own.y * ex2_approx(own.x - ref);
    const float sum = wa + wb;
    const float per = sum == 0.f ? 0.f : 1.f / sum;
    const float ua = wa * per, ub = wb * per;
    uint32_t out[kN / 2];
#pragma unroll
    for (int e = 0; e < kN; e += 2)
      out[e / 2] = pack2<kBf16>(x[e] * ua + y[e] * ub, x[e + 1] * ua + y[e + 1] * ub);
    uint16_t* dst = static_cast<uint16_t*>(p.o) + row * p.o_token + head * p.o_head + lane * kN;
    if constexpr (kN == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[kN / 2 - 1]);
    else *reinterpret_cast<uint32_t*>(dst) = out[0];
    if (lane == 0)
      p.lse[stat] = sum == 0.f ? -INFINITY : (top + lg2_approx(sum)) * 0.6931471805599453f;
  }
}

template <int D, bool kBf16>
cudaError_t launch_join_t(const SharedJoin& a, cudaStream_t s) {
  int sms = 0;
  const cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const long long blocks = (static_cast<long long>(a.total) * a.heads + 3) / 4;
  return launch_pdl(shared_join_kernel<D, kBf16>,
                    static_cast<unsigned>(blocks < 16LL * sms ? blocks : 16LL * sms),
                    kSharedThreads, 0, s, a);
}

}  // namespace

cudaError_t launch_shared_setup(const SharedSetup& a, cudaStream_t s) {
  return launch_pdl(shared_setup_kernel, static_cast<unsigned>(a.groups), kSetupThreads, 0, s, a);
}

cudaError_t launch_shared_join(const SharedJoin& a, cudaStream_t s) {
  if (a.D == 64)
    return a.elem == kElemBf16 ? launch_join_t<64, true>(a, s) : launch_join_t<64, false>(a, s);
  return a.elem == kElemBf16 ? launch_join_t<128, true>(a, s) : launch_join_t<128, false>(a, s);
}

}  // namespace fa
