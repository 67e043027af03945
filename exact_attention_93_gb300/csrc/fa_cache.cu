// fa_cache.cu -- writing keys and values into a paged cache, as 16-bit copies
// or as e4m3 rows with a power-of-two scale each, and reading them back.
//
// Quantisation of one (token, head) row x: the scale is the smallest power of
// two 2^k with max |x| <= 448 * 2^k (448: e4m3's largest value), taken from the
// bits of the maximum; the codes are x * 2^-k (an exact product) rounded to
// nearest even.  e4m3 is a floating format, so a scale between the powers of
// two would buy no precision for normal codes; a power of two makes every
// cached value exactly representable in bf16, so reading back and the
// attention kernels' products lose nothing more.
//
// Both directions move each byte once and compute next to nothing: HBM is
// the bound (and latency, for a few tokens).  A warp takes the keys or the
// values of one token: D / 8 lanes hold a head's row, 8 elements (16 bytes of
// 16-bit rows) each, kUnroll rows in flight per lane; the row loads are issued
// before the page lookup (sequence, length, page: three dependent loads), which
// they hide.
#include "fa_ragged.cuh"
#include "fa_serve.h"
#include "sm103_primitives.cuh"

namespace fa {
namespace {

constexpr int kCacheThreads = 128;
constexpr int kUnroll = 4;

struct Slot {
  long long row;      // element offset of head 0's row in the cache
  long long exp;      // offset of head 0's exponent byte
  bool ok;
};

// Where key `pos` of sequence b lives (whole warp or single threads alike).
__device__ __forceinline__ Slot find_slot(const CacheLaunch& p, int w, int b, long long pos) {
  Slot s{0, 0, false};
  if (pos < 0 || pos >= (static_cast<long long>(p.r.max_pages) << p.c.page_log2)) return s;
  const int page = p.r.table[b * p.r.table_stride + (pos >> p.c.page_log2)];
  if (page < 0 || page >= p.c.pages) return s;
  const long long off = pos & (p.c.page_size - 1);
  s.row = page * p.c.page[w] + off * p.c.token[w];
  s.exp = static_cast<long long>(page) * p.c.heads * p.c.page_size + off;
  s.ok = true;
  return s;
}

template <bool kBf16>
__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = unpack2<kBf16>(w[i]);
    f[2 * i] = u.x;
    f[2 * i + 1] = u.y;
  }
}

template <int D, bool kBf16, bool kFp8>
__global__ void __launch_bounds__(kCacheThreads)
    cache_append_kernel(const __grid_constant__ CacheLaunch p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  const long long item = blockIdx.x * (kCacheThreads / 32LL) + (threadIdx.x >> 5);
  const int w = static_cast<int>(item & 1), row = static_cast<int>(item >> 1);
  if (row >= p.r.total) return;
  const int lane = threadIdx.x & 31, sub = lane % kLanes, slot = lane / kLanes;
  const uint16_t* src = static_cast<const uint16_t*>(p.rows[w]) + row * p.row_token[w] + sub * 8;
  Slot at{0, 0, false};
  for (int h0 = slot; h0 - slot < p.c.heads; h0 += kRows * kUnroll) {
    uint4 v[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * kRows;
      v[u] = h < p.c.heads ? __ldg(reinterpret_cast<const uint4*>(src + h * p.row_head[w]))
                           : make_uint4(0u, 0u, 0u, 0u);
    }
    if (h0 == slot) {
      const int b = warp_find_seq(p.r.cu, p.r.batch, row);
      if (b < 0) return;  // behind the last sequence
      const int c0 = p.r.cu[b], c1 = p.r.cu[b + 1];
      const long long pos = static_cast<long long>(p.r.lens[b]) - c1 + row;
      at = find_slot(p, w, b, pos);
      if (!at.ok) {
        // no slot for this row; a sequence shorter than its rows is the caller's right
        if ((pos >= 0 || c1 < c0) && lane == 0) atomicExch(p.err, kDevErrBadIndex);
        return;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * kRows;
      if constexpr (!kFp8) {
        if (h < p.c.heads)
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.c.p[w]) + at.row +
                                    h * p.c.head[w] + sub * 8) = v[u];
      } else {
        float f[8];
        unpack8<kBf16>(v[u], f);
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float a = fabsf(f[i]);
          top = fmaxf(top, a < INFINITY ? a : 0.f);  // (false for NaN)
        }
#pragma unroll
        for (int m = 1; m < kLanes; m <<= 1)
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        const uint32_t bits = __float_as_uint(top);
        int e = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
        e = max(e, 1);  // a finite maximum keeps e below 248
        const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
        const uint2 code = make_uint2(
            pack2_e4m3(f[0] * inv, f[1] * inv) | pack2_e4m3(f[2] * inv, f[3] * inv) << 16,
            pack2_e4m3(f[4] * inv, f[5] * inv) | pack2_e4m3(f[6] * inv, f[7] * inv) << 16);
        // a row without finite nonzero values is marked as zeros, unless it holds
        // infinities or NaN, which keep the smallest scale
        bool odd = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) odd |= !(fabsf(f[i]) < INFINITY);
#pragma unroll
        for (int m = 1; m < kLanes; m <<= 1) odd |= __shfl_xor_sync(0xffffffffu, odd, m) != 0;
        if (h < p.c.heads) {
          *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.c.p[w]) + at.row + h * p.c.head[w] +
                                    sub * 8) = code;
          if (sub == 0)
            p.c.exp[w][at.exp + static_cast<long long>(h) * p.c.page_size] =
                static_cast<uint8_t>(top > 0.f || odd ? e : 0);
        }
      }
    }
  }
}

template <int D, bool kBf16, bool kFp8>
__global__ void __launch_bounds__(kCacheThreads)
    cache_read_kernel(const __grid_constant__ CacheLaunch p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes;
  const long long item = blockIdx.x * (kCacheThreads / 32LL) + (threadIdx.x >> 5);
  const int w = static_cast<int>(item & 1), row = static_cast<int>(item >> 1);
  if (row >= p.r.total) return;
  const int lane = threadIdx.x & 31, sub = lane % kLanes, slot = lane / kLanes;
  const int b = warp_find_seq(p.r.cu, p.r.batch, row);
  if (b < 0) return;  // behind the last sequence
  const long long pos = (p.r.lens ? p.r.lens[b] : 0LL) + row - p.r.cu[b];
  const Slot at = find_slot(p, w, b, pos);
  if (!at.ok && lane == 0) atomicExch(p.err, kDevErrBadIndex);
  uint16_t* dst = static_cast<uint16_t*>(p.rows[w]) + row * p.row_token[w] + sub * 8;
  for (int h0 = slot; h0 < p.c.heads; h0 += kRows * kUnroll) {
    uint4 v[kUnroll];
    uint32_t e[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * kRows;
      v[u] = make_uint4(0u, 0u, 0u, 0u);
      e[u] = 0u;
      if (!at.ok || h >= p.c.heads) continue;
      if constexpr (kFp8) {
        const uint2 c = __ldg(reinterpret_cast<const uint2*>(
            static_cast<const uint8_t*>(p.c.p[w]) + at.row + h * p.c.head[w] + sub * 8));
        v[u].x = c.x;
        v[u].y = c.y;
        e[u] = p.c.exp[w][at.exp + static_cast<long long>(h) * p.c.page_size];
      } else {
        v[u] = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.c.p[w]) +
                                                    at.row + h * p.c.head[w] + sub * 8));
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * kRows;
      if (h >= p.c.heads) continue;
      if constexpr (kFp8) {
        const float scale = __uint_as_float(e[u] << 23);
        uint32_t out[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t two = ((i & 2) ? v[u].y : v[u].x) >> ((i & 1) * 16);
          const float2 f = unpack2<false>(e4m3x2_to_f16x2(two));
          out[i] = e[u] ? pack2<kBf16>(f.x * scale, f.y * scale) : 0u;
        }
        v[u] = make_uint4(out[0], out[1], out[2], out[3]);
      }
      *reinterpret_cast<uint4*>(dst + h * p.row_head[w]) = v[u];
    }
  }
}

template <typename K>
cudaError_t launch_rows(K kern, const CacheLaunch& a, cudaStream_t s) {
  const long long per_block = kCacheThreads / 32;
  const long long blocks = (2LL * a.r.total + per_block - 1) / per_block;
  kern<<<static_cast<unsigned>(blocks), kCacheThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_append(const CacheLaunch& a, cudaStream_t s) {
  const bool fp8 = a.c.elem == kElemE4m3, bf16 = a.elem == kElemBf16;
  if (a.c.D == 64)
    return !fp8 ? launch_rows(cache_append_kernel<64, true, false>, a, s)
           : bf16 ? launch_rows(cache_append_kernel<64, true, true>, a, s)
                  : launch_rows(cache_append_kernel<64, false, true>, a, s);
  return !fp8 ? launch_rows(cache_append_kernel<128, true, false>, a, s)
         : bf16 ? launch_rows(cache_append_kernel<128, true, true>, a, s)
                : launch_rows(cache_append_kernel<128, false, true>, a, s);
}

cudaError_t launch_cache_read(const CacheLaunch& a, cudaStream_t s) {
  const bool fp8 = a.c.elem == kElemE4m3, bf16 = a.elem == kElemBf16;
  if (a.c.D == 64)
    return !fp8 ? launch_rows(cache_read_kernel<64, true, false>, a, s)
           : bf16 ? launch_rows(cache_read_kernel<64, true, true>, a, s)
                  : launch_rows(cache_read_kernel<64, false, true>, a, s);
  return !fp8 ? launch_rows(cache_read_kernel<128, true, false>, a, s)
         : bf16 ? launch_rows(cache_read_kernel<128, true, true>, a, s)
                : launch_rows(cache_read_kernel<128, false, true>, a, s);
}

}  // namespace fa
