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
// the bound (and latency, for a few tokens).  A warp takes the keys and the values
// of one token to append, the keys or the values to read: D / 8 lanes hold a
// head's row, 8 elements (16 bytes of 16-bit rows) each, kUnroll rows in flight per
// lane; appending, the row loads are issued before the page lookup (sequence,
// length, page: three dependent loads), which they hide.  Many warps with little
// each hide those loads best: four tokens a warp took 10 % longer, one lookup for a
// block of tokens and a barrier 30 %.  With at most kUnroll heads each lane group
// takes a token of its own instead of every kRows-th head of one.
//
// What is left beside the bytes is instruction issue, so a row's maximum is taken
// on packed 16-bit magnitudes (ordered like their values), two rows' at a time
// across the lanes, rows that hold infinities or NaN take a path of their own, and
// one lookup serves keys and values (a warp for each: 36 us instead of 33).
//
// Measured, 30111 tokens of 8 heads of 128: 16-bit 38 us to append and 39 to
// read, 6.3 to 6.4 TB/s; e4m3 33 and 32 us, 5.6 and 5.8 TB/s.
#include "fa_ragged.cuh"
#include "fa_serve.h"
#include "sm103_primitives.cuh"

namespace fa {
namespace {

constexpr int kCacheThreads = 128;
constexpr int kUnroll = 4;

// The page of key `pos` of sequence b; -1 when there is none.
__device__ __forceinline__ int find_page(const CacheLaunch& p, int b, long long pos) {
  if (pos < 0 || pos >= (static_cast<long long>(p.r.max_pages) << p.c.page_log2)) return -1;
  const int page = p.r.table[b * p.r.table_stride + (pos >> p.c.page_log2)];
  return page < p.c.pages ? page : -1;
}

// Where a key's rows (w = 0) or a value's (w = 1) live in a page.
struct Slot {
  long long row = 0;  // element offset of head 0's row in the cache
  long long exp = 0;  // offset of head 0's exponent byte
  Slot() = default;
  __device__ __forceinline__ Slot(const CacheLaunch& p, int w, int page, long long pos) {
    const long long off = pos & (p.c.page_size - 1);
    row = page * p.c.page[w] + off * p.c.token[w];
    exp = static_cast<long long>(page) * p.c.heads * p.c.page_size + off;
  }
};

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

// One row as e4m3 codes beside its exponent byte; top: its largest magnitude's
// 16 bits.
template <bool kBf16, int kLanes>
__device__ __forceinline__ uint2 quantise(const uint4& v, uint32_t top, int slot, uint32_t& exp) {
  const uint32_t x[4] = {v.x, v.y, v.z, v.w};
  const bool zeros = top == 0;
  constexpr uint32_t kInf = kBf16 ? 0x7f80u : 0x7c00u;
  if (top >= kInf) {  // the same for all lanes of the row
    top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t m = (x[i >> 1] >> ((i & 1) * 16)) & 0x7fffu;
      top = m < kInf ? max(top, m) : top;
    }
    const uint32_t row = ((1u << kLanes) - 1u) << (slot * kLanes);
#pragma unroll
    for (int m = 1; m < kLanes; m <<= 1) top = max(top, __shfl_xor_sync(row, top, m));
  }
  // the smallest 2^(e - 127) with top <= 448 * 2^(e - 127); a finite
  // maximum keeps e below 248
  const uint32_t bits = __float_as_uint(unpack2<kBf16>(top).x);
  const int e =
      max(static_cast<int>(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0), 1);
  const float inv = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
  exp = zeros ? 0u : static_cast<uint32_t>(e);
  float f[8];
  unpack8<kBf16>(v, f);
  return make_uint2(pack2_e4m3(f[0] * inv, f[1] * inv) | pack2_e4m3(f[2] * inv, f[3] * inv) << 16,
                    pack2_e4m3(f[4] * inv, f[5] * inv) | pack2_e4m3(f[6] * inv, f[7] * inv) << 16);
}

template <int D, bool kBf16, bool kFp8, bool kFewHeads>
__global__ void __launch_bounds__(kCacheThreads)
    cache_append_kernel(const __grid_constant__ CacheLaunch p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kStep = kFewHeads ? 1 : kRows;
  const long long first = (blockIdx.x * (kCacheThreads / 32LL) + (threadIdx.x >> 5)) *
                          (kFewHeads ? kRows : 1);
  if (first >= p.r.total) return;
  const int lane = threadIdx.x & 31, sub = lane % kLanes, slot = lane / kLanes;
  const int row = static_cast<int>(first) + (kFewHeads ? slot : 0);
  const int h_first = kFewHeads ? 0 : slot, heads = row < p.r.total ? p.c.heads : 0;
  bool ok = false;
  Slot at[2];
  for (int h0 = h_first; h0 - h_first < p.c.heads; h0 += kStep * kUnroll) {
    uint4 v[2][kUnroll];
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const uint16_t* src =
          static_cast<const uint16_t*>(p.rows[w]) + row * p.row_token[w] + sub * 8;
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = h0 + u * kStep;
        v[w][u] = h < heads ? __ldg(reinterpret_cast<const uint4*>(src + h * p.row_head[w]))
                            : make_uint4(0u, 0u, 0u, 0u);
      }
    }
    if (h0 == h_first && p.slots) {
      if (row < p.r.total) {
        const long long slot = p.slots[row], page = slot >> p.c.page_log2;
        ok = slot >= 0 && page < p.c.pages;
        at[0] = Slot(p, 0, static_cast<int>(page), slot);
        at[1] = Slot(p, 1, static_cast<int>(page), slot);
        if (!ok && slot >= 0 && sub == 0) atomicExch(p.err, kDevErrBadIndex);
      }
    } else if (h0 == h_first) {
      const int b = warp_find_seq(p.r.cu, p.r.batch, static_cast<int>(first), row);
      if (b >= 0 && row < p.r.total) {  // (not behind the last sequence)
        const int c0 = p.r.cu[b], c1 = p.r.cu[b + 1];
        const long long pos = static_cast<long long>(p.r.lens[b]) - c1 + row;
        const int page = find_page(p, b, pos);
        ok = page >= 0;
        at[0] = Slot(p, 0, page, pos);
        at[1] = Slot(p, 1, page, pos);
        // no page: a sequence shorter than its rows is the caller's right
        if (!ok && (pos >= 0 || c1 < c0) && sub == 0) atomicExch(p.err, kDevErrBadIndex);
      }
    }
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      // the rows' largest magnitudes, two rows to a word
      [[maybe_unused]] uint32_t tops[kUnroll / 2];
      if constexpr (kFp8) {
#pragma unroll
        for (int i = 0; i < kUnroll / 2; ++i) {
          uint32_t half[2];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4& x = v[w][2 * i + j];
            half[j] = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                               __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
          }
          tops[i] = __vmaxu2(__byte_perm(half[0], half[1], 0x5410),
                             __byte_perm(half[0], half[1], 0x7632));
#pragma unroll
          for (int m = 1; m < kLanes; m <<= 1)
            tops[i] = __vmaxu2(tops[i], __shfl_xor_sync(0xffffffffu, tops[i], m));
        }
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int h = h0 + u * kStep;
        const long long to = at[w].row + h * p.c.head[w] + sub * 8;
        if constexpr (!kFp8) {
          if (ok && h < heads)
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.c.p[w]) + to) = v[w][u];
        } else {
          uint32_t e;
          const uint2 codes = quantise<kBf16, kLanes>(
              v[w][u], (tops[u >> 1] >> ((u & 1) * 16)) & 0xffffu, slot, e);
          if (ok && h < heads) {
            *reinterpret_cast<uint2*>(static_cast<uint8_t*>(p.c.p[w]) + to) = codes;
            if (sub == 0)
              p.c.exp[w][at[w].exp + static_cast<long long>(h) * p.c.page_size] =
                  static_cast<uint8_t>(e);
          }
        }
      }
    }
  }
}

template <int D, bool kBf16, bool kFp8, bool kFewHeads>
__global__ void __launch_bounds__(kCacheThreads)
    cache_read_kernel(const __grid_constant__ CacheLaunch p) {
  constexpr int kLanes = D / 8, kRows = 32 / kLanes, kStep = kFewHeads ? 1 : kRows;
  const long long item = blockIdx.x * (kCacheThreads / 32LL) + (threadIdx.x >> 5);
  const int w = static_cast<int>(item & 1);
  const long long first = (item >> 1) * (kFewHeads ? kRows : 1);
  if (first >= p.r.total) return;
  const int lane = threadIdx.x & 31, sub = lane % kLanes, slot = lane / kLanes;
  const int row = static_cast<int>(first) + (kFewHeads ? slot : 0);
  const int b = warp_find_seq(p.r.cu, p.r.batch, static_cast<int>(first), row);
  if (b < 0 || row >= p.r.total) return;  // behind the last sequence
  const long long pos = (p.r.lens ? p.r.lens[b] : 0LL) + row - p.r.cu[b];
  const int page = find_page(p, b, pos);
  const Slot at(p, w, page, pos);
  if (page < 0 && sub == 0) atomicExch(p.err, kDevErrBadIndex);
  uint16_t* dst = static_cast<uint16_t*>(p.rows[w]) + row * p.row_token[w] + sub * 8;
  for (int h0 = kFewHeads ? 0 : slot; h0 < p.c.heads; h0 += kStep * kUnroll) {
    uint4 v[kUnroll];
    uint32_t e[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int h = h0 + u * kStep;
      v[u] = make_uint4(0u, 0u, 0u, 0u);
      e[u] = 0u;
      if (page < 0 || h >= p.c.heads) continue;
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
      const int h = h0 + u * kStep;
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

// `ways`: warps for a token's keys and values.
template <typename K>
cudaError_t launch_rows(K kern, K few_heads, const CacheLaunch& a, int ways, cudaStream_t s) {
  const bool few = a.c.heads <= kUnroll;
  const long long tokens = few ? 32 / (a.c.D / 8) : 1, per_block = kCacheThreads / 32;
  const long long items = ways * ((a.r.total + tokens - 1) / tokens);
  const long long blocks = (items + per_block - 1) / per_block;
  (few ? few_heads : kern)<<<static_cast<unsigned>(blocks), kCacheThreads, 0, s>>>(a);
  return cudaGetLastError();
}

template <int D, bool kBf16, bool kFp8>
cudaError_t append_t(const CacheLaunch& a, cudaStream_t s) {
  return launch_rows(cache_append_kernel<D, kBf16, kFp8, false>,
                     cache_append_kernel<D, kBf16, kFp8, true>, a, 1, s);
}

template <int D, bool kBf16, bool kFp8>
cudaError_t read_t(const CacheLaunch& a, cudaStream_t s) {
  return launch_rows(cache_read_kernel<D, kBf16, kFp8, false>,
                     cache_read_kernel<D, kBf16, kFp8, true>, a, 2, s);
}

}  // namespace

// (a 16-bit cache's rows are copied, whichever type they are)
cudaError_t launch_cache_append(const CacheLaunch& a, cudaStream_t s) {
  const bool fp8 = a.c.elem == kElemE4m3, bf16 = a.elem == kElemBf16;
  if (a.c.D == 64)
    return !fp8 ? append_t<64, true, false>(a, s)
           : bf16 ? append_t<64, true, true>(a, s) : append_t<64, false, true>(a, s);
  return !fp8 ? append_t<128, true, false>(a, s)
         : bf16 ? append_t<128, true, true>(a, s) : append_t<128, false, true>(a, s);
}

cudaError_t launch_cache_read(const CacheLaunch& a, cudaStream_t s) {
  const bool fp8 = a.c.elem == kElemE4m3, bf16 = a.elem == kElemBf16;
  if (a.c.D == 64)
    return !fp8 ? read_t<64, true, false>(a, s)
           : bf16 ? read_t<64, true, true>(a, s) : read_t<64, false, true>(a, s);
  return !fp8 ? read_t<128, true, false>(a, s)
         : bf16 ? read_t<128, true, true>(a, s) : read_t<128, false, true>(a, s);
}

}  // namespace fa
