// fa_tables.cu -- the tables of a decoder's step, from the sequences' lengths: new
// pages taken from a stack of free ones, running sums, positions and slots; and the
// pages' way back.
//
//   need_b = ceil((len_b + new_b) / page) - ceil(len_b / page)
//   cu_b = sum of new before b,  first_b = sum of need before b
//   page j of sequence b = free[count - 1 - first_b - (j - ceil(len_b / page))]
//
// What bounds it.  A few bytes a token: latency, two dependent loads and the sums
// between them.  So one launch does it all: every CTA takes the sums over all sequences
// (they fit shared memory, kChunk sequences at a time) and writes a share of the results.
// Which sequence a row or a page belongs to is a binary search among sums in shared
// memory.  A page is taken from the free list where its rows need it; nobody waits for
// the table to be written.  Written in place, lengths and count must have been read by all
// CTAs before: these are one cluster then, and meet at its barrier.
//
// All or nothing: the totals are known before the first write.
//
// Measured (in a graph): 64 single tokens 3.9 us, 48 prompts of 111000 tokens in pages of
// 16 8.1 us.
#include <cooperative_groups.h>

#include <climits>

#include "fa_tables.h"
#include "sm103_primitives.cuh"

namespace fa {
namespace {

namespace cg = cooperative_groups;

// One CTA for a step of few tokens, several larger ones for prompts: a cluster of eight, or,
// where nothing is written in place, as many as there are rows for.  (48 prompts, 111000
// tokens: 8 CTAs of 512 threads, a row a thread, 16.3 us; four rows a thread 11.5.)
constexpr int kFewThreads = 512, kManyThreads = 1024, kClusterCtas = 8, kMostCtas = 32;
constexpr int kChunk = 2048;  // sequences at a time

struct ChunkSums {
  int a[kChunk + 1], b[kChunk + 1];  // running sums, from the chunk's beginning
};

// Exclusive sums of two counts of each of the block's kChunk sequences, kPer of them a
// thread's: 32 bits, as the totals are known to fit.
template <int kThreads>
__device__ __forceinline__ void block_sums(const int (&x)[kChunk / kThreads],
                                           const int (&y)[kChunk / kThreads], ChunkSums& out,
                                           int2 (&warps)[kThreads / 32]) {
  constexpr int kPer = kChunk / kThreads;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int sx = 0, sy = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    sx += x[i];
    sy += y[i];
  }
  int ux = sx, uy = sy;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int ox = __shfl_up_sync(0xffffffffu, ux, d), oy = __shfl_up_sync(0xffffffffu, uy, d);
    if (lane >= d) {
      ux += ox;
      uy += oy;
    }
  }
  if (lane == 31) warps[warp] = make_int2(ux, uy);
  __syncthreads();
  int px = ux - sx, py = uy - sy;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w)
    if (w < warp) {
      px += warps[w].x;
      py += warps[w].y;
    }
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    out.a[threadIdx.x * kPer + i] = px;
    out.b[threadIdx.x * kPer + i] = py;
    px += x[i];
    py += y[i];
  }
  if (threadIdx.x == kThreads - 1) {
    out.a[kChunk] = px;
    out.b[kChunk] = py;
  }
  __syncthreads();
}

// The last of sums[0 .. kChunk - 1] that is at most v (sums[0] = 0 <= v): the
// sequence that element v belongs to, as those without elements share their sum with
// the next.
__device__ __forceinline__ int find(const int* sums, int v) {
  int at = 0;
#pragma unroll
  for (int step = kChunk / 2; step > 0; step >>= 1)
    if (sums[at + step] <= v) at += step;
  return at;
}

struct Totals {
  long long x, y;
  int bad;
};

template <int kThreads>
__device__ __forceinline__ Totals block_totals(Totals t, Totals (&warps)[kThreads / 32]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) {
    t.x += __shfl_xor_sync(0xffffffffu, t.x, m);
    t.y += __shfl_xor_sync(0xffffffffu, t.y, m);
    t.bad |= __shfl_xor_sync(0xffffffffu, t.bad, m);
  }
  if (lane == 0) warps[warp] = t;
  __syncthreads();
  t = Totals{0, 0, 0};
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    t.x += warps[w].x;
    t.y += warps[w].y;
    t.bad |= warps[w].bad;
  }
  return t;
}

__device__ __forceinline__ int pages_of(int keys, int page_log2) {
  return (keys + (1 << page_log2) - 1) >> page_log2;
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads)
    reserve_kernel(const __grid_constant__ ReserveLaunch p) {
  __shared__ ChunkSums sums;  // a: new tokens, b: new pages
  __shared__ int len[kChunk];
  constexpr int kPer = kChunk / kThreads;
  __shared__ int2 warps[kThreads / 32];
  __shared__ Totals totals[kThreads / 32];
  const int me = blockIdx.x * kThreads + threadIdx.x, all = gridDim.x * kThreads;
  const int most = p.max_pages << p.page_log2;
  const int count = *p.free_count;
  // -- what is asked for, and whether it can be had; the first chunk stays at hand
  Totals t{0, 0, count < 0 || count > p.capacity};
  const auto add = [&](int n, int l) {
    if (n < 0 || l < 0 || l > most || n > most - l) {
      t.bad = 1;
      return;
    }
    t.x += n;
    t.y += pages_of(l + n, p.page_log2) - pages_of(l, p.page_log2);
  };
  int n[kPer], l[kPer];
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    const int b = threadIdx.x * kPer + i;
    n[i] = b < p.batch ? p.fresh[b] : 0;
    l[i] = b < p.batch ? p.lens[b] : 0;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) add(n[i], l[i]);
  for (int b = kChunk + threadIdx.x; b < p.batch; b += kThreads) add(p.fresh[b], p.lens[b]);
  t = block_totals<kThreads>(t, totals);
  if (t.x > p.total) t.bad = 1;
  const int missing = t.bad ? -1 : static_cast<int>(max(0LL, t.y - count));
  if (missing != 0) {
    if (p.in_place) cg::this_cluster().sync();
    for (int b = me; b < p.batch; b += all) {
      p.cu[b + 1] = 0;
      if (p.lens_out != p.lens) p.lens_out[b] = p.lens[b];
    }
    for (int i = me; i < p.total; i += all) {
      p.positions[i] = 0;
      p.slots[i] = -1;
    }
    if (me == 0) {
      p.cu[0] = 0;
      *p.free_count_out = count;
      *p.missing = missing;
      if (t.bad) atomicExch(p.err, kDevErrBadIndex);
    }
    return;
  }
  const bool aligned = ((reinterpret_cast<uintptr_t>(p.positions) |
                         reinterpret_cast<uintptr_t>(p.slots)) & 15) == 0;
  // -- kChunk sequences at a time
  int row0 = 0, taken = 0;  // rows and pages of the chunks before
  for (int b0 = 0; b0 < p.batch; b0 += kChunk) {
    if (b0) __syncthreads();  // (the sums before have been read)
    int need[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int j = threadIdx.x * kPer + i, b = b0 + j;
      if (b0) {
        n[i] = b < p.batch ? p.fresh[b] : 0;
        l[i] = b < p.batch ? p.lens[b] : 0;
      }
      need[i] = pages_of(l[i] + n[i], p.page_log2) - pages_of(l[i], p.page_log2);
      len[j] = l[i];
    }
    block_sums<kThreads>(n, need, sums, warps);
    if (p.in_place) cg::this_cluster().sync();  // everyone has read this chunk's lengths
    const int rows = sums.a[kChunk], pages = sums.b[kChunk];
    const int top = count - 1 - taken;  // this chunk's first page in the free list
    for (int j = me; j < min(kChunk, p.batch - b0); j += all) {
      p.cu[b0 + j + 1] = row0 + sums.a[j + 1];
      p.lens_out[b0 + j] = len[j] + sums.a[j + 1] - sums.a[j];
    }
    for (int m = me; m < pages; m += all) {
      const int j = find(sums.b, m);
      const int col = pages_of(len[j], p.page_log2) + m - sums.b[j];
      p.table[(b0 + j) * p.table_stride + col] = p.free_pages[top - m];
    }
    // Four rows a thread where there are more rows than threads: what one has looked up
    // mostly serves the next, and a search and a page's load, one after the other, are the
    // time that this takes.
    const int each = rows > all ? 4 : 1;
    const bool wide = each == 4 && row0 % 4 == 0 && aligned;
    for (int i0 = each * me; i0 < rows; i0 += each * all) {
      int pos[4] = {};
      long long slot[4] = {};
      int j = 0, ends = -1, held = 0, col = -1, page = 0;
#pragma unroll
      for (int t4 = 0; t4 < 4; ++t4) {
        const int i = i0 + t4;
        if (t4 >= each || i >= rows) break;
        if (i >= ends) {
          j = find(sums.a, i);
          ends = sums.a[j + 1];
          held = pages_of(len[j], p.page_log2);
          col = -1;
        }
        pos[t4] = len[j] + i - sums.a[j];
        const int c = pos[t4] >> p.page_log2;
        if (c != col) {
          col = c;
          page = c < held ? p.table[(b0 + j) * p.table_stride + c]
                          : p.free_pages[top - sums.b[j] - (c - held)];
          // (a slot below zero says that a row is not to be written: its key would be lost)
          if (page < 0) atomicExch(p.err, kDevErrBadIndex);
        }
        slot[t4] = page < 0 ? -1
                            : (static_cast<long long>(page) << p.page_log2) +
                                  (pos[t4] & ((1 << p.page_log2) - 1));
      }
      int* const to = p.positions + row0 + i0;
      long long* const at = p.slots + row0 + i0;
      if (wide && i0 + 4 <= rows) {
        *reinterpret_cast<int4*>(to) = make_int4(pos[0], pos[1], pos[2], pos[3]);
        *reinterpret_cast<longlong2*>(at) = make_longlong2(slot[0], slot[1]);
        *reinterpret_cast<longlong2*>(at + 2) = make_longlong2(slot[2], slot[3]);
      } else {
#pragma unroll
        for (int t4 = 0; t4 < 4; ++t4)
          if (t4 < each && i0 + t4 < rows) {
            to[t4] = pos[t4];
            at[t4] = slot[t4];
          }
      }
    }
    row0 += rows;
    taken += pages;
  }
  for (int i = row0 + me; i < p.total; i += all) {
    p.positions[i] = 0;
    p.slots[i] = -1;
  }
  if (me == 0) {
    p.cu[0] = 0;
    *p.free_count_out = count - taken;
    *p.missing = 0;
  }
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads)
    release_kernel(const __grid_constant__ ReleaseLaunch p) {
  __shared__ ChunkSums sums;  // b: pages given back
  __shared__ int keep[kChunk];
  constexpr int kPer = kChunk / kThreads;
  __shared__ int2 warps[kThreads / 32];
  __shared__ Totals totals[kThreads / 32];
  const int me = blockIdx.x * kThreads + threadIdx.x, all = gridDim.x * kThreads;
  const int most = p.max_pages << p.page_log2;
  const int count = *p.free_count;
  Totals t{0, 0, count < 0 || count > p.capacity};
  for (int b = threadIdx.x; b < p.batch; b += kThreads) {
    if (!p.done[b]) continue;
    const int l = p.lens[b], k = p.keep ? p.keep[b] : 0;
    if (l < 0 || l > most || k < 0) t.bad = 1;
    else t.y += max(0, pages_of(l, p.page_log2) - k);
  }
  t = block_totals<kThreads>(t, totals);
  if (t.bad || t.y > p.capacity - count) {
    if (me == 0) atomicExch(p.err, kDevErrBadIndex);
    return;  // (the same in every CTA)
  }
  int given = 0;
  for (int b0 = 0; b0 < p.batch; b0 += kChunk) {
    if (b0) __syncthreads();
    const int none[kPer] = {};
    int give[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int j = threadIdx.x * kPer + i, b = b0 + j;
      const bool mine = b < p.batch && p.done[b];
      keep[j] = mine && p.keep ? p.keep[b] : 0;
      give[i] = mine ? max(0, pages_of(p.lens[b], p.page_log2) - keep[j]) : 0;
    }
    block_sums<kThreads>(none, give, sums, warps);
    cg::this_cluster().sync();  // everyone has read this chunk's lengths, and the count
    const int pages = sums.b[kChunk];
    for (int m = me; m < pages; m += all) {
      const int j = find(sums.b, m);
      p.free_pages[count + given + m] =
          p.table[(b0 + j) * p.table_stride + keep[j] + m - sums.b[j]];
    }
    for (int j = me; j < min(kChunk, p.batch - b0); j += all)
      if (p.done[b0 + j]) p.lens[b0 + j] = 0;
    given += pages;
  }
  if (me == 0) *p.free_count = count + given;
}

// `cluster`: the CTAs wait for one another.
template <typename L>
cudaError_t launch_tables(void (*kern)(L), const L& a, int ctas, int threads, bool cluster,
                          cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {static_cast<unsigned>(ctas), 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = cluster ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

// Items (tokens, table entries) from which several CTAs pay.
constexpr long long kLarge = 1024;

}  // namespace

cudaError_t launch_reserve(const ReserveLaunch& a, cudaStream_t s) {
  if (a.total <= kLarge)
    return launch_tables(reserve_kernel<kFewThreads>, a, 1, kFewThreads, true, s);
  const int ctas = a.in_place ? kClusterCtas
                              : std::min(kMostCtas, (a.total - 1) / (4 * kManyThreads) + 1);
  return launch_tables(reserve_kernel<kManyThreads>, a, ctas, kManyThreads, a.in_place, s);
}

cudaError_t launch_release(const ReleaseLaunch& a, cudaStream_t s) {
  // (the pages are the kernel's to count: at most the table's)
  const long long entries = static_cast<long long>(a.batch) * a.max_pages;
  if (std::min<long long>(entries, a.capacity) <= kLarge)
    return launch_tables(release_kernel<kFewThreads>, a, 1, kFewThreads, true, s);
  return launch_tables(release_kernel<kManyThreads>, a, kClusterCtas, kManyThreads, true, s);
}

}  // namespace fa
