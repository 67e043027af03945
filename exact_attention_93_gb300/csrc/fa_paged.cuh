// fa_paged.cuh -- what the attention-over-pages kernels share: which keys a
// block of queries sees, how the work is split over the CTAs, and the joining
// of blocks that several CTAs worked on.
//
// Units.  A unit is one block of query rows (kRows of the rows token * group +
// head-in-group of one sequence) against one key head.  It walks tiles of 128
// keys.  All units of a sequence are given the same weight, the number of key
// tiles that any of its queries sees (at least 1, so that rows without keys
// are written too).  Units are laid end to end, sequence by sequence, and each
// CTA takes an equal stretch of the whole, cutting units where the stretch
// ends: a long context over few rows is spread over every SM, ragged batches
// stay balanced, and a CTA leaves at most two cut pieces whatever the batch.
// Cut pieces go to the workspace in fp32 (unnormalised O, maximum, sum) and
// paged_join_kernel adds them up in a fixed order.
#pragma once

#include "fa_ragged.cuh"

namespace fa {

constexpr float kPagedLn2 = 0.6931471805599453f;

// Keys [lo, hi) that some query of tokens [t0, t1) of the sequence sees.
__device__ __forceinline__ void visible_span(const PagedLaunch& p, const Seq& s, int t0, int t1,
                                             int& lo, int& hi) {
  lo = p.win_left < 0 ? 0 : max(0, s.pos0 + t0 - p.win_left);
  const long long last = static_cast<long long>(s.pos0) + t1 - 1 + p.win_right;
  hi = p.win_right < 0 ? s.len : static_cast<int>(max(0LL, min(static_cast<long long>(s.len), last + 1)));
  if (lo >= hi) lo = hi = 0;
}

// A sequence as the work split sees it.
template <int kRows>
struct SeqWork {
  Seq s;
  int blocks;      // query blocks per key head
  int first_tile;  // key tiles first_tile .. first_tile + weight - 1
  int weight;
  __device__ __forceinline__ void load(const PagedLaunch& p, int b, uint32_t* err = nullptr) {
    s = load_seq(p.r, p.page_log2, b, err);
    blocks = (s.rows * p.group + kRows - 1) / kRows;
    int lo, hi;
    visible_span(p, s, 0, s.rows, lo, hi);
    first_tile = lo / kTile;
    weight = max(1, (hi + kTile - 1) / kTile - first_tile);
  }
  __device__ __forceinline__ long long work(const PagedLaunch& p) const {
    return static_cast<long long>(weight) * blocks * p.heads_k;
  }
};

// A place in the laid-out work: sequence b, unit u of it, tile `off` of that.
struct Place {
  int b, unit, off;
  long long left;   // of this CTA's stretch
  long long begin;  // of this CTA's stretch
  long long total;
};

__device__ __forceinline__ long long stretch(long long total, int n, int c) {
  return total * c / n;
}

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// The whole work, by one warp.
template <int kRows>
__device__ __forceinline__ long long warp_total_work(const PagedLaunch& p) {
  long long sum = 0;
  for (int b = threadIdx.x & 31; b < p.r.batch; b += 32) {
    SeqWork<kRows> w;
    w.load(p, b, blockIdx.x == 0 ? p.err : nullptr);
    sum += w.work(p);
  }
  return warp_sum(sum);
}

// The sequence, unit and tile at position `at` (< the whole work), by one
// warp; unit_start gets the position of the unit's first tile.
template <int kRows>
__device__ __forceinline__ void warp_locate(const PagedLaunch& p, long long at, Place& out,
                                            long long& unit_start) {
  const int lane = threadIdx.x & 31;
  long long before = 0;
  for (int b0 = 0; b0 < p.r.batch; b0 += 32) {
    SeqWork<kRows> w;
    w.weight = 1;
    long long mine = 0;
    if (b0 + lane < p.r.batch) {
      w.load(p, b0 + lane);
      mine = w.work(p);
    }
    long long upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, before + upto > at);
    if (past) {
      const int src = __ffs(past) - 1;
      const long long start = before + __shfl_sync(0xffffffffu, upto - mine, src);
      const int weight = __shfl_sync(0xffffffffu, w.weight, src);
      const long long in = at - start;
      out.b = b0 + src;
      out.unit = static_cast<int>(in / weight);
      out.off = static_cast<int>(in - static_cast<long long>(out.unit) * weight);
      unit_start = at - out.off;
      return;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  out.b = p.r.batch;
  out.unit = out.off = 0;
  unit_start = at;
}

// A CTA's next piece of work.
struct Piece {
  int b, hk, block;
  int t0, t1;            // the block's tokens
  int rows;              // valid rows of the block
  int lo, hi;            // keys some row of the block sees
  int tile0, tile1;      // key tiles to walk (none: tile0 >= tile1)
  bool whole;            // the piece covers its unit
  int slot;              // of the CTA's two partial results, when it does not
};

// Walks a CTA's stretch.  Every role of the CTA runs its own copy.
template <int kRows>
struct WorkWalk {
  Place at;
  SeqWork<kRows> w;
  bool loaded;
  __device__ __forceinline__ explicit WorkWalk(const Place& start) : at(start), loaded(false) {}
  __device__ __forceinline__ bool next(const PagedLaunch& p, Piece& x, Seq& seq) {
    if (at.left <= 0) return false;
    if (!loaded) {
      w.load(p, at.b);
      loaded = true;
    }
    while (at.unit >= w.blocks * p.heads_k) {  // (a sequence without rows has no units)
      at.unit = 0;
      if (++at.b >= p.r.batch) return false;
      w.load(p, at.b);
    }
    const int take = static_cast<int>(min(at.left, static_cast<long long>(w.weight - at.off)));
    x.b = at.b;
    x.hk = at.unit / w.blocks;
    x.block = at.unit - x.hk * w.blocks;
    x.rows = min(kRows, w.s.rows * p.group - x.block * kRows);
    x.t0 = x.block * kRows / p.group;
    x.t1 = (x.block * kRows + x.rows - 1) / p.group + 1;
    visible_span(p, w.s, x.t0, x.t1, x.lo, x.hi);
    x.whole = take == w.weight;
    x.slot = at.off > 0 ? 0 : 1;
    x.tile0 = max(w.first_tile + at.off, x.lo / kTile);
    x.tile1 = min(w.first_tile + at.off + take, (x.hi + kTile - 1) / kTile);
    seq = w.s;
    at.off += take;
    at.left -= take;
    if (at.off == w.weight) {
      at.off = 0;
      ++at.unit;
    }
    return true;
  }
};

// Row r of a piece: its token's index in the sequence and its query head.
__device__ __forceinline__ void row_of(const PagedLaunch& p, int first_row, int r, int hk,
                                       int& token, int& head) {
  token = (first_row + r) / p.group;
  head = hk * p.group + (first_row + r) - token * p.group;
}

__device__ __forceinline__ float paged_slope2(const PagedLaunch& p, int b, int head) {
  return -1.4426950408889634f * p.alibi[static_cast<long long>(b) * p.alibi_bstride + head];
}

template <bool kBf16, int kN>
__device__ __forceinline__ void store16(uint16_t* dst, const float (&o)[kN], float scale) {
  if constexpr (kN == 4) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack2<kBf16>(o[0] * scale, o[1] * scale),
                                                pack2<kBf16>(o[2] * scale, o[3] * scale));
  } else {
    *reinterpret_cast<uint32_t*>(dst) = pack2<kBf16>(o[0] * scale, o[1] * scale);
  }
}

// Adds up the units that several CTAs worked on.  Block c looks at the unit
// its CTA c began and did not finish; the pieces are CTA c's second partial
// result and the first ones of the CTAs after it.  Warp w takes rows w,
// w + 8, ...; its lanes the D columns.  Launched to overlap the end of the
// kernel before it; the split is worked out again before waiting for it.
template <int kRows, int D, bool kBf16>
__global__ void __launch_bounds__(256) paged_join_kernel(const __grid_constant__ PagedLaunch p,
                                                         int n) {
  __shared__ Place sh;
  __shared__ long long sh_start;
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    Place at{};
    long long start = 0;
    at.total = warp_total_work<kRows>(p);
    at.begin = stretch(at.total, n, c);
    const long long end = stretch(at.total, n, c + 1);
    at.left = end - at.begin;
    if (at.left > 0) warp_locate<kRows>(p, end - 1, at, start);
    if (lane == 0) {
      sh = at;
      sh_start = start;
    }
  }
  __syncthreads();
  const Place at = sh;
  const long long start = sh_start, end = at.begin + at.left;
  pdl_wait();
  if (at.left <= 0 || at.b >= p.r.batch) return;
  SeqWork<kRows> w;
  w.load(p, at.b);
  if (start < at.begin || start + w.weight <= end) return;
  int last = c;  // CTAs c .. last hold pieces
  while (stretch(at.total, n, last + 1) < start + w.weight) ++last;
  const int hk = at.unit / w.blocks, block = at.unit - hk * w.blocks;
  const int rows = min(kRows, w.s.rows * p.group - block * kRows);
  constexpr int kN = D / 32;
  for (int r = warp; r < rows; r += 8) {
    auto piece = [&](int i) {
      return (2LL * i + (i == c ? 1 : 0)) * kRows + r;
    };
    // (a CTA with an empty stretch wrote nothing)
    auto empty = [&](int i) { return stretch(at.total, n, i) == stretch(at.total, n, i + 1); };
    float m = -INFINITY;
    for (int i = c + lane; i <= last; i += 32)
      if (!empty(i)) m = fmaxf(m, p.part_ml[piece(i)].x);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
    const float ref = m == -INFINITY ? 0.f : m;
    float o[kN] = {}, l = 0.f;
#pragma unroll 4
    for (int i = c; i <= last; ++i) {
      if (empty(i)) continue;
      const float2 ml = p.part_ml[piece(i)];
      const float a = ex2_approx(ml.x - ref);
      l = fmaf(ml.y, a, l);
      const float* src = p.part_o + piece(i) * D + lane * kN;
      float x[kN];
      if constexpr (kN == 4) {
        const float4 v = *reinterpret_cast<const float4*>(src);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
      } else {
        const float2 v = *reinterpret_cast<const float2*>(src);
        x[0] = v.x; x[1] = v.y;
      }
#pragma unroll
      for (int e = 0; e < kN; ++e) o[e] = fmaf(x[e], a, o[e]);
    }
    int token, head;
    row_of(p, block * kRows, r, hk, token, head);
    const long long row = w.s.start + token;
    store16<kBf16>(static_cast<uint16_t*>(p.o) + row * p.o_token + head * p.o_head + lane * kN, o,
                   l == 0.f ? 0.f : 1.f / l);
    if (lane == 0)
      p.lse[static_cast<long long>(head) * p.r.total + row] =
          l == 0.f ? -INFINITY : (m + lg2_approx(l)) * kPagedLn2;
  }
}

}  // namespace fa
