// fa_paged.cuh -- what the attention-over-pages kernels share: which keys a
// block of queries sees, how the work is split over the CTAs, and the joining
// of blocks that several CTAs worked on.
//
// Units.  A unit is one block of query rows (rows token * group +
// head-in-group of one sequence) against one key head.  It walks tiles of 128
// keys.  Units are laid end to end by their weights, key head by key head and
// within a head sequence by sequence, and each CTA takes an equal stretch of the
// whole, cutting units where the stretch ends: a long context over few rows is
// spread over every SM, ragged batches stay balanced, and a CTA leaves at most two
// cut pieces whatever the batch.  Cut pieces go to the workspace in fp32
// (unnormalised O, maximum, sum) and paged_join_kernel adds them up in a fixed
// order.  Where no sequence of the table can be long (PagedLaunch::whole), units
// stay whole instead, each with the CTA whose stretch it begins in, and nothing
// is left to join.
//
// Heads come first in that order because a token's rows of all heads lie side by
// side: the CTAs of the heads then walk the same tokens at about the same time,
// and what one leaves in an open DRAM page the others find there.
//
// Weights.  The few-row kernel gives all units of a sequence the number of key
// tiles that any of its queries sees, at least 1 (a sequence usually is one
// block).  The many-row kernel counts each block's own tiles, plus kUnitCost
// for what a unit costs beside its tiles: under a causal mask the blocks of a
// prompt see from one tile to all of them.  The sums over blocks that this
// needs are sums of floor((a + i b) / 128), taken in closed form.
#pragma once

#include "fa_ragged.cuh"

namespace fa {

constexpr float kPagedLn2 = 0.6931471805599453f;
// Loading Q, filling the pipeline and writing O take the many-row kernel about
// as long as three key tiles.
constexpr int kUnitCost = 3;

// Keys [lo, hi) that some query of tokens [t0, t1) of the sequence sees.
__device__ __forceinline__ void visible_span(const PagedLaunch& p, const Seq& s, int t0, int t1,
                                             int& lo, int& hi) {
  lo = p.win_left < 0 ? 0 : max(0, s.pos0 + t0 - p.win_left);
  const long long last = static_cast<long long>(s.pos0) + t1 - 1 + p.win_right;
  hi = p.win_right < 0 ? s.len
                       : static_cast<int>(max(0LL, min(static_cast<long long>(s.len), last + 1)));
  if (lo >= hi) lo = hi = 0;
}

// sum over i < n of floor((a i + b) / m), a and b not negative: the lattice points
// under a line, counted by the reciprocity of such sums (Graham, Knuth and Patashnik,
// Concrete Mathematics, section 3.5), which takes (a, m) through the steps of Euclid's
// algorithm.  m starts at 128 and n below 2^23, so that a n + b, with a and b reduced,
// fits 32 bits throughout.
__device__ __forceinline__ long long floor_sum(uint32_t n, uint32_t m, uint32_t a, uint32_t b) {
  long long sum = 0;
  while (n > 0) {
    if (a >= m) {
      sum += static_cast<long long>(n) * (n - 1) / 2 * (a / m);
      a %= m;
    }
    if (b >= m) {
      sum += static_cast<long long>(n) * (b / m);
      b %= m;
    }
    const uint32_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y - n * m;
    const uint32_t t = m;
    m = a;
    a = t;
  }
  return sum;
}

// sum over i < n of max(0, floor((a + i b) / 128)).
__device__ __forceinline__ long long tile_sum(int n, int a, int b) {
  const int skip = a < 0 ? min(n, (-a + b - 1) / b) : 0;
  return floor_sum(static_cast<uint32_t>(n - skip), kTile, static_cast<uint32_t>(b),
                   static_cast<uint32_t>(a + skip * b));
}

// A sequence as the work split sees it.
template <bool kMany>
struct SeqWork {
  Seq s;
  int blocks;  // query blocks per key head
  int flat;    // few rows: the weight of every unit
  int first;   // few rows: the first key tile
  __device__ __forceinline__ void load(const PagedLaunch& p, int b, uint32_t* err = nullptr) {
    s = load_seq(p.r, p.page_log2, b, err);
    const int rows = s.rows * p.group;
    blocks = rows < p.min_rows || rows > p.max_rows ? 0 : (rows + p.block_rows - 1) / p.block_rows;
    if constexpr (!kMany) {
      int lo, hi;
      visible_span(p, s, 0, s.rows, lo, hi);
      first = lo / kTile;
      flat = max(1, (hi + kTile - 1) / kTile - first);
    }
  }
  // Weight of the blocks before block i of a head.
  __device__ __forceinline__ long long before(const PagedLaunch& p, int i) const {
    if constexpr (!kMany) return static_cast<long long>(flat) * i;
    const int bt = p.block_rows / p.group;  // tokens of a block
    long long sum = static_cast<long long>(kUnitCost) * i;
    int open = 0;  // leading blocks whose keys end before the sequence's
    if (p.win_right >= 0) {
      const int end = s.len - s.pos0 - p.win_right;
      open = min(i, max(0, (end + bt - 1) / bt - 1));
      sum += tile_sum(open, s.pos0 + bt + p.win_right + kTile - 1, bt);
    }
    sum += static_cast<long long>(i - open) * ((s.len + kTile - 1) / kTile);
    if (p.win_left >= 0) sum -= tile_sum(i, s.pos0 - p.win_left, bt);
    return sum;
  }
};

// A CTA's place in the laid-out work.
struct Place {
  int b, hk, block;
  long long off;    // into the unit
  long long pos;    // into the whole
  long long left;   // of this CTA's stretch
  long long total;
};

// a / b for a >= 0, b > 0; a 64-bit division is a long instruction sequence.
__device__ __forceinline__ long long divide(long long a, long long b) {
  if (((a | b) >> 32) == 0)
    return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// floor(total c / n)
__device__ __forceinline__ long long stretch(long long total, int n, int c) {
  const long long q = divide(total, n);
  const uint32_t r = static_cast<uint32_t>(total - q * n);
  return q * c + r * static_cast<uint32_t>(c) / static_cast<uint32_t>(n);
}

__device__ __forceinline__ long long warp_sum(long long v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

// Where CTA c of n begins, by one warp.
template <bool kMany>
__device__ __forceinline__ Place warp_place(const PagedLaunch& p, int n, int c) {
  const int lane = threadIdx.x & 31;
  Place at{};
  // lane i sums over sequences i, i + 32, ...; the first 32 stay at hand
  SeqWork<kMany> w;
  long long seq0 = 0;
  for (int b = lane; b < p.r.batch; b += 32) {
    w.load(p, b, c == 0 ? p.err : nullptr);
    const long long mine = w.blocks ? w.before(p, w.blocks) : 0;
    if (b == lane) seq0 = mine;
    at.total += mine;
  }
  const long long head = warp_sum(at.total);  // the work of one key head
  at.total = head * p.heads_k;
  at.pos = stretch(at.total, n, c);
  at.left = stretch(at.total, n, c + 1) - at.pos;
  if (at.left == 0) return at;
  at.hk = static_cast<int>(divide(at.pos, head));
  const long long in = at.pos - at.hk * head;  // in that head's work
  long long ahead = 0;
  for (int b0 = 0; b0 < p.r.batch; b0 += 32) {
    long long mine = seq0;
    if (b0 > 0) {
      mine = 0;
      if (b0 + lane < p.r.batch) {
        w.load(p, b0 + lane);
        if (w.blocks) mine = w.before(p, w.blocks);
      }
    }
    long long upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += o;
    }
    const uint32_t past = __ballot_sync(0xffffffffu, ahead + upto > in);
    if (past) {
      const int src = __ffs(past) - 1;
      at.b = b0 + src;
      const long long rem = in - ahead - __shfl_sync(0xffffffffu, upto - mine, src);
      w.load(p, at.b);
      // the last block whose predecessors weigh at most rem: 32 tries at once
      int lo = 0, hi = w.blocks;  // it is in [lo, hi)
      while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int i = lo + lane * step;
        const uint32_t ok = __ballot_sync(0xffffffffu, i < hi && w.before(p, i) <= rem);
        lo += (__popc(ok) - 1) * step;
        hi = min(hi, lo + step);
      }
      at.block = lo;
      const long long start = lo ? w.before(p, lo) : 0;
      at.off = rem - start;
      if (p.whole && at.off > 0) {  // the unit belongs to a CTA before this one
        const long long rest = w.before(p, lo + 1) - rem;
        at.pos += rest;
        at.left = max(0LL, at.left - rest);
        at.off = 0;
        ++at.block;
      }
      return at;
    }
    ahead += __shfl_sync(0xffffffffu, upto, 31);
  }
  at.left = 0;  // not reached
  return at;
}

// A CTA's next piece of work.
struct Piece {
  int b, hk, block;
  int t0, t1;        // the block's tokens
  int rows;          // valid rows of the block
  int lo, hi;        // keys some row of the block sees
  int tile0, tile1;  // key tiles to walk (none: tile0 >= tile1)
  bool whole;        // the piece covers its unit
  int slot;          // of the CTA's two partial results, when it does not
  int last;          // when the unit begins here and goes on: the CTA that ends it
};

// What paged_join_kernel does for a CTA: add up the unit that it began and
// did not finish.
struct JoinTask {
  int rows;  // 0: nothing to do; -1: the CTA had no work at all
  int start, first_row, hk, last;
};

// Walks a CTA's stretch.  Every role of the CTA runs its own copy.
template <bool kMany>
struct WorkWalk {
  Place at;
  SeqWork<kMany> w;
  bool loaded;
  __device__ __forceinline__ explicit WorkWalk(const Place& start) : at(start), loaded(false) {}
  __device__ __forceinline__ bool next(const PagedLaunch& p, Piece& x) {
    if (at.left <= 0) return false;
    if (!loaded) {
      w.load(p, at.b);
      loaded = true;
    }
    while (at.block >= w.blocks) {  // (a sequence without rows has no blocks)
      at.block = 0;
      if (++at.b >= p.r.batch) {
        at.b = 0;
        if (++at.hk >= p.heads_k) return false;
      }
      w.load(p, at.b);
    }
    x.b = at.b;
    x.hk = at.hk;
    x.block = at.block;
    const int row0 = x.block * p.block_rows;
    x.rows = min(p.block_rows, w.s.rows * p.group - row0);
    x.t0 = row0 / p.group;
    x.t1 = (row0 + x.rows - 1) / p.group + 1;
    visible_span(p, w.s, x.t0, x.t1, x.lo, x.hi);
    const int lo_tile = x.lo / kTile, hi_tile = (x.hi + kTile - 1) / kTile;
    const int weight = kMany ? kUnitCost + hi_tile - lo_tile : w.flat;
    const int off = static_cast<int>(at.off);
    const int take =
        p.whole ? weight : static_cast<int>(min(at.left, static_cast<long long>(weight - off)));
    x.whole = take == weight;
    x.slot = off > 0 ? 0 : 1;
    const int base = kMany ? lo_tile - kUnitCost : w.first;
    x.tile0 = max(base + off, lo_tile);
    x.tile1 = min(base + off + take, hi_tile);
    x.last = -1;
    if (off == 0 && take < weight)
      x.last = static_cast<int>(((at.pos + weight) * static_cast<long long>(gridDim.x) - 1) /
                                at.total);
    at.off += take;
    at.pos += take;
    at.left -= take;
    if (off + take == weight) {
      at.off = 0;
      ++at.block;
    }
    return true;
  }
};

// By one thread of the CTA: the task for its last piece.
__device__ __forceinline__ JoinTask join_task(const PagedLaunch& p, const Piece& x, const Seq& s) {
  return JoinTask{x.last >= 0 ? x.rows : 0, s.start, x.block * p.block_rows, x.hk, x.last};
}

// The pages of a piece's tiles, for a producer warp: 32 table entries at a time,
// the next 32 on their way, so that no tile waits for a load of its entries.
struct PageFeed {
  const int* table;
  int first;       // page index that lane 0's entry belongs to
  int lo, hi;      // pages that hold a visible key
  int cur, next;
  __device__ __forceinline__ int load(int i) const { return i >= lo && i <= hi ? table[i] : -1; }
  __device__ __forceinline__ void start(const PagedLaunch& p, int b, int tile, int key_lo,
                                        int key_hi) {
    table = p.r.table + b * p.r.table_stride;
    first = (tile * kTile) >> p.page_log2;
    lo = key_lo >> p.page_log2;
    hi = (key_hi - 1) >> p.page_log2;
    cur = load(first + (threadIdx.x & 31));
    next = load(first + 32 + (threadIdx.x & 31));
  }
  // The page of the box of a tile that starts at key k0 (this lane's); tiles
  // come in order.  A tile's pages never straddle two sets of 32: they are
  // at most eight, a power of two, and the first set starts with a tile.
  __device__ __forceinline__ int get(const PagedLaunch& p, int tile, int k0) {
    if (((tile * kTile) >> p.page_log2) - first >= 32) {
      first += 32;
      cur = next;
      next = load(first + 32 + (threadIdx.x & 31));
    }
    return __shfl_sync(0xffffffffu, cur, ((k0 >> p.page_log2) - first) & 31);
  }
};

// Row r of a block that starts at row first_row of its sequence: its token
// and its query head.
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

// Adds up the units that several CTAs worked on.  Block (c, y) takes a share of
// the rows of the unit that CTA c began and did not finish; its pieces are CTA
// c's second partial result and the first ones of the CTAs after it.  A warp's
// lanes are the D columns of kRowsAtOnce rows, kPieces pieces of which it loads
// side by side: the loads' latency is all this costs.  A long context over few
// rows has up to a hundred pieces of a handful of rows, a prompt two or three
// pieces of 256.
constexpr int kJoinThreads = 64;

template <int D, bool kBf16, int kRowsAtOnce, int kPieces>
__global__ void __launch_bounds__(kJoinThreads)
    paged_join_kernel(const __grid_constant__ PagedLaunch p) {
  pdl_wait_and_release();
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const JoinTask task = p.tasks[c];
  constexpr int kN = D / 32, kWarps = kJoinThreads / 32;
  const int step = gridDim.y * kWarps * kRowsAtOnce;
  for (int r0 = (blockIdx.y * kWarps + warp) * kRowsAtOnce; r0 < task.rows; r0 += step) {
    float m[kRowsAtOnce], l[kRowsAtOnce] = {}, o[kRowsAtOnce][kN] = {};
#pragma unroll
    for (int q = 0; q < kRowsAtOnce; ++q) m[q] = -INFINITY;
    // up to 32 CTAs at a time: lane i knows whether CTA first + i had work
    for (int first = c; first <= task.last; first += 32) {
      uint32_t live = __ballot_sync(
          0xffffffffu, first + lane <= task.last && p.tasks[min(first + lane, task.last)].rows >= 0);
      while (live) {
        float2 ml[kPieces][kRowsAtOnce];
        float x[kPieces][kRowsAtOnce][kN];
#pragma unroll
        for (int k = 0; k < kPieces; ++k) {
          const bool some = live != 0;
          const int i = first + (some ? __ffs(live) - 1 : 0);
          live &= live - 1;
          const long long at = (2LL * i + (i == c ? 1 : 0)) * p.block_rows + r0;
#pragma unroll
          for (int q = 0; q < kRowsAtOnce; ++q) {
            const bool valid = some && r0 + q < task.rows;
            ml[k][q] = valid ? p.part_ml[at + q] : make_float2(-INFINITY, 0.f);
            // (of pieces without keys there is a maximum alone, -inf; what this
            // finds there is not used)
            const float* src = p.part_o + (at + q) * D + lane * kN;
            if constexpr (kN == 4) {
              const float4 v = valid ? *reinterpret_cast<const float4*>(src)
                                     : make_float4(0.f, 0.f, 0.f, 0.f);
              x[k][q][0] = v.x; x[k][q][1] = v.y; x[k][q][2] = v.z; x[k][q][3] = v.w;
            } else {
              const float2 v =
                  valid ? *reinterpret_cast<const float2*>(src) : make_float2(0.f, 0.f);
              x[k][q][0] = v.x; x[k][q][1] = v.y;
            }
          }
        }
#pragma unroll
        for (int k = 0; k < kPieces; ++k)
#pragma unroll
          for (int q = 0; q < kRowsAtOnce; ++q) {
            const float m_new = fmaxf(m[q], ml[k][q].x);
            const float ref = m_new == -INFINITY ? 0.f : m_new;
            const float a = ex2_approx(m[q] - ref), b = ex2_approx(ml[k][q].x - ref);
            m[q] = m_new;
            l[q] = l[q] * a + ml[k][q].y * b;
#pragma unroll
            for (int e = 0; e < kN; ++e)
              o[q][e] = o[q][e] * a + (ml[k][q].x == -INFINITY ? 0.f : x[k][q][e] * b);
          }
      }
    }
#pragma unroll
    for (int q = 0; q < kRowsAtOnce; ++q) {
      if (r0 + q >= task.rows) continue;
      int token, head;
      row_of(p, task.first_row, r0 + q, task.hk, token, head);
      const long long row = task.start + token;
      store16<kBf16>(static_cast<uint16_t*>(p.o) + row * p.o_token + head * p.o_head + lane * kN,
                     o[q], l[q] == 0.f ? 0.f : 1.f / l[q]);
      if (lane == 0)
        p.lse[static_cast<long long>(head) * p.r.total + row] =
            l[q] == 0.f ? -INFINITY : (m[q] + lg2_approx(l[q])) * kPagedLn2;
    }
  }
}

template <int D, bool kBf16>
cudaError_t launch_join(const PagedLaunch& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  // few rows in a block: many pieces at a time; many rows: some of each
  const bool few = a.block_rows <= 16;
  const int rows = kJoinThreads / 32 * (few ? 1 : 2);
  cfg.gridDim = dim3(static_cast<unsigned>(a.sms),
                     static_cast<unsigned>((a.block_rows + rows - 1) / rows));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return few ? cudaLaunchKernelEx(&cfg, paged_join_kernel<D, kBf16, 1, 8>, a)
             : cudaLaunchKernelEx(&cfg, paged_join_kernel<D, kBf16, 2, 2>, a);
}

}  // namespace fa
