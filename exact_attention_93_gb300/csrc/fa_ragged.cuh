// fa_ragged.cuh -- device side of a packed ragged batch over a paged cache:
// which sequence a packed row belongs to, and where its keys live.  Nothing
// here trusts the device arrays: whatever they hold, the results index inside
// the caller's buffers or say that there is nothing to index.
#pragma once

#include "fa_serve.h"
#include "sm103_primitives.cuh"

namespace fa {

// The sequence of packed row `row`, or -1 when it belongs to none (before
// cu[0], or from cu[batch] on).  The lanes' rows ascend and lie close together:
// the whole warp looks for `first`, the least of them, sampling 32 boundaries at
// a step, so that 1024 sequences take two dependent loads, and each lane goes on
// from there.
__device__ __forceinline__ int warp_find_seq(const int* __restrict__ cu, int batch, int first,
                                             int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = batch;  // the number of b in 1 .. batch with cu[b] <= row is in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + (lane + 1) * step - 1;
    const int n = __popc(__ballot_sync(0xffffffffu, i < hi && cu[1 + min(i, batch - 1)] <= first));
    lo += n * step;
    hi = min(hi, lo + step - 1);
  }
  while (lo < batch && cu[lo + 1] <= row) ++lo;
  return lo < batch && cu[0] <= row ? lo : -1;
}

// One sequence of the batch, its bounds clamped to the arrays'.
struct Seq {
  int start, rows;  // packed rows start .. start + rows - 1
  int len;          // keys in the cache
  int pos0;         // position of row `start`: len - rows (negative: rows without keys)
};

__device__ __forceinline__ Seq load_seq(const Ragged& r, int page_log2, int b, uint32_t* err) {
  Seq s;
  const int c0 = r.cu[b], c1 = r.cu[b + 1], n = r.lens[b];
  s.start = min(max(c0, 0), r.total);
  s.rows = min(max(c1, s.start), r.total) - s.start;
  const long long most = static_cast<long long>(r.max_pages) << page_log2;
  s.len = static_cast<int>(min(static_cast<long long>(max(n, 0)), most));
  s.pos0 = s.len - s.rows;
  if (err && (n < 0 || n > most || c0 < 0 || c1 < c0 || c1 > r.total))
    atomicExch(err, kDevErrBadIndex);
  return s;
}

}  // namespace fa
