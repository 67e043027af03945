// fa_serve.h -- launch interface of the rotary, paged-cache and
// paged-attention kernels (include/fattn_cache.h): the argument blocks the
// kernels take and the launchers fa_serve_api.cu calls.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "fa_internal.h"

namespace fa {

// Element types, with fa_elem's values.
enum : int { kElemBf16 = 0, kElemFp16 = 1, kElemFp32 = 2, kElemE4m3 = 3 };

struct RotaryLaunch {
  const void* x[2];
  void* y[2];
  RowStrides xs[2], ys[2];
  int heads[2];  // heads[1] == 0: one operand
  int B, N, D, rotary;
  const double* inv_freq;
  const void* positions;
  int position_bits;
  long long position_bstride;
  float magnitude;
  int interleaved, inverse, elem;
};

cudaError_t launch_rotary(const RotaryLaunch& a, cudaStream_t s);

// The packed batch: who owns which rows, and where their keys live.
struct Ragged {
  const int* table;
  long long table_stride;
  int max_pages;
  const int* cu;
  const int* lens;  // append, attention: lengths; read: first positions (may be null)
  int batch, total;
};

// Strides in elements of the cache's type.
struct Pages {
  void* p[2];  // keys, values
  uint8_t* exp[2];
  long long page[2], token[2], head[2];
  int pages, page_size, page_log2, heads, D, elem;
};

struct CacheLaunch {
  Pages c;
  Ragged r;
  void* rows[2];  // packed keys, values
  long long row_token[2], row_head[2];
  int elem;  // of the packed rows
  uint32_t* err;
};

cudaError_t launch_cache_append(const CacheLaunch& a, cudaStream_t s);
cudaError_t launch_cache_read(const CacheLaunch& a, cudaStream_t s);

struct JoinTask;

// Attention over pages.  Scores work in log2 units.
struct PagedLaunch {
  // keys and values: {D, page_size, heads, pages}, box {128 bytes (64 for
  // 64-byte rows), min(page_size, 128), 1, 1}
  CUtensorMap map_k, map_v;
  // queries of the many-row kernel: {D, heads, total}, box {64, group, tokens of a tile}
  CUtensorMap map_q;
  const void* q;
  long long q_token, q_head;
  void* o;
  long long o_token, o_head;
  float* lse;  // [heads][total]
  const uint8_t *k_exp, *v_exp;
  Ragged r;
  int heads, heads_k, group, D;
  int pages, page_size, page_log2;
  int cache_elem, elem;
  float scale_log2;
  int win_left, win_right;  // causal: win_right = 0
  const float* alibi;
  int alibi_bstride;
  int block_rows;   // query rows of a unit
  int min_rows, max_rows;  // sequences of other numbers of rows (tokens x group) are left out
  int whole;        // units are not cut
  // unless whole:
  float* part_o;    // [2 sms][block_rows][D]
  float2* part_ml;  // [2 sms][block_rows]: maximum, sum
  JoinTask* tasks;  // [sms]
  int sms;          // CTAs of the grid
  uint32_t* err;
};

// Query rows (tokens x group) of a block of the few-row kernel, for sequences of
// `rows` rows on average, and of the many-row kernel.
int paged_few_rows(double rows);
int paged_many_rows(int group);
cudaError_t launch_paged_many(const PagedLaunch& a, cudaStream_t s);
cudaError_t launch_paged_few(const PagedLaunch& a, cudaStream_t s);

}  // namespace fa
