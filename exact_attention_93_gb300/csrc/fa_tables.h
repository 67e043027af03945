// fa_tables.h -- launch interface of the kernels that build a paged cache's tables.
#pragma once

#include <algorithm>

#include "fa_serve.h"

namespace fa {

struct ReserveLaunch {
  const int *fresh, *lens;  // new tokens, lengths before
  int* table;
  long long table_stride;
  int max_pages, page_log2, batch, total, capacity;
  const int *free_pages, *free_count;
  int *cu, *lens_out, *positions, *free_count_out, *missing;
  long long* slots;
  int in_place;  // lens_out is lens, or free_count_out free_count
  uint32_t* err;
};

struct ReleaseLaunch {
  const uint8_t* done;
  int* lens;
  const int* keep;  // or null
  const int* table;
  long long table_stride;
  int max_pages, page_log2, batch, capacity;
  int *free_pages, *free_count;
  uint32_t* err;
};

cudaError_t launch_reserve(const ReserveLaunch& a, cudaStream_t s);
cudaError_t launch_release(const ReleaseLaunch& a, cudaStream_t s);

}  // namespace fa
