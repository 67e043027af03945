// fa_decoder_api.cu -- the C ABI of include/fattn_decoder.h but for attention: argument
// checks and kernel launches.  No arithmetic of the operators lives here.
#include <algorithm>
#include <cmath>

#include "fa_checks.h"
#include "fa_norm.h"
#include "fa_tables.h"

namespace fa {
namespace {

fa_status norm_arguments(NormLaunch& a, const fa_rotary_operand* q, const fa_rotary_operand* k,
                         const void* q_weight, const void* k_weight, fa_elem weight_dtype,
                         float eps, int B, int N, int D, int rotary_dim, const double* inv_freq,
                         const fa_positions* positions, float magnitude, int interleaved,
                         fa_elem dtype, bool& done) {
  if (!positions) return FA_ERR_INVALID_ARG;
  const fa_status st = rotary_arguments(a.rot, q, k, B, N, D, rotary_dim, inv_freq, *positions,
                                        magnitude, dtype, done);
  if (st != FA_OK) return st;
  if (weight_dtype != dtype && weight_dtype != FA_ELEM_FP32) return FA_ERR_UNSUPPORTED;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return FA_ERR_INVALID_ARG;
  if ((q_weight && !aligned(q_weight, 8)) || (k_weight && (!aligned(k_weight, 8) || !k)))
    return FA_ERR_INVALID_ARG;
  a.rot.interleaved = interleaved != 0;
  a.weight[0] = q_weight;
  a.weight[1] = k_weight;
  a.weight_elem = weight_dtype;
  a.eps = eps;
  return FA_OK;
}

bool table_ok(const int* table, long long stride, int max_pages, int batch, int page_size,
              const int* free_pages, int capacity) {
  return batch >= 1 && batch <= (1 << 20) && max_pages >= 1 && stride >= max_pages &&
         stride <= kMaxBytes && page_size >= 16 && page_size <= 256 &&
         (page_size & (page_size - 1)) == 0 && capacity >= 0 &&
         static_cast<long long>(max_pages) * page_size <= kMaxRows && aligned(table, 4) &&
         (capacity == 0 || aligned(free_pages, 4));
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_rotary_axes(const fa_rotary_operand* q, const fa_rotary_operand* k, int B, int N,
                         int D, int rotary_dim, const double* inv_freq,
                         const fa_positions* positions, float magnitude, int interleaved,
                         int inverse, fa_elem dtype, void* stream) {
  if (!positions) return FA_ERR_INVALID_ARG;
  RotaryLaunch a{};
  bool done;
  const fa_status st =
      rotary_arguments(a, q, k, B, N, D, rotary_dim, inv_freq, *positions, magnitude, dtype, done);
  if (st != FA_OK || done) return st;
  a.interleaved = interleaved != 0;
  a.inverse = inverse != 0;
  return launch_rotary(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_qk_norm_rotary(const fa_rotary_operand* q, const fa_rotary_operand* k,
                            const void* q_weight, const void* k_weight, fa_elem weight_dtype,
                            float eps, int B, int N, int D, int rotary_dim,
                            const double* inv_freq, const fa_positions* positions,
                            float magnitude, int interleaved, fa_elem dtype, void* stream) {
  NormLaunch a{};
  bool done;
  const fa_status st =
      norm_arguments(a, q, k, q_weight, k_weight, weight_dtype, eps, B, N, D, rotary_dim, inv_freq,
                     positions, magnitude, interleaved, dtype, done);
  if (st != FA_OK || done) return st;
  return launch_norm_rotary(a, false, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? FA_OK
             : FA_ERR_CUDA;
}

fa_status fa_qk_norm_rotary_bwd_workspace_size(int D, size_t* bytes) {
  if (!bytes) return FA_ERR_INVALID_ARG;
  *bytes = 0;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  int sms = 0;
  if (sm_count(&sms) != cudaSuccess) sms = 160;  // no device: sizes for the checks alone
  *bytes = round256(sizeof(float) * kNormBlocks * sms * D);
  return FA_OK;
}

fa_status fa_qk_norm_rotary_bwd(const fa_rotary_operand* q, const fa_rotary_operand* k,
                                const void* dq_out, fa_strides dq_strides, const void* dk_out,
                                fa_strides dk_strides, const void* q_weight,
                                const void* k_weight, void* dq_weight, void* dk_weight,
                                fa_elem weight_dtype, float eps, int B, int N, int D,
                                int rotary_dim, const double* inv_freq,
                                const fa_positions* positions, float magnitude, int interleaved,
                                fa_elem dtype, void* workspace, size_t workspace_bytes,
                                void* stream) {
  NormLaunch a{};
  bool done;
  fa_status st =
      norm_arguments(a, q, k, q_weight, k_weight, weight_dtype, eps, B, N, D, rotary_dim, inv_freq,
                     positions, magnitude, interleaved, dtype, done);
  if (st != FA_OK) return st;
  if ((dq_weight && !aligned(dq_weight, 8)) || (dk_weight && (!aligned(dk_weight, 8) || !k)) ||
      (dq_weight && dq_weight == dk_weight))
    return FA_ERR_INVALID_ARG;
  size_t need = 0;
  if ((st = fa_qk_norm_rotary_bwd_workspace_size(D, &need)) != FA_OK) return st;
  if (!aligned(workspace, 256) || workspace_bytes < need) return FA_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (done) {  // no rows: sums of nothing
    const size_t bytes = static_cast<size_t>(D) * elem_bytes(weight_dtype);
    for (void* w : {dq_weight, dk_weight})
      if (w && cudaMemsetAsync(w, 0, bytes, s) != cudaSuccess) return FA_ERR_CUDA;
    return FA_OK;
  }
  const void* dy[2] = {dq_out, dk_out};
  const fa_strides strides[2] = {dq_strides, dk_strides};
  const int es = elem_bytes(dtype);
  for (int i = 0; i < (k ? 2 : 1); ++i) {
    const long long extent[3] = {B, a.rot.heads[i], N};
    const long long st3[3] = {strides[i].batch, strides[i].head, strides[i].seq};
    if (!aligned(dy[i], 16) || !strides_ok(st3, extent, 3, D, es, 16) || a.rot.x[i] == a.rot.y[i] ||
        dy[i] == a.rot.y[i])
      return FA_ERR_INVALID_ARG;
    a.dy[i] = dy[i];
    a.dys[i] = RowStrides{strides[i].batch, strides[i].head, strides[i].seq};
  }
  a.rot.inverse = 1;
  a.dweight[0] = dq_weight;
  a.dweight[1] = dk_weight;
  a.partial = static_cast<float*>(workspace);
  return launch_norm_rotary(a, true, s) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_cache_reserve(const fa_reserve* r, void* stream) {
  if (!r || r->total < 0 || r->total > kMaxRows ||
      !table_ok(r->block_table, r->table_stride, r->max_pages, r->batch, r->page_size,
                r->free_pages, r->capacity))
    return FA_ERR_INVALID_ARG;
  for (const void* p : {static_cast<const void*>(r->new_tokens), static_cast<const void*>(r->seqlens),
                        static_cast<const void*>(r->free_count), static_cast<const void*>(r->cu_seqlens),
                        static_cast<const void*>(r->seqlens_out),
                        static_cast<const void*>(r->free_count_out),
                        static_cast<const void*>(r->missing)})
    if (!aligned(p, 4)) return FA_ERR_INVALID_ARG;
  if (r->total > 0 && (!aligned(r->positions, 4) || !aligned(r->slots, 8)))
    return FA_ERR_INVALID_ARG;
  ReserveLaunch a{};
  a.fresh = r->new_tokens;
  a.lens = r->seqlens;
  a.table = r->block_table;
  a.table_stride = r->table_stride;
  a.max_pages = r->max_pages;
  a.page_log2 = log2_of(r->page_size);
  a.batch = r->batch;
  a.total = r->total;
  a.capacity = r->capacity;
  a.free_pages = r->free_pages;
  a.free_count = r->free_count;
  a.cu = r->cu_seqlens;
  a.lens_out = r->seqlens_out;
  a.positions = r->positions;
  a.free_count_out = r->free_count_out;
  a.missing = r->missing;
  a.slots = r->slots;
  a.in_place = a.lens_out == a.lens || a.free_count_out == a.free_count;
  a.err = device_error_word();
  if (!a.err) return FA_ERR_CUDA;
  return launch_reserve(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_cache_release(const unsigned char* done, int* seqlens, const int* keep_pages,
                           const int* block_table, long long table_stride, int max_pages,
                           int* free_pages, int capacity, int* free_count, int batch,
                           int page_size, void* stream) {
  if (!done || !aligned(seqlens, 4) || (keep_pages && !aligned(keep_pages, 4)) ||
      !aligned(free_count, 4) ||
      !table_ok(block_table, table_stride, max_pages, batch, page_size, free_pages, capacity))
    return FA_ERR_INVALID_ARG;
  ReleaseLaunch a{done,      seqlens,  keep_pages, block_table,           table_stride,
                  max_pages, log2_of(page_size), batch, capacity, free_pages, free_count,
                  device_error_word()};
  if (!a.err) return FA_ERR_CUDA;
  return launch_release(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_cache_write(const fa_kv_pages* cache, const long long* slots, int total,
                         const void* k, long long k_token, long long k_head, const void* v,
                         long long v_token, long long v_head, fa_elem dtype, void* stream) {
  if (total < 0 || total > kMaxRows || (total > 0 && !aligned(slots, 8))) return FA_ERR_INVALID_ARG;
  fa_ragged batch{};
  batch.total = total;
  return cache_rows(cache, &batch, nullptr, slots, k, k_token, k_head, v, v_token, v_head, dtype,
                    stream, true);
}

}  // extern "C"
