// fa_serve_api.cu -- the C ABI of include/fattn_cache.h: argument checks, TMA
// descriptor set-up, workspace layout and kernel launches.  No arithmetic of
// the operators lives here.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "fa_internal.h"
#include "fa_serve.h"
#include "fattn_cache.h"
#include "host_tmap.hpp"

namespace fa {
namespace {

constexpr long long kMaxBytes = 1ll << 40;  // every operand lies below this from its base
constexpr int kMaxRows = 1 << 29;           // packed rows, keys of a sequence, window bounds
constexpr float kLog2e = 1.4426950408889634f;
// Keys up to which units stay whole.  (us, cut and whole: one sequence of 1000
// keys 9.9 and 9.6, of 1500 10.8 and 11.9, 8 of 1000 13.7 and 10.4; prompts of
// 4 x 300 tokens 28.2 and 16.9, of 1500 tokens 39.4 and 31.9.)  The keys alone decide,
// and with fewer units than SMs whole units leave some without work: 9 chunks of 1 to
// 500 tokens under a window of 1000, 72 units, take 35 us; cut, they were not measured.
constexpr int kWholeKeysFew = 1536, kWholeKeysMany = 1536;

bool aligned(const void* p, uintptr_t n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

int elem_bytes(int elem) { return elem == FA_ELEM_FP32 ? 4 : elem == FA_ELEM_E4M3 ? 1 : 2; }

bool is16(int elem) { return elem == FA_ELEM_BF16 || elem == FA_ELEM_FP16; }

// Strides of one operand: non-negative, `unit`-byte multiples, and the last
// element below kMaxBytes.
bool strides_ok(const long long* st, const long long* extent, int n, int D, int es, int unit) {
  double last = D;
  for (int i = 0; i < n; ++i) {
    if (st[i] < 0 || (st[i] * es) % unit != 0 || st[i] > kMaxBytes) return false;
    last += static_cast<double>(extent[i] - 1) * st[i];
  }
  return last * es < static_cast<double>(kMaxBytes);
}

// An operand that is written: every index has elements of its own (strides below
// a row would let rows share them).
bool apart(const long long* st, const long long* extent, int n, int D) {
  for (int i = 0; i < n; ++i)
    if (extent[i] > 1 && st[i] < D) return false;
  return true;
}

fa_status check_batch(const fa_ragged* b, bool lens_needed) {
  if (!b || b->batch < 1 || b->total < 0 || b->total > kMaxRows || b->max_pages < 1)
    return FA_ERR_INVALID_ARG;
  if (!aligned(b->block_table, 4) || !aligned(b->cu_seqlens, 4) || b->table_stride < b->max_pages)
    return FA_ERR_INVALID_ARG;
  if (lens_needed && !aligned(b->seqlens, 4)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

fa_status check_pages(const fa_kv_pages* c, const fa_ragged* b, fa_elem dtype) {
  if (!c) return FA_ERR_INVALID_ARG;
  if (c->head_dim != 64 && c->head_dim != 128) return FA_ERR_UNSUPPORTED;
  if (!is16(dtype) || (!is16(c->type) && c->type != FA_ELEM_E4M3)) return FA_ERR_UNSUPPORTED;
  if (is16(c->type) && c->type != static_cast<int>(dtype)) return FA_ERR_UNSUPPORTED;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)))
    return FA_ERR_UNSUPPORTED;
  if (c->pages < 1 || c->heads < 1 || c->heads > 65535) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(b->max_pages) * c->page_size > kMaxRows) return FA_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16)) return FA_ERR_INVALID_ARG;
  if (c->type == FA_ELEM_E4M3 && (!aligned(c->k_exp, 16) || !aligned(c->v_exp, 16)))
    return FA_ERR_INVALID_ARG;
  const long long extent[3] = {c->pages, c->page_size, c->heads};
  const long long ks[3] = {c->k_page, c->k_token, c->k_head};
  const long long vs[3] = {c->v_page, c->v_token, c->v_head};
  const int es = elem_bytes(c->type);
  if (!strides_ok(ks, extent, 3, c->head_dim, es, 16) ||
      !strides_ok(vs, extent, 3, c->head_dim, es, 16))
    return FA_ERR_INVALID_ARG;
  return FA_OK;
}

// A packed [total][heads][D] operand of 16-bit elements.
bool packed_ok(const void* p, long long token, long long head, int total, int heads, int D) {
  const long long extent[2] = {total, heads}, st[2] = {token, head};
  return aligned(p, 16) && strides_ok(st, extent, 2, D, 2, 16);
}

int log2_of(int x) {
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

Ragged ragged_of(const fa_ragged* b, const int* lens) {
  return Ragged{b->block_table, b->table_stride, b->max_pages, b->cu_seqlens, lens, b->batch,
                b->total};
}

fa_status cache_rows(const fa_kv_pages* cache, const fa_ragged* batch, const int* lens,
                     const void* k, long long k_token, long long k_head, const void* v,
                     long long v_token, long long v_head, fa_elem dtype, void* stream,
                     bool append) {
  fa_status st;
  if ((st = check_pages(cache, batch, dtype)) != FA_OK) return st;
  if (batch->total == 0) return FA_OK;
  if (!packed_ok(k, k_token, k_head, batch->total, cache->heads, cache->head_dim) ||
      !packed_ok(v, v_token, v_head, batch->total, cache->heads, cache->head_dim))
    return FA_ERR_INVALID_ARG;
  const long long pages[3] = {cache->pages, cache->page_size, cache->heads};
  const long long rows[2] = {batch->total, cache->heads};
  const long long st_k[3] = {cache->k_page, cache->k_token, cache->k_head};
  const long long st_v[3] = {cache->v_page, cache->v_token, cache->v_head};
  const long long st_rk[2] = {k_token, k_head}, st_rv[2] = {v_token, v_head};
  const int D = cache->head_dim;
  const bool distinct =
      append ? cache->k != cache->v &&
                   (cache->type != FA_ELEM_E4M3 || cache->k_exp != cache->v_exp) &&
                   apart(st_k, pages, 3, D) && apart(st_v, pages, 3, D)
             : k != v && apart(st_rk, rows, 2, D) && apart(st_rv, rows, 2, D);
  if (!distinct) return FA_ERR_INVALID_ARG;
  CacheLaunch a{};
  a.c = Pages{{cache->k, cache->v},
              {cache->k_exp, cache->v_exp},
              {cache->k_page, cache->v_page},
              {cache->k_token, cache->v_token},
              {cache->k_head, cache->v_head},
              cache->pages,
              cache->page_size,
              log2_of(cache->page_size),
              cache->heads,
              cache->head_dim,
              cache->type};
  a.r = ragged_of(batch, lens);
  a.rows[0] = const_cast<void*>(k);
  a.rows[1] = const_cast<void*>(v);
  a.row_token[0] = k_token;
  a.row_token[1] = v_token;
  a.row_head[0] = k_head;
  a.row_head[1] = v_head;
  a.elem = dtype;
  a.err = device_error_word();
  if (!a.err) return FA_ERR_CUDA;
  const auto launch = append ? launch_cache_append : launch_cache_read;
  return launch(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// One launch of a call: the few-row or the many-row kernel over the sequences of
// min_rows to max_rows query rows (tokens x group).
struct PagedPart {
  bool many, whole;
  int block_rows, min_rows, max_rows;
};

struct PagedPlan {
  int parts;
  PagedPart part[2];
  size_t o_bytes, ml_bytes, total_bytes;
};

// Which kernel a call takes.  The lengths are on the device; what the host knows
// is the mean.  (us, few-row and many-row kernel, 32 / 8 heads of 128, contexts
// up to 16000 keys, 16-bit and e4m3: 64 sequences of 2 tokens, 8 rows, 146 and
// 160, 92 and 184; of 4 tokens, 16 rows, 156 and 162, 142 and 185.  Blocks of 32
// rows in the few-row kernel spilled: 968 us for 8 tokens, 207 in the other.)
//
// Single tokens may come together with a chunk of a prompt.  Where that is likely
// (the sequences cannot be equally long, as total is no multiple of batch, and one of
// them could be) and there are enough single tokens for it to pay, each kernel takes
// its own sequences; a launch that finds none costs 15 us.  (Few rows alone, many rows alone, both: 256
// single tokens and a chunk of 512 over 4000 keys 447, 346 and 298, e4m3 609, 411
// and 227; 256 and 100 252, 283 and 278, e4m3 219, 347 and 205; 64 and 512 218,
// 192 and 195, e4m3 289, 230 and 149; 64 and 64 153, 163 and 185, e4m3 104, 190
// and 135; 8 and 200, e4m3, 45, 24 and 32.)  Unequal sequences whose rows happen to
// divide evenly are not seen, as equal ones (a few drafted tokens each) are the far
// likelier reason: 255 single tokens and a chunk of 513 over 4000 keys each take 741 us
// in e4m3, 256 and 512 464 (16-bit 696 and 691).
constexpr int kFewRows = 16, kMixedMean = 512;
constexpr int mixed_batch(bool fp8) { return fp8 ? 32 : 128; }
constexpr int mixed_longest(bool fp8) { return fp8 ? 384 : 768; }

PagedPlan paged_plan(int batch, int total, int heads, int heads_k, int D, long long max_keys,
                     bool fp8) {
  int sms = 0;
  if (sm_count(&sms) != cudaSuccess) sms = 160;  // no device: sizes for the checks alone
  const int group = heads / heads_k;
  const double mean = static_cast<double>(total) * group / batch;
  // rows of the longest sequence when the others are single tokens
  const long long longest = (static_cast<long long>(total) - batch + 1) * group;
  const bool mixed = total % batch != 0 && batch >= mixed_batch(fp8) && group <= kFewRows &&
                     mean <= kMixedMean && longest > mixed_longest(fp8);
  PagedPlan plan{};
  size_t rows = 0;
  auto add = [&](bool many, int block_rows, int min_rows, int max_rows) {
    const bool whole = max_keys <= (many ? kWholeKeysMany : kWholeKeysFew);
    plan.part[plan.parts++] = PagedPart{many, whole, block_rows, min_rows, max_rows};
    if (!whole) rows = std::max(rows, size_t(2) * sms * block_rows);
  };
  if (mixed || mean <= kFewRows)
    add(false, paged_few_rows(mixed ? group : mean), 0, mixed ? kFewRows : INT_MAX);
  if (mixed || mean > kFewRows)
    add(true, paged_many_rows(group), mixed ? kFewRows + 1 : 0, INT_MAX);
  plan.o_bytes = round256(rows * D * sizeof(float));
  plan.ml_bytes = round256(rows * sizeof(float2));
  plan.total_bytes = rows ? plan.o_bytes + plan.ml_bytes + round256(32ull * sms) : 0;
  return plan;
}

bool paged_sizes_ok(int batch, int total, int heads, int heads_k, int D) {
  return batch >= 1 && total >= 0 && total <= kMaxRows && heads_k >= 1 && heads >= heads_k &&
         heads % heads_k == 0 && heads / heads_k <= 128 && (D == 64 || D == 128) &&
         static_cast<long long>(total) * heads < (1ll << 30);
}

// One cache tensor for the kernels' boxes of min(page_size, 128) rows.
bool page_map(CUtensorMap* m, const void* base, const fa_kv_pages* c, long long page,
              long long token, long long head) {
  const bool fp8 = c->type == FA_ELEM_E4M3;
  // A row is followed by another head's, which another CTA wants: fetching 256
  // bytes for rows of 128 gained 2 % with 8 heads (122 and 120 us for 64 contexts
  // of 256 to 16000 keys, e4m3, D = 128) and lost 10 % with 3 (61 and 67).
  const int row = c->head_dim * (fp8 ? 1 : 2);
  const CUtensorMapL2promotion promotion = row >= 256   ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B
                                           : row >= 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B
                                                        : CU_TENSOR_MAP_L2_PROMOTION_L2_64B;
  const uint32_t rows = static_cast<uint32_t>(c->page_size < kTile ? c->page_size : kTile);
  return make_tmap_4d(
      m, base,
      fp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8
          : c->type == FA_ELEM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                    : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
      static_cast<uint64_t>(c->head_dim), static_cast<uint64_t>(c->page_size),
      static_cast<uint64_t>(c->heads), static_cast<uint64_t>(c->pages),
      static_cast<uint64_t>(token), static_cast<uint64_t>(head), static_cast<uint64_t>(page),
      fp8 ? static_cast<uint32_t>(c->head_dim) : 64u, rows,
      fp8 && c->head_dim == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
      fp8 ? 1 : 2, 1, promotion);
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_rotary(const fa_rotary_operand* q, const fa_rotary_operand* k, int B, int N, int D,
                    int rotary_dim, const double* inv_freq, const void* positions,
                    int position_bits, long long position_batch_stride, float magnitude,
                    int interleaved, int inverse, fa_elem dtype, void* stream) {
  if (!q || B < 0 || N < 0 || B > kMaxRows || N > kMaxRows) return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  if (!is16(dtype) && dtype != FA_ELEM_FP32) return FA_ERR_UNSUPPORTED;
  if (rotary_dim < 16 || rotary_dim > D || rotary_dim % 16) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * N > (1ll << 40)) return FA_ERR_INVALID_ARG;
  if (!aligned(inv_freq, 8) || !std::isfinite(magnitude)) return FA_ERR_INVALID_ARG;
  if (positions ? (position_bits != 32 && position_bits != 64) ||
                      !aligned(positions, position_bits / 8) || position_batch_stride < 0
                : position_bits != 0)
    return FA_ERR_INVALID_ARG;
  RotaryLaunch a{};
  const fa_rotary_operand* ops[2] = {q, k};
  for (int i = 0; i < 2; ++i) {
    const fa_rotary_operand* t = ops[i];
    if (!t) continue;
    if (t->heads < 1 || t->heads > 65535) return FA_ERR_INVALID_ARG;
    if (B == 0 || N == 0) continue;
    const long long extent[3] = {B, t->heads, N};
    const long long xs[3] = {t->xs.batch, t->xs.head, t->xs.seq};
    const long long ys[3] = {t->ys.batch, t->ys.head, t->ys.seq};
    const int es = elem_bytes(dtype);
    if (!aligned(t->x, 16) || !aligned(t->y, 16) || !strides_ok(xs, extent, 3, D, es, 16) ||
        !strides_ok(ys, extent, 3, D, es, 16))
      return FA_ERR_INVALID_ARG;
    if (t->x == t->y && (xs[0] != ys[0] || xs[1] != ys[1] || xs[2] != ys[2]))
      return FA_ERR_INVALID_ARG;
    if (!apart(ys, extent, 3, D) || (i == 1 && t->y == a.y[0])) return FA_ERR_INVALID_ARG;
    a.x[i] = t->x;
    a.y[i] = t->y;
    a.xs[i] = RowStrides{t->xs.batch, t->xs.head, t->xs.seq};
    a.ys[i] = RowStrides{t->ys.batch, t->ys.head, t->ys.seq};
    a.heads[i] = t->heads;
  }
  if (B == 0 || N == 0) return FA_OK;
  a.B = B;
  a.N = N;
  a.D = D;
  a.rotary = rotary_dim;
  a.inv_freq = inv_freq;
  a.positions = positions;
  a.position_bits = position_bits;
  a.position_bstride = position_batch_stride;
  a.magnitude = magnitude;
  a.interleaved = interleaved != 0;
  a.inverse = inverse != 0;
  a.elem = dtype;
  return launch_rotary(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_cache_append(const fa_kv_pages* cache, const fa_ragged* batch, const void* k,
                          long long k_token, long long k_head, const void* v, long long v_token,
                          long long v_head, fa_elem dtype, void* stream) {
  const fa_status st = check_batch(batch, true);
  if (st != FA_OK) return st;
  return cache_rows(cache, batch, batch->seqlens, k, k_token, k_head, v, v_token, v_head, dtype,
                    stream, true);
}

fa_status fa_cache_read(const fa_kv_pages* cache, const fa_ragged* batch, const int* starts,
                        void* k, long long k_token, long long k_head, void* v, long long v_token,
                        long long v_head, fa_elem dtype, void* stream) {
  const fa_status st = check_batch(batch, false);
  if (st != FA_OK) return st;
  if (starts && !aligned(starts, 4)) return FA_ERR_INVALID_ARG;
  return cache_rows(cache, batch, starts, k, k_token, k_head, v, v_token, v_head, dtype, stream,
                    false);
}

fa_status fa_fwd_paged_workspace_size(int batch, int total, int heads, int heads_k, int D,
                                      long long max_keys, size_t* bytes) {
  if (!bytes) return FA_ERR_INVALID_ARG;
  *bytes = 0;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  if (!paged_sizes_ok(batch, total, heads, heads_k, D) || max_keys < 0) return FA_ERR_INVALID_ARG;
  for (const bool fp8 : {false, true})  // whatever the cache holds
    *bytes = std::max(
        *bytes, paged_plan(batch, total, heads, heads_k, D, max_keys, fp8).total_bytes);
  return FA_OK;
}

fa_status fa_fwd_paged(const void* q, long long q_token, long long q_head, void* o,
                       long long o_token, long long o_head, float* lse, const fa_kv_pages* cache,
                       const fa_ragged* batch, int heads, const fa_options* options, float scale,
                       int causal, fa_elem dtype, void* workspace, size_t workspace_bytes,
                       void* stream) {
  fa_status st;
  if ((st = check_batch(batch, true)) != FA_OK) return st;
  if ((st = check_pages(cache, batch, dtype)) != FA_OK) return st;
  if (!paged_sizes_ok(batch->batch, batch->total, heads, cache->heads, cache->head_dim) ||
      !std::isfinite(scale))
    return FA_ERR_INVALID_ARG;
  PagedLaunch a{};
  a.win_left = a.win_right = -1;
  if (options) {
    if (options->block_mask) return FA_ERR_UNSUPPORTED;
    if (options->window_left < -1 || options->window_right < -1) return FA_ERR_INVALID_ARG;
    if (options->alibi_slopes && !aligned(options->alibi_slopes, 4)) return FA_ERR_INVALID_ARG;
    a.win_left = options->window_left < kMaxRows ? options->window_left : -1;
    a.win_right = options->window_right < kMaxRows ? options->window_right : -1;
    a.alibi = options->alibi_slopes;
    a.alibi_bstride = options->alibi_per_batch ? heads : 0;
  }
  if (causal) a.win_right = 0;
  if (batch->total == 0) return FA_OK;
  const int D = cache->head_dim;
  if (!packed_ok(q, q_token, q_head, batch->total, heads, D) ||
      !packed_ok(o, o_token, o_head, batch->total, heads, D) || !aligned(lse, 4))
    return FA_ERR_INVALID_ARG;
  const long long extent[2] = {batch->total, heads}, o_st[2] = {o_token, o_head};
  if (o == q || !apart(o_st, extent, 2, D)) return FA_ERR_INVALID_ARG;
  const PagedPlan plan =
      paged_plan(batch->batch, batch->total, heads, cache->heads, D,
                 static_cast<long long>(batch->max_pages) * cache->page_size,
                 cache->type == FA_ELEM_E4M3);
  if (plan.total_bytes &&
      (!aligned(workspace, 256) || workspace_bytes < plan.total_bytes))
    return FA_ERR_INVALID_ARG;
  if (!page_map(&a.map_k, cache->k, cache, cache->k_page, cache->k_token, cache->k_head) ||
      !page_map(&a.map_v, cache->v, cache, cache->v_page, cache->v_token, cache->v_head))
    return FA_ERR_CUDA;
  a.q = q;
  a.q_token = q_token;
  a.q_head = q_head;
  a.o = o;
  a.o_token = o_token;
  a.o_head = o_head;
  a.lse = lse;
  a.k_exp = cache->k_exp;
  a.v_exp = cache->v_exp;
  a.r = ragged_of(batch, batch->seqlens);
  a.heads = heads;
  a.heads_k = cache->heads;
  a.group = heads / cache->heads;
  a.D = D;
  a.pages = cache->pages;
  a.page_size = cache->page_size;
  a.page_log2 = log2_of(cache->page_size);
  a.cache_elem = cache->type;
  a.elem = dtype;
  a.scale_log2 = scale * kLog2e;
  if (plan.total_bytes) {
    auto* base = static_cast<uint8_t*>(workspace);
    a.part_o = reinterpret_cast<float*>(base);
    a.part_ml = reinterpret_cast<float2*>(base + plan.o_bytes);
    a.tasks = reinterpret_cast<JoinTask*>(base + plan.o_bytes + plan.ml_bytes);
  }
  if (sm_count(&a.sms) != cudaSuccess) return FA_ERR_CUDA;
  a.err = device_error_word();
  if (!a.err) return FA_ERR_CUDA;
  // {D, heads, total}: a box is the heads of one key head for a tile's tokens
  if (plan.part[plan.parts - 1].many &&
      !make_tmap_4d(&a.map_q, q,
                    dtype == FA_ELEM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                          : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                    static_cast<uint64_t>(D), static_cast<uint64_t>(heads),
                    static_cast<uint64_t>(batch->total), 1, static_cast<uint64_t>(q_head),
                    static_cast<uint64_t>(q_token), static_cast<uint64_t>(q_token), 64,
                    static_cast<uint32_t>(a.group), CU_TENSOR_MAP_SWIZZLE_128B, 2,
                    static_cast<uint32_t>(kTile / a.group)))
    return FA_ERR_CUDA;
  for (int i = 0; i < plan.parts; ++i) {  // one after the other: they share the workspace
    const PagedPart& part = plan.part[i];
    a.block_rows = part.block_rows;
    a.min_rows = part.min_rows;
    a.max_rows = part.max_rows;
    // (a window bounds what a unit walks as well as the table does)
    const long long unit_keys =
        a.win_left < 0 || a.win_right < 0
            ? kMaxRows
            : static_cast<long long>(a.win_left) + a.win_right + a.block_rows / a.group + kTile;
    a.whole = part.whole || unit_keys <= (part.many ? kWholeKeysMany : kWholeKeysFew);
    const auto launch = part.many ? launch_paged_many : launch_paged_few;
    if (launch(a, static_cast<cudaStream_t>(stream)) != cudaSuccess) return FA_ERR_CUDA;
  }
  return FA_OK;
}

}  // extern "C"
