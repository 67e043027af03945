// fa_checks.h -- argument checks that the entry points of include/fattn_cache.h and
// include/fattn_decoder.h share.  Host-side only.
#pragma once

#include <climits>
#include <cmath>
#include <cstdint>

#include "fa_internal.h"
#include "fa_serve.h"
#include "fattn_decoder.h"

namespace fa {

constexpr long long kMaxBytes = 1ll << 40;  // every operand lies below this from its base
constexpr int kMaxRows = 1 << 29;           // packed rows, keys of a sequence, window bounds

inline bool aligned(const void* p, uintptr_t n) { return p && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline size_t round256(size_t x) { return (x + 255) & ~size_t(255); }

inline int elem_bytes(int elem) { return elem == FA_ELEM_FP32 ? 4 : elem == FA_ELEM_E4M3 ? 1 : 2; }

inline bool is16(int elem) { return elem == FA_ELEM_BF16 || elem == FA_ELEM_FP16; }

// Strides of one operand: non-negative, `unit`-byte multiples, and the last
// element below kMaxBytes.
inline bool strides_ok(const long long* st, const long long* extent, int n, int D, int es, int unit) {
  double last = D;
  for (int i = 0; i < n; ++i) {
    if (st[i] < 0 || (st[i] * es) % unit != 0 || st[i] > kMaxBytes) return false;
    last += static_cast<double>(extent[i] - 1) * st[i];
  }
  return last * es < static_cast<double>(kMaxBytes);
}

// An operand that is written: every index has elements of its own (strides below
// a row would let rows share them).
inline bool apart(const long long* st, const long long* extent, int n, int D) {
  for (int i = 0; i < n; ++i)
    if (extent[i] > 1 && st[i] < D) return false;
  return true;
}

inline fa_status check_batch(const fa_ragged* b, bool lens_needed) {
  if (!b || b->batch < 1 || b->total < 0 || b->total > kMaxRows || b->max_pages < 1)
    return FA_ERR_INVALID_ARG;
  if (!aligned(b->block_table, 4) || !aligned(b->cu_seqlens, 4) || b->table_stride < b->max_pages)
    return FA_ERR_INVALID_ARG;
  if (lens_needed && !aligned(b->seqlens, 4)) return FA_ERR_INVALID_ARG;
  return FA_OK;
}

inline fa_status check_pages(const fa_kv_pages* c, const fa_ragged* b, fa_elem dtype) {
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
inline bool packed_ok(const void* p, long long token, long long head, int total, int heads, int D) {
  const long long extent[2] = {total, heads}, st[2] = {token, head};
  return aligned(p, 16) && strides_ok(st, extent, 2, D, 2, 16);
}

inline int log2_of(int x) {
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

inline Ragged ragged_of(const fa_ragged* b, const int* lens) {
  return Ragged{b->block_table, b->table_stride, b->max_pages, b->cu_seqlens, lens, b->batch,
                b->total};
}

// Fills the arguments of a rotation (but for interleaved and inverse) from those of an
// entry point.  done: there is nothing to turn.
inline fa_status rotary_arguments(RotaryLaunch& a, const fa_rotary_operand* q,
                                  const fa_rotary_operand* k, int B, int N, int D, int rotary_dim,
                                  const double* inv_freq, const fa_positions& pos, float magnitude,
                                  fa_elem dtype, bool& done) {
  done = false;
  if (!q || B < 0 || N < 0 || B > kMaxRows || N > kMaxRows) return FA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return FA_ERR_UNSUPPORTED;
  if (!is16(dtype) && dtype != FA_ELEM_FP32) return FA_ERR_UNSUPPORTED;
  if (rotary_dim < 16 || rotary_dim > D || rotary_dim % 16) return FA_ERR_INVALID_ARG;
  if (static_cast<long long>(B) * N > (1ll << 40)) return FA_ERR_INVALID_ARG;
  if (!aligned(inv_freq, 8) || !std::isfinite(magnitude)) return FA_ERR_INVALID_ARG;
  if (pos.positions ? (pos.bits != 32 && pos.bits != 64) ||
                          !aligned(pos.positions, pos.bits / 8) || pos.batch_stride < 0
                    : pos.bits != 0)
    return FA_ERR_INVALID_ARG;
  if (pos.axes < 1 || pos.axes > 8) return FA_ERR_INVALID_ARG;
  if (pos.axes > 1) {
    // (no tokens: no positions either)
    if ((!pos.positions && B > 0 && N > 0) || !pos.axis_of_pair || pos.axis_stride < 0)
      return FA_ERR_INVALID_ARG;
    for (int i = 0; i < rotary_dim / 2; ++i) {
      if (pos.axis_of_pair[i] >= pos.axes) return FA_ERR_INVALID_ARG;
      a.axis[i] = pos.axis_of_pair[i];
    }
  }
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
  done = B == 0 || N == 0;
  a.B = B;
  a.N = N;
  a.D = D;
  a.rotary = rotary_dim;
  a.inv_freq = inv_freq;
  a.positions = pos.positions;
  a.position_bits = pos.bits;
  a.position_bstride = pos.batch_stride;
  a.position_axes = pos.axes;
  a.position_astride = pos.axis_stride;
  a.magnitude = magnitude;
  a.elem = dtype;
  return FA_OK;
}

// Appends packed rows to the cache (by slots, or, where they are null, by tables and
// lengths), or reads them back.
inline fa_status cache_rows(const fa_kv_pages* cache, const fa_ragged* batch, const int* lens,
                            const long long* slots, const void* k, long long k_token,
                            long long k_head, const void* v, long long v_token, long long v_head,
                            fa_elem dtype, void* stream, bool append) {
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
  a.slots = slots;
  a.err = device_error_word();
  if (!a.err) return FA_ERR_CUDA;
  const auto launch = append ? launch_cache_append : launch_cache_read;
  return launch(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace fa
