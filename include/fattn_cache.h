/*
 * fattn_cache.h -- libfattn: rotary positions, a paged key/value cache and
 * exact attention of new tokens over it, on one sm_103a GPU (C ABI).
 *
 * These entry points stand beside those of fattn.h and share its conventions:
 * device pointers the caller owns, no device memory allocated by the library,
 * calls that only enqueue work on `stream`, arguments checked before anything
 * is enqueued (FA_ERR_INVALID_ARG, FA_ERR_UNSUPPORTED), fp32 sums and softmax
 * statistics, bounded waits.  All work goes to the current device, which must
 * be the one the pointers belong to.
 *
 * What the kernels read from device memory (page tables, lengths) cannot be
 * checked by the host.  The kernels clamp it so that no access leaves the
 * caller's arrays, and record it: fa_device_error() of fattn.h then gives
 * FA_ERR_INVALID_ARG.
 */
#ifndef FATTN_CACHE_H
#define FATTN_CACHE_H

#include "fattn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types; the first two have fa_dtype's values. */
typedef enum { FA_ELEM_BF16 = 0, FA_ELEM_FP16 = 1, FA_ELEM_FP32 = 2, FA_ELEM_E4M3 = 3 } fa_elem;

/*
 * One operand of fa_rotary: [batch][seq][head][D] elements at x + b*xs.batch +
 * n*xs.seq + h*xs.head + d, written to y with the strides ys.  y == x (with
 * equal strides) rotates in place; otherwise x and y must not overlap, and the
 * two operands' y never do.
 * Strides are non-negative and keep every 8 elements 16-byte aligned
 * (multiples of 8; of 4 for fp32).
 */
typedef struct {
  const void* x;
  void* y;
  int heads;
  fa_strides xs, ys;
} fa_rotary_operand;

/*
 * Rotary positions.  Pair i of the first `rotary_dim` elements of each head
 * (elements i and i + rotary_dim/2, or 2i and 2i + 1 when interleaved) at
 * position p is turned by the angle a = p * inv_freq[i] and scaled:
 *
 *   y1 = magnitude * (x1 cos a - x2 sin a),   y2 = magnitude * (x1 sin a + x2 cos a)
 *
 * The other elements are copied.  inverse != 0 turns by -a, which is the
 * gradient of the forward (the rotation's transpose).
 *
 *   q, k        operands; k may be NULL.  D is 64 or 128, the same for both;
 *               dtype FA_ELEM_BF16, FP16 or FP32.  Arithmetic in fp32.
 *   rotary_dim  a multiple of 16, at most D.
 *   inv_freq    device fp64 [rotary_dim / 2], radians per position.  The angle
 *               is reduced to a fraction of a turn in 64-bit fixed point, so
 *               far positions lose nothing.
 *   positions   device int32 or int64 (position_bits 32 or 64), position of
 *               (b, n) at positions[b * position_batch_stride + n]; NULL
 *               (position_bits 0): n itself.
 */
fa_status fa_rotary(const fa_rotary_operand* q, const fa_rotary_operand* k, int B, int N, int D,
                    int rotary_dim, const double* inv_freq, const void* positions,
                    int position_bits, long long position_batch_stride, float magnitude,
                    int interleaved, int inverse, fa_elem dtype, void* stream);

/*
 * A paged cache.  Keys and values are [pages][page_size][heads][D] in any
 * strides with D contiguous (element strides page / token / head, multiples of
 * 16 bytes).  page_size is 16, 32, 64, 128 or 256; D is 64 or 128; type is
 * FA_ELEM_BF16, FA_ELEM_FP16 or FA_ELEM_E4M3.
 *
 * An e4m3 cache holds for each (page, head, token) row an exponent byte e in
 * k_exp / v_exp, contiguous [pages][heads][page_size], 16-byte aligned: the
 * row's values are code * 2^(e - 127), 1 <= e <= 254; e = 0 marks a row of zeros,
 * whatever its codes (a cache of zero bytes reads as zeros).
 */
typedef struct {
  void *k, *v;
  unsigned char *k_exp, *v_exp;
  long long k_page, k_token, k_head;
  long long v_page, v_token, v_head;
  int pages, page_size, heads, head_dim;
  int type;
} fa_kv_pages;

/*
 * A batch of sequences packed along their tokens.  Rows cu_seqlens[b] ..
 * cu_seqlens[b + 1] - 1 of a packed [total][heads][D] array belong to sequence
 * b; rows from cu_seqlens[batch] on belong to none and are never written.
 * Key j of sequence b lives in slot j % page_size of page
 * block_table[b * table_stride + j / page_size].  seqlens[b] is the length of
 * sequence b in the cache, its rows of the packed array (the newest tokens)
 * included.  All int32 on the device.  A sequence may have no rows, or a
 * length of zero.
 *
 * batch, max_pages and the cache's pages are at least 1, total at most 2^29, and so
 * is max_pages * page_size.
 */
typedef struct {
  const int* block_table;
  long long table_stride;
  int max_pages;
  const int* cu_seqlens;
  const int* seqlens;
  int batch, total;
} fa_ragged;

/*
 * Writes the packed rows k, v ([total][heads][D], bf16 or fp16, element
 * strides token / head) into the cache: row i of sequence b becomes key
 * seqlens[b] - rows(b) + i.  A 16-bit cache has the rows' type and gets a
 * copy.  An e4m3 cache gets each (token, head) row at its own scale, the
 * smallest power of two 2^(e - 127), 1 <= e <= 254, with which the row's
 * largest finite magnitude is at most 448; values are rounded to nearest even,
 * infinities become +-448 * 2^(e - 127), NaN stays NaN.
 * The cache's strides are at least D where there is more than one of a kind, and
 * k and v (and their exponents) do not overlap.  Rows whose position is negative
 * or beyond the table, or whose page is not in 0 .. pages - 1, are not written.  The slots that one call writes must be
 * distinct; a slot that two rows share holds either one's bytes.
 */
fa_status fa_cache_append(const fa_kv_pages* cache, const fa_ragged* batch, const void* k,
                          long long k_token, long long k_head, const void* v, long long v_token,
                          long long v_head, fa_elem dtype, void* stream);

/*
 * Reads cached rows back: packed row i of sequence b gets key starts[b] + i
 * (starts NULL: key i), as k and v in `dtype` (bf16 or fp16; a 16-bit cache's
 * own type).  Rows outside the table, or of a page outside 0 .. pages - 1, read
 * as zeros.  batch->seqlens is not used.  k and v do not overlap, and their
 * strides are at least D where there is more than one of a kind.
 */
fa_status fa_cache_read(const fa_kv_pages* cache, const fa_ragged* batch, const int* starts,
                        void* k, long long k_token, long long k_head, void* v, long long v_token,
                        long long v_head, fa_elem dtype, void* stream);

/*
 * Workspace bytes that fa_fwd_paged needs for these sizes, max_keys being
 * max_pages * page_size of its batch and cache.  Zero where it needs none
 * (short tables: no sequence's work is divided); otherwise room for the partial
 * results that are joined at the end.
 */
fa_status fa_fwd_paged_workspace_size(int batch, int total, int heads, int heads_k, int D,
                                      long long max_keys, size_t* bytes);

/*
 * Exact attention of packed new tokens over the paged cache (which already
 * holds their keys and values):
 *
 *   o[r,h,:] = sum_j P_rj V[j,h/G,:],   P = softmax_j(scale * q[r,h] . K[j,h/G] - slope_h |p - j|)
 *   lse[h,r] = the natural log of the softmax's sum
 *
 * for row r of sequence b at position p = seqlens[b] - rows(b) + (r -
 * cu_seqlens[b]), over the keys j < seqlens[b] inside p - window_left ..
 * p + window_right (options; -1: no bound), with causal != 0 also j <= p.
 * G = heads / cache->heads query heads, 128 at most, share a key head; total *
 * heads is below 2^30.  A row that sees no key gets o = 0 and lse = -inf.
 *
 *   q, o     [total][heads][D] in `dtype` (bf16 or fp16; a 16-bit cache's own
 *            type), element strides token / head, multiples of 8, 16-byte
 *            aligned.
 *            o does not overlap q, and its strides are at least D where there
 *            is more than one of a kind.
 *   lse      fp32 [heads][total].
 *   options  NULL, or window and ALiBi as for fa_fwd_ex (slopes [heads] or
 *            [batch][heads]); block_mask must be NULL.
 *   workspace  fa_fwd_paged_workspace_size bytes, 256-byte aligned (NULL when
 *            that is zero).  Calls that may overlap on the GPU need one each.
 *
 * Keys and values beyond a sequence's length, and pages that no visible key
 * lies in, are not looked at, whatever they hold.  Inside the span of keys that
 * some query of a row block sees, a NaN or infinity in a value reaches every
 * query of that block that sees any key (its weight 0 times NaN is NaN), as in
 * the dense product.
 * Deterministic: the same inputs give bit-identical outputs.
 *
 * Weights are rounded to q's type before they multiply the values (fp16 ones keep
 * 11 bits down to 2^-20 of the largest), over an e4m3 cache to fp16; all sums are
 * fp32.
 *
 * Under an e4m3 cache the products run on fp16 numbers under powers of two, a row
 * of q under its own.  What that costs goes by the kernel that a sequence takes.
 * With e a row's exponent byte and R the largest among those (of keys, of values)
 * that a row block has walked:
 *   - up to 16 rows (tokens x G; the mean over the batch, or the sequence's own
 *     where single tokens come beside a chunk of a prompt): keys lose nothing; a
 *     weight times 2^(e - R) is rounded to 11 bits down to 2^-29, and off by 2^-40
 *     at most below.
 *   - more rows: keys and values with e >= R - 22 lose nothing, those with e > R -
 *     32 are off by 2^-32 * 2^(R - 127) at most, others count as zeros; weights are
 *     rounded to 11 bits down to 2^-18 of the largest, and off by 2^-29 of it at
 *     most below.
 */
fa_status fa_fwd_paged(const void* q, long long q_token, long long q_head, void* o,
                       long long o_token, long long o_head, float* lse, const fa_kv_pages* cache,
                       const fa_ragged* batch, int heads, const fa_options* options, float scale,
                       int causal, fa_elem dtype, void* workspace, size_t workspace_bytes,
                       void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FATTN_CACHE_H */
