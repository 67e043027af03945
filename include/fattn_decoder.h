/*
 * fattn_decoder.h -- libfattn: what stands around attention in a decoder's step,
 * on one sm_103a GPU (C ABI): rotary positions along several axes, norms of queries
 * and keys with the rotation in the same pass, the tables of a paged cache built on
 * the GPU, writing by slots, and attention over prefixes that sequences share.
 *
 * These entry points stand beside those of fattn_cache.h, whose types and
 * conventions they share: device pointers the caller owns, no device memory
 * allocated by the library, calls that only enqueue work on `stream`, arguments
 * checked before anything is enqueued.  What the kernels read from device memory
 * (tables, lengths, slots) is clamped so that no access leaves the caller's arrays,
 * and recorded: fa_device_error() then gives FA_ERR_INVALID_ARG.
 */
#ifndef FATTN_DECODER_H
#define FATTN_DECODER_H

#include "fattn_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Positions of (b, n) along one axis or several (text: one; images: row and column;
 * video: time, row, column): positions[axis * axis_stride + b * batch_stride + n],
 * device int32 or int64 (bits 32 or 64).  axis_of_pair, on the host, names the axis
 * (0 .. axes - 1) of each of the rotary_dim / 2 pairs; it is read by the call.  axes
 * is 1 to 8; with one axis axis_of_pair is not looked at, and positions may be NULL
 * (bits 0): n itself.  Strides are not negative.
 */
typedef struct {
  const void* positions;
  int bits;
  int axes;
  long long axis_stride, batch_stride;
  const unsigned char* axis_of_pair;
} fa_positions;

/* fa_rotary with pair i turned by positions[axis_of_pair[i]] * inv_freq[i]. */
fa_status fa_rotary_axes(const fa_rotary_operand* q, const fa_rotary_operand* k, int B, int N,
                         int D, int rotary_dim, const double* inv_freq,
                         const fa_positions* positions, float magnitude, int interleaved,
                         int inverse, fa_elem dtype, void* stream);

/*
 * Each head's row normed, weighted and turned:
 *
 *   y = rotate(x * w / sqrt(mean(x^2) + eps))
 *
 * with the mean over the head's D elements and the rotation (magnitude included) of
 * fa_rotary_axes; elements beyond rotary_dim are normed alone.
 *
 *   q_weight, k_weight  [D], of weight_dtype (dtype, or FA_ELEM_FP32), or NULL for
 *                       ones; k_weight belongs to k.  8-byte aligned at least.
 *   eps                 not negative, finite.
 *
 * Squares are summed in fp32: a row of magnitudes beyond 2^60 may come out as zeros, and
 * one below 2^-60 loses bits where eps is as small.  With eps = 0 a row of zeros gives NaN.
 * The other arguments as for fa_rotary_axes.
 */
fa_status fa_qk_norm_rotary(const fa_rotary_operand* q, const fa_rotary_operand* k,
                            const void* q_weight, const void* k_weight, fa_elem weight_dtype,
                            float eps, int B, int N, int D, int rotary_dim,
                            const double* inv_freq, const fa_positions* positions,
                            float magnitude, int interleaved, fa_elem dtype, void* stream);

/* Workspace bytes of fa_qk_norm_rotary_bwd for head dimension D on the current device. */
fa_status fa_qk_norm_rotary_bwd_workspace_size(int D, size_t* bytes);

/*
 * Its gradients.  q and k are operands x -> dx (x the forward's input, not
 * overlapping dx); dq_out and dk_out the gradients of the forward's results, [batch][seq][head][D]
 * with the strides dq_strides / dk_strides (multiples of 8, of 4 for fp32, 16-byte
 * aligned; a stride may be zero).  dq_weight, dk_weight: [D] of weight_dtype, or NULL
 * where they are not wanted; sums are fp32 in a fixed order, so that the same call
 * gives the same bits.
 *
 *   workspace  fa_qk_norm_rotary_bwd_workspace_size bytes, 256-byte aligned.  Calls
 *              that may overlap on the GPU need one each.
 */
fa_status fa_qk_norm_rotary_bwd(const fa_rotary_operand* q, const fa_rotary_operand* k,
                                const void* dq_out, fa_strides dq_strides, const void* dk_out,
                                fa_strides dk_strides, const void* q_weight,
                                const void* k_weight, void* dq_weight, void* dk_weight,
                                fa_elem weight_dtype, float eps, int B, int N, int D,
                                int rotary_dim, const double* inv_freq,
                                const fa_positions* positions, float magnitude, int interleaved,
                                fa_elem dtype, void* workspace, size_t workspace_bytes,
                                void* stream);

/*
 * The tables of one step, built on the GPU from the sequences' lengths: sequence b,
 * seqlens[b] keys long, brings new_tokens[b] more, and gets the pages that it lacks
 * for them from a stack of free ones.
 *
 *   new_tokens, seqlens  int32 [batch].
 *   block_table   int32 [batch][table_stride], max_pages columns.  Entry j of row b
 *                 names the page of keys j * page_size and on; entries of pages that
 *                 the sequence holds (ceil(seqlens / page_size)) are read, those of its
 *                 new pages written, the others left alone.
 *   free_pages    int32 [capacity], of which the first *free_count are free.  Pages are
 *                 taken from the end, in the order of the sequences and of their keys.
 *   page_size     16, 32, 64, 128 or 256.
 *   total         rows of positions and slots.
 *
 * Results (device):
 *   cu_seqlens    int32 [batch + 1]: 0 and the running sum of new_tokens.
 *   seqlens_out   int32 [batch]: seqlens + new_tokens.  May be seqlens.
 *   positions     int32 [total]: of packed row i, its position in its sequence.
 *   slots         int64 [total]: page * page_size + position % page_size, where its key
 *                 goes.  Rows behind the last sequence get position 0 and slot -1.  A page
 *                 below zero where a new key goes, in the table or among the free ones, is
 *                 recorded as a device error, and its rows get slot -1 too.
 *   free_count_out  int32 [1]: *free_count less the pages taken.  May be free_count.
 *   missing       int32 [1]: 0; or, when free pages do not suffice, how many more it
 *                 takes; or -1 when an argument on the device is bad: a negative length,
 *                 one beyond the table, more new tokens than `total`, a free_count outside
 *                 0 .. capacity (recorded as a device error).  Unless it is 0 nothing is
 *                 taken: the table, seqlens and free_count stay, cu_seqlens is all zeros,
 *                 and every row is one behind the last sequence, so that the calls that
 *                 follow in the same step find nothing to do.
 *
 * batch is 1 to 2^20, total 0 to 2^29, max_pages * page_size at most 2^29.  Outputs do
 * not overlap one another or the inputs but as said.
 */
typedef struct {
  const int* new_tokens;
  const int* seqlens;
  int* block_table;
  long long table_stride;
  int max_pages;
  const int* free_pages;
  int capacity;
  const int* free_count;
  int batch, page_size, total;
  int* cu_seqlens;
  int* seqlens_out;
  int* positions;
  long long* slots;
  int* free_count_out;
  int* missing;
} fa_reserve;

fa_status fa_cache_reserve(const fa_reserve* r, void* stream);

/*
 * Gives pages back: those of every sequence b with done[b] != 0 (bytes, [batch]) but
 * its first keep_pages[b] (int32 [batch], NULL: none kept; shared ones, say) go to
 * the end of free_pages, in the order of the sequences and of their keys; *free_count
 * grows by their number, and seqlens[b] becomes 0.  A length outside the table, a
 * negative keep_pages, or more pages than free_pages has room for is recorded as a
 * device error, and then nothing changes.  The table's entries stay as they are.
 */
fa_status fa_cache_release(const unsigned char* done, int* seqlens, const int* keep_pages,
                           const int* block_table, long long table_stride, int max_pages,
                           int* free_pages, int capacity, int* free_count, int batch,
                           int page_size, void* stream);

/*
 * fa_cache_append by slots: packed row i of k and v ([total][heads][D]) becomes the
 * key of slot slots[i] (int64 [total], page * page_size + place in the page).  Rows of
 * negative slots are not written, nor those beyond the cache, which are recorded.
 */
fa_status fa_cache_write(const fa_kv_pages* cache, const long long* slots, int total,
                         const void* k, long long k_token, long long k_head, const void* v,
                         long long v_token, long long v_head, fa_elem dtype, void* stream);

/*
 * fa_fwd_paged for sequences in groups that share their first pages: the results are
 * those of fa_fwd_paged, causal, without window and biases, with the shared keys
 * walked once for all rows of a group instead of once for each sequence.
 *
 *   cu_groups     int32 [groups + 1], ascending: group g is the sequences cu_groups[g] ..
 *                 cu_groups[g + 1] - 1.  Sequences in no group share nothing.
 *   shared_pages  int32 [groups]: how many first entries the rows of block_table of group
 *                 g's sequences have in common.  No more are taken than lie before every
 *                 new token of the group.  That the rows agree is the caller's word: the
 *                 group's first sequence with rows has its entries read.
 *   groups        0 to batch.
 *   workspace     fa_fwd_paged_shared_workspace_size bytes, 256-byte aligned.
 *
 * Which way is taken goes by the sizes that the host knows (for the prefix the width of the
 * table, and every sequence is taken to be in a group): where sharing would cost more than it
 * saves, each sequence walks all of its keys.  A call most of whose sequences are in no group,
 * or whose table is far wider than its prefixes, may be better off without groups.
 * The other arguments as for fa_fwd_paged.  The parts are joined in fp32 before the one
 * rounding of the result.  Deterministic.  Under an e4m3 cache what the products keep
 * goes by the kernel that the shared and the own part take, as stated there.
 */
fa_status fa_fwd_paged_shared_workspace_size(int batch, int total, int heads, int heads_k, int D,
                                             long long max_keys, int groups, size_t* bytes);

fa_status fa_fwd_paged_shared(const void* q, long long q_token, long long q_head, void* o,
                              long long o_token, long long o_head, float* lse,
                              const fa_kv_pages* cache, const fa_ragged* batch,
                              const int* cu_groups, const int* shared_pages, int groups,
                              int heads, float scale, fa_elem dtype, void* workspace,
                              size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FATTN_DECODER_H */
