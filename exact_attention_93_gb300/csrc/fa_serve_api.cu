// fa_serve_api.cu -- the C ABI of include/fattn_cache.h, and attention over shared
// prefixes of include/fattn_decoder.h: argument checks, TMA descriptor set-up,
// workspace layout and kernel launches.  No arithmetic of the operators lives here.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstdint>

#include "fa_checks.h"
#include "fa_internal.h"
#include "fa_serve.h"
#include "fattn_decoder.h"
#include "host_tmap.hpp"

namespace fa {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
// Keys up to which units stay whole.  (us, cut and whole: one sequence of 1000
// keys 9.9 and 9.6, of 1500 10.8 and 11.9, 8 of 1000 13.7 and 10.4; prompts of
// 4 x 300 tokens 28.2 and 16.9, of 1500 tokens 39.4 and 31.9.)  The keys alone decide,
// and with fewer units than SMs whole units leave some without work: 9 chunks of 1 to
// 500 tokens under a window of 1000, 72 units, take 35 us; cut, they were not measured.
constexpr int kWholeKeysFew = 1536, kWholeKeysMany = 1536;

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

PagedPlan plan_of(const PagedLaunch& a, const Ragged& r) {
  return paged_plan(r.batch, r.total, a.heads, a.heads_k, a.D,
                    static_cast<long long>(r.max_pages) * a.page_size, a.cache_elem == kElemE4m3);
}

bool plan_many(const PagedPlan& plan) { return plan.part[plan.parts - 1].many; }

// Checks the arguments of attention over pages, and fills all of the kernels' but what
// comes from the device and the workspace.
fa_status paged_arguments(PagedLaunch& a, const void* q, long long q_token, long long q_head,
                          void* o, long long o_token, long long o_head, float* lse,
                          const fa_kv_pages* cache, const fa_ragged* batch, int heads,
                          const fa_options* options, float scale, int causal, fa_elem dtype) {
  fa_status st;
  if ((st = check_batch(batch, true)) != FA_OK) return st;
  if ((st = check_pages(cache, batch, dtype)) != FA_OK) return st;
  if (!paged_sizes_ok(batch->batch, batch->total, heads, cache->heads, cache->head_dim) ||
      !std::isfinite(scale))
    return FA_ERR_INVALID_ARG;
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
  return FA_OK;
}

// What comes from the device and its driver; many: queries go by tensor map.
bool paged_device(PagedLaunch& a, const fa_kv_pages* cache, bool many) {
  if (sm_count(&a.sms) != cudaSuccess || !(a.err = device_error_word())) return false;
  if (!page_map(&a.map_k, cache->k, cache, cache->k_page, cache->k_token, cache->k_head) ||
      !page_map(&a.map_v, cache->v, cache, cache->v_page, cache->v_token, cache->v_head))
    return false;
  // {D, heads, total}: a box is the heads of one key head for a tile's tokens
  return !many ||
         make_tmap_4d(&a.map_q, a.q,
                      a.elem == kElemBf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                          : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                      static_cast<uint64_t>(a.D), static_cast<uint64_t>(a.heads),
                      static_cast<uint64_t>(a.r.total), 1, static_cast<uint64_t>(a.q_head),
                      static_cast<uint64_t>(a.q_token), static_cast<uint64_t>(a.q_token), 64,
                      static_cast<uint32_t>(a.group), CU_TENSOR_MAP_SWIZZLE_128B, 2,
                      static_cast<uint32_t>(kTile / a.group));
}

// All rows of all units are at most this share of what the CTAs' tasks could hold.
constexpr int kFewJoins = 4;

fa_status paged_launch(PagedLaunch a, const PagedPlan& plan, void* workspace, cudaStream_t s) {
  if (plan.total_bytes) {
    auto* base = static_cast<uint8_t*>(workspace);
    a.part_o = reinterpret_cast<float*>(base);
    a.part_ml = reinterpret_cast<float2*>(base + plan.o_bytes);
    a.tasks = reinterpret_cast<JoinTask*>(base + plan.o_bytes + plan.ml_bytes);
  }
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
    // rows of the units that can be cut, one per CTA at most, for sequences of the mean length
    const double rows = static_cast<double>(a.r.total) * a.group;
    a.few_joins = rows * a.heads_k * kFewJoins <= static_cast<double>(a.sms) * a.block_rows;
    a.whole = part.whole || unit_keys <= (part.many ? kWholeKeysMany : kWholeKeysFew);
    const auto launch = part.many ? launch_paged_many : launch_paged_few;
    if (launch(a, s) != cudaSuccess) return FA_ERR_CUDA;
  }
  return FA_OK;
}

// Whether walking the shared keys once per group is worth two parts and their joining.
// Sequences that share pages find one another's in L2, so that the whole cost of not
// sharing is the key tiles that each walks again; but where the groups' keys together do
// not stay in L2, HBM's reads are.  The lengths are on the device: the table's width
// stands for the prefix, and a table far wider than that leads to sharing, as asked for.  So
// are the groups' ends: every sequence is taken to be in one.  (Two of 512 sequences of 8
// tokens over 2048 keys, 1024 of them shared, not shared 715 us, shared 778; 8 of 64 single
// tokens over 4096 keys, all shared, 147 and 164.)
//
// The model, in us: without sharing kOwnTile for each of a CTA's tiles; with it kSetOut for
// the kernels before the own part (which costs the same either way) and kSharedTile for
// each tile of up to 256 rows.  Measured, not shared and shared, 32 / 8 heads of 128, 200
// keys of their own: 64 single tokens, prefix of 1024 keys 36 and 47, 4096 69 and 61, 16384
// 218 and 72 (e4m3 38 and 53, 86 and 61, 272 and 76); 16 single tokens, 4096 24 and 41, 16384
// 66 and 55; 8 groups of 8, 1024 37 and 48, 4096 121 and 70; 32 groups of 2, 4096 172 and
// 114; 64 x 8 tokens, 4096 187 and 102, x 16 186 and 131, x 32 189 and 184; 16 x 16 tokens,
// 4096 66 and 73.  12 / 4 heads of 64, 24 x 4 tokens, 6000 keys 31 and 41.
struct SharedCost {
  double own_tile, shared_tile, set_out;
};

SharedCost shared_cost(double rows, double group_rows, int D, bool fp8) {
  SharedCost c{};
  const double small = D == 64 ? 0.7 : 1.0;
  c.own_tile = small * (rows <= 8         ? (fp8 ? 0.58 : 0.46)
                        : rows <= kFewRows ? (fp8 ? 0.92 : 0.7)
                                           : (fp8 ? 1.7 : 1.43));
  if (group_rows <= kFewRows) {
    c.shared_tile = small * (fp8 ? 0.92 : 0.7);
    c.set_out = 12;
  } else {
    c.shared_tile = small * (fp8 ? 3.4 : 2.8);
    c.set_out = 30;
  }
  if (rows > kFewRows) c.set_out += 12;  // the own part does not join them itself
  return c;
}

constexpr double kSharedRows = 64;  // rows (tokens x group) of a sequence
constexpr double kCopyBytesPerUs = 6.7e6, kStaysInL2 = 64e6;

bool sharing_pays(int batch, int total, int heads, int heads_k, int D, long long max_keys,
                  int groups, bool fp8) {
  const int group = heads / heads_k;
  const double rows = static_cast<double>(total) * group / batch;
  if (groups < 1 || groups >= batch || rows > kSharedRows) return false;
  int sms = 0;
  if (sm_count(&sms) != cudaSuccess) sms = 160;  // no device: sizes for the checks alone
  const double group_rows = rows * batch / groups;
  const SharedCost c = shared_cost(rows, group_rows, D, fp8);
  const double tiles = std::ceil(static_cast<double>(max_keys) / kTile) * heads_k / sms;
  const double key_bytes = static_cast<double>(max_keys) * heads_k * D * (fp8 ? 2 : 4);
  const double hbm = groups * key_bytes > kStaysInL2 ? key_bytes / kCopyBytesPerUs : 0;
  const double blocks = group_rows <= kFewRows ? 1 : std::ceil(group_rows / (2 * kTile));
  return std::max(c.own_tile * tiles, hbm) * batch >
         c.set_out + std::max(c.shared_tile * tiles * blocks, hbm) * groups;
}

// Behind a shared prefix most sequences have few keys of their own, so what a unit costs
// beside its tiles counts in sharing out the work.  (us, a whole call, in tiles 0, 1, 2, 3 and
// 5: 64 sequences of 16 to 2000 own keys 87, 86, 83, 84 and 83; 128 of 1 to 1500, e4m3, 100,
// 97, 94, 93 and 93.)
constexpr int kOwnUnitCost = 3;

// The workspace of attention over shared prefixes, in front of the kernels' own.
struct SharedLayout {
  size_t o1, o2, ml1, ml2, cu, lens, rows, skip, bytes;
};

SharedLayout shared_layout(int batch, int total, int heads, int D, int groups) {
  const size_t rows = static_cast<size_t>(total) * heads;
  SharedLayout at{};
  size_t end = 0;
  const auto take = [&](size_t bytes) {
    const size_t begin = end;
    end += round256(bytes);
    return begin;
  };
  at.o1 = take(sizeof(float) * rows * D);
  at.o2 = take(sizeof(float) * rows * D);
  at.ml1 = take(sizeof(float2) * rows);
  at.ml2 = take(sizeof(float2) * rows);
  at.cu = take(sizeof(int) * (groups + 1));
  at.lens = take(sizeof(int) * groups);
  at.rows = take(sizeof(int) * groups);
  at.skip = take(sizeof(int) * batch);
  at.bytes = end;
  return at;
}

}  // namespace
}  // namespace fa

using namespace fa;

extern "C" {

fa_status fa_rotary(const fa_rotary_operand* q, const fa_rotary_operand* k, int B, int N, int D,
                    int rotary_dim, const double* inv_freq, const void* positions,
                    int position_bits, long long position_batch_stride, float magnitude,
                    int interleaved, int inverse, fa_elem dtype, void* stream) {
  RotaryLaunch a{};
  bool done;
  const fa_positions pos{positions, position_bits, 1, 0, position_batch_stride, nullptr};
  const fa_status st =
      rotary_arguments(a, q, k, B, N, D, rotary_dim, inv_freq, pos, magnitude, dtype, done);
  if (st != FA_OK || done) return st;
  a.interleaved = interleaved != 0;
  a.inverse = inverse != 0;
  return launch_rotary(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status fa_cache_append(const fa_kv_pages* cache, const fa_ragged* batch, const void* k,
                          long long k_token, long long k_head, const void* v, long long v_token,
                          long long v_head, fa_elem dtype, void* stream) {
  const fa_status st = check_batch(batch, true);
  if (st != FA_OK) return st;
  return cache_rows(cache, batch, batch->seqlens, nullptr, k, k_token, k_head, v, v_token, v_head, dtype,
                    stream, true);
}

fa_status fa_cache_read(const fa_kv_pages* cache, const fa_ragged* batch, const int* starts,
                        void* k, long long k_token, long long k_head, void* v, long long v_token,
                        long long v_head, fa_elem dtype, void* stream) {
  const fa_status st = check_batch(batch, false);
  if (st != FA_OK) return st;
  if (starts && !aligned(starts, 4)) return FA_ERR_INVALID_ARG;
  return cache_rows(cache, batch, starts, nullptr, k, k_token, k_head, v, v_token, v_head, dtype, stream,
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
  PagedLaunch a{};
  const fa_status st = paged_arguments(a, q, q_token, q_head, o, o_token, o_head, lse, cache, batch,
                                       heads, options, scale, causal, dtype);
  if (st != FA_OK || batch->total == 0) return st;
  const PagedPlan plan = plan_of(a, a.r);
  if (plan.total_bytes && (!aligned(workspace, 256) || workspace_bytes < plan.total_bytes))
    return FA_ERR_INVALID_ARG;
  if (!paged_device(a, cache, plan_many(plan))) return FA_ERR_CUDA;
  return paged_launch(a, plan, workspace, static_cast<cudaStream_t>(stream));
}

fa_status fa_fwd_paged_shared_workspace_size(int batch, int total, int heads, int heads_k, int D,
                                             long long max_keys, int groups, size_t* bytes) {
  const fa_status st =
      fa_fwd_paged_workspace_size(batch, total, heads, heads_k, D, max_keys, bytes);
  if (st != FA_OK) return st;
  if (groups < 0 || groups > batch) return FA_ERR_INVALID_ARG;
  const size_t plain = *bytes;
  for (const bool fp8 : {false, true}) {  // whatever the cache holds
    if (!sharing_pays(batch, total, heads, heads_k, D, max_keys, groups, fp8)) continue;
    const size_t parts = std::max(
        plain, paged_plan(groups, total, heads, heads_k, D, max_keys, fp8).total_bytes);
    *bytes = std::max(*bytes, shared_layout(batch, total, heads, D, groups).bytes + parts);
  }
  return FA_OK;
}

fa_status fa_fwd_paged_shared(const void* q, long long q_token, long long q_head, void* o,
                              long long o_token, long long o_head, float* lse,
                              const fa_kv_pages* cache, const fa_ragged* batch,
                              const int* cu_groups, const int* shared_pages, int groups,
                              int heads, float scale, fa_elem dtype, void* workspace,
                              size_t workspace_bytes, void* stream) {
  PagedLaunch a{};
  fa_status st = paged_arguments(a, q, q_token, q_head, o, o_token, o_head, lse, cache, batch,
                                 heads, nullptr, scale, 1, dtype);
  if (st != FA_OK) return st;
  if (groups < 0 || groups > batch->batch ||
      (groups > 0 && (!aligned(cu_groups, 4) || !aligned(shared_pages, 4))))
    return FA_ERR_INVALID_ARG;
  if (batch->total == 0) return FA_OK;
  if (!sharing_pays(batch->batch, batch->total, heads, a.heads_k, a.D,
                    static_cast<long long>(a.r.max_pages) * a.page_size, groups,
                    a.cache_elem == kElemE4m3))
    return fa_fwd_paged(q, q_token, q_head, o, o_token, o_head, lse, cache, batch, heads, nullptr,
                        scale, 1, dtype, workspace, workspace_bytes, stream);
  const SharedLayout at = shared_layout(batch->batch, batch->total, heads, a.D, groups);
  auto* base = static_cast<uint8_t*>(workspace);
  const auto ints = [&](size_t offset) { return reinterpret_cast<int*>(base + offset); };
  const auto floats = [&](size_t offset) { return reinterpret_cast<float*>(base + offset); };
  const auto stats = [&](size_t offset) { return reinterpret_cast<float2*>(base + offset); };
  // the groups as sequences: all of their rows see all of the shared keys
  PagedLaunch first = a;
  first.r = Ragged{a.r.table, a.r.table_stride, a.r.max_pages, ints(at.cu), ints(at.lens),
                   groups,    a.r.total,        nullptr,       ints(at.rows)};
  first.win_right = -1;
  first.parts = a.parts = 1;
  a.r.skip = ints(at.skip);
  const PagedPlan plan1 = plan_of(first, first.r), plan2 = plan_of(a, a.r);
  if (!aligned(workspace, 256) ||
      workspace_bytes < at.bytes + std::max(plan1.total_bytes, plan2.total_bytes))
    return FA_ERR_INVALID_ARG;
  if (!paged_device(a, cache, plan_many(plan1) || plan_many(plan2))) return FA_ERR_CUDA;
  first.sms = a.sms;
  first.err = a.err;
  first.map_k = a.map_k;
  first.map_v = a.map_v;
  first.map_q = a.map_q;
  const auto s = static_cast<cudaStream_t>(stream);
  Ragged whole = a.r;
  whole.skip = nullptr;
  if (launch_shared_setup(
          SharedSetup{whole, cu_groups, shared_pages, groups, a.page_log2, ints(at.cu),
                      ints(at.lens), ints(at.rows), ints(at.skip), a.err},
          s) != cudaSuccess)
    return FA_ERR_CUDA;
  first.o32 = floats(at.o1);
  first.ml32 = stats(at.ml1);
  // one after the other: they share the workspace
  if ((st = paged_launch(first, plan1, base + at.bytes, s)) != FA_OK) return st;
  if (!plan_many(plan2)) {  // few rows: the own part's kernels join the two
    a.add_o = first.o32;
    a.add_ml = first.ml32;
    a.add_first = ints(at.cu);
    a.add_end = ints(at.cu) + groups;
    a.unit_cost = kOwnUnitCost;
    return paged_launch(a, plan2, base + at.bytes, s);
  }
  a.o32 = floats(at.o2);
  a.ml32 = stats(at.ml2);
  if ((st = paged_launch(a, plan2, base + at.bytes, s)) != FA_OK) return st;
  const SharedJoin join{first.o32,   a.o32,     first.ml32, a.ml32,  ints(at.cu), ints(at.cu) + groups,
                        a.r.cu,      a.r.batch, a.r.total, a.heads, a.D,         a.elem,
                        o,           o_token,   o_head,    lse};
  return launch_shared_join(join, s) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // extern "C"
