// fa_paged_many.cu -- attention over a paged cache for many query rows per
// sequence: chunks of prompts over long contexts, whole packed prompts.
//
// What bounds it.  A unit's 2 x 128 query rows make 4 * 256 * D operations of
// each 4 * D byte key and value: the tensor cores are the bound, and beside
// them the exponentials.  The kernel is the design of the dense forward
// (fa_fwd.cu: two 128-row tiles in turn, S and O in tensor memory, P written
// over S) fed from pages:
//
//   - The rows of a tile are tokens x the G query heads that share a key head
//     (row = token * G + head), so K and V are staged once for all of them.  A
//     tile holds floor(128 / G) tokens; with a G that does not divide 128 its
//     last rows idle.
//   - K and V tiles of 128 keys are gathered by TMA page by page: one lane of
//     the producer warp per page.  Only pages that hold a key some row of the
//     unit sees are touched.
//   - CTAs stay resident and walk a stretch of the units laid end to end
//     (fa_paged.cuh); a unit that a stretch's end cuts leaves its partial O,
//     maximum and sum in fp32 for the joining kernel.
//   - One warp works out the units ahead of the others and hands them over
//     through a ring in shared memory: the arithmetic is long and rarely run,
//     and in every role's path it cost some 4 us a unit, mostly fetching its
//     instructions.
//   - O goes from tensor memory to the caller's rows by plain stores: a packed
//     batch's tiles end anywhere, and a tensor-map store would run into the
//     next sequence.
//
// Values outside the visible span (behind the sequence's end, in pages not
// loaded) may be anything, and 0 * NaN is NaN: a spare warp makes those rows of
// a tile zeros before the P V product reads it.
//
// e4m3 caches: four warps convert each 8-bit tile to fp16 in shared
// memory (exactly, relative to the largest row exponent so far, which scales
// the scores, and O, in fp32), and bf16 queries to fp16 under a power-of-two
// scale per row; both products then run in fp16.
//
// Warps: 0-3 softmax of tile A, 4-7 of tile B, 8 producer, 9 MMA issue, 10 the
// units, 11 zeroing (12 warps), or 12-15 conversion (e4m3 caches, 16 warps).
//
// Measured (D = 128, 32 query and 8 key heads, bf16): a prompt of 8192 tokens
// 381 us, 1442 TFLOP/s, tensor pipe 61 % active (the dense forward over 32 heads
// 415 us); 32768 tokens of 8 heads 1447 us, 1520 TFLOP/s (dense 1381); four
// prompts of 9429 tokens in all 227 us; four chunks of 137 tokens over 20000 keys
// 188 us.  Beside its key tiles a unit costs about 3 us (reading O out, filling
// the pipeline again) and a call about 10.  e4m3: 466 and 208 us for the first
// and the last.  (With other inputs in every call 412 and 197, e4m3 479 and 217.)
// There registers are the limit: 16 warps share what 12 have in the 16-bit kernel,
// and a split with more for the softmax or more for the conversion made both slower
// (200 / 56: 481 us, 184 / 72: 482).  Queries take 25 us of the 466, a unit's rows
// being converted before its first product.  The chunks are at half the tensor rate:
// 4 x 137 rows of a key head are two full blocks and one of 36 rows for each, and
// that one walks every key with one query tile and nothing to alternate with.
#include <type_traits>

#include "fa_paged.cuh"
#include "fa_serve.h"
#include "sm103_primitives.cuh"

namespace fa {
namespace {

// Threads, and registers per thread after the softmax warps have taken the
// others': 12 warps launch with 168 (2 x 208 + 80 <= 3 x 168 on each
// sub-partition), 16 with 128 (2 x 192 + 2 x 64 = 4 x 128).
template <bool kFp8>
struct ManyWarps {
  static constexpr int kThreads = kFp8 ? 512 : 384;
  static constexpr uint32_t kLow = kFp8 ? 64 : 80, kHigh = kFp8 ? 192 : 208;
  static constexpr int kFirst = kFp8 ? 12 : 11;  // zeroing or converting warps
  static constexpr int kConverters = kThreads - 32 * kFirst;  // their threads
};
constexpr int kUnitRing = 4;
// references of key and value exponents, one per key tile: a softmax group is
// never more than three tiles behind the conversion's stages (a tile pair's
// ranges end within two tiles of each other)
constexpr int kRefs = 8;

template <int D, bool kFp8>
struct ManySmem {
  static constexpr int kBlocks = D / 64;               // 64-column blocks of a 16-bit tile
  static constexpr int kBlockBytes = kTile * 128;
  static constexpr int kTileBytes = kBlocks * kBlockBytes;
  // K and V tiles alternate through one ring: tile g's K is number 2 g, its V
  // 2 g + 1
  static constexpr int kStages = kFp8 ? (D == 128 ? 5 : 6) : (D == 128 ? 4 : 8);
  // e4m3, D = 128: a raw tile lands in the upper half of its stage, where each
  // of its rows lies under the upper half of its own converted row
  static constexpr bool kInPlace = D == 128;
  static constexpr int kRawBytes = kTile * D;
  alignas(1024) uint8_t q[2][kTileBytes];
  alignas(1024) uint8_t kv[kStages][kTileBytes];
  alignas(1024) uint8_t raw_tiles[kFp8 && !kInPlace ? kStages : 1][kFp8 && !kInPlace ? kRawBytes : 16];
  alignas(16) uint8_t exps[kFp8 ? kStages : 1][kTile];
  int8_t qshift[2][kFp8 ? 2 * kTile : 1];  // [unit & 1]: rows of q were scaled by 2^this
  int kref[kRefs], vref[kRefs];
  int4 unit[kUnitRing][4];  // ManyUnit
  uint64_t unit_full[kUnitRing], unit_empty[kUnitRing];
  uint64_t q_full, q_empty, q_ready;
  uint64_t full[kStages], empty[kStages];
  // tiles that need work before the tensor cores may read them land here first:
  // e4m3 ones, and V tiles with rows to make zeros
  uint64_t raw_full[kStages];
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t drain;
  __device__ __forceinline__ uint8_t* raw(int st) {
    return kInPlace ? kv[st] + kRawBytes : raw_tiles[kInPlace ? 0 : st];
  }
  uint32_t tmem_base;
  int abort_flag;
  // 16-bit caches: O on its way out, 32 rows x 128 bytes per softmax warp
  alignas(16) uint8_t stage[kFp8 ? 1 : 8][kFp8 ? 16 : 4096];
};

__device__ __forceinline__ bool many_warp_wait(uint64_t* bar, uint32_t parity, uint32_t* err,
                                               volatile int* abort_flag) {
  const bool ok = mbar_wait(bar, parity, err, abort_flag);
  return __all_sync(0xffffffffu, ok);
}

// A piece of work as the roles need it.  Key tiles: of query tile t [lo_t,
// hi_t], none when lo_t > hi_t, and the K/V stream first .. last over their
// union (first > last: nothing to multiply).
struct ManyUnit {
  int lo0, hi0, lo1, hi1;
  int first, last;
  int key_lo, key_hi;  // keys that some row sees
  int start;           // packed row of the block's first token
  int tokens;          // of the block
  int pos;             // position of its first token
  int len;             // keys of the sequence
  int b, hk;
  int slot;            // of the partial result; -1: the piece covers its unit
  int valid;           // 0: no more work

  __device__ __forceinline__ bool two(int tile_tokens) const { return tokens > tile_tokens; }
  __device__ __forceinline__ int count(int t) const {
    return t ? max(0, hi1 - lo1 + 1) : max(0, hi0 - lo0 + 1);
  }
  __device__ __forceinline__ int streamed() const { return max(0, last - first + 1); }
  // key tile j has rows that no query sees
  __device__ __forceinline__ bool ragged(int j) const {
    return j * kTile < key_lo || (j + 1) * kTile > key_hi;
  }
};
static_assert(sizeof(ManyUnit) == 64, "four 16-byte words");

__device__ __forceinline__ void many_range(const PagedLaunch& p, const Piece& x, const Seq& s,
                                           int t0, int t1, int& lo, int& hi) {
  int a, b;
  visible_span(p, s, t0, t1, a, b);
  lo = max(a / kTile, x.tile0);
  hi = min((b + kTile - 1) / kTile, x.tile1) - 1;
  if (t0 >= t1 || lo > hi) {
    lo = 1;
    hi = 0;
  }
}

// The next entry of the ring, for a whole warp.  False on a timeout; valid is
// 0 in the last entry.
template <class Smem>
__device__ __forceinline__ bool take_unit(Smem& s, uint32_t n, ManyUnit& u, uint32_t* err,
                                          volatile int* abort_flag) {
  const int slot = n % kUnitRing;
  const bool ok = __all_sync(
      0xffffffffu, mbar_wait(&s.unit_full[slot], (n / kUnitRing) & 1, err, abort_flag));
  if (!ok) return false;
  int4 w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = s.unit[slot][i];
  u = ManyUnit{w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w,
               w[2].x, w[2].y, w[2].z, w[2].w, w[3].x, w[3].y, w[3].z, w[3].w};
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(&s.unit_empty[slot]);
  return u.valid != 0;
}

// 2^(n - 127) for an exponent field n, 0 below the normal range.
__device__ __forceinline__ float many_exp2_field(int n) {
  return __uint_as_float(static_cast<uint32_t>(min(max(n, 0), 254)) << 23);
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <int D, bool kFp8, bool kBf16, bool kAlibi, bool kParts>
__global__ void __launch_bounds__(ManyWarps<kFp8>::kThreads, 1)
    paged_many_kernel(const __grid_constant__ PagedLaunch p) {
  pdl_wait_and_release();
  using Smem = ManySmem<D, kFp8>;
  constexpr bool kMmaBf16 = kBf16 && !kFp8;  // type of the products
  // P = 2^(x - m + kPOffset [+ up to 3, e4m3]), the reference m lagging the
  // true maximum by at most kThreshold.  bf16 has the range for no offset; fp16
  // P stays below 2^15 (e4m3) or 2^14 and normal down to 2^-18 or 2^-20 of m:
  // without the offset, keys of weight 2^-15 lost most of their bits.
  constexpr float kThreshold = 8.0f;
  constexpr int kPOffset = kMmaBf16 ? 0 : kFp8 ? 4 : 6;
  extern __shared__ uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>(smem_raw + (-smem_u32(smem_raw) & 1023u));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int tile_tokens = p.block_rows / p.group / 2, tile_rows = tile_tokens * p.group;
  constexpr int kConverters = ManyWarps<kFp8>::kConverters, kStages = Smem::kStages;
  if (tid == 0) {
    mbar_init(&s.q_full, 1);
    mbar_init(&s.q_empty, 1);
    mbar_init(&s.q_ready, kConverters / 32);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_full[i], 128);
      mbar_init(&s.o_done[i], 1);
    }
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&s.full[i], kFp8 ? kConverters / 32 : 1);
      mbar_init(&s.empty[i], 1);
      mbar_init(&s.raw_full[i], 1);
    }
    for (int i = 0; i < kUnitRing; ++i) {
      mbar_init(&s.unit_full[i], 1);
      mbar_init(&s.unit_empty[i], 10 + kConverters / 32);  // warps that read it
    }
    mbar_init(&s.drain, 1);
    s.abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 8) {
    tmem_alloc(&s.tmem_base, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = s.tmem_base;
  volatile int* abort_flag = &s.abort_flag;
  ManyUnit u;
  uint32_t taken = 0;  // entries of the unit ring

  if (warp >= 8) {
    setmaxnreg_dec<ManyWarps<kFp8>::kLow>();
    if (warp == 8) {
      // ------------------------------------------------------------ producer
      if (lane == 0) {
        tma_prefetch_desc(&p.map_q);
        tma_prefetch_desc(&p.map_k);
        tma_prefetch_desc(&p.map_v);
      }
      constexpr int kRowBytes = kFp8 ? D : 2 * D;
      const int box_rows = min(p.page_size, kTile), per_tile = kTile / box_rows;
      uint32_t units = 0;   // Q loads
      uint32_t n = 0;       // K and V tiles loaded
      uint32_t cut = 0;     // 16-bit, bit st: parity of the next tile in raw_full[st]
      uint32_t to_raw = 0;  // bit st: stage st's last load was one
      bool stop = false;
      while (!stop && take_unit(s, taken++, u, p.err, abort_flag)) {
        if (u.first > u.last) continue;
        PageFeed feed;
        feed.start<kParts>(p, u.b, u.first, u.key_lo, u.key_hi);
        // Q once the last S product of the unit before has read it
        if (units > 0 && !many_warp_wait(&s.q_empty, (units - 1) & 1, p.err, abort_flag)) break;
        if (lane == 0) {
          const int n_q = u.two(tile_tokens) ? 2 : 1;
          mbar_arrive_expect_tx(&s.q_full, n_q * tile_rows * 2 * D);
          for (int t = 0; t < n_q; ++t)
            for (int kb = 0; kb < Smem::kBlocks; ++kb)
              tma_load_4d(s.q[t] + kb * Smem::kBlockBytes, &p.map_q, &s.q_full, kb * 64,
                          u.hk * p.group, u.start + t * tile_tokens, 0);
        }
        ++units;
        for (int j = u.first; j <= u.last; ++j) {
          const int k0 = j * kTile + lane * box_rows;
          const bool mine = lane < per_tile && k0 < u.key_hi && k0 + box_rows > u.key_lo;
          const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, mine));
          int page = feed.get(p, j, k0);
          if (mine && (page < 0 || page >= p.pages)) {
            atomicExch(p.err, kDevErrBadIndex);
            page = p.pages;  // out of range for the tensor map: reads as zeros
          }
          const int row = k0 & (p.page_size - 1);
#pragma unroll
          for (int kv = 0; kv < 2 && !stop; ++kv) {
            const int st = n % kStages;
            uint64_t* full = kFp8 ? &s.raw_full[st] : &s.full[st];
            if constexpr (!kFp8) {
              to_raw &= ~(1u << st);
              if (kv && u.ragged(j)) {
                full = &s.raw_full[st];
                cut ^= 1u << st;
                to_raw |= 1u << st;
              }
            }
            if (n >= kStages &&
                !many_warp_wait(&s.empty[st], (n / kStages - 1) & 1, p.err, abort_flag)) {
              stop = true;
              break;
            }
            if (lane == 0)
              mbar_arrive_expect_tx(full, boxes * box_rows * (kRowBytes + (kFp8 ? 1 : 0)));
            __syncwarp();
            if (mine) {
              uint8_t* dst = (kFp8 ? s.raw(st) : s.kv[st]) +
                             lane * box_rows * (kRowBytes < 128 ? kRowBytes : 128);
#pragma unroll
              for (int kb = 0; kb < (kRowBytes + 127) / 128; ++kb)
                tma_load_4d(dst + kb * Smem::kBlockBytes, kv ? &p.map_v : &p.map_k, full, kb * 64,
                            row, u.hk, page);
              if constexpr (kFp8) {
                const uint8_t* e = (kv ? p.v_exp : p.k_exp) +
                                   (static_cast<long long>(page < p.pages ? page : 0) * p.heads_k +
                                    u.hk) * p.page_size + row;
                bulk_load(s.exps[st] + lane * box_rows, e, box_rows, full);
              }
            }
            ++n;
          }
          if (stop) break;
        }
      }
      if (*abort_flag && lane == 0) {
        // Copies already in flight land before the CTA's shared memory goes away.
        int zero = 0;
        if (units > 0) mbar_wait(&s.q_full, (units - 1) & 1, p.err, &zero, 100000000ull);
        for (uint32_t i = n > kStages ? n - kStages : 0; i < n; ++i) {
          const int st = i % kStages;
          const bool cut_tile = !kFp8 && ((to_raw >> st) & 1);
          mbar_wait(kFp8 || cut_tile ? &s.raw_full[st] : &s.full[st],
                    cut_tile ? ((cut >> st) & 1) ^ 1 : (i / kStages) & 1, p.err, &zero,
                    100000000ull);
        }
      }
      __syncwarp();
    } else if (warp == 9) {
      // ---------------------------------------------------------- MMA issuer
      // Every lane computes the same descriptors and waits; one issues.
      const bool leader = elect_one_sync();
      auto commit = [&](uint64_t* bar) {
        if (leader) tc_commit(bar);
      };
      constexpr uint32_t ab = kMmaBf16 ? 1u : 0u;
      constexpr uint32_t idS = idesc_f16(128, 128, ab, 0, 0);
      constexpr uint32_t idPV = idesc_f16(128, D, ab, 0, 1);
      const uint64_t dq0 = smem_desc_sw128(smem_u32(s.q[0]), 16, 1024);
      const uint64_t dk0 = smem_desc_sw128(smem_u32(s.kv[0]), 16, 1024);
      const uint64_t dv0 = smem_desc_sw128(smem_u32(s.kv[0]), Smem::kBlockBytes, 1024);
      uint32_t units = 0, ring = 0;
      int base0 = 0, base1 = 0;  // P V products of tiles A, B in earlier units
      bool ok = true;
      while (ok && take_unit(s, taken++, u, p.err, abort_flag)) {
        if (u.first > u.last) continue;
        int s_left = u.count(0) + u.count(1);
        auto issue_s = [&](int t, uint32_t g) {  // K of streamed tile g
          const uint64_t dq = desc_add(dq0, t * Smem::kTileBytes);
          const uint64_t dk = desc_add(dk0, (2 * g) % kStages * Smem::kTileBytes);
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * Smem::kBlockBytes + (kk & 3) * 32;
            if (leader)
              tc_mma_ss(tbase + t * 128, desc_add(dq, off), desc_add(dk, off), idS,
                        kk > 0 ? 1u : 0u);
          }
          commit(&s.s_full[t]);
          if (--s_left == 0) commit(&s.q_empty);  // the next unit's Q may come
        };
        auto k_wait = [&](uint32_t g) {
          return mbar_wait_poll(&s.full[(2 * g) % kStages], (2 * g) / kStages & 1, p.err,
                                abort_flag);
        };
        ok = mbar_wait_poll(kFp8 && kBf16 ? &s.q_ready : &s.q_full, units & 1, p.err,
                            abort_flag) &&
             k_wait(ring);
        ++units;
        if (!ok) break;
        tc_fence_after();
        if (u.first >= u.lo0 && u.first <= u.hi0) issue_s(0, ring);
        if (u.first >= u.lo1 && u.first <= u.hi1) issue_s(1, ring);
        commit(&s.empty[(2 * ring) % kStages]);
        for (int j = u.first; ok && j <= u.last; ++j) {
          const uint32_t g = ring + static_cast<uint32_t>(j - u.first);
          const int st = (2 * g + 1) % kStages;
          ok = mbar_wait_poll(&s.full[st], (2 * g + 1) / kStages & 1, p.err, abort_flag);
          if (!ok) break;
          bool k_next = false;  // K_{j+1} has landed
          for (int t = 0; ok && t < 2; ++t) {
            const int lt = t ? u.lo1 : u.lo0, ht = t ? u.hi1 : u.hi0;
            const bool active = j >= lt && j <= ht;
            // S_t(j + 1) is next: after P V of tile j, or as the first product
            // of a tile whose range starts there
            const bool s_next = active ? j + 1 <= ht : (j + 1 == lt && lt <= ht);
            if (active) {
              ok = mbar_wait_poll(&s.p_full[t], ((t ? base1 : base0) + j - lt) & 1, p.err,
                                  abort_flag);
              if (!ok) break;
              tc_fence_after();
              const uint64_t dv = desc_add(dv0, st * Smem::kTileBytes);
#pragma unroll
              for (int kk = 0; kk < kTile / 16; ++kk)
                if (leader)
                  tc_mma_ts(tbase + 256 + t * D, tbase + t * 128 + kk * 8,
                            desc_add(dv, kk * 16 * 128), idPV, (j > lt || kk > 0) ? 1u : 0u);
              commit(&s.o_done[t]);
            }
            if (s_next) {
              if (!k_next) {
                ok = k_wait(g + 1);
                if (!ok) break;
                tc_fence_after();
                k_next = true;
              }
              issue_s(t, g + 1);
            }
          }
          commit(&s.empty[st]);
          if (k_next) commit(&s.empty[(2 * g + 2) % kStages]);
        }
        ring += static_cast<uint32_t>(u.streamed());
        base0 += u.count(0);
        base1 += u.count(1);
      }
      // Every product issued above completes before TMEM is released.
      commit(&s.drain);
      int zero = 0;
      mbar_wait(&s.drain, 0, p.err, &zero, 100000000ull);
    } else if (warp == 10) {
      // -------------------------------------------------------------- units
      const Place at = warp_place<true, kParts>(p, gridDim.x, blockIdx.x);
      if (lane == 0 && at.left == 0 && !p.whole) p.tasks[blockIdx.x] = JoinTask{-1, 0, 0, 0, 0};
      WorkWalk<true, kParts> walk(at);
      Piece x;
      for (uint32_t n = 0;; ++n) {
        const bool more = walk.next(p, x);
        ManyUnit v{};
        if (more) {
          const Seq& q = walk.w.s;
          many_range(p, x, q, x.t0, min(x.t1, x.t0 + tile_tokens), v.lo0, v.hi0);
          many_range(p, x, q, x.t0 + tile_tokens, x.t1, v.lo1, v.hi1);
          v.first = v.lo0 <= v.hi0 ? v.lo0 : v.lo1;
          v.last = max(v.hi0, v.hi1);
          if (v.lo0 > v.hi0 && v.lo1 > v.hi1) {
            v.first = 1;
            v.last = 0;
          }
          v.key_lo = x.lo;
          v.key_hi = x.hi;
          v.start = q.start + x.t0;
          v.tokens = x.t1 - x.t0;
          v.pos = q.pos0 + x.t0;
          v.len = q.len;
          v.b = x.b;
          v.hk = x.hk;
          v.slot = x.whole ? -1 : x.slot;
          v.valid = 1;
          if (lane == 0 && !p.whole) p.tasks[blockIdx.x] = join_task(p, x, q);
        }
        const int slot = n % kUnitRing;
        if (n >= kUnitRing && !many_warp_wait(&s.unit_empty[slot], (n / kUnitRing - 1) & 1, p.err,
                                              abort_flag))
          break;
        if (lane == 0) {
          s.unit[slot][0] = make_int4(v.lo0, v.hi0, v.lo1, v.hi1);
          s.unit[slot][1] = make_int4(v.first, v.last, v.key_lo, v.key_hi);
          s.unit[slot][2] = make_int4(v.start, v.tokens, v.pos, v.len);
          s.unit[slot][3] = make_int4(v.b, v.hk, v.slot, v.valid);
          mbar_arrive(&s.unit_full[slot]);
        }
        __syncwarp();
        if (!more) break;
      }
    } else if (warp >= ManyWarps<kFp8>::kFirst) {
      // ---------------------- zeroing (warp 11), or conversion (warps 12-15)
      [[maybe_unused]] const int cv = tid - 32 * ManyWarps<kFp8>::kFirst;
      [[maybe_unused]] uint32_t units = 0;
      uint32_t ring = 0;
      [[maybe_unused]] uint32_t fixed = 0;  // bit st: parity of the next tile in raw_full[st]
      bool ok = true;
      while (ok && take_unit(s, taken++, u, p.err, abort_flag)) {
        if (u.first > u.last) continue;
        if constexpr (!kFp8) {
          for (int j = u.first; ok && j <= u.last; ++j, ++ring) {
            if (!u.ragged(j)) continue;
            const int st = (2 * ring + 1) % kStages;
            // (a barrier of its own: this warp skips the other tiles, whose phases
            // it would lose count of)
            ok = many_warp_wait(&s.raw_full[st], (fixed >> st) & 1, p.err, abort_flag);
            if (!ok) break;
            fixed ^= 1u << st;
            for (int i = lane; i < kTile * (2 * D / 16); i += 32) {
              const int r = i & (kTile - 1), c = i >> 7;  // 16-byte chunk c of row r
              const int key = j * kTile + r;
              if (key < u.key_lo || key >= u.key_hi)
                *reinterpret_cast<uint4*>(s.kv[st] + (c >> 3) * Smem::kBlockBytes + r * 128 +
                                          (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.full[st]);
          }
        } else {
          if constexpr (kBf16) {
            // Q to fp16, each row under the power of two that takes its largest
            // magnitude into [2^14, 2^15)
            ok = many_warp_wait(&s.q_full, units & 1, p.err, abort_flag);
            if (!ok) break;
            for (int i = cv; i < 2 * kTile; i += kConverters) {
              uint8_t* row = s.q[i >> 7] + (i & 127) * 128;
              float top = 0.f;
#pragma unroll 4
              for (int c = 0; c < 2 * D / 16; ++c) {
                const uint4 v = *reinterpret_cast<const uint4*>(
                    row + (c >> 3) * Smem::kBlockBytes + (((c & 7) ^ (i & 7)) << 4));
                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float2 f = unpack2<true>(u[e]);
                  top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                }
              }
              const int e = static_cast<int>(__float_as_uint(top) >> 23);
              const int shift = min(max(141 - e, -112), 126);
              const float down = many_exp2_field(127 + shift);
              s.qshift[units & 1][i] = static_cast<int8_t>(shift);
#pragma unroll 4
              for (int c = 0; c < 2 * D / 16; ++c) {
                uint4* at = reinterpret_cast<uint4*>(row + (c >> 3) * Smem::kBlockBytes +
                                                     (((c & 7) ^ (i & 7)) << 4));
                const uint4 v = *at;
                const uint32_t u[4] = {v.x, v.y, v.z, v.w};
                uint32_t h[4];
#pragma unroll
                for (int e2 = 0; e2 < 4; ++e2) {
                  const float2 f = unpack2<true>(u[e2]);
                  h[e2] = pack2<false>(f.x * down, f.y * down);
                }
                *at = make_uint4(h[0], h[1], h[2], h[3]);
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s.q_ready);
          }
          ++units;
          // Two warps convert K tiles and two V tiles, side by side.  All four
          // see every tile land and arrive for it, so that V's barrier covers
          // what the others have written for its key tile too.
          const int my_kv = (warp - ManyWarps<kFp8>::kFirst) >> 1;
          // Largest exponent of the piece's keys, or values, so far, or 12: 2^(ref - 11
          // - 127), by which the results are scaled back, stays a normal number.  (Rows
          // of exponent 1 lose nothing under it.)
          uint32_t ref = 12;
          for (int j = u.first; ok && j <= u.last; ++j, ++ring) {
            const bool cut = u.ragged(j);
#pragma unroll 1
            for (int kv = 0; kv < 2; ++kv) {
              const uint32_t n = 2 * ring + kv;
              const int st = n % kStages;
              ok = many_warp_wait(&s.raw_full[st], (n / kStages) & 1, p.err, abort_flag);
              if (!ok) break;
              if (kv != my_kv) {
                if (lane == 0) mbar_arrive(&s.full[st]);
                continue;
              }
              {
                uint32_t four = reinterpret_cast<const uint32_t*>(s.exps[st])[lane];
                if (cut) {
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const int key = j * kTile + lane * 4 + i;
                    if (key < u.key_lo || key >= u.key_hi) four &= ~(0xffu << (8 * i));
                  }
                }
                const uint32_t top = max(max(four & 0xffu, (four >> 8) & 0xffu),
                                         max((four >> 16) & 0xffu, four >> 24));
                ref = max(ref, __reduce_max_sync(0xffffffffu, top));
              }
              const int base_e = static_cast<int>(ref);
              if ((cv & 63) == 0) (kv ? s.vref : s.kref)[ring % kRefs] = base_e;
              // Eight lanes share a row, lane c with codes 8 c .. 8 c + 7 of each
              // 64: they become chunk c of the row in that column block.  A
              // warp's rows are 8 apart, so that their swizzle is the same and
              // every address a constant away from the first; it reads kBatch
              // of them before it writes any: in place, a row's raw bytes lie
              // under its converted ones.  Odd rows take the 64s in the other
              // order, for the banks' sake.
              constexpr int kPieces = D / 64, kBatch = 4, kStep = 8;
              const int c = lane & 7, r0 = (warp & 1) * 4 + (lane >> 3);
              const int flip = r0 & (kPieces - 1);
              const uint8_t* from[kPieces];
              uint8_t* to[kPieces];
#pragma unroll
              for (int h = 0; h < kPieces; ++h) {
                const int x = (h ^ flip) * 8 + c;  // 8-byte piece of the raw row
                from[h] = s.raw(st) + (x & 1) * 8 +
                          (D == 128 ? r0 * 128 + (((x >> 1) ^ (r0 & 7)) << 4)
                                    : r0 * 64 + (((x >> 1) ^ ((r0 >> 1) & 3)) << 4));
                to[h] = s.kv[st] + (h ^ flip) * Smem::kBlockBytes + r0 * 128 +
                        ((c ^ (r0 & 7)) << 4);
              }
              // Factors 2^(e - ref + 7), which keep codes below 448 * 128, as fp16
              // pairs: this lane's are of rows 8 (lane >> 2) + (lane & 3) of the
              // warp's fours, and 64 on.  e = 0 (and rows to leave out) make
              // zeros whatever the codes; -0 stands for that.
              uint32_t f2[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int r = (warp & 1) * 4 + (lane & 3) + (lane >> 2) * kStep + i * 64;
                const int key = j * kTile + r, e = s.exps[st][r];
                const float f = many_exp2_field(134 + e - base_e);
                f2[i] = e == 0 || (cut && (key < u.key_lo || key >= u.key_hi)) ? 0x80008000u
                                                                              : pack2<false>(f, f);
              }
              const bool empty =
                  __any_sync(0xffffffffu, f2[0] == 0x80008000u || f2[1] == 0x80008000u);
              auto rows = [&](auto some_empty) {
#pragma unroll 1
                for (int m = 0; m < kTile / kStep; m += kBatch) {
                  uint2 v[kBatch][kPieces];
#pragma unroll
                  for (int i = 0; i < kBatch; ++i)
#pragma unroll
                    for (int h = 0; h < kPieces; ++h)
                      v[i][h] = *reinterpret_cast<const uint2*>(from[h] + (m + i) * kStep * D);
                  if constexpr (Smem::kInPlace) __syncwarp();
#pragma unroll
                  for (int i = 0; i < kBatch; ++i) {
                    const uint32_t f = __shfl_sync(0xffffffffu, m < 8 ? f2[0] : f2[1],
                                                   ((m + i) & 7) * 4 + (lane >> 3));
#pragma unroll
                    for (int h = 0; h < kPieces; ++h) {
                      uint32_t w0 = v[i][h].x, w1 = v[i][h].y;
                      if (some_empty && f == 0x80008000u) w0 = w1 = 0u;
                      *reinterpret_cast<uint4*>(to[h] + (m + i) * kStep * 128) =
                          make_uint4(mul_f16x2(e4m3x2_to_f16x2(w0), f),
                                     mul_f16x2(e4m3x2_to_f16x2(w0 >> 16), f),
                                     mul_f16x2(e4m3x2_to_f16x2(w1), f),
                                     mul_f16x2(e4m3x2_to_f16x2(w1 >> 16), f));
                    }
                  }
                }
              };
              if (empty)
                rows(std::true_type{});
              else
                rows(std::false_type{});
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&s.full[st]);
            }
          }
        }
      }
    }
  } else {
    setmaxnreg_inc<ManyWarps<kFp8>::kHigh>();
    // -------------------------------------------------------------- softmax
    const int t = warp >> 2, r = tid & 127;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tbase + t * 128, tO = tbase + 256 + t * D;
    const int row_token = r / p.group, row_head = r - row_token * p.group;
    int base = 0;  // key tiles of this query tile in earlier units
    uint32_t ring = 0, units = 0;
    bool ok = true;
    while (ok && take_unit(s, taken++, u, p.err, abort_flag)) {
      const int lt = t ? u.lo1 : u.lo0, n_tiles = u.count(t);
      const int token = t * tile_tokens + row_token;    // of the block
      const bool mine = r < tile_rows && token < u.tokens;  // a row to write
      // rows that are none see what the tile's last token sees
      const int first_token = t * tile_tokens;
      const int last_token = min(u.tokens, first_token + tile_tokens) - 1;
      const int pos = u.pos + min(token, last_token);
      const int head = u.hk * p.group + row_head;
      const float nslope2 = kAlibi && mine ? paged_slope2(p, u.b, head) : 0.f;
      // visible keys: of this row, and those that every row of the tile sees
      const int first = p.win_left < 0 ? 0 : pos - p.win_left;
      const int last = p.win_right < 0 ? u.len - 1 : min(u.len - 1, pos + p.win_right);
      const int pos_a = u.pos + first_token, pos_b = u.pos + last_token;
      const int all_first = p.win_left < 0 ? 0 : pos_b - p.win_left;
      const int all_last = p.win_right < 0 ? u.len - 1 : min(u.len - 1, pos_a + p.win_right);
      // some row of the tile sees at most 128 keys (the count is concave in the
      // row, so an end row has the fewest): see lo below
      const bool few_keys = [&] {
        auto count = [&](int q) {
          return min(u.len - 1, p.win_right < 0 ? u.len - 1 : q + p.win_right) -
                 max(0, p.win_left < 0 ? 0 : q - p.win_left) + 1;
        };
        return min(count(pos_a), count(pos_b)) <= kTile;
      }();
      float sl2 = p.scale_log2;
      int vbase = 0;  // e4m3: the value exponent that O is relative to
      float m = -INFINITY;  // reference maximum, log2 units
      float l = 0.f;        // sum of 2^(t - m)
      // The sum O is divided by: the largest weight of each tile enters as
      // rounded to 16 bits, and in cut tiles of rows with few keys every weight,
      // so that the weights that dominate O sum to one as rounded (as in the
      // dense forward).  The LSE keeps the exact sum l.
      float lo = 0.f;
      for (int jj = 0, j = lt; jj < n_tiles; ++jj, ++j) {
        ok = many_warp_wait(&s.s_full[t], (base + jj) & 1, p.err, abort_flag);
        if (!ok) break;
        tc_fence_after();
        const uint32_t g = ring + static_cast<uint32_t>(j - u.first);
        float mult = sl2;   // scores -> log2 units
        int vshift = 0;     // e4m3: this tile's value exponent over vbase
        bool rebase = false;
        float down = 1.f;
        if constexpr (kFp8) {
          // converted V comes after K and Q by the same threads
          ok = many_warp_wait(&s.full[(2 * g + 1) % kStages], (2 * g + 1) / kStages & 1, p.err,
                              abort_flag);
          if (!ok) break;
          if (jj == 0 && kBf16) sl2 *= many_exp2_field(127 - s.qshift[units & 1][t * kTile + r]);
          // K was scaled by 2^(127 - kref + 7)
          mult = sl2 * many_exp2_field(s.kref[g % kRefs] - 7);
          const int vr = s.vref[g % kRefs];
          if (jj == 0) vbase = vr;
          if (vr - vbase > 3) {
            down = many_exp2_field(127 + vbase - vr);
            vbase = vr;
            rebase = jj > 0;
          }
          vshift = vr - vbase;
        }
        const bool pos_scale = mult > 0.f;
        float sv[kTile];
        {
          uint32_t raw[kTile / 32][32];
#pragma unroll
          for (int c = 0; c < kTile / 32; ++c) tmem_ld32(tS + lane_off + c * 32, raw[c]);
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < kTile / 32; ++c)
#pragma unroll
            for (int e = 0; e < 32; ++e) sv[c * 32 + e] = __uint_as_float(raw[c][e]);
        }
        const int k0 = j * kTile;
        const bool prescale = kAlibi || !pos_scale;
        if (kAlibi) {
          const float d0 = static_cast<float>(k0 - pos);
#pragma unroll
          for (int c = 0; c < kTile; ++c)
            sv[c] = fmaf(sv[c], mult, nslope2 * fabsf(d0 + static_cast<float>(c)));
        } else if (!pos_scale) {
#pragma unroll
          for (int c = 0; c < kTile; ++c) sv[c] *= mult;
        }
        const bool masked = k0 < all_first || k0 + kTile - 1 > all_last;
        if (masked) {
          // visible columns cf .. cl of this row; 32 columns at a time, as a
          // warp's rows agree about most of them
          const int cf = first - k0, cl = last - k0;
#pragma unroll
          for (int c = 0; c < kTile; c += 32) {
            if (__any_sync(0xffffffffu, cl < c + 31)) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (c + e > cl) sv[c + e] = -INFINITY;
            }
            if (p.win_left >= 0 && __any_sync(0xffffffffu, cf > c)) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (c + e < cf) sv[c + e] = -INFINITY;
            }
          }
        }
        float mxs[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) mxs[e] = sv[e];
#pragma unroll
        for (int c = 8; c < kTile; c += 16)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            mxs[e] = c + 8 < kTile ? fmax3(mxs[e], sv[c + e], sv[c + 8 + e])
                                   : fmaxf(mxs[e], sv[c + e]);
        const float mx = fmax3(fmax3(mxs[0], mxs[1], mxs[2]), fmax3(mxs[3], mxs[4], mxs[5]),
                               fmaxf(mxs[6], mxs[7]));
        // (a masked score times a positive scale stays -inf)
        const float m_tile = prescale ? mx : mx * mult;
        const float m_new = fmaxf(m, m_tile);
        const bool need = m_new > m + kThreshold;
        float alpha = 1.f;
        if (need) {
          alpha = ex2_approx(m - m_new);  // 0 on the first tile (m = -inf)
          l *= alpha;
          lo *= alpha;
          m = m_new;
        }
        if (jj > 0 && __any_sync(0xffffffffu, need || rebase)) {
          ok = many_warp_wait(&s.o_done[t], (base + jj - 1) & 1, p.err, abort_flag);
          if (!ok) break;
          tc_fence_after();
          alpha *= down;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + lane_off + c * 32, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tmem_st32(tO + lane_off + c * 32, o);
          }
        }
        // the tile's P is 2^(kPOffset + vshift) times the weights; unscale
        // brings their sum back
        const float offset = static_cast<float>(kPOffset + vshift);
        const float unscale = many_exp2_field(127 - kPOffset - vshift);
        const float mneg = (m == -INFINITY) ? 0.f : offset - m;
        const float em = prescale ? 1.f : mult;
        const uint64_t mult2 = f32x2(em, em), mneg2 = f32x2(mneg, mneg);
        const float pmax = ex2_approx(fmaf(mx, em, mneg));
        const float pmax_corr = unpack2<kMmaBf16>(pack2<kMmaBf16>(pmax, 0.f)).x - pmax;
        uint64_t sums[2] = {f32x2(0.f, 0.f), f32x2(0.f, 0.f)};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const float2 z = split_f32x2(
                fma_f32x2(f32x2(sv[h * 64 + 2 * c], sv[h * 64 + 2 * c + 1]), mult2, mneg2));
            const float p0 = ex2_approx(z.x), p1 = ex2_approx(z.y);
            sums[c & 1] = add_f32x2(sums[c & 1], f32x2(p0, p1));
            pk[c] = pack2<kMmaBf16>(p0, p1);
          }
          tmem_st32(tS + lane_off + h * 32, pk);
        }
        const float2 s0 = split_f32x2(sums[0]), s1 = split_f32x2(sums[1]);
        const float tile_sum = (s0.x + s0.y) + (s1.x + s1.y);
        l = fmaf(tile_sum, unscale, l);
        if (masked && few_keys) {
          tmem_st_wait();
          uint64_t rs = f32x2(0.f, 0.f);
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t pr[32];
            tmem_ld32(tS + lane_off + h * 32, pr);
            tmem_ld_wait();
#pragma unroll
            for (int c = 0; c < 32; ++c) {
              const float2 q2 = unpack2<kMmaBf16>(pr[c]);
              rs = add_f32x2(rs, f32x2(q2.x, q2.y));
            }
          }
          const float2 r2 = split_f32x2(rs);
          lo = fmaf(r2.x + r2.y, unscale, lo);
        } else {
          lo = fmaf(tile_sum + pmax_corr, unscale, lo);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(&s.p_full[t]);
      }
      if (!ok) break;

      // ------------------------------------------------------------ epilogue
      const bool have = n_tiles > 0;
      if (have) {
        ok = many_warp_wait(&s.o_done[t], (base + n_tiles - 1) & 1, p.err, abort_flag);
        if (!ok) break;
        tc_fence_after();
      }
      if (t == 0 || u.two(tile_tokens)) {
        // O in tensor memory is 2^kPOffset (e4m3: and 2^(127 + 7 - vbase)) times
        // the sum of weights times values
        // (of small values in two steps, as the first divides by a sum of many weights)
        const bool small = kFp8 && vbase < 64;
        const float back =
            many_exp2_field((kFp8 ? vbase - 7 + (small ? 64 : 0) : 127) - kPOffset);
        const float per = lo == 0.f ? 0.f : back / lo;
        const bool whole = u.slot < 0;
        // partial results are divided by their sum as rounded and multiplied by
        // the exact one, which is what they are joined with
        const float scale = whole ? per : per * l;
        const long long at =
            (2LL * blockIdx.x + max(u.slot, 0)) * p.block_rows + t * tile_rows + r;
        const long long row = u.start + token;
        if (mine) {
          if (whole) store_stats<kParts>(p, row, head, m, l);
          else p.part_ml[at] = make_float2(m, l);
        }
        // This row's 128-byte pieces in the output: D / 64 of 16-bit elements,
        // D / 32 of fp32.  (The loops stay rolled: unrolled, the epilogue spent
        // most of its 2.5 us waiting for its own instructions.)
        const bool narrow = whole && !(kParts && p.o32);
        uint8_t* out = narrow ? reinterpret_cast<uint8_t*>(static_cast<uint16_t*>(p.o) +
                                                           row * p.o_token + head * p.o_head)
                       : whole ? reinterpret_cast<uint8_t*>(p.o32 + (row * p.heads + head) * D)
                               : reinterpret_cast<uint8_t*>(p.part_o + at * D);
        if (!mine) out = nullptr;
        // the rows this lane writes 16 bytes of: rr = lane / 8 + 4 i
        unsigned long long rows[kFp8 ? 1 : 8];
        if constexpr (!kFp8) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            rows[i] = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(out),
                                  (lane >> 3) + 4 * i);
        }
        // (a cut piece without tiles leaves its maximum, -inf, alone)
        const int chunks = whole || have ? D / 32 : 0;
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {  // 32 columns
          uint32_t o[32];
          if (have) {
            tmem_ld32(tO + lane_off + c * 32, o);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * scale);
          if (lo == 0.f) {  // no key: zeros, also where other rows saw a NaN value
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          if (small) {
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = __float_as_uint(__uint_as_float(o[e]) * many_exp2_field(127 - 64));
          }
          // 16-bit: half a piece, fp32: a whole one
          const int half = narrow ? (c & 1) * 4 : 0, n = narrow ? 4 : 8;
          if (narrow) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              o[e] = pack2<kBf16>(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
          }
          if constexpr (kFp8) {
            if (mine) {
#pragma unroll
              for (int q = 0; q < 8; ++q)
                if (q < n)
                  *reinterpret_cast<uint4*>(out + (half + q) * 16) =
                      make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
            }
          } else {
            // through shared memory, so that eight lanes write a row's 128 bytes
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (q < n)
                *reinterpret_cast<uint4*>(s.stage[warp] + lane * 128 +
                                          (((half + q) ^ (lane & 7)) << 4)) =
                    make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
          }
          if (narrow && !(c & 1)) continue;  // the piece's other half comes next
          if constexpr (!kFp8) {
            __syncwarp();
            uint4 v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int rr = (lane >> 3) + 4 * i;
              v[i] = *reinterpret_cast<const uint4*>(s.stage[warp] + rr * 128 +
                                                     (((lane ^ rr) & 7) << 4));
            }
            const int piece = narrow ? c >> 1 : c;
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (rows[i])
                *reinterpret_cast<uint4*>(rows[i] + piece * 128 + (lane & 7) * 16) = v[i];
            __syncwarp();
          } else {
            out += 128;
          }
        }
      }
      if (u.first <= u.last) ++units;
      ring += static_cast<uint32_t>(u.streamed());
      base += n_tiles;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tbase, 512);
  }
}

template <int D, bool kFp8, bool kBf16, bool kAlibi, bool kParts = false>
cudaError_t launch_many_t(const PagedLaunch& a, cudaStream_t s) {
  auto kern = paged_many_kernel<D, kFp8, kBf16, kAlibi, kParts>;
  const int smem = static_cast<int>(sizeof(ManySmem<D, kFp8>)) + 1024;
  static_assert(sizeof(ManySmem<D, kFp8>) + 1024 <= 232448, "shared memory of one CTA");
  static AttrCache configured;
  cudaError_t e = ensure_dynamic_smem(kern, smem, configured);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, static_cast<unsigned>(a.sms), ManyWarps<kFp8>::kThreads, smem, s, a);
  return e != cudaSuccess || a.whole ? e : launch_join<D, kBf16, kParts>(a, s);
}

template <int D, bool kFp8>
cudaError_t launch_many_d(const PagedLaunch& a, cudaStream_t s) {
  const bool bf16 = a.elem == kElemBf16, alibi = a.alibi != nullptr;
  if (a.parts)  // (without biases)
    return bf16 ? launch_many_t<D, kFp8, true, false, true>(a, s)
                : launch_many_t<D, kFp8, false, false, true>(a, s);
  return bf16 ? (alibi ? launch_many_t<D, kFp8, true, true>(a, s)
                       : launch_many_t<D, kFp8, true, false>(a, s))
              : (alibi ? launch_many_t<D, kFp8, false, true>(a, s)
                       : launch_many_t<D, kFp8, false, false>(a, s));
}

}  // namespace

int paged_many_rows(int group) { return 2 * (kTile / group) * group; }

cudaError_t launch_paged_many(const PagedLaunch& a, cudaStream_t s) {
  const bool fp8 = a.cache_elem == kElemE4m3;
  if (a.D == 64) return fp8 ? launch_many_d<64, true>(a, s) : launch_many_d<64, false>(a, s);
  return fp8 ? launch_many_d<128, true>(a, s) : launch_many_d<128, false>(a, s);
}

}  // namespace fa
