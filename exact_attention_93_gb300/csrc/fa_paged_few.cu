// fa_paged_few.cu -- attention over a paged cache for few query rows per
// sequence: single tokens being generated, short runs of drafted tokens.
//
//   s_j = scale * q . k_j - slope |p - j|,  m = max_j s_j,
//   l = sum_j 2^(s_j - m),  o = sum_j 2^(s_j - m) v_j / l   (log2 units)
//
// What bounds it.  Every cached key and value is read once for 2 G
// multiply-adds per element (G query heads to a key head): at 8 bytes moved
// per 1000 products the tensor cores idle and HBM is the bound.  So the kernel
// is a stream: one CTA per SM walks its stretch of the work (fa_paged.cuh) and
// four producer warps keep rings of K and V tiles (128 keys each) in flight by
// TMA, page by page.  (One warp took 0.3 us to issue a tile's boxes, which an
// e4m3 cache streams in 0.4 us.)
//
// Eight consumer warps in two groups take alternate tiles, 32 keys of a tile
// each, with a running maximum, sum and O of their own that are joined once per
// piece of work: no barrier among them inside the key loop, and two tiles of
// dependent steps in flight.  (With every warp on the same tile, 16 keys each,
// an e4m3 batch of 64 contexts took 9 % longer; three groups of four warps, with
// one producer each, gained nothing there and lost 20 % on 128 shorter contexts.)
// The products are turned around, S^T = K Q^T and O^T = V^T P^T, on mma.sync
// m16n8k16: keys and head columns fill the 16 rows, so the padding of the query
// side is to 8 rows, and the operands go from shared memory to registers to the
// tensor core without a detour through tensor memory, which a tile of 8 columns
// would not fill.  P^T moves from the accumulator to the operand layout by an
// in-register 8 x 8 transpose.  The tensor cores take P in 16 bits, so weights are
// rounded (by 2^-8 of themselves at most in bf16, 2^-11 in fp16), each on its own;
// O is divided by the sum of the unrounded ones.
//
// e4m3 caches.  Codes convert exactly to fp16 in registers, so an 8-bit cache
// costs half the HBM bytes and no precision beyond its own: q is scaled by a
// power of two per row to fit fp16, key exponents scale the scores in fp32,
// and value exponents go into P relative to the largest one seen so far, R:
// P' = 2^(s - m) * 2^(e_v - R + 15), at most 2^15.  Weights and exponents share
// fp16's range that way: P' is normal down to a product of 2^-29.  (Scaling V
// instead would leave the range to each, at a multiply for every value; with the
// rows' magnitudes within some 2^10 of one another, weights keep their 11 bits down
// to 2^-19.)  The order of the head columns (keys) and of columns and keys (values)
// inside an operand is chosen so that a lane reads 16 contiguous bytes.
//
// Measured (32 query and 8 key heads): 64 contexts of 256 to 16000 keys, D = 128,
// 16-bit 188 us, 6.6 TB/s of keys and values, 97 % of the measured copy rate;
// D = 64 108 us, 5.7 TB/s.  e4m3, D = 128, 118 us, 5.3 TB/s (the same stream
// without its products 107 us, of which 13 are the start and the joining), and
// D = 64 84 us, where the conversions bound it (the stream alone 62).  Sixteen rows (4
// tokens a sequence) take half as long again as eight over an e4m3 cache, a tenth
// longer over a 16-bit one: the second eight columns double the products, softmax and
// transposes of each warp's chain, which over e4m3 is nearly as long as the stream
// already with eight.  One context of 1000 keys 9 to 12 us, by the machine, of 4000 12
// to 15, of 32000 30 to 37: launch, the look at the batch, and the joining of the
// pieces.
#include "fa_paged.cuh"
#include "fa_serve.h"
#include "sm103_primitives.cuh"

namespace fa {
namespace {

constexpr int kConsumers = 8;                       // warps
constexpr int kProducers = 4;                       // K and V of either group
constexpr int kFewThreads = (kConsumers + kProducers) * 32;
// registers: 12 warps launch with kFewRegs each, 2 x kFewHigh + kFewLow = 3 x
// kFewRegs on each sub-partition.  That leaves room on the SM for blocks of the
// joining kernel, which wait there for this one's end instead of starting after
// it (1000 keys, one sequence: 16.5 -> 13.2 us).
constexpr uint32_t kFewLow = 80, kFewHigh = 176, kFewRegs = 144;
constexpr int kGroups = 2, kGroupWarps = kConsumers / kGroups;
constexpr int kSlices = kTile / kGroupWarps / 16;    // 16-key slices of a tile per warp
constexpr int kRingBytes = 192 * 1024;

template <int D, bool kFp8, int NB>
struct FewSmem {
  static constexpr int kRowBytes = kFp8 ? D : 2 * D;
  static constexpr int kSlotBytes = kTile * kRowBytes;
  // Each group of consumers has a ring of its own, through which the K and V of
  // its tiles alternate: a slot's uses then follow one another in one group's
  // sight, and none can be mistaken for the one before it.
  static constexpr int kSlots = kRingBytes / kSlotBytes, kRing = kSlots / kGroups;
  // a row of the joining buffer: 16-bit, its columns; e4m3, where a lane holds
  // columns (D / 8) g + 2 mb and the next of every block mb, pair mb of lane group g
  // at 2 (10 mb + g): stores of pairs and loads of a lane's columns meet no bank twice
  static constexpr int kMergePitch = kFp8 ? D / 16 * 20 + 4 : D + 4;
  static constexpr int kSteps = D / 16;
  alignas(1024) uint8_t ring[kSlots][kSlotBytes];
  alignas(16) uint8_t exps[kFp8 ? kSlots : 1][kTile];
  // joining the warps' results: eight query rows of one group's warps at a time
  alignas(16) float merge[kGroupWarps][8][kMergePitch];
  float m[kConsumers][8 * NB], l[kConsumers][8 * NB];
  int vref[kConsumers];
  uint64_t full[kSlots], empty[kSlots];
  Place place;
  int abort_flag;
};

// Waits like mbar_wait, but at once when some thread of the CTA has given up:
// the walk then goes on over whatever is in shared memory, so that every
// barrier keeps its count, and the error word tells the caller.
__device__ __forceinline__ void ring_wait(uint64_t* bar, uint32_t parity, uint32_t* err,
                                          volatile int* abort_flag) {
  if (*abort_flag) return;
  mbar_wait(bar, parity, err, abort_flag);
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

template <bool kBf16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if constexpr (kBf16) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  }
}

// 2^(n - 127) for an exponent field n, 0 below the normal range.
__device__ __forceinline__ float exp2_field(int n) {
  return __uint_as_float(static_cast<uint32_t>(min(max(n, 0), 254)) << 23);
}

template <int D, bool kFp8, bool kBf16, int NB>
__global__ void __maxnreg__(kFewRegs)
    paged_few_kernel(const __grid_constant__ PagedLaunch p) {
  pdl_wait_and_release();
  using Smem = FewSmem<D, kFp8, NB>;
  constexpr int kRows = 8 * NB, kRowBytes = Smem::kRowBytes;
  constexpr int kSlots = Smem::kSlots, kRing = Smem::kRing;
  constexpr int kSteps = Smem::kSteps;      // k16 steps over the head, and m16 blocks of V^T
  constexpr bool kMmaBf16 = kBf16 && !kFp8;  // type of the products
  // weights are kept as 2^(s - m + kLift): fp16 ones reach up to 2^15 and stay
  // normal down to 2^-29 of the largest (e4m3: see pfac)
  constexpr float kLift = !kFp8 && !kBf16 ? 15.f : 0.f;
  extern __shared__ uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>(smem_raw + (-smem_u32(smem_raw) & 1023u));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    const Place at = warp_place<false>(p, gridDim.x, blockIdx.x);
    if (lane == 0) {
      s.place = at;
      if (at.left == 0 && !p.whole) p.tasks[blockIdx.x] = JoinTask{-1, 0, 0, 0, 0};
    }
  }
  if (threadIdx.x == 32) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], kGroupWarps);
    }
    s.abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  volatile int* abort_flag = &s.abort_flag;
  WorkWalk<false> walk(s.place);
  Piece x;

  if (warp >= kConsumers) {
    // --------------------------------------------------------------- producers
    setmaxnreg_dec<kFewLow>();
    const int group = (warp - kConsumers) >> 1, kv = (warp - kConsumers) & 1;
    const CUtensorMap* map = kv ? &p.map_v : &p.map_k;
    const uint8_t* exps = kv ? p.v_exp : p.k_exp;
    const int box_rows = min(p.page_size, kTile);
    const int per_tile = kTile / box_rows;
    if (lane == 0) tma_prefetch_desc(map);
    uint32_t tiles = 0;  // of the pieces before this one
    uint32_t loads = 0;  // this warp's
    while (walk.next(p, x)) {
      PageFeed feed;
      feed.start(p, x.b, x.tile0, x.lo, x.hi);
      for (int tile = x.tile0 + ((group - static_cast<int>(tiles)) & (kGroups - 1));
           tile < x.tile1; tile += kGroups) {
        const int k0 = tile * kTile + lane * box_rows;
        // lane i < per_tile: the i-th box of the tile, if a visible key lies in it
        const bool mine = lane < per_tile && k0 < x.hi && k0 + box_rows > x.lo;
        const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, mine));
        int page = feed.get(p, tile, k0);
        if (mine && (page < 0 || page >= p.pages)) {
          atomicExch(p.err, kDevErrBadIndex);
          page = p.pages;  // out of range for the tensor map: reads as zeros
        }
        const int row = k0 & (p.page_size - 1);
        const uint32_t n = 2 * loads + kv;  // in the group's ring
        const int slot = group * kRing + n % kRing;
        if (n >= kRing) ring_wait(&s.empty[slot], (n / kRing - 1) & 1, p.err, abort_flag);
        if (__any_sync(0xffffffffu, *abort_flag)) goto stopped;
        if (lane == 0)
          mbar_arrive_expect_tx(&s.full[slot], boxes * box_rows * (kRowBytes + (kFp8 ? 1 : 0)));
        __syncwarp();
        if (mine) {
          uint8_t* dst = s.ring[slot] + lane * box_rows * (kRowBytes < 128 ? kRowBytes : 128);
#pragma unroll
          for (int kb = 0; kb < (kRowBytes + 127) / 128; ++kb)
            tma_load_4d(dst + kb * kTile * 128, map, &s.full[slot], kb * 64, row, x.hk, page);
          if constexpr (kFp8)  // (of a page that does not exist, any exponents will do)
            bulk_load(s.exps[slot] + lane * box_rows,
                      exps + (static_cast<long long>(page < p.pages ? page : 0) * p.heads_k +
                              x.hk) * p.page_size + row,
                      box_rows, &s.full[slot]);
        }
        ++loads;
      }
      tiles += static_cast<uint32_t>(max(0, x.tile1 - x.tile0));
    }
  stopped:
    if (*abort_flag) {
      // Copies in flight land before the CTA's shared memory goes away.
      int zero = 0;
      if (lane == 0)
        for (uint32_t i = loads > kRing ? loads - kRing : 0; i < loads; ++i) {
          const uint32_t n = 2 * i + kv;
          if (n + kRing >= 2 * loads)  // (earlier ones have been read)
            mbar_wait(&s.full[group * kRing + n % kRing], (n / kRing) & 1, p.err, &zero,
                      100000000ull);
        }
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------------- consumers
    setmaxnreg_inc<kFewHigh>();
    const int g = lane >> 2, t = lane & 3;
    const int group = warp / kGroupWarps;
    const int slice0 = (warp % kGroupWarps) * kSlices * 16;  // this warp's first row of a tile
    // This lane's offsets into a tile, for its first slice; the others lie 16
    // rows on, with the same swizzle.  K as A operand (m16 x k16), V^T as A
    // operand; e4m3: 16 key bytes are chunks 2 t + h of rows g and g + 8 (four
    // steps of four columns each), values are D / 8 columns of rows 2 t and
    // 2 t + 1 (and 8 on).
    uint32_t koff[kFp8 ? 2 : 4], voff[kFp8 ? 2 : 4];
#pragma unroll
    for (int i = 0; i < (kFp8 ? 2 : 4); ++i) {
      if constexpr (!kFp8) {
        koff[i] = (slice0 + (lane & 15)) * 128 + (((i * 2 + (lane >> 4)) ^ (lane & 7)) << 4);
        voff[i] = (slice0 + (lane >> 4) * 8 + (lane & 7)) * 128 +
                  (((i * 2 + ((lane >> 3) & 1)) ^ (lane & 7)) << 4);
      } else if constexpr (D == 128) {
        koff[i] = (slice0 + g) * 128 + (((2 * t + i) ^ g) << 4);
        voff[i] = (slice0 + 2 * t + i) * 128 + ((g ^ (2 * t + i)) << 4);
      } else {
        koff[i] = (slice0 + g) * 64 + ((t ^ ((g >> 1) & 3)) << 4);
        voff[i] = (slice0 + 2 * t + i) * 64 + (((g >> 1) ^ t) << 4) + (g & 1) * 8;
      }
    }
    uint32_t tiles = 0;  // of the pieces before this one
    while (walk.next(p, x)) {
      const Seq& seq = walk.w.s;
      const int row0 = x.block * kRows;
      if (threadIdx.x == 0 && !p.whole) p.tasks[blockIdx.x] = join_task(p, x, seq);
      // -- queries as B operands, and what each of this lane's columns sees
      uint32_t qf[NB][kSteps][2];
      float qscale[NB][2];
      {
        float mine[NB];  // scale of query row 8 nb + g
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          uint32_t f[kSteps][2];
          const int r = nb * 8 + g;
          const uint16_t* src = nullptr;
          if (r < x.rows) {
            int token, head;
            row_of(p, row0, r, x.hk, token, head);
            src = static_cast<const uint16_t*>(p.q) +
                  static_cast<long long>(seq.start + token) * p.q_token + head * p.q_head;
          }
#pragma unroll
          for (int kk = 0; kk < kSteps; ++kk) {
            if constexpr (kFp8) {
              // a lane's 16 key bytes are four steps of four columns
              const uint2 v = src ? __ldg(reinterpret_cast<const uint2*>(
                                        src + (D == 128 ? 32 * t + 4 * kk : 16 * t + 4 * kk)))
                                  : make_uint2(0u, 0u);
              f[kk][0] = v.x;
              f[kk][1] = v.y;
            } else {
              f[kk][0] = src ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * kk + 2 * t)) : 0u;
              f[kk][1] =
                  src ? __ldg(reinterpret_cast<const uint32_t*>(src + 16 * kk + 8 + 2 * t)) : 0u;
            }
          }
          mine[nb] = 1.f;
          if constexpr (kFp8 && kBf16) {
            // bf16 -> fp16 under a power-of-two scale that takes the row's
            // largest magnitude into [2^14, 2^15): what falls below fp16's
            // normal range is under 2^-28 of that
            float top = 0.f;
#pragma unroll
            for (int kk = 0; kk < kSteps; ++kk)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float2 u = unpack2<true>(f[kk][i]);
                top = fmaxf(top, fmaxf(fabsf(u.x), fabsf(u.y)));
              }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const int e = static_cast<int>(__float_as_uint(top) >> 23);  // biased
            // down by 2^(e - 127 - 14) in two exact steps, each a normal number
            const int shift = min(max(141 - e, -112), 126);
            const float down = exp2_field(127 + shift);
            mine[nb] = exp2_field(127 - shift);
#pragma unroll
            for (int kk = 0; kk < kSteps; ++kk)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float2 u = unpack2<true>(f[kk][i]);
                f[kk][i] = pack2<false>(u.x * down, u.y * down);
              }
          }
#pragma unroll
          for (int kk = 0; kk < kSteps; ++kk) {
            qf[nb][kk][0] = f[kk][0];
            qf[nb][kk][1] = f[kk][1];
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int c = 0; c < 2; ++c)  // from the lanes of row 8 nb + 2 t + c
            qscale[nb][c] =
                p.scale_log2 * __shfl_sync(0xffffffffu, mine[nb], (2 * t + c) * 4);
      }
      int pos[NB][2];
      float slope[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          int token, head;
          row_of(p, row0, min(nb * 8 + 2 * t + c, x.rows - 1), x.hk, token, head);
          pos[nb][c] = seq.pos0 + token;
          slope[nb][c] = p.alibi ? paged_slope2(p, x.b, head) : 0.f;
        }
      // keys that every row of the block sees need no mask
      const int all_lo = p.win_left < 0 ? 0 : seq.pos0 + x.t1 - 1 - p.win_left;
      const int all_hi = p.win_right < 0 ? seq.len : min(seq.len, seq.pos0 + x.t0 + p.win_right + 1);

      float m[NB][2], l[NB][2], o[kSteps][NB][4];
      int vref = 16;  // R: the largest value exponent so far, or 16: 2^(R - 142) stays normal
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        m[nb][0] = m[nb][1] = -INFINITY;
        l[nb][0] = l[nb][1] = 0.f;
#pragma unroll
        for (int mb = 0; mb < kSteps; ++mb)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[mb][nb][i] = 0.f;
      }

      for (int tile = x.tile0 + ((group - static_cast<int>(tiles)) & (kGroups - 1));
           tile < x.tile1; tile += kGroups) {
        const uint32_t n = 2 * ((tiles + static_cast<uint32_t>(tile - x.tile0)) / kGroups);
        const int ks = group * kRing + n % kRing, vs = group * kRing + (n + 1) % kRing;
        const int k0 = tile * kTile + slice0;  // this warp's first key
        // -- S^T = K Q^T
        ring_wait(&s.full[ks], (n / kRing) & 1, p.err, abort_flag);
        __syncwarp();
        float acc[kSlices][NB][4];
        float kfac[kSlices][2];
#pragma unroll
        for (int sl = 0; sl < kSlices; ++sl) {
          // two independent chains of products per slice and eight queries
          float half[NB][4];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[sl][nb][i] = half[nb][i] = 0.f;
          auto step = [&](int kk, const uint32_t (&a)[4]) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              if (kk & 1)
                mma16816<kMmaBf16>(half[nb], a, qf[nb][kk][0], qf[nb][kk][1]);
              else
                mma16816<kMmaBf16>(acc[sl][nb], a, qf[nb][kk][0], qf[nb][kk][1]);
            }
          };
          if constexpr (!kFp8) {
            const uint32_t base = smem_u32(s.ring[ks]) + sl * 16 * 128;
#pragma unroll
            for (int kk = 0; kk < kSteps; ++kk) {
              uint32_t a[4];
              ldmatrix4(a, base + koff[kk & 3] + (kk >> 2) * kTile * 128);
              step(kk, a);
            }
          } else {
            const uint8_t* base = s.ring[ks] + sl * 16 * kRowBytes;
#pragma unroll
            for (int h = 0; h < kSteps / 4; ++h) {
              const uint4 lo = *reinterpret_cast<const uint4*>(base + koff[h]);
              const uint4 hi = *reinterpret_cast<const uint4*>(base + koff[h] + 8 * kRowBytes);
              const uint32_t lw[4] = {lo.x, lo.y, lo.z, lo.w}, hw[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const uint32_t a[4] = {e4m3x2_to_f16x2(lw[w]), e4m3x2_to_f16x2(hw[w]),
                                       e4m3x2_to_f16x2(lw[w] >> 16), e4m3x2_to_f16x2(hw[w] >> 16)};
                step(4 * h + w, a);
              }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)  // 2^(e - 127)
              kfac[sl][i] = __uint_as_float(
                  static_cast<uint32_t>(s.exps[ks][slice0 + sl * 16 + g + 8 * i]) << 23);
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[sl][nb][i] += half[nb][i];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.empty[ks]);

        if constexpr (kFp8) {
          // Rows marked as zeros (e = 0) are zeros whatever their codes, which may be
          // NaN: their products are those of a row of zero codes.  (Rows outside the
          // span, often such ones, are left alone here and below: at the end of every
          // sequence this code's own instructions would be fetched, 14 us of 110 in
          // the batch of 64 contexts; the look itself costs 1 to 2 us.)
          bool none = false;
#pragma unroll
          for (int sl = 0; sl < kSlices; ++sl)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int key = k0 + sl * 16 + g + 8 * i;
              none |= kfac[sl][i] == 0.f && key >= x.lo && key < x.hi;
            }
          if (__any_sync(0xffffffffu, none)) {
            const uint32_t a[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              float zero[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int kk = 0; kk < kSteps; ++kk)
                mma16816<kMmaBf16>(zero, a, qf[nb][kk][0], qf[nb][kk][1]);
#pragma unroll
              for (int sl = 0; sl < kSlices; ++sl)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (kfac[sl][i >> 1] == 0.f) acc[sl][nb][i] = zero[i];
            }
          }
        }

        // -- scores, maximum, weights
        const bool masked = k0 < all_lo || k0 + kSlices * 16 > all_hi;
        float alpha[NB][2];
        bool moved = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int sl = 0; sl < kSlices; ++sl)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              // (the powers of two first: beside small keys a query may be so large
              // that its product alone leaves the range)
              const float f =
                  kFp8 ? qscale[nb][i & 1] * kfac[sl][i >> 1] : qscale[nb][i & 1];
              acc[sl][nb][i] *= f;
            }
          if (p.alibi || masked) {
#pragma unroll
            for (int sl = 0; sl < kSlices; ++sl)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int c = i & 1, key = k0 + sl * 16 + g + (i >> 1) * 8;
                float z = acc[sl][nb][i];
                if (p.alibi)
                  z = fmaf(slope[nb][c], fabsf(static_cast<float>(key - pos[nb][c])), z);
                if (masked) {
                  const bool seen = key < seq.len &&
                                    (p.win_left < 0 || key >= pos[nb][c] - p.win_left) &&
                                    (p.win_right < 0 || key <= pos[nb][c] + p.win_right);
                  if (!seen) z = -INFINITY;
                }
                acc[sl][nb][i] = z;
              }
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float top = m[nb][c];
#pragma unroll
            for (int sl = 0; sl < kSlices; ++sl)
              top = fmax3(top, acc[sl][nb][c], acc[sl][nb][c + 2]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            alpha[nb][c] = top > m[nb][c] ? ex2_approx(m[nb][c] - top) : 1.f;
            moved |= top > m[nb][c];
            m[nb][c] = top;
            const float ref = top == -INFINITY ? 0.f : top - kLift;
            float sum = 0.f;
#pragma unroll
            for (int sl = 0; sl < kSlices; ++sl) {
              acc[sl][nb][c] = ex2_approx(acc[sl][nb][c] - ref);
              acc[sl][nb][c + 2] = ex2_approx(acc[sl][nb][c + 2] - ref);
              sum += acc[sl][nb][c] + acc[sl][nb][c + 2];
            }
            l[nb][c] = fmaf(l[nb][c], alpha[nb][c], sum);
          }
        }

        // -- O^T = O^T diag(alpha) + V^T P^T
        ring_wait(&s.full[vs], ((n + 1) / kRing) & 1, p.err, abort_flag);
        __syncwarp();
        const bool ragged = k0 < x.lo || k0 + kSlices * 16 > x.hi;
        if (ragged) {
          // rows outside the visible span hold anything: make them zeros
          for (int r = 0; r < kSlices * 16; ++r)
            if (k0 + r < x.lo || k0 + r >= x.hi)
              for (int i = lane; i < kRowBytes / 16; i += 32) {
                const int blk = i >> 3;  // 128-byte column blocks
                uint8_t* row = s.ring[vs] + blk * kTile * 128 +
                               (slice0 + r) * (kRowBytes < 128 ? kRowBytes : 128);
                *reinterpret_cast<uint4*>(row + (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
              }
          fence_proxy_async_smem();
          __syncwarp();
        }
        if constexpr (kFp8) {
          uint32_t e[kSlices][2], top = 0;
          bool none = false;
#pragma unroll
          for (int sl = 0; sl < kSlices; ++sl)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int key = k0 + sl * 16 + g + 8 * i;
              e[sl][i] = s.exps[vs][slice0 + sl * 16 + g + 8 * i];
              const bool outside = ragged && (key < x.lo || key >= x.hi);
              none |= e[sl][i] == 0 && !outside;
              if (outside) e[sl][i] = 0;
              top = max(top, e[sl][i]);
            }
          top = __reduce_max_sync(0xffffffffu, top);
          if (__any_sync(0xffffffffu, none)) {  // values marked as zeros
            for (int r = slice0; r < slice0 + kSlices * 16; ++r)
              if (s.exps[vs][r] == 0 && lane < kRowBytes / 16)
                *reinterpret_cast<uint4*>(s.ring[vs] + r * kRowBytes + lane * 16) =
                    make_uint4(0u, 0u, 0u, 0u);
            fence_proxy_async_smem();
            __syncwarp();
          }
          if (static_cast<int>(top) > vref) {
            const float down = exp2_field(127 + vref - static_cast<int>(top));
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              alpha[nb][0] *= down;
              alpha[nb][1] *= down;
            }
            moved = true;
            vref = static_cast<int>(top);
          }
#pragma unroll
          for (int sl = 0; sl < kSlices; ++sl)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float f =
                  e[sl][i] ? exp2_field(127 + 15 + static_cast<int>(e[sl][i]) - vref) : 0.f;
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                acc[sl][nb][2 * i] *= f;
                acc[sl][nb][2 * i + 1] *= f;
              }
            }
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int mb = 0; mb < kSteps; ++mb)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[mb][nb][i] *= alpha[nb][i & 1];
        }
#pragma unroll
        for (int sl = 0; sl < kSlices; ++sl) {
          uint32_t pf[NB][2];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              pf[nb][i] =
                  transpose8x8(pack2<kMmaBf16>(acc[sl][nb][2 * i], acc[sl][nb][2 * i + 1]));
          if constexpr (!kFp8) {
            const uint32_t base = smem_u32(s.ring[vs]) + sl * 16 * 128;
#pragma unroll
            for (int mb = 0; mb < kSteps; ++mb) {
              uint32_t a[4];
              ldmatrix4_trans(a, base + voff[mb & 3] + (mb >> 2) * kTile * 128);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
                mma16816<kMmaBf16>(o[mb][nb], a, pf[nb][0], pf[nb][1]);
            }
          } else {
            // keys 2t, 2t+1, 2t+8, 2t+9 of the slice, D / 8 columns each
            constexpr int kWords = D / 32;
            uint32_t v8[4][kWords];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint8_t* row =
                  s.ring[vs] + voff[i & 1] + (sl * 16 + (i >> 1) * 8) * kRowBytes;
              if constexpr (D == 128) {
                const uint4 v = *reinterpret_cast<const uint4*>(row);
                v8[i][0] = v.x;
                v8[i][1] = v.y;
                v8[i][kWords - 2] = v.z;
                v8[i][kWords - 1] = v.w;
              } else {
                const uint2 v = *reinterpret_cast<const uint2*>(row);
                v8[i][0] = v.x;
                v8[i][1] = v.y;
              }
            }
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
              const uint32_t x0 = __byte_perm(v8[0][w], v8[1][w], 0x5140),
                             x1 = __byte_perm(v8[0][w], v8[1][w], 0x7362),
                             y0 = __byte_perm(v8[2][w], v8[3][w], 0x5140),
                             y1 = __byte_perm(v8[2][w], v8[3][w], 0x7362);
              const uint32_t a0[4] = {e4m3x2_to_f16x2(x0), e4m3x2_to_f16x2(x0 >> 16),
                                      e4m3x2_to_f16x2(y0), e4m3x2_to_f16x2(y0 >> 16)};
              const uint32_t a1[4] = {e4m3x2_to_f16x2(x1), e4m3x2_to_f16x2(x1 >> 16),
                                      e4m3x2_to_f16x2(y1), e4m3x2_to_f16x2(y1 >> 16)};
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                mma16816<kMmaBf16>(o[2 * w][nb], a0, pf[nb][0], pf[nb][1]);
                mma16816<kMmaBf16>(o[2 * w + 1][nb], a1, pf[nb][0], pf[nb][1]);
              }
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.empty[vs]);
      }
      tiles += static_cast<uint32_t>(max(0, x.tile1 - x.tile0));

      // -- join the warps: row q of each group of eight is summed by warp q
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float sum = l[nb][c];
          sum += __shfl_xor_sync(0xffffffffu, sum, 4);
          sum += __shfl_xor_sync(0xffffffffu, sum, 8);
          sum += __shfl_xor_sync(0xffffffffu, sum, 16);
          if (g == 0) {
            s.m[warp][nb * 8 + 2 * t + c] = m[nb][c] - kLift;
            s.l[warp][nb * 8 + 2 * t + c] = sum;
          }
        }
      if (lane == 0) s.vref[warp] = vref;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const int r = nb * 8 + warp;
        constexpr int kN = D / 32;
        float top = -INFINITY, sum = 0.f, out[kN] = {};
        [[maybe_unused]] int vtop = 0;
#pragma unroll
        for (int gr = 0; gr < kGroups; ++gr) {
          if (group == gr)
#pragma unroll
            for (int mb = 0; mb < kSteps; ++mb)
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                float* row = s.merge[warp % kGroupWarps][2 * t + c];
                if constexpr (kFp8) {
                  *reinterpret_cast<float2*>(row + 2 * (10 * mb + g)) =
                      make_float2(o[mb][nb][c], o[mb][nb][c + 2]);
                } else {
                  row[16 * mb + g] = o[mb][nb][c];
                  row[16 * mb + g + 8] = o[mb][nb][c + 2];
                }
              }
          named_bar_sync(1, kConsumers * 32);
          if (gr == 0)
#pragma unroll
            for (int w = 0; w < kConsumers; ++w) {
              top = fmaxf(top, s.m[w][r]);
              if constexpr (kFp8) vtop = max(vtop, s.vref[w]);
            }
          const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
          for (int w = 0; w < kGroupWarps; ++w) {
            const int from = gr * kGroupWarps + w;
            const float a = ex2_approx(s.m[from][r] - ref);
            sum = fmaf(s.l[from][r], a, sum);
            const float av = kFp8 ? a * exp2_field(127 + s.vref[from] - vtop) : a;
            const float* src = s.merge[w][warp];
#pragma unroll
            for (int e = 0; e < kN; e += 2) {  // columns lane * kN + e and the next
              constexpr int kPairs = D / 16;   // of a lane group's columns
              const int pair = (lane * kN + e) / 2;
              const float2 v = *reinterpret_cast<const float2*>(
                  src + (kFp8 ? 2 * (10 * (pair % kPairs) + pair / kPairs) : 2 * pair));
              out[e] = fmaf(v.x, av, out[e]);
              out[e + 1] = fmaf(v.y, av, out[e + 1]);
            }
          }
          named_bar_sync(1, kConsumers * 32);
        }
        if constexpr (kFp8) {
          const float back = exp2_field(vtop - 15);
#pragma unroll
          for (int e = 0; e < kN; ++e) out[e] *= back;
        }
        if (r < x.rows) {
          if (x.whole) {
            int token, head;
            row_of(p, row0, r, x.hk, token, head);
            const long long row = seq.start + token;
            if (sum == 0.f) {  // no key: zeros, also where other rows saw a NaN value
#pragma unroll
              for (int e = 0; e < kN; ++e) out[e] = 0.f;
            }
            store16<kBf16>(static_cast<uint16_t*>(p.o) + row * p.o_token + head * p.o_head +
                               lane * kN,
                           out, sum == 0.f ? 0.f : 1.f / sum);
            if (lane == 0)
              p.lse[static_cast<long long>(head) * p.r.total + row] =
                  sum == 0.f ? -INFINITY : (top + lg2_approx(sum)) * kPagedLn2;
          } else {
            const long long at = (2LL * blockIdx.x + x.slot) * kRows + r;
            float* dst = p.part_o + at * D + lane * kN;
#pragma unroll
            for (int e = 0; e < kN; ++e) dst[e] = out[e];
            if (lane == 0) p.part_ml[at] = make_float2(top, sum);
          }
        }
      }
    }
  }
}

template <int D, bool kFp8, bool kBf16, int NB>
cudaError_t launch_few_t(const PagedLaunch& a, cudaStream_t s) {
  auto kern = paged_few_kernel<D, kFp8, kBf16, NB>;
  const int smem = static_cast<int>(sizeof(FewSmem<D, kFp8, NB>)) + 1024;
  static_assert(sizeof(FewSmem<D, kFp8, NB>) + 1024 <= 232448, "shared memory of one CTA");
  static AttrCache configured;
  cudaError_t e = ensure_dynamic_smem(kern, smem, configured);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, static_cast<unsigned>(a.sms), kFewThreads, smem, s, a);
  return e != cudaSuccess || a.whole ? e : launch_join<D, kBf16>(a, s);
}

template <int D, bool kFp8, bool kBf16>
cudaError_t launch_few_n(const PagedLaunch& a, cudaStream_t s) {
  return a.block_rows == 8 ? launch_few_t<D, kFp8, kBf16, 1>(a, s)
                           : launch_few_t<D, kFp8, kBf16, 2>(a, s);
}

template <int D>
cudaError_t launch_few_d(const PagedLaunch& a, cudaStream_t s) {
  const bool fp8 = a.cache_elem == kElemE4m3, bf16 = a.elem == kElemBf16;
  return fp8 ? (bf16 ? launch_few_n<D, true, true>(a, s)
                     : launch_few_n<D, true, false>(a, s))
             : (bf16 ? launch_few_n<D, false, true>(a, s)
                     : launch_few_n<D, false, false>(a, s));
}

}  // namespace

int paged_few_rows(double rows) { return rows <= 8 ? 8 : 16; }

cudaError_t launch_paged_few(const PagedLaunch& a, cudaStream_t s) {
  return a.D == 64 ? launch_few_d<64>(a, s) : launch_few_d<128>(a, s);
}

}  // namespace fa
