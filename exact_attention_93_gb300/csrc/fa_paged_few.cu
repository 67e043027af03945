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
// one producer warp keeps a ring of K and V tiles (128 keys each) in flight by
// TMA, page by page.
//
// Eight consumer warps share each tile, 16 keys each, with a running maximum,
// sum and O of their own that are joined once per piece of work: no barrier
// among them inside the key loop.  The products are turned around, S^T = K Q^T
// and O^T = V^T P^T, on mma.sync m16n8k16: keys and head columns fill the 16
// rows, so the padding of the query side is to 8 rows, and the operands go
// from shared memory to registers to the tensor core without a detour through
// tensor memory, which a tile of 8 columns would not fill.  P^T moves from the
// accumulator to the operand layout by an in-register 8 x 8 transpose.
//
// e4m3 caches.  Codes convert exactly to fp16 in registers, so an 8-bit cache
// costs half the HBM bytes and no precision beyond its own: q is scaled by a
// power of two per row to fit fp16, key exponents scale the scores in fp32,
// and value exponents go into P relative to the largest one seen so far, R:
// P' = 2^(s - m) * 2^(e_v - R + 15), at most 2^15.  The order of the head
// columns (keys) and of columns and keys (values) inside an operand is chosen
// so that a lane reads 16 contiguous bytes.
#include "fa_paged.cuh"
#include "fa_serve.h"
#include "sm103_primitives.cuh"

namespace fa {
namespace {

constexpr int kConsumers = 8;                        // warps
constexpr int kFewThreads = (kConsumers + 1) * 32;   // and the producer
constexpr int kSliceKeys = kTile / kConsumers;       // keys of a tile per warp
constexpr int kRingBytes = 160 * 1024;

template <int D, bool kFp8, int NB>
struct FewSmem {
  static constexpr int kRowBytes = kFp8 ? D : 2 * D;
  static constexpr int kSlotBytes = kTile * kRowBytes;
  static constexpr int kSlots = kRingBytes / kSlotBytes;  // K and V tiles alternate
  static constexpr int kMergePitch = D + 4;
  static constexpr int kSteps = D / 16;
  alignas(1024) uint8_t ring[kSlots][kSlotBytes];
  alignas(16) uint8_t exps[kFp8 ? kSlots : 1][kTile];
  // joining the warps' results, eight query rows at a time
  alignas(16) float merge[kConsumers][8][kMergePitch];
  float m[kConsumers][8 * NB], l[kConsumers][8 * NB];
  float vscale[kConsumers];
  // queries as operand fragments, where registers do not hold them
  uint2 q[NB >= 4 ? kSteps : 1][NB >= 4 ? NB : 1][32];
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
__global__ void __launch_bounds__(kFewThreads, 1)
    paged_few_kernel(const __grid_constant__ PagedLaunch p) {
  pdl_wait_and_release();
  using Smem = FewSmem<D, kFp8, NB>;
  constexpr int kRows = 8 * NB, kRowBytes = Smem::kRowBytes, kSlots = Smem::kSlots;
  constexpr int kSteps = Smem::kSteps;      // k16 steps over the head, and m16 blocks of V^T
  constexpr bool kMmaBf16 = kBf16 && !kFp8;  // type of the products
  constexpr bool kQRegs = NB < 4;
  // weights are kept as 2^(s - m + kLift): fp16 ones reach up to 2^15 and stay
  // normal down to 2^-29 of the largest (e4m3: see pfac)
  constexpr float kLift = !kFp8 && !kBf16 ? 15.f : 0.f;
  extern __shared__ uint8_t smem_raw[];
  Smem& s = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                     ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    const Place at = warp_place<false>(p, gridDim.x, blockIdx.x);
    if (lane == 0) {
      s.place = at;
      if (at.left == 0) p.tasks[blockIdx.x] = JoinTask{-1, 0, 0, 0, 0};
    }
  }
  if (threadIdx.x == 32) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], kConsumers);
    }
    s.abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
  volatile int* abort_flag = &s.abort_flag;
  WorkWalk<false> walk(s.place);
  Piece x;

  if (warp == kConsumers) {
    // ---------------------------------------------------------------- producer
    const int box_rows = min(p.page_size, kTile);
    const int per_tile = kTile / box_rows;
    if (lane == 0) {
      tma_prefetch_desc(&p.map_k);
      tma_prefetch_desc(&p.map_v);
    }
    uint32_t n = 0;  // slots filled
    while (walk.next(p, x)) {
      const int* table = p.r.table + x.b * p.r.table_stride;
      // lane i < per_tile: the i-th box of a tile, if a visible key lies in it
      auto page_of = [&](int tile) {
        const int k0 = tile * kTile + lane * box_rows;
        const bool wanted = lane < per_tile && tile < x.tile1 && k0 < x.hi && k0 + box_rows > x.lo;
        return wanted ? table[k0 >> p.page_log2] : -2;
      };
      int page = page_of(x.tile0);
      for (int tile = x.tile0; tile < x.tile1; ++tile) {
        const int k0 = tile * kTile + lane * box_rows;
        const bool mine = lane < per_tile && k0 < x.hi && k0 + box_rows > x.lo;
        const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, mine));
        const int next_page = page_of(tile + 1);
        if (mine && (page < 0 || page >= p.pages)) {
          atomicExch(p.err, kDevErrBadIndex);
          page = p.pages;  // out of range for the tensor map: reads as zeros
        }
        const int row = k0 & (p.page_size - 1);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv, ++n) {
          const int slot = n % kSlots;
          if (n >= kSlots) ring_wait(&s.empty[slot], (n / kSlots - 1) & 1, p.err, abort_flag);
          if (__any_sync(0xffffffffu, *abort_flag)) goto stopped;
          if (lane == 0)
            mbar_arrive_expect_tx(&s.full[slot],
                                  boxes * box_rows * (kRowBytes + (kFp8 ? 1 : 0)));
          __syncwarp();
          if (mine) {
            uint8_t* dst = s.ring[slot] + lane * box_rows * (kRowBytes < 128 ? kRowBytes : 128);
#pragma unroll
            for (int kb = 0; kb < (kRowBytes + 127) / 128; ++kb)
              tma_load_4d(dst + kb * kTile * 128, kv ? &p.map_v : &p.map_k, &s.full[slot],
                          kb * 64, row, x.hk, page);
            if constexpr (kFp8) {
              // (of a page that does not exist, any exponents will do)
              const uint8_t* e = (kv ? p.v_exp : p.k_exp) +
                                 (static_cast<long long>(page < p.pages ? page : 0) * p.heads_k +
                                  x.hk) * p.page_size + row;
              bulk_load(s.exps[slot] + lane * box_rows, e, box_rows, &s.full[slot]);
            }
          }
        }
        page = next_page;
      }
    }
  stopped:
    if (*abort_flag) {
      // Copies in flight land before the CTA's shared memory goes away.
      int zero = 0;
      if (lane == 0)
        for (uint32_t i = n > kSlots ? n - kSlots : 0; i < n; ++i)
          mbar_wait(&s.full[i % kSlots], (i / kSlots) & 1, p.err, &zero, 100000000ull);
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------------- consumers
    const int g = lane >> 2, t = lane & 3;
    uint32_t n = 0;  // slots consumed
    while (walk.next(p, x)) {
      const Seq& seq = walk.w.s;
      const int row0 = x.block * kRows;
      if (threadIdx.x == 0) p.tasks[blockIdx.x] = join_task(p, x, seq);
      // -- queries as B operands, and what each of this lane's columns sees
      uint32_t qf[kQRegs ? NB : 1][kSteps][2];
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
                                        src + (kk >> 2) * 64 + 16 * t + 4 * (kk & 3)))
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
            if constexpr (kQRegs) {
              qf[nb][kk][0] = f[kk][0];
              qf[nb][kk][1] = f[kk][1];
            } else if (kk % kConsumers == warp) {
              s.q[kk][nb][lane] = make_uint2(f[kk][0], f[kk][1]);
            }
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int c = 0; c < 2; ++c)  // from the lanes of row 8 nb + 2 t + c
            qscale[nb][c] =
                p.scale_log2 * __shfl_sync(0xffffffffu, mine[nb], (2 * t + c) * 4);
        if constexpr (!kQRegs) named_bar_sync(1, kConsumers * 32);
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
      int vref = 0;  // R: the largest value exponent so far
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        m[nb][0] = m[nb][1] = -INFINITY;
        l[nb][0] = l[nb][1] = 0.f;
#pragma unroll
        for (int mb = 0; mb < kSteps; ++mb)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[mb][nb][i] = 0.f;
      }

      for (int tile = x.tile0; tile < x.tile1; ++tile, n += 2) {
        const int ks = n % kSlots, vs = (n + 1) % kSlots;
        const int k0 = tile * kTile + warp * kSliceKeys;  // this warp's keys k0 .. k0 + 15
        // -- S^T = K Q^T
        ring_wait(&s.full[ks], (n / kSlots) & 1, p.err, abort_flag);
        __syncwarp();
        float acc[NB][4];
        {
          float half[4] = {0.f, 0.f, 0.f, 0.f};  // NB = 1: a second, independent chain
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[nb][i] = 0.f;
          auto step = [&](int kk, const uint32_t (&a)[4]) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              uint32_t b0, b1;
              if constexpr (kQRegs) {
                b0 = qf[nb][kk][0];
                b1 = qf[nb][kk][1];
              } else {
                const uint2 v = s.q[kk][nb][lane];
                b0 = v.x;
                b1 = v.y;
              }
              if (NB == 1 && (kk & 1))
                mma16816<kMmaBf16>(half, a, b0, b1);
              else
                mma16816<kMmaBf16>(acc[nb], a, b0, b1);
            }
          };
          if constexpr (!kFp8) {
            const int r = warp * kSliceKeys + (lane & 15);
            const uint32_t base = smem_u32(s.ring[ks]) + r * 128;
#pragma unroll
            for (int kk = 0; kk < kSteps; ++kk) {
              const int chunk = (kk & 3) * 2 + (lane >> 4);
              uint32_t a[4];
              ldmatrix4(a, base + (kk >> 2) * kTile * 128 + ((chunk ^ (r & 7)) << 4));
              step(kk, a);
            }
          } else {
            // rows g and g + 8 of the slice, 16 bytes per 64 columns
            constexpr int kHalves = D / 64;
            uint4 k8[2][kHalves];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int r = warp * kSliceKeys + g + 8 * i;
              const uint8_t* row = s.ring[ks] + r * kRowBytes;
              if constexpr (D == 128) {
                // odd rows take their halves in the other order (the swizzle
                // would put both rows' 64 bytes on the same banks)
                const uint4 u = *reinterpret_cast<const uint4*>(
                    row + (((t + ((g & 1) << 2)) ^ (r & 7)) << 4));
                const uint4 v = *reinterpret_cast<const uint4*>(
                    row + (((t + (((g & 1) ^ 1) << 2)) ^ (r & 7)) << 4));
                k8[i][0] = (g & 1) ? v : u;
                k8[i][kHalves - 1] = (g & 1) ? u : v;
              } else {
                k8[i][0] = *reinterpret_cast<const uint4*>(row + ((t ^ ((r >> 1) & 3)) << 4));
              }
            }
#pragma unroll
            for (int kk = 0; kk < kSteps; ++kk) {
              const uint4 &lo = k8[0][kk >> 2], &hi = k8[1][kk >> 2];
              const uint32_t w0 = (kk & 3) == 0 ? lo.x : (kk & 3) == 1 ? lo.y
                                  : (kk & 3) == 2 ? lo.z : lo.w;
              const uint32_t w1 = (kk & 3) == 0 ? hi.x : (kk & 3) == 1 ? hi.y
                                  : (kk & 3) == 2 ? hi.z : hi.w;
              const uint32_t a[4] = {e4m3x2_to_f16x2(w0), e4m3x2_to_f16x2(w1),
                                     e4m3x2_to_f16x2(w0 >> 16), e4m3x2_to_f16x2(w1 >> 16)};
              step(kk, a);
            }
          }
          if (NB == 1)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[0][i] += half[i];
        }
        float kfac[2] = {1.f, 1.f};
        if constexpr (kFp8) {
          kfac[0] = exp2_field(s.exps[ks][warp * kSliceKeys + g]);
          kfac[1] = exp2_field(s.exps[ks][warp * kSliceKeys + g + 8]);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.empty[ks]);

        // -- scores, maximum, weights
        const bool masked = k0 < all_lo || k0 + kSliceKeys > all_hi;
        float alpha[NB][2];
        bool moved = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = i & 1, key = k0 + g + (i >> 1) * 8;
            float z = acc[nb][i] * (kFp8 ? qscale[nb][c] * kfac[i >> 1] : qscale[nb][c]);
            if (p.alibi)
              z = fmaf(slope[nb][c], fabsf(static_cast<float>(key - pos[nb][c])), z);
            if (masked) {
              const bool seen = key < seq.len && (p.win_left < 0 || key >= pos[nb][c] - p.win_left) &&
                                (p.win_right < 0 || key <= pos[nb][c] + p.win_right);
              if (!seen) z = -INFINITY;
            }
            acc[nb][i] = z;
          }
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float top = fmaxf(acc[nb][c], acc[nb][c + 2]);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
            const float m_new = fmaxf(m[nb][c], top);
            alpha[nb][c] = m_new > m[nb][c] ? ex2_approx(m[nb][c] - m_new) : 1.f;
            moved |= m_new > m[nb][c];
            m[nb][c] = m_new;
            const float ref = m_new == -INFINITY ? 0.f : m_new - kLift;
            acc[nb][c] = ex2_approx(acc[nb][c] - ref);
            acc[nb][c + 2] = ex2_approx(acc[nb][c + 2] - ref);
            l[nb][c] = fmaf(l[nb][c], alpha[nb][c], acc[nb][c] + acc[nb][c + 2]);
          }
        }

        // -- O^T = O^T diag(alpha) + V^T P^T
        ring_wait(&s.full[vs], ((n + 1) / kSlots) & 1, p.err, abort_flag);
        __syncwarp();
        const bool ragged = k0 < x.lo || k0 + kSliceKeys > x.hi;
        if (ragged) {
          // rows outside the visible span hold anything: make them zeros
          for (int r = 0; r < kSliceKeys; ++r)
            if (k0 + r < x.lo || k0 + r >= x.hi)
              for (int i = lane; i < kRowBytes / 16; i += 32) {
                const int blk = i >> 3;  // 128-byte column blocks
                uint8_t* row = s.ring[vs] + blk * kTile * 128 +
                               (warp * kSliceKeys + r) * (kRowBytes < 128 ? kRowBytes : 128);
                *reinterpret_cast<uint4*>(row + (i & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
              }
          fence_proxy_async_smem();
          __syncwarp();
        }
        float pfac[2] = {1.f, 1.f};
        if constexpr (kFp8) {
          int e[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int key = k0 + g + 8 * i;
            e[i] = key >= x.lo && key < x.hi ? s.exps[vs][warp * kSliceKeys + g + 8 * i] : 0;
          }
          int top = max(e[0], e[1]);
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 4));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 8));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));
          if (top > vref) {
            const float down = exp2_field(127 + vref - top);
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) {
              alpha[nb][0] *= down;
              alpha[nb][1] *= down;
            }
            moved = true;
            vref = top;
          }
          pfac[0] = e[0] ? exp2_field(127 + e[0] - vref + 15) : 0.f;
          pfac[1] = e[1] ? exp2_field(127 + e[1] - vref + 15) : 0.f;
        }
        if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
          for (int mb = 0; mb < kSteps; ++mb)
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
#pragma unroll
              for (int i = 0; i < 4; ++i) o[mb][nb][i] *= alpha[nb][i & 1];
        }
        uint32_t pf[NB][2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            pf[nb][i] = transpose8x8(
                pack2<kMmaBf16>(kFp8 ? acc[nb][2 * i] * pfac[i] : acc[nb][2 * i],
                                kFp8 ? acc[nb][2 * i + 1] * pfac[i] : acc[nb][2 * i + 1]));
        if constexpr (!kFp8) {
          const int r = warp * kSliceKeys + (lane >> 4) * 8 + (lane & 7);
          const uint32_t base = smem_u32(s.ring[vs]) + r * 128;
#pragma unroll
          for (int mb = 0; mb < kSteps; ++mb) {
            const int chunk = (mb & 3) * 2 + ((lane >> 3) & 1);
            uint32_t a[4];
            ldmatrix4_trans(a, base + (mb >> 2) * kTile * 128 + ((chunk ^ (r & 7)) << 4));
#pragma unroll
            for (int nb = 0; nb < NB; ++nb) mma16816<kMmaBf16>(o[mb][nb], a, pf[nb][0], pf[nb][1]);
          }
        } else {
          // keys 2t, 2t+1, 2t+8, 2t+9 of the slice, D / 8 columns each
          constexpr int kWords = D / 32;
          uint32_t v8[4][kWords];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int r = warp * kSliceKeys + 2 * t + (i & 1) + (i >> 1) * 8;
            const uint8_t* row = s.ring[vs] + r * kRowBytes;
            if constexpr (D == 128) {
              const uint4 v = *reinterpret_cast<const uint4*>(row + ((g ^ (r & 7)) << 4));
              v8[i][0] = v.x;
              v8[i][1] = v.y;
              v8[i][kWords - 2] = v.z;
              v8[i][kWords - 1] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(
                  row + (((g >> 1) ^ ((r >> 1) & 3)) << 4) + (g & 1) * 8);
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
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.empty[vs]);
      }

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
      if (lane == 0) s.vscale[warp] = kFp8 ? exp2_field(vref - 15) : 1.f;
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
        for (int mb = 0; mb < kSteps; ++mb)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            // 16-bit: column 16 mb + g (+ 8); e4m3: column (D / 8) g + 2 mb (+ 1)
            const int d = kFp8 ? (D / 8) * g + 2 * mb + (i >> 1) : 16 * mb + g + 8 * (i >> 1);
            s.merge[warp][2 * t + (i & 1)][d] = o[mb][nb][i];
          }
        named_bar_sync(1, kConsumers * 32);
        const int r = nb * 8 + warp;
        if (r < x.rows) {
          float top = -INFINITY;
#pragma unroll
          for (int w = 0; w < kConsumers; ++w) top = fmaxf(top, s.m[w][r]);
          const float ref = top == -INFINITY ? 0.f : top;
          constexpr int kN = D / 32;
          float sum = 0.f, out[kN] = {};
#pragma unroll
          for (int w = 0; w < kConsumers; ++w) {
            const float a = ex2_approx(s.m[w][r] - ref);
            sum = fmaf(s.l[w][r], a, sum);
            const float av = kFp8 ? a * s.vscale[w] : a;
            const float* src = &s.merge[w][warp][lane * kN];
#pragma unroll
            for (int e = 0; e < kN; ++e) out[e] = fmaf(src[e], av, out[e]);
          }
          if (x.whole) {
            int token, head;
            row_of(p, row0, r, x.hk, token, head);
            const long long row = seq.start + token;
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
        named_bar_sync(1, kConsumers * 32);
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
  return a.block_rows == 8    ? launch_few_t<D, kFp8, kBf16, 1>(a, s)
         : a.block_rows == 16 ? launch_few_t<D, kFp8, kBf16, 2>(a, s)
                            : launch_few_t<D, kFp8, kBf16, 4>(a, s);
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

int paged_few_rows(long long rows, int batch) {
  return rows <= 8LL * batch ? 8 : rows <= 16LL * batch ? 16 : 32;
}

cudaError_t launch_paged_few(const PagedLaunch& a, cudaStream_t s) {
  return a.D == 64 ? launch_few_d<64>(a, s) : launch_few_d<128>(a, s);
}

}  // namespace fa
