// Input gradient of a packed projection on the 5th-generation tensor cores:
//   dx[m][k] = add[m][k] + sum_n dy[m][n] w[n][k],   w[n][k] = sw[n][k / 128] q[n][k].
//
// The contraction runs over the output features n, whose scales differ from row
// to row, so a scale cannot be taken out of the sum: the packed codes are
// dequantized on chip and the products run in bf16 with fp32 accumulation.
// dy is bf16 already.  w, 18 bits, enters as T bf16 terms:
//   T = 1  rounded once, 2^-8 relative at most and independent from row to row, so about
//          the error that the rounding of a bf16 dx adds (2.35e-3 of the norm for
//          1.66e-3).  What a bf16 dx takes.
//   T = 3  hi + mid + lo = w exactly, each term a step of its own over the same codes and
//          dY, and sums of 512 rows n at a time are added to an fp32 dx in its own memory
//          (tensor memory rounds every addition towards zero: 1.3e-6 of the norm with 512
//          rows, 9.6e-6 with 4096; a bf16 dx is summed there throughout).  What an fp32 dx
//          takes, at three times the products and more of the conversion (2048 tokens x
//          1280 k x 9728 n: 325 us for 50).
// The caller may choose either for either dx.
//
// A work unit is (128 columns k: one tile column; NT tokens; a range of n).  Per
// step of 64 rows n:
//   D[128 k][NT tokens] += W'[64 n][128 k]^T dY[NT tokens][64 n]^T
// with W' as the A operand, MN-major, so that the codes keep the packed order
// (k contiguous) and no transposition is needed, and dY as the B operand,
// K-major as it lies in memory.  Long sequences run in pairs of CTAs (cta_group::2),
// a tile column each and half of the tokens' dY, which both use.
//
// Roles in one CTA (persistent over work units, every role walks the same
// sequence of steps g = 0, 1, 2, ...):
//   warp 0       weight producer: labels and tile indices of 32 steps at a time,
//                one step per lane, the next 32 in flight; codes (TMA) and the 64
//                row scales (bulk copy) into the raw ring
//   warp 1       allocates tensor memory; issues tcgen05.mma (kind::f16, K = 16) four times
//                per step and 256 tokens, in a pair for both CTAs
//   warp 3       dY producer (TMA, 128-byte swizzle), after the previous kernel
//   warps 4-     transform: codes -> sw q in bf16 -> the swizzled A slot, in two or three
//                groups of four warps that take steps in turn (one step's chain of waits and
//                latencies, 1000 cycles, is longer than its MMAs, 512 for 256 tokens)
//   the rest     epilogue: tensor memory -> add -> dx, while the next unit runs in
//                the other accumulator buffer; units of 384 or 512 tokens take both, and
//                have a group of four warps for each
// The weights are read before the previous kernel has finished; dY, add, dx and
// the workspace are not touched before.
//
// What bounds it: the transform with 256 tokens a unit (step 810 cycles), the tensor pipe
// with 512 (step 1100 of 1024 cycles; each dequantized tile serves twice the products), and
// for long calls the power.  The kernels' own times, in graphs with the form forced (calls take
// 780 and 100 us): 8192 tokens x 14336 k x 4096 n 1010 us in single CTAs, 910 in pairs with 256
// tokens and 740 with 512 (1.3 PFLOP/s; a library product sustains 1.38); 2048 x 2560 x 9728 101,
// 95 and 84; 2048 x 9728 x 2560 102, 92 and 98, and 87 with 384.
//
// Whole units go to the CTAs as long as every CTA gets one; the units that are left
// (all of them for short sequences) may be split over n so that they fill the GPU once
// more, their partial sums go to the workspace, and a second launch adds them in
// split order.  (Summed by the unit's
// last CTA instead, 77 x 2560 x 1088 took 60 us: one CTA's loads wait for one
// another, a grid's do not.)
// Every wait is bounded, as in tc_linear_kernel.
#include <algorithm>
#include <cstring>

#include "aq_internal.cuh"
#include "tc_bf16.cuh"

namespace aq {
namespace {

constexpr int kStep = 64;       // rows n per step
constexpr int kRawBytes = kStep * kTileK + 256;  // INT8 codes, then 64 fp16 scales
constexpr int kXfWarp0 = 4, kXfWarps = 4, kXfThreads = 32 * kXfWarps;  // groups of four warps
constexpr int kEpiWarps = 4;
constexpr int kMaxBwdSplits = 16;
constexpr int kSumRows = 512;   // rows n summed in tensor memory for an exact fp32 dx

template <int NT, int CG>
struct BwdShape {
  static constexpr int kHalves = NT > 256 ? 2 : 1, kN = NT / kHalves;  // products of a step, their N
  static constexpr int kXfGroups = CG == 2 && kHalves == 1 ? 3 : 2, kEpiWarp0 = kXfWarp0 + kXfGroups * kXfWarps;
  static constexpr int kThreads = 32 * (kEpiWarp0 + kEpiWarps * kHalves);
  static constexpr int kA = kStep * kTileK * 2;  // W' slot: two 64-column halves of 64 rows x 128 bytes
  static constexpr int kB = NT / CG * kStep * 2;  // dY slot: this CTA's rows x 128 bytes
  // Rings of W', dY and packed codes.  Copies take 1 to 1.5 us to land, as long as two
  // to four steps: codes and dY each need that many slots on their way.
  static constexpr int kSA = NT / CG <= 128 ? 4 : 3, kSB = NT / CG <= 128 ? 6 : 4, kRaw = NT / CG <= 128 ? 7 : 6;
  static constexpr int kTmemCols = 2 * kN <= 64 ? 64 : 2 * kN <= 128 ? 128 : 2 * kN <= 256 ? 256 : 512;  // two accumulators
  static constexpr int kCtrl = 512;
  static constexpr int kSmem = 1024 + kSA * kA + kSB * kB + kRaw * kRawBytes + kCtrl;
  static constexpr uint32_t kIdesc = idesc_bf16(kN, true, false, 128 * CG);
  static_assert(kN % 16 == 0 && kN >= 32 && kN <= 256, "MMA N");
  static_assert(kSmem <= 227 * 1024, "shared memory");
  // A parity says which of two phases is over, so a waiter must know the one before to be
  // over.  A group that turns to step i has seen the MMAs of step i - kXfGroups - kSA
  // complete; that has to cover the last but one use of its slots.
  static_assert(kXfGroups <= kSA && kXfGroups + kSA <= kRaw, "phases");
  static_assert((2 * kRaw + 2 * kSA + 2 * kSB + 4 + 1) * 8 + kRaw * 4 + 3 * 4 <= kCtrl, "control area");
};

struct BwdMaps {
  CUtensorMap w8, w4, dy;
};

struct BwdArgs {
  const uint8_t* bitmap;
  const int32_t* tile_idx;
  const uint16_t* scales;
  int N, K, bN, C, T4, T8;
  int M, ntb, steps;   // steps of a unit: T times N / 64
  int chunk;           // steps summed in tensor memory (T = 3)
  int whole, S, units;  // units done whole, splits of the others, work items in all
  const void* add;
  void* dx;
  int ldadd, lddx, f32;
  void* ws;
  float* partial;  // [split work item][NT][128]
  Stall stall;     // (of a pair, the second CTA's weight producer stops)
};

struct BwdUnit {
  int kb, tb, i0, i1;  // kb: with pairs, of two tile columns
  int part;  // index among the split work items, or -1
};

__device__ __forceinline__ BwdUnit bwd_unit(const BwdArgs& a, int u) {
  BwdUnit x;
  x.part = u - a.whole;
  x.i0 = 0;
  x.i1 = a.steps;
  if (x.part >= 0) {
    const int s = x.part % a.S;
    u = a.whole + x.part / a.S;
    x.i0 = (int)((long long)a.steps * s / a.S);
    x.i1 = (int)((long long)a.steps * (s + 1) / a.S);
  }
  x.tb = u % a.ntb;
  x.kb = u / a.ntb;
  return x;
}

// ---- two CTAs on one tile: the leader (rank 0) issues the products of both
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t lead_addr(const void* p) {  // the same place in the leader's shared memory
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
  return r;
}
__device__ __forceinline__ void tmem_alloc2(uint32_t* slot_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot_smem)), "r"(ncols)
               : "memory");
}
__device__ __forceinline__ void tmem_relinquish2() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc2(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols) : "memory");
}
// Load into this CTA's memory that completes on the leader's barrier.
__device__ __forceinline__ void tma_load_2d_lead(void* dst, const CUtensorMap* map, int x, int y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
      "[%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(lead_addr(bar))
      : "memory");
}
// Arrive at the leader's barrier.  Its products read tiles that this CTA wrote into its own
// memory, so what came before is released at cluster scope; only for shared memory, which is all
// that the leader reads.  (With a release of all memory each step waited for the copies and stores
// under way: 8192 x 14336 x 4096 took 820 us for 677.)
template <int CG>
__device__ __forceinline__ void arrive_lead(uint64_t* bar) {
  if constexpr (CG == 1)
    mbar_arrive(bar);
  else
    asm volatile(
        "fence.release.sync_restrict::shared::cta.cluster;\n\t"
        "mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(lead_addr(bar))
        : "memory");
}
// The leader's mbar_wait on what the other CTA of the pair arrives at or its copies complete:
// acquires at cluster scope.
template <int CG>
__device__ __forceinline__ bool pair_wait(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned long long limit_ns) {
  if constexpr (CG == 1) return mbar_wait(bar, parity, abort, limit_ns);
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  if (ok) return true;
  const unsigned long long t0 = globaltimer_ns();
  for (;;) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "r"(kWaitSuspendNs)
        : "memory");
    if (ok) return true;
    if (*abort || globaltimer_ns() - t0 > limit_ns) return false;
  }
}
// Arrive at the barriers of both CTAs when every MMA issued so far is done.
template <int CG>
__device__ __forceinline__ void mma_commit_all(uint64_t* bar) {
  if constexpr (CG == 1)
    mma_commit(bar);
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// What the bf16 value of v leaves, exactly.
__device__ __forceinline__ float2 bf16_rest(float2 v) {
  const __nv_bfloat162 b = __floats2bfloat162_rn(v.x, v.y);
  const uint32_t w = *reinterpret_cast<const uint32_t*>(&b) ^ 0x80008000u;  // - b
  return __fadd2_rn(v, make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)));
}

// Four codes (two's-complement bytes) times sw, as two bf16 pairs.  The byte
// b = q + 128 in the middle of a mantissa is 32768 + b, and 32896 sw is exact (9 + 11
// bits), so one fused multiply-add gives sw q exactly.
__device__ __forceinline__ void codes4(uint32_t w, float2 sw, float2 off, float2& p, float2& q) {
  const uint32_t x = w ^ 0x80808080u;
  p = __ffma2_rn(make_float2(__uint_as_float(__byte_perm(x, 0x47000000u, 0x7604)),
                                    __uint_as_float(__byte_perm(x, 0x47000000u, 0x7614))), sw, off);
  q = __ffma2_rn(make_float2(__uint_as_float(__byte_perm(x, 0x47000000u, 0x7624)),
                                    __uint_as_float(__byte_perm(x, 0x47000000u, 0x7634))), sw, off);
}
__device__ __forceinline__ uint2 round4(float2 p, float2 q) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(p.x, p.y), b = __floats2bfloat162_rn(q.x, q.y);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

template <int NT, int CG, int T>
__global__ void __launch_bounds__(BwdShape<NT, CG>::kThreads, 1)
    linear_backward_kernel(const __grid_constant__ BwdMaps maps, const __grid_constant__ BwdArgs a) {
  using Sh = BwdShape<NT, CG>;
  constexpr int SA = Sh::kSA, SB = Sh::kSB, RW = Sh::kRaw, H = Sh::kHalves;
  static_assert(T == 1 || H == 1, "sums of part of a unit alternate between two accumulators");
  constexpr int kXfGroups = Sh::kXfGroups, kEpiWarp0 = Sh::kEpiWarp0;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  auto stage_a = [&](int i) { return smem + i * Sh::kA; };
  auto stage_b = [&](int i) { return smem + SA * Sh::kA + i * Sh::kB; };
  auto raw_slot = [&](int i) { return smem + SA * Sh::kA + SB * Sh::kB + i * kRawBytes; };
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(raw_slot(RW));
  uint64_t* raw_empty = raw_full + RW;
  uint64_t* a_full = raw_empty + RW;   // transform warps done with the slot
  uint64_t* a_done = a_full + SA;      // the slot's MMAs are complete
  uint64_t* b_full = a_done + SA;      // dY landed
  uint64_t* b_done = b_full + SB;
  uint64_t* acc_full = b_done + SB;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  volatile uint32_t* raw_int4 = reinterpret_cast<volatile uint32_t*>(drain + 1);
  uint32_t* tmem_slot = const_cast<uint32_t*>(raw_int4 + RW);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* never_flag = abort_flag + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = CG == 1 ? 0 : blockIdx.x & 1, first_unit = blockIdx.x / CG, stride = gridDim.x / CG;
  if (threadIdx.x == 0) {
    for (int i = 0; i < RW; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], kXfWarps);
    }
    for (int i = 0; i < SA; ++i) {
      mbar_init(&a_full[i], kXfWarps * CG);
      mbar_init(&a_done[i], 1);
    }
    for (int i = 0; i < SB; ++i) {
      mbar_init(&b_full[i], 1);
      mbar_init(&b_done[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], kEpiWarps * CG);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *never_flag = 0;
    fence_mbar_init();
    if (a.T8 > 0) prefetch_tmap(&maps.w8);
    if (a.T4 > 0) prefetch_tmap(&maps.w4);
    prefetch_tmap(&maps.dy);
  }
  if (warp == 1) {
    if constexpr (CG == 1) {
      tmem_alloc(tmem_slot, Sh::kTmemCols);
      tmem_relinquish();
    } else {
      tmem_alloc2(tmem_slot, Sh::kTmemCols);
      tmem_relinquish2();
    }
  }
  tc_fence_before();
  __syncthreads();
  if (CG == 2) cluster_sync();  // the other's barriers are set up
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_launch_dependents();

  auto fail = [&](int info) {
    *abort_flag = 1;
    record_error(a.ws, AQ_ERR_TIMEOUT, info, 0);
  };

  if (warp == 0) {
    // ------------------------------------------------------------ weight producer
    int u = first_unit;  // unit that holds this lane's next step, and the step it starts at
    uint32_t base = 0, g = lane;
    BwdUnit x = bwd_unit(a, u);
    // first row in its precision's buffer, offset of the scales, INT4 label: 2 = past the end
    auto fetch = [&](uint32_t& row, uint32_t& sc, uint32_t& kind) {
      while (u < a.units && g >= base + (uint32_t)(x.i1 - x.i0)) {
        base += x.i1 - x.i0;
        u += stride;
        if (u < a.units) x = bwd_unit(a, u);
      }
      kind = 2;
      row = sc = 0;
      if (u < a.units) {
        const int n0 = (x.i0 + (int)(g - base)) / T * kStep, r = n0 / a.bN, in = n0 - r * a.bN;
        const int t = r * a.C + x.kb * CG + rank;
        kind = __ldg(a.bitmap + (t >> 3)) >> (t & 7) & 1;
        row = (uint32_t)__ldg(a.tile_idx + t) * a.bN + in;
        sc = (uint32_t)t * a.bN + in;
      }
      g += 32;
    };
    uint32_t row[2], sc[2], kind[2];
    fetch(row[0], sc[0], kind[0]);
    Ring rr{0, 0};
    bool more = true, ok = true;
    int steps = 0;
    while (more && ok) {
      fetch(row[1], sc[1], kind[1]);
      for (int i = 0; i < 32 && ok; ++i) {
        const uint32_t k = __shfl_sync(0xffffffffu, kind[0], i), r = __shfl_sync(0xffffffffu, row[0], i),
                       s = __shfl_sync(0xffffffffu, sc[0], i);
        if (k == 2) {
          more = false;
          break;
        }
        if (a.stall.stop_after >= 0 && rank == CG - 1 && steps++ == a.stall.stop_after) {
          stalled(abort_flag, a.stall.wait_ns);
          ok = false;
          break;
        }
        if (!__all_sync(0xffffffffu, lane != 0 || mbar_wait(&raw_empty[rr.i], rr.ph ^ 1u, abort_flag, a.stall.wait_ns))) {
          fail(1);
          ok = false;
        } else if (lane == 0) {
          raw_int4[rr.i] = k;
          uint8_t* dst = raw_slot(rr.i);
          mbar_arrive_expect_tx(&raw_full[rr.i], (k ? kStep * kTileK / 2 : kStep * kTileK) + kStep * 2);
          tma_load_2d(dst, k ? &maps.w4 : &maps.w8, 0, (int)r, &raw_full[rr.i]);
          bulk_load(dst + kStep * kTileK, a.scales + s, kStep * 2, &raw_full[rr.i]);
        }
        rr.template next<RW>();
      }
      row[0] = row[1];
      sc[0] = sc[1];
      kind[0] = kind[1];
    }
    if (lane == 0 && (!ok || *abort_flag)) grace();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (rank == 0) {
      const uint64_t adesc0 = mn_desc(smem_u32(stage_a(0)), kStep * 128), bdesc0 = sw128_desc(smem_u32(stage_b(0)));
      const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
      Ring sr{0, 0}, br{0, 0}, ar{0, 0};
      bool ok = true, any = false;
      for (int u = first_unit; ok && u < a.units; u += stride) {
        const BwdUnit x = bwd_unit(a, u);
        int left = 0;  // steps of the sum that is being formed
        for (int i = x.i0; ok && i < x.i1; ++i) {
          const bool first = T == 1 ? i == x.i0 : left == 0;
          if (T > 1) left = (left == 0 ? min(a.chunk, x.i1 - i) : left) - 1;
          const bool last = T == 1 ? i + 1 == x.i1 : left == 0;
          if (!__all_sync(0xffffffffu, pair_wait<CG>(&b_full[br.i], br.ph, abort_flag, a.stall.wait_ns) &&
                                           pair_wait<CG>(&a_full[sr.i], sr.ph, abort_flag, a.stall.wait_ns))) {
            fail(3);
            ok = false;
            break;
          }
#pragma unroll
          for (int h = 0; h < H; ++h) {
            const int buf = H == 2 ? h : ar.i;
            if (first && !__all_sync(0xffffffffu, pair_wait<CG>(&acc_empty[buf], ar.ph ^ 1u, abort_flag, a.stall.wait_ns))) {
              fail(2);
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t d = tmem + buf * Sh::kN;
            const uint64_t ao = adesc0 + (uint64_t)((sr.i * Sh::kA) >> 4),
                           bo = bdesc0 + (uint64_t)((br.i * Sh::kB + h * (Sh::kB / H)) >> 4);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < kStep / 16; ++k)  // 16 rows: two groups of A, 32 bytes of B
                mma_bf16<CG>(d, ao + 128 * k, bo + 2 * k, Sh::kIdesc, !first || k > 0);
              if (h == H - 1) {
                mma_commit_all<CG>(&a_done[sr.i]);
                mma_commit_all<CG>(&b_done[br.i]);
              }
              if (last) mma_commit_all<CG>(&acc_full[buf]);
            }
            __syncwarp();
            any = true;
          }
          sr.template next<SA>();
          br.template next<SB>();
          if (H == 1 && last) ar.template next<2>();
        }
        if (H == 2) ar.ph ^= 1u;
      }
      if (any || CG == 2) {  // every MMA issued is complete before tensor memory is freed
        if (elect_one()) mma_commit_all<CG>(drain);
        __syncwarp();
        mbar_wait(drain, 0, never_flag, a.stall.wait_ns);
      }
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ dY producer
    if (lane == 0) {
      pdl_wait();
      Ring br{0, 0};
      bool ok = true;
      for (int u = first_unit; ok && u < a.units; u += stride) {
        const BwdUnit x = bwd_unit(a, u);
        for (int i = x.i0; i < x.i1; ++i) {
          if (!mbar_wait(&b_done[br.i], br.ph ^ 1u, abort_flag, a.stall.wait_ns)) {
            fail(4);
            ok = false;
            break;
          }
          // one barrier, the leader's, for both halves of the tokens
          if (rank == 0) mbar_arrive_expect_tx(&b_full[br.i], Sh::kB * CG);
#pragma unroll
          for (int h = 0; h < H; ++h) {
            uint8_t* dst = stage_b(br.i) + h * (Sh::kB / H);
            const int m = x.tb * NT + h * Sh::kN + rank * (Sh::kN / CG);
            if constexpr (CG == 1) tma_load_2d(dst, &maps.dy, i / T * kStep, m, &b_full[br.i]);
            else tma_load_2d_lead(dst, &maps.dy, i / T * kStep, m, &b_full[br.i]);
          }
          br.template next<SB>();
        }
      }
      if (!ok || *abort_flag) grace();
    }
  } else if (warp >= kXfWarp0 && warp < kEpiWarp0) {
    // ------------------------------------------------------------ transform
    // 16 codes of one row per thread and round, eight threads a row, rows 16 apart: a
    // thread's chunks sit at fixed offsets, and its row scale serves 16 codes.  Threads
    // of the second 64 columns write their two chunks in the other order, so that the
    // eight threads of a row always write eight different 16-byte columns.
    const int t = (threadIdx.x - 32 * kXfWarp0) % kXfThreads, group = (warp - kXfWarp0) / kXfWarps;
    const int c = t & 7, r0 = t >> 3, late = c >> 2;
    const int first = late * (kStep * 128) + r0 * 128 + (((2 * (c & 3) + late) ^ (r0 & 7)) << 4);
    const int second = late * (kStep * 128) + r0 * 128 + (((2 * (c & 3) + 1 - late) ^ (r0 & 7)) << 4);
    Ring sr{0, 0}, rr{0, 0};
    bool ok = true;
    int turn = 0;
    for (int u = first_unit; ok && u < a.units; u += stride) {
      const BwdUnit x = bwd_unit(a, u);
      for (int i = x.i0; i < x.i1; ++i) {
        if (turn == group) {
          if (!__all_sync(0xffffffffu, mbar_wait(&raw_full[rr.i], rr.ph, abort_flag, a.stall.wait_ns) &&
                                           mbar_wait(&a_done[sr.i], sr.ph ^ 1u, abort_flag, a.stall.wait_ns))) {
            fail(5);
            ok = false;
            break;
          }
          const uint8_t* src = raw_slot(rr.i);
          const uint16_t* scl = reinterpret_cast<const uint16_t*>(src + kStep * kTileK);
          uint8_t* dst = stage_a(sr.i);
          // (rotated, so that no group has the longest conversion throughout)
          const int term = (i + i / T) % T;
          auto put = [&](int k, uint4 v, float s) {
            const float o = -32896.f * s;
            const float2 s2 = make_float2(s, s), o2 = make_float2(o, o);
            float2 f[8];
            codes4(v.x, s2, o2, f[0], f[1]);
            codes4(v.y, s2, o2, f[2], f[3]);
            codes4(v.z, s2, o2, f[4], f[5]);
            codes4(v.w, s2, o2, f[6], f[7]);
#pragma unroll 1
            for (int t = 0; T > 1 && t < term; ++t)
#pragma unroll
              for (int j = 0; j < 8; ++j) f[j] = bf16_rest(f[j]);
            const uint2 e0 = round4(f[0], f[1]), e1 = round4(f[2], f[3]), e2 = round4(f[4], f[5]), e3 = round4(f[6], f[7]);
            const uint4 lo = make_uint4(e0.x, e0.y, e1.x, e1.y), hi = make_uint4(e2.x, e2.y, e3.x, e3.y);
            *reinterpret_cast<uint4*>(dst + first + k * 2048) = late ? hi : lo;
            *reinterpret_cast<uint4*>(dst + second + k * 2048) = late ? lo : hi;
          };
          // (compact with several terms: unrolled, and a copy of the code for each term, a step took twice as long)
          constexpr int kUnrolled = T == 1 ? kStep / 16 : 1;
          if (raw_int4[rr.i]) {
#pragma unroll kUnrolled
            for (int k = 0; k < kStep / 16; ++k) {  // nibbles as 16 q: see tc_linear.cu
              const uint2 w = *reinterpret_cast<const uint2*>(src + (r0 + 16 * k) * (kTileK / 2) + c * 8);
              const uint32_t l0 = (w.x << 4) & 0xF0F0F0F0u, h0 = w.x & 0xF0F0F0F0u;
              const uint32_t l1 = (w.y << 4) & 0xF0F0F0F0u, h1 = w.y & 0xF0F0F0F0u;
              put(k, make_uint4(__byte_perm(l0, h0, 0x5140), __byte_perm(l0, h0, 0x7362), __byte_perm(l1, h1, 0x5140),
                                __byte_perm(l1, h1, 0x7362)),
                  __half2float(__ushort_as_half(scl[r0 + 16 * k])) * 0.0625f);
            }
          } else {
#pragma unroll kUnrolled
            for (int k = 0; k < kStep / 16; ++k)
              put(k, *reinterpret_cast<const uint4*>(src + (r0 + 16 * k) * kTileK + c * 16),
                  __half2float(__ushort_as_half(scl[r0 + 16 * k])));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (CG == 1 || rank == 0) mbar_arrive(&a_full[sr.i]);
            else arrive_lead<CG>(&a_full[sr.i]);
            mbar_arrive(&raw_empty[rr.i]);
          }
        }
        turn = turn == kXfGroups - 1 ? 0 : turn + 1;
        sr.template next<SA>();
        rr.template next<RW>();
      }
    }
  } else if (warp >= kEpiWarp0) {
    // ------------------------------------------------------------ epilogue
    // (two halves have a group of four warps each)
    const int quad = warp & 3, half = (warp - kEpiWarp0) / kEpiWarps;
    const size_t kcol = 32 * quad + lane;
    pdl_wait();
    int ui = 0;  // sums taken over
    bool ok = true;
    for (int u = first_unit; ok && u < a.units; u += stride) {
      const BwdUnit x = bwd_unit(a, u);
      for (int i = x.i0; i < x.i1; i = T == 1 ? x.i1 : i + a.chunk, ++ui) {
        const int buf = H == 2 ? half : ui & 1, phase = H == 2 ? ui & 1 : ui >> 1 & 1, m0 = x.tb * NT + half * Sh::kN;
        const size_t k = (size_t)(x.kb * CG + rank) * kTileK + kcol;
        if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[buf], phase, abort_flag, a.stall.wait_ns))) {
          fail(6);
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t taddr = tmem_base + ((uint32_t)(32 * quad) << 16) + buf * Sh::kN;
        // a lane holds one column k of every token: a warp's stores cover 32 columns
        float* fp = x.part >= 0 ? a.partial + ((size_t)(x.part * CG + rank) * NT + half * Sh::kN) * kTileK + kcol
                                : static_cast<float*>(a.dx) + (size_t)m0 * a.lddx + k;
        __nv_bfloat16* bp = static_cast<__nv_bfloat16*>(a.dx) + (size_t)m0 * a.lddx + k;
        const size_t fld = x.part >= 0 ? kTileK : a.lddx;
        // A unit's later sums (T = 3, fp32 throughout) are added to what the same thread has stored, at L2, in the
        // order of its stores, so the result is the same on every run.  (A value below 2^-126 may become zero there.)
        const bool f32 = a.f32 || x.part >= 0, more = T > 1 && i > x.i0, add = a.add && x.part < 0 && !more;
        const int cols = min(Sh::kN, a.M - m0);  // (none: below 0)
        for (int c0 = 0; c0 < cols; c0 += 16) {
          uint32_t v[16];
          tmem_ld16(taddr + c0, v);
          const int left = cols - c0;
          float y[16];
          if (add)
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (e < left)
                y[e] = a.f32 ? static_cast<const float*>(a.add)[(size_t)(m0 + c0 + e) * a.ldadd + k]
                             : bf16_bits_to_float(static_cast<const uint16_t*>(a.add)[(size_t)(m0 + c0 + e) * a.ldadd + k]);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            asm volatile("" : "+r"(v[e]));
            if (add && e < left) v[e] = __float_as_uint(__uint_as_float(v[e]) + y[e]);
          }
          if (more) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (e < left) atomicAdd(fp + (size_t)e * fld, __uint_as_float(v[e]));
          } else if (f32) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (e < left) fp[(size_t)e * fld] = __uint_as_float(v[e]);
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (e < left) bp[(size_t)e * a.lddx] = __float2bfloat16_rn(__uint_as_float(v[e]));
          }
          fp += 16 * fld;
          bp += (size_t)16 * a.lddx;
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_lead<CG>(&acc_empty[buf]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (CG == 2) {
    cluster_sync();  // the other's products may read this CTA's memory until here
    // The leader's last arrival has come to this CTA too.  (After the barrier: the leader, should it have
    // given up later than this CTA, has issued it by then, and this wait cannot run out before it.)
    if (warp == 1) mbar_wait(drain, 0, never_flag, a.stall.wait_ns);
    __syncwarp();
  }
  if (warp == 1) {
    tc_fence_after();
    if constexpr (CG == 1) tmem_dealloc(tmem_base, Sh::kTmemCols);
    else tmem_dealloc2(tmem_base, Sh::kTmemCols);
  }
}

// dx = add + the partial sums of the split units, splits in increasing order; four
// columns of a token per thread, blockIdx.y the split unit.
__global__ void __launch_bounds__(256) linear_backward_sum_kernel(const BwdArgs a, int nt, int cg) {
  const int i = blockIdx.x * 256 + threadIdx.x, c = i / (kTileK / 4), col = blockIdx.y % cg, j = blockIdx.y / cg,
            u = a.whole + j;
  const int m = u % a.ntb * nt + c, k = (u / a.ntb * cg + col) * kTileK + i % (kTileK / 4) * 4;
  pdl_launch_dependents();
  pdl_wait();
  if (c >= nt || m >= a.M) return;
  const float4* p = reinterpret_cast<const float4*>(a.partial) + ((size_t)j * a.S * cg + col) * nt * (kTileK / 4) + i;
  const size_t step = (size_t)cg * nt * (kTileK / 4);
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int s = 0; s < a.S; ++s) {
    const float4 w = __ldcg(p + s * step);
    v.x += w.x;
    v.y += w.y;
    v.z += w.z;
    v.w += w.w;
  }
  if (a.f32) {
    if (a.add) {
      const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(a.add) + (size_t)m * a.ldadd + k);
      v.x += w.x;
      v.y += w.y;
      v.z += w.z;
      v.w += w.w;
    }
    *reinterpret_cast<float4*>(static_cast<float*>(a.dx) + (size_t)m * a.lddx + k) = v;
  } else {
    if (a.add) {
      const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.add) + (size_t)m * a.ldadd + k);
      v.x += bf16_bits_to_float(w.x & 0xFFFFu);
      v.y += bf16_bits_to_float(w.x >> 16);
      v.z += bf16_bits_to_float(w.y & 0xFFFFu);
      v.w += bf16_bits_to_float(w.y >> 16);
    }
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.dx) + (size_t)m * a.lddx + k) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
}

// ---------------------------------------------------------------- host side
struct BwdPlan {
  int cg, nt, ntb;  // CTAs and tokens of a unit, units along the tokens
  long long whole;  // units done whole
  int rest, S;      // units that are split, and their splits
};

// The forms of a unit, with the time of a step and of a unit's epilogue where the next
// unit cannot cover it, in 10 ns (a fit over sizes from 64 x 2560 x 2560 to 4096 x 2048 x
// 2048 to within 10%).
struct BwdForm {
  int cg, nt, step, unit;
};
constexpr BwdForm kBwdForms[] = {{1, 32, 40, 30},   {1, 64, 40, 40},   {1, 128, 40, 60},
                                 {1, 256, 45, 120}, {2, 256, 41, 120}, {2, 384, 50, 300}, {2, 512, 60, 400}};

// The form and the splits of least time: the steps of the CTA that has most, its units'
// ends, and for a split the second launch with its 4 bytes written and read per sum.
BwdPlan plan_bwd(int M, int N, int C, int terms) {
  const int steps = N / kStep * terms;
  BwdPlan best{0, 0, 0, 0, 0, 1};
  long long best_cost = 0;
  for (const BwdForm& f : kBwdForms) {
    if (C % f.cg || (terms > 1 && f.nt > 256)) continue;
    const int ntb = (M + f.nt - 1) / f.nt, slots = num_sms() / f.cg;
    const long long units = (long long)C / f.cg * ntb, rounds = units / slots;
    const int rest = (int)(units % slots), most = rest ? std::max(1, std::min({slots / rest, steps / 4, kMaxBwdSplits})) : 1;
    for (int S = 1; S <= most; ++S) {
      const bool split = S > 1;
      long long cost = (rounds * steps + (rest ? (steps + S - 1) / S : 0)) * f.step + (rounds + (rest > 0)) * f.unit;
      if (split) cost += 300 + (rounds ? 500 : 0) + (long long)rest * S * f.cg * f.nt * kTileK * 4 * 30 / 1000000;
      if (best.nt == 0 || cost < best_cost) {
        best = split ? BwdPlan{f.cg, f.nt, ntb, rounds * slots, rest, S} : BwdPlan{f.cg, f.nt, ntb, units, 0, 1};
        best_cost = cost;
      }
    }
  }
  return best;
}

template <int NT, int CG, int T>
cudaError_t launch_bwd(const aq_packed* w, const uint16_t* dy, int ldd, const BwdArgs& a, cudaStream_t st) {
  using Sh = BwdShape<NT, CG>;
  cudaError_t e = ensure_smem_attr<linear_backward_kernel<NT, CG, T>>(Sh::kSmem);
  if (e != cudaSuccess) return e;
  BwdMaps maps;
  memset(&maps, 0, sizeof(maps));
  bool ok = map_2d(&maps.dy, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dy, a.N, a.M, (uint64_t)ldd * 2, kStep, Sh::kN / CG, true);
  if (ok && w->T8 > 0)
    ok = map_2d(&maps.w8, CU_TENSOR_MAP_DATA_TYPE_UINT8, w->w8, kTileK, (uint64_t)w->T8 * w->bN, kTileK, kTileK, kStep, false);
  if (ok && w->T4 > 0)
    ok = map_2d(&maps.w4, CU_TENSOR_MAP_DATA_TYPE_UINT8, w->w4, kTileK / 2, (uint64_t)w->T4 * w->bN, kTileK / 2,
                kTileK / 2, kStep, false);
  if (!ok) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(CG * std::min(a.units, num_sms() / CG));
  cfg.blockDim = dim3(Sh::kThreads);
  cfg.dynamicSmemBytes = Sh::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // as launch_pdl
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = CG;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = CG == 1 ? 1 : 2;
  return cudaLaunchKernelEx(&cfg, linear_backward_kernel<NT, CG, T>, maps, a);
}

template <int T>
cudaError_t launch_form(const BwdPlan& p, const aq_packed* w, const uint16_t* dy, int ldd, const BwdArgs& a,
                        cudaStream_t st) {
  switch (p.cg * 1000 + p.nt) {
    case 1032: return launch_bwd<32, 1, T>(w, dy, ldd, a, st);
    case 1064: return launch_bwd<64, 1, T>(w, dy, ldd, a, st);
    case 1128: return launch_bwd<128, 1, T>(w, dy, ldd, a, st);
    case 1256: return launch_bwd<256, 1, T>(w, dy, ldd, a, st);
    case 2256: return launch_bwd<256, 2, T>(w, dy, ldd, a, st);
  }
  if constexpr (T == 1) {
    if (p.cg * 1000 + p.nt == 2384) return launch_bwd<384, 2, 1>(w, dy, ldd, a, st);
    if (p.cg * 1000 + p.nt == 2512) return launch_bwd<512, 2, 1>(w, dy, ldd, a, st);
  }
  return cudaErrorInvalidValue;
}

// Terms of the weights for dxdtype (see aq_linear_backward); 0: not a valid one.
int bwd_terms(int dxdtype) {
  const int type = dxdtype & 0xFF, weights = dxdtype - type;
  if (type != AQ_F32 && type != AQ_BF16) return 0;
  if (weights == 0) return type == AQ_F32 ? 3 : 1;
  return weights == AQ_WEIGHTS_EXACT ? 3 : weights == AQ_WEIGHTS_BF16 ? 1 : 0;
}

constexpr int kMaxBwdTokens = 1 << 21;

}  // namespace
}  // namespace aq

using namespace aq;

extern "C" size_t aq_linear_backward_workspace_bytes(int M, const aq_packed* w) {
  if (validate_packed(w) != AQ_OK || M < 1 || M > kMaxBwdTokens) return 0;
  size_t most = 0;
  for (int terms : {1, 3}) {
    const BwdPlan p = plan_bwd(M, w->N, w->C, terms);
    most = std::max(most, (size_t)p.rest * p.S * p.cg * p.nt * kTileK * sizeof(float));
  }
  return kWsHeader + most;
}

static int linear_backward(const aq_packed* w, const uint16_t* dy, int ldd, int M, const void* add, int ldadd, void* dx,
                           int lddx, int dxdtype, void* ws, size_t ws_bytes, const Stall& stall, void* stream) {
  int rc = validate_packed(w);
  if (rc != AQ_OK) return rc;
  if (!dy || !dx || M < 1 || M > kMaxBwdTokens || ldd < w->N || ldd % 8 || ((uintptr_t)dy & 15)) return AQ_ERR_ARG;
  const int terms = bwd_terms(dxdtype);
  if (terms == 0) return AQ_ERR_ARG;
  dxdtype &= 0xFF;
  const int per16 = dxdtype == AQ_F32 ? 4 : 8;
  if (lddx < w->K || lddx % per16 || ((uintptr_t)dx & 15)) return AQ_ERR_ARG;
  if (add && (ldadd < w->K || ldadd % per16 || ((uintptr_t)add & 15))) return AQ_ERR_ARG;
  if (add == dx && ldadd != lddx && M > 1) return AQ_ERR_ARG;  // in place is row by row
  if (!ws || ws_bytes < aq_linear_backward_workspace_bytes(M, w)) return AQ_ERR_WORKSPACE;
  if ((uintptr_t)ws & 15) return AQ_ERR_ARG;
  // units end in any order: what one writes over dy, others would still read
  const size_t elt = dxdtype == AQ_F32 ? 4 : 2, width = w->K * elt;
  const Span outs[] = {{dx, lddx * elt, width, M}};
  const Span ins[] = {{dy, (size_t)ldd * 2, (size_t)w->N * 2, M}, {add == dx ? nullptr : add, ldadd * elt, width, M}};
  if (outputs_overlap(outs, ins)) return AQ_ERR_ARG;
  const BwdPlan p = plan_bwd(M, w->N, w->C, terms);
  BwdArgs a;
  memset(&a, 0, sizeof(a));
  a.bitmap = w->bitmap; a.tile_idx = w->tile_idx; a.scales = w->scales;
  a.N = w->N; a.K = w->K; a.bN = w->bN; a.C = w->C; a.T4 = w->T4; a.T8 = w->T8;
  a.M = M; a.ntb = p.ntb; a.S = p.S; a.steps = w->N / kStep * terms;
  a.chunk = dxdtype == AQ_F32 ? kSumRows / kStep * terms : 1 << 30;
  if (p.whole > 0x7FFF0000ll) return AQ_ERR_ARG;
  a.whole = (int)p.whole;
  a.units = a.whole + p.rest * p.S;
  a.add = add; a.dx = dx; a.ldadd = ldadd; a.lddx = lddx; a.f32 = dxdtype == AQ_F32;
  a.ws = ws;
  a.stall = stall;
  a.partial = reinterpret_cast<float*>(static_cast<char*>(ws) + kWsHeader);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = terms == 3 ? launch_form<3>(p, w, dy, ldd, a, st) : launch_form<1>(p, w, dy, ldd, a, st);
  if (e == cudaSuccess && p.rest > 0)
    e = launch_pdl(linear_backward_sum_kernel, dim3((p.nt * (kTileK / 4) + 255) / 256, p.rest * p.cg), dim3(256), 0, st, a,
                   p.nt, p.cg);
  return e == cudaSuccess ? AQ_OK : AQ_ERR_CUDA;
}

extern "C" int aq_linear_backward(const aq_packed* w, const uint16_t* dy, int ldd, int M, const void* add, int ldadd,
                                  void* dx, int lddx, int dxdtype, void* ws, size_t ws_bytes, void* stream) {
  return linear_backward(w, dy, ldd, M, add, ldadd, dx, lddx, dxdtype, ws, ws_bytes, Stall{}, stream);
}

extern "C" int aq_debug_linear_backward_stalled(const aq_packed* w, const uint16_t* dy, int ldd, int M, void* dx, int lddx,
                                                int dxdtype, void* ws, size_t ws_bytes, unsigned long long wait_ns,
                                                int stop_after, void* stream) {
  if (!stall_ok(wait_ns, stop_after)) return AQ_ERR_ARG;
  return linear_backward(w, dy, ldd, M, nullptr, 0, dx, lddx, dxdtype, ws, ws_bytes, Stall{wait_ns, stop_after}, stream);
}
