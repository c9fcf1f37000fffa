// Weight gradients of the adapters on the 5th-generation tensor cores:
//   g_l[r][d] = sum over the tokens m of adapter l of T[m][r] x[m][d]
// with x the activations (8-bit codes or bf16; then T holds dS, times the token
// scale for codes) or the output's gradient (then T holds S).
//
// T is fp32 and enters as three bf16 terms, 24 bits, side by side along N:
//   D[128 d][hi | mid | lo] += x[64 tokens][128 d]^T [T_hi | T_mid | T_lo][64 tokens]
// so one pass over x serves all three; codes are exact in bf16.  Both operands are
// MN-major, that is, as they lie in memory.  A first kernel, or the expansion of dx beside
// its own work, writes the terms (zeros behind a token's rank) and says of each 64 tokens
// whether one adapter has them all.  On paper the bytes of x bound it, 64 x 128 of them per
// step against 64 x 128 x 3r multiplications; in practice a step's chain of waits and its
// conversion (940 of 2000 cycles, two CTAs per SM): both gradients of 8192 x 14336 codes and 8192 x 4096, ranks 16 to 32, take
// 70 us, 40% of the copy rate.
//
// A CTA takes 128 columns and a range of tokens, whoever's they are, so that
// unequal adapters do not make unequal CTAs; where that leaves room on the GPU (short
// batches), several share a range's adapters (30 tokens of 22 adapters: 126 -> 74 us).  It lists its steps beforehand, (adapter,
// 64 tokens) pairs ordered by adapter, and runs through them without a pause at an
// adapter's end (a pause cost 5 us).  Where a 64 holds
// other adapters' tokens too, their rows are cleared in shared memory on both sides,
// so that nothing of them, not even an infinity, reaches the sum.  Tensor memory
// sums 512 tokens at a time; the epilogue adds those sums in fp32 registers,
// rounding to nearest.  Partial sums of the ranges are added in range order.
//
// Roles: warp 0 codes or bf16 activations (TMA), warp 1 tensor memory and MMA, warp 2
// terms (TMA), warps 4-7 codes -> bf16 and the clearing, warps 8-11 epilogue.
// Every wait is bounded; one that gives up is recorded in the workspace.
#include <algorithm>
#include <cstring>

#include "lora.cuh"
#include "tc_bf16.cuh"

namespace aq {
namespace {

constexpr int kTok = 64;       // tokens of a step
constexpr int kD = 128;        // columns of a CTA
constexpr int kThreads = 384;
constexpr int kUnit = 8;       // steps summed in tensor memory
constexpr int kXf = 4, kEpi = 4;  // warps
constexpr int kMaxAdapters = 16384;
constexpr int kListCap = 512, kSlotCap = 64;  // steps and adapters listed at once

// A listed step: which 64 tokens of the range, whether others' tokens are among them, the
// bounds of a unit and of its adapter, and the adapter's slot.
constexpr uint32_t kMixed = 1u << 9, kUnitStart = 1u << 10, kUnitEnd = 1u << 11, kLast = 1u << 12;
constexpr int kSlotShift = 13;

// ---------------------------------------------------------------- terms
__global__ void __launch_bounds__(256) lora_terms_kernel(const TermsArgs a) {
  __shared__ int rank[kTok];
  const int tid = threadIdx.x, m0 = blockIdx.x * kTok;
  const TermsJob& j = a.job[blockIdx.y];
  pdl_launch_dependents();
  pdl_wait();
  if (tid < kTok) {
    const int n = min(kTok, a.M - m0);
    int v = tid < n ? __ldg(a.ids + m0 + tid) : -1, r = 0;
    if (v < 0 || v >= a.L) v = -1;
    if (v >= 0) {
      const int b = min(max(__ldg(a.off + v), 0), a.R);
      r = min(min(max(__ldg(a.off + v + 1), b), a.R) - b, a.max_rank) - a.rb0;
    }
    rank[tid] = r;
    int lead = __ldg(a.ids + m0);
    if (lead < 0 || lead >= a.L) lead = -1;
    const bool same = __all_sync(0xffffffffu, tid >= n || v == lead);
    const bool none = __all_sync(0xffffffffu, v < 0);
    __shared__ int kind[2];
    if ((tid & 31) == 0) kind[tid >> 5] = none ? 1 : same ? 2 : 0;
    asm volatile("bar.sync 1, 64;" ::: "memory");
    if (tid == 0 && blockIdx.y == 0 && a.rb0 == 0) {
      const bool all_same = n > 32 ? kind[0] && kind[0] == kind[1] : kind[0] != 0;
      a.info[blockIdx.x] = !all_same ? -2 : kind[0] == 1 ? -1 : lead;
    }
  }
  __syncthreads();
  const int per_row = a.rc / 8;
  for (int i = tid; i < kTok * per_row; i += 256) {
    const int t = i / per_row, c = (i - t * per_row) * 8, m = m0 + t;
    if (m >= a.M) break;
    write_terms(a, j, m, c, rank[t]);
  }
}

// ---------------------------------------------------------------- gradients
template <int NB, bool CODES>
struct GradShape {
  static constexpr int kRanks = NB / 3;
  static constexpr int kAtoms = (NB + 63) / 64;       // 64 terms x 64 tokens, 8 KiB each
  static constexpr int kA = kTok * kD * 2, kB = kAtoms * 8192;
  // two CTAs per SM up to 32 ranks: a CTA's start and end are then covered by the other
  static constexpr int kPerSm = NB <= 96 ? 2 : 1;
  // rings: activations in bf16 (filled from the codes, or by TMA), terms, codes
  static constexpr int kSA = CODES ? (NB <= 96 ? 2 : 3) : NB <= 48 ? 4 : NB <= 96 ? 3 : 4;
  static constexpr int kSB = NB <= 48 ? (CODES ? 6 : 4) : NB <= 96 ? 3 : 5;
  static constexpr int kRaw = CODES ? (NB <= 96 ? 3 : 5) : 0;  // 8 KiB each
  static constexpr int kTmem = 2 * NB <= 128 ? 128 : 2 * NB <= 256 ? 256 : 512;
  static constexpr int kCtrl = 512 + kListCap * 4 + 4 * kSlotCap * 4 + kThreads * 4 + kMaxAdapters / 8;
  static constexpr int kSmem = 1024 + kSA * kA + kSB * kB + kRaw * kTok * kD + kCtrl;
  static constexpr uint32_t kIdesc = idesc_bf16(NB, true, true);
  static_assert(kPerSm * (kSmem + 1024) <= 228 * 1024, "shared memory");
  // the transform warps look at the terms' barriers in mixed steps only: the use of a slot
  // before must be over by then (they have seen the MMAs of step i - kSA complete)
  static_assert(kSB >= kSA, "phases");
  static_assert(kPerSm * kTmem <= 512, "tensor memory");
};

struct GradMaps {
  CUtensorMap x, terms;
};

struct GradArgs {
  const int32_t* ids;
  const int32_t* off;
  const int32_t* info;
  int M, D, L, R, max_rank, rb0;
  float* g;       // [splits][R][D]
  int splits;
  int blocks, shares;  // CTAs along the columns, and those that share a range's adapters
  uint8_t* has;   // [L][splits]: whether the range has tokens of the adapter
  void* ws;
  Stall stall;    // (the activations' producer stops)
};

// Eight codes (bytes) as bf16: 128 + the low seven bits, less 128 or 256 by the sign, exact.
__device__ __forceinline__ uint4 widen_codes8(uint2 w) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = __byte_perm(i < 2 ? w.x : w.y, 0x43434343u, (i & 1) ? 0x4342 : 0x4140);
    const uint32_t lo = h & 0xFF7FFF7Fu, hi = h & 0xFF80FF80u;
    const __nv_bfloat162 v =
        __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&lo), *reinterpret_cast<const __nv_bfloat162*>(&hi));
    o[i] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int NB, bool CODES>
__device__ __forceinline__ void grad_cta(const GradMaps& maps, const GradArgs& a, int index) {
  using Sh = GradShape<NB, CODES>;
  constexpr int SA = Sh::kSA, SB = Sh::kSB, RW = CODES ? Sh::kRaw : 1;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  auto stage_a = [&](int st) { return smem + st * Sh::kA; };
  auto stage_b = [&](int st) { return smem + SA * Sh::kA + st * Sh::kB; };
  auto raw_slot = [&](int s) { return smem + SA * Sh::kA + SB * Sh::kB + s * kTok * kD; };
  uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + SA * Sh::kA + SB * Sh::kB + Sh::kRaw * kTok * kD);
  uint64_t* raw_empty = raw_full + RW;
  uint64_t* a_full = raw_empty + RW;   // transform warps done with the stage
  uint64_t* a_tma = a_full + SA;       // bf16 activations landed
  uint64_t* a_done = a_tma + SA;       // the stage's MMAs are complete
  uint64_t* b_full = a_done + SA;      // terms landed
  uint64_t* b_done = b_full + SB;
  uint64_t* acc_full = b_done + SB;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* never_flag = abort_flag + 1;
  volatile uint32_t* list = reinterpret_cast<volatile uint32_t*>(reinterpret_cast<uint8_t*>(raw_full) + 512);
  volatile int* slot_id = reinterpret_cast<volatile int*>(list + kListCap);  // adapter, first gradient row, ranks
  volatile int* slot_row = slot_id + kSlotCap;
  volatile int* slot_nr = slot_row + kSlotCap;
  volatile int* slot_steps = slot_nr + kSlotCap;
  volatile int* kinds = slot_steps + kSlotCap;  // `info` of the range's 64s
  uint32_t* present = reinterpret_cast<uint32_t*>(const_cast<int*>(kinds + kThreads));

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int block = index % a.blocks, share = index / a.blocks % a.shares, split = index / a.blocks / a.shares;
  const int d0 = block * kD, shares = a.shares;
  if (tid == 0) {
    for (int i = 0; i < RW; ++i) {
      mbar_init(&raw_full[i], 1);
      mbar_init(&raw_empty[i], kXf);
    }
    for (int i = 0; i < SA; ++i) {
      mbar_init(&a_full[i], kXf);
      mbar_init(&a_tma[i], 1);
      mbar_init(&a_done[i], 1);
    }
    for (int i = 0; i < SB; ++i) {
      mbar_init(&b_full[i], 1);
      mbar_init(&b_done[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], kEpi);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *never_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.x);
    prefetch_tmap(&maps.terms);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, Sh::kTmem);
    tmem_relinquish();
  }
  for (int i = tid; i < (a.L + 31) / 32; i += kThreads) present[i] = 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  // not earlier: a later kernel's CTA that held this one's tensor memory while it
  // waits for this one to end would never see it end
  pdl_launch_dependents();

  auto fail = [&](int info) {
    *abort_flag = 1;
    record_error(a.ws, AQ_ERR_TIMEOUT, info, 0);
  };

  pdl_wait();
  // the adapters of this range's (at most 384) 64s, one of which each thread looks after
  const int chunks = (a.M + kTok - 1) / kTok;
  const int c0 = (int)((long long)chunks * split / a.splits), c1 = (int)((long long)chunks * (split + 1) / a.splits);
  const int own = c0 + tid < c1 ? __ldg(a.info + c0 + tid) : -1;
  kinds[tid] = own;
  if (own >= 0) atomicOr(&present[own >> 5], 1u << (own & 31));
  for (unsigned left = __ballot_sync(0xffffffffu, own == -2); left; left &= left - 1) {  // a warp reads a mixed 64 together
    const int m0 = (c0 + 32 * warp + __ffs(left) - 1) * kTok;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int m = m0 + 32 * h + lane, v = m < a.M ? __ldg(a.ids + m) : -1;
      if (v >= 0 && v < a.L) atomicOr(&present[v >> 5], 1u << (v & 31));
    }
  }
  __syncthreads();
  // which of the 64s base .. base + 31 have tokens of adapter l
  auto steps_of = [&](int l, int base) {
    const int kind = kinds[base + lane];
    bool take = kind == l;
    for (unsigned left = __ballot_sync(0xffffffffu, kind == -2); left; left &= left - 1) {
      const int m = (c0 + base + __ffs(left) - 1) * kTok + lane;
      const bool has = (m < a.M && __ldg(a.ids + m) == l) || (m + 32 < a.M && __ldg(a.ids + m + 32) == l);
      if (__any_sync(0xffffffffu, has) && lane == __ffs(left) - 1) take = true;
    }
    return __ballot_sync(0xffffffffu, take);
  };

  Ring sr{0, 0}, br{0, 0}, rr{0, 0}, ar{0, 0};  // activations, terms, codes, accumulator
  bool ok = true, issued = false;
  int loads = 0;
  float tot[Sh::kRanks];
#pragma unroll
  for (int r = 0; r < Sh::kRanks; ++r) tot[r] = 0.f;

  for (int done = 0;;) {
    // The next of this CTA's adapters (every shares-th of the present ones); each warp finds
    // them for itself ...
    int seen = 0;
    for (int w0 = 0; w0 < (a.L + 31) / 32; w0 += 32) {
      uint32_t bits = w0 + lane < (a.L + 31) / 32 ? present[w0 + lane] : 0u;
      const int mine = __popc(bits);
      int upto = mine;
      if (a.L > 32) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += v;
        }
      }
      for (int i = seen + upto - mine; bits; bits &= bits - 1, ++i) {
        const int slot = i / shares - done;
        if (i % shares == share && slot >= 0 && slot < kSlotCap) slot_id[slot] = 32 * (w0 + lane) + __ffs(bits) - 1;
      }
      seen += __shfl_sync(0xffffffffu, upto, a.L > 32 ? 31 : 0);
    }
    __syncwarp();
    const int left = (seen > share ? (seen - share + shares - 1) / shares : 0) - done, named = min(left, kSlotCap);
    if (left <= 0) break;
    auto ranks_of = [&](int l, int& row0) {
      row0 = min(max(__ldg(a.off + l), 0), a.R);
      return min(min(min(max(__ldg(a.off + l + 1), row0), a.R) - row0, a.max_rank) - a.rb0, Sh::kRanks);
    };
    // lane's 64, the at-th of an adapter with `steps`
    auto put = [&](int first, int at, int steps, int slot, int k) {
      list[first + at] = (uint32_t)k | (kinds[k] == -2 ? kMixed : 0u) | (at % kUnit == 0 ? kUnitStart : 0u) |
                         (at % kUnit == kUnit - 1 || at + 1 == steps ? kUnitEnd : 0u) | (at + 1 == steps ? kLast : 0u) |
                         ((uint32_t)slot << kSlotShift);
    };
    const unsigned below = (1u << lane) - 1;
    int slots = 1, n = 0;
    if (named == 1) {
      // ... one: each warp counts its steps and lists those of 32 64s ...
      const int l = slot_id[0];
      int row0, before = 0;
      unsigned which = 0;
      const int nr = ranks_of(l, row0);
      for (int base = 0; base < c1 - c0; base += 32) {
        const unsigned steps = nr > 0 ? steps_of(l, base) : 0u;
        if (base == 32 * warp) {
          which = steps;
          before = n;
        }
        n += __popc(steps);
      }
      if (which >> lane & 1u) put(0, before + __popc(which & below), n, 0, 32 * warp + lane);
      if (tid == 0) {
        slot_row[0] = row0 + a.rb0;
        slot_nr[0] = nr;
      }
    } else {
      // ... several: their rows and the number of their steps, an adapter per warp ...
      for (int i = warp; i < named; i += kThreads / 32) {
        const int l = slot_id[i];
        int row0, steps = 0;
        const int nr = ranks_of(l, row0);
        if (nr > 0)
          for (int base = 0; base < c1 - c0; base += 32) steps += __popc(steps_of(l, base));
        if (lane == 0) {
          slot_row[i] = row0 + a.rb0;
          slot_nr[i] = nr;
          slot_steps[i] = steps;
        }
      }
      __syncthreads();
      // ... and the steps, of as many adapters as the list holds (384 steps of one at most)
      int end0 = lane < named ? slot_steps[lane] : 0, end1 = lane + 32 < named ? slot_steps[lane + 32] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v0 = __shfl_up_sync(0xffffffffu, end0, o), v1 = __shfl_up_sync(0xffffffffu, end1, o);
        if (lane >= o) {
          end0 += v0;
          end1 += v1;
        }
      }
      end1 += __shfl_sync(0xffffffffu, end0, 31);
      slots = __popc(__ballot_sync(0xffffffffu, lane < named && end0 <= kListCap)) +
              __popc(__ballot_sync(0xffffffffu, lane + 32 < named && end1 <= kListCap));
      n = __shfl_sync(0xffffffffu, slots > 32 ? end1 : end0, (slots - 1) & 31);
      for (int i = warp; i < slots; i += kThreads / 32) {
        const int l = slot_id[i], steps = slot_steps[i];
        const int first = __shfl_sync(0xffffffffu, i < 32 ? end0 : end1, i & 31) - steps;
        int before = 0;
        for (int base = 0; before < steps && base < c1 - c0; base += 32) {
          const unsigned which = steps_of(l, base);
          if (which >> lane & 1u) put(first, before + __popc(which & below), steps, i, base + lane);
          before += __popc(which);
        }
      }
    }
    __syncthreads();
    done += slots;
    const int base = c0;

    if (warp == 0) {
      // ------------------------------------------------------------ codes, or bf16 activations
      if (lane == 0) {
        for (int i = 0; ok && i < n; ++i) {
          const int m0 = (base + (int)(list[i] & 0x1FF)) * kTok;
          if (a.stall.stop_after >= 0 && loads++ == a.stall.stop_after) {
            stalled(abort_flag, a.stall.wait_ns);
            ok = false;
            break;
          }
          if (!(CODES ? mbar_wait(&raw_empty[rr.i], rr.ph ^ 1u, abort_flag, a.stall.wait_ns)
                      : mbar_wait(&a_done[sr.i], sr.ph ^ 1u, abort_flag, a.stall.wait_ns))) {
            fail(21);
            ok = false;
            break;
          }
          if (CODES) {
            mbar_arrive_expect_tx(&raw_full[rr.i], kTok * kD);
            tma_load_2d(raw_slot(rr.i), &maps.x, d0, m0, &raw_full[rr.i]);
            rr.template next<RW>();
          } else {
            mbar_arrive_expect_tx(&a_tma[sr.i], Sh::kA);
            tma_load_2d(stage_a(sr.i), &maps.x, d0, m0, &a_tma[sr.i]);
            tma_load_2d(stage_a(sr.i) + 8192, &maps.x, d0 + 64, m0, &a_tma[sr.i]);
            sr.template next<SA>();
          }
        }
      }
    } else if (warp == 1) {
      // ------------------------------------------------------------ MMA
      const uint64_t adesc0 = mn_desc(smem_u32(stage_a(0)), kTok * 128), bdesc0 = mn_desc(smem_u32(stage_b(0)), kTok * 128);
      const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
      for (int i = 0; ok && i < n; ++i) {
        const uint32_t step = __shfl_sync(0xffffffffu, list[i], 0);
        if ((step & kUnitStart) && !__all_sync(0xffffffffu, mbar_wait(&acc_empty[ar.i], ar.ph ^ 1u, abort_flag, a.stall.wait_ns))) {
          fail(22);
          ok = false;
          break;
        }
        if (!__all_sync(0xffffffffu, mbar_wait(&b_full[br.i], br.ph, abort_flag, a.stall.wait_ns) &&
                                         mbar_wait(&a_full[sr.i], sr.ph, abort_flag, a.stall.wait_ns) &&
                                         (CODES || mbar_wait(&a_tma[sr.i], sr.ph, abort_flag, a.stall.wait_ns)))) {
          fail(23);
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t ao = adesc0 + (uint64_t)((sr.i * Sh::kA) >> 4), bo = bdesc0 + (uint64_t)((br.i * Sh::kB) >> 4);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < kTok / 16; ++k)  // 16 tokens: two groups of eight rows
            mma_bf16(tmem + ar.i * NB, ao + 128 * k, bo + 128 * k, Sh::kIdesc, !(step & kUnitStart) || k > 0);
          mma_commit(&a_done[sr.i]);
          mma_commit(&b_done[br.i]);
          if (step & kUnitEnd) mma_commit(&acc_full[ar.i]);
        }
        __syncwarp();
        issued = true;
        sr.template next<SA>();
        br.template next<SB>();
        if (step & kUnitEnd) ar.template next<2>();
      }
    } else if (warp == 2) {
      // ------------------------------------------------------------ terms
      if (lane == 0) {
        for (int i = 0; ok && i < n; ++i) {
          if (!mbar_wait(&b_done[br.i], br.ph ^ 1u, abort_flag, a.stall.wait_ns)) {
            fail(24);
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&b_full[br.i], Sh::kB);
#pragma unroll
          for (int c = 0; c < Sh::kAtoms; ++c)
            tma_load_2d(stage_b(br.i) + c * 8192, &maps.terms, 64 * c, (base + (int)(list[i] & 0x1FF)) * kTok, &b_full[br.i]);
          br.template next<SB>();
        }
      }
    } else if (warp >= 4 && warp < 4 + kXf) {
      // ------------------------------------------------------------ transform
      // 16 codes of a row per thread and round, rows 16 apart: two chunks at fixed offsets.
      // Threads of the second 64 columns write theirs in the other order, so that the
      // eight threads of a row always write eight different 16-byte columns.
      const int t = tid - 128, c = t & 7, r0 = t >> 3, late = c >> 2;
      const int first = late * (kTok * 128) + r0 * 128 + (((2 * (c & 3) + late) ^ (r0 & 7)) << 4);
      const int second = late * (kTok * 128) + r0 * 128 + (((2 * (c & 3) + 1 - late) ^ (r0 & 7)) << 4);
      for (int i = 0; ok && i < n; ++i) {
        const bool mixed = list[i] & kMixed;
        const int m0 = (base + (int)(list[i] & 0x1FF)) * kTok;
        bool got = mbar_wait(&a_done[sr.i], sr.ph ^ 1u, abort_flag, a.stall.wait_ns);
        if (CODES) got = got && mbar_wait(&raw_full[rr.i], rr.ph, abort_flag, a.stall.wait_ns);
        if (mixed) got = got && mbar_wait(&b_full[br.i], br.ph, abort_flag, a.stall.wait_ns);
        if (mixed && !CODES) got = got && mbar_wait(&a_tma[sr.i], sr.ph, abort_flag, a.stall.wait_ns);
        if (!__all_sync(0xffffffffu, got)) {
          fail(25);
          ok = false;
          break;
        }
        if (CODES) {
          const uint8_t* src = raw_slot(rr.i) + r0 * kD + c * 16;
          uint8_t* dst = stage_a(sr.i);
          uint4 v[kTok / 16];
#pragma unroll
          for (int k = 0; k < kTok / 16; ++k) v[k] = *reinterpret_cast<const uint4*>(src + k * 16 * kD);
#pragma unroll
          for (int k = 0; k < kTok / 16; ++k) {
            const uint4 lo = widen_codes8(make_uint2(v[k].x, v[k].y)), hi = widen_codes8(make_uint2(v[k].z, v[k].w));
            *reinterpret_cast<uint4*>(dst + first + k * 2048) = late ? hi : lo;
            *reinterpret_cast<uint4*>(dst + second + k * 2048) = late ? lo : hi;
          }
        }
        if (mixed) {
          // rows of tokens that this adapter does not have: two lanes per row, the
          // rows that this warp itself has written
          __syncwarp();
          const int r = 4 * (warp - 4) + (lane >> 1 & 3) + 16 * (lane >> 3), half = lane & 1, m = m0 + r;
          if (m >= a.M || __ldg(a.ids + m) != slot_id[list[i] >> kSlotShift]) {
            const uint4 zero = make_uint4(0, 0, 0, 0);
            for (int q = 0; q < 8; ++q) *reinterpret_cast<uint4*>(stage_a(sr.i) + half * 8192 + r * 128 + q * 16) = zero;
            for (int q = half; q < 8 * Sh::kAtoms; q += 2)
              *reinterpret_cast<uint4*>(stage_b(br.i) + (q >> 3) * 8192 + r * 128 + (q & 7) * 16) = zero;
          }
        }
        if (CODES || mixed) fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&a_full[sr.i]);
          if (CODES) mbar_arrive(&raw_empty[rr.i]);
        }
        sr.template next<SA>();
        br.template next<SB>();
        if (CODES) rr.template next<RW>();
      }
    } else if (warp >= 4 + kXf) {
      // ------------------------------------------------------------ epilogue
      for (int i = 0; ok && i < n; ++i) {
        const uint32_t step = list[i];
        if (!(step & kUnitEnd)) continue;
        if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[ar.i], ar.ph, abort_flag, a.stall.wait_ns))) {
          fail(26);
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t taddr = tmem_base + ((uint32_t)(32 * (warp & 3)) << 16) + ar.i * NB;
#pragma unroll
        for (int r = 0; r < Sh::kRanks; r += 16) {
#pragma unroll
          for (int sp = 2; sp >= 0; --sp) {
            uint32_t v[16];
            tmem_ld16(taddr + sp * Sh::kRanks + r, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              asm volatile("" : "+r"(v[e]));
              tot[r + e] += __uint_as_float(v[e]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[ar.i]);
        ar.template next<2>();
        if (step & kLast) {
          const int d = d0 + 32 * (warp & 3) + lane, nr = slot_nr[step >> kSlotShift];
          float* g = a.g + ((size_t)split * a.R + slot_row[step >> kSlotShift]) * a.D + d;
#pragma unroll
          for (int r = 0; r < Sh::kRanks; ++r) {
            if (r < nr && d < a.D) g[(size_t)r * a.D] = tot[r];
            tot[r] = 0.f;
          }
        }
      }
    }
    __syncthreads();  // the list may be written anew
  }

  // adapters without tokens here: noted for the sum, or zeros where there is none
  if (a.splits > 1) {
    if (block == 0 && share == 0 && a.rb0 == 0)
      for (int l = tid; l < a.L; l += kThreads) a.has[(size_t)l * a.splits + split] = (present[l >> 5] >> (l & 31)) & 1u;
  } else {
    // a warp per adapter, four columns a lane (D is a multiple of 8)
    const int d = d0 + 4 * lane;
    for (int l = warp + share * (kThreads / 32); l < a.L; l += shares * (kThreads / 32)) {
      if ((present[l >> 5] >> (l & 31)) & 1u) continue;
      const int row0 = min(max(__ldg(a.off + l), 0), a.R);
      const int nr = min(min(min(max(__ldg(a.off + l + 1), row0), a.R) - row0, a.max_rank) - a.rb0, Sh::kRanks);
      for (int r = 0; d < a.D && r < nr; ++r)
        *reinterpret_cast<float4*>(a.g + (size_t)(row0 + a.rb0 + r) * a.D + d) = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  if (warp == 1 && issued) {
    if (elect_one()) mma_commit(drain);
    __syncwarp();
    mbar_wait(drain, 0, never_flag, a.stall.wait_ns);
  }
  if ((warp == 0 || warp == 2) && lane == 0 && (!ok || *abort_flag)) {
    grace();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, Sh::kTmem);
  }
}

// Both gradients in one launch, that of A first.
struct GradJobs {
  GradMaps maps[2];
  GradArgs args[2];
};
template <int NB, bool CODES>
__global__ void __launch_bounds__(kThreads, GradShape<NB, CODES>::kPerSm)
    lora_grad_kernel(const __grid_constant__ GradJobs j) {
  const int first = j.args[0].blocks * j.args[0].shares * j.args[0].splits, side = (int)blockIdx.x >= first;
  if (CODES && side == 0)
    grad_cta<NB, CODES>(j.maps[0], j.args[0], blockIdx.x);
  else
    grad_cta<NB, false>(j.maps[side], j.args[side], blockIdx.x - (side ? first : 0));
}

// g = the sum of the ranges' partial sums in range order, for one adapter and 1024 columns
// of one of the two gradients.
struct SumJob {
  const float* p;       // [splits][R][D]
  const uint8_t* has;   // [L][splits]
  float* g;
  int splits, D, blocks;  // blocks of 1024 columns; 0: nothing to sum
};
struct SumArgs {
  SumJob job[2];
  const int32_t* off;
  int R, max_rank;
};

__global__ void __launch_bounds__(256) lora_sum_kernel(const __grid_constant__ SumArgs a) {
  const bool second = blockIdx.x >= a.job[0].blocks;
  const SumJob& j = a.job[second];
  const int l = blockIdx.y, d = ((blockIdx.x - (second ? a.job[0].blocks : 0)) * 256 + threadIdx.x) * 4;
  pdl_launch_dependents();
  pdl_wait();
  if (d >= j.D) return;
  const int row0 = min(max(__ldg(a.off + l), 0), a.R),
            row1 = min(row0 + a.max_rank, min(max(__ldg(a.off + l + 1), row0), a.R));
  const uint8_t* mine = j.has + (size_t)l * j.splits;
  const size_t step = (size_t)a.R * j.D;
  for (int r = row0 + blockIdx.z; r < row1; r += gridDim.z) {
    const float* p = j.p + (size_t)r * j.D + d;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k0 = 0; k0 < j.splits; k0 += 8) {  // eight loads on their way
      float4 w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i] = k0 + i < j.splits && mine[k0 + i] ? __ldcg(reinterpret_cast<const float4*>(p + (k0 + i) * step))
                                                 : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v.x += w[i].x;
        v.y += w[i].y;
        v.z += w[i].z;
        v.w += w[i].w;
      }
    }
    *reinterpret_cast<float4*>(j.g + (size_t)r * j.D + d) = v;
  }
}

// ---------------------------------------------------------------- host side
int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }
size_t align256(size_t b) { return (b + 255) / 256 * 256; }

int rank_blocks(int max_rank) { return ceil_div(max_rank, 64); }
int block_ranks(int max_rank, int rb) { return (std::min(64, max_rank - 64 * rb) + 15) / 16 * 16; }
int block_pad(int max_rank, int rb) { return (3 * block_ranks(max_rank, rb) + 63) / 64 * 64; }
size_t terms_bytes(int M, int max_rank) {
  size_t b = 0;
  for (int rb = 0; rb < rank_blocks(max_rank); ++rb) b += align256((size_t)M * block_pad(max_rank, rb) * 2);
  return b;
}

int grad_slots(int max_rank) { return (max_rank <= 32 ? 2 : 1) * num_sms(); }  // see GradShape

// Token ranges, the same for both gradients: at most 384 64s each; the fewest steps on the
// longest path, counting a CTA's start and end as ten.
int grad_splits(const aq_lora* ad, int M) {
  const int chunks = ceil_div(M, kTok), blocks = ceil_div(ad->K, kD) + ceil_div(ad->N, kD), slots = grad_slots(ad->max_rank);
  const int least = ceil_div(chunks, kThreads);
  int best = least;
  long long cost = 0;
  for (int s = least; s <= std::max(least, std::min(chunks, 16)); ++s) {
    // (a launch for the sum counts as eight)
    const long long c = (long long)ceil_div((long long)blocks * s, slots) * (ceil_div(chunks, s) + 10) + (s > 1 ? 8 : 0);
    if (cost == 0 || c < cost) {
      cost = c;
      best = s;
    }
  }
  return best;
}

// CTAs that share the adapters of one range and column block: as many as fit in one wave.
// (Rows of the gradients are an adapter's own, so there is nothing to sum.)
int grad_shares(const aq_lora* ad, int splits) {
  const int blocks = ceil_div(ad->K, kD) + ceil_div(ad->N, kD);
  return std::max(1, std::min(ad->L, grad_slots(ad->max_rank) / std::max(1, blocks * splits)));
}

size_t part_bytes(const aq_lora* ad, int M, int D) {
  const int s = grad_splits(ad, M);
  return s > 1 ? align256((size_t)s * ad->R * D * sizeof(float)) + align256((size_t)ad->L * s) : 0;
}

template <int NB, bool CODES>
cudaError_t launch_shape(const GradJobs& j, cudaStream_t st) {
  constexpr int smem = std::max(GradShape<NB, CODES>::kSmem, GradShape<NB, false>::kSmem);
  cudaError_t e = ensure_smem_attr<lora_grad_kernel<NB, CODES>>(smem);
  if (e != cudaSuccess) return e;
  int ctas = 0;
  for (const GradArgs& a : j.args) ctas += a.blocks * a.shares * a.splits;
  return launch_pdl(lora_grad_kernel<NB, CODES>, dim3(ctas), dim3(kThreads), (size_t)smem, st, j);
}

template <bool CODES>
cudaError_t launch_ranks(int ranks, const GradJobs& j, cudaStream_t st) {
  switch (ranks) {
    case 16: return launch_shape<48, CODES>(j, st);
    case 32: return launch_shape<96, CODES>(j, st);
    case 48: return launch_shape<144, CODES>(j, st);
    case 64: return launch_shape<192, CODES>(j, st);
  }
  return cudaErrorInvalidValue;
}

}  // namespace

size_t lora_grad_ws_bytes(const aq_lora* ad, int M) {
  return align256((size_t)ceil_div(M, kTok) * 4) + 2 * terms_bytes(M, ad->max_rank) +
         part_bytes(ad, M, ad->K) + part_bytes(ad, M, ad->N);
}

TermsArgs lora_grad_terms(const aq_lora* ad, const int32_t* ids, int M, int rb, const float* t, int tsplits, int ldt,
                          const float* sx, const float* s, void* ws) {
  char* at = static_cast<char*>(ws);
  int32_t* info = reinterpret_cast<int32_t*>(at);
  at += align256((size_t)ceil_div(M, kTok) * 4);
  for (int i = 0; i < rb; ++i) at += align256((size_t)M * block_pad(ad->max_rank, i) * 2);
  return {{{t, tsplits, ldt, sx, reinterpret_cast<uint16_t*>(at)},
           {s, 1, ad->max_rank, nullptr, reinterpret_cast<uint16_t*>(at + terms_bytes(M, ad->max_rank))}},
          ids, ad->off, M, ad->L, ad->R, ad->max_rank, 64 * rb, block_ranks(ad->max_rank, rb), block_pad(ad->max_rank, rb), info};
}

cudaError_t launch_lora_grad(const aq_lora* ad, const int32_t* ids, int M, const float* t, int tsplits, int ldt, const void* x,
                             int ldx, const float* sx, float* da, const float* s, const uint16_t* dy, int ldd,
                             float* dbt, bool have_terms, void* header, void* ws, const Stall& stall, cudaStream_t st) {
  char* at = static_cast<char*>(ws);
  int32_t* info = reinterpret_cast<int32_t*>(at);
  at += align256((size_t)ceil_div(M, kTok) * 4);
  char* terms[2] = {at, at + terms_bytes(M, ad->max_rank)};
  at += 2 * terms_bytes(M, ad->max_rank);
  SumArgs sum;
  memset(&sum, 0, sizeof(sum));
  cudaError_t e = cudaSuccess;
  for (int rb = 0; rb < rank_blocks(ad->max_rank) && e == cudaSuccess && !have_terms; ++rb)
    e = launch_pdl(lora_terms_kernel, dim3(ceil_div(M, kTok), 2), dim3(256), 0, st,
                   lora_grad_terms(ad, ids, M, rb, t, tsplits, ldt, sx, s, ws));
  const int splits = grad_splits(ad, M), shares = grad_shares(ad, splits);
  size_t off = 0;
  for (int rb = 0; rb < rank_blocks(ad->max_rank) && e == cudaSuccess; ++rb) {
    const int rc = block_ranks(ad->max_rank, rb), npad = block_pad(ad->max_rank, rb);
    GradJobs j;
    memset(&j, 0, sizeof(j));
    char* part = at;
    for (int side = 0; side < 2; ++side) {
      const int D = side ? ad->N : ad->K;
      const bool codes = !side && sx;
      float* out = side ? dbt : da;
      uint8_t* has = reinterpret_cast<uint8_t*>(part) + align256((size_t)splits * ad->R * D * sizeof(float));
      if (splits > 1) sum.job[side] = {reinterpret_cast<float*>(part), has, out, splits, D, ceil_div(D, 1024)};
      GradMaps& maps = j.maps[side];
      bool ok = map_2d(&maps.terms, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, terms[side] + off, npad, M, (uint64_t)npad * 2,
                       64, kTok, true);
      ok = ok && (codes ? map_2d(&maps.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, x, D, M, ldx, kD, kTok, false)
                  : side ? map_2d(&maps.x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dy, D, M, (uint64_t)ldd * 2, 64, kTok, true)
                         : map_2d(&maps.x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, D, M, (uint64_t)ldx * 2, 64, kTok, true));
      if (!ok) return cudaErrorInvalidValue;
      j.args[side] = {ids, ad->off, info, M, D, ad->L, ad->R, ad->max_rank, 64 * rb,
                      splits > 1 ? reinterpret_cast<float*>(part) : out, splits, ceil_div(D, kD), shares, has, header, stall};
      part += part_bytes(ad, M, D);
    }
    e = sx ? launch_ranks<true>(rc, j, st) : launch_ranks<false>(rc, j, st);
    off += align256((size_t)M * npad * 2);
  }
  if (e == cudaSuccess && sum.job[0].blocks + sum.job[1].blocks > 0) {
    sum.off = ad->off;
    sum.R = ad->R;
    sum.max_rank = ad->max_rank;
    e = launch_pdl(lora_sum_kernel, dim3(sum.job[0].blocks + sum.job[1].blocks, ad->L, std::min(ad->max_rank, 16)), dim3(256),
                   0, st, sum);
  }
  return e;
}

}  // namespace aq
