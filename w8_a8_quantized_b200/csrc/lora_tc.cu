// Adapters of more than 64 tokens (prefill, training) on the 5th-generation tensor
// cores, ranks up to 64: the two contractions of lora.cu over tiles of 128 tokens.
// Both are bound by the bytes of the long axis (x; y and out), so everything around
// the products is there to keep TMA copies in flight.  Expanding 8192 tokens to 14336 columns
// (bf16) takes 90 us: at the copy rate while it runs, after 8 us of waiting, list and terms.
//
// A tile's adapters are listed once.  Products of each adapter go to accumulator
// columns of its own and a token's row takes those of its adapter: a row is never
// mixed with another adapter's, whatever that holds.
#include <algorithm>
#include <cstring>

#include "lora.cuh"
#include "tc_bf16.cuh"

namespace aq {
namespace {

constexpr int kTok = 128;      // tokens of a tile
constexpr int kMaxTcRank = 64;

struct TcTable {
  const uint16_t* w;   // [R][D]
  const int32_t* off;
  const float* scale;
  int D, L, R, max_rank;
  int rp;              // max_rank rounded up to 16
};

struct TcList {
  int n;
  int row0[kTok], rank[kTok];
  float scale[kTok];
  uint32_t mask[kTok][4];  // rows of the tile that have the adapter, a word per 32
  int slot[kTok];          // of each row: list index or -1
  int id[kTok];
  int first[kTok];
  int count[4];
};

// By the first 128 threads of the block; all threads call it.
__device__ void list_tile(const TcTable& t, const int32_t* ids, int m0, int M, TcList& q) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int v = -1, row0 = 0, rank = 0;
  if (tid < kTok) {
    if (m0 + tid < M) v = __ldg(ids + m0 + tid);
    if (v < 0 || v >= t.L) v = -1;
    if (v >= 0) {
      row0 = min(max(__ldg(t.off + v), 0), t.R);
      rank = min(min(max(__ldg(t.off + v + 1), row0), t.R) - row0, t.max_rank);
      if (rank == 0) v = -1;
    }
    q.id[tid] = v;
  }
  __syncthreads();
  uint32_t mk[4] = {};
  bool first = false;
  unsigned vote = 0;
  int lead = 0;
  if (tid < kTok) {
#pragma unroll
    for (int w = 3; w >= 0; --w) {
      // lanes of word w with this id, read 32 ids at a time
      const int other = q.id[32 * w + lane];
      uint32_t bits = 0;
#pragma unroll
      for (int j = 0; j < 32; ++j) bits |= (uint32_t)(__shfl_sync(0xffffffffu, other, j) == v) << j;
      mk[w] = bits;
      if (bits) lead = 32 * w + __ffs(bits) - 1;
    }
    first = v >= 0 && lead == tid;
    vote = __ballot_sync(0xffffffffu, first);
    if (lane == 0) q.count[warp] = __popc(vote);
  }
  __syncthreads();
  if (tid < kTok) {
    int idx = __popc(vote & ((1u << lane) - 1));
    for (int w = 0; w < warp; ++w) idx += q.count[w];
    if (first) {
      q.first[tid] = idx;
      q.row0[idx] = row0;
      q.rank[idx] = rank;
      q.scale[idx] = __ldg(t.scale + v);
#pragma unroll
      for (int w = 0; w < 4; ++w) q.mask[idx][w] = mk[w];
    }
    if (tid == 0) q.n = q.count[0] + q.count[1] + q.count[2] + q.count[3];
  }
  __syncthreads();
  if (tid < kTok) q.slot[tid] = v >= 0 ? q.first[lead] : -1;
  __syncthreads();
}

// ---------------------------------------------------------------- shrink
// P[split][m][i] = c_l sum over the split's columns of x[m][k] A_l[i][k]:
// D[128 tokens][ranks of the pass's adapters] += x[128][64 k] A[ranks][64 k]^T.
// Tensor memory sums 1024 columns at a time, registers (rounding to nearest) the rest.
constexpr int kSThreads = 256;
constexpr int kSX = 4, kSW = 4;        // rings of activations and of table rows
constexpr int kSCols = 128;            // accumulator columns of one buffer
constexpr int kSUnit = 16;             // steps summed in tensor memory

struct ShrinkMaps {
  CUtensorMap x, w;
};
struct ShrinkTcArgs {
  TcTable t;
  const int32_t* ids;
  int M, splits;
  float* p;
  int32_t* counts;  // [tiles]: adapters of a tile, for the expansion
  void* ws;
  Stall stall;      // (the activations' producer stops)
};

template <int RC>
struct ShrinkShape {
  static constexpr int kX = kTok * 128, kW = RC * 128;
  static constexpr int kCap = kSCols / RC;  // adapters of a pass
  static constexpr int kCtrl = 512;
  static constexpr int kSmem = 1024 + kSX * kX + kSW * kMaxTcRank * 128 + kCtrl + (int)sizeof(TcList);
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs per SM");
};

template <int RC>
__global__ void __launch_bounds__(kSThreads, 2)
    lora_shrink_tc_kernel(const __grid_constant__ ShrinkMaps maps, const __grid_constant__ ShrinkTcArgs a) {
  using Sh = ShrinkShape<RC>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  auto xbuf = [&](int i) { return smem + i * Sh::kX; };
  auto wbuf = [&](int i) { return smem + kSX * Sh::kX + i * kMaxTcRank * 128; };
  uint8_t* ctrl = smem + kSX * Sh::kX + kSW * kMaxTcRank * 128;
  uint64_t* x_full = reinterpret_cast<uint64_t*>(ctrl);
  uint64_t* x_free = x_full + kSX;
  uint64_t* w_full = x_free + kSX;
  uint64_t* w_free = w_full + kSW;
  uint64_t* acc_full = w_free + kSW;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drain = acc_empty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* never_flag = abort_flag + 1;
  TcList& q = *reinterpret_cast<TcList*>(ctrl + Sh::kCtrl);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int m0 = blockIdx.x * kTok, split = blockIdx.y;
  const TcTable& t = a.t;
  if (tid == 0) {
    for (int i = 0; i < kSX; ++i) {
      mbar_init(&x_full[i], 1);
      mbar_init(&x_free[i], 1);
    }
    for (int i = 0; i < kSW; ++i) {
      mbar_init(&w_full[i], 1);
      mbar_init(&w_free[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 4);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *never_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.x);
    prefetch_tmap(&maps.w);
  }
  pdl_wait();
  list_tile(t, a.ids, m0, a.M, q);
  const int na = q.n;
  if (tid == 0 && split == 0) a.counts[blockIdx.x] = na;
  if (na == 0) return;
  if (warp == 1) {
    tmem_alloc(tmem_slot, 2 * kSCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_launch_dependents();  // after the allocation: see lora_grad_kernel
  auto fail = [&](int info) {
    *abort_flag = 1;
    record_error(a.ws, AQ_ERR_TIMEOUT, info, 0);
  };
  const int steps = (t.D + 63) / 64;
  const int s0 = (int)((long long)steps * split / a.splits), s1 = (int)((long long)steps * (split + 1) / a.splits);
  bool ok = true;

  if (warp == 0) {
    if (lane == 0) {
      Ring xr{0, 0};
      int loads = 0;
      for (int p0 = 0; ok && p0 < na; p0 += Sh::kCap)
        for (int s = s0; s < s1; ++s) {
          if (a.stall.stop_after >= 0 && loads++ == a.stall.stop_after) {
            stalled(abort_flag, a.stall.wait_ns);
            ok = false;
            break;
          }
          if (!mbar_wait(&x_free[xr.i], xr.ph ^ 1u, abort_flag, a.stall.wait_ns)) {
            fail(31);
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&x_full[xr.i], Sh::kX);
          tma_load_2d(xbuf(xr.i), &maps.x, 64 * s, m0, &x_full[xr.i]);
          xr.template next<kSX>();
        }
      if (!ok || *abort_flag) grace();
    }
  } else if (warp == 2) {
    if (lane == 0) {
      Ring wr{0, 0};
      for (int p0 = 0; ok && p0 < na; p0 += Sh::kCap) {
        const int p1 = min(p0 + Sh::kCap, na);
        for (int s = s0; ok && s < s1; ++s)
          for (int i = p0; i < p1; ++i) {
            if (!mbar_wait(&w_free[wr.i], wr.ph ^ 1u, abort_flag, a.stall.wait_ns)) {
              fail(32);
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&w_full[wr.i], Sh::kW);
            tma_load_2d(wbuf(wr.i), &maps.w, 64 * s, q.row0[i], &w_full[wr.i]);
            wr.template next<kSW>();
          }
      }
      if (!ok || *abort_flag) grace();
    }
  } else if (warp == 1) {
    constexpr uint32_t idesc = idesc_bf16(RC, false, false);
    const uint64_t xdesc = sw128_desc(smem_u32(xbuf(0))), wdesc = sw128_desc(smem_u32(wbuf(0)));
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
    Ring xr{0, 0}, wr{0, 0}, ar{0, 0};
    bool issued = false;
    for (int p0 = 0; ok && p0 < na; p0 += Sh::kCap) {
      const int p1 = min(p0 + Sh::kCap, na);
      for (int s = s0; ok && s < s1; ++s) {
        const int in_unit = (s - s0) % kSUnit;
        if (in_unit == 0 && !__all_sync(0xffffffffu, mbar_wait(&acc_empty[ar.i], ar.ph ^ 1u, abort_flag, a.stall.wait_ns))) {
          fail(33);
          ok = false;
          break;
        }
        if (!__all_sync(0xffffffffu, mbar_wait(&x_full[xr.i], xr.ph, abort_flag, a.stall.wait_ns))) {
          fail(34);
          ok = false;
          break;
        }
        for (int i = p0; i < p1; ++i) {
          if (!__all_sync(0xffffffffu, mbar_wait(&w_full[wr.i], wr.ph, abort_flag, a.stall.wait_ns))) {
            fail(35);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem + ar.i * kSCols + (i - p0) * RC;
          const uint64_t xo = xdesc + (uint64_t)((xr.i * Sh::kX) >> 4), wo = wdesc + (uint64_t)((wr.i * kMaxTcRank * 128) >> 4);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_bf16(d, xo + 2 * k, wo + 2 * k, idesc, in_unit > 0 || k > 0);
            mma_commit(&w_free[wr.i]);
          }
          __syncwarp();
          issued = true;
          wr.template next<kSW>();
        }
        if (!ok) break;
        const bool last = in_unit == kSUnit - 1 || s + 1 == s1;
        if (elect_one()) {
          mma_commit(&x_free[xr.i]);
          if (last) mma_commit(&acc_full[ar.i]);
        }
        __syncwarp();
        xr.template next<kSX>();
        if (last) ar.template next<2>();
      }
    }
    if (issued) {
      if (elect_one()) mma_commit(drain);
      __syncwarp();
      mbar_wait(drain, 0, never_flag, a.stall.wait_ns);
    }
  } else if (warp >= 4) {
    const int w = warp & 3, row = 32 * w + lane, mine = q.slot[row];
    float tot[RC];
#pragma unroll
    for (int c = 0; c < RC; ++c) tot[c] = 0.f;
    Ring ar{0, 0};
    for (int p0 = 0; ok && p0 < na; p0 += Sh::kCap) {
      const int p1 = min(p0 + Sh::kCap, na);
      for (int s = s0; s < s1; s += kSUnit) {
        if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[ar.i], ar.ph, abort_flag, a.stall.wait_ns))) {
          fail(36);
          ok = false;
          break;
        }
        tc_fence_after();
        for (int i = p0; i < p1; ++i) {
          if (q.mask[i][w] == 0) continue;
          const uint32_t taddr = tmem_base + ((uint32_t)(32 * w) << 16) + ar.i * kSCols + (i - p0) * RC;
#pragma unroll
          for (int c = 0; c < RC; c += 16) {
            uint32_t v[16];
            tmem_ld16(taddr + c, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              asm volatile("" : "+r"(v[e]));
              if (mine == i) tot[c + e] += __uint_as_float(v[e]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[ar.i]);
        ar.template next<2>();
      }
    }
    if (mine >= 0 && ok) {
      const int rank = q.rank[mine];
      const float sc = q.scale[mine];
      float4* dst = reinterpret_cast<float4*>(a.p + ((size_t)split * a.M + m0 + row) * RC);
#pragma unroll
      for (int c = 0; c < RC; c += 4)
        dst[c / 4] = make_float4(c < rank ? sc * tot[c] : 0.f, c + 1 < rank ? sc * tot[c + 1] : 0.f,
                                 c + 2 < rank ? sc * tot[c + 2] : 0.f, c + 3 < rank ? sc * tot[c + 3] : 0.f);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 2 * kSCols);
  }
}

// ---------------------------------------------------------------- expand
// out = y + S B^T:  D[128 tokens][block of columns] = S_terms[128][ranks] B^T[ranks][block],
// S (fp32) as three bf16 terms, 24 bits, in shared memory for the whole CTA (two, 2^-17 of a
// product, where out is rounded to bf16 and ranks above 48 leave the third no room: it would
// take a slot of y, 4001 x 4096 -> 14336 73 us for 65, and bring nothing that shows beside
// out's rounding, 1.7e-3 of the norm), table rows by asynchronous
// copies that clear the rows behind the adapter's rank, y and out by TMA through
// the same buffer.  Blocks of 128 bf16 or 64 fp32 columns: 32 KiB of y.
// Eight epilogue warps: four per half block, each half with its own stores, so that
// a warp's chain per block (y, sums, back) is short.
constexpr int kEThreads = 512;
constexpr int kEY = 4, kEAcc = 4;
constexpr int kYBytes = 2 * kTok * 128;

struct ExpandMaps {
  CUtensorMap y, out;
};
struct ExpandTcArgs {
  TcTable t;
  const int32_t* ids;
  const int32_t* counts;
  int M, splits, has_y, in_place;
  int tiles, g, extra;  // CTAs of a tile, and those left for tiles of several adapters
  TermsArgs terms;      // rc 0: not wanted
  const float* p;  // [splits][M][rp]
  float* s;        // [M][max_rank] or null
  void* ws;
  Stall stall;     // (y's producer stops)
};

// kEW: slots of table rows, as many as fit (3 for 64 ranks, 5 up to 32): with k slots
// k - 1 loads are on their way.
template <bool F32, int EW, int T>
struct ExpandTcShape {
  static constexpr int kEW = EW;
  static constexpr int kBN = F32 ? 64 : 128, kTerms = T, kPer16 = F32 ? 4 : 8;
  static constexpr int kHalf = 8 * kPer16;  // columns of 128 bytes
  static constexpr int kCtrl = 512;
  static constexpr int smem(int rp) {
    return 1024 + kEY * kYBytes + kTerms * kTok * 128 + kEW * rp * kBN * 2 + kCtrl + (int)sizeof(TcList);
  }
};

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(x), "r"(y)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ void copy16(void* dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}

template <bool F32, int kEW, int T>
__global__ void __launch_bounds__(kEThreads, 1)
    lora_expand_tc_kernel(const __grid_constant__ ExpandMaps maps, const __grid_constant__ ExpandTcArgs a) {
  using Sh = ExpandTcShape<F32, kEW, T>;
  constexpr int BN = Sh::kBN;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  const TcTable& t = a.t;
  const int wslot = t.rp * BN * 2;  // BN / 64 halves of rp rows x 128 bytes
  auto ybuf = [&](int i) { return smem + i * kYBytes; };
  uint8_t* terms = smem + kEY * kYBytes;
  uint8_t* wbase = terms + Sh::kTerms * kTok * 128;
  uint8_t* ctrl = wbase + kEW * wslot;
  uint64_t* y_full = reinterpret_cast<uint64_t*>(ctrl);
  uint64_t* y_free = y_full + kEY;
  uint64_t* w_full = y_free + kEY;
  uint64_t* w_free = w_full + kEW;
  uint64_t* acc_full = w_free + kEW;
  uint64_t* acc_empty = acc_full + kEAcc;
  uint64_t* epi = acc_empty + kEAcc;  // [2]
  uint64_t* drain = epi + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  volatile int* never_flag = abort_flag + 1;
  TcList& q = *reinterpret_cast<TcList*>(ctrl + Sh::kCtrl);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  __shared__ int place[3], sums[2][kEThreads / 32];
  if (tid == 0) {
    for (int i = 0; i < kEY; ++i) {
      mbar_init(&y_full[i], 1);
      mbar_init(&y_free[i], 2);
    }
    for (int i = 0; i < kEW; ++i) {
      mbar_init(&w_full[i], 4);
      mbar_init(&w_free[i], 1);
    }
    for (int i = 0; i < kEAcc; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 8);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&epi[i], 4);
    mbar_init(drain, 1);
    *abort_flag = 0;
    *never_flag = 0;
    fence_mbar_init();
    if (a.has_y) prefetch_tmap(&maps.y);
    prefetch_tmap(&maps.out);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kEAcc * BN);
    tmem_relinquish();
  }
  pdl_wait();
  // This CTA's tile and its part of the tile's columns.  A block of columns takes as much
  // again for every further adapter of the tile, so the CTAs that g per tile leave go to
  // tiles of several adapters, in proportion to those beyond the first.  (4001 tokens of six
  // requests, 4096 -> 14336, five of 32 tiles with two: 66 us, 77 without.)
  int tile = (int)blockIdx.x < a.tiles * a.g ? (int)blockIdx.x / a.g : -1, part = (int)blockIdx.x % a.g, parts = a.g;
  if (a.extra > 0) {
    const int more = tid < a.tiles ? max(__ldcg(a.counts + tid) - 1, 0) : 0;
    const int of_warp = __reduce_add_sync(0xffffffffu, more);
    if (lane == 0) sums[0][warp] = of_warp;
    if (tid == 0) place[0] = -1;
    __syncthreads();
    int total = 0;
    for (int i = 0; i < kEThreads / 32; ++i) total += sums[0][i];
    const int share = total > 0 ? a.extra * more / total : 0;
    int end = share;  // of the tiles up to this thread's
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, end, o);
      if (lane >= o) end += v;
    }
    if (lane == 31) sums[1][warp] = end;
    __syncthreads();
    for (int i = 0; i < warp; ++i) end += sums[1][i];
    const int j = (int)blockIdx.x - a.tiles * a.g;
    if (tile >= 0 ? tid == tile : j >= end - share && j < end) {
      place[0] = tid;
      place[1] = tile >= 0 ? part : a.g + j - (end - share);
      place[2] = a.g + share;
    }
    __syncthreads();
    tile = place[0];
    part = place[1];
    parts = place[2];
  }
  const int M = tile >= 0 ? a.M : 0;  // (a CTA without a part has no tokens and no columns)
  const int m0 = max(tile, 0) * kTok, blocks = tile >= 0 ? (t.D + BN - 1) / BN : 0;
  const int b0 = tile >= 0 ? (int)((long long)blocks * part / parts) : 0;
  const int b1 = tile >= 0 ? (int)((long long)blocks * (part + 1) / parts) : 0;
  list_tile(t, a.ids, m0, M, q);
  const int na = q.n;

  // S as bf16 terms in the 128-byte swizzle, eight ranks per thread and round
  const int per_row = t.rp / 8;
  for (int i = tid; i < kTok * per_row; i += kEThreads) {
    const int r = i / per_row, c8 = i - r * per_row, m = m0 + r;
    if (m >= M) continue;
    const int mine = q.slot[r], rank = mine >= 0 ? q.rank[mine] : 0;
    float v[8] = {};
    if (8 * c8 < rank) {
      const float4* src = reinterpret_cast<const float4*>(a.p + (size_t)m * t.rp) + 2 * c8;
      const size_t step = (size_t)a.M * t.rp / 4;
#pragma unroll 4
      for (int k = 0; k < a.splits; ++k) {
        const float4 x = __ldg(src + k * step), y = __ldg(src + k * step + 1);
        v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
        v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
      }
    }
    uint16_t h[3][8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (8 * c8 + e >= rank) v[e] = 0.f;
      split3(v[e], h[0][e], h[1][e], h[2][e]);
      if (a.s && part == 0 && 8 * c8 + e < t.max_rank) a.s[(size_t)m * t.max_rank + 8 * c8 + e] = v[e];
    }
#pragma unroll
    for (int k = 0; k < Sh::kTerms; ++k) {
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = h[k][2 * e] | ((uint32_t)h[k][2 * e + 1] << 16);
      *reinterpret_cast<uint4*>(terms + k * kTok * 128 + r * 128 + ((c8 ^ (r & 7)) << 4)) =
          make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  fence_proxy_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  pdl_launch_dependents();  // after the allocation: see lora_grad_kernel
  auto fail = [&](int info) {
    *abort_flag = 1;
    record_error(a.ws, AQ_ERR_TIMEOUT, info, 0);
  };
  bool ok = true;
  const bool idle = na == 0 && a.in_place;  // nothing changes

  if ((warp == 2 || warp == 3) && a.terms.rc > 0 && tile >= 0) {
    // ------------------------------------------------------------ terms of the weight gradients, shared by the tile's CTAs
    const int ranks8 = a.terms.rc / 8;
    for (int i = 64 * part + tid - 64; i < 2 * kTok * ranks8; i += 64 * parts) {
      const int job = i / (kTok * ranks8), k = i - job * kTok * ranks8, r = k / ranks8, m = m0 + r;
      if (m < M) write_terms(a.terms, a.terms.job[job], m, (k - r * ranks8) * 8, q.slot[r] >= 0 ? q.rank[q.slot[r]] : 0);
    }
    const int first = m0 + 64 * (warp - 2), n = min(64, M - first);
    if (n > 0 && part == 0) {
      auto id = [&](int i) {
        const int v = i < n ? __ldg(a.ids + first + i) : -1;
        return v >= 0 && v < t.L ? v : -1;
      };
      const int lead = id(0), v0 = id(lane), v1 = id(lane + 32);
      const bool same = __all_sync(0xffffffffu, (lane >= n || v0 == lead) && (lane + 32 >= n || v1 == lead));
      if (lane == 0) a.terms.info[first / 64] = same ? lead : -2;
    }
  }
  if (idle) {
  } else if (warp == 0) {
    // ------------------------------------------------------------ y
    if (lane == 0) {
      Ring yr{0, 0};
      for (int b = b0; b < b1; ++b) {
        if (a.stall.stop_after >= 0 && b - b0 == a.stall.stop_after) {
          stalled(abort_flag, a.stall.wait_ns);
          ok = false;
          break;
        }
        if (!mbar_wait(&y_free[yr.i], yr.ph ^ 1u, abort_flag, a.stall.wait_ns)) {
          fail(41);
          ok = false;
          break;
        }
        if (a.has_y) {
          // (a half that starts behind the last column is not copied)
          const bool two = b * BN + Sh::kHalf < t.D;
          mbar_arrive_expect_tx(&y_full[yr.i], two ? kYBytes : kYBytes / 2);
          tma_load_2d(ybuf(yr.i), &maps.y, b * BN, m0, &y_full[yr.i]);
          if (two) tma_load_2d(ybuf(yr.i) + kYBytes / 2, &maps.y, b * BN + Sh::kHalf, m0, &y_full[yr.i]);
        } else {
          mbar_arrive(&y_full[yr.i]);
        }
        yr.template next<kEY>();
      }
      if (!ok || *abort_flag) grace();
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA
    constexpr uint32_t idesc = idesc_bf16(BN, false, true);
    const uint64_t sdesc = sw128_desc(smem_u32(terms)), wdesc = mn_desc(smem_u32(wbase), t.rp * 128);
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_base, 0);
    Ring wr{0, 0}, ar{0, 0};
    bool issued = false;
    for (int b = b0; ok && b < b1; ++b)
      for (int i = 0; i < na; ++i) {
        if (!__all_sync(0xffffffffu, mbar_wait(&acc_empty[ar.i], ar.ph ^ 1u, abort_flag, a.stall.wait_ns) &&
                                         mbar_wait(&w_full[wr.i], wr.ph, abort_flag, a.stall.wait_ns))) {
          fail(42);
          ok = false;
          break;
        }
        tc_fence_after();
        const int ks = __shfl_sync(0xffffffffu, (q.rank[i] + 15) / 16, 0);
        const uint64_t wo = wdesc + (uint64_t)((wr.i * wslot) >> 4);
        if (elect_one()) {
          for (int sp = Sh::kTerms - 1; sp >= 0; --sp)
            for (int k = 0; k < ks; ++k)
              mma_bf16(tmem + ar.i * BN, sdesc + (uint64_t)((sp * kTok * 128) >> 4) + 2 * k, wo + 128 * k, idesc,
                       sp < Sh::kTerms - 1 || k > 0);
          mma_commit(&w_free[wr.i]);
          mma_commit(&acc_full[ar.i]);
        }
        __syncwarp();
        issued = true;
        wr.template next<kEW>();
        ar.template next<kEAcc>();
      }
    if (issued) {
      if (elect_one()) mma_commit(drain);
      __syncwarp();
      mbar_wait(drain, 0, never_flag, a.stall.wait_ns);
    }
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------ table rows
    const int lt = tid - 128;
    Ring wr{0, 0}, pr{0, 0};  // the slot being filled, the slot being published
    int pending = 0;          // loads on their way
    auto publish = [&]() {    // the oldest has landed
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&w_full[pr.i]);
      pr.template next<kEW>();
      --pending;
    };
    for (int b = b0; ok && b < b1; ++b)
      for (int i = 0; i < na; ++i) {
        if (pending == kEW - 1) {
          asm volatile("cp.async.wait_group %0;" ::"n"(kEW - 2) : "memory");
          publish();
        }
        if (!__all_sync(0xffffffffu, mbar_wait(&w_free[wr.i], wr.ph ^ 1u, abort_flag, a.stall.wait_ns))) {
          fail(43);
          ok = false;
          break;
        }
        const int rank = q.rank[i], rows = (rank + 15) & ~15;
        uint8_t* dst = wbase + wr.i * wslot;
        const uint16_t* src = t.w + (size_t)q.row0[i] * t.D + b * BN;
        for (int j = lt; j < rows * (BN / 8); j += 128) {
          const int r = j / (BN / 8), c = j % (BN / 8);
          const bool in = r < rank && b * BN + 8 * c < t.D;
          copy16(dst + (c >> 3) * t.rp * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4), in ? src + (size_t)r * t.D + 8 * c : t.w,
                 in);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        wr.template next<kEW>();
        ++pending;
      }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    while (pending) publish();
  } else if (warp >= 8) {
    // ------------------------------------------------------------ epilogue
    const int w = warp & 3, half = (warp - 8) >> 2, row = 32 * w + lane, mine = q.slot[row];
    const bool stores = w == 0 && lane == 0;
    constexpr int HC = BN / 2, kLd = HC / 16, kPer = 16 / Sh::kPer16;  // columns, loads, chunks per load
    Ring yr{0, 0}, ar{0, 0};
    uint32_t phase = 0;
    int freed = 0;  // next y buffer to hand back
    for (int b = b0; ok && b < b1; ++b) {
      uint8_t* ybase = ybuf(yr.i) + half * (kYBytes / 2);
      uint4* yrow = reinterpret_cast<uint4*>(ybase + row * 128);  // chunk c of the row at c ^ (row & 7)
      if (!__all_sync(0xffffffffu, mbar_wait(&y_full[yr.i], yr.ph, abort_flag, a.stall.wait_ns))) {
        fail(44);
        ok = false;
        break;
      }
      uint4 y[8];
#pragma unroll
      for (int c = 0; c < 8; ++c) y[c] = a.has_y ? yrow[c ^ (row & 7)] : make_uint4(0, 0, 0, 0);
      for (int i = 0; i < na; ++i) {
        if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[ar.i], ar.ph, abort_flag, a.stall.wait_ns))) {
          fail(45);
          ok = false;
          break;
        }
        tc_fence_after();
        if (q.mask[i][w]) {
          const uint32_t taddr = tmem_base + ((uint32_t)(32 * w) << 16) + ar.i * BN + half * HC;
          uint32_t v[kLd][16];
#pragma unroll
          for (int c = 0; c < kLd; ++c) tmem_ld16(taddr + 16 * c, v[c]);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < kLd; ++c)
#pragma unroll
            for (int e = 0; e < 16; ++e) asm volatile("" : "+r"(v[c][e]));
          if (mine == i) {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const uint32_t* d = &v[c / kPer][(c % kPer) * Sh::kPer16];
              uint32_t o[4] = {y[c].x, y[c].y, y[c].z, y[c].w};
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                if constexpr (F32) {
                  o[e] = __float_as_uint(__uint_as_float(o[e]) + __uint_as_float(d[e]));
                } else {
                  const __nv_bfloat162 s2 =
                      __floats2bfloat162_rn(__uint_as_float(o[e] << 16) + __uint_as_float(d[2 * e]),
                                            __uint_as_float(o[e] & 0xFFFF0000u) + __uint_as_float(d[2 * e + 1]));
                  o[e] = *reinterpret_cast<const uint32_t*>(&s2);
                }
              }
              y[c] = make_uint4(o[0], o[1], o[2], o[3]);
            }
          }
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&acc_empty[ar.i]);
        ar.template next<kEAcc>();
      }
      if (!ok) break;
      if (mine >= 0 || !a.has_y)
#pragma unroll
        for (int c = 0; c < 8; ++c) yrow[c ^ (row & 7)] = y[c];
      fence_proxy_async_smem();
      __syncwarp();
      // every warp waits: one that ran ahead would arrive for the next block in place of
      // one that has not finished this block
      if (lane == 0) mbar_arrive(&epi[half]);
      if (!__all_sync(0xffffffffu, mbar_wait(&epi[half], phase, abort_flag, a.stall.wait_ns))) {
        fail(46);
        break;
      }
      if (stores) {
        if (b * BN + half * Sh::kHalf < t.D) tma_store_2d(&maps.out, ybase, b * BN + half * Sh::kHalf, m0);
        bulk_commit();
        if (b > b0) {  // the store before this one has read its buffer
          bulk_wait_read<1>();
          mbar_arrive(&y_free[freed]);
          freed = freed + 1 == kEY ? 0 : freed + 1;
        }
      }
      phase ^= 1u;
      __syncwarp();
      yr.template next<kEY>();
    }
    if (stores) bulk_wait_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kEAcc * BN);
  }
}

// ---------------------------------------------------------------- host side
int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }

TcTable table(const aq_lora* ad, bool b_side) {
  const int rp = (ad->max_rank + 15) / 16 * 16;
  return b_side ? TcTable{ad->bt, ad->off, ad->scale, ad->N, ad->L, ad->R, ad->max_rank, rp}
                : TcTable{ad->a, ad->off, ad->scale, ad->K, ad->L, ad->R, ad->max_rank, rp};
}

template <int RC>
cudaError_t launch_shrink(const ShrinkMaps& maps, const ShrinkTcArgs& a, cudaStream_t st) {
  using Sh = ShrinkShape<RC>;
  cudaError_t e = ensure_smem_attr<lora_shrink_tc_kernel<RC>>(Sh::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(lora_shrink_tc_kernel<RC>, dim3(ceil_div(a.M, kTok), a.splits), dim3(kSThreads), (size_t)Sh::kSmem, st,
                    maps, a);
}

template <bool F32, int EW, int T>
cudaError_t launch_expand(const ExpandMaps& maps, ExpandTcArgs a, cudaStream_t st) {
  using Sh = ExpandTcShape<F32, EW, T>;
  constexpr int most = EW == 5 ? 32 : F32 || T == 2 ? kMaxTcRank : 48;  // ranks
  static_assert(Sh::smem(most) + 512 <= 227 * 1024, "shared memory");
  cudaError_t e = ensure_smem_attr<lora_expand_tc_kernel<F32, EW, T>>(Sh::smem(most));
  if (e != cudaSuccess) return e;
  // column ranges per tile: the fewest blocks on the longest path, counting the
  // start of a CTA (list, terms, first copies) as four blocks
  const int tiles = ceil_div(a.M, kTok), blocks = ceil_div(a.t.D, Sh::kBN), sms = num_sms();
  a.tiles = tiles;
  a.g = 1;
  long long cost = 0;
  for (int waves = 1; waves <= 6; ++waves) {
    const int g = std::max(1, std::min(blocks, waves * sms / tiles));
    const long long c = (long long)ceil_div((long long)tiles * g, sms) * (ceil_div(blocks, g) + 4);
    if (cost == 0 || c < cost) {
      cost = c;
      a.g = g;
    }
  }
  // the rest of the last wave (a thread of the kernel looks after each tile)
  a.extra = a.t.L > 1 && tiles <= kEThreads && a.g < blocks ? ceil_div((long long)tiles * a.g, sms) * sms - tiles * a.g : 0;
  return launch_pdl(lora_expand_tc_kernel<F32, EW, T>, dim3(tiles * a.g + a.extra), dim3(kEThreads), (size_t)Sh::smem(a.t.rp), st,
                    maps, a);
}

}  // namespace

bool lora_tc_fits(const aq_lora* ad, int M) { return M > 64 && ad->max_rank <= kMaxTcRank; }

int lora_tc_splits(int M, int D) {
  // two CTAs per SM, eight or more steps each
  const int tiles = ceil_div(M, kTok), steps = ceil_div(D, 64);
  return std::max(1, std::min({2 * num_sms() / tiles, steps / 8, 16}));
}

size_t lora_tc_count_bytes(int M) { return (size_t)ceil_div(M, kTok) * 4; }

cudaError_t launch_lora_shrink_tc(const aq_lora* ad, bool b_side, const uint16_t* x, int ldx, const int32_t* ids, int M,
                                  float* p, int32_t* counts, void* header, const Stall& stall, cudaStream_t st) {
  const TcTable t = table(ad, b_side);
  ShrinkMaps maps;
  memset(&maps, 0, sizeof(maps));
  if (!map_2d(&maps.x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, x, t.D, M, (uint64_t)ldx * 2, 64, kTok, true) ||
      !map_2d(&maps.w, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, t.w, t.D, t.R, (uint64_t)t.D * 2, 64, t.rp, true))
    return cudaErrorInvalidValue;
  const ShrinkTcArgs a{t, ids, M, lora_tc_splits(M, t.D), p, counts, header, stall};
  switch (t.rp) {
    case 16: return launch_shrink<16>(maps, a, st);
    case 32: return launch_shrink<32>(maps, a, st);
    case 48: return launch_shrink<48>(maps, a, st);
    case 64: return launch_shrink<64>(maps, a, st);
  }
  return cudaErrorInvalidValue;
}

cudaError_t launch_lora_expand_tc(const aq_lora* ad, bool b_side, const int32_t* ids, int M, const float* p, int splits,
                                  const int32_t* counts, const void* y, int ldy, void* out, int ldo, bool f32, float* s,
                                  const TermsArgs* terms, void* header, const Stall& stall, cudaStream_t st) {
  const TcTable t = table(ad, b_side);
  ExpandMaps maps;
  memset(&maps, 0, sizeof(maps));
  const auto type = f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int elt = f32 ? 4 : 2;
  if (!map_2d(&maps.out, type, out, t.D, M, (uint64_t)ldo * elt, 128 / elt, kTok, true) ||
      (y && !map_2d(&maps.y, type, y, t.D, M, (uint64_t)ldy * elt, 128 / elt, kTok, true)))
    return cudaErrorInvalidValue;
  const ExpandTcArgs a{t, ids, counts, M, splits, y != nullptr, y == out, 0, 0, 0, terms ? *terms : TermsArgs{}, p, s, header, stall};
  if (t.rp <= 32) return f32 ? launch_expand<true, 5, 3>(maps, a, st) : launch_expand<false, 5, 3>(maps, a, st);
  if (f32) return launch_expand<true, 3, 3>(maps, a, st);
  return t.rp <= 48 ? launch_expand<false, 3, 3>(maps, a, st) : launch_expand<false, 3, 2>(maps, a, st);
}

}  // namespace aq
