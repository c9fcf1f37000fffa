// Low-rank adapters of many requests beside a shared projection, and their
// gradients.
//
// Token m has the adapter l = ids[m] (none when ids[m] is outside [0, L)) of
// rank r_l, with A_l [r_l][K] and B_l^T [r_l][N] stored as rows
// off[l] .. off[l+1]-1 of two bf16 tables:
//   forward   S[m][r] = c_l sum_k x[m][k] A_l[r][k]
//             out[m][n] = y[m][n] + sum_r S[m][r] B_l^T[r][n]
//   backward  T[m][r] = c_l sum_n dy[m][n] B_l^T[r][n]
//             dx[m][k] = add[m][k] + sum_r T[m][r] A_l[r][k]
//             dA_l[r][k] = sum_m T[m][r] x[m][k];  dB_l^T[r][n] = sum_m S[m][r] dy[m][n]
// so three kernels serve both: contract a long axis to the rank (shrink),
// the rank to a long axis (expand), and the tokens (lora_grad.cu).
//
// Products run on mma.sync (bf16 in, fp32 out): the tables and x, dy are bf16
// (8-bit codes are exact in bf16), and S and T, fp32, enter as three bf16 terms
// (24 significant bits).  Sums are fp32.
//
// A tile is 64 consecutive tokens.  A kernel lists the adapters that occur in
// its tile and runs them one after another on the same activations: requests
// are contiguous in a batch, so a tile has one or two; a decode batch has up to
// 64 in its one tile, which `kz` CTAs share out.  Rows of other adapters are
// never added in but selected out, so that an infinity or NaN in one request's
// adapter or activations stays with that request.
#include <algorithm>

#include "aq_internal.cuh"
#include "lora.cuh"

namespace aq {
namespace {

typedef unsigned long long u64;

constexpr int kTok = 64;       // tokens of a tile
constexpr int kRank = 64;      // ranks of a block
constexpr int kMaxRank = 256;  // largest rank of an adapter
constexpr int kThreads = 256;  // 8 warps
constexpr int kDC = 128;       // columns of a chunk of the long axis
constexpr int kLd = kDC + 8;   // row pitch in shared memory: 17 x 16 bytes, conflict-free for ldmatrix

struct Table {  // one of the two tables of an adapter set
  const uint16_t* w;   // [R][D]
  const int32_t* off;  // [L + 1]
  const float* scale;  // [L]
  int D, L, R, max_rank;
};

// Rows of adapter l, kept inside the table whatever `off` holds.
__device__ __forceinline__ void rows_of(const Table& t, int l, int& row0, int& rank) {
  const int a = min(max(__ldg(t.off + l), 0), t.R), b = min(max(__ldg(t.off + l + 1), a), t.R);
  row0 = a;
  rank = min(b - a, t.max_rank);
}

// The adapters of a tile that this CTA handles.
struct TileList {
  int n;             // adapters
  int row0[kTok];    // first table row of the rank block
  int rank[kTok];    // ranks of the block
  float scale[kTok];
  u64 mask[kTok];    // tokens of the tile that have it
  int slot[kTok];    // of each token: list index, -1 another CTA's, -2 no adapter (or none in this rank block)
  int id[kTok];
  int first[kTok];
  int count[2];
};

// Ranks from rb0 on; of the adapters that have some, those with index = zi mod kz.
__device__ void list_tile(const Table& t, const int32_t* ids, int m0, int M, int rb0, int zi, int kz, TileList& q) {
  const int tid = threadIdx.x, lane = tid & 31;
  int v = -1, row0 = 0, rank = 0;
  if (tid < kTok) {
    if (m0 + tid < M) v = __ldg(ids + m0 + tid);
    if (v < 0 || v >= t.L) v = -1;
    if (v >= 0) {
      rows_of(t, v, row0, rank);
      rank -= rb0;
      if (rank <= 0) v = -1;
    }
    q.id[tid] = v;
  }
  __syncthreads();
  u64 mk = 0;
  bool first = false;
  unsigned vote = 0;
  if (tid < kTok) {
#pragma unroll 8
    for (int j = 0; j < kTok; ++j) mk |= (u64)(q.id[j] == v) << j;
    first = v >= 0 && __ffsll((long long)mk) - 1 == tid;
    vote = __ballot_sync(0xffffffffu, first);
    if (lane == 0) q.count[tid >> 5] = __popc(vote);
  }
  __syncthreads();
  if (tid < kTok) {
    const int idx = (tid >= 32 ? q.count[0] : 0) + __popc(vote & ((1u << lane) - 1));
    if (first) {
      q.first[tid] = idx;
      if (idx % kz == zi) {
        const int a = idx / kz;
        q.row0[a] = row0 + rb0;
        q.rank[a] = rank;
        q.scale[a] = __ldg(t.scale + v);
        q.mask[a] = mk;
      }
    }
    if (tid == 0) {
      const int all = q.count[0] + q.count[1];
      q.n = all > zi ? (all - zi + kz - 1) / kz : 0;
    }
  }
  __syncthreads();
  if (tid < kTok) {
    int s = -2;
    if (v >= 0) {
      const int idx = q.first[__ffsll((long long)mk) - 1];
      s = idx % kz == zi ? idx / kz : -1;
    }
    q.slot[tid] = s;
  }
  __syncthreads();
}

__device__ __forceinline__ void cp16(void* dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(in ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p)));
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], const void* p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(smem_u32(p)));
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ---------------------------------------------------------------- shrink
struct ShrinkArgs {
  Table t;
  const uint16_t* x;
  int ldx, M;
  const int32_t* ids;
  float* p;  // [splits][M][max_rank]
  int splits, kz;
};

struct ShrinkSmem {
  uint16_t x[3][kTok][kLd];
  uint16_t w[3][kRank][kLd];
  float s[2][kTok][kRank];
  TileList q;
};

__global__ void __launch_bounds__(kThreads) lora_shrink_kernel(const ShrinkArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  ShrinkSmem& sm = *reinterpret_cast<ShrinkSmem*>(raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int m0 = blockIdx.x * kTok, split = blockIdx.y, zi = blockIdx.z % a.kz, rb0 = blockIdx.z / a.kz * kRank;
  const Table& t = a.t;
  pdl_launch_dependents();
  pdl_wait();
  list_tile(t, a.ids, m0, a.M, rb0, zi, a.kz, sm.q);
  const int na = sm.q.n;
  if (na == 0) return;
  const int chunks = (t.D + kDC - 1) / kDC;
  const int c0 = (int)((long long)chunks * split / a.splits), c1 = (int)((long long)chunks * (split + 1) / a.splits);
  for (int i = tid; i < 2 * kTok * kRank; i += kThreads) (&sm.s[0][0][0])[i] = 0.f;

  // items: (chunk, adapter), adapters inside
  const int items = (c1 - c0) * na;
  int ic = c0, ia = 0, is = 0, ix = 2;  // next item to issue: its chunk, adapter, table slot, activation slot
  auto issue = [&]() {
    if (ic < c1) {
      const int d0 = ic * kDC;
      if (ia == 0) {
        ix = ix == 2 ? 0 : ix + 1;
        for (int i = tid; i < kTok * (kDC / 8); i += kThreads) {
          const int r = i / (kDC / 8), c = i % (kDC / 8) * 8;
          const bool in = m0 + r < a.M && d0 + c < t.D;
          cp16(&sm.x[ix][r][c], in ? a.x + (size_t)(m0 + r) * a.ldx + d0 + c : a.x, in);
        }
      }
      const int nr = min(sm.q.rank[ia], kRank), row0 = sm.q.row0[ia];
      const int rows = (nr + 15) & ~15;
      for (int i = tid; i < rows * (kDC / 8); i += kThreads) {
        const int r = i / (kDC / 8), c = i % (kDC / 8) * 8;
        const bool in = r < nr && d0 + c < t.D;
        cp16(&sm.w[is][r][c], in ? t.w + (size_t)(row0 + r) * t.D + d0 + c : t.w, in);
      }
      is = is == 2 ? 0 : is + 1;
      if (++ia == na) {
        ia = 0;
        ++ic;
      }
    }
    cp_commit();
  };
  issue();
  issue();
  const int sub = warp & 3, kh = warp >> 2;
  float acc[kRank / 8][4];
#pragma unroll
  for (int j = 0; j < kRank / 8; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
  int al = 0, ws = 0, xs = 0, run = 0;
  for (int it = 0; it < items; ++it) {
    cp_wait<1>();
    __syncthreads();
    issue();
    const u64 mask = sm.q.mask[al];
    const uint32_t mine = (uint32_t)(mask >> (16 * sub)) & 0xFFFFu;
    if (mine) {
      const int nt = (min(sm.q.rank[al], kRank) + 15) / 16;  // pairs of 8-rank tiles
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        const int k0 = 64 * kh + 16 * ks;
        uint32_t fa[4];
        ldsm4(fa, &sm.x[xs][16 * sub + (lane & 7) + 8 * ((lane >> 3) & 1)][k0 + 8 * (lane >> 4)]);
#pragma unroll
        for (int j = 0; j < kRank / 16; ++j) {
          if (j < nt) {
            uint32_t fb[4];
            ldsm4(fb, &sm.w[ws][16 * j + (lane & 7) + 8 * (lane >> 4)][k0 + 8 * ((lane >> 3) & 1)]);
            mma16816(acc[2 * j], fa, fb[0], fb[1]);
            mma16816(acc[2 * j + 1], fa, fb[2], fb[3]);
          }
        }
      }
      // the tokens of this adapter take the products over (a run of 8 chunks
      // where the tile has one adapter)
      if (na > 1 || ++run == 8 || it + 1 == items) {
        run = 0;
#pragma unroll
        for (int j = 0; j < kRank / 8; ++j) {
          if (j < 2 * nt) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int r = (lane >> 2) + 8 * (e >> 1);
              if ((mine >> r) & 1u) sm.s[kh][16 * sub + r][8 * j + 2 * (lane & 3) + (e & 1)] += acc[j][e];
              acc[j][e] = 0.f;
            }
          }
        }
      }
    }
    ws = ws == 2 ? 0 : ws + 1;
    if (++al == na) {
      al = 0;
      xs = xs == 2 ? 0 : xs + 1;
    }
  }
  cp_wait<0>();
  __syncthreads();
  for (int i = tid; i < kTok * kRank; i += kThreads) {
    const int r = i / kRank, c = i % kRank, s = sm.q.slot[r];
    if (s >= 0 && c < sm.q.rank[s])
      a.p[((size_t)split * a.M + m0 + r) * t.max_rank + rb0 + c] = sm.q.scale[s] * (sm.s[0][r][c] + sm.s[1][r][c]);
  }
}

// ---------------------------------------------------------------- expand
struct ExpandArgs {
  Table t;
  const int32_t* ids;
  int M;
  const float* p;  // [splits][M][max_rank]
  int splits, kz;
  const void* y;   // or null
  void* out;
  int ldy, ldo;
  float* s;        // [M][max_rank] or null: the summed products
  int rp;          // ranks of a tile's products in shared memory: max_rank rounded up to 16
  int wrows;       // table rows per slot: min(rp, kRank)
};

// A CTA takes one tile of tokens and a range of column blocks: the list of
// adapters and the products' bf16 terms are made once, then the blocks stream
// through two buffers of table rows and two of y (16-byte copies, one item
// ahead); sums go into the y buffer and leave it as 16-byte stores.
// F32: fp32 y and out, 64 columns a block; otherwise bf16, 128 columns.  Three terms
// of S, 24 bits.
template <bool F32>
struct ExpandShape {
  static constexpr int kBN = F32 ? 64 : 128, kTerms = 3;
  static constexpr int kLdW = kBN + 8;                // bf16 elements
  static constexpr int kElt = F32 ? 4 : 2, kPer16 = 16 / kElt;
  static constexpr int kLdY = kBN + kPer16;           // elements of y: rows of 272 bytes
  static constexpr int kYBytes = kTok * kLdY * kElt;
  static constexpr int kNt = kBN / 16;                // 8-column tiles of a warp (half the block)
  static size_t smem(int rp) {
    return sizeof(TileList) + 2 * kYBytes + 2 * (size_t)std::min(rp, kRank) * kLdW * 2 +
           (size_t)kTerms * kTok * (rp + 8) * 2;
  }
};

template <bool F32>
__global__ void __launch_bounds__(kThreads, 2) lora_expand_kernel(const ExpandArgs a) {
  using Sh = ExpandShape<F32>;
  constexpr int BN = Sh::kBN, NT = Sh::kNt;
  extern __shared__ __align__(16) uint8_t raw[];
  TileList& q = *reinterpret_cast<TileList*>(raw);
  uint8_t* ybuf = raw + sizeof(TileList);
  uint16_t* wbuf = reinterpret_cast<uint16_t*>(ybuf + 2 * Sh::kYBytes);
  uint16_t* terms = wbuf + 2 * a.wrows * Sh::kLdW;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int m0 = blockIdx.y * kTok, zi = blockIdx.z;
  const Table& t = a.t;
  const int lds = a.rp + 8, plane = kTok * lds;
  const int blocks = (t.D + BN - 1) / BN;
  const int b0 = (int)((long long)blocks * blockIdx.x / gridDim.x);
  const int b1 = (int)((long long)blocks * (blockIdx.x + 1) / gridDim.x);
  pdl_launch_dependents();
  pdl_wait();
  list_tile(t, a.ids, m0, a.M, 0, zi, a.kz, q);
  const int na = q.n;

  // items: (column block, adapter, block of 64 ranks); a block without an
  // adapter has one empty item
  int ib = b0, ia = 0, ir = 0, is = 0;  // next item to issue
  auto issue = [&]() {
    if (ib < b1) {
      const int n0 = ib * BN;
      if (ia == 0 && ir == 0 && a.y) {
        uint8_t* dst = ybuf + (ib & 1) * Sh::kYBytes;
        for (int i = tid; i < kTok * 16; i += kThreads) {
          const int r = i >> 4, c = (i & 15) * Sh::kPer16, s = q.slot[r];
          const bool in = m0 + r < a.M && n0 + c < t.D && (s >= 0 || (s == -2 && zi == 0));
          const uint8_t* src = static_cast<const uint8_t*>(a.y);
          cp16(dst + (r * Sh::kLdY + c) * Sh::kElt,
               in ? src + ((size_t)(m0 + r) * a.ldy + n0 + c) * Sh::kElt : src, in);
        }
      }
      if (ia < na) {
        const int nr = min(q.rank[ia] - ir, kRank), row0 = q.row0[ia] + ir;
        const int rows = (nr + 15) & ~15;
        uint16_t* dst = wbuf + is * a.wrows * Sh::kLdW;
        for (int i = tid; i < rows * (BN / 8); i += kThreads) {
          const int r = i / (BN / 8), c = i % (BN / 8) * 8;
          const bool in = r < nr && n0 + c < t.D;
          cp16(dst + r * Sh::kLdW + c, in ? t.w + (size_t)(row0 + r) * t.D + n0 + c : t.w, in);
        }
      }
      is ^= 1;
      ir += kRank;
      if (ia >= na || ir >= q.rank[ia]) {
        ir = 0;
        if (++ia >= na) {
          ia = 0;
          ++ib;
        }
      }
    }
    cp_commit();
  };
  issue();

  // S of this tile as bf16 terms, zero behind the token's rank
  for (int r = tid >> 4; r < kTok; r += kThreads / 16) {
    const int s = q.slot[r], m = m0 + r;
    if (s == -1 || m >= a.M) continue;
    const int rank = s >= 0 ? q.rank[s] : 0;
    for (int c = tid & 15; c < a.rp; c += 16) {
      float v = 0.f;
      if (c < rank) {
        const float* src = a.p + (size_t)m * t.max_rank + c;
        const size_t step = (size_t)a.M * t.max_rank;
#pragma unroll 8
        for (int k = 0; k < a.splits; ++k) v += __ldg(src + k * step);
      }
      if (a.s && blockIdx.x == 0 && c < t.max_rank && (s >= 0 || zi == 0)) a.s[(size_t)m * t.max_rank + c] = v;
      uint16_t hi, mid, lo;
      split3(v, hi, mid, lo);
      uint16_t* d = terms + r * lds + c;
      d[0] = hi;
      d[plane] = mid;
      d[2 * plane] = lo;
    }
  }

  const int sub = warp & 3, nh = warp >> 2;
  float delta[NT][4], acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
  int ws = 0;
  for (int b = b0; b < b1; ++b) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) delta[j][e] = 0.f;
    for (int al = 0; al < max(na, 1); ++al) {
      const int rank = al < na ? q.rank[al] : 1;
      const uint32_t mine = al < na ? (uint32_t)(q.mask[al] >> (16 * sub)) & 0xFFFFu : 0u;
      for (int r0 = 0; r0 < rank; r0 += kRank) {
        cp_wait<0>();
        __syncthreads();
        issue();
        if (mine) {
          const uint16_t* w = wbuf + ws * a.wrows * Sh::kLdW;
          const int ksteps = (min(rank - r0, kRank) + 15) / 16;
          for (int ks = 0; ks < ksteps; ++ks) {
            uint32_t fa[Sh::kTerms][4];
#pragma unroll
            for (int sp = 0; sp < Sh::kTerms; ++sp)
              ldsm4(fa[sp], terms + sp * plane + (16 * sub + (lane & 15)) * lds + r0 + 16 * ks + 8 * (lane >> 4));
#pragma unroll
            for (int j = 0; j < NT / 2; ++j) {
              uint32_t fb[4];
              ldsm4t(fb, w + (16 * ks + (lane & 15)) * Sh::kLdW + (BN / 2) * nh + 16 * j + 8 * (lane >> 4));
#pragma unroll
              for (int sp = Sh::kTerms - 1; sp >= 0; --sp) {
                mma16816(acc[2 * j], fa[sp], fb[0], fb[1]);
                mma16816(acc[2 * j + 1], fa[sp], fb[2], fb[3]);
              }
            }
          }
        }
        ws ^= 1;
      }
      if (mine) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if ((mine >> ((lane >> 2) + 8 * (e >> 1))) & 1u) delta[j][e] = acc[j][e];
            acc[j][e] = 0.f;
          }
      }
    }
    uint8_t* yb = ybuf + (b & 1) * Sh::kYBytes;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = 16 * sub + (lane >> 2) + 8 * h;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int c = (BN / 2) * nh + 8 * j + 2 * (lane & 3);
        float v0 = delta[j][2 * h], v1 = delta[j][2 * h + 1];
        if constexpr (F32) {
          float2* d = reinterpret_cast<float2*>(yb + (r * Sh::kLdY + c) * 4);
          const float2 y = a.y ? *d : make_float2(0.f, 0.f);
          *d = make_float2(y.x + v0, y.y + v1);
        } else {
          uint32_t* d = reinterpret_cast<uint32_t*>(yb + (r * Sh::kLdY + c) * 2);
          const uint32_t y = a.y ? *d : 0u;
          const __nv_bfloat162 o =
              __floats2bfloat162_rn(bf16_bits_to_float(y & 0xFFFFu) + v0, bf16_bits_to_float(y >> 16) + v1);
          *d = *reinterpret_cast<const uint32_t*>(&o);
        }
      }
    }
    __syncthreads();
    for (int i = tid; i < kTok * 16; i += kThreads) {
      const int r = i >> 4, c = (i & 15) * Sh::kPer16, s = q.slot[r], n = b * BN + c;
      if (m0 + r < a.M && n < t.D && (s >= 0 || (s == -2 && zi == 0)))
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.out) + ((size_t)(m0 + r) * a.ldo + n) * Sh::kElt) =
            *reinterpret_cast<const uint4*>(yb + (r * Sh::kLdY + c) * Sh::kElt);
    }
  }
  cp_wait<0>();
}

// ---------------------------------------------------------------- host side
int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }
size_t align256(size_t b) { return (b + 255) / 256 * 256; }

Table table_a(const aq_lora* ad) { return {ad->a, ad->off, ad->scale, ad->K, ad->L, ad->R, ad->max_rank}; }
Table table_b(const aq_lora* ad) { return {ad->bt, ad->off, ad->scale, ad->N, ad->L, ad->R, ad->max_rank}; }

// CTAs that share the adapters of one tile: a single tile may hold 64.  An expanding CTA
// makes the terms of all its tokens first, so fewer share there (30 tokens of 22 adapters with
// gradients: 82 us with 8 contracting and 4 expanding, 84 with 4 and 4, 91 with 8 and 8).
int share(int M, const Table& t, int most) { return M <= kTok && t.L > 1 ? std::min(most, t.L) : 1; }

int shrink_splits(int M, const Table& t) {
  const int tiles = ceil_div(M, kTok), chunks = ceil_div(t.D, kDC);
  // at most 16: whoever takes the products adds the parts up, a load after the other (64 tokens,
  // D 14336, with gradients: 37 us with 16, 84 with 112)
  return std::max(1, std::min({chunks, ceil_div(2 * num_sms(), tiles), 16}));
}

// Partial sums of the products: as the kernels that write and read them split the long axis and pitch the rows.
struct Products {
  int splits, ld;
};
Products products(const aq_lora* ad, int M, bool b_side) {
  const Table t = b_side ? table_b(ad) : table_a(ad);
  return lora_tc_fits(ad, M) ? Products{lora_tc_splits(M, t.D), (t.max_rank + 15) / 16 * 16}
                             : Products{shrink_splits(M, t), t.max_rank};
}
size_t sum_bytes(const aq_lora* ad, int M, bool b_side) {
  const Products p = products(ad, M, b_side);
  return align256((size_t)p.splits * M * p.ld * sizeof(float));
}
// with the tiles' adapter counts behind them
size_t p_bytes(const aq_lora* ad, int M, bool b_side) {
  return sum_bytes(ad, M, b_side) + (lora_tc_fits(ad, M) ? align256(lora_tc_count_bytes(M)) : 0);
}

cudaError_t shrink(const Table& t, const uint16_t* x, int ldx, const int32_t* ids, int M, float* p, cudaStream_t st) {
  ShrinkArgs a{t, x, ldx, M, ids, p, shrink_splits(M, t), share(M, t, 8)};
  cudaError_t e = ensure_smem_attr<lora_shrink_kernel>(sizeof(ShrinkSmem));
  if (e != cudaSuccess) return e;
  const dim3 grid(ceil_div(M, kTok), a.splits, a.kz * ceil_div(t.max_rank, kRank));
  return launch_pdl(lora_shrink_kernel, grid, dim3(kThreads), sizeof(ShrinkSmem), st, a);
}

template <bool F32>
cudaError_t launch_expand(const ExpandArgs& a, cudaStream_t st) {
  using Sh = ExpandShape<F32>;
  cudaError_t e = ensure_smem_attr<lora_expand_kernel<F32>>((int)Sh::smem(kMaxRank));
  if (e != cudaSuccess) return e;
  // about six CTAs per SM in all: the last wave is short, and the work that a
  // CTA does once stays a small part of it
  const int tiles = ceil_div(a.M, kTok), blocks = ceil_div(a.t.D, Sh::kBN);
  const dim3 grid(std::max(1, std::min(blocks, ceil_div(6 * num_sms(), tiles * a.kz))), tiles, a.kz);
  return launch_pdl(lora_expand_kernel<F32>, grid, dim3(kThreads), Sh::smem(a.rp), st, a);
}

cudaError_t expand(const Table& t, const int32_t* ids, int M, const float* p, int splits, const void* y, int ldy,
                   void* out, int ldo, int dtype, float* s, cudaStream_t st) {
  const int rp = (t.max_rank + 15) / 16 * 16;
  const ExpandArgs a{t, ids, M, p, splits, share(M, t, 4), y, out, ldy, ldo, s, rp, std::min(rp, kRank)};
  return dtype == AQ_F32 ? launch_expand<true>(a, st) : launch_expand<false>(a, st);
}

// p = the products of x with the a (or b) side; out = y + p's sums times the other side.
cudaError_t shrink_any(const aq_lora* ad, bool b_side, const uint16_t* x, int ldx, const int32_t* ids, int M, float* p,
                       void* header, const Stall& stall, cudaStream_t st) {
  int32_t* counts = reinterpret_cast<int32_t*>(reinterpret_cast<char*>(p) + sum_bytes(ad, M, b_side));
  return lora_tc_fits(ad, M) ? launch_lora_shrink_tc(ad, b_side, x, ldx, ids, M, p, counts, header, stall, st)
                             : shrink(b_side ? table_b(ad) : table_a(ad), x, ldx, ids, M, p, st);
}
cudaError_t expand_any(const aq_lora* ad, bool b_side, const int32_t* ids, int M, const float* p, const void* y, int ldy,
                       void* out, int ldo, int dtype, float* s, const TermsArgs* terms, void* header,
                       const Stall& stall, cudaStream_t st) {
  const int splits = products(ad, M, !b_side).splits;
  const int32_t* counts = reinterpret_cast<const int32_t*>(reinterpret_cast<const char*>(p) + sum_bytes(ad, M, !b_side));
  return lora_tc_fits(ad, M)
             ? launch_lora_expand_tc(ad, b_side, ids, M, p, splits, counts, y, ldy, out, ldo, dtype == AQ_F32, s, terms, header,
                                     stall, st)
             : expand(b_side ? table_b(ad) : table_a(ad), ids, M, p, splits, y, ldy, out, ldo, dtype, s, st);
}

int check_lora(const aq_lora* ad) {
  if (!ad || !ad->a || !ad->bt || !ad->off || !ad->scale) return AQ_ERR_ARG;
  if (ad->N < 8 || ad->K < 8 || ad->N % 8 || ad->K % 8 || ad->N > (1 << 20) || ad->K > (1 << 20)) return AQ_ERR_SHAPE;
  if (ad->L < 1 || ad->R < 1 || ad->max_rank < 1 || ad->max_rank > kMaxRank || ad->max_rank > ad->R) return AQ_ERR_SHAPE;
  if (ad->L > 16383) return AQ_ERR_SHAPE;  // grid rows: up to four rank blocks per adapter
  if (((uintptr_t)ad->a | (uintptr_t)ad->bt) & 15) return AQ_ERR_ARG;
  if (((uintptr_t)ad->off | (uintptr_t)ad->scale) & 3) return AQ_ERR_ARG;
  return AQ_OK;
}

constexpr int kMaxTokens = 65535 * kTok;  // grid rows of the expand kernel

// Rows read or written as 16-byte vectors.
bool bad_rows(const void* p, int ld, int width, int per16) { return !p || ((uintptr_t)p & 15) || ld < width || ld % per16; }
// In place is row by row: the same pointer with another pitch would overwrite rows still to be read.
bool skewed(const void* in, int ldi, const void* out, int ldo, int M) { return in == out && ldi != ldo && M > 1; }
// Any other overlap of an output is refused too: kernels of a call run one after another and CTAs in any order, so
// what was written over an input would be read as the input.
Span rows_at(const void* p, int ld, int width, int elt, int M) { return {p, (size_t)ld * elt, (size_t)width * elt, M}; }

}  // namespace
}  // namespace aq

using namespace aq;

extern "C" size_t aq_lora_workspace_bytes(const aq_lora* ad, int M, int backward) {
  if (check_lora(ad) != AQ_OK || M < 1 || M > kMaxTokens) return 0;
  if (!backward) return lora_decode_fits(ad, M) ? 16 : kWsHeader + p_bytes(ad, M, false);
  return kWsHeader + p_bytes(ad, M, true) + lora_grad_ws_bytes(ad, M);
}

extern "C" int aq_lora_apply(const aq_lora* ad, const uint16_t* x, int ldx, const int32_t* ids, int M, const void* y,
                             int ldy, void* out, int ldo, int ydtype, float* s, void* ws, size_t ws_bytes,
                             void* stream) {
  int rc = check_lora(ad);
  if (rc != AQ_OK) return rc;
  if (M < 1 || M > kMaxTokens || !ids || ((uintptr_t)ids & 3) || ((uintptr_t)s & 3)) return AQ_ERR_ARG;
  if (ydtype != AQ_F32 && ydtype != AQ_BF16) return AQ_ERR_ARG;
  const int per16 = ydtype == AQ_F32 ? 4 : 8;
  if (bad_rows(x, ldx, ad->K, 8) || bad_rows(out, ldo, ad->N, per16) || (y && bad_rows(y, ldy, ad->N, per16)) ||
      skewed(y, ldy, out, ldo, M))
    return AQ_ERR_ARG;
  if (!ws || ws_bytes < aq_lora_workspace_bytes(ad, M, 0)) return AQ_ERR_WORKSPACE;
  if ((uintptr_t)ws & 15) return AQ_ERR_ARG;
  const int elt = ydtype == AQ_F32 ? 4 : 2;
  const Span outs[] = {rows_at(out, ldo, ad->N, elt, M), flat(s, (size_t)M * ad->max_rank * 4)};
  const Span ins[] = {rows_at(y == out ? nullptr : y, ldy, ad->N, elt, M), rows_at(x, ldx, ad->K, 2, M),
                      flat(ids, (size_t)M * 4),
                      flat(ad->a, (size_t)ad->R * ad->K * 2), flat(ad->bt, (size_t)ad->R * ad->N * 2),
                      flat(ad->off, (size_t)(ad->L + 1) * 4), flat(ad->scale, (size_t)ad->L * 4)};
  if (outputs_overlap(outs, ins)) return AQ_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (lora_decode_fits(ad, M))
    return launch_lora_decode(ad, x, ldx, ids, M, y, ldy, out, ldo, ydtype == AQ_F32, s, st) == cudaSuccess ? AQ_OK
                                                                                                            : AQ_ERR_CUDA;
  float* p = reinterpret_cast<float*>(static_cast<char*>(ws) + kWsHeader);
  cudaError_t e = shrink_any(ad, false, x, ldx, ids, M, p, ws, Stall{}, st);
  if (e == cudaSuccess) e = expand_any(ad, true, ids, M, p, y, ldy, out, ldo, ydtype, s, nullptr, ws, Stall{}, st);
  return e == cudaSuccess ? AQ_OK : AQ_ERR_CUDA;
}

// `stalls`: of the contraction, the expansion and the weight gradients.
static int lora_backward(const aq_lora* ad, const uint16_t* dy, int ldd, const int32_t* ids, int M, const float* s,
                         const void* x, int ldx, const float* sx, float* da, float* dbt, const void* add, int ldadd,
                         void* dx, int lddx, int dxdtype, void* ws, size_t ws_bytes, const Stall (&stalls)[3],
                         void* stream) {
  int rc = check_lora(ad);
  if (rc != AQ_OK) return rc;
  if (M < 1 || M > kMaxTokens || !ids || !da || !dbt || !s) return AQ_ERR_ARG;
  if (((uintptr_t)ids | (uintptr_t)s | (uintptr_t)sx) & 3 || ((uintptr_t)da | (uintptr_t)dbt) & 15) return AQ_ERR_ARG;
  if (bad_rows(dy, ldd, ad->N, 8) || bad_rows(x, ldx, ad->K, sx ? 16 : 8)) return AQ_ERR_ARG;
  if (sx && ad->K % 16) return AQ_ERR_SHAPE;  // codes are read 16 at a time
  if (!dx && add) return AQ_ERR_ARG;
  if (dx) {
    if (dxdtype != AQ_F32 && dxdtype != AQ_BF16) return AQ_ERR_ARG;
    const int per16 = dxdtype == AQ_F32 ? 4 : 8;
    if (bad_rows(dx, lddx, ad->K, per16) || (add && bad_rows(add, ldadd, ad->K, per16)) || skewed(add, ldadd, dx, lddx, M))
      return AQ_ERR_ARG;
  }
  if (!ws || ws_bytes < aq_lora_workspace_bytes(ad, M, 1)) return AQ_ERR_WORKSPACE;
  if ((uintptr_t)ws & 15) return AQ_ERR_ARG;
  const int elt = dxdtype == AQ_F32 ? 4 : 2;
  const Span outs[] = {flat(da, (size_t)ad->R * ad->K * 4), flat(dbt, (size_t)ad->R * ad->N * 4),
                       rows_at(dx, lddx, ad->K, elt, M)};
  const Span ins[] = {rows_at(add == dx ? nullptr : add, ldadd, ad->K, elt, M), rows_at(dy, ldd, ad->N, 2, M),
                      rows_at(x, ldx, ad->K, sx ? 1 : 2, M), flat(ids, (size_t)M * 4), flat(sx, (size_t)M * 4),
                      flat(s, (size_t)M * ad->max_rank * 4),
                      flat(ad->a, (size_t)ad->R * ad->K * 2), flat(ad->bt, (size_t)ad->R * ad->N * 2),
                      flat(ad->off, (size_t)(ad->L + 1) * 4), flat(ad->scale, (size_t)ad->L * 4)};
  if (outputs_overlap(outs, ins)) return AQ_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  float* p = reinterpret_cast<float*>(static_cast<char*>(ws) + kWsHeader);
  const Products t = products(ad, M, true);
  cudaError_t e = shrink_any(ad, true, dy, ldd, ids, M, p, ws, stalls[0], st);
  char* rest = reinterpret_cast<char*>(p) + p_bytes(ad, M, true);
  const bool beside = dx && lora_tc_fits(ad, M);
  const TermsArgs terms = lora_grad_terms(ad, ids, M, 0, p, t.splits, t.ld, sx, s, rest);
  if (e == cudaSuccess && dx)
    e = expand_any(ad, false, ids, M, p, add, ldadd, dx, lddx, dxdtype, nullptr, beside ? &terms : nullptr, ws, stalls[1],
                   st);
  if (e == cudaSuccess)
    e = launch_lora_grad(ad, ids, M, p, t.splits, t.ld, x, ldx, sx, da, s, dy, ldd, dbt, beside, ws, rest, stalls[2],
                         st);
  return e == cudaSuccess ? AQ_OK : AQ_ERR_CUDA;
}

extern "C" int aq_lora_backward(const aq_lora* ad, const uint16_t* dy, int ldd, const int32_t* ids, int M,
                                const float* s, const void* x, int ldx, const float* sx, float* da, float* dbt,
                                const void* add, int ldadd, void* dx, int lddx, int dxdtype, void* ws, size_t ws_bytes,
                                void* stream) {
  const Stall stalls[3];
  return lora_backward(ad, dy, ldd, ids, M, s, x, ldx, sx, da, dbt, add, ldadd, dx, lddx, dxdtype, ws, ws_bytes, stalls,
                       stream);
}

extern "C" int aq_debug_lora_backward_stalled(const aq_lora* ad, const uint16_t* dy, int ldd, const int32_t* ids, int M,
                                              const float* s, const void* x, int ldx, const float* sx, float* da,
                                              float* dbt, void* dx, int lddx, int dxdtype, void* ws, size_t ws_bytes,
                                              int kernel, unsigned long long wait_ns, int stop_after, void* stream) {
  if (check_lora(ad) != AQ_OK || !dx || kernel < 0 || kernel > 2 || (kernel < 2 && !lora_tc_fits(ad, M)) ||
      !stall_ok(wait_ns, stop_after))
    return AQ_ERR_ARG;
  Stall stalls[3];
  stalls[kernel] = Stall{wait_ns, stop_after};
  return lora_backward(ad, dy, ldd, ids, M, s, x, ldx, sx, da, dbt, nullptr, 0, dx, lddx, dxdtype, ws, ws_bytes, stalls,
                       stream);
}
