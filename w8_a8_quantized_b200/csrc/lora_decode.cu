// Adapters of a decode batch (at most 64 tokens) in one launch:
//   S[i] = c_l sum_k x[k] A_l[i][k];   out[n] = y[n] + sum_i S[i] B_l^T[i][n]
//
// A few tokens read each adapter's rows once for next to no arithmetic, so the
// work is a stream of table rows whose time is the latency of two dependent
// passes.  Both run here in one cluster of eight CTAs per (adapter, up to two of
// its tokens): each CTA takes an eighth of the columns k of A_l, the partial sums
// are exchanged through distributed shared memory, and each CTA takes an eighth
// of the columns n of B_l^T.  The cluster of token m serves it and the next
// token of the same adapter if an even number of them comes before it, and returns
// otherwise.  Sums are fp32, in a fixed order.
//
// B's columns are cut into as many clusters as the GPU has room for in one wave (each
// forms S anew, from L2): what a CTA does one row after another is what takes its time
// (rank 64, N 9728, K 2560, one token: 12 us with one cluster, 7.8 with five, 6.3 with two rows of a half warp at once).  For the
// same reason a cluster takes two tokens of an adapter and not four, whose sums would
// leave registers for half the rows on their way.
#include <algorithm>

#include "aq_internal.cuh"
#include "lora.cuh"

namespace aq {
namespace {

constexpr int kCl = 8;         // CTAs of a cluster
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kT = 2;          // tokens of a cluster
constexpr int kVec = 8;        // columns of a 16-byte load
constexpr int kWide = 32 * kVec;  // columns of a warp's load
constexpr int kMaxSlice = 5120;   // columns of A in a CTA
constexpr int kRedBytes = kWarps * kT * kWide * 4;  // sums of the row groups

struct DecodeArgs {
  const uint16_t* a;
  const uint16_t* bt;
  const int32_t* off;
  const float* scale;
  int N, K, L, R, max_rank;
  const uint16_t* x;
  int ldx, M;
  const int32_t* ids;
  const void* y;
  void* out;
  int ldy, ldo;
  float* s;
  int kslice, nslice;  // columns of a CTA, multiples of 8
};

__device__ __forceinline__ uint32_t peer_smem(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void store_peer(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

__device__ __forceinline__ void widen8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

// out[0..7] = y[0..7] + v
template <bool F32>
__device__ __forceinline__ void put8(const DecodeArgs& a, int m, int n, const float (&v)[8]) {
  if constexpr (F32) {
    float4 p = make_float4(v[0], v[1], v[2], v[3]), q = make_float4(v[4], v[5], v[6], v[7]);
    if (a.y) {
      const float4* y = reinterpret_cast<const float4*>(static_cast<const float*>(a.y) + (size_t)m * a.ldy + n);
      const float4 y0 = y[0], y1 = y[1];
      p.x += y0.x; p.y += y0.y; p.z += y0.z; p.w += y0.w;
      q.x += y1.x; q.y += y1.y; q.z += y1.z; q.w += y1.w;
    }
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(a.out) + (size_t)m * a.ldo + n);
    o[0] = p;
    o[1] = q;
  } else {
    float y[8] = {};
    if (a.y)
      widen8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.y) + (size_t)m * a.ldy + n), y);
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 p = __floats2bfloat162_rn(y[2 * i] + v[2 * i], y[2 * i + 1] + v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&p);
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + (size_t)m * a.ldo + n) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// This CTA's columns k0 .. k0 + kn of S for TT tokens: 16 lanes per table row, RP rows
// per half warp with U loads each on their way; sent to every CTA of the cluster.
template <int TT, int RP, int U>
__device__ __forceinline__ void contract(const DecodeArgs& a, const uint16_t* xs, uint32_t part_addr, int c, int row0,
                                         int rank, int k0, int kn, float scale, int T) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane & 15;
  for (int r0 = 2 * warp; r0 < rank; r0 += 2 * kWarps * RP) {
    const int r = r0 + (lane >> 4);
    const uint16_t* row = a.a + (size_t)(row0 + r) * a.K + k0;
    float acc[RP][TT];
#pragma unroll
    for (int j = 0; j < RP; ++j)
#pragma unroll
      for (int t = 0; t < TT; ++t) acc[j][t] = 0.f;
    for (int kb = sub * kVec; kb < kn; kb += U * 16 * kVec) {
      uint4 w[RP][U];
#pragma unroll
      for (int j = 0; j < RP; ++j)
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int k = kb + i * 16 * kVec;
          w[j][i] = k < kn && r + 2 * kWarps * j < rank
                        ? __ldg(reinterpret_cast<const uint4*>(row + (size_t)(2 * kWarps * j) * a.K + k))
                        : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int k = kb + i * 16 * kVec;
        if (k < kn) {
#pragma unroll
          for (int t = 0; t < TT; ++t) {
            if (t < T) {
              float xf[8];
              widen8(*reinterpret_cast<const uint4*>(xs + t * a.kslice + k), xf);
#pragma unroll
              for (int j = 0; j < RP; ++j) {
                float wf[8];
                widen8(w[j][i], wf);
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[j][t] = fmaf(wf[e], xf[e], acc[j][t]);
              }
            }
          }
        }
      }
    }
#pragma unroll
    for (int j = 0; j < RP; ++j)
#pragma unroll
      for (int t = 0; t < TT; ++t) {
        const int rj = r + 2 * kWarps * j;
        if (r0 + 2 * kWarps * j >= rank) continue;
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) acc[j][t] += __shfl_xor_sync(0xffffffffu, acc[j][t], o);
        if (t < T && rj < rank && sub < kCl)
          store_peer(peer_smem(part_addr + (uint32_t)(((c * a.max_rank + rj) * kT + t) * 4), sub), scale * acc[j][t]);
      }
  }
}

// Columns n0 .. n1 of the result for TT tokens: warps share them out by 256 columns,
// then by rows (rgs row groups), ROWS table rows on their way, the first of them
// during the exchange of the sums.
template <bool F32, int TT, int ROWS>
__device__ __forceinline__ void spread(const DecodeArgs& a, const float* part, float* sums, float* red, int row0, int rank,
                                       int n0, int n1, const int (&tok)[kT], int T, bool keep) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ncg = max(1, (n1 - n0 + kWide - 1) / kWide);
  const int rgs = ncg >= kWarps ? 1 : kWarps / ncg;
  const int rg = ncg >= kWarps ? 0 : warp / ncg;
  const bool works = rg < rgs;
  int cg = ncg >= kWarps ? warp : warp % ncg;
  uint4 w[ROWS];
  auto load = [&](int r0, int n) {
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int r = r0 + i * rgs;
      w[i] = r < rank && n < n1 ? __ldg(reinterpret_cast<const uint4*>(a.bt + (size_t)(row0 + r) * a.N + n))
                                : make_uint4(0, 0, 0, 0);
    }
  };
  if (works) load(rg, n0 + cg * kWide + lane * kVec);
  cluster_arrive();
  cluster_wait();
  for (int i = tid; i < rank * kT; i += kThreads) {
    float s = 0.f;
    if (i % kT < T)
#pragma unroll
      for (int k = 0; k < kCl; ++k) s += part[k * a.max_rank * kT + i];
    sums[i] = s;
  }
  __syncthreads();
  if (keep)
#pragma unroll
    for (int t = 0; t < TT; ++t)
      if (t < T)
        for (int i = tid; i < a.max_rank; i += kThreads)
          a.s[(size_t)tok[t] * a.max_rank + i] = i < rank ? sums[i * kT + t] : 0.f;
  bool head = true;
  for (; cg < ncg && works; cg += kWarps) {
    const int n = n0 + cg * kWide + lane * kVec;
    float acc[TT][8];
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[t][e] = 0.f;
    for (int r0 = rg; r0 < rank; r0 += ROWS * rgs) {
      if (!head) load(r0, n);
      head = false;
#pragma unroll
      for (int i = 0; i < ROWS; ++i) {
        const int r = r0 + i * rgs;
        if (r < rank) {
          float wf[8];
          widen8(w[i], wf);
#pragma unroll
          for (int t = 0; t < TT; ++t) {
            const float s = sums[r * kT + t];
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[t][e] = fmaf(s, wf[e], acc[t][e]);
          }
        }
      }
    }
    if (rgs == 1) {
      if (n < n1)
#pragma unroll
        for (int t = 0; t < TT; ++t)
          if (t < T) put8<F32>(a, tok[t], n, acc[t]);
    } else {
#pragma unroll
      for (int t = 0; t < TT; ++t)
        if (t < T) {
          float4* d = reinterpret_cast<float4*>(red + ((rg * kT + t) * ncg + cg) * kWide + lane * kVec);
          d[0] = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
          d[1] = make_float4(acc[t][4], acc[t][5], acc[t][6], acc[t][7]);
        }
    }
  }
  if (rgs > 1) {
    __syncthreads();
    const int vecs = ncg * 32;
    for (int i = tid; i < T * vecs; i += kThreads) {
      const int t = i / vecs, n = n0 + (i - t * vecs) * kVec;
      if (n >= n1) continue;
      float s[8] = {};
      for (int g = 0; g < rgs; ++g) {
        const float4* d = reinterpret_cast<const float4*>(red + (g * kT + t) * ncg * kWide + (n - n0));
        const float4 p = d[0], q = d[1];
        s[0] += p.x; s[1] += p.y; s[2] += p.z; s[3] += p.w;
        s[4] += q.x; s[5] += q.y; s[6] += q.z; s[7] += q.w;
      }
      put8<F32>(a, t == 0 ? tok[0] : tok[1], n, s);
    }
  }
}

template <bool F32>
__global__ void __cluster_dims__(kCl, 1, 1) __launch_bounds__(kThreads, 3) lora_decode_kernel(const DecodeArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  uint16_t* xs = reinterpret_cast<uint16_t*>(raw + kRedBytes);          // [kT][kslice]
  float* part = reinterpret_cast<float*>(xs + kT * a.kslice);           // [kCl][max_rank][kT]
  float* sums = part + kCl * a.max_rank * kT;                           // [max_rank][kT]
  float* red = reinterpret_cast<float*>(raw);                           // [rgs][kT][ncg * kWide]
  __shared__ unsigned votes[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c = blockIdx.x, m = blockIdx.y;
  pdl_launch_dependents();
  pdl_wait();
  const int v = __ldg(a.ids + m);
  if (tid < 64) {
    const unsigned b = __ballot_sync(0xffffffffu, tid < a.M && __ldg(a.ids + min(tid, a.M - 1)) == v);
    if (lane == 0) votes[warp] = b;
  }
  int row0 = 0, rank = 0;
  if (v >= 0 && v < a.L) {
    row0 = min(max(__ldg(a.off + v), 0), a.R);
    rank = min(min(max(__ldg(a.off + v + 1), row0), a.R) - row0, a.max_rank);
  }
  const int n0 = min((blockIdx.z * kCl + c) * a.nslice, a.N), n1 = min(n0 + a.nslice, a.N);
  const bool keep = a.s && c == 0 && blockIdx.z == 0;
  if (rank == 0) {  // no adapter: y itself
    if (keep)
      for (int i = tid; i < a.max_rank; i += kThreads) a.s[(size_t)m * a.max_rank + i] = 0.f;
    if (a.out != a.y) {
      const float zero[8] = {};
      for (int n = n0 + tid * kVec; n < n1; n += kThreads * kVec) put8<F32>(a, m, n, zero);
    }
    return;
  }
  __syncthreads();
  unsigned long long mask = votes[0] | ((unsigned long long)votes[1] << 32);
  if (__popcll(mask & ((1ull << m) - 1)) % kT != 0) return;  // another token's cluster serves it
  mask &= ~((1ull << m) - 1);
  int tok[kT], T = 0;
#pragma unroll
  for (int t = 0; t < kT; ++t) {
    tok[t] = mask ? __ffsll((long long)mask) - 1 : m;
    if (mask) ++T;
    mask &= mask - 1;
  }
  const int k0 = c * a.kslice, kn = max(0, min(a.kslice, a.K - k0));
  cluster_arrive();  // the others' shared memory may be written once all have come this far
#pragma unroll
  for (int t = 0; t < kT; ++t)
    if (t < T)
      for (int k = tid * kVec; k < kn; k += kThreads * kVec)
        *reinterpret_cast<uint4*>(xs + t * a.kslice + k) =
            __ldg(reinterpret_cast<const uint4*>(a.x + (size_t)tok[t] * a.ldx + k0 + k));
  const float scale = __ldg(a.scale + v);
  cluster_wait();
  __syncthreads();
  // as many rows on their way as a row's columns leave room for (64 tokens of 40 adapters, K
  // 2560: 17.9 us with two rows of four loads, 20.4 with one of eight)
  if (T == 1) {
    if (a.kslice <= 512) contract<1, 2, 4>(a, xs, smem_u32(part), c, row0, rank, k0, kn, scale, T);
    else contract<1, 1, 8>(a, xs, smem_u32(part), c, row0, rank, k0, kn, scale, T);
    spread<F32, 1, 8>(a, part, sums, red, row0, rank, n0, n1, tok, T, keep);
  } else {
    if (a.kslice <= 512) contract<kT, 2, 4>(a, xs, smem_u32(part), c, row0, rank, k0, kn, scale, T);
    else contract<kT, 1, 8>(a, xs, smem_u32(part), c, row0, rank, k0, kn, scale, T);
    spread<F32, kT, 8>(a, part, sums, red, row0, rank, n0, n1, tok, T, keep);
  }
}

// Columns of a CTA where `parts` of them share d.
int slice(int d, int parts) { return ((d + parts - 1) / parts + 7) / 8 * 8; }
// Clusters that share the columns of B^T: as many as give one wave of three CTAs per
// SM, with 256 to 2048 columns of a CTA.
int column_clusters(int M, int N) {
  const int least = (N + kCl * kWarps * kWide - 1) / (kCl * kWarps * kWide), most = (N + kCl * kWide - 1) / (kCl * kWide);
  return std::max(least, std::min(most, 3 * num_sms() / (kCl * M)));
}

template <bool F32>
cudaError_t launch(const DecodeArgs& a, size_t smem, cudaStream_t st) {
  cudaError_t e = ensure_smem_attr<lora_decode_kernel<F32>>((int)(kRedBytes + kT * kMaxSlice * 2 + (kCl + 1) * 256 * kT * 4));
  if (e != cudaSuccess) return e;
  return launch_pdl(lora_decode_kernel<F32>, dim3(kCl, a.M, column_clusters(a.M, a.N)), dim3(kThreads), smem, st, a);
}

size_t smem_bytes(int K, int max_rank) {
  return kRedBytes + (size_t)kT * slice(K, kCl) * 2 + (size_t)(kCl + 1) * max_rank * kT * 4;
}

}  // namespace

bool lora_decode_fits(const aq_lora* ad, int M) { return M <= 64 && slice(ad->K, kCl) <= kMaxSlice; }

cudaError_t launch_lora_decode(const aq_lora* ad, const uint16_t* x, int ldx, const int32_t* ids, int M, const void* y,
                               int ldy, void* out, int ldo, bool f32, float* s, cudaStream_t st) {
  const DecodeArgs a{ad->a, ad->bt, ad->off, ad->scale, ad->N, ad->K, ad->L, ad->R, ad->max_rank, x, ldx, M,
                     ids, y, out, ldy, ldo, s, slice(ad->K, kCl), slice(ad->N, kCl * column_clusters(M, ad->N))};
  const size_t smem = smem_bytes(ad->K, ad->max_rank);
  return f32 ? launch<true>(a, smem, st) : launch<false>(a, smem, st);
}

}  // namespace aq
