// Gated activation between the gate/up and the down projection, with the codes
// and the 8-bit checkpoints it leaves behind, and its backward pass.
//
// Forward, per token (row) of F features:
//   h = silu(g) u = g / (1 + exp(-g)) * u
//   s = max(max|h| R, 1e-12), R = fl64(1 / 127);  hq = clamp(rint(h / s), -127, 127)
// and, when asked for, checkpoints of g and u by the same rule with one scale
// per 128 features of a row.  (aq_quant_act's rule but for the scale's last fp64
// bit: a product with R in place of the quotient.)  Backward, from the checkpoints g~ = gs gq, u~ = us uq:
//   p = 1 / (1 + exp(-g~));  dg = dh u~ p (1 + g~ (1 - p));  du = dh g~ p.
//
// Both are bound by HBM: 4 bytes read and 1 (3 with checkpoints) written per
// element forward, 4 read and 4 written backward.
//
// The codes are those of h, s and the quotient in fp64.  h is formed in fp32
// first; everything that fp32 cannot decide is redone in fp64:
//  - the row's largest |h|: every element within 2e-6 of the fp32 maximum;
//  - a code whose fp32 quotient lies within its error bound of a half-integer.
// fp32 error bound: expf 2 ulp, and one rounding each of 1 + e, the reciprocal,
// two products, fp32(s), its reciprocal and the last product: 11 * 2^-24 <
// 6.6e-7 relative; 1e-6 is used.
#include "aq_internal.cuh"

namespace aq {
namespace {

constexpr int kGroup = 128;  // features per scale of a checkpoint: 16 threads x 8
constexpr float kHMaxFast = 1e37f;  // rows with a larger |h| take fp64 throughout

__device__ __forceinline__ double gated64(float g, float u) {
  const double gd = g;
  return gd * (1.0 / (1.0 + exp(-gd))) * static_cast<double>(u);
}

// fp32 h within 6.6e-7 relative of gated64 (below -80 exp overflows towards
// fp32's limit: there the fp64 value, rounded).
__device__ __forceinline__ float gated32(float g, float u) {
  if (g < -80.f) return static_cast<float>(gated64(g, u));
  return g * __frcp_rn(1.f + expf(-g)) * u;
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = bf16_bits_to_float((i & 1) ? (w[i >> 1] >> 16) : (w[i >> 1] & 0xFFFFu));
}

__device__ __forceinline__ double scale64(double amax) { return fmax(amax * (1.0 / 127.0), 1e-12); }

// Codes and scale of one 128-feature group held by 16 neighbouring lanes.
__device__ __forceinline__ void checkpoint8(const uint4& v, bool in, int8_t* q, float* s, size_t qi, size_t si) {
  float amax = in ? abs_max8(v, 0.f) : 0.f;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  const double sd = scale64(amax);
  if (in) {
    *reinterpret_cast<uint2*>(q + qi) = quantize8(v, sd, act_recip(sd));
    if ((threadIdx.x & 15) == 0) s[si] = static_cast<float>(sd);
  }
}

// One CTA per row; a thread holds CV vectors of 8 h values in registers.
template <int CV, int THREADS, bool KEEP>
__global__ void __launch_bounds__(THREADS)
    silu_mul_quant_kernel(const uint16_t* __restrict__ gate, int ldg, const uint16_t* __restrict__ up, int ldu, int F,
                          int8_t* __restrict__ hq, float* __restrict__ sh, int8_t* __restrict__ gq,
                          float* __restrict__ gs, int8_t* __restrict__ uq, float* __restrict__ us) {
  __shared__ float red[THREADS / 32];
  __shared__ unsigned long long top;  // bits of the row's largest fp64 |h| (non-negative doubles order as integers)
  const int m = blockIdx.x;
  const uint4* grow = reinterpret_cast<const uint4*>(gate + (size_t)m * ldg);
  const uint4* urow = reinterpret_cast<const uint4*>(up + (size_t)m * ldu);
  const int nvec = F / 8, groups = (F + kGroup - 1) / kGroup;
  if (threadIdx.x == 0) top = 0;
  pdl_launch_dependents();
  pdl_wait();

  float h[CV][8];
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < CV; ++i) {
    const int v = threadIdx.x + i * THREADS;
    const bool in = v < nvec;
    const uint4 gv = in ? __ldg(grow + v) : make_uint4(0, 0, 0, 0);
    const uint4 uv = in ? __ldg(urow + v) : make_uint4(0, 0, 0, 0);
    float g[8], u[8];
    unpack8(gv, g);
    unpack8(uv, u);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[i][e] = gated32(g[e], u[e]);
      amax = fmaxf(amax, fabsf(h[i][e]));
    }
    if (KEEP) {
      checkpoint8(gv, in, gq, gs, (size_t)m * F + (size_t)v * 8, (size_t)m * groups + v / 16);
      checkpoint8(uv, in, uq, us, (size_t)m * F + (size_t)v * 8, (size_t)m * groups + v / 16);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = amax;
  __syncthreads();
  amax = red[0];
#pragma unroll
  for (int w = 1; w < THREADS / 32; ++w) amax = fmaxf(amax, red[w]);
  const bool wide = !(amax < kHMaxFast);

  // the exact maximum: redo every element that may be it (none where the scale
  // is at its floor: 1e-11 / 127 < 1e-12)
  const float near = wide ? 0.f : amax * (1.f - 2e-6f);
  const bool floored = amax <= 1e-11f;
  double best = 0.0;
#pragma unroll
  for (int i = 0; i < CV; ++i) {
    const int v = threadIdx.x + i * THREADS;
    bool any = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) any = any || !(fabsf(h[i][e]) < near);
    if (v < nvec && any && !floored) {
      float g[8], u[8];
      unpack8(__ldg(grow + v), g);
      unpack8(__ldg(urow + v), u);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (!(fabsf(h[i][e]) < near)) best = fmax(best, fabs(gated64(g[e], u[e])));
    }
  }
  if (best > 0.0) atomicMax(&top, static_cast<unsigned long long>(__double_as_longlong(best)));
  __syncthreads();
  const double amax64 = __longlong_as_double(static_cast<long long>(top));
  const double s = scale64(amax64);
  const float r32 = act_recip(s);
  if (threadIdx.x == 0) sh[m] = static_cast<float>(s);

  constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: see quantize8
#pragma unroll
  for (int i = 0; i < CV; ++i) {
    const int v = threadIdx.x + i * THREADS;
    if (v >= nvec) continue;
    uint32_t c[8];
    uint32_t slow = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float t = h[i][e] * r32;
      const float r = __fadd_rn(fminf(fmaxf(t, -127.f), 127.f), kRound);
      const float k = __fsub_rn(r, kRound);
      slow |= (0.5f - fabsf(t - k) > 1.0e-6f * fabsf(t) ? 0u : 1u) << e;
      c[e] = __float_as_uint(r);
    }
    if (wide) slow = 0xFFu;
    if (slow) {
      float g[8], u[8];
      unpack8(__ldg(grow + v), g);
      unpack8(__ldg(urow + v), u);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if ((slow >> e) & 1u)
          c[e] = static_cast<uint32_t>(static_cast<int>(fmin(fmax(rint(gated64(g[e], u[e]) / s), -127.0), 127.0)));
    }
    const uint32_t l0 = __byte_perm(c[0], c[1], 0x0040), h0 = __byte_perm(c[2], c[3], 0x0040);
    const uint32_t l1 = __byte_perm(c[4], c[5], 0x0040), h1 = __byte_perm(c[6], c[7], 0x0040);
    reinterpret_cast<uint2*>(hq + (size_t)m * F)[v] =
        make_uint2(__byte_perm(l0, h0, 0x5410), __byte_perm(l1, h1, 0x5410));
  }
}

// 16 features per thread.
constexpr int kBwdThreads = 256;

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__global__ void __launch_bounds__(kBwdThreads)
    silu_mul_backward_kernel(const uint16_t* __restrict__ dh, int ldd, const int8_t* __restrict__ gq,
                             const float* __restrict__ gs, const int8_t* __restrict__ uq, const float* __restrict__ us,
                             int M, int F, uint16_t* __restrict__ dgate, int ldg, uint16_t* __restrict__ dup,
                             int ldu) {
  const int nv = F / 16, groups = (F + kGroup - 1) / kGroup;
  pdl_launch_dependents();
  pdl_wait();
  const long long total = (long long)M * nv;
  for (long long i = (long long)blockIdx.x * kBwdThreads + threadIdx.x; i < total;
       i += (long long)gridDim.x * kBwdThreads) {
    const int m = (int)(i / nv), v = (int)(i - (long long)m * nv);
    const uint4 gv = __ldg(reinterpret_cast<const uint4*>(gq + (size_t)m * F) + v);
    const uint4 uv = __ldg(reinterpret_cast<const uint4*>(uq + (size_t)m * F) + v);
    const uint4* drow = reinterpret_cast<const uint4*>(dh + (size_t)m * ldd) + 2 * v;
    const uint4 d0 = __ldg(drow), d1 = __ldg(drow + 1);
    const float sg = __ldg(gs + (size_t)m * groups + v / 8), su = __ldg(us + (size_t)m * groups + v / 8);
    float d[16];
    {
      float a[8], b[8];
      unpack8(d0, a);
      unpack8(d1, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d[e] = a[e];
        d[8 + e] = b[e];
      }
    }
    const uint32_t gw[4] = {gv.x, gv.y, gv.z, gv.w}, uw[4] = {uv.x, uv.y, uv.z, uv.w};
    uint32_t og[8], ou[8];
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      float rg[2], ru[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int b = e + k;
        const float g = sg * static_cast<float>(static_cast<int8_t>(gw[b >> 2] >> (8 * (b & 3))));
        const float u = su * static_cast<float>(static_cast<int8_t>(uw[b >> 2] >> (8 * (b & 3))));
        // from exp(-|g|) both p and 1 - p keep their bits wherever g lies
        const float x = expf(-fabsf(g)), r = __frcp_rn(1.f + x), xr = x * r;
        const float p = g < 0.f ? xr : r, np = g < 0.f ? r : xr;
        rg[k] = d[b] * (u * (p * fmaf(g, np, 1.f)));
        ru[k] = d[b] * (g * p);
      }
      og[e / 2] = pack_bf16(rg[0], rg[1]);
      ou[e / 2] = pack_bf16(ru[0], ru[1]);
    }
    uint4* go = reinterpret_cast<uint4*>(dgate + (size_t)m * ldg) + 2 * v;
    uint4* uo = reinterpret_cast<uint4*>(dup + (size_t)m * ldu) + 2 * v;
    go[0] = make_uint4(og[0], og[1], og[2], og[3]);
    go[1] = make_uint4(og[4], og[5], og[6], og[7]);
    uo[0] = make_uint4(ou[0], ou[1], ou[2], ou[3]);
    uo[1] = make_uint4(ou[4], ou[5], ou[6], ou[7]);
  }
}

template <bool KEEP>
cudaError_t launch_fwd(const uint16_t* gate, int ldg, const uint16_t* up, int ldu, int M, int F, int8_t* hq, float* sh,
                       int8_t* gq, float* gs, int8_t* uq, float* us, cudaStream_t st) {
  const int nvec = F / 8;
#define AQ_GATED(CV, T)                                                                                            \
  return launch_pdl(silu_mul_quant_kernel<CV, T, KEEP>, dim3(M), dim3(T), 0, st, gate, ldg, up, ldu, F, hq, sh, gq, \
                    gs, uq, us)
  if (nvec <= 256) AQ_GATED(1, 256);
  if (nvec <= 512) AQ_GATED(2, 256);
  if (nvec <= 1024) AQ_GATED(4, 256);
  if (nvec <= 2048) AQ_GATED(4, 512);
  if (nvec <= 4096) AQ_GATED(4, 1024);
  AQ_GATED(8, 1024);
#undef AQ_GATED
}

}  // namespace
}  // namespace aq

using namespace aq;

// a row of h is held in the registers of one CTA
static constexpr int kGatedMaxF = 65536;

extern "C" int aq_silu_mul_quant(const uint16_t* gate, int ldg, const uint16_t* up, int ldu, int M, int F, int8_t* hq,
                                 float* sh, int8_t* gq, float* gs, int8_t* uq, float* us, void* stream) {
  if (!gate || !up || !hq || !sh || M < 1 || F < 16 || F % 16 || F > kGatedMaxF) return AQ_ERR_ARG;
  if (ldg < F || ldu < F || ldg % 8 || ldu % 8) return AQ_ERR_ARG;
  const bool keep = gq || gs || uq || us;
  if (keep && (!gq || !gs || !uq || !us)) return AQ_ERR_ARG;
  if (((uintptr_t)gate | (uintptr_t)up | (uintptr_t)hq | (uintptr_t)gq | (uintptr_t)uq) & 15) return AQ_ERR_ARG;
  if (((uintptr_t)sh | (uintptr_t)gs | (uintptr_t)us) & 3) return AQ_ERR_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = keep ? launch_fwd<true>(gate, ldg, up, ldu, M, F, hq, sh, gq, gs, uq, us, st)
                             : launch_fwd<false>(gate, ldg, up, ldu, M, F, hq, sh, gq, gs, uq, us, st);
  return e == cudaSuccess ? AQ_OK : AQ_ERR_CUDA;
}

extern "C" int aq_silu_mul_backward(const uint16_t* dh, int ldd, const int8_t* gq, const float* gs, const int8_t* uq,
                                    const float* us, int M, int F, uint16_t* dgate, int ldg, uint16_t* dup, int ldu,
                                    void* stream) {
  if (!dh || !gq || !gs || !uq || !us || !dgate || !dup || M < 1 || F < 16 || F % 16 || F > kGatedMaxF)
    return AQ_ERR_ARG;
  if (ldd < F || ldg < F || ldu < F || ldd % 8 || ldg % 8 || ldu % 8) return AQ_ERR_ARG;
  if (((uintptr_t)dh | (uintptr_t)gq | (uintptr_t)uq | (uintptr_t)dgate | (uintptr_t)dup) & 15) return AQ_ERR_ARG;
  if (((uintptr_t)gs | (uintptr_t)us) & 3) return AQ_ERR_ARG;
  const long long blocks = ((long long)M * (F / 16) + kBwdThreads - 1) / kBwdThreads;
  const int grid = (int)(blocks < 65535ll * 16 ? blocks : 65535ll * 16);
  return launch_pdl(silu_mul_backward_kernel, dim3(grid), dim3(kBwdThreads), 0, static_cast<cudaStream_t>(stream), dh,
                    ldd, gq, gs, uq, us, M, F, dgate, ldg, dup, ldu) == cudaSuccess
             ? AQ_OK
             : AQ_ERR_CUDA;
}
