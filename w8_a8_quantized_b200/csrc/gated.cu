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
// Both are bound by HBM on paper (4 bytes read and 1, with checkpoints 3, written
// per element forward; 4 and 4 backward).  Backward gets there: 4096 x 14336 in 79 us in a graph, 91%
// of the copy rate by the call's bytes.  Forward is bound by its instructions, 33 an element with three codes (46
// when the checkpoints' codes were tested and redone): 83 us in a graph, 76%.
// Hence float2 arithmetic, two multifunction operations per sigmoid, no clamps (a
// quotient cannot pass 127 by more than its rounding), and one comparison per
// eight codes; what that cannot decide is redone one element at a time.
//
// The codes are those of h, s and the quotient in fp64.  fp32 decides all but:
//  - the row's largest |h|: every element within 2e-6 of the fp32 maximum is redone;
//  - a code whose fp32 quotient lies within its error bound of a half-integer.
// Error bounds in units of 2^-24, relative.  exp(-g) = 2^(-g L1) (1 - c g), L1 the
// leading 16 bits of log2 e (with a bf16 g an exact product) and c = (log2 e - L1)
// ln 2: ex2.approx 4, the dropped (c g)^2 / 2 below 2 for |g| <= 88, two roundings.
// Then 1 + e: 1, rcp.approx 2, two products 2: h within 13.  The row's maximum
// likewise, its product with R 2, the reciprocal 2: a quotient within 30, 1.8e-6.
// The checkpoints' codes need no test: see biased_inverse.
#include <algorithm>

#include "aq_internal.cuh"

namespace aq {
namespace {

constexpr int kGroup = 128;  // features per scale of a checkpoint: 16 threads x 8
constexpr float kHMaxFast = 1e37f;  // rows with a larger |h| take fp64 throughout
constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: added, leaves the nearest integer in the low mantissa bits
constexpr float kNearH = 1.85e-6f;  // relative error of a quotient of h

__device__ __forceinline__ double gated64(float g, float u) {
  const double gd = g;
  return gd * (1.0 / (1.0 + exp(-gd))) * static_cast<double>(u);
}

__device__ __forceinline__ float ex2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

constexpr float kL1 = 1.44268798828125f;       // log2 e to 16 bits
constexpr float kLc = 4.888495152129525e-06f;  // (log2 e - kL1) ln 2

// exp(-g) of two bf16 values.
__device__ __forceinline__ float2 exp_neg2(float2 g) {
  const float2 y = __fmul2_rn(g, make_float2(-kL1, -kL1));
  const float2 c = __ffma2_rn(g, make_float2(-kLc, -kLc), make_float2(1.f, 1.f));
  return __fmul2_rn(make_float2(ex2_approx(y.x), ex2_approx(y.y)), c);
}

__device__ __forceinline__ float2 widen2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ uint32_t word(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
// Element e of eight bf16 values, e not known to the compiler.
__device__ __forceinline__ float pick(const uint4& v, int e) {
  const uint32_t w = word(v, e >> 1);
  return __uint_as_float((e & 1) ? (w & 0xFFFF0000u) : (w << 16));
}

__device__ __forceinline__ double scale64(double amax) { return fmax(amax * (1.0 / 127.0), 1e-12); }

__device__ __forceinline__ int code64(double x, double s) {
  return static_cast<int>(fmin(fmax(rint(x / s), -127.0), 127.0));
}

// max(a, b, c) in one instruction.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ uint2 pack_codes(const uint32_t (&c)[8]) {
  return make_uint2(__byte_perm(__byte_perm(c[0], c[1], 0x0040), __byte_perm(c[2], c[3], 0x0040), 0x5410),
                    __byte_perm(__byte_perm(c[4], c[5], 0x0040), __byte_perm(c[6], c[7], 0x0040), 0x5410));
}

// Codes of eight values; bit e of the result: element e is too near a half-integer.
// `limit`: 0.5 less the quotients' error bound.
__device__ __forceinline__ uint32_t codes8(const float2 (&x)[4], float r32, float limit, uint2& out) {
  const float2 r2 = make_float2(r32, r32), round2 = make_float2(kRound, kRound), back2 = make_float2(-kRound, -kRound);
  uint32_t c[8];
  float2 d[4];
  float far = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 r = __ffma2_rn(x[i], r2, round2);
    const float2 k = __fadd2_rn(r, back2);
    d[i] = __ffma2_rn(x[i], r2, make_float2(-k.x, -k.y));
    far = max3(far, fabsf(d[i].x), fabsf(d[i].y));
    c[2 * i] = __float_as_uint(r.x);
    c[2 * i + 1] = __float_as_uint(r.y);
  }
  out = pack_codes(c);
  uint32_t slow = 0;
  if (!(far <= limit)) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      slow |= (fabsf(d[i].x) <= limit ? 0u : 1u << (2 * i)) | (fabsf(d[i].y) <= limit ? 0u : 2u << (2 * i));
  }
  return slow;
}

// Scale of a checkpoint group: fp32 of max(amax R, 1e-12) in fp64.  R1 has 16
// bits, so with a bf16 amax both products are exact and the sum is rounded once
// (checked against the fp64 form for every bf16 amax).
__device__ __forceinline__ float scale32(float amax) {
  constexpr float kR1 = 0x1.0204p-7f, kR2 = 0x1.020408p-28f;
  return fmaxf(fmaf(amax, kR2, amax * kR1), 1e-12f);
}

// v >> n, 0 for any n above 31.
__device__ __forceinline__ uint32_t shr_clamped(uint32_t v, uint32_t n) {
  uint32_t r;
  asm("shr.u32 %0, %1, %2;" : "=r"(r) : "r"(v), "r"(n));
  return r;
}

// Reciprocal of a checkpoint's scale `s` (fp32) that decides every code without a test.
// With 8-bit mantissas the quotient x / s, about 127 x / amax, is either a half-integer
// b up to the roundings of s and of the quotient, or 2^-16 b away from it.  127 is prime, so
// the half-integers are b = 63.5, x = amax / 2, and all of them where amax has the mantissa
// 254 / 128.  There s is a power of two and the quotients are exact: ties go to even by
// themselves.  For the other mantissas the fp64 quotient at amax / 2 is below 63.5 for six
// and not for the rest, so 1 / s is made 2^-19 smaller or larger: more than its own
// error, 2^-22, and less than what would move any other quotient over a half-integer.  (Where
// s is at its floor, 1e-12, none comes nearer than 8e-6 b.)
__device__ __forceinline__ float biased_inverse(float s, float amax) {
  constexpr uint32_t kBelow0 = 1u << 9 | 1u << 10 | 1u << 24 | 1u << 25;  // mantissas 128 + 9, 10, 24, 25
  constexpr uint32_t kBelow1 = 1u << (41 - 32) | 1u << (56 - 32);        // 128 + 41, 56
  const uint32_t i = __float_as_uint(amax) >> 16 & 127;
  const uint32_t below = (shr_clamped(kBelow0, i) | shr_clamped(kBelow1, i - 32u)) & 1u;
  const float r = rcp_approx(s) * (below ? 1.f - 0x1p-19f : 1.f + 0x1p-19f);
  return (__float_as_uint(s) & 0x7FFFFFu) == 0 ? __uint_as_float(0x7F000000u - __float_as_uint(s)) : r;  // 2^-e of 2^e
}

// Codes of eight values by a reciprocal that decides them.
__device__ __forceinline__ uint2 decided8(const float2 (&x)[4], float r) {
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = __ffma2_rn(x[i], make_float2(r, r), make_float2(kRound, kRound));
    c[2 * i] = __float_as_uint(t.x);
    c[2 * i + 1] = __float_as_uint(t.y);
  }
  return pack_codes(c);
}

// The largest |x| of eight bf16 values, one of each half.
__device__ __forceinline__ uint32_t max_abs2(const uint4& v) {
  const __nv_bfloat162* p = reinterpret_cast<const __nv_bfloat162*>(&v);
  const __nv_bfloat162 m = __hmax2(__hmax2(__habs2(p[0]), __habs2(p[1])), __hmax2(__habs2(p[2]), __habs2(p[3])));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// Checkpoints of g and u: codes and scales of one 128-feature group of each,
// held by 16 neighbouring lanes.
__device__ __forceinline__ void checkpoint8(uint32_t gmax, uint32_t umax, const float2 (&g)[4], const float2 (&u)[4],
                                            bool in, bool group_in, int8_t* gq, float* gs, int8_t* uq, float* us, size_t qi,
                                            size_t si) {
  uint32_t m = __vmaxu2(__byte_perm(gmax, umax, 0x5410), __byte_perm(gmax, umax, 0x7632));  // both maxima in one word
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
  // the first eight lanes see to g's scale, the others to u's
  const bool us_half = threadIdx.x & 8;
  const float amax = __uint_as_float(us_half ? m & 0xFFFF0000u : m << 16), scale = scale32(amax);
  const float r = biased_inverse(scale, amax);
  const float rg = __shfl_sync(0xffffffffu, r, 0, 16), ru = __shfl_sync(0xffffffffu, r, 8, 16);
  if (in) {
    *reinterpret_cast<uint2*>(gq + qi) = decided8(g, rg);
    *reinterpret_cast<uint2*>(uq + qi) = decided8(u, ru);
  }
  if ((threadIdx.x & 7) == 0 && group_in) *(us_half ? us + si : gs + si) = scale;
}

// One CTA per row; a thread holds CV vectors of 8 h values in registers.  The
// block is as wide as the row needs (whole warps).
template <int CV, int MAXT, int MINB, bool KEEP>
__global__ void __launch_bounds__(MAXT, MINB)
    silu_mul_quant_kernel(const uint16_t* __restrict__ gate, int ldg, const uint16_t* __restrict__ up, int ldu, int F,
                          int8_t* __restrict__ hq, float* __restrict__ sh, int8_t* __restrict__ gq,
                          float* __restrict__ gs, int8_t* __restrict__ uq, float* __restrict__ us) {
  __shared__ uint32_t red[MAXT / 32];  // the warps' largest |h|
  __shared__ unsigned long long top;  // bits of the row's largest fp64 |h| (non-negative doubles order as integers)
  const int m = blockIdx.x, threads = blockDim.x;
  const uint4* grow = reinterpret_cast<const uint4*>(gate + (size_t)m * ldg);
  const uint4* urow = reinterpret_cast<const uint4*>(up + (size_t)m * ldu);
  const int nvec = F / 8, groups = (F + kGroup - 1) / kGroup;
  if (threadIdx.x == 0) top = 0;
  pdl_launch_dependents();
  pdl_wait();

  // all loads first: the checkpoints' rounds below would keep later ones waiting
  uint4 gl[CV], ul[CV];
#pragma unroll
  for (int i = 0; i < CV; ++i) {
    const int v = min(threadIdx.x + i * threads, nvec - 1);  // behind the end: the last again, in its own group
    gl[i] = __ldg(grow + v);
    ul[i] = __ldg(urow + v);
  }
  float2 h[CV][4];
  float big[CV], amax = 0.f;  // the vectors' largest |h|, the row's
#pragma unroll
  for (int i = 0; i < CV; ++i) {
    const int v = threadIdx.x + i * threads;
    const bool in = v < nvec;
    const uint4 gv = gl[i], uv = ul[i];
    const float2 g[4] = {widen2(gv.x), widen2(gv.y), widen2(gv.z), widen2(gv.w)};
    const float2 u[4] = {widen2(uv.x), widen2(uv.y), widen2(uv.z), widen2(uv.w)};
    const uint32_t gmax = max_abs2(gv);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 x = __fadd2_rn(exp_neg2(g[e]), make_float2(1.f, 1.f));
      h[i][e] = __fmul2_rn(__fmul2_rn(g[e], make_float2(rcp_approx(x.x), rcp_approx(x.y))), u[e]);
    }
    if ((gmax & 0xFFFFu) > 0x42A0u || gmax > 0x42A0FFFFu) {  // |g| > 80: exp may leave fp32's range: the fp64 value, rounded
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (g[e].x < -80.f) h[i][e].x = static_cast<float>(gated64(g[e].x, u[e].x));
        if (g[e].y < -80.f) h[i][e].y = static_cast<float>(gated64(g[e].y, u[e].y));
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) big[i] = max3(e ? big[i] : 0.f, fabsf(h[i][e].x), fabsf(h[i][e].y));
    amax = fmaxf(amax, big[i]);
    if (KEEP)
      checkpoint8(gmax, max_abs2(uv), g, u, in, (v & ~15) < nvec, gq, gs, uq, us, (size_t)m * F + (size_t)v * 8, (size_t)m * groups + v / 16);
  }
  // (non-negative floats order as integers)
  const uint32_t of_warp = __reduce_max_sync(0xffffffffu, __float_as_uint(amax));
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[threadIdx.x >> 5] = of_warp;
  __syncthreads();
  amax = __uint_as_float(__reduce_max_sync(0xffffffffu, lane < threads / 32 ? red[lane] : 0u));
  const bool wide = !(amax < kHMaxFast);

  // the exact maximum: redo every element that may be it (none where the scale
  // is at its floor: 1e-11 / 127 < 1e-12)
  const float near = wide ? 0.f : amax * (1.f - 2e-6f);
  if (amax > 1e-11f || wide) {
    double best = 0.0;
#pragma unroll
    for (int i = 0; i < CV; ++i) {
      const int v = threadIdx.x + i * threads;
      if (v < nvec && !(big[i] < near)) {
        const uint4 gv = __ldg(grow + v), uv = __ldg(urow + v);
        for (int e = 0; e < 8; ++e) {
          const float2 p = e < 4 ? (e < 2 ? h[i][0] : h[i][1]) : (e < 6 ? h[i][2] : h[i][3]);
          if (!(fabsf(e & 1 ? p.y : p.x) < near)) best = fmax(best, fabs(gated64(pick(gv, e), pick(uv, e))));
        }
      }
    }
    if (best > 0.0) atomicMax(&top, static_cast<unsigned long long>(__double_as_longlong(best)));
  }

  // codes by the fp32 scale; undecided ones are noted
  const float r32 = rcp_approx(fmaxf(amax * (1.f / 127.f), 1e-12f));
  uint32_t undecided[(CV + 3) / 4];
#pragma unroll
  for (int i = 0; i < (CV + 3) / 4; ++i) undecided[i] = 0;
#pragma unroll
  for (int i = 0; i < CV; ++i) {
    const int v = threadIdx.x + i * threads;
    if (v < nvec) {
      uint2 c;
      const uint32_t slow = codes8(h[i], r32, fmaf(big[i] * r32, -kNearH, 0.5f - 1e-6f), c);
      undecided[i / 4] |= (wide ? 0xFFu : slow) << (8 * (i & 3));
      reinterpret_cast<uint2*>(hq + (size_t)m * F)[v] = c;
    }
  }
  __syncthreads();
  const double s = scale64(__longlong_as_double(static_cast<long long>(top)));
  if (threadIdx.x == 0) sh[m] = static_cast<float>(s);
#pragma unroll
  for (int j = 0; j < (CV + 3) / 4; ++j)
    for (uint32_t w = undecided[j]; w; w &= w - 1) {
      const int i = __ffs(w) - 1;
      const size_t f = (size_t)(threadIdx.x + (4 * j + (i >> 3)) * threads) * 8 + (i & 7);
      const float g = bf16_bits_to_float(__ldg(gate + (size_t)m * ldg + f)), u = bf16_bits_to_float(__ldg(up + (size_t)m * ldu + f));
      hq[(size_t)m * F + f] = static_cast<int8_t>(code64(gated64(g, u), s));
    }
}

__device__ __forceinline__ uint32_t pack2(float2 v) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(v.x, v.y);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// Two codes (bytes 2i, 2i + 1 of x, offset by 128) times their scale.
template <int I>
__device__ __forceinline__ float2 restore2(uint32_t x, float2 s) {
  constexpr uint32_t sel = 0x7440u | (I ? 0x2u : 0u);
  const float2 p = make_float2(__uint_as_float(__byte_perm(x, 0x4B000000u, sel)),
                               __uint_as_float(__byte_perm(x, 0x4B000000u, sel + 1)));
  return __fmul2_rn(__fadd2_rn(p, make_float2(-8388736.f, -8388736.f)), s);
}

// Gradients of two elements.  x = exp(-|g|), so that p and 1 - p keep their bits
// wherever g lies (formed 2^24 too large, since ex2.approx flushes subnormals);
// its relative error, |g| 2^-24 and a few units, is far below bf16's rounding.
__device__ __forceinline__ void back2(float2 g, float2 u, float2 d, float2& dg, float2& du) {
  constexpr float kL = 1.4426950408889634f;
  const float2 one = make_float2(1.f, 1.f);
  float2 x = make_float2(ex2_approx(fmaf(fabsf(g.x), -kL, 24.f)), ex2_approx(fmaf(fabsf(g.y), -kL, 24.f)));
  x = __fmul2_rn(x, make_float2(0x1p-24f, 0x1p-24f));
  const float2 y = __fadd2_rn(x, one);
  const float2 r = make_float2(rcp_approx(y.x), rcp_approx(y.y));
  const float2 xr = __fmul2_rn(x, r);
  const float2 p = make_float2(g.x < 0.f ? xr.x : r.x, g.y < 0.f ? xr.y : r.y);
  const float2 np = make_float2(g.x < 0.f ? r.x : xr.x, g.y < 0.f ? r.y : xr.y);
  dg = __fmul2_rn(d, __fmul2_rn(u, __fmul2_rn(p, __ffma2_rn(g, np, one))));
  du = __fmul2_rn(d, __fmul2_rn(g, p));
}

// A load of what the same thread may overwrite afterwards (dgate or dup in place of dh): not by way of the read-only
// cache.
__device__ __forceinline__ uint4 load16(const uint4* p) {
  uint4 v;
  asm("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

// One CTA per row, 16 features per thread and round.
__global__ void __launch_bounds__(256)
    silu_mul_backward_kernel(const uint16_t* __restrict__ dh, int ldd, const int8_t* __restrict__ gq,
                             const float* __restrict__ gs, const int8_t* __restrict__ uq, const float* __restrict__ us,
                             int F, uint16_t* __restrict__ dgate, int ldg, uint16_t* __restrict__ dup, int ldu) {
  const int m = blockIdx.x, nv = F / 16, groups = (F + kGroup - 1) / kGroup;
  const uint4* grow = reinterpret_cast<const uint4*>(gq + (size_t)m * F);
  const uint4* urow = reinterpret_cast<const uint4*>(uq + (size_t)m * F);
  const uint4* drow = reinterpret_cast<const uint4*>(dh + (size_t)m * ldd);
  uint4* go = reinterpret_cast<uint4*>(dgate + (size_t)m * ldg);
  uint4* uo = reinterpret_cast<uint4*>(dup + (size_t)m * ldu);
  pdl_launch_dependents();
  pdl_wait();
#pragma unroll 2
  for (int v = threadIdx.x; v < nv; v += blockDim.x) {
    const uint4 gv = __ldg(grow + v), uv = __ldg(urow + v), d0 = load16(drow + 2 * v), d1 = load16(drow + 2 * v + 1);
    const float sg = __ldg(gs + (size_t)m * groups + v / 8), su = __ldg(us + (size_t)m * groups + v / 8);
    const float2 sg2 = make_float2(sg, sg), su2 = make_float2(su, su);
    uint32_t og[8], ou[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t gw = word(gv, i) ^ 0x80808080u, uw = word(uv, i) ^ 0x80808080u;
      const uint32_t da = word(i < 2 ? d0 : d1, 2 * (i & 1)), db = word(i < 2 ? d0 : d1, 2 * (i & 1) + 1);
      float2 dg, du;
      back2(restore2<0>(gw, sg2), restore2<0>(uw, su2), widen2(da), dg, du);
      og[2 * i] = pack2(dg);
      ou[2 * i] = pack2(du);
      back2(restore2<1>(gw, sg2), restore2<1>(uw, su2), widen2(db), dg, du);
      og[2 * i + 1] = pack2(dg);
      ou[2 * i + 1] = pack2(du);
    }
    go[2 * v] = make_uint4(og[0], og[1], og[2], og[3]);
    go[2 * v + 1] = make_uint4(og[4], og[5], og[6], og[7]);
    uo[2 * v] = make_uint4(ou[0], ou[1], ou[2], ou[3]);
    uo[2 * v + 1] = make_uint4(ou[4], ou[5], ou[6], ou[7]);
  }
}

template <int CV, int MAXT, int MINB, bool KEEP>
cudaError_t launch_row(const uint16_t* gate, int ldg, const uint16_t* up, int ldu, int M, int F, int8_t* hq, float* sh,
                       int8_t* gq, float* gs, int8_t* uq, float* us, cudaStream_t st) {
  const int per = (F / 8 + CV - 1) / CV, threads = std::max(32, (per + 31) / 32 * 32);
  return launch_pdl(silu_mul_quant_kernel<CV, MAXT, MINB, KEEP>, dim3(M), dim3(threads), 0, st, gate, ldg, up, ldu, F,
                    hq, sh, gq, gs, uq, us);
}

template <bool KEEP>
cudaError_t launch_fwd(const uint16_t* gate, int ldg, const uint16_t* up, int ldu, int M, int F, int8_t* hq, float* sh,
                       int8_t* gq, float* gs, int8_t* uq, float* us, cudaStream_t st) {
  // Vectors a thread, threads of a CTA, CTAs per SM.  With few tokens as few vectors as the row allows, since a thread's
  // work is a chain; with many as many as leave registers for two CTAs per SM, as far as that goes (14336 features).
  // us in graphs, without and with checkpoints, here and with another variant:
  //      1 token    2048:   1.9   2.2  (two vectors    2.0   2.4)
  //                14336:   3.0   3.7  (four vectors   3.4   4.4)
  //                17408:   5.0   6.6  (1024 threads   6.7   8.9)
  //   4096 tokens   2048:  13.0  17.3  (two vectors    9.5  13.0: the one bound that many tokens would move)
  //                 4096:  18.3  27.7  (four vectors  21.6  30.7)
  //                 9728:    51    69  (two, 75 and 93; eight, 71 and 97)
  //                14336:    60    83  (two, 89 and 112; eight, 92 and 132)
  //                17408:   145   211  (1024 threads, 133 and 202): one CTA per SM either way, at 116 to 126 registers
  // Above 32768 features the last variant spills 388 bytes (1 token of 65536: 12.9 and 16.9).
  const int nvec = F / 8;
#define AQ_GATED(CV, T, B) return launch_row<CV, T, B, KEEP>(gate, ldg, up, ldu, M, F, hq, sh, gq, gs, uq, us, st)
  if (nvec <= 256) AQ_GATED(1, 256, 4);
  if (M <= num_sms() && nvec <= 2048) AQ_GATED(2, 1024, 1);  // a row per SM: the shortest chain per thread
  if (nvec <= 512) AQ_GATED(2, 256, 4);
  if (nvec <= 1792) AQ_GATED(4, 448, 2);
  if (nvec <= 4096) AQ_GATED(8, 512, 1);
  AQ_GATED(8, 1024, 1);
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
  const size_t codes = (size_t)M * F, scales = (size_t)M * ((F + kGroup - 1) / kGroup) * 4;
  const Span outs[] = {flat(hq, codes), flat(sh, (size_t)M * 4), flat(gq, codes), flat(gs, scales), flat(uq, codes),
                       flat(us, scales)};
  const Span ins[] = {{gate, (size_t)ldg * 2, (size_t)F * 2, M}, {up, (size_t)ldu * 2, (size_t)F * 2, M}};
  if (outputs_overlap(outs, ins)) return AQ_ERR_ARG;
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
  const size_t codes = (size_t)M * F, scales = (size_t)M * ((F + kGroup - 1) / kGroup) * 4, width = (size_t)F * 2;
  const Span outs[] = {{dgate, (size_t)ldg * 2, width, M}, {dup, (size_t)ldu * 2, width, M}};
  // in place of dh: a thread stores what it has made of its own loads, so rows of one pitch are as good as apart
  const bool in_place = (dgate == dh && (ldg == ldd || M == 1)) || (dup == dh && (ldu == ldd || M == 1));
  const Span ins[] = {{in_place ? nullptr : dh, (size_t)ldd * 2, width, M}, flat(gq, codes), flat(gs, scales), flat(uq, codes), flat(us, scales)};
  if (outputs_overlap(outs, ins)) return AQ_ERR_ARG;
  // whole warps, ceil(F / 4096) rounds a thread
  const int nv = F / 16, rounds = (nv + 255) / 256, threads = ((nv + rounds - 1) / rounds + 31) / 32 * 32;
  return launch_pdl(silu_mul_backward_kernel, dim3(M), dim3(threads), 0, static_cast<cudaStream_t>(stream), dh, ldd, gq,
                    gs, uq, us, F, dgate, ldg, dup, ldu) == cudaSuccess
             ? AQ_OK
             : AQ_ERR_CUDA;
}
