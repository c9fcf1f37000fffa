// Shared by the adapter kernels.
#pragma once

#include "aq_internal.cuh"

namespace aq {

// Decode batches (lora_decode.cu): whether the one-launch kernel takes the call, and the call.
bool lora_decode_fits(const aq_lora* ad, int M);
cudaError_t launch_lora_decode(const aq_lora* ad, const uint16_t* x, int ldx, const int32_t* ids, int M, const void* y,
                               int ldy, void* out, int ldo, bool f32, float* s, cudaStream_t st);

// The bf16 terms of S and T for the weight gradients (lora_grad.cu), of `rc` ranks from rb0 on.
struct TermsJob {
  const float* p;     // [splits][M][ld]
  int splits, ld;
  const float* sx;    // [M] or null
  uint16_t* terms;    // [M][npad]: hi, mid, lo of `rc` ranks each
};
struct TermsArgs {
  TermsJob job[2];
  const int32_t* ids;
  const int32_t* off;
  int M, L, R, max_rank;
  int rb0, rc, npad;
  int32_t* info;      // per 64 tokens: the adapter that has them all, -1 none has any, -2 mixed
};

// More than 64 tokens, ranks up to 64 (lora_tc.cu).  Shrink: p [splits][M][rp] (rp =
// max_rank rounded up to 16) from the a side or the b side of the tables; expand:
// out = y + p's sums times the other side.  `counts`: lora_tc_count_bytes, written by the
// one for the other.  `terms`, if any: to be written beside out.  `header`: the error word of the call's workspace.
bool lora_tc_fits(const aq_lora* ad, int M);
int lora_tc_splits(int M, int D);
size_t lora_tc_count_bytes(int M);
cudaError_t launch_lora_shrink_tc(const aq_lora* ad, bool b_side, const uint16_t* x, int ldx, const int32_t* ids, int M,
                                  float* p, int32_t* counts, void* header, const Stall& stall, cudaStream_t st);
cudaError_t launch_lora_expand_tc(const aq_lora* ad, bool b_side, const int32_t* ids, int M, const float* p, int splits,
                                  const int32_t* counts, const void* y, int ldy, void* out, int ldo, bool f32, float* s,
                                  const TermsArgs* terms, void* header, const Stall& stall, cudaStream_t st);

// Weight gradients (lora_grad.cu): t [tsplits][M][ldt] partial sums of the
// output's gradient times B, s [M][max_rank] the forward products.  `header`: the
// error word of a call's workspace; `ws`: lora_grad_ws_bytes, 256-byte aligned
// behind a workspace that starts on 16 bytes.
size_t lora_grad_ws_bytes(const aq_lora* ad, int M);
cudaError_t launch_lora_grad(const aq_lora* ad, const int32_t* ids, int M, const float* t, int tsplits, int ldt, const void* x,
                             int ldx, const float* sx, float* da, const float* s, const uint16_t* dy, int ldd,
                             float* dbt, bool have_terms, void* header, void* ws, const Stall& stall, cudaStream_t st);
// What the terms of rank block rb are made of, and where they go in `ws`.
TermsArgs lora_grad_terms(const aq_lora* ad, const int32_t* ids, int M, int rb, const float* t, int tsplits, int ldt,
                          const float* sx, const float* s, void* ws);

#if defined(__CUDACC__)
// v as three bf16 terms: hi + mid + lo = v to 24 bits.  A non-finite v stays in hi.
__device__ __forceinline__ void split3(float v, uint16_t& hi, uint16_t& mid, uint16_t& lo) {
  const __nv_bfloat16 h = __float2bfloat16_rn(v);
  float r = v - __bfloat162float(h);
  if (!(fabsf(r) < 3e38f)) r = 0.f;
  const __nv_bfloat16 m = __float2bfloat16_rn(r);
  const __nv_bfloat16 l = __float2bfloat16_rn(r - __bfloat162float(m));
  hi = __bfloat16_as_ushort(h);
  mid = __bfloat16_as_ushort(m);
  lo = __bfloat16_as_ushort(l);
}

// Eight ranks from c on of token m, which has `rank` from a.rb0 on.
__device__ __forceinline__ void write_terms(const TermsArgs& a, const TermsJob& j, int m, int c, int rank) {
  const int left = rank - c;
  float v[8] = {};
  if (left > 0) {
    const float* src = j.p + (size_t)m * j.ld + a.rb0 + c;
    const size_t step = (size_t)a.M * j.ld;
#pragma unroll 4
    for (int k = 0; k < j.splits; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e < left) v[e] += __ldg(src + k * step + e);
    if (j.sx) {
      const float scale = __ldg(j.sx + m);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= scale;
    }
  }
  uint16_t h[3][8];
#pragma unroll
  for (int e = 0; e < 8; ++e) split3(v[e], h[0][e], h[1][e], h[2][e]);
  uint16_t* d = j.terms + (size_t)m * a.npad + c;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = h[k][2 * e] | ((uint32_t)h[k][2 * e + 1] << 16);
    *reinterpret_cast<uint4*>(d + k * a.rc) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}
#endif

}  // namespace aq
