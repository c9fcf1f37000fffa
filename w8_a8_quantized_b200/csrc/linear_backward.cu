// Input gradient of a packed projection:
//   dx[m][k] = add[m][k] + sum_n dy[m][n] sw[n][j(k)] q[n][k],   j(k) = k / 128.
// One CTA per 64 tokens x 64 columns; 16 x 64 slices of dy and of the
// dequantized weights pass through shared memory, sums in fp32.
#include "aq_internal.cuh"

namespace aq {
namespace {

constexpr int kT = 64, kN = 16;

struct BwdArgs {
  aq_packed w;
  const uint16_t* dy;
  int ldd, M;
  const void* add;
  void* dx;
  int ldadd, lddx, f32;
};

__global__ void __launch_bounds__(256) linear_backward_kernel(const BwdArgs a) {
  __shared__ float sd[kN][kT + 1], sw[kN][kT + 1];
  const int tid = threadIdx.x, m0 = blockIdx.y * kT, k0 = blockIdx.x * kT, j = k0 / kTileK;
  const aq_packed& w = a.w;
  pdl_launch_dependents();
  pdl_wait();
  float acc[4][4] = {};
  for (int n0 = 0; n0 < w.N; n0 += kN) {
    const int r = n0 / w.bN, tile = r * w.C + j;
    const bool is4 = (w.bitmap[tile >> 3] >> (tile & 7)) & 1;
    const size_t base = (size_t)w.tile_idx[tile] * w.bN * kTileK;
    for (int i = tid; i < kN * kT; i += 256) {
      const int n = i / kT, k = i % kT, in_row = n0 + n - r * w.bN, in_col = k0 + k - j * kTileK;
      const size_t e = base + (size_t)in_row * kTileK + in_col;
      int q;
      if (is4) {
        const int b = w.w4[e >> 1];
        q = (int)(int8_t)((e & 1) ? (b & 0xF0) : (b << 4)) >> 4;
      } else {
        q = w.w8[e];
      }
      sw[n][k] = __half2float(__ushort_as_half(w.scales[(size_t)tile * w.bN + in_row])) * (float)q;
      const int m = i / kN, c = i % kN;
      sd[c][m] = m0 + m < a.M ? bf16_bits_to_float(a.dy[(size_t)(m0 + m) * a.ldd + n0 + c]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < kN; ++n)
#pragma unroll
      for (int y = 0; y < 4; ++y)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[y][x] = fmaf(sd[n][(tid / 16) * 4 + y], sw[n][(tid % 16) + 16 * x], acc[y][x]);
    __syncthreads();
  }
  for (int y = 0; y < 4; ++y) {
    const int m = m0 + (tid / 16) * 4 + y;
    if (m >= a.M) continue;
    for (int x = 0; x < 4; ++x) {
      const int k = k0 + tid % 16 + 16 * x;
      float v = acc[y][x];
      if (a.f32) {
        if (a.add) v += static_cast<const float*>(a.add)[(size_t)m * a.ldadd + k];
        static_cast<float*>(a.dx)[(size_t)m * a.lddx + k] = v;
      } else {
        if (a.add) v += bf16_bits_to_float(static_cast<const uint16_t*>(a.add)[(size_t)m * a.ldadd + k]);
        static_cast<__nv_bfloat16*>(a.dx)[(size_t)m * a.lddx + k] = __float2bfloat16_rn(v);
      }
    }
  }
}

}  // namespace
}  // namespace aq

using namespace aq;

static constexpr int kMaxBwdTokens = 1 << 21;

extern "C" size_t aq_linear_backward_workspace_bytes(int M, const aq_packed* w) {
  if (validate_packed(w) != AQ_OK || M < 1 || M > kMaxBwdTokens) return 0;
  return kWsHeader;
}

extern "C" int aq_linear_backward(const aq_packed* w, const uint16_t* dy, int ldd, int M, const void* add, int ldadd,
                                  void* dx, int lddx, int dxdtype, void* ws, size_t ws_bytes, void* stream) {
  int rc = validate_packed(w);
  if (rc != AQ_OK) return rc;
  if (!dy || !dx || M < 1 || M > kMaxBwdTokens || ldd < w->N || ldd % 8 || ((uintptr_t)dy & 15)) return AQ_ERR_ARG;
  if (dxdtype != AQ_F32 && dxdtype != AQ_BF16) return AQ_ERR_ARG;
  const int per16 = dxdtype == AQ_F32 ? 4 : 8;
  if (lddx < w->K || lddx % per16 || ((uintptr_t)dx & 15)) return AQ_ERR_ARG;
  if (add && (ldadd < w->K || ldadd % per16 || ((uintptr_t)add & 15))) return AQ_ERR_ARG;
  if (!ws || ws_bytes < aq_linear_backward_workspace_bytes(M, w)) return AQ_ERR_WORKSPACE;
  if ((uintptr_t)ws & 15) return AQ_ERR_ARG;
  BwdArgs a{*w, dy, ldd, M, add, dx, ldadd, lddx, dxdtype == AQ_F32};
  return launch_pdl(linear_backward_kernel, dim3(w->K / kT, (M + kT - 1) / kT), dim3(256), 0,
                    static_cast<cudaStream_t>(stream), a) == cudaSuccess
             ? AQ_OK
             : AQ_ERR_CUDA;
}
