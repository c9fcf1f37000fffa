// Shared by the bf16 tensor-core kernels (tcgen05, kind::f16).
#pragma once

#include "aq_internal.cuh"

namespace aq {
namespace {

#if defined(__CUDACC__)
// D[tmem] (+)= A[smem] * B[smem]^T, bf16 x bf16 -> fp32, by one CTA or a pair of them.
template <int CG = 1>
__device__ __forceinline__ void mma_bf16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}

// Descriptor of an MN-major operand in the 128-byte swizzle: groups of 8 rows
// (contraction) 1024 bytes apart, the next 64 columns `lead` bytes on.
__device__ __forceinline__ uint64_t mn_desc(uint32_t smem_addr, uint32_t lead) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr >> 4) & 0x3FFF);
  d |= (uint64_t)(lead >> 4) << 16;  // leading: the next 64 columns
  d |= (uint64_t)(1024 >> 4) << 32;           // stride: the next 8 rows
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// Instruction descriptor: D fp32, A and B bf16, M = 128 (256 for a pair); mn_a / mn_b: the operand is MN-major.
__host__ __device__ constexpr uint32_t idesc_bf16(int n, bool mn_a, bool mn_b, int m = 128) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)mn_a << 15) | ((uint32_t)mn_b << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// One lane of a converged warp.  MMAs and commits issued under it take 130 + 50 cycles per
// four + two of them; under `lane == 0` in a diverged warp they took 360 + 220, since
// their operands are then not known to be uniform.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Ring position with its phase parity.
struct Ring {
  uint32_t i, ph;
  template <int N>
  __device__ __forceinline__ void next() {
    if (++i == N) {
      i = 0;
      ph ^= 1u;
    }
  }
};

// A producer that has stopped (see Stall) stays until the other roles have given up.
__device__ __forceinline__ void stalled(volatile int* abort, unsigned long long wait_ns) {
  const unsigned long long t0 = globaltimer_ns();
  while (!*abort && globaltimer_ns() - t0 < 2 * wait_ns) __nanosleep(1000);
}

// Copies in flight when a CTA gives up get this long to land.
__device__ __forceinline__ void grace() {
  const unsigned long long t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < 200000ull) __nanosleep(1000);
}

#endif

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<EncodeFn>(p) : nullptr;
  }();
  return fn;
}

bool map_2d(CUtensorMap* m, CUtensorMapDataType type, const void* base, uint64_t cols, uint64_t rows, uint64_t pitch,
            uint32_t box_cols, uint32_t box_rows, bool swizzle) {
  EncodeFn fn = encode();
  if (!fn) return false;
  const cuuint64_t dims[2] = {cols, rows}, strides[1] = {pitch};
  const cuuint32_t box[2] = {box_cols, box_rows}, one[2] = {1, 1};
  return fn(m, type, 2, const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            swizzle ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace aq
