// Shared by the adapter kernels.
#pragma once

#include "aq_internal.cuh"

namespace aq {

// Decode batches (lora_decode.cu): whether the one-launch kernel takes the call, and the call.
bool lora_decode_fits(const aq_lora* ad, int M);
cudaError_t launch_lora_decode(const aq_lora* ad, const uint16_t* x, int ldx, const int32_t* ids, int M, const void* y,
                               int ldy, void* out, int ldo, bool f32, float* s, cudaStream_t st);

}  // namespace aq
