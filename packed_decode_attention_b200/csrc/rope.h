// Launch parameters of the rotary positions over several axes (rope.cu),
// shared by the kernel and the C ABI (api_rope.cu).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

namespace bgtq {

struct RopeAxesArgs {
  double turns[64];                    // base^(-2j/128) / (2 pi)
  uint8_t axis[64];
  const int32_t* pos;                  // [axes][tokens]
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;  // elements from a token to the next
  int64_t tokens;
  int32_t hq, hkv, pairing;
  int32_t parts, part_heads;           // set by the launch
};

cudaError_t launch_rope_axes(RopeAxesArgs& a, int bf16, int n_sms, cudaStream_t stream);

}  // namespace bgtq
