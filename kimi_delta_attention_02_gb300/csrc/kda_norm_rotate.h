// kda_norm_rotate.h -- host side of the norm and rotation of queries and keys (kda_norm_rotate.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace kda {

constexpr int kRotateMaxD = 256, kRotateMaxAxes = 4;

struct RotateArgs {
  const void *x[2];        // q, k
  void *out[2];
  const float *weight[2];  // or null
  int64_t stride[2], out_stride[2];  // elements from token to token
  int32_t heads[2];
  const void *positions;   // [axes][tokens], or null (no rotation)
  const float *inv_freq;
  int64_t tokens;
  int32_t d, half, norm, pos64;
  float eps, per;  // the norm's factor is 1 / sqrt(per sum(x^2) + eps)
  uint8_t axis[kRotateMaxD / 2];
};

cudaError_t launch_norm_rotate(const RotateArgs &a, bool in_bf16, bool out_bf16, bool interleaved, cudaStream_t stream);

}  // namespace kda
