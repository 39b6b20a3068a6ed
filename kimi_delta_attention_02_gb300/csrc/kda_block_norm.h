// kda_block_norm.h -- arguments of the block norm kernel (kda_block_norm.cu).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace kda {

constexpr int kBlockNormMaxD = 16384;  // 512 threads x 32 channels in registers

struct BlockNormArgs {
  const void *x, *y, *gate;  // y, gate: null without
  const float *post_weight, *channel_scale, *pre_weight;
  void *residual_out, *out;
  int64_t rows;
  int D;
  int gate_form;  // 0 none, 1 per channel, 2 per row
  int post_norm;
  float scale, post_eps, pre_eps;
  int threads_per_row, stages;  // set by the launcher
};

cudaError_t launch_block_norm(BlockNormArgs a, bool x_bf16, bool y_bf16, bool out_bf16, cudaStream_t stream);

}  // namespace kda
