// kda_delta.cuh -- what the kernels of the gated delta rule with one decay per head share:
// S_t = (I - beta_t k_t k_t^T) e^{g_t} S_{t-1} + beta_t k_t v_t^T, o_t = scale S_t^T q_t per sequence
// and value head, with the query / key head h / (H / H_k).
#pragma once

#include "kda_linear.cuh"

namespace kda {

struct DeltaArgs {
  const void *q, *k, *v;
  const float *log_decay;   // [T, H], or [H] when !per_token
  const float *beta;        // [T, H]
  const int32_t *cu;
  const float *init_state;  // [num_seqs, H, d_k, d_v] or null
  void *out;
  float *final_state;       // or null
  int num_seqs, H, H_k, d_k, d_v, per_token;
  int64_t total;
  float scale;
};

cudaError_t launch_delta_recurrent(const DeltaArgs &a, bool in_bf16, bool out_bf16, cudaStream_t stream);
cudaError_t launch_delta_decode(const void *q, const void *k, const void *v, const float *log_decay, bool per_token,
                                const float *beta, float *state, void *out, int B, int H, int H_k, int d_k, int d_v,
                                bool in_bf16, bool out_bf16, float scale, cudaStream_t stream);

}  // namespace kda
