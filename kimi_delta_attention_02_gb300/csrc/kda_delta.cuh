// kda_delta.cuh -- what the kernels of the gated delta rule with one decay per head share:
// S_t = (I - beta_t k_t k_t^T) e^{g_t} S_{t-1} + beta_t k_t v_t^T, o_t = scale S_t^T q_t per sequence
// and value head, with the query / key head h / (H / H_k).
//
// The state a segment of tokens leaves is affine in the one it enters with, S_end = M S_start + B: M is
// what the segment makes of the identity with v = 0, B what it makes of zero. A sequence cut into
// segments runs in three passes (the slots are those of linear attention, kda_linear.cuh): pass 1 runs
// every sequence's first segment to the end, outputs included, and forms M and B of the segments between
// the first and the last; pass 2 chains them; pass 3 runs the segments behind the first from their
// entering states. Sequences that are not cut are done in pass 1.
#pragma once

#include "kda_linear.cuh"

namespace kda {

struct DeltaPlan {
  bool tensor = false;   // tensor-core kernel, else the token kernel
  int32_t few = -1;      // sequences of up to this many tokens are the decode kernel's (-1: none)
  bool order = false;    // longest sequences first, by a list in the workspace
  bool pad = false;      // q, k, v by copies whose head sizes are padded to multiples of 8
  int32_t seg_len = 0;   // tokens between cuts (0: none)
  int32_t inner = 0;     // total / seg_len
  size_t pad_q = 0, pad_k = 0, pad_v = 0;  // in the workspace: the copies;
  size_t ends = 0;       // [inner, H, d_k, d_v] fp32 (padded sizes), the states that segments leave, or the list,
  size_t maps = 0;       // [inner, H, d_k, d_k] fp32 (padded sizes), their M
  size_t bytes = 0;      // of the workspace that the plan uses
};

struct DeltaArgs {
  const void *q, *k, *v;
  const float *log_decay;   // [T, H], or [H] when !per_token
  const float *beta;        // [T, H]
  const int32_t *cu;
  const float *init_state;  // [num_seqs, H, d_k, d_v] or null
  void *out;
  float *final_state;       // or null
  uint8_t *workspace;       // or null
  int num_seqs, H, H_k, d_k, d_v, per_token;
  int64_t total;
  float scale;
  DeltaPlan plan;
};

// The place in the workspace of a segment with a successor: its own number among the multiples of the
// segment length (see LinearPlan). Its predecessor's is one less.
__device__ __forceinline__ int64_t delta_place(const DeltaArgs &a, const LinearSlot &s) {
  const int64_t bos = a.cu[s.n];
  return a.plan.seg_len == 0 ? 0 : bos / a.plan.seg_len + (s.t0 - bos) / a.plan.seg_len;
}

__host__ __device__ constexpr int delta_up8(int d) { return (d + 7) & ~7; }

// The plan for a call that has this much workspace (SIZE_MAX: what it would like to have).
DeltaPlan delta_plan(int64_t total, int num_seqs, int H, int H_k, int d_k, int d_v, bool in_bf16, bool out_bf16,
                     bool recurrent, size_t workspace_bytes);
cudaError_t launch_delta_recurrent(const DeltaArgs &a, bool in_bf16, bool out_bf16, cudaStream_t stream);
cudaError_t launch_delta_short(const DeltaArgs &a, bool in_bf16, bool out_bf16, cudaStream_t stream);
cudaError_t launch_delta_chunked(const DeltaArgs &a, bool out_bf16, cudaStream_t stream);
cudaError_t launch_delta_chain(const DeltaArgs &a, cudaStream_t stream);
cudaError_t launch_delta_decode(const void *q, const void *k, const void *v, const float *log_decay, bool per_token,
                                const float *beta, float *state, void *out, int B, int H, int H_k, int d_k, int d_v,
                                bool in_bf16, bool out_bf16, float scale, cudaStream_t stream);

}  // namespace kda
