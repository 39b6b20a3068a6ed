// kda_linear.cuh -- what the linear-attention kernels share: the plan that cuts packed
// sequences into segments, and a kernel's way from its block to its segment.
//
// Per sequence and head: S_t = e^{g_t} S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t. The state a
// segment of tokens leaves is affine in the state it enters with a scalar factor,
// S_end = e^{sum g} S_start + B (B: the state it leaves from zero), so segments of one sequence
// can run side by side: pass 1 forms B of every segment but a sequence's last, pass 2 chains
// them, pass 3 runs all segments from their entering states.
#pragma once

#include "kda_common.cuh"

namespace kda {

// Where a call's work is cut. seg_len = 0: every (sequence, head) is one piece and slot n is
// sequence n. Otherwise sequence n owns the slots cu[n] / L + n .. cu[n + 1] / L + n (L =
// seg_len): the first ceil(len / L) of them hold its segments (an empty sequence holds one empty
// segment), the others are idle. A slot is found from cu_seqlens alone, so the host needs no
// lengths and the grid is total / L + num_seqs slots.
struct LinearPlan {
  int32_t seg_len = 0;
  int32_t slots = 0;
  int32_t col_tile = 0;     // value columns per CTA
  bool tensor = false;      // tensor-core kernel (bf16), else the token-recurrent one
  size_t state_bytes = 0;   // workspace: [slots, H, d_k, d_v] fp32 entering states, then
  size_t bytes = 0;         // [slots, H] fp32 summed log-decays
};

struct LinearSlot {
  int n;              // sequence
  int64_t t0, t1;     // its tokens [t0, t1)
  bool first, last;   // of its sequence
};

// False for an idle slot. Called by whole warps.
__device__ __forceinline__ bool linear_slot(const int32_t *__restrict__ cu, int num_seqs, int seg_len, int slot,
                                            LinearSlot &s) {
  if (seg_len == 0) {
    s.n = slot;
    s.t0 = cu[slot];
    s.t1 = cu[slot + 1];
    s.first = s.last = true;
    return true;
  }
  // The last n whose first slot cu[n] / L + n is <= slot: a warp tries 32 candidates at a time (two
  // dependent reads for up to 1024 sequences, where halving takes ten). All lanes take part.
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = num_seqs - 1;
  while (lo < hi) {
    const int stride = (hi - lo + 32) / 32, n = lo + lane * stride;
    const bool fits = n <= hi && cu[n] / seg_len + n <= slot;  // true for lane 0, then false from some lane on
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, fits));
    lo += last * stride;
    hi = stride == 1 ? lo : (lo + stride - 1 < hi ? lo + stride - 1 : hi);
  }
  const int64_t bos = cu[lo], eos = cu[lo + 1];
  const int j = slot - (int(bos) / seg_len + lo);
  s.n = lo;
  s.t0 = bos + int64_t(j) * seg_len;
  s.t1 = s.t0 + seg_len < eos ? s.t0 + seg_len : eos;
  s.first = j == 0;
  s.last = s.t0 + seg_len >= eos;
  return s.first || s.t0 < eos;
}

// One decay step of a state entry: e^g s, as s + (e^g - 1) s. e^g itself, rounded to fp32, would
// be off by up to 2^-25 in the same direction at every token of a head with a constant decay,
// which a memory of thousands of tokens adds up; e^g - 1 carries its error relative to itself.
__device__ __forceinline__ float decay_step(float s, float expm1_g) { return fmaf(expm1_g, s, s); }

struct LinearArgs {
  const void *q, *k, *v;
  const float *log_decay;   // [T, H], or [H] when !per_token
  const int32_t *cu;
  const float *init_state;  // [num_seqs, H, d_k, d_v] or null
  void *out;
  float *final_state;       // or null
  float *seg_states;        // workspace, or null (seg_len = 0)
  float *seg_decay;
  int num_seqs, H, H_k, d_k, d_v, per_token;
  int64_t total;
  float scale;
  LinearPlan plan;
};

LinearPlan linear_plan(int64_t total, int num_seqs, int H, int d_k, int d_v, bool in_bf16, bool out_bf16,
                       bool recurrent);
cudaError_t launch_linear_recurrent(const LinearArgs &a, bool in_bf16, bool out_bf16, cudaStream_t stream);
bool linear_chunked_supported(int d_k, int d_v, bool in_bf16);
cudaError_t launch_linear_chunked(const LinearArgs &a, bool out_bf16, cudaStream_t stream);
cudaError_t launch_linear_scan(const LinearArgs &a, cudaStream_t stream);

}  // namespace kda
