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

// Where a call's work is cut. seg_len = 0: every (sequence, head) is one piece. Otherwise sequences
// are cut every L = seg_len tokens from their start, and sequence n keeps its segment j at place
// cu[n] / L + n + j of the workspace (total / L + num_seqs places are enough). Every segment but a
// sequence's last is found from a multiple of L: i L (i = 1 .. total / L) lies in exactly one such
// segment, behind its first token and at most at its end. So the host needs no lengths: total / L
// pieces for those, of which some stay idle, and one piece per sequence for the last segments.
struct LinearPlan {
  int32_t seg_len = 0;
  int32_t inner = 0;        // total / L
  int32_t col_tile = 0;     // value columns per CTA
  bool tensor = false;      // tensor-core kernel (bf16), else the token-recurrent one
  bool pad = false;         // runs on copies whose head sizes are padded to multiples of 8
  size_t states = 0;        // places in the workspace: [places, H, d_k, d_v] fp32 entering states,
  size_t decays = 0;        // [places, H] fp32 summed log-decays, the padded copies
  size_t pad_q = 0, pad_k = 0, pad_v = 0, pad_out = 0, pad_states = 0;
  size_t bytes = 0;         // of the workspace that the plan uses
};

constexpr int64_t kLinearMaxTokens = 0x7fffff80;  // 2^31 - 128: token indexes rounded up to chunks stay 32-bit
constexpr int kLinearSMs = 152;       // a GB300's (fixed: the workspace query needs no device)
constexpr int kLinearTokenCols = 64;  // value columns per CTA of the token-recurrent kernel

struct LinearSlot {
  int n;              // sequence
  int64_t place;      // in the workspace
  int64_t t0, t1;     // its tokens [t0, t1)
  bool first, last;   // of its sequence
};

// Piece `index`: the pieces for segments with a successor come first (they are the longest). False
// for an idle piece. Called by whole warps.
__device__ __forceinline__ bool linear_slot(const int32_t *__restrict__ cu, int num_seqs, int L, int inner, int index,
                                            LinearSlot &s) {
  if (index >= inner) {
    s.n = index - inner;
    const int64_t bos = cu[s.n], eos = cu[s.n + 1];
    const int j = L == 0 || eos == bos ? 0 : int((eos - bos - 1) / L);
    s.place = L == 0 ? 0 : bos / L + s.n + j;
    s.t0 = bos + int64_t(j) * L;
    s.t1 = eos;
    s.first = j == 0;
    s.last = true;
    return true;
  }
  // The last n that starts before (index + 1) L: a warp tries 32 candidates at a time (two
  // dependent reads for up to 1024 sequences, where halving takes ten). All lanes take part.
  const int64_t mark = int64_t(index + 1) * L;
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = num_seqs - 1;
  while (lo < hi) {
    const int stride = (hi - lo + 32) / 32, n = lo + lane * stride;
    const bool before = n <= hi && cu[n] < mark;  // true for lane 0, then false from some lane on
    const int last = 31 - __clz(__ballot_sync(0xffffffffu, before));
    lo += last * stride;
    hi = stride == 1 ? lo : (lo + stride - 1 < hi ? lo + stride - 1 : hi);
  }
  const int64_t bos = cu[lo], eos = cu[lo + 1];
  const int j = index - int(bos / L);
  s.n = lo;
  s.place = bos / L + lo + j;
  s.t0 = bos + int64_t(j) * L;
  s.t1 = s.t0 + L;
  s.first = j == 0;
  s.last = false;
  return s.t1 < eos;
}

// One decay step of a state entry, e^g s. Where e^g is one half or more it is s + (e^g - 1) s: e^g
// itself, rounded to fp32, would be off by up to 2^-25 in the same direction at every token of a head
// with a constant decay, which a memory of thousands of tokens adds up; e^g - 1 carries its error
// relative to itself. Below one half it is e^g s: there e^g - 1, near -1, would be off by 2^-25 of
// the state before the step, however little of it is left, and no memory is long. (For a choice at
// every token of a loop over rows see the token-recurrent kernel's own form.)
struct Decay {
  float c;    // e^g - 1, or e^g
  bool keep;  // whether s itself is added
};
__device__ __forceinline__ Decay decay_of(float g) {
  const float m = expm1f(g);
  return m < -0.5f ? Decay{expf(g), false} : Decay{m, true};  // a NaN keeps
}
__device__ __forceinline__ float decay_step(float s, Decay d) { return fmaf(d.c, s, d.keep ? s : 0.f); }

// The factor of the n-th decay step of a run, e^g in fp32, for loops that multiply by it. Simply
// rounded, the factors of a constant decay would all be off the same way, which a memory of thousands
// of tokens adds up. So the step takes a whole ulp more or less where `rest`, what one rounding loses in
// ulps, times the steps so far passes a half: factors of a constant decay stay within an ulp of e to the
// sum, others round either way without a bias. (Decay's choice between two forms, made in the token
// kernel's loop over rows, costs 2.07 ms at T = 4096, 96 heads of 128 in fp32; this 1.57.)
__device__ __forceinline__ float unbiased_decay(float g, int64_t step) {
  const Decay d = decay_of(g);
  if (!d.keep) return d.c;  // e^g below one half: no memory to drift
  const float e = 1.f + d.c;
  const uint32_t exponent = __float_as_uint(e) & 0x7f800000u;  // an ulp is 2^-23 of its power of two
  const float rest = (d.c - (e - 1.f)) * __uint_as_float(0x8a800000u - exponent);
  const float n = float(step & 4095);
  return fmaf(rintf((n + 1.f) * rest) - rintf(n * rest), __uint_as_float(exponent - 0x0b800000u), e);
}

struct LinearArgs {
  const void *q, *k, *v;
  const float *log_decay;   // [T, H], or [H] when !per_token
  const int32_t *cu;
  const float *init_state;  // [num_seqs, H, d_k, d_v] or null
  void *out;
  float *final_state;       // or null
  uint8_t *workspace;       // or null
  float *seg_states;        // in the workspace, or null (seg_len = 0)
  float *seg_decay;
  int num_seqs, H, H_k, d_k, d_v, per_token;
  int64_t total;
  float scale;
  LinearPlan plan;
};

// The passes of a segmented call are launched so that one may begin while the one before it drains: a
// kernel lets its successor begin once all its CTAs run, and a thread that reads what an earlier pass
// wrote waits for that pass to have ended. Pass 3 only does so for segments that enter with the
// workspace's states; sequences that are not cut, and first segments, run beside passes 1 and 2.
// Every CTA that has a piece waits before it ends (idle ones return at once), and pass 3 always has some, a
// last segment for each sequence, so that it never ends before an earlier pass; all CTAs of pass 2 wait.
__device__ __forceinline__ void let_next_pass_begin() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_earlier_passes() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_pass_kernel(void (*kern)(P...), dim3 grid, unsigned threads, size_t smem, bool overlap,
                               cudaStream_t stream, const A &...args) {
  cudaLaunchConfig_t c{};
  c.gridDim = grid, c.blockDim = dim3(threads), c.dynamicSmemBytes = smem, c.stream = stream;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &attr, c.numAttrs = overlap ? 1 : 0;
  return cudaLaunchKernelEx(&c, kern, args...);
}

// A cut sequence's first segment enters with the initial state; where the final one takes its place,
// pass 2 leaves a copy in the workspace, because the last segment may end before the first begins.
__host__ __device__ __forceinline__ bool linear_in_place(const LinearArgs &a) {
  return a.init_state != nullptr && a.init_state == a.final_state;
}
// The state that a segment enters with, or null (zeros), in pass 3. Waits for it.
__device__ __forceinline__ const float *linear_entering(const LinearArgs &a, const LinearSlot &s, int h) {
  const int64_t dd = int64_t(a.d_k) * a.d_v;
  if (!s.first || (!s.last && linear_in_place(a))) {
    wait_for_earlier_passes();
    return a.seg_states + (s.place * a.H + h) * dd;
  }
  return a.init_state != nullptr ? a.init_state + (int64_t(s.n) * a.H + h) * dd : nullptr;
}

// The plan for a call that has this much workspace (SIZE_MAX: what it would like to have).
LinearPlan linear_plan(int64_t total, int num_seqs, int H, int H_k, int d_k, int d_v, bool in_bf16, bool out_bf16,
                       bool recurrent, size_t workspace_bytes);
// Copies what needs padding and points `a` at the copies (d_v becomes the padded one; d_k stays, the
// states have that many rows), and brings the output and the final states back.
cudaError_t launch_linear_pad(LinearArgs &a, cudaStream_t stream);
cudaError_t launch_linear_unpad(const LinearArgs &a, bool out_bf16, void *out, float *final_state, int d_v,
                                cudaStream_t stream);
cudaError_t launch_linear_recurrent(const LinearArgs &a, bool in_bf16, bool out_bf16, cudaStream_t stream);
cudaError_t launch_linear_chunked(const LinearArgs &a, bool out_bf16, cudaStream_t stream);
cudaError_t launch_linear_scan(const LinearArgs &a, cudaStream_t stream);

}  // namespace kda
