// kda_api.cu -- the C ABI of libkda (declared in include/kda.h): argument
// validation on the host, dispatch to the kernels, the device error word.
#include <cmath>
#include <cstdint>

#include "kda_block_norm.h"
#include "kda_common.cuh"
#include "kda_delta.cuh"
#include "kda_linear.cuh"
#include "kda_norm_rotate.h"

#include <atomic>
#include <mutex>

namespace kda {

namespace {
__device__ uint32_t g_device_error = 0;
// what the last kda_check_device_error took out of g_device_error (read back by the host)
__device__ uint32_t g_device_error_taken = 0;
constexpr int kMaxDevices = 64;
std::atomic<uint32_t *> g_error_word[kMaxDevices];
std::mutex g_error_word_mu;
std::mutex g_check_mu;  // one kda_check_device_error at a time: they share g_device_error_taken

// Read and clear the error word in one step, behind the work already on the stream.
__global__ void take_device_error_kernel() { g_device_error_taken = atomicExch(&g_device_error, 0u); }
}  // namespace

uint32_t *device_error_word() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  uint32_t *p = g_error_word[dev].load(std::memory_order_acquire);
  if (p != nullptr) return p;
  std::lock_guard<std::mutex> lock(g_error_word_mu);
  p = g_error_word[dev].load(std::memory_order_relaxed);
  if (p == nullptr) {
    void *addr = nullptr;
    if (cudaGetSymbolAddress(&addr, g_device_error) != cudaSuccess) return nullptr;
    p = static_cast<uint32_t *>(addr);
    g_error_word[dev].store(p, std::memory_order_release);
  }
  return p;
}

// ---------------------------------------------------------------------------------------------
// Scratch of kda_prefill_noalloc, for callers that cannot hand the library a workspace. It is a
// file-scope device array, so every GPU that loads this library holds these 16 MiB until the
// process exits. Host code may not use its name as a device address (on the host it names a
// stand-in): noalloc_scratch() looks the address up once per device, with that device current.
// ---------------------------------------------------------------------------------------------
constexpr size_t kNoAllocScratchBytes = size_t(16) << 20;
static __device__ __align__(256) uint8_t g_noalloc_scratch[kNoAllocScratchBytes];

namespace {
std::atomic<void *> g_noalloc_ptr[kMaxDevices];
std::mutex g_noalloc_mu;

// Device address of g_noalloc_scratch on the current device (nullptr if the lookup failed). The
// first call on a device does the lookup, which may load the library's device code: it must not
// happen inside a stream capture.
void *noalloc_scratch() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
  void *p = g_noalloc_ptr[dev].load(std::memory_order_acquire);
  if (p != nullptr) return p;
  std::lock_guard<std::mutex> lock(g_noalloc_mu);
  p = g_noalloc_ptr[dev].load(std::memory_order_relaxed);
  if (p == nullptr) {
    void *addr = nullptr;
    if (cudaGetSymbolAddress(&addr, g_noalloc_scratch) != cudaSuccess || addr == nullptr) return nullptr;
    p = addr;
    g_noalloc_ptr[dev].store(p, std::memory_order_release);
  }
  return p;
}
}  // namespace

// Each launcher takes the decay input as `decay` + `A_log`: log_alpha (fp32) with A_log null
// (the clamped form), or the gated form's logits z (input dtype) with A_log [H]; and the output
// gate as `out_gate` (gate logits, input dtype; null = plain read-out) + `norm_weight` + `norm_eps`.
cudaError_t launch_decode(const void *q, const void *k, const void *v, const void *decay, int decay_form,
                          const float *A_log, const float *beta, float *state, const void *out_gate,
                          const float *norm_weight, float norm_eps, const float *conv_w, void *conv_state,
                          float l2_eps, void *out, int B, int H, int d_k, int d_v, bool in_bf16, bool out_bf16,
                          float lb, float scale, cudaStream_t stream);
cudaError_t launch_prologue(const void *q_raw, const void *k_raw, const void *v_raw, const float *conv_w,
                            const int32_t *cu_seqlens, int num_seqs, int64_t total_tokens, int H, int d_k, int d_v,
                            bool bf16, const void *conv_init, float eps, void *q, void *k, void *v,
                            void *conv_final, cudaStream_t stream);
cudaError_t launch_recurrent(const void *q, const void *k, const void *v, const void *decay, int decay_form,
                             const float *A_log, const float *beta, const int32_t *cu_seqlens, int num_seqs, int H,
                             int d_k, int d_v, bool in_bf16, bool out_bf16, float lb, float scale,
                             const float *init_state, const void *out_gate, const float *norm_weight,
                             float norm_eps, void *out, float *final_state, cudaStream_t stream);
bool chunked_supported(int d_k, int d_v, bool in_bf16, float lb, int decay_form);
size_t prefill_workspace_bytes(int64_t total_tokens, int32_t num_seqs, int32_t H, int32_t d_k, int32_t d_v);
kda_status launch_chunked(const void *q, const void *k, const void *v, const void *decay, int decay_form,
                          const float *A_log, const float *beta, const int32_t *cu_seqlens, int num_seqs,
                          int64_t total_tokens, int H, bool out_bf16, float lb, float scale, const float *init_state,
                          const void *out_gate, const float *norm_weight, float norm_eps, void *out,
                          float *final_state, void *workspace, size_t workspace_bytes, cudaStream_t stream);
cudaError_t launch_linear_decode(const void *q, const void *k, const void *v, const float *log_decay, bool per_token,
                                 float *state, void *out, int B, int H, int H_k, int d_k, int d_v, bool in_bf16,
                                 bool out_bf16, float scale, cudaStream_t stream);

namespace {

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
bool finite_nonneg(float x) { return x >= 0.f && x < INFINITY; }  // false for NaN

// whether the byte ranges [a, a + na) and [b, b + nb) intersect (null or empty never does)
bool overlaps(const void *a, size_t na, const void *b, size_t nb) {
  if (!a || !b || !na || !nb) return false;
  const char *pa = static_cast<const char *>(a), *pb = static_cast<const char *>(b);
  return pa < pb + nb && pb < pa + na;
}

// decay: log_alpha (fp32) when A_log is null, else the gated form's logits z (in_dtype)
kda_status check_prefill_args(const void *q, const void *k, const void *v, const void *decay, const float *A_log,
                              const float *beta, const int32_t *cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                              int32_t H, int32_t d_k, int32_t d_v, kda_dtype in_dtype, kda_dtype out_dtype,
                              const float *init_state, const void *out, const float *final_state,
                              const void *out_gate = nullptr, const float *norm_weight = nullptr) {
  if (in_dtype != KDA_F32 && in_dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (out_dtype != KDA_F32 && out_dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (num_seqs < 0 || total_tokens < 0 || H < 1 || d_k < 1 || d_v < 1) return KDA_ERR_INVALID_ARG;
  if (d_k > 128 || d_v > 128) return KDA_ERR_UNSUPPORTED;
  if (total_tokens > INT32_MAX) return KDA_ERR_UNSUPPORTED;  // cu_seqlens are int32
  if (int64_t(num_seqs) * H > INT32_MAX / 4) return KDA_ERR_UNSUPPORTED;
  if (cu_seqlens == nullptr || !aligned4(cu_seqlens)) return KDA_ERR_INVALID_ARG;
  if (total_tokens > 0) {
    if (!q || !k || !v || !decay || !beta || !out) return KDA_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(decay) || !aligned16(out) ||
        !aligned4(beta))
      return KDA_ERR_INVALID_ARG;
  }
  if (init_state && !aligned16(init_state)) return KDA_ERR_INVALID_ARG;
  if (final_state && !aligned16(final_state)) return KDA_ERR_INVALID_ARG;
  // outputs must not overlap the inputs (final_state == init_state is allowed)
  const size_t es = in_dtype == KDA_BF16 ? 2 : 4, eo = out_dtype == KDA_BF16 ? 2 : 4;
  const size_t nk = size_t(total_tokens) * H * d_k, nv = size_t(total_tokens) * H * d_v;
  const size_t ns = size_t(num_seqs) * H * d_k * d_v * 4;
  if (total_tokens > 0 && out_gate != nullptr && !aligned16(out_gate)) return KDA_ERR_INVALID_ARG;
  if (norm_weight != nullptr && !aligned4(norm_weight)) return KDA_ERR_INVALID_ARG;
  const void *ins[8] = {q, k, v, decay, beta, A_log, out_gate, norm_weight};
  const size_t in_bytes[8] = {nk * es, nk * es, nv * es, nk * (A_log ? es : 4), size_t(total_tokens) * H * 4,
                              A_log ? size_t(H) * 4 : 0, out_gate ? nv * es : 0,
                              norm_weight ? size_t(d_v) * 4 : 0};
  for (int i = 0; i < 8; ++i) {
    if (overlaps(out, nv * eo, ins[i], in_bytes[i])) return KDA_ERR_INVALID_ARG;
    if (overlaps(final_state, ns, ins[i], in_bytes[i])) return KDA_ERR_INVALID_ARG;
  }
  if (overlaps(out, nv * eo, init_state, ns) || overlaps(out, nv * eo, final_state, ns))
    return KDA_ERR_INVALID_ARG;
  if (final_state != init_state && overlaps(final_state, ns, init_state, ns)) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

// The workspace: NULL with 0 bytes, or a 16-byte-aligned device range that overlaps no tensor argument.
kda_status check_workspace(const void *ws, size_t ws_bytes, const void *q, const void *k, const void *v,
                           const void *decay, const float *A_log, const float *beta, const int32_t *cu_seqlens,
                           int32_t num_seqs, int64_t total_tokens, int32_t H, int32_t d_k, int32_t d_v,
                           kda_dtype in_dtype, kda_dtype out_dtype, const float *init_state, const void *out,
                           const float *final_state, const void *out_gate, const float *norm_weight) {
  if (ws == nullptr) return ws_bytes == 0 ? KDA_OK : KDA_ERR_INVALID_ARG;
  if (ws_bytes == 0 || !aligned16(ws)) return KDA_ERR_INVALID_ARG;
  const size_t es = in_dtype == KDA_BF16 ? 2 : 4, eo = out_dtype == KDA_BF16 ? 2 : 4;
  const size_t nk = size_t(total_tokens) * H * d_k, nv = size_t(total_tokens) * H * d_v;
  const size_t ns = size_t(num_seqs) * H * d_k * d_v * 4;
  const void *args[12] = {q, k, v, decay, beta, A_log, out_gate, norm_weight, cu_seqlens, init_state, out,
                          final_state};
  const size_t bytes[12] = {nk * es, nk * es, nv * es, nk * (A_log ? es : 4), size_t(total_tokens) * H * 4,
                            A_log ? size_t(H) * 4 : 0, out_gate ? nv * es : 0, norm_weight ? size_t(d_v) * 4 : 0,
                            size_t(num_seqs + 1) * 4, init_state ? ns : 0, nv * eo, final_state ? ns : 0};
  for (int i = 0; i < 12; ++i)
    if (overlaps(ws, ws_bytes, args[i], bytes[i])) return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

// the gated form's parameters: A_log [H] fp32 on the device, g_min finite and <= 0
kda_status check_gate_args(const float *A_log, float g_min) {
  if (A_log == nullptr || !aligned4(A_log)) return KDA_ERR_INVALID_ARG;
  if (!(g_min <= 0.f) || !(g_min > -INFINITY)) return KDA_ERR_INVALID_ARG;  // rejects NaN and -inf
  return KDA_OK;
}

// the output gate's parameters: the weight only with gate logits, eps finite and >= 0
kda_status check_out_gate_args(const void *out_gate, const float *norm_weight, float norm_eps) {
  if (out_gate == nullptr) return norm_weight == nullptr ? KDA_OK : KDA_ERR_INVALID_ARG;
  if (!(norm_eps >= 0.f) || !(norm_eps < INFINITY)) return KDA_ERR_INVALID_ARG;  // rejects NaN and inf
  return KDA_OK;
}

kda_status prefill_impl(const void *q, const void *k, const void *v, const void *decay, const float *A_log,
                        const float *beta, const int32_t *cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                        int32_t H, int32_t d_k, int32_t d_v, kda_dtype in_dtype, kda_dtype out_dtype, float lb,
                        float scale, const float *init_state, void *out, float *final_state, void *stream,
                        bool force_recurrent, const void *out_gate = nullptr, const float *norm_weight = nullptr,
                        float norm_eps = 0.f, int decay_form = -1, void *workspace = nullptr,
                        size_t workspace_bytes = 0) {
  if (decay_form < 0) decay_form = A_log != nullptr ? DECAY_GATED : DECAY_CLAMPED;
  kda_status st = check_out_gate_args(out_gate, norm_weight, norm_eps);
  if (st != KDA_OK) return st;
  st = check_prefill_args(q, k, v, decay, A_log, beta, cu_seqlens, num_seqs, total_tokens, H, d_k, d_v, in_dtype,
                          out_dtype, init_state, out, final_state, out_gate, norm_weight);
  if (st != KDA_OK) return st;
  st = check_workspace(workspace, workspace_bytes, q, k, v, decay, A_log, beta, cu_seqlens, num_seqs, total_tokens,
                       H, d_k, d_v, in_dtype, out_dtype, init_state, out, final_state, out_gate, norm_weight);
  if (st != KDA_OK) return st;
  if (num_seqs == 0) return KDA_OK;
  if (total_tokens == 0) out_gate = norm_weight = nullptr;  // nothing is read out
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  // the chunked kernels: bf16 inputs, d = 128; a bounded map with a lower bound >= -5, or the
  // unbounded map
  if (!force_recurrent && total_tokens > 0 && chunked_supported(d_k, d_v, in_dtype == KDA_BF16, lb, decay_form))
    return launch_chunked(q, k, v, decay, decay_form, A_log, beta, cu_seqlens, num_seqs, total_tokens, H,
                          out_dtype == KDA_BF16, lb, scale, init_state, out_gate, norm_weight, norm_eps, out,
                          final_state, workspace, workspace_bytes, s);
  const cudaError_t err = launch_recurrent(q, k, v, decay, decay_form, A_log, beta, cu_seqlens, num_seqs, H, d_k, d_v,
                                           in_dtype == KDA_BF16, out_dtype == KDA_BF16, lb, scale, init_state,
                                           out_gate, norm_weight, norm_eps, out, final_state, s);
  return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status decode_impl(const void *q, const void *k, const void *v, const void *decay, const float *A_log,
                       const float *beta, float *state, void *out, int32_t B, int32_t H, int32_t d_k, int32_t d_v,
                       kda_dtype in_dtype, kda_dtype out_dtype, float lb, float scale, void *stream,
                       const void *out_gate = nullptr, const float *norm_weight = nullptr, float norm_eps = 0.f,
                       const float *conv_weight = nullptr, void *conv_state = nullptr, float l2_eps = 0.f,
                       int decay_form = -1) {
  if (decay_form < 0) decay_form = A_log != nullptr ? DECAY_GATED : DECAY_CLAMPED;
  if (in_dtype != KDA_F32 && in_dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (out_dtype != KDA_F32 && out_dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (B < 1 || H < 1 || d_k < 1 || d_v < 1) return KDA_ERR_INVALID_ARG;
  if (d_k > 128 || d_v > 128 || (d_v & 3) != 0) return KDA_ERR_UNSUPPORTED;
  if (int64_t(B) * H > INT32_MAX) return KDA_ERR_UNSUPPORTED;
  if (!q || !k || !v || !decay || !beta || !state || !out) return KDA_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(decay) || !aligned16(state) ||
      !aligned16(out) || !aligned4(beta))
    return KDA_ERR_INVALID_ARG;
  const kda_status st = check_out_gate_args(out_gate, norm_weight, norm_eps);
  if (st != KDA_OK) return st;
  if ((out_gate && !aligned16(out_gate)) || (norm_weight && !aligned4(norm_weight))) return KDA_ERR_INVALID_ARG;
  {  // state (read and rewritten) and out (written) must not overlap each other or any input
    const size_t es = in_dtype == KDA_BF16 ? 2 : 4, eo = out_dtype == KDA_BF16 ? 2 : 4;
    const size_t nk = size_t(B) * H * d_k, nv = size_t(B) * H * d_v, ns = size_t(B) * H * d_k * d_v * 4;
    const void *ins[8] = {q, k, v, decay, beta, A_log, out_gate, norm_weight};
    const size_t in_bytes[8] = {nk * es, nk * es, nv * es, nk * (A_log ? es : 4), size_t(B) * H * 4,
                                A_log ? size_t(H) * 4 : 0, out_gate ? nv * es : 0, norm_weight ? size_t(d_v) * 4 : 0};
    for (int i = 0; i < 8; ++i)
      if (overlaps(state, ns, ins[i], in_bytes[i]) || overlaps(out, nv * eo, ins[i], in_bytes[i]))
        return KDA_ERR_INVALID_ARG;
    if (overlaps(out, nv * eo, state, ns)) return KDA_ERR_INVALID_ARG;
  }
  if (conv_state != nullptr) {  // the prologue: weights and state on the device, eps finite
    if (conv_weight == nullptr || !aligned16(conv_weight) || !aligned16(conv_state) || !finite_nonneg(l2_eps))
      return KDA_ERR_INVALID_ARG;
    const size_t es = in_dtype == KDA_BF16 ? 2 : 4, eo = out_dtype == KDA_BF16 ? 2 : 4;
    const size_t ncs = size_t(B) * H * 3 * (2 * d_k + d_v) * es;
    const size_t nk = size_t(B) * H * d_k, nv = size_t(B) * H * d_v;
    if (overlaps(conv_state, ncs, state, size_t(B) * H * d_k * d_v * 4) ||
        overlaps(conv_state, ncs, out, nv * eo) || overlaps(conv_state, ncs, q, nk * es) ||
        overlaps(conv_state, ncs, k, nk * es) || overlaps(conv_state, ncs, v, nv * es) ||
        overlaps(conv_state, ncs, conv_weight, size_t(H) * (2 * d_k + d_v) * 16) ||
        overlaps(state, size_t(B) * H * d_k * d_v * 4, conv_weight, size_t(H) * (2 * d_k + d_v) * 16) ||
        overlaps(out, nv * eo, conv_weight, size_t(H) * (2 * d_k + d_v) * 16))
      return KDA_ERR_INVALID_ARG;
  } else if (conv_weight != nullptr) {
    return KDA_ERR_INVALID_ARG;  // weights without a state
  }
  const cudaError_t err = launch_decode(q, k, v, decay, decay_form, A_log, beta, state, out_gate, norm_weight, norm_eps,
                                        conv_weight, conv_state, l2_eps, out, B, H, d_k, d_v, in_dtype == KDA_BF16,
                                        out_dtype == KDA_BF16, lb, scale, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

// the decay form of a parameter block: the clamped form takes no A_log, the gated ones need it
// (the unbounded one has no bound to check)
kda_status check_decay_form(kda_decay_form form, const float *A_log, float bound) {
  if (form == KDA_DECAY_CLAMPED) return A_log == nullptr ? KDA_OK : KDA_ERR_INVALID_ARG;
  if (form == KDA_DECAY_GATED) return check_gate_args(A_log, bound);
  if (form == KDA_DECAY_UNBOUNDED) return (A_log != nullptr && aligned4(A_log)) ? KDA_OK : KDA_ERR_INVALID_ARG;
  return KDA_ERR_INVALID_ARG;
}

bool valid_dtype(kda_dtype d) { return d == KDA_F32 || d == KDA_BF16; }

// Sizes of a linear-attention call: rows of q, k, v (tokens, or decode's B) and states.
kda_status check_linear_sizes(int64_t rows, int64_t states, int32_t H, int32_t H_k, int32_t d_k, int32_t d_v,
                              int32_t per_token, kda_dtype in_dtype, kda_dtype out_dtype) {
  if (!valid_dtype(in_dtype) || !valid_dtype(out_dtype)) return KDA_ERR_INVALID_ARG;
  if (rows < 0 || states < 0 || H < 1 || H_k < 1 || d_k < 1 || d_v < 1) return KDA_ERR_INVALID_ARG;
  if (H % H_k != 0 || (per_token != 0 && per_token != 1)) return KDA_ERR_INVALID_ARG;
  if (d_k > 128 || d_v > 128 || rows > kLinearMaxTokens || states * H > INT32_MAX / 4) return KDA_ERR_UNSUPPORTED;
  if (rows * H > INT64_MAX / 1024) return KDA_ERR_UNSUPPORTED;  // bytes of a tensor
  return KDA_OK;
}

// A byte range of a tensor argument (null: none). No output may overlap an input or another output.
struct Range {
  const void *p;
  size_t bytes;
};
bool outputs_clear(const Range *outs, int n_out, const Range *ins, int n_in) {
  for (int o = 0; o < n_out; ++o) {
    for (int i = 0; i < n_in; ++i)
      if (overlaps(outs[o].p, outs[o].bytes, ins[i].p, ins[i].bytes)) return false;
    for (int o2 = o + 1; o2 < n_out; ++o2)
      if (overlaps(outs[o].p, outs[o].bytes, outs[o2].p, outs[o2].bytes)) return false;
  }
  return true;
}

// A tensor's rows, one per token, `stride` bytes apart (at least `bytes`). Two such tensors of T tokens
// may lie inside each other's range, like the parts of a fused projection: with one stride they share
// a byte only if some row of one meets a row of the other.
struct Rows {
  const void *p;
  int64_t bytes, stride;
};
bool rows_overlap(const Rows &x, const Rows &y, int64_t T) {
  if (!overlaps(x.p, size_t((T - 1) * x.stride + x.bytes), y.p, size_t((T - 1) * y.stride + y.bytes))) return false;
  if (x.stride != y.stride) return true;
  const int64_t between = reinterpret_cast<intptr_t>(y.p) - reinterpret_cast<intptr_t>(x.p);
  const int64_t off = ((between % x.stride) + x.stride) % x.stride;
  return !(off >= x.bytes && off + y.bytes <= x.stride);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" {

kda_status kda_prefill_recurrent(const void *q, const void *k, const void *v, const float *log_alpha,
                                 const float *beta, const int32_t *cu_seqlens, int32_t num_seqs,
                                 int64_t total_tokens, int32_t H, int32_t d_k, int32_t d_v, kda_dtype in_dtype,
                                 kda_dtype out_dtype, float lower_bound, float scale, const float *init_state,
                                 void *out, float *final_state, void *stream) {
  return prefill_impl(q, k, v, log_alpha, nullptr, beta, cu_seqlens, num_seqs, total_tokens, H, d_k, d_v, in_dtype,
                      out_dtype, lower_bound, scale, init_state, out, final_state, stream, true);
}

kda_status kda_prefill(const void *q, const void *k, const void *v, const float *log_alpha, const float *beta,
                       const int32_t *cu_seqlens, int32_t num_seqs, int64_t total_tokens, int32_t H, int32_t d_k,
                       int32_t d_v, kda_dtype in_dtype, kda_dtype out_dtype, float lower_bound, float scale,
                       const float *init_state, void *out, float *final_state, void *workspace,
                       size_t workspace_bytes, void *stream) {
  return prefill_impl(q, k, v, log_alpha, nullptr, beta, cu_seqlens, num_seqs, total_tokens, H, d_k, d_v, in_dtype,
                      out_dtype, lower_bound, scale, init_state, out, final_state, stream, false, nullptr, nullptr,
                      0.f, -1, workspace, workspace_bytes);
}

size_t kda_prefill_workspace_size(int64_t total_tokens, int32_t num_seqs, int32_t H, int32_t d_k, int32_t d_v) {
  return prefill_workspace_bytes(total_tokens, num_seqs, H, d_k, d_v);
}

// kda_prefill with its scratch in g_noalloc_scratch instead of a caller's workspace: the same
// validation, schedule and kernels, and no allocation of any kind. Sizes whose schedule needs more
// scratch than the array holds are refused before anything is enqueued.
kda_status kda_prefill_noalloc(const void *q, const void *k, const void *v, const float *log_alpha,
                               const float *beta, const int32_t *cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                               int32_t H, int32_t d_k, int32_t d_v, kda_dtype in_dtype, kda_dtype out_dtype,
                               float lower_bound, float scale, const float *init_state, void *out,
                               float *final_state, void *stream) {
  const kda_status st = check_prefill_args(q, k, v, log_alpha, nullptr, beta, cu_seqlens, num_seqs, total_tokens, H,
                                           d_k, d_v, in_dtype, out_dtype, init_state, out, final_state);
  if (st != KDA_OK) return st;
  if (prefill_workspace_bytes(total_tokens, num_seqs, H, d_k, d_v) > kNoAllocScratchBytes) return KDA_ERR_UNSUPPORTED;
  void *scratch = noalloc_scratch();
  if (scratch == nullptr) return KDA_ERR_CUDA;
  return prefill_impl(q, k, v, log_alpha, nullptr, beta, cu_seqlens, num_seqs, total_tokens, H, d_k, d_v, in_dtype,
                      out_dtype, lower_bound, scale, init_state, out, final_state, stream, false, nullptr, nullptr,
                      0.f, -1, scratch, kNoAllocScratchBytes);
}

kda_status kda_prefill_gated(const void *q, const void *k, const void *v, const void *z, const float *A_log,
                             const float *beta, const int32_t *cu_seqlens, int32_t num_seqs, int64_t total_tokens,
                             int32_t H, int32_t d_k, int32_t d_v, kda_dtype in_dtype, kda_dtype out_dtype,
                             float g_min, float scale, const float *init_state, void *out, float *final_state,
                             void *stream) {
  const kda_status st = check_gate_args(A_log, g_min);
  if (st != KDA_OK) return st;
  return prefill_impl(q, k, v, z, A_log, beta, cu_seqlens, num_seqs, total_tokens, H, d_k, d_v, in_dtype, out_dtype,
                      g_min, scale, init_state, out, final_state, stream, false);
}

kda_status kda_prefill_gated_recurrent(const void *q, const void *k, const void *v, const void *z,
                                       const float *A_log, const float *beta, const int32_t *cu_seqlens,
                                       int32_t num_seqs, int64_t total_tokens, int32_t H, int32_t d_k, int32_t d_v,
                                       kda_dtype in_dtype, kda_dtype out_dtype, float g_min, float scale,
                                       const float *init_state, void *out, float *final_state, void *stream) {
  const kda_status st = check_gate_args(A_log, g_min);
  if (st != KDA_OK) return st;
  return prefill_impl(q, k, v, z, A_log, beta, cu_seqlens, num_seqs, total_tokens, H, d_k, d_v, in_dtype, out_dtype,
                      g_min, scale, init_state, out, final_state, stream, true);
}

kda_status kda_decode(const void *q, const void *k, const void *v, const float *log_alpha, const float *beta,
                      float *state, void *out, int32_t B, int32_t H, int32_t d_k, int32_t d_v, kda_dtype in_dtype,
                      kda_dtype out_dtype, float lower_bound, float scale, void *stream) {
  return decode_impl(q, k, v, log_alpha, nullptr, beta, state, out, B, H, d_k, d_v, in_dtype, out_dtype,
                     lower_bound, scale, stream);
}

kda_status kda_decode_gated(const void *q, const void *k, const void *v, const void *z, const float *A_log,
                            const float *beta, float *state, void *out, int32_t B, int32_t H, int32_t d_k,
                            int32_t d_v, kda_dtype in_dtype, kda_dtype out_dtype, float g_min, float scale,
                            void *stream) {
  const kda_status st = check_gate_args(A_log, g_min);
  if (st != KDA_OK) return st;
  return decode_impl(q, k, v, z, A_log, beta, state, out, B, H, d_k, d_v, in_dtype, out_dtype, g_min, scale, stream);
}

kda_status kda_prefill_ex(const kda_prefill_params *p, void *stream) {
  if (p == nullptr || p->struct_size != sizeof(kda_prefill_params)) return KDA_ERR_INVALID_ARG;
  const kda_status st = check_decay_form(p->decay_form, p->A_log, p->decay_bound);
  if (st != KDA_OK) return st;
  return prefill_impl(p->q, p->k, p->v, p->decay, p->A_log, p->beta, p->cu_seqlens, p->num_seqs, p->total_tokens,
                      p->H, p->d_k, p->d_v, p->in_dtype, p->out_dtype, p->decay_bound, p->scale, p->init_state,
                      p->out, p->final_state, stream, p->force_recurrent != 0, p->out_gate, p->norm_weight,
                      p->norm_eps, int(p->decay_form), p->workspace, p->workspace_bytes);
}

kda_status kda_decode_ex(const kda_decode_params *p, void *stream) {
  if (p == nullptr || p->struct_size != sizeof(kda_decode_params)) return KDA_ERR_INVALID_ARG;
  const kda_status st = check_decay_form(p->decay_form, p->A_log, p->decay_bound);
  if (st != KDA_OK) return st;
  return decode_impl(p->q, p->k, p->v, p->decay, p->A_log, p->beta, p->state, p->out, p->B, p->H, p->d_k, p->d_v,
                     p->in_dtype, p->out_dtype, p->decay_bound, p->scale, stream, p->out_gate, p->norm_weight,
                     p->norm_eps, p->conv_weight, p->conv_state, p->l2_eps, int(p->decay_form));
}

kda_status kda_prologue(const void *q_raw, const void *k_raw, const void *v_raw, const float *conv_weight,
                        const int32_t *cu_seqlens, int32_t num_seqs, int64_t total_tokens, int32_t H, int32_t d_k,
                        int32_t d_v, kda_dtype dtype, const void *conv_init, float l2_eps, void *q, void *k, void *v,
                        void *conv_final, void *stream) {
  if (dtype != KDA_F32 && dtype != KDA_BF16) return KDA_ERR_INVALID_ARG;
  if (num_seqs < 0 || total_tokens < 0 || H < 1 || d_k < 1 || d_v < 1) return KDA_ERR_INVALID_ARG;
  if (d_k > 128 || d_v > 128) return KDA_ERR_UNSUPPORTED;
  if (total_tokens > INT32_MAX || H > 65535) return KDA_ERR_UNSUPPORTED;
  if (num_seqs == 0 && total_tokens > 0) return KDA_ERR_INVALID_ARG;
  if (!finite_nonneg(l2_eps)) return KDA_ERR_INVALID_ARG;
  if (cu_seqlens == nullptr || !aligned4(cu_seqlens)) return KDA_ERR_INVALID_ARG;
  if (conv_weight == nullptr || !aligned16(conv_weight)) return KDA_ERR_INVALID_ARG;
  if (total_tokens > 0) {
    if (!q_raw || !k_raw || !v_raw || !q || !k || !v) return KDA_ERR_INVALID_ARG;
    if (!aligned16(q_raw) || !aligned16(k_raw) || !aligned16(v_raw) || !aligned16(q) || !aligned16(k) ||
        !aligned16(v))
      return KDA_ERR_INVALID_ARG;
  }
  if ((conv_init && !aligned16(conv_init)) || (conv_final && !aligned16(conv_final))) return KDA_ERR_INVALID_ARG;
  const size_t es = dtype == KDA_BF16 ? 2 : 4;
  const size_t nk = size_t(total_tokens) * H * d_k * es, nv = size_t(total_tokens) * H * d_v * es;
  const size_t ns = size_t(num_seqs) * H * 3 * (2 * d_k + d_v) * es;
  const void *ins[6] = {q_raw, k_raw, v_raw, conv_weight, cu_seqlens, conv_init};
  const size_t in_bytes[6] = {nk, nk, nv, size_t(H) * (2 * d_k + d_v) * 16, size_t(num_seqs + 1) * 4, ns};
  const void *outs[4] = {q, k, v, conv_final};
  const size_t out_bytes[4] = {nk, nk, nv, conv_final ? ns : 0};
  for (int o = 0; o < 4; ++o) {
    for (int i = 0; i < 6; ++i)
      if (overlaps(outs[o], out_bytes[o], ins[i], in_bytes[i])) return KDA_ERR_INVALID_ARG;
    for (int o2 = o + 1; o2 < 4; ++o2)
      if (overlaps(outs[o], out_bytes[o], outs[o2], out_bytes[o2])) return KDA_ERR_INVALID_ARG;
  }
  if (num_seqs == 0) return KDA_OK;
  const cudaError_t err = launch_prologue(q_raw, k_raw, v_raw, conv_weight, cu_seqlens, num_seqs, total_tokens, H,
                                          d_k, d_v, dtype == KDA_BF16, conv_init, l2_eps, q, k, v, conv_final,
                                          static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_linear_prefill_workspace_size(int64_t total_tokens, int32_t num_seqs, int32_t H, int32_t H_k, int32_t d_k,
                                         int32_t d_v, kda_dtype in_dtype, kda_dtype out_dtype,
                                         int32_t force_recurrent) {
  if (check_linear_sizes(total_tokens, num_seqs, H, H_k, d_k, d_v, 1, in_dtype, out_dtype) != KDA_OK) return 0;
  if (total_tokens == 0 || num_seqs == 0) return 0;
  return linear_plan(total_tokens, num_seqs, H, H_k, d_k, d_v, in_dtype == KDA_BF16, out_dtype == KDA_BF16,
                     force_recurrent != 0, SIZE_MAX)
      .bytes;
}

kda_status kda_linear_prefill(const kda_linear_prefill_params *p, void *stream) {
  if (p == nullptr || p->struct_size != sizeof(kda_linear_prefill_params)) return KDA_ERR_INVALID_ARG;
  const kda_status st = check_linear_sizes(p->total_tokens, p->num_seqs, p->H, p->H_k, p->d_k, p->d_v,
                                           p->decay_per_token, p->in_dtype, p->out_dtype);
  if (st != KDA_OK) return st;
  const int64_t T = p->total_tokens;
  if (T > 0 && p->num_seqs == 0) return KDA_ERR_INVALID_ARG;
  if (p->cu_seqlens == nullptr || !aligned4(p->cu_seqlens)) return KDA_ERR_INVALID_ARG;
  if (T > 0) {
    if (!p->q || !p->k || !p->v || !p->log_decay || !p->out) return KDA_ERR_INVALID_ARG;
    if (!aligned16(p->q) || !aligned16(p->k) || !aligned16(p->v) || !aligned16(p->out) || !aligned4(p->log_decay))
      return KDA_ERR_INVALID_ARG;
  }
  if (!aligned16(p->init_state) || !aligned16(p->final_state)) return KDA_ERR_INVALID_ARG;
  if ((p->workspace == nullptr) != (p->workspace_bytes == 0) || !aligned16(p->workspace)) return KDA_ERR_INVALID_ARG;
  const size_t es = p->in_dtype == KDA_BF16 ? 2 : 4, eo = p->out_dtype == KDA_BF16 ? 2 : 4;
  const size_t nk = size_t(T) * p->H_k * p->d_k * es, nv = size_t(T) * p->H * p->d_v;
  const size_t ns = size_t(p->num_seqs) * p->H * p->d_k * p->d_v * 4;
  const bool in_place = p->final_state != nullptr && p->final_state == p->init_state;
  const Range ins[6] = {{p->q, nk}, {p->k, nk}, {p->v, nv * es},
                        {p->log_decay, size_t(p->decay_per_token ? T : 1) * p->H * 4},
                        {p->cu_seqlens, (size_t(p->num_seqs) + 1) * 4}, {in_place ? nullptr : p->init_state, ns}};
  const Range outs[3] = {{p->out, nv * eo}, {p->final_state, ns}, {p->workspace, p->workspace_bytes}};
  if (!outputs_clear(outs, 3, ins, 6)) return KDA_ERR_INVALID_ARG;
  if (p->num_seqs == 0) return KDA_OK;
  if (T == 0 && p->final_state == nullptr) return KDA_OK;

  LinearArgs a{};
  a.q = p->q, a.k = p->k, a.v = p->v, a.log_decay = p->log_decay, a.cu = p->cu_seqlens;
  a.init_state = p->init_state, a.out = p->out, a.final_state = p->final_state;
  a.num_seqs = p->num_seqs, a.H = p->H, a.H_k = p->H_k, a.d_k = p->d_k, a.d_v = p->d_v;
  a.per_token = p->decay_per_token, a.total = T, a.scale = p->scale;
  const bool in_bf16 = p->in_dtype == KDA_BF16, out_bf16 = p->out_dtype == KDA_BF16;
  a.plan = linear_plan(T, p->num_seqs, p->H, p->H_k, p->d_k, p->d_v, in_bf16, out_bf16, p->force_recurrent != 0,
                       p->workspace_bytes);
  a.workspace = static_cast<uint8_t *>(p->workspace);
  if (a.plan.seg_len != 0) {
    a.seg_states = reinterpret_cast<float *>(a.workspace + a.plan.states);
    a.seg_decay = reinterpret_cast<float *>(a.workspace + a.plan.decays);
  }
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const cudaError_t err = a.plan.tensor ? launch_linear_chunked(a, out_bf16, cs)
                                        : launch_linear_recurrent(a, in_bf16, out_bf16, cs);
  return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_linear_decode(const kda_linear_decode_params *p, void *stream) {
  if (p == nullptr || p->struct_size != sizeof(kda_linear_decode_params)) return KDA_ERR_INVALID_ARG;
  if (p->B < 1) return KDA_ERR_INVALID_ARG;
  const kda_status st =
      check_linear_sizes(p->B, p->B, p->H, p->H_k, p->d_k, p->d_v, p->decay_per_token, p->in_dtype, p->out_dtype);
  if (st != KDA_OK) return st;
  if (!p->q || !p->k || !p->v || !p->log_decay || !p->state || !p->out) return KDA_ERR_INVALID_ARG;
  if (!aligned16(p->q) || !aligned16(p->k) || !aligned16(p->v) || !aligned16(p->state) || !aligned16(p->out) ||
      !aligned4(p->log_decay))
    return KDA_ERR_INVALID_ARG;
  const size_t es = p->in_dtype == KDA_BF16 ? 2 : 4, eo = p->out_dtype == KDA_BF16 ? 2 : 4;
  const size_t nk = size_t(p->B) * p->H_k * p->d_k * es, nv = size_t(p->B) * p->H * p->d_v;
  const Range ins[4] = {{p->q, nk}, {p->k, nk}, {p->v, nv * es},
                        {p->log_decay, size_t(p->decay_per_token ? p->B : 1) * p->H * 4}};
  const Range outs[2] = {{p->out, nv * eo}, {p->state, nv * p->d_k * 4}};
  if (!outputs_clear(outs, 2, ins, 4)) return KDA_ERR_INVALID_ARG;
  const cudaError_t err = launch_linear_decode(p->q, p->k, p->v, p->log_decay, p->decay_per_token != 0, p->state,
                                               p->out, p->B, p->H, p->H_k, p->d_k, p->d_v, p->in_dtype == KDA_BF16,
                                               p->out_dtype == KDA_BF16, p->scale, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_block_norm(const kda_block_norm_params *p, void *stream) {
  if (p == nullptr || p->struct_size != sizeof(kda_block_norm_params)) return KDA_ERR_INVALID_ARG;
  if (!valid_dtype(p->x_dtype) || !valid_dtype(p->y_dtype) || !valid_dtype(p->out_dtype)) return KDA_ERR_INVALID_ARG;
  if (p->rows < 0 || p->D < 1) return KDA_ERR_INVALID_ARG;
  if (p->D > kBlockNormMaxD || p->rows > INT32_MAX) return KDA_ERR_UNSUPPORTED;
  if (p->gate_form != KDA_GATE_NONE && p->gate_form != KDA_GATE_CHANNEL && p->gate_form != KDA_GATE_ROW)
    return KDA_ERR_INVALID_ARG;
  if (p->post_norm != 0 && p->post_norm != 1) return KDA_ERR_INVALID_ARG;
  if (!finite_nonneg(p->pre_eps) || !finite_nonneg(p->post_eps)) return KDA_ERR_INVALID_ARG;
  if (p->rows > 0) {
    if (p->x == nullptr || (p->residual_out == nullptr && p->out == nullptr)) return KDA_ERR_INVALID_ARG;
    if ((p->gate_form != KDA_GATE_NONE) != (p->gate != nullptr)) return KDA_ERR_INVALID_ARG;
    if (p->y == nullptr && (p->gate || p->post_weight || p->channel_scale || p->post_norm)) return KDA_ERR_INVALID_ARG;
    if ((p->post_weight != nullptr && p->post_norm == 0) || (p->pre_weight != nullptr && p->out == nullptr))
      return KDA_ERR_INVALID_ARG;
  }
  const void *all[8] = {p->x, p->y, p->gate, p->post_weight, p->channel_scale, p->pre_weight, p->residual_out, p->out};
  for (const void *q : all)
    if (!aligned16(q)) return KDA_ERR_INVALID_ARG;
  const size_t ex = p->x_dtype == KDA_BF16 ? 2 : 4, ey = p->y_dtype == KDA_BF16 ? 2 : 4;
  const size_t n = size_t(p->rows) * p->D, w = size_t(p->D) * 4;
  const bool in_place = p->residual_out != nullptr && p->residual_out == p->x;
  const Range ins[6] = {{in_place ? nullptr : p->x, n * ex}, {p->y, n * ey},
                        {p->gate, (p->gate_form == KDA_GATE_ROW ? size_t(p->rows) : n) * ey},
                        {p->post_weight, w}, {p->channel_scale, w}, {p->pre_weight, w}};
  const Range outs[2] = {{p->residual_out, n * ex}, {p->out, n * (p->out_dtype == KDA_BF16 ? 2 : 4)}};
  if (!outputs_clear(outs, 2, ins, 6)) return KDA_ERR_INVALID_ARG;
  if (p->rows == 0) return KDA_OK;
  BlockNormArgs a{};
  a.x = p->x, a.y = p->y, a.gate = p->gate;
  a.post_weight = p->post_weight, a.channel_scale = p->channel_scale, a.pre_weight = p->pre_weight;
  a.residual_out = p->residual_out, a.out = p->out, a.rows = p->rows, a.D = p->D;
  a.gate_form = int(p->gate_form), a.post_norm = p->post_norm;
  a.scale = p->scale, a.post_eps = p->post_eps, a.pre_eps = p->pre_eps;
  const cudaError_t err = launch_block_norm(a, p->x_dtype == KDA_BF16, p->y_dtype == KDA_BF16,
                                            p->out_dtype == KDA_BF16, static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

size_t kda_delta_prefill_workspace_size(int64_t total_tokens, int32_t num_seqs, int32_t H, int32_t H_k, int32_t d_k,
                                        int32_t d_v, kda_dtype in_dtype, kda_dtype out_dtype,
                                        int32_t force_recurrent) {
  if (check_linear_sizes(total_tokens, num_seqs, H, H_k, d_k, d_v, 1, in_dtype, out_dtype) != KDA_OK) return 0;
  if (total_tokens == 0 || num_seqs == 0) return 0;
  return delta_plan(total_tokens, num_seqs, H, H_k, d_k, d_v, in_dtype == KDA_BF16, out_dtype == KDA_BF16,
                    force_recurrent != 0, SIZE_MAX)
      .bytes;
}

kda_status kda_delta_prefill(const kda_delta_prefill_params *p, void *stream) {
  if (p == nullptr || p->struct_size != sizeof(kda_delta_prefill_params)) return KDA_ERR_INVALID_ARG;
  const kda_status st = check_linear_sizes(p->total_tokens, p->num_seqs, p->H, p->H_k, p->d_k, p->d_v,
                                           p->decay_per_token, p->in_dtype, p->out_dtype);
  if (st != KDA_OK) return st;
  const int64_t T = p->total_tokens;
  if (T > 0 && p->num_seqs == 0) return KDA_ERR_INVALID_ARG;
  if (p->cu_seqlens == nullptr || !aligned4(p->cu_seqlens)) return KDA_ERR_INVALID_ARG;
  if (T > 0) {
    if (!p->q || !p->k || !p->v || !p->log_decay || !p->beta || !p->out) return KDA_ERR_INVALID_ARG;
    if (!aligned16(p->q) || !aligned16(p->k) || !aligned16(p->v) || !aligned16(p->out) || !aligned4(p->log_decay) ||
        !aligned4(p->beta))
      return KDA_ERR_INVALID_ARG;
  }
  if (!aligned16(p->init_state) || !aligned16(p->final_state)) return KDA_ERR_INVALID_ARG;
  if ((p->workspace == nullptr) != (p->workspace_bytes == 0) || !aligned16(p->workspace)) return KDA_ERR_INVALID_ARG;
  const size_t es = p->in_dtype == KDA_BF16 ? 2 : 4, eo = p->out_dtype == KDA_BF16 ? 2 : 4;
  const size_t nk = size_t(T) * p->H_k * p->d_k * es, nv = size_t(T) * p->H * p->d_v;
  const size_t ns = size_t(p->num_seqs) * p->H * p->d_k * p->d_v * 4;
  const bool in_place = p->final_state != nullptr && p->final_state == p->init_state;
  const Range ins[7] = {{p->q, nk}, {p->k, nk}, {p->v, nv * es},
                        {p->log_decay, size_t(p->decay_per_token ? T : 1) * p->H * 4}, {p->beta, size_t(T) * p->H * 4},
                        {p->cu_seqlens, (size_t(p->num_seqs) + 1) * 4}, {in_place ? nullptr : p->init_state, ns}};
  const Range outs[3] = {{p->out, nv * eo}, {p->final_state, ns}, {p->workspace, p->workspace_bytes}};
  if (!outputs_clear(outs, 3, ins, 7)) return KDA_ERR_INVALID_ARG;
  if (p->num_seqs == 0) return KDA_OK;
  if (T == 0 && p->final_state == nullptr) return KDA_OK;

  DeltaArgs a{};
  a.q = p->q, a.k = p->k, a.v = p->v, a.log_decay = p->log_decay, a.beta = p->beta, a.cu = p->cu_seqlens;
  a.init_state = p->init_state, a.out = p->out, a.final_state = p->final_state;
  a.num_seqs = p->num_seqs, a.H = p->H, a.H_k = p->H_k, a.d_k = p->d_k, a.d_v = p->d_v;
  a.per_token = p->decay_per_token, a.total = T, a.scale = p->scale;
  const bool in_bf16 = p->in_dtype == KDA_BF16, out_bf16 = p->out_dtype == KDA_BF16;
  a.plan = delta_plan(T, p->num_seqs, p->H, p->H_k, p->d_k, p->d_v, in_bf16, out_bf16, p->force_recurrent != 0,
                      p->workspace_bytes);
  a.workspace = static_cast<uint8_t *>(p->workspace);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  cudaError_t err = a.plan.few >= 0 ? launch_delta_short(a, in_bf16, out_bf16, cs) : cudaSuccess;
  if (err == cudaSuccess)
    err = a.plan.tensor ? launch_delta_chunked(a, out_bf16, cs) : launch_delta_recurrent(a, in_bf16, out_bf16, cs);
  return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_delta_decode(const kda_delta_decode_params *p, void *stream) {
  if (p == nullptr || p->struct_size != sizeof(kda_delta_decode_params)) return KDA_ERR_INVALID_ARG;
  if (p->B < 1) return KDA_ERR_INVALID_ARG;
  const kda_status st =
      check_linear_sizes(p->B, p->B, p->H, p->H_k, p->d_k, p->d_v, p->decay_per_token, p->in_dtype, p->out_dtype);
  if (st != KDA_OK) return st;
  if (!p->q || !p->k || !p->v || !p->log_decay || !p->beta || !p->state || !p->out) return KDA_ERR_INVALID_ARG;
  if (!aligned16(p->q) || !aligned16(p->k) || !aligned16(p->v) || !aligned16(p->state) || !aligned16(p->out) ||
      !aligned4(p->log_decay) || !aligned4(p->beta))
    return KDA_ERR_INVALID_ARG;
  const size_t es = p->in_dtype == KDA_BF16 ? 2 : 4, eo = p->out_dtype == KDA_BF16 ? 2 : 4;
  const size_t nk = size_t(p->B) * p->H_k * p->d_k * es, nv = size_t(p->B) * p->H * p->d_v;
  const Range ins[5] = {{p->q, nk}, {p->k, nk}, {p->v, nv * es},
                        {p->log_decay, size_t(p->decay_per_token ? p->B : 1) * p->H * 4},
                        {p->beta, size_t(p->B) * p->H * 4}};
  const Range outs[2] = {{p->out, nv * eo}, {p->state, nv * p->d_k * 4}};
  if (!outputs_clear(outs, 2, ins, 5)) return KDA_ERR_INVALID_ARG;
  const cudaError_t err =
      launch_delta_decode(p->q, p->k, p->v, p->log_decay, p->decay_per_token != 0, p->beta, p->state, p->out, p->B,
                          p->H, p->H_k, p->d_k, p->d_v, p->in_dtype == KDA_BF16, p->out_dtype == KDA_BF16, p->scale,
                          static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_norm_rotate(const kda_norm_rotate_params *p, void *stream) {
  if (p == nullptr || p->struct_size != sizeof(kda_norm_rotate_params)) return KDA_ERR_INVALID_ARG;
  if (!valid_dtype(p->in_dtype) || !valid_dtype(p->out_dtype)) return KDA_ERR_INVALID_ARG;
  if (p->norm != KDA_NORM_NONE && p->norm != KDA_NORM_RMS && p->norm != KDA_NORM_L2) return KDA_ERR_INVALID_ARG;
  if (p->tokens < 0 || p->H_q < 1 || p->H_k < 0 || p->d < 1) return KDA_ERR_INVALID_ARG;
  if (p->rot_dim < 0 || p->rot_dim > p->d || p->rot_dim % 2 != 0) return KDA_ERR_INVALID_ARG;
  if ((p->interleaved != 0 && p->interleaved != 1) || !finite_nonneg(p->eps)) return KDA_ERR_INVALID_ARG;
  if (p->d > kRotateMaxD || p->num_axes > kRotateMaxAxes || p->tokens > INT32_MAX || p->H_q > 65535 || p->H_k > 65535)
    return KDA_ERR_UNSUPPORTED;
  const int half = p->rot_dim / 2;
  if (half > 0) {
    if (p->num_axes < 1 || (p->position_bytes != 4 && p->position_bytes != 8)) return KDA_ERR_INVALID_ARG;
    for (int i = 0; i < half; ++i)
      if (p->pair_axis[i] >= p->num_axes) return KDA_ERR_INVALID_ARG;
  }
  if (p->norm != KDA_NORM_RMS && (p->q_weight != nullptr || p->k_weight != nullptr)) return KDA_ERR_INVALID_ARG;
  if ((p->H_k == 0) != (p->k == nullptr && p->k_out == nullptr)) return KDA_ERR_INVALID_ARG;
  const int64_t wq = int64_t(p->H_q) * p->d, wk = int64_t(p->H_k) * p->d;
  if (p->q_stride < wq || p->q_out_stride < wq || p->k_stride < wk || p->k_out_stride < wk) return KDA_ERR_INVALID_ARG;
  const int64_t most = INT64_MAX / 16 / (p->tokens > 0 ? p->tokens : 1);  // bytes of a tensor
  if (p->q_stride > most || p->q_out_stride > most || p->k_stride > most || p->k_out_stride > most)
    return KDA_ERR_UNSUPPORTED;
  if (p->tokens == 0) return KDA_OK;
  const int64_t ei = p->in_dtype == KDA_BF16 ? 2 : 4, eo = p->out_dtype == KDA_BF16 ? 2 : 4;
  const auto aligned = [](const void *x, int64_t bytes) { return reinterpret_cast<uintptr_t>(x) % uintptr_t(bytes) == 0; };
  if (p->q == nullptr || p->q_out == nullptr || (p->H_k > 0 && (p->k == nullptr || p->k_out == nullptr)))
    return KDA_ERR_INVALID_ARG;
  if (half > 0 && (p->positions == nullptr || p->inv_freq == nullptr || !aligned(p->positions, p->position_bytes)))
    return KDA_ERR_INVALID_ARG;
  if (!aligned(p->q, ei) || !aligned(p->k, ei) || !aligned(p->q_out, eo) || !aligned(p->k_out, eo) ||
      !aligned4(p->q_weight) || !aligned4(p->k_weight) || !aligned4(p->inv_freq))
    return KDA_ERR_INVALID_ARG;
  // rows of a token, in bytes: outputs share none with inputs (their own in place excepted) or each other
  const Rows q{p->q, wq * ei, p->q_stride * ei}, k{p->k, wk * ei, p->k_stride * ei};
  const Rows qo{p->q_out, wq * eo, p->q_out_stride * eo}, ko{p->k_out, wk * eo, p->k_out_stride * eo};
  const auto same = [&](const Rows &x, const Rows &y) { return x.p == y.p && x.stride == y.stride && ei == eo; };
  const int64_t T = p->tokens;
  if (!same(q, qo) && rows_overlap(q, qo, T)) return KDA_ERR_INVALID_ARG;
  if (p->H_k > 0) {
    if (!same(k, ko) && rows_overlap(k, ko, T)) return KDA_ERR_INVALID_ARG;
    if (rows_overlap(q, ko, T) || rows_overlap(k, qo, T) || rows_overlap(qo, ko, T)) return KDA_ERR_INVALID_ARG;
  }
  const Range small[4] = {{p->q_weight, size_t(p->d) * 4}, {p->k_weight, size_t(p->d) * 4},
                          {half > 0 ? p->positions : nullptr, size_t(p->num_axes) * T * p->position_bytes},
                          {half > 0 ? p->inv_freq : nullptr, size_t(half) * 4}};
  const Range outs[2] = {{p->q_out, size_t((T - 1) * qo.stride + qo.bytes)},
                         {p->k_out, size_t(p->H_k > 0 ? (T - 1) * ko.stride + ko.bytes : 0)}};
  for (const Range &o : outs)
    for (const Range &i : small)
      if (overlaps(o.p, o.bytes, i.p, i.bytes)) return KDA_ERR_INVALID_ARG;
  RotateArgs a{};
  a.x[0] = p->q, a.x[1] = p->k, a.out[0] = p->q_out, a.out[1] = p->k_out;
  a.weight[0] = p->q_weight, a.weight[1] = p->k_weight;
  a.stride[0] = p->q_stride, a.stride[1] = p->k_stride, a.out_stride[0] = p->q_out_stride, a.out_stride[1] = p->k_out_stride;
  a.heads[0] = p->H_q, a.heads[1] = p->H_k;
  a.positions = p->positions, a.inv_freq = p->inv_freq, a.tokens = T;
  a.d = p->d, a.half = half, a.norm = int(p->norm), a.pos64 = p->position_bytes == 8, a.eps = p->eps;
  a.per = p->norm == KDA_NORM_RMS ? 1.f / float(p->d) : 1.f;
  for (int i = 0; i < half; ++i) a.axis[i] = p->pair_axis[i];
  const cudaError_t err = launch_norm_rotate(a, p->in_dtype == KDA_BF16, p->out_dtype == KDA_BF16, p->interleaved != 0,
                                             static_cast<cudaStream_t>(stream));
  return err == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

kda_status kda_check_device_error(void *stream) {
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  std::lock_guard<std::mutex> lock(g_check_mu);
  take_device_error_kernel<<<1, 1, 0, s>>>();
  if (cudaGetLastError() != cudaSuccess) return KDA_ERR_CUDA;
  uint32_t word = 0;
  if (cudaMemcpyFromSymbolAsync(&word, g_device_error_taken, sizeof word, 0, cudaMemcpyDeviceToHost, s) !=
          cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return KDA_ERR_CUDA;
  if (word & (DEVERR_TMA_TIMEOUT | DEVERR_MMA_TIMEOUT)) return KDA_ERR_TIMEOUT;
  if (word & DEVERR_RANGE) return KDA_ERR_RANGE;
  return KDA_OK;
}

const char *kda_status_string(kda_status status) {
  switch (status) {
    case KDA_OK: return "KDA_OK";
    case KDA_ERR_INVALID_ARG: return "KDA_ERR_INVALID_ARG";
    case KDA_ERR_UNSUPPORTED: return "KDA_ERR_UNSUPPORTED";
    case KDA_ERR_CUDA: return "KDA_ERR_CUDA";
    case KDA_ERR_TIMEOUT: return "KDA_ERR_TIMEOUT";
    case KDA_ERR_RANGE: return "KDA_ERR_RANGE";
  }
  return "KDA_ERR_UNKNOWN";
}

int32_t kda_version(void) { return 100; }

}  // extern "C"
