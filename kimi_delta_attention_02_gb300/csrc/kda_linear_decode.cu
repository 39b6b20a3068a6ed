// kda_linear_decode.cu -- one token of linear attention with one decay per head, states updated in
// place: S <- e^g S + k v^T, o = scale S^T q, for B sequences and H heads.
//
// One read and one write of the d_k x d_v fp32 state per (sequence, head) against about one flop
// per byte: bound by HBM bandwidth, and by latency when few states are in flight. No entry of the
// new state needs another entry of the old one, so the state streams through registers: each
// thread owns kVec neighbouring value columns of one key row in 256 / kTX, loads eight rows'
// pieces before it uses the first, and only the read-out is summed over the CTA.
#include "kda_linear.cuh"

namespace kda {
namespace {

constexpr int kThr = 256;
constexpr int kBatch = 8;  // rows in flight per thread

// kTX threads side by side along the value columns, kVec columns each; 256 / kTX key rows at a time.
template <bool kInBF16, bool kOutBF16, int kVec, int kTX>
__global__ void __launch_bounds__(kThr)
    linear_decode_kernel(const void *__restrict__ q, const void *__restrict__ k, const void *__restrict__ v,
                         const float *__restrict__ log_decay, int per_token, float *__restrict__ state,
                         void *__restrict__ out, int H, int H_k, int d_k, int d_v, int tiles, float scale) {
  constexpr int kRG = kThr / kTX;  // row groups
  constexpr int kCols = kTX * kVec;
  __shared__ float s_k[128], s_q[128];
  __shared__ float s_o[kThr / 32][kCols];
  const int tid = threadIdx.x, tx = tid % kTX, ty = tid / kTX;
  const int tile = blockIdx.x % tiles;
  const int64_t bh = blockIdx.x / tiles;
  const int h = int(bh % H);
  const int64_t bk = bh / H * H_k + h / (H / H_k);
  const int c = tx * kVec, col = tile * kCols + c;  // this thread's columns: col .. col + kVec - 1
  const bool ok = col < d_v;                        // kVec divides d_v
  float *S = state + bh * int64_t(d_k) * d_v + col;

  float st[kBatch][kVec];
  auto load = [&](int r0) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int r = r0 + ty + kRG * j;
      if (ok && r < d_k) {
        if constexpr (kVec == 4) {
          const float4 x = __ldcs(reinterpret_cast<const float4 *>(S + int64_t(r) * d_v));
          st[j][0] = x.x, st[j][1] = x.y, st[j][2] = x.z, st[j][3] = x.w;
        } else {
          st[j][0] = __ldcs(S + int64_t(r) * d_v);
        }
      } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) st[j][e] = 0.f;
      }
    }
  };
  load(0);
  const float em1 = expm1f(log_decay[per_token ? bh : h]);
  float vv[kVec];
#pragma unroll
  for (int e = 0; e < kVec; ++e) vv[e] = ok ? load_elem<kInBF16>(v, bh * d_v + col + e) : 0.f;
  if (tid < 128) s_k[tid] = tid < d_k ? load_elem<kInBF16>(k, bk * d_k + tid) : 0.f;
  else s_q[tid - 128] = tid - 128 < d_k ? load_elem<kInBF16>(q, bk * d_k + tid - 128) : 0.f;
  __syncthreads();

  float o[kVec] = {};
  for (int r0 = 0; r0 < d_k; r0 += kRG * kBatch) {
    if (r0 != 0) load(r0);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int r = r0 + ty + kRG * j;
      if (r < d_k) {
        const float kr = s_k[r], qr = s_q[r];
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          st[j][e] = fmaf(kr, vv[e], decay_step(st[j][e], em1));
          o[e] = fmaf(qr, st[j][e], o[e]);
        }
        if (ok) {
          if constexpr (kVec == 4)
            __stcs(reinterpret_cast<float4 *>(S + int64_t(r) * d_v), make_float4(st[j][0], st[j][1], st[j][2], st[j][3]));
          else __stcs(S + int64_t(r) * d_v, st[j][0]);
        }
      }
    }
  }
  // the read-out: row groups of a warp by shuffles, then the warps
#pragma unroll
  for (int off = 16; off >= kTX; off >>= 1)
#pragma unroll
    for (int e = 0; e < kVec; ++e) o[e] += __shfl_xor_sync(0xffffffffu, o[e], off);
  if ((tid & 31) < kTX) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) s_o[tid >> 5][c + e] = o[e];
  }
  __syncthreads();
  if (tid < kCols && tile * kCols + tid < d_v) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < kThr / 32; ++w) x += s_o[w][tid];
    store_elem<kOutBF16>(out, bh * d_v + tile * kCols + tid, scale * x);
  }
}

}  // namespace

cudaError_t launch_linear_decode(const void *q, const void *k, const void *v, const float *log_decay, bool per_token,
                                 float *state, void *out, int B, int H, int H_k, int d_k, int d_v, bool in_bf16,
                                 bool out_bf16, float scale, cudaStream_t stream) {
  // four columns per thread where rows of the state start on 16-byte boundaries
  const bool vec = d_v % 4 == 0;
  const int64_t pairs = int64_t(B) * H;
  const int cols = vec ? 128 : 32;
  const int tiles = (d_v + cols - 1) / cols;
  using Kern = void (*)(const void *, const void *, const void *, const float *, int, float *, void *, int, int, int,
                        int, int, float);
#define KDA_LDEC(v_, tx) \
  { linear_decode_kernel<false, false, v_, tx>, linear_decode_kernel<false, true, v_, tx>, \
    linear_decode_kernel<true, false, v_, tx>, linear_decode_kernel<true, true, v_, tx> }
  static const Kern table[2][4] = {KDA_LDEC(4, 32), KDA_LDEC(1, 32)};
#undef KDA_LDEC
  table[vec ? 0 : 1][2 * int(in_bf16) + int(out_bf16)]<<<unsigned(pairs * tiles), kThr, 0, stream>>>(
      q, k, v, log_decay, int(per_token), state, out, H, H_k, d_k, d_v, tiles, scale);
  return cudaGetLastError();
}

}  // namespace kda
