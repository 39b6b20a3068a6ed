// kda_linear_decode.cu -- one token of linear attention with one decay per head, states updated in
// place: S <- e^g S + k v^T, o = scale S^T q, for B sequences and H heads.
//
// One read and one write of the d_k x d_v fp32 state per (sequence, head) against about one flop
// per byte: bound by HBM bandwidth, and by latency when few states are in flight. No entry of the
// new state needs another entry of the old one, so the state streams through registers: each
// thread owns kVec neighbouring value columns of one key row in kThr / kTX, loads 8 rows' pieces (16
// of single columns) before it uses the first, and only the read-out is summed over the CTA.
//
// 256 sequences, 96 heads of 128 x 128: 464 us, 6.94 TB/s of states. One sequence: 8.7 us.
#include "kda_linear.cuh"

namespace kda {
namespace {


// kTX threads side by side along the value columns, kVec columns each; kThr / kTX key rows at a time.
template <bool kInBF16, bool kOutBF16, int kVec, int kTX, int kThr>
__global__ void __launch_bounds__(kThr)
    linear_decode_kernel(const void *__restrict__ q, const void *__restrict__ k, const void *__restrict__ v,
                         const float *__restrict__ log_decay, int per_token, float *__restrict__ state,
                         void *__restrict__ out, int H, int H_k, int d_k, int d_v, int tiles, float scale) {
  constexpr int kBatch = kVec == 4 ? 8 : 16;  // rows in flight per thread
  constexpr int kRG = kThr / kTX;             // row groups
  constexpr int kSide = kTX > 32 ? kTX : 32;  // threads that store their sums side by side
  constexpr int kCols = kTX * kVec;
  __shared__ float s_k[128], s_q[128];
  __shared__ float s_o[kThr / kSide][kCols];
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
  const Decay decay = decay_of(log_decay[per_token ? bh : h]);
  float vv[kVec];
#pragma unroll
  for (int e = 0; e < kVec; ++e) vv[e] = ok ? load_elem<kInBF16>(v, bh * d_v + col + e) : 0.f;
#pragma unroll
  for (int i = tid; i < 256; i += kThr) {
    const int r = i & 127;
    if (r < d_k) (i < 128 ? s_k : s_q)[r] = load_elem<kInBF16>(i < 128 ? k : q, bk * d_k + r);
  }
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
          st[j][e] = fmaf(kr, vv[e], decay_step(st[j][e], decay));
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
  for (int off = 16; off >= kTX; off >>= 1)  // none from 32 threads on
#pragma unroll
    for (int e = 0; e < kVec; ++e) o[e] += __shfl_xor_sync(0xffffffffu, o[e], off);
  if (tid % kSide < kTX) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) s_o[tid / kSide][c + e] = o[e];
  }
  __syncthreads();
#pragma unroll
  for (int i = tid; i < kCols; i += kThr) {
    if (tile * kCols + i >= d_v) break;
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < kThr / kSide; ++w) x += s_o[w][i];
    store_elem<kOutBF16>(out, bh * d_v + tile * kCols + i, scale * x);
  }
}

}  // namespace

cudaError_t launch_linear_decode(const void *q, const void *k, const void *v, const float *log_decay, bool per_token,
                                 float *state, void *out, int B, int H, int H_k, int d_k, int d_v, bool in_bf16,
                                 bool out_bf16, float scale, cudaStream_t stream) {
  // Four columns per thread where rows of the state start on 16-byte boundaries, and as few threads
  // side by side as cover the columns: 8192 states of 128 x 64 take 84 us with 16 threads, 95 with 32,
  // of 53 x 53 (single columns) 46 us in one tile, 56 in two. While that makes fewer CTAs than there are
  // SMs, half as many: 96 states of 128 x 128 take 8.7 us in tiles of 64 columns, 10.8 in whole rows.
  const bool vec = d_v % 4 == 0;
  const int64_t pairs = int64_t(B) * H;
  int size = d_v <= 32 ? 0 : d_v <= 64 ? 1 : 2;  // 32, 64 or 128 columns per CTA
  const auto tiles_of = [&](int x) { return (d_v + (32 << x) - 1) / (32 << x); };
  while (size > 0 && pairs * tiles_of(size) < kLinearSMs) --size;
  const int tiles = tiles_of(size);
  // Small states take smaller CTAs, whose threads each have several rows to load at once: 16384 states of
  // 16 x 16 take 21 us with 64 threads, 31 with 128, 62 with 256; 8192 of 64 x 64 take 48, 46 and 54
  // us, 8192 of 128 x 64 91, 87 and 85.
  const int entries = d_k * d_v;
  const int least = !vec && size == 2 ? 1 : 0;  // 128 threads side by side
  const int threads = entries > 4096 ? 2 : entries > 2048 ? 1 : least;  // 64, 128 or 256
  using Kern = void (*)(const void *, const void *, const void *, const float *, int, float *, void *, int, int, int,
                        int, int, float);
#define KDA_LDEC(v_, tx, t) \
  { linear_decode_kernel<false, false, v_, tx, t>, linear_decode_kernel<false, true, v_, tx, t>, \
    linear_decode_kernel<true, false, v_, tx, t>, linear_decode_kernel<true, true, v_, tx, t> }
  static const Kern one[3][3][4] = {{KDA_LDEC(1, 32, 64), KDA_LDEC(1, 32, 128), KDA_LDEC(1, 32, 256)},
                                    {KDA_LDEC(1, 64, 64), KDA_LDEC(1, 64, 128), KDA_LDEC(1, 64, 256)},
                                    {{}, KDA_LDEC(1, 128, 128), KDA_LDEC(1, 128, 256)}};
  static const Kern four[3][3][4] = {{KDA_LDEC(4, 8, 64), KDA_LDEC(4, 8, 128), KDA_LDEC(4, 8, 256)},
                                     {KDA_LDEC(4, 16, 64), KDA_LDEC(4, 16, 128), KDA_LDEC(4, 16, 256)},
                                     {KDA_LDEC(4, 32, 64), KDA_LDEC(4, 32, 128), KDA_LDEC(4, 32, 256)}};
#undef KDA_LDEC
  (vec ? four : one)[size][threads][2 * int(in_bf16) + int(out_bf16)]<<<unsigned(pairs * tiles), 64 << threads, 0,
                                                                        stream>>>(
      q, k, v, log_decay, int(per_token), state, out, H, H_k, d_k, d_v, tiles, scale);
  return cudaGetLastError();
}

}  // namespace kda
