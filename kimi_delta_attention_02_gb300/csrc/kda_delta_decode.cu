// kda_delta_decode.cu -- one token of the gated delta rule with one decay per head, states updated in
// place: S' = e^g S, u = beta (v - S'^T k), S <- S' + k u^T, o = scale (S'^T q + (k . q) u), for B
// sequences and H heads.
//
// One read and one write of the d_k x d_v fp32 state per (sequence, head) against 1.2 flops per byte:
// bound by HBM bandwidth (256 sequences, 96 heads of 128: 3.25 GB in 470 to 484 us, the copy rate), and by
// latency when few states are in flight (one sequence: 6 us, 2 at the copy rate). A new entry needs its whole old
// column (S'^T k), so a CTA holds all key rows of its value columns, 32 entries per thread: kRows rows of
// kVec neighbouring columns, every load issued before the first is used. Where rows of the state start on
// 16-byte boundaries the entries come to shared memory by cp.async (each thread reads back only what it
// copied), so that they take no registers and six CTAs of 32 KB share an SM (603 us with the entries in
// registers and two CTAs); single columns are held in registers. The two row sums meet once, by shuffles and through shared memory, and every thread forms its
// own columns' u.
#include "kda_delta.cuh"

namespace kda {
namespace {

// kTX threads side by side along the value columns, kVec columns each; kThr / kTX key rows at a time.
template <bool kInBF16, bool kOutBF16, int kVec, int kTX, int kThr>
__global__ void __launch_bounds__(kThr, kVec == 4 ? 1536 / kThr : 512 / kThr)
    delta_decode_kernel(const void *__restrict__ q, const void *__restrict__ k, const void *__restrict__ v,
                        const float *__restrict__ log_decay, int per_token, const float *__restrict__ beta,
                        float *__restrict__ state, void *__restrict__ out, int H, int H_k, int d_k, int d_v,
                        int tiles, float scale) {
  constexpr int kRows = 32 / kVec;  // rows per thread
  constexpr int kRG = kThr / kTX;   // row groups
  constexpr int kWarps = kThr / 32;
  constexpr int kGroup = kTX < 32 ? kTX : 32;       // neighbouring threads of one row group in a warp
  constexpr int kParts = kTX < 32 ? kWarps : kRG;   // partial sums that meet in shared memory
  constexpr int kCols = kTX * kVec;
  __shared__ float s_k[kRG * kRows], s_q[kRG * kRows];
  __shared__ __align__(16) float s_y[kParts][kCols], s_z[kParts][kCols];
  __shared__ float s_kq[kParts];
  const int tid = threadIdx.x, tx = tid % kTX, ty = tid / kTX;
  const int tile = blockIdx.x % tiles;
  const int64_t bh = blockIdx.x / tiles;
  const int h = int(bh % H);
  const int64_t bk = bh / H * H_k + h / (H / H_k);
  const int c = tx * kVec, col = tile * kCols + c;  // this thread's columns: col .. col + kVec - 1
  const bool ok = col < d_v;                        // kVec divides d_v
  float *S = state + bh * int64_t(d_k) * d_v + col;

  __shared__ __align__(16) float s_st[kVec == 4 ? kRG * kRows * kCols : 4];
  float st[kVec == 4 ? 1 : kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int r = ty + kRG * j;
    const bool on = ok && r < d_k;
    if constexpr (kVec == 4) cp_async_16_zfill(&s_st[(kThr * j + tid) * 4], on ? S + int64_t(r) * d_v : state, on);
    else st[j] = on ? __ldcs(S + int64_t(r) * d_v) : 0.f;
  }
  // the decayed entries of row j
  auto get = [&](int j, Decay decay, float (&x)[kVec]) {
    if constexpr (kVec == 4) {
      const float4 v = *reinterpret_cast<const float4 *>(&s_st[(kThr * j + tid) * 4]);
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
      x[0] = st[j];
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) x[e] = decay_step(x[e], decay);
  };
  const Decay decay = decay_of(log_decay[per_token ? bh : h]);
  const float b = beta[bh];
  float vv[kVec];
#pragma unroll
  for (int e = 0; e < kVec; ++e) vv[e] = ok ? load_elem<kInBF16>(v, bh * d_v + col + e) : 0.f;
#pragma unroll
  for (int i = tid; i < kRG * kRows; i += kThr) {
    s_k[i] = i < d_k ? load_elem<kInBF16>(k, bk * d_k + i) : 0.f;
    s_q[i] = i < d_k ? load_elem<kInBF16>(q, bk * d_k + i) : 0.f;
  }
  __syncthreads();

  float y[kVec] = {}, z[kVec] = {}, kq = 0.f;
  if constexpr (kVec == 4) cp_async_wait_all();
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const float kr = s_k[ty + kRG * j], qr = s_q[ty + kRG * j];
    kq = fmaf(kr, qr, kq);
    float x[kVec];
    get(j, decay, x);
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      y[e] = fmaf(kr, x[e], y[e]);
      z[e] = fmaf(qr, x[e], z[e]);
    }
  }
#pragma unroll
  for (int off = 16; off >= kTX; off >>= 1) {  // the row groups of a warp; none from 32 threads on
    kq += __shfl_xor_sync(0xffffffffu, kq, off);
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      y[e] += __shfl_xor_sync(0xffffffffu, y[e], off);
      z[e] += __shfl_xor_sync(0xffffffffu, z[e], off);
    }
  }
  const int part = kTX < 32 ? tid >> 5 : ty;
  if ((tid & 31) < kGroup) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) s_y[part][c + e] = y[e], s_z[part][c + e] = z[e];
    if (tx == 0) s_kq[part] = kq;
  }
  __syncthreads();
  float u[kVec];
#pragma unroll
  for (int e = 0; e < kVec; ++e) {
    float sum = 0.f;
#pragma unroll
    for (int p = 0; p < kParts; ++p) sum += s_y[p][c + e];
    u[e] = b * (vv[e] - sum);
  }
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int r = ty + kRG * j;
    const float kr = s_k[r];
    float x[kVec];
    get(j, decay, x);
#pragma unroll
    for (int e = 0; e < kVec; ++e) x[e] = fmaf(kr, u[e], x[e]);
    if (ok && r < d_k) {
      if constexpr (kVec == 4) __stcs(reinterpret_cast<float4 *>(S + int64_t(r) * d_v), make_float4(x[0], x[1], x[2], x[3]));
      else __stcs(S + int64_t(r) * d_v, x[0]);
    }
  }
  if (ty == 0 && ok) {
    kq = 0.f;
#pragma unroll
    for (int p = 0; p < kParts; ++p) kq += s_kq[p];
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      float sum = 0.f;
#pragma unroll
      for (int p = 0; p < kParts; ++p) sum += s_z[p][c + e];
      store_elem<kOutBF16>(out, bh * d_v + col + e, scale * fmaf(kq, u[e], sum));
    }
  }
}

}  // namespace

cudaError_t launch_delta_decode(const void *q, const void *k, const void *v, const float *log_decay, bool per_token,
                                const float *beta, float *state, void *out, int B, int H, int H_k, int d_k, int d_v,
                                bool in_bf16, bool out_bf16, float scale, cudaStream_t stream) {
  // Four columns per thread where rows of the state start on 16-byte boundaries, tiles as narrow as the
  // columns need and the fewest threads that hold all key rows: 32, 64 or 128. Narrower tiles while there are
  // fewer than two for each SM (us at 16 / 32 / 64 columns: 96 pairs of 128 8.3 / 6.2 / 7.7, 384 pairs
  // 14.4 / 12.3 / 12.3, 24576 pairs 545 / 511 / 470).
  const bool vec = d_v % 4 == 0;
  const int64_t pairs = int64_t(B) * H;
  int size = d_v <= 16 ? 0 : d_v <= 32 ? 1 : 2;  // 16, 32 or 64 columns per CTA
  const auto tiles_of = [&](int x) { return (d_v + (16 << x) - 1) / (16 << x); };
  while (size > 0 && pairs * tiles_of(size) < 2 * kLinearSMs) --size;
  const int tiles = tiles_of(size), rows = d_k <= 32 ? 0 : d_k <= 64 ? 1 : 2;
  using Kern = void (*)(const void *, const void *, const void *, const float *, int, const float *, float *, void *,
                        int, int, int, int, int, float);
#define KDA_DDEC(v_, tx, t) \
  { delta_decode_kernel<false, false, v_, tx, t>, delta_decode_kernel<false, true, v_, tx, t>, \
    delta_decode_kernel<true, false, v_, tx, t>, delta_decode_kernel<true, true, v_, tx, t> }
  // threads: kTX x (key rows / rows per thread)
  static const Kern one[3][3][4] = {{KDA_DDEC(1, 16, 32), KDA_DDEC(1, 16, 32), KDA_DDEC(1, 16, 64)},
                                    {KDA_DDEC(1, 32, 32), KDA_DDEC(1, 32, 64), KDA_DDEC(1, 32, 128)},
                                    {KDA_DDEC(1, 64, 64), KDA_DDEC(1, 64, 128), KDA_DDEC(1, 64, 256)}};
  static const Kern four[3][3][4] = {{KDA_DDEC(4, 4, 32), KDA_DDEC(4, 4, 32), KDA_DDEC(4, 4, 64)},
                                     {KDA_DDEC(4, 8, 32), KDA_DDEC(4, 8, 64), KDA_DDEC(4, 8, 128)},
                                     {KDA_DDEC(4, 16, 64), KDA_DDEC(4, 16, 128), KDA_DDEC(4, 16, 256)}};
  static const int threads[3][3] = {{32, 32, 64}, {32, 64, 128}, {64, 128, 256}};
#undef KDA_DDEC
  (vec ? four : one)[size][rows][2 * int(in_bf16) + int(out_bf16)]<<<unsigned(pairs * tiles), threads[size][rows], 0,
                                                                     stream>>>(
      q, k, v, log_decay, int(per_token), beta, state, out, H, H_k, d_k, d_v, tiles, scale);
  return cudaGetLastError();
}

}  // namespace kda
