// kda_delta_decode.cu -- one token of the gated delta rule with one decay per head, states updated in
// place: S' = e^g S, u = beta (v - S'^T k), S <- S' + k u^T, o = scale (S'^T q + (k . q) u), for B
// sequences and H heads; and prompts of a few tokens, one token after the other on the state in shared memory.
//
// One read and one write of the d_k x d_v fp32 state per (sequence, head) against 1.2 flops per byte:
// bound by HBM bandwidth (256 sequences, 96 heads of 128: 3.25 GB in 465 to 484 us, the copy rate), and by
// latency when few states are in flight (one sequence: 6 us, 2 at the copy rate). A new entry needs its whole
// old column (S'^T k), so a CTA holds all key rows of its value columns, 32 entries per thread: kRows rows of
// kVec neighbouring columns, every load issued before the first is used. Where rows of the state start on
// 16-byte boundaries the entries come to shared memory by cp.async (each thread reads back only what it
// copied), so that they take no registers and six CTAs of 32 KB share an SM (603 us with the entries in
// registers and two CTAs); single columns are held in registers. The two row sums meet once, by shuffles and
// through shared memory, and every thread forms its own columns' u.
#include "kda_delta.cuh"

namespace kda {
namespace {

struct TokenArgs {
  const void *q, *k, *v;
  const float *log_decay, *beta, *from;  // from: the entering states, or null
  float *to;                             // or null
  void *out;
  const int32_t *cu;  // kMany: the sequences' tokens
  int per_token, H, H_k, d_k, d_v, tiles, most;
  float scale;
};

// kTX threads side by side along the value columns, kVec columns each; kThr / kTX key rows at a time. kMany: the
// sequences of up to `most` tokens, one after the other; else one token each.
template <bool kInBF16, bool kOutBF16, int kVec, int kTX, int kThr, bool kMany>
__global__ void __launch_bounds__(kThr, kVec == 4 ? 1536 / kThr : 512 / kThr) delta_decode_kernel(const TokenArgs a) {
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
  const int d_k = a.d_k, d_v = a.d_v;
  const int tile = blockIdx.x % a.tiles;
  const int64_t bh = blockIdx.x / a.tiles, n = bh / a.H;
  const int h = int(bh % a.H), hk = h / (a.H / a.H_k);
  const int64_t t0 = kMany ? a.cu[n] : n, t1 = kMany ? a.cu[n + 1] : n + 1;
  if (kMany && t1 - t0 > a.most) return;
  const int c = tx * kVec, col = tile * kCols + c;  // this thread's columns: col .. col + kVec - 1
  const bool ok = col < d_v;                        // kVec divides d_v
  const int64_t at = bh * int64_t(d_k) * d_v + col;
  float *const to = a.to;
  const void *const nothing = to != nullptr ? to : a.out;  // an address for copies of no bytes

  __shared__ __align__(16) float s_st[kVec == 4 ? kRG * kRows * kCols : 4];
  float st[kVec == 4 ? 1 : kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    const int r = ty + kRG * j;
    const bool on = ok && r < d_k && (!kMany || a.from != nullptr);
    if constexpr (kVec == 4) cp_async_16_zfill(&s_st[(kThr * j + tid) * 4], on ? a.from + at + int64_t(r) * d_v : nothing, on);
    else st[j] = on ? __ldcs(a.from + at + int64_t(r) * d_v) : 0.f;
  }
  auto entry = [&](int j) { return reinterpret_cast<float4 *>(&s_st[(kThr * j + tid) * 4]); };
  // the decayed entries of row j
  auto get = [&](int j, Decay decay, float (&x)[kVec]) {
    if constexpr (kVec == 4) {
      const float4 v = *entry(j);
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
      x[0] = st[j];
    }
#pragma unroll
    for (int e = 0; e < kVec; ++e) x[e] = decay_step(x[e], decay);
  };
  auto write = [&](int j, const float (&x)[kVec]) {
    const int r = ty + kRG * j;
    if (!ok || r >= d_k) return;
    if constexpr (kVec == 4) __stcs(reinterpret_cast<float4 *>(to + at + int64_t(r) * d_v), make_float4(x[0], x[1], x[2], x[3]));
    else __stcs(to + at + int64_t(r) * d_v, x[0]);
  };
#pragma unroll 1
  for (int64_t t = t0; t < t1; ++t) {
    if (kMany && t > t0) __syncthreads();  // the token before is done with what is shared
    const Decay decay = decay_of(a.log_decay[a.per_token ? t * a.H + h : h]);
    const float b = a.beta[t * a.H + h];
    float vv[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) vv[e] = ok ? load_elem<kInBF16>(a.v, (t * a.H + h) * d_v + col + e) : 0.f;
#pragma unroll
    for (int i = tid; i < kRG * kRows; i += kThr) {
      s_k[i] = i < d_k ? load_elem<kInBF16>(a.k, (t * a.H_k + hk) * d_k + i) : 0.f;
      s_q[i] = i < d_k ? load_elem<kInBF16>(a.q, (t * a.H_k + hk) * d_k + i) : 0.f;
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
      const float kr = s_k[ty + kRG * j];
      float x[kVec];
      get(j, decay, x);
#pragma unroll
      for (int e = 0; e < kVec; ++e) x[e] = fmaf(kr, u[e], x[e]);
      if constexpr (!kMany) {
        write(j, x);
      } else if constexpr (kVec == 4) {
        *entry(j) = make_float4(x[0], x[1], x[2], x[3]);
      } else {
        st[j] = x[0];
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
        store_elem<kOutBF16>(a.out, (t * a.H + h) * d_v + col + e, a.scale * fmaf(kq, u[e], sum));
      }
    }
  }
  if constexpr (kMany) {
    if (to == nullptr) return;
    if constexpr (kVec == 4) cp_async_wait_all();  // (a sequence without tokens)
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      if constexpr (kVec == 4) {
        const float4 v = *entry(j);
        const float x[4] = {v.x, v.y, v.z, v.w};
        write(j, x);
      } else {
        const float x[1] = {st[j]};
        write(j, x);
      }
    }
  }
}

}  // namespace

namespace {

cudaError_t launch_tokens(TokenArgs a, int64_t pairs, bool in_bf16, bool out_bf16, cudaStream_t stream) {
  // Four columns per thread where rows of the state start on 16-byte boundaries, tiles as narrow as the
  // columns need and the fewest threads that hold all key rows: 32, 64 or 128. Narrower tiles while there are
  // fewer than two for each SM (us at 16 / 32 / 64 columns: 96 pairs of 128 8.3 / 6.2 / 7.7, 384 pairs
  // 14.4 / 12.3 / 12.3, 24576 pairs 545 / 511 / 470).
  const bool vec = a.d_v % 4 == 0;
  int size = a.d_v <= 16 ? 0 : a.d_v <= 32 ? 1 : 2;  // 16, 32 or 64 columns per CTA
  const auto tiles_of = [&](int x) { return (a.d_v + (16 << x) - 1) / (16 << x); };
  while (size > 0 && pairs * tiles_of(size) < 2 * kLinearSMs) --size;
  a.tiles = tiles_of(size);
  const int rows = a.d_k <= 32 ? 0 : a.d_k <= 64 ? 1 : 2;
  using Kern = void (*)(const TokenArgs);
#define KDA_DDEC(v_, tx, t) \
  { KDA_DDEC_IO(v_, tx, t, false), KDA_DDEC_IO(v_, tx, t, true) }
#define KDA_DDEC_IO(v_, tx, t, m) \
  { delta_decode_kernel<false, false, v_, tx, t, m>, delta_decode_kernel<false, true, v_, tx, t, m>, \
    delta_decode_kernel<true, false, v_, tx, t, m>, delta_decode_kernel<true, true, v_, tx, t, m> }
  // threads: kTX x (key rows / rows per thread)
  static const Kern one[3][3][2][4] = {{KDA_DDEC(1, 16, 32), KDA_DDEC(1, 16, 32), KDA_DDEC(1, 16, 64)},
                                       {KDA_DDEC(1, 32, 32), KDA_DDEC(1, 32, 64), KDA_DDEC(1, 32, 128)},
                                       {KDA_DDEC(1, 64, 64), KDA_DDEC(1, 64, 128), KDA_DDEC(1, 64, 256)}};
  static const Kern four[3][3][2][4] = {{KDA_DDEC(4, 4, 32), KDA_DDEC(4, 4, 32), KDA_DDEC(4, 4, 64)},
                                        {KDA_DDEC(4, 8, 32), KDA_DDEC(4, 8, 64), KDA_DDEC(4, 8, 128)},
                                        {KDA_DDEC(4, 16, 64), KDA_DDEC(4, 16, 128), KDA_DDEC(4, 16, 256)}};
  static const int threads[3][3] = {{32, 32, 64}, {32, 64, 128}, {64, 128, 256}};
#undef KDA_DDEC
#undef KDA_DDEC_IO
  (vec ? four : one)[size][rows][int(a.cu != nullptr)][2 * int(in_bf16) + int(out_bf16)]
      <<<unsigned(pairs * a.tiles), threads[size][rows], 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_delta_decode(const void *q, const void *k, const void *v, const float *log_decay, bool per_token,
                                const float *beta, float *state, void *out, int B, int H, int H_k, int d_k, int d_v,
                                bool in_bf16, bool out_bf16, float scale, cudaStream_t stream) {
  const TokenArgs a{q, k, v, log_decay, beta, state, state, out, nullptr, int(per_token), H, H_k, d_k, d_v, 0, 0, scale};
  return launch_tokens(a, int64_t(B) * H, in_bf16, out_bf16, stream);
}

cudaError_t launch_delta_short(const DeltaArgs &d, bool in_bf16, bool out_bf16, cudaStream_t stream) {
  const TokenArgs a{d.q, d.k, d.v, d.log_decay, d.beta, d.init_state, d.final_state, d.out, d.cu, d.per_token,
                    d.H, d.H_k, d.d_k, d.d_v, 0, d.plan.few, d.scale};
  return launch_tokens(a, int64_t(d.num_seqs) * d.H, in_bf16, out_bf16, stream);
}

}  // namespace kda
