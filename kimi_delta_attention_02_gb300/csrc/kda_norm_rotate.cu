// kda_norm_rotate.cu -- the norm of each query and key head and its rotary positions in one pass.
// y = r (a (*) x + b (*) x_partner) per head row, with r = 1 / sqrt(mean(x^2) + eps) (or of the sum, or
// one), a = w cos p and b = -+ w_partner sin p of the token's angles, which all heads share.
//
// Reads and writes q and k once at about 7 flops per element: bound by HBM bandwidth. The angles of a
// token are formed once per CTA, in shared memory; a row's lanes then keep a and b of their channels
// in registers while they go through the token's heads.
//
// Angles. p = position * f can be millions of radians, where fp32 is off by tenths. A turn is a number
// modulo one: F = f / (2 pi) modulo one as a 64-bit fraction (formed in fp64, off by 2^-53 of itself, so
// the angle is off by 2^-53 of itself too), and the wrapping 64-bit product position * F is the angle's
// fraction of a turn whatever the position, negative ones among them. Its top 32 bits, as a signed number
// of half turns, go to sincospi: off by 2^-32 of a turn.
#include "kda_common.cuh"
#include "kda_norm_rotate.h"

namespace kda {
namespace {

constexpr int kThr = 256;

// One channel per lane and step: rows that start anywhere, head sizes that are no multiple of 8.
template <bool kInBF16, bool kOutBF16, bool kNeighbours>
__global__ void __launch_bounds__(kThr) rotate_any_kernel(const RotateArgs a) {
  constexpr int kPer = kRotateMaxD / 32;
  __shared__ uint64_t s_turn[kRotateMaxD / 2];
  __shared__ float2 s_cs[kRotateMaxD / 2];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  for (int i = tid; i < a.half; i += kThr) {
    const double f = double(a.inv_freq[i]) * 0.15915494309189533577;  // turns per position
    s_turn[i] = __double2ull_rz((f - floor(f)) * 18446744073709551616.);
  }
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    __syncthreads();
    for (int i = tid; i < a.half; i += kThr) {
      const int64_t at = a.axis[i] * a.tokens + t;
      const int64_t pos = a.pos64 ? static_cast<const int64_t *>(a.positions)[at]
                                  : int64_t(static_cast<const int32_t *>(a.positions)[at]);
      const int32_t turn = int32_t((uint64_t(pos) * s_turn[i]) >> 32);
      float s, c;
      sincospif(float(turn) * 0x1p-31f, &s, &c);
      if (!isfinite(a.inv_freq[i])) s = c = __int_as_float(0x7fc00000);
      s_cs[i] = make_float2(c, s);
    }
    __syncthreads();
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      const int64_t from = t * a.stride[which], to = t * a.out_stride[which];
      float ca[kPer], cb[kPer];
      int partner[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        const int c = lane + 32 * j;
        const bool turned = c < 2 * a.half;
        const bool first = kNeighbours ? (c & 1) == 0 : c < a.half;
        partner[j] = !turned ? c : kNeighbours ? c ^ 1 : first ? c + a.half : c - a.half;
        const float2 cs = turned ? s_cs[kNeighbours ? c >> 1 : first ? c : c - a.half] : make_float2(1.f, 0.f);
        const float *weight = a.weight[which];
        const bool on = c < a.d;
        ca[j] = (weight != nullptr && on ? weight[c] : 1.f) * cs.x;
        cb[j] = (weight != nullptr && on ? weight[partner[j]] : 1.f) * (first ? -cs.y : cs.y);
      }
#pragma unroll 1
      for (int h = w; h < a.heads[which]; h += kThr / 32) {
        const int64_t row = from + int64_t(h) * a.d;
        float x[kPer], xp[kPer], sum = 0.f;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int c = lane + 32 * j;
          x[j] = c < a.d ? load_elem<kInBF16>(a.x[which], row + c) : 0.f;
          xp[j] = c < 2 * a.half ? load_elem<kInBF16>(a.x[which], row + partner[j]) : 0.f;
          sum = fmaf(x[j], x[j], sum);
        }
        float r = 1.f;
        if (a.norm != KDA_NORM_NONE) {
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
          r = 1.f / sqrtf((a.norm == KDA_NORM_RMS ? sum / float(a.d) : sum) + a.eps);
        }
        __syncwarp();  // in place: every lane has read the row
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const int c = lane + 32 * j;
          const float y = c < 2 * a.half ? fmaf(xp[j], cb[j], x[j] * ca[j]) : x[j] * ca[j];
          if (c < a.d) store_elem<kOutBF16>(a.out[which], to + int64_t(h) * a.d + c, r * y);
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_norm_rotate(const RotateArgs &a, bool in_bf16, bool out_bf16, bool interleaved, cudaStream_t stream) {
  using Kern = void (*)(const RotateArgs);
#define KDA_ROT(ib, ob) {rotate_any_kernel<ib, ob, false>, rotate_any_kernel<ib, ob, true>}
  static const Kern any[4][2] = {KDA_ROT(false, false), KDA_ROT(false, true), KDA_ROT(true, false), KDA_ROT(true, true)};
#undef KDA_ROT
  const int64_t fit = 152 * 8;
  any[2 * int(in_bf16) + int(out_bf16)][int(interleaved)]<<<unsigned(a.tokens < fit ? a.tokens : fit), kThr, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kda
