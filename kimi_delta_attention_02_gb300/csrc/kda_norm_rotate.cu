// kda_norm_rotate.cu -- the norm of each query and key head and its rotary positions in one pass.
// y = r (a (*) x + b (*) x_partner) per head row, with r = 1 / sqrt(mean(x^2) + eps) (or of the sum, or
// one), a = w cos p and b = -+ w_partner sin p of the token's angles, which all heads share.
//
// Reads and writes q and k once at about 7 flops per element: bound by HBM bandwidth (4096 tokens, 192 heads
// of 128, bf16: 403 MB in 82 us, 4.9 TB/s; the copy rate would be 60 us), by latency for a few tokens (one token:
// 6 us). The angles of a token are formed once per CTA, in shared memory. A head row takes as many lanes as it
// has pieces of 8 channels, so that a warp works on up to 32 rows at once (10007 tokens, 20 heads of 72: 23 us; 31
// with lanes in powers of two). A lane keeps the factors of its channels in registers while it goes through the
// token's heads, two at a time. A turned channel's partner is in the same lane (neighbours), in another one,
// or comes by a second load, which finds its line in L1.
//
// Angles. p = position * f can be millions of radians, where fp32 is off by tenths. A turn is a number
// modulo one: F = f / (2 pi) modulo one as a 128-bit fraction (off by 2^-104 while f is below 2^24), and the
// upper 64 bits of the wrapping product |position| F are the angle's fraction of a turn, off by 2^-41 at the
// furthest of 64-bit positions. The nearest quarter turn is taken off in integers, so that what fp32 holds of
// the rest, at most an eighth, is off by 2^-28 of a turn (all of a turn's fraction in 24 bits by 2^-26).
#include "kda_common.cuh"
#include "kda_norm_rotate.h"

namespace kda {
namespace {

constexpr int kThr = 256;

using Turns = unsigned __int128;  // the fraction of a turn, behind the point

__device__ __forceinline__ Turns turns_per_position(float inv_freq) {
  // |f| = m 2^-s with a whole m, times 1 / (2 pi) with 128 bits behind the point; all in integers
  const uint32_t bits = __float_as_uint(inv_freq) & 0x7fffffffu, exponent = bits >> 23;
  const uint64_t m = (bits & 0x7fffffu) | (exponent != 0 ? 0x800000u : 0u);
  const int s = 150 - int(exponent != 0 ? exponent : 1);
  constexpr uint64_t k1 = 0x28be60db9391054aull, k0 = 0x7f09d5f47d4d3770ull;  // 1 / (2 pi)
  const Turns upper = Turns(m) * k1 + __umul64hi(m, k0);
  const Turns low = (upper << 64) | (m * k0), high = upper >> 64;  // m / (2 pi) 2^128
  const Turns f = s <= 0 ? (s > -128 ? low << -s : 0) : s < 128 ? (low >> s) | (high << (128 - s)) : high >> (s - 128);
  return inv_freq < 0.f ? 0 - f : f;
}
// The angle of pair i at token t as (cos, sin); `turns` is the pair's F.
__device__ __forceinline__ float2 angle(const RotateArgs &a, int i, int64_t t, Turns turns) {
  const int64_t at = a.axis[i] * a.tokens + t;
  const int64_t pos = a.pos64 ? static_cast<const int64_t *>(a.positions)[at]
                              : int64_t(static_cast<const int32_t *>(a.positions)[at]);
  const uint64_t far = pos < 0 ? uint64_t(0) - uint64_t(pos) : uint64_t(pos);
  uint64_t turn = far * uint64_t(turns >> 64) + __umul64hi(far, uint64_t(turns));
  if (pos < 0) turn = uint64_t(0) - turn;
  const uint32_t quarter = uint32_t((turn + (uint64_t(1) << 61)) >> 62);  // the nearest; 4 is 0
  const int32_t rest = int32_t(int64_t(turn - (uint64_t(quarter) << 62)) >> 30);  // in 2^-34 of a turn
  float s, c;
  sincospif(float(rest) * 0x1p-33f, &s, &c);
  if (quarter & 1) {
    const float x = c;
    c = -s, s = x;
  }
  if (quarter & 2) c = -c, s = -s;
  if (!isfinite(a.inv_freq[i])) s = c = __int_as_float(0x7fc00000);
  return make_float2(c, s);
}
__device__ __forceinline__ float norm_factor(const RotateArgs &a, float sum) {
  return a.norm == KDA_NORM_NONE ? 1.f : rsqrtf(fmaf(sum, a.per, a.eps));
}

// 8 channels as stored: N 16-byte words
template <bool kBF16>
struct Piece {
  uint4 w[kBF16 ? 1 : 2];
  __device__ __forceinline__ void get(float (&x)[8]) const {
    if constexpr (kBF16) {
      const float2 p[4] = {unpack_bf16x2(w[0].x), unpack_bf16x2(w[0].y), unpack_bf16x2(w[0].z), unpack_bf16x2(w[0].w)};
#pragma unroll
      for (int e = 0; e < 4; ++e) x[2 * e] = p[e].x, x[2 * e + 1] = p[e].y;
    } else {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        x[4 * e] = __uint_as_float(w[e].x), x[4 * e + 1] = __uint_as_float(w[e].y);
        x[4 * e + 2] = __uint_as_float(w[e].z), x[4 * e + 3] = __uint_as_float(w[e].w);
      }
    }
  }
};
// four neighbouring elements
template <bool kBF16>
__device__ __forceinline__ void load4(const void *base, int64_t at, float *x) {
  if constexpr (kBF16) {
    const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(base) + at);
    const float2 a = unpack_bf16x2(w.x), b = unpack_bf16x2(w.y);
    x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
  } else {
    const float4 w = *reinterpret_cast<const float4 *>(static_cast<const float *>(base) + at);
    x[0] = w.x, x[1] = w.y, x[2] = w.z, x[3] = w.w;
  }
}

// Rows of whole pieces of 8 channels on 16-byte boundaries. kPart: partners are neighbours (0), or lie rot / 2
// channels away: whole pieces (8) come from their lane, half pieces (4) by a load, others (1) by a load each. With
// 1 and 2 (neighbours) a piece may turn in part; else it turns as a whole or not at all. `lanes` threads per
// row, `group` rows of a token side by side; `pairs` threads form a token's angles. (65536 tokens, 18 heads of 64 of
// which 20 channels turn: 117 us as halves, 70 as neighbours; 155 by the kernel below.)
template <bool kInBF16, bool kOutBF16, int kPart>
__global__ void __launch_bounds__(kThr, 3) rotate_kernel(const RotateArgs a, int lanes, int group, int pairs) {
  constexpr int kEi = kInBF16 ? 2 : 4, kEo = kOutBF16 ? 2 : 4;
  constexpr int kU = kInBF16 ? 2 : 1;  // rows at a time, and as many on their way
  constexpr bool kNear = kPart == 0 || kPart == 2, kSome = kPart == 1 || kPart == 2;
  __shared__ Turns s_turn[kRotateMaxD / 2];
  __shared__ __align__(16) float2 s_cs[2][kThr * 4];  // tokens x rot / 2: a row has at most 8 channels per lane
  const int tid = threadIdx.x, lane = tid & 31;
  const int per_warp = 32 / lanes, slots = kThr / 32 * per_warp;  // (lanes behind a warp's last row take part in shuffles only)
  const int piece = lane % lanes, slot = lane < per_warp * lanes ? (tid >> 5) * per_warp + lane / lanes : slots;
  const int tokens = slots / group, token = slot / group;
  const int c0 = 8 * piece, first = slot % group + group * blockIdx.y, stride = group * gridDim.y;
  const bool turns = c0 < 2 * a.half, upper = c0 >= a.half;
  const int partner = turns ? (upper ? c0 - a.half : c0 + a.half) : c0;  // of a whole piece, and its lane
  const int from_lane = lane + (partner - c0) / 8;
  int half_way = 1;  // half of the next power of two
  while (2 * half_way < lanes) half_way *= 2;
  if (lanes == 1) half_way = 0;
  for (int i = tid; i < a.half; i += kThr) s_turn[i] = turns_per_position(a.inv_freq[i]);
  __syncthreads();
  int buf = 0;
#pragma unroll 1
  for (int64_t t0 = int64_t(blockIdx.x) * tokens; t0 < a.tokens; t0 += int64_t(gridDim.x) * tokens, buf ^= 1) {
    const int here = a.tokens - t0 < tokens ? int(a.tokens - t0) : tokens;
    const int64_t t = t0 + token;
    const bool mine = token < here;
    // the first row is on its way while the angles are formed
    const uint8_t *src;
    Piece<kInBF16> next[kU] = {};
    auto fetch = [&](int h, int rows) {
#pragma unroll
      for (int u = 0; u < kU; ++u)
        if (mine && h + u * stride < rows) {
#pragma unroll
          for (int e = 0; e < kEi / 2; ++e)
            next[u].w[e] = reinterpret_cast<const uint4 *>(src + uint32_t(u * stride) * a.d * kEi + c0 * kEi)[e];
        }
    };
    src = static_cast<const uint8_t *>(a.x[0]) + (t * a.stride[0] + int64_t(first) * a.d) * kEi;
    fetch(first, a.heads[0]);
    const int p = tid & (pairs - 1);
#pragma unroll 1
    for (int i = tid / pairs; i < here; i += kThr / pairs)
      if (p < a.half) s_cs[buf][i * a.half + p] = angle(a, p, t0 + i, s_turn[p]);
    __syncthreads();  // (the other buffer's readers are past it when this one is written again)
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      const int rows = a.heads[which];
      if (which == 1) {
        src = static_cast<const uint8_t *>(a.x[1]) + (t * a.stride[1] + int64_t(first) * a.d) * kEi;
        fetch(first, rows);
      }
      // the factors of this lane's channels and of their partners
      const float *w = a.weight[which];
      float2 ca[4], cb[4];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = c0 + e;
        const bool up = kNear ? (e & 1) != 0 : c >= a.half;
        const int p = kNear ? c ^ 1 : up ? c - a.half : c + a.half;
        float x = 1.f, y = 0.f;
        if (mine && (kSome ? c < 2 * a.half : turns)) {
          const float2 cs = s_cs[buf][token * a.half + (kNear ? c >> 1 : up ? p : c)];
          x = cs.x, y = up ? cs.y : -cs.y;
          if (w != nullptr) y *= w[p];
        }
        if (mine && w != nullptr) x *= w[c];
        if (e & 1) ca[e >> 1].y = x, cb[e >> 1].y = y;
        else ca[e >> 1].x = x, cb[e >> 1].x = y;
      }
      uint8_t *dst = static_cast<uint8_t *>(a.out[which]) + (t * a.out_stride[which] + int64_t(first) * a.d + c0) * kEo;
      const uint32_t row_in = uint32_t(stride) * a.d * kEi, row_out = uint32_t(stride) * a.d * kEo;
#pragma unroll 1
      for (int h = first; h - first < rows; h += kU * stride, dst += kU * row_out) {  // (all rows of a warp go round together)
        Piece<kInBF16> raw[kU];
        const uint8_t *row = src;
        src += kU * row_in;
#pragma unroll
        for (int u = 0; u < kU; ++u) raw[u] = next[u];
        fetch(h + kU * stride, rows);
        float sum[kU];
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          float x[8];
          raw[u].get(x);
          float2 s2 = make_float2(0.f, 0.f);
#pragma unroll
          for (int e = 0; e < 8; e += 2) s2 = f2_fma(make_float2(x[e], x[e + 1]), make_float2(x[e], x[e + 1]), s2);
          sum[u] = s2.x + s2.y;
        }
        // to a row's first lane, and from there to all
#pragma unroll 1
        for (int off = half_way; off > 0; off >>= 1) {
#pragma unroll
          for (int u = 0; u < kU; ++u) {
            const float other = __shfl_down_sync(0xffffffffu, sum[u], off);
            if (piece + off < lanes) sum[u] += other;
          }
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) sum[u] = __shfl_sync(0xffffffffu, sum[u], lane - piece);
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          const bool ok = mine && h + u * stride < rows;
          float x[8], xp[8];
          raw[u].get(x);
          if constexpr (kNear) {
#pragma unroll
            for (int e = 0; e < 8; ++e) xp[e] = kSome && c0 + e >= 2 * a.half ? 0.f : x[e ^ 1];
          } else if constexpr (kPart == 1) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const int c = c0 + e;
              xp[e] = ok && c < 2 * a.half ? load_elem<kInBF16>(row + u * row_in, c < a.half ? c + a.half : c - a.half) : 0.f;
            }
          } else if constexpr (kPart == 8) {
            Piece<kInBF16> p;
#pragma unroll
            for (int e = 0; e < kEi / 2; ++e) {
              p.w[e].x = __shfl_sync(0xffffffffu, raw[u].w[e].x, from_lane), p.w[e].y = __shfl_sync(0xffffffffu, raw[u].w[e].y, from_lane);
              p.w[e].z = __shfl_sync(0xffffffffu, raw[u].w[e].z, from_lane), p.w[e].w = __shfl_sync(0xffffffffu, raw[u].w[e].w, from_lane);
            }
            p.get(xp);
          } else {
#pragma unroll
            for (int e = 0; e < 8; e += 4) {
              if (ok && turns)
                load4<kInBF16>(row + u * row_in, c0 + e < a.half ? c0 + e + a.half : c0 + e - a.half, &xp[e]);
            }
          }
          __syncwarp();  // in place: every lane of the row has read it
          const float r = norm_factor(a, sum[u]);
          float2 y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            y[e] = f2_mul(make_float2(x[2 * e], x[2 * e + 1]), ca[e]);
            // (left out or zero, not multiplied by zero, where nothing turns: the partner may be infinite)
            if (turns) y[e] = f2_fma(make_float2(xp[2 * e], xp[2 * e + 1]), cb[e], y[e]);
            y[e] = f2_mul(y[e], make_float2(r, r));
          }
          if (ok) {
            uint8_t *to = dst + u * row_out;
            if constexpr (kOutBF16) {
              *reinterpret_cast<uint4 *>(to) = make_uint4(pack_bf16x2(y[0].x, y[0].y), pack_bf16x2(y[1].x, y[1].y),
                                                          pack_bf16x2(y[2].x, y[2].y), pack_bf16x2(y[3].x, y[3].y));
            } else {
              reinterpret_cast<float4 *>(to)[0] = make_float4(y[0].x, y[0].y, y[1].x, y[1].y);
              reinterpret_cast<float4 *>(to)[1] = make_float4(y[2].x, y[2].y, y[3].x, y[3].y);
            }
          }
        }
      }
    }
  }
}

// Rows that start anywhere, head sizes that are no multiple of 8: a warp per row, a pair of channels per lane
// and step (kPer of them: the pairs that turn, then neighbours of those that do not), element by element. A
// warp keeps a token's factors in registers while it goes through its share of the token's heads (blockIdx.y).
// Bound by its 2-byte accesses: the sizes above take 189 us here, and 10007 tokens of 20 heads of 72 take 45 us
// (23 us by whole pieces), so rows that allow it go there.
template <bool kInBF16, bool kOutBF16, int kPer>
__global__ void __launch_bounds__(kThr) rotate_any_kernel(const RotateArgs a, int interleaved) {
  const int lane = threadIdx.x & 31;
  Turns turns[kPer];
  int ch[kPer], ph[kPer];  // the pair's channels, or the row's end
#pragma unroll
  for (int j = 0; j < kPer; ++j) {
    const int p = lane + 32 * j;
    const bool turned = p < a.half;
    turns[j] = turned ? turns_per_position(a.inv_freq[p]) : 0;
    ch[j] = turned && interleaved == 0 ? p : 2 * p;
    ph[j] = turned && interleaved == 0 ? p + a.half : 2 * p + 1;
    if (ch[j] > a.d) ch[j] = a.d;
    if (ph[j] > a.d) ph[j] = a.d;
  }
#pragma unroll 1
  for (int64_t t = blockIdx.x * int64_t(kThr / 32) + (threadIdx.x >> 5); t < a.tokens; t += gridDim.x * int64_t(kThr / 32)) {
    float2 cs[kPer];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int p = lane + 32 * j;
      cs[j] = p < a.half ? angle(a, p, t, turns[j]) : make_float2(1.f, 0.f);
    }
#pragma unroll 1
    for (int which = 0; which < 2; ++which) {
      const float *weight = a.weight[which];
      float w[kPer], wp[kPer];
#pragma unroll
      for (int j = 0; j < kPer; ++j) {
        w[j] = weight != nullptr && ch[j] < a.d ? weight[ch[j]] : 1.f;
        wp[j] = weight != nullptr && ph[j] < a.d ? weight[ph[j]] : 1.f;
      }
#pragma unroll 1
      for (int h = blockIdx.y; h < a.heads[which]; h += gridDim.y) {
        const int64_t from = t * a.stride[which] + int64_t(h) * a.d, to = t * a.out_stride[which] + int64_t(h) * a.d;
        float x[kPer], xp[kPer], sum = 0.f;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          x[j] = ch[j] < a.d ? load_elem<kInBF16>(a.x[which], from + ch[j]) : 0.f;
          xp[j] = ph[j] < a.d ? load_elem<kInBF16>(a.x[which], from + ph[j]) : 0.f;
        }
#pragma unroll
        for (int j = 0; j < kPer; ++j) sum = fmaf(x[j], x[j], fmaf(xp[j], xp[j], sum));
        if (a.norm != KDA_NORM_NONE) {
#pragma unroll
          for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        }
        const float r = norm_factor(a, sum);
        __syncwarp();  // in place: every lane has read the row
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
          const bool turned = lane + 32 * j < a.half;
          const float n = w[j] * x[j], np = wp[j] * xp[j];
          // (left as they are, not multiplied by zero, where nothing turns: the neighbour may be infinite)
          const float y = turned ? fmaf(n, cs[j].x, -np * cs[j].y) : n, yp = turned ? fmaf(np, cs[j].x, n * cs[j].y) : np;
          if (ch[j] < a.d) store_elem<kOutBF16>(a.out[which], to + ch[j], r * y);
          if (ph[j] < a.d) store_elem<kOutBF16>(a.out[which], to + ph[j], r * yp);
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_norm_rotate(const RotateArgs &a, bool in_bf16, bool out_bf16, bool interleaved, cudaStream_t stream) {
  const auto whole = [&](const void *p, int64_t stride, int size) {
    return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && (a.tokens == 1 || stride * size % 16 == 0));
  };
  const int si = in_bf16 ? 2 : 4, so = out_bf16 ? 2 : 4;
  if (a.d % 8 == 0 && whole(a.x[0], a.stride[0], si) && whole(a.x[1], a.stride[1], si) &&
      whole(a.out[0], a.out_stride[0], so) && whole(a.out[1], a.out_stride[1], so)) {
    using Kern = void (*)(const RotateArgs, int, int, int);
#define KDA_ROT(ib, ob) \
  {rotate_kernel<ib, ob, 0>, rotate_kernel<ib, ob, 2>, rotate_kernel<ib, ob, 8>, rotate_kernel<ib, ob, 4>, rotate_kernel<ib, ob, 1>}
    static const Kern kernels[4][5] = {KDA_ROT(false, false), KDA_ROT(false, true), KDA_ROT(true, false), KDA_ROT(true, true)};
#undef KDA_ROT
    const int lanes = a.d / 8, slots = kThr / 32 * (32 / lanes);
    int pairs = 1, group = 1;
    while (pairs < a.half) pairs *= 2;
    const int rows = a.heads[0] > a.heads[1] ? a.heads[0] : a.heads[1];
    const int64_t fit = 152 * 3;
    // A lane's factors serve up to twelve rows of a token (us at 1 / 3 / 6 / 12 / 24 rows: 4096 tokens, 192 heads of 128
    // 82 / 82 / 82 / 79 / 83; 80 heads 59 / 59 / 43 / 40 / 45).
    while (2 * group <= slots && group * 12 < rows) group *= 2;
    const int64_t tokens = slots / group, passes = (a.tokens + tokens - 1) / tokens;
    // Few tokens: their heads over several CTAs.
    const int64_t most = (rows + group - 1) / group, spare = fit / passes;
    const unsigned parts = unsigned(spare < 1 ? 1 : spare < most ? spare : most);
    kernels[2 * int(in_bf16) + int(out_bf16)][interleaved ? (a.half % 4 == 0 ? 0 : 1) : a.half % 8 == 0 ? 2 : a.half % 4 == 0 ? 3 : 4]<<<
        dim3(unsigned(passes < fit ? passes : fit), parts), kThr, 0, stream>>>(a, lanes, group, pairs);
    return cudaGetLastError();
  }
  using Kern = void (*)(const RotateArgs, int);
#define KDA_ROT(ib, ob) {rotate_any_kernel<ib, ob, 1>, rotate_any_kernel<ib, ob, 2>, rotate_any_kernel<ib, ob, 4>}
  static const Kern any[4][3] = {KDA_ROT(false, false), KDA_ROT(false, true), KDA_ROT(true, false), KDA_ROT(true, true)};
#undef KDA_ROT
  const int64_t fit = 152 * 6, passes = (a.tokens + kThr / 32 - 1) / (kThr / 32);
  const int64_t rows = a.heads[0] > a.heads[1] ? a.heads[0] : a.heads[1], spare = fit / passes;
  const unsigned parts = unsigned(spare < 1 ? 1 : spare < rows ? spare : rows);
  any[2 * int(in_bf16) + int(out_bf16)][a.d <= 64 ? 0 : a.d <= 128 ? 1 : 2]<<<
      dim3(unsigned(passes < fit ? passes : fit), parts), kThr, 0, stream>>>(a, int(interleaved));
  return cudaGetLastError();
}

}  // namespace kda
