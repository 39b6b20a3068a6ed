// kda_block_norm.cu -- between two blocks of a residual stream, in one pass over each row of D
// channels:
//     n  = w_post (*) y / sqrt(mean(y^2) + eps)      (or n = y without the norm after the block)
//     x' = x + scale c (*) Sigmoid(r) (*) n          (r: one gate logit per channel or per row)
//     h  = w_pre (*) x' / sqrt(mean(x'^2) + eps)     (x' in fp32, before it is rounded for storage)
// Each tensor is read once and written once, the row in registers between its two sums: bound by
// HBM bandwidth, or by latency when there are few rows.
#include "kda_common.cuh"
#include "kda_block_norm.h"

namespace kda {
namespace {

// eight neighbouring elements; p is 16-byte aligned
template <bool kBF16>
__device__ __forceinline__ void load8(const void *base, int64_t at, float (&v)[8]) {
  if constexpr (kBF16) {
    const uint4 u = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + at);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack_bf16x2(w[i]);
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  } else {
    const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(base) + at);
    const float4 a = p[0], b = p[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
}
template <bool kBF16>
__device__ __forceinline__ void store8(void *base, int64_t at, const float (&v)[8]) {
  if constexpr (kBF16) {
    *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(base) + at) =
        make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else {
    float4 *p = reinterpret_cast<float4 *>(static_cast<float *>(base) + at);
    p[0] = make_float4(v[0], v[1], v[2], v[3]);
    p[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// Sum over the threads of a row: the warp's, then, with several warps per row (one row per CTA),
// the CTA's. `slot` keeps two sums of one row apart.
__device__ __forceinline__ float row_sum(float x, int warps, float *s_part, int slot) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  if (warps == 1) return x;
  if ((threadIdx.x & 31) == 0) s_part[slot * 32 + (threadIdx.x >> 5)] = x;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  x = lane < warps ? s_part[slot * 32 + lane] : 0.f;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// A row's threads hold its channels in kG pieces of 8 each: with kWide 8 neighbouring channels per
// piece (16-byte accesses; D a multiple of 8), else 8 channels a row's threads apart.
template <bool kXB, bool kYB, bool kOB, int kG, bool kWide>
__global__ void __launch_bounds__(kG > 1 ? 512 : 1024) block_norm_kernel(const BlockNormArgs a) {
  __shared__ float s_part[64];
  const int tpr = a.threads_per_row, warps = tpr >> 5;
  const int lane = threadIdx.x % tpr;
  const int64_t row = int64_t(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
  if (row >= a.rows) return;  // whole warps: with several rows per CTA a row is one warp
  const int64_t base = row * a.D;
  const int D = a.D;
  auto channel = [&](int g, int e) { return kWide ? (g * tpr + lane) * 8 + e : (g * 8 + e) * tpr + lane; };

  float x[kG][8], u[kG][8];
  float gate[kG][8];
  const bool has_y = a.y != nullptr;
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    if constexpr (kWide) {
      const int c = channel(g, 0);
      if (c < D) {
        load8<kXB>(a.x, base + c, x[g]);
        if (has_y) load8<kYB>(a.y, base + c, u[g]);
        if (a.gate_form == 1) load8<kYB>(a.gate, base + c, gate[g]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[g][e] = u[g][e] = gate[g][e] = 0.f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = channel(g, e);
        x[g][e] = u[g][e] = gate[g][e] = 0.f;
        if (c < D) {
          x[g][e] = load_elem<kXB>(a.x, base + c);
          if (has_y) u[g][e] = load_elem<kYB>(a.y, base + c);
          if (a.gate_form == 1) gate[g][e] = load_elem<kYB>(a.gate, base + c);
        }
      }
    }
  }
  auto weight = [&](const float *w, int g, float (&v)[8]) {  // ones without a weight
    if (w == nullptr) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 1.f;
      return;
    }
    if constexpr (kWide) {
      const int c = channel(g, 0);
      if (c < D) load8<false>(w, c, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = channel(g, e) < D ? w[channel(g, e)] : 0.f;
    }
  };

  if (has_y) {
    float rstd = 1.f;
    if (a.post_norm) {
      float ss = 0.f;
#pragma unroll
      for (int g = 0; g < kG; ++g)
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(u[g][e], u[g][e], ss);
      rstd = 1.f / sqrtf(row_sum(ss, warps, s_part, 0) / float(D) + a.post_eps);
    }
    float f = a.scale * rstd;
    if (a.gate_form == 2) f *= sigmoid_approx(load_elem<kYB>(a.gate, row));
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      float w[8], c[8];
      weight(a.post_weight, g, w);
      weight(a.channel_scale, g, c);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float s = f * w[e] * c[e];
        if (a.gate_form == 1) s *= sigmoid_approx(gate[g][e]);
        if (kWide ? channel(g, 0) < D : channel(g, e) < D) x[g][e] = fmaf(s, u[g][e], x[g][e]);
      }
    }
  }
  if (a.residual_out != nullptr) {
#pragma unroll
    for (int g = 0; g < kG; ++g) {
      if constexpr (kWide) {
        if (channel(g, 0) < D) store8<kXB>(a.residual_out, base + channel(g, 0), x[g]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (channel(g, e) < D) store_elem<kXB>(a.residual_out, base + channel(g, e), x[g][e]);
      }
    }
  }
  if (a.out == nullptr) return;
  float ss = 0.f;
#pragma unroll
  for (int g = 0; g < kG; ++g)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fmaf(x[g][e], x[g][e], ss);
  const float rstd = 1.f / sqrtf(row_sum(ss, warps, s_part, 1) / float(D) + a.pre_eps);
#pragma unroll
  for (int g = 0; g < kG; ++g) {
    float w[8];
    weight(a.pre_weight, g, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] *= x[g][e] * rstd;
    if constexpr (kWide) {
      if (channel(g, 0) < D) store8<kOB>(a.out, base + channel(g, 0), w);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (channel(g, e) < D) store_elem<kOB>(a.out, base + channel(g, e), w[e]);
    }
  }
}

}  // namespace

cudaError_t launch_block_norm(BlockNormArgs a, bool x_bf16, bool y_bf16, bool out_bf16, cudaStream_t stream) {
  using Kern = void (*)(const BlockNormArgs);
  // pieces per thread 1, 2, 4; wide
#define KDA_BN(x, y, o, w) \
  block_norm_kernel<x, y, o, 1, w>, block_norm_kernel<x, y, o, 2, w>, block_norm_kernel<x, y, o, 4, w>
#define KDA_BN8(w)                                                                                              \
  {                                                                                                             \
    KDA_BN(false, false, false, w), KDA_BN(false, false, true, w), KDA_BN(false, true, false, w),               \
        KDA_BN(false, true, true, w), KDA_BN(true, false, false, w), KDA_BN(true, false, true, w),              \
        KDA_BN(true, true, false, w), KDA_BN(true, true, true, w)                                               \
  }
  static const Kern table[2][24] = {KDA_BN8(false), KDA_BN8(true)};
#undef KDA_BN8
#undef KDA_BN
  const int pieces = (a.D + 7) / 8;
  int g, tpr;
  if (pieces <= 128) {  // a warp per row, four rows per CTA
    tpr = 32;
    g = pieces <= 32 ? 0 : pieces <= 64 ? 1 : 2;
  } else {
    g = pieces <= 1024 && a.rows <= 152 ? 0 : 2;
    tpr = (((pieces + (1 << g) - 1) >> g) + 31) & ~31;
  }
  a.threads_per_row = tpr;
  const int rows_per_cta = tpr == 32 ? 4 : 1;
  const unsigned grid = unsigned((a.rows + rows_per_cta - 1) / rows_per_cta);
  table[a.D % 8 == 0][12 * int(x_bf16) + 6 * int(y_bf16) + 3 * int(out_bf16) + g]<<<grid, tpr * rows_per_cta, 0,
                                                                                    stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kda
