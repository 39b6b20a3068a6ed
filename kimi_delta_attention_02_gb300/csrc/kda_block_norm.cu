// kda_block_norm.cu -- between two blocks of a residual stream, in one pass over each row of D
// channels:
//     n  = w_post (*) y / sqrt(mean(y^2) + eps)      (or n = y without the norm after the block)
//     x' = x + scale c (*) Sigmoid(r) (*) n          (r: one gate logit per channel or per row)
//     h  = w_pre (*) x' / sqrt(mean(x'^2) + eps)     (x' in fp32, before it is rounded for storage)
// Each tensor is read once and written once, the row in registers between its two sums: bound by
// HBM bandwidth, or by latency when there are few rows.
//
// A thread owns the same 8 channels of every row its CTA takes, so its weights stay in registers,
// and the next rows travel while one is summed (a barrier per sum):
//  * rows of 1032 to 8192 channels that start on 16-byte boundaries come into shared memory by bulk
//    copies, two rows ahead (one when three do not fit);
//  * other rows of up to 8192 channels are loaded into registers one row ahead;
//  * longer rows take four pieces per thread, one row per CTA, weights from L1.
//
// Measured: 4096 x 7168, fp32 stream, bf16 blocks with a gate per channel 65 us (6.4 TB/s, 95 % of the
// HBM copy rate; without shared memory 137 us); 16384 x 776 of the same 48 us, x 777 60 us (rows that
// start anywhere: 4-byte and 2-byte accesses); 8192 x 5000 in bf16 93 us; one row 7 us.
#include <atomic>

#include "kda_block_norm.h"
#include "kda_common.cuh"

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

template <bool B>
struct Bool {
  static constexpr bool value = B;
};

// Sum over the threads of a row: the warp's (or its kLanes neighbouring lanes'), then,
// with several warps per row (one row per CTA), the CTA's. `slot` keeps two sums of one row apart.
template <int kLanes = 32>
__device__ __forceinline__ float row_sum(float x, int warps, float *s_part, int slot) {
#pragma unroll
  for (int off = kLanes / 2; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  if (kLanes < 32 || warps == 1) return x;
  if ((threadIdx.x & 31) == 0) s_part[slot * 32 + (threadIdx.x >> 5)] = x;
  __syncthreads();
  const int lane = threadIdx.x & 31;
  x = lane < warps ? s_part[slot * 32 + lane] : 0.f;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
  return x;
}

// A thread's piece of a row as it was loaded: 8 neighbouring channels with kWide (16-byte accesses;
// D a multiple of 8), else 8 channels a row's threads apart. `lane`: the piece's place in the row, of
// `places`.
template <bool kBF16, bool kWide>
struct Piece {
  static constexpr int kWords = kWide && kBF16 ? 4 : 8;
  uint32_t w[kWords] = {};  // zeros past the row
  __device__ __forceinline__ void load(const void *base, int64_t row, int lane, int places, int D) {
    if constexpr (kWide) {
      if (lane * 8 < D) {
        const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(base) + (row + lane * 8) * (kBF16 ? 2 : 4));
        const uint4 a = __ldcs(p);
        w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
        if constexpr (!kBF16) {
          const uint4 b = __ldcs(p + 1);
          w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (e * places + lane < D) {  // as stored: a conversion here would wait for the load
          const int64_t at = row + e * places + lane;
          if constexpr (kBF16) w[e] = __ldcs(static_cast<const uint16_t *>(base) + at);
          else w[e] = __ldcs(static_cast<const uint32_t *>(base) + at);
        }
    }
  }
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (kWide && kBF16) return __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
    else return __uint_as_float(kBF16 ? w[e] << 16 : w[e]);
  }
};

// Rows of up to 8 x 1024 channels: threads_per_row threads with kG pieces each per row, several rows
// per CTA when a row is one warp's or less (8 or 16 lanes); CTA i takes rows i, i + grid, ... (in units of its rows).
// kG = 1: up to 768 threads, 80 registers; kG = 2: up to 512 threads, 128 registers.
template <bool kXB, bool kYB, bool kOB, int kG, bool kWide, int kLanes>
__global__ void __launch_bounds__(kG == 1 ? 768 : 512) block_norm_rows_kernel(const BlockNormArgs a) {
  __shared__ float s_part[2 * 64];
  constexpr bool kSub = kLanes < 32;  // a warp has several rows
  const int tpr = kSub ? kLanes : a.threads_per_row, warps = tpr >> 5, places = tpr * kG, D = a.D;
  const int lane = threadIdx.x % tpr;
  const int64_t first = int64_t(blockIdx.x) * (blockDim.x / tpr) + threadIdx.x / tpr;
  const int64_t stride = int64_t(gridDim.x) * (blockDim.x / tpr);
  auto channel = [&](int i, int e) { return kWide ? (i * tpr + lane) * 8 + e : e * places + i * tpr + lane; };
  auto on = [&](int i, int e) { return kWide ? (i * tpr + lane) * 8 < D : e * places + i * tpr + lane < D; };

  // scale * post_weight * channel_scale and pre_weight of this thread's channels
  float w1[kG][8], w2[kG][8];
#pragma unroll
  for (int i = 0; i < kG; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      w1[i][e] = a.scale, w2[i][e] = 1.f;
      if (on(i, e)) {
        if (a.post_weight != nullptr) w1[i][e] *= a.post_weight[channel(i, e)];
        if (a.channel_scale != nullptr) w1[i][e] *= a.channel_scale[channel(i, e)];
        if (a.pre_weight != nullptr) w2[i][e] = a.pre_weight[channel(i, e)];
      }
    }
  const bool has_y = a.y != nullptr;
  Piece<kXB, kWide> nx[kG];
  Piece<kYB, kWide> ny[kG], ng[kG];
  float next_gate = 0.f;
  auto load = [&](int64_t row) {
    if (row >= a.rows) return;  // of a warp's rows some may lie past the last one
#pragma unroll
    for (int i = 0; i < kG; ++i) {
      nx[i].load(a.x, row * D, i * tpr + lane, places, D);
      if (has_y) ny[i].load(a.y, row * D, i * tpr + lane, places, D);
      if (a.gate_form == 1) ng[i].load(a.gate, row * D, i * tpr + lane, places, D);
    }
    if (a.gate_form == 2) next_gate = load_elem<kYB>(a.gate, row);
  };
  load(first);
  int slot = 0;  // the sums alternate between two places each, so that one barrier each is enough
  const int ahead = kSub ? (threadIdx.x & 31) / tpr : 0;  // a warp's rows run together
  for (int64_t row = first; row - ahead < a.rows; row += stride, slot ^= 2) {
    float v[kG][8];
    float f = 1.f;
    if (has_y && a.post_norm) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < kG; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(ny[i][e], ny[i][e], ss);
      f = 1.f / sqrtf(row_sum<kLanes>(ss, warps, s_part, slot) / float(D) + a.post_eps);
    }
    if (has_y && a.gate_form == 2) f *= sigmoid_approx(next_gate);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < kG; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[i][e] = nx[i][e];
        if (has_y && on(i, e)) {
          float s = f * w1[i][e];
          if (a.gate_form == 1) s *= sigmoid_approx(ng[i][e]);
          v[i][e] = fmaf(s, ny[i][e], v[i][e]);
        }
        ss = fmaf(v[i][e], v[i][e], ss);
      }
    load(row + stride);  // travels while this row is summed and stored
    auto store = [&](auto kB, void *base) {
      if (kSub && row >= a.rows) return;
#pragma unroll
      for (int i = 0; i < kG; ++i) {
        if constexpr (kWide) {
          if (on(i, 0)) store8<decltype(kB)::value>(base, row * D + channel(i, 0), v[i]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (on(i, e)) store_elem<decltype(kB)::value>(base, row * D + channel(i, e), v[i][e]);
        }
      }
    };
    if (a.residual_out != nullptr) store(Bool<kXB>{}, a.residual_out);
    if (a.out != nullptr) {
      const float rstd = 1.f / sqrtf(row_sum<kLanes>(ss, warps, s_part, slot + 1) / float(D) + a.pre_eps);
#pragma unroll
      for (int i = 0; i < kG; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) v[i][e] *= rstd * w2[i][e];
      store(Bool<kOB>{}, a.out);
    }
  }
}

// One bulk copy global -> shared memory (16-byte aligned, a multiple of 16 bytes), completing on bar.
__device__ __forceinline__ void bulk_load(void *smem, const void *gmem, uint32_t bytes, uint64_t *bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(smem)),
               "l"(gmem), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

constexpr int kMaxStages = 3;

// four neighbouring elements (8-byte or 16-byte accesses)
template <bool kBF16>
__device__ __forceinline__ void load4(const void *base, int at, float *v) {
  if constexpr (kBF16) {
    const uint2 u = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(base) + at);
    const float2 a = unpack_bf16x2(u.x), b = unpack_bf16x2(u.y);
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
  } else {
    const float4 a = *reinterpret_cast<const float4 *>(static_cast<const float *>(base) + at);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  }
}
template <bool kBF16>
__device__ __forceinline__ void store4(void *base, int64_t at, const float *v) {
  if constexpr (kBF16)
    __stcs(reinterpret_cast<uint2 *>(static_cast<uint16_t *>(base) + at),
           make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])));
  else __stcs(reinterpret_cast<float4 *>(static_cast<float *>(base) + at), make_float4(v[0], v[1], v[2], v[3]));
}

// Rows that pass through shared memory (D a multiple of 8), one at a time per CTA; a.stages rows are in
// shared memory, a.stages - 1 of them ahead. A thread owns the channels 4 t .. + 3 and 4 (t + threads)
// .. + 3, so that a warp's accesses of either type are contiguous.
template <bool kXB, bool kYB, bool kOB>
__global__ void __launch_bounds__(1024) block_norm_piped_kernel(const BlockNormArgs a, uint32_t *err_word) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float s_part[64];
  __shared__ uint64_t full[kMaxStages];
  const int tid = threadIdx.x, warps = blockDim.x >> 5, D = a.D;
  const int c[2] = {4 * tid, 4 * (tid + int(blockDim.x))};
  const bool on[2] = {c[0] < D, c[1] < D}, has_y = a.y != nullptr, has_g = a.gate_form == 1;
  const uint32_t xb = uint32_t(D) * (kXB ? 2 : 4), yb = uint32_t(D) * (kYB ? 2 : 4);
  const uint32_t stage_bytes = xb + (has_y ? yb : 0) + (has_g ? yb : 0);
  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) mbar_init(&full[i], 1);
    fence_mbarrier_init();
  }
  auto issue = [&](int64_t row, int stage) {  // by thread 0
    uint8_t *dst = smem + stage * stage_bytes;
    mbar_arrive_expect_tx(&full[stage], stage_bytes);
    bulk_load(dst, static_cast<const uint8_t *>(a.x) + row * xb, xb, &full[stage]);
    if (has_y) bulk_load(dst + xb, static_cast<const uint8_t *>(a.y) + row * yb, yb, &full[stage]);
    if (has_g) bulk_load(dst + xb + yb, static_cast<const uint8_t *>(a.gate) + row * yb, yb, &full[stage]);
  };
  const int64_t stride = gridDim.x;
  int in_flight = 0;  // thread 0: copies of rows not waited for yet
  if (tid == 0)
    for (; in_flight + 1 < a.stages && blockIdx.x + in_flight * stride < a.rows; ++in_flight)
      issue(blockIdx.x + in_flight * stride, in_flight);
  float w1[8], w2[8];  // scale * post_weight * channel_scale, pre_weight
#pragma unroll
  for (int e = 0; e < 8; ++e) w1[e] = a.scale, w2[e] = 1.f;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (!on[i]) continue;
    float t[4];
    if (a.post_weight != nullptr) {
      load4<false>(a.post_weight, c[i], t);
#pragma unroll
      for (int e = 0; e < 4; ++e) w1[4 * i + e] *= t[e];
    }
    if (a.channel_scale != nullptr) {
      load4<false>(a.channel_scale, c[i], t);
#pragma unroll
      for (int e = 0; e < 4; ++e) w1[4 * i + e] *= t[e];
    }
    if (a.pre_weight != nullptr) load4<false>(a.pre_weight, c[i], w2 + 4 * i);
  }
  __syncthreads();  // the barriers are initialised
  int stage = 0, parity = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += stride) {
    const bool ok = mbar_wait(&full[stage], uint32_t(parity), err_word, DEVERR_TMA_TIMEOUT);
    // all threads leave together; and all are done with the row before, whose place the copy of a
    // later row may take
    if (__syncthreads_or(!ok)) break;
    const int64_t ahead = row + int64_t(a.stages - 1) * stride;
    if (tid == 0) {
      --in_flight;
      if (ahead < a.rows) {
        issue(ahead, stage == 0 ? a.stages - 1 : stage - 1);
        ++in_flight;
      }
    }
    const uint8_t *src = smem + stage * stage_bytes;
    if (++stage == a.stages) stage = 0, parity ^= 1;

    float f = 1.f, v[8], y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = y[e] = 0.f;
    if (has_y) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (on[i]) load4<kYB>(src + xb, c[i], y + 4 * i);
      if (a.post_norm) {
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
        f = 1.f / sqrtf(row_sum(ss, warps, s_part, 0) / float(D) + a.post_eps);
      }
      if (a.gate_form == 2) f *= sigmoid_approx(load_elem<kYB>(a.gate, row));
    }
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if (!on[i]) continue;
      load4<kXB>(src, c[i], v + 4 * i);
      if (has_y) {
        float g[4] = {1.f, 1.f, 1.f, 1.f};
        if (has_g) {
          load4<kYB>(src + xb + yb, c[i], g);
#pragma unroll
          for (int e = 0; e < 4; ++e) g[e] = sigmoid_approx(g[e]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * i + e] = fmaf(f * w1[4 * i + e] * g[e], y[4 * i + e], v[4 * i + e]);
      }
      if (a.residual_out != nullptr) store4<kXB>(a.residual_out, row * D + c[i], v + 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) ss = fmaf(v[4 * i + e], v[4 * i + e], ss);
    }
    if (a.out != nullptr) {
      const float rstd = 1.f / sqrtf(row_sum(ss, warps, s_part, 1) / float(D) + a.pre_eps);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (!on[i]) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[4 * i + e] *= rstd * w2[4 * i + e];
        store4<kOB>(a.out, row * D + c[i], v + 4 * i);
      }
    }
  }
  // left early: the copies still in flight land before the CTA ends
  for (; tid == 0 && in_flight > 0; --in_flight) {
    mbar_wait(&full[stage], uint32_t(parity), err_word, DEVERR_TMA_TIMEOUT);
    if (++stage == a.stages) stage = 0, parity ^= 1;
  }
}

// Longer rows, one per CTA: a thread holds kG pieces of 8 channels.
template <bool kXB, bool kYB, bool kOB, bool kWide>
__global__ void __launch_bounds__(512) block_norm_long_kernel(const BlockNormArgs a) {
  constexpr int kG = 4;
  __shared__ float s_part[64];
  const int tpr = a.threads_per_row, warps = tpr >> 5;
  const int lane = threadIdx.x;
  const int64_t row = blockIdx.x;
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
#define KDA_BN8(kern, ...)                                                                        \
  {                                                                                               \
    kern<false, false, false, __VA_ARGS__>, kern<false, false, true, __VA_ARGS__>,                \
        kern<false, true, false, __VA_ARGS__>, kern<false, true, true, __VA_ARGS__>,              \
        kern<true, false, false, __VA_ARGS__>, kern<true, false, true, __VA_ARGS__>,              \
        kern<true, true, false, __VA_ARGS__>, kern<true, true, true, __VA_ARGS__>                 \
  }
  static const Kern rows_kernel[4][2][8] = {  // 8 or 16 lanes a row, warps with one and two pieces a thread
      {KDA_BN8(block_norm_rows_kernel, 1, false, 8), KDA_BN8(block_norm_rows_kernel, 1, true, 8)},
      {KDA_BN8(block_norm_rows_kernel, 1, false, 16), KDA_BN8(block_norm_rows_kernel, 1, true, 16)},
      {KDA_BN8(block_norm_rows_kernel, 1, false, 32), KDA_BN8(block_norm_rows_kernel, 1, true, 32)},
      {KDA_BN8(block_norm_rows_kernel, 2, false, 32), KDA_BN8(block_norm_rows_kernel, 2, true, 32)}};
  static const Kern long_kernel[2][8] = {KDA_BN8(block_norm_long_kernel, false), KDA_BN8(block_norm_long_kernel, true)};
#undef KDA_BN8
  const int wide = a.D % 8 == 0, types = 4 * int(x_bf16) + 2 * int(y_bf16) + int(out_bf16);
  const int pieces = (a.D + 7) / 8;
  if (pieces > 1024) {
    a.threads_per_row = ((pieces + 3) / 4 + 31) & ~31;
    long_kernel[wide][types]<<<unsigned(a.rows), a.threads_per_row, 0, stream>>>(a);
    return cudaGetLastError();
  }
  constexpr int kSMs = 152;
  if (wide && pieces > 128) {
    using Piped = void (*)(const BlockNormArgs, uint32_t *);
    static const Piped piped[8] = {
        block_norm_piped_kernel<false, false, false>, block_norm_piped_kernel<false, false, true>,
        block_norm_piped_kernel<false, true, false>,  block_norm_piped_kernel<false, true, true>,
        block_norm_piped_kernel<true, false, false>,  block_norm_piped_kernel<true, false, true>,
        block_norm_piped_kernel<true, true, false>,   block_norm_piped_kernel<true, true, true>};
    constexpr int kMaxSmem = 224 * 1024;
    const int ex = x_bf16 ? 2 : 4, ey = y_bf16 ? 2 : 4;
    const int row_bytes = a.D * (ex + (a.y != nullptr ? ey : 0) + (a.gate_form == 1 ? ey : 0));
    const int threads = (a.D / 8 + 31) & ~31;
    a.stages = row_bytes * kMaxStages <= kMaxSmem ? kMaxStages : 2;
    const int smem = row_bytes * a.stages;
    int per_sm = 2048 / threads < kMaxSmem / (smem + 1024) ? 2048 / threads : kMaxSmem / (smem + 1024);
    if (per_sm > 1024 / threads) per_sm = 1024 / threads;  // 64 registers per thread
    if (per_sm < 1) per_sm = 1;
    static std::atomic<uint64_t> granted[8];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (bit == 0 || (granted[types].load(std::memory_order_acquire) & bit) == 0) {
      e = cudaFuncSetAttribute(piped[types], cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
      if (e != cudaSuccess) return e;
      granted[types].fetch_or(bit, std::memory_order_release);
    }
    const int64_t fit = int64_t(kSMs) * per_sm;
    piped[types]<<<unsigned(a.rows < fit ? a.rows : fit), threads, smem, stream>>>(a, device_error_word());
    return cudaGetLastError();
  }
  const int two = pieces > 768, threads_per_sm = two ? 512 : 768;
  // (37395 rows of 80 channels: 17 us with 16 lanes a row, 23 with a warp; odd rows, bf16, of 777 and 2047
  // channels reach 3.3 and 2.2 TB/s, rows of 776 and 2048 4.3 and 3.3)
  const int kind = pieces <= 8 ? 0 : pieces <= 16 ? 1 : two ? 3 : 2;
  a.threads_per_row = kind < 2 ? 8 << kind : ((two ? (pieces + 1) / 2 : pieces) + 31) & ~31;
  const int rows_per_cta = a.threads_per_row <= 32 ? 256 / a.threads_per_row : 1, threads = a.threads_per_row * rows_per_cta;
  const int64_t need = (a.rows + rows_per_cta - 1) / rows_per_cta, fit = int64_t(kSMs) * (threads_per_sm / threads);
  rows_kernel[kind][wide][types]<<<unsigned(need < fit ? need : fit), threads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kda
