// kda_delta_plan.cu -- how a prefill of the gated delta rule is cut (host), and the kernel that chains the
// segments' states.
#include <atomic>

#include "kda_delta.cuh"

namespace kda {
namespace {

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

constexpr int kChainCols = 16, kChainThreads = 256, kChainStride = 132;  // (floats per row of M: conflict-free)
constexpr int kChainBytes = (2 * 128 * kChainStride + 128 * kChainCols) * 4;

// Pass 2: E_{j+1} = M_j E_j + B_j for the segments between a sequence's first and last, in fp32. The
// first segment's end state is E_1; B_j gives way to E_{j+1}. The CTAs of a sequence's first segment
// (blockIdx.y is the piece) walk its segments, 16 value columns each: thread (rg, cg) forms rows rg, rg + 32,
// .. of columns 2 cg, + 1, with E and M in shared memory and the next M on its way (5 us a step; 13 us with
// M read through L1 as it is used).
__global__ void __launch_bounds__(kChainThreads) delta_chain_kernel(const DeltaArgs a) {
  extern __shared__ __align__(16) float chain_smem[];
  float *const E = chain_smem + 2 * 128 * kChainStride;  // [128][16]
  LinearSlot s;
  if (!linear_slot(a.cu, a.num_seqs, a.plan.seg_len, a.plan.inner, blockIdx.y, s) || !s.first) return;
  const int segs = (a.cu[s.n + 1] - a.cu[s.n] - 1) / a.plan.seg_len + 1;
  const int h = blockIdx.x % a.H, cg = threadIdx.x & 7, rg = threadIdx.x >> 3;
  const int c = int(blockIdx.x) / a.H * kChainCols + 2 * cg;
  const int64_t place = delta_place(a, s);
  float *ends = reinterpret_cast<float *>(a.workspace + a.plan.ends);
  const float *maps = reinterpret_cast<const float *>(a.workspace + a.plan.maps);
  const int pk = delta_up8(a.d_k), pv = delta_up8(a.d_v);
  auto at = [&](int64_t p, int r) { return ends + ((p * a.H + h) * pk + r) * pv + c; };
  auto fetch = [&](int j) {  // M_j; one group of copies per call, also where there is none
    if (j + 1 < segs) {
      const float *M = maps + ((place + j) * a.H + h) * int64_t(pk) * pk;
      const int per_row = pk >> 2;
      for (int i = threadIdx.x; i < a.d_k * per_row; i += kChainThreads) {
        const int r = i / per_row, k = i % per_row * 4;
        cp_async_16_zfill(&chain_smem[(j & 1) * 128 * kChainStride + r * kChainStride + k], M + i * 4, true);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto on = [&](int i) { return rg + 32 * i < a.d_k && c < a.d_v; };  // (an odd d_v's last pair is in the row: pv)
  fetch(1);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = on(i) ? *reinterpret_cast<const float2 *>(at(place, rg + 32 * i)) : make_float2(0.f, 0.f);
    *reinterpret_cast<float2 *>(&E[(rg + 32 * i) * kChainCols + 2 * cg]) = x;
  }
  for (int j = 1; j + 1 < segs; ++j) {
    fetch(j + 1);
    float2 acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc[i] = on(i) ? *reinterpret_cast<const float2 *>(at(place + j, rg + 32 * i)) : make_float2(0.f, 0.f);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    const float *M = chain_smem + (j & 1) * 128 * kChainStride + rg * kChainStride;
#pragma unroll 4
    for (int k = 0; k < pk; k += 4) {  // (behind d_k, M's columns and E's rows are zero)
      float2 x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = *reinterpret_cast<const float2 *>(&E[(k + e) * kChainCols + 2 * cg]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (rg + 32 * i >= a.d_k) break;
        const float4 m = *reinterpret_cast<const float4 *>(&M[32 * i * kChainStride + k]);
        acc[i] = f2_fma(make_float2(m.x, m.x), x[0], acc[i]);
        acc[i] = f2_fma(make_float2(m.y, m.y), x[1], acc[i]);
        acc[i] = f2_fma(make_float2(m.z, m.z), x[2], acc[i]);
        acc[i] = f2_fma(make_float2(m.w, m.w), x[3], acc[i]);
      }
    }
    __syncthreads();  // every thread is past E and M before they are overwritten
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      *reinterpret_cast<float2 *>(&E[(rg + 32 * i) * kChainCols + 2 * cg]) = acc[i];
      if (on(i)) *reinterpret_cast<float2 *>(at(place + j, rg + 32 * i)) = acc[i];
    }
  }
}

}  // namespace

cudaError_t launch_delta_chain(const DeltaArgs &a, cudaStream_t stream) {
  static std::atomic<uint64_t> granted;  // as in the other kernels
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (bit == 0 || (granted.load(std::memory_order_acquire) & bit) == 0) {
    e = cudaFuncSetAttribute(delta_chain_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kChainBytes);
    if (e != cudaSuccess) return e;
    granted.fetch_or(bit, std::memory_order_release);
  }
  const dim3 grid(unsigned(a.H * ((a.d_v + kChainCols - 1) / kChainCols)), unsigned(a.plan.inner));
  delta_chain_kernel<<<grid, kChainThreads, kChainBytes, stream>>>(a);
  return cudaGetLastError();
}

// The tensor-core kernel takes a chunk of 64 tokens' time for the shortest sequence, so calls of short ones go
// to the token kernel: below `least` tokens a sequence on average. us by the token kernel / this one at 8, 16,
// 32, 64 and 100 tokens; 16 sequences of 64 heads: 128 x 128 103/93, 132/93, 198/94, 326/97; 64 x 128 70/86, 86/86,
// 133/88; 128 x 64 54/90, 70/90, 106/92, 172/93; 64 x 64, where a warp holds a whole state, 36/84, 43/84,
// 66/85, 111/86. Fewer chains than SMs (3 sequences of 8 heads): 128 x 128 9/15, 11/15, 13/15, 19/15; 64 x 64
// 7/14, 7/14, 9/14, 13/13, 17/17. TMA needs rows of whole 16-byte pieces, so other head sizes run on padded
// copies of q, k and v in the workspace, or without one in the token kernel (4096 tokens, 96 heads of 100: 348 us
// by copies, 2087 by the token kernel; 32 heads of 68: 215, 828).
//
// Few key channels stay in the token kernel, for the precision: random keys of a chunk are far from orthogonal, so
// that T' V and T'' X are larger than their sum, and their pairs' roundings reach 1.1e-5 of fp32 outputs and 1.0e-5 of
// states in the 2-norm (d_k = 5 and 6; from 9 on 8.3e-6 of states, from 17 on 9.1e-6 of outputs; 3e-7 by the token
// kernel). 4096 tokens, 96 heads of 16 x 128: 1197 us there, 237 here. It is a rule for random keys: ones that share a
// direction are no more orthogonal in 128 channels than in few, and come to 3e-5 of outputs and 2e-5 of states at any d_k.
//
// The shortest sequences go to the decode kernel, which holds no more than a state and is bound by its bytes, where
// there are more chains than SMs and the mean length says that there may be some: those of up to `few` tokens. us
// by the token kernel / that one at 1, 4, 8 and 16 tokens, 128 sequences of 64 heads: 128 x 128 754/219, 764/468,
// 798/808, 1019/1499 (the tensor cores: 651); 64 x 64 250/72, 252/121, 277/195, 336/347 (597 by the tensor cores).
//
// A CTA holds one (sequence, head) from end to end, one CTA per SM, so few long sequences leave SMs idle. A
// sequence cut into m segments runs 2 m - 3 of them side by side in pass 1 and m - 1 in pass 3: two segments'
// time instead of m, for up to three times the work. Of a single sequence m is that of the least time by
// waves of CTAs: a chunk of 64 tokens takes some 4 us, a step of pass 2 five, a pass ten to begin and end (T =
// 65536, 16 heads: m = 10, 1268 us; m = 6: 1354 us; not cut: 3870). Of several the lengths are not known
// here, and cuts lie so far apart that pass 1 fills the SMs at most twice. Sequences in more chains than SMs run
// longest first.
DeltaPlan delta_plan(int64_t total, int num_seqs, int H, int H_k, int d_k, int d_v, bool in_bf16, bool out_bf16,
                     bool recurrent, size_t workspace_bytes) {
  DeltaPlan p;
  const bool idle = int64_t(num_seqs) * H <= kLinearSMs;
  const int64_t least = d_k <= 64 && d_v <= 64 ? (idle ? 88 : 44) : idle ? 44 : d_v <= 64 ? 24 : d_k <= 64 ? 16 : 6;
  if (!recurrent && !idle && total < 64 * int64_t(num_seqs)) p.few = d_k <= 64 && d_v <= 64 ? 12 : 5;
  p.tensor = in_bf16 && !recurrent && d_k > (out_bf16 ? 8 : 16) && total >= least * num_seqs &&
             int64_t(H) * d_v <= 1 << 25;  // (its output addresses)
  const int pk = delta_up8(d_k), pv = delta_up8(d_v);
  const auto room = [&](int64_t len) {  // for cuts of this length
    const int64_t inner = total / len;
    const size_t ends = align256(size_t(inner) * H * pk * pv * 4), maps = align256(size_t(inner) * H * pk * pk * 4);
    if (p.bytes + ends + maps > workspace_bytes) return false;
    p.seg_len = int32_t(len), p.inner = int32_t(inner);
    p.maps = p.ends + ends;
    p.bytes += ends + maps;
    return true;
  };
  if (!p.tensor) {
    // One long sequence in the token kernel, where the cuts save a fifth at least. ns a token by CTAs of 32 columns:
    // with 38 of them, 76, 152 and more, in segments (a tenth less in one run). T = 16384, fp32, heads of 128: 1 head
    // 1405 us in one run, 572 in segments; 4 heads 1405, 1301; 16 heads 2245, 3808; 8 heads of 64 1400, 712.
    if (!recurrent && num_seqs == 1) {
      const auto ns = [&](int64_t ctas) -> int64_t {
        return ctas <= kLinearSMs / 4 ? 95 : ctas <= kLinearSMs / 2 ? 145 : ctas * 135 / 100 > 236 ? ctas * 135 / 100 : 236;
      };
      const int64_t tv = (d_v + 31) / 32, tk = (pk + 31) / 32;
      int64_t best = total * ns(tv * H) * 4 / 5, len = 0;
      for (int64_t m = 3; m <= 64 && total >= m * 128; ++m) {
        const int64_t each = (total + m - 1) / m;
        const int64_t time = each * (ns(((m - 1) * tv + (m - 2) * tk) * H) + ns((m - 1) * tv * H)) + 30000 + 6000 * m;
        if (time < best) best = time, len = each;
      }
      if (len > 0) room(len);
    }
    return p;
  }
  if (pk != d_k || pv != d_v) {
    const size_t qk = pk != d_k ? align256(size_t(total) * H_k * pk * 2) : 0;
    p.pad_k = qk, p.pad_v = 2 * qk;
    p.bytes = p.ends = p.pad_v + (pv != d_v ? align256(size_t(total) * H * pv * 2) : 0);
    p.pad = p.bytes <= workspace_bytes;
    if (!p.pad) {
      DeltaPlan token;
      token.few = p.few;
      return token;
    }
  }
  int64_t len = 0;
  if (num_seqs == 1) {
    const auto waves = [&](int64_t pieces) { return (pieces * H + kLinearSMs - 1) / kLinearSMs; };
    int64_t best = total / 64 * 4 * waves(1);
    for (int64_t m = 3; m <= 64 && total >= m * 512; ++m) {
      const int64_t us = (waves(2 * m - 3) + waves(m - 1)) * (total / (m * 64) * 4 + 10) + 5 * m;
      if (us < best) best = us, len = (total + m - 1) / m;
    }
  } else {
    len = (2 * total * H + kLinearSMs - 1) / kLinearSMs;
  }
  len = (len + 63) / 64 * 64;
  if (len > 0 && len < 512) len = 512;
  // (room for three segments; and cuts that most sequences are too short for would only cost the order of the
  // others: 301 us instead of 273 for prompts of 4096 tokens and less on 32 heads, cut at 4672)
  if (len > 0 && total >= 3 * len - 63 * 3 && 8 * total >= len * num_seqs) {
    if (room(len)) return p;
  }
  const size_t list = align256(size_t(num_seqs) * 4);
  if (num_seqs > 1 && num_seqs <= 8192 && !idle && p.bytes + list <= workspace_bytes) {
    p.order = true;
    p.bytes += list;
  }
  return p;
}

}  // namespace kda
