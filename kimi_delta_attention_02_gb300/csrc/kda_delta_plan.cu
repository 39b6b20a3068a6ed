// kda_delta_plan.cu -- how a prefill of the gated delta rule is cut (host), and the kernel that chains the
// segments' states.
#include "kda_delta.cuh"

namespace kda {
namespace {

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

constexpr int kChainCols = 32, kChainThreads = 256;

// Pass 2: E_{j+1} = M_j E_j + B_j for the segments between a sequence's first and last, in fp32. The
// first segment's end state is E_1; B_j gives way to E_{j+1}. The CTAs of a sequence's first segment
// (blockIdx.y is the piece) walk its segments, 32 value columns each: thread (rg, cg) forms rows
// 4 rg .. + 3 of columns 4 cg .. + 3, E in shared memory, M through L1.
__global__ void __launch_bounds__(kChainThreads) delta_chain_kernel(const DeltaArgs a) {
  __shared__ __align__(16) float E[128][kChainCols];
  LinearSlot s;
  if (!linear_slot(a.cu, a.num_seqs, a.plan.seg_len, a.plan.inner, blockIdx.y, s) || !s.first) return;
  const int segs = (a.cu[s.n + 1] - a.cu[s.n] - 1) / a.plan.seg_len + 1;
  const int h = blockIdx.x % a.H, c = int(blockIdx.x) / a.H * kChainCols + 4 * (threadIdx.x & 7);
  const int rg = threadIdx.x >> 3, r0 = 4 * rg, cs = 4 * (threadIdx.x & 7);
  const bool ok = c < a.d_v && r0 < a.d_k;  // (d_k and d_v are multiples of 8)
  const int64_t place = delta_place(a, s);
  float *ends = reinterpret_cast<float *>(a.workspace + a.plan.ends);
  const float *maps = reinterpret_cast<const float *>(a.workspace + a.plan.maps);
  auto at = [&](int64_t p, int r) { return ends + ((p * a.H + h) * a.d_k + r) * a.d_v + c; };
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (ok) *reinterpret_cast<float4 *>(&E[r0 + i][cs]) = *reinterpret_cast<const float4 *>(at(place, r0 + i));
  for (int j = 1; j + 1 < segs; ++j) {
    __syncthreads();
    const float *M = maps + ((place + j) * a.H + h) * int64_t(a.d_k) * a.d_k + r0 * a.d_k;
    float4 acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc[i] = ok ? *reinterpret_cast<const float4 *>(at(place + j, r0 + i)) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int k = 0; k < a.d_k; k += 4) {
      float4 m[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        m[i] = ok ? *reinterpret_cast<const float4 *>(M + i * a.d_k + k) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float4 x = *reinterpret_cast<const float4 *>(&E[k + e][cs]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y = e == 0 ? m[i].x : e == 1 ? m[i].y : e == 2 ? m[i].z : m[i].w;
          acc[i].x = fmaf(y, x.x, acc[i].x), acc[i].y = fmaf(y, x.y, acc[i].y);
          acc[i].z = fmaf(y, x.z, acc[i].z), acc[i].w = fmaf(y, x.w, acc[i].w);
        }
      }
    }
    __syncthreads();  // every thread is past E before it is overwritten
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (ok) {
        *reinterpret_cast<float4 *>(&E[r0 + i][cs]) = acc[i];
        *reinterpret_cast<float4 *>(at(place + j, r0 + i)) = acc[i];
      }
  }
}

}  // namespace

cudaError_t launch_delta_chain(const DeltaArgs &a, cudaStream_t stream) {
  const dim3 grid(unsigned(a.H * ((a.d_v + kChainCols - 1) / kChainCols)), unsigned(a.plan.inner));
  delta_chain_kernel<<<grid, kChainThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

// A CTA of the tensor-core kernel holds one (sequence, head) from end to end, one CTA per SM, so few long
// sequences leave SMs idle. A sequence cut into m segments runs 2 m - 3 of them side by side in pass 1 and
// m - 1 in pass 3: two segments' time instead of m, for up to three times the work. Of a single sequence
// m is the largest that fits; of several the lengths are not known here, and cuts lie so far apart that
// pass 1 fills the SMs at most twice. Sequences in more chains than SMs run longest first.
DeltaPlan delta_plan(int64_t total, int num_seqs, int H, int d_k, int d_v, bool in_bf16, bool out_bf16, bool recurrent,
                     size_t workspace_bytes) {
  DeltaPlan p;
  // TMA addresses rows of a multiple of 16 bytes
  const int64_t least = d_k <= 64 && d_v <= 64 ? 44 : d_k <= 64 || d_v <= 64 ? 16 : 6;
  p.tensor = in_bf16 && !recurrent && d_k % 8 == 0 && d_v % 8 == 0 && total >= least * num_seqs &&
             int64_t(H) * d_v <= 1 << 25;  // (its output addresses)
  if (!p.tensor) return p;
  (void)out_bf16;
  int64_t len = 0;
  if (num_seqs == 1) {
    const int64_t m = (kLinearSMs / H + 3) / 2;
    if (m >= 3) len = (total + m - 1) / m;
  } else {
    len = (2 * total * H + kLinearSMs - 1) / kLinearSMs;
  }
  len = (len + 63) / 64 * 64;
  if (len > 0 && len < 512) len = 512;
  if (len > 0 && total >= 3 * len - 63 * 3 && 8 * total >= len * num_seqs) {
    const int64_t inner = total / len;
    const size_t ends = align256(size_t(inner) * H * d_k * d_v * 4), maps = align256(size_t(inner) * H * d_k * d_k * 4);
    if (ends + maps <= workspace_bytes) {
      p.seg_len = int32_t(len);
      p.inner = int32_t(inner);
      p.maps = ends;
      p.bytes = ends + maps;
      return p;
    }
  }
  const size_t list = align256(size_t(num_seqs) * 4);
  if (num_seqs > 1 && num_seqs <= 8192 && int64_t(num_seqs) * H > kLinearSMs && list <= workspace_bytes) {
    p.order = true;
    p.bytes = list;
  }
  return p;
}

}  // namespace kda
