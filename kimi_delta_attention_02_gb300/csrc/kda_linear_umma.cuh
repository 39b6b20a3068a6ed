// kda_linear_umma.cuh -- what the tensor-core kernels of linear attention and of the gated delta rule
// share beside kda_common.cuh: MMAs issued by one elected lane of a whole warp, tile descriptors, and
// some small device functions.
#pragma once

#include <cuda.h>

#include "kda_common.cuh"

namespace kda {
namespace {

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float *v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "f"(v[0]),
               "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap *map, int32_t x, int32_t y, int32_t z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map), "r"(x), "r"(y), "r"(z)
               : "memory");
}

// An MMA warp runs as a whole, so that descriptors stay in uniform registers (a lone lane has to
// move each one there), and its elected lane alone issues.
__device__ __forceinline__ bool elect_lane() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(p));
  return p != 0;
}
//   D[tmem] (+)= A[smem] x B[smem], bf16
__device__ __forceinline__ void mma_ss(bool leader, uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(uint32_t(leader))
      : "memory");
}
//   D[tmem] (+)= A[tmem] x B[smem]: A's row m in lane m, two elements of K per 32-bit column
__device__ __forceinline__ void mma_ts(bool leader, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n setp.ne.b32 q, %5, 0;\n"
      " @q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(uint32_t(leader))
      : "memory");
}
__device__ __forceinline__ void mma_commit(bool leader, uint64_t &bar) {
  asm volatile(
      "{\n .reg .pred q;\n setp.ne.b32 q, %1, 0;\n"
      " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(&bar)),
      "r"(uint32_t(leader))
      : "memory");
}

// K-major tile (128-byte rows of 64 elements, 8-row atoms); MN-major tile with `lbo` between its
// 64-element blocks.
__device__ __forceinline__ uint64_t desc_k(uint32_t addr) { return umma_desc(addr, 16, 1024, kSwizzle128B); }
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr, uint32_t lbo) {
  return umma_desc(addr, lbo, 1024, kSwizzle128B);
}

}  // namespace
}  // namespace kda
