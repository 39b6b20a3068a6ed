// kda_linear_chunked.cu -- linear attention with one decay per head on the tensor cores (bf16
// inputs): S_t = e^{g_t} S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t, in chunks of 128 tokens. Rows of
// q, k and v are multiples of 16 bytes (the launch pads copies of others).
//
// With G the cumulative log-decay inside a chunk and S the state that enters it,
//     O  = (D (*) Q K^T) V + diag(e^G) Q S,      D_ij = e^{G_i - G_j} for j <= i, else 0,
//     S <- e^{G_C} S + K^T V',                   V'_j = e^{G_C - G_j} v_j .
// All four products are tcgen05 MMAs with fp32 accumulators in tensor memory; the state itself
// stays in fp32 registers. One CTA owns one segment of one (sequence, head) and kDV value columns.
//
// Roundings. P = D (*) Q K^T and the state enter their products as bf16 (each off by at most 2^-8
// of the value, like the bf16 output they end in); with an fp32 output they enter as a bf16 pair
// hi + lo (2^-16). V' is always such a pair, because the fp32 state adds it up over the whole sequence.
//
// Decays. A chunk has four blocks of 32 tokens. a_i is the sum of g from its block's start to i,
// s_j from behind j to its block's end, t_B a whole block's (log2 units). Then e^{G_i - G_j} is
// 2^{a_i - a_j} within a block and 2^{a_i + t_{J+1} + ... + t_{I-1}} 2^{s_j} across: no factor is
// the difference of two long sums, none exceeds one while g <= 0, and only the diagonal blocks
// take an exponential per entry, of a difference of two sums a. Each sum is made in five levels: off by
// at most 5 x 2^-24 of itself, and 2^-24 for its terms' own roundings, so their difference is off by
// 11 x 2^-24 x ln 2 of the block's sum: less than 2^-16 while its 32 tokens decay by 2^-32 or less. In a block that
// decays by more every entry takes its own sum if the output is fp32 (T = 4096, 96 heads of 128 that
// all do: 255 us, 218 without); a bf16 output bears the difference (sums up to 32 x 127, off by at
// most 2^-9, seen 2^-10.4, next to P's 2^-8; without the branch the loop is 4 % faster). A decay below
// 2^-127 per token counts as 2^-127, which leaves nothing in fp32 either unless a state of 2^100 entered it
// or growth follows (up to e^40 by the header, so e^-48 is left), so g = -infinity needs no case of its own.
//
// Shared memory holds five 32 KB buffers that the chunks' tiles take in turn, Q V K Q V K ..., so that
// a tile waits for the one five places before it: Q of chunk n for V of n - 2, V for K of n - 2, K for
// Q of n - 1. The output needs no buffer: it goes from tensor memory through registers to global
// memory, 32 bytes (a whole sector) per thread and store. The states come and go through the place of
// their own bf16 tile.
//
// Pass 1 of a segmented call (kStateOnly) forms a segment's end state from zero, sum over its chunks of
// e^(decay behind the chunk) K^T V', last chunk first: once that factor is below 2^-127, and so zero in
// fp32, no earlier token leaves anything and the rest of the segment is not read. (With a positive g
// before, some would be left: the header counts what enters a run of tokens that sums below -87 as forgotten.)
//
// Warps (20): 0 loads (TMA), 1 issues the MMAs Q K^T, Q S, P V, 2 makes the decay tables, 3 issues
// K^T V' (on its own, so that either's waits are filled by the other's work), 4-7 form P (one
// query row per thread, in place in tensor memory: P is the A operand of its product), 8-11 convert
// V to V' in quarters of 32 tokens, 12-19 keep the state (one key row and half the columns per
// thread) and write the output (one token and half the columns). Per chunk the tensor pipe runs
// Q K^T, K^T V' (hi, lo), P V, Q S: 2560 cycles for 128 value columns; everything else runs beside.
//
// Measured (bf16, d = 128): T = 4096, 96 heads 109 us (3.8 TB/s, 57 % of the HBM copy rate, on the 96
// SMs that have a chain; tensor pipe 63 % busy there); T = 65536, 16 heads 290 us (3.7 TB/s); 64 prompts
// of 40 to 250 tokens, 16 heads 93 us. What bounds a chunk is the way from one state to the next (D to
// registers, the bf16 tile, Q S, P V, the output), 3.3 us, against 1.3 us of MMAs and 1.9 us of HBM
// traffic with 96 SMs at it; the output's row-per-thread stores keep the load/store pipe for a third of it.
#include <atomic>

#include "kda_linear.cuh"
#include "kda_tma_host.h"

namespace kda {
namespace {

constexpr int kC = 128;            // tokens per chunk
constexpr int kThreads = 640;
constexpr uint32_t kBuf = 32768;   // 128 tokens x 128 channels bf16, two 64-channel blocks
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kMinLog2 = -127.f;
constexpr uint32_t kProbes = 2000000;
constexpr float kFarLog2 = -32.f;  // of a block's 32 tokens

template <int kDV, bool kOutBF16, bool kStateOnly>
struct Cfg {
  static constexpr bool kPair = !kOutBF16 && !kStateOnly;  // P and S as hi + lo
  static constexpr int kBufs = kStateOnly ? 4 : 5;         // pass 1: K V K V
  static constexpr uint32_t kTileV = 256u * kDV;
  static constexpr uint32_t kTileS = 256u * kDV;                    // 128 key rows x kDV bf16; stages states too
  static constexpr uint32_t kTileVP = 64u * kDV;                    // a quarter of V': 32 tokens
  static constexpr uint32_t oS = kBufs * kBuf, oVP = oS + (kPair ? 2 : 1) * kTileS, oTab = oVP + 4 * kTileVP;
};

// The buffers of chunk n's tiles (tile i of the call in buffer i mod 5, in pass 1 i mod 4); step()
// goes to the next chunk.
template <bool kStateOnly>
struct Bufs {
  static constexpr uint32_t kBufs = kStateOnly ? 4 : 5;
  uint32_t first = 0;
  __device__ __forceinline__ uint32_t at(uint32_t i) const {
    const uint32_t b = first + i;
    return (b >= kBufs ? b - kBufs : b) * kBuf;
  }
  __device__ __forceinline__ uint32_t Q() const { return at(0); }
  __device__ __forceinline__ uint32_t K() const { return at(kStateOnly ? 0 : 2); }
  __device__ __forceinline__ uint32_t V() const { return at(1); }
  __device__ __forceinline__ void step() {
    first += kStateOnly ? 2 : 3;
    if (first >= kBufs) first -= kBufs;
  }
};

struct Table {  // decays of one chunk, log2 units unless said otherwise
  float a[kC];       // from the block's start to the token, itself included
  float es[96];      // 2^(from behind the token to the block's end), blocks 0 .. 2
  uint32_t f[kC];    // e^{G_C - G_j} as a pair: the nearest bf16 (low half), what is left
  float e1;          // e^{G_C} - 1, or e^{G_C} below one half; in pass 1 e^(everything behind the chunk)
  float keep;        // 1 or 0: how often the state itself is added to e1 times the state (see Decay)
  uint32_t stop;     // pass 1: no chunk before this one leaves anything
  float pad;
  __device__ __forceinline__ float block(int B) const { return a[32 * B + 31]; }
};
static_assert(sizeof(Table) % 16 == 0, "128-bit reads of the second table");

struct Control {
  uint64_t q_full[2], k_full[2], v_full[2];            // by chunk parity
  uint64_t qs_done[2], d_done[2], pv_done[2];          // Q S (and Q K^T before it), K^T V', P V
  uint64_t vp_full[2], vp_free[2], tab_full[2], tab_free[2];
  uint64_t qk_done, p_full, d_free, s_full, o_read, zeroed, drain;
  uint32_t tmem;
  volatile uint32_t abort;
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// bf16 pairs: a b and a b + c, rounded to nearest-even
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t fma_bf16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}

// A warp's part of a state, 32 rows of kCols columns with one row per lane in registers, from or to
// global memory (row stride d_v, the first `rows` rows and `cols` columns) through 64 kCols bytes of
// shared memory, half of the columns at a time, so that global memory sees whole lines: a row per
// thread costs the load/store pipe three cycles for every 32 bytes (64 prompts of 40 to 250 tokens:
// 108 us so, 96 us through shared memory).
template <int kCols>
struct StateRows {
  static constexpr int kR = kCols / 2, kPer = kR / 4, kStep = 32 / kPer;  // columns, float4 per row, rows per access
  static __device__ __forceinline__ int slot(int row, int j) { return row * kPer + (j ^ ((kPer == 8 ? row : row >> 1) & (kPer - 1))); }
  static __device__ __forceinline__ void load(const float *src, int d_v, int rows, int cols, float4 *stage, float *S) {
    const int lane = threadIdx.x & 31, row0 = lane / kPer, j = lane % kPer;
    float4 x[2][kPer];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int row = row0 + i * kStep, c = h * kR + 4 * j;
        x[h][i] = row < rows && c < cols ? *reinterpret_cast<const float4 *>(src + int64_t(row) * d_v + c)
                                         : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kPer; ++i) stage[slot(row0 + i * kStep, j)] = x[h][i];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const float4 v = stage[slot(lane, i)];
        S[h * kR + 4 * i] = v.x, S[h * kR + 4 * i + 1] = v.y, S[h * kR + 4 * i + 2] = v.z, S[h * kR + 4 * i + 3] = v.w;
      }
    }
  }
  static __device__ __forceinline__ void store(float *dst, int d_v, int rows, int cols, float4 *stage, const float *S) {
    const int lane = threadIdx.x & 31, row0 = lane / kPer, j = lane % kPer;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kPer; ++i)
        stage[slot(lane, i)] = make_float4(S[h * kR + 4 * i], S[h * kR + 4 * i + 1], S[h * kR + 4 * i + 2], S[h * kR + 4 * i + 3]);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        const int row = row0 + i * kStep, c = h * kR + 4 * j;
        if (row < rows && c < cols) *reinterpret_cast<float4 *>(dst + int64_t(row) * d_v + c) = stage[slot(row, j)];
      }
    }
  }
};

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

template <int kDV, bool kOutBF16, bool kStateOnly>
__global__ void __launch_bounds__(kThreads, 1)
    linear_chunked_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                          const __grid_constant__ CUtensorMap mv, const LinearArgs a, uint32_t *err_word) {
  using F = Cfg<kDV, kOutBF16, kStateOnly>;
  constexpr bool kPair = F::kPair;
  extern __shared__ __align__(1024) uint8_t smem[];
  Table *tab = reinterpret_cast<Table *>(smem + F::oTab);
  Control *ctl = reinterpret_cast<Control *>(smem + F::oTab + 2 * sizeof(Table));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x % a.H, hk = h / (a.H / a.H_k);
  const int col0 = blockIdx.y * kDV;

  if (tid == 0) {
    if (!kStateOnly) tma_prefetch_desc(&mq);
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
  }
  if constexpr (kStateOnly) let_next_pass_begin();
  LinearSlot s;
  if (!linear_slot(a.cu, a.num_seqs, a.plan.seg_len, a.plan.inner, blockIdx.x / a.H, s)) return;
  const int len = int(s.t1 - s.t0), chunks = (len + kC - 1) / kC;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->q_full[i], 1), mbar_init(&ctl->k_full[i], 1), mbar_init(&ctl->v_full[i], 1);
      mbar_init(&ctl->qs_done[i], 1), mbar_init(&ctl->d_done[i], 1), mbar_init(&ctl->pv_done[i], 1);
      mbar_init(&ctl->vp_full[i], 4), mbar_init(&ctl->vp_free[i], 1);
      mbar_init(&ctl->tab_full[i], 1), mbar_init(&ctl->tab_free[i], kStateOnly ? 14 : 16);
    }
    mbar_init(&ctl->qk_done, 1), mbar_init(&ctl->p_full, 4), mbar_init(&ctl->d_free, 8);
    mbar_init(&ctl->s_full, 8), mbar_init(&ctl->o_read, 8), mbar_init(&ctl->zeroed, 4), mbar_init(&ctl->drain, kStateOnly ? 1 : 2);
    ctl->abort = 0;
    fence_mbarrier_init();
  }
  if (warp == 1) tmem_alloc(&ctl->tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  const uint32_t tQK = tmem, tOI = tmem + 128, tOX = tOI + kDV, tD = tOX + kDV, tPL = tD + kDV;  // tPL: low half of P

  // A bounded wait; false once any role has given up, so that all leave together. `wait` is for
  // the single-lane roles, `wait_warp` gives all lanes of a warp one answer.
  auto wait = [&](uint64_t &bar, uint32_t parity, uint32_t code) -> bool {
    if (mbar_try_wait(&bar, parity & 1)) return true;
#pragma unroll 1
    for (uint32_t i = 0; i < kSleepLimit; ++i) {
      if (mbar_try_wait_sleep(&bar, parity & 1, kSleepNs)) return true;
      if (ctl->abort != 0) return false;
    }
    ctl->abort = 1;
    raise_device_error(err_word, code);
    return false;
  };
  // (T = 65536, 16 heads, in one run: 292 us with plain probes on the MMA warps, 310 without, 301 on all warps; a
  // failing probe takes 1 us, so kProbes are 2 s)
  auto wait_warp = [&](uint64_t &bar, uint32_t parity, uint32_t code) -> bool {
    if (warp == 1 || warp == 3) {  // the MMA warps: plain probes, shorter code
      bool ok = false;
#pragma unroll 1
      for (uint32_t i = 0; i < kProbes; ++i) {
        ok = mbar_try_wait(&bar, parity & 1);
        if (ok || ctl->abort != 0) break;
      }
      if (__all_sync(0xffffffffu, ok)) return true;
      ctl->abort = 1;
      raise_device_error(err_word, code);
      return false;
    }
    return __all_sync(0xffffffffu, wait(bar, parity, code)) != 0;
  };

  if (warp == 0) {
    // ---- loads: chunk n's V, Q and K, each when its buffer is free
    if (lane == 0) {
      Bufs<kStateOnly> at;
      int issued = 0;
#pragma unroll 1
      for (int n = 0; n < chunks; ++n, at.step()) {
        const int32_t t = int32_t(s.t0) + (kStateOnly ? chunks - 1 - n : n) * kC;
        const int s2 = n & 1;
        if (kStateOnly && n > 0) {
          if (!wait(ctl->tab_full[s2 ^ 1], (n - 1) >> 1, DEVERR_MMA_TIMEOUT)) break;
          const bool stop = tab[s2 ^ 1].stop != 0;
          mbar_arrive(&ctl->tab_free[s2 ^ 1]);
          if (stop) break;
        }
        if (n >= 2) {  // everything with chunk n - 2's K and V is done
          if (!wait(ctl->d_done[s2], (n >> 1) - 1, DEVERR_MMA_TIMEOUT)) break;
          if (!kStateOnly && !wait(ctl->pv_done[s2], (n >> 1) - 1, DEVERR_MMA_TIMEOUT)) break;
        }
        mbar_arrive_expect_tx(&ctl->v_full[s2], F::kTileV);
#pragma unroll
        for (int b = 0; b < kDV / 64; ++b)
          tma_load_3d(smem + at.V() + b * 16384, &mv, &ctl->v_full[s2], col0 + 64 * b, h, t);
        issued = 3 * n + 1;
        if constexpr (!kStateOnly) {
          mbar_arrive_expect_tx(&ctl->q_full[s2], kBuf);
#pragma unroll
          for (int b = 0; b < 2; ++b) tma_load_3d(smem + at.Q() + b * 16384, &mq, &ctl->q_full[s2], 64 * b, hk, t);
          issued = 3 * n + 2;
          if (n >= 1) {  // K's place is Q's of chunk n - 1; meanwhile it comes as far as L2
#pragma unroll
            for (int b = 0; b < 2; ++b) tma_prefetch_3d(&mk, 64 * b, hk, t);
            if (!wait(ctl->qs_done[s2 ^ 1], (n - 1) >> 1, DEVERR_MMA_TIMEOUT)) break;
          }
        }
        mbar_arrive_expect_tx(&ctl->k_full[s2], kBuf);
#pragma unroll
        for (int b = 0; b < 2; ++b) tma_load_3d(smem + at.K() + b * 16384, &mk, &ctl->k_full[s2], 64 * b, hk, t);
        issued = 3 * n + 3;
      }
      // every load issued has landed before the CTA may end: the last two of each tensor
      const int nv = (issued + 2) / 3, nq = (issued + 1) / 3, nk = issued / 3;
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {
        if (!kStateOnly && nq > i) mbar_wait(&ctl->q_full[(nq - 1 - i) & 1], ((nq - 1 - i) >> 1) & 1, err_word, DEVERR_TMA_TIMEOUT);
        if (nk > i) mbar_wait(&ctl->k_full[(nk - 1 - i) & 1], ((nk - 1 - i) >> 1) & 1, err_word, DEVERR_TMA_TIMEOUT);
        if (nv > i) mbar_wait(&ctl->v_full[(nv - 1 - i) & 1], ((nv - 1 - i) >> 1) & 1, err_word, DEVERR_TMA_TIMEOUT);
      }
    }
  } else if (warp == 1) {
    // ---- Q K^T, Q S, P V
    if constexpr (!kStateOnly) {
      constexpr uint32_t iQK = umma_idesc_bf16(128, 128, false, false, false);
      constexpr uint32_t iPV = umma_idesc_bf16(128, kDV, false, true, false);  // P V and Q S
      const bool leader = elect_lane();
      const uint32_t base = smem_u32(smem);
      // Descriptors of the first buffers; an operand elsewhere is `bytes / 16` further (addresses
      // stay below 2^18, so the address field never carries).
      const uint64_t dBuf = desc_k(base), dBufT = desc_mn(base, 16384), dS = desc_mn(base + F::oS, 16384);
      Bufs<kStateOnly> at;
#pragma unroll 1
      for (int n = 0; n < chunks; ++n, at.step()) {
        const uint64_t dQ = dBuf + (at.Q() >> 4), dK = dBuf + (at.K() >> 4), dV = dBufT + (at.V() >> 4);
        if (!wait_warp(ctl->k_full[n & 1], n >> 1, DEVERR_TMA_TIMEOUT)) break;
        if (!wait_warp(ctl->q_full[n & 1], n >> 1, DEVERR_TMA_TIMEOUT)) break;
        // P of chunk n - 1 has been read out of the columns Q K^T goes to
        if (n > 0 && !wait_warp(ctl->pv_done[(n - 1) & 1], (n - 1) >> 1, DEVERR_MMA_TIMEOUT)) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          const uint32_t o = (ks >> 2) * 1024 + (ks & 3) * 2;
          mma_ss(leader, tQK, dQ + o, dK + o, iQK, ks > 0);
        }
        mma_commit(leader, ctl->qk_done);
        if (!wait_warp(ctl->s_full, n, DEVERR_MMA_TIMEOUT)) break;
        if (n > 0 && !wait_warp(ctl->o_read, n - 1, DEVERR_MMA_TIMEOUT)) break;  // O of chunk n - 1 is read out
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < (kPair ? 16 : 8); ++ks)
          mma_ss(leader, tOX, dQ + (((ks & 7) >> 2) * 1024 + (ks & 3) * 2),
                 dS + ((ks >> 3) * (F::kTileS >> 4) + (ks & 7) * 128), iPV, ks > 0);
        mma_commit(leader, ctl->qs_done[n & 1]);
        if (!wait_warp(ctl->v_full[n & 1], n >> 1, DEVERR_TMA_TIMEOUT)) break;
        if (!wait_warp(ctl->p_full, n, DEVERR_MMA_TIMEOUT)) break;
        // the last chunk's rows behind the segment are zeroed in V
        if ((n + 1) * kC > len && !wait_warp(ctl->zeroed, 0, DEVERR_MMA_TIMEOUT)) break;
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < (kPair ? 16 : 8); ++ks)
          mma_ts(leader, tOI, (ks < 8 ? tQK : tPL) + 8 * (ks & 7), dV + (ks & 7) * 128, iPV, ks > 0);
        mma_commit(leader, ctl->pv_done[n & 1]);
      }
      // no MMA is in flight when tensor memory is freed
      mma_commit(leader, ctl->drain);
      if (leader) mbar_wait(&ctl->drain, 0, err_word, DEVERR_MMA_TIMEOUT);
    }
  } else if (warp == 3) {
    // ---- K^T V', 32 tokens at a time
    constexpr uint32_t iD = umma_idesc_bf16(128, kDV, true, true, false);
    const bool leader = elect_lane();
    const uint32_t base = smem_u32(smem);
    const uint64_t dBufT = desc_mn(base, 16384), dVP = desc_mn(base + F::oVP, 4096);
    Bufs<kStateOnly> at;
    bool ok = true;
#pragma unroll 1
    for (int n = 0; ok && n < chunks; ++n, at.step()) {
      if (!wait_warp(ctl->k_full[n & 1], n >> 1, DEVERR_TMA_TIMEOUT)) break;
      if (n > 0 && !wait_warp(ctl->d_free, n - 1, DEVERR_MMA_TIMEOUT)) break;
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        const int u = 4 * n + q;
        ok = wait_warp(ctl->vp_full[u & 1], u >> 1, DEVERR_MMA_TIMEOUT);
        if (!ok) break;
        tc_fence_after();
        const uint64_t ak = dBufT + ((at.K() >> 4) + q * 256), bv = dVP + uint32_t(u & 1) * (2 * F::kTileVP >> 4);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)  // hi, lo
          mma_ss(leader, tD, ak + (ks & 1) * 128, bv + ((ks >> 1) * (F::kTileVP >> 4) + (ks & 1) * 128), iD,
                 q > 0 || ks > 0);
        mma_commit(leader, ctl->vp_free[u & 1]);
      }
      if (!ok) break;
      mma_commit(leader, ctl->d_done[n & 1]);
      if constexpr (kStateOnly) {
        if (!wait_warp(ctl->tab_full[n & 1], n >> 1, DEVERR_MMA_TIMEOUT)) break;
        const bool stop = tab[n & 1].stop != 0;
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->tab_free[n & 1]);
        if (stop) break;
      }
    }
    mma_commit(leader, ctl->drain);
    if (leader) mbar_wait(&ctl->drain, 0, err_word, DEVERR_MMA_TIMEOUT);
  } else if (warp == 2) {
    // ---- decay tables
    double total = 0.;
    const bool per_token = a.per_token != 0;
    const float constant = per_token ? 0.f : a.log_decay[h];
    float g[4];
    auto fetch = [&](int n) {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int i = (kStateOnly ? chunks - 1 - n : n) * kC + 32 * b + lane;
        g[b] = i < len ? (per_token ? a.log_decay[(s.t0 + i) * a.H + h] : constant) : 0.f;
      }
    };
    fetch(0);
#pragma unroll 1
    for (int n = 0; n < chunks; ++n) {
      float p[4], x[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const float v = g[b] * kLog2e;
        p[b] = v < kMinLog2 ? kMinLog2 : v;  // a NaN stays
        x[b] = __shfl_down_sync(0xffffffffu, p[b], 1);
        if (lane == 31) x[b] = 0.f;  // from behind the token
      }
      if (n + 1 < chunks) fetch(n + 1);
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          const float up = __shfl_up_sync(0xffffffffu, p[b], o), down = __shfl_down_sync(0xffffffffu, x[b], o);
          if (lane >= o) p[b] += up;
          if (lane + o < 32) x[b] += down;
        }
      }
      float t[4];
#pragma unroll
      for (int b = 0; b < 4; ++b) t[b] = __shfl_sync(0xffffffffu, p[b], 31);
      const float all = (t[0] + t[1]) + (t[2] + t[3]);
      const float before = kStateOnly ? ex2(float(total)) : 0.f;  // of what lies behind the chunk
      total += double(all);
      Table &w = tab[n & 1];
      if (!wait_warp(ctl->tab_free[n & 1], (n >> 1) ^ 1, DEVERR_MMA_TIMEOUT)) break;
      const float behind[4] = {t[1] + t[2] + t[3], t[2] + t[3], t[3], 0.f};
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        w.a[32 * b + lane] = p[b];
        const float es = ex2(x[b]);
        if (b < 3) w.es[32 * b + lane] = es;
        const float f = es * ex2(behind[b]);
        const uint32_t f1 = pack_bf16x2(f, 0.f) & 0xffffu;
        w.f[32 * b + lane] = f1 | (pack_bf16x2(f - bf16_to_f32(uint16_t(f1)), 0.f) << 16);
      }
      const bool stop = kStateOnly && total <= double(kMinLog2);  // a NaN goes on
      if (lane == 0) {
        if constexpr (kStateOnly) {
          w.e1 = before;
        } else {
          const bool keep = !(all < -1.f);  // a NaN keeps
          w.e1 = keep ? expm1f(all * kLn2) : ex2(all);
          w.keep = keep ? 1.f : 0.f;
        }
        w.stop = stop;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->tab_full[n & 1]);
      if (stop) break;
    }
    if (kStateOnly && lane == 0 && blockIdx.y == 0)
      a.seg_decay[s.place * a.H + h] = float(total * 0.6931471805599453);
  } else if (warp >= 4 && warp < 8) {
    // ---- P: row i of Q K^T in lane i; the decays, then bf16 in place
    if constexpr (!kStateOnly) {
      const int w = warp & 3;
      const uint32_t row = uint32_t(32 * w) << 16;
#pragma unroll 1
      for (int n = 0; n < chunks; ++n) {
        const Table &tb = tab[n & 1];
        if (!wait_warp(ctl->tab_full[n & 1], n >> 1, DEVERR_MMA_TIMEOUT)) break;
        const float ai = tb.a[32 * w + lane];
        if (!wait_warp(ctl->qk_done, n, DEVERR_MMA_TIMEOUT)) break;
        tc_fence_after();
        // bf16 of 32 columns over columns that have been read already
        auto put = [&](int J, const float2(&p)[16]) {
          float hi[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) hi[j] = __uint_as_float(pack_bf16x2(p[j].x, p[j].y));
          tmem_st16(tQK + row + 16 * J, hi);
          if constexpr (kPair) {
            float lo[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              const float2 b = unpack_bf16x2(__float_as_uint(hi[j]));
              lo[j] = __uint_as_float(pack_bf16x2(p[j].x - b.x, p[j].y - b.y));
            }
            tmem_st16(tPL + row + 16 * J, lo);
          }
        };
        auto get = [&](int J, float2(&p)[16]) {
          float x[2][16];
          tmem_ld16(tQK + row + 32 * J, x[0]);
          tmem_ld16(tQK + row + 32 * J + 16, x[1]);
          tmem_ld_wait(x[0], x[1]);
#pragma unroll
          for (int j = 0; j < 16; ++j) p[j] = make_float2(x[j >> 3][(2 * j) & 15], x[j >> 3][(2 * j + 1) & 15]);
        };
#pragma unroll 1
        for (int J = 0; J < w; ++J) {  // blocks before the row's: row factor x column factor
          float e = ai;  // from the end of block J to the row
          if (J + 1 < w) e += tb.block(J + 1);
          if (J + 2 < w) e += tb.block(J + 2);
          e = ex2(e);
          float2 p[16];
          get(J, p);
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 c = *reinterpret_cast<const float4 *>(&tb.es[32 * J + j]);
            p[j >> 1] = f2_mul(p[j >> 1], f2_mul(make_float2(c.x, c.y), make_float2(e, e)));
            p[(j >> 1) + 1] = f2_mul(p[(j >> 1) + 1], f2_mul(make_float2(c.z, c.w), make_float2(e, e)));
          }
          put(J, p);
        }
        if (kPair && tb.block(w) < kFarLog2) {
          // long sums, whose differences would lose what lies behind a token that forgets: each entry
          // takes the sum of its own, of the tokens from behind its column to the row
          const int i = n * kC + 32 * w + lane;
          float g = i < len ? a.log_decay[a.per_token ? (s.t0 + i) * a.H + h : h] * kLog2e : 0.f;
          g = g < kMinLog2 ? kMinLog2 : g;
#pragma unroll 1
          for (int j0 = 0; j0 < 32; j0 += 16) {
            float sum = 0.f, x[16], hi[8], lo[8];
#pragma unroll 1
            for (int j = 31; j >= j0 + 16; --j) {
              const float next = __shfl_sync(0xffffffffu, g, j);
              if (j <= lane) sum += next;
            }
            tmem_ld16_wait(tQK + row + 32 * w + j0, x);
#pragma unroll
            for (int j = 15; j >= 0; --j) {
              x[j] = j0 + j <= lane ? x[j] * ex2(sum) : 0.f;
              const float next = __shfl_sync(0xffffffffu, g, j0 + j);
              if (j0 + j <= lane) sum += next;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint32_t u = pack_bf16x2(x[2 * j], x[2 * j + 1]);
              const float2 b = unpack_bf16x2(u);
              hi[j] = __uint_as_float(u);
              lo[j] = __uint_as_float(pack_bf16x2(x[2 * j] - b.x, x[2 * j + 1] - b.y));
            }
            tmem_st8(tQK + row + 16 * w + j0 / 2, hi);
            tmem_st8(tPL + row + 16 * w + j0 / 2, lo);
          }
        } else {  // the row's own block; selected away, not multiplied: what lies above may be infinite
          float2 p[16];
          get(w, p);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 c = *reinterpret_cast<const float2 *>(&tb.a[32 * w + j]);
            p[j >> 1].x = j <= lane ? p[j >> 1].x * ex2(ai - c.x) : 0.f;
            p[j >> 1].y = j + 1 <= lane ? p[j >> 1].y * ex2(ai - c.y) : 0.f;
          }
          put(w, p);
        }
#pragma unroll 1
        for (int J = w + 1; J < 4; ++J) {
          float zero[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) zero[j] = 0.f;
          tmem_st16(tQK + row + 16 * J, zero);
          if constexpr (kPair) tmem_st16(tPL + row + 16 * J, zero);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&ctl->p_full);
          mbar_arrive(&ctl->tab_free[n & 1]);
        }
      }
    }
  } else if (warp >= 8 && warp < 12) {
    // ---- V': quarters of 32 tokens, two buffers
    const int wt = tid - 256;
    // this thread's pieces: 8 columns (piece j) of tokens t0, t0 + step, ... of a quarter
    constexpr int step = 1024 / kDV;
    const int j = wt % (kDV / 8), t0 = wt / (kDV / 8);
    const uint32_t src_off = sw128_chunk(t0, j & 7, j >> 3, 128), dst_off = sw128_chunk(t0, j & 7, j >> 3, 32);
    Bufs<kStateOnly> at;
    bool ok = true;
#pragma unroll 1
    for (int n = 0; ok && n < chunks; ++n, at.step()) {
      const Table &tb = tab[n & 1];
      ok = wait_warp(ctl->tab_full[n & 1], n >> 1, DEVERR_MMA_TIMEOUT) &&
           wait_warp(ctl->v_full[n & 1], n >> 1, DEVERR_TMA_TIMEOUT);
      if (!ok) break;
      uint8_t *V = smem + at.V() + src_off;
      const int part = len - n * kC;
      if (part < kC) {
        // rows from here on hold another sequence's tokens: zeros in V and K, since 0 times another
        // sequence's infinity would not vanish in the products
        if (!wait_warp(ctl->k_full[n & 1], n >> 1, DEVERR_TMA_TIMEOUT)) break;
        uint8_t *K = smem + at.K();
#pragma unroll 1
        for (int m = 0; m < kC / step; ++m) {  // each thread its own pieces of V, and K's beside
          const int tt = t0 + m * step;
          if (tt < part) continue;
          const uint4 zero = make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4 *>(V + m * step * 128) = zero;
          for (int b = 0; b < 128 / kDV; ++b)
            *reinterpret_cast<uint4 *>(K + sw128_chunk(tt, j & 7, kDV == 128 ? j >> 3 : b, 128)) = zero;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (!kStateOnly && lane == 0) mbar_arrive(&ctl->zeroed);
      }
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        const int u = 4 * n + q;
        uint8_t *src = V + q * 4096, *dst = smem + F::oVP + (u & 1) * 2 * F::kTileVP + dst_off;
        ok = wait_warp(ctl->vp_free[u & 1], (u >> 1) ^ 1, DEVERR_MMA_TIMEOUT);
        if (!ok) break;
#pragma unroll
        for (int m = 0; m < 32 / step; ++m) {
          // V' = f v with f = f1 + f2: hi = bf16(f1 v), whose error fits in bf16 itself, and lo =
          // bf16(that error + f2 v)
          const uint32_t f = tb.f[32 * q + t0 + m * step];
          const uint32_t f1 = __byte_perm(f, 0, 0x1010), f2 = __byte_perm(f, 0, 0x3232);
          const uint4 x = *reinterpret_cast<const uint4 *>(src + m * step * 128);
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
          uint32_t h4[4], l4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            h4[e] = mul_bf16x2(f1, xs[e]);
            l4[e] = fma_bf16x2(f2, xs[e], fma_bf16x2(f1, xs[e], h4[e] ^ 0x80008000u));
          }
          *reinterpret_cast<uint4 *>(dst + m * step * 128) = make_uint4(h4[0], h4[1], h4[2], h4[3]);
          *reinterpret_cast<uint4 *>(dst + F::kTileVP + m * step * 128) = make_uint4(l4[0], l4[1], l4[2], l4[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->vp_full[u & 1]);
      }
      const bool stop = kStateOnly && tb.stop != 0;
      __syncwarp();
      if (ok && lane == 0) mbar_arrive(&ctl->tab_free[n & 1]);
      if (stop) break;
    }
  } else if (warp >= 12) {
    // ---- the state and the output
    constexpr int kHalf = kDV / 2;  // columns per thread
    const int half = (warp - 12) >> 2, w = warp & 3, r = 32 * w + lane;
    const uint32_t row = uint32_t(32 * w) << 16;
    const int cb = half * kHalf;  // first column within the tile
    const int64_t dd = int64_t(a.d_k) * a.d_v;
    float S[kHalf];
    float4 *const stage = reinterpret_cast<float4 *>(smem + F::oS + (warp - 12) * (F::kTileS / 8));
    const int64_t part = int64_t(32 * w) * a.d_v + col0 + cb;  // this warp's part of a state
    const int rows = a.d_k - 32 * w, width = a.d_v - col0 - cb;
    const float *src = kStateOnly ? nullptr : linear_entering(a, s, h);
    if (src != nullptr) {
      StateRows<kHalf>::load(src + part, a.d_v, rows, width, stage, S);
    } else {
#pragma unroll
      for (int c = 0; c < kHalf; ++c) S[c] = 0.f;
    }
    // the tile takes the place of what all eight warps have staged
    if (!kStateOnly) named_bar_sync(1, 256);
    const uint32_t state_off = sw128_chunk(r, 0, cb >> 6, 128);
    auto write_state_tile = [&]() {  // the B operand of Q S: rows k, MN-major
#pragma unroll
      for (int c = 0; c < kHalf; c += 8) {
        uint32_t u[4], l[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          u[e] = pack_bf16x2(S[c + 2 * e], S[c + 2 * e + 1]);
          if constexpr (kPair) {
            const float2 b = unpack_bf16x2(u[e]);
            l[e] = pack_bf16x2(S[c + 2 * e] - b.x, S[c + 2 * e + 1] - b.y);
          }
        }
        const uint32_t o = state_off ^ ((((cb + c) >> 3) & 7) << 4);
        *reinterpret_cast<uint4 *>(smem + F::oS + o) = make_uint4(u[0], u[1], u[2], u[3]);
        if constexpr (kPair)
          *reinterpret_cast<uint4 *>(smem + F::oS + F::kTileS + o) = make_uint4(l[0], l[1], l[2], l[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->s_full);
    };
    if (!kStateOnly && chunks > 0) write_state_tile();
    // rows of the output that start on 32-byte boundaries take 32-byte stores
    const bool wide = ((reinterpret_cast<uintptr_t>(a.out) | (uint32_t(a.d_v) * (kOutBF16 ? 2 : 4))) & 31) == 0;
#pragma unroll 1
    for (int n = 0; n < chunks; ++n) {
      const Table &tb = tab[n & 1];
      if (!wait_warp(ctl->tab_full[n & 1], n >> 1, DEVERR_MMA_TIMEOUT)) break;
      const float e1 = tb.e1, keep = kStateOnly ? 0.f : tb.keep;
      const bool stop = kStateOnly && tb.stop != 0;
      float eG = 0.f;  // e^{G_r}, the decay of the entering state at token r
      if constexpr (!kStateOnly) {
        eG = tb.a[r];
#pragma unroll
        for (int B = 0; B < 3; ++B)
          if (B < w) eG += tb.block(B);
        eG = a.scale * ex2(eG);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->tab_free[n & 1]);
      // the state: S <- e^{G_C} S + K^T V' (in pass 1, S <- S + e^(behind) K^T V')
      if (!wait_warp(ctl->d_done[n & 1], n >> 1, DEVERR_MMA_TIMEOUT)) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < kHalf; c += 16) {
        float d[16];
        tmem_ld16_wait(tD + row + cb + c, d);
#pragma unroll
        for (int e = 0; e < 16; e += 2) {
          const float2 x = make_float2(S[c + e], S[c + e + 1]), dd2 = make_float2(d[e], d[e + 1]);
          const float2 y = kStateOnly ? f2_fma(make_float2(e1, e1), dd2, x)
                                      : f2_fma(make_float2(e1, e1), x, f2_fma(make_float2(keep, keep), x, dd2));
          S[c + e] = y.x, S[c + e + 1] = y.y;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->d_free);
      if (stop) break;
      if constexpr (!kStateOnly) {
        if (n + 1 < chunks) {
          if (!wait_warp(ctl->qs_done[n & 1], n >> 1, DEVERR_MMA_TIMEOUT)) break;
          write_state_tile();
        }
        if (!wait_warp(ctl->pv_done[n & 1], n >> 1, DEVERR_MMA_TIMEOUT)) break;
        tc_fence_after();
        // the output: O = scale (P V + e^G Q S), token r in lane r
        constexpr int kPer = kOutBF16 ? 16 : 8;  // columns of 32 bytes
        constexpr int kEs = kOutBF16 ? 2 : 4;
        const int64_t t = s.t0 + int64_t(n) * kC + r;
        uint8_t *out = static_cast<uint8_t *>(a.out) + ((t * a.H + h) * a.d_v + col0 + cb) * kEs;
        const int cols = t < s.t1 ? a.d_v - col0 - cb : 0;  // this row's columns from cb on
#pragma unroll
        for (int c = 0; c < kHalf; c += kPer) {
          uint32_t u[8];
#pragma unroll
          for (int i = 0; i < kPer; i += 8) {
            float oi[8], ox[8];
            tmem_ld8(tOI + row + cb + c + i, oi);
            tmem_ld8(tOX + row + cb + c + i, ox);
            tmem_ld_wait(oi, ox);
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float2 y = f2_fma(make_float2(eG, eG), make_float2(ox[e], ox[e + 1]),
                                      f2_mul(make_float2(a.scale, a.scale), make_float2(oi[e], oi[e + 1])));
              if constexpr (kOutBF16) u[(i + e) >> 1] = pack_bf16x2(y.x, y.y);
              else u[e] = __float_as_uint(y.x), u[e + 1] = __float_as_uint(y.y);
            }
          }
          if (wide && c < cols) {  // whole: cols is then a multiple of kPer
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out + c * kEs), "r"(u[0]),
                         "r"(u[1]), "r"(u[2]), "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                         : "memory");
          } else {
            if (c < cols) *reinterpret_cast<uint4 *>(out + c * kEs) = make_uint4(u[0], u[1], u[2], u[3]);
            if (c + kPer / 2 < cols) *reinterpret_cast<uint4 *>(out + c * kEs + 16) = make_uint4(u[4], u[5], u[6], u[7]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->o_read);
      }
    }
    float *dst = kStateOnly ? a.seg_states + (s.place * a.H + h) * dd
                 : (s.last && a.final_state != nullptr) ? a.final_state + (int64_t(s.n) * a.H + h) * dd : nullptr;
    // (P V of the last chunk is done, and Q S before it, so nobody reads the tile)
    if (dst != nullptr) StateRows<kHalf>::store(dst + part, a.d_v, rows, width, stage, S);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tmem_relinquish();
    tmem_dealloc(tmem, 512);
  }
  if constexpr (!kStateOnly) wait_for_earlier_passes();
}

template <int kDV, bool kOutBF16, bool kStateOnly>
cudaError_t launch_one(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const LinearArgs &a,
                       cudaStream_t stream) {
  using F = Cfg<kDV, kOutBF16, kStateOnly>;
  constexpr uint32_t smem = F::oTab + 2 * sizeof(Table) + sizeof(Control);
  static_assert(smem <= 232448, "shared memory of one CTA");
  const auto kern = linear_chunked_kernel<kDV, kOutBF16, kStateOnly>;
  // the kernel's shared memory, granted once per device (bit d for device d; past 63 at every launch)
  static std::atomic<uint64_t> granted;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (bit == 0 || (granted.load(std::memory_order_acquire) & bit) == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
    if (e != cudaSuccess) return e;
    granted.fetch_or(bit, std::memory_order_release);
  }
  const unsigned pieces = unsigned(a.plan.inner) + (kStateOnly ? 0u : unsigned(a.num_seqs));
  const dim3 grid(pieces * unsigned(a.H), unsigned((a.d_v + kDV - 1) / kDV));
  return launch_pass_kernel(kern, grid, kThreads, smem, !kStateOnly && a.plan.seg_len != 0, stream, mq, mk, mv, a,
                            device_error_word());
}

}  // namespace

namespace {
cudaError_t launch_passes(const LinearArgs &a, bool out_bf16, cudaStream_t stream) {
  CUtensorMap mq, mk, mv;
  const int d_k = (a.d_k + 7) & ~7;
  if (!tensor_map_3d(&mq, a.q, true, a.total, a.H_k, d_k, 64, kC, true) ||
      !tensor_map_3d(&mk, a.k, true, a.total, a.H_k, d_k, 64, kC, true) ||
      !tensor_map_3d(&mv, a.v, true, a.total, a.H, a.d_v, 64, kC, true))
    return cudaErrorInvalidValue;
  const bool wide = a.plan.col_tile == 128;
  if (a.plan.seg_len != 0) {
    cudaError_t e = wide ? launch_one<128, true, true>(mq, mk, mv, a, stream)
                         : launch_one<64, true, true>(mq, mk, mv, a, stream);
    if (e == cudaSuccess) e = launch_linear_scan(a, stream);
    if (e != cudaSuccess) return e;
  }
  if (wide) return launch_one<128, true, false>(mq, mk, mv, a, stream);
  return out_bf16 ? launch_one<64, true, false>(mq, mk, mv, a, stream)
                  : launch_one<64, false, false>(mq, mk, mv, a, stream);
}
}  // namespace

cudaError_t launch_linear_chunked(const LinearArgs &a, bool out_bf16, cudaStream_t stream) {
  if (!a.plan.pad) return launch_passes(a, out_bf16, stream);
  LinearArgs b = a;
  cudaError_t e = launch_linear_pad(b, stream);
  if (e == cudaSuccess) e = launch_passes(b, out_bf16, stream);
  if (e == cudaSuccess && a.d_v % 8 != 0)
    e = launch_linear_unpad(b, out_bf16, a.out, a.final_state, a.d_v, stream);
  return e;
}

}  // namespace kda
