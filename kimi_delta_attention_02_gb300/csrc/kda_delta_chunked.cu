// kda_delta_chunked.cu -- the gated delta rule with one decay per head on the tensor cores (bf16
// inputs; head sizes that are no multiple of 8 by padded copies), in chunks of 64 tokens.
//
// With G the cumulative log-decay inside a chunk, D_ti = e^{G_t - G_i}, and S the state that enters it,
//     A_ti = beta_t D_ti (k_t . k_i), i < t;      T' = (I + A)^-1 diag(beta),   T'' = -T' diag(e^G)
//     U    = T' V + T'' X,                        X = K S
//     O    = scale diag(e^G) Q S + P U,           P_ti = scale D_ti (q_t . k_i), i <= t
//     S   <- e^{G_C} S + K^T U',                  U'_i = e^{G_C - G_i} u_i .
// Everything that touches the state is formed transposed, with the value channels as the 128 rows of
// the MMA: X^T = S^T K^T, U^T = V^T T'^T + X^T T''^T, S^T += U'^T K, O^T = U^T P^T. So the state's way from
// one chunk to the next (S -> X -> U -> U' -> S) stays in one lane of tensor memory per value channel: each
// product's accumulator is read by a thread that owns its lane, split into the next product's A operand
// and written back over the same columns. Shared memory only holds B operands (K and Q as they come, T', T''
// and P) and V, the A operand of T' V, which runs ahead of the chain. The state itself stays in fp32 registers.
//
// Roundings. The operands of what reaches the state (S, X, T', T'', U') are pairs of bf16, hi + lo, each
// pair off by at most 2^-17 of the value, and the products take hi hi + hi lo + lo hi (K, Q and V are bf16
// as given). The read-out takes S, U and P as the same kind of pairs, for bf16 outputs too: where keys are alike, P U
// is a small sum of large terms, and a single bf16 P (2^-9) put outputs off by up to 0.0065. A is formed in fp32. Its inverse
// starts from blocks of 8 by forward substitution in fp32, joined to 16 in fp32, and to 32 and 64 by
// products of blocks in pairs of tf32 (2^-20) on the tensor cores. No power of A is formed, which with keys
// alike would grow like binomials. At T = 4096, 96 heads of 128: bf16 output off by 0.0017 in the 2-norm, its
// own rounding, fp32 output by 7e-6, state by 5e-6.
//
// Decays. G is summed in fp64 and kept as a pair of floats, so that no entry of D loses to long sums.
// A log-decay below -88 counts as -88 (2^-127), as in linear attention.
//
// Warps (24): 0 loads (TMA), 1 issues the chain's products X, U, S, 2 makes the decay tables, 3 issues
// the others (K K^T with Q K^T, Q S, P U) into the gaps of the chain; 4-7 and 8-11 make A, its inverse and P of
// every other chunk each, one to two chunks ahead; 12-15 write the output; 16-23 keep the state (a value
// channel and half of the key rows per thread) and form the chain's operands.
//
// What bounds it: the chain's latency. A chunk takes 4.1 us (T = 4096, 96 heads of 128: 262 us for 64 of them,
// against 63 us to move the bytes and 2.0 ms of the token kernel), of which the three products take 0.8 us
// and the hand-overs between MMA and warps (six, 0.15 to 0.2 us each) and the splitting of X, U' and S the
// rest, in competition with warps 4 to 11 for the issue slots: 203 us of 256 with those idle. (4.7 us a chunk with all
// SMs busy: the roles' 85 KB of code share an instruction cache.) Hence two halves per
// hand-over, so that a product starts on the first half, and V's product and the read-out off the chain.
#include <atomic>

#include "kda_delta.cuh"
#include "kda_linear_umma.cuh"
#include "kda_tma_host.h"

namespace kda {
namespace {

constexpr int kC = 64;             // tokens per chunk
constexpr int kThreads = 768;
constexpr int kKQ = 3, kP = 3, kTabs = 4;  // buffers (with two of P, A and P wait for them: 291 us instead of 263)
constexpr uint32_t kTileKQ = 32768;        // 64 rows of K, then 64 of Q, x 128 channels, two 64-channel blocks
constexpr uint32_t kBlockV = 8192;         // 64 rows of V x 64 channels: two buffers of one block, or one of two
constexpr uint32_t kTileT = 8192;          // 64 x 64 bf16
// P's pair in 96 rows. It is lower triangular, so lo takes the place of what would be zero in hi, 32 x 32 at a time:
//     rows  0 .. 31: hi of P's rows  0 .. 31, columns 0 .. 31 | lo of the same
//     rows 32 .. 63: hi of P's rows 32 .. 63, columns 0 .. 31 | columns 32 .. 63
//     rows 64 .. 95: lo of the same
constexpr uint32_t kTileP = 12288;
constexpr int kStrideA = 68;       // floats per row of A
constexpr uint32_t kProbes = 2000000;
constexpr double kLog2e = 1.4426950408889634, kLn2 = 0.6931471805599453, kMinLog2 = -127.;

struct Table {  // decays of one chunk; sums in log2 units
  float g[kC], g_lo[kC];  // G_t, as a pair
  float f[kC];            // -e^{G_t}
  float out[kC];          // scale e^{G_t}
  float w[kC];            // e^{G_C - G_t}
  float beta[kC];
  float cross[kC];        // e^{G_31 - G_i} for i < 32, e^{G_t - G_31} from there on
  float whole;            // e^{G_C} as the state's factor
  float pad[3];
};

struct Control {
  uint64_t kq_full[kKQ], v_full[2], tab_full[kTabs], tab_free[kTabs];
  // A wait tells phases by their parity, so it must not come two phases late, nor before the phase before
  // it has ended. Where one side may be two ahead, or a waiter takes every other chunk, there is a barrier
  // for each buffer, or for even and odd chunks.
  uint64_t kq_free[kKQ], v_free[2], p_free[3], gram_done[2], t_free[2];
  uint64_t gram_read, t_full, zeroed;
  uint64_t s_full[2], r_full[2], up_full[2];  // the first and second half of each thread's columns
  uint64_t x_done, xq_done, u_done, d_done, o_done, o_read, drain;
  uint32_t tmem;
  volatile uint32_t gave_up;
};

// in shared memory
constexpr uint32_t kAtV = kKQ * kTileKQ, kAtT = kAtV + 2 * kBlockV, kAtP = kAtT + 4 * kTileT, kAtA = kAtP + kP * kTileP,
                   kAtTab = kAtA + 2 * kC * kStrideA * 4, kAtCtl = kAtTab + kTabs * sizeof(Table),
                   kBytes = kAtCtl + sizeof(Control);
static_assert(kBytes <= 232448, "shared memory of one CTA");

// a run of tokens on one CTA
struct Run {
  int64_t t0;
  int len, chunks;
  bool emit;           // with outputs
  bool identity;       // from the identity, with v = 0
  const float *from;   // entering state, or null: zero
  float *to;           // or null
  int from_width, width;  // columns of `from` and `to`: d_v, or padded to a multiple of 8 in the workspace
};

// Probes (a failing one takes about 1 us) until the phase of this parity is complete; false, and `gave_up`
// set, after kProbes of them.
__device__ __forceinline__ bool bounded_wait(uint64_t &bar, uint32_t parity, volatile uint32_t &gave_up) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p, q;\n .reg .b32 i;\n mov.b32 i, %4;\n"
      "PROBE:\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n @p bra DONE;\n"
      " sub.u32 i, i, 1;\n setp.ne.u32 q, i, 0;\n @q bra PROBE;\n st.volatile.shared.b32 [%3], 1;\n"
      "DONE:\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(smem_u32(&bar)), "r"(parity), "r"(smem_u32(const_cast<const uint32_t *>(&gave_up))), "n"(kProbes)
      : "memory");
  return ok != 0;
}

// Two values as a pair of bf16 each: the nearest, and what is left.
__device__ __forceinline__ void split_pair(float x, float y, uint32_t &hi, uint32_t &lo) {
  hi = pack_bf16x2(x, y);
  const float2 rest = f2_fma(unpack_bf16x2(hi), make_float2(-1.f, -1.f), make_float2(x, y));
  lo = pack_bf16x2(rest.x, rest.y);
}

template <int kRegs>
__device__ __forceinline__ void registers_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegs)); }
template <int kRegs>
__device__ __forceinline__ void registers_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegs)); }

// D += A B of 16 x 8 x 8 in tf32 with fp32 sums
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}
// One warp: to = +- x m for 16 rows and 8 kN columns, over 16 kK inner entries, of fp32 blocks in rows of
// kStrideA. Each operand is a pair of tf32, cut off, not rounded (2^-20, with the range of fp32: where keys
// are not unit vectors or the decay grows, the entries do), whose low parts' product is left out. Unrolled by two: in full it is code enough to slow the whole CTA by 6 %.
template <int kK, int kN>
__device__ __forceinline__ void block_product(const float *x, const float *m, float *to, bool negate, int lane) {
  const int g = lane >> 2, t = lane & 3;
  auto split = [](float v, uint32_t &hi, uint32_t &lo) {
    hi = __float_as_uint(v) & 0xffffe000u;
    lo = __float_as_uint(v - __uint_as_float(hi)) & 0xffffe000u;
  };
  float d[kN][3][4] = {};
  // (inner entries 2 t and 2 t + 1 stand where the instruction has t and t + 4, in both operands)
  const float *xr = x + g * kStrideA + 2 * t, *mr = m + 2 * t * kStrideA + g;
#pragma unroll 2
  for (int k = 0; k < 2 * kK; ++k, xr += 8, mr += 8 * kStrideA) {
    uint32_t ah[4], al[4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float2 v = *reinterpret_cast<const float2 *>(xr + e * 8 * kStrideA);
      split(v.x, ah[e], al[e]);
      split(v.y, ah[e + 2], al[e + 2]);
    }
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      uint32_t bh[2], bl[2];
      split(mr[8 * j], bh[0], bl[0]);
      split(mr[kStrideA + 8 * j], bh[1], bl[1]);
      mma_tf32(d[j][0], ah, bh);
      mma_tf32(d[j][1], ah, bl);
      mma_tf32(d[j][2], al, bh);
    }
  }
  const float sign = negate ? -1.f : 1.f;
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    float y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) y[e] = sign * (d[j][0][e] + (d[j][1][e] + d[j][2][e]));
    *reinterpret_cast<float2 *>(&to[g * kStrideA + 8 * j + 2 * t]) = make_float2(y[0], y[1]);
    *reinterpret_cast<float2 *>(&to[(g + 8) * kStrideA + 8 * j + 2 * t]) = make_float2(y[2], y[3]);
  }
}

template <bool kOutBF16>
__global__ void __launch_bounds__(kThreads, 1)
    delta_chunked_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                         const __grid_constant__ CUtensorMap mv, const DeltaArgs a, int pass, uint32_t *err_word) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Table *tab = reinterpret_cast<Table *>(smem + kAtTab);
  Control *ctl = reinterpret_cast<Control *>(smem + kAtCtl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x % a.H, hk = h / (a.H / a.H_k);

  if (tid == 0) {
    tma_prefetch_desc(&mq);
    tma_prefetch_desc(&mk);
    tma_prefetch_desc(&mv);
  }
  Run run;
  {
    int index = blockIdx.x / a.H;
    const bool map = index >= a.plan.inner + a.num_seqs;  // pass 1: the pieces once more, for their M
    if (map) index -= a.plan.inner + a.num_seqs;
    if (a.plan.order) index = reinterpret_cast<const int32_t *>(a.workspace + a.plan.ends)[index];
    LinearSlot s;
    if (!linear_slot(a.cu, a.num_seqs, a.plan.seg_len, a.plan.inner, index, s)) return;
    if ((pass == 3 || map) ? s.first : s.last && !s.first) return;
    if (s.first && s.last && s.t1 - s.t0 <= a.plan.few) return;  // done by the decode kernel
    const int pk = delta_up8(a.d_k), pv = delta_up8(a.d_v);
    const int64_t dd = int64_t(a.d_k) * a.d_v, ee = int64_t(pk) * pv;
    float *ends = reinterpret_cast<float *>(a.workspace + a.plan.ends);
    const int64_t place = delta_place(a, s);
    run.t0 = s.t0, run.len = int(s.t1 - s.t0), run.chunks = (run.len + kC - 1) / kC;
    run.emit = s.first || pass == 3;
    run.identity = map;
    run.from_width = s.first ? a.d_v : pv;
    run.width = pv;
    run.from = !s.first ? (pass == 3 ? ends + ((place - 1) * a.H + h) * ee : nullptr)
               : a.init_state != nullptr ? a.init_state + (int64_t(s.n) * a.H + h) * dd : nullptr;
    if (run.emit && s.last) {
      run.width = a.d_v;
      run.to = a.final_state != nullptr ? a.final_state + (int64_t(s.n) * a.H + h) * dd : nullptr;
    } else {
      run.to = pass == 3 ? nullptr : ends + (place * a.H + h) * ee;
    }
    if (map) {
      run.width = pk;
      run.to = reinterpret_cast<float *>(a.workspace + a.plan.maps) + (place * a.H + h) * int64_t(pk) * pk;
    }
  }
  const int chunks = run.chunks, len = run.len;
  const int nk = (a.d_k + 15) >> 4;       // steps of 16 key channels
  const int kb = (a.d_k + 63) >> 6, vb = (a.d_v + 63) >> 6;  // blocks of 64 channels
  const int v_last = vb == 1 ? 1 : 0;     // V's buffers less one

  if (tid == 0) {
    for (int i = 0; i < kKQ; ++i) mbar_init(&ctl->kq_full[i], 1), mbar_init(&ctl->kq_free[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&ctl->v_full[i], 1), mbar_init(&ctl->v_free[i], 1);
    for (int i = 0; i < kP; ++i) mbar_init(&ctl->p_free[i], 1);
    for (int i = 0; i < 2; ++i) mbar_init(&ctl->gram_done[i], 1), mbar_init(&ctl->t_free[i], 1);
    for (int i = 0; i < kTabs; ++i) mbar_init(&ctl->tab_full[i], 1), mbar_init(&ctl->tab_free[i], run.emit ? 16 : 12);
    mbar_init(&ctl->t_full, 4), mbar_init(&ctl->gram_read, 4), mbar_init(&ctl->zeroed, 4);
    for (int i = 0; i < 2; ++i) mbar_init(&ctl->s_full[i], 8), mbar_init(&ctl->r_full[i], 8), mbar_init(&ctl->up_full[i], 8);
    mbar_init(&ctl->x_done, 1), mbar_init(&ctl->xq_done, 1), mbar_init(&ctl->u_done, 1), mbar_init(&ctl->d_done, 1);
    mbar_init(&ctl->o_done, 1), mbar_init(&ctl->o_read, 4), mbar_init(&ctl->drain, 2);
    ctl->gave_up = 0;
    fence_mbarrier_init();
  }
  if (warp == 1) tmem_alloc(&ctl->tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ctl->tmem;
  // S and K^T U' (128 columns), X, U and U', Q S, O, K K^T and Q K^T, U for the read-out (hi, lo)
  const uint32_t tS = tmem, tX = tmem + 128, tU = tmem + 192, tXQ = tmem + 256, tO = tmem + 320, tG = tmem + 384,
                 tUH = tmem + 448;

  // A bounded wait. Its role leaves when it is false, and with it every role that waits for that one, each
  // after its own limit; the end of the kernel reports it. `wait` is for single lanes, `wait_warp` gives all
  // lanes of a warp one answer. Their code is short because it stands at forty places.
  auto wait = [&](uint64_t &bar, uint32_t parity) -> bool { return bounded_wait(bar, parity & 1, ctl->gave_up); };
  auto wait_warp = [&](uint64_t &bar, uint32_t parity) -> bool { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
  const bool partial = len % kC != 0;  // the last chunk's rows behind the run are zeroed in K and V

  // registers by warpgroup, out of the 80 each that the launch holds: 56 + 2 x 72 + 40 + 2 x 120 = 6 x 80
  if (warp < 4) {
    registers_down<56>();
    if (warp == 0) {
      // ---- loads
      if (lane == 0) {
        int kq = 0, vs = 0;  // issued
        uint32_t ks = 0, vs_ = 0, ks_turn = 1, vs_turn = 1;  // buffers, and the parity of the use before
        const uint32_t kq_bytes = kb * (run.emit ? 16384 : 8192);
#pragma unroll 1
        for (int32_t t = int32_t(run.t0), n = 0; n < chunks; ++n, t += kC) {
          if (!wait(ctl->kq_free[ks], ks_turn)) break;
          uint8_t *dst = smem + ks * kTileKQ;
          uint64_t &full = ctl->kq_full[ks];
          mbar_arrive_expect_tx(&full, kq_bytes);
#pragma unroll 1
          for (int b = 0; b < kb; ++b) {
            tma_load_3d(dst + b * 16384, &mk, &full, 64 * b, hk, t);
            if (run.emit) tma_load_3d(dst + b * 16384 + 8192, &mq, &full, 64 * b, hk, t);
          }
          ++kq;
          if (++ks == kKQ) ks = 0, ks_turn ^= 1;
          if (run.identity) continue;
          if (!wait(ctl->v_free[vs_], vs_turn)) break;
          mbar_arrive_expect_tx(&ctl->v_full[vs_], vb * kBlockV);
#pragma unroll 1
          for (int b = 0; b < vb; ++b)
            tma_load_3d(smem + kAtV + (vs_ + b) * kBlockV, &mv, &ctl->v_full[vs_], 64 * b, h, t);
          ++vs;
          if (vs_ == uint32_t(v_last)) vs_ = 0, vs_turn ^= 1;
          else ++vs_;
        }
        // every load issued has landed before the CTA may end
#pragma unroll 1
        for (int i = kq > kKQ ? kq - kKQ : 0; i < kq; ++i) wait(ctl->kq_full[i % kKQ], i / kKQ);
#pragma unroll 1
        for (int i = vs > v_last ? vs - v_last - 1 : 0; i < vs; ++i) wait(ctl->v_full[i & v_last], i >> v_last);
      }
    } else if (warp == 1) {
      // ---- the chain: X = K S, U = T' V + T'' X, K^T U'
      const bool leader = elect_lane();
      const uint32_t base = smem_u32(smem);
      constexpr uint32_t i64 = umma_idesc_bf16(128, 64, false, false, false);
      const uint32_t iD = umma_idesc_bf16(128, a.d_k > 64 ? 128 : 64, false, true, false);
      constexpr uint32_t iV = umma_idesc_bf16(128, 64, true, false, false);
      uint32_t stage = 0;
#pragma unroll 1
      for (int n = 0; n < chunks; ++n) {
        // nothing, as the compiler does not see: addresses made with it are not kept in registers over the loop,
        // forty of them
        const uint32_t none = uint32_t(n) >> 28;
        const uint32_t tS = tmem + none, tX = tS + 128, tU = tS + 192;
        const uint64_t dT = desc_k(base + none + kAtT), dTW = dT + (2 * kTileT >> 4);  // T', then T'', each hi and lo
        const uint32_t tile = base + stage * kTileKQ;
        const uint64_t dK = desc_k(tile), dKT = desc_mn(tile, 16384);
        uint64_t &kq_full = ctl->kq_full[stage], &kq_free = ctl->kq_free[stage];
        if (!wait_warp(kq_full, n / kKQ)) break;
        if (++stage == kKQ) stage = 0;
        if (partial && n + 1 == chunks && !wait_warp(ctl->zeroed, 0)) break;
        // T' V, while S is made
        if (!wait_warp(ctl->t_full, n)) break;
        if (!run.identity && !wait_warp(ctl->v_full[n & v_last], n >> v_last)) break;
        if (n > 0 && !wait_warp(ctl->d_done, n - 1)) break;  // U' of chunk n - 1 is read
        if (!run.identity) {
          tc_fence_after();
          const uint64_t dV = desc_mn(base + kAtV + (n & v_last) * kBlockV, kBlockV);
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            mma_ss(leader, tU, dV + 128 * ks, dT + 2 * ks, iV, ks > 0);
            mma_ss(leader, tU, dV + 128 * ks, dT + (kTileT >> 4) + 2 * ks, iV, 1);
          }
          mma_commit(leader, ctl->v_free[n & v_last]);
        }
        // Each product begins with the steps whose operands come first: S, X and U' by halves of each thread's
        // columns (steps 0, 1, 4, 5 of S, then 2, 3, 6, 7; steps 0, 2, then 1, 3 of the tokens).
        bool ok = true;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          ok = ok && wait_warp(ctl->s_full[p], n);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int m = 0; m < 4; ++m) {
            const int ks = 4 * (m >> 1) + 2 * p + (m & 1);
            if (ks >= nk) break;
            const uint64_t b = dK + ((ks >> 2) * 1024 + (ks & 3) * 2);
            mma_ts(leader, tX, tS + 16 * ks, b, i64, ks > 0);
            mma_ts(leader, tX, tS + 16 * ks + 8, b, i64, 1);
          }
        }
        if (!ok) break;
        mma_commit(leader, ctl->x_done);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          ok = ok && wait_warp(ctl->r_full[p], n);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int ks = p; ks < 4; ks += 2) {
            mma_ts(leader, tU, tX + 16 * ks, dTW + 2 * ks, i64, ks > 0 || !run.identity);
            mma_ts(leader, tU, tX + 16 * ks, dTW + (kTileT >> 4) + 2 * ks, i64, 1);
            mma_ts(leader, tU, tX + 16 * ks + 8, dTW + 2 * ks, i64, 1);
          }
        }
        if (!ok) break;
        mma_commit(leader, ctl->u_done);
        mma_commit(leader, ctl->t_free[n & 1]);
        if (run.emit && !wait_warp(ctl->xq_done, n)) break;  // Q S has read S
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          ok = ok && wait_warp(ctl->up_full[p], n);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int ks = p; ks < 4; ks += 2) {
            mma_ts(leader, tS, tU + 16 * ks, dKT + 128 * ks, iD, ks > 0);
            mma_ts(leader, tS, tU + 16 * ks + 8, dKT + 128 * ks, iD, 1);
          }
        }
        if (!ok) break;
        mma_commit(leader, ctl->d_done);
        mma_commit(leader, kq_free);  // (K K^T, Q K^T and Q S were done before)
      }
      // no MMA is in flight when tensor memory is freed
      mma_commit(leader, ctl->drain);
      if (leader) mbar_wait(&ctl->drain, 0, err_word, DEVERR_MMA_TIMEOUT);
    } else if (warp == 3) {
      // ---- the other products
      const bool leader = elect_lane();
      const uint32_t base = smem_u32(smem);
      constexpr uint32_t i64 = umma_idesc_bf16(128, 64, false, false, false);
      constexpr uint32_t i32 = umma_idesc_bf16(128, 32, false, false, false);
      const uint64_t dKQ = desc_k(base);
      auto gram = [&](int n) -> bool {  // rows 0 .. 63: K K^T, 64 .. 127: Q K^T
        if (!wait_warp(ctl->kq_full[n % kKQ], n / kKQ)) return false;
        if (partial && n + 1 == chunks && !wait_warp(ctl->zeroed, 0)) return false;
        if (n > 0 && !wait_warp(ctl->gram_read, n - 1)) return false;
        tc_fence_after();
        const uint64_t d = dKQ + (n % kKQ) * (kTileKQ >> 4);
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          if (ks >= nk) break;
          const uint64_t b = d + ((ks >> 2) * 1024 + (ks & 3) * 2);
          mma_ss(leader, tG, b, b, i64, ks > 0);
        }
        mma_commit(leader, ctl->gram_done[n & 1]);
        return true;
      };
      // K K^T and Q K^T two chunks ahead, while X is split; Q S while U becomes U'; P U while S is made
#pragma unroll 1
      for (int n = -2; n < chunks; ++n) {
        const bool here = run.emit && n >= 0;
        if (here && !wait_warp(ctl->x_done, n)) break;
        if (n + 2 < chunks && !gram(n + 2)) break;
        if (!here) continue;
        if (!wait_warp(ctl->u_done, n)) break;
        if (n > 0 && !wait_warp(ctl->o_read, n - 1)) break;
        tc_fence_after();
        const uint64_t d = dKQ + ((n % kKQ) * (kTileKQ >> 4) + (8192 >> 4));
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          if (ks >= nk) break;
          const uint64_t b = d + ((ks >> 2) * 1024 + (ks & 3) * 2);
          mma_ts(leader, tXQ, tS + 16 * ks, b, i64, ks > 0);
          mma_ts(leader, tXQ, tS + 16 * ks + 8, b, i64, 1);
        }
        mma_commit(leader, ctl->xq_done);
        const uint64_t dPn = desc_k(base + kAtP) + n % kP * (kTileP >> 4);
        if (!wait_warp(ctl->d_done, n)) break;  // (U for the read-out came before)
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const uint32_t hi = tUH + 8 * ks, lo = hi + 32;
          if (ks < 2) {  // both halves of the rows; then lo's upper half
            mma_ts(leader, tO, hi, dPn + 2 * ks, i64, ks > 0);
            mma_ts(leader, tO, lo, dPn + 2 * ks, i64, 1);
            mma_ts(leader, tO, hi, dPn + 2 * ks + 4, i32, 1);
          } else {
            mma_ts(leader, tO + 32, hi, dPn + 2 * ks + (4096 >> 4), i32, 1);
            mma_ts(leader, tO + 32, lo, dPn + 2 * ks + (4096 >> 4), i32, 1);
          }
          mma_ts(leader, tO + 32, hi, dPn + 2 * ks + (8192 >> 4), i32, 1);
        }
        mma_commit(leader, ctl->o_done);
        mma_commit(leader, ctl->p_free[n % kP]);
      }
      mma_commit(leader, ctl->drain);
      if (leader) mbar_wait(&ctl->drain, 0, err_word, DEVERR_MMA_TIMEOUT);
    } else if (warp == 2) {
      // ---- decay tables: tokens 2 lane and 2 lane + 1
      const bool per_token = a.per_token != 0;
      const float constant = per_token ? 0.f : a.log_decay[h];
      float g[2] = {}, b[2] = {};
#pragma unroll 1
      for (int n = -1; n < chunks; ++n) {
        double G[2];
        const float beta[2] = {b[0], b[1]};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const double x = double(g[e]) * kLog2e;
          G[e] = x < kMinLog2 ? kMinLog2 : x;  // a NaN stays
          const int i = (n + 1) * kC + 2 * lane + e;  // the next chunk's
          g[e] = i < len ? (per_token ? a.log_decay[(run.t0 + i) * a.H + h] : constant) : 0.f;
          b[e] = i < len ? a.beta[(run.t0 + i) * a.H + h] : 0.f;
        }
        if (n < 0) continue;
        double sum = G[0] + G[1];
#pragma unroll 1
        for (int o = 1; o < 32; o <<= 1) {
          const double up = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += up;
        }
        const double end = __shfl_sync(0xffffffffu, sum, 31), middle = __shfl_sync(0xffffffffu, sum, 15);
        G[0] = sum - G[1], G[1] = sum;
        Table &w = tab[n % kTabs];
        if (!wait_warp(ctl->tab_free[n % kTabs], (n / kTabs) ^ 1)) break;
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {
          const int i = 2 * lane + e;
          const double x = e == 0 ? G[0] : G[1];
          const float hi = float(x), f = ex2(hi);
          w.g[i] = hi, w.g_lo[i] = float(x - double(hi));
          w.f[i] = -f;
          w.out[i] = a.scale * f;
          w.cross[i] = ex2(float(lane < 16 ? middle - x : x - middle));
          w.w[i] = ex2(float(end - x));
          w.beta[i] = e == 0 ? beta[0] : beta[1];
        }
        if (lane == 0) w.whole = unbiased_decay(float(end * kLn2), n);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->tab_full[n % kTabs]);
      }
    }
  } else if (warp < 12) {
    registers_down<72>();
    // ---- A, its inverse and P: warps 4 to 7 of the even chunks, 8 to 11 of the odd ones
    const int w = warp & 3, group = (warp >> 2) - 1, wt = tid & 127;
    float *const sA = reinterpret_cast<float *>(smem + kAtA) + group * (kC * kStrideA);
    const uint32_t row = uint32_t(32 * w) << 16;
    const int hb = w & 1, t = 32 * hb + lane;  // this thread's row of K K^T (warps 0, 1) or Q K^T (2, 3)
    auto sync = [&]() { named_bar_sync(1 + group, 128); };
    auto sync_pair = [&]() { named_bar_sync(3 + 2 * group + (w >> 1), 64); };
    // what lies above the diagonal blocks of T' and T'' is zero and stays it (both groups write it)
    for (int i = wt; i < 4 * 32 * 4; i += 128)
      *reinterpret_cast<uint4 *>(smem + kAtT + (i >> 7) * kTileT + sw128_chunk((i >> 2) & 31, 4 + (i & 3), 0, kC)) =
          make_uint4(0, 0, 0, 0);
    // rows of the last chunk behind the run: another sequence's, whose infinities times zero would not vanish
    auto clear_rows = [&](uint8_t *tile, uint32_t block, int blocks, int part) {
#pragma unroll 1
      for (int i = part * 8 + wt; i < kC * 8; i += 128) {  // 16-byte pieces of a 64-channel block
        *reinterpret_cast<uint4 *>(tile + i * 16) = make_uint4(0, 0, 0, 0);
        if (blocks > 1) *reinterpret_cast<uint4 *>(tile + block + i * 16) = make_uint4(0, 0, 0, 0);
      }
      fence_proxy_async_smem();
    };
#pragma unroll 1
    for (int n = group; n < chunks; n += 2) {
      bool ok = true;  // a warp whose wait gives up comes to the next barrier, where all learn of it
      const bool clear = partial && n + 1 == chunks;
      if (clear) {
        ok = wait_warp(ctl->kq_full[n % kKQ], n / kKQ);
        if (ok) clear_rows(smem + n % kKQ * kTileKQ, 16384, kb, len - n * kC);
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->zeroed);
      }
      const Table &tb = tab[n % kTabs];
      ok = ok && wait_warp(ctl->tab_full[n % kTabs], n / kTabs) && wait_warp(ctl->gram_done[n & 1], n >> 1) &&
           (!run.emit || n < kP || wait_warp(ctl->p_free[n % kP], n / kP - 1));
      tc_fence_after();
      if (named_bar_or(1 + group, 128, !ok)) break;
      // row t of A or P, entries i < t or i <= t; selected away, not multiplied, behind them, where an
      // exponential may be infinite
      const int end = w < 2 ? t : run.emit ? t + 1 : 0;
      const float factor = w < 2 ? tb.beta[t] : a.scale;
      const float2 g2 = make_float2(tb.g[t], tb.g[t]), l2 = make_float2(tb.g_lo[t], tb.g_lo[t]);
      uint8_t *P = smem + kAtP + n % kP * kTileP;
#pragma unroll 1
      for (int c = 0; c < 32 * hb + 32; c += 16) {
        float x[16];
        tmem_ld16_wait(tG + row + c, x);
        if (c < 32 * hb) {  // across the middle: a factor of the row times one of the column, none above one while g <= 0
          const float e = factor * tb.cross[t];
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(&tb.cross[c + j]);
            const float2 y0 = f2_mul(make_float2(x[j], x[j + 1]), f2_mul(make_float2(f.x, f.y), make_float2(e, e)));
            const float2 y1 = f2_mul(make_float2(x[j + 2], x[j + 3]), f2_mul(make_float2(f.z, f.w), make_float2(e, e)));
            x[j] = y0.x, x[j + 1] = y0.y, x[j + 2] = y1.x, x[j + 3] = y1.y;
          }
        } else {
          constexpr float2 minus = {-1.f, -1.f};
#pragma unroll
          for (int j = 0; j < 16; j += 4) {
            const float4 g = *reinterpret_cast<const float4 *>(&tb.g[c + j]), l = *reinterpret_cast<const float4 *>(&tb.g_lo[c + j]);
            const float2 d0 = f2_add(f2_fma(make_float2(g.x, g.y), minus, g2), f2_fma(make_float2(l.x, l.y), minus, l2));
            const float2 d1 = f2_add(f2_fma(make_float2(g.z, g.w), minus, g2), f2_fma(make_float2(l.z, l.w), minus, l2));
            const float d[4] = {d0.x, d0.y, d1.x, d1.y};
#pragma unroll
            for (int e = 0; e < 4; ++e) x[j + e] = c + j + e < end ? factor * ex2(d[e]) * x[j + e] : 0.f;
          }
        }
        if (w < 2) {
#pragma unroll
          for (int j = 0; j < 16; j += 4)
            *reinterpret_cast<float4 *>(&sA[t * kStrideA + c + j]) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
        } else if (run.emit) {
#pragma unroll
          for (int j = 0; j < 16; j += 8) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) split_pair(x[j + 2 * e], x[j + 2 * e + 1], hi[e], lo[e]);
            const uint32_t o = sw128_chunk(t, (c + j) >> 3, 0, kC);
            *reinterpret_cast<uint4 *>(P + o) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            *reinterpret_cast<uint4 *>(P + (hb == 0 ? o ^ 64 : o + 4096)) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&ctl->gram_read);
      sync();
      // The inverse of I + A in place: T_21 = -T_22 (A_21 T_11) from blocks of 8 to 16, 32 and 64. A_21 T_11
      // stands at Y, the block above the diagonal, which nobody else uses.
      float *const Y = sA + 32;
      {  // warp w: its block of 16
        float *const D = sA + 16 * w * (kStrideA + 1);
        const int b8 = lane & 8, j = lane & 7;
        const float *L = D + b8 * (kStrideA + 1);
        float4 l[7][2];
#pragma unroll
        for (int r = 1; r < 8; ++r) {
          l[r - 1][0] = *reinterpret_cast<const float4 *>(&L[r * kStrideA]);
          l[r - 1][1] = *reinterpret_cast<const float4 *>(&L[r * kStrideA + 4]);
        }
        float x[8];
        x[0] = j == 0 ? 1.f : 0.f;
#pragma unroll
        for (int r = 1; r < 8; ++r) {
          const float ls[8] = {l[r - 1][0].x, l[r - 1][0].y, l[r - 1][0].z, l[r - 1][0].w,
                               l[r - 1][1].x, l[r - 1][1].y, l[r - 1][1].z, l[r - 1][1].w};
          float sum = j == r ? 1.f : 0.f;
#pragma unroll
          for (int i = 0; i < r; ++i) sum = fmaf(-ls[i], x[i], sum);
          x[r] = sum;
        }
        __syncwarp();
        if (lane < 16) {
#pragma unroll
          for (int r = 0; r < 8; ++r) D[(b8 + r) * kStrideA + b8 + j] = x[r];
        }
        __syncwarp();
        const int r = lane >> 2, c = 2 * (lane & 3);
        auto product = [&](const float *x, const float *m, int stride, float sign) {
          float2 y = make_float2(0.f, 0.f);
          const float4 a0 = *reinterpret_cast<const float4 *>(&x[r * kStrideA]);
          const float4 a1 = *reinterpret_cast<const float4 *>(&x[r * kStrideA + 4]);
          const float as[8] = {a0.x, a0.y, a0.z, a0.w, a1.x, a1.y, a1.z, a1.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 b = *reinterpret_cast<const float2 *>(&m[i * stride + c]);
            y.x = fmaf(sign * as[i], b.x, y.x), y.y = fmaf(sign * as[i], b.y, y.y);
          }
          return y;
        };
        float *const y8 = Y + 8 * w * kStrideA;
        const float2 y = product(D + 8 * kStrideA, D, kStrideA, 1.f);
        *reinterpret_cast<float2 *>(&y8[r * kStrideA + c]) = y;
        __syncwarp();
        const float2 z = product(D + 8 * (kStrideA + 1), y8, kStrideA, -1.f);
        *reinterpret_cast<float2 *>(&D[(8 + r) * kStrideA + c]) = z;
      }
      sync_pair();
      {  // pairs of warps: a block of 32, eight columns each; T_11's columns from 8 on have no rows above 8
        float *const D = sA + 32 * (w >> 1) * (kStrideA + 1), *const y16 = Y + 16 * (w >> 1) * kStrideA;
        const int c = 8 * (w & 1);
#pragma unroll 1
        for (int p = 0; p < 2; ++p) {
          block_product<1, 1>(D + 16 * kStrideA + 16 * p, (p == 0 ? D : y16) + c, (p == 0 ? y16 : D + 16 * kStrideA) + c,
                              p != 0, lane);
          if (p == 0) sync_pair();
        }
      }
      sync();
      {  // all: 16 rows and 16 columns each
        const int r = 16 * (w & 1), c = 16 * (w >> 1);
#pragma unroll 1
        for (int p = 0; p < 2; ++p) {
          block_product<2, 2>(sA + (32 + r) * kStrideA + 32 * p, (p == 0 ? sA : Y) + c,
                              (p == 0 ? Y + r * kStrideA : sA + (32 + r) * kStrideA) + c, p != 0, lane);
          if (p == 0) sync();
        }
      }
      // T' = T diag(beta) and T'' = -T' diag(e^G) as pairs, 8 columns at a time: 4 pieces of each upper row, 8 of
      // each lower one. Their buffers: the products of chunk n - 1 are done.
      ok = n == 0 || wait_warp(ctl->t_free[(n - 1) & 1], (n - 1) >> 1);
      if (clear && !run.identity) {
        ok = ok && wait_warp(ctl->v_full[n & v_last], n >> v_last);
        if (ok) clear_rows(smem + kAtV + (n & v_last) * kBlockV, kBlockV, vb, len - n * kC);
      }
      if (named_bar_or(1 + group, 128, !ok)) break;
#pragma unroll 1
      for (int m = 0; m < 3; ++m) {
        const int r = m == 0 ? wt >> 2 : 32 + (((m - 1) * 128 + wt) >> 3), c = 8 * (m == 0 ? wt & 3 : wt & 7);
        uint8_t *T = smem + kAtT + sw128_chunk(r, c >> 3, 0, kC);
        float2 y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          y[e] = f2_mul(*reinterpret_cast<const float2 *>(&sA[r * kStrideA + c + 2 * e]), *reinterpret_cast<const float2 *>(&tb.beta[c + 2 * e]));
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            split_pair(y[e].x, y[e].y, hi[e], lo[e]);
            y[e] = f2_mul(y[e], *reinterpret_cast<const float2 *>(&tb.f[c + 2 * e]));
          }
          *reinterpret_cast<uint4 *>(T + which * 2 * kTileT) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4 *>(T + which * 2 * kTileT + kTileT) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      fence_proxy_async_smem();
      sync();  // A is free again
      if (lane == 0) {
        mbar_arrive(&ctl->t_full);
        mbar_arrive(&ctl->tab_free[n % kTabs]);
      }
    }
  } else if (warp < 16) {
    registers_down<40>();
    // ---- the output: value channel c, O = scale (Q S) + P U
    if (run.emit) {
      const int w = warp & 3, c = 32 * w + lane;
      const uint32_t row = uint32_t(32 * w) << 16;
      constexpr int kEs = kOutBF16 ? 2 : 4;
      const uint32_t step = uint32_t(a.H) * uint32_t(a.d_v) * kEs;  // from token to token; 16 of them are below 2^32 (see delta_plan)
      uint8_t *out = static_cast<uint8_t *>(a.out) + ((run.t0 * a.H + h) * a.d_v + c) * kEs;
#pragma unroll 1
      for (int n = 0; n < chunks; ++n) {
        const Table &tb = tab[n % kTabs];
        if (!wait_warp(ctl->tab_full[n % kTabs], n / kTabs)) break;
        if (!wait_warp(ctl->o_done, n)) break;
        tc_fence_after();
#pragma unroll 1
        for (int t = 0; t < kC; t += 8, out += uint64_t(step) * 8) {
          const int part = c < a.d_v ? len - n * kC - t : 0;
          float x[8], o[8];
          tmem_ld8(tXQ + row + t, x);
          tmem_ld8(tO + row + t, o);
          tmem_ld_wait(x, o);
#pragma unroll
          for (int j = 0; j < 8; j += 4) {
            const float4 f = *reinterpret_cast<const float4 *>(&tb.out[t + j]);
            const float2 y0 = f2_fma(make_float2(f.x, f.y), make_float2(x[j], x[j + 1]), make_float2(o[j], o[j + 1]));
            const float2 y1 = f2_fma(make_float2(f.z, f.w), make_float2(x[j + 2], x[j + 3]), make_float2(o[j + 2], o[j + 3]));
            x[j] = y0.x, x[j + 1] = y0.y, x[j + 2] = y1.x, x[j + 3] = y1.y;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < part) store_elem<kOutBF16>(out + uint64_t(uint32_t(j) * step), 0, x[j]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&ctl->o_read);
          mbar_arrive(&ctl->tab_free[n % kTabs]);
        }
      }
    }
  } else {
    registers_up<120>();
    // ---- the state: value channel c, key rows 64 half .. + 63; tokens 32 half .. + 31 of X and U'
    const int w = warp & 3, half = (warp - 16) >> 2, c = 32 * w + lane;
    const uint32_t row = uint32_t(32 * w) << 16;
    const uint32_t rS = tS + row + 64 * half, rX = tX + row + 32 * half, rU = tU + row + 32 * half;
    const uint32_t rUH = tUH + row + 16 * half;
    const bool rows_on = 64 * half < a.d_k;  // else this half of the state is zero throughout
    // The entering state goes to where K^T U' of a chunk before would be, for the first step to take it from.
    // (By loops over 16 rows, like the way out: code that runs once is fetched once, from far.)
    if (rows_on) {
#pragma unroll 1
      for (int i = 0; i < 64; i += 16) {
        float x[16];
        const int r0 = 64 * half + i;
        const float *from = run.from + int64_t(r0) * run.from_width + c;
        const int rows = run.from != nullptr && c < a.d_v ? a.d_k - r0 : 0;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          x[j] = run.identity && r0 + j == c ? 1.f : 0.f;
          if (j < rows) x[j] = from[uint32_t(j) * uint32_t(run.from_width)];
        }
        tmem_st16(rS + i, x);
      }
      tmem_st_wait();
    }
    float S[64];
#pragma unroll
    for (int i = 0; i < 64; ++i) S[i] = 0.f;
    // 16 values as the A operand of one step: 8 columns of hi pairs, 8 of lo pairs
    auto put_pair = [&](uint32_t at, const float *x) {
      float hi[8], lo[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t h, l;
        split_pair(x[2 * j], x[2 * j + 1], h, l);
        hi[j] = __uint_as_float(h), lo[j] = __uint_as_float(l);
      }
      tmem_st8(at, hi);
      tmem_st8(at + 8, lo);
    };
    auto give = [&](uint64_t &bar) {  // what this warp wrote to tensor memory is there for the MMAs
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar);
    };
#pragma unroll 1
    for (int n = -1;; ++n) {
      const Table &tb = tab[n & (kTabs - 1)];
      if (n >= 0) {
        if (n >= chunks) break;
        if (!wait_warp(ctl->tab_full[n % kTabs], n / kTabs)) break;
        if (run.emit && n > 0 && !wait_warp(ctl->o_done, n - 1)) break;  // the read-out's U of chunk n - 1 is read
        // X = K S, split where it stands
        if (!wait_warp(ctl->x_done, n)) break;
        tc_fence_after();
#pragma unroll 1
        for (int p = 0; p < 2; ++p) {
          float x[16];
          tmem_ld16_wait(rX + 16 * p, x);
          put_pair(rX + 16 * p, x);
          give(ctl->r_full[p]);
        }
        // U, and U' over it
        if (!wait_warp(ctl->u_done, n)) break;
        tc_fence_after();
#pragma unroll 1
        for (int p = 0; p < 2; ++p) {
          float x[16];
          tmem_ld16_wait(rU + 16 * p, x);
          if (run.emit) {
            float hi[8], lo[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              uint32_t h, l;
              split_pair(x[2 * j], x[2 * j + 1], h, l);
              hi[j] = __uint_as_float(h), lo[j] = __uint_as_float(l);
            }
            tmem_st8(rUH + 8 * p, hi);
            tmem_st8(rUH + 32 + 8 * p, lo);
          }
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            const float2 y = f2_mul(make_float2(x[j], x[j + 1]), *reinterpret_cast<const float2 *>(&tb.w[32 * half + 16 * p + j]));
            x[j] = y.x, x[j + 1] = y.y;
          }
          put_pair(rU + 16 * p, x);
          give(ctl->up_full[p]);
        }
        if (!wait_warp(ctl->d_done, n)) break;
        tc_fence_after();
      }
      // S <- e^{G_C} S + K^T U'
      const float2 whole = make_float2(n < 0 ? 0.f : tb.whole, n < 0 ? 0.f : tb.whole);
#pragma unroll
      for (int i = 0; i < 64; i += 32) {
        if (rows_on) {
          float d[32];
          tmem_ld16(rS + i, d);
          tmem_ld16(rS + i + 16, d + 16);
          tmem_ld_wait(d);
#pragma unroll
          for (int j = 0; j < 32; j += 2) {
            const float2 y = f2_fma(whole, make_float2(S[i + j], S[i + j + 1]), make_float2(d[j], d[j + 1]));
            S[i + j] = y.x, S[i + j + 1] = y.y;
          }
          if (n + 1 < chunks) put_pair(rS + i, &S[i]), put_pair(rS + i + 16, &S[i + 16]);
        }
        if (n + 1 < chunks) give(ctl->s_full[i >> 5]);
      }
      if (n >= 0) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->tab_free[n % kTabs]);
      }
    }
    if (run.to != nullptr && rows_on) {
#pragma unroll
      for (int i = 0; i < 64; i += 16) tmem_st16(rS + i, &S[i]);
      tmem_st_wait();
#pragma unroll 1
      for (int i = 0; i < 64; i += 16) {
        float x[16];
        tmem_ld16_wait(rS + i, x);
        const int r0 = 64 * half + i, rows = c < run.width ? a.d_k - r0 : 0;
        float *to = run.to + int64_t(r0) * run.width + c;
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (j < rows) to[uint32_t(j) * uint32_t(run.width)] = x[j];
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && ctl->gave_up != 0) raise_device_error(err_word, DEVERR_MMA_TIMEOUT);
  if (warp == 1) {
    tmem_relinquish();
    tmem_dealloc(tmem, 512);
  }
}

template <bool kOutBF16>
cudaError_t launch_pass(const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv, const DeltaArgs &a, int pass,
                        cudaStream_t stream) {
  const auto kern = delta_chunked_kernel<kOutBF16>;
  // the kernel's shared memory, granted once per device (bit d for device d; past 63 at every launch)
  static std::atomic<uint64_t> granted;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (bit == 0 || (granted.load(std::memory_order_acquire) & bit) == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kBytes));
    if (e != cudaSuccess) return e;
    granted.fetch_or(bit, std::memory_order_release);
  }
  const unsigned pieces = unsigned(a.plan.inner + a.num_seqs) + (pass == 1 && a.plan.seg_len != 0 ? unsigned(a.plan.inner) : 0u);
  kern<<<pieces * unsigned(a.H), kThreads, kBytes, stream>>>(mq, mk, mv, a, pass, device_error_word());
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_order_longest_first(const int32_t *cu_seqlens, int num_seqs, int32_t *order, cudaStream_t stream);

cudaError_t launch_delta_chunked(const DeltaArgs &a, bool out_bf16, cudaStream_t stream) {
  LinearArgs in{};  // q, k, v or their padded copies
  in.q = a.q, in.k = a.k, in.v = a.v;
  cudaError_t e = cudaSuccess;
  if (a.plan.pad) {
    in.workspace = a.workspace, in.total = a.total;
    in.H = a.H, in.H_k = a.H_k, in.d_k = a.d_k, in.d_v = a.d_v;
    in.plan.pad_q = a.plan.pad_q, in.plan.pad_k = a.plan.pad_k, in.plan.pad_v = a.plan.pad_v;
    e = launch_linear_pad(in, stream);
    if (e != cudaSuccess) return e;
  }
  const int pk = delta_up8(a.d_k), pv = delta_up8(a.d_v);
  CUtensorMap mq, mk, mv;
  if (!tensor_map_3d(&mq, in.q, true, a.total, a.H_k, pk, 64, kC, true) ||
      !tensor_map_3d(&mk, in.k, true, a.total, a.H_k, pk, 64, kC, true) ||
      !tensor_map_3d(&mv, in.v, true, a.total, a.H, pv, 64, kC, true))
    return cudaErrorInvalidValue;
  const auto pass = [&](int which) {
    return out_bf16 ? launch_pass<true>(mq, mk, mv, a, which, stream) : launch_pass<false>(mq, mk, mv, a, which, stream);
  };
  if (a.plan.order) e = launch_order_longest_first(a.cu, a.num_seqs, reinterpret_cast<int32_t *>(a.workspace + a.plan.ends), stream);
  if (e == cudaSuccess) e = pass(1);
  if (e != cudaSuccess || a.plan.seg_len == 0) return e;
  e = launch_delta_chain(a, stream);
  return e == cudaSuccess ? pass(3) : e;
}

}  // namespace kda
