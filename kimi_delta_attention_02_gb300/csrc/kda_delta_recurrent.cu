// kda_delta_recurrent.cu -- the gated delta rule with one decay per head in fp32 on the CUDA cores,
// four tokens at a time. It takes every size and both dtypes (fp32 inputs, short sequences, head sizes
// that TMA cannot address); the tensor-core kernel is the fast path of long bf16 sequences.
//
// For tokens 0 .. 3 of a block that enters with S, E_t = e^{g_0 + .. + g_t} and D_ti = e^{g_{i+1} + .. + g_t}:
//     y_t = S^T k_t,  z_t = S^T q_t
//     u_t = beta_t (v_t - E_t y_t) - sum_{i<t} beta_t D_ti (k_t . k_i) u_i
//     o_t = scale (E_t z_t + sum_{i<=t} D_ti (q_t . k_i) u_i)
//     S  <- E_3 S + sum_i k_i (D_3i u_i)
// so the eight row sums of a block meet in one exchange and the state is read and written once: 13
// multiply-adds per entry for four tokens (16 one by one) and a quarter of the waits. No decay is the
// difference of two sums.
//
// A warp holds 4 kNC value columns: lane (cl, rl) owns kNC of them and the key rows 32 j + 4 rl + 0..3,
// two rows to a packed fp32 instruction. q, k, v pass through shared memory 16 tokens at a time, the
// next 16 waiting in registers; warp w forms the products k.k and q.k of the stage's block w.
#include <type_traits>

#include "kda_delta.cuh"

namespace kda {
namespace {

constexpr int kTok = 16;  // tokens per stage
constexpr int kThr = 128;

struct Block {  // of four tokens
  float E[4];       // from the block's start
  float beta[4];
  float rest[4];    // D_3i
  float whole;      // E_3 as the state's factor
  float pad[3];
  float kk[4][4];   // beta_t D_ti (k_t . k_i), i < t
  float qk[4][4];   // D_ti (q_t . k_i), i <= t
};

template <bool kInBF16, bool kOutBF16, int kRows, int kNC>
__global__ void __launch_bounds__(kThr) delta_recurrent_kernel(const DeltaArgs a) {
  constexpr int kDK = 8 * kRows, kCols = 16 * kNC;
  __shared__ __align__(16) float s_k[2][kTok][kDK], s_q[2][kTok][kDK];
  __shared__ __align__(16) float s_v[2][kTok][kCols];
  __shared__ __align__(16) Block s_block[kTok / 4];
  __shared__ float s_g[2][kTok], s_beta[2][kTok];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int rl = lane & 7, cl = lane >> 3;
  const int h = blockIdx.x % a.H, n = blockIdx.x / a.H, hk = h / (a.H / a.H_k);
  const int col0 = blockIdx.y * kCols, cw = 4 * kNC * w + kNC * cl, col = col0 + cw;
  const int64_t t0 = a.cu[n], t1 = a.cu[n + 1];

  // the state: S[c][2 j + p] holds rows 32 j + 4 rl + 2 p, + 1 of column col + c
  float2 S[kNC][kRows / 2];
  const int64_t at_state = (int64_t(n) * a.H + h) * a.d_k * a.d_v;
#pragma unroll
  for (int p = 0; p < kRows / 2; ++p) {
    const int r = 32 * (p >> 1) + 4 * rl + 2 * (p & 1);
    auto at = [&](int row, int c) {
      return a.init_state != nullptr && row < a.d_k && col + c < a.d_v
                 ? a.init_state[at_state + int64_t(row) * a.d_v + col + c] : 0.f;
    };
#pragma unroll
    for (int c = 0; c < kNC; ++c) S[c][p] = make_float2(at(r, c), at(r + 1, c));
  }

  // global -> registers -> shared memory, a stage of kTok tokens at a time (as stored: a conversion
  // here would wait for the load)
  using Elem = std::conditional_t<kInBF16, uint16_t, float>;
  auto raw = [](const void *p, int64_t at) { return static_cast<const Elem *>(p)[at]; };
  auto value = [](Elem x) {
    if constexpr (kInBF16) return bf16_to_f32(x);
    else return x;
  };
  constexpr int kKeys = kTok * kDK / kThr, kVals = kTok * kCols / kThr;
  Elem rk[kKeys], rq[kKeys], rv[kVals];
  float r_g = 0.f, r_beta = 0.f;
  auto fetch = [&](int64_t t) {  // tokens t .. t + kTok - 1; zeros past the sequence
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const int64_t tt = t + i * (kThr / kDK) + tid / kDK;
      const int c = tid % kDK;
      const bool ok = tt < t1 && c < a.d_k;
      const int64_t at = (tt * a.H_k + hk) * a.d_k + c;
      rk[i] = ok ? raw(a.k, at) : Elem(0);
      rq[i] = ok ? raw(a.q, at) : Elem(0);
    }
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      const int64_t tt = t + (i * kThr + tid) / kCols;
      const int c = col0 + tid % kCols;
      rv[i] = tt < t1 && c < a.d_v ? raw(a.v, (tt * a.H + h) * a.d_v + c) : Elem(0);
    }
    if (tid < kTok) {
      const bool ok = t + tid < t1;
      r_g = ok ? a.log_decay[a.per_token ? (t + tid) * a.H + h : h] : 0.f;
      r_beta = ok ? a.beta[(t + tid) * a.H + h] : 0.f;
    }
  };
  auto stage = [&](int b) {
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      s_k[b][i * (kThr / kDK) + tid / kDK][tid % kDK] = value(rk[i]);
      s_q[b][i * (kThr / kDK) + tid / kDK][tid % kDK] = value(rq[i]);
    }
#pragma unroll
    for (int i = 0; i < kVals; ++i) s_v[b][(i * kThr + tid) / kCols][tid % kCols] = value(rv[i]);
    if (tid < kTok) s_g[b][tid] = r_g, s_beta[b][tid] = r_beta;
  };
  // warp w: the products and decays of the stage's block w
  auto form_block = [&](int b, int64_t step) {
    Block &B = s_block[w];
    float4 k4[4], q4[4];
    const bool on = 4 * lane < kDK;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      k4[t] = on ? *reinterpret_cast<const float4 *>(&s_k[b][4 * w + t][4 * lane]) : make_float4(0.f, 0.f, 0.f, 0.f);
      q4[t] = on ? *reinterpret_cast<const float4 *>(&s_q[b][4 * w + t][4 * lane]) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    auto dot = [](float4 x, float4 y) { return fmaf(x.x, y.x, x.y * y.y) + fmaf(x.z, y.z, x.w * y.w); };
    float sums[16];  // 10 of q.k (row t from t (t + 1) / 2), then 6 of k.k (row t from t (t - 1) / 2)
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i <= t; ++i) {
        sums[t * (t + 1) / 2 + i] = dot(q4[t], k4[i]);
        if (i < t) sums[10 + t * (t - 1) / 2 + i] = dot(k4[t], k4[i]);
      }
    const float sum = lane_sums<16>(sums, lane);  // lanes 2 e, 2 e + 1: entry e
    const int e = lane >> 1;
    const bool is_qk = e < 10;
    const int m = is_qk ? e : e - 10;
    int t = is_qk ? (m >= 6 ? 3 : m >= 3 ? 2 : m >= 1 ? 1 : 0) : (m >= 3 ? 3 : m >= 1 ? 2 : 1);
    int i = m - (is_qk ? t * (t + 1) / 2 : t * (t - 1) / 2);
    float g[4], decay = 0.f, from = 0.f, rest = 0.f, whole = 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      g[j] = s_g[b][4 * w + j];
      if (j > i && j <= t) decay += g[j];
      if (j <= (lane & 3)) from += g[j];
      if (j > (lane & 3)) rest += g[j];
      whole += g[j];
    }
    if ((lane & 1) == 0) {
      if (is_qk) B.qk[t][i] = expf(decay) * sum;
      else B.kk[t][i] = s_beta[b][4 * w + t] * expf(decay) * sum;
    }
    if (lane < 4) {
      B.E[lane] = expf(from);
      B.rest[lane] = expf(rest);
      B.beta[lane] = s_beta[b][4 * w + lane];
    }
    if (lane == 4) B.whole = unbiased_decay(whole, step);
  };

  if (t0 < t1) {
    fetch(t0);
    stage(0);
  }
  int b = 0;
  for (int64_t t = t0; t < t1; t += kTok, b ^= 1) {
    __syncthreads();  // stage b is written; every thread is done with stage b ^ 1 and the blocks
    const bool more = t + kTok < t1;
    if (more) fetch(t + kTok);
    form_block(b, (t - t0) / 4 + w);
    __syncthreads();
    const int len = t1 - t < kTok ? int(t1 - t) : kTok;
#pragma unroll 1
    for (int i0 = 0; i0 < len; i0 += 4) {
      const Block &B = s_block[i0 >> 2];
      float2 acc[kNC][8];
#pragma unroll
      for (int c = 0; c < kNC; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[c][e] = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < kRows / 4; ++j) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float4 x = *reinterpret_cast<const float4 *>(&(e < 4 ? s_k : s_q)[b][i0 + (e & 3)][32 * j + 4 * rl]);
#pragma unroll
          for (int c = 0; c < kNC; ++c)
            acc[c][e] = f2_fma(make_float2(x.z, x.w), S[c][2 * j + 1],
                               f2_fma(make_float2(x.x, x.y), S[c][2 * j], acc[c][e]));
        }
      }
      float u[kNC][4];
#pragma unroll
      for (int c = 0; c < kNC; ++c) {
        // the sums over the eight lanes rl: lane rl ends with y_rl, or z_{rl - 4}
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = acc[c][e].x + acc[c][e].y;
#pragma unroll
        for (int half = 4; half >= 1; half >>= 1) {
          const bool up = (rl & half) != 0;
#pragma unroll
          for (int e = 0; e < half; ++e)
            x[e] = (up ? x[e + half] : x[e]) + __shfl_xor_sync(0xffffffffu, up ? x[e] : x[e + half], half);
        }
        const float mine = x[0];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float y = __shfl_sync(0xffffffffu, mine, e, 8);
          float r = B.beta[e] * (s_v[b][i0 + e][cw + c] - B.E[e] * y);
#pragma unroll
          for (int i = 0; i < e; ++i) r = fmaf(-B.kk[e][i], u[c][i], r);
          u[c][e] = i0 + e < len ? r : 0.f;
        }
        const int e = rl & 3;
        float o = B.E[e] * mine;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i <= e) o = fmaf(B.qk[e][i], u[c][i], o);
        if (rl >= 4 && i0 + e < len && col + c < a.d_v)
          store_elem<kOutBF16>(a.out, ((t + i0 + e) * a.H + h) * a.d_v + col + c, a.scale * o);
      }
      const float2 whole = make_float2(B.whole, B.whole);
#pragma unroll
      for (int c = 0; c < kNC; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) u[c][e] *= B.rest[e];
#pragma unroll
      for (int j = 0; j < kRows / 4; ++j) {
#pragma unroll
        for (int c = 0; c < kNC; ++c) {
          S[c][2 * j] = f2_mul(whole, S[c][2 * j]);
          S[c][2 * j + 1] = f2_mul(whole, S[c][2 * j + 1]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float4 x = *reinterpret_cast<const float4 *>(&s_k[b][i0 + e][32 * j + 4 * rl]);
#pragma unroll
          for (int c = 0; c < kNC; ++c) {
            const float2 uu = make_float2(u[c][e], u[c][e]);
            S[c][2 * j] = f2_fma(make_float2(x.x, x.y), uu, S[c][2 * j]);
            S[c][2 * j + 1] = f2_fma(make_float2(x.z, x.w), uu, S[c][2 * j + 1]);
          }
        }
      }
    }
    if (more) stage(b ^ 1);
  }

  if (a.final_state != nullptr) {
#pragma unroll
    for (int p = 0; p < kRows / 2; ++p) {
      const int r = 32 * (p >> 1) + 4 * rl + 2 * (p & 1);
#pragma unroll
      for (int c = 0; c < kNC; ++c) {
        float *dst = a.final_state + at_state + int64_t(r) * a.d_v + col + c;
        if (col + c < a.d_v && r < a.d_k) dst[0] = S[c][p].x;
        if (col + c < a.d_v && r + 1 < a.d_k) dst[a.d_v] = S[c][p].y;
      }
    }
  }
}

}  // namespace

cudaError_t launch_delta_recurrent(const DeltaArgs &a, bool in_bf16, bool out_bf16, cudaStream_t stream) {
  using Kern = void (*)(const DeltaArgs);
  const int64_t chains = int64_t(a.num_seqs) * a.H;
  int nc = 4;
  while (nc > 1 && chains * ((a.d_v + 16 * nc - 1) / (16 * nc)) < 2 * kLinearSMs) nc >>= 1;
  const bool wide = a.d_k > 64;
#define KDA_DELTA(ib, ob)                                                                                     \
  {delta_recurrent_kernel<ib, ob, 8, 1>, delta_recurrent_kernel<ib, ob, 8, 2>, delta_recurrent_kernel<ib, ob, 8, 4>, \
   delta_recurrent_kernel<ib, ob, 16, 1>, delta_recurrent_kernel<ib, ob, 16, 2>, delta_recurrent_kernel<ib, ob, 16, 4>}
  static const Kern kernels[4][6] = {KDA_DELTA(false, false), KDA_DELTA(false, true), KDA_DELTA(true, false),
                                     KDA_DELTA(true, true)};
#undef KDA_DELTA
  const dim3 grid(unsigned(chains), unsigned((a.d_v + 16 * nc - 1) / (16 * nc)));
  kernels[2 * int(in_bf16) + int(out_bf16)][3 * int(wide) + (nc == 4 ? 2 : nc - 1)]<<<grid, kThr, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace kda
