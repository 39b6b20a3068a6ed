// kda_linear_recurrent.cu -- linear attention with one decay per head, a token at a time, in fp32
// on the CUDA cores: S = e^{g_t} S + k_t v_t^T, o_t = scale S^T q_t. It takes every size and both
// dtypes (fp32 inputs, short sequences, bf16 head sizes that lack the workspace to be padded); the
// tensor-core kernel is the fast path of long bf16 sequences.
//
// A CTA of 128 threads holds 64 value columns of one segment's state in registers: lane
// (pair, rg) of warp w owns columns 16 w + 2 pair, + 1 and the key rows 16 j + 4 rg + 0..3, so a
// row sum ends with two shuffles inside a warp and the tokens need no CTA barrier. q, k, v pass
// through shared memory 16 tokens at a time (fp32), the next 16 waiting in registers. Two rows
// go through one packed fp32 instruction: 3 per row pair, column and token (k v, decay,
// read-out), which bound the kernel where it fills the SMs; with few heads the chain of tokens does,
// 0.35 us each (prompts of 700 and 333 tokens, 6 heads of 100 x 72 in fp32: 43 us in segments; 128
// sequences of 4 tokens and 64 heads of 64, bf16: 99 us, 2.7 TB/s of states; T = 4096, 96 heads of 128 in
// fp32: 1.57 ms, of it 1.11 in pass 3, whose load/store pipe is 67 % busy, fp32 58 % and issue 47 %).
#include <type_traits>

#include "kda_linear.cuh"

namespace kda {
namespace {

constexpr int kTok = 16;    // tokens per stage
constexpr int kCols = kLinearTokenCols;
constexpr int kThr = 128;

// kRows: key rows per thread (16 for d_k <= 64, else 32). kStateOnly: pass 1 of a segmented call,
// which leaves the state from zero and the summed log-decay in the workspace.
template <bool kInBF16, bool kOutBF16, int kRows, bool kStateOnly>
__global__ void __launch_bounds__(kThr, 3) linear_recurrent_kernel(const LinearArgs a) {
  __shared__ __align__(16) float s_k[2][kTok][4 * kRows], s_q[2][kTok][4 * kRows];
  __shared__ __align__(16) float s_v[2][kTok][kCols];
  __shared__ float s_e[2][kTok], s_g[2][kTok];  // e^g; g (pass 1)
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int rg = lane & 3, pair = lane >> 2;
  const int h = blockIdx.x % a.H;
  const int col0 = blockIdx.y * kCols;
  if constexpr (kStateOnly) let_next_pass_begin();
  LinearSlot s;
  if (!linear_slot(a.cu, a.num_seqs, a.plan.seg_len, a.plan.inner, blockIdx.x / a.H, s)) return;
  const int hk = h / (a.H / a.H_k);
  const int col = col0 + 16 * w + 2 * pair;  // this thread's columns: col, col + 1
  const bool ok0 = col < a.d_v, ok1 = col + 1 < a.d_v;

  // the state: S[c][p] holds rows (row(2 p), row(2 p) + 1) of column col + c
  float2 S[2][kRows / 2];
  auto row_of = [&](int p) { return 16 * (p >> 1) + 4 * rg + 2 * (p & 1); };
  const int64_t dd = int64_t(a.d_k) * a.d_v;
  const float *S0 = kStateOnly ? nullptr : linear_entering(a, s, h);
#pragma unroll
  for (int p = 0; p < kRows / 2; ++p) {
    const int r = row_of(p);
    auto at = [&](int row, int c) {
      return S0 != nullptr && row < a.d_k && col + c < a.d_v ? S0[int64_t(row) * a.d_v + col + c] : 0.f;
    };
    S[0][p] = make_float2(at(r, 0), at(r + 1, 0));
    S[1][p] = make_float2(at(r, 1), at(r + 1, 1));
  }

  // global -> registers -> shared memory, a stage of kTok tokens at a time
  // (as stored: a conversion here would wait for the load)
  using Elem = std::conditional_t<kInBF16, uint16_t, float>;
  auto raw = [](const void *p, int64_t at) { return static_cast<const Elem *>(p)[at]; };
  auto value = [](Elem x) {
    if constexpr (kInBF16) return bf16_to_f32(x);
    else return x;
  };
  Elem rk[kTok], rq[kTok], rv[kTok * kCols / kThr];
  float rg_ = 0.f;
  auto fetch = [&](int64_t t) {  // tokens t .. t + kTok - 1; zeros past the segment
#pragma unroll
    for (int i = 0; i < kTok; ++i) {
      const bool ok = t + i < s.t1 && tid < a.d_k;
      const int64_t at = ((t + i) * a.H_k + hk) * a.d_k + tid;
      rk[i] = ok ? raw(a.k, at) : Elem(0);
      if constexpr (!kStateOnly) rq[i] = ok ? raw(a.q, at) : Elem(0);
    }
#pragma unroll
    for (int i = 0; i < kTok * kCols / kThr; ++i) {
      const int64_t tt = t + 2 * i + (tid >> 6);
      const int c = col0 + (tid & 63);
      rv[i] = tt < s.t1 && c < a.d_v ? raw(a.v, (tt * a.H + h) * a.d_v + c) : Elem(0);
    }
    if (tid < kTok) rg_ = t + tid < s.t1 ? a.log_decay[a.per_token ? (t + tid) * a.H + h : h] : 0.f;
  };
  // The factor of a token's decay, e^g in fp32. Simply rounded, the factors of a constant decay would
  // all be off the same way, which a memory of thousands of tokens adds up. So the token takes a whole
  // ulp more or less where `rest`, what one rounding loses in ulps, times the tokens so far passes a
  // half: factors of a constant decay stay within an ulp of e to the sum, others round either way
  // without a bias. (Decay's choice between two forms, made in the loop over rows, costs 2.07 ms at
  // T = 4096, 96 heads of 128 in fp32; this 1.57.)
  auto factor = [&](float g, int64_t t) {
    const Decay d = decay_of(g);
    if (!d.keep) return d.c;  // e^g below one half: no memory to drift
    const float e = 1.f + d.c;
    const uint32_t exponent = __float_as_uint(e) & 0x7f800000u;  // an ulp is 2^-23 of its power of two
    const float rest = (d.c - (e - 1.f)) * __uint_as_float(0x8a800000u - exponent);
    const float n = float((t - s.t0) & 4095);
    return fmaf(rintf((n + 1.f) * rest) - rintf(n * rest), __uint_as_float(exponent - 0x0b800000u), e);
  };
  auto stage = [&](int b, int64_t t) {
    if (tid < 4 * kRows) {
#pragma unroll
      for (int i = 0; i < kTok; ++i) {
        s_k[b][i][tid] = value(rk[i]);
        if constexpr (!kStateOnly) s_q[b][i][tid] = value(rq[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < kTok * kCols / kThr; ++i) s_v[b][2 * i + (tid >> 6)][tid & 63] = value(rv[i]);
    if (tid < kTok) {
      s_e[b][tid] = factor(rg_, t + tid);
      if constexpr (kStateOnly) s_g[b][tid] = rg_;
    }
  };

  double decay_sum = 0.;  // of the segment, pass 1 (all threads alike)
  if (s.t0 < s.t1) {
    fetch(s.t0);
    stage(0, s.t0);
  }
  int b = 0;
  for (int64_t t = s.t0; t < s.t1; t += kTok, b ^= 1) {
    __syncthreads();  // stage b is written; every thread is done with stage b ^ 1
    const bool more = t + kTok < s.t1;
    if (more) fetch(t + kTok);
    const int len = s.t1 - t < kTok ? int(s.t1 - t) : kTok;
    if constexpr (kStateOnly) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kTok; ++i) sum += s_g[b][i];
      decay_sum += double(sum);
    }
    for (int i = 0; i < len; i += 2) {  // two tokens: their four row sums meet in one exchange
      float part[4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float2 o[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        const float2 e2 = make_float2(s_e[b][i + u], s_e[b][i + u]);
        const float2 v2 = *reinterpret_cast<const float2 *>(&s_v[b][i + u][16 * w + 2 * pair]);
        const float2 v0 = make_float2(v2.x, v2.x), v1 = make_float2(v2.y, v2.y);
#pragma unroll
        for (int j = 0; j < kRows / 4; ++j) {
          const float4 k4 = *reinterpret_cast<const float4 *>(&s_k[b][i + u][16 * j + 4 * rg]);
          const float2 ka = make_float2(k4.x, k4.y), kb = make_float2(k4.z, k4.w);
          S[0][2 * j] = f2_fma(e2, S[0][2 * j], f2_mul(ka, v0));
          S[0][2 * j + 1] = f2_fma(e2, S[0][2 * j + 1], f2_mul(kb, v0));
          S[1][2 * j] = f2_fma(e2, S[1][2 * j], f2_mul(ka, v1));
          S[1][2 * j + 1] = f2_fma(e2, S[1][2 * j + 1], f2_mul(kb, v1));
          if constexpr (!kStateOnly) {
            const float4 q4 = *reinterpret_cast<const float4 *>(&s_q[b][i + u][16 * j + 4 * rg]);
            const float2 qa = make_float2(q4.x, q4.y), qb = make_float2(q4.z, q4.w);
            o[0] = f2_fma(qb, S[0][2 * j + 1], f2_fma(qa, S[0][2 * j], o[0]));
            o[1] = f2_fma(qb, S[1][2 * j + 1], f2_fma(qa, S[1][2 * j], o[1]));
          }
        }
        part[2 * u] = o[0].x + o[0].y;
        part[2 * u + 1] = o[1].x + o[1].y;
      }
      if constexpr (!kStateOnly) {
        // sums over the four lanes rg: each ends with one of (token u, column c)
        const bool up2 = (rg & 2) != 0, up1 = (rg & 1) != 0;
        float x0 = (up2 ? part[2] : part[0]) + __shfl_xor_sync(0xffffffffu, up2 ? part[0] : part[2], 2);
        float x1 = (up2 ? part[3] : part[1]) + __shfl_xor_sync(0xffffffffu, up2 ? part[1] : part[3], 2);
        const float x = (up1 ? x1 : x0) + __shfl_xor_sync(0xffffffffu, up1 ? x0 : x1, 1);
        const int u = rg >> 1, c = rg & 1;
        if (i + u < len && (c ? ok1 : ok0))
          store_elem<kOutBF16>(a.out, ((t + i + u) * a.H + h) * a.d_v + col + c, a.scale * x);
      }
    }
    if (more) stage(b ^ 1, t + kTok);
  }

  float *dst = kStateOnly ? a.seg_states + (s.place * a.H + h) * dd
               : (s.last && a.final_state != nullptr) ? a.final_state + (int64_t(s.n) * a.H + h) * dd : nullptr;
  if (dst != nullptr) {
#pragma unroll
    for (int p = 0; p < kRows / 2; ++p) {
      const int r = row_of(p);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        if (!(c ? ok1 : ok0)) continue;
        if (r < a.d_k) dst[int64_t(r) * a.d_v + col + c] = S[c][p].x;
        if (r + 1 < a.d_k) dst[int64_t(r + 1) * a.d_v + col + c] = S[c][p].y;
      }
    }
  }
  if (kStateOnly && tid == 0 && blockIdx.y == 0) a.seg_decay[s.place * a.H + h] = float(decay_sum);
}

template <bool kStateOnly>
cudaError_t launch_pass(const LinearArgs &a, bool in_bf16, bool out_bf16, cudaStream_t stream) {
  const unsigned pieces = unsigned(a.plan.inner) + (kStateOnly ? 0u : unsigned(a.num_seqs));
  const dim3 grid(pieces * unsigned(a.H), unsigned((a.d_v + kCols - 1) / kCols));
  const bool wide = a.d_k > 64;
  using Kern = void (*)(const LinearArgs);
#define KDA_LIN(ib, ob) \
  wide ? Kern(linear_recurrent_kernel<ib, ob, 32, kStateOnly>) : Kern(linear_recurrent_kernel<ib, ob, 16, kStateOnly>)
  Kern kern;
  if constexpr (kStateOnly) kern = in_bf16 ? (KDA_LIN(true, false)) : (KDA_LIN(false, false));
  else
    kern = in_bf16 ? (out_bf16 ? (KDA_LIN(true, true)) : (KDA_LIN(true, false)))
                   : (out_bf16 ? (KDA_LIN(false, true)) : (KDA_LIN(false, false)));
#undef KDA_LIN
  // Pass 3 does not begin early here: beside pass 1 it takes the issue slots that pass 1 waits for (prompts
  // of 700 and 333 tokens, 6 heads: 46 us, early 50).
  kern<<<grid, kThr, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_recurrent(const LinearArgs &a, bool in_bf16, bool out_bf16, cudaStream_t stream) {
  if (a.plan.seg_len != 0) {
    cudaError_t e = launch_pass<true>(a, in_bf16, out_bf16, stream);
    if (e == cudaSuccess) e = launch_linear_scan(a, stream);
    if (e != cudaSuccess) return e;
  }
  return launch_pass<false>(a, in_bf16, out_bf16, stream);
}

}  // namespace kda
