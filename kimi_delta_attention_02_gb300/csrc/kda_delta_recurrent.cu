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
// kLanes lanes share a column's key rows, so a warp holds 32 / kLanes kNC value columns: lane (cl, rl) owns
// kNC of them and the key rows 4 kLanes j + 4 rl + 0..3, two rows to a packed fp32 instruction. Four warps do
// this. Four others go ahead of them: they bring q, k, v to shared memory 16 tokens at a time (the next 16
// waiting in registers) and form the products k.k and q.k and the decays of the next 16 tokens' blocks.
//
// What bounds it: the latency of a block of four tokens where chains are few (0.13 us a token: 700 and 333
// tokens, 6 heads of 100 x 72, fp32: 97 us, 137 without warps that go ahead), issue where they are many
// (4096 tokens, 96 heads of 128: 1.98 ms, 2.41 without; the 21 G multiply-adds are a quarter of the fp32
// rate, beside the reads of k and q from shared memory and the exchange of the sums).
#include <atomic>
#include <type_traits>

#include "kda_delta.cuh"

namespace kda {
namespace {

constexpr int kTok = 16;  // tokens per stage
constexpr int kThr = 128;  // of each half: those that keep the state, those that go ahead

struct Block {  // of four tokens
  float E[4];       // from the block's start
  float beta[4];
  float rest[4];    // D_3i
  float whole;      // E_3 as the state's factor
  float pad[3];
  float kk[4][4];   // beta_t D_ti (k_t . k_i), i < t
  float qk[4][4];   // D_ti (q_t . k_i), i <= t
};

template <int kDK, int kCols>
struct Shared {
  float k[3][kTok][kDK], q[3][kTok][kDK], v[3][kTok][kCols];
  Block block[2][kTok / 4];
  float g[3][kTok], beta[3][kTok];
};

// kCut: pieces of a cut sequence, in passes 1 and 3 (in one kernel with the others, its addresses cost them
// spills: 4096 tokens, 96 heads of 128 2362 us instead of 1963).
template <bool kInBF16, bool kOutBF16, int kLanes, int kRows, int kNC, bool kCut>
__global__ void __launch_bounds__(2 * kThr, 2) delta_recurrent_kernel(const DeltaArgs a, int pass) {
  constexpr int kDK = kLanes * kRows, kCols = kThr / kLanes * kNC;
  constexpr int kEach = kLanes / 8;  // lanes that end with the same one of a block's eight sums
  extern __shared__ __align__(16) uint8_t smem[];
  Shared<kDK, kCols> &sh = *reinterpret_cast<Shared<kDK, kCols> *>(smem);
  const int tid = threadIdx.x % kThr, lane = tid & 31, w = tid >> 5;
  const int rl = lane % kLanes, cl = lane / kLanes;
  const int h = blockIdx.x % a.H, hk = h / (a.H / a.H_k);
  const int col0 = blockIdx.y * kCols, cw = 32 / kLanes * kNC * w + kNC * cl, col = col0 + cw;
  int index = blockIdx.x / a.H;
  LinearSlot s;
  bool map = false, emit = true;
  if constexpr (kCut) {  // as in the tensor-core kernel
    map = index >= a.plan.inner + a.num_seqs;  // pass 1: the pieces once more, for their M
    if (map) index -= a.plan.inner + a.num_seqs;
    if (!linear_slot(a.cu, a.num_seqs, a.plan.seg_len, a.plan.inner, index, s)) return;
    if ((pass == 3 || map) ? s.first : s.last && !s.first) return;
    emit = s.first || pass == 3;
  } else {
    s.n = index, s.t0 = a.cu[index], s.t1 = a.cu[index + 1];
    if (s.t1 - s.t0 <= a.plan.few) return;  // done by the decode kernel
  }
  const int64_t t0 = s.t0, t1 = s.t1;
  const int pk = delta_up8(a.d_k), cols = map ? pk : a.d_v;  // (M has zeros behind d_k)
  const int v_cols = map ? 0 : a.d_v, out_cols = emit ? a.d_v : 0;
  if (kCut && col0 >= cols) return;

  // global -> registers -> shared memory, a stage of kTok tokens at a time (as stored: a conversion here
  // would wait for the load). Rows of q and k that are whole 16-byte pieces take 16-byte loads: a load
  // per element and its address are half of a stage's instructions where a warp has one column.
  using Elem = std::conditional_t<kInBF16, uint16_t, float>;
  auto value = [](Elem x) {
    if constexpr (kInBF16) return bf16_to_f32(x);
    else return x;
  };
  constexpr int kPer = 16 / int(sizeof(Elem)), kPieces = kTok * kDK / kPer / kThr, kRowPieces = kDK / kPer;
  constexpr int kVals = (kTok * kCols + kThr - 1) / kThr;
  union Raw {
    uint4 w;
    Elem e[kPer];
  };
  Raw rk[kPieces], rq[kPieces];
  Elem rv[kVals];
  const bool whole = a.d_k % kPer == 0;
  float r_g = 0.f, r_beta = 0.f;
  auto fetch = [&](int64_t t) {  // tokens t .. t + kTok - 1; zeros past the sequence
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int64_t tt = t + (i * kThr + tid) / kRowPieces;
      const int c = tid % kRowPieces * kPer;
      const int64_t at = (tt * a.H_k + hk) * a.d_k + c;
      const Elem *k = static_cast<const Elem *>(a.k) + at, *q = static_cast<const Elem *>(a.q) + at;
      rk[i].w = rq[i].w = make_uint4(0, 0, 0, 0);
      if (tt >= t1 || c >= a.d_k) continue;
      if (whole) {
        rk[i].w = *reinterpret_cast<const uint4 *>(k), rq[i].w = *reinterpret_cast<const uint4 *>(q);
      } else {
#pragma unroll
        for (int e = 0; e < kPer; ++e)
          if (c + e < a.d_k) rk[i].e[e] = k[e], rq[i].e[e] = q[e];
      }
    }
#pragma unroll
    for (int i = 0; i < kVals; ++i) {
      const int64_t tt = t + (i * kThr + tid) / kCols;
      const int c = col0 + tid % kCols;
      rv[i] = i * kThr + tid < kTok * kCols && tt < t1 && c < v_cols
                  ? static_cast<const Elem *>(a.v)[(tt * a.H + h) * a.d_v + c] : Elem(0);
    }
    if (tid < kTok) {
      const bool ok = t + tid < t1;
      r_g = ok ? a.log_decay[a.per_token ? (t + tid) * a.H + h : h] : 0.f;
      r_beta = ok ? a.beta[(t + tid) * a.H + h] : 0.f;
    }
  };
  auto stage = [&](int b) {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int row = (i * kThr + tid) / kRowPieces, c = tid % kRowPieces * kPer;
#pragma unroll
      for (int e = 0; e < kPer; e += 4) {
        *reinterpret_cast<float4 *>(&sh.k[b][row][c + e]) =
            make_float4(value(rk[i].e[e]), value(rk[i].e[e + 1]), value(rk[i].e[e + 2]), value(rk[i].e[e + 3]));
        *reinterpret_cast<float4 *>(&sh.q[b][row][c + e]) =
            make_float4(value(rq[i].e[e]), value(rq[i].e[e + 1]), value(rq[i].e[e + 2]), value(rq[i].e[e + 3]));
      }
    }
#pragma unroll
    for (int i = 0; i < kVals; ++i)
      if (i * kThr + tid < kTok * kCols) sh.v[b][(i * kThr + tid) / kCols][tid % kCols] = value(rv[i]);
    if (tid < kTok) sh.g[b][tid] = r_g, sh.beta[b][tid] = r_beta;
  };
  // warp w: the products and decays of the stage's block w
  auto form_block = [&](int b, Block &B, int64_t step) {
    float4 k4[4], q4[4];
    const bool on = 4 * lane < kDK;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      k4[t] = on ? *reinterpret_cast<const float4 *>(&sh.k[b][4 * w + t][4 * lane]) : make_float4(0.f, 0.f, 0.f, 0.f);
      q4[t] = on ? *reinterpret_cast<const float4 *>(&sh.q[b][4 * w + t][4 * lane]) : make_float4(0.f, 0.f, 0.f, 0.f);
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
      g[j] = sh.g[b][4 * w + j];
      if (j > i && j <= t) decay += g[j];
      if (j <= (lane & 3)) from += g[j];
      if (j > (lane & 3)) rest += g[j];
      whole += g[j];
    }
    if ((lane & 1) == 0) {
      if (is_qk) B.qk[t][i] = expf(decay) * sum;
      else B.kk[t][i] = sh.beta[b][4 * w + t] * expf(decay) * sum;
    }
    if (lane < 4) {
      B.E[lane] = expf(from);
      B.rest[lane] = expf(rest);
      B.beta[lane] = sh.beta[b][4 * w + lane];
    }
    if (lane == 4) B.whole = unbiased_decay(whole, step);
  };

  if (threadIdx.x >= kThr) {
    // stage i + 2 comes to shared memory and the blocks of stage i + 1 are formed while stage i is worked on
    if (t0 >= t1) return;
    fetch(t0);
    stage(0);
    fetch(t0 + kTok);
    stage(1);
    fetch(t0 + 2 * kTok);
    named_bar_sync(1, kThr);
    form_block(0, sh.block[0][w], w);
    int b1 = 1, b2 = 2;
    for (int64_t t = t0, i = 1; t < t1; t += kTok, ++i) {
      __syncthreads();
      stage(b2);
      fetch(t + 3 * kTok);
      form_block(b1, sh.block[i & 1][w], i * (kTok / 4) + w);
      b1 = b2;
      if (++b2 == 3) b2 = 0;
    }
    return;
  }

  // the state: S[c][2 j + p] holds rows 4 kLanes j + 4 rl + 2 p, + 1 of column col + c
  float2 S[kNC][kRows / 2];
  const int64_t at_state = (int64_t(s.n) * a.H + h) * a.d_k * a.d_v;
  const float *from = a.init_state != nullptr ? a.init_state + at_state : nullptr;
  float *to = a.final_state != nullptr ? a.final_state + at_state : nullptr;
  int from_width = a.d_v, to_width = a.d_v;
  if constexpr (kCut) {
    const int pv = delta_up8(a.d_v);
    const int64_t place = delta_place(a, s), each = int64_t(pk) * pv;
    float *ends = reinterpret_cast<float *>(a.workspace + a.plan.ends);
    if (!s.first) from = pass == 3 ? ends + ((place - 1) * a.H + h) * each : nullptr, from_width = pv;
    if (map) to = reinterpret_cast<float *>(a.workspace + a.plan.maps) + (place * a.H + h) * (int64_t(pk) * pk), to_width = pk;
    else if (!emit || !s.last) to = pass == 3 ? nullptr : ends + (place * a.H + h) * each, to_width = pv;
  }
#pragma unroll
  for (int p = 0; p < kRows / 2; ++p) {
    const int r = 4 * kLanes * (p >> 1) + 4 * rl + 2 * (p & 1);
    auto at = [&](int row, int c) {
      if (map) return row == col + c && row < a.d_k ? 1.f : 0.f;
      return from != nullptr && row < a.d_k && col + c < a.d_v ? from[int64_t(row) * from_width + col + c] : 0.f;
    };
#pragma unroll
    for (int c = 0; c < kNC; ++c) S[c][p] = make_float2(at(r, c), at(r + 1, c));
  }

  int b = 0, turn = 0;
  for (int64_t t = t0; t < t1; t += kTok, turn ^= 1) {
    __syncthreads();
    const int len = t1 - t < kTok ? int(t1 - t) : kTok;
#pragma unroll 1
    for (int i0 = 0; i0 < len; i0 += 4) {
      const Block &B = sh.block[turn][i0 >> 2];
      float2 acc[kNC][8];
#pragma unroll
      for (int c = 0; c < kNC; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[c][e] = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < kRows / 4; ++j) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float4 x = *reinterpret_cast<const float4 *>(&(e < 4 ? sh.k : sh.q)[b][i0 + (e & 3)][4 * kLanes * j + 4 * rl]);
#pragma unroll
          for (int c = 0; c < kNC; ++c)
            acc[c][e] = f2_fma(make_float2(x.z, x.w), S[c][2 * j + 1],
                               f2_fma(make_float2(x.x, x.y), S[c][2 * j], acc[c][e]));
        }
      }
      float u[kNC][4];
#pragma unroll
      for (int c = 0; c < kNC; ++c) {
        // the sums over the lanes rl: lane rl ends with y_{rl / kEach}, or z_{rl / kEach - 4}
        float x[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = acc[c][e].x + acc[c][e].y;
#pragma unroll
        for (int half = 4; half >= 1; half >>= 1) {
          const bool up = (rl & half * kEach) != 0;
#pragma unroll
          for (int e = 0; e < half; ++e)
            x[e] = (up ? x[e + half] : x[e]) + __shfl_xor_sync(0xffffffffu, up ? x[e] : x[e + half], half * kEach);
        }
        float mine = x[0];
#pragma unroll
        for (int off = kEach >> 1; off >= 1; off >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, off);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float y = __shfl_sync(0xffffffffu, mine, e * kEach, kLanes);
          float r = B.beta[e] * (sh.v[b][i0 + e][cw + c] - B.E[e] * y);
#pragma unroll
          for (int i = 0; i < e; ++i) r = fmaf(-B.kk[e][i], u[c][i], r);
          u[c][e] = i0 + e < len ? r : 0.f;
        }
        const int e = rl / kEach & 3;
        float o = B.E[e] * mine;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (i <= e) o = fmaf(B.qk[e][i], u[c][i], o);
        if (rl >= 4 * kEach && rl % kEach == 0 && i0 + e < len && col + c < out_cols)
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
          const float4 x = *reinterpret_cast<const float4 *>(&sh.k[b][i0 + e][4 * kLanes * j + 4 * rl]);
#pragma unroll
          for (int c = 0; c < kNC; ++c) {
            const float2 uu = make_float2(u[c][e], u[c][e]);
            S[c][2 * j] = f2_fma(make_float2(x.x, x.y), uu, S[c][2 * j]);
            S[c][2 * j + 1] = f2_fma(make_float2(x.z, x.w), uu, S[c][2 * j + 1]);
          }
        }
      }
    }
    if (++b == 3) b = 0;
  }

  if (to != nullptr) {
#pragma unroll
    for (int p = 0; p < kRows / 2; ++p) {
      const int r = 4 * kLanes * (p >> 1) + 4 * rl + 2 * (p & 1);
#pragma unroll
      for (int c = 0; c < kNC; ++c) {
        float *dst = to + int64_t(r) * to_width + col + c;
        if (col + c < cols && r < a.d_k) dst[0] = S[c][p].x;
        if (col + c < cols && r + 1 < a.d_k) dst[to_width] = S[c][p].y;
      }
    }
  }
}

template <bool kInBF16, bool kOutBF16, int kLanes, int kRows, int kNC, bool kCut>
cudaError_t launch_one_of(const DeltaArgs &a, int pass, int64_t pieces, int cols, cudaStream_t stream) {
  constexpr int kCols = kThr / kLanes * kNC;
  constexpr int smem = int(sizeof(Shared<kLanes * kRows, kCols>));
  const auto kern = delta_recurrent_kernel<kInBF16, kOutBF16, kLanes, kRows, kNC, kCut>;
  if (smem > 49152) {  // granted once per device (bit d for device d; past 63 at every launch)
    static std::atomic<uint64_t> granted;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (bit == 0 || (granted.load(std::memory_order_acquire) & bit) == 0) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e != cudaSuccess) return e;
      granted.fetch_or(bit, std::memory_order_release);
    }
  }
  const dim3 grid(unsigned(pieces * a.H), unsigned((cols + kCols - 1) / kCols));
  kern<<<grid, 2 * kThr, smem, stream>>>(a, pass);
  return cudaGetLastError();
}

template <bool kInBF16, bool kOutBF16, int kLanes, int kRows, int kNC>
cudaError_t launch_one(const DeltaArgs &a, int pass, int64_t pieces, int cols, cudaStream_t stream) {
  return a.plan.seg_len != 0 ? launch_one_of<kInBF16, kOutBF16, kLanes, kRows, kNC, true>(a, pass, pieces, cols, stream)
                             : launch_one_of<kInBF16, kOutBF16, kLanes, kRows, kNC, false>(a, pass, pieces, cols, stream);
}

}  // namespace

cudaError_t launch_delta_recurrent(const DeltaArgs &a, bool in_bf16, bool out_bf16, cudaStream_t stream) {
  // A warp per column while that leaves at most two CTAs for an SM: a block's way is shorter, but 16 columns per
  // CTA are less work. Two columns per thread once 16 per CTA are more CTAs than SMs: a CTA's block takes half
  // as long again, and one SM's two CTAs twice as long. 1000 tokens in fp32, us by 4 / 16 / 32 columns per
  // CTA: 8 heads of 128 134 / 144 / 205, 16 heads 261 / 146 / 205, 28 heads 388 / 231 / 205, 48 heads 756 / 455 / 315,
  // 96 heads 1432 / 682 / 497; 48 heads of 64 383 / 152 / 122.
  const auto pass = [&](int which) {
    const bool cut = a.plan.seg_len != 0;
    const int64_t pieces = int64_t(a.num_seqs) + a.plan.inner + (cut && which == 1 ? a.plan.inner : 0);
    // (pass 1 writes all of M's columns, those behind d_k too: pass 2 multiplies them by zeros, and what the workspace
    // held there may be a NaN)
    const int pk = delta_up8(a.d_k), cols = cut && which == 1 && pk > a.d_v ? pk : a.d_v;
    const auto ctas = [&](int width) { return pieces * a.H * ((cols + width - 1) / width); };
    const auto run = [&](auto in, auto out) {
      constexpr bool ib = decltype(in)::value, ob = decltype(out)::value;
      if (ctas(4) <= 2 * kLinearSMs) return launch_one<ib, ob, 32, 4, 1>(a, which, pieces, cols, stream);
      const bool wide = a.d_k > 64, two = ctas(16) > kLinearSMs;
      if (wide)
        return two ? launch_one<ib, ob, 8, 16, 2>(a, which, pieces, cols, stream)
                   : launch_one<ib, ob, 8, 16, 1>(a, which, pieces, cols, stream);
      return two ? launch_one<ib, ob, 8, 8, 2>(a, which, pieces, cols, stream)
                 : launch_one<ib, ob, 8, 8, 1>(a, which, pieces, cols, stream);
    };
    const std::true_type yes;
    const std::false_type no;
    return in_bf16 ? (out_bf16 ? run(yes, yes) : run(yes, no)) : (out_bf16 ? run(no, yes) : run(no, no));
  };
  cudaError_t e = pass(1);
  if (e != cudaSuccess || a.plan.seg_len == 0) return e;
  e = launch_delta_chain(a, stream);
  return e == cudaSuccess ? pass(3) : e;
}

}  // namespace kda
