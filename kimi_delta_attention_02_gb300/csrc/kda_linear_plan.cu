// kda_linear_plan.cu -- how a linear-attention prefill is cut (host), and its two small kernels: the scan
// that chains the segments' states, and the copies that pad head sizes to what TMA can address.
#include "kda_linear.cuh"

namespace kda {
namespace {

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }
int up8(int x) { return (x + 7) & ~7; }

// Pass 2: a segment's end state from zero, B_j, gives way to its successor's entering state in the
// successor's place, E_0 = initial state (read where it is), E_{j+1} = e^{D_j} E_j + B_j. The CTAs of
// a sequence's first segment (blockIdx.y is the piece) walk its segments, kVec entries per thread, the
// next segments' entries on their way meanwhile.
template <int kVec>
__global__ void __launch_bounds__(256) linear_scan_kernel(const LinearArgs a) {
  let_next_pass_begin();
  LinearSlot s;
  const bool some = linear_slot(a.cu, a.num_seqs, a.plan.seg_len, a.plan.inner, blockIdx.y, s) && s.first;
  wait_for_earlier_passes();
  if (!some) return;
  const int segs = (a.cu[s.n + 1] - a.cu[s.n] - 1) / a.plan.seg_len + 1;  // (a sum could pass 2^31)
  const int64_t dd = int64_t(a.d_k) * a.d_v, step = int64_t(a.H) * dd;
  struct alignas(4 * kVec) Vec {
    float v[kVec];
  };
  for (int64_t e = (int64_t(blockIdx.x) * blockDim.x + threadIdx.x) * kVec; e < step;
       e += int64_t(gridDim.x) * blockDim.x * kVec) {
    float *p = a.seg_states + s.place * step + e;
    const float *d = a.seg_decay + s.place * a.H + e / dd;
    auto read = [&](int j) { return *reinterpret_cast<const Vec *>(p + j * step); };
    Vec S = {};
    if (a.init_state != nullptr) S = *reinterpret_cast<const Vec *>(a.init_state + s.n * step + e);
    constexpr int kAhead = 4;
    Vec b[kAhead] = {};
    float D[kAhead] = {};
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i + 1 < segs) b[i] = read(i), D[i] = d[i * a.H];
    if (linear_in_place(a)) *reinterpret_cast<Vec *>(p) = S;  // B_0 has been read
    for (int j0 = 0; j0 + 1 < segs; j0 += kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int j = j0 + i;
        if (j + 1 >= segs) break;
        const Decay decay = decay_of(D[i]);
#pragma unroll
        for (int v = 0; v < kVec; ++v) S.v[v] = decay_step(S.v[v], decay) + b[i].v[v];
        if (j + kAhead + 1 < segs) b[i] = read(j + kAhead), D[i] = d[(j + kAhead) * a.H];
        // B_{j+1} of this place, if there is one, was read above (kAhead >= 2)
        *reinterpret_cast<Vec *>(p + (j + 1) * step) = S;
      }
    }
  }
}

// Rows of d elements to rows padded with zeros to a multiple of 8, or back. Each thread moves one
// piece of 8 elements, aligned on the padded side.
struct PadJob {
  const void *src;
  void *dst;
  int64_t rows;       // of the whole tensor; with cu only up to the last sequence's end
  const int32_t *cu;  // or null
  int32_t per_token;  // rows per token
  int32_t d, bytes;   // element size: 2 or 4
};
struct PadArgs {
  PadJob job[4];
  int num_seqs, jobs;
};

template <typename T, bool kBack>
__device__ __forceinline__ void pad_rows(const PadJob &job, int64_t rows) {
  struct alignas(16) Piece {
    T v[8];
  };
  const int per_row = (job.d + 7) >> 3;
  for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < rows * per_row;
       i += int64_t(gridDim.x) * blockDim.x) {
    const int64_t row = i / per_row;
    const int c = int(i - row * per_row) * 8;
    if constexpr (kBack) {
      const Piece x = static_cast<const Piece *>(job.src)[i];
      T *y = static_cast<T *>(job.dst) + row * job.d + c;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e < job.d) y[e] = x.v[e];
    } else {
      const T *x = static_cast<const T *>(job.src) + row * job.d + c;
      Piece y{};
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e < job.d) y.v[e] = x[e];
      static_cast<Piece *>(job.dst)[i] = y;
    }
  }
}

template <bool kBack>
__global__ void __launch_bounds__(256) linear_pad_kernel(const PadArgs a) {
  const PadJob &job = a.job[blockIdx.y];
  const int64_t rows = job.cu == nullptr ? job.rows : int64_t(job.cu[a.num_seqs]) * job.per_token;
  if (job.bytes == 2) pad_rows<uint16_t, kBack>(job, rows);
  else pad_rows<uint32_t, kBack>(job, rows);
}

template <bool kBack>
cudaError_t launch_pad(const PadArgs &a, cudaStream_t stream) {
  int64_t most = 0;
  for (int i = 0; i < a.jobs; ++i) {
    const int64_t pieces = a.job[i].rows * (up8(a.job[i].d) / 8);
    most = pieces > most ? pieces : most;
  }
  const int64_t need = (most + 255) / 256, fit = kLinearSMs * 16;
  linear_pad_kernel<kBack><<<dim3(unsigned(need < fit ? need : fit), unsigned(a.jobs)), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_scan(const LinearArgs &a, cudaStream_t stream) {
  const int64_t dd = int64_t(a.d_k) * a.d_v;
  const int vec = dd % 4 == 0 ? 4 : 1;  // states start on 16-byte boundaries
  // One wave of CTAs (8 per SM) for all pieces, because most may be idle: 64 short prompts, of which none is
  // cut, take 108 us with one wave, 110 with four. (`inner` is at most one and a half times the plan's
  // `tasks`, far below the grid's limit.)
  const int64_t need = (a.H * dd + 256 * vec - 1) / (256 * vec), fit = 8 * kLinearSMs / a.plan.inner;
  const dim3 grid(unsigned(need < fit ? need : fit > 1 ? fit : 1), unsigned(a.plan.inner));
  return launch_pass_kernel(vec == 4 ? linear_scan_kernel<4> : linear_scan_kernel<1>, grid, 256, 0, true, stream, a);
}

cudaError_t launch_linear_pad(LinearArgs &a, cudaStream_t stream) {
  const LinearPlan &p = a.plan;
  PadArgs pad{};
  auto add = [&](const void *src, size_t at, int64_t rows, int d, int bytes) -> void * {
    void *to = a.workspace + at;
    pad.job[pad.jobs++] = {src, to, rows, nullptr, 0, d, bytes};
    return to;
  };
  if (a.d_k % 8 != 0) {
    a.q = add(a.q, p.pad_q, a.total * a.H_k, a.d_k, 2);
    a.k = add(a.k, p.pad_k, a.total * a.H_k, a.d_k, 2);
  }
  if (a.d_v % 8 != 0) {
    a.v = add(a.v, p.pad_v, a.total * a.H, a.d_v, 2);
    const int64_t rows = int64_t(a.num_seqs) * a.H * a.d_k;
    if (a.init_state != nullptr)
      a.init_state = static_cast<float *>(add(a.init_state, p.pad_states, rows, a.d_v, 4));
    if (a.final_state != nullptr) a.final_state = reinterpret_cast<float *>(a.workspace + p.pad_states);
    a.out = a.workspace + p.pad_out;
    a.d_v = up8(a.d_v);
  }
  return launch_pad<false>(pad, stream);
}

cudaError_t launch_linear_unpad(const LinearArgs &a, bool out_bf16, void *out, float *final_state, int d_v,
                                cudaStream_t stream) {
  PadArgs pad{};
  pad.num_seqs = a.num_seqs;
  pad.job[pad.jobs++] = {a.out, out, a.total * a.H, a.cu, a.H, d_v, out_bf16 ? 2 : 4};
  if (final_state != nullptr)
    pad.job[pad.jobs++] = {a.final_state, final_state, int64_t(a.num_seqs) * a.H * a.d_k, nullptr, 0, d_v, 4};
  return launch_pad<true>(pad, stream);
}

// Segments are as long as two thirds of the call's tokens x heads x column tiles divided among
// `tasks` CTAs, so that a sequence longer than a CTA's share is split and the others stay whole. (8
// ragged sequences of up to 4096 tokens, 32 heads of 64: 154 us with the whole share, 149 with half of
// it, 129 with two thirds.) Of a single sequence the length is known: it is cut into as many equal
// segments as CTAs fit beside each other.
//
// A chunk costs the tensor-core kernel the same however few tokens it holds, the token-recurrent one
// goes by tokens, so the mean length decides. Microseconds, tensor cores / token-recurrent, at
// sequences of 4, 16, 32 and 64 tokens:
//   16 of 64 heads of 128, bf16 out   71/53   72/75   73/113  88/189    128 of them  488/295 511/466 512/748  520/1332
//   the same, fp32 out               103/52  103/75  103/113 120/190                 728/295 760/466 758/747  791/1332
//   16 of 64 heads of 64              51/32   50/31   50/44   56/69                  311/99  332/150 335/243  345/429
// and of padded head sizes at 32, 48, 72 and 96 tokens:
//   16 of 64 heads of 100, bf16 out  142/108 161/147 176/209 194/265    128 of them 1018/723 1081/1000 1197/1473 1314/1900
//   the same, fp32 out               180/108 201/147 219/209 236/266               1327/723 1412/1000 1536/1473 1670/1898
//   16 of 64 heads of 53              78/44   89/57   98/77  111/94                 537/238  575/328  634/479  694/608
// The mean counts empty sequences, and hides a long one among short ones: one of 8192 tokens beside 600
// empty ones, 32 heads of 128, takes the token-recurrent kernel, 1400 us of which the states' traffic is 400
// (alone 100 us on the tensor cores). The host knows no lengths.
LinearPlan linear_plan(int64_t total, int num_seqs, int H, int H_k, int d_k, int d_v, bool in_bf16, bool out_bf16,
                       bool recurrent, size_t workspace_bytes) {
  LinearPlan p;
  // TMA addresses rows of a multiple of 16 bytes; other head sizes are padded into the workspace
  const bool odd = d_k % 8 != 0 || d_v % 8 != 0, wide = out_bf16 && d_v > 64;
  const bool small = d_k <= 64 && d_v <= 64;
  const int64_t least = (small ? 48 : wide && d_k > 64 ? 16 : 24) * (!odd ? 1 : small ? 2 : 3);
  p.tensor = in_bf16 && !recurrent && total >= least * num_seqs;
  const bool pad = p.tensor && odd;
  size_t at = 0;
  if (pad) {
    auto take = [&](size_t bytes) {
      const size_t was = at;
      at += align256(bytes);
      return was;
    };
    if (d_k % 8 != 0) {
      p.pad_q = take(size_t(total) * H_k * up8(d_k) * 2);
      p.pad_k = take(size_t(total) * H_k * up8(d_k) * 2);
    }
    if (d_v % 8 != 0) {
      p.pad_v = take(size_t(total) * H * up8(d_v) * 2);
      p.pad_out = take(size_t(total) * H * up8(d_v) * (out_bf16 ? 2 : 4));
      p.pad_states = take(size_t(num_seqs) * H * d_k * up8(d_v) * 4);
    }
    p.pad = at <= workspace_bytes;
    if (!p.pad) p.tensor = false, at = 0;
  }
  p.bytes = at;
  p.col_tile = !p.tensor ? kLinearTokenCols : wide ? 128 : 64;
  const int64_t tiles = (d_v + p.col_tile - 1) / p.col_tile;
  const int64_t unit = p.tensor ? 128 : 16, min_len = p.tensor ? 512 : 48;
  const int64_t tasks = p.tensor ? kLinearSMs : 3 * kLinearSMs;
  int64_t len = 0;
  if (num_seqs == 1) {
    const int64_t m = tasks / (H * tiles);
    if (m >= 2) len = (total + m - 1) / m;
  } else {
    len = (total * H * tiles * 2 + 3 * tasks - 1) / (3 * tasks);
  }
  len = (len + unit - 1) / unit * unit;
  if (len > 0 && len < min_len) len = min_len;
  if (len > 0 && len < total) {
    const int64_t places = total / len + num_seqs;
    const size_t states = align256(size_t(places) * H * d_k * (p.pad ? up8(d_v) : d_v) * 4);
    const size_t decays = align256(size_t(places) * H * 4);
    if (places * H <= INT32_MAX / 4 && at + states + decays <= workspace_bytes) {
      p.seg_len = int32_t(len);
      p.inner = int32_t(total / len);
      p.states = at;
      p.decays = at + states;
      p.bytes = at + states + decays;
    }
  }
  return p;
}

}  // namespace kda
