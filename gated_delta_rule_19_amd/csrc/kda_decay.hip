// Linear attention with one decay a head, for packed prompts and for single
// tokens:  S_t = exp(g_t) S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t.
#include "kda_block.h"
#include "kda_device.h"

#include <algorithm>
#include <type_traits>

namespace kda {

namespace {

struct DecayArgs {
  int32_t H, num_slots, dk, dv, rq, rk, rv; // r*: heads that share one of q, k, v
  float scale;
  int64_t qs, ks, vs, gs, os;
  const float *g, *init;
  float *fin;
  const int32_t *slots;
};

// exp(g), 0 from -150 down (and for -inf)
__device__ __forceinline__ float decay_of(float g) { return expf(fmaxf(g, -150.f)); }

// One workgroup per (sequence, head, 64 columns): token by token, a column's
// state spread over four lanes.
template <typename T, int D4>
__global__ __launch_bounds__(256) void decay_kernel(SeqTable tab, DecayArgs a, int cols,
                                                    const T *__restrict__ q,
                                                    const T *__restrict__ k,
                                                    const T *__restrict__ v, T *__restrict__ o) {
  const SeqView sv(tab);
  __shared__ float qk[2][256];
  __shared__ float part[256];
  const int n = blockIdx.x / (a.H * cols), hc = blockIdx.x - n * a.H * cols;
  const int h = hc / cols, col = (hc - h * cols) * 64 + (threadIdx.x & 63);
  const int d0 = (threadIdx.x >> 6) * D4;
  const int seq = sv.seq(n), len = sv.len(n);
  const int64_t tok0 = sv.tok0(n);
  const int64_t slot = a.slots ? a.slots[seq] : seq;
  const bool kept = slot >= 0 && slot < a.num_slots, in = col < a.dv;
  const int64_t at = (slot * a.H + h) * a.dk * a.dv + col;
  float S[D4];
#pragma unroll
  for (int d = 0; d < D4; ++d)
    S[d] = a.init && kept && in && d0 + d < a.dk ? a.init[at + (int64_t)(d0 + d) * a.dv] : 0.f;
  for (int t = 0; t < len; ++t) {
    const int64_t row = tok0 + t;
    __syncthreads();
    if (threadIdx.x < a.dk) {
      qk[0][threadIdx.x] = to_f32(q[row * a.qs + (int64_t)(h / a.rq) * a.dk + threadIdx.x]);
      qk[1][threadIdx.x] = to_f32(k[row * a.ks + (int64_t)(h / a.rk) * a.dk + threadIdx.x]);
    }
    const float decay = decay_of(a.g[row * a.gs + h]);
    const float x = in ? to_f32(v[row * a.vs + (int64_t)(h / a.rv) * a.dv + col]) : 0.f;
    __syncthreads();
    float sum = 0.f;
#pragma unroll
    for (int d = 0; d < D4; ++d) {
      if (d0 + d >= a.dk)
        break;
      S[d] = fmaf(qk[1][d0 + d], x, decay * S[d]);
      sum = fmaf(qk[0][d0 + d], S[d], sum);
    }
    part[threadIdx.x] = sum;
    __syncthreads();
    if (threadIdx.x < 64 && in)
      o[row * a.os + (int64_t)h * a.dv + col] =
          from_f32<T>(a.scale * (part[threadIdx.x] + part[threadIdx.x + 64] +
                                 part[threadIdx.x + 128] + part[threadIdx.x + 192]));
  }
  if (a.fin && kept && in)
#pragma unroll
    for (int d = 0; d < D4; ++d)
      if (d0 + d < a.dk)
        a.fin[at + (int64_t)(d0 + d) * a.dv] = S[d];
}

// ---- single tokens ----------------------------------------------------------------

typedef f32x4 f32x4_any __attribute__((aligned(4)));
constexpr int kStepRows = 16; // state rows a lane has in flight

// A workgroup per (row, head): 2^lanes_log2 lanes a state row, four columns
// each, so that the state is read and written in whole lines; 8 dk dv bytes
// for 4 dk dv operations: bound by HBM.
template <typename T>
__global__ __launch_bounds__(256) void decay_step_kernel(DecayArgs a, int lanes_log2,
                                                         const T *__restrict__ q,
                                                         const T *__restrict__ k,
                                                         const T *__restrict__ v,
                                                         T *__restrict__ o) {
  __shared__ float qk[2][KDA_DECAY_MAX_DIM];
  __shared__ float part[4][KDA_DECAY_MAX_DIM];
  const int64_t row = blockIdx.x / a.H;
  const int h = (int)(blockIdx.x - row * a.H);
  const int64_t slot = a.slots ? a.slots[row] : row;
  if (slot < 0 || slot >= a.num_slots)
    return; // a padding entry
  const int lanes = 1 << lanes_log2, col = (threadIdx.x & (lanes - 1)) * 4;
  const int first = threadIdx.x >> lanes_log2, step = 256 >> lanes_log2;
  const int left = a.dv - col; // columns from this lane's on
  float *S = a.fin + (slot * a.H + h) * a.dk * a.dv + col;

  for (int d = threadIdx.x; d < a.dk; d += 256) {
    qk[0][d] = to_f32(q[row * a.qs + (int64_t)(h / a.rq) * a.dk + d]);
    qk[1][d] = to_f32(k[row * a.ks + (int64_t)(h / a.rk) * a.dk + d]);
  }
  const float decay = decay_of(a.g[row * a.gs + h]);
  float x[4], sum[4] = {};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    x[j] = j < left ? to_f32(v[row * a.vs + (int64_t)(h / a.rv) * a.dv + col + j]) : 0.f;
  bool staged = false;
  for (int d0 = first; d0 - first < a.dk; d0 += kStepRows * step) {
    f32x4 s[kStepRows];
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
      const int d = d0 + i * step;
      s[i] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (d < a.dk && left > 0) {
        const float *p = S + d * a.dv;
        if (left >= 4)
          s[i] = *reinterpret_cast<const f32x4_any *>(p);
        else
          s[i] = f32x4{p[0], left > 1 ? p[1] : 0.f, left > 2 ? p[2] : 0.f, 0.f};
      }
    }
    if (!staged)
      lds_barrier();
    staged = true;
#pragma unroll
    for (int i = 0; i < kStepRows; ++i) {
      const int d = d0 + i * step;
      if (d < a.dk && left > 0) {
        const float qd = qk[0][d], kd = qk[1][d];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[i][j] = fmaf(kd, x[j], decay * s[i][j]);
          sum[j] = fmaf(qd, s[i][j], sum[j]);
        }
        float *p = S + d * a.dv;
        if (left >= 4) {
          *reinterpret_cast<f32x4_any *>(p) = s[i];
        } else {
          p[0] = s[i][0];
          if (left > 1)
            p[1] = s[i][1];
          if (left > 2)
            p[2] = s[i][2];
        }
      }
    }
  }
  // the rows' partial sums: lanes of one column, then the waves
  for (int b = lanes; b < 64; b <<= 1)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      sum[j] += __shfl_xor(sum[j], b);
  if ((threadIdx.x & 63) < lanes)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < left)
        part[threadIdx.x >> 6][col + j] = sum[j];
  __syncthreads();
  for (int e = threadIdx.x; e < a.dv; e += 256)
    o[row * a.os + (int64_t)h * a.dv + e] =
        from_f32<T>(a.scale * (part[0][e] + part[1][e] + (part[2][e] + part[3][e])));
}

DecayArgs decay_args(const DecayCall &c) {
  DecayArgs a{};
  a.H = c.H;
  a.num_slots = c.num_slots;
  a.dk = c.io.dk;
  a.dv = c.io.dv;
  a.rq = c.H / c.io.Hq;
  a.rk = c.H / c.io.Hk;
  a.rv = c.H / c.io.Hv;
  a.scale = c.io.scale;
  a.qs = c.io.q_stride;
  a.ks = c.io.k_stride;
  a.vs = c.io.v_stride;
  a.gs = c.io.g_stride;
  a.os = c.io.o_stride;
  a.g = c.io.g;
  a.init = c.init;
  a.fin = c.fin;
  a.slots = c.slots;
  return a;
}

} // namespace

DecayPlan decay_plan(int32_t num_seqs, const int64_t *, int32_t, int32_t, int32_t, int, int32_t) {
  DecayPlan p{};
  p.total = seq_table_bytes(num_seqs);
  return p;
}

hipError_t launch_decay(int elt, const DecayCall &c, int32_t num_seqs, const int64_t *cu,
                        const DecayPlan &, void *ws, hipStream_t s) {
  const DecayArgs a = decay_args(c);
  const int cols = (a.dv + 63) / 64;
  const int64_t grid = (int64_t)num_seqs * a.H * cols;
  if (grid * 256 > UINT32_MAX)
    return hipErrorInvalidConfiguration;
  SeqTable tab;
  const hipError_t e = make_seq_table(
      tab, num_seqs, cu, [](int64_t, int) { return (int64_t)1; }, ws, s);
  if (e != hipSuccess)
    return e;
  const auto run = [&](auto tag, auto d4) {
    using T = decltype(tag);
    decay_kernel<T, decltype(d4)::value><<<(unsigned)grid, 256, 0, s>>>(
        tab, a, cols, (const T *)c.io.q, (const T *)c.io.k, (const T *)c.io.v, (T *)c.io.o);
    return hipGetLastError();
  };
  const auto sized = [&](auto tag) {
    using std::integral_constant;
    if (a.dk <= 64)
      return run(tag, integral_constant<int, 16>());
    if (a.dk <= 128)
      return run(tag, integral_constant<int, 32>());
    return run(tag, integral_constant<int, 64>());
  };
  return elt == 1 ? sized(bf16()) : sized(float());
}

hipError_t launch_decay_step(int elt, const DecayCall &c, int32_t rows, hipStream_t s) {
  const DecayArgs a = decay_args(c);
  const int64_t grid = (int64_t)rows * a.H;
  if (grid * 256 > UINT32_MAX)
    return hipErrorInvalidConfiguration;
  int lanes_log2 = 0;
  while ((4 << lanes_log2) < a.dv)
    ++lanes_log2;
  const auto run = [&](auto tag) {
    using T = decltype(tag);
    decay_step_kernel<T><<<(unsigned)grid, 256, 0, s>>>(a, lanes_log2, (const T *)c.io.q,
                                                        (const T *)c.io.k, (const T *)c.io.v,
                                                        (T *)c.io.o);
    return hipGetLastError();
  };
  return elt == 1 ? run(bf16()) : run(float());
}

} // namespace kda
