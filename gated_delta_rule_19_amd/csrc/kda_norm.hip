// Norm after a block, its gate and scaled residual, and the norm in front of
// the next block, in one pass over the rows:
//   u = x * post_weight / sqrt(mean(x^2) + post_eps), u = u * sigmoid(gate)
//   r = residual + scale * u,  y = r * weight / sqrt(mean(r^2) + eps)
//
// A few operations on every element moved: bound by HBM.  A row stays in the
// registers of the lanes that read it, 16 bytes of the widest type at a time,
// so that each input is read once although both means need the whole row;
// the gate and the residual are requested before the first mean is formed.
// Rows of up to 256 groups take one wave or a part of one, longer ones a
// workgroup, whose waves join their sums in LDS.  Sums are fp32: each lane's
// own of up to 64 elements, then the lanes' in a tree: 74 roundings deep at most.
//
// 8192 x 12288 bf16 with all parts: 184 us for 1.01 GB, 5.5 TB/s, what a large
// copy reaches on the same card.  Two groups a lane keep more rows in flight
// than four (194 us then, 205), and non-temporal accesses, here larger than all
// caches, gain as much (cached: 216 us).  20000 x 1002 fp32: 81 us for 401 MB (5.0
// TB/s): rows that end inside a 128-byte line cost a tenth (1024 columns: 5.5).
// One row: 5.0 us on the GPU, the latency of three rounds to memory and two
// joins of sums.
#include "kda_block.h"
#include "kda_device.h"

#include <type_traits>

namespace kda {

namespace {

struct NormArgs {
  int32_t rows, D, lanes_log2; // lanes_log2: of a row in a wave
  int64_t xs, gs, rs, os, ys;
  const float *post_weight, *weight, *scale;
  float post_eps, eps, scale_all, inv_D;
};

// E neighbouring elements, with their type's alignment only: 16 bytes of the
// widest type, so that a wave's access is one run of memory.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
template <typename T, int E> struct GroupOf;
template <> struct GroupOf<bf16, 8> { typedef u32x4 type; typedef u32x4_any any; };
template <> struct GroupOf<bf16, 4> { typedef u32x2 type; typedef u32x2_any any; };
template <> struct GroupOf<float, 4> { typedef f32x4 type; typedef f32x4_any any; };
template <typename T, int E> using Group = typename GroupOf<T, E>::type;

__device__ __forceinline__ void widen(const u32x4 &g, float *x) { widen8(g, x); }
__device__ __forceinline__ void widen(const u32x2 &g, float *x) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = __builtin_bit_cast(float, i % 2 ? g[i / 2] & 0xffff0000u : g[i / 2] << 16);
}
__device__ __forceinline__ void widen(const f32x4 &g, float *x) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = g[i];
}
template <typename T, int E> __device__ __forceinline__ Group<T, E> rounded(const float *x) {
  typedef T Vec __attribute__((ext_vector_type(E)));
  Vec v;
#pragma unroll
  for (int i = 0; i < E; ++i)
    v[i] = from_f32<T>(x[i]);
  return __builtin_bit_cast(Group<T, E>, v);
}

// n of E elements of a row (n >= E: all; the others read 0)
template <int E, typename T>
__device__ __forceinline__ Group<T, E> load_part(const T *p, int n) {
  if (n >= E)
    return __builtin_nontemporal_load(reinterpret_cast<const typename GroupOf<T, E>::any *>(p));
  float x[E];
  for (int i = 0; i < E; ++i)
    x[i] = i < n ? to_f32(p[i]) : 0.f;
  return rounded<T, E>(x);
}
template <int E, typename T>
__device__ __forceinline__ void store_part(T *p, int n, const float *x) {
  if (n >= E) {
    __builtin_nontemporal_store(rounded<T, E>(x),
                                reinterpret_cast<typename GroupOf<T, E>::any *>(p));
  } else {
    for (int i = 0; i < E; ++i)
      if (i < n)
        p[i] = from_f32<T>(x[i]);
  }
}
// E of a parameter's fp32 values (16-byte aligned at whole groups)
template <int E> __device__ __forceinline__ void load_param(const float *p, int n, float *x) {
  if (n >= E) {
#pragma unroll
    for (int i = 0; i < E; i += 4)
      widen(*reinterpret_cast<const f32x4 *>(p + i), x + i);
  } else {
    for (int i = 0; i < E; ++i)
      x[i] = i < n ? p[i] : 0.f;
  }
}

// 1 / (1 + e^-w): exp2 of the rounded product t with log2(e), and to first order
// what t leaves of it (that alone would be |w| 2^-24 of the result).  Not where
// all outputs are bf16, half a step of which is hundreds of times that even at the
// ends of fp32's range (4 rows of 65536: 18.9 us, with it 21.1).
template <bool EXACT> __device__ __forceinline__ float sigmoid(float w) {
  constexpr float c1 = 0x1.715476p+0f, c2 = 0x1.4ae0bep-26f; // c1 + c2: log2(e)
  constexpr float ln2 = 0x1.62e43p-1f;
  const float t = -w * c1, e = __builtin_amdgcn_exp2f(t);
  if constexpr (!EXACT)
    return __builtin_amdgcn_rcpf(1.f + e);
  const float left = fmaf(-w, c2, fmaf(-w, c1, -t));
  // (past fp32's range e is infinity or nothing, whatever is left)
  return __builtin_amdgcn_rcpf(1.f + (fabsf(t) < 127.f ? fmaf(e, left * ln2, e) : e));
}

// The sum over the lanes of a row: 2^lanes_log2 lanes of a wave, or with
// BLOCK the whole workgroup (`at`: which of the two sums' LDS).
template <bool BLOCK> __device__ __forceinline__ float row_sum(float v, int lanes_log2, int at) {
  for (int b = 0; b < (BLOCK ? 6 : lanes_log2); ++b)
    v += __shfl_xor(v, 1 << b);
  if constexpr (BLOCK) {
    __shared__ alignas(16) float part[2][16];
    const int waves = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0)
      part[at][threadIdx.x >> 6] = v;
    if (threadIdx.x < 16 && (int)threadIdx.x >= waves)
      part[at][threadIdx.x] = 0.f;
    lds_barrier();
    const f32x4 *p = reinterpret_cast<const f32x4 *>(part[at]);
    const f32x4 w = (p[0] + p[1]) + (p[2] + p[3]);
    v = (w[0] + w[1]) + (w[2] + w[3]);
  }
  return v;
}

// Elements of a group.
template <typename T, typename R> constexpr int kGroup = sizeof(T) + sizeof(R) == 4 ? 8 : 4;

// NV groups a lane.  Rows of more than 32768 elements leave no registers to
// hold x, the gate and the residual at once: these two are read behind the
// first mean.
template <typename T, typename R, int NV, bool BLOCK>
__global__ __launch_bounds__(BLOCK ? 1024 : 256) void norm_kernel(
    NormArgs a, const T *x, const T *gate, const R *residual, R *residual_out, T *y) {
  constexpr int E = kGroup<T, R>;
  constexpr bool AHEAD = NV * E <= 32;
  int64_t row;
  int lane, lanes;
  if constexpr (BLOCK) {
    row = blockIdx.x;
    lane = threadIdx.x;
    lanes = blockDim.x;
  } else {
    lanes = 1 << a.lanes_log2;
    lane = threadIdx.x & (lanes - 1);
    row = ((int64_t)blockIdx.x * 256 + threadIdx.x) >> a.lanes_log2;
  }
  const bool real = row < a.rows;
  int left[NV]; // elements from each group's start on that the row has
  Group<T, E> xr[NV], gr[NV];
  Group<R, E> rr[NV];
  const auto load_others = [&](int i) __attribute__((always_inline)) {
    const int c = (i * lanes + lane) * E;
    gr[i] = gate && left[i] > 0 ? load_part<E>(gate + row * a.gs + c, left[i]) : Group<T, E>{};
    rr[i] = residual && left[i] > 0 ? load_part<E>(residual + row * a.rs + c, left[i])
                                    : Group<R, E>{};
  };
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * lanes + lane) * E;
    left[i] = real ? a.D - c : 0;
    xr[i] = left[i] > 0 ? load_part<E>(x + row * a.xs + c, left[i]) : Group<T, E>{};
    if constexpr (AHEAD)
      load_others(i);
  }
  float u[NV][E];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    widen(xr[i], u[i]);
#pragma unroll
    for (int j = 0; j < E; ++j)
      sum = fmaf(u[i][j], u[i][j], sum);
  }
  float inv = 1.f;
  if (a.post_weight)
    inv = 1.f / sqrtf(row_sum<BLOCK>(sum, a.lanes_log2, 0) * a.inv_D + a.post_eps);
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * lanes + lane) * E;
    if (left[i] <= 0)
      continue;
    if constexpr (!AHEAD)
      load_others(i);
    float w[E], res[E];
    if (a.post_weight) {
      load_param<E>(a.post_weight + c, left[i], w);
#pragma unroll
      for (int j = 0; j < E; ++j)
        u[i][j] *= inv * w[j];
    }
    if (gate) {
      widen(gr[i], w);
#pragma unroll
      for (int j = 0; j < E; ++j)
        u[i][j] *= sigmoid<sizeof(T) + sizeof(R) != 4>(w[j]);
    }
    if (a.scale)
      load_param<E>(a.scale + c, left[i], w);
    widen(rr[i], res);
#pragma unroll
    for (int j = 0; j < E; ++j) {
      const float su = (a.scale ? w[j] : a.scale_all) * u[i][j];
      u[i][j] = residual ? res[j] + su : su;
      if (j < left[i])
        sum = fmaf(u[i][j], u[i][j], sum);
    }
    if (residual_out)
      store_part<E>(residual_out + row * a.os + c, left[i], u[i]);
  }
  if (!y)
    return;
  inv = 1.f / sqrtf(row_sum<BLOCK>(sum, a.lanes_log2, 1) * a.inv_D + a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * lanes + lane) * E;
    if (left[i] <= 0)
      continue;
    float w[E];
    load_param<E>(a.weight + c, left[i], w);
#pragma unroll
    for (int j = 0; j < E; ++j)
      w[j] *= inv * u[i][j];
    store_part<E>(y + row * a.ys + c, left[i], w);
  }
}

} // namespace

hipError_t launch_block_norm(int elt, int32_t rows, int32_t D, const kda_norm_io &io,
                             hipStream_t s) {
  NormArgs a{};
  a.rows = rows;
  a.D = D;
  a.xs = io.x_stride;
  a.gs = io.gate_stride;
  a.rs = io.residual_stride;
  a.os = io.residual_out_stride;
  a.ys = io.y_stride;
  a.post_weight = io.post_weight;
  a.weight = io.weight;
  a.scale = io.scale;
  a.post_eps = io.post_eps;
  a.eps = io.eps;
  a.scale_all = io.scale_all;
  a.inv_D = 1.f / (float)D;
  const auto typed = [&](auto xt, auto rt) {
    using T = decltype(xt);
    using R = decltype(rt);
    constexpr int E = kGroup<T, R>;
    const int need = (D + E - 1) / E; // groups
    const auto run = [&](auto nv, auto block, int64_t grid, int threads) {
      // (the device's grids: 2^32 - 1 threads)
      if (grid * threads > UINT32_MAX)
        return hipErrorInvalidConfiguration;
      norm_kernel<T, R, decltype(nv)::value, decltype(block)::value>
          <<<(unsigned)grid, threads, 0, s>>>(a, (const T *)io.x, (const T *)io.gate,
                                              (const R *)io.residual, (R *)io.residual_out,
                                              (T *)io.y);
      return hipGetLastError();
    };
    using std::false_type;
    using std::integral_constant;
    using std::true_type;
    if (need <= 256) { // a wave or less per row
      while ((1 << a.lanes_log2) < need && a.lanes_log2 < 6)
        ++a.lanes_log2;
      const int64_t grid = ((int64_t)rows * (1 << a.lanes_log2) + 255) / 256;
      if (need <= 64)
        return run(integral_constant<int, 1>(), false_type(), grid, 256);
      if (need <= 128)
        return run(integral_constant<int, 2>(), false_type(), grid, 256);
      return run(integral_constant<int, 4>(), false_type(), grid, 256);
    }
    const auto block = [&](auto nv) {
      const int threads = ((need + decltype(nv)::value - 1) / decltype(nv)::value + 63) / 64 * 64;
      return threads <= 1024 ? run(nv, true_type(), rows, threads) : hipErrorInvalidConfiguration;
    };
    if (need <= 2048)
      return block(integral_constant<int, 2>());
    if (need <= 4096)
      return block(integral_constant<int, 4>());
    if (E == 8 || need <= 8192)
      return block(integral_constant<int, 8>());
    return block(integral_constant<int, 64 / E>());
  };
  if (elt == 1)
    return io.residual_dt == KDA_BF16 ? typed(bf16(), bf16()) : typed(bf16(), float());
  return io.residual_dt == KDA_BF16 ? typed(float(), bf16()) : typed(float(), float());
}

} // namespace kda
