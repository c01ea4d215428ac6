// Norm after a block, its gate and scaled residual, and the norm in front of
// the next block, in one pass over the rows:
//   u = x * post_weight / sqrt(mean(x^2) + post_eps), u = u * sigmoid(gate)
//   r = residual + scale * u,  y = r * weight / sqrt(mean(r^2) + eps)
//
// A few operations on every element moved: bound by HBM.  A row stays in the
// registers of the lanes that read it, eight neighbouring elements at a time,
// so that each input is read once although both means need the whole row;
// the gate and the residual are requested before the first mean is formed.
// Rows of up to 2048 elements take one wave or a part of one, longer ones a
// workgroup, whose waves join their sums in LDS.  Sums are fp32: each lane's
// own, then the lanes' in a tree, so at most 8 NV + 10 roundings deep.
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

// eight elements with their type's alignment only
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
template <typename T> struct Oct;
template <> struct Oct<bf16> { u32x4 r; };
template <> struct Oct<float> { f32x4 lo, hi; };

__device__ __forceinline__ void load_oct(const bf16 *p, Oct<bf16> &o) {
  o.r = *reinterpret_cast<const u32x4_any *>(p);
}
__device__ __forceinline__ void load_oct(const float *p, Oct<float> &o) {
  o.lo = *reinterpret_cast<const f32x4_any *>(p);
  o.hi = *reinterpret_cast<const f32x4_any *>(p + 4);
}
__device__ __forceinline__ void widen(const Oct<bf16> &o, float *x) { widen8(o.r, x); }
__device__ __forceinline__ void widen(const Oct<float> &o, float *x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = o.lo[i];
    x[4 + i] = o.hi[i];
  }
}
__device__ __forceinline__ void store_oct(bf16 *p, const float *x) {
  bf16x8 v;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = static_cast<bf16>(x[i]);
  *reinterpret_cast<u32x4_any *>(p) = __builtin_bit_cast(u32x4, v);
}
__device__ __forceinline__ void store_oct(float *p, const float *x) {
  *reinterpret_cast<f32x4_any *>(p) = f32x4{x[0], x[1], x[2], x[3]};
  *reinterpret_cast<f32x4_any *>(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
}

// n of eight elements of a row (n >= 8: all; the others read 0)
template <typename T> __device__ __forceinline__ void load_part(const T *p, int n, Oct<T> &o) {
  o = Oct<T>{};
  if (n >= 8) {
    load_oct(p, o);
  } else {
    float x[8] = {};
    for (int i = 0; i < 8; ++i)
      if (i < n)
        x[i] = to_f32(p[i]);
    if constexpr (std::is_same<T, float>::value) {
      o.lo = f32x4{x[0], x[1], x[2], x[3]};
      o.hi = f32x4{x[4], x[5], x[6], x[7]};
    } else {
      bf16x8 v;
      for (int i = 0; i < 8; ++i)
        v[i] = static_cast<bf16>(x[i]);
      o.r = __builtin_bit_cast(u32x4, v);
    }
  }
}
template <typename T> __device__ __forceinline__ void store_part(T *p, int n, const float *x) {
  if (n >= 8) {
    store_oct(p, x);
  } else {
    for (int i = 0; i < 8; ++i)
      if (i < n)
        p[i] = from_f32<T>(x[i]);
  }
}
// eight of a parameter's fp32 values (16-byte aligned at whole groups)
__device__ __forceinline__ void load_param(const float *p, int n, float *x) {
  if (n >= 8) {
    load8f(p, x);
  } else {
    for (int i = 0; i < 8; ++i)
      x[i] = i < n ? p[i] : 0.f;
  }
}

// The sum over the lanes of a row: 2^lanes_log2 lanes of a wave, or with
// BLOCK the whole workgroup (`at`: which of the two sums' LDS).
template <bool BLOCK> __device__ __forceinline__ float row_sum(float v, int lanes_log2, int at) {
  for (int b = 0; b < (BLOCK ? 6 : lanes_log2); ++b)
    v += __shfl_xor(v, 1 << b);
  if constexpr (BLOCK) {
    __shared__ float part[2][16];
    const int waves = blockDim.x >> 6;
    if ((threadIdx.x & 63) == 0)
      part[at][threadIdx.x >> 6] = v;
    lds_barrier();
    v = 0.f;
    for (int w = 0; w < waves; ++w)
      v += part[at][w];
  }
  return v;
}

template <typename T, typename R, int NV, bool BLOCK>
__global__ __launch_bounds__(BLOCK ? 1024 : 256) void norm_kernel(
    NormArgs a, const T *x, const T *gate, const R *residual, R *residual_out, T *y) {
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
  int left[NV]; // elements of each group of eight that the row has
  Oct<T> xr[NV], gr[NV];
  Oct<R> rr[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * lanes + lane) * 8;
    left[i] = real ? a.D - c : 0;
    xr[i] = Oct<T>{};
    gr[i] = Oct<T>{};
    rr[i] = Oct<R>{};
    if (left[i] > 0) {
      load_part(x + row * a.xs + c, left[i], xr[i]);
      if (gate)
        load_part(gate + row * a.gs + c, left[i], gr[i]);
      if (residual)
        load_part(residual + row * a.rs + c, left[i], rr[i]);
    }
  }
  float u[NV][8];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    widen(xr[i], u[i]);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      sum = fmaf(u[i][j], u[i][j], sum);
  }
  float inv = 1.f;
  if (a.post_weight)
    inv = 1.f / sqrtf(row_sum<BLOCK>(sum, a.lanes_log2, 0) * a.inv_D + a.post_eps);
  sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * lanes + lane) * 8;
    if (left[i] <= 0)
      continue;
    float w[8], res[8];
    if (a.post_weight) {
      load_param(a.post_weight + c, left[i], w);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        u[i][j] *= inv * w[j];
    }
    if (gate) {
      widen(gr[i], w);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        u[i][j] *= __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-w[j] * 1.4426950408889634f));
    }
    if (a.scale)
      load_param(a.scale + c, left[i], w);
    widen(rr[i], res);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float su = (a.scale ? w[j] : a.scale_all) * u[i][j];
      u[i][j] = residual ? res[j] + su : su;
      if (j < left[i])
        sum = fmaf(u[i][j], u[i][j], sum);
    }
    if (residual_out)
      store_part(residual_out + row * a.os + c, left[i], u[i]);
  }
  if (!y)
    return;
  inv = 1.f / sqrtf(row_sum<BLOCK>(sum, a.lanes_log2, 1) * a.inv_D + a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * lanes + lane) * 8;
    if (left[i] <= 0)
      continue;
    float w[8];
    load_param(a.weight + c, left[i], w);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      w[j] *= inv * u[i][j];
    store_part(y + row * a.ys + c, left[i], w);
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
  const int need = (D + 7) / 8; // groups of eight
  const auto typed = [&](auto xt, auto rt) {
    using T = decltype(xt);
    using R = decltype(rt);
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
    const auto threads = [&](int nv) { return ((need + nv - 1) / nv + 63) / 64 * 64; };
    if (threads(4) <= 1024)
      return run(integral_constant<int, 4>(), true_type(), rows, threads(4));
    return run(integral_constant<int, 8>(), true_type(), rows, threads(8));
  };
  if (elt == 1)
    return io.residual_dt == KDA_BF16 ? typed(bf16(), bf16()) : typed(bf16(), float());
  return io.residual_dt == KDA_BF16 ? typed(float(), bf16()) : typed(float(), float());
}

} // namespace kda
