// 8-bit state cache: fp32 state rows quantised as they are written, and read
// back.
//
// A row is L consecutive values that share one fp32 scale (KDA: the 128
// value channels of one key channel; the selective scan: the N states of one
// channel -- the decay acts on whole rows, so their magnitudes differ from
// row to row far more than within one):
//   scale = amax / qmax (at least 2^-126),  code = round_to_nearest_even(x * (1 / scale))
//   x'    = code * scale,              qmax = 127 (int8) or 448 (e4m3)
// A row that holds an infinity or a NaN has no scale: it is stored as NaN
// with codes 0 and reads back as NaN.  All arithmetic is fp32; the code is
// the only rounding to fewer bits (half a step: amax / 254 for int8, 2^-4 of
// the value for e4m3 above its subnormals).
//
// 5 bytes move per value and a few operations are done on it: bound by HBM.
// A row is spread over `lanes` neighbouring lanes (a power of two) with VEC
// values each, so a wave reads and writes whole lines, and the row maximum
// crosses the lanes in registers.
#include "kda_device.h"
#include "kda_recurrent.h"

#include <type_traits>

namespace kda {

namespace {

struct CacheArgs {
  int32_t L, lanes_log2, num_src, num_dst;
  int64_t R;
  int64_t waves;   // all waves
  int64_t per;     // waves per item
  const int32_t *src, *dst;
};

// The largest scales whose product with qmax stays finite: the quotient of
// the largest finite value rounds up past the one for 127.
constexpr float kTopInt8 = 0x1.020406p+121f, kTopE4M3 = 0x1.249248p+119f;

// kRows row groups per wave: their loads are in flight together.  Stores are
// non-temporal (what is written is as large as the states of a batch).  64
// KDA states of 96 heads to e4m3: 107, 89, 91, 95 us with 1, 2, 4, 8 groups,
// 84 us with 2 and non-temporal stores (6.06 TB/s); 250 x 8192 rows of 16
// int8 read back: 37.6 us, 25.6 us non-temporal (6.7 TB/s).
constexpr int kRows = 2;

__device__ __forceinline__ unsigned umax_lanes(unsigned m, int lanes_log2) {
  // (uniform trip count)
  for (int b = 0; b < lanes_log2; ++b)
    m = max(m, (unsigned)__shfl_xor((int)m, 1 << b));
  return m;
}

__device__ __forceinline__ int encode_int8(float v) { return (int)__builtin_rintf(v); }

// VEC values a lane, K times: value (k * lanes + lane) * VEC + i of the row.
template <int VEC, int K, bool E4M3>
__global__ __launch_bounds__(256) void store_kernel(CacheArgs a, const float *__restrict__ state,
                                                    uint8_t *__restrict__ codes,
                                                    float *__restrict__ scales) {
  const int64_t wave = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (wave >= a.waves)
    return;
  const int item = (int)(wave / a.per);
  const int64_t from = a.src ? a.src[item] : item, to = a.dst ? a.dst[item] : item;
  if (from < 0 || from >= a.num_src || to < 0 || to >= a.num_dst)
    return; // a padding entry
  const int lanes = 1 << a.lanes_log2;
  const int lane = threadIdx.x & (lanes - 1);
  const int group = (threadIdx.x & 63) >> a.lanes_log2;
  const int rows = 64 >> a.lanes_log2; // rows of a row group
  const int64_t row0 = (wave - item * a.per) * (kRows * rows) + group;

  float v[kRows][K][VEC];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int64_t row = row0 + r * rows;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * lanes + lane) * VEC;
      const float *p = state + (from * a.R + row) * a.L + c;
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        v[r][k][i] = 0.f;
      if (row < a.R && c < a.L) {
        if constexpr (VEC == 4) {
          const f32x4 x = __builtin_nontemporal_load(reinterpret_cast<const f32x4 *>(p));
#pragma unroll
          for (int i = 0; i < 4; ++i)
            v[r][k][i] = x[i];
        } else
          v[r][k][0] = *p;
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int64_t row = row0 + r * rows;
    // magnitudes as integers: their order is the values', with infinity and
    // NaN above every finite value
    unsigned m = 0;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        m = max(m, __builtin_bit_cast(unsigned, v[r][k][i]) & 0x7fffffffu);
    m = umax_lanes(m, a.lanes_log2);
    const bool finite = m < 0x7f800000u;
    const float amax = __builtin_bit_cast(float, m);
    const float scale =
        fminf(fmaxf(amax / (E4M3 ? 448.f : 127.f), 0x1p-126f), E4M3 ? kTopE4M3 : kTopInt8);
    const float inv = finite ? 1.f / scale : 0.f;
    if (row >= a.R)
      continue;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * lanes + lane) * VEC;
      if (c >= a.L)
        continue;
      uint8_t *p = codes + (to * a.R + row) * a.L + c;
      float q[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        q[i] = finite ? v[r][k][i] * inv : 0.f;
      int w;
      if constexpr (E4M3) {
        w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
        if constexpr (VEC == 4)
          w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
      } else {
        w = encode_int8(q[0]) & 255;
        if constexpr (VEC == 4)
          w |= (encode_int8(q[1]) & 255) << 8 | (encode_int8(q[2]) & 255) << 16 |
               encode_int8(q[3]) << 24;
      }
      if constexpr (VEC == 4)
        __builtin_nontemporal_store(w, reinterpret_cast<int *>(p));
      else
        *p = (uint8_t)w;
    }
    if (lane == 0)
      scales[to * a.R + row] = finite ? scale : __builtin_nanf("");
  }
}

template <int VEC, int K, bool E4M3>
__global__ __launch_bounds__(256) void load_kernel(CacheArgs a, const uint8_t *__restrict__ codes,
                                                   const float *__restrict__ scales,
                                                   float *__restrict__ state) {
  const int64_t wave = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (wave >= a.waves)
    return;
  const int item = (int)(wave / a.per);
  const int64_t from = a.src ? a.src[item] : item, to = a.dst ? a.dst[item] : item;
  if (from < 0 || from >= a.num_src || to < 0 || to >= a.num_dst)
    return; // a padding entry
  const int lanes = 1 << a.lanes_log2;
  const int lane = threadIdx.x & (lanes - 1);
  const int group = (threadIdx.x & 63) >> a.lanes_log2;
  const int rows = 64 >> a.lanes_log2;
  const int64_t row0 = (wave - item * a.per) * (kRows * rows) + group;

  int w[kRows][K];
  float sc[kRows];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int64_t row = row0 + r * rows;
    sc[r] = row < a.R ? scales[from * a.R + row] : 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * lanes + lane) * VEC;
      const uint8_t *p = codes + (from * a.R + row) * a.L + c;
      w[r][k] = 0;
      if (row < a.R && c < a.L) {
        if constexpr (VEC == 4)
          w[r][k] = *reinterpret_cast<const int *>(p);
        else
          w[r][k] = *p;
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int64_t row = row0 + r * rows;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int c = (k * lanes + lane) * VEC;
      if (row >= a.R || c >= a.L)
        continue;
      float x[4];
      if constexpr (E4M3) {
        x[0] = __builtin_amdgcn_cvt_f32_fp8(w[r][k], 0);
        x[1] = __builtin_amdgcn_cvt_f32_fp8(w[r][k], 1);
        x[2] = __builtin_amdgcn_cvt_f32_fp8(w[r][k], 2);
        x[3] = __builtin_amdgcn_cvt_f32_fp8(w[r][k], 3);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          x[i] = (float)(int8_t)(w[r][k] >> (8 * i));
      }
      float *p = state + (to * a.R + row) * a.L + c;
      if constexpr (VEC == 4)
        __builtin_nontemporal_store(
            f32x4{x[0] * sc[r], x[1] * sc[r], x[2] * sc[r], x[3] * sc[r]},
            reinterpret_cast<f32x4 *>(p));
      else
        *p = x[0] * sc[r];
    }
  }
}

// Launch shape: VEC values per lane (4 when every row is 16-byte aligned in
// the state and 4-byte aligned in the codes), the smallest power-of-two lane
// count that holds a row, and for rows of more than 64 VEC values several
// passes.  Rows of other lengths pay for single elements: store and load of 64
// x 12288 rows of 13 take 30 and 21 us (8.8 at the copy's rate), of 127 155 to
// 158 and 145 (int8: 197; 82), of 128 84 to 99 and 90.
template <typename F>
hipError_t cache_launch(const CacheCall &c, const float *state, const void *codes, F &&run) {
  const bool wide = c.L % 4 == 0 && ((uintptr_t)state & 15u) == 0 && ((uintptr_t)codes & 3u) == 0;
  const int per_lane = wide ? 4 : 1;
  const int need = (c.L + per_lane - 1) / per_lane;
  CacheArgs a{};
  a.L = c.L;
  while ((1 << a.lanes_log2) < need && a.lanes_log2 < 6)
    ++a.lanes_log2;
  a.num_src = c.num_src;
  a.num_dst = c.num_dst;
  a.R = c.R;
  a.src = c.src;
  a.dst = c.dst;
  const int64_t rows = (int64_t)kRows * (64 >> a.lanes_log2);
  a.per = (c.R + rows - 1) / rows;
  a.waves = a.per * c.n;
  if (a.waves > (int64_t)(UINT32_MAX / 256) * 4) // (the threads' count may pass 64 bits)
    return hipErrorInvalidConfiguration;
  const dim3 grid((unsigned)((a.waves + 3) / 4));
  auto k = [&](auto vec, auto kk) {
    if (c.format == 1)
      run(vec, kk, std::true_type(), a, grid);
    else
      run(vec, kk, std::false_type(), a, grid);
    return hipGetLastError();
  };
  using std::integral_constant;
  if (wide)
    return k(integral_constant<int, 4>(), integral_constant<int, 1>());
  if (need <= 64)
    return k(integral_constant<int, 1>(), integral_constant<int, 1>());
  if (need <= 128)
    return k(integral_constant<int, 1>(), integral_constant<int, 2>());
  return k(integral_constant<int, 1>(), integral_constant<int, 4>());
}

} // namespace

hipError_t launch_state_store(const CacheCall &c, hipStream_t s) {
  return cache_launch(c, c.state_in, c.codes_out,
                      [&](auto vec, auto k, auto e4m3, const CacheArgs &a, dim3 grid) {
                        store_kernel<decltype(vec)::value, decltype(k)::value,
                                     decltype(e4m3)::value><<<grid, 256, 0, s>>>(
                            a, c.state_in, (uint8_t *)c.codes_out, c.scales_out);
                      });
}

hipError_t launch_state_load(const CacheCall &c, hipStream_t s) {
  return cache_launch(c, c.state_out, c.codes_in,
                      [&](auto vec, auto k, auto e4m3, const CacheArgs &a, dim3 grid) {
                        load_kernel<decltype(vec)::value, decltype(k)::value,
                                    decltype(e4m3)::value><<<grid, 256, 0, s>>>(
                            a, (const uint8_t *)c.codes_in, c.scales_in, c.state_out);
                      });
}

} // namespace kda
