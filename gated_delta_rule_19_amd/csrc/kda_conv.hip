// Short causal depthwise convolution in front of the recurrence, for packed
// prompts and for single tokens.
//
//   y[t, d] = act(bias[d] + sum_{j < W} w[d, j] x[t - (W - 1) + j, d])
//
// where the W - 1 positions before a sequence's first token are the rows of
// its state (oldest first), and the state after the sequence is its last
// W - 1 inputs.  2 W flops for two elements moved: bound by HBM.  A lane owns
// VEC neighbouring channels (16 bytes) with their weights and the window of
// W - 1 inputs in registers and walks down a run of tokens, so each input is
// read once (plus W - 1 rows of run-in per tile, which the neighbouring tile
// has just brought into L2) and nothing passes through LDS.
#include "kda_device.h"
#include "kda_recurrent.h"
#include "kda_seqtab.h"

#include <type_traits>

namespace kda {

// ---- the packed-sequence table of long batches -------------------------------
__global__ __launch_bounds__(kTablePart) void seq_table_kernel(TablePart part, int count,
                                                               SeqEntry *__restrict__ dst) {
  const int i = threadIdx.x;
  if (i < count)
    dst[i] = part.e[i];
}

hipError_t launch_table_part(const TablePart &part, int count, SeqEntry *dst, hipStream_t s) {
  seq_table_kernel<<<1, kTablePart, 0, s>>>(part, count, dst);
  return hipGetLastError();
}

// ---- element vectors ------------------------------------------------------------
// A 16-byte vector with its elements' alignment only: rows may start anywhere
// (this target's unaligned access mode serves such loads).  8192 tokens of
// 12289 bf16 channels take 84 us, 108 with one element a lane; 12288: 75.
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
template <typename T, int VEC> struct Pack;
template <> struct Pack<bf16, 8> { u32x4_any r; };
template <> struct Pack<float, 4> { f32x4_any r; };
template <> struct Pack<bf16, 1> { bf16 r; };
template <> struct Pack<float, 1> { float r; };

__device__ __forceinline__ void unpack(const Pack<bf16, 8> &p, float *x) { widen8(p.r, x); }
__device__ __forceinline__ void unpack(const Pack<float, 4> &p, float *x) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    x[i] = p.r[i];
}
__device__ __forceinline__ void unpack(const Pack<bf16, 1> &p, float *x) { x[0] = to_f32(p.r); }
__device__ __forceinline__ void unpack(const Pack<float, 1> &p, float *x) { x[0] = p.r; }

template <typename T, int VEC> __device__ __forceinline__ Pack<T, VEC> load_pack(const T *p) {
  return *reinterpret_cast<const Pack<T, VEC> *>(p);
}
template <typename T, int VEC>
__device__ __forceinline__ void store_pack(T *p, const Pack<T, VEC> &v) {
  *reinterpret_cast<Pack<T, VEC> *>(p) = v;
}
template <typename T, int VEC> __device__ __forceinline__ Pack<T, VEC> zero_pack() {
  Pack<T, VEC> p;
  __builtin_memset(&p, 0, sizeof(p));
  return p;
}
// (non-temporal: the prompt's outputs are larger than a die's L2; 222 -> 212 us
// at 8192 x 36864 bf16, 52 -> 48 us at 20000 x 1536 fp32)
template <typename T, int VEC> __device__ __forceinline__ void store_f32(T *p, const float *x) {
  if constexpr (VEC == 8) {
    bf16x8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = static_cast<bf16>(x[i]);
    __builtin_nontemporal_store(__builtin_bit_cast(u32x4, v), reinterpret_cast<u32x4_any *>(p));
  } else if constexpr (VEC == 4) {
    __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]},
                                reinterpret_cast<f32x4_any *>(p));
  } else {
    *p = from_f32<T>(x[0]);
  }
}

// Weights [D, W] and bias of a lane's VEC channels.
template <typename T, int VEC, int W> struct Taps {
  float w[W][VEC], b[VEC];

  __device__ __forceinline__ void load(const T *weight, const T *bias, int64_t d) {
    // one lane's VEC * W weights are contiguous
    float f[VEC * W];
#pragma unroll
    for (int i = 0; i < W; ++i)
      unpack(load_pack<T, VEC>(weight + d * W + i * VEC), f + i * VEC);
#pragma unroll
    for (int i = 0; i < VEC * W; ++i)
      w[i % W][i / W] = f[i];
    unpack(bias ? load_pack<T, VEC>(bias + d) : zero_pack<T, VEC>(), b);
  }
  // win: the W - 1 inputs before x, oldest first
  __device__ __forceinline__ void apply(const float (&win)[W - 1][VEC], const float *x, bool act,
                                        float *y) const {
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      float s = b[i];
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
        s = fmaf(w[j][i], win[j][i], s);
      s = fmaf(w[W - 1][i], x[i], s);
      y[i] = act ? silu(s) : s;
    }
  }
};

template <int VEC, int W>
__device__ __forceinline__ void shift(float (&win)[W - 1][VEC], const float *x) {
#pragma unroll
  for (int j = 0; j + 1 < W - 1; ++j)
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      win[j][i] = win[j + 1][i];
#pragma unroll
  for (int i = 0; i < VEC; ++i)
    win[W - 2][i] = x[i];
}

// Tokens per tile.  Short tiles keep the rows in flight close together: 8192
// x 36864 bf16 runs in 222, 229, 248, 257 us with tiles of 8, 16, 32, 64,
// though a tile of 8 reads W - 1 run-in rows for its 8 (from L2 or the
// memory-side cache, where the tile before has just brought them).
constexpr int kConvTile = 8;
static_assert(kConvTile >= 7, "a tile's run-in lies within the tile before");

struct ConvArgs {
  int32_t D, cw;      // channels; waves per row of channels
  int32_t full;       // lanes with VEC channels; the D % VEC others have a lane each
  int32_t act;        // 1: silu
  int32_t num_slots;
  int64_t xs, ys;     // row strides
  int64_t waves;      // all waves with work
  const int32_t *slots;
};

// One tile of one sequence, VEC channels from d.
template <typename T, int VEC, int W>
__device__ __forceinline__ void conv_tile(const ConvArgs &a, const T *x, const T *weight,
                                          const T *bias, const T *init, T *fin, T *y, int64_t d,
                                          int t0, int len, int64_t slot, bool kept) {
  constexpr int kW1 = W - 1;
  using P = Pack<T, VEC>;
  x += d;
  y += d;
  float win[kW1][VEC];
  if (t0 > 0) {
    // (a tile is at least W - 1 tokens)
#pragma unroll
    for (int j = 0; j < kW1; ++j)
      unpack(load_pack<T, VEC>(x + (int64_t)(t0 - kW1 + j) * a.xs), win[j]);
  } else {
    P first[kW1];
#pragma unroll
    for (int j = 0; j < kW1; ++j) {
      first[j] = init && kept ? load_pack<T, VEC>(init + (slot * kW1 + j) * a.D + d)
                              : zero_pack<T, VEC>();
      unpack(first[j], win[j]);
    }
    if (fin && kept) {
#pragma unroll
      for (int j = 0; j < kW1; ++j) {
        const int p = len - kW1 + j; // position of row j of the final state
        P v = zero_pack<T, VEC>();
        if (p >= 0)
          v = load_pack<T, VEC>(x + (int64_t)p * a.xs);
        else {
#pragma unroll
          for (int r = j; r < kW1; ++r)
            if (r == p + kW1)
              v = first[r];
        }
        store_pack<T, VEC>(fin + (slot * kW1 + j) * a.D + d, v);
      }
    }
  }
  Taps<T, VEC, W> taps;
  taps.load(weight, bias, d);

  // a whole tile's loads are in flight together
  if (len - t0 >= kConvTile) {
    P in[kConvTile];
#pragma unroll
    for (int u = 0; u < kConvTile; ++u)
      in[u] = load_pack<T, VEC>(x + (int64_t)(t0 + u) * a.xs);
#pragma unroll
    for (int u = 0; u < kConvTile; ++u) {
      float xv[VEC], yv[VEC];
      unpack(in[u], xv);
      taps.apply(win, xv, a.act != 0, yv);
      shift<VEC, W>(win, xv);
      store_f32<T, VEC>(y + (int64_t)(t0 + u) * a.ys, yv);
    }
    return;
  }
  for (int t = t0; t < len; ++t) {
    float xv[VEC], yv[VEC];
    unpack(load_pack<T, VEC>(x + (int64_t)t * a.xs), xv);
    taps.apply(win, xv, a.act != 0, yv);
    shift<VEC, W>(win, xv);
    store_f32<T, VEC>(y + (int64_t)t * a.ys, yv);
  }
}

// Lane l of a row of channels: the VEC channels from l VEC, or (REST, past
// the `full` lanes with VEC of them) one of the D % VEC others.  run(vec, d).
template <int VEC, bool REST, typename F>
__device__ __forceinline__ void by_channels(const ConvArgs &a, int64_t l, F &&run) {
  if (l < a.full) {
    run(std::integral_constant<int, VEC>(), l * VEC);
  } else if constexpr (REST) {
    const int64_t d = (int64_t)a.full * VEC + (l - a.full);
    if (d < a.D)
      run(std::integral_constant<int, 1>(), d);
  }
}

// One wave per (tile of one sequence, 64 lanes of channels).  The wave of a
// sequence's first tile also reads the initial state and writes the final
// one, so the two may be the same buffer.
template <typename T, int VEC, int W, bool REST>
__global__ __launch_bounds__(256) void conv_kernel(SeqTable tab, ConvArgs a,
                                                   const T *__restrict__ x,
                                                   const T *__restrict__ weight,
                                                   const T *__restrict__ bias, const T *init,
                                                   T *fin, T *__restrict__ y) {
  const int64_t wave = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (wave >= a.waves)
    return;
  const int blk = (int)(wave / a.cw);
  const int64_t l = (wave - (int64_t)blk * a.cw) * 64 + (threadIdx.x & 63);
  const SeqView seqs(tab);
  const int n = seqs.find(blk, 0);
  const int t0 = (blk - seqs.blk(n, 0)) * kConvTile;
  const int len = seqs.len(n);
  const int64_t tok0 = seqs.tok0(n);
  int64_t slot = seqs.seq(n);
  bool kept = true;
  if (a.slots) {
    slot = a.slots[slot];
    kept = slot >= 0 && slot < a.num_slots;
  }
  by_channels<VEC, REST>(a, l, [&](auto vec, int64_t d) {
    conv_tile<T, decltype(vec)::value, W>(a, x + tok0 * a.xs, weight, bias, init, fin,
                                          y + tok0 * a.ys, d, t0, len, slot, kept);
  });
}

// Single tokens: one wave per (row, 64 lanes of channels); reads the W - 1
// rows of the row's state and the input, writes the output and the shifted
// state.
template <typename T, int VEC, int W>
__device__ __forceinline__ void conv_token(const ConvArgs &a, const T *x, const T *weight,
                                           const T *bias, T *st, T *y, int64_t d) {
  constexpr int kW1 = W - 1;
  using P = Pack<T, VEC>;
  st += d;
  P old[kW1];
#pragma unroll
  for (int j = 0; j < kW1; ++j)
    old[j] = load_pack<T, VEC>(st + (int64_t)j * a.D);
  const P xin = load_pack<T, VEC>(x + d);
  Taps<T, VEC, W> taps;
  taps.load(weight, bias, d);
  float win[kW1][VEC], xv[VEC], yv[VEC];
#pragma unroll
  for (int j = 0; j < kW1; ++j)
    unpack(old[j], win[j]);
  unpack(xin, xv);
  taps.apply(win, xv, a.act != 0, yv);
  store_f32<T, VEC>(y + d, yv);
#pragma unroll
  for (int j = 0; j + 1 < kW1; ++j)
    store_pack<T, VEC>(st + (int64_t)j * a.D, old[j + 1]);
  store_pack<T, VEC>(st + (int64_t)(kW1 - 1) * a.D, xin);
}

template <typename T, int VEC, int W, bool REST>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvArgs a, const T *x,
                                                        const T *__restrict__ weight,
                                                        const T *__restrict__ bias,
                                                        T *__restrict__ state, T *y) {
  const int64_t wave = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (wave >= a.waves)
    return;
  const int row = (int)(wave / a.cw);
  const int64_t l = (wave - (int64_t)row * a.cw) * 64 + (threadIdx.x & 63);
  const int64_t slot = a.slots ? a.slots[row] : row;
  if (slot < 0 || slot >= a.num_slots)
    return; // a padding row: nothing is read or written
  by_channels<VEC, REST>(a, l, [&](auto vec, int64_t d) {
    conv_token<T, decltype(vec)::value, W>(a, x + row * a.xs, weight, bias,
                                           state + slot * (W - 1) * a.D, y + row * a.ys, d);
  });
}

// ---- launches -------------------------------------------------------------------
namespace {

template <typename F> hipError_t with_width(int W, F &&f) {
  switch (W) {
  case 2: return f(std::integral_constant<int, 2>());
  case 3: return f(std::integral_constant<int, 3>());
  case 4: return f(std::integral_constant<int, 4>());
  case 5: return f(std::integral_constant<int, 5>());
  case 6: return f(std::integral_constant<int, 6>());
  case 7: return f(std::integral_constant<int, 7>());
  case 8: return f(std::integral_constant<int, 8>());
  default: return hipErrorInvalidValue;
  }
}

template <typename F> hipError_t with_type(int elt, bool rest, F &&f) {
  using std::integral_constant;
  if (elt == 1)
    return rest ? f(bf16(), integral_constant<int, 8>(), std::true_type())
                : f(bf16(), integral_constant<int, 8>(), std::false_type());
  return rest ? f(float(), integral_constant<int, 4>(), std::true_type())
              : f(float(), integral_constant<int, 4>(), std::false_type());
}

ConvArgs conv_args(const ConvCall &c, int vec) {
  ConvArgs a{};
  a.D = c.D;
  a.full = c.D / vec;
  a.cw = (a.full + c.D % vec + 63) / 64;
  a.act = c.act;
  a.num_slots = c.num_slots;
  a.xs = c.x_stride;
  a.ys = c.y_stride;
  a.slots = c.slots;
  return a;
}

} // namespace

hipError_t launch_conv(int elt, const ConvCall &c, int32_t num_seqs, const int64_t *cu, void *ws,
                       hipStream_t s) {
  const int vec = elt == 1 ? 8 : 4;
  ConvArgs a = conv_args(c, vec);
  const auto tiles = [](int64_t len, int w) -> int64_t {
    return w ? 0 : (len > kConvTile ? (len + kConvTile - 1) / kConvTile : 1);
  };
  int64_t total[kCounts];
  if (!seq_totals(num_seqs, cu, tiles, total))
    return hipErrorInvalidConfiguration;
  a.waves = total[0] * a.cw;
  if ((a.waves + 3) / 4 * 256 > UINT32_MAX)
    return hipErrorInvalidConfiguration;
  SeqTable tab;
  const hipError_t e = make_seq_table(tab, num_seqs, cu, tiles, ws, s);
  if (e != hipSuccess)
    return e;
  return with_type(elt, c.D % vec != 0, [&](auto tag, auto v, auto rest) {
    return with_width(c.W, [&](auto w) {
      using T = decltype(tag);
      conv_kernel<T, decltype(v)::value, decltype(w)::value, decltype(rest)::value>
          <<<(unsigned)((a.waves + 3) / 4), 256, 0, s>>>(
              tab, a, (const T *)c.x, (const T *)c.weight, (const T *)c.bias, (const T *)c.init,
              (T *)c.fin, (T *)c.y);
      return hipGetLastError();
    });
  });
}

hipError_t launch_conv_step(int elt, const ConvCall &c, int32_t rows, hipStream_t s) {
  const int vec = elt == 1 ? 8 : 4;
  ConvArgs a = conv_args(c, vec);
  a.waves = (int64_t)rows * a.cw;
  if ((a.waves + 3) / 4 * 256 > UINT32_MAX)
    return hipErrorInvalidConfiguration;
  return with_type(elt, c.D % vec != 0, [&](auto tag, auto v, auto rest) {
    return with_width(c.W, [&](auto w) {
      using T = decltype(tag);
      conv_step_kernel<T, decltype(v)::value, decltype(w)::value, decltype(rest)::value>
          <<<(unsigned)((a.waves + 3) / 4), 256, 0, s>>>(a, (const T *)c.x, (const T *)c.weight,
                                                         (const T *)c.bias, (T *)c.fin,
                                                         (T *)c.y);
      return hipGetLastError();
    });
  });
}

} // namespace kda
