// Selective state space scan: a diagonal linear recurrence with N states per
// channel whose decay, input and read-out all come from the token.
//
//   delta = softplus(dt + bias)          (or dt itself)
//   h[d, n] <- exp(delta A[d, n]) h[d, n] + delta x[d] B[n]
//   y[d]    = sum_n C[n] h[d, n] + Dskip[d] x[d],   then y *= silu(z)
//
// Bound.  Per (token, channel) four elements move, but each of the N states
// takes two products, an exponential and two more products and sums: 24
// cycles of a SIMD for 64 of them (the exponential 8, the others 4 each; no
// fp32 pairs are used).  With N = 16 the vector ALU is the limit, not HBM:
// 8192 tokens x 8192 channels are 164 us of those instructions alone,
// against 88 us of traffic.  All arithmetic is fp32; y is the only rounding
// to fewer bits.
//
// The recurrence is serial in the tokens, so what fills the chip are channels
// and states, and when those do not suffice, pieces of the sequence.  Two
// kernels, chosen by ssm_plan from the times of both:
//   row kernel   a channel's states across 16 lanes: 16 times the waves of
//                the other, for one reduction across lanes a token (some 43
//                cycles a state and token in all);
//   lane kernel  all states of a channel in one lane (some 34 cycles), where
//                there are sequences and channels enough.
// Either runs long sequences of few channels cut into segments.
// The cut: the decay over a segment is exp(A sum(delta)), so a segment's
// effect on the state that enters it is known from its end state from zero
// and its sum of delta.  The first launch runs every first segment (from the
// true initial state) beside the end states of the middle ones (some 25
// cycles: no read-out), a second folds those pairs into entry states, the
// third runs all segments but the first.  The middle segments' exponentials
// are evaluated twice, which is what the cut costs: 131072 tokens x 1536
// channels take 1.32 ms (65 cycles a state and token), 4.5 ms uncut.
#include "kda_device.h"
#include "kda_recurrent.h"
#include "kda_seqtab.h"

#include <algorithm>
#include <type_traits>

namespace kda {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// log(1 + exp(x)) = max(x, 0) + log1p(e), e = exp(-|x|) in (0, 1], with
// log1p(e) = 2 atanh(s), s = e / (2 + e) <= 1/3, and atanh(s) / s a polynomial
// in s^2 (degree 4, fitted for the smallest relative error over [0, 1/9]:
// 8e-9).  (The logarithm of 1 + e itself would lose the small steps: at
// delta = 0.001 its argument keeps 13 of e's 23 bits.)
__device__ __forceinline__ float softplus(float x) {
  const float e = exp2_hw(-fabsf(x) * kLog2e);
  const float s = e * __builtin_amdgcn_rcpf(2.f + e);
  const float q = s * s;
  float p = 0.14089167f;
  p = fmaf(p, q, 0.139803007f);
  p = fmaf(p, q, 0.200124547f);
  p = fmaf(p, q, 0.333331585f);
  p = fmaf(p, q, 1.f);
  return fmaf(s + s, p, fmaxf(x, 0.f));
}

// A in log2 units.  An infinite A is taken as the largest finite one, by
// prompts and single tokens alike: its decay is the same, and a step of 0
// (which the prompt kernels take past a segment's end) leaves the state as it
// is instead of making 0 * inf.
__device__ __forceinline__ float finite_rate(float r) {
  return fabsf(r) == __builtin_inff() ? copysignf(3.4028235e38f, r) : r;
}
__device__ __forceinline__ float log2_rate(float a) { return finite_rate(a * kLog2e); }

// A sum of finite steps as a finite number: its decay is the same, and a rate
// of 0 keeps its state.  (A step that is not finite itself shows in the state
// that the sum goes with.)
__device__ __forceinline__ float finite_sum(float x) {
  return fmaxf(fminf(x, 3.4028235e38f), -3.4028235e38f);
}

// x, or 0 without a thought of what x is (mask: all ones or 0).
__device__ __forceinline__ float masked(float x, int mask) {
  return __builtin_bit_cast(float, __builtin_bit_cast(int, x) & mask);
}

// Infinity or NaN in any lane.
__device__ __forceinline__ bool any_nonfinite(float x) {
  return __builtin_amdgcn_ballot_w64(__builtin_amdgcn_classf(x, 0x207)) != 0;
}

struct SsmArgs {
  int32_t D, N, G, softplus, num_slots;
  int32_t Dg;      // channels per group
  int32_t cb;      // 64-channel blocks per group
  int32_t seg;     // tokens per segment
  int64_t xs, dls, zs, ys, Bs, Cs;
  const float *A, *skip, *bias;
  const float *init;
  float *fin;
  const int32_t *slots;
  float *pend;         // [pairs][G cb][SN][64] end states of the segments
  float *psum;         // [pairs][G cb][64] their sums of delta
};

// ---- raw elements --------------------------------------------------------------------
// The loaded bits (of P = 1 or 2 neighbouring elements) are kept as they are
// and widened where they are used, so that nothing waits for a load before
// then.
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
template <typename T, int P> struct RawOf;
template <> struct RawOf<bf16, 1> { typedef unsigned short type; };
template <> struct RawOf<bf16, 2> { typedef unsigned type; };
template <> struct RawOf<float, 1> { typedef unsigned type; };
template <> struct RawOf<float, 2> { typedef u32x2 type; };
template <typename T, int P = 1> using Raw = typename RawOf<T, P>::type;

template <typename T, int P> __device__ __forceinline__ float widen(Raw<T, P> r, int j) {
  unsigned u;
  if constexpr (sizeof(T) == 2)
    u = P == 1 || j == 0 ? (unsigned)r << 16 : (unsigned)r & 0xffff0000u;
  else if constexpr (P == 1)
    u = r;
  else
    u = j == 0 ? r.x : r.y;
  return __builtin_bit_cast(float, u);
}
// The elements at byte voff + soff (soff wave-uniform).  voff -1 reads 0 and
// writes nothing.
template <typename T, int P>
__device__ __forceinline__ Raw<T, P> buffer_raw(__amdgpu_buffer_rsrc_t r, int voff, int soff) {
  if constexpr (sizeof(T) * P == 2)
    return __builtin_amdgcn_raw_buffer_load_b16(r, voff, soff, 0);
  else if constexpr (sizeof(T) * P == 4)
    return __builtin_amdgcn_raw_buffer_load_b32(r, voff, soff, 0);
  else
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, voff, soff, 0));
}
template <typename T, int P>
__device__ __forceinline__ void buffer_put(__amdgpu_buffer_rsrc_t r, const float (&v)[P], int voff,
                                           int soff) {
  if constexpr (P == 1) {
    buffer_store(r, from_f32<T>(v[0]), voff, soff);
  } else if constexpr (sizeof(T) == 2) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 w = {static_cast<bf16>(v[0]), static_cast<bf16>(v[1])};
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, w), r, voff, soff, 0);
  } else {
    const f32x2_t w = {v[0], v[1]};
    __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, w), r, voff, soff, 0);
  }
}

// ---- a channel's states across a row of 16 lanes -------------------------------------
// Lane (c, i) of a wave, c = lane / 16, i = lane % 16, holds states i, 16 + i,
// ... (E of them) of channel c, and for every 16 tokens computes delta and
// delta x of token i of that channel; a token's pair reaches the other lanes
// of the row as the DPP row broadcast of the two products it enters, at no
// cost.  The read-out leaves 16 partial products a lane, one for each token,
// and row_reduce16 adds them across the row so that token i's sum ends in
// lane i: 33 instructions for 16 tokens instead of 64.
//
// A workgroup's four waves stage tiles of TT tokens for their 16 channels
// through LDS, because a wave's own loads would be 16 rows of 8 bytes (620 us
// instead of 415 at 8192 x 8192 bf16): the threads go down the channels of a
// row, evaluate softplus and gate there, and take the read-outs back the same
// way for skip, gate and store.  391 us at that size, with two waves a SIMD:
// 9.5 instructions a state and token, the vector ALU busy 75% of the time.
// Tiles of 32 and 128 tokens: 417 and 406 us; eight waves (32 channels): 388;
// one barrier a tile with both buffers doubled: 430.
// Where N fills no 16 E, a tile with an infinite delta x goes through a copy
// of the loop that keeps the states that are not there 0 (PAD; the test and
// the copy cost 2% at N = 20 and 13).

// Token I's value of every row, in all of the row's lanes.
template <int I> __device__ __forceinline__ float row_bcast(float x) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x150 + I, 0xf, 0xf, true));
}

template <int CTRL> __device__ __forceinline__ float quad_swap(float x) {
  return __builtin_bit_cast(
      float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), CTRL, 0xf, 0xf, true));
}

// Sum of p[i] over the 16 lanes of each row, in the row's lane i.  Each step
// halves both the tokens and the lanes still to be added: lanes whose bit is
// 0 go on with the lower token of a pair, the others with the upper one, each
// adding its partner's share.  The first two steps write their two halves by
// DPP bank masks (4 lanes a bank).  (s_nop 1: a DPP operand must be two
// instructions old, which the compiler does not see inside or around asm.
// "+&v": the sums are written before the last operand is read.)
__device__ __forceinline__ float row_reduce16(float (&p)[16], int lane) {
  asm volatile(
      "s_nop 1\n\t"
      "v_add_f32_dpp %0, %0, %0 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
      "v_add_f32_dpp %1, %1, %1 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
      "v_add_f32_dpp %2, %2, %2 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
      "v_add_f32_dpp %3, %3, %3 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
      "v_add_f32_dpp %4, %4, %4 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
      "v_add_f32_dpp %5, %5, %5 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
      "v_add_f32_dpp %6, %6, %6 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
      "v_add_f32_dpp %7, %7, %7 row_ror:8 row_mask:0xf bank_mask:0x3\n\t"
      "v_add_f32_dpp %0, %8, %8 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %1, %9, %9 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %2, %10, %10 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %3, %11, %11 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %4, %12, %12 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %5, %13, %13 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %6, %14, %14 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "v_add_f32_dpp %7, %15, %15 row_ror:8 row_mask:0xf bank_mask:0xc\n\t"
      "s_nop 1\n\t"
      "v_add_f32_dpp %0, %0, %0 row_shl:4 row_mask:0xf bank_mask:0x5\n\t"
      "v_add_f32_dpp %1, %1, %1 row_shl:4 row_mask:0xf bank_mask:0x5\n\t"
      "v_add_f32_dpp %2, %2, %2 row_shl:4 row_mask:0xf bank_mask:0x5\n\t"
      "v_add_f32_dpp %3, %3, %3 row_shl:4 row_mask:0xf bank_mask:0x5\n\t"
      "v_add_f32_dpp %0, %4, %4 row_shr:4 row_mask:0xf bank_mask:0xa\n\t"
      "v_add_f32_dpp %1, %5, %5 row_shr:4 row_mask:0xf bank_mask:0xa\n\t"
      "v_add_f32_dpp %2, %6, %6 row_shr:4 row_mask:0xf bank_mask:0xa\n\t"
      "v_add_f32_dpp %3, %7, %7 row_shr:4 row_mask:0xf bank_mask:0xa\n\t"
      "s_nop 1"
      : "+&v"(p[0]), "+&v"(p[1]), "+&v"(p[2]), "+&v"(p[3]), "+&v"(p[4]), "+&v"(p[5]), "+&v"(p[6]),
        "+&v"(p[7])
      : "v"(p[8]), "v"(p[9]), "v"(p[10]), "v"(p[11]), "v"(p[12]), "v"(p[13]), "v"(p[14]),
        "v"(p[15]));
  const bool b1 = lane & 2, b0 = lane & 1;
  float r[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const float keep = b1 ? p[j + 2] : p[j], give = b1 ? p[j] : p[j + 2];
    r[j] = keep + quad_swap<0x4e>(give); // quad_perm [2, 3, 0, 1]
  }
  const float keep = b0 ? r[1] : r[0], give = b0 ? r[0] : r[1];
  return keep + quad_swap<0xb1>(give); // quad_perm [1, 0, 3, 2]
}

// One token of the recurrence in all rows: I-th of its 16, k-th of its 4.
// The lane's states from `states` on are not there: rate, B and C are 0 and so
// is the state, without a thought until delta x is infinite or NaN; MASK then
// keeps them 0.
template <int I, int E, bool FULL, bool MASK>
__device__ __forceinline__ void row_token(float delta, float u, int states, const float (&A2)[E],
                                          float (&h)[E], const f32x4 (&b)[E], const f32x4 (&c)[E],
                                          float &p) {
  const float d = row_bcast<I>(delta), ui = row_bcast<I>(u);
#pragma unroll
  for (int e = 0; e < E; ++e) {
    h[e] = fmaf(exp2_hw(d * A2[e]), h[e], ui * b[e][I & 3]);
    if (MASK)
      h[e] = 16 * e < states ? h[e] : 0.f;
    if (FULL)
      p = e == 0 ? c[e][I & 3] * h[e] : fmaf(c[e][I & 3], h[e], p);
  }
}

constexpr int row_tile(int E) { return E >= 4 ? 16 : 64 / E; }

// Four waves a workgroup: 16 channels; workgroups of one 64-channel stretch.
constexpr int kRowChans = 16, kRowNear = 64 / kRowChans;

// TT tokens of a workgroup's channels.  (Row pads: the staging threads
// go down the channels, 64 / CH tokens side by side.)
template <int E> struct __align__(16) RowLds {
  static constexpr int TT = row_tile(E), CH = kRowChans;
  float bc[2][16 * E][TT + 4];       // B, C by state
  float2 du[CH][TT + 32 / CH];       // (delta, delta x)
  float y[CH][TT + 64 / CH];         // read-outs
  alignas(16) int odd[4];                  // a wave staged a delta x that is not finite
};

// Values a thread stages from a matrix: rows r0, r0 + kStep, ... of a tile, P
// neighbouring columns.  Rows past the segment and columns past the matrix
// read 0.
template <typename T, int P, int kN, int kStep> struct Stage {
  const T *p;     // the tile's first row
  int64_t stride; // elements
  int voff;       // this thread's byte offset in the tile, -1: no column
  int r0;
  Raw<T, P> r[kN];

  __device__ __forceinline__ Stage(const T *p_, int64_t s, int row, int col, bool on)
      : p(p_), stride(s), voff(on ? (row * (int)s + col) * (int)sizeof(T) : -1), r0(row) {}
  // rows: how many of the tile's lie in the segment
  __device__ __forceinline__ void fetch(int rows) {
    const __amdgpu_buffer_rsrc_t rs = buffer_rsrc(p, rows > 0 ? 0x7fffffff : 0);
    const int step = kStep * (int)stride * (int)sizeof(T);
    if (rows >= kN * kStep) {
#pragma unroll
      for (int k = 0; k < kN; ++k)
        r[k] = buffer_raw<T, P>(rs, voff, k * step);
    } else {
#pragma unroll
      for (int k = 0; k < kN; ++k)
        r[k] = buffer_raw<T, P>(rs, r0 + k * kStep < rows ? voff : -1, k * step);
    }
  }
  __device__ __forceinline__ float at(int k, int j) const { return widen<T, P>(r[k], j); }
  __device__ __forceinline__ void next(int rows) { p += rows * stride; }
};

template <typename T, int E, int P, bool PAD, bool FULL>
__device__ __forceinline__ float row_segment(const SsmArgs &a, RowLds<E> &lds, float (&h)[E],
                                             const float (&A2)[E], const T *x, const T *dl,
                                             const T *z, const T *B, const T *C, T *y, int ntok,
                                             int chans, const float (&bias)[P],
                                             const float (&skip)[P]) {
  constexpr int TT = row_tile(E), CH = kRowChans, NP = 16 * E;
  constexpr int kStep = 256 * P / CH;       // rows the threads stage at a time
  constexpr int kRows = TT / kStep;         // elements (or pairs) of a thread
  constexpr int kBcStep = 256 * P / NP;     // likewise for B and C
  constexpr int kBc = TT / kBcStep;
  static_assert(kRows >= 1 && kBc >= 1, "the threads cover at most a tile");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int sc = tid % (CH / P) * P, sr = tid / (CH / P); // channel and first row it stages
  const int sn = tid % (NP / P) * P, st = tid / (NP / P); // state and first token of B and C
  const int rc = wave * 4 + (lane >> 4), ri = lane & 15;
  const int states = a.N - ri, has_skip = a.skip ? -1 : 0;
  const bool in = sc < chans;
  Stage<T, P, kRows, kStep> sx(x, a.xs, sr, sc, in), sd(dl, a.dls, sr, sc, in),
      sz(z, a.zs, sr, sc, in);
  Stage<T, P, kBc, kBcStep> sb(B, a.Bs, st, sn, sn < a.N), scc(C, a.Cs, st, sn, sn < a.N);
  const int yoff = in ? (sr * (int)a.ys + sc) * (int)sizeof(T) : -1;
  const int ystep = kStep * (int)a.ys * (int)sizeof(T);
  float xk[kRows][P];
  float sum = 0.f;

  const auto fetch = [&](int rows) {
    sx.fetch(rows);
    sd.fetch(rows);
    sb.fetch(rows);
    if (FULL) {
      scc.fetch(rows);
      if (z)
        sz.fetch(rows);
    }
    sx.next(TT);
    sd.next(TT);
    sz.next(TT);
    sb.next(TT);
    scc.next(TT);
  };

  fetch(ntok);
  for (int t0 = 0; t0 < ntok; t0 += TT) {
    const int n = min(TT, ntok - t0);
    float d[kRows][P], gate[kRows][P];
#pragma unroll
    for (int k = 0; k < kRows; ++k)
#pragma unroll
      for (int j = 0; j < P; ++j) {
        xk[k][j] = sx.at(k, j);
        d[k][j] = sd.at(k, j) + bias[j];
        gate[k][j] = 1.f;
      }
    if (a.softplus) {
#pragma unroll
      for (int k = 0; k < kRows; ++k)
#pragma unroll
        for (int j = 0; j < P; ++j)
          d[k][j] = softplus(d[k][j]);
    }
    if (FULL && z) {
#pragma unroll
      for (int k = 0; k < kRows; ++k)
#pragma unroll
        for (int j = 0; j < P; ++j)
          gate[k][j] = silu(sz.at(k, j));
    }
    // past the segment's end a step of 0 (with x and B 0) leaves h as it is
    if (n < TT) {
#pragma unroll
      for (int k = 0; k < kRows; ++k)
#pragma unroll
        for (int j = 0; j < P; ++j)
          d[k][j] = sr + kStep * k < n ? d[k][j] : 0.f;
    }
    float worst = 0.f; // not finite where one of its products is not
#pragma unroll
    for (int k = 0; k < kRows; ++k)
#pragma unroll
      for (int j = 0; j < P; ++j) {
        const float u = d[k][j] * xk[k][j];
        lds.du[sc + j][sr + kStep * k] = float2{d[k][j], u};
        worst = fmaf(0.f, u, worst);
      }
    if (PAD) {
      const int odd = any_nonfinite(worst);
      if (lane == 0)
        lds.odd[wave] = odd;
    }
#pragma unroll
    for (int k = 0; k < kBc; ++k)
#pragma unroll
      for (int j = 0; j < P; ++j) {
        lds.bc[0][sn + j][st + k * kBcStep] = sb.at(k, j);
        if (FULL)
          lds.bc[1][sn + j][st + k * kBcStep] = scc.at(k, j);
      }
    __syncthreads();
    fetch(ntok - t0 - TT); // in flight during the recurrence

    // (a step that is not finite makes delta x not finite)
    bool odd = false;
    if (PAD) {
      const int4 o = *reinterpret_cast<const int4 *>(lds.odd);
      odd = __builtin_amdgcn_readfirstlane(o.x | o.y | o.z | o.w) != 0;
    }
    const auto tokens16 = [&](int s0, auto mask) {
      const float2 du = lds.du[rc][s0 + ri];
      float p[16];
      const auto quad = [&](auto q) {
        constexpr int Q = decltype(q)::value;
        constexpr bool M = decltype(mask)::value;
        f32x4 b[E], c[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
          b[e] = *reinterpret_cast<const f32x4 *>(&lds.bc[0][16 * e + ri][s0 + 4 * Q]);
          if (FULL)
            c[e] = *reinterpret_cast<const f32x4 *>(&lds.bc[1][16 * e + ri][s0 + 4 * Q]);
        }
        row_token<4 * Q, E, FULL, M>(du.x, du.y, states, A2, h, b, c, p[4 * Q]);
        row_token<4 * Q + 1, E, FULL, M>(du.x, du.y, states, A2, h, b, c, p[4 * Q + 1]);
        row_token<4 * Q + 2, E, FULL, M>(du.x, du.y, states, A2, h, b, c, p[4 * Q + 2]);
        row_token<4 * Q + 3, E, FULL, M>(du.x, du.y, states, A2, h, b, c, p[4 * Q + 3]);
      };
      quad(std::integral_constant<int, 0>());
      quad(std::integral_constant<int, 1>());
      quad(std::integral_constant<int, 2>());
      quad(std::integral_constant<int, 3>());
      if (FULL)
        lds.y[rc][s0 + ri] = row_reduce16(p, lane);
      else
        sum += du.x; // (lane i: the tokens i of every 16)
    };
    if (PAD && odd)
      for (int s0 = 0; s0 < n; s0 += 16)
        tokens16(s0, std::true_type());
    else
      for (int s0 = 0; s0 < n; s0 += 16)
        tokens16(s0, std::false_type());
    __syncthreads();

    if (FULL) {
      const __amdgpu_buffer_rsrc_t ry = buffer_rsrc(y, 0x7fffffff);
#pragma unroll
      for (int k = 0; k < kRows; ++k) {
        const int row = sr + kStep * k;
        float v[P];
#pragma unroll
        for (int j = 0; j < P; ++j) {
          v[j] = lds.y[sc + j][row];
          v[j] = fmaf(skip[j], masked(xk[k][j], has_skip), v[j]);
          if (z)
            v[j] *= gate[k][j];
        }
        buffer_put<T, P>(ry, v, row < n ? yoff : -1, k * ystep);
      }
      y += TT * a.ys;
    }
  }
  return sum;
}

// PAD: fewer than 16 E states.
template <typename T, int E, int P, bool PAD>
__global__ __launch_bounds__(256) void ssm_row_kernel(SeqTable tab, SsmArgs a, int pass,
                                                          int64_t grid,
                                                          const T *__restrict__ x,
                                                          const T *__restrict__ dl,
                                                          const T *__restrict__ z,
                                                          const T *__restrict__ B,
                                                          const T *__restrict__ C,
                                                          T *__restrict__ y) {
  __shared__ RowLds<E> lds;
  constexpr int CH = kRowChans;
  // Workgroups go round the eight dies; those of one 64-channel stretch, which
  // share its cache lines, are put on one die.
  constexpr int kNear = kRowNear;
  const int64_t bid =
      ((int64_t)(blockIdx.x / (8 * kNear)) * 8 + blockIdx.x % 8) * kNear + blockIdx.x / 8 % kNear;
  if (bid >= grid)
    return;
  const int rb = (a.Dg + CH - 1) / CH, blocks = a.G * rb;
  const int sb = (int)(bid / blocks), gr = (int)(bid - (int64_t)sb * blocks);
  const int g = gr / rb, c0 = (gr - g * rb) * CH; // first channel in its group
  const SeqView seqs(tab);
  const int n = seqs.find(sb, pass);
  const int len = seqs.len(n);
  const int64_t tok0 = seqs.tok0(n);
  const int nseg = len > a.seg ? (len + a.seg - 1) / a.seg : 1;
  const int j = sb - seqs.blk(n, pass) + pass;
  const int64_t pair0 = seqs.blk(n, 1);
  const int s0 = j * a.seg, ntok = min(a.seg, len - s0);

  const int tid = threadIdx.x, lane = tid & 63;
  const int ri = lane & 15;
  const int dg = c0 + (tid >> 6) * 4 + (lane >> 4); // the channel whose states it holds
  const bool in = dg < a.Dg;
  const int64_t d = (int64_t)g * a.Dg + dg;
  float A2[E], h[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    A2[e] = in && 16 * e + ri < a.N ? log2_rate(a.A[d * a.N + 16 * e + ri]) : 0.f;
    h[e] = 0.f;
  }
  int64_t slot = seqs.seq(n);
  bool kept = true;
  if (a.slots) {
    slot = a.slots[slot];
    kept = slot >= 0 && slot < a.num_slots;
  }
  // states in segment pairs: [pair][64-channel block][state][channel]
  const int64_t at = ((int64_t)(g * a.cb + dg / 64) * (16 * E) + ri) * 64 + dg % 64;
  const int64_t pstep = (int64_t)a.G * a.cb * (16 * E) * 64;
  if (j == 0) {
    if (a.init && kept && in) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (16 * e + ri < a.N)
          h[e] = a.init[(slot * a.D + d) * a.N + 16 * e + ri];
    }
  } else if (pass == 1 && in) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      h[e] = a.pend[(pair0 + j - 1) * pstep + at + e * 16 * 64];
  }

  const int64_t t0 = tok0 + s0, d0 = (int64_t)g * a.Dg + c0;
  const int chans = min(CH, a.Dg - c0);
  const int sc = tid % (CH / P) * P; // the channels it stages
  float bias[P], skip[P];
#pragma unroll
  for (int q = 0; q < P; ++q) {
    bias[q] = a.bias && sc + q < chans ? a.bias[d0 + sc + q] : 0.f;
    skip[q] = a.skip && sc + q < chans ? a.skip[d0 + sc + q] : 0.f;
  }
  x += t0 * a.xs + d0;
  dl += t0 * a.dls + d0;
  B += t0 * a.Bs + g * a.N;
  C += t0 * a.Cs + g * a.N;
  float sum = 0.f;
  if (pass == 1 || j == 0)
    row_segment<T, E, P, PAD, true>(a, lds, h, A2, x, dl, z ? z + t0 * a.zs + d0 : nullptr, B, C,
                                y + t0 * a.ys + d0, ntok, chans, bias, skip);
  else
    sum = row_segment<T, E, P, PAD, false>(a, lds, h, A2, x, dl, nullptr, B, C, nullptr, ntok, chans,
                                       bias, skip);

  if (j == nseg - 1) {
    if (a.fin && kept && in) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (16 * e + ri < a.N)
          a.fin[(slot * a.D + d) * a.N + 16 * e + ri] = h[e];
    }
  } else if (pass == 0) {
    sum = row_scan16(sum); // lane 15: the whole segment's
    if (in) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        a.pend[(pair0 + j) * pstep + at + e * 16 * 64] = h[e];
      if (j > 0 && ri == 15)
        a.psum[((pair0 + j) * a.G * a.cb + g * a.cb + dg / 64) * 64 + dg % 64] = finite_sum(sum);
    }
  }
}

// ---- all states of a channel in one lane --------------------------------------------
// No exchange between waves and no barrier: a wave streams its 64 channels'
// tokens, U at a time with the next U tokens' inputs in flight.  B and C come
// through an LDS area of the wave's own: kBcTokens tokens' values, widened,
// loaded a whole area ahead; every lane then reads the same 16 bytes.  (As
// scalar operands from a table of scalar loads they saved the LDS reads, but
// a wave then stood still for every miss: 567 us against 467 at 8192 x 8192,
// 138 against 67 us at 256 x 1536.)  131072 x 1536 bf16, cut into 171
// segments: 1.32 ms, 65 cycles a state and token where the instructions of
// both passes come to 59.
// There is a kernel for every N up to 16: a state too many would cost its
// instructions (8192 tokens of 64 sequences x 1536 with N = 5: 84 us, 96 with
// 8 states), and would have to be kept from making 0 * inf of an infinite
// input.
constexpr int kBcTokens = 16;

// Places for the N values of B or C of a token: 4, 8 or 16.
constexpr int lane_places(int N) { return N <= 4 ? 4 : (N <= 8 ? 8 : 16); }

template <int NP> struct __align__(16) LaneBc {
  float v[2][kBcTokens][2 * NP]; // B then C of each token, two areas in turn
};

// One element per lane of a row of channels; lanes at or past `bytes` (the
// row's end, or 0 for a token past the segment) read 0 and write nothing.
template <typename T>
__device__ __forceinline__ Raw<T> row_load(const T *p, int bytes, int lane) {
  return buffer_raw<T, 1>(buffer_rsrc(p, bytes), lane * (int)sizeof(T), 0);
}
template <typename T>
__device__ __forceinline__ void row_store(T *p, int bytes, int lane, float v) {
  buffer_store(buffer_rsrc(p, bytes), from_f32<T>(v), lane * (int)sizeof(T), 0);
}

// The values of B and C a lane brings in per area: state i of every kStep-th
// token.  Tokens past the segment and states past N read 0.
template <typename T, int NP> struct BcLoader {
  static constexpr int kStep = 64 / NP;
  static constexpr int kPer = kBcTokens / kStep;
  const T *B, *C;
  int64_t Bs, Cs;
  int t0, i;
  bool on;
  Raw<T> b[kPer], c[kPer];

  __device__ __forceinline__ BcLoader(const T *B_, const T *C_, int64_t Bs_, int64_t Cs_, int N,
                                      int lane)
      : B(B_), C(C_), Bs(Bs_), Cs(Cs_) {
    t0 = lane / NP;
    i = lane % NP;
    on = i < N;
  }
  __device__ __forceinline__ void fetch(int tok, int ntok) {
    // (an area's rows lie within 2^31 bytes)
    constexpr int kSpan = 0x7fffffff;
    const __amdgpu_buffer_rsrc_t rb = buffer_rsrc(B + tok * Bs, kSpan);
    const __amdgpu_buffer_rsrc_t rc = buffer_rsrc(C + tok * Cs, kSpan);
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      const int t = t0 + k * kStep;
      const bool ok = on && tok + t < ntok;
      b[k] = buffer_raw<T, 1>(rb, ok ? (t * (int)Bs + i) * (int)sizeof(T) : -1, 0);
      c[k] = buffer_raw<T, 1>(rc, ok ? (t * (int)Cs + i) * (int)sizeof(T) : -1, 0);
    }
  }
  __device__ __forceinline__ void put(float (*area)[2 * NP]) const {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      area[t0 + k * kStep][i] = widen<T, 1>(b[k], 0);
      area[t0 + k * kStep][NP + i] = widen<T, 1>(c[k], 0);
    }
  }
};

template <typename T, int NS, bool FULL>
__device__ __forceinline__ float lane_segment(const SsmArgs &a, LaneBc<lane_places(NS)> &lds,
                                              float (&h)[NS], const float (&A2)[NS],
                                              BcLoader<T, lane_places(NS)> bc,
                                              const T *x, const T *dl, const T *z, T *y, int ntok,
                                              int row_bytes, int lane, float bias, float skip) {
  constexpr int U = 4, NP = lane_places(NS);
  Raw<T> xr[U], dr[U], zr[U];
  float sum = 0.f;
  const auto bytes = [&](int t) { return t < ntok ? row_bytes : 0; };
  const auto fetch = [&](int t0) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int64_t t = t0 + k;
      xr[k] = row_load(x + t * a.xs, bytes(t0 + k), lane);
      dr[k] = row_load(dl + t * a.dls, bytes(t0 + k), lane);
    }
    if (FULL && z) {
#pragma unroll
      for (int k = 0; k < U; ++k)
        zr[k] = row_load(z + (t0 + k) * a.zs, bytes(t0 + k), lane);
    }
  };
  bc.fetch(0, ntok);
  fetch(0);
  for (int b0 = 0; b0 < ntok; b0 += kBcTokens) {
    // this wave's reads of the area two before are done: its LDS
    // instructions run in order
    float(*area)[2 * NP] = lds.v[(b0 / kBcTokens) & 1];
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    bc.put(area);
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
    bc.fetch(b0 + kBcTokens, ntok);
    for (int t0 = b0; t0 < min(b0 + kBcTokens, ntok); t0 += U) {
      float xk[U], d[U], gate[U], acc[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        xk[k] = widen<T, 1>(xr[k], 0);
        d[k] = widen<T, 1>(dr[k], 0) + bias;
        gate[k] = 1.f;
      }
      if (a.softplus) {
#pragma unroll
        for (int k = 0; k < U; ++k)
          d[k] = softplus(d[k]);
      }
      if (FULL && z) {
#pragma unroll
        for (int k = 0; k < U; ++k)
          gate[k] = silu(widen<T, 1>(zr[k], 0));
      }
      // past the segment's end a step of 0 (with x and B 0) leaves h as it is
      if (ntok - t0 < U) {
#pragma unroll
        for (int k = 0; k < U; ++k)
          d[k] = t0 + k < ntok ? d[k] : 0.f;
      }
      fetch(t0 + U);
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const float *row = area[t0 - b0 + k];
        const float u = d[k] * xk[k];
        acc[k] = 0.f;
#pragma unroll
        for (int q = 0; q < NS; q += 4) {
          const f32x4 bv = *reinterpret_cast<const f32x4 *>(row + q);
          f32x4 cv;
          if (FULL)
            cv = *reinterpret_cast<const f32x4 *>(row + NP + q);
#pragma unroll
          for (int i = 0; i < 4 && q + i < NS; ++i) {
            h[q + i] = fmaf(exp2_hw(d[k] * A2[q + i]), h[q + i], u * bv[i]);
            if (FULL)
              acc[k] = fmaf(cv[i], h[q + i], acc[k]);
          }
        }
        if (!FULL)
          sum += d[k];
      }
      if (FULL) {
        if (a.skip) { // (without one, an infinite x adds no 0 * inf)
#pragma unroll
          for (int k = 0; k < U; ++k)
            acc[k] = fmaf(skip, xk[k], acc[k]);
        }
#pragma unroll
        for (int k = 0; k < U; ++k)
          row_store(y + (t0 + k) * a.ys, bytes(t0 + k), lane, z ? acc[k] * gate[k] : acc[k]);
      }
    }
  }
  return sum;
}

template <typename T, int NS>
__global__ __launch_bounds__(256, 4) void ssm_lane_kernel(SeqTable tab, SsmArgs a, int pass,
                                                       const T *__restrict__ x,
                                                       const T *__restrict__ dl,
                                                       const T *__restrict__ z,
                                                       const T *__restrict__ B,
                                                       const T *__restrict__ C,
                                                       T *__restrict__ y) {
  __shared__ LaneBc<lane_places(NS)> lds[4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int blocks = a.G * a.cb, quads = (blocks + 3) / 4;
  const int sb = blockIdx.x / quads, gc = (blockIdx.x - sb * quads) * 4 + wave;
  if (gc >= blocks)
    return;
  const int g = gc / a.cb, cbi = gc - g * a.cb;
  const SeqView seqs(tab);
  const int n = seqs.find(sb, pass);
  const int len = seqs.len(n);
  const int64_t tok0 = seqs.tok0(n);
  const int nseg = len > a.seg ? (len + a.seg - 1) / a.seg : 1;
  const int j = sb - seqs.blk(n, pass) + pass;
  const int64_t pair0 = seqs.blk(n, 1);
  const int s0 = j * a.seg, ntok = min(a.seg, len - s0);

  const int dg = cbi * 64 + lane;
  const bool in = dg < a.Dg;
  const int64_t d = (int64_t)g * a.Dg + dg;
  float A2[NS], h[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    A2[i] = in ? log2_rate(a.A[d * NS + i]) : 0.f;
    h[i] = 0.f;
  }
  int64_t slot = seqs.seq(n);
  bool kept = true;
  if (a.slots) {
    slot = a.slots[slot];
    kept = slot >= 0 && slot < a.num_slots;
  }
  if (j == 0) {
    if (a.init && kept && in) {
      const float *p = a.init + (slot * a.D + d) * NS;
#pragma unroll
      for (int i = 0; i < NS; ++i)
        h[i] = p[i];
    }
  } else if (pass == 1) {
    const float *pe = a.pend + ((pair0 + j - 1) * blocks + gc) * NS * 64 + lane;
#pragma unroll
    for (int i = 0; i < NS; ++i)
      h[i] = pe[i * 64];
  }

  const int64_t t0 = tok0 + s0;
  const BcLoader<T, lane_places(NS)> bc(B + t0 * a.Bs + g * NS, C + t0 * a.Cs + g * NS, a.Bs,
                                        a.Cs, NS, lane);
  const float bias = in && a.bias ? a.bias[d] : 0.f;
  const float skip = in && a.skip ? a.skip[d] : 0.f;
  const int64_t d0 = (int64_t)g * a.Dg + cbi * 64; // the wave's first channel
  const int row_bytes = min(64, a.Dg - cbi * 64) * (int)sizeof(T);
  float sum = 0.f;
  if (pass == 1 || j == 0)
    lane_segment<T, NS, true>(a, lds[wave], h, A2, bc, x + t0 * a.xs + d0, dl + t0 * a.dls + d0,
                              z ? z + t0 * a.zs + d0 : nullptr, y + t0 * a.ys + d0, ntok,
                              row_bytes, lane, bias, skip);
  else
    sum = lane_segment<T, NS, false>(a, lds[wave], h, A2, bc, x + t0 * a.xs + d0,
                                     dl + t0 * a.dls + d0, nullptr, nullptr, ntok, row_bytes,
                                     lane, bias, skip);

  if (j == nseg - 1) {
    if (a.fin && kept && in) {
      float *p = a.fin + (slot * a.D + d) * NS;
#pragma unroll
      for (int i = 0; i < NS; ++i)
        p[i] = h[i];
    }
  } else if (pass == 0) {
    float *pe = a.pend + ((pair0 + j) * blocks + gc) * NS * 64 + lane;
#pragma unroll
    for (int i = 0; i < NS; ++i)
      pe[i * 64] = h[i];
    if (j > 0)
      a.psum[((pair0 + j) * blocks + gc) * 64 + lane] = finite_sum(sum);
  }
}

// ---- the segments' entry states -------------------------------------------------------
// pend[0] is the state after the first segment; pend[j] becomes
// pend[j] + exp(A sum_j) pend[j - 1], the state after segment j.  A workgroup
// folds one state of 64 channels: its waves take a run of the pairs each,
// first from zero; the runs' ends and sums of delta (again a pair each) give
// every run its entry state, from which it is folded once more and written.
// (One wave over all pairs took 45 us for 490 of them, the loads of 16 in
// flight at a time.)
constexpr int kFoldWaves = 8;

// The state after a segment, from the one before it, its sum of steps and its
// end state from zero.  The decay 2^e, e = sum A2, is the product of the
// steps' decays and may lie outside fp32 where the state does not: with A > 0
// or negative steps a state of 0 or 1e-30 may grow by e^100, and an infinite
// one outlasts a decay of e^-100.  So only 2^(e - ceil(e)), in (1/2, 1], is
// multiplied, and the rest moves the state's exponent.  (512 passes the way
// from the largest fp32 number to the smallest.  Over an infinite step, and
// at an infinite rate, both of which stand here as the largest number, the
// decay is what that of a step would be: 0, or infinite, with the NaN that
// they make.)
__device__ __forceinline__ float fold_segment(float sum, float A2, float h, float end) {
  constexpr float kMax = 3.4028235e38f;
  if (fabsf(sum) < kMax && fabsf(A2) < kMax) {
    const float e = fminf(fmaxf(sum * A2, -512.f), 512.f), whole = ceilf(e);
    return ldexpf(exp2_hw(e - whole) * h, (int)whole) + end;
  }
  return fmaf(exp2_hw(sum * A2), h, end);
}

__global__ __launch_bounds__(64 * kFoldWaves) void ssm_fold_kernel(SeqTable tab, SsmArgs a,
                                                                   int SN) {
  __shared__ float s_end[kFoldWaves][64], s_sum[kFoldWaves][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int blocks = a.G * a.cb, per = blocks * SN;
  const int f = blockIdx.x / per, rest = blockIdx.x - f * per;
  const int gc = rest / SN, i = rest - gc * SN;
  if (i >= a.N)
    return;
  const SeqView seqs(tab);
  const int n = seqs.find(f, 2);
  const int64_t pair0 = seqs.blk(n, 1);
  const int pairs = (int)(seqs.blk(n + 1, 1) - pair0);
  const int g = gc / a.cb, dg = (gc - g * a.cb) * 64 + lane;
  const float A2 = dg < a.Dg ? log2_rate(a.A[((int64_t)g * a.Dg + dg) * a.N + i]) : 0.f;
  float *pe = a.pend + ((pair0 * blocks + gc) * SN + i) * 64 + lane;
  const float *ps = a.psum + (pair0 * blocks + gc) * 64 + lane;
  const int64_t pstep = (int64_t)blocks * SN * 64, sstep = (int64_t)blocks * 64;
  const int run = (pairs - 1 + kFoldWaves - 1) / kFoldWaves;
  const int j0 = 1 + wave * run, j1 = min(pairs, j0 + run);
  float sum = 0.f;
  const auto fold = [&](float h, bool write) {
    for (int j = j0; j < j1; j += 8) {
      float e[8], sd[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int q = min(j + k, j1 - 1);
        e[k] = pe[q * pstep];
        sd[k] = ps[q * sstep];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (j + k < j1) {
          h = fold_segment(sd[k], A2, h, e[k]);
          if (write)
            pe[(j + k) * pstep] = h;
          else
            sum += sd[k];
        }
    }
    return h;
  };
  s_end[wave][lane] = fold(0.f, false);
  s_sum[wave][lane] = finite_sum(sum);
  __syncthreads();
  float h = pe[0];
  for (int w = 0; w < wave; ++w)
    h = fold_segment(s_sum[w][lane], A2, h, s_end[w][lane]);
  fold(h, true);
}

// ---- single tokens ------------------------------------------------------------------
// A wave takes 64 channels of one row.  The state is read once and written
// once, so HBM bounds the call as long as little else goes through the memory
// pipe: x, delta, z and y move one channel a lane (softplus and gate are
// evaluated there), B and C once a wave; the states pass in chunks of 64 / W
// channels, W lanes a channel with VEC states on each (K times), which get
// their channel's delta and delta x from its lane and give their sum back to
// it.  256 rows x 12288 bf16, N = 16: 69 to 74 us, 5.6 to 6.0 TB/s.  Where N
// is no multiple of 4 a lane takes one state at a time: N = 13 83 us (3.9
// TB/s), N = 5 40 us (3.1).
struct StepArgs {
  int32_t D, N, G, Dg, cb, rows, softplus, num_slots, wlog, bcvec;
  int64_t xs, dls, zs, ys, Bs, Cs;
  const float *A, *skip, *bias;
  float *state;
  const int32_t *slots;
};

// Sum over groups of 2^wlog neighbouring lanes, in every lane of the group.
__device__ __forceinline__ float group_sum(float x, int wlog) {
  if (wlog > 0)
    x += quad_swap<0xb1>(x); // lane ^ 1
  if (wlog > 1)
    x += quad_swap<0x4e>(x); // lane ^ 2
  if (wlog > 2)
    x += quad_swap<0x141>(x); // mirrored in 8 lanes: the other quad
  if (wlog > 3)
    x += quad_swap<0x140>(x); // mirrored in 16 lanes: the other eight
  if (wlog > 4)
    x = add_xor16(x);
  if (wlog > 5)
    x = add_xor32(x);
  return x;
}

// Four consecutive values of B or C.
__device__ __forceinline__ void load4(const bf16 *p, float (&v)[4]) {
  const bf16x4 r = *reinterpret_cast<const bf16x4 *>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = to_f32(r[i]);
}
__device__ __forceinline__ void load4(const float *p, float (&v)[4]) {
  const f32x4 r = *reinterpret_cast<const f32x4 *>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    v[i] = r[i];
}

template <typename T, int VEC, int K>
__global__ __launch_bounds__(256) void ssm_step_kernel(StepArgs a, const T *__restrict__ x,
                                                       const T *__restrict__ dl,
                                                       const T *__restrict__ B,
                                                       const T *__restrict__ C,
                                                       const T *__restrict__ z, T *y) {
  // the waves of a workgroup: four rows of the same channels, whose A they
  // share in the compute unit's cache
  const int64_t wv = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t blocks = (int64_t)a.G * a.cb, q = wv / (4 * blocks);
  const int64_t row = q * 4 + wv % 4, gc = wv / 4 % blocks;
  if (row >= a.rows)
    return;
  const int64_t slot = a.slots ? a.slots[row] : row;
  if (slot < 0 || slot >= a.num_slots)
    return; // a padding row: nothing is read or written
  const int lane = threadIdx.x & 63;
  const int64_t g = gc / a.cb;
  const int c0 = (int)(gc - g * a.cb) * 64; // first channel, in its group
  const int64_t d0 = g * a.Dg + c0;
  const int chans = min(64, a.Dg - c0);
  const int W = 1 << a.wlog, per = 64 >> a.wlog; // lanes a channel, channels a chunk
  const int w = lane & (W - 1), cc = lane >> a.wlog;

  // this lane's channel
  float xv = 0.f, delta = 0.f, zv = 0.f, skip = 0.f;
  if (lane < chans) {
    xv = to_f32(x[row * a.xs + d0 + lane]);
    delta = to_f32(dl[row * a.dls + d0 + lane]) + (a.bias ? a.bias[d0 + lane] : 0.f);
    if (z)
      zv = to_f32(z[row * a.zs + d0 + lane]);
    if (a.skip)
      skip = a.skip[d0 + lane];
  }
  // this lane's states in every chunk
  float b[K][VEC], c[K][VEC];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int n = (k * W + w) * VEC;
    const T *pb = B + row * a.Bs + g * a.N + n, *pc = C + row * a.Cs + g * a.N + n;
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      b[k][i] = c[k][i] = 0.f;
    if (n < a.N) {
      bool done = false;
      if constexpr (VEC == 4)
        if (a.bcvec) {
          load4(pb, b[k]);
          load4(pc, c[k]);
          done = true;
        }
      if (!done) {
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          b[k][i] = to_f32(pb[i]);
          c[k][i] = to_f32(pc[i]);
        }
      }
    }
  }
  if (a.softplus)
    delta = softplus(delta);
  const float u = delta * xv;
  // An infinite rate counts as the largest finite one, as in the prompt
  // kernels.  That shows in steps of (nearly) 0 alone, so only waves with one
  // replace it (in all of them: 256 x 12288, N = 16 takes 74 us, not 68; 64 x
  // 8192, N = 65 114, not 78).
  const bool still =
      __builtin_amdgcn_ballot_w64(lane < chans && fabsf(delta) < 1e-35f) != 0;

  float *st = a.state + (slot * a.D + d0) * a.N;
  const float *Ad = a.A + d0 * a.N;
  float out = 0.f;
  constexpr int kU = K == 1 ? 4 : 2; // chunks whose states are in flight together
  for (int k0 = 0; k0 < W; k0 += kU) {
    float h[kU][K][VEC], A[kU][K][VEC];
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      const int ch = (k0 + j) * per + cc;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int n = (k * W + w) * VEC;
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          h[j][k][i] = A[j][k][i] = 0.f;
        if (k0 + j < W && ch < chans && n < a.N) {
          if constexpr (VEC == 4) {
            const f32x4 hv = __builtin_nontemporal_load(
                reinterpret_cast<const f32x4 *>(st + ch * a.N + n));
            const f32x4 av = *reinterpret_cast<const f32x4 *>(Ad + ch * a.N + n);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              h[j][k][i] = hv[i];
              A[j][k][i] = av[i];
            }
          } else {
            h[j][k][0] = st[ch * a.N + n];
            A[j][k][0] = Ad[ch * a.N + n];
          }
        }
      }
    }
    if (still) {
#pragma unroll
      for (int j = 0; j < kU; ++j)
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int i = 0; i < VEC; ++i)
            A[j][k][i] = finite_rate(A[j][k][i]);
    }
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      if (k0 + j >= W)
        break;
      const int ch = (k0 + j) * per + cc;
      const float dj = __shfl(delta, ch) * kLog2e, uj = __shfl(u, ch);
      float acc = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const int n = (k * W + w) * VEC;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          h[j][k][i] = fmaf(exp2_hw(dj * A[j][k][i]), h[j][k][i], uj * b[k][i]);
          // (a state that is not there adds no 0 * inf)
          acc = n < a.N ? fmaf(c[k][i], h[j][k][i], acc) : acc;
        }
        if (ch < chans && n < a.N) {
          if constexpr (VEC == 4)
            __builtin_nontemporal_store(f32x4{h[j][k][0], h[j][k][1], h[j][k][2], h[j][k][3]},
                                        reinterpret_cast<f32x4 *>(st + ch * a.N + n));
          else
            st[ch * a.N + n] = h[j][k][0];
        }
      }
      acc = group_sum(acc, a.wlog);
      // channel's lane l: chunk l / per, whose lanes (l % per) W .. hold it
      const float mine = __shfl(acc, (lane & (per - 1)) << a.wlog);
      out = lane >> (6 - a.wlog) == k0 + j ? mine : out;
    }
  }
  if (lane < chans) {
    float v = a.skip ? fmaf(skip, xv, out) : out;
    if (z)
      v *= silu(zv);
    y[row * a.ys + d0 + lane] = from_f32<T>(v);
  }
}

// ---- host ---------------------------------------------------------------------------
// States a lane of the row kernel holds.
int row_states(int N) { return N <= 16 ? 1 : (N <= 32 ? 2 : (N <= 64 ? 4 : 8)); }
constexpr int kLaneMaxStates = 16;

constexpr size_t kAlign = 256;
size_t up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

int64_t chan_blocks(int32_t D, int32_t G) { return (int64_t)G * ((D / G + 63) / 64); }

template <int N = 1, typename F> hipError_t with_lane(int states, F &&f) {
  if constexpr (N < kLaneMaxStates)
    if (states != N)
      return with_lane<N + 1>(states, f);
  return f(std::integral_constant<int, N>());
}

template <typename F> hipError_t with_row(int E, bool pairs, bool pad, F &&f) {
  using std::integral_constant;
  const auto padded = [&](auto e, auto p) {
    return pad ? f(e, p, std::true_type()) : f(e, p, std::false_type());
  };
  using one = integral_constant<int, 1>;
  using two = integral_constant<int, 2>;
  switch (E) {
  case 1: return pairs ? padded(one(), two()) : padded(one(), one());
  case 2: return pairs ? padded(two(), two()) : padded(two(), one());
  case 4: return padded(integral_constant<int, 4>(), one());
  default: return padded(integral_constant<int, 8>(), one());
  }
}

} // namespace

int64_t ssm_num_segments(int64_t len, const SsmPlan &p) {
  return len > p.seg ? (len + p.seg - 1) / p.seg : 1;
}

// Which kernel, and the cut.  Times in us, fitted to runs over D = 1536 ..
// 12288, 1 .. 128 sequences and 1024 .. 32768 tokens with N = 16:
//   row kernel, uncut: 36 ns a token of the longest sequence where its waves
//     have a SIMD each to themselves; a wave more on the SIMD adds 16.5 ns.
//     A sequence costs some 80 tokens to begin (tiles of 64).
//   lane kernel, uncut: 0.24 ns per token and 64 channels at full occupancy
//     (a sequence costs some 24 tokens to begin), 0.4 us a token of the
//     longest sequence for a wave alone.
//   either one, cut into segments (six row waves a SIMD, four lane waves):
//     two such runs, the middle segments' first one without read-outs (row:
//     0.7 of a run; lane: 0.18 ns per token and 64 channels), and 15 or 25 us
//     for the launches between.
// Both sides: 8192 tokens x 8192 channels: row 391, lane cut 463.  131072 x
// 1536: row 4500, lane cut 1320.  4096 x 1536: row 139, row cut 66, lane cut
// 92.  64 sequences of 16 tokens x 8192: row 189, lane 81.  128 sequences of
// 64 x 12288: row 742, lane 513.
// Other N scale these times by their share of the instructions; that was not
// fitted, but measured on both sides for N = 1 .. 128 (bf16, gate; and fp32 for
// N = 5 and 8) at 8192 x 8192, 4096 x 1536, 65536 x 1024, 16 sequences of 1024
// x 2048 and 64 of 128 x 4096.  8192 x 8192, N = 1, 4, 5, 8, 13: row 458, 406,
// 430, 401, 441, lane cut 234, 247, 273, 315, 481; 65536 x 1024: row cut 604,
// 599, 615, 611, 633, lane cut 238, 270, 306, 347, 478.  The choice is the
// faster side, or within a tenth of it, at all but one: 16 sequences of 1024 x
// 2048 with N = 1 .. 5 run uncut on the lane kernel in 235 .. 300, where the
// row kernel takes 173 .. 183 and the cut lane kernel 127 .. 178.  (A lane
// wave alone takes some 0.20 + 0.0125 N us a token, of which the model below
// leaves out the part without N.)
SsmPlan ssm_plan(int32_t num_seqs, const int64_t *cu, int32_t D, int32_t N, int32_t G,
                 int32_t split_hint) {
  SsmPlan p{};
  const int64_t blocks = chan_blocks(D, G), tokens = cu[num_seqs];
  int64_t longest = 0;
  for (int32_t n = 0; n < num_seqs; ++n)
    longest = std::max(longest, cu[n + 1] - cu[n]);
  // multiples of 32 tokens: whole tiles
  const auto whole = [](int64_t x) { return std::max<int64_t>(32, (x + 31) / 32 * 32); };
  p.seg = whole(longest);
  const int E = row_states(N);
  const double T = (double)tokens, L = (double)longest, W = (double)blocks, n = num_seqs;
  // (the states' share of each kernel's instructions, beside N = 16)
  const double row_scale = (33. * E + 15.) / 48., full = (24. * N + 150.) / 534. * 0.24e-3,
               half = (20. * N + 90.) / 410. * 0.18e-3;
  // row waves a SIMD, one sequence
  const double per_simd = (double)G * ((D / G + kRowChans - 1) / kRowChans) * 4. / 1024.;
  const auto row_time = [&](double longest_run, double tokens_run) {
    return row_scale * std::max(0.036 * longest_run,
                                0.020 * longest_run + 0.0165 * per_simd * tokens_run);
  };
  const auto lane_time = [&](double longest_run, double work) {
    const double alone = 0.40 * longest_run * N / 16.;
    return std::max(alone, work) + 0.15 * std::min(alone, work);
  };
  const bool lane_fits = N <= kLaneMaxStates;
  const double row = row_time(L, T + 80. * n);
  const double lane = lane_fits ? lane_time(L, W * (T + 24. * n) * full) : 1e30;
  const double uncut = std::min(row, lane);
  p.lane = lane < row;
  if (split_hint > 1) {
    p.lane = lane_fits;
    p.seg = whole((longest + split_hint - 1) / split_hint);
  } else if (split_hint == 0) {
    const int64_t row_seg = std::max<int64_t>(128, whole((int64_t)(T * per_simd / 6.)));
    const int64_t lane_seg = std::max<int64_t>(64, whole(tokens * blocks / 4096));
    int64_t first = 0, middle = 0; // tokens of first and of middle segments
    for (int32_t i = 0; i < num_seqs; ++i) {
      const int64_t len = cu[i + 1] - cu[i];
      first += std::min(len, lane_seg);
      middle += std::max<int64_t>(0, len - 2 * lane_seg);
    }
    const double row_cut = 15. + 1.7 * row_time((double)row_seg, T + 80. * n);
    const double lane_cut =
        lane_fits ? 25. +
                        lane_time((double)lane_seg, W * (((double)first + 24. * n) * full +
                                                         (double)middle * half)) +
                        lane_time((double)lane_seg, W * (T - (double)first) * full)
                  : 1e30;
    const bool cut_lane = lane_cut < row_cut;
    const int64_t seg = cut_lane ? lane_seg : row_seg;
    if (std::min(lane_cut, row_cut) < 0.85 * uncut && seg * 3 <= longest) {
      p.lane = cut_lane;
      p.seg = seg;
    }
  }
  p.states = p.lane ? N : E;
  for (int32_t n = 0; n < num_seqs; ++n)
    p.pairs += ssm_num_segments(cu[n + 1] - cu[n], p) - 1;
  const size_t SN = (size_t)p.states * (p.lane ? 1 : 16);
  size_t o = seq_table_bytes(num_seqs);
  p.off_end = o;
  o = up(o + (size_t)p.pairs * blocks * 64 * SN * sizeof(float));
  p.off_sum = o;
  o = up(o + (size_t)p.pairs * blocks * 64 * sizeof(float));
  p.total = o;
  return p;
}

hipError_t launch_ssm(int elt, const SsmCall &c, int32_t num_seqs, const int64_t *cu,
                      const SsmPlan &plan, void *ws, hipStream_t s) {
  const int64_t tokens = cu[num_seqs];
  const int64_t blocks = chan_blocks(c.D, c.G);
  const int SN = plan.states * (plan.lane ? 1 : 16);
  uint8_t *w = (uint8_t *)ws;

  SsmArgs a{};
  a.D = c.D;
  a.N = c.N;
  a.G = c.G;
  a.softplus = c.softplus;
  a.num_slots = c.num_slots;
  a.Dg = c.D / c.G;
  a.cb = (a.Dg + 63) / 64;
  a.seg = (int32_t)plan.seg;
  a.xs = c.x_stride;
  a.dls = c.delta_stride;
  a.zs = c.z_stride;
  a.ys = c.y_stride;
  a.Bs = c.B_stride;
  a.Cs = c.C_stride;
  a.A = c.A;
  a.skip = c.skip;
  a.bias = c.bias;
  a.init = c.init;
  a.fin = c.fin;
  a.slots = c.slots;
  a.pend = (float *)(w + plan.off_end);
  a.psum = (float *)(w + plan.off_sum);

  // segments in each pass, and (2) whether there are pairs to fold
  const auto tiles = [&](int64_t len, int w) -> int64_t {
    const int64_t nseg = ssm_num_segments(len, plan);
    return w == 0 ? std::max<int64_t>(1, nseg - 1) : (w == 1 ? nseg - 1 : nseg > 2);
  };
  int64_t total[kCounts];
  if (!seq_totals(num_seqs, cu, tiles, total))
    return hipErrorInvalidConfiguration;
  // workgroups per (segment, all channels); the row kernel's grid is rounded
  // up to whole rounds over the dies
  const int64_t per = plan.lane ? (blocks + 3) / 4 : (int64_t)c.G * ((a.Dg + kRowChans - 1) / kRowChans);
  const int64_t round = plan.lane ? 1 : 8 * kRowNear;
  int64_t grid[2];
  for (int pass = 0; pass < 2; ++pass) {
    grid[pass] = (total[pass] * per + round - 1) / round * round;
    if (grid[pass] * 256 > UINT32_MAX)
      return hipErrorInvalidConfiguration;
  }
  const int64_t fold = total[2] * blocks * SN;
  if (fold * 64 * kFoldWaves > UINT32_MAX)
    return hipErrorInvalidConfiguration;
  SeqTable tab;
  hipError_t e = make_seq_table(tab, num_seqs, cu, tiles, ws, s);
  if (e != hipSuccess)
    return e;

  // the row kernel stages two neighbouring elements at a time where every
  // pair is one aligned load (8192 x 8192 bf16: 391 us against 415)
  const auto paired = [elt](const void *p, int64_t stride) {
    return ((uintptr_t)p & (elt == 1 ? 3u : 7u)) == 0 && stride % 2 == 0;
  };
  const bool pairs = a.Dg % 2 == 0 && c.N % 2 == 0 && paired(c.x, c.x_stride) &&
                     paired(c.delta, c.delta_stride) && paired(c.z, c.z ? c.z_stride : 0) &&
                     paired(c.y, c.y_stride) && paired(c.B, c.B_stride) && paired(c.C, c.C_stride);

  const auto typed = [&](auto tag) {
    using T = decltype(tag);
    const T *x = (const T *)c.x, *dl = (const T *)c.delta, *z = (const T *)c.z;
    const T *B = (const T *)c.B, *C = (const T *)c.C;
    T *y = (T *)c.y;
    const auto passes = [&](auto &&run) {
      run(0, (unsigned)grid[0]);
      if (fold > 0)
        ssm_fold_kernel<<<(unsigned)fold, 64 * kFoldWaves, 0, s>>>(tab, a, SN);
      if (total[1] > 0)
        run(1, (unsigned)grid[1]);
      return hipGetLastError();
    };
    if (plan.lane)
      return with_lane(plan.states, [&](auto ns) {
        return passes([&](int pass, unsigned n) {
          ssm_lane_kernel<T, decltype(ns)::value><<<n, 256, 0, s>>>(tab, a, pass, x, dl, z, B, C, y);
        });
      });
    return with_row(plan.states, pairs, c.N < SN, [&](auto e, auto p2, auto pad) {
      return passes([&](int pass, unsigned n) {
        ssm_row_kernel<T, decltype(e)::value, decltype(p2)::value, decltype(pad)::value>
            <<<n, 256, 0, s>>>(tab, a, pass, total[pass] * per, x, dl, z, B, C, y);
      });
    });
  };
  return elt == 1 ? typed(bf16()) : typed(float());
}

hipError_t launch_ssm_step(int elt, const SsmCall &c, int32_t rows, hipStream_t s) {
  StepArgs a{};
  a.D = c.D;
  a.N = c.N;
  a.Dg = c.D / c.G;
  a.softplus = c.softplus;
  a.num_slots = c.num_slots;
  a.xs = c.x_stride;
  a.dls = c.delta_stride;
  a.zs = c.z_stride;
  a.ys = c.y_stride;
  a.Bs = c.B_stride;
  a.Cs = c.C_stride;
  a.A = c.A;
  a.skip = c.skip;
  a.bias = c.bias;
  a.state = c.fin;
  a.slots = c.slots;
  a.G = c.G;
  a.cb = (a.Dg + 63) / 64;
  a.rows = rows;
  const bool wide = c.N % 4 == 0; // (the state and A are 16-byte aligned)
  const int need = wide ? c.N / 4 : c.N;
  while ((1 << a.wlog) < need && a.wlog < 6)
    ++a.wlog;
  const uintptr_t quad = elt == 1 ? 8 : 16;
  a.bcvec = (uintptr_t)c.B % quad == 0 && (uintptr_t)c.C % quad == 0 && c.B_stride % 4 == 0 &&
            c.C_stride % 4 == 0;
  const int64_t grid = ((int64_t)rows + 3) / 4 * c.G * a.cb;
  if (grid * 256 > UINT32_MAX)
    return hipErrorInvalidConfiguration;
  const auto run = [&](auto tag, auto vec, auto k) {
    using T = decltype(tag);
    ssm_step_kernel<T, decltype(vec)::value, decltype(k)::value><<<(unsigned)grid, 256, 0, s>>>(
        a, (const T *)c.x, (const T *)c.delta, (const T *)c.B, (const T *)c.C, (const T *)c.z,
        (T *)c.y);
    return hipGetLastError();
  };
  const auto shaped = [&](auto tag) {
    using std::integral_constant;
    if (wide)
      return run(tag, integral_constant<int, 4>(), integral_constant<int, 1>());
    if (need <= 64)
      return run(tag, integral_constant<int, 1>(), integral_constant<int, 1>());
    return run(tag, integral_constant<int, 1>(), integral_constant<int, 2>());
  };
  return elt == 1 ? shaped(bf16()) : shaped(float());
}

} // namespace kda
