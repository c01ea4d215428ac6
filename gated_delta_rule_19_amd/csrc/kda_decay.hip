// Linear attention with one decay a head, for packed prompts and for single
// tokens:  S_t = exp(g_t) S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t.
//
// Prompts run in chunks of 64 tokens.  With G the sum of g from a chunk's
// start, S the state that enters it and L its last token:
//   o_i = scale (e^{G_i} S^T q_i + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j)
//   S'  = e^{G_L} S + sum_j k_j (e^{G_L - G_j} v_j)^T
// that is four matrix products a chunk.  A workgroup carries the state of one
// (sequence, head) and 64 value columns through the tokens in registers; wave
// w owns 16 columns of the state (all dk rows) and the scores and outputs of
// tokens 16 w .. 16 w + 15.  K and V of a chunk and the state that enters it
// are shared through LDS; the next chunk's K, V, q and g are requested before
// a chunk is worked on and wait in registers.
//
// Layout: every product takes its tokens (the summed index of S' and of the
// second part of o) in the order 32 s + 16 h + 4 g + r for element 4 h + r of
// lane group g, which is how two tiles of scores come out of the matrix
// instruction: the scores go into the next product from the registers they
// are in, and K and V are read transposed in that order.  Column tiles take
// the columns 32 (t / 2) + 8 (m / 4) + 4 (t % 2) + m % 4, so that a lane holds
// eight neighbouring columns of o.
//
// Roundings: the state is fp32 and its update takes v e^{G_L - G_j} as the sum
// of three bf16 numbers (24 bits; one alone would leave the state 2^-9 off),
// beside k as it is; the scores and the entering state are rounded to bf16
// once each for o, which is rounded to bf16 itself.  fp32 calls round nothing.
// G is summed in 64 bits and kept as two fp32 numbers, so that differences
// within a chunk keep their accuracy beside a decay of e^-150.
//
// An infinity or NaN in k or v would reach earlier tokens of its chunk as
// 0 * inf: a chunk is ended in front of such a token, which is then worked on
// alone, its update as an outer product.
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
  // prompts
  int32_t slices, seg; // 64-column slices of dv, tokens per segment
  int64_t units;       // (segment, head) pairs of this launch
  float *pair_state;   // [pairs, H, slices, DK / 16, 256] of four
  double *pair_decay;  // [pairs, H]: log2 of a segment's decay
};

constexpr float kMinDecay = -150.f; // fp32's exp is 0 there
constexpr double kLog2E = 1.4426950408889634074;

// exp(g), 0 from kMinDecay down (and for -inf)
__device__ __forceinline__ float decay_of(float g) { return expf(fmaxf(g, kMinDecay)); }

// 2^x of a 64-bit exponent, to an fp32 rounding or two
__device__ __forceinline__ float exp2_of(double x) {
  x = x < -1000. ? -1000. : x > 1000. ? 1000. : x; // (a NaN stays one)
  const double n = rint(x);
  return ldexpf(__builtin_amdgcn_exp2f((float)(x - n)), (int)n);
}

// ---- prompts ----------------------------------------------------------------------

constexpr int kDC = 64;   // tokens per chunk
constexpr int kDCols = 64; // value columns per workgroup

// Eight elements of a row, as loaded.
template <typename T> struct Oct;
template <> struct Oct<bf16> { u32x4 r; };
template <> struct Oct<float> { f32x4 lo, hi; };
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));

// n of eight elements from p (n >= 8: all, n <= 0: none; the others are 0)
__device__ __forceinline__ Oct<bf16> load_oct(const bf16 *p, int n) {
  Oct<bf16> o{};
  if (n >= 8) {
    o.r = *reinterpret_cast<const u32x4_any *>(p);
  } else if (n > 0) {
    bf16x8 v{};
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n)
        v[i] = p[i];
    o.r = __builtin_bit_cast(u32x4, v);
  }
  return o;
}
__device__ __forceinline__ Oct<float> load_oct(const float *p, int n) {
  Oct<float> o{};
  if (n >= 8) {
    o.lo = *reinterpret_cast<const f32x4_any *>(p);
    o.hi = *reinterpret_cast<const f32x4_any *>(p + 4);
  } else if (n > 0) {
    float v[8] = {};
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n)
        v[i] = p[i];
    o.lo = f32x4{v[0], v[1], v[2], v[3]};
    o.hi = f32x4{v[4], v[5], v[6], v[7]};
  }
  return o;
}
__device__ __forceinline__ void to_lds(bf16 *p, const Oct<bf16> &o) {
  *reinterpret_cast<u32x4 *>(p) = o.r;
}
__device__ __forceinline__ void to_lds(float *p, const Oct<float> &o) {
  *reinterpret_cast<f32x4 *>(p) = o.lo;
  *reinterpret_cast<f32x4 *>(p + 4) = o.hi;
}
__device__ __forceinline__ Frag<bf16> as_frag(const Oct<bf16> &o) {
  return {__builtin_bit_cast(bf16x8, o.r)};
}
__device__ __forceinline__ Frag<float> as_frag(const Oct<float> &o) { return {o.lo, o.hi}; }

// Nonzero where an element has an exponent of all ones.
__device__ __forceinline__ uint32_t non_finite(const Oct<bf16> &o) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) // (the sums of the halves do not carry over)
    m |= (o.r[i] & 0x7f807f80u) + 0x00800080u;
  return m & 0x80008000u;
}
__device__ __forceinline__ uint32_t non_finite(const Oct<float> &o) {
  const u32x4 lo = __builtin_bit_cast(u32x4, o.lo), hi = __builtin_bit_cast(u32x4, o.hi);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m |= ((lo[i] & 0x7f800000u) + 0x00800000u) | ((hi[i] & 0x7f800000u) + 0x00800000u);
  return m & 0x80000000u;
}

// The operand of eight tokens (element 4 h + r: row0 + 16 h + 4 lg + r) and
// the 16 columns col(m) of a tile, from a token-major LDS matrix.  bf16: two
// transposed reads; in each 16-lane group, lane 4 a + b of ds_read_b64_tr_b16
// receives element b of the 4-element reads of lanes a, a + 4, a + 8, a + 12,
// so lane L reads four columns of row L / 4, from the one of m = 4 (L % 4) on.
template <typename Col>
__device__ __forceinline__ Frag<bf16> tr_frag(const bf16 *m, int ld, int row0, int lr, int lg,
                                              Col &&col) {
  typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
  const bf16 *p = m + (row0 + 4 * lg + (lr >> 2)) * ld + col(4 * (lr & 3));
  const bf16x4 r0 = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4 *)p);
  const bf16x4 r1 = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4 *)(p + 16 * ld));
  return {__builtin_shufflevector(r0, r1, 0, 1, 2, 3, 4, 5, 6, 7)};
}
template <typename Col>
__device__ __forceinline__ Frag<float> tr_frag(const float *m, int ld, int row0, int lr, int lg,
                                               Col &&col) {
  const float *p = m + (row0 + 4 * lg) * ld + col(lr);
  Frag<float> f;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    f.lo[r] = p[r * ld];
    f.hi[r] = p[(16 + r) * ld];
  }
  return f;
}

__device__ __forceinline__ Frag<bf16> pack_scores(const f32x4 &lo, const f32x4 &hi, bf16) {
  return pack_acc2(lo, hi);
}
__device__ __forceinline__ Frag<float> pack_scores(const f32x4 &lo, const f32x4 &hi, float) {
  return {lo, hi};
}

// An operand times a weight per element, as a sum of operands.
struct Split3 {
  Frag<bf16> part[3];
};
__device__ __forceinline__ Split3 weigh(const Frag<bf16> &v, const f32x4 &w0, const f32x4 &w1) {
  Split3 s;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float x = static_cast<float>(v.v[i]) * (i < 4 ? w0[i & 3] : w1[i & 3]);
#pragma unroll
    for (int p = 0; p < 3; ++p) {
      const bf16 b = static_cast<bf16>(x);
      s.part[p].v[i] = b;
      x = x == static_cast<float>(b) ? 0.f : x - static_cast<float>(b);
    }
  }
  return s;
}
struct Whole {
  Frag<float> part[1];
};
__device__ __forceinline__ Whole weigh(const Frag<float> &v, const f32x4 &w0, const f32x4 &w1) {
  return {{{v.lo * w0, v.hi * w1}}};
}

template <typename T> struct Tiles; // rows of the LDS matrices, padded
template <> struct Tiles<bf16> { static constexpr int k = 8, v = 8, s = 8; };
template <> struct Tiles<float> { static constexpr int k = 4, v = 4, s = 4; };

// Launch `pass` 0: all segments but each sequence's last (all of them where a
// sequence is not cut): the first segments in full, the others only their
// state from zero.  Pass 1: the other segments from the states that enter
// them.
template <typename T, int DK>
__global__ __launch_bounds__(256) void decay_chunk_kernel(SeqTable tab, DecayArgs a, int pass,
                                                          const T *__restrict__ q,
                                                          const T *__restrict__ k,
                                                          const T *__restrict__ v,
                                                          T *__restrict__ o) {
  const SeqView sv(tab);
  constexpr int kLdK = DK + Tiles<T>::k, kLdV = kDCols + Tiles<T>::v, kLdS = DK + Tiles<T>::s;
  constexpr int kGK = DK / 32, kGV = 2; // groups of eight of K and V a lane stages
  constexpr int kTD = DK / 16;          // state tiles of a wave
  __shared__ alignas(16) T Ks[kDC * kLdK], Vs[kDC * kLdV], Ss[kDCols * kLdS];
  __shared__ alignas(16) float Ghi[kDC], Glo[kDC], wts[kDC], eG[kDC];
  __shared__ float total;
  __shared__ int first_bad[4];

  // block b: unit (b / 8 / slices) * 8 + b % 8, slice b / 8 % slices: slices
  // of one unit, which share q and k, are on one die
  const int64_t unit = (int64_t)(blockIdx.x / (8 * a.slices)) * 8 + blockIdx.x % 8;
  if (unit >= a.units)
    return;
  const int slice = blockIdx.x / 8 % a.slices;
  const int h = (int)(unit % a.H), blk = (int)(unit / a.H);
  const int n = sv.find(blk, pass);
  const int seq = sv.seq(n), len = sv.len(n);
  const int nseg = sv.blk(n + 1, 1) - sv.blk(n, 1) + 1; // (pairs in front: pass 1's blocks)
  const int seg = blk - sv.blk(n, pass) + pass;
  const int64_t pair0 = sv.blk(n, 1);
  const bool outputs = pass == 1 || seg == 0;
  int pos = seg * a.seg;
  const int end = min(len, pos + a.seg);
  const int64_t slot = a.slots ? a.slots[seq] : seq;
  const bool kept = slot >= 0 && slot < a.num_slots;

  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lg = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col0 = slice * kDCols;
  const auto row_col = [](int d) { return [d](int m) { return 16 * d + m; }; };
  const auto val_col = [](int e) {
    return [e](int m) { return 32 * (e >> 1) + 8 * (m >> 2) + 4 * (e & 1) + (m & 3); };
  };
  const int my_col = val_col(w)(lr); // of the state this lane holds

  // the state that enters: lane (lr, lg) element r of tile d is row 16 d + 4
  // lg + r of column my_col
  f32x4 S[kTD];
  const int64_t global = (slot * a.H + h) * a.dk * a.dv + col0 + my_col;
  float *pairs = a.pair_state + ((pair0 * a.H + h) * a.slices + slice) * (kTD * 1024) + tid * 4;
  const int64_t pair_step = (int64_t)a.H * a.slices * (kTD * 1024);
  if (pass == 1) {
#pragma unroll
    for (int d = 0; d < kTD; ++d)
      S[d] = *reinterpret_cast<const f32x4 *>(pairs + (seg - 1) * pair_step + d * 1024);
  } else {
    const bool from = seg == 0 && a.init && kept && col0 + my_col < a.dv;
#pragma unroll
    for (int d = 0; d < kTD; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * d + 4 * lg + r;
        S[d][r] = from && row < a.dk ? a.init[global + (int64_t)row * a.dv] : 0.f;
      }
  }

  // staging: what a lane loads of a tile of `cnt` tokens from token `at` on
  Oct<T> kr[kGK], vr[kGV], qn[kGK];
  float gn = 0.f;
  const int64_t tok0 = sv.tok0(n);
  const auto load_tile = [&](int at, int cnt) {
    const T *kb = k + (tok0 + at) * a.ks + (int64_t)(h / a.rk) * a.dk;
    const T *vb = v + (tok0 + at) * a.vs + (int64_t)(h / a.rv) * a.dv + col0;
#pragma unroll
    for (int i = 0; i < kGK; ++i) {
      const int row = (i * 256 + tid) / (DK / 8), c = (i * 256 + tid) % (DK / 8) * 8;
      kr[i] = load_oct(kb + row * (int)a.ks + c, row < cnt ? a.dk - c : 0);
    }
#pragma unroll
    for (int i = 0; i < kGV; ++i) {
      const int row = (i * 256 + tid) / 8, c = (i * 256 + tid) % 8 * 8;
      vr[i] = load_oct(vb + row * (int)a.vs + c, row < cnt ? a.dv - col0 - c : 0);
    }
    if (w == 0)
      gn = lane < cnt ? a.g[(tok0 + at + lane) * a.gs + h] : 0.f;
    if (outputs) {
      const T *qb = q + (tok0 + at) * a.qs + (int64_t)(h / a.rq) * a.dk;
      const int row = 16 * w + lr;
#pragma unroll
      for (int i = 0; i < kGK; ++i)
        qn[i] = load_oct(qb + row * (int)a.qs + 32 * i + 8 * lg, row < cnt ? a.dk - 32 * i - 8 * lg : 0);
    }
  };
  // wave 0: log2 of the decay from the tile's start to each of its tokens
  double G = 0.;
  const auto scan_decays = [&](int cnt) {
    G = lane < cnt ? (double)fmaxf(gn, kMinDecay) * kLog2E : 0.;
    if (gn != gn)
      G = __builtin_nan("");
#pragma unroll
    for (int b = 1; b < 64; b <<= 1) {
      const double up = __shfl_up(G, b);
      G += lane >= b ? up : 0.;
    }
  };
  const auto put_decays = [&](int cnt) {
    const double last = __shfl(G, cnt - 1);
    const float hi = (float)G;
    Ghi[lane] = hi;
    Glo[lane] = (float)(G - (double)hi);
    eG[lane] = exp2_of(G);
    wts[lane] = lane < cnt ? exp2_of(last - G) : 0.f;
    if (lane == 0)
      total = exp2_of(last);
  };
  const auto put_state = [&]() {
#pragma unroll
    for (int d = 0; d < kTD; ++d)
      store4(Ss + my_col * kLdS + 16 * d + 4 * lg, S[d][0], S[d][1], S[d][2], S[d][3]);
  };
  // the tile into LDS; what it holds beside finite numbers is noted
  const auto put_tile = [&]() {
    int bad = kDC;
#pragma unroll
    for (int i = 0; i < kGK; ++i) {
      const int row = (i * 256 + tid) / (DK / 8), c = (i * 256 + tid) % (DK / 8) * 8;
      to_lds(Ks + row * kLdK + c, kr[i]);
      if (non_finite(kr[i]))
        bad = min(bad, row);
    }
#pragma unroll
    for (int i = 0; i < kGV; ++i) {
      const int row = (i * 256 + tid) / 8, c = (i * 256 + tid) % 8 * 8;
      to_lds(Vs + row * kLdV + c, vr[i]);
      if (non_finite(vr[i]))
        bad = min(bad, row);
    }
    if (__any(bad < kDC))
      for (int b = 1; b < 64; b <<= 1)
        bad = min(bad, __shfl_xor(bad, b));
    if (lane == 0)
      first_bad[w] = bad;
  };

  double decay_sum = 0.; // (wave 0, lane 0) of the segment
  int cnt = min(kDC, end - pos);
  if (cnt > 0) {
    load_tile(pos, cnt);
    if (w == 0)
      scan_decays(cnt);
  }
  while (cnt > 0) {
    // (every wave is done with the tile before)
    put_tile();
    if (outputs)
      put_state();
    if (w == 0)
      put_decays(cnt);
    lds_barrier();
    const int bad = min(min(first_bad[0], first_bad[1]), min(first_bad[2], first_bad[3]));
    if (bad < cnt) {
      cnt = max(1, bad);
      lds_barrier();
      for (int i = tid; i < (kDC - cnt) * kLdK; i += 256)
        Ks[cnt * kLdK + i] = from_f32<T>(0.f);
      for (int i = tid; i < (kDC - cnt) * kLdV; i += 256)
        Vs[cnt * kLdV + i] = from_f32<T>(0.f);
      if (w == 0)
        put_decays(cnt);
      lds_barrier();
    }
    if (w == 0)
      decay_sum += __shfl(G, cnt - 1);
    Frag<T> qf[kGK];
#pragma unroll
    for (int i = 0; i < kGK; ++i)
      qf[i] = as_frag(qn[i]);
    const int next = pos + cnt, next_cnt = min(kDC, end - next);
    if (next_cnt > 0)
      load_tile(next, next_cnt);

    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    if (outputs && 16 * w < cnt) {
      // o^T of this wave's tokens: tile e, lane (lr, lg) element r is column
      // 32 (e / 2) + 8 lg + 4 (e % 2) + r of token 16 w + lr
      f32x4 O[4] = {zero, zero, zero, zero};
#pragma unroll
      for (int s = 0; s < kGK; ++s)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mma(O[e], load_frag(Ss + val_col(e)(lr) * kLdS + 32 * s + 8 * lg), qf[s]);
      const int i = 16 * w + lr;
      const float ei = eG[i], hi = Ghi[i], lo = Glo[i];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        O[e] *= ei;
      for (int c = 0; c <= w >> 1; ++c) {
        f32x4 P[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          P[t] = zero;
          const int j0 = 32 * c + 16 * t;
          if (j0 > 16 * w)
            continue;
#pragma unroll
          for (int s = 0; s < kGK; ++s)
            mma(P[t], load_frag(Ks + (j0 + lr) * kLdK + 32 * s + 8 * lg), qf[s]);
          const f32x4 jh = *reinterpret_cast<const f32x4 *>(Ghi + j0 + 4 * lg);
          const f32x4 jl = *reinterpret_cast<const f32x4 *>(Glo + j0 + 4 * lg);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float d = __builtin_amdgcn_exp2f((hi - jh[r]) + (lo - jl[r]));
            P[t][r] = j0 + 4 * lg + r <= i ? P[t][r] * d : 0.f;
          }
        }
        const Frag<T> pf = pack_scores(P[0], P[1], T());
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mma(O[e], tr_frag(Vs, kLdV, 32 * c, lr, lg, val_col(e)), pf);
      }
      if (i < cnt) {
        T *op = o + (tok0 + pos + i) * a.os + (int64_t)h * a.dv + col0;
#pragma unroll
        for (int e = 0; e < 4; e += 2) {
          const int c = 32 * (e >> 1) + 8 * lg, left = a.dv - col0 - c;
          float x[8];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            x[r] = O[e][r] * a.scale;
            x[4 + r] = O[e + 1][r] * a.scale;
          }
          if (left >= 8) {
            if constexpr (std::is_same<T, float>::value) {
              *reinterpret_cast<f32x4_any *>(op + c) = f32x4{x[0], x[1], x[2], x[3]};
              *reinterpret_cast<f32x4_any *>(op + c + 4) = f32x4{x[4], x[5], x[6], x[7]};
            } else {
              *reinterpret_cast<u32x4_any *>(op + c) = __builtin_bit_cast(u32x4, pack8(x).v);
            }
          } else {
#pragma unroll
            for (int r = 0; r < 7; ++r)
              if (r < left)
                op[c + r] = from_f32<T>(x[r]);
          }
        }
      }
    }

    const float all = total;
    if (cnt == 1) { // a token alone: its products are exact
      const float x = to_f32(Vs[my_col]);
#pragma unroll
      for (int d = 0; d < kTD; ++d)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          S[d][r] = fmaf(to_f32(Ks[16 * d + 4 * lg + r]), x, all * S[d][r]);
    } else {
#pragma unroll
      for (int d = 0; d < kTD; ++d)
        S[d] *= all;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const f32x4 w0 = *reinterpret_cast<const f32x4 *>(wts + 32 * s + 4 * lg);
        const f32x4 w1 = *reinterpret_cast<const f32x4 *>(wts + 32 * s + 16 + 4 * lg);
        const auto vw = weigh(tr_frag(Vs, kLdV, 32 * s, lr, lg, val_col(w)), w0, w1);
#pragma unroll
        for (int d = 0; d < kTD; ++d) {
          const Frag<T> kf = tr_frag(Ks, kLdK, 32 * s, lr, lg, row_col(d));
#pragma unroll
          for (const auto &p : vw.part)
            mma(S[d], kf, p);
        }
      }
    }
    pos = next;
    cnt = next_cnt;
    if (cnt > 0 && w == 0)
      scan_decays(cnt);
    lds_barrier();
  }

  if (seg < nseg - 1) { // (pass 0)
    float *to = pairs + seg * pair_step;
#pragma unroll
    for (int d = 0; d < kTD; ++d)
      *reinterpret_cast<f32x4 *>(to + d * 1024) = S[d];
    if (tid == 0 && slice == 0)
      a.pair_decay[(pair0 + seg) * a.H + h] = decay_sum;
  } else if (a.fin && kept && col0 + my_col < a.dv) {
#pragma unroll
    for (int d = 0; d < kTD; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * d + 4 * lg + r;
        if (row < a.dk)
          a.fin[global + (int64_t)row * a.dv] = S[d][r];
      }
  }
}

// The states of a sequence's segments from zero become the states after them:
// one by one, an element of the state per lane.
__global__ __launch_bounds__(256) void decay_fold_kernel(SeqTable tab, DecayArgs a, int per) {
  const SeqView sv(tab);
  const int64_t b = blockIdx.x; // (sequence with middle segments, head, 1024 elements)
  const int x = (int)(b % per);
  const int h = (int)(b / per % a.H);
  const int n = sv.find((int)(b / per / a.H), 2);
  const int64_t pair0 = sv.blk(n, 1), last = sv.blk(n + 1, 1);
  const int64_t step = (int64_t)a.H * per * 256;
  f32x4 *p = reinterpret_cast<f32x4 *>(a.pair_state) + (pair0 * a.H + h) * per * 256 + x * 256 +
             threadIdx.x;
  f32x4 S = *p;
  for (int64_t i = pair0 + 1; i < last; ++i) {
    p += step;
    S = *p + exp2_of(a.pair_decay[i * a.H + h]) * S;
    *p = S;
  }
}

// ---- single tokens ----------------------------------------------------------------

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

namespace {
size_t up(size_t x) { return (x + 255) / 256 * 256; }
int padded_dk(int dk) { return dk <= 64 ? 64 : dk <= 128 ? 128 : 256; }
int64_t num_segments(int64_t len, int64_t seg) { return len <= seg ? 1 : (len + seg - 1) / seg; }
} // namespace

DecayPlan decay_plan(int32_t num_seqs, const int64_t *cu, int32_t H, int32_t dk, int32_t dv,
                     int, int32_t split_hint) {
  DecayPlan p{};
  const int64_t slices = (dv + kDCols - 1) / kDCols;
  int64_t longest = 0;
  for (int32_t n = 0; n < num_seqs; ++n)
    longest = std::max(longest, cu[n + 1] - cu[n]);
  const auto whole = [](int64_t x) { return std::max<int64_t>(kDC, (x + kDC - 1) / kDC * kDC); };
  p.seg = whole(longest);
  if (split_hint > 1) {
    p.seg = whole((longest + split_hint - 1) / split_hint);
  } else if (split_hint == 0) {
    const int64_t seg =
        std::max<int64_t>(256, whole((cu[num_seqs] * H * slices + 511) / 512));
    if (longest >= 3 * seg)
      p.seg = seg;
  }
  for (int32_t n = 0; n < num_seqs; ++n)
    p.pairs += num_segments(cu[n + 1] - cu[n], p.seg) - 1;
  size_t at = seq_table_bytes(num_seqs);
  p.off_state = at;
  at = up(at + (size_t)p.pairs * H * slices * kDCols * padded_dk(dk) * sizeof(float));
  p.off_decay = at;
  p.total = up(at + (size_t)p.pairs * H * sizeof(double));
  return p;
}

hipError_t launch_decay(int elt, const DecayCall &c, int32_t num_seqs, const int64_t *cu,
                        const DecayPlan &plan, void *ws, hipStream_t s) {
  DecayArgs a = decay_args(c);
  a.slices = (a.dv + kDCols - 1) / kDCols;
  a.seg = (int32_t)plan.seg;
  a.pair_state = (float *)((uint8_t *)ws + plan.off_state);
  a.pair_decay = (double *)((uint8_t *)ws + plan.off_decay);
  // blocks: segments in each pass, and (2) whether there are pairs to fold
  const auto tiles = [&](int64_t len, int w) -> int64_t {
    const int64_t nseg = num_segments(len, plan.seg);
    return w == 0 ? std::max<int64_t>(1, nseg - 1) : (w == 1 ? nseg - 1 : nseg > 2);
  };
  int64_t total[kCounts];
  if (!seq_totals(num_seqs, cu, tiles, total))
    return hipErrorInvalidConfiguration;
  int64_t grid[2];
  for (int pass = 0; pass < 2; ++pass) {
    grid[pass] = (total[pass] * a.H + 7) / 8 * 8 * a.slices;
    if (grid[pass] * 256 > UINT32_MAX)
      return hipErrorInvalidConfiguration;
  }
  const int per = a.slices * padded_dk(a.dk) / 16; // blocks of a state
  const int64_t fold = total[2] * a.H * per;
  if (fold * 256 > UINT32_MAX)
    return hipErrorInvalidConfiguration;
  SeqTable tab;
  const hipError_t e = make_seq_table(tab, num_seqs, cu, tiles, ws, s);
  if (e != hipSuccess)
    return e;
  const auto run = [&](auto tag, auto dk) {
    using T = decltype(tag);
    const auto chunks = [&](int pass) {
      a.units = total[pass] * a.H;
      decay_chunk_kernel<T, decltype(dk)::value><<<(unsigned)grid[pass], 256, 0, s>>>(
          tab, a, pass, (const T *)c.io.q, (const T *)c.io.k, (const T *)c.io.v, (T *)c.io.o);
    };
    chunks(0);
    if (fold > 0)
      decay_fold_kernel<<<(unsigned)fold, 256, 0, s>>>(tab, a, per);
    if (total[1] > 0)
      chunks(1);
    return hipGetLastError();
  };
  const auto sized = [&](auto tag) {
    using std::integral_constant;
    if (a.dk <= 64)
      return run(tag, integral_constant<int, 64>());
    if (a.dk <= 128)
      return run(tag, integral_constant<int, 128>());
    return run(tag, integral_constant<int, 256>());
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
