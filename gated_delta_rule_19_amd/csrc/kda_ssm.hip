// Selective state space scan: a diagonal linear recurrence with N states per
// channel whose decay, input and read-out all come from the token.
//
//   delta = softplus(dt + bias)          (or dt itself)
//   h[d, n] <- exp(delta A[d, n]) h[d, n] + delta x[d] B[n]
//   y[d]    = sum_n C[n] h[d, n] + Dskip[d] x[d],   then y *= silu(z)
//
// Bound.  Per (token, channel) four elements move, but N states each take a
// product, an exponential and three more products and sums: with N = 16 the
// vector ALU is the limit, not HBM, and the kernel is built to issue nothing
// per state but those five instructions.
//   - A lane owns one channel, so delta, delta x, x, z and y need no
//     broadcast, and B and C are the same for the whole wave: they come as
//     scalar loads from an fp32 table that bc_kernel lays out first (per
//     wave: consecutive tokens, its states' B then C) and enter the products
//     as scalar operands.
//   - The states of a channel are dealt to the S waves of a workgroup, NS
//     each, in registers.  The waves share delta and delta x through LDS (one
//     of them evaluates the softplus of a token) and leave their partial
//     sums of y there, which one wave per token then adds up.
//
// Few chains.  The recurrence is serial in the tokens.  When the sequences'
// channels do not fill the chip, a sequence is cut into segments: the decay
// over a segment is exp(A sum(delta)), so a segment's effect on the state
// that enters it is known from its end state from zero and its sum of delta.
// The first launch runs every first segment (from the true initial state)
// beside the end states of the middle ones; the second runs all others, each
// folding the pairs before it into its entry state.  The middle segments'
// exponentials are evaluated twice, which is what the cut costs.
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

__device__ __forceinline__ float silu(float x) {
  return x * __builtin_amdgcn_rcpf(1.f + exp2_hw(-x * kLog2e));
}

struct SsmArgs {
  int32_t D, N, G, softplus, num_slots;
  int32_t Dg;      // channels per group
  int32_t cb;      // 64-channel blocks per group
  int32_t seg;     // tokens per segment
  int32_t vec_state; // a channel's states may be read and written NS at a time
  int64_t T;       // tokens (rows of the B / C table)
  int64_t xs, dls, zs, ys, Bs, Cs;
  const float *A, *skip, *bias;
  const float *init;
  float *fin;
  const int32_t *slots;
  const float *bc;     // [G][S][T][2 NS]
  float *pend;         // [pairs][G cb][S NS][64] end states of the segments
  float *psum;         // [pairs][G cb][64] their sums of delta
};

// ---- B and C as fp32, per wave ---------------------------------------------------
// Entry (g, w, t): the NS values of B, then of C, that wave w uses for token
// t and group g; states past N read 0.
template <typename T, int NS>
__global__ __launch_bounds__(256) void bc_kernel(const T *__restrict__ B, const T *__restrict__ C,
                                                 int64_t Bs, int64_t Cs, int64_t tokens, int G,
                                                 int N, int S, float *__restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  // neighbouring lanes: the waves of one token, so a row of B is read whole
  const int64_t t = i / (G * S);
  if (t >= tokens)
    return;
  const int gw = (int)(i - t * (G * S)), g = gw / S, w = gw - g * S;
  float v[2 * NS];
#pragma unroll
  for (int k = 0; k < NS; ++k) {
    const int n = w * NS + k;
    v[k] = n < N ? to_f32(B[t * Bs + g * N + n]) : 0.f;
    v[NS + k] = n < N ? to_f32(C[t * Cs + g * N + n]) : 0.f;
  }
  float *o = out + ((int64_t)gw * tokens + t) * (2 * NS);
#pragma unroll
  for (int k = 0; k < 2 * NS; ++k)
    o[k] = v[k];
}

// ---- one segment of one sequence, 64 channels -------------------------------------
template <int NS> struct BcVec {
  float b[NS], c[NS];
};

template <int TT, int S> struct SsmLds {
  f32x4 dx[TT / 2][64];        // (delta, delta x) of two tokens, per channel
  f32x4 y[S][TT / 4][64];      // partial sums of four tokens, per channel
};

// FULL: outputs and (last segment) the final state.  Otherwise only the end
// state from h = 0 and the sum of delta.
template <typename T, int S, int NS, int TT, bool FULL>
__device__ __forceinline__ float scan_segment(const SsmArgs &a, SsmLds<TT, S> &lds,
                                              float (&h)[NS], const float (&A2)[NS],
                                              const KDA_CONST_AS float *bc, const T *x,
                                              const T *dl, const T *z, T *y, int ntok, int wave,
                                              int lane, bool in, float bias, float skip) {
  constexpr int RP = TT / S > 0 ? TT / S : 1; // tokens a wave stages and finishes
  constexpr int kBusy = TT / RP;              // waves that do
  const bool stager = wave < kBusy;
  const int r0 = wave * RP;
  T xr[RP], dr[RP], zr[RP];
  float xk[RP];
  float sum = 0.f;

  const auto fetch = [&](int t0) {
    const int n = ntok - t0;
#pragma unroll
    for (int r = 0; r < RP; ++r) {
      const int64_t t = t0 + r0 + r;
      xr[r] = T(0.f);
      dr[r] = T(0.f);
      if (stager && r0 + r < n && in) {
        xr[r] = x[t * a.xs];
        dr[r] = dl[t * a.dls];
      }
    }
  };

  fetch(0);
  for (int t0 = 0; t0 < ntok; t0 += TT) {
    const int n = min(TT, ntok - t0);
    // stage this tile's delta and delta x
    if (stager) {
      float pair[RP][2];
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        const float xv = to_f32(xr[r]);
        float d = to_f32(dr[r]) + bias;
        if (a.softplus)
          d = softplus(d);
        xk[r] = xv;
        pair[r][0] = d;
        pair[r][1] = d * xv;
      }
      if constexpr (RP % 2 == 0) {
#pragma unroll
        for (int r = 0; r < RP; r += 2)
          lds.dx[(r0 + r) / 2][lane] =
              f32x4{pair[r][0], pair[r][1], pair[r + 1][0], pair[r + 1][1]};
      } else {
        float *p = reinterpret_cast<float *>(&lds.dx[r0 / 2][lane]) + (r0 & 1) * 2;
        p[0] = pair[0][0];
        p[1] = pair[0][1];
      }
    }
    __syncthreads();

    // in flight during the recurrence: the next tile's inputs, this one's gate
    fetch(t0 + TT);
    if (FULL && z) {
#pragma unroll
      for (int r = 0; r < RP; ++r)
        if (stager && r0 + r < n && in)
          zr[r] = z[(int64_t)(t0 + r0 + r) * a.zs];
    }

    const KDA_CONST_AS float *tb = bc + (int64_t)t0 * (2 * NS);
    int t = 0;
    for (; t + 4 <= n; t += 4) {
      const f32x4 p0 = lds.dx[t / 2][lane], p1 = lds.dx[t / 2 + 1][lane];
      const float d[4] = {p0[0], p0[2], p1[0], p1[2]};
      const float u[4] = {p0[1], p0[3], p1[1], p1[3]};
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const KDA_CONST_AS float *row = tb + (t + k) * (2 * NS);
#pragma unroll
        for (int i = 0; i < NS; ++i) {
          h[i] = fmaf(exp2_hw(d[k] * A2[i]), h[i], u[k] * row[i]);
          if (FULL)
            acc[k] = fmaf(row[NS + i], h[i], acc[k]);
        }
        if (!FULL)
          sum += d[k];
      }
      if (FULL)
        lds.y[wave][t / 4][lane] = acc;
    }
    for (; t < n; ++t) { // the last tokens of a segment, one by one
      const f32x4 p0 = lds.dx[t / 2][lane];
      const float d = t & 1 ? p0[2] : p0[0], u = t & 1 ? p0[3] : p0[1];
      const KDA_CONST_AS float *row = tb + t * (2 * NS);
      float acc = 0.f;
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        h[i] = fmaf(exp2_hw(d * A2[i]), h[i], u * row[i]);
        if (FULL)
          acc = fmaf(row[NS + i], h[i], acc);
      }
      if (FULL)
        reinterpret_cast<float *>(&lds.y[wave][t / 4][lane])[t & 3] = acc;
      else
        sum += d;
    }
    __syncthreads();

    if (FULL && stager) {
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        const int row = r0 + r;
        if (row >= n)
          break;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < S; ++w)
          v += reinterpret_cast<const float *>(&lds.y[w][row / 4][lane])[row & 3];
        v = fmaf(skip, xk[r], v);
        if (z)
          v *= silu(to_f32(zr[r]));
        if (in)
          y[(int64_t)(t0 + row) * a.ys] = from_f32<T>(v);
      }
    }
  }
  return sum;
}

// pass 0: first segments (full) and middle ones (end states); pass 1: every
// segment but the first, in full.
template <typename T, int S, int NS, int TT>
__global__ __launch_bounds__(64 * S) void ssm_kernel(SeqTable tab, SsmArgs a, int pass,
                                                     const T *__restrict__ x,
                                                     const T *__restrict__ dl,
                                                     const T *__restrict__ z,
                                                     T *__restrict__ y) {
  __shared__ SsmLds<TT, S> lds;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int blocks = a.G * a.cb;
  const int sb = blockIdx.x / blocks, gc = blockIdx.x - sb * blocks;
  const int g = gc / a.cb, cbi = gc - g * a.cb;
  const SeqView seqs(tab);
  const int n = seqs.find(sb, pass);
  const int len = seqs.len(n);
  const int64_t tok0 = seqs.tok0(n);
  const int nseg = len > a.seg ? (len + a.seg - 1) / a.seg : 1;
  const int j = sb - seqs.blk(n, pass) + pass;
  const int64_t pair0 = seqs.blk(n, 1); // its nseg - 1 transition pairs
  const int s0 = j * a.seg, ntok = min(a.seg, len - s0);
  const bool full = pass == 1 || j == 0;

  const int dg = cbi * 64 + lane; // channel in its group
  const bool in = dg < a.Dg;
  const int64_t d = (int64_t)g * a.Dg + dg;
  const int n0 = wave * NS;

  float A2[NS], h[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    A2[i] = in && n0 + i < a.N ? a.A[d * a.N + n0 + i] * kLog2e : 0.f;
    h[i] = 0.f;
  }
  int64_t slot = n;
  bool kept = true;
  if (a.slots) {
    slot = a.slots[n];
    kept = slot >= 0 && slot < a.num_slots;
  }
  if (j == 0) {
    if (a.init && kept && in) {
      const float *p = a.init + (slot * a.D + d) * a.N + n0;
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (n0 + i < a.N)
          h[i] = p[i];
    }
  } else if (full) {
    const float *pe = a.pend + (((pair0 + j - 1) * blocks + gc) * S + wave) * NS * 64 + lane;
#pragma unroll
    for (int i = 0; i < NS; ++i)
      h[i] = pe[i * 64];
  }

  const KDA_CONST_AS float *bc =
      (const KDA_CONST_AS float *)(uintptr_t)(a.bc +
                                              (((int64_t)g * S + wave) * a.T + tok0 + s0) * 2 * NS);
  const int64_t t0 = tok0 + s0;
  const float bias = in && a.bias ? a.bias[d] : 0.f;
  const float skip = in && a.skip ? a.skip[d] : 0.f;
  float sum = 0.f;
  if (full)
    scan_segment<T, S, NS, TT, true>(a, lds, h, A2, bc, x + t0 * a.xs + d, dl + t0 * a.dls + d,
                                     z ? z + t0 * a.zs + d : nullptr, y + t0 * a.ys + d, ntok,
                                     wave, lane, in, bias, skip);
  else
    sum = scan_segment<T, S, NS, TT, false>(a, lds, h, A2, bc, x + t0 * a.xs + d,
                                            dl + t0 * a.dls + d, nullptr, nullptr, ntok, wave,
                                            lane, in, bias, skip);

  if (j == nseg - 1) {
    if (a.fin && kept && in) {
      float *p = a.fin + (slot * a.D + d) * a.N + n0;
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (n0 + i < a.N)
          p[i] = h[i];
    }
  } else if (pass == 0) {
    float *pe = a.pend + (((pair0 + j) * blocks + gc) * S + wave) * NS * 64 + lane;
#pragma unroll
    for (int i = 0; i < NS; ++i)
      pe[i * 64] = h[i];
    if (j > 0 && wave == 0)
      a.psum[((pair0 + j) * blocks + gc) * 64 + lane] = sum;
  }
}

// ---- all states of a channel in one lane --------------------------------------------
// No exchange between waves and no barrier: a wave streams its 64 channels'
// tokens, U at a time with the next U tokens' inputs in flight.  B and C come
// through an LDS area of the wave's own: kBcTokens tokens' values, widened,
// loaded a whole area ahead; every lane then reads the same 16 bytes.
constexpr int kBcTokens = 16;

template <int NS> struct LaneBc {
  float v[2][kBcTokens][2 * NS]; // B then C of each token, two areas in turn
};

// One element per lane of a row of channels; lanes at or past `bytes` (the
// row's end, or 0 for a token past the segment) read 0 and write nothing.
// The loaded bits are kept as they are and widened where they are used, so
// that nothing waits for a load before then.
template <typename T> struct RawOf { typedef unsigned short type; };
template <> struct RawOf<float> { typedef unsigned type; };
template <typename T> using Raw = typename RawOf<T>::type;
__device__ __forceinline__ float widen(unsigned short r) {
  return __builtin_bit_cast(float, (unsigned)r << 16);
}
__device__ __forceinline__ float widen(unsigned r) { return __builtin_bit_cast(float, r); }
__device__ __forceinline__ unsigned short buffer_raw(__amdgpu_buffer_rsrc_t r, int voff,
                                                     const bf16 *) {
  return __builtin_amdgcn_raw_buffer_load_b16(r, voff, 0, 0);
}
__device__ __forceinline__ unsigned buffer_raw(__amdgpu_buffer_rsrc_t r, int voff,
                                               const float *) {
  return __builtin_amdgcn_raw_buffer_load_b32(r, voff, 0, 0);
}
template <typename T>
__device__ __forceinline__ Raw<T> row_load(const T *p, int bytes, int lane) {
  return buffer_raw(buffer_rsrc(p, bytes), lane * (int)sizeof(T), p);
}
template <typename T>
__device__ __forceinline__ void row_store(T *p, int bytes, int lane, float v) {
  buffer_store(buffer_rsrc(p, bytes), from_f32<T>(v), lane * (int)sizeof(T), 0);
}

// The values of B and C a lane brings in per area: state i of every kStep-th
// token.  Tokens past the segment and states past N read 0.
template <typename T, int NS> struct BcLoader {
  static constexpr int kStep = 64 / NS;
  static constexpr int kPer = kBcTokens / kStep;
  const T *B, *C;
  int64_t Bs, Cs;
  int t0, i;
  bool on;
  Raw<T> b[kPer], c[kPer];

  __device__ __forceinline__ BcLoader(const T *B_, const T *C_, int64_t Bs_, int64_t Cs_, int N,
                                      int lane)
      : B(B_), C(C_), Bs(Bs_), Cs(Cs_) {
    t0 = lane / NS;
    i = lane % NS;
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
      b[k] = buffer_raw(rb, ok ? (t * (int)Bs + i) * (int)sizeof(T) : -1, B);
      c[k] = buffer_raw(rc, ok ? (t * (int)Cs + i) * (int)sizeof(T) : -1, C);
    }
  }
  __device__ __forceinline__ void put(float (*area)[2 * NS]) const {
#pragma unroll
    for (int k = 0; k < kPer; ++k) {
      area[t0 + k * kStep][i] = widen(b[k]);
      area[t0 + k * kStep][NS + i] = widen(c[k]);
    }
  }
};

template <typename T, int NS, bool FULL>
__device__ __forceinline__ float lane_segment(const SsmArgs &a, LaneBc<NS> &lds, float (&h)[NS],
                                              const float (&A2)[NS], BcLoader<T, NS> bc,
                                              const T *x, const T *dl, const T *z, T *y, int ntok,
                                              int row_bytes, int lane, float bias, float skip) {
  constexpr int U = 4;
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
    float(*area)[2 * NS] = lds.v[(b0 / kBcTokens) & 1];
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
        xk[k] = widen(xr[k]);
        d[k] = widen(dr[k]) + bias;
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
          gate[k] = silu(widen(zr[k]));
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
            cv = *reinterpret_cast<const f32x4 *>(row + NS + q);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            h[q + i] = fmaf(exp2_hw(d[k] * A2[q + i]), h[q + i], u * bv[i]);
            if (FULL)
              acc[k] = fmaf(cv[i], h[q + i], acc[k]);
          }
        }
        if (FULL)
          acc[k] = fmaf(skip, xk[k], acc[k]);
        else
          sum += d[k];
      }
      if (FULL) {
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
  __shared__ LaneBc<NS> lds[4];
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
    A2[i] = in && i < a.N ? a.A[d * a.N + i] * kLog2e : 0.f;
    h[i] = 0.f;
  }
  int64_t slot = n;
  bool kept = true;
  if (a.slots) {
    slot = a.slots[n];
    kept = slot >= 0 && slot < a.num_slots;
  }
  if (j == 0) {
    if (a.init && kept && in) {
      const float *p = a.init + (slot * a.D + d) * a.N;
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (i < a.N)
          h[i] = p[i];
    }
  } else if (pass == 1) {
    const float *pe = a.pend + ((pair0 + j - 1) * blocks + gc) * NS * 64 + lane;
#pragma unroll
    for (int i = 0; i < NS; ++i)
      h[i] = pe[i * 64];
  }

  const int64_t t0 = tok0 + s0;
  const BcLoader<T, NS> bc(B + t0 * a.Bs + g * a.N, C + t0 * a.Cs + g * a.N, a.Bs, a.Cs, a.N,
                           lane);
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
      float *p = a.fin + (slot * a.D + d) * a.N;
#pragma unroll
      for (int i = 0; i < NS; ++i)
        if (i < a.N)
          p[i] = h[i];
    }
  } else if (pass == 0) {
    float *pe = a.pend + ((pair0 + j) * blocks + gc) * NS * 64 + lane;
#pragma unroll
    for (int i = 0; i < NS; ++i)
      pe[i * 64] = h[i];
    if (j > 0)
      a.psum[((pair0 + j) * blocks + gc) * 64 + lane] = sum;
  }
}

// ---- the segments' entry states -------------------------------------------------------
// pend[0] is the state after the first segment; pend[j] becomes
// pend[j] + exp(A sum_j) pend[j - 1], the state after segment j.  One wave per
// (cut sequence, 64 channels, state); the pairs of 16 segments are in flight
// together.
__global__ __launch_bounds__(256) void ssm_fold_kernel(SeqTable tab, SsmArgs a, int SN) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int blocks = a.G * a.cb;
  const int64_t wv = (int64_t)blockIdx.x * 4 + wave;
  const int n = (int)(wv / ((int64_t)blocks * SN));
  if (n >= tab.num_seqs)
    return;
  const int rest = (int)(wv - (int64_t)n * blocks * SN);
  const int gc = rest / SN, i = rest - gc * SN;
  const SeqView seqs(tab);
  const int64_t pair0 = seqs.blk(n, 1);
  const int pairs = (int)(seqs.blk(n + 1, 1) - pair0);
  if (pairs <= 1 || i >= a.N)
    return;
  const int g = gc / a.cb, dg = (gc - g * a.cb) * 64 + lane;
  const float A2 = dg < a.Dg ? a.A[((int64_t)g * a.Dg + dg) * a.N + i] * kLog2e : 0.f;
  float *pe = a.pend + ((pair0 * blocks + gc) * SN + i) * 64 + lane;
  const float *ps = a.psum + (pair0 * blocks + gc) * 64 + lane;
  const int64_t pstep = (int64_t)blocks * SN * 64, sstep = (int64_t)blocks * 64;
  float h = pe[0];
  for (int j = 1; j < pairs; j += 16) {
    float e[16], sd[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int q = min(j + k, pairs - 1);
      e[k] = pe[q * pstep];
      sd[k] = ps[q * sstep];
    }
#pragma unroll
    for (int k = 0; k < 16; ++k)
      if (j + k < pairs) {
        h = fmaf(exp2_hw(sd[k] * A2), h, e[k]);
        pe[(j + k) * pstep] = h;
      }
  }
}

// ---- single tokens ------------------------------------------------------------------
// A channel's N states lie side by side on `lanes` neighbouring lanes, VEC on
// each, K times; a wave takes 64 / lanes channels of one row.  The state is
// read once and written once: bound by HBM.
struct StepArgs {
  int32_t D, N, Dg, softplus, num_slots, lanes_log2;
  int64_t cw, waves; // waves per row, all waves
  int64_t xs, dls, zs, ys, Bs, Cs;
  const float *A, *skip, *bias;
  float *state;
  const int32_t *slots;
};

template <typename T, int VEC, int K>
__global__ __launch_bounds__(256) void ssm_step_kernel(StepArgs a, const T *__restrict__ x,
                                                       const T *__restrict__ dl,
                                                       const T *__restrict__ B,
                                                       const T *__restrict__ C,
                                                       const T *__restrict__ z, T *y) {
  const int64_t wv = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (wv >= a.waves)
    return;
  const int row = (int)(wv / a.cw);
  const int64_t slot = a.slots ? a.slots[row] : row;
  if (slot < 0 || slot >= a.num_slots)
    return; // a padding row: nothing is read or written
  const int lanes = 1 << a.lanes_log2;
  const int lane = threadIdx.x & (lanes - 1);
  const int64_t d =
      (wv - row * a.cw) * (64 >> a.lanes_log2) + ((threadIdx.x & 63) >> a.lanes_log2);
  const bool in = d < a.D;
  const int64_t g = in ? d / a.Dg : 0;

  float h[K][VEC], A[K][VEC], b[K][VEC], c[K][VEC];
  float *st = a.state + (slot * a.D + d) * a.N;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int n = (k * lanes + lane) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      h[k][i] = A[k][i] = b[k][i] = c[k][i] = 0.f;
    if (in && n < a.N) {
      if constexpr (VEC == 4) {
        const f32x4 hv = *reinterpret_cast<const f32x4 *>(st + n);
        const f32x4 av = *reinterpret_cast<const f32x4 *>(a.A + d * a.N + n);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          h[k][i] = hv[i];
          A[k][i] = av[i];
        }
      } else {
        h[k][0] = st[n];
        A[k][0] = a.A[d * a.N + n];
      }
#pragma unroll
      for (int i = 0; i < VEC; ++i) {
        b[k][i] = to_f32(B[row * a.Bs + g * a.N + n + i]);
        c[k][i] = to_f32(C[row * a.Cs + g * a.N + n + i]);
      }
    }
  }
  float xv = 0.f, dv = 0.f;
  if (in) {
    xv = to_f32(x[row * a.xs + d]);
    dv = to_f32(dl[row * a.dls + d]) + (a.bias ? a.bias[d] : 0.f);
  }
  if (a.softplus)
    dv = softplus(dv);
  const float u = dv * xv;
  float acc = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int n = (k * lanes + lane) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) {
      h[k][i] = fmaf(exp2_hw(dv * (A[k][i] * kLog2e)), h[k][i], u * b[k][i]);
      acc = fmaf(c[k][i], h[k][i], acc);
    }
    if (in && n < a.N) {
      if constexpr (VEC == 4)
        *reinterpret_cast<f32x4 *>(st + n) = f32x4{h[k][0], h[k][1], h[k][2], h[k][3]};
      else
        st[n] = h[k][0];
    }
  }
  for (int m = 0; m < a.lanes_log2; ++m)
    acc += __shfl_xor(acc, 1 << m);
  if (in && lane == 0) {
    float v = fmaf(a.skip ? a.skip[d] : 0.f, xv, acc);
    if (z)
      v *= silu(to_f32(z[row * a.zs + d]));
    y[row * a.ys + d] = from_f32<T>(v);
  }
}

// ---- host ---------------------------------------------------------------------------
// Waves per workgroup and states per wave of the wide kernel (states dealt to
// the waves), and states of the lane kernel.
struct Shape {
  int S, NS;
};
Shape wide_shape(int N) {
  if (N <= 8)
    return {2, 4};
  if (N <= 16)
    return {4, 4};
  if (N <= 32)
    return {8, 4};
  if (N <= 64)
    return {16, 4};
  return {16, 8};
}
int lane_states(int N) { return N <= 4 ? 4 : (N <= 8 ? 8 : 16); }
constexpr int kLaneMaxStates = 16;

constexpr size_t kAlign = 256;
size_t up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

int64_t chan_blocks(int32_t D, int32_t G) { return (int64_t)G * ((D / G + 63) / 64); }

template <typename F> hipError_t with_wide(Shape sh, F &&f) {
  using std::integral_constant;
  using i2 = integral_constant<int, 2>;
  using i4 = integral_constant<int, 4>;
  using i8 = integral_constant<int, 8>;
  using i16 = integral_constant<int, 16>;
  using i32 = integral_constant<int, 32>;
  if (sh.NS == 8)
    return f(i16(), i8(), i16());
  switch (sh.S) {
  case 2: return f(i2(), i4(), i16());
  case 4: return f(i4(), i4(), i32());
  case 8: return f(i8(), i4(), i32());
  default: return f(i16(), i4(), i16());
  }
}

template <typename F> hipError_t with_lane(int NS, F &&f) {
  using std::integral_constant;
  if (NS == 4)
    return f(integral_constant<int, 4>());
  if (NS == 8)
    return f(integral_constant<int, 8>());
  return f(integral_constant<int, 16>());
}

} // namespace

int64_t ssm_num_segments(int64_t len, const SsmPlan &p) {
  return len > p.seg ? (len + p.seg - 1) / p.seg : 1;
}

SsmPlan ssm_plan(int32_t num_seqs, const int64_t *cu, int32_t D, int32_t N, int32_t G,
                 int32_t split_hint) {
  SsmPlan p{};
  const int64_t blocks = chan_blocks(D, G), tokens = cu[num_seqs];
  int64_t longest = 0;
  for (int32_t n = 0; n < num_seqs; ++n)
    longest = std::max(longest, cu[n + 1] - cu[n]);
  // multiples of 32 tokens: whole tiles
  const auto whole = [](int64_t x) { return std::max<int64_t>(32, (x + 31) / 32 * 32); };
  const Shape sh = wide_shape(N);
  p.seg = whole(longest);
  p.lane = N <= kLaneMaxStates;
  if (split_hint > 1) {
    p.seg = whole((longest + split_hint - 1) / split_hint);
  } else if (split_hint == 0) {
    const int64_t want = p.lane ? tokens * blocks / 4096 : tokens * blocks / 1024;
    p.seg = std::min(p.seg, std::max<int64_t>(64, whole(want)));
  }
  p.S = p.lane ? 1 : sh.S;
  p.NS = p.lane ? lane_states(N) : sh.NS;
  for (int32_t n = 0; n < num_seqs; ++n)
    p.pairs += ssm_num_segments(cu[n + 1] - cu[n], p) - 1;
  const size_t SN = (size_t)p.S * p.NS;
  size_t o = seq_table_bytes(num_seqs);
  p.off_bc = o;
  o = up(o + (p.lane ? 0 : (size_t)tokens * G * SN * 2 * sizeof(float)));
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
  const int SN = plan.S * plan.NS;
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
  a.T = tokens;
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
  a.bc = (const float *)(w + plan.off_bc);
  a.pend = (float *)(w + plan.off_end);
  a.psum = (float *)(w + plan.off_sum);

  const auto tiles = [&](int64_t len, int pass) -> int64_t {
    const int64_t nseg = ssm_num_segments(len, plan);
    return pass ? nseg - 1 : std::max<int64_t>(1, nseg - 1);
  };
  int64_t total[2];
  if (!seq_totals(num_seqs, cu, tiles, total))
    return hipErrorInvalidConfiguration;
  // workgroups per (segment, all channels) and threads per workgroup
  const int64_t per = plan.lane ? (blocks + 3) / 4 : blocks;
  const int64_t threads = plan.lane ? 256 : 64 * plan.S;
  for (int pass = 0; pass < 2; ++pass)
    if (total[pass] * per > INT32_MAX || total[pass] * per * threads > UINT32_MAX)
      return hipErrorInvalidConfiguration;
  const int64_t bcb = (tokens * c.G * plan.S + 255) / 256;
  const int64_t fold = plan.pairs > 0 ? ((int64_t)num_seqs * blocks * SN + 3) / 4 : 0;
  if (bcb * 256 > UINT32_MAX || fold * 256 > UINT32_MAX)
    return hipErrorInvalidConfiguration;
  SeqTable tab;
  hipError_t e = make_seq_table(tab, num_seqs, cu, tiles, ws, s);
  if (e != hipSuccess)
    return e;

  const auto typed = [&](auto tag) {
    using T = decltype(tag);
    const T *x = (const T *)c.x, *dl = (const T *)c.delta, *z = (const T *)c.z;
    T *y = (T *)c.y;
    const auto table = [&](auto ns) {
      if (tokens > 0)
        bc_kernel<T, decltype(ns)::value><<<(unsigned)bcb, 256, 0, s>>>(
            (const T *)c.B, (const T *)c.C, c.B_stride, c.C_stride, tokens, c.G, c.N, plan.S,
            (float *)(w + plan.off_bc));
    };
    const auto passes = [&](auto &&run) {
      run(0, (unsigned)(total[0] * per));
      if (total[1] > 0) {
        ssm_fold_kernel<<<(unsigned)fold, 256, 0, s>>>(tab, a, SN);
        run(1, (unsigned)(total[1] * per));
      }
      return hipGetLastError();
    };
    if (plan.lane)
      return with_lane(plan.NS, [&](auto ns) {
        return passes([&](int pass, unsigned grid) {
          ssm_lane_kernel<T, decltype(ns)::value>
              <<<grid, 256, 0, s>>>(tab, a, pass, x, dl, z, (const T *)c.B, (const T *)c.C, y);
        });
      });
    return with_wide({plan.S, plan.NS}, [&](auto cs, auto ns, auto tt) {
      table(ns);
      return passes([&](int pass, unsigned grid) {
        ssm_kernel<T, decltype(cs)::value, decltype(ns)::value, decltype(tt)::value>
            <<<grid, 64 * decltype(cs)::value, 0, s>>>(tab, a, pass, x, dl, z, y);
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
  const bool wide = c.N % 4 == 0; // (the state and A are 16-byte aligned)
  const int need = wide ? c.N / 4 : c.N;
  while ((1 << a.lanes_log2) < need && a.lanes_log2 < 6)
    ++a.lanes_log2;
  const int per = 64 >> a.lanes_log2;
  a.cw = (c.D + per - 1) / per;
  a.waves = a.cw * rows;
  if ((a.waves + 3) / 4 * 256 > UINT32_MAX)
    return hipErrorInvalidConfiguration;
  const auto run = [&](auto tag, auto vec, auto k) {
    using T = decltype(tag);
    ssm_step_kernel<T, decltype(vec)::value, decltype(k)::value>
        <<<(unsigned)((a.waves + 3) / 4), 256, 0, s>>>(a, (const T *)c.x, (const T *)c.delta,
                                                       (const T *)c.B, (const T *)c.C,
                                                       (const T *)c.z, (T *)c.y);
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
