// Beam search's selection over beams and vocabulary, and the reordering of the
// states that the chosen beams continue from.
//
// Selection.  Token v of beam w is worth score[w] + x[w, v] - lse[w], with
// lse[w] = log(sum_u exp(x[w, u])).  Within a beam that is the order of the
// logits themselves, so each logit is read once, by the first of two kernels:
//   part kernel: a workgroup holds 16 KB of one beam's logits in registers and
//     finds their maximum, the sum of exp(x - maximum), and the K largest in
//     order (larger first, equal ones by the lower token);
//   merge kernel: a workgroup per batch joins the parts' sums into lse, values
//     the parts' candidates in 64 bits, and takes the K best of them.
// The part kernel finds its K largest without sorting them all: the K-th
// largest of the lanes' own maxima has K elements at or above it, so only what
// is above it is collected and ranked (elements of fewer than K lanes), and
// where these are fewer than K the first ones equal to it follow.  A logit of
// -inf is never collected: where fewer than K candidates are above -inf, the
// lowest (w, v) that are not among them fill up the selection.
//
// Sums: exp from fp32 with its argument's rounding put back (about 2^-23
// relative a term), four of them added in fp32 and the fours in 64 bits; so two
// beams' candidates change places only if their values are that near.
//
// Reordering.  One pass in place: a lane holds the same 16 bytes of all rows
// of its group that change, loads them all, then stores them, so no order of
// rows can overwrite what is still to be read, whatever the table.
#include "kda_block.h"
#include "kda_device.h"

#include <algorithm>
#include <type_traits>

namespace kda {

namespace {

// ---- selection: parts ---------------------------------------------------------

constexpr int kPartBytes = 16384; // of logits per workgroup
template <typename T> constexpr int kPart = kPartBytes / (int)sizeof(T);

struct BeamArgs {
  int32_t B, W, V, K, eos, order;
  int32_t parts;
  int32_t lanes_log2;           // lanes that join a beam's parts
  double inv_parts, inv_places; // 1 / parts, 1 / (W parts)
  int64_t row_stride;
};

struct Cand { // a candidate of a part: token < 0 marks none
  float x;
  int32_t v;
};
struct PartSum {
  double sum;
  float max;
  int32_t pad;
};

// The order of a type's values as unsigned numbers (-0 as 0).
template <typename T> struct OrderOf;
template <> struct OrderOf<bf16> {
  static constexpr int kBits = 16;
  static __device__ __forceinline__ uint32_t make(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.f) >> 16;
    return u ^ (u & 0x8000u ? 0xffffu : 0x8000u);
  }
  static __device__ __forceinline__ float value(uint32_t u) {
    return __builtin_bit_cast(float, (u ^ (u & 0x8000u ? 0x8000u : 0xffffu)) << 16);
  }
};
template <> struct OrderOf<float> {
  static constexpr int kBits = 32;
  static __device__ __forceinline__ uint32_t make(float x) {
    const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.f);
    return u ^ (u & 0x80000000u ? 0xffffffffu : 0x80000000u);
  }
  static __device__ __forceinline__ float value(uint32_t u) {
    return __builtin_bit_cast(float, u ^ (u & 0x80000000u ? 0x80000000u : 0xffffffffu));
  }
};
// Keys in the order of the selection: the value's order above the complement
// of the place in the part.
template <typename T> struct KeyOf {
  typedef std::conditional_t<sizeof(T) == 2, uint32_t, uint64_t> type;
  static constexpr int kPlaces = kPart<T>;
  static __device__ __forceinline__ type make(float x, int at) {
    return (type)OrderOf<T>::make(x) * kPlaces + (type)(kPlaces - 1 - at);
  }
  static __device__ __forceinline__ int place(type k) {
    return kPlaces - 1 - (int)(k & (kPlaces - 1));
  }
  static __device__ __forceinline__ float value(type k) {
    return OrderOf<T>::value((uint32_t)(k / kPlaces));
  }
};
// eight elements with their type's alignment only
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_any __attribute__((aligned(4)));
__device__ __forceinline__ void load8(const bf16 *p, float *x) {
  widen8(*reinterpret_cast<const u32x4_any *>(p), x);
}
__device__ __forceinline__ void load8(const float *p, float *x) {
  const f32x4 a = *reinterpret_cast<const f32x4_any *>(p);
  const f32x4 b = *reinterpret_cast<const f32x4_any *>(p + 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[i] = a[i];
    x[4 + i] = b[i];
  }
}

// the largest of a wave's values
template <int CTRL, int ROWS> __device__ __forceinline__ float dpp_max(float x) {
  const int u = __builtin_bit_cast(int, x);
  return fmaxf(x, __builtin_bit_cast(
                      float, __builtin_amdgcn_update_dpp(u, u, CTRL, ROWS, 0xf, false)));
}
__device__ __forceinline__ float wave_max(float x) {
  x = dpp_max<0x111, 0xf>(x); // 1, 2, 4, 8 lanes within rows of 16
  x = dpp_max<0x112, 0xf>(x);
  x = dpp_max<0x114, 0xf>(x);
  x = dpp_max<0x118, 0xf>(x);
  x = dpp_max<0x142, 0xa>(x); // ends of rows to those behind
  x = dpp_max<0x143, 0xc>(x);
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), 63));
}
// The K-th largest of 256 numbers, four a lane, bit by bit from the top, or with
// `parts` any number that parts the K largest from the others.
__device__ __forceinline__ uint32_t kth_of_256(const uint32_t (&of)[4], int K, int bits,
                                               bool &parts) {
  uint32_t low = 0;
  parts = false;
  for (int bit = bits - 1; bit >= 0 && !parts; --bit) {
    const uint32_t at = low | 1u << bit;
    int reach = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      reach += __popcll(__ballot(of[i] >= at));
    if (reach >= K) {
      low = at;
      parts = reach == K;
    }
  }
  return low;
}

// exp(d) for d <= 0 (0 from -104 down, -inf too; NaN for NaN): exp2 of the
// rounded product t with log2(e), and to first order what t leaves of d,
// d - t ln(2) in one operation (fp32's ln(2) is 3e-9 off).
__device__ __forceinline__ float exp_neg(float d) {
  d = __builtin_elementwise_maximum(d, -104.f);
  const float t = d * 0x1.715476p+0f;
  const float e = __builtin_amdgcn_exp2f(t);
  return fmaf(e, fmaf(t, -0x1.62e43p-1f, d), e);
}

// 64 x 8 beams of 128001 bf16 logits: 8192 workgroups, 41 us (3.2 TB/s), bound
// by the vector units: some 520 instructions a wave for 32 logits a lane, nine
// for each exp with its sum, about 33 us; the loads of the eight workgroups of a
// CU hide behind them.  The threshold from 256 lanes' maxima by bits costs one
// wave 16 (32) steps of four ballots; from groups of each wave's lanes, and an
// LDS atomic for each element found, all of it took 66 us.
template <typename T>
__global__ __launch_bounds__(256) void beam_part_kernel(BeamArgs a, const T *__restrict__ logits,
                                                        Cand *__restrict__ cand,
                                                        PartSum *__restrict__ sums) {
  typedef KeyOf<T> KO;
  typedef typename KO::type Key;
  typedef OrderOf<T> Order;
  constexpr int kN = kPart<T> / 256 / 8; // groups of eight a lane
  __shared__ Key keys[KDA_BEAM_MAX * 8 * kN];
  __shared__ float lane_max[256], wave_top[4];
  __shared__ double lane_sum[256];
  __shared__ float bar_at, tie_at;
  __shared__ int count, wave_ties[2][4];
  const int row = blockIdx.x / a.parts, part = blockIdx.x - row * a.parts;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int first = part * kPart<T>;
  const int left = a.V - first; // elements from the part's start on
  const T *p = logits + row * a.row_stride + first;

  float x[kN][8];
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    const int c = (i * 256 + tid) * 8;
    if (c + 8 <= left) {
      load8(p + c, x[i]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        x[i][j] = c + j < left ? to_f32(p[c + j]) : -__builtin_inff();
    }
  }
  float m = -__builtin_inff(), most[kN]; // of each eight
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    most[i] = x[i][0];
#pragma unroll
    for (int j = 1; j < 8; ++j)
      most[i] = fmaxf(most[i], x[i][j]); // (a NaN is found by the sum)
    m = fmaxf(m, most[i]);
  }
  lane_max[tid] = m;
  m = wave_max(m);
  if (lane == 0)
    wave_top[wv] = m;
  if (tid == 0)
    count = 0;
  __syncthreads();
  const float top = fmaxf(fmaxf(wave_top[0], wave_top[1]), fmaxf(wave_top[2], wave_top[3]));

  if (wv == 0) {
    uint32_t of[4];
    bool parts;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      of[i] = Order::make(lane_max[i * 64 + lane]);
    const uint32_t low = kth_of_256(of, a.K, Order::kBits, parts);
    if (lane == 0) {
      // (the next number above infinity is a NaN: nothing reaches it)
      bar_at = Order::value(parts ? low : low + 1);
      const bool none = parts || low <= Order::make(-__builtin_inff());
      tie_at = none ? __builtin_nanf("") : Order::value(low);
    }
  }

  double sum = 0.;
  if (top > -__builtin_inff()) {
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
      for (int j = 0; j < 8; j += 4) {
        const auto e = [&](int l) { return exp_neg(x[i][j + l] - top); };
        sum += (double)((e(0) + e(1)) + (e(2) + e(3)));
      }
  } else {
    // nothing, unless a NaN hides there
#pragma unroll
    for (int i = 0; i < kN; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (x[i][j] != x[i][j])
          sum = __builtin_nan("");
  }
  lane_sum[tid] = sum;
  __syncthreads();

  // what reaches the threshold, in any order: the keys are ordered below
  const float bar = bar_at, tie = tie_at;
#pragma unroll
  for (int i = 0; i < kN; ++i)
    if (most[i] >= bar) {
      int n = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        n += x[i][j] >= bar;
      int at = atomicAdd(&count, n);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (x[i][j] >= bar)
          keys[at++] = KO::make(x[i][j], (i * 256 + tid) * 8 + j);
    }
  if (wv == 3) { // (each lane's sum is there since the barrier)
    sum = (lane_sum[lane] + lane_sum[64 + lane]) + (lane_sum[128 + lane] + lane_sum[192 + lane]);
#pragma unroll
    for (int b = 1; b < 64; b <<= 1)
      sum += __shfl_xor(sum, b);
    if (lane == 0)
      sums[blockIdx.x] = {sum, top, 0};
  }
  __syncthreads();

  const int n = __builtin_amdgcn_readfirstlane(count);
  Cand *out = cand + (int64_t)blockIdx.x * a.K;
  for (int i = tid; i < n; i += 256) { // by rank
    const Key k = keys[i];
    int above = 0;
    for (int j = 0; j < n; ++j)
      above += keys[j] > k;
    if (above < a.K)
      out[above] = {KO::value(k), first + KO::place(k)};
  }
  int have = n;
  if (have < a.K && tie == tie) { // the first elements that are equal to it
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      int mine = 0, upto;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        mine += x[i][j] == tie;
      upto = mine; // of the lanes up to this one
#pragma unroll
      for (int b = 1; b < 64; b <<= 1) {
        const int o = __shfl_up(upto, b);
        upto += lane >= b ? o : 0;
      }
      if (lane == 63)
        wave_ties[i & 1][wv] = upto;
      __syncthreads();
      int at = have + upto - mine;
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        at += s < wv ? wave_ties[i & 1][s] : 0;
        have += wave_ties[i & 1][s];
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (x[i][j] == tie) {
          if (at < a.K)
            out[at] = {tie, first + (i * 256 + tid) * 8 + j};
          ++at;
        }
      if (have >= a.K)
        break;
    }
  }
  if (tid >= have && tid < a.K)
    out[tid] = {0.f, -1};
}

// ---- selection: merge -----------------------------------------------------------

constexpr int kMergeCap = 1024;
constexpr int kHeld = 4; // candidates a lane holds at a time
constexpr int kTurn = 79; // lanes that a block of 256 candidates is turned by

// A valued candidate.  Before another one: the larger value, then the lower
// beam, then (where 64 bits do not tell a beam's values apart) the larger
// logit, then the lower token.
struct Valued {
  double val;
  float x;
  int32_t w, v;
};
__device__ __forceinline__ bool before(const Valued &p, const Valued &q) {
  const bool tail = (p.x > q.x) | ((p.x == q.x) & (p.v < q.v)); // (all at once: no branches)
  return (p.val > q.val) |
         ((p.val == q.val) & ((p.w < q.w) | ((p.w == q.w) & tail)));
}

// A chain of latencies, a workgroup a batch: 8 us for 64 batches of 8 beams in
// 16 parts, 5 us for one of 4 beams in 8; so the candidates are asked for
// before the sums, a beam's parts are joined by as many lanes, and the ranks
// are counted by all four waves without branches (one lane each, with
// branches: 22 us).
//
// What is ranked is what reaches the K-th largest of the 256 lanes' own maxima:
// some 1.2 K candidates if each lane's are a fair draw of all.  So a lane takes
// them across beams, parts and ranks alike: rank by rank, each block of 256 turned
// against the one before, lest a lane meet one part's at all ranks (W and parts
// are often powers of two).  Taken as they lie, with the ranks of a part side by
// side, a K of 16 or more that divides 256 let thousands through: 64 beams of
// 128001, K = 64: 4280 us, now 135; 16 of 200000 in fp32, K = 32: 320 to 900, now
// 64.
__global__ __launch_bounds__(256) void beam_merge_kernel(
    BeamArgs a, const Cand *__restrict__ cand, const PartSum *__restrict__ sums,
    const float *__restrict__ scores, const uint8_t *__restrict__ finished,
    float *__restrict__ out_scores, int32_t *__restrict__ out_parents,
    int32_t *__restrict__ out_tokens, uint8_t *__restrict__ out_finished) {
  __shared__ double lse[KDA_BEAM_MAX], base[KDA_BEAM_MAX]; // base NaN: beam without value
  __shared__ bool done[KDA_BEAM_MAX];
  __shared__ double open_base[KDA_BEAM_MAX]; // base, NaN for a finished beam too
  __shared__ uint32_t lane_key[256];
  __shared__ int rank[kMergeCap];
  __shared__ Valued buf[kMergeCap];
  __shared__ Valued sel[KDA_BEAM_MAX];
  __shared__ Valued wave_best[4];
  __shared__ int count;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 63;
  const int wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int K = a.K, W = a.W, P = a.parts;
  const double inf = __builtin_inf();
  const PartSum *ps = sums + (int64_t)b * W * P;
  const Cand *cs = cand + (int64_t)b * W * P * K;

  // Candidate i: of place i % (W P), that is beam and part, the i / (W P)-th.  The
  // first ones are asked for before all else, so that their way from memory and
  // the sums' is one.  (Quotients: the double is off by less than half of what
  // parts i + 1/2 from a multiple.)
  const int places = W * P, all = places * K;
  const auto index = [&](int block) { return block * 256 + ((tid + kTurn * block) & 255); };
  Cand held[kHeld];
  int place[kHeld];
  const auto load = [&](Cand(&c)[kHeld], int i0) {
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      const int i = index(i0 / 256 + j);
      const int r = (int)(((double)i + 0.5) * a.inv_places);
      place[j] = i - r * places;
      c[j] = i < all ? cs[place[j] * K + r] : Cand{0.f, -1};
    }
  };
  load(held, 0);

  // lse: 2^lanes_log2 lanes a beam
  const int wide = 1 << a.lanes_log2;
  for (int w0 = 0; w0 < W; w0 += 256 >> a.lanes_log2) {
    const int w = w0 + (tid >> a.lanes_log2), p0 = tid & (wide - 1);
    const bool in = w < W;
    const float sc = in ? scores[b * W + w] : 0.f;
    const bool fin = in && finished && finished[b * W + w];
    const PartSum none{0., -__builtin_inff(), 0};
    const PartSum q0 = in && p0 < P ? ps[w * P + p0] : none;
    float top = q0.max;
    for (int p = p0 + wide; p < P && in; p += wide)
      top = fmaxf(top, ps[w * P + p].max);
    for (int s = 1; s < wide; s <<= 1)
      top = fmaxf(top, __shfl_xor(top, s));
    double sum = 0.;
    PartSum q = q0;
    for (int p = p0;;) { // (a part of -inf only has the sum 0, or NaN)
      sum += q.max > -__builtin_inff() ? q.sum * exp((double)q.max - (double)top) : q.sum;
      p += wide;
      if (p >= P || !in)
        break;
      q = ps[w * P + p];
    }
    for (int s = 1; s < wide; s <<= 1)
      sum += __shfl_xor(sum, s);
    if (in && p0 == 0) {
      const double l = (double)top + log(sum);
      const bool has = sc - sc == 0.f && (fin || l - l == 0.); // finite
      done[w] = fin;
      lse[w] = l;
      base[w] = has ? (double)sc : __builtin_nan("");
      open_base[w] = has && !fin ? (double)sc : __builtin_nan("");
    }
  }
  if (tid == 0)
    count = 0;
  __syncthreads();

  const auto of_done = [&](int w) { // the one candidate of a finished beam
    return Valued{base[w], 0.f, w, a.eos};
  };
  // What the held candidates are worth, NaN if nothing.
  double worth[kHeld];
  int beam[kHeld];
  const auto rate = [&]() {
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
      beam[j] = held[j].v >= 0 ? (int)(((double)place[j] + 0.5) * a.inv_parts) : 0;
      const double v = open_base[beam[j]] + ((double)held[j].x - lse[beam[j]]);
      worth[j] = held[j].v >= 0 ? v : __builtin_nan("");
    }
  };
  // goes over the candidates that have a value
  rate();
  const auto for_all = [&](auto &&f) {
    for (int i0 = 0;;) {
#pragma unroll
      for (int j = 0; j < kHeld; ++j)
        if (worth[j] == worth[j])
          f(Valued{worth[j], held[j].x, beam[j], held[j].v});
      if (all <= kHeld * 256) // (they stay for the next time)
        break;
      i0 += kHeld * 256;
      const bool more = i0 < all;
      i0 = more ? i0 : 0;
      load(held, i0);
      rate();
      if (!more)
        break;
    }
  };
  double best = -inf;
  for_all([&](const Valued &v) { best = fmax(best, v.val); });
  double bar;
  {
    // (in fp32, rounded down: a lane's best still reaches it)
    typedef OrderOf<float> Order;
    const float near = (float)best;
    lane_key[tid] = Order::make(near) - ((double)near > best);
    __syncthreads();
    uint32_t of[4];
    bool parts;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      of[i] = lane_key[i * 64 + lane];
    const uint32_t low = kth_of_256(of, K, Order::kBits, parts);
    bar = low > Order::make(-__builtin_inff()) ? (double)Order::value(low) : -inf;
  }
  const auto push = [&](const Valued &v) {
    const int at = atomicAdd(&count, 1);
    if (at < kMergeCap)
      buf[at] = v;
  };
  for_all([&](const Valued &v) {
    if (v.val >= bar)
      push(v);
  });
  if (tid < W && done[tid] && base[tid] == base[tid])
    push(of_done(tid));
  __syncthreads();

  const int n = count;
  if (n <= kMergeCap) {
    // by rank: wave wv counts every fourth one
    for (int i = tid; i < n; i += 256)
      rank[i] = 0;
    __syncthreads();
    for (int i = lane; i < n; i += 64) {
      const Valued v = buf[i];
      int above = 0;
      for (int j = wv; j < n; j += 4)
        above += before(buf[j], v);
      atomicAdd(&rank[i], above);
    }
    __syncthreads();
    for (int i = tid; i < n; i += 256)
      if (rank[i] < K)
        sel[rank[i]] = buf[i];
  } else {
    // more than the buffer holds (thousands of equal values): one by one, each
    // time the best of all candidates that come after the last one
    Valued last{inf, 0.f, -1, -1};
    for (int k = 0; k < K; ++k) {
      Valued mine{-inf, 0.f, W, 0};
      const auto take = [&](const Valued &v) {
        if (before(last, v) && before(v, mine))
          mine = v;
      };
      for_all(take);
      if (tid < W && done[tid] && base[tid] == base[tid])
        take(of_done(tid));
      for (int s = 1; s < 64; s <<= 1) {
        const Valued o{__shfl_xor(mine.val, s), __shfl_xor(mine.x, s), __shfl_xor(mine.w, s),
                       __shfl_xor(mine.v, s)};
        if (before(o, mine))
          mine = o;
      }
      if (lane == 0)
        wave_best[wv] = mine;
      __syncthreads();
      for (int s = 0; s < 4; ++s)
        if (before(wave_best[s], mine))
          mine = wave_best[s];
      last = mine;
      if (tid == 0)
        sel[k] = mine;
      __syncthreads();
    }
  }
  __syncthreads();
  if (wv != 0)
    return;

  // one wave from here on: entry `lane` of the selection
  const int have = min(n, K);
  Valued v{-inf, 0.f, 0, 0};
  if (lane < have)
    v = sel[lane];
  if (have < K) {
    // the lowest (w, v) that are not chosen: of the first K places at most
    // `have` are
    bool open_place = lane < K;
    for (int i = 0; i < have; ++i)
      open_place = open_place && (int64_t)sel[i].w * a.V + sel[i].v != lane;
    uint64_t places = __ballot(open_place);
    if (lane >= have && lane < K) {
      for (int i = lane - have; i > 0; --i)
        places &= places - 1;
      const int at = __builtin_ctzll(places);
      v.w = at / a.V;
      v.v = at % a.V;
    }
  }
  int to = lane;
  if (a.order == KDA_BEAM_BY_ROW) {
    bool stays = lane < K;
    uint64_t taken = 0;
    for (int i = 0; i < K; ++i) {
      const int w = __builtin_amdgcn_readlane(v.w, i);
      taken |= 1ull << w;
      stays = stays && !(i < lane && w == v.w);
    }
    const uint64_t moves = __ballot(lane < K && !stays);
    if (stays) {
      to = v.w;
    } else {
      uint64_t spare = ~taken;
      for (int i = __popcll(moves & ((1ull << lane) - 1)); i > 0; --i)
        spare &= spare - 1;
      to = spare ? __builtin_ctzll(spare) : 0;
    }
  }
  if (lane < K) {
    const int64_t at = (int64_t)b * K + to;
    out_scores[at] = (float)v.val;
    out_parents[at] = v.w;
    out_tokens[at] = v.v;
    out_finished[at] = done[v.w] || v.v == a.eos;
  }
}

// ---- reordering ----------------------------------------------------------------

typedef u32x4 u32x4_byte __attribute__((aligned(1)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef u32x2 u32x2_byte __attribute__((aligned(1)));

// States of the size of the card's last cache and below are left in it for the
// step that reads them next; the stores of larger ones go past it (2 groups of 4
// rows of 96 x 128 x 128 fp32, reorder and step: 30 us, 33; 32 groups: 471, 445).
constexpr int64_t kLastCache = 256 << 20;

// KM: rows that change, at most; U: bytes a lane holds of each, in turns of
// STEP rows without a branch (a place behind the last row repeats it).
//
// 32 groups of 4 rows of 6.3 MB, of which 64 change: 135 us, 5.96 TB/s, what
// memory gives.  One piece a lane: with four, one after the other, 144 us.
template <int KM, int STEP, bool PAST, typename U>
__global__ __launch_bounds__(256) void reorder_kernel(ReorderCall c) {
  __shared__ int64_t from[KDA_BEAM_MAX], to[KDA_BEAM_MAX];
  __shared__ int moved;
  constexpr int64_t kSpan = 256 * (int64_t)sizeof(U);
  // state, group and block of columns
  int64_t blk = c.first + blockIdx.x;
  int s = 0;
  int64_t per = 0;
  for (; s < c.num_states; ++s) {
    per = (c.bytes[s] + kSpan - 1) / kSpan;
    if (blk < per * c.groups)
      break;
    blk -= per * c.groups;
  }
  if (s == c.num_states)
    return;
  const int group = (int)(blk / per);
  const int64_t col = (blk - group * per) * kSpan + threadIdx.x * (int64_t)sizeof(U);
  const int64_t bytes = c.bytes[s];
  if (threadIdx.x < 64) {
    const int r = threadIdx.x;
    const int64_t row = (int64_t)group * c.K + r;
    int64_t f = 0, t = 0;
    bool moves = false;
    if (r < c.K) {
      const int p = c.parents[row];
      if (p >= 0 && p < c.K && p != r) {
        f = c.slots ? c.slots[row - r + p] : row - r + p;
        t = c.slots ? c.slots[row] : row;
        moves = f >= 0 && f < c.num_slots[s] && t >= 0 && t < c.num_slots[s];
      }
    }
    const uint64_t which = __ballot(moves);
    if (moves) {
      const int at = __popcll(which & ((1ull << r) - 1));
      from[at] = f * bytes;
      to[at] = t * bytes;
    }
    if (r == 0)
      moved = __popcll(which);
  }
  __syncthreads();
  const int n = __builtin_amdgcn_readfirstlane(moved);
  if (n == 0)
    return;
  uint8_t *base = (uint8_t *)c.state[s];
  if (col + (int64_t)sizeof(U) <= bytes) {
    typedef std::conditional_t<sizeof(U) == 16, u32x4_byte, u32x2_byte> Any;
    U v[KM];
#pragma unroll
    for (int i0 = 0; i0 < KM; i0 += STEP)
      if (i0 < n)
#pragma unroll
        for (int i = i0; i < i0 + STEP; ++i)
          v[i] = *reinterpret_cast<const Any *>(base + from[min(i, n - 1)] + col);
#pragma unroll
    for (int i0 = 0; i0 < KM; i0 += STEP)
      if (i0 < n)
#pragma unroll
        for (int i = i0; i < i0 + STEP; ++i) {
          Any *p = reinterpret_cast<Any *>(base + to[min(i, n - 1)] + col);
          if constexpr (PAST)
            __builtin_nontemporal_store(v[i], p);
          else
            *p = v[i];
        }
  } else {
    // the last bytes of a slice whose size is no multiple of the unit
#pragma unroll 1
    for (int64_t at = col; at < bytes; ++at) {
      uint8_t v[KM];
#pragma unroll
      for (int i = 0; i < KM; ++i)
        v[i] = base[from[min(i, n - 1)] + at];
#pragma unroll
      for (int i = 0; i < KM; ++i)
        base[to[min(i, n - 1)] + at] = v[i];
    }
  }
}

template <typename T> int part_count(int32_t V) { return (V - 1) / kPart<T> + 1; }

size_t up(size_t x) { return (x + 255) / 256 * 256; }

} // namespace

size_t beam_workspace(int elt, int32_t B, int32_t W, int32_t V, int32_t K) {
  const size_t parts = elt == 1 ? part_count<bf16>(V) : part_count<float>(V);
  const size_t n = (size_t)B * W * parts;
  return up(n * sizeof(PartSum)) + up(n * K * sizeof(Cand));
}

hipError_t launch_beam_select(int elt, const BeamCall &c, void *ws, hipStream_t s) {
  BeamArgs a{};
  a.B = c.B;
  a.W = c.W;
  a.V = c.V;
  a.K = c.K;
  a.eos = c.eos;
  a.order = c.order;
  a.row_stride = c.row_stride;
  a.parts = elt == 1 ? part_count<bf16>(c.V) : part_count<float>(c.V);
  while ((1 << a.lanes_log2) < a.parts && a.lanes_log2 < 6)
    ++a.lanes_log2;
  a.inv_parts = 1. / (double)a.parts;
  a.inv_places = 1. / ((double)c.W * a.parts);
  const int64_t n = (int64_t)c.B * c.W * a.parts;
  if (n * 256 > UINT32_MAX)
    return hipErrorInvalidConfiguration;
  PartSum *sums = (PartSum *)ws;
  Cand *cand = (Cand *)((uint8_t *)ws + up((size_t)n * sizeof(PartSum)));
  if (elt == 1)
    beam_part_kernel<bf16><<<(unsigned)n, 256, 0, s>>>(a, (const bf16 *)c.logits, cand, sums);
  else
    beam_part_kernel<float><<<(unsigned)n, 256, 0, s>>>(a, (const float *)c.logits, cand, sums);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess)
    return e;
  beam_merge_kernel<<<(unsigned)c.B, 256, 0, s>>>(a, cand, sums, c.scores, c.finished,
                                                  c.out_scores, c.out_parents, c.out_tokens,
                                                  c.out_finished);
  return hipGetLastError();
}

hipError_t launch_state_reorder(const ReorderCall &call, hipStream_t s) {
  ReorderCall c = call;
  int64_t held = 0;
  for (int i = 0; i < c.num_states; ++i)
    held += c.bytes[i] * c.groups * c.K;
  const auto run = [&](auto km, auto step, auto unit) {
    typedef decltype(unit) U;
    constexpr int KM = decltype(km)::value, STEP = decltype(step)::value;
    const int64_t span = 256 * (int64_t)sizeof(U);
    int64_t blocks = 0;
    for (int i = 0; i < c.num_states; ++i)
      blocks += (c.bytes[i] + span - 1) / span * c.groups;
    const auto kernel = held > kLastCache ? reorder_kernel<KM, STEP, true, U>
                                          : reorder_kernel<KM, STEP, false, U>;
    // (the device's grids: 2^32 - 1 threads)
    constexpr int64_t kMost = UINT32_MAX / 256;
    for (c.first = 0; c.first < blocks; c.first += kMost) {
      kernel<<<(unsigned)std::min(kMost, blocks - c.first), 256, 0, s>>>(c);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess)
        return e;
    }
    return hipSuccess;
  };
  using std::integral_constant;
  typedef integral_constant<int, 1> Single;
  typedef integral_constant<int, 8> Eight;
  if (c.K <= 4)
    return run(integral_constant<int, 4>(), Single(), u32x4());
  if (c.K <= 8) // (one by one, the compiler spends 234 registers: 32 groups of 8, 715 us, 443)
    return run(integral_constant<int, 8>(), integral_constant<int, 2>(), u32x4());
  if (c.K <= 16)
    return run(integral_constant<int, 16>(), Single(), u32x4());
  if (c.K <= 32)
    return run(integral_constant<int, 32>(), Eight(), u32x4());
  return run(integral_constant<int, 64>(), Eight(), u32x2());
}

} // namespace kda
