// Linear attention with one decay a head, for packed prompts and for single
// tokens:  S_t = exp(g_t) S_{t-1} + k_t v_t^T,  o_t = scale S_t^T q_t.
//
// Prompts run in chunks of 64 tokens.  With G the sum of g from a chunk's
// start, S the state that enters it and L its last token:
//   o_i = scale (e^{G_i} S^T q_i + sum_{j <= i} e^{G_i - G_j} (q_i . k_j) v_j)
//   S'  = e^{G_L} S + sum_j k_j (e^{G_L - G_j} v_j)^T
// that is four matrix products a chunk.  A workgroup carries the state of one
// (sequence, head) and 64 or 128 value columns through the tokens; each of its
// waves holds 16 columns of the state (all dk rows) in registers and forms
// these columns of o.  The scores of a chunk are formed once, 16 tokens by 32
// a wave, and shared through LDS as operands; q, k and v of a chunk lie in LDS
// as they come.
//
// Layout: what one product leaves in registers is the next one's operand.  A
// lane holds eight neighbouring rows of its state column in two accumulators
// (tiles of rows take the rows 32 (t / 2) + 8 (m / 4) + 4 (t % 2) + m % 4), so
// the state, rounded, is the operand of S^T q beside rows of q as they are.
// The scores come out with the tokens 32 s + 16 h + 4 g + r in element 4 h + r
// of lane group g; K and V are read transposed in that order.
//
// Roundings: the state is fp32 and its update takes v e^{G_L - G_j} as the sum
// of three bf16 numbers (24 bits; one alone would leave the state 2^-9 off, for
// the rest of the prompt), beside k as it is.  For o, which is bf16 itself, the
// scores and the entering state are rounded to bf16 once each: o is then 2.3e-3
// of its size off (root mean square), 1.7e-3 of it by its own rounding.  Both in
// two parts leave its own alone, but take 22 products more of a wave's 70 (8192
// tokens of 96 heads 291 us against 264, 131072 of 12 777 against 702, 16 x 2048
// of 96 1030 against 884): who needs the bits has fp32 calls, which round nothing.
// G is summed and kept as two fp32 numbers, so that differences within a chunk
// keep their accuracy beside a decay of e^-150.
//
// Ends of fp32's range.  Where an infinity or a NaN in q, k or v, or growth past
// fp32, would meet a 0 in these products (an infinity in k or v would even reach
// earlier tokens of its chunk), a wave's columns of the chunk go by the
// recurrence, token by token.  Infinities and NaN of q and k show in the scores,
// which are looked at as they are formed (launches that form only states look at
// k); those of v each wave finds in its columns.
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
  int32_t slices, seg; // slices of dv (a workgroup's columns), tokens per segment
  int64_t units;       // (segment, head) pairs of this launch
  float *seg_state;    // [segments of cut sequences, H, slices, DK / 16, lanes] of four
  double *pair_decay;  // [segments of pass 0, H]: log2 of a segment's decay
};

constexpr float kMinDecay = -150.f; // fp32's exp is 0 there
// exp(g), 0 from kMinDecay down (and for -inf); NaN for NaN
__device__ __forceinline__ float decay_of(float g) { return expf(g < kMinDecay ? kMinDecay : g); }

// Numbers of some 48 bits as the sum of two fp32 ones, hi the sum rounded.
struct Pair {
  float hi, lo;
};
__device__ __forceinline__ Pair operator+(const Pair &a, const Pair &b) {
  const float s = a.hi + b.hi, t = s - a.hi;
  const float e = (a.hi - (s - t)) + (b.hi - t) + (a.lo + b.lo);
  const float h = s + e;
  return {h, e - (h - s)};
}
__device__ __forceinline__ Pair operator-(const Pair &a) { return {-a.hi, -a.lo}; }
// 2^x to an fp32 rounding or two, whatever the size of x
__device__ __forceinline__ float exp2_of(const Pair &x) {
  const float e = __builtin_amdgcn_exp2f(x.hi);
  return fmaf(e, x.lo * 0.693147181f, e);
}
// log2 of a token's decay: g log2(e)
__device__ __forceinline__ Pair log2_decay(float g) {
  constexpr float c1 = 0x1.715476p+0f, c2 = 0x1.4ae0bep-26f; // log2(e)
  g = g < kMinDecay ? kMinDecay : g; // (a NaN stays one)
  const float hi = g * c1;
  return {hi, fmaf(g, c2, fmaf(g, c1, -hi))};
}
// Whether the decays of a chunk (a token a lane; 0 behind the last) grow a
// state by more than some 2^64 on the way: by tokens then, lest factors of 2^127
// and more meet small k and v.
__device__ __forceinline__ bool grows(float g) {
  if (__builtin_expect(!__any(g > 0.f), 1))
    return false;
  float up = fmaxf(g, 0.f);
  for (int b = 1; b < 64; b <<= 1)
    up += __shfl_xor(up, b);
  return !(up < 44.f);
}
constexpr float kNone = -104.f; // fp32's exp is 0 below

// What a chunk takes of its decays, from G (log2 of the decay from its start to
// each token), the last of them, and the tokens' g (0 behind the last; `real`:
// this lane's is not behind).
struct ChunkDecay {
  float to_token, to_end, all;
};
__device__ __forceinline__ ChunkDecay chunk_decay(const Pair &G, const Pair &last, float g,
                                                  bool real) {
  // A product of decays that underflows is the least number above 0, so that an
  // infinite state outlasts it, as it does token by token; 0 with a token that
  // forgets everything.
  constexpr float kLeast = 0x1p-149f;
  const auto product = [](float e, bool none) { return e < kLeast ? none ? 0.f : kLeast : e; };
  const uint64_t none = __ballot(g < kNone), upto = (2ull << (threadIdx.x & 63)) - 1;
  return {product(exp2_of(G), (none & upto) != 0), real ? exp2_of(last + -G) : 0.f,
          grows(g) ? __builtin_inff() : product(exp2_of(last), none != 0)};
}
// log2 of a chunk's decay, from the sum over its tokens: -inf where one is 0.
__device__ __forceinline__ double log2_total(const Pair &sum, float g) {
  if (__builtin_expect(!__any(!(g >= kNone && g < __builtin_inff())), 1))
    return (double)sum.hi + (double)sum.lo;
  return (__any(g < kNone) ? -__builtin_inf() : 0.) +
         (__any(g == __builtin_inff()) ? __builtin_inf() : 0.) +
         (__any(g != g) ? __builtin_nan("") : 0.);
}
// Sum over lanes 0 .. of a wave up to each (DPP: 1, 2, 4 and 8 lanes within
// rows of 16, then the ends of rows to those behind).
template <int CTRL, int ROWS> __device__ __forceinline__ Pair dpp_pair(const Pair &x) {
  return {__builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                        0, __builtin_bit_cast(int, x.hi), CTRL, ROWS, 0xf, true)),
          __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(
                                        0, __builtin_bit_cast(int, x.lo), CTRL, ROWS, 0xf, true))};
}
__device__ __forceinline__ Pair prefix_sum(Pair x) {
  x = x + dpp_pair<0x111, 0xf>(x);
  x = x + dpp_pair<0x112, 0xf>(x);
  x = x + dpp_pair<0x114, 0xf>(x);
  x = x + dpp_pair<0x118, 0xf>(x);
  x = x + dpp_pair<0x142, 0xa>(x);
  return x + dpp_pair<0x143, 0xc>(x);
}
__device__ __forceinline__ Pair lane_pair(const Pair &x, int lane) {
  lane = __builtin_amdgcn_readfirstlane(lane);
  const auto read = [lane](float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
  };
  return {read(x.hi), read(x.lo)};
}

// ---- prompts ----------------------------------------------------------------------

constexpr int kDC = 64; // tokens per chunk

// Tiles are staged in pieces of 16 bytes.
template <typename T> constexpr int kPiece = 16 / (int)sizeof(T);
typedef u32x4 u32x4_any __attribute__((aligned(2)));

// n elements of a piece from p (n >= the piece's: all, n <= 0: none; else 0)
__device__ __forceinline__ u32x4 load_piece(const bf16 *p, int n) {
  if (n >= 8)
    return *reinterpret_cast<const u32x4_any *>(p);
  bf16x8 v{};
#pragma unroll
  for (int i = 0; i < 7; ++i)
    if (i < n)
      v[i] = p[i];
  return __builtin_bit_cast(u32x4, v);
}
__device__ __forceinline__ u32x4 load_piece(const float *p, int n) {
  if (n >= 4)
    return *reinterpret_cast<const u32x4_any *>(p);
  f32x4 v{};
#pragma unroll
  for (int i = 0; i < 3; ++i)
    if (i < n)
      v[i] = p[i];
  return __builtin_bit_cast(u32x4, v);
}

// The sum of 0 * x over a piece: NaN where an element is not finite.
__device__ __forceinline__ float zero_sum(const u32x4 &x, bf16) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  const bf16x8 v = __builtin_bit_cast(bf16x8, x);
  const bf16x2_t z = {static_cast<bf16>(0.f), static_cast<bf16>(0.f)};
  float a = __builtin_amdgcn_fdot2_f32_bf16(__builtin_shufflevector(v, v, 0, 1), z, 0.f, false);
  float b = __builtin_amdgcn_fdot2_f32_bf16(__builtin_shufflevector(v, v, 2, 3), z, 0.f, false);
  a = __builtin_amdgcn_fdot2_f32_bf16(__builtin_shufflevector(v, v, 4, 5), z, a, false);
  b = __builtin_amdgcn_fdot2_f32_bf16(__builtin_shufflevector(v, v, 6, 7), z, b, false);
  return a + b;
}
__device__ __forceinline__ float zero_sum(const u32x4 &x, float) {
  const f32x4 v = __builtin_bit_cast(f32x4, x) * 0.f;
  return (v[0] + v[1]) + (v[2] + v[3]);
}

// LDS matrices.  Rows have no padding; the pieces of a row are permuted by an
// exclusive-or with bits of the row, so that the same piece of the rows of a tile
// lies in different banks.  K and q have rows of LD = DK elements, V of the
// workgroup's columns.  Counted one kind of read at a time (SQ_LDS_BANK_CONFLICT):
// none for rows of fp32 fragments, V transposed, scores, decays and weights; but 4
// of the 8 cycles of a row fragment in bf16, and half of those of K transposed (2
// of 4, fp32 4 of 8): its lanes take one half of their pieces, half the banks.
template <typename T, int LD> __device__ __forceinline__ int row_flip(int row) {
  if constexpr (sizeof(T) == 4)
    return row & 15;
  else if constexpr (LD == 64) // (two rows meet all banks)
    return ((row >> 1) & 3) << 1 | ((row >> 3) & 1);
  else
    return (row & 7) << 1 | ((row >> 3) & 1);
}
template <typename T, int LD> __device__ __forceinline__ int lds_at(int row, int col) {
  constexpr int kP = kPiece<T>;
  return row * LD + (((col / kP) ^ row_flip<T, LD>(row)) * kP | (col & (kP - 1)));
}
// Because only low bits of the row enter the permutation, 16 rows further is a
// constant distance; and where bits of a column index above those of a lane's
// own change, the place changes by an exclusive-or with them: with at =
// lds_at(row, col), fragment s of a row is at ^ 32 s, row tile t of the state
// (columns of K) at ^ state_tile(t), wave w's columns of V at ^ 16 w.
__device__ __forceinline__ constexpr int state_tile(int t) { return 32 * (t >> 1) + 4 * (t & 1); }
// Row m of tile 0 of the state's rows.
__device__ __forceinline__ int state_row(int m) { return 8 * (m >> 2) + (m & 3); }

// The operand of eight tokens (element 4 h + r: row0 + 16 h + 4 lg + r) and
// the 16 columns of a tile; `ld` elements a row.  bf16: two transposed reads;
// in each 16-lane group, lane 4 a + b of ds_read_b64_tr_b16 receives element b
// of the 4-element reads of lanes a, a + 4, a + 8, a + 12, so lane L reads
// four columns of row L / 4, from the one of m = 4 (L % 4) on (tr_row, tr_col).
// fp32: element by element; at[r]: row 4 lg + r, column lr.
template <typename T> constexpr int kTrAt = sizeof(T) == 4 ? 4 : 1;
__device__ __forceinline__ Frag<bf16> tr_frag(const bf16 *m, int ld, const int (&at)[1], int flip) {
  typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
  const bf16 *p = m + (at[0] ^ flip);
  const bf16x4 r0 = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4 *)p);
  const bf16x4 r1 = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4 *)(p + 16 * ld));
  return {__builtin_shufflevector(r0, r1, 0, 1, 2, 3, 4, 5, 6, 7)};
}
__device__ __forceinline__ Frag<float> tr_frag(const float *m, int ld, const int (&at)[4],
                                               int flip) {
  Frag<float> f;
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    f.lo[r] = m[at[r] ^ flip];
    f.hi[r] = m[(at[r] ^ flip) + 16 * ld];
  }
  return f;
}

// Eight neighbouring elements of a row (fp32: two pieces).
__device__ __forceinline__ Frag<bf16> lds_frag(const bf16 *m, int at) { return load_frag(m + at); }
__device__ __forceinline__ Frag<float> lds_frag(const float *m, int at) {
  return {*reinterpret_cast<const f32x4 *>(m + at), *reinterpret_cast<const f32x4 *>(m + (at ^ 4))};
}

__device__ __forceinline__ Frag<bf16> pack_scores(const f32x4 &lo, const f32x4 &hi, bf16) {
  return pack_acc2(lo, hi);
}
__device__ __forceinline__ Frag<float> pack_scores(const f32x4 &lo, const f32x4 &hi, float) {
  return {lo, hi};
}

// A fragment kept in LDS as an operand, lane by lane.
__device__ __forceinline__ void put_frag(bf16 *p, int lane, const Frag<bf16> &f) {
  *reinterpret_cast<bf16x8 *>(p + lane * 8) = f.v;
}
__device__ __forceinline__ void put_frag(float *p, int lane, const Frag<float> &f) {
  *reinterpret_cast<f32x4 *>(p + lane * 4) = f.lo;
  *reinterpret_cast<f32x4 *>(p + 256 + lane * 4) = f.hi;
}
__device__ __forceinline__ Frag<bf16> get_frag(const bf16 *p, int lane) {
  return load_frag(p + lane * 8);
}
__device__ __forceinline__ Frag<float> get_frag(const float *p, int lane) {
  return {*reinterpret_cast<const f32x4 *>(p + lane * 4),
          *reinterpret_cast<const f32x4 *>(p + 256 + lane * 4)};
}

// An operand times a weight per element, as a sum of operands.
struct Split3 {
  Frag<bf16> part[3];
};
__device__ __forceinline__ Split3 weigh(const Frag<bf16> &v, const f32x4 &w0, const f32x4 &w1) {
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  const u32x4 raw = __builtin_bit_cast(u32x4, v.v);
  u32x4 out[3];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float x = __builtin_bit_cast(float, raw[i] << 16) * (i < 2 ? w0[2 * i] : w1[2 * i - 4]);
    float y = __builtin_bit_cast(float, raw[i] & 0xffff0000u) *
              (i < 2 ? w0[2 * i + 1] : w1[2 * i - 3]);
#pragma unroll
    for (int p = 0; p < 3; ++p) { // (a pair is rounded by one instruction)
      const uint32_t b = __builtin_bit_cast(
          uint32_t, bf16x2_t{static_cast<bf16>(x), static_cast<bf16>(y)});
      out[p][i] = b;
      x -= __builtin_bit_cast(float, b << 16);
      y -= __builtin_bit_cast(float, b & 0xffff0000u);
    }
  }
  return {{{__builtin_bit_cast(bf16x8, out[0])},
           {__builtin_bit_cast(bf16x8, out[1])},
           {__builtin_bit_cast(bf16x8, out[2])}}};
}
struct Whole {
  Frag<float> part[1];
};
__device__ __forceinline__ Whole weigh(const Frag<float> &v, const f32x4 &w0, const f32x4 &w1) {
  return {{{v.lo * w0, v.hi * w1}}};
}

// ... of 0 * x over eight numbers, added to z
__device__ __forceinline__ float zero_sum(const f32x4 &a, const f32x4 &b, float z) {
#pragma unroll
  for (int r = 0; r < 4; ++r)
    z = fmaf(a[r], 0.f, z);
  float y = 0.f;
#pragma unroll
  for (int r = 0; r < 4; ++r)
    y = fmaf(b[r], 0.f, y);
  return z + y;
}
__device__ __forceinline__ float zero_sum(const Frag<bf16> &f) {
  return zero_sum(__builtin_bit_cast(u32x4, f.v), bf16());
}
__device__ __forceinline__ float zero_sum(const Frag<float> &f) {
  return zero_sum(__builtin_bit_cast(u32x4, f.lo), 0.f) +
         zero_sum(__builtin_bit_cast(u32x4, f.hi), 0.f);
}

// ---- tokens one by one ------------------------------------------------------------

// One head's tokens from a place on.
template <typename T> struct Tokens {
  const T *q, *k, *v;
  const float *g;
  T *o;
};

// `count` of them by the recurrence, in fp32 and straight from memory: this
// lane's column `col` of the state (`in`: there is one), and with OUT o from the
// state after a token (this lane's rows, summed over the four lane groups).  Some
// 100 us for a chunk of 64 (heads of 128), against 2 to 4.
template <bool OUT, typename T, int TD>
__device__ __forceinline__ void by_token(f32x4 (&S)[TD], const DecayArgs &a, const Tokens<T> &s,
                                         int count, int col, bool in) {
#pragma unroll 1
  for (int i = 0; i < count; ++i) {
    // (rare: opaque, lest its addresses and conditions be kept in registers)
    const int group = opaque_lane() >> 4;
    const float decay = decay_of(s.g[i * a.gs]), x = in ? to_f32(s.v[i * a.vs + col]) : 0.f;
    float sum = 0.f;
    const auto rk = buffer_rsrc(s.k + i * a.ks, a.dk * (uint32_t)sizeof(T));
    const auto rq = buffer_rsrc(s.q + i * a.qs, a.dk * (uint32_t)sizeof(T));
#pragma unroll
    for (int d = 0; d < TD; ++d) { // (rows behind dk read 0)
      float kr[4], qr[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int at = (state_tile(d) + 8 * group + r) * (int)sizeof(T);
        kr[r] = buffer_load1(rk, at, (const T *)nullptr);
        if constexpr (OUT)
          qr[r] = buffer_load1(rq, at, (const T *)nullptr);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        // (... and stay 0 beside an infinite x or decay)
        const bool real = state_tile(d) + 8 * group + r < a.dk;
        S[d][r] = fmaf(kr[r], real ? x : 0.f, (real ? decay : 0.f) * S[d][r]);
        if constexpr (OUT)
          sum = fmaf(qr[r], S[d][r], sum);
      }
    }
    if constexpr (OUT) {
      sum = add_xor32(add_xor16(sum));
      if (group == 0 && in)
        s.o[i * a.os + col] = from_f32<T>(sum * a.scale);
    }
  }
}

// Whether a wave takes a chunk by the recurrence: for q or k (`met`: a score was
// not finite), its columns of V (vf), or growth (all is infinite).  Not for the
// state that enters or a NaN among the decays: these the products carry on as the
// recurrence does, and a sequence that has met a NaN or an infinity stays as fast
// as others.
template <typename T>
__device__ __forceinline__ bool by_recurrence(const Frag<T> (&vf)[2], int met, float all) {
  const float z = zero_sum(vf[0]) + zero_sum(vf[1]);
  return __any((z != z) | (met != 0) | (all == __builtin_inff()));
}

// ---- the chunks -------------------------------------------------------------------

// A raw buffer's descriptor over `bytes` bytes at p (wave-uniform), in four
// scalars.
__device__ __forceinline__ u32x4 raw_rsrc(const void *p, uint32_t bytes) {
  const uint64_t at = (uint64_t)(uintptr_t)p;
  return u32x4{(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)at),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)((uint32_t)(at >> 32) & 0xffffu)),
               (uint32_t)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
}
// 16 bytes per lane from a raw buffer straight into LDS, lane l's to byte 16 l
// after `to` (wave-uniform).  In assembly because the compiler, which sees such
// a load as a store to any of LDS, would wait for it before each transposed
// read; the walk below waits for vmcnt(0) and a barrier before it reads what
// was loaded.  Nothing is returned in registers.  m0 cannot be named as changed
// (the compiler reserves it); a test on the listing holds that nothing else in
// these kernels uses it.
__device__ __forceinline__ void lds_request16(const u32x4 &r, int at, const void *to) {
  // (the low half of a generic LDS address is the offset in LDS)
  const uint32_t m0 = (uint32_t)(uintptr_t)to;
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane(m0)), "v"(at), "s"(r));
}
constexpr int kNowhere = 0x7fffffe0; // a byte offset past every buffer's end

// LDS and memory reads in front of and behind this are not exchanged (the
// scheduler would otherwise raise all of a chunk's, and spill registers).
__device__ __forceinline__ void reads_stay() { __builtin_amdgcn_sched_barrier(0x000f); }

// Launch `pass` 0, of cut sequences: all segments but the last, only their
// states: the first from the state that enters the sequence, which is put into
// the workspace as it is, the others from zero.  Pass 1: all segments in full
// from the states that enter them.  NW waves, 16 value columns each.  FAST: dk,
// dv and the rows' addresses are multiples of 16 bytes: everything moves through
// raw buffers, whose bounds take the place of branches at a chunk's end, and q, K
// and V straight into LDS.  AHEAD: a chunk ahead into the other one of two copies;
// TURNS, where LDS holds no two: each of the three as its place gets free;
// without either, the loads of the one copy are waited for (heads of 128 in bf16:
// 8.2 us a chunk, FAST 3.9; of 255 in fp32 28.6, of 256 FAST 17.3; fp32 heads of
// 128, eight waves, spill two registers there).
//
// 131072 tokens, 12 heads of 128, bf16: 21 segments a head, 275 us for their
// states and 450 for the outputs (3.6 TB/s of q, k, v and o).  No unit is full
// (matrix cores 22 %): what is seen of its bound is the chain of a chunk's
// products, barriers and LDS round trips, 3.9 us for 128 columns with 96 CUs
// busy, 4.6 with all.  Chunks requested two ahead (a third copy, 158 KB of LDS)
// gain 2 % there and lose 15 % on sequences of two chunks.
//
// fp32 multiplies on the fp32 matrix instructions, at a sixteenth of bf16's
// rate: 9.4 of the 13.1 us of a chunk of eight waves are theirs, rows that pad dk
// and columns that pad dv included.  With all loads waited for, without TURNS, a
// chunk took 14.8; one of bf16 heads of 256 5.5 us, now 4.4.
template <typename T, int DK, int NW> constexpr int kCopyBytes =
    kDC * (2 * DK + 16 * NW) * (int)sizeof(T);
template <typename T, int DK, int NW, bool FAST>
__global__ __launch_bounds__(64 * NW, NW == 8 ? 2 : 1) void decay_chunk_kernel(
    SeqTable tab, DecayArgs a, int pass, const T *__restrict__ q, const T *__restrict__ k,
    const T *__restrict__ v, T *__restrict__ o) {
  const SeqView sv(tab);
  constexpr int kEs = (int)sizeof(T), kP = kPiece<T>;
  constexpr int kCols = 16 * NW;                // value columns
  constexpr int kGQ = DK / 32;                  // fragments of a row of q or K
  constexpr int kTD = DK / 16;                  // row tiles of a wave's state
  constexpr int kNK = DK * kEs / (16 * NW);     // pieces of K (q) a lane stages
  constexpr int kNV = kEs;                      // pieces of V a lane stages
  constexpr bool AHEAD = FAST && 2 * kCopyBytes<T, DK, NW> <= 98304;
  // TURNS: K alone has two copies; V is free once every wave holds its columns,
  // q once the scores and S^T q are formed.
  constexpr bool TURNS =
      FAST && !AHEAD && kCopyBytes<T, DK, NW> + kDC * (DK + kDC) * kEs <= 155648;
  constexpr int kBufs = AHEAD ? 2 : 1, kKBufs = AHEAD || TURNS ? 2 : 1;
  // (bf16 has room for the scores beside q; fp32 puts them in its place)
  constexpr bool OWN_P = kEs == 2;
  __shared__ alignas(16) T Qs[kBufs][kDC * DK], Ks[kKBufs][kDC * DK], Vs[kBufs][kDC * kCols];
  __shared__ alignas(16) T Ps[OWN_P ? kDC * kDC : 8];
  __shared__ alignas(16) float Ghi[2][kDC], Glo[2][kDC], wts[2][kDC], eG[2][kDC];
  __shared__ float total[2];
  __shared__ int strange[2][NW];

  // block b: unit (b / 8 / slices) * 8 + b % 8, slice b / 8 % slices: slices
  // of one unit, which share q and k, are on one die
  const int64_t unit = (int64_t)(blockIdx.x / (8 * a.slices)) * 8 + blockIdx.x % 8;
  if (unit >= a.units)
    return;
  const int slice = blockIdx.x / 8 % a.slices;
  const int h = (int)(unit % a.H), blk = (int)(unit / a.H);
  const int n = sv.find(blk, pass);
  const int seq = sv.seq(n), len = sv.len(n);
  const int nseg = sv.blk(n + 1, 1) - sv.blk(n, 1), seg = blk - sv.blk(n, pass);
  // (states in front: of each cut sequence one more than its blocks in pass 0)
  const int64_t pair0 = sv.blk(n, 0), state0 = pair0 + sv.blk(n, 2);
  int pos = seg * a.seg;
  const int end = min(len, pos + a.seg);
  const int64_t slot = a.slots ? a.slots[seq] : seq;
  const bool kept = slot >= 0 && slot < a.num_slots;

  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lg = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col0 = slice * kCols;
  const int cols = min(kCols, a.dv - col0);
  const int my_col = 16 * w + lr; // of the state this lane holds

  // the state that enters: element r of tile d is row state_tile(d) + 8 lg + r
  // of column my_col
  f32x4 S[kTD];
  const int64_t global = (slot * a.H + h) * a.dk * a.dv + col0 + my_col;
  const int64_t seg_step = (int64_t)a.H * a.slices * (kTD * 256 * NW);
  // the state that enters this segment
  float *entry = a.seg_state + (state0 + seg) * seg_step +
                 ((int64_t)h * a.slices + slice) * (kTD * 256 * NW) + tid * 4;
  const auto put_state = [&](float *to) __attribute__((always_inline)) {
#pragma unroll
    for (int d = 0; d < kTD; ++d)
      *reinterpret_cast<f32x4 *>(to + d * 256 * NW) = S[d];
  };
  if (pass == 1 && nseg > 1) {
#pragma unroll
    for (int d = 0; d < kTD; ++d)
      S[d] = *reinterpret_cast<const f32x4 *>(entry + d * 256 * NW);
  } else {
    const bool from = seg == 0 && a.init && kept && my_col < cols;
#pragma unroll
    for (int d = 0; d < kTD; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = state_tile(d) + 8 * lg + r;
        S[d][r] = from && row < a.dk ? a.init[global + (int64_t)row * a.dv] : 0.f;
      }
    if (pass == 0 && seg == 0) // (pass 1 may write the last state in its place)
      put_state(entry);
  }

  // Staging.  Wave w's piece i is the (pieces a lane) * w + i-th kilobyte of
  // an LDS copy, 16 bytes a lane; where that is in the matrix follows from the
  // flips.  `at`: the places of the next tile in memory.
  struct Source {
    const T *q, *k, *v;
    const float *g;
  };
  const int64_t tok0 = sv.tok0(n);
  const int ks = (int)a.ks, vs = (int)a.vs, qs = (int)a.qs, os = (int)a.os, gs = (int)a.gs;
  const auto source = [&](int at) __attribute__((always_inline)) {
    return Source{q + (tok0 + at) * a.qs + (int64_t)(h / a.rq) * a.dk,
                  k + (tok0 + at) * a.ks + (int64_t)(h / a.rk) * a.dk,
                  v + (tok0 + at) * a.vs + (int64_t)(h / a.rv) * a.dv + col0,
                  a.g + (tok0 + at) * a.gs + h};
  };
  const auto piece = [&](auto ld, int per_lane, int i, int &row, int &col)
      __attribute__((always_inline)) {
    constexpr int LD = decltype(ld)::value, per = LD / kP;
    const int at = (w * per_lane + i) * 64 + lane;
    row = at / per;
    col = ((at % per) ^ row_flip<T, LD>(row)) * kP;
  };
  const auto stage = [&](auto ld, T *copy, const T *from, int stride, int width, int cnt,
                         int per_lane, int i) __attribute__((always_inline)) {
    int row, c;
    piece(ld, per_lane, i, row, c);
    T *to = copy + (w * per_lane + i) * 64 * kP;
    if constexpr (FAST)
      lds_request16(
          raw_rsrc(from, cnt > 0 ? (uint32_t)(((cnt - 1) * stride + width) * kEs) : 0u),
          c < width ? (row * stride + c) * kEs : kNowhere, to);
    else
      *reinterpret_cast<u32x4 *>(to + lane * kP) =
          load_piece(from + row * stride + c, row < cnt ? width - c : 0);
  };
  using std::integral_constant;
  typedef integral_constant<int, DK> RowDK;
  typedef integral_constant<int, kCols> RowV;
  // load i of a tile's 2 kNK + kNV (without q: the last kNK are left out)
  const auto stage_one = [&](const Source &s, int cnt, int buf, int i)
      __attribute__((always_inline)) {
    if (i < kNK)
      stage(RowDK(), Ks[buf], s.k, ks, a.dk, cnt, kNK, i);
    else if (i < kNK + kNV)
      stage(RowV(), Vs[AHEAD ? buf : 0], s.v, vs, cols, cnt, kNV, i - kNK);
    else
      stage(RowDK(), Qs[AHEAD ? buf : 0], s.q, qs, a.dk, cnt, kNK, i - kNK - kNV);
  };
  float gn = 0.f;
  constexpr int kScan = NW - 1; // the wave that sums the decays (8 waves: it has no scores)
  const auto load_g = [&](const Source &s, int cnt) __attribute__((always_inline)) {
    if (w == kScan)
      gn = lane < cnt ? s.g[lane * gs] : 0.f;
  };

  // The scan wave: G = log2 of the decay from the tile's start to each of its
  // tokens, and what the chunk takes of it.
  Pair G;
  ChunkDecay ends;
  double decay_sum = 0.; // of the segment
  const auto scan_decays = [&](auto out_tag, int cnt) __attribute__((always_inline)) {
    if (w != kScan)
      return;
    G = prefix_sum(lane < cnt ? log2_decay(gn) : Pair{0.f, 0.f});
    const Pair last = lane_pair(G, cnt - 1);
    ends = chunk_decay(G, last, gn, lane < cnt);
    if constexpr (!decltype(out_tag)::value)
      decay_sum += log2_total(last, gn);
  };
  const auto put_decays = [&](int par) __attribute__((always_inline)) {
    Ghi[par][lane] = G.hi;
    Glo[par][lane] = G.lo;
    eG[par][lane] = ends.to_token;
    wts[par][lane] = ends.to_end;
    if (lane == 0)
      total[par] = ends.all;
  };
  // Whether the staged tile holds other than finite numbers in k or v (each wave
  // looks at what it has staged itself).
  const auto look = [&](int buf, int par) __attribute__((always_inline)) {
    const auto at = [&](const T *copy, int per_lane, int i) __attribute__((always_inline)) {
      return zero_sum(
          *reinterpret_cast<const u32x4 *>(copy + ((w * per_lane + i) * 64 + lane) * kP), T());
    };
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < kNK; ++i)
      z += at(Ks[buf], kNK, i);
#pragma unroll
    for (int i = 0; i < kNV; ++i)
      z += at(Vs[AHEAD ? buf : 0], kNV, i);
    const bool met = __any(z != z);
    if (lane == 0)
      strange[par][w] = met;
  };

  // this lane's places in the LDS matrices: rows of fragments, and transposed
  const int frag0 = lds_at<T, DK>(lr, 8 * lg);
  int k_tr[kTrAt<T>], v_tr[kTrAt<T>];
#pragma unroll
  for (int r = 0; r < kTrAt<T>; ++r) {
    const int row = 4 * lg + (sizeof(T) == 4 ? r : lr >> 2), m = sizeof(T) == 4 ? lr : 4 * (lr & 3);
    k_tr[r] = lds_at<T, DK>(row, state_row(m));
    v_tr[r] = lds_at<T, kCols>(row, 16 * w + m);
  }

  // Walks the segment's tokens; OUT: with outputs.
  const auto walk = [&](auto out_tag) __attribute__((always_inline)) {
    constexpr bool OUT = decltype(out_tag)::value;
    constexpr int kLoads = kNK + kNV + (OUT ? kNK : 0);
    int cnt = min(kDC, end - pos), buf = 0, par = 0;
    if (cnt <= 0)
      return;
    {
      const Source s = source(pos);
      if constexpr (AHEAD || TURNS)
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          stage_one(s, cnt, buf, i);
      load_g(s, cnt);
      scan_decays(out_tag, cnt);
    }
    while (true) {
      if constexpr (!AHEAD && !TURNS) { // (every wave is done with the tile before)
        const Source s = source(pos);
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
          stage_one(s, cnt, buf, i);
      }
      if (w == kScan)
        put_decays(par);
      wait_vmem_all(); // this wave's pieces are in LDS
      if constexpr (!OUT)
        look(buf, par);
      lds_barrier();
      const float all = total[par];
      bool one_by_one = false; // this wave's columns of the chunk by the recurrence
      if constexpr (!OUT) {
        int met = 0;
#pragma unroll
        for (int i = 0; i < NW; ++i)
          met |= strange[par][i];
        one_by_one = __any(met != 0 || all == __builtin_inff());
      }
      // The next chunk's loads, one here and one there: all at once, they wait
      // for each other.
      const int next = pos + cnt, next_cnt = min(kDC, end - next);
      const Source s = source(next);
      constexpr int kSteps = OUT ? 16 : 4;
      const auto request = [&](int step) __attribute__((always_inline)) {
        if constexpr (AHEAD)
#pragma unroll
          for (int i = 0; i < kLoads; ++i)
            if (i * kSteps / kLoads == step)
              stage_one(s, next_cnt, buf ^ 1, i);
        if constexpr (TURNS)
#pragma unroll
          for (int i = 0; i < kNK; ++i) { // K; with outputs q in the second half
            if (i * (OUT ? 8 : kSteps) / kNK == step)
              stage_one(s, next_cnt, buf ^ 1, i);
            if (OUT && 8 + i * 8 / kNK == step)
              stage_one(s, next_cnt, buf, kNK + kNV + i);
          }
      };
      const auto request_v = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < kNV; ++i)
          stage_one(s, next_cnt, buf, kNK + i);
      };
      load_g(s, next_cnt);
      const T *Qb = Qs[AHEAD ? buf : 0], *Kb = Ks[buf], *Vb = Vs[AHEAD ? buf : 0];
      const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
      Frag<T> vf[2]; // this wave's columns of V, tokens 0 .. 31 and 32 .. 63
#pragma unroll
      for (int c = 0; c < 2; ++c)
        vf[c] = tr_frag(Vb + 32 * c * kCols, kCols, v_tr, 0);
      if constexpr (TURNS && !OUT) {
        lds_barrier(); // every wave holds its columns of V
        request_v();
      }

      // o^T of this wave's columns: tile t, element r is column 4 lg + r of token
      // 16 t + lr
      f32x4 O[4] = {zero, zero, zero, zero};
      T *Pb = OWN_P ? Ps : Qs[AHEAD ? buf : 0];
      if constexpr (OUT) {
        // Scores: unit u is tokens 16 t .. of q against tokens 32 c .. of k,
        // (t, c) = (u, 0), and (2, 1), (3, 1) for u = 4, 5; the others are
        // above the diagonal.  Unit u is wave u % NW's.
        f32x4 P[2][2];
        const auto unit_of = [&](int y, int &t, int &c) __attribute__((always_inline)) {
          const int u = w + y * NW;
          t = u < 4 ? u : u - 2;
          c = u < 4 ? 0 : 1;
          return u < 6;
        };
        constexpr int kUnits = NW == 8 ? 1 : 2;
        float zp = 0.f; // NaN where a score is not finite
#pragma unroll
        for (int y = 0; y < kUnits; ++y) {
          int t, c;
          P[y][0] = P[y][1] = zero;
          if (unit_of(y, t, c)) {
#pragma unroll
            for (int x = 0; x < kGQ; ++x) {
              const Frag<T> qf = lds_frag(Qb + 16 * t * DK, frag0 ^ 32 * x);
#pragma unroll
              for (int g = 0; g < 2; ++g)
                mma(P[y][g], lds_frag(Kb + (32 * c + 16 * g) * DK, frag0 ^ 32 * x), qf);
            }
          }
          zp = zero_sum(P[y][0], P[y][1], zp);
        }
        // ... and o from the entering state
        {
          Frag<T> f[2][4];
          const auto read_q = [&](int x) __attribute__((always_inline)) {
#pragma unroll
            for (int t = 0; t < 4; ++t)
              f[x & 1][t] = lds_frag(Qb + 16 * t * DK, frag0 ^ 32 * x);
          };
          read_q(0);
#pragma unroll
          for (int x = 0; x < kGQ; ++x) {
            reads_stay();
            if (x + 1 < kGQ)
              read_q(x + 1);
#pragma unroll
            for (int y = x * 8 / kGQ; y < (x + 1) * 8 / kGQ; ++y)
              request(y);
            const Frag<T> sf = pack_scores(S[2 * x], S[2 * x + 1], T());
#pragma unroll
            for (int t = 0; t < 4; ++t)
              mma(O[t], sf, f[x & 1][t]);
          }
          reads_stay();
        }
        const bool unlike = __any(zp != zp);
        if (lane == 0)
          strange[par][w] = unlike;
        const float *gh = Ghi[par], *gl = Glo[par];
        if constexpr (!OWN_P)
          lds_barrier(); // every wave has read q
#pragma unroll
        for (int y = 0; y < kUnits; ++y) {
          int t, c;
          if (unit_of(y, t, c)) {
            const int i = 16 * t + lr;
            const float hi = gh[i], lo = gl[i];
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              const int j0 = 32 * c + 16 * g + 4 * lg;
              const f32x4 jh = *reinterpret_cast<const f32x4 *>(gh + j0);
              const f32x4 jl = *reinterpret_cast<const f32x4 *>(gl + j0);
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const float d = __builtin_amdgcn_exp2f((hi - jh[r]) + (lo - jl[r]));
                P[y][g][r] = j0 + r <= i ? P[y][g][r] * d : 0.f;
              }
            }
            put_frag(Pb + (2 * t + c) * 512, lane, pack_scores(P[y][0], P[y][1], T()));
          }
        }
        lds_barrier(); // the scores are there
        if constexpr (TURNS)
          request_v();
        int met = 0;
#pragma unroll
        for (int i = 0; i < NW; ++i)
          met |= strange[par][i];
        one_by_one = by_recurrence(vf, met, all);
      }

      constexpr int kFirst = OUT ? 8 : 0, kHere = kSteps - kFirst; // requests left
      T *ob = o + (tok0 + pos) * a.os + (int64_t)h * a.dv + col0;
      if (__builtin_expect(one_by_one, 0)) {
        if constexpr (OUT && TURNS && !OWN_P)
          lds_barrier(); // (as below)
#pragma unroll
        for (int y = kFirst; y < kSteps; ++y)
          request(y);
        const Source t = source(pos);
        by_token<OUT>(S, a, Tokens<T>{t.q, t.k, t.v, t.g, ob}, cnt, my_col, my_col < cols);
      } else {
        if constexpr (OUT) {
          const auto ro =
              buffer_rsrc(ob, (uint32_t)(((cnt - 1) * os + cols) * kEs));
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const int i = 16 * t + lr;
            O[t] *= eG[par][i];
#pragma unroll
            for (int c = 0; c <= t >> 1; ++c)
              mma(O[t], vf[c], get_frag(Pb + (2 * t + c) * 512, lane));
            O[t] *= a.scale;
            const int c = 16 * w + 4 * lg;
            if constexpr (FAST) {
              const int at = c < cols ? (i * os + c) * kEs : kNowhere;
              if constexpr (kEs == 2) {
                typedef __bf16 bf16x4_t __attribute__((ext_vector_type(4)));
                typedef uint32_t u32x2_t4 __attribute__((ext_vector_type(2)));
                bf16x4_t y;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                  y[r] = static_cast<bf16>(O[t][r]);
                __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2_t4, y), ro, at, 0,
                                                      0);
              } else {
                __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, O[t]), ro, at, 0,
                                                       0);
              }
            } else if (i < cnt) {
#pragma unroll
              for (int r = 0; r < 4; ++r)
                if (c + r < cols)
                  ob[i * os + c + r] = from_f32<T>(O[t][r]);
            }
          }
          if constexpr (TURNS && !OWN_P)
            lds_barrier(); // the scores are read: q may come in their place
        }

        // The state's update, four row tiles at a time, each four's operands
        // read while the ones before are multiplied.
#pragma unroll
        for (int d = 0; d < kTD; ++d)
          S[d] *= all;
        constexpr int kBatch = kTD / 4;
        Frag<T> kf[2][4];
        const auto read_k = [&](int b) __attribute__((always_inline)) {
#pragma unroll
          for (int d = 0; d < 4; ++d)
            kf[b & 1][d] = tr_frag(Kb + 32 * (b / kBatch) * DK, DK, k_tr,
                                   state_tile(b % kBatch * 4 + d));
        };
        read_k(0);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const f32x4 w0 = *reinterpret_cast<const f32x4 *>(wts[par] + 32 * x + 4 * lg);
          const f32x4 w1 = *reinterpret_cast<const f32x4 *>(wts[par] + 32 * x + 16 + 4 * lg);
          const auto vw = weigh(vf[x], w0, w1);
#pragma unroll
          for (int b = x * kBatch; b < (x + 1) * kBatch; ++b) {
            reads_stay();
            if (b + 1 < 2 * kBatch)
              read_k(b + 1);
#pragma unroll
            for (int y = b * kHere / (2 * kBatch); y < (b + 1) * kHere / (2 * kBatch); ++y)
              request(kFirst + y);
#pragma unroll
            for (const auto &p : vw.part)
#pragma unroll
              for (int d = 0; d < 4; ++d)
                mma(S[b % kBatch * 4 + d], kf[b & 1][d], p);
          }
        }
      }
      if (next_cnt <= 0)
        break;
      pos = next;
      cnt = next_cnt;
      par ^= 1;
      scan_decays(out_tag, cnt);
      if constexpr (AHEAD || TURNS)
        buf ^= 1;
      else
        lds_barrier();
    }
  };
  if (pass == 1)
    walk(std::true_type());
  else
    walk(std::false_type());
  wait_vmem_all(); // (nothing lands in LDS behind the workgroup's end)

  if (pass == 0) {
    put_state(entry + seg_step);
    if (tid == 64 * kScan && slice == 0)
      a.pair_decay[(pair0 + seg) * a.H + h] = decay_sum;
  } else if (seg == nseg - 1 && a.fin && kept && my_col < cols) {
#pragma unroll
    for (int d = 0; d < kTD; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = state_tile(d) + 8 * lg + r;
        if (row < a.dk)
          a.fin[global + (int64_t)row * a.dv] = S[d][r];
      }
  }
}

// Streams: uncut bf16 sequences of aligned rows and up to 128 keys a head, with
// the work of a chunk spread over two kinds of waves, so that the chain of
// chunks runs at the pace of the state's own products.  Four waves carry 16
// columns of the state each (o from the entering state and from the scores, the
// update).  Eight others are a chunk ahead of them and look at k and v and form
// the scores, and two chunks ahead request q, K and V (straight into LDS) and
// sum the decays.  One barrier a chunk.  Three copies of q, K, V and the decays
// (chunk i % 3), two of the scores.
//
// 8192 tokens, 96 heads of 128: 192 workgroups, 269 us on the GPU, 2.1 us a chunk
// (1.7 with 64 workgroups).  With the same waves doing both in turn a chunk took
// 1.6 times as long.  Four score waves: 1.1 times; a score wave of two units and
// the wait for the decays behind it set the pace.
template <int DK>
__global__ __launch_bounds__(768, 3) void decay_stream_kernel(SeqTable tab, DecayArgs a,
                                                              const bf16 *__restrict__ q,
                                                              const bf16 *__restrict__ k,
                                                              const bf16 *__restrict__ v,
                                                              bf16 *__restrict__ o) {
  typedef bf16 T;
  const SeqView sv(tab);
  constexpr int kEs = 2, kP = 8, NW = 4, NS = 8, kCols = 64;
  constexpr int kGQ = DK / 32, kTD = DK / 16;
  constexpr int kNK = DK / 64, kNV = 1; // pieces of K (q) and V a lane stages
  __shared__ alignas(16) T Qs[3][kDC * DK], Ks[3][kDC * DK], Vs[3][kDC * kCols];
  __shared__ alignas(16) T Ps[2][kDC * kDC];
  __shared__ alignas(16) float Ghi[3][kDC], Glo[3][kDC], wts[3][kDC], eG[3][kDC];
  __shared__ float total[3];
  __shared__ int strange[2][8];

  const int64_t unit = (int64_t)(blockIdx.x / (8 * a.slices)) * 8 + blockIdx.x % 8;
  if (unit >= a.units)
    return;
  const int slice = blockIdx.x / 8 % a.slices;
  const int h = (int)(unit % a.H), blk = (int)(unit / a.H);
  const int n = sv.find(blk, 1);
  const int seq = sv.seq(n), end = sv.len(n);
  int pos = 0;
  const int64_t slot = a.slots ? a.slots[seq] : seq;
  const bool kept = slot >= 0 && slot < a.num_slots;

  const int tid = threadIdx.x, lane = tid & 63, lr = lane & 15, lg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), w = wave < NW ? wave : wave - NW;
  const int col0 = slice * kCols;
  const int cols = min(kCols, a.dv - col0);
  const int64_t tok0 = sv.tok0(n);
  const int ks = (int)a.ks, vs = (int)a.vs, qs = (int)a.qs, os = (int)a.os, gs = (int)a.gs;
  const T *q0 = q + tok0 * a.qs + (int64_t)(h / a.rq) * a.dk;
  const T *k0 = k + tok0 * a.ks + (int64_t)(h / a.rk) * a.dk;
  const T *v0 = v + tok0 * a.vs + (int64_t)(h / a.rv) * a.dv + col0;
  const float *g0 = a.g + tok0 * a.gs + h;
  T *o0 = o + tok0 * a.os + (int64_t)h * a.dv + col0;
  const int frag0 = lds_at<T, DK>(lr, 8 * lg);
  const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
  if (wave >= NW) {
    // ---- scores ----
    const auto stage = [&](auto ld, T *copy, const T *from, int stride, int width, int cnt,
                           int per_lane, int i) __attribute__((always_inline)) {
      constexpr int LD = decltype(ld)::value, per = LD / kP;
      const int at = (w * per_lane + i) * 64 + lane, row = at / per;
      const int c = ((at % per) ^ row_flip<T, LD>(row)) * kP;
      lds_request16(raw_rsrc(from, (uint32_t)(((cnt - 1) * stride + width) * kEs)),
                    c < width ? (row * stride + c) * kEs : kNowhere,
                    copy + (w * per_lane + i) * 64 * kP);
    };
    using std::integral_constant;
    const auto request = [&](int at, int copy) __attribute__((always_inline)) {
      const int cnt = min(kDC, end - at);
      if (cnt <= 0)
        return;
#pragma unroll
      for (int i = 0; i < kNK; ++i)
        stage(integral_constant<int, DK>(), Ks[copy], k0 + (int64_t)at * ks, ks, a.dk, cnt, kNK, i);
#pragma unroll
      for (int i = 0; i < kNK; ++i)
        stage(integral_constant<int, DK>(), Qs[copy], q0 + (int64_t)at * qs, qs, a.dk, cnt, kNK, i);
#pragma unroll
      for (int i = 0; i < kNV; ++i)
        stage(integral_constant<int, kCols>(), Vs[copy], v0 + (int64_t)at * vs, vs, cols, cnt, kNV,
              i);
    };
    const auto load_g = [&](int at) __attribute__((always_inline)) {
      return w == NS - 1 && lane < end - at ? g0[(int64_t)(at + lane) * gs] : 0.f;
    };
    const auto decays = [&](float gn, int at, int copy) __attribute__((always_inline)) {
      if (w != NS - 1)
        return;
      const int cnt = max(1, min(kDC, end - at));
      const Pair G = prefix_sum(lane < cnt ? log2_decay(gn) : Pair{0.f, 0.f});
      const Pair last = lane_pair(G, cnt - 1);
      const ChunkDecay ends = chunk_decay(G, last, gn, lane < cnt);
      Ghi[copy][lane] = G.hi;
      Glo[copy][lane] = G.lo;
      eG[copy][lane] = ends.to_token;
      wts[copy][lane] = ends.to_end;
      if (lane == 0)
        total[copy] = ends.all;
    };
    // a chunk's scores as operands: unit u is tokens 16 t .. of q against tokens
    // 32 c .. of k, (t, c) = (u, 0), and (2, 1), (3, 1) for u = 4, 5; the others
    // are above the diagonal
    const auto scores = [&](int par, int copy) __attribute__((always_inline)) {
      const float *gh = Ghi[copy], *gl = Glo[copy];
      const auto one = [&](int t, int c) __attribute__((always_inline)) {
        f32x4 P[2] = {zero, zero};
#pragma unroll
        for (int x = 0; x < kGQ; ++x) {
          const Frag<T> qf = lds_frag(Qs[copy] + 16 * t * DK, frag0 ^ 32 * x);
#pragma unroll
          for (int g = 0; g < 2; ++g)
            mma(P[g], lds_frag(Ks[copy] + (32 * c + 16 * g) * DK, frag0 ^ 32 * x), qf);
        }
        const float z = zero_sum(P[0], P[1], 0.f);
        const bool unlike = __any(z != z); // a score is not finite
        if (lane == 0)
          strange[par][w] = unlike;
        const int i = 16 * t + lr;
        const float hi = gh[i], lo = gl[i];
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          const int j0 = 32 * c + 16 * g + 4 * lg;
          const f32x4 jh = *reinterpret_cast<const f32x4 *>(gh + j0);
          const f32x4 jl = *reinterpret_cast<const f32x4 *>(gl + j0);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float d = __builtin_amdgcn_exp2f((hi - jh[r]) + (lo - jl[r]));
            P[g][r] = j0 + r <= i ? P[g][r] * d : 0.f;
          }
        }
        put_frag(&Ps[par][(2 * t + c) * 512], lane, pack_scores(P[0], P[1], T()));
      };
      if (w < 6)
        one(w < 4 ? w : w - 2, w >> 2);
    };
    if (end == 0)
      return;
    request(pos, 0);
    request(pos + kDC, 1);
    const float ga = load_g(pos), gb = load_g(pos + kDC);
    float gn = load_g(pos + 2 * kDC);
    decays(ga, pos, 0);
    decays(gb, pos + kDC, 1);
    wait_vmem_all(); // this wave's pieces are in LDS
    lds_barrier();
    scores(0, 0);
    lds_barrier();
    // copies of the chunks at hand, after it, and after that
    for (int par = 0, c1 = 1, c2 = 2; pos < end; par ^= 1) {
      const float gc = gn; // (the next one's request early: it is waited for below)
      gn = load_g(pos + 3 * kDC);
      request(pos + 2 * kDC, c2);
      if (pos + kDC < end)
        scores(par ^ 1, c1);
      decays(gc, pos + 2 * kDC, c2);
      pos += kDC;
      c1 = c2;
      c2 = c2 == 2 ? 0 : c2 + 1;
      wait_vmem_all();
      lds_barrier();
    }
    return;
  }

  // ---- states ----
  const int my_col = 16 * w + lr; // of the state this lane holds
  // the state that enters: element r of tile d is row state_tile(d) + 8 lg + r
  // of column my_col
  f32x4 S[kTD];
  const int64_t global = (slot * a.H + h) * a.dk * a.dv + col0 + my_col;
#pragma unroll
  for (int d = 0; d < kTD; ++d)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int row = state_tile(d) + 8 * lg + r;
      S[d][r] = a.init && kept && my_col < cols && row < a.dk
                    ? a.init[global + (int64_t)row * a.dv]
                    : 0.f;
    }
  int k_tr[1], v_tr[1];
  k_tr[0] = lds_at<T, DK>(4 * lg + (lr >> 2), state_row(4 * (lr & 3)));
  v_tr[0] = lds_at<T, kCols>(4 * lg + (lr >> 2), 16 * w + 4 * (lr & 3));
  if (end > 0) { // (as the score waves)
    lds_barrier();
    lds_barrier();
  }
  for (int par = 0, c0 = 0; pos < end; par ^= 1) {
    const T *Qb = Qs[c0], *Kb = Ks[c0], *Vb = Vs[c0];
    Frag<T> vf[2]; // this wave's columns of V, tokens 0 .. 31 and 32 .. 63
#pragma unroll
    for (int c = 0; c < 2; ++c)
      vf[c] = tr_frag(Vb + 32 * c * kCols, kCols, v_tr, 0);
    const float all = total[c0];
    // o^T of this wave's columns: tile t, element r is column 4 lg + r
    // of token 16 t + lr
    f32x4 O[4] = {zero, zero, zero, zero};
    Frag<T> f[2][4];
    const auto read_q = [&](int x) __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < 4; ++t)
        f[x & 1][t] = lds_frag(Qb + 16 * t * DK, frag0 ^ 32 * x);
    };
    Frag<T> pf[4][2];
    float ei[4];
    const auto read_p = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        ei[t] = eG[c0][16 * t + lr];
#pragma unroll
        for (int c = 0; c <= t >> 1; ++c)
          pf[t][c] = get_frag(&Ps[par][(2 * t + c) * 512], lane);
      }
    };
    read_q(0);
#pragma unroll
    for (int x = 0; x < kGQ; ++x) {
      reads_stay();
      if (x + 1 < kGQ)
        read_q(x + 1);
      const Frag<T> sf = pack_acc2(S[2 * x], S[2 * x + 1]);
#pragma unroll
      for (int t = 0; t < 4; ++t)
        mma(O[t], sf, f[x & 1][t]);
    }
    reads_stay();
    const auto ro = buffer_rsrc(o0 + (int64_t)pos * os,
                                (uint32_t)(((min(kDC, end - pos) - 1) * os + cols) * kEs));
    int met = 0;
#pragma unroll
    for (int i = 0; i < 6; ++i) // (the units' waves)
      met |= strange[par][i];
    const bool one_by_one = by_recurrence(vf, met, all);
    if (__builtin_expect(one_by_one, 0)) {
      by_token<true>(S, a,
                     Tokens<T>{q0 + pos * a.qs, k0 + pos * a.ks, v0 + pos * a.vs, g0 + pos * a.gs,
                               o0 + pos * a.os},
                     min(kDC, end - pos), my_col, my_col < cols);
    } else {
      read_p();
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        O[t] *= ei[t];
#pragma unroll
        for (int c = 0; c <= t >> 1; ++c)
          mma(O[t], vf[c], pf[t][c]);
      }
      // (the stores by themselves: spread over the update by the compiler, they
      // cost 8192 tokens of 96 heads 288 us, not 280)
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int i = 16 * t + lr;
        O[t] *= a.scale;
        const int c = 16 * w + 4 * lg;
        typedef uint32_t u32x2_o __attribute__((ext_vector_type(2)));
        bf16x4 y;
#pragma unroll
        for (int r = 0; r < 4; ++r)
          y[r] = static_cast<bf16>(O[t][r]);
        __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2_o, y), ro,
                                              c < cols ? (i * os + c) * kEs : kNowhere, 0, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
      // The state's update, four row tiles at a time, each four's operands
      // read while the ones before are multiplied.
#pragma unroll
      for (int d = 0; d < kTD; ++d)
        S[d] *= all;
      constexpr int kBatch = kTD / 4;
      Frag<T> kf[2][4];
      const auto read_k = [&](int b) __attribute__((always_inline)) {
#pragma unroll
        for (int d = 0; d < 4; ++d)
          kf[b & 1][d] = tr_frag(Kb + 32 * (b / kBatch) * DK, DK, k_tr,
                                 state_tile(b % kBatch * 4 + d));
      };
      read_k(0);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const f32x4 w0 = *reinterpret_cast<const f32x4 *>(wts[c0] + 32 * x + 4 * lg);
        const f32x4 w1 = *reinterpret_cast<const f32x4 *>(wts[c0] + 32 * x + 16 + 4 * lg);
        const Split3 vw = weigh(vf[x], w0, w1);
#pragma unroll
        for (int b = x * kBatch; b < (x + 1) * kBatch; ++b) {
          reads_stay();
          if (b + 1 < 2 * kBatch)
            read_k(b + 1);
#pragma unroll
          for (const auto &p : vw.part)
#pragma unroll
            for (int d = 0; d < 4; ++d)
              mma(S[b % kBatch * 4 + d], kf[b & 1][d], p);
        }
      }
    }
    pos += kDC;
    c0 = c0 == 2 ? 0 : c0 + 1;
    lds_barrier();
  }

  if (a.fin && kept && my_col < cols) {
#pragma unroll
    for (int d = 0; d < kTD; ++d)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = state_tile(d) + 8 * lg + r;
        if (row < a.dk)
          a.fin[global + (int64_t)row * a.dv] = S[d][r];
      }
  }
}

// The states of a sequence's segments from zero become the states after them:
// one by one, an element of the state per lane.
__global__ __launch_bounds__(256) void decay_fold_kernel(SeqTable tab, DecayArgs a, int per) {
  const SeqView sv(tab);
  const int64_t b = blockIdx.x; // (cut sequence, head, 1024 elements)
  const int x = (int)(b % per);
  const int h = (int)(b / per % a.H);
  const int n = sv.find((int)(b / per / a.H), 2);
  const int64_t pair0 = sv.blk(n, 0), last = sv.blk(n + 1, 0); // (the segments of pass 0)
  const int64_t step = (int64_t)a.H * per * 256;
  f32x4 *p = reinterpret_cast<f32x4 *>(a.seg_state) + (pair0 + sv.blk(n, 2) + 1) * step +
             (h * (int64_t)per + x) * 256 + threadIdx.x;
  f32x4 S = *p;
  for (int64_t i = pair0 + 1; i < last; ++i) {
    p += step;
    // 2^(e - ceil(e)), in (1/2, 1], times S, then the whole powers of 2: a state
    // that is 0 or infinite stays so whatever the size of e.
    const double e = a.pair_decay[i * a.H + h], whole = ceil(e);
    const f32x4 in = *p;
    if (e - e == 0.) {
      const float part = __builtin_amdgcn_exp2f((float)(e - whole));
      const int n = (int)fmin(fmax(whole, -1e6), 1e6);
#pragma unroll
      for (int r = 0; r < 4; ++r)
        S[r] = ldexpf(part * S[r], n) + in[r];
    } else { // a token's decay of 0 or infinity, or a NaN
      S = in + (e < 0. ? 0.f : (float)e) * S;
    }
    *p = S;
  }
}

// ---- single tokens ----------------------------------------------------------------

typedef f32x4 f32x4_any __attribute__((aligned(4)));
constexpr int kStepRows = 16; // state rows a lane has in flight

// A workgroup per (row, head): 2^lanes_log2 lanes a state row, four columns
// each, so that the state is read and written in whole lines; 8 dk dv bytes
// for 4 dk dv operations: bound by HBM.  PAST: non-temporal, for states beyond
// the card's last cache (see kLastCache).
template <typename T, bool PAST>
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
          s[i] = PAST ? __builtin_nontemporal_load(reinterpret_cast<const f32x4_any *>(p))
                      : *reinterpret_cast<const f32x4_any *>(p);
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
          if constexpr (PAST)
            __builtin_nontemporal_store(s[i], reinterpret_cast<f32x4_any *>(p));
          else
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

// How a call runs.  Measured (MI355X, 96 heads of 128, bf16 unless told):
//
// - Streams (four state waves, 64 columns a workgroup, one workgroup a CU) take
//   1.7 to 2.1 us a chunk of 64 tokens, eight waves of the other kernel 3.9 us
//   for 128 columns, four 3.4 us for 64.  A stream for each chain is the fastest
//   while all of them run at once: 8192 tokens, 192 streams: 264 us, the
//   chunk kernel uncut 499, cut in two 433.  With more chains than CUs the
//   others' wider blocks are: 16 x 2048 tokens: 880 us, streams 930.  Four waves
//   are for value heads that eight would leave half empty (32 sequences of 256
//   tokens, 16 heads of 64: 25 us, eight waves 36, streams 29).
// - Of a cut sequence k and v are read twice, in three launches: 2.8 us a chunk
//   for the states alone, 4.6 for all of it with every CU busy, some 20 us
//   beside.  A stream takes the whole in 2.0 us a chunk, so that cuts begin to
//   pay at four segments and 256 tokens (32 heads: 1024 tokens in four segments
//   43 us, uncut 37; 2048 in eight 50, 62; 8192 133, 219; 48 heads and 32768
//   tokens in five 693, 943), where the chunk kernel would take a whole
//   sequence from two and a half on.  Rows off 16 bytes have the chunk kernel
//   alone, and its rule (1024 tokens of 32 heads: uncut 133 us, cut 65).
// - fp32: 13.1 us a chunk with eight waves and 128 columns, 9.8 with four and
//   64: four where the longest sequence sets the time (9001 tokens in 37 ragged
//   sequences, 10 heads of 100 x 72, the longest 743: 149 us against 166, 1009:
//   163 and 216), eight where the number of workgroups does (37 sequences of 243:
//   123 us against 138).  In between four may be the slower one (616: 152, 141).
constexpr int64_t kCUs = 256;

bool decay_even(int elt, const kda_decay_io &io) {
  const int64_t es = elt == 1 ? 2 : 4;
  const auto even = [es](const void *p, int64_t stride) {
    return ((uintptr_t)p & 15u) == 0 && stride * es % 16 == 0;
  };
  return io.dk * es % 16 == 0 && io.dv * es % 16 == 0 && even(io.q, io.q_stride) &&
         even(io.k, io.k_stride) && even(io.v, io.v_stride) && even(io.o, io.o_stride);
}

DecayPlan decay_plan(int elt, int32_t num_seqs, const int64_t *cu, int32_t H, int32_t dk,
                     int32_t dv, int32_t split_hint, bool even) {
  DecayPlan p{};
  int64_t longest = 0;
  for (int32_t n = 0; n < num_seqs; ++n)
    longest = std::max(longest, cu[n + 1] - cu[n]);
  const auto whole = [](int64_t x) { return std::max<int64_t>(kDC, (x + kDC - 1) / kDC * kDC); };
  const auto slices = [dv](int waves) { return (dv + 16 * waves - 1) / (16 * waves); };
  // tokens that each CU has to take when all are busy
  const auto share = [&](int waves) {
    return (cu[num_seqs] * H * slices(waves) + kCUs - 1) / kCUs;
  };
  // (heads of more than 128 keys leave no registers, in fp32 no LDS, for eight)
  p.waves = dk > 128 || dv <= 64 ? 4 : 8;
  p.streams = even && elt == 1 && dk <= 128 && (int64_t)num_seqs * H * slices(4) <= kCUs;
  p.seg = whole(longest);
  if (split_hint > 1) {
    p.seg = whole((longest + split_hint - 1) / split_hint);
  } else if (split_hint == 0) {
    // (the shortest segments whose workgroups run at once, if sequences that
    // are shorter share CUs as their tokens let them)
    const auto blocks = [&](int64_t seg) {
      int64_t cut = 0, rest = 0;
      for (int32_t n = 0; n < num_seqs; ++n) {
        const int64_t len = cu[n + 1] - cu[n];
        cut += len > seg ? num_segments(len, seg) : 0;
        rest += len > seg ? 0 : len;
      }
      return (cut + (rest + seg - 1) / seg) * H * slices(p.waves);
    };
    int64_t seg = std::max<int64_t>(256, whole(share(p.waves)));
    while (seg < longest && blocks(seg) > kCUs)
      seg += whole(seg / 32);
    if (p.streams ? longest >= 4 * seg + 256 : 2 * longest >= 5 * seg)
      p.seg = seg;
  }
  int64_t states = 0;
  for (int32_t n = 0; n < num_seqs; ++n) {
    const int64_t nseg = num_segments(cu[n + 1] - cu[n], p.seg);
    p.pairs += nseg - 1;
    states += nseg > 1 ? nseg : 0;
  }
  p.streams = p.streams && p.pairs == 0;
  if (elt != 1 && p.pairs == 0 && 3 * std::max(longest, share(4)) < 4 * std::max(longest, share(8)))
    p.waves = 4;
  size_t at = seq_table_bytes(num_seqs);
  p.off_state = at;
  const size_t state = (size_t)slices(p.waves) * 16 * p.waves * padded_dk(dk) * sizeof(float);
  at = up(at + (size_t)states * H * state);
  p.off_decay = at;
  p.total = up(at + (size_t)p.pairs * H * sizeof(double));
  return p;
}

hipError_t launch_decay(int elt, const DecayCall &c, int32_t num_seqs, const int64_t *cu,
                        const DecayPlan &plan, void *ws, hipStream_t s) {
  DecayArgs a = decay_args(c);
  const bool fast = decay_even(elt, c.io);
  const int waves = plan.streams ? 4 : plan.waves;
  a.slices = (a.dv + 16 * waves - 1) / (16 * waves);
  a.seg = (int32_t)plan.seg;
  a.seg_state = (float *)((uint8_t *)ws + plan.off_state);
  a.pair_decay = (double *)((uint8_t *)ws + plan.off_decay);
  // blocks: segments in each pass, and (2) whether the sequence is cut
  const auto tiles = [&](int64_t len, int w) -> int64_t {
    const int64_t nseg = num_segments(len, plan.seg);
    return w == 0 ? nseg - 1 : (w == 1 ? nseg : nseg > 1);
  };
  int64_t total[kCounts];
  if (!seq_totals(num_seqs, cu, tiles, total))
    return hipErrorInvalidConfiguration;
  const int threads = plan.streams ? 768 : 64 * waves;
  int64_t grid[2];
  for (int pass = 0; pass < 2; ++pass) {
    grid[pass] = (total[pass] * a.H + 7) / 8 * 8 * a.slices;
    if (grid[pass] * threads > UINT32_MAX)
      return hipErrorInvalidConfiguration;
  }
  const int per = a.slices * waves * padded_dk(a.dk) / 64; // blocks of a state
  const int64_t fold = total[2] * a.H * per;
  if (fold * 256 > UINT32_MAX)
    return hipErrorInvalidConfiguration;
  SeqTable tab;
  const hipError_t e = make_seq_table(tab, num_seqs, cu, tiles, ws, s);
  if (e != hipSuccess)
    return e;
  if (plan.streams) {
    a.units = total[1] * a.H;
    const auto kernel = a.dk <= 64 ? decay_stream_kernel<64> : decay_stream_kernel<128>;
    kernel<<<(unsigned)grid[1], threads, 0, s>>>(tab, a, (const bf16 *)c.io.q, (const bf16 *)c.io.k,
                                                 (const bf16 *)c.io.v, (bf16 *)c.io.o);
    return hipGetLastError();
  }
  const auto run = [&](auto tag, auto dk, auto nw) {
    using T = decltype(tag);
    constexpr int DK = decltype(dk)::value, NW = decltype(nw)::value;
    const auto chunks = [&](int pass) {
      a.units = total[pass] * a.H;
      const auto kernel =
          fast ? decay_chunk_kernel<T, DK, NW, true> : decay_chunk_kernel<T, DK, NW, false>;
      kernel<<<(unsigned)grid[pass], threads, 0, s>>>(tab, a, pass, (const T *)c.io.q,
                                                      (const T *)c.io.k, (const T *)c.io.v,
                                                      (T *)c.io.o);
    };
    if (plan.pairs > 0) {
      chunks(0);
      decay_fold_kernel<<<(unsigned)fold, 256, 0, s>>>(tab, a, per);
    }
    chunks(1);
    return hipGetLastError();
  };
  using std::integral_constant;
  const auto wide = [&](auto tag, auto dk) {
    if (waves == 4)
      return run(tag, dk, integral_constant<int, 4>());
    if constexpr (decltype(dk)::value <= 128)
      return run(tag, dk, integral_constant<int, 8>());
    return hipErrorInvalidConfiguration; // (the plan gives these four)
  };
  const auto sized = [&](auto tag) {
    if (a.dk <= 64)
      return wide(tag, integral_constant<int, 64>());
    if (a.dk <= 128)
      return wide(tag, integral_constant<int, 128>());
    return wide(tag, integral_constant<int, 256>());
  };
  return elt == 1 ? sized(bf16()) : sized(float());
}

// The states of a decoding batch are read again a token later.  Up to the size
// of the last cache they may still be there (32 rows of 96 heads of 128 x 128,
// 201 MB, over and over: 63 us, non-temporal 78), beyond it a cached pass only
// drives out what it is about to read (256 rows, 3.2 GB of reads and writes:
// 633 us, non-temporal 593, 5.4 TB/s; 64 rows: 166 us, 154).
constexpr int64_t kLastCache = 256 << 20;

hipError_t launch_decay_step(int elt, const DecayCall &c, int32_t rows, hipStream_t s) {
  const DecayArgs a = decay_args(c);
  const int64_t grid = (int64_t)rows * a.H;
  if (grid * 256 > UINT32_MAX)
    return hipErrorInvalidConfiguration;
  int lanes_log2 = 0;
  while ((4 << lanes_log2) < a.dv)
    ++lanes_log2;
  const bool past = grid * a.dk * a.dv * (int64_t)sizeof(float) > kLastCache;
  const auto run = [&](auto tag) {
    using T = decltype(tag);
    const auto kernel = past ? decay_step_kernel<T, true> : decay_step_kernel<T, false>;
    kernel<<<(unsigned)grid, 256, 0, s>>>(a, lanes_log2, (const T *)c.io.q, (const T *)c.io.k,
                                          (const T *)c.io.v, (T *)c.io.o);
    return hipGetLastError();
  };
  return elt == 1 ? run(bf16()) : run(float());
}

} // namespace kda
