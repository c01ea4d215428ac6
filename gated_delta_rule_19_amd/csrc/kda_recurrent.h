// Launchers of the calls around the KDA recurrence that keep a state of
// their own: the short convolution, the selective scan, and the 8-bit state
// cache (internal; arguments already validated).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kda_seqtab.h"

namespace kda {

// x sigmoid(x) with the hardware's exponential and reciprocal: the activation
// of the convolution and the gate of the scan.  -inf gives NaN (-inf * 0).
__device__ __forceinline__ float silu(float x) {
  return x * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-x * 1.4426950408889634f));
}

// Short convolution, prompts and single tokens.  Strides in elements.
struct ConvCall {
  int32_t D, W, act, num_slots;
  const void *x;
  int64_t x_stride;
  const void *weight, *bias; // [D, W], [D] or null
  const void *init;          // [num_slots, W - 1, D] or null
  void *fin;                 // likewise (step: the state, updated in place)
  const int32_t *slots;      // device [num_seqs] or null (identity)
  void *y;
  int64_t y_stride;
};

// cu: num_seqs + 1 host bounds; ws: seq_table_bytes(num_seqs) of device memory.
hipError_t launch_conv(int elt, const ConvCall &c, int32_t num_seqs, const int64_t *cu, void *ws,
                       hipStream_t s);
hipError_t launch_conv_step(int elt, const ConvCall &c, int32_t rows, hipStream_t s);

// Selective scan, prompts and single tokens.
struct SsmCall {
  int32_t D, N, G, softplus, num_slots;
  const void *x, *delta, *B, *C, *z;
  int64_t x_stride, delta_stride, B_stride, C_stride, z_stride;
  void *y;
  int64_t y_stride;
  const float *A, *skip, *bias;
  const float *init; // [num_slots, D, N] or null
  float *fin;        // likewise (step: the state, updated in place)
  const int32_t *slots;
};

// How a call's sequences are cut: seg tokens per segment (a sequence of at
// most seg tokens is not cut).
struct SsmPlan {
  int64_t seg;    // tokens per segment
  int64_t pairs;  // transition pairs of all cut sequences
  bool lane;      // all states of a channel in one lane, or across 16
  int32_t states; // of a lane
  size_t off_end, off_sum, total; // workspace layout (the table first)
};
SsmPlan ssm_plan(int32_t num_seqs, const int64_t *cu, int32_t D, int32_t N, int32_t G,
                 int32_t split_hint);
int64_t ssm_num_segments(int64_t len, const SsmPlan &p);

hipError_t launch_ssm(int elt, const SsmCall &c, int32_t num_seqs, const int64_t *cu,
                      const SsmPlan &plan, void *ws, hipStream_t s);
hipError_t launch_ssm_step(int elt, const SsmCall &c, int32_t rows, hipStream_t s);

// 8-bit state cache: n items of R rows of L values; item i is src[i] of the
// num_src items read and dst[i] of the num_dst items written (null: i).
struct CacheCall {
  int32_t n, L, format, num_src, num_dst;
  int64_t R;
  const int32_t *src, *dst;
  const float *state_in;
  float *state_out;
  const void *codes_in;
  void *codes_out;
  const float *scales_in;
  float *scales_out;
};
hipError_t launch_state_store(const CacheCall &c, hipStream_t s);
hipError_t launch_state_load(const CacheCall &c, hipStream_t s);

} // namespace kda
