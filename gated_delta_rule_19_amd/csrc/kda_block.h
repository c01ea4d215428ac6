// Launchers of a decoder block's calls beside the KDA layer: the decayed
// attention, the block norm, beam selection and state reordering (internal;
// arguments already validated).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kda.h"
#include "kda_seqtab.h"

namespace kda {

// Decayed attention, prompts and single tokens.  Strides in elements.
struct DecayCall {
  int32_t H, num_slots;
  kda_decay_io io;
  const float *init; // [num_slots, H, dk, dv] or null
  float *fin;        // likewise (step: the state, updated in place)
  const int32_t *slots;
};

// How a call's sequences are cut: seg tokens per segment (a sequence of at
// most seg tokens is not cut).
struct DecayPlan {
  int64_t seg;
  int64_t pairs; // transition pairs of all cut sequences
  int waves;     // of a workgroup, 16 value columns each
  bool streams;  // a workgroup for each chain, none cut
  size_t off_state, off_decay, total; // workspace layout (the table first)
};
// `even`: whether all rows start at multiples of 16 bytes, as decay_even has it
// of a call; what its workspace has to hold is more with the one or the other.
DecayPlan decay_plan(int elt, int32_t num_seqs, const int64_t *cu, int32_t H, int32_t dk,
                     int32_t dv, int32_t split_hint, bool even);
bool decay_even(int elt, const kda_decay_io &io);

hipError_t launch_decay(int elt, const DecayCall &c, int32_t num_seqs, const int64_t *cu,
                        const DecayPlan &plan, void *ws, hipStream_t s);
hipError_t launch_decay_step(int elt, const DecayCall &c, int32_t rows, hipStream_t s);

hipError_t launch_block_norm(int elt, int32_t rows, int32_t D, const kda_norm_io &io,
                             hipStream_t s);

struct BeamCall {
  int32_t B, W, V, K, eos, order;
  const void *logits;
  int64_t row_stride;
  const float *scores;
  const uint8_t *finished;
  float *out_scores;
  int32_t *out_parents, *out_tokens;
  uint8_t *out_finished;
};
size_t beam_workspace(int elt, int32_t B, int32_t W, int32_t V, int32_t K);
hipError_t launch_beam_select(int elt, const BeamCall &c, void *ws, hipStream_t s);

// One launch's argument block: the buffers by value.
struct ReorderCall {
  int32_t groups, K, num_states;
  int64_t first; // block of this launch's first one
  const int32_t *parents, *slots;
  void *state[KDA_REORDER_MAX_STATES];
  int64_t bytes[KDA_REORDER_MAX_STATES];
  int32_t num_slots[KDA_REORDER_MAX_STATES];
};
hipError_t launch_state_reorder(const ReorderCall &c, hipStream_t s);

} // namespace kda
