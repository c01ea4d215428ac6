// Host side of a decoder block's calls beside the KDA layer: the decayed
// attention, the block norm, beam selection and state reordering.  Argument
// checks, then the launches; nothing here allocates or throws, and every
// check runs before anything is enqueued.
#include "kda.h"
#include "kda_block.h"
#include "kda_checks.h"

#include <algorithm>

using namespace kda;

static_assert(sizeof(kda_decay_io) == 104, "kda_decay_io layout");
static_assert(sizeof(kda_norm_io) == 120, "kda_norm_io layout");

namespace {

bool good_dt(kda_dtype dt) { return dt == KDA_F32 || dt == KDA_BF16; }
int elt_of(kda_dtype dt) { return dt == KDA_BF16 ? 1 : 0; }

// ---- decayed attention --------------------------------------------------------

kda_status check_decay(int32_t H, int32_t dk, int32_t dv, kda_dtype dt) {
  if (!good_dt(dt) || dk > KDA_DECAY_MAX_DIM || dv > KDA_DECAY_MAX_DIM)
    return KDA_ERR_UNSUPPORTED;
  return H < 1 || H > (1 << 24) || dk < 1 || dv < 1 ? KDA_ERR_INVALID_ARG : KDA_OK;
}

kda_status check_decay_io(int64_t rows, int32_t H, kda_dtype dt, const kda_decay_io *io) {
  if (!io)
    return KDA_ERR_INVALID_ARG;
  const kda_status st = check_decay(H, io->dk, io->dv, dt);
  if (st != KDA_OK)
    return st;
  for (int32_t few : {io->Hq, io->Hk, io->Hv})
    if (few < 1 || few > H || H % few != 0)
      return KDA_ERR_INVALID_ARG;
  if (rows == 0)
    return KDA_OK;
  const int64_t dk = io->dk, dv = io->dv;
  if (!good_rows(io->q, io->q_stride, io->Hq * dk, dt) ||
      !good_rows(io->k, io->k_stride, io->Hk * dk, dt) ||
      !good_rows(io->v, io->v_stride, io->Hv * dv, dt) ||
      !good_rows(io->o, io->o_stride, H * dv, dt) || !io->g || !aligned4(io->g) ||
      (io->g_stride != 0 && (io->g_stride < H || io->g_stride > kMaxStride)))
    return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

struct DecayRegions {
  Region in[5], o;
};
DecayRegions decay_regions(int64_t rows, int32_t H, kda_dtype dt, const kda_decay_io *io,
                           const int32_t *slots, int32_t count) {
  const int64_t es = elt_size(dt), dk = io->dk, dv = io->dv;
  return {{rows_of(io->q, rows, io->q_stride, io->Hq * dk, es),
           rows_of(io->k, rows, io->k_stride, io->Hk * dk, es),
           rows_of(io->v, rows, io->v_stride, io->Hv * dv, es),
           rows_of(io->g, io->g_stride ? rows : rows > 0, io->g_stride ? io->g_stride : H, H, 4),
           dense(slots, (wide)count * 4)},
          rows_of(io->o, rows, io->o_stride, H * dv, es)};
}

DecayCall decay_call(int32_t H, const kda_decay_io *io, const int32_t *slots, int32_t num_slots) {
  DecayCall c{};
  c.H = H;
  c.num_slots = num_slots;
  c.io = *io;
  c.slots = slots;
  return c;
}

} // namespace

extern "C" {

size_t kda_decay_attention_workspace_size(int32_t num_seqs, const int64_t *cu_seqlens_host,
                                          int32_t H, int32_t dk, int32_t dv, kda_dtype dt,
                                          int32_t split_hint) {
  if (!good_cu(num_seqs, cu_seqlens_host) || check_decay(H, dk, dv, dt) != KDA_OK ||
      split_hint < 0)
    return 0;
  size_t most = 0; // (a call's pointers and strides are not known yet)
  for (bool even : {false, true})
    most = std::max(most, decay_plan(elt_of(dt), num_seqs, cu_seqlens_host, H, dk, dv, split_hint,
                                     even).total);
  return most;
}

kda_status kda_decay_attention(int32_t num_seqs, const int64_t *cu_seqlens_host, int32_t H,
                               kda_dtype dt, const kda_decay_io *io, const float *initial_state,
                               float *final_state, const int32_t *slots, int32_t num_slots,
                               int32_t split_hint, void *workspace, size_t workspace_bytes,
                               void *stream) {
  if (!good_dt(dt))
    return KDA_ERR_UNSUPPORTED;
  if (!good_cu(num_seqs, cu_seqlens_host) || split_hint < 0 ||
      !good_slots(slots, num_slots, num_seqs, initial_state || final_state))
    return KDA_ERR_INVALID_ARG;
  const int64_t T = cu_seqlens_host[num_seqs];
  kda_status st = check_decay_io(T, H, dt, io);
  if (st != KDA_OK || num_seqs == 0)
    return st;
  if (!aligned16(initial_state) || !aligned16(final_state))
    return KDA_ERR_INVALID_ARG;
  const DecayRegions r = decay_regions(T, H, dt, io, slots, num_seqs);
  const wide pool = bytes_of(num_slots, H, (int64_t)io->dk * io->dv, sizeof(float));
  const Region init = dense(initial_state, pool), fin = dense(final_state, pool);
  if (overlaps_any(r.o, r.in) || overlaps_any(fin, r.in) || overlaps_any(r.o, {init, fin}) ||
      (initial_state != final_state && overlap(init, fin)))
    return KDA_ERR_INVALID_ARG;
  const DecayPlan plan = decay_plan(elt_of(dt), num_seqs, cu_seqlens_host, H, io->dk, io->dv,
                                    split_hint, decay_even(elt_of(dt), *io));
  st = check_workspace(plan.total, workspace, workspace_bytes);
  if (st != KDA_OK)
    return st;
  const Region ws = dense(workspace, plan.total);
  if (overlaps_any(ws, r.in) || overlaps_any(ws, {r.o, init, fin}))
    return KDA_ERR_INVALID_ARG;
  DecayCall c = decay_call(H, io, slots, num_slots);
  c.init = initial_state;
  c.fin = final_state;
  return result(launch_decay(elt_of(dt), c, num_seqs, cu_seqlens_host, plan, workspace,
                             (hipStream_t)stream));
}

kda_status kda_decay_attention_step(int32_t rows, int32_t H, kda_dtype dt, const kda_decay_io *io,
                                    float *state, const int32_t *slots, int32_t num_slots,
                                    void *stream) {
  if (!good_dt(dt))
    return KDA_ERR_UNSUPPORTED;
  if (rows < 0 || !good_slots(slots, num_slots, rows, true))
    return KDA_ERR_INVALID_ARG;
  const kda_status st = check_decay_io(rows, H, dt, io);
  if (st != KDA_OK || rows == 0)
    return st;
  if (!state || !aligned16(state))
    return KDA_ERR_INVALID_ARG;
  const DecayRegions r = decay_regions(rows, H, dt, io, slots, rows);
  const Region pool =
      dense(state, bytes_of(num_slots, H, (int64_t)io->dk * io->dv, sizeof(float)));
  if (overlaps_any(r.o, r.in) || overlaps_any(pool, r.in) || overlap(r.o, pool))
    return KDA_ERR_INVALID_ARG;
  DecayCall c = decay_call(H, io, slots, num_slots);
  c.fin = state;
  return result(launch_decay_step(elt_of(dt), c, rows, (hipStream_t)stream));
}

// ---- block norm ------------------------------------------------------------------

kda_status kda_block_norm(int32_t rows, int32_t D, kda_dtype dt, const kda_norm_io *io,
                          void *stream) {
  if (!good_dt(dt) || D > KDA_NORM_MAX_WIDTH)
    return KDA_ERR_UNSUPPORTED;
  if (rows < 0 || D < 1 || !io)
    return KDA_ERR_INVALID_ARG;
  if (rows == 0)
    return KDA_OK;
  if ((!io->y && !io->residual_out) || (io->y && !io->weight))
    return KDA_ERR_INVALID_ARG;
  if ((io->residual || io->residual_out) && !good_dt(io->residual_dt))
    return KDA_ERR_UNSUPPORTED;
  const kda_dtype rt = io->residual_dt;
  const auto bad = [&](const void *p, int64_t stride, kda_dtype t) {
    return p && !good_rows(p, stride, D, t);
  };
  if (!io->x || bad(io->x, io->x_stride, dt) || bad(io->gate, io->gate_stride, dt) ||
      bad(io->residual, io->residual_stride, rt) ||
      bad(io->residual_out, io->residual_out_stride, rt) || bad(io->y, io->y_stride, dt) ||
      !aligned16(io->post_weight) || !aligned16(io->weight) || !aligned16(io->scale))
    return KDA_ERR_INVALID_ARG;
  const int64_t es = elt_size(dt), rs = elt_size(rt);
  const Region x = rows_of(io->x, rows, io->x_stride, D, es),
               gate = rows_of(io->gate, rows, io->gate_stride, D, es),
               res = rows_of(io->residual, rows, io->residual_stride, D, rs),
               ro = rows_of(io->residual_out, rows, io->residual_out_stride, D, rs),
               y = rows_of(io->y, rows, io->y_stride, D, es);
  const Region w[3] = {dense(io->post_weight, (wide)D * 4), dense(io->weight, (wide)D * 4),
                       dense(io->scale, (wide)D * 4)};
  // an output may be an input itself: every element is read by the lane that
  // writes it, before it does
  const auto clash = [&](const Region &out, kda_dtype ot, int64_t ostride, const Region &in,
                         kda_dtype it, int64_t istride) {
    return !(out.p == in.p && ot == it && ostride == istride) && overlap(out, in);
  };
  const auto clashes = [&](const Region &out, kda_dtype ot, int64_t stride) {
    return overlaps_any(out, w) || clash(out, ot, stride, x, dt, io->x_stride) ||
           clash(out, ot, stride, gate, dt, io->gate_stride) ||
           clash(out, ot, stride, res, rt, io->residual_stride);
  };
  if (clashes(ro, rt, io->residual_out_stride) || clashes(y, dt, io->y_stride) || overlap(ro, y))
    return KDA_ERR_INVALID_ARG;
  return result(launch_block_norm(elt_of(dt), rows, D, *io, (hipStream_t)stream));
}

// ---- beams -------------------------------------------------------------------------

static kda_status check_beam(int32_t B, int32_t W, int32_t V, int32_t K, kda_dtype dt) {
  if (!good_dt(dt) || W > KDA_BEAM_MAX || K > KDA_BEAM_MAX)
    return KDA_ERR_UNSUPPORTED;
  return B < 0 || B > (1 << 24) || W < 1 || V < 1 || K < 1 || (int64_t)W * V < K
             ? KDA_ERR_INVALID_ARG
             : KDA_OK;
}

size_t kda_beam_select_workspace_size(int32_t B, int32_t W, int32_t V, int32_t K, kda_dtype dt) {
  return check_beam(B, W, V, K, dt) != KDA_OK ? 0 : beam_workspace(elt_of(dt), B, W, V, K);
}

kda_status kda_beam_select(int32_t B, int32_t W, int32_t V, int32_t K, kda_dtype dt,
                           const void *logits, int64_t row_stride, const float *scores,
                           const uint8_t *finished, int32_t eos, int32_t order,
                           float *out_scores, int32_t *out_parents, int32_t *out_tokens,
                           uint8_t *out_finished, void *workspace, size_t workspace_bytes,
                           void *stream) {
  kda_status st = check_beam(B, W, V, K, dt);
  if (st != KDA_OK)
    return st;
  if ((order != KDA_BEAM_BY_SCORE && order != KDA_BEAM_BY_ROW) ||
      (order == KDA_BEAM_BY_ROW && K < W) || eos < -1 || eos >= V || (eos < 0 && finished))
    return KDA_ERR_INVALID_ARG;
  if (B == 0)
    return KDA_OK;
  if (!logits || !aligned_elt(logits, dt) || row_stride < V || row_stride > ((int64_t)1 << 31) ||
      !scores || !aligned4(scores) || !out_scores || !out_parents || !out_tokens ||
      !out_finished || !aligned4(out_scores) || !aligned4(out_parents) || !aligned4(out_tokens))
    return KDA_ERR_INVALID_ARG;
  const size_t need = beam_workspace(elt_of(dt), B, W, V, K);
  st = check_workspace(need, workspace, workspace_bytes);
  if (st != KDA_OK)
    return st;
  const wide bw = (wide)B * W, bk = (wide)B * K;
  const Region in[3] = {rows_of(logits, (int64_t)bw, row_stride, V, elt_size(dt)),
                        dense(scores, bw * 4), dense(finished, bw)};
  const Region out[5] = {dense(out_scores, bk * 4), dense(out_parents, bk * 4),
                         dense(out_tokens, bk * 4), dense(out_finished, bk),
                         dense(workspace, need)};
  for (int i = 0; i < 5; ++i) {
    if (overlaps_any(out[i], in))
      return KDA_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(out[i], out[j]))
        return KDA_ERR_INVALID_ARG;
  }
  BeamCall c{};
  c.B = B;
  c.W = W;
  c.V = V;
  c.K = K;
  c.eos = eos;
  c.order = order;
  c.logits = logits;
  c.row_stride = row_stride;
  c.scores = scores;
  c.finished = finished;
  c.out_scores = out_scores;
  c.out_parents = out_parents;
  c.out_tokens = out_tokens;
  c.out_finished = out_finished;
  return result(launch_beam_select(elt_of(dt), c, workspace, (hipStream_t)stream));
}

kda_status kda_state_reorder(int32_t groups, int32_t K, const int32_t *parents,
                             const int32_t *slots, int32_t num_states, void *const *states_host,
                             const int64_t *slice_bytes_host, const int32_t *num_slots_host,
                             void *stream) {
  if (K > KDA_BEAM_MAX || num_states > KDA_REORDER_MAX_STATES)
    return KDA_ERR_UNSUPPORTED;
  if (groups < 0 || K < 1 || num_states < 0 ||
      (num_states > 0 && (!states_host || !slice_bytes_host || !num_slots_host)))
    return KDA_ERR_INVALID_ARG;
  if (groups == 0 || num_states == 0)
    return KDA_OK;
  const int64_t rows = (int64_t)groups * K;
  if (!parents || !aligned4(parents) || !aligned4(slots) || rows > INT32_MAX)
    return KDA_ERR_INVALID_ARG;
  ReorderCall c{};
  c.groups = groups;
  c.K = K;
  c.parents = parents;
  c.slots = slots;
  Region r[KDA_REORDER_MAX_STATES];
  const Region tables[2] = {dense(parents, (wide)rows * 4), dense(slots, (wide)rows * 4)};
  for (int i = 0; i < num_states; ++i) {
    const int64_t bytes = slice_bytes_host[i];
    const int32_t held = num_slots_host[i];
    if (bytes < 0 || bytes > ((int64_t)1 << 46) || held < 0 || (!slots && held < rows))
      return KDA_ERR_INVALID_ARG;
    if (bytes == 0 || held == 0)
      continue;
    if (!states_host[i])
      return KDA_ERR_INVALID_ARG;
    const Region s = dense(states_host[i], bytes_of(held, bytes, 1, 1));
    if (overlaps_any(s, tables))
      return KDA_ERR_INVALID_ARG;
    for (int j = 0; j < c.num_states; ++j)
      if (overlap(s, r[j]))
        return KDA_ERR_INVALID_ARG;
    r[c.num_states] = s;
    c.state[c.num_states] = states_host[i];
    c.bytes[c.num_states] = bytes;
    c.num_slots[c.num_states++] = held;
  }
  if (c.num_states == 0 || K == 1) // (one row has no other parent)
    return KDA_OK;
  return result(launch_state_reorder(c, (hipStream_t)stream));
}

} // extern "C"
