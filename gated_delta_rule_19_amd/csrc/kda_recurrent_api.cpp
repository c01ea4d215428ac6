// Host side of the short convolution, the selective scan and the 8-bit state
// cache: argument checks, then the launches.  Nothing here allocates or
// throws; every check runs before anything is enqueued.
#include "kda.h"
#include "kda_checks.h"
#include "kda_recurrent.h"

using namespace kda;

static_assert(sizeof(kda_ssm_io) == 128, "kda_ssm_io layout");

namespace {

kda_status check_conv(int32_t D, int32_t W, kda_dtype dt, int32_t act) {
  if (dt != KDA_F32 && dt != KDA_BF16)
    return KDA_ERR_UNSUPPORTED;
  if (W < 2 || W > KDA_CONV_MAX_WIDTH)
    return KDA_ERR_UNSUPPORTED;
  if (D < 1 || (act != KDA_ACT_NONE && act != KDA_ACT_SILU))
    return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

kda_status check_ssm(int32_t D, int32_t N, int32_t G, kda_dtype dt, const kda_ssm_io *io) {
  if (dt != KDA_F32 && dt != KDA_BF16)
    return KDA_ERR_UNSUPPORTED;
  if (N > KDA_SSM_MAX_STATES)
    return KDA_ERR_UNSUPPORTED;
  if (D < 1 || N < 1 || G < 1 || D % G != 0 || !io || io->reserved != 0 ||
      (io->delta_softplus != 0 && io->delta_softplus != 1))
    return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

// What a scan reads beside its initial state, and its y.
constexpr size_t kScanInputs = 9;
struct ScanRegions {
  Region in[kScanInputs], y;
};
ScanRegions scan_regions(int64_t rows, int32_t D, int32_t N, int32_t G, kda_dtype dt,
                         const kda_ssm_io *io, const int32_t *slots, int32_t count) {
  const int64_t gn = (int64_t)G * N, es = elt_size(dt);
  return {{rows_of(io->x, rows, io->x_stride, D, es),
           rows_of(io->delta, rows, io->delta_stride, D, es),
           rows_of(io->B, rows, io->B_stride, gn, es), rows_of(io->C, rows, io->C_stride, gn, es),
           rows_of(io->z, rows, io->z_stride, D, es), dense(io->A, bytes_of(D, N, 1, 4)),
           dense(io->D_skip, (wide)D * 4), dense(io->delta_bias, (wide)D * 4),
           dense(slots, (wide)count * 4)},
          rows_of(io->y, rows, io->y_stride, D, es)};
}

// The matrices and parameters of a scan over `rows` tokens.
kda_status check_ssm_io(int64_t rows, int32_t D, int32_t N, int32_t G, kda_dtype dt,
                        const kda_ssm_io *io) {
  const int64_t gn = (int64_t)G * N;
  if (rows > 0 &&
      (!good_rows(io->x, io->x_stride, D, dt) || !good_rows(io->delta, io->delta_stride, D, dt) ||
       !good_rows(io->B, io->B_stride, gn, dt) || !good_rows(io->C, io->C_stride, gn, dt) ||
       !good_rows(io->y, io->y_stride, D, dt) ||
       (io->z && !good_rows(io->z, io->z_stride, D, dt))))
    return KDA_ERR_INVALID_ARG;
  if (!io->A || !aligned16(io->A) || !aligned16(io->D_skip) || !aligned16(io->delta_bias))
    return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

SsmCall ssm_call(int32_t D, int32_t N, int32_t G, const kda_ssm_io *io) {
  SsmCall c{};
  c.D = D;
  c.N = N;
  c.G = G;
  c.softplus = io->delta_softplus;
  c.x = io->x;
  c.delta = io->delta;
  c.B = io->B;
  c.C = io->C;
  c.z = io->z;
  c.y = io->y;
  c.x_stride = io->x_stride;
  c.delta_stride = io->delta_stride;
  c.B_stride = io->B_stride;
  c.C_stride = io->C_stride;
  c.z_stride = io->z_stride;
  c.y_stride = io->y_stride;
  c.A = io->A;
  c.skip = io->D_skip;
  c.bias = io->delta_bias;
  return c;
}

kda_status check_cache(int32_t n, int64_t R, int32_t L, int32_t format, const int32_t *src,
                       int32_t num_src, const int32_t *dst, int32_t num_dst) {
  if (format != KDA_CODE_INT8 && format != KDA_CODE_E4M3)
    return KDA_ERR_UNSUPPORTED;
  if (L > 256)
    return KDA_ERR_UNSUPPORTED;
  if (n < 0 || R < 1 || R > ((int64_t)1 << 31) || L < 1 || num_src < 0 || num_dst < 0 ||
      !aligned4(src) || !aligned4(dst) || (!src && num_src < n) || (!dst && num_dst < n))
    return KDA_ERR_INVALID_ARG;
  return KDA_OK;
}

} // namespace

extern "C" {

size_t kda_short_conv_workspace_size(int32_t num_seqs) {
  return num_seqs < 0 ? 0 : seq_table_bytes(num_seqs);
}

kda_status kda_short_conv(int32_t num_seqs, const int64_t *cu_seqlens_host, int32_t D, int32_t W,
                          kda_dtype dt, const void *x, int64_t x_stride, const void *weight,
                          const void *bias, int32_t act, const void *initial_state,
                          void *final_state, const int32_t *slots, int32_t num_slots, void *y,
                          int64_t y_stride, void *workspace, size_t workspace_bytes,
                          void *stream) {
  kda_status st = check_conv(D, W, dt, act);
  if (st != KDA_OK)
    return st;
  if (!good_cu(num_seqs, cu_seqlens_host) ||
      !good_slots(slots, num_slots, num_seqs, initial_state || final_state))
    return KDA_ERR_INVALID_ARG;
  if (num_seqs == 0)
    return KDA_OK;
  const int64_t T = cu_seqlens_host[num_seqs], es = elt_size(dt);
  if (T > 0 && (!good_rows(x, x_stride, D, dt) || !good_rows(y, y_stride, D, dt)))
    return KDA_ERR_INVALID_ARG;
  if (!weight || !aligned16(weight) || !aligned16(bias) || !aligned16(initial_state) ||
      !aligned16(final_state))
    return KDA_ERR_INVALID_ARG;
  const size_t need = seq_table_bytes(num_seqs);
  const wide pool = bytes_of(num_slots, W - 1, D, es);
  const Region in_x = rows_of(x, T, x_stride, D, es), out_y = rows_of(y, T, y_stride, D, es),
               in_w = dense(weight, bytes_of(D, W, 1, es)), in_b = dense(bias, (wide)D * es),
               init = dense(initial_state, pool), fin = dense(final_state, pool),
               table = dense(slots, (wide)num_seqs * 4);
  if (overlaps_any(out_y, {in_x, in_w, in_b, init, fin, table}) ||
      overlaps_any(fin, {in_x, in_w, in_b, table}) ||
      (initial_state != final_state && overlap(init, fin)))
    return KDA_ERR_INVALID_ARG;
  st = check_workspace(need, workspace, workspace_bytes);
  if (st != KDA_OK)
    return st;
  if (overlaps_any(dense(workspace, need), {in_x, out_y, in_w, in_b, init, fin, table}))
    return KDA_ERR_INVALID_ARG;
  ConvCall c{};
  c.D = D;
  c.W = W;
  c.act = act;
  c.num_slots = num_slots;
  c.x = x;
  c.x_stride = x_stride;
  c.weight = weight;
  c.bias = bias;
  c.init = initial_state;
  c.fin = final_state;
  c.slots = slots;
  c.y = y;
  c.y_stride = y_stride;
  return result(launch_conv(dt == KDA_BF16 ? 1 : 0, c, num_seqs, cu_seqlens_host, workspace,
                            (hipStream_t)stream));
}

kda_status kda_short_conv_step(int32_t N, int32_t D, int32_t W, kda_dtype dt, const void *x,
                               int64_t x_stride, const void *weight, const void *bias,
                               int32_t act, void *state, const int32_t *slots, int32_t num_slots,
                               void *y, int64_t y_stride, void *stream) {
  const kda_status st = check_conv(D, W, dt, act);
  if (st != KDA_OK)
    return st;
  if (N < 0 || !good_slots(slots, num_slots, N, true))
    return KDA_ERR_INVALID_ARG;
  if (N == 0)
    return KDA_OK;
  if (!good_rows(x, x_stride, D, dt) || !good_rows(y, y_stride, D, dt) || !weight || !state ||
      !aligned16(weight) || !aligned16(bias) || !aligned16(state))
    return KDA_ERR_INVALID_ARG;
  const int64_t es = elt_size(dt);
  const Region in_x = rows_of(x, N, x_stride, D, es), out_y = rows_of(y, N, y_stride, D, es),
               in_w = dense(weight, bytes_of(D, W, 1, es)), in_b = dense(bias, (wide)D * es),
               pool = dense(state, bytes_of(num_slots, W - 1, D, es)),
               table = dense(slots, (wide)N * 4);
  if (overlaps_any(out_y, {in_w, in_b, pool, table}) ||
      overlaps_any(pool, {in_x, in_w, in_b, table}) ||
      (!(x == y && x_stride == y_stride) && overlap(out_y, in_x)))
    return KDA_ERR_INVALID_ARG;
  ConvCall c{};
  c.D = D;
  c.W = W;
  c.act = act;
  c.num_slots = num_slots;
  c.x = x;
  c.x_stride = x_stride;
  c.weight = weight;
  c.bias = bias;
  c.fin = state;
  c.slots = slots;
  c.y = y;
  c.y_stride = y_stride;
  return result(launch_conv_step(dt == KDA_BF16 ? 1 : 0, c, N, (hipStream_t)stream));
}

size_t kda_selective_scan_workspace_size(int32_t num_seqs, const int64_t *cu_seqlens_host,
                                         int32_t D, int32_t N, int32_t G, int32_t split_hint) {
  if (!good_cu(num_seqs, cu_seqlens_host) || D < 1 || N < 1 || N > KDA_SSM_MAX_STATES || G < 1 ||
      D % G != 0 || split_hint < 0)
    return 0;
  return ssm_plan(num_seqs, cu_seqlens_host, D, N, G, split_hint).total;
}

kda_status kda_selective_scan(int32_t num_seqs, const int64_t *cu_seqlens_host, int32_t D,
                              int32_t N, int32_t G, kda_dtype dt, const kda_ssm_io *io,
                              const float *initial_state, float *final_state,
                              const int32_t *slots, int32_t num_slots, int32_t split_hint,
                              void *workspace, size_t workspace_bytes, void *stream) {
  kda_status st = check_ssm(D, N, G, dt, io);
  if (st != KDA_OK)
    return st;
  if (!good_cu(num_seqs, cu_seqlens_host) || split_hint < 0 ||
      !good_slots(slots, num_slots, num_seqs, initial_state || final_state))
    return KDA_ERR_INVALID_ARG;
  if (num_seqs == 0)
    return KDA_OK;
  const int64_t T = cu_seqlens_host[num_seqs];
  st = check_ssm_io(T, D, N, G, dt, io);
  if (st != KDA_OK)
    return st;
  if (!aligned16(initial_state) || !aligned16(final_state))
    return KDA_ERR_INVALID_ARG;
  const ScanRegions r = scan_regions(T, D, N, G, dt, io, slots, num_seqs);
  const wide pool = bytes_of(num_slots, D, N, sizeof(float));
  const Region init = dense(initial_state, pool), fin = dense(final_state, pool);
  if (overlaps_any(r.y, r.in) || overlaps_any(fin, r.in) || overlaps_any(r.y, {init, fin}) ||
      (initial_state != final_state && overlap(init, fin)))
    return KDA_ERR_INVALID_ARG;
  const SsmPlan plan = ssm_plan(num_seqs, cu_seqlens_host, D, N, G, split_hint);
  st = check_workspace(plan.total, workspace, workspace_bytes);
  if (st != KDA_OK)
    return st;
  const Region ws = dense(workspace, plan.total);
  if (overlaps_any(ws, r.in) || overlaps_any(ws, {r.y, init, fin}))
    return KDA_ERR_INVALID_ARG;
  SsmCall c = ssm_call(D, N, G, io);
  c.init = initial_state;
  c.fin = final_state;
  c.slots = slots;
  c.num_slots = num_slots;
  return result(launch_ssm(dt == KDA_BF16 ? 1 : 0, c, num_seqs, cu_seqlens_host, plan, workspace,
                           (hipStream_t)stream));
}

kda_status kda_selective_scan_step(int32_t rows, int32_t D, int32_t N, int32_t G, kda_dtype dt,
                                   const kda_ssm_io *io, float *state, const int32_t *slots,
                                   int32_t num_slots, void *stream) {
  kda_status st = check_ssm(D, N, G, dt, io);
  if (st != KDA_OK)
    return st;
  if (rows < 0 || !good_slots(slots, num_slots, rows, true))
    return KDA_ERR_INVALID_ARG;
  if (rows == 0)
    return KDA_OK;
  st = check_ssm_io(rows, D, N, G, dt, io);
  if (st != KDA_OK)
    return st;
  if (!state || !aligned16(state))
    return KDA_ERR_INVALID_ARG;
  const ScanRegions r = scan_regions(rows, D, N, G, dt, io, slots, rows);
  const Region pool = dense(state, bytes_of(num_slots, D, N, sizeof(float)));
  if (overlaps_any(r.y, r.in) || overlaps_any(pool, r.in) || overlap(r.y, pool))
    return KDA_ERR_INVALID_ARG;
  SsmCall c = ssm_call(D, N, G, io);
  c.fin = state;
  c.slots = slots;
  c.num_slots = num_slots;
  return result(launch_ssm_step(dt == KDA_BF16 ? 1 : 0, c, rows, (hipStream_t)stream));
}

kda_status kda_state_store(int32_t n, int64_t R, int32_t L, int32_t format, const float *state,
                           const int32_t *src, int32_t num_src, void *codes, float *scales,
                           const int32_t *dst, int32_t num_dst, void *stream) {
  const kda_status st = check_cache(n, R, L, format, src, num_src, dst, num_dst);
  if (st != KDA_OK)
    return st;
  if (n == 0)
    return KDA_OK;
  if (!state || !codes || !scales || !aligned4(state) || !aligned4(scales))
    return KDA_ERR_INVALID_ARG;
  const Region st_r = dense(state, bytes_of(num_src, R, L, sizeof(float))),
               codes_r = dense(codes, bytes_of(num_dst, R, L, 1)),
               scales_r = dense(scales, bytes_of(num_dst, R, 1, sizeof(float))),
               src_r = dense(src, (wide)n * 4), dst_r = dense(dst, (wide)n * 4);
  if (overlaps_any(codes_r, {st_r, scales_r, src_r, dst_r}) ||
      overlaps_any(scales_r, {st_r, src_r, dst_r}))
    return KDA_ERR_INVALID_ARG;
  CacheCall c{};
  c.n = n;
  c.R = R;
  c.L = L;
  c.format = format;
  c.src = src;
  c.num_src = num_src;
  c.dst = dst;
  c.num_dst = num_dst;
  c.state_in = state;
  c.codes_out = codes;
  c.scales_out = scales;
  return result(launch_state_store(c, (hipStream_t)stream));
}

kda_status kda_state_load(int32_t n, int64_t R, int32_t L, int32_t format, const void *codes,
                          const float *scales, const int32_t *src, int32_t num_src, float *state,
                          const int32_t *dst, int32_t num_dst, void *stream) {
  const kda_status st = check_cache(n, R, L, format, src, num_src, dst, num_dst);
  if (st != KDA_OK)
    return st;
  if (n == 0)
    return KDA_OK;
  if (!state || !codes || !scales || !aligned4(state) || !aligned4(scales))
    return KDA_ERR_INVALID_ARG;
  const Region st_r = dense(state, bytes_of(num_dst, R, L, sizeof(float))),
               codes_r = dense(codes, bytes_of(num_src, R, L, 1)),
               scales_r = dense(scales, bytes_of(num_src, R, 1, sizeof(float))),
               src_r = dense(src, (wide)n * 4), dst_r = dense(dst, (wide)n * 4);
  if (overlaps_any(st_r, {codes_r, scales_r, src_r, dst_r}))
    return KDA_ERR_INVALID_ARG;
  CacheCall c{};
  c.n = n;
  c.R = R;
  c.L = L;
  c.format = format;
  c.src = src;
  c.num_src = num_src;
  c.dst = dst;
  c.num_dst = num_dst;
  c.codes_in = codes;
  c.scales_in = scales;
  c.state_out = state;
  return result(launch_state_load(c, (hipStream_t)stream));
}

} // extern "C"
