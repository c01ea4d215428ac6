// Argument checks that the calls beside the KDA recurrence share (internal).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kda.h"

namespace kda {

inline bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
inline bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }
inline bool aligned_elt(const void *p, kda_dtype dt) {
  return ((uintptr_t)p & (dt == KDA_BF16 ? 1u : 3u)) == 0;
}
inline int64_t elt_size(kda_dtype dt) { return dt == KDA_BF16 ? 2 : 4; }

// Row strides up to 2^22 elements keep the rows of one tile (64 tokens of at
// most 4 bytes) within the 31-bit offsets the kernels form inside it; offsets
// of whole tiles are 64-bit.
constexpr int64_t kMaxStride = (int64_t)1 << 22;
constexpr int64_t kMaxTokens = (int64_t)1 << 40;

// Packed bounds: 0 first, nondecreasing, no sequence of 2^30 tokens or more.
inline bool good_cu(int32_t num_seqs, const int64_t *cu) {
  if (num_seqs < 0 || num_seqs > (1 << 24) || !cu || cu[0] != 0)
    return false;
  for (int32_t n = 0; n < num_seqs; ++n)
    if (cu[n + 1] < cu[n] || cu[n + 1] - cu[n] >= ((int64_t)1 << 30))
      return false;
  return cu[num_seqs] < kMaxTokens;
}

// A token matrix the call reads or writes.
inline bool good_rows(const void *p, int64_t stride, int64_t width, kda_dtype dt) {
  return p && aligned_elt(p, dt) && stride >= width && stride <= kMaxStride;
}

// What a call reads or writes, as byte ranges: `rows` rows of `width` bytes,
// `pitch` bytes apart.  A dense buffer is one row.  Sizes that the arguments
// merely name may pass 64 bits, so distances are kept in 128.
typedef __int128 wide;
struct Region {
  const void *p;
  wide rows, pitch, width;
};
inline Region rows_of(const void *p, int64_t rows, int64_t stride, int64_t width, int64_t es) {
  return {p, rows, (wide)stride * es, (wide)width * es};
}
inline Region dense(const void *p, wide bytes) { return {p, 1, bytes, bytes}; }
inline wide bytes_of(int64_t a, int64_t b, int64_t c, int64_t es) { return (wide)a * b * c * es; }

// Whether two regions share a byte.  Matrices with one pitch may interleave
// (column ranges of one buffer), and a dense buffer may lie between rows; two
// matrices of different pitch are taken to meet where their extents do.
inline bool overlap(const Region &a, const Region &b) {
  if (!a.p || !b.p || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0)
    return false;
  if (a.rows == 1 && b.rows > 1)
    return overlap(b, a);
  const wide at = (wide)(uintptr_t)b.p - (wide)(uintptr_t)a.p; // b's start in a
  const wide a_end = (a.rows - 1) * a.pitch + a.width;
  const wide end = at + (b.rows - 1) * b.pitch + b.width;
  if (end <= 0 || at >= a_end)
    return false;
  if (a.rows == 1)
    return true;
  if (b.rows == 1) { // in a gap between two rows of a, or not
    const wide lo = at > 0 ? at : 0, row = lo / a.pitch;
    return lo - row * a.pitch < a.width || (row + 1) * a.pitch < end;
  }
  if (a.pitch != b.pitch)
    return true;
  wide off = at % a.pitch; // b's column offset in a's rows
  if (off < 0)
    off += a.pitch;
  return off < a.width || off + b.width > a.pitch;
}

template <size_t N> inline bool overlaps_any(const Region &out, const Region (&in)[N]) {
  for (const Region &r : in)
    if (overlap(out, r))
      return true;
  return false;
}

// Slot table: the state buffers' slice count against the batch's.
inline bool good_slots(const int32_t *slots, int32_t num_slots, int32_t count, bool states) {
  if (!aligned4(slots))
    return false;
  return !states || (num_slots >= 0 && (slots || num_slots >= count));
}

inline kda_status result(hipError_t e) {
  if (e == hipSuccess)
    return KDA_OK;
  // (the launchers' own refusal of a grid past the device's limits)
  return e == hipErrorInvalidConfiguration ? KDA_ERR_INVALID_ARG : KDA_ERR_HIP;
}

inline kda_status check_workspace(size_t need, const void *ws, size_t bytes) {
  if (need == 0)
    return KDA_OK;
  if (!ws || bytes < need)
    return KDA_ERR_WORKSPACE;
  return ((uintptr_t)ws & 255u) == 0 ? KDA_OK : KDA_ERR_INVALID_ARG;
}

} // namespace kda
