// Packed-sequence tables that travel with the launch.
//
// The calls that walk packed sequences tile by tile need, on the device, the
// sequences' bounds and the number of tiles before each of them.  Up to
// kInlineSeqs sequences the tables are the kernel's first argument, by value:
// nothing is uploaded, the call takes no workspace and may be captured into a
// graph (the argument block is part of the recorded launch).  Above that,
// seq_table_kernel launches write them to the workspace, kTablePart
// sequences each, from their own argument blocks; the tables are again part
// of the recorded launches, never of a host buffer that a later call reuses.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace kda {

constexpr int kInlineSeqs = 64;  // 65 entries of 32 bytes: 2080 of the 4096 argument bytes
constexpr int kTablePart = 100;  // entries per table-writing launch: 3200 bytes
constexpr int kCounts = 3;

// One sequence: its first token, length and number, and the blocks of the
// entries before it in each of a call's (at most three) launches.  The entry
// past the last holds the totals.  Inline tables put the longest sequences
// first, so that the longest serial work starts first and the short ones
// fill in behind it; longer tables keep the sequences' order.
struct SeqEntry {
  int64_t tok0;
  int32_t len, seq;
  int32_t blk[kCounts];
  int32_t pad;
};
static_assert(sizeof(SeqEntry) == 32, "SeqEntry layout");

struct SeqTable {
  const SeqEntry *ws; // null: the entries are `in`
  int32_t num_seqs;
  int32_t pad;
  SeqEntry in[kInlineSeqs + 1];
};

struct TablePart {
  SeqEntry e[kTablePart];
};

inline size_t seq_table_bytes(int32_t num_seqs) {
  return num_seqs <= kInlineSeqs
             ? 0
             : (((size_t)num_seqs + 1) * sizeof(SeqEntry) + 255) / 256 * 256;
}

hipError_t launch_table_part(const TablePart &part, int count, SeqEntry *dst, hipStream_t s);

// The table's totals: tiles(length, w) is how many blocks a sequence has in
// launch w.  False when a total passes 2^31 - 1.
template <typename F>
bool seq_totals(int32_t num_seqs, const int64_t *cu, F &&tiles, int64_t (&total)[kCounts]) {
  for (int w = 0; w < kCounts; ++w)
    total[w] = 0;
  for (int32_t n = 0; n < num_seqs; ++n)
    for (int w = 0; w < kCounts; ++w) {
      total[w] += tiles(cu[n + 1] - cu[n], w);
      if (total[w] > INT32_MAX)
        return false;
    }
  return true;
}

// Fills `t` from the host bounds; a long table's launches to `ws`
// (seq_table_bytes of it) are enqueued.
template <typename F>
hipError_t make_seq_table(SeqTable &t, int32_t num_seqs, const int64_t *cu, F &&tiles, void *ws,
                          hipStream_t s) {
  t.num_seqs = num_seqs;
  t.pad = 0;
  t.ws = num_seqs <= kInlineSeqs ? nullptr : (const SeqEntry *)ws;
  int32_t order[kInlineSeqs];
  if (!t.ws)
    for (int32_t n = 0; n < num_seqs; ++n) { // by length, stable
      const int64_t len = cu[n + 1] - cu[n];
      int32_t i = n;
      for (; i > 0 && cu[order[i - 1] + 1] - cu[order[i - 1]] < len; --i)
        order[i] = order[i - 1];
      order[i] = n;
    }
  int64_t at[kCounts] = {};
  TablePart part;
  for (int32_t i = 0; i <= num_seqs; ++i) {
    SeqEntry &e = t.ws ? part.e[i % kTablePart] : t.in[i];
    const int32_t n = t.ws || i == num_seqs ? i : order[i];
    e.tok0 = cu[n];
    e.seq = n;
    e.len = i < num_seqs ? (int32_t)(cu[n + 1] - cu[n]) : 0;
    e.pad = 0;
    for (int w = 0; w < kCounts; ++w) {
      e.blk[w] = (int32_t)at[w];
      at[w] += i < num_seqs ? tiles(cu[n + 1] - cu[n], w) : 0;
    }
    const int filled = i % kTablePart + 1;
    if (t.ws && (filled == kTablePart || i == num_seqs)) {
      const hipError_t err = launch_table_part(part, filled, (SeqEntry *)ws + (i + 1 - filled), s);
      if (err != hipSuccess)
        return err;
    }
  }
  return hipSuccess;
}

#ifdef __HIP_DEVICE_COMPILE__
#define KDA_CONST_AS __attribute__((address_space(4)))
#else
#define KDA_CONST_AS
#endif

// The table as the kernel sees it.  The SeqTable is the kernel's first
// parameter, so inline entries are read straight from the argument block;
// reads are wave-uniform and go through scalar loads.
struct SeqView {
  const KDA_CONST_AS SeqEntry *e;
  int32_t num_seqs;

  __device__ __forceinline__ explicit SeqView(const SeqTable &t) {
#ifdef __HIP_DEVICE_COMPILE__
    const KDA_CONST_AS char *args = (const KDA_CONST_AS char *)__builtin_amdgcn_kernarg_segment_ptr();
    const KDA_CONST_AS SeqEntry *in =
        (const KDA_CONST_AS SeqEntry *)(args + offsetof(SeqTable, in));
    e = t.ws ? (const KDA_CONST_AS SeqEntry *)(uintptr_t)t.ws : in;
#else
    e = nullptr;
#endif
    num_seqs = t.num_seqs;
  }
  __device__ __forceinline__ int64_t tok0(int n) const { return e[n].tok0; }
  __device__ __forceinline__ int32_t len(int n) const { return e[n].len; }
  __device__ __forceinline__ int32_t seq(int n) const { return e[n].seq; }
  __device__ __forceinline__ int32_t blk(int n, int w) const { return e[n].blk[w]; }

  // The entry that block b of launch w belongs to: the last n with
  // blk(n) <= b (entries without blocks share their successor's count).
  __device__ __forceinline__ int find(int b, int w) const {
    int lo = 0, hi = num_seqs;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (e[mid].blk[w] <= b)
        lo = mid;
      else
        hi = mid;
    }
    return lo;
  }
};

} // namespace kda
