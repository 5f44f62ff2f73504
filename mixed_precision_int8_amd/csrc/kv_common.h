// Shared by the kernels of the int8 key/value cache: the cache and batch as the
// kernels see them, and the mapping from a workgroup to its sequence.
#pragma once

#include "device_util.h"
#include "internal.h"

namespace llmint8 {

// Tokens of sequence b in this call: rows [row0, row0 + n), positions
// [len - n, len). Every number is cut to what the buffers hold, so that no
// content of cu, len or table makes a kernel leave them: cu to [0, T], n to
// >= 0, len to [0, width * page].
struct KvSeq {
  int b, row0, n, len;
};

__device__ __forceinline__ KvSeq kv_seq(const KvBatch& s, int page_shift, int b) {
  KvSeq q;
  const int c0 = min(max(s.cu[b], 0), s.T), c1 = min(max(s.cu[b + 1], 0), s.T);
  q.b = b;
  q.row0 = c0;
  q.n = max(c1 - c0, 0);
  const int64_t room = (int64_t)s.width << page_shift;
  q.len = (int)min((int64_t)max(s.len[b], 0), room);
  return q;
}

// The sequence that work item `item` belongs to, where sequence b owns the items
// from (cu[b] * per >> shift) + slack * b on. A sequence of n rows then has at
// least (n * per >> shift) + slack items, which covers the tiles of 2^shift that
// its n * per rows fill (slack 1) or the pages of 2^shift that n tokens reach
// (slack 2), with no table of tile counts. Whole workgroup: the sequences
// are counted in parallel, one round of loads for every kThreads of them.
// Returns b and sets *first to its first item; -1 where no sequence owns the item
// (cu starts late, or falls).
template <int kThreads>
__device__ __forceinline__ int kv_find(const KvBatch& s, int item, int per, int shift, int slack,
                                       int* first) {
  int b = -1;
  for (int b0 = 0; b0 < s.B; b0 += kThreads) {
    const int i = b0 + (int)threadIdx.x;
    bool mine = false;
    if (i < s.B) {
      const int64_t c = min(max(s.cu[i], 0), s.T);
      mine = (c * per >> shift) + (int64_t)slack * i <= item;
    }
    b += __syncthreads_count(mine);
  }
  if (b < 0) return b;
  const int64_t c = min(max(s.cu[b], 0), s.T);
  *first = (int)((c * per >> shift) + (int64_t)slack * b);
  return b;
}

// Page of token `tok` of sequence b, or -1 where the table names none that exists.
__device__ __forceinline__ int kv_page(const KvBatch& s, int b, int entry, int64_t pages) {
  const int p = s.table[(int64_t)b * s.width + min(entry, s.width - 1)];
  return (entry < s.width && (uint32_t)p < (uint64_t)pages) ? p : -1;
}

}  // namespace llmint8
