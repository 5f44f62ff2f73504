// Shared by the kernels of the int8 key/value cache: the cache and batch as the
// kernels see them, and the mapping from a workgroup to its sequence.
#pragma once

#include "device_util.h"
#include "kv_internal.h"

namespace llmint8 {

typedef int v2i __attribute__((ext_vector_type(2)));

// A value that all lanes hold, moved to a scalar register.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32));
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// the larger of two, NaN if one of them is (fmaxf takes the other)
__device__ __forceinline__ float max_or_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }

__device__ __forceinline__ KvSeq kv_seq(const KvBatch& s, int page_shift, int b) {
  return kv_seq_of(b, s.cu[b], s.cu[b + 1], s.len[b], s.T, (int64_t)s.width << page_shift);
}

// kv_seq of a sequence that all lanes ask for
__device__ __forceinline__ KvSeq kv_seq_uniform(const KvBatch& s, int page_shift, int b) {
  KvSeq q = kv_seq(s, page_shift, b);
  q.b = uniform(q.b);
  q.row0 = uniform(q.row0);
  q.n = uniform(q.n);
  q.len = uniform(q.len);
  q.pos0 = uniform(q.pos0);
  return q;
}

// The sequence that owns work item `item` (kv_items), found with no table of counts.
// Whole workgroup: the sequences are counted in parallel, one round of loads for
// every kThreads of them, and the owner hands its numbers, loaded in the same
// round, to the others (sh). Sets *index to the item's number in the sequence and
// *count to the sequence's items; false where no sequence owns the item (it is
// past the last one's, or cu starts late or falls).
template <int kThreads>
__device__ __forceinline__ bool kv_find(const KvBatch& s, int page_shift, int item, int per, int shift,
                                        int (&sh)[6], KvSeq* out, int* index, int* count) {
  if (s.B == 1) {
    *out = kv_seq_uniform(s, page_shift, 0);
    const KvItems own = kv_items(0, out->row0, out->n, per, shift);
    *index = kv_item_index(own, item);
    *count = own.count;
    return *index >= 0;
  }
  int b = -1;
  for (int b0 = 0; b0 < s.B; b0 += kThreads) {
    const int i = b0 + (int)threadIdx.x;
    const int lane = min(i, s.B - 1);
    const KvSeq q = kv_seq(s, page_shift, lane);
    const KvItems own = kv_items(lane, q.row0, q.n, per, shift);
    const int mine = __syncthreads_count(i < s.B && own.first <= item);
    if (mine > 0 && (int)threadIdx.x == mine - 1) {
      sh[0] = q.row0;
      sh[1] = q.n;
      sh[2] = q.len;
      sh[3] = own.first;
      sh[4] = own.count;
      sh[5] = q.pos0;
    }
    b += mine;
    if (mine < min(kThreads, s.B - b0)) break;
  }
  if (b < 0) return false;
  __syncthreads();
  out->b = b;
  out->row0 = uniform(sh[0]);
  out->n = uniform(sh[1]);
  out->len = uniform(sh[2]);
  out->pos0 = uniform(sh[5]);
  const KvItems own{uniform(sh[3]), uniform(sh[4])};
  *index = kv_item_index(own, item);
  *count = own.count;
  return *index >= 0;
}

// Page that the table names for the tokens of an entry; may be any number. Past the
// table's end, where a tile may reach but no token is, the last one's.
__device__ __forceinline__ int kv_entry(const KvBatch& s, int b, int entry) {
  return s.table[(int64_t)b * s.width + min(entry, s.width - 1)];
}
// The page itself, or -1 where there is none of that number.
__device__ __forceinline__ int kv_page(int number, int64_t pages) {
  return (uint32_t)number < (uint64_t)pages ? number : -1;
}
// The page of an entry that may be past the table's end, where there is none.
__device__ __forceinline__ int kv_entry_page(const KvBatch& s, int b, int entry, int64_t pages) {
  return entry < s.width ? kv_page(kv_entry(s, b, entry), pages) : -1;
}

}  // namespace llmint8
