// The int8 key/value cache's part of internal.h: admission limits, what the
// kernels take, launchers.
#pragma once

#include "internal.h"
#include "ranges.h"

namespace llmint8 {

// api.cpp: the status of a HIP result (kept for llmint8_last_hip_error), the device's CUs
int abi_hip_status(hipError_t e);
int abi_cu_count();

// The kernels index tokens, rows and work items in 32 bits (a launch has fewer than
// rows + seqs items; positions are below len)
constexpr int64_t kKvMax = int64_t(1) << 29;
constexpr int64_t kKvMaxQHeads = 65536;
constexpr int64_t kKvMaxQRows = int64_t(1) << 30;  // rows times query heads of an attention call
inline int admit_kv_cache(int64_t pages, int64_t heads, int64_t page, int64_t dim) {
  if (pages <= 0 || heads <= 0 || page <= 0 || dim <= 0) return LLMINT8_ERR_INVALID_ARG;
  if (page != 16 && page != 32 && page != 64 && page != 128) return LLMINT8_ERR_UNSUPPORTED;
  if (dim % 16 != 0 || dim > 256 || heads > 4096 || pages >= kTwo31) return LLMINT8_ERR_UNSUPPORTED;
  return LLMINT8_OK;
}
inline int admit_kv_batch(int64_t seqs, int64_t rows, int64_t width, int64_t page) {
  if (seqs < 0 || rows < 0 || width <= 0) return LLMINT8_ERR_INVALID_ARG;
  if (rows > kKvMax || width > kKvMax / page || seqs > kKvMax / (2 * page)) return LLMINT8_ERR_UNSUPPORTED;
  return LLMINT8_OK;
}

// The cache: codes K [pages, heads, page, dim], V [pages, heads, dim, page] and the
// largest magnitudes aK, aV [pages, heads].
struct KvCache {
  int8_t* K;
  int8_t* V;
  float* aK;
  float* aV;
  int64_t pages;
  int heads, dim, page_shift;
};
// The sequences of a call (device arrays) and their sizes.
struct KvBatch {
  const int32_t* cu;     // [B + 1]
  const int32_t* len;    // [B]
  const int32_t* table;  // [B, width]
  int B, T, width;
};
// Tokens of sequence b in this call: rows [row0, row0 + n), positions from pos0 on
// (below 0: rows without one), of a sequence that has tokens [0, len) in pages that
// the table has entries for. Every number is cut to what the buffers hold, so that
// no content of cu, len or table makes a kernel leave them: cu to [0, T], n to >= 0,
// len to [0, width * page]. Positions are those of the whole length: a token past
// the table has no page, and the ones before it keep their places.
struct KvSeq {
  int b, row0, n, len, pos0;
};
__host__ __device__ inline KvSeq kv_seq_of(int b, int cu0, int cu1, int length, int T, int64_t room) {
  KvSeq q;
  cu0 = cu0 < 0 ? 0 : cu0 > T ? T : cu0;
  cu1 = cu1 < 0 ? 0 : cu1 > T ? T : cu1;
  length = length < 0 ? 0 : length;
  q.b = b;
  q.row0 = cu0;
  q.n = cu1 > cu0 ? cu1 - cu0 : 0;
  q.len = length < room ? length : (int)room;
  q.pos0 = length - q.n;
  return q;
}
// The tokens of a sequence's rows that are on page `entry` of its table: positions
// [t0, t1), slot 0 at base; none if t0 >= t1. There may be no such entry.
struct KvOnPage {
  int base, t0, t1;
};
__host__ __device__ inline KvOnPage kv_on_page(const KvSeq& q, int entry, int page_shift) {
  const int end = q.pos0 + q.n;
  if (entry > (end - 1) >> page_shift) return {0, 0, 0};  // where base could leave 32 bits
  const int base = entry << page_shift, left = end - base;
  return {base, q.pos0 > base ? q.pos0 : base, base + (left < 1 << page_shift ? left : 1 << page_shift)};
}

// The work items of a launch: sequence b with rows [row0, row0 + n) owns `count` of
// them from `first` on, enough for the tiles of 2^shift that its n * per rows fill,
// and one less at most than the pages of 2^shift that n tokens reach. With rows
// that follow each other the sequences' items do too; what a launch has beyond the
// last sequence's (rows past cu[seqs]) belongs to none.
struct KvItems {
  int first, count;
};
__host__ __device__ inline KvItems kv_items(int b, int row0, int n, int per, int shift) {
  KvItems i;
  i.first = (int)(((int64_t)row0 * per) >> shift) + b;
  i.count = (int)(((int64_t)(row0 + n) * per) >> shift) + b + 1 - i.first;
  return i;
}
// An item's number in its sequence, -1 if it is not one of its own.
__host__ __device__ inline int kv_item_index(const KvItems& i, int item) {
  return item >= i.first && item - i.first < i.count ? item - i.first : -1;
}
// The pages of an item where per = 1 and a tile is a page: the sequence's last item
// takes the page past the others' as well, if there is one.
struct KvEntries {
  int first, count;
};
__host__ __device__ inline KvEntries kv_item_entries(int pos0, int index, int count, int page_shift) {
  return {((pos0 > 0 ? pos0 : 0) >> page_shift) + index, index + 1 == count ? 2 : 1};
}
// 16-bit rows [T, heads, dim]: strides in elements, channels dense
struct KvRows {
  uint16_t* p;
  int64_t token, head;
};
struct KvAppendArgs {
  KvCache c;
  KvBatch s;
  KvRows k, v, q, qo;  // q.p null: no q
  const float* rope;   // [rope_rows, rot] (cos, then sin), or null
  int q_heads, rope_rows, rot, interleaved;
};
hipError_t launch_kv_append(const KvAppendArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_kv_gather(const KvCache& c, const KvBatch& s, const KvRows& k, const KvRows& v, bool bf16,
                            int num_cus, hipStream_t stream);
// rope[p][i] = mag cos(p f[i]), rope[p][n + i] = mag sin(p f[i])
constexpr int kRopeMaxPairs = 128;
struct RopeFreq {
  double f[kRopeMaxPairs];
};
hipError_t launch_rope_table(const RopeFreq& f, int pairs, int rows, double mag, float* table,
                             hipStream_t stream);
struct KvAttnArgs {
  KvCache c;
  KvBatch s;
  KvRows q, o;
  float* lse;  // [T, q_heads] or null
  float scale;
  int bf16, q_heads, causal, window, sinks;
  // Runs of rows with long contexts are cut into parts, for `extra` workgroups at
  // most beyond one to each run and head (0: not cut); `slots` workgroups run at
  // once. What the parts leave for the join: [max_parts, run, dim] and
  // [max_parts, run, 2], and notes [T * q_heads, 2] of each row's parts.
  int prompt;  // kv_prompt instead of kv_step; splits: parts of its tokens (1: not cut)
  int splits;
  int run, extra, slots, max_parts;
  float* part_o;
  float* part_ml;
  int* notes;
};
// A row's note for the join: slot of its first part << shift | its place in a run,
// and how many parts there are; no parts if the two name none of the workspace (a
// row that no run of this call holds has whatever the workspace held).
constexpr int kKvNoteShift = 8;
struct KvNote {
  int slot, place, parts;
};
__host__ __device__ inline KvNote kv_note(int where, int parts, int run, int max_parts) {
  const KvNote n{where >> kKvNoteShift, where & ((1 << kKvNoteShift) - 1), parts};
  const bool there = where >= 0 && n.place < run && n.slot < max_parts && parts >= 1 && parts <= max_parts - n.slot;
  return there ? n : KvNote{0, 0, 0};
}
int kv_attention_run(const KvBatch& s, int heads, int q_heads);  // rows of a run: 16 or 32
int kv_attention_extra(const KvBatch& s, int heads, int q_heads, int dim, int64_t max_span, int num_cus,
                       int* slots);
bool kv_attention_prompt(const KvBatch& s, int heads, int q_heads);
int kv_prompt_splits(const KvBatch& s, int heads, int q_heads, int dim, int page_shift, int64_t max_span,
                     int num_cus, int* run, int* max_parts);
hipError_t launch_kv_prompt(const KvAttnArgs& a, hipStream_t stream);
hipError_t launch_kv_attention(const KvAttnArgs& a, hipStream_t stream);

}  // namespace llmint8
