// The packed attention's part of internal.h: limits, what the kernels take,
// launchers. A call's rows are sequences one after the other; every token of a
// sequence is a row of q, k and v.
#pragma once

#include "kv_internal.h"

namespace llmint8 {

// Rows and (row, head) pairs are counted in 32 bits; a tile of 64 rows has to lie
// within a buffer window of 2^31 bytes, so strides are limited as well.
constexpr int64_t kAttnMaxStride = int64_t(1) << 23;
constexpr int64_t kMaxWorkItems = int64_t(1) << 32;  // of a launch, and fewer
inline int admit_attention(int64_t seqs, int64_t rows, int64_t q_heads, int64_t heads, int64_t dim) {
  if (seqs < 0 || rows < 0 || q_heads <= 0 || heads <= 0 || dim <= 0) return LLMINT8_ERR_INVALID_ARG;
  if (q_heads % heads != 0) return LLMINT8_ERR_INVALID_ARG;
  if (dim % 8 != 0 || dim > 256 || heads > 4096 || q_heads > 65536) return LLMINT8_ERR_UNSUPPORTED;
  if (rows > kKvMax || seqs > (int64_t(1) << 24)) return LLMINT8_ERR_UNSUPPORTED;
  if (rows * q_heads > kKvMaxQRows) return LLMINT8_ERR_UNSUPPORTED;
  return LLMINT8_OK;
}

// The launches of a call: workgroups that take 128 rows of a sequence and key/value head (forward, dq), or
// 128 or 64 of its tokens (dk and dv). A launch has fewer than 2^32 work items.
struct AttnGrid {
  int64_t blocks;
  int threads;
  bool fits() const { return blocks * threads < kMaxWorkItems; }
};
inline AttnGrid attn_row_grid(int64_t rows, int64_t q_heads, int64_t heads, int64_t seqs) {
  return {((rows * (q_heads / heads) >> 7) + seqs) * heads, 256};
}
inline AttnGrid attn_col_grid(int64_t rows, int64_t heads, int64_t seqs, int64_t dim) {
  return {((rows >> (dim <= 128 ? 7 : 6)) + seqs) * heads, dim > 96 && dim <= 128 ? 512 : 256};
}

struct AttnArgs {
  const int32_t* cu;  // [B + 1]
  int B, T;
  KvRows q, k, v, o;
  float* lse;  // [T, q_heads] or null
  float scale;
  int q_heads, heads, dim, causal, window, sinks;
  // backward
  KvRows d_o, dq, dk, dv;
  float* stat;  // [2][q_heads][T]: what a row's logits (in powers of two) are short of, and delta
};

// Rows [row0, row0 + n) of sequence b, cut to the call's rows whatever cu holds.
struct AttnSeq {
  int row0, n;
};
__host__ __device__ inline AttnSeq attn_seq_of(int cu0, int cu1, int T) {
  cu0 = cu0 < 0 ? 0 : cu0 > T ? T : cu0;
  cu1 = cu1 < 0 ? 0 : cu1 > T ? T : cu1;
  return AttnSeq{cu0, cu1 > cu0 ? cu1 - cu0 : 0};
}

// A tile of 64 rows of a head in LDS (attn_common.h): where rows begin, and at which chunk of
// 16 bytes of its row a chunk is kept.
template <int DP>
struct AttnTile {
  static constexpr int kPitch = DP <= 64 ? 128 : DP <= 96 ? 192 : DP <= 128 ? 256 : 512;  // bytes of a row
  static constexpr int kChunks = kPitch / 16;
  static constexpr bool kNarrow = kPitch == 128, kMiddle = kPitch == 192;
  static constexpr int kSixteen = 16 * kPitch + (kMiddle ? 0 : 64);  // bytes of 16 rows
  static constexpr int kBytes = 4 * kSixteen;
  static constexpr int NQ = DP / 16;  // 16-channel steps
  static constexpr int ND = DP / 32;  // 32-channel blocks
  static __host__ __device__ constexpr int swizzle(int row) {
    return kNarrow ? (row >> 1 & 1) << 2 | (row >> 2 & 1) : kMiddle ? row >> 2 & 3 : (row & 3) << 2;
  }
  static __host__ __device__ constexpr int at(int row) {
    return (row >> 4) * kSixteen + (row & 15) * kPitch +
           (kNarrow ? (row >> 3 & 1) * 32 : kMiddle ? 0 : (row >> 2 & 3) * 16);
  }
  // where the 64 chunks of a wavefront's copy go: copy number `copy` of a tile, the copies of W
  // wavefronts one after the other
  static __host__ __device__ constexpr int copy_at(int copy) {
    return kMiddle ? copy * 1024 : at(copy * (1024 / kPitch));
  }
};

hipError_t launch_attention(const AttnArgs& a, bool bf16, hipStream_t stream);
hipError_t launch_attention_backward(const AttnArgs& a, bool bf16, hipStream_t stream);

}  // namespace llmint8
