// Shared by the packed attention's kernels: a workgroup's sequence, tiles of 64
// rows of one head in LDS, and the operands read from them.
//
// A tile is 64 rows of 16-bit channels as they lie in memory, copied straight to
// LDS (buffer loads that go there without registers; rows past the sequence and
// channels past the head read as zero by the buffer's range check). It serves as
// operand A of v_mfma_f32_32x32x16 in both directions:
//   rows      (32 rows x 16 channels) one ds_read_b128 a lane
//   channels  (32 channels x 16 rows) two ds_read_b64_tr_b16 a lane, which
//             transpose 4 x 16 values on the way
// The rows of a "rows" operand are taken with bits 2 and 3 of their number swapped,
// so that a lane's 16 results are rows 8 hf .. 8 hf + 7 of each sixteen: as they
// stand, operand B of the next product, which sums over these rows.
//
// 16-byte chunks of a row are stored at chunk ^ swizzle(row): 16 rows' reads at one
// chunk fall on all 64 banks, and so do the four rows x 32 bytes that a
// transposing read takes for 16 lanes.
#pragma once

#include "attn_internal.h"
#include "kv_common.h"

namespace llmint8 {

constexpr float kAttnNegInf = -__builtin_inff();

template <int DP>
struct AttnTile {
  static constexpr int kPitch = DP <= 64 ? 128 : DP <= 128 ? 256 : 512;  // bytes of a row
  static constexpr int kChunks = kPitch / 16;
  static constexpr int kBytes = 64 * kPitch;
  static constexpr int NQ = DP / 16;  // 16-channel steps
  static constexpr int ND = DP / 32;  // 32-channel blocks
  static __device__ __forceinline__ int swizzle(int row) {
    if constexpr (kPitch == 128) return ((row >> 1) & 3) << 1 | ((row >> 3) & 1);
    return (row & 7) << 1 | ((row >> 3) & 1);
  }
};

// Copies to LDS: 64 x 16 bytes (64 x 4) from the lanes' offsets to `to` on. (Functions of
// their own, not of a template's: the host pass drops kernels whose instances use the
// 16-byte form.)
__device__ __forceinline__ void attn_copy16(__amdgpu_buffer_rsrc_t r, char* to, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)to, 16, off, 0, 0, 0);
}
__device__ __forceinline__ void attn_copy4(__amdgpu_buffer_rsrc_t r, float* to, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)to, 4, off, 0, 0, 0);
}

// A matrix of rows in memory: the window that starts at a row, and the offsets at
// which this thread's copies of a tile stand in it.
template <int DP, int W>
struct AttnCopy {
  using Tile = AttnTile<DP>;
  static constexpr int kIssues = Tile::kBytes / 1024 / W;  // of 1 KB to a wavefront and tile
  uint32_t off[kIssues];
  __device__ __forceinline__ AttnCopy(int64_t token, int dim) {
    const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
#pragma unroll
    for (int i = 0; i < kIssues; ++i) {
      const int at = (i * W + wave) * 64 + lane;
      const int row = at / Tile::kChunks, chunk = at % Tile::kChunks ^ Tile::swizzle(row);
      off[i] = chunk * 8 < dim ? (uint32_t)(row * (int)token * 2 + chunk * 16) : kOobOffset;
    }
  }
  // rows [first, first + 64) of `rows` (an address and its row count) into LDS at `to`
  __device__ __forceinline__ void issue(const uint16_t* p, int64_t token, int first, int n, char* to) const {
    const int wave = uniform((int)threadIdx.x >> 6);
    const int left = min(n - first, 64);
    const __amdgpu_buffer_rsrc_t r = make_rsrc(p + (int64_t)first * token, (uint32_t)(max(left, 0) * (int)token * 2));
#pragma unroll
    for (int i = 0; i < kIssues; ++i)
      attn_copy16(r, to + (i * W + wave) * 1024, off[i]);
  }
};

__device__ __forceinline__ void attn_wait_copies() { __builtin_amdgcn_s_waitcnt(0x0f70); }  // vmcnt(0)

// Operands from a tile.
template <int DP>
struct AttnRead {
  using Tile = AttnTile<DP>;
  int row_at, row_x, tr_at, tr_x;
  __device__ __forceinline__ AttnRead() {
    const int lane = threadIdx.x & 63, hf = lane >> 5, nn = lane & 31;
    const int row = (nn & 0x13) | (nn & 4) << 1 | (nn & 8) >> 1;
    row_at = row * Tile::kPitch;
    row_x = (hf ^ Tile::swizzle(row)) * 16;
    const int i = lane & 15, t = 8 * hf + (i >> 2), c = 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
    tr_at = t * Tile::kPitch + 8 * (i & 1);
    tr_x = (c ^ Tile::swizzle(t)) * 16;
  }
  // rows [32 block, +32) x channels [16 step, +16)
  __device__ __forceinline__ uint4 rows(const char* tile, int block, int step) const {
    return *reinterpret_cast<const uint4*>(tile + row_at + (row_x ^ step * 32) + block * 32 * Tile::kPitch);
  }
  // channels [32 block, +32) x rows [16 step, +16)
  __device__ __forceinline__ uint4 channels(const char* tile, int block, int step) const {
    typedef short v4s __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) v4s* lds_v4s;
    // four rows on, bit 2 of the row is the swizzle's bit 3 (2 where a row has eight chunks)
    constexpr int kNext = Tile::kPitch == 128 ? 64 : 128;
    const int x = tr_x ^ block * 64;
    const char* p = tile + tr_at + step * 16 * Tile::kPitch;
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(p + x));
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(p + 4 * Tile::kPitch + (x ^ kNext)));
    const uint2 a = __builtin_bit_cast(uint2, lo), b = __builtin_bit_cast(uint2, hi);
    return make_uint4(a.x, a.y, b.x, b.y);
  }
};

// The sequence that owns work item `item` (kv_items), as kv_find does it, for rows alone.
template <int kThreads>
__device__ __forceinline__ bool attn_find(const AttnArgs& a, int item, int per, int shift, int (&sh)[4], AttnSeq* out,
                                          int* index) {
  if (a.B == 1) {
    const AttnSeq q = attn_seq_of(a.cu[0], a.cu[1], a.T);
    out->row0 = uniform(q.row0);
    out->n = uniform(q.n);
    *index = kv_item_index(kv_items(0, out->row0, out->n, per, shift), item);
    return *index >= 0;
  }
  int b = -1;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int i = b0 + (int)threadIdx.x, lane = min(i, a.B - 1);
    const AttnSeq q = attn_seq_of(a.cu[lane], a.cu[lane + 1], a.T);
    const KvItems own = kv_items(lane, q.row0, q.n, per, shift);
    const int mine = __syncthreads_count(i < a.B && own.first <= item);
    if (mine > 0 && (int)threadIdx.x == mine - 1) {
      sh[0] = q.row0;
      sh[1] = q.n;
      sh[2] = kv_item_index(own, item);
    }
    b += mine;
    if (mine < min(kThreads, a.B - b0)) break;
  }
  if (b < 0) return false;
  __syncthreads();
  out->row0 = uniform(sh[0]);
  out->n = uniform(sh[1]);
  *index = uniform(sh[2]);
  return *index >= 0;
}

// with the other half's lane of the same column (lanes n and n + 32)
__device__ __forceinline__ float attn_other(float v, float* other) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  *other = __uint_as_float(r[1]);
  return __uint_as_float(r[0]);
}
__device__ __forceinline__ float attn_pair_max(float v) {
  float o;
  v = attn_other(v, &o);
  return fmaxf(v, o);
}
__device__ __forceinline__ float attn_pair_sum(float v) {
  float o;
  v = attn_other(v, &o);
  return v + o;
}

__device__ __forceinline__ v16f_t attn_zero() {
  v16f_t z;
#pragma unroll
  for (int i = 0; i < 16; ++i) z[i] = 0.0f;
  return z;
}

// What a row sees of its sequence: tokens up to `last` that are past `from` or
// below `sinks` (from = -1: all of them).
struct AttnSees {
  int last, from, sinks;
  __device__ __forceinline__ AttnSees(const AttnArgs& a, int pos, int n)
      : last(a.causal ? min(pos, n - 1) : n - 1), from(a.window > 0 ? pos - a.window : -1), sinks(a.sinks) {}
  __device__ __forceinline__ bool operator()(int j) const { return (j <= last) & ((j > from) | (j < sinks)); }
};

// A product whose weights are exactly zero where a column does not see a row must not
// take that row's values that are not finite (0 times them is NaN). Where a tile has
// masked rows its operands pass attn_finite, which zeroes such values and notes that
// there were any; attn_others then adds them to the sums of the columns that see them.
template <bool BF16>
__device__ __forceinline__ uint4 attn_finite(const uint4& x, uint32_t* odd) {
  constexpr uint32_t kUp = BF16 ? 0x00800080u : 0x04000400u;  // carries an exponent of ones into bit 15
  uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t bad = ((v[j] & 0x7fff7fffu) + kUp) & 0x80008000u;
    *odd |= bad;
    v[j] &= ~((bad >> 15) * 0xffffu);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}
// Rows of the tile go by `see(row)`: whether this lane's column sees that row of the 64.
template <int DP, bool BF16, class See>
__device__ __forceinline__ void attn_others(v16f_t (&acc)[DP / 32], const char* tile, See&& see) {
  using Tile = AttnTile<DP>;
  constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u;
  const int lane = threadIdx.x & 63, hf = lane >> 5;
#pragma unroll 1
  for (int t = 0; t < 64; ++t) {
    const bool sees = see(t);
#pragma unroll 1
    for (int c0 = 0; c0 < Tile::kPitch / 2; c0 += 64) {
      const int at = (c0 + lane) >> 3;
      const uint16_t v = *reinterpret_cast<const uint16_t*>(tile + t * Tile::kPitch + ((at ^ Tile::swizzle(t)) * 16) + (lane & 7) * 2);
      uint64_t left = __ballot((v & kInf) == kInf);
      while (left) {
        const int from = __builtin_ctzll(left);
        left &= left - 1;
        const float x = Act16<BF16>::to_f32((uint32_t)__builtin_amdgcn_readlane((int)v, from));
        const int c = c0 + from;
#pragma unroll
        for (int d = 0; d < DP / 32; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (sees && c == 32 * d + 8 * (i >> 2) + 4 * hf + (i & 3)) acc[d][i] += x;
      }
    }
  }
}

}  // namespace llmint8
