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
// Rows of 16 are laid out so that the 16-byte reads of 16 rows at one chunk fall on all 64
// banks, and so do the four rows x 32 bytes that a transposing read takes for 16 lanes:
// chunks are stored at chunk ^ 2 (row % 4) and every four rows begin 16, 128 or 144 bytes
// later (rows of 128 bytes: chunk ^ 2 (row / 2 % 4), 16 bytes later every eight rows). The
// exclusive or touches three bits of a chunk's number, so that four addresses to a lane
// serve all "rows" operands and two all "channels" operands: the rest of an address is a
// constant of the instruction. (With the usual one over all bits each step had an address
// of its own; the 128-channel kernels spilled 90 registers.)
#pragma once

#include "attn_internal.h"
#include "kv_common.h"

namespace llmint8 {

constexpr float kAttnNegInf = -__builtin_inff();

template <int DP>
struct AttnTile {
  static constexpr int kPitch = DP <= 64 ? 128 : DP <= 128 ? 256 : 512;  // bytes of a row
  static constexpr int kChunks = kPitch / 16;
  static constexpr bool kNarrow = kPitch == 128;
  static constexpr int kSixteen = 16 * kPitch + (kNarrow ? 32 : 256);  // bytes of 16 rows
  static constexpr int kBytes = 4 * kSixteen;
  static constexpr int NQ = DP / 16;  // 16-channel steps
  static constexpr int ND = DP / 32;  // 32-channel blocks
  static __device__ __forceinline__ constexpr int swizzle(int row) {
    return kNarrow ? ((row >> 1) & 3) << 1 : (row & 3) << 1;
  }
  static __device__ __forceinline__ constexpr int at(int row) {
    const int pad = kNarrow ? (row >> 3 & 1) * 16 : (row >> 2 & 1) * 16 + (row >> 3 & 1) * 128;
    return (row >> 4) * kSixteen + (row & 15) * kPitch + pad;
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

// A matrix of rows in memory: the offset at which this thread's copies of a tile begin.
template <int DP, int W>
struct AttnCopy {
  using Tile = AttnTile<DP>;
  static constexpr int kIssues = 64 * Tile::kPitch / 1024 / W;  // of 1 KB to a wavefront and tile
  static constexpr int kRows = 1024 / Tile::kPitch;             // of an issue
  static_assert(kRows * W % 4 == 0, "the rows of a thread's issues have one swizzle");
  uint32_t off, step;
  __device__ __forceinline__ AttnCopy(int64_t token, int dim) {
    const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
    const int row = wave * kRows + lane / Tile::kChunks, chunk = lane % Tile::kChunks ^ Tile::swizzle(row);
    off = chunk * 8 < dim ? (uint32_t)(row * (int)token * 2 + chunk * 16) : kOobOffset;
    step = (uint32_t)(kRows * W * (int)token * 2);
  }
  // rows [first, first + 64) of the n at p into LDS at `to`; those from n on are zeros
  __device__ __forceinline__ void issue(const uint16_t* p, int64_t token, int first, int n, char* to) const {
    const int wave = uniform((int)threadIdx.x >> 6);
    const int left = min(n - first, 64);
    const __amdgpu_buffer_rsrc_t r = make_rsrc(p + (int64_t)first * token, (uint32_t)(max(left, 0) * (int)token * 2));
#pragma unroll
    for (int i = 0; i < kIssues; ++i) attn_copy16(r, to + Tile::at((i * W + wave) * kRows), off + i * step);
  }
};

__device__ __forceinline__ void attn_wait_copies() { __builtin_amdgcn_s_waitcnt(0x0f70); }  // vmcnt(0)

// Operands from tiles: `tile` is the place of one among the tiles of a workgroup, a
// constant; the addresses move between its stages (`next`).
template <int DP>
struct AttnRead {
  using Tile = AttnTile<DP>;
  const char* row[4];
  const char* tr[2];
  __device__ __forceinline__ explicit AttnRead(const char* smem) {
    const int lane = threadIdx.x & 63, hf = lane >> 5, nn = lane & 31;
    const int r = (nn & 0x13) | (nn & 4) << 1 | (nn & 8) >> 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) row[i] = smem + Tile::at(r) + ((2 * i + hf) ^ Tile::swizzle(r)) * 16;
    const int i = lane & 15, t = 8 * hf + (i >> 2), c = 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
#pragma unroll
    for (int d = 0; d < 2; ++d) tr[d] = smem + Tile::at(t) + ((4 * d + c) ^ Tile::swizzle(t)) * 16 + 8 * (i & 1);
  }
  __device__ __forceinline__ void next_rows(int by) {
#pragma unroll
    for (int i = 0; i < 4; ++i) row[i] += by;
  }
  __device__ __forceinline__ void next_channels(int by) {
    tr[0] += by;
    tr[1] += by;
  }
  __device__ __forceinline__ void next(int by) {
    next_rows(by);
    next_channels(by);
  }
  // rows [32 block, +32) x channels [16 step, +16)
  __device__ __forceinline__ uint4 rows(int tile, int block, int step) const {
    return *reinterpret_cast<const uint4*>(row[step & 3] + (tile * Tile::kBytes + (step >> 2) * 128 + block * 2 * Tile::kSixteen));
  }
  // channels [32 block, +32) x rows [16 step, +16)
  __device__ __forceinline__ uint4 channels(int tile, int block, int step) const {
    typedef short v4s __attribute__((ext_vector_type(4)));
    typedef __attribute__((address_space(3))) v4s* lds_v4s;
    const int at = tile * Tile::kBytes + (block >> 1) * 128 + step * Tile::kSixteen;
    // four rows on, the exclusive or of narrow rows has its bit 2 turned
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(tr[block & 1] + at));
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)(tr[(block ^ (int)Tile::kNarrow) & 1] + at + Tile::at(4)));
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

// The largest of three, NaN if one of them is (one instruction; fmaxf costs two more, as it
// takes the other one and quiets its operands first).
__device__ __forceinline__ float attn_max(float a, float b, float c) {
  return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}

// A product whose weights are exactly zero where a column does not see a row must not
// take that row's values that are not finite (0 times them is NaN). Where a tile has
// masked rows the workgroup zeroes such values in LDS first; if there were any (the
// result), attn_others adds them, from memory, to the sums of the columns that see them.
template <int DP, bool BF16, int W>
__device__ __forceinline__ bool attn_finite(char* tile) {
  using Tile = AttnTile<DP>;
  constexpr uint32_t kUp = BF16 ? 0x00800080u : 0x04000400u;  // carries an exponent of ones into bit 15
  uint32_t odd = 0;
#pragma unroll
  for (int i = 0; i < 64 * Tile::kChunks / (64 * W); ++i) {
    const int u = i * 64 * W + (int)threadIdx.x;
    uint4* at = reinterpret_cast<uint4*>(tile + Tile::at(u / Tile::kChunks) + u % Tile::kChunks * 16);
    const uint4 x = *at;
    uint32_t v[4] = {x.x, x.y, x.z, x.w}, any = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t bad = ((v[j] & 0x7fff7fffu) + kUp) & 0x80008000u;
      any |= bad;
      v[j] &= ~((bad >> 15) * 0xffffu);
    }
    if (any) *at = make_uint4(v[0], v[1], v[2], v[3]);
    odd |= any;
  }
  return __syncthreads_or(odd != 0);
}
// Rows [first, first + 64) of the n at p; `see(row)`: whether this lane's column sees that
// row of the 64.
template <int DP, bool BF16, class See>
__device__ __forceinline__ void attn_others(v16f_t (&acc)[DP / 32], const uint16_t* p, int64_t token, int first, int n,
                                            int dim, See&& see) {
  constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u;
  const int lane = threadIdx.x & 63, hf = lane >> 5, rows = min(n - first, 64);
#pragma unroll 1
  for (int t = 0; t < rows; ++t) {
    const bool sees = see(t);
#pragma unroll 1
    for (int c0 = 0; c0 < dim; c0 += 64) {
      const uint32_t v = c0 + lane < dim ? p[(int64_t)(first + t) * token + c0 + lane] : 0u;
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

// s += the tile's rows [32 block, +32) times b, operands read two steps ahead
template <int DP, bool BF16>
__device__ __forceinline__ v16f_t attn_rows_product(const AttnRead<DP>& rd, int tile, int block, const uint4 (&b)[DP / 16]) {
  constexpr int NQ = DP / 16, kAhead = 2;
  uint4 x[kAhead + 1];
#pragma unroll
  for (int st = 0; st < kAhead; ++st) x[st] = rd.rows(tile, block, st);
  v16f_t s;
#pragma unroll
  for (int st = 0; st < NQ; ++st) {
    if (st + kAhead < NQ) x[(st + kAhead) % (kAhead + 1)] = rd.rows(tile, block, st + kAhead);
    s = Act16<BF16>::mma32(x[st % (kAhead + 1)], b[st], st == 0 ? attn_zero() : s);
    __builtin_amdgcn_sched_barrier(0);
  }
  return s;
}

// values 8 k .. 8 k + 7 as an operand
template <bool BF16>
__device__ __forceinline__ uint4 attn_pack(const v16f_t& t, int k) {
  using A = Act16<BF16>;
  return make_uint4(A::pack2(t[8 * k], t[8 * k + 1]), A::pack2(t[8 * k + 2], t[8 * k + 3]),
                    A::pack2(t[8 * k + 4], t[8 * k + 5]), A::pack2(t[8 * k + 6], t[8 * k + 7]));
}

// acc += the tile's channels x rows [32 block, +32) times t, operands read two products ahead
template <int DP, bool BF16>
__device__ __forceinline__ void attn_channels_product(const AttnRead<DP>& rd, int tile, int block, const v16f_t& t,
                                                      v16f_t (&acc)[DP / 32]) {
  constexpr int ND = DP / 32, kAhead = 2;
  uint4 x[kAhead + 1];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) x[i] = rd.channels(tile, i % ND, 2 * block + i / ND);
  uint4 p;
#pragma unroll
  for (int i = 0; i < 2 * ND; ++i) {
    if (i + kAhead < 2 * ND) x[(i + kAhead) % (kAhead + 1)] = rd.channels(tile, (i + kAhead) % ND, 2 * block + (i + kAhead) / ND);
    if (i % ND == 0) p = attn_pack<BF16>(t, i / ND);
    acc[i % ND] = Act16<BF16>::mma32(x[i % (kAhead + 1)], p, acc[i % ND]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

}  // namespace llmint8
