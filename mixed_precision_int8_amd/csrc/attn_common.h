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
// An instruction of either kind takes LDS four cycles where no bank is asked twice: 16
// rows of one chunk of 16 bytes, or four rows of four chunks. Chunks are stored at
// chunk ^ 4 (row % 4), and every four rows begin 16 bytes later (rows of 128 bytes: at
// chunk ^ 4 (row / 2 % 2) ^ (row / 4 % 2), 32 bytes later every eight rows; rows of 192 bytes begin
// at four different places of 256 as they are: at chunk ^ (row / 4 % 4)). The exclusive
// or touches few bits of a chunk's number, so that four addresses to a lane serve all
// "rows" operands and four all "channels" operands: the rest of an address is a constant of
// the instruction. (With one over all bits each step had an address of its own; the
// 128-channel kernels spilled 90 registers.)
#pragma once

#include "attn_internal.h"
#include "kv_common.h"

namespace llmint8 {

constexpr float kAttnNegInf = -__builtin_inff();

// Copies to LDS: 64 x 16 bytes (64 x 4) from the lanes' offsets to `to` on. (Functions of
// their own, not of a template's: the host pass drops kernels whose instances use the
// 16-byte form.)
//
// The compiler makes a read of LDS wait for every copy in flight unless it is told that the
// two do not meet: the reads have to carry what it knows of types or scopes (a read of a
// vector type does, one of uint4 does not, a transposing read does from a function with a
// restricted pointer), and LDS has to be one array. Then the kernels' own waits are the only
// ones: attn_wait_copies before a barrier that hands a tile over.
__device__ __forceinline__ void attn_copy16(__amdgpu_buffer_rsrc_t r, char* to, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)to, 16, off, 0, 0, 0);
}
__device__ __forceinline__ void attn_copy4(__amdgpu_buffer_rsrc_t r, char* to, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)to, 4, off, 0, 0, 0);
}
__device__ __forceinline__ void attn_wait_copies() { __builtin_amdgcn_s_waitcnt(0x0f70); }  // vmcnt(0)
// This wavefront's writes to LDS are done, then the workgroup's barrier. __syncthreads
// would wait for the copies in flight as well.
__device__ __forceinline__ void attn_barrier() {
  __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0)
  asm volatile("s_barrier" ::: "memory");
}
typedef short v4s __attribute__((ext_vector_type(4)));
__device__ __forceinline__ v4s attn_read_tr(const char* __restrict p) {
  typedef __attribute__((address_space(3))) v4s* lds_v4s;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s)p);
}

// A matrix of rows in memory: the offset at which this thread's copies of a tile begin.
template <int DP, int W>
struct AttnCopy {
  using Tile = AttnTile<DP>;
  static constexpr int kIssues = 64 * Tile::kPitch / 1024 / W;  // of 64 chunks to a wavefront and tile
  static constexpr int kRows = 1024 / Tile::kPitch;             // of an issue, where they are whole
  static_assert(Tile::kMiddle || kRows * W % 8 == 0, "the rows of a thread's issues have one swizzle and copy_at adds up");
  uint32_t off[Tile::kMiddle ? kIssues : 1], step;
  int to_mine;  // of this wavefront's first issue in a tile
  __device__ __forceinline__ AttnCopy(int64_t token, int dim) {
    const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
#pragma unroll
    for (int i = 0; i < (Tile::kMiddle ? kIssues : 1); ++i) {
      const int n = (i * W + wave) * 64 + lane, row = n / Tile::kChunks, chunk = n % Tile::kChunks ^ Tile::swizzle(row);
      off[i] = chunk * 8 < dim ? (uint32_t)(row * (int)token * 2 + chunk * 16) : kOobOffset;
    }
    step = (uint32_t)(kRows * W * (int)token * 2);
    to_mine = Tile::copy_at(wave);
  }
  // The tile at address `at` into LDS at `to`; what is `bytes` or more from its start on reads
  // as zeros. The window's numbers are the same in all lanes and have to be in scalar
  // registers: of vector ones the compiler makes a loop around each copy.
  __device__ __forceinline__ void issue(int64_t at, int bytes, char* to) const {
    const __amdgpu_buffer_rsrc_t r = make_rsrc(reinterpret_cast<const void*>(uniform(at)), (uint32_t)uniform(bytes));
#pragma unroll
    for (int i = 0; i < kIssues; ++i)
      attn_copy16(r, to + (to_mine + Tile::copy_at(i * W)), Tile::kMiddle ? off[i] : off[0] + i * step);
  }
  // A product whose weights are exactly zero where a column does not see a row must not take
  // that row's values that are not finite (0 times them is NaN). Where a tile has masked rows
  // every wavefront zeroes such values in the pieces that it copied, once they are there and
  // before the barrier that hands the tile over, and sets *flag if there were any; attn_others
  // then adds them, from memory, at the end, to the sums of the columns that see them.
  template <bool BF16>
  __device__ __forceinline__ void finite(char* to, int* flag) const {
    constexpr uint32_t kUp = BF16 ? 0x00800080u : 0x04000400u;  // carries an exponent of ones into bit 15
    v4i x[kIssues];
    char* const at = to + to_mine + (threadIdx.x & 63) * 16;
#pragma unroll
    for (int i = 0; i < kIssues; ++i) x[i] = *reinterpret_cast<const v4i*>(at + Tile::copy_at(i * W));
#pragma unroll
    for (int i = 0; i < kIssues; ++i) {
      uint32_t odd = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t v = (uint32_t)x[i][j], bad = ((v & 0x7fff7fffu) + kUp) & 0x80008000u;
        odd |= bad;
        x[i][j] = (int)(v & ~((bad >> 15) * 0xffffu));
      }
      if (__builtin_expect(odd != 0, 0)) {
        *reinterpret_cast<v4i*>(at + Tile::copy_at(i * W)) = x[i];
        *flag = 1;
      }
    }
  }
};

// Tiles of a matrix one after the other, by address (a product of 64 bits for each would be a
// dozen scalar instructions): `step` on from tile to tile, but `jump` where a caller says so.
template <int DP, int W>
struct AttnStream : AttnCopy<DP, W> {
  int64_t at, step_by, jump_by;
  int row;  // bytes of a token
  // from row `first` on; a jump goes from one tile's begin to `jump` elements on
  __device__ __forceinline__ AttnStream(const uint16_t* p, int64_t token, int dim, int64_t first, int64_t jump)
      : AttnCopy<DP, W>(token, dim),
        at(reinterpret_cast<int64_t>(p + first * token)),
        step_by(128 * token),
        jump_by(2 * jump),
        row((int)(2 * token)) {}
  __device__ __forceinline__ void rewind(const uint16_t* p, int64_t token, int64_t first) {
    at = reinterpret_cast<int64_t>(p + first * token);
  }
  __device__ __forceinline__ void next(int rows, char* to, bool jump) {
    this->issue(at, rows * row, to);
    at += jump ? jump_by : step_by;
  }
};

// Operands from tiles: `tile` is the place of one among the tiles of a workgroup, a
// constant; the addresses move between its stages (`next`).
template <int DP>
struct AttnRead {
  using Tile = AttnTile<DP>;
  // addresses that differ by the exclusive or
  static constexpr int kRowAt = Tile::kNarrow || Tile::kMiddle ? 2 : 4, kTrAt = Tile::kMiddle ? 2 : 4;
  const char* row[kRowAt];
  const char* tr[kTrAt];
  __device__ __forceinline__ explicit AttnRead(const char* smem) {
    const int lane = threadIdx.x & 63, hf = lane >> 5, nn = lane & 31;
    const int r = (nn & 0x13) | (nn & 4) << 1 | (nn & 8) >> 1;
#pragma unroll
    for (int i = 0; i < kRowAt; ++i)
      row[i] = smem + Tile::at(r) + (((Tile::kMiddle ? 2 : 4) * i + hf) ^ Tile::swizzle(r)) * 16;
    const int i = lane & 15, t = 8 * hf + (i >> 2), c = 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
#pragma unroll
    for (int d = 0; d < kTrAt; ++d) {
      // narrow: 32-channel block d / 2, and four rows on where d is odd; middle: four rows on
      const int u = Tile::kNarrow || Tile::kMiddle ? t + 4 * (d & 1) : t;
      const int block = Tile::kNarrow ? d >> 1 : Tile::kMiddle ? 0 : d;
      tr[d] = smem + Tile::at(u) + ((4 * block + c) ^ Tile::swizzle(u)) * 16 + 8 * (i & 1);
    }
  }
  __device__ __forceinline__ void next_rows(int by) {
#pragma unroll
    for (int i = 0; i < kRowAt; ++i) row[i] += by;
  }
  __device__ __forceinline__ void next_channels(int by) {
#pragma unroll
    for (int i = 0; i < kTrAt; ++i) tr[i] += by;
  }
  __device__ __forceinline__ void next(int by) {
    next_rows(by);
    next_channels(by);
  }
  // rows [32 block, +32) x channels [16 step, +16)
  __device__ __forceinline__ uint4 rows(int tile, int block, int step) const {
    const int at = tile * Tile::kBytes + block * 2 * Tile::kSixteen +
                   (Tile::kMiddle ? (step >> 1) * 64 : (step & 1) * 32 + (step >> 3) * 256);
    const v4i x = *reinterpret_cast<const v4i*>(row[Tile::kMiddle ? step & 1 : (step >> 1) % kRowAt] + at);
    return __builtin_bit_cast(uint4, x);
  }
  // channels [32 block, +32) x rows [16 step, +16)
  __device__ __forceinline__ uint4 channels(int tile, int block, int step) const {
    const int at = tile * Tile::kBytes + step * Tile::kSixteen +
                   (Tile::kNarrow ? 0 : Tile::kMiddle ? block * 64 : (block >> 2) * 256);
    const char* first = tr[Tile::kNarrow ? 2 * block : Tile::kMiddle ? 0 : block & 3] + at;
    const char* second = Tile::kNarrow   ? tr[(2 * block + 1) % kTrAt] + at
                         : Tile::kMiddle ? tr[1] + at
                                         : first + Tile::at(4);
    const v4s lo = attn_read_tr(first);
    const v4s hi = attn_read_tr(second);
    const uint2 a = __builtin_bit_cast(uint2, lo), b = __builtin_bit_cast(uint2, hi);
    return make_uint4(a.x, a.y, b.x, b.y);
  }
};

// The sequence and tile of 2^shift rows (tokens times `per`) that is a workgroup's work, by
// one wavefront alone: no LDS, no barrier. False where there is none (a launch has a few
// workgroups more than there is work).
//   Up to 64 sequences: a lane has one, and the tiles of all go by how many their sequence
// has below (DOWN) or above them, most first: with a causal mask that is their length, and
// the longest start first. The level of item x is the largest l with x < F(l), where F(l) =
// sum max(0, tiles - l) tiles have l or more.
//   More: in the order of the sequences, the owner found by 64 probes at a time of where
// their items begin (kv_items).
template <bool DOWN>
__device__ __forceinline__ bool attn_place(const AttnArgs& a, int item, int per, int shift, AttnSeq* out, int* run) {
  const int lane = threadIdx.x & 63;
  if (a.B <= 64) {
    const int b = min(lane, a.B - 1);
    const AttnSeq q = attn_seq_of(a.cu[b], a.cu[b + 1], a.T);
    const int tiles = lane < a.B ? (int)(((int64_t)q.n * per + (1 << shift) - 1) >> shift) : 0;
    auto at_least = [&](int l) { return __builtin_amdgcn_readlane(wave_incl_sum(max(tiles - l, 0)), 63); };
    if (item >= at_least(0)) return false;
    int lo = 0, hi = (int)(((int64_t)a.T * per >> shift) + 1), above = 0;  // F(lo) > item >= F(hi)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1, f = at_least(mid);
      if (f > item) lo = mid;
      else hi = mid, above = f;
    }
    const uint64_t have = __ballot(tiles > lo);
    const int before = __builtin_amdgcn_mbcnt_hi((uint32_t)(have >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)have, 0));
    const uint64_t mine = __ballot(tiles > lo && before == item - above);
    if (mine == 0) return false;  // cu falls somewhere
    const int owner = __builtin_ctzll(mine);
    out->row0 = __builtin_amdgcn_readlane(q.row0, owner);
    out->n = __builtin_amdgcn_readlane(q.n, owner);
    *run = DOWN ? lo : __builtin_amdgcn_readlane(tiles, owner) - 1 - lo;
    return true;
  }
  int lo = 0, hi = a.B;
  while (true) {
    const int step = (hi - lo + 63) >> 6, b = min(lo + lane * step, hi - 1);
    const AttnSeq q = attn_seq_of(a.cu[b], a.cu[b + 1], a.T);
    const KvItems own = kv_items(b, q.row0, q.n, per, shift);
    const int below = __popcll(__ballot(lo + lane * step < hi && own.first <= item));
    if (below == 0) return false;
    if (step == 1) {
      out->row0 = __builtin_amdgcn_readlane(q.row0, below - 1);
      out->n = __builtin_amdgcn_readlane(q.n, below - 1);
      const int at = __builtin_amdgcn_readlane(kv_item_index(own, item), below - 1);
      const int tiles = (int)(((int64_t)out->n * per + (1 << shift) - 1) >> shift);
      if (at < 0 || at >= tiles) return false;
      *run = DOWN ? tiles - 1 - at : at;
      return true;
    }
    lo += (below - 1) * step;
    hi = min(hi, lo + step);
  }
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

// What a row sees of its sequence: `count` tokens from `first` on (of a window; else from 0), and
// those below `sinks`.
struct AttnSees {
  int first, sinks;
  uint32_t count;
  __device__ __forceinline__ AttnSees(const AttnArgs& a, int pos, int n) {
    const int end = a.causal ? min(pos + 1, n) : n;
    first = a.window > 0 ? pos - a.window + 1 : 0;
    count = (uint32_t)(end - first);
    sinks = min(a.sinks, end);
  }
  __device__ __forceinline__ bool operator()(int j) const { return ((uint32_t)j - (uint32_t)first < count) | (j < sinks); }
};

// What rows at tokens lo .. hi of a sequence of n see: `last` and `begin` bound what any of them
// does, all_end and all_begin what all do (but for sinks).
struct AttnSpan {
  int last, begin, all_end, all_begin, sinks;
  __device__ __forceinline__ AttnSpan(const AttnArgs& a, int lo, int hi, int n)
      : last(a.causal ? min(hi, n - 1) : n - 1),
        begin(a.window > 0 ? lo - a.window + 1 : 0),
        all_end(a.causal ? min(lo, n - 1) : n - 1),
        all_begin(a.window > 0 ? hi - a.window + 1 : 0),
        sinks(a.sinks) {}
  // of the tile of 64 tokens from base on some row does not see some token
  __device__ __forceinline__ bool masked(int base) const { return (base + 63 > all_end) | (base < all_begin); }
  // no row sees any of `len` tokens from base on
  __device__ __forceinline__ bool none(int base, int len) const {
    return (base > last) | ((base + len <= begin) & (base >= sinks));
  }
};

// The largest of three, NaN if one of them is (one instruction; fmaxf costs two more, as it
// takes the other one and quiets its operands first).
__device__ __forceinline__ float attn_max(float a, float b, float c) {
  return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}

// Rows [first, first + 64) of the n at p; `see(row)`: whether this lane's column sees that
// row of the 64. `weight`: the products' weights are of one sign, and an infinity is added as it
// is (its weight is taken not to vanish); others may have either sign, or be 0 or NaN: NaN.
template <int DP, bool BF16, class See>
__device__ __forceinline__ void attn_others(v16f_t (&acc)[DP / 32], const uint16_t* p, int64_t token, int first, int n,
                                            int dim, bool weight, See&& see) {
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
        const float value = Act16<BF16>::to_f32((uint32_t)__builtin_amdgcn_readlane((int)v, from));
        const float x = weight ? value : value - value;
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

// Logits of 32 of the n rows at p, from `first` on, formed from a tile that `finite` has cleared:
// a row that holds an infinity or NaN gets -infinity, weight 0. Its logit was that or, of a column whose
// lse is NaN, anything; a cleared tile has some other number for it.
template <bool BF16>
__device__ __forceinline__ void attn_hide(v16f_t& s, const uint16_t* p, int64_t token, int first, int n, int dim) {
  constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u;
  const int hf = (threadIdx.x & 63) >> 5;
  uint32_t odd = 0;
#pragma unroll 1
  for (int x = 0; x < 16; ++x) {
    const int row = first + 16 * (x >> 3) + 8 * hf + (x & 7);
#pragma unroll 1
    for (int c = 0; row < n && c < dim; c += 2) {
      const uint32_t v = *reinterpret_cast<const uint32_t*>(p + (int64_t)row * token + c);
      if ((v & kInf) == kInf || (v >> 16 & kInf) == kInf) odd |= 1u << x;
    }
  }
#pragma unroll
  for (int x = 0; x < 16; ++x)
    if (odd >> x & 1) s[x] = kAttnNegInf;
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

// What rounding values to the type leaves of them, nothing where they are not finite: a second
// product with it takes away the rounding of the first.
template <bool BF16>
__device__ __forceinline__ void attn_residual(v16f_t& t) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint4 p = attn_pack<BF16>(t, k);
    const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float left = t[8 * k + j] - Act16<BF16>::to_f32(j & 1 ? w[j >> 1] >> 16 : w[j >> 1] & 0xffffu);
      t[8 * k + j] = __builtin_isfinite(left) ? left : 0.0f;
    }
  }
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
