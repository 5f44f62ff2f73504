// The int8 key/value cache on gfx950: writing it (with rotary positions) and
// reading it back.
//
// Cache: page p of head h holds P tokens as codes K[p, h, token, channel] and
// V[p, h, channel, token] with one magnitude each, aK[p, h] and aV[p, h]; a code
// c stands for fl32(c * fl32(a / 127)). V is held channel-major because the
// attention's second product runs over tokens: 16 tokens of a channel are then
// one 16-byte load that is an operand of the matrix instruction as it stands.
//
// Writing tokens into a page, per head:
//   a'   = max(a, max |new values|)      (a counts as 0 where slot 0 is written)
//   c'   = rne(fl32(c * fl32(a / a')))   for the tokens that were there, if a' > a
//   code = rne(fl32(x * fl32(127 / a'))) for the new ones
// The magnitude of a page only grows, and the codes that it held are moved to
// the new scale in the same pass, so that a page always has one scale whatever
// the steps it was written in. Magnitudes under 2^-64 count as zero, so
// that reciprocals and ratios of magnitudes stay in fp32. A NaN or infinity makes
// the page's magnitude one, its codes zeros, and all that is read of them NaN.
#include <algorithm>

#include "kv_common.h"

namespace llmint8 {

namespace {

constexpr float kTiny = 5.42101086242752217e-20f;  // 2^-64

// rne(x) for |x| < 2^22 in the low byte of the result's bits
__device__ __forceinline__ uint32_t rne_bits(float x) {
  return __builtin_bit_cast(uint32_t, x + 12582912.0f);
}

// low bytes of four words, packed
__device__ __forceinline__ uint32_t pack_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0c0c0400u);
  const uint32_t hi = __builtin_amdgcn_perm(d, c, 0x0c0c0400u);
  return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}

// four codes times r, rounded half to even
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float r) {
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = rne_bits((float)(int)(int8_t)(w >> (8 * i)) * r);
  return pack_bytes(v[0], v[1], v[2], v[3]);
}

template <bool BF16>
__device__ __forceinline__ void widen8(const uint4& v, float f[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = Act16<BF16>::to_f32((w[i >> 1] >> (16 * (i & 1))) & 0xffffu);
}

// Rotary positions over the first `rot` channels: pairs are (i, i + rot / 2), or
// (2 i, 2 i + 1) interleaved; products and sums are rounded one by one. A row is
// worked on in units of 16 channels: 16 neighbours, or, with the halves apart, 8
// channels and the 8 that they pair with.
//
// VEC: rot is a multiple of 16 (0: no rotation), so that a unit's pairs are its own
// and its angles are vectors. Otherwise units are 16 neighbours and partners and
// angles are read one by one.
template <bool VEC>
struct Rope {
  const float* table;  // [rows, rot]: cosines, then sines; null: none
  int rows, rot, interleaved;
  __device__ __forceinline__ bool turned(int u) const { return table && 16 * u < rot; }
  __device__ __forceinline__ bool paired(int u) const { return VEC && !interleaved && turned(u); }
  __device__ __forceinline__ int low(int u) const { return paired(u) ? u << 3 : u << 4; }  // channels of f[0..7]
  __device__ __forceinline__ int high(int u) const { return paired(u) ? (u << 3) + (rot >> 1) : (u << 4) + 8; }
  __device__ __forceinline__ const float* row(int pos) const { return table + (int64_t)min(max(pos, 0), rows - 1) * rot; }
};

// Cosines and sines of a unit's eight pairs.
struct Angles {
  float c[8], s[8];
};
__device__ __forceinline__ void load4(const float* p, float* f) {
  const v4f v = *reinterpret_cast<const v4f*>(p);
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = v[i];
}
template <bool VEC>
__device__ __forceinline__ void angles_of(const Rope<VEC>& r, int u, int pos, Angles* a) {
  if (!VEC || !r.turned(u)) return;
  const float* cs = r.row(pos);
  const int half = r.rot >> 1;
  load4(cs + 8 * u, a->c);
  load4(cs + 8 * u + 4, a->c + 4);
  load4(cs + half + 8 * u, a->s);
  load4(cs + half + 8 * u + 4, a->s + 4);
}

template <bool VEC>
__device__ __forceinline__ void load_unit(const Rope<VEC>& r, const uint16_t* row, int u, uint4 raw[2]) {
  raw[0] = *reinterpret_cast<const uint4*>(row + r.low(u));
  raw[1] = *reinterpret_cast<const uint4*>(row + r.high(u));
}
template <bool BF16, bool VEC>
__device__ __forceinline__ void turn_unit(const Rope<VEC>& r, const uint16_t* row, int u, int pos, const Angles& a,
                                          const uint4 raw[2], float f[16]) {
  widen8<BF16>(raw[0], f);
  widen8<BF16>(raw[1], f + 8);
  if (!r.turned(u)) return;
  if constexpr (VEC) {
    if (r.interleaved) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x1 = f[2 * j], x2 = f[2 * j + 1];
        f[2 * j] = x1 * a.c[j] - x2 * a.s[j];
        f[2 * j + 1] = x2 * a.c[j] + x1 * a.s[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float x1 = f[j], x2 = f[8 + j];
        f[j] = x1 * a.c[j] - x2 * a.s[j];
        f[8 + j] = x2 * a.c[j] + x1 * a.s[j];
      }
    }
  } else {
    const float* cs = r.row(pos);
    const int half = r.rot >> 1;
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int ch = 16 * u + j;
      if (ch >= r.rot) break;
      const bool first = r.interleaved ? (ch & 1) == 0 : ch < half;
      const int i = r.interleaved ? ch >> 1 : first ? ch : ch - half;
      const float x = Act16<BF16>::to_f32(row[ch]);
      const float g = Act16<BF16>::to_f32(row[r.interleaved ? ch ^ 1 : first ? ch + half : ch - half]);
      f[j] = first ? x * cs[i] - g * cs[half + i] : x * cs[i] + g * cs[half + i];
    }
  }
}

template <bool BF16>
__device__ __forceinline__ uint4 round8(const float f[8]) {
  return make_uint4(Act16<BF16>::pack2(f[0], f[1]), Act16<BF16>::pack2(f[2], f[3]), Act16<BF16>::pack2(f[4], f[5]),
                    Act16<BF16>::pack2(f[6], f[7]));
}

// Bytes j of eight words -> for each j (0..3), the eight bytes as two words.
__device__ __forceinline__ void transpose8x4(const uint32_t w[8], uint32_t lo[4], uint32_t hi[4]) {
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const uint32_t* x = w + 4 * p;
    uint32_t* out = p ? hi : lo;
    const uint32_t a = __builtin_amdgcn_perm(x[1], x[0], 0x05010400u);  // x0.0 x1.0 x0.1 x1.1
    const uint32_t b = __builtin_amdgcn_perm(x[3], x[2], 0x05010400u);
    const uint32_t c = __builtin_amdgcn_perm(x[1], x[0], 0x07030602u);  // x0.2 x1.2 x0.3 x1.3
    const uint32_t d = __builtin_amdgcn_perm(x[3], x[2], 0x07030602u);
    out[0] = __builtin_amdgcn_perm(b, a, 0x05040100u);
    out[1] = __builtin_amdgcn_perm(b, a, 0x07060302u);
    out[2] = __builtin_amdgcn_perm(d, c, 0x05040100u);
    out[3] = __builtin_amdgcn_perm(d, c, 0x07060302u);
  }
}

}  // namespace

// A page that the call writes to (found by kv_find) and one of `across` parts of
// its heads, neighbours in the grid: NT threads to a head's K or V, 256 / NT of
// these to a workgroup; the rest of the parts rotate q.
//
// HBM-bound for prompts (NT 256): every input is read once, as what a thread holds
// of a page stays in registers between the maximum and the codes, and the angles
// of a token once for four heads of q. 7495 tokens of 32 and 8 heads of 128 take 42
// us, 169 MB at 4.0 TB/s. A step writes few tokens (NT 64): there the time is that
// of the loads that wait for each other (one token 4.4 us, one of each of 256
// sequences 9.9 us), and a wavefront takes a head, a thread one unit of q. Measured
// with the gather of the open pages (us, NT 64 / 256): 256 sequences of one token
// 26 / 44; 64 of four 18 / 21, of six 19 / 21, of eight 23 / 21, of 32 46 / 27.
//
// VEC: Rope's. Partners and angles that are read one by one take registers that
// the vectors of the other form need, so the two are kept apart. The form without
// is slow (the same tokens with 24 of 128 channels turned 192 us, with all turned
// 35, both from the caches; 150 scalars spilled); head sizes in use have vectors.
template <int NT, bool VEC>
__host__ __device__ constexpr int q_heads_of(int dim) { return NT == 64 ? 256 / (dim >> 4) : VEC ? 4 : 1; }

template <bool BF16, int NT, bool VEC>
__global__ __launch_bounds__(256, VEC ? 4 : 2) void kc_append(KvAppendArgs a, int across) {
  __shared__ float red[4];
  __shared__ int sh_seq[6];
  const int P = 1 << a.c.page_shift, D = a.c.dim, H = a.c.heads;
  const int block = (int)(blockIdx.x % across);
  int index, count;
  KvSeq q;
  if (!kv_find<256>(a.s, a.c.page_shift, blockIdx.x / across, 1, a.c.page_shift, sh_seq, &q, &index, &count)) return;
  const int pos0 = q.pos0;
  auto write_page = [&](int entry) {
    const KvOnPage on = kv_on_page(q, entry, a.c.page_shift);
    const int t0 = on.t0, t1 = on.t1;
    if (t0 >= t1) return;
    const int n = t1 - t0, s0 = t0 - on.base;
    const Rope<VEC> rope{a.rope, a.rope_rows, a.rot, a.interleaved};
    const int units = D >> 4;
    constexpr int kPer = 256 / NT;
    const int kv_blocks = (2 * H + kPer - 1) / kPer;
    if (block >= kv_blocks) {
      constexpr int kTogether = NT == 256 && VEC ? 4 : 1;  // heads of a thread
      const int per = 256 / units, mine = threadIdx.x / units, u = threadIdx.x - mine * units;
      const int h0 = (block - kv_blocks) * q_heads_of<NT, VEC>(D) + (NT == 256 ? 0 : mine);
      const int t_step = NT == 256 ? per : 1;
      for (int t = 0; t < n; t += t_step) {
        const int pos = t0 + t + (NT == 256 ? mine : 0);
        const bool live = mine < per && pos < t1;
        const int64_t row = q.row0 + (pos - pos0);
        const uint16_t* from = a.q.p + row * a.q.token + (int64_t)h0 * a.q.head;
        uint16_t* to = a.qo.p + row * a.qo.token + (int64_t)h0 * a.qo.head;
        Angles ang;
        uint4 raw[kTogether][2];
        if (live) {
#pragma unroll
          for (int k = 0; k < kTogether; ++k)
            if (h0 + k < a.q_heads) load_unit(rope, from + (int64_t)k * a.q.head, u, raw[k]);
          angles_of(rope, u, pos, &ang);
        }
#pragma unroll
        for (int k = 0; k < kTogether; ++k) {
          float f[16];
          const bool in = live && h0 + k < a.q_heads;
          if (in) turn_unit<BF16>(rope, from + (int64_t)k * a.q.head, u, pos, ang, raw[k], f);
          // where partners are read one by one, all of a row (whole rows are a step's) has been read before
          // any of it is written: q may be turned where it stands
          if (!VEC) __syncthreads();
          if (!in) continue;
          *reinterpret_cast<uint4*>(to + (int64_t)k * a.qo.head + rope.low(u)) = round8<BF16>(f);
          *reinterpret_cast<uint4*>(to + (int64_t)k * a.qo.head + rope.high(u)) = round8<BF16>(f + 8);
        }
      }
      return;
    }
    const int tid = threadIdx.x % NT;
    const int y = block * kPer + (int)threadIdx.x / NT;
    if (y >= 2 * H) return;  // whole wavefronts, and no barrier follows where they are parts of a workgroup
    const bool isv = y >= H;
    const int h = isv ? y - H : y;
    const int page = kv_entry_page(a.s, q.b, entry, a.c.pages);
    if (page < 0) return;
    const KvRows src = isv ? a.v : a.k;
    const int64_t ph = (int64_t)page * H + h;
    int8_t* codes = (isv ? a.c.V : a.c.K) + ph * ((int64_t)P * D);
    float* amax = (isv ? a.c.aV : a.c.aK) + ph;
    const uint16_t* rows = src.p + (int64_t)(q.row0 + (t0 - pos0)) * src.token + (int64_t)h * src.head;
    const float old = s0 > 0 ? *amax : 0.0f;
    float m = 0.0f;
    auto reduce = [&]() {
#pragma unroll
      for (int o = 32; o > 0; o >>= 1) m = max_or_nan(m, __shfl_xor(m, o, 64));
      if constexpr (NT == 256) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
        __syncthreads();
        m = max_or_nan(max_or_nan(red[0], red[1]), max_or_nan(red[2], red[3]));
      }
    };
    float now = 0.0f, scale = 0.0f;
    auto settle = [&]() {  // the page's new magnitude, and the codes that were there moved to it
      reduce();
      now = max_or_nan(old, m);
      now = now < kTiny ? 0.0f : now;
      scale = now > 0.0f ? 127.0f / now : 0.0f;
      if (tid == 0) *amax = now;
      if (!(now > old) || s0 == 0) return;
      const float r = old / now;
      if (!isv) {
        uint32_t* w = reinterpret_cast<uint32_t*>(codes);
        for (int i = tid; i < (s0 * D) >> 2; i += NT) w[i] = rescale4(w[i], r);
      } else {  // whole words of four tokens, then the one that the new tokens begin in
        const int quads = s0 >> 2;
        for (int i = tid; i < D * quads; i += NT) {
          const int c = i / quads;
          uint32_t* w = reinterpret_cast<uint32_t*>(codes + (int64_t)c * P) + (i - c * quads);
          *w = rescale4(*w, r);
        }
        for (int i = tid; i < D * (s0 & 3); i += NT) {
          const int c = i / (s0 & 3);
          int8_t* at = codes + (int64_t)c * P + (s0 & ~3) + (i - c * (s0 & 3));
          *at = (int8_t)rne_bits((float)*at * r);
        }
      }
    };
    if (!isv) {
      const int total = n * units;
      auto put = [&](int t, int u, const float f[16]) {
        uint32_t r[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) r[j] = rne_bits(f[j] * scale);
        int8_t* to = codes + (int64_t)(s0 + t) * D;
        *reinterpret_cast<uint2*>(to + rope.low(u)) =
            make_uint2(pack_bytes(r[0], r[1], r[2], r[3]), pack_bytes(r[4], r[5], r[6], r[7]));
        *reinterpret_cast<uint2*>(to + rope.high(u)) =
            make_uint2(pack_bytes(r[8], r[9], r[10], r[11]), pack_bytes(r[12], r[13], r[14], r[15]));
      };
      auto turn = [&](int t, int u, const Angles& ang, const uint4 raw[2], float f[16]) {
        turn_unit<BF16>(rope, rows + (int64_t)t * src.token, u, t0 + t, ang, raw, f);
#pragma unroll
        for (int j = 0; j < 16; ++j) m = max_or_nan(m, fabsf(f[j]));
      };
      auto get = [&](int t, int u, float f[16]) {
        Angles ang;
        uint4 raw[2];
        load_unit(rope, rows + (int64_t)t * src.token, u, raw);
        angles_of(rope, u, t0 + t, &ang);
        turn(t, u, ang, raw, f);
      };
      constexpr int kHold = NT == 256 && VEC ? 2 : 1;  // units of a thread that stay in registers
      if (total <= kHold * NT) {
        float f[kHold][16];
        uint4 raw[kHold][2];
        Angles ang[kHold];
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
          const int x = tid + NT * i, t = x / units;
          if (x < total) {
            load_unit(rope, rows + (int64_t)t * src.token, x - t * units, raw[i]);
            angles_of(rope, x - t * units, t0 + t, &ang[i]);
          }
        }
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
          const int x = tid + NT * i, t = x / units;
          if (x < total) turn(t, x - t * units, ang[i], raw[i], f[i]);
        }
        settle();
#pragma unroll
        for (int i = 0; i < kHold; ++i) {
          const int x = tid + NT * i, t = x / units;
          if (x < total) put(t, x - t * units, f[i]);
        }
      } else {  // pages of more: read again for the codes
        float f[16];
        for (int x = tid; x < total; x += NT) get(x / units, x % units, f);
        settle();
        for (int x = tid; x < total; x += NT) {
          get(x / units, x % units, f);
          put(x / units, x % units, f);
        }
      }
      return;
    }
    // V: four tokens (a word of V's rows) of eight channels to a thread
    const int cpr = D >> 3, q0 = s0 >> 2, quads = ((s0 + n + 3) >> 2) - q0, total = quads * cpr;
    auto get = [&](int x, uint4 raw[4]) {
      const int quad = x / cpr, c0 = (x - quad * cpr) * 8, t = 4 * (q0 + quad) - s0;  // t: token of the call, may begin before it
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        raw[j] = make_uint4(0, 0, 0, 0);
        if (t + j >= 0 && t + j < n) raw[j] = *reinterpret_cast<const uint4*>(rows + (int64_t)(t + j) * src.token + c0);
      }
    };
    auto top = [&](const uint4 raw[4]) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float f[8];
        widen8<BF16>(raw[j], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) m = max_or_nan(m, fabsf(f[k]));
      }
    };
    auto put = [&](int x, const uint4 raw[4]) {
      const int quad = x / cpr, c0 = (x - quad * cpr) * 8, t = 4 * (q0 + quad) - s0;
      uint32_t w[8];  // a word per channel
      uint32_t r[4][8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float f[8];
        widen8<BF16>(raw[j], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) r[j][k] = rne_bits(f[k] * scale);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) w[k] = pack_bytes(r[0][k], r[1][k], r[2][k], r[3][k]);
      int8_t* to = codes + (int64_t)c0 * P + 4 * (q0 + quad);
      if (t >= 0 && t + 4 <= n) {
#pragma unroll
        for (int k = 0; k < 8; ++k) *reinterpret_cast<uint32_t*>(to + (int64_t)k * P) = w[k];
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (t + j >= 0 && t + j < n)
#pragma unroll
            for (int k = 0; k < 8; ++k) to[(int64_t)k * P + j] = (int8_t)(w[k] >> (8 * j));
      }
    };
    uint4 raw[4];
    if (total <= NT) {
      if (tid < total) {
        get(tid, raw);
        top(raw);
      }
      settle();
      if (tid < total) put(tid, raw);
    } else {
      for (int x = tid; x < total; x += NT) {
        get(x, raw);
        top(raw);
      }
      settle();
      for (int x = tid; x < total; x += NT) {
        get(x, raw);
        put(x, raw);
      }
    }
  };
  const KvEntries own = kv_item_entries(pos0, index, count, a.c.page_shift);
  write_page(own.first);
  if (own.count > 1) {
    __syncthreads();
    write_page(own.first + 1);
  }
}

template <int NT, bool VEC>
static hipError_t launch_append(const KvAppendArgs& a, bool bf16, hipStream_t stream) {
  const int items = (a.s.T >> a.c.page_shift) + a.s.B, per = 256 / NT, qh = q_heads_of<NT, VEC>(a.c.dim);
  const int across = (2 * a.c.heads + per - 1) / per + (a.q.p ? (a.q_heads + qh - 1) / qh : 0);
  if ((int64_t)items * across > INT32_MAX) return hipErrorInvalidConfiguration;
  const dim3 grid(items * across);
  if (bf16)
    hipLaunchKernelGGL((kc_append<true, NT, VEC>), grid, dim3(256), 0, stream, a, across);
  else
    hipLaunchKernelGGL((kc_append<false, NT, VEC>), grid, dim3(256), 0, stream, a, across);
  return hipGetLastError();
}

hipError_t launch_kv_append(const KvAppendArgs& a, bool bf16, hipStream_t stream) {
  const bool few = a.s.T <= 6 * (int64_t)a.s.B, vec = !a.rope || a.rot % 16 == 0;
  if (vec) return few ? launch_append<64, true>(a, bf16, stream) : launch_append<256, true>(a, bf16, stream);
  return few ? launch_append<64, false>(a, bf16, stream) : launch_append<256, false>(a, bf16, stream);
}

// A page that holds some of the asked tokens; K and V of `per` heads to a
// workgroup. HBM-bound: 16-byte stores of whole rows (streamed: nothing reads them
// here), K from 8-byte loads, V from words of four tokens that are transposed in
// registers, 8 channels and 4 tokens to a thread. 128000 tokens of 8 heads of 128,
// 788 MB: 157 us, 5.0 TB/s (a large copy: 5.2). Small calls wait for cu, table and
// codes one after the other: 5.2 us for one page, 18.8 for 256 pages of 51 MB.
template <bool BF16>
__global__ __launch_bounds__(256) void kc_gather(KvCache c, KvBatch s, KvRows k, KvRows v, int per, int across) {
  __shared__ int sh_seq[6];
  const int P = 1 << c.page_shift, D = c.dim, H = c.heads, tid = threadIdx.x;
  const int block = (int)(blockIdx.x % across);
  int index, count;
  KvSeq q;
  if (!kv_find<256>(s, c.page_shift, blockIdx.x / across, 1, c.page_shift, sh_seq, &q, &index, &count)) return;
  const int pos0 = q.pos0;
  auto read_page = [&](int entry) {
    const KvOnPage on = kv_on_page(q, entry, c.page_shift);
    const int t0 = on.t0, t1 = on.t1;
    if (t0 >= t1) return;
    const int page = kv_entry_page(s, q.b, entry, c.pages);
    const int cpr = D >> 3, n = t1 - t0, s0 = t0 - on.base;
    const int64_t row = q.row0 + (t0 - pos0);
    const int step = 256 / cpr, r0 = tid / cpr, c0 = (tid - r0 * cpr) * 8;  // a thread's row of a step, and channels
    if (r0 >= step) return;
    // a page that does not exist: any codes times zero
    auto out = [&](uint16_t* to, uint32_t x, uint32_t y, float st) {
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = (float)(int)(int8_t)((j < 4 ? x : y) >> (8 * (j & 3))) * st;
      const uint4 o = round8<BF16>(f);
      __builtin_nontemporal_store(v4i{(int)o.x, (int)o.y, (int)o.z, (int)o.w}, reinterpret_cast<v4i*>(to));
    };
    for (int h = block * per; h < min((block + 1) * per, H); ++h) {
      const int64_t ph = (int64_t)max(page, 0) * H + h;
      const float sk = page < 0 ? 0.0f : c.aK[ph] / 127.0f, sv = page < 0 ? 0.0f : c.aV[ph] / 127.0f;
      const int8_t* kc = c.K + ph * ((int64_t)P * D) + (int64_t)s0 * D + c0;
      const int8_t* vc = c.V + ph * ((int64_t)P * D) + (int64_t)c0 * P;
      uint16_t* kt = k.p + row * k.token + (int64_t)h * k.head + c0;
      uint16_t* vt = v.p + row * v.token + (int64_t)h * v.head + c0;
      const int q0 = s0 >> 2, q1 = (s0 + n + 3) >> 2;
      // 4 step tokens of K and 4 step slots of V at a time: all loads, then the stores
      for (int t = r0, quad = q0 + r0; t < n || quad < q1; t += 4 * step, quad += step) {
        uint2 x[4];
        uint32_t w[8], lo[4], hi[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const uint2*>(kc + (int64_t)min(t + i * step, n - 1) * D);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] = *reinterpret_cast<const uint32_t*>(vc + (int64_t)j * P + 4 * min(quad, q1 - 1));
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (t + i * step < n) out(kt + (t + i * step) * k.token, x[i].x, x[i].y, sk);
        if (quad >= q1) continue;
        transpose8x4(w, lo, hi);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = 4 * quad + i - s0;
          if (at >= 0 && at < n) out(vt + (int64_t)at * v.token, lo[i], hi[i], sv);
        }
      }
    }
  };
  const KvEntries own = kv_item_entries(pos0, index, count, c.page_shift);
  read_page(own.first);
  if (own.count > 1) read_page(own.first + 1);
}

hipError_t launch_kv_gather(const KvCache& c, const KvBatch& s, const KvRows& k, const KvRows& v, bool bf16,
                            int num_cus, hipStream_t stream) {
  const int items = (s.T >> c.page_shift) + s.B;
  // heads to a workgroup: one while that gives the chip no more than 32 to a CU (128000 tokens: 157 us, and
  // 165 with 16, 249 with 8; 64 as 32)
  const int per = (int)std::min<int64_t>(std::max<int64_t>(1, (int64_t)items * c.heads / (32 * num_cus)), c.heads);
  const int across = (c.heads + per - 1) / per;
  if ((int64_t)items * across > INT32_MAX) return hipErrorInvalidConfiguration;
  const dim3 grid(items * across);
  if (bf16)
    hipLaunchKernelGGL(kc_gather<true>, grid, dim3(256), 0, stream, c, s, k, v, per, across);
  else
    hipLaunchKernelGGL(kc_gather<false>, grid, dim3(256), 0, stream, c, s, k, v, per, across);
  return hipGetLastError();
}

// The angles are formed and reduced in 64 bits: p * f is exact to 2^-53 of
// itself, where 32 bits would be off by 0.06 radian at position 10^6.
__global__ __launch_bounds__(256) void kc_rope_table(RopeFreq f, int pairs, int rows, double mag,
                                                     float* __restrict__ table) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= (int64_t)rows * pairs) return;
  const int p = (int)(i / pairs), j = (int)(i - (int64_t)p * pairs);
  double s, c;
  sincos((double)p * f.f[j], &s, &c);
  table[(int64_t)p * 2 * pairs + j] = (float)(mag * c);
  table[(int64_t)p * 2 * pairs + pairs + j] = (float)(mag * s);
}

hipError_t launch_rope_table(const RopeFreq& f, int pairs, int rows, double mag, float* table,
                             hipStream_t stream) {
  const int64_t n = (int64_t)rows * pairs;
  hipLaunchKernelGGL(kc_rope_table, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, stream, f, pairs, rows,
                     mag, table);
  return hipGetLastError();
}

}  // namespace llmint8
