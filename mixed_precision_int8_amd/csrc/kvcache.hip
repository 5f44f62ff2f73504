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
// that reciprocals and ratios of magnitudes stay in fp32.
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

// Channels [c0, c0 + 8) of one row, rotated by the angles of position `pos`
// where they are among the first `rot`. Pairs are (i, i + rot / 2) or, in the
// interleaved layout, (2 i, 2 i + 1); products and sums are rounded one by one.
template <bool BF16>
__device__ __forceinline__ void load_rotated8(const uint16_t* row, int c0, const float* rope, int rope_rows,
                                              int rot, int interleaved, int pos, float f[8]) {
  widen8<BF16>(*reinterpret_cast<const uint4*>(row + c0), f);
  if (!rope || c0 >= rot) return;
  const float* cs = rope + (int64_t)min(max(pos, 0), rope_rows - 1) * rot;
  const int half = rot >> 1;
  if (interleaved) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      if (c0 + j >= rot) break;
      const float c = cs[(c0 + j) >> 1], s = cs[half + ((c0 + j) >> 1)];
      const float x1 = f[j], x2 = f[j + 1];
      f[j] = x1 * c - x2 * s;
      f[j + 1] = x2 * c + x1 * s;
    }
    return;
  }
  if ((half & 7) == 0) {  // the partners are one aligned vector
    const bool first = c0 < half;
    const int i0 = first ? c0 : c0 - half;
    float g[8];
    widen8<BF16>(*reinterpret_cast<const uint4*>(row + (first ? c0 + half : c0 - half)), g);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float c = cs[i0 + j], s = cs[half + i0 + j];
      f[j] = first ? f[j] * c - g[j] * s : f[j] * c + g[j] * s;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int ch = c0 + j;
    if (ch >= rot) break;
    const bool first = ch < half;
    const int i = first ? ch : ch - half;
    const float g = Act16<BF16>::to_f32(row[first ? ch + half : ch - half]);
    const float c = cs[i], s = cs[half + i];
    f[j] = first ? f[j] * c - g * s : f[j] * c + g * s;
  }
}

__device__ __forceinline__ float block_max(float m, float* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  return fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
}

}  // namespace

// One workgroup per (page that the call writes to, head, K or V); the rest of
// the grid's second axis rotates q, four heads of the page's tokens at a time.
template <bool BF16>
__global__ __launch_bounds__(256) void kc_append(KvAppendArgs a) {
  __shared__ float red[4];
  const int P = 1 << a.c.page_shift, D = a.c.dim, H = a.c.heads;
  __shared__ int sh_seq[4];
  int first;
  KvSeq q;
  if (!kv_find<256>(a.s, a.c.page_shift, blockIdx.x, 1, a.c.page_shift, 2, sh_seq, &q, &first)) return;
  const int b = q.b;
  const int pos0 = q.len - q.n;                             // position of row0 (< 0: those rows are dropped)
  const int entry = (max(pos0, 0) >> a.c.page_shift) + ((int)blockIdx.x - first);
  const int base = entry << a.c.page_shift;                 // position of slot 0
  const int t0 = max(pos0, base), t1 = min(q.len, base + P);  // positions written
  if (q.n == 0 || t0 >= t1) return;
  const int cpr = D >> 3;  // 8-channel chunks per row
  const int y = blockIdx.y;
  const int tid = threadIdx.x;
  if (y >= 2 * H) {
    const int h0 = (y - 2 * H) * 4, hn = min(4, a.q_heads - h0);
    const int per = hn * cpr, total = (t1 - t0) * per;
    // whole heads to a step, and every load of a step before its first store: q may be turned in place
    const int step = 256 / cpr * cpr;
    for (int i0 = 0; i0 < total; i0 += step) {
      const int i = i0 + tid;
      const bool mine = tid < step && i < total;
      const int t = i / per, r = i - t * per;
      const int h = h0 + r / cpr, c0 = (r % cpr) * 8;
      const int64_t row = q.row0 + (t0 + t - pos0);
      float f[8] = {};
      if (mine)
        load_rotated8<BF16>(a.q.p + row * a.q.token + (int64_t)h * a.q.head, c0, a.rope, a.rope_rows, a.rot,
                            a.interleaved, t0 + t, f);
      __syncthreads();
      if (!mine) continue;
      uint4 o;
      o.x = Act16<BF16>::pack2(f[0], f[1]);
      o.y = Act16<BF16>::pack2(f[2], f[3]);
      o.z = Act16<BF16>::pack2(f[4], f[5]);
      o.w = Act16<BF16>::pack2(f[6], f[7]);
      *reinterpret_cast<uint4*>(a.qo.p + row * a.qo.token + (int64_t)h * a.qo.head + c0) = o;
    }
    return;
  }
  const bool isv = y >= H;
  const int h = isv ? y - H : y;
  const int page = kv_page(kv_entry(a.s, b, entry), a.c.pages);
  if (page < 0) return;
  const KvRows src = isv ? a.v : a.k;
  const float* rope = isv ? nullptr : a.rope;
  const int64_t ph = (int64_t)page * H + h;
  int8_t* codes = (isv ? a.c.V : a.c.K) + ph * ((int64_t)P * D);
  float* amax = (isv ? a.c.aV : a.c.aK) + ph;
  const uint16_t* rows = src.p + (int64_t)(q.row0 + (t0 - pos0)) * src.token + (int64_t)h * src.head;
  const int n = t1 - t0, s0 = t0 - base;
  float m = 0.0f;
  for (int i = tid; i < n * cpr; i += 256) {
    const int t = i / cpr, c0 = (i - t * cpr) * 8;
    float f[8];
    load_rotated8<BF16>(rows + (int64_t)t * src.token, c0, rope, a.rope_rows, a.rot, a.interleaved, t0 + t, f);
#pragma unroll
    for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
  }
  const float old = s0 > 0 ? *amax : 0.0f;
  m = block_max(m, red);
  float now = fmaxf(old, m);
  now = now < kTiny ? 0.0f : now;
  const float s = now > 0.0f ? 127.0f / now : 0.0f;
  // the tokens that were there, moved to the new scale
  if (now > old && s0 > 0) {
    const float r = old / now;
    if (!isv) {
      uint32_t* w = reinterpret_cast<uint32_t*>(codes);
      for (int i = tid; i < (s0 * D) >> 2; i += 256) w[i] = rescale4(w[i], r);
    } else {
      for (int i = tid; i < D * s0; i += 256) {
        const int c = i / s0, t = i - c * s0;
        int8_t* at = codes + (int64_t)c * P + t;
        *at = (int8_t)rne_bits((float)*at * r);
      }
    }
  }
  __syncthreads();  // amax has been read by all
  if (tid == 0) *amax = now;
  for (int i = tid; i < n * cpr; i += 256) {
    const int t = i / cpr, c0 = (i - t * cpr) * 8;
    float f[8];
    load_rotated8<BF16>(rows + (int64_t)t * src.token, c0, rope, a.rope_rows, a.rot, a.interleaved, t0 + t, f);
    uint32_t r[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) r[j] = rne_bits(f[j] * s);
    if (!isv) {
      *reinterpret_cast<uint2*>(codes + (int64_t)(s0 + t) * D + c0) =
          make_uint2(pack_bytes(r[0], r[1], r[2], r[3]), pack_bytes(r[4], r[5], r[6], r[7]));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) codes[(int64_t)(c0 + j) * P + s0 + t] = (int8_t)r[j];
    }
  }
}

hipError_t launch_kv_append(const KvAppendArgs& a, bool bf16, hipStream_t stream) {
  const int items = (a.s.T >> a.c.page_shift) + 2 * a.s.B;
  const int qy = a.q.p ? (a.q_heads + 3) / 4 : 0;
  const dim3 grid(items, 2 * a.c.heads + qy);
  if (bf16)
    hipLaunchKernelGGL(kc_append<true>, grid, dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL(kc_append<false>, grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

// One workgroup per (page that holds some of the asked tokens, head, K or V).
template <bool BF16>
__global__ __launch_bounds__(256) void kc_gather(KvCache c, KvBatch s, KvRows k, KvRows v) {
  const int P = 1 << c.page_shift, D = c.dim, H = c.heads;
  __shared__ int sh_seq[4];
  int first;
  KvSeq q;
  if (!kv_find<256>(s, c.page_shift, blockIdx.x, 1, c.page_shift, 2, sh_seq, &q, &first)) return;
  const int b = q.b;
  const int pos0 = q.len - q.n;
  const int entry = (max(pos0, 0) >> c.page_shift) + ((int)blockIdx.x - first);
  const int base = entry << c.page_shift;
  const int t0 = max(pos0, base), t1 = min(q.len, base + P);
  if (q.n == 0 || t0 >= t1) return;
  const bool isv = (int)blockIdx.y >= H;
  const int h = isv ? blockIdx.y - H : blockIdx.y;
  const int page = kv_page(kv_entry(s, b, entry), c.pages);
  const int64_t ph = (int64_t)max(page, 0) * H + h;
  const int8_t* codes = (isv ? c.V : c.K) + ph * ((int64_t)P * D);
  const float st = page < 0 ? 0.0f : (isv ? c.aV : c.aK)[ph] / 127.0f;
  const KvRows dst = isv ? v : k;
  const int cpr = D >> 3, n = t1 - t0, s0 = t0 - base;
  uint16_t* rows = dst.p + (int64_t)(q.row0 + (t0 - pos0)) * dst.token + (int64_t)h * dst.head;
  for (int i = threadIdx.x; i < n * cpr; i += 256) {
    const int t = i / cpr, c0 = (i - t * cpr) * 8;
    float f[8];
    if (!isv) {
      const uint2 w = *reinterpret_cast<const uint2*>(codes + (int64_t)(s0 + t) * D + c0);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = (float)(int)(int8_t)((j < 4 ? w.x : w.y) >> (8 * (j & 3))) * st;
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = (float)(int)codes[(int64_t)(c0 + j) * P + s0 + t] * st;
    }
    uint4 o;
    o.x = Act16<BF16>::pack2(f[0], f[1]);
    o.y = Act16<BF16>::pack2(f[2], f[3]);
    o.z = Act16<BF16>::pack2(f[4], f[5]);
    o.w = Act16<BF16>::pack2(f[6], f[7]);
    *reinterpret_cast<uint4*>(rows + (int64_t)t * dst.token + c0) = o;
  }
}

hipError_t launch_kv_gather(const KvCache& c, const KvBatch& s, const KvRows& k, const KvRows& v, bool bf16,
                            hipStream_t stream) {
  const dim3 grid((s.T >> c.page_shift) + 2 * s.B, 2 * c.heads);
  if (bf16)
    hipLaunchKernelGGL(kc_gather<true>, grid, dim3(256), 0, stream, c, s, k, v);
  else
    hipLaunchKernelGGL(kc_gather<false>, grid, dim3(256), 0, stream, c, s, k, v);
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
