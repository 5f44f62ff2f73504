// Attention of long runs of rows over the int8 key/value cache on gfx950: the
// same function as kv_step (kvattn.hip), for calls that the matrix cores bound.
//
// A workgroup takes 128 rows of a sequence and head group (tokens times the
// group's heads), 32 to a wavefront, and goes over the tokens in tiles of 64.
// Here a code is used by 128 rows, so it is converted once: int8 codes are exact
// in fp16, the tile goes to LDS as fp16 without its scales, and both products run
// on v_mfma_f32_32x32x16_f16.
//   S^T = K . q^T   A = 32 tokens x 16 channels from LDS, B = q in registers, fp16
//                   (bf16 rows times a power of two that brings the largest
//                   channel to 2^13: exact but for channels under 2^-30 of it,
//                   whose last bits are below fp16's 2^-24)
//   O^T = V^T . P^T A = 32 channels x 16 tokens from LDS, B = the weights as fp16
// Tokens are assigned to the rows of S^T so that a lane's weights are, in order,
// its operand of the second product (bits 2 and 3 of the row swapped). Scales
// enter between the products: 16 tokens of a tile share a page at least, and
//   u = s * (unit aK) + log2(aV / 127),  w = exp2(u - m + 8)
// is one multiply-add and one exponential a token; m is the row's running
// maximum, left where it is until a tile exceeds it by 2^7, so that a weight is at
// most 2^15 in fp16 and those down to 2^-32 of it count.
//
// A tile's codes are loaded to registers while the one before is computed, and
// go to the other half of LDS, converted, between its products: one barrier to a
// tile.
//
// Bound by the SIMDs' issue of vector and matrix instructions together (55% and
// 40-45% of the time on long prompts; the softmax, the conversion and about a dozen
// of 49 spilled scalars read back to a tile are what the first are) and by LDS: a
// tile's products read it once for every wavefront, 160 KB with the stores, 1280
// cycles of a CU at 128 bytes a cycle where its matrix instructions take 1024, and
// the stores' lanes, 16 bytes at a stride of 32, conflict. One prompt of 16384 tokens of 32 heads of 128 runs at 1040 TFLOP/s,
// prompts of 2000-4096 behind 5000 at 880-920 (their last tiles are masked, the last
// workgroups alone, and the rows that start first are the last sequence's, not the
// longest of the call), where a large product of the library runs at 1530.
#include <algorithm>
#include <type_traits>

#include "kv_common.h"

namespace llmint8 {

namespace {

typedef _Float16 v2h __attribute__((ext_vector_type(2)));

constexpr float kNegInf = -__builtin_inff();
constexpr float kMinMag = 5.42101086242752217e-20f;  // 2^-64, as in kvattn.hip

// 16 codes -> fp16: 1024 + (c + 128) is a byte under the exponent of 1024
__device__ __forceinline__ void widen16(const v4i& c, uint4* lo, uint4* hi) {
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = (uint32_t)c[i] ^ 0x80808080u;
    const v2h off = {(_Float16)1152.0f, (_Float16)1152.0f};
    r[2 * i] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, __builtin_amdgcn_perm(0x64646464u, x, 0x04010400u)) - off);
    r[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, __builtin_amdgcn_perm(0x64646464u, x, 0x04030402u)) - off);
  }
  *lo = make_uint4(r[0], r[1], r[2], r[3]);
  *hi = make_uint4(r[4], r[5], r[6], r[7]);
}

__device__ __forceinline__ v16f_t mfma(const uint4& a, const uint4& b, const v16f_t& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// with the other half's lane of the same row (lanes n and n + 32)
__device__ __forceinline__ float other_half(float v, float* other) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  *other = __uint_as_float(r[1]);
  return __uint_as_float(r[0]);
}
__device__ __forceinline__ float pair_max(float v) {
  float o;
  v = other_half(v, &o);
  return fmaxf(v, o);
}
__device__ __forceinline__ float pair_sum(float v) {
  float o;
  v = other_half(v, &o);
  return v + o;
}

}  // namespace

// FULL: dim = DP. ONE: a tile is within one page. W: wavefronts.
template <int DP, bool FULL, bool ONE, int W>
__global__ __launch_bounds__(64 * W, DP <= 128 ? 2 : 1) void kv_prompt(KvAttnArgs a) {
  constexpr int kThreads = 64 * W, kRows = 32 * W;
  constexpr int NQ = DP / 16;   // 16-channel steps of the first product
  constexpr int ND = DP / 32;   // 32-channel blocks of the second
  constexpr int NU = 4 * DP / kThreads;  // 16-byte pieces of a tile's K (and V) for a thread
  // rows in LDS: a 16-byte chunk more than their values, so that 16 rows' reads at one place of the row
  // fall on different banks
  constexpr int kKPitch = 2 * DP + 16, kVPitch = 2 * 64 + 16;
  constexpr int kKBytes = 64 * kKPitch, kVBytes = DP * kVPitch;
  __shared__ __attribute__((aligned(16))) char smem_k[2 * kKBytes], smem_v[2 * kVBytes];
  __shared__ int sh_seq[6];
  const int D = FULL ? DP : a.c.dim;
  const int shift = a.c.page_shift, P = 1 << shift, H = a.c.heads, G = a.q_heads / H;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int hf = lane >> 5, nn = lane & 31;
  int run, count;
  KvSeq sq;
  // the last rows of a sequence see the most: they start first
  const unsigned whole = gridDim.x / a.splits, at = blockIdx.x % whole;
  const int h = (int)(at % H), item = (int)((whole - 1 - at) / H), part = (int)(blockIdx.x / whole);
  if (!kv_find<kThreads>(a.s, shift, item, G, W == 4 ? 7 : 8, sh_seq, &sq, &run, &count)) return;
  const int64_t rows = (int64_t)sq.n * G, row0 = (int64_t)run * kRows;
  if (row0 >= rows) return;
  const int b = sq.b;
  const int r = (int)min(row0 + wave * 32 + nn, rows - 1);
  const int tok = r / G, qh = h * G + (r - tok * G);
  const int pos = sq.pos0 + tok;
  const int64_t qrow = sq.row0 + tok;
  const int pos_lo = sq.pos0 + (int)row0 / G;
  const int pos_hi = sq.pos0 + (int)(min(row0 + kRows, rows) - 1) / G;

  // tiles that any of the rows sees
  const int end = a.causal ? min(sq.len, pos_hi + 1) : sq.len;
  const int hi = end > 0 ? (end + 63) >> 6 : 0;
  const int lo = min(a.window > 0 ? max(pos_lo - a.window + 1, 0) >> 6 : 0, hi);
  const int sink = a.window > 0 ? min((int)(((int64_t)a.sinks + 63) >> 6), lo) : 0;
  const int all = sink + hi - lo;
  const int i0 = (int)((int64_t)all * part / a.splits), tiles = (int)((int64_t)all * (part + 1) / a.splits) - i0;
  auto base_of = [&](int i) { return (i0 + i < sink ? i0 + i : lo + i0 + i - sink) << 6; };

  // q in fp16, and what one unit of S stands for
  uint4 q[NQ];
  float unit;
  {
    const uint16_t* qp = a.q.p + qrow * a.q.token + (int64_t)qh * a.q.head;
#pragma unroll
    for (int ks = 0; ks < NQ; ++ks) {
      const int c0 = ks * 16 + hf * 8;
      q[ks] = make_uint4(0, 0, 0, 0);
      if (FULL || c0 < D) q[ks] = *reinterpret_cast<const uint4*>(qp + c0);
    }
    unit = fabsf(a.scale) * 1.44269504088896341f * (1.0f / 127.0f);
    if (a.bf16) {
      uint32_t top = 0;
#pragma unroll
      for (int ks = 0; ks < NQ; ++ks) {
        const uint32_t w[4] = {q[ks].x, q[ks].y, q[ks].z, q[ks].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max(top, max(w[j] & 0x7fffu, (w[j] >> 16) & 0x7fffu));
      }
      const float m = pair_max(bf16_bits_to_float(top));
      // powers of two 2^(13 - e) and its inverse, e the exponent of the row's largest channel
      const int e = min(max((int)(__float_as_uint(m) >> 23) - 127, -100), 127);
      const float up = __uint_as_float((uint32_t)(13 - e + 127) << 23);
      unit *= __uint_as_float((uint32_t)(e - 13 + 127) << 23);
#pragma unroll
      for (int ks = 0; ks < NQ; ++ks) {
        const uint32_t w[4] = {q[ks].x, q[ks].y, q[ks].z, q[ks].w};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = Act16<false>::pack2(bf16_bits_to_float(w[j] & 0xffffu) * up, bf16_bits_to_float(w[j] >> 16) * up);
        q[ks] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    if (a.scale < 0.0f) {
#pragma unroll
      for (int ks = 0; ks < NQ; ++ks)
        q[ks] = make_uint4(q[ks].x ^ 0x80008000u, q[ks].y ^ 0x80008000u, q[ks].z ^ 0x80008000u, q[ks].w ^ 0x80008000u);
    }
  }

  // Pieces of 16 codes: K piece u is channels 16 (u % (DP / 16)) of token u / (DP / 16), V piece u is
  // tokens 16 (u % 4) of channel u / 4.
  // Page numbers of a tile, asked for a tile before they are needed.
  constexpr int NG = ONE ? 1 : 4;  // groups of 16 tokens that may be on pages of their own
  struct Numbers {
    int of[ONE ? 1 : NU > 4 ? NU : 4];
  };
  auto base_at = [&](int i) { return base_of(min(i, tiles - 1)); };
  auto k_numbers = [&](int i) {  // of this thread's K pieces
    Numbers n;
#pragma unroll
    for (int k = 0; k < (ONE ? 1 : NU); ++k)
      n.of[k] = kv_entry(a.s, b, (base_at(i) + (ONE ? 0 : (tid + kThreads * k) / (DP / 16))) >> shift);
    return n;
  };
  auto g_numbers = [&](int i) {  // of the groups
    Numbers n;
#pragma unroll
    for (int k = 0; k < NG; ++k) n.of[k] = kv_entry(a.s, b, (base_at(i) + 16 * k) >> shift);
    return n;
  };
  const int64_t page_bytes = (int64_t)P * D;
  v4i tk[NU], tv[NU];
  auto load_k = [&](int i, const Numbers& n) {
    const int base = base_at(i);
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int u = tid + kThreads * k;
      const int row = u / (DP / 16), c = (u % (DP / 16)) * 16;
      const int page = kv_page(ONE ? uniform(n.of[0]) : n.of[k], a.c.pages);
      const int8_t* p = a.c.K + ((int64_t)max(page, 0) * H + h) * page_bytes + (ONE ? base & (P - 1) : 0) * D;
      const uint32_t off = (uint32_t)(ONE ? row : (base + row) & (P - 1)) * D + (FULL || c < D ? c : 0);
      tk[k] = *reinterpret_cast<const v4i*>(p + off);
      if (!FULL && c >= D) tk[k] = v4i{0, 0, 0, 0};
    }
  };
  auto load_v = [&](int i, const Numbers& n) {
    const int base = base_at(i);
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int u = tid + kThreads * k;
      const int row = u >> 2, g = u & 3;
      int number = ONE ? uniform(n.of[0]) : n.of[0];
      if constexpr (!ONE) number = g == 0 ? n.of[0] : g == 1 ? n.of[1] : g == 2 ? n.of[2] : n.of[3];
      const int page = kv_page(number, a.c.pages);
      const int8_t* p = a.c.V + ((int64_t)max(page, 0) * H + h) * page_bytes + (ONE ? base & (P - 1) : 0);
      const uint32_t off = (uint32_t)(FULL || row < D ? row : 0) * P + (ONE ? 16 * g : (base + 16 * g) & (P - 1));
      tv[k] = *reinterpret_cast<const v4i*>(p + off);
    }
  };
  struct Scales {
    float ak[NG], av[NG];
    bool gone[NG];  // a page that does not exist
  };
  auto scales_of = [&](const Numbers& n) {
    Scales x;
#pragma unroll
    for (int k = 0; k < NG; ++k) {
      const int page = kv_page(uniform(n.of[k]), a.c.pages);
      const int64_t at = (int64_t)max(page, 0) * H + h;
      x.ak[k] = a.c.aK[at];
      x.av[k] = a.c.aV[at];
      x.gone[k] = page < 0;
    }
    return x;
  };
  // Pieces into LDS: K to the tokens' rows, V to the channels'.
  auto store_k = [&](auto stage) {
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int u = tid + kThreads * k;
      uint4 x, y;
      widen16(tk[k], &x, &y);
      char* to = smem_k + (u / (DP / 16) * kKPitch + u % (DP / 16) * 32) + stage * kKBytes;
      *reinterpret_cast<uint4*>(to) = x;
      *reinterpret_cast<uint4*>(to + 16) = y;
    }
  };
  auto store_v = [&](auto stage) {
#pragma unroll
    for (int k = 0; k < NU; ++k) {
      const int u = tid + kThreads * k;
      uint4 x, y;
      widen16(tv[k], &x, &y);
      char* to = smem_v + ((u >> 2) * kVPitch + (u & 3) * 32) + stage * kVBytes;
      *reinterpret_cast<uint4*>(to) = x;
      *reinterpret_cast<uint4*>(to + 16) = y;
    }
  };

  v16f_t acc[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;
  float m_run = kNegInf, l_run = 0.0f;  // l_run: of this lane's tokens
  const int last = a.causal ? min(pos, sq.len - 1) : sq.len - 1;
  const int all_end = a.causal ? min(pos_lo, sq.len - 1) : sq.len - 1;
  const int all_begin = a.window > 0 ? pos_hi - a.window + 1 : 0;
  // row of S^T nn is token nn with bits 2 and 3 swapped
  const char* k_from = smem_k + ((nn & 0x13) | (nn & 4) << 1 | (nn & 8) >> 1) * kKPitch + hf * 16;
  const char* v_from = smem_v + nn * kVPitch + hf * 16;

  constexpr std::integral_constant<int, 0> kEven;
  constexpr std::integral_constant<int, 1> kOdd;
  const v16f_t zero = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  auto scores = [&](v16f_t (&s)[2], auto stage) {
#pragma unroll
    for (int st = 0; st < NQ; ++st)
#pragma unroll
      for (int sb = 0; sb < 2; ++sb)
        s[sb] = mfma(*reinterpret_cast<const uint4*>(k_from + (stage * kKBytes + sb * 32 * kKPitch + st * 32)), q[st],
                     st == 0 ? zero : s[sb]);
  };
  Numbers kn, gn;
  Scales sc, sc1;
  auto tile = [&](int i, auto here, auto there) {
    __syncthreads();
    v16f_t s[2];
    scores(s, here);
    // the next tile's codes to the other half of LDS, and those of the one after it on their way
    store_k(there);
    store_v(there);
    load_k(i + 2, kn);
    load_v(i + 2, gn);
    const Scales sc2 = scales_of(gn);
    kn = k_numbers(i + 3);
    gn = g_numbers(i + 3);
    const int base = base_of(i);
    // a lane's values 8 k .. 8 k + 7 are tokens 16 k + 8 hf .. of the tile
    float f[4], lv[4], rv[4];
    bool gone = false;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int x = ONE ? 0 : k;
      const float v = (sc.av[x] < kMinMag ? kMinMag : sc.av[x]) * (1.0f / 127.0f);
      f[k] = unit * sc.ak[x];
      lv[k] = __builtin_amdgcn_logf(v);  // log2
      rv[k] = __builtin_amdgcn_rcpf(v);
      gone |= sc.gone[x];
    }
    if (base + 63 > all_end || base < all_begin || gone) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        bool any = false;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int x = base + 16 * k + 8 * hf + j;
          const bool see = !sc.gone[ONE ? 0 : k] && x <= last && (a.window <= 0 || x > pos - a.window || x < a.sinks);
          const float u = __builtin_fmaf(s[k >> 1][(k & 1) * 8 + j], f[k], lv[k]);
          s[k >> 1][(k & 1) * 8 + j] = see ? u : kNegInf;
          any |= see;
        }
        f[k] = 1.0f;
        lv[k] = 0.0f;
        rv[k] = any ? rv[k] : 0.0f;  // a page that the row does not see may have any magnitude
      }
    }
    float mt = kNegInf;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float x = s[k >> 1][(k & 1) * 8];
#pragma unroll
      for (int j = 1; j < 8; ++j) x = fmaxf(x, s[k >> 1][(k & 1) * 8 + j]);
      mt = fmaxf(mt, __builtin_fmaf(x, f[k], lv[k]));  // f >= 0
    }
    mt = pair_max(mt);
    if (__any(mt > m_run + 7.0f)) {  // a row has outgrown its maximum: what was summed moves to the new one
      const float m_new = fmaxf(m_run, mt);
      const float alpha = m_run == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m_run - m_new);
      m_run = m_new;
      l_run *= alpha;
#pragma unroll
      for (int d = 0; d < ND; ++d) acc[d] *= alpha;
    }
    const float ref = m_run == kNegInf ? 0.0f : m_run - 8.0f;
    uint4 p[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float w[8], sum = 0.0f;
      const float off = lv[k] - ref;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        w[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[k >> 1][(k & 1) * 8 + j], f[k], off));
        sum += w[j];
      }
      l_run = __builtin_fmaf(sum, rv[k], l_run);
      p[k] = make_uint4(Act16<false>::pack2(w[0], w[1]), Act16<false>::pack2(w[2], w[3]),
                        Act16<false>::pack2(w[4], w[5]), Act16<false>::pack2(w[6], w[7]));
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int d = 0; d < ND; ++d)
        acc[d] = mfma(*reinterpret_cast<const uint4*>(v_from + (here * kVBytes + d * 32 * kVPitch + k * 32)), p[k], acc[d]);
    sc = sc1;
    sc1 = sc2;
  };
  if (tiles > 0) {
    const Numbers k0 = k_numbers(0), g0 = g_numbers(0), k1 = k_numbers(1), g1 = g_numbers(1);
    load_k(0, k0);
    load_v(0, g0);
    sc = scales_of(g0);
    store_k(kEven);
    store_v(kEven);
    load_k(1, k1);
    load_v(1, g1);
    sc1 = scales_of(g1);
    kn = k_numbers(2);
    gn = g_numbers(2);
    for (int i = 0; i < tiles; i += 2) {
      tile(i, kEven, kOdd);
      if (i + 1 < tiles) tile(i + 1, kOdd, kEven);
    }
  }

  l_run = pair_sum(l_run);
  const int mine = wave * 32 + nn;
  if (row0 + mine >= rows) return;
  const int64_t row = qrow * a.q_heads + qh;
  if (a.splits > 1) {  // to be joined; weights are 2^8 times what the maximum stands for
    const int slot = (item * H + h) * a.splits + part;
    const int64_t to = (int64_t)slot * kRows + mine;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = d * 32 + 8 * k + 4 * hf;
        if (FULL || c < D)
          *reinterpret_cast<v4f*>(a.part_o + to * D + c) = v4f{acc[d][4 * k], acc[d][4 * k + 1], acc[d][4 * k + 2], acc[d][4 * k + 3]};
      }
    if (hf == 0) {
      *reinterpret_cast<v2f*>(a.part_ml + to * 2) = v2f{m_run - 8.0f, l_run};
      if (part == 0) *reinterpret_cast<v2i*>(a.notes + row * 2) = v2i{slot << kKvNoteShift | mine, a.splits};
    }
    return;
  }
  const float inv = l_run == 0.0f ? 0.0f : 1.0f / l_run;
  uint16_t* op = a.o.p + qrow * a.o.token + (int64_t)qh * a.o.head;
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = d * 32 + 8 * k + 4 * hf;
      if (!FULL && c >= D) continue;
      const float x0 = acc[d][4 * k] * inv, x1 = acc[d][4 * k + 1] * inv, x2 = acc[d][4 * k + 2] * inv,
                  x3 = acc[d][4 * k + 3] * inv;
      *reinterpret_cast<uint2*>(op + c) = a.bf16 ? make_uint2(Act16<true>::pack2(x0, x1), Act16<true>::pack2(x2, x3))
                                                 : make_uint2(Act16<false>::pack2(x0, x1), Act16<false>::pack2(x2, x3));
    }
  if (a.lse && hf == 0) a.lse[row] = l_run == 0.0f ? kNegInf : (m_run - 8.0f + log2f(l_run)) * 0.693147180559945309f;
}

// Wavefronts of a workgroup: four, two workgroups to a CU. Heads of 65 to 128
// channels on pages smaller than a tile need more registers for the addresses of
// a tile's codes, and eight wavefronts to share them out (three prompts of 4000
// tokens on pages of 32: 515 us, 555 with four; on pages of 64 four take 352, eight
// 358).
static int prompt_waves(int dim, int page_shift) { return page_shift < 6 && dim > 64 && dim <= 128 ? 8 : 4; }

static int64_t prompt_items(const KvBatch& s, int G, int waves) { return (int64_t)s.T * G / (32 * waves) + s.B; }

// Parts that the tokens are cut into where the call has too few rows to fill the
// chip: as many as fill it, of eight tiles at least. Measured (32 query and 8
// key/value heads of 128, us cut / uncut): 64 rows at the end of 4000 tokens 27 /
// 86, 256 of 16000 86 / 321, 600 of 4000 64 / 89, 1000 of 16000 288 / 325; about
// even where a sequence's rows and tokens are near in number (2 of 330 rows and
// 4000 tokens 89 / 89, of 500 and 3000 77 / 71). Sets the rows of a part's result
// and how many parts there are in all.
int kv_prompt_splits(const KvBatch& s, int heads, int q_heads, int dim, int page_shift, int64_t max_span,
                     int num_cus, int* run, int* max_parts) {
  const int G = q_heads / heads, waves = prompt_waves(dim, page_shift);
  const int64_t rows = 32 * waves;
  const int64_t works = std::max<int64_t>(s.B, ((int64_t)s.T * G + rows - 1) / rows) * heads;
  const int64_t slots = (int64_t)num_cus * (waves == 8 || dim > 128 ? 1 : dim <= 64 ? 3 : 2);
  const int64_t n = std::min<int64_t>(slots / works, (max_span + 511) / 512);
  *run = (int)rows;
  *max_parts = n > 1 ? (int)(prompt_items(s, G, waves) * heads * n) : 0;
  return (int)std::max<int64_t>(1, n);
}

template <int DP, bool FULL, bool ONE, int W>
static hipError_t launch_prompt(const KvAttnArgs& a, hipStream_t stream) {
  const int64_t blocks = prompt_items(a.s, a.q_heads / a.c.heads, W) * a.c.heads * a.splits;
  if (blocks > INT32_MAX) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((kv_prompt<DP, FULL, ONE, W>), dim3((unsigned)blocks), dim3(64 * W), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_kv_prompt(const KvAttnArgs& a, hipStream_t stream) {
  const bool one = a.c.page_shift >= 6;
  if (a.c.dim == 64)
    return one ? launch_prompt<64, true, true, 4>(a, stream) : launch_prompt<64, true, false, 4>(a, stream);
  if (a.c.dim < 64)
    return one ? launch_prompt<64, false, true, 4>(a, stream) : launch_prompt<64, false, false, 4>(a, stream);
  if (a.c.dim == 128)
    return one ? launch_prompt<128, true, true, 4>(a, stream) : launch_prompt<128, true, false, 8>(a, stream);
  if (a.c.dim < 128)
    return one ? launch_prompt<128, false, true, 4>(a, stream) : launch_prompt<128, false, false, 8>(a, stream);
  return one ? launch_prompt<256, false, true, 4>(a, stream) : launch_prompt<256, false, false, 4>(a, stream);
}

}  // namespace llmint8
