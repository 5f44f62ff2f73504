// Attention over the int8 key/value cache on gfx950.
//
//   s_j = scale * q . k_j over the tokens j that the row sees,
//   o   = sum_j softmax(s)_j v_j,     lse = log sum_j exp(s_j)
// with k_j = K codes * aK / 127 and v_j = V codes * aV / 127 of the token's page
// and head, the codes read as they are stored.
//
// kv_step: both products run on v_mfma_i32_16x16x64_i8, so that no code is ever
// converted: a tile is 64 tokens against 16 query rows (the heads of a group,
// times the call's tokens of the sequence), a wavefront to a tile.
//   S^T = K . q^T   A = 16 tokens x 64 channels of codes, as loaded; B = q, held
//                   as 16-bit integers in two int8 planes (q = qi * max|q| /
//                   32639, qi = 256 hi + lo): the error of a channel is 2^-16 of
//                   the row's largest, below the inputs' own rounding, and the
//                   sums are exact (dim * 127 * 32639 < 2^31).
//   O^T = V^T . P^T A = 16 channels x 64 tokens of codes, as loaded; B = the
//                   weights exp2(u - tile max) as 16-bit integers in two planes.
// The tokens of a tile are assigned to the rows of S^T so that the weights a lane
// gets out of the first product (token 16 g + 4 t + i of query row n, lane 16 g +
// n) are the operand it needs for the second one: nothing moves between lanes.
// The scale of V's page goes into the exponent: u = s log2(e) + log2(aV / 127),
// so pages of any scale share a tile, and the row's sum takes each weight
// without it.
#include <math.h>

#include "kv_common.h"

namespace llmint8 {

namespace {

constexpr float kMinMag = 5.42101086242752217e-20f;  // 2^-64: the least magnitude of a page that is not zero
constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ v4i mfma_i8(const v4i& a, const v4i& b, const v4i& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ v4i load16(const int8_t* p) { return *reinterpret_cast<const v4i*>(p); }

// over the four lanes that hold one query row (lanes n, n + 16, n + 32, n + 48)
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, __shfl_xor(v, 16, 64));
  return fmaxf(v, __shfl_xor(v, 32, 64));
}
__device__ __forceinline__ float row_sum(float v) {
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

// The tiles of 64 tokens that a run of rows at positions [pos_lo, pos_hi] sees:
// the first `sink` ones, then [lo, hi).
struct Span {
  int sink, lo, hi;
  __device__ __forceinline__ int count() const { return sink + max(hi - lo, 0); }
  __device__ __forceinline__ int tile(int i) const { return i < sink ? i : lo + (i - sink); }
};

__device__ __forceinline__ Span visible_span(int len, int pos_lo, int pos_hi, int causal, int window, int sinks) {
  Span s;
  const int end = causal ? min(len, pos_hi + 1) : len;
  s.hi = end > 0 ? (end + 63) >> 6 : 0;
  s.lo = window > 0 ? max(pos_lo - window + 1, 0) >> 6 : 0;
  s.lo = min(s.lo, s.hi);
  s.sink = window > 0 ? min((int)(((int64_t)sinks + 63) >> 6), s.lo) : 0;
  return s;
}

}  // namespace

template <int DP, bool BF16>
__global__ __launch_bounds__(256) void kv_step(KvAttnArgs a) {
  constexpr int NK = DP / 64;  // 64-channel steps of the first product
  constexpr int ND = DP / 16;  // 16-channel blocks of the second
  __shared__ float sh_o[2][16][DP];
  __shared__ float sh_ml[4][16][2];
  const int P = 1 << a.c.page_shift, D = a.c.dim, H = a.c.heads, G = a.q_heads / H;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int g = lane >> 4, nn = lane & 15;
  int first;
  const int b = kv_find<256>(a.s, blockIdx.x, G, 4, 1, &first);
  if (b < 0) return;
  const KvSeq sq = kv_seq(a.s, a.c.page_shift, b);
  const int h = blockIdx.y;
  const int row_tile = (int)blockIdx.x - first;
  const int rows = sq.n * G;
  if (row_tile * 16 >= rows) return;
  const int r = row_tile * 16 + nn;
  const bool live = r < rows;
  const int tok = min(r, rows - 1) / G, head = min(r, rows - 1) - tok * G;
  const int pos = sq.len - sq.n + tok;
  const int64_t qrow = sq.row0 + tok;
  const int qh = h * G + head;

  // q: 16-bit integers in two planes, and what one unit of S stands for
  v4i qhi[NK], qlo[NK];
  float unit;
  {
    const uint16_t* qp = a.q.p + qrow * a.q.token + (int64_t)qh * a.q.head;
    float f[NK][16], m = 0.0f;
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) {
      const int c0 = ks * 64 + g * 16;
      uint4 w[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
      if (c0 < D) {
        w[0] = *reinterpret_cast<const uint4*>(qp + c0);
        w[1] = *reinterpret_cast<const uint4*>(qp + c0 + 8);
      }
      const uint32_t* u = &w[0].x;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        f[ks][j] = Act16<BF16>::to_f32((u[j >> 1] >> (16 * (j & 1))) & 0xffffu);
        m = fmaxf(m, fabsf(f[ks][j]));
      }
    }
    m = row_max(m);
    const float sc = m > 0.0f ? 32639.0f / m : 0.0f;
    unit = m * (1.0f / 32639.0f) * a.scale * 1.44269504088896341f * (1.0f / 127.0f);
#pragma unroll
    for (int ks = 0; ks < NK; ++ks) {
      uint32_t hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int v = (int)rintf(f[ks][j] * sc);
        const int vh = (v + 128) >> 8;
        hi[j >> 2] |= (uint32_t)(vh & 0xff) << (8 * (j & 3));
        lo[j >> 2] |= (uint32_t)((v - (vh << 8)) & 0xff) << (8 * (j & 3));
      }
      qhi[ks] = v4i{(int)hi[0], (int)hi[1], (int)hi[2], (int)hi[3]};
      qlo[ks] = v4i{(int)lo[0], (int)lo[1], (int)lo[2], (int)lo[3]};
    }
  }

  // this part's share of the tiles that any row of the run sees
  const int pos_lo = sq.len - sq.n + row_tile * 16 / G;
  const int pos_hi = sq.len - sq.n + (min(row_tile * 16 + 15, rows - 1)) / G;
  const Span span = visible_span(sq.len, pos_lo, pos_hi, a.causal, a.window, a.sinks);
  const int total = span.count();
  const int share = max(a.split_tiles, (total + a.splits - 1) / a.splits);
  const int i0 = min((int)blockIdx.z * share, total), i1 = min(i0 + share, total);

  v4f acc[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) acc[d] = v4f{0, 0, 0, 0};
  float m_run = kNegInf, l_run = 0.0f;
  const int64_t page_bytes = (int64_t)P * D;
  for (int it = i0 + wave; it < i1; it += 4) {
    const int base = span.tile(it) << 6;
    // pages of the token rows that this lane loads and of the tokens that it holds
    const int tk = base + 16 * (nn >> 2), tv = base + 16 * g;
    const int pk = kv_page(a.s, b, tk >> a.c.page_shift, a.c.pages);
    const int pv = kv_page(a.s, b, tv >> a.c.page_shift, a.c.pages);
    const int8_t* kp = a.c.K + ((int64_t)max(pk, 0) * H + h) * page_bytes +
                       ((tk & (P - 1)) + (nn & 3)) * D;
    const int64_t hv = (int64_t)max(pv, 0) * H + h;
    const int8_t* vp = a.c.V + hv * page_bytes + (tv & (P - 1));
    v4i kf[4][NK], vf[ND];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int ks = 0; ks < NK; ++ks) {
        const int c0 = ks * 64 + g * 16;
        kf[t][ks] = load16(kp + 4 * t * D + (c0 < D ? c0 : 0));
      }
#pragma unroll
    for (int d = 0; d < ND; ++d) vf[d] = load16(vp + (int64_t)min(d * 16 + nn, D - 1) * P);
    const float ak = a.c.aK[hv], av = a.c.aV[hv];

    // S in units of q's and the page's scales
    float u[16];
    const float fk = unit * ak;
    // a page of zeros takes the smallest scale there is: its weights only enter the row's sum, and
    // must not set the scale of the others'
    const float vs = (av > kMinMag ? av : kMinMag) * (1.0f / 127.0f);
    const float lv = __builtin_amdgcn_logf(vs);  // log2
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      v4i s = {0, 0, 0, 0};
#pragma unroll
      for (int ks = 0; ks < NK; ++ks) s = mfma_i8(kf[t][ks], qhi[ks], s);
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] <<= 8;
#pragma unroll
      for (int ks = 0; ks < NK; ++ks) s = mfma_i8(kf[t][ks], qlo[ks], s);
#pragma unroll
      for (int i = 0; i < 4; ++i) u[4 * t + i] = __builtin_fmaf((float)s[i], fk, lv);
    }
    // what the row does not see
    const int last = a.causal ? min(pos, sq.len - 1) : sq.len - 1;  // < 0: nothing
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const int t = tv + j;
      const bool see = pv >= 0 && t <= last && (a.window <= 0 || t > pos - a.window || t < a.sinks);
      u[j] = see ? u[j] : kNegInf;
    }
    float mt = u[0];
#pragma unroll
    for (int j = 1; j < 16; ++j) mt = fmaxf(mt, u[j]);
    mt = row_max(mt);
    const float mt0 = mt == kNegInf ? 0.0f : mt;
    const float m_new = fmaxf(m_run, mt);
    const float m0 = m_new == kNegInf ? 0.0f : m_new;
    const float alpha = __builtin_amdgcn_exp2f(m_run - m0), beta = __builtin_amdgcn_exp2f(mt - m0);
    m_run = m_new;
    float sum = 0.0f;
    uint32_t w[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float e = __builtin_amdgcn_exp2f(u[j] - mt0);
      sum += e;
      // rne(32639 e) + 128 in the low 16 bits: high plane, and low plane + 128
      w[j] = __builtin_bit_cast(uint32_t, __builtin_fmaf(e, 32639.0f, 12582912.0f + 128.0f));
    }
    l_run = l_run * alpha + sum * beta * __builtin_amdgcn_rcpf(vs);
    v4i phi, plo;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t h01 = __builtin_amdgcn_perm(w[4 * t + 1], w[4 * t], 0x0c0c0501u);
      const uint32_t h23 = __builtin_amdgcn_perm(w[4 * t + 3], w[4 * t + 2], 0x0c0c0501u);
      const uint32_t l01 = __builtin_amdgcn_perm(w[4 * t + 1], w[4 * t], 0x0c0c0400u);
      const uint32_t l23 = __builtin_amdgcn_perm(w[4 * t + 3], w[4 * t + 2], 0x0c0c0400u);
      phi[t] = (int)__builtin_amdgcn_perm(h23, h01, 0x05040100u);
      plo[t] = (int)(__builtin_amdgcn_perm(l23, l01, 0x05040100u) ^ 0x80808080u);
    }
    const float bu = beta * (1.0f / 32639.0f);
#pragma unroll
    for (int d = 0; d < ND; ++d) {
      v4i o = mfma_i8(vf[d], phi, v4i{0, 0, 0, 0});
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] <<= 8;
      o = mfma_i8(vf[d], plo, o);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[d][i] = __builtin_fmaf((float)o[i], bu, acc[d][i] * alpha);
    }
  }

  // join the four wavefronts
  l_run = row_sum(l_run);
  if (g == 0) {
    sh_ml[wave][nn][0] = m_run;
    sh_ml[wave][nn][1] = l_run;
  }
  __syncthreads();
  float m_all = sh_ml[0][nn][0];
#pragma unroll
  for (int w = 1; w < 4; ++w) m_all = fmaxf(m_all, sh_ml[w][nn][0]);
  const float m0 = m_all == kNegInf ? 0.0f : m_all;
  float l_all = 0.0f;
#pragma unroll
  for (int w = 0; w < 4; ++w) l_all += sh_ml[w][nn][1] * __builtin_amdgcn_exp2f(sh_ml[w][nn][0] - m0);
  const float mine = __builtin_amdgcn_exp2f(m_run - m0);
#pragma unroll
  for (int d = 0; d < ND; ++d) acc[d] *= mine;
#pragma unroll
  for (int half = 2; half > 0; half >>= 1) {
    if (wave >= half && wave < 2 * half)
#pragma unroll
      for (int d = 0; d < ND; ++d) *reinterpret_cast<v4f*>(&sh_o[wave - half][nn][d * 16 + 4 * g]) = acc[d];
    __syncthreads();
    if (wave < half)
#pragma unroll
      for (int d = 0; d < ND; ++d) acc[d] += *reinterpret_cast<const v4f*>(&sh_o[wave][nn][d * 16 + 4 * g]);
    __syncthreads();
  }
  if (wave != 0 || !live) return;
  const int64_t row = qrow * a.q_heads + qh;
  if (a.splits > 1) {
    const int64_t at = (int64_t)blockIdx.z * ((int64_t)a.s.T * a.q_heads) + row;
#pragma unroll
    for (int d = 0; d < ND; ++d)
      if (d * 16 < D) *reinterpret_cast<v4f*>(a.part_o + at * D + d * 16 + 4 * g) = acc[d];
    if (g == 0) {
      a.part_ml[at * 2] = m_all;
      a.part_ml[at * 2 + 1] = l_all;
    }
    return;
  }
  const float inv = l_all > 0.0f ? 1.0f / l_all : 0.0f;
  uint16_t* op = a.o.p + qrow * a.o.token + (int64_t)qh * a.o.head;
#pragma unroll
  for (int d = 0; d < ND; ++d)
    if (d * 16 < D)
      *reinterpret_cast<uint2*>(op + d * 16 + 4 * g) = make_uint2(Act16<BF16>::pack2(acc[d][0] * inv, acc[d][1] * inv),
                                                                 Act16<BF16>::pack2(acc[d][2] * inv, acc[d][3] * inv));
  if (a.lse && g == 0) a.lse[row] = l_all > 0.0f ? (m_all + log2f(l_all)) * 0.693147180559945309f : kNegInf;
}

// Joins the parts of a row: a wavefront to a row.
template <bool BF16>
__global__ __launch_bounds__(256) void kv_join(KvAttnArgs a) {
  const int64_t rows = (int64_t)a.s.T * a.q_heads;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (row >= rows) return;
  const int t = (int)(row / a.q_heads);
  const int last = min(max(a.s.cu[a.s.B], 0), a.s.T);
  if (t >= last) return;  // rows past the batch are not written
  float m = kNegInf;
  for (int s = 0; s < a.splits; ++s) m = fmaxf(m, a.part_ml[(s * rows + row) * 2]);
  const float m0 = m == kNegInf ? 0.0f : m;
  const int D = a.c.dim;
  float l = 0.0f;
  v4f o = {0, 0, 0, 0};
  for (int s = 0; s < a.splits; ++s) {
    const float w = __builtin_amdgcn_exp2f(a.part_ml[(s * rows + row) * 2] - m0);
    if (w == 0.0f) continue;
    l += w * a.part_ml[(s * rows + row) * 2 + 1];
    if (lane * 4 < D) {
      const v4f p = *reinterpret_cast<const v4f*>(a.part_o + (s * rows + row) * D + lane * 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] += w * p[i];
    }
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  const int h = (int)(row - (int64_t)t * a.q_heads);
  if (lane * 4 < D)
    *reinterpret_cast<uint2*>(a.o.p + t * a.o.token + h * a.o.head + lane * 4) =
        make_uint2(Act16<BF16>::pack2(o[0] * inv, o[1] * inv), Act16<BF16>::pack2(o[2] * inv, o[3] * inv));
  if (a.lse && lane == 0) a.lse[row] = l > 0.0f ? (m + log2f(l)) * 0.693147180559945309f : kNegInf;
}

int kv_attention_splits(const KvBatch& s, int heads, int q_heads, int64_t max_span, int num_cus,
                        int* split_tiles) {
  const int64_t items = (((int64_t)s.T * (q_heads / heads)) >> 4) + s.B;
  const int64_t tiles = (max_span + 63) / 64;
  // enough parts for 8 workgroups a CU, none under 4 tiles (one for each wavefront)
  int64_t n = (8 * num_cus) / (items * heads);
  n = std::max<int64_t>(1, std::min<int64_t>(n, (tiles + 3) / 4));
  n = std::min<int64_t>(n, 256);
  *split_tiles = (int)std::max<int64_t>(1, (tiles + n - 1) / n);
  return (int)n;
}

hipError_t launch_kv_attention(const KvAttnArgs& a, bool bf16, hipStream_t stream) {
  const int G = a.q_heads / a.c.heads;
  const dim3 grid((unsigned)((((int64_t)a.s.T * G) >> 4) + a.s.B), a.c.heads, a.splits);
#define STEP(DP)                                                                     \
  do {                                                                               \
    if (bf16)                                                                        \
      hipLaunchKernelGGL((kv_step<DP, true>), grid, dim3(256), 0, stream, a);        \
    else                                                                             \
      hipLaunchKernelGGL((kv_step<DP, false>), grid, dim3(256), 0, stream, a);       \
  } while (0)
  if (a.c.dim <= 64)
    STEP(64);
  else if (a.c.dim <= 128)
    STEP(128);
  else
    STEP(256);
#undef STEP
  if (a.splits > 1) {
    const unsigned blocks = (unsigned)(((int64_t)a.s.T * a.q_heads + 3) / 4);
    if (bf16)
      hipLaunchKernelGGL(kv_join<true>, dim3(blocks), dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL(kv_join<false>, dim3(blocks), dim3(256), 0, stream, a);
  }
  return hipGetLastError();
}

}  // namespace llmint8
