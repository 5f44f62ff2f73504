// Attention over packed sequences on gfx950, forward: o = softmax(scale q k^T) v of
// each sequence's rows over its own tokens, with grouped heads, causal masks,
// sliding windows and sinks, or none.
//
// A workgroup takes 128 rows of a sequence and key/value head (tokens times the
// group's query heads, so that a tile of k and v serves all of them), 32 to a
// wavefront, and goes over the tokens in tiles of 64, the next one on its way to
// the other half of LDS while one is computed:
//   S^T = K . q^T    A = 32 tokens x 16 channels from LDS, B = q in registers
//   O^T = V^T . P^T  A = 32 channels x 16 tokens from LDS, transposed by the read,
//                    B = the weights, in the lane that computed them
// Softmax over the tiles with a running maximum m, left where it is until a tile
// exceeds it by 2^7: w = exp2(u - m + 8) is at most 2^15, so that in fp16 weights
// down to 2^-32 of the largest count. Statistics and sums are fp32, a weight is
// rounded to the inputs' type (2^-11 or 2^-8 of itself at most) for the product.
//
// Bound by the SIMDs' issue: matrix instructions and the softmax's vector instructions run
// side by side only from different wavefronts, so two to four share a SIMD. 18000 tokens of
// 32/8 heads of 128: 880 us, 1010 TFLOP/s (a large product reaches 1531; the counters of 15000
// tokens have the matrix cores busy in 43% of the cycles, LDS in 22%, without a conflict).
// Without exponentials, maximum or sums it takes 3 to 6% less each, with all copies from one
// tile 1%: none of them alone is what it waits for.
#include <type_traits>

#include "attn_common.h"

namespace llmint8 {

template <int DP, bool BF16>
__global__ __launch_bounds__(256, DP <= 64 ? 4 : DP <= 128 ? 2 : 1) void ka_attention(AttnArgs a) {
  using Tile = AttnTile<DP>;
  constexpr int W = 4, kRows = 32 * W, NQ = Tile::NQ, ND = Tile::ND;
  constexpr int kStage = 2 * Tile::kBytes;  // k, v
  __shared__ __attribute__((aligned(1024))) char smem[2 * kStage + 16];
  int* const flag = reinterpret_cast<int*>(smem + 2 * kStage);
  const int D = a.dim, H = a.heads, G = a.q_heads / H;
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
  const int hf = lane >> 5, nn = lane & 31;
  const int h = (int)(blockIdx.x % H), item = (int)(blockIdx.x / H);
  AttnSeq sq;
  int run;
  if (!attn_place<true>(a, item, G, 7, &sq, &run)) return;
  const int64_t rows = (int64_t)sq.n * G, row0 = (int64_t)run * kRows;
  // the token and head of a lane's row
  auto place = [&](int n, int* pos, int* qh) {
    const int r = (int)min(row0 + wave * 32 + n, rows - 1);
    *pos = r / G;
    *qh = h * G + (r - *pos * G);
  };
  int pos, qh;
  place(nn, &pos, &qh);
  auto span_of = [&](int64_t from, int64_t to) {  // of rows [from, to)
    return AttnSpan(a, (int)(min(from, rows) / G), (int)((min(to, rows) - 1) / G), sq.n);
  };
  const AttnSpan all = span_of(row0, row0 + kRows);
  const bool idle = row0 + wave * 32 >= rows;  // this wavefront has no row
  const AttnSpan own = span_of(row0 + wave * 32, row0 + wave * 32 + 32);

  // tiles that any of the rows sees
  const int hi = (all.last >> 6) + 1, lo = min(max(all.begin, 0) >> 6, hi);
  const int sink = min((int)(((int64_t)a.sinks + 63) >> 6), lo);
  const int tiles = sink + hi - lo;
  auto base_of = [&](int i) { return (i < sink ? i : lo + i - sink) << 6; };

  const uint16_t* kp = a.k.p + (int64_t)sq.row0 * a.k.token + (int64_t)h * a.k.head;
  const uint16_t* vp = a.v.p + (int64_t)sq.row0 * a.v.token + (int64_t)h * a.v.head;
  const int start = base_of(0), past = (lo - sink + 1) * 64;  // past: from the last tile of the sinks to the next
  AttnStream<DP, W> ck(kp, a.k.token, D, start, past * a.k.token), cv(vp, a.v.token, D, start, past * a.v.token);
  auto copy = [&](int i, int stage) {
    const int n = i < tiles ? min(sq.n - base_of(i), 64) : 0;  // past the last tile: zeros, to keep the loop free of branches
    ck.next(n, smem + stage * kStage, i + 1 == sink);
    cv.next(n, smem + stage * kStage + Tile::kBytes, i + 1 == sink);
  };
  copy(0, 0);
  if (threadIdx.x == 0) *flag = 0;
  attn_barrier();

  uint4 q[NQ];
  {
    const uint16_t* qp = a.q.p + (int64_t)(sq.row0 + pos) * a.q.token + (int64_t)qh * a.q.head;
    const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
    for (int ks = 0; ks < NQ; ++ks) {
      const int c0 = ks * 16 + hf * 8;
      q[ks] = make_uint4(0, 0, 0, 0);
      if (c0 < D) {
        q[ks] = *reinterpret_cast<const uint4*>(qp + c0);
        q[ks] = make_uint4(q[ks].x ^ flip, q[ks].y ^ flip, q[ks].z ^ flip, q[ks].w ^ flip);
      }
    }
  }
  // u = s f; never zero, so that a masked logit stays -infinity
  const float f = fmaxf(fabsf(a.scale) * 1.44269504088896341f, 1e-37f);

  v16f_t acc[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) acc[d] = attn_zero();
  float m_run = kAttnNegInf, l_run = 0.0f;  // l_run: of this lane's tokens
  AttnRead<DP> rd(smem);
  const AttnSees sees(a, pos, sq.n);

  for (int i = 0; i < tiles; ++i) {
    const int stage = i & 1, base = base_of(i);
    const bool masked = all.masked(base);
    attn_wait_copies();
    if (masked) cv.template finite<BF16>(smem + stage * kStage + Tile::kBytes, flag);
    attn_barrier();
    copy(i + 1, stage ^ 1);

    if (!(idle | own.none(base, 64))) {
      // operands are read two steps ahead of their products
      uint4 x[3][2];
#pragma unroll
      for (int st = 0; st < 2; ++st)
#pragma unroll
        for (int sb = 0; sb < 2; ++sb) x[st][sb] = rd.rows(0, sb, st);
      v16f_t s[2];
#pragma unroll
      for (int st = 0; st < NQ; ++st) {
#pragma unroll
        for (int sb = 0; sb < 2; ++sb) {
          if (st + 2 < NQ) x[(st + 2) % 3][sb] = rd.rows(0, sb, st + 2);
          s[sb] = Act16<BF16>::mma32(x[st % 3][sb], q[st], st == 0 ? attn_zero() : s[sb]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      uint4 y[2][ND];
#pragma unroll
      for (int d = 0; d < ND; ++d) y[0][d] = rd.channels(1, d, 0);
      // a lane's values 8 k .. 8 k + 7 are tokens 16 k + 8 hf .. of the tile
      if (own.masked(base)) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (!sees(base + 16 * k + 8 * hf + j)) s[k >> 1][(k & 1) * 8 + j] = kAttnNegInf;
      }
      float mt = s[0][0];
#pragma unroll
      for (int j = 0; j < 16; ++j) mt = attn_max(mt, s[0][j], s[1][j]);
      mt = attn_pair_max(mt) * f;
      // a row that has outgrown its maximum: what was summed moves to the new one (its own row
      // decides, so that results do not depend on the rows beside it)
      if (__any(mt > m_run + 7.0f)) {
        const float m_new = mt > m_run + 7.0f ? mt : m_run;
        const float alpha = m_run == kAttnNegInf ? 0.0f : __builtin_amdgcn_exp2f(m_run - m_new);
        m_run = m_new;
        l_run *= alpha;
#pragma unroll
        for (int d = 0; d < ND; ++d) acc[d] *= alpha;
      }
      const float off = m_run == kAttnNegInf ? 0.0f : 8.0f - m_run;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (k < 3) {
#pragma unroll
          for (int d = 0; d < ND; ++d) y[(k + 1) & 1][d] = rd.channels(1, d, k + 1);
        }
        float w[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          w[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[k >> 1][(k & 1) * 8 + j], f, off));
          l_run += w[j];
        }
        const uint4 p = make_uint4(Act16<BF16>::pack2(w[0], w[1]), Act16<BF16>::pack2(w[2], w[3]),
                                   Act16<BF16>::pack2(w[4], w[5]), Act16<BF16>::pack2(w[6], w[7]));
#pragma unroll
        for (int d = 0; d < ND; ++d) acc[d] = Act16<BF16>::mma32(y[k & 1][d], p, acc[d]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    rd.next(stage ? -kStage : kStage);
  }
  attn_wait_copies();
  if (__builtin_expect(uniform(*flag), 0)) {
#pragma unroll 1
    for (int i = 0; i < tiles; ++i) {
      const int base = base_of(i);
      if (all.masked(base))
        attn_others<DP, BF16>(acc, vp, a.v.token, base, sq.n, D, true, [&](int t) { return sees(base + t); });
    }
  }

  l_run = attn_pair_sum(l_run);
  int n = threadIdx.x & 31;
  asm volatile("" : "+v"(n));  // computed again rather than kept in registers (64 channels have 128 of them)
  if (row0 + wave * 32 + n >= rows) return;
  place(n, &pos, &qh);
  const int64_t qrow = (int64_t)sq.row0 + pos;
  const float inv = 1.0f / l_run;  // l_run is zero where all of a row's logits are -infinity: o is NaN, lse -infinity
  uint16_t* op = a.o.p + qrow * a.o.token + (int64_t)qh * a.o.head;
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = d * 32 + 8 * k + 4 * hf;
      if (c >= D) continue;
      *reinterpret_cast<uint2*>(op + c) =
          make_uint2(Act16<BF16>::pack2(acc[d][4 * k] * inv, acc[d][4 * k + 1] * inv),
                     Act16<BF16>::pack2(acc[d][4 * k + 2] * inv, acc[d][4 * k + 3] * inv));
    }
  if (a.lse && hf == 0)
    a.lse[qrow * a.q_heads + qh] = (m_run - 8.0f + log2f(l_run)) * 0.693147180559945309f;
}

template <int DP, bool BF16>
static hipError_t launch_fwd(const AttnArgs& a, hipStream_t stream) {
  const AttnGrid g = attn_row_grid(a.T, a.q_heads, a.heads, a.B);
  if (!g.fits()) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((ka_attention<DP, BF16>), dim3((unsigned)g.blocks), dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_attention(const AttnArgs& a, bool bf16, hipStream_t stream) {
  if (a.dim <= 64) return bf16 ? launch_fwd<64, true>(a, stream) : launch_fwd<64, false>(a, stream);
  if (a.dim <= 96) return bf16 ? launch_fwd<96, true>(a, stream) : launch_fwd<96, false>(a, stream);
  if (a.dim <= 128) return bf16 ? launch_fwd<128, true>(a, stream) : launch_fwd<128, false>(a, stream);
  return bf16 ? launch_fwd<256, true>(a, stream) : launch_fwd<256, false>(a, stream);
}

}  // namespace llmint8
