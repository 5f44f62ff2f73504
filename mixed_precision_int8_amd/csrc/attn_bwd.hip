// The gradients of attention over packed sequences on gfx950. With P the softmax
// weights of the forward pass and delta_i = sum_c do_ic o_ic,
//   dV = P^T do,  dS = P (do V^T - delta),  dq = scale dS K,  dk = scale dS^T q
// (dk and dv summed over the query heads of a group). Two kernels, each of which
// forms S and do V^T anew, so that every sum is one wavefront's, in registers, in
// a fixed order; a single kernel would save two of seven products and add the rows'
// sums of dq in memory, by atomics or in copies.
//   ka_dq   rows of q to lanes, tiles of k and v in LDS, like the forward pass; it
//           also leaves each row's lse and delta for the second
//   ka_dkv  tokens of k and v to lanes, tiles of q and do in LDS, over the heads of
//           the group one after the other
// P and dS are rounded to the inputs' type for their products. fp16 has too small a
// range for dS as it comes: P carries a factor of 2^15, and dS a power of two for
// each column that brings the largest so far to 2^8..2^15, lowered (with the sums)
// when a tile exceeds it. bf16 needs neither.
#include <type_traits>

#include "attn_common.h"

namespace llmint8 {

namespace {

// A column's power of two for dS in fp16.
template <bool BF16, int ND>
struct Reach {
  float g = BF16 ? 1.0f : 8.507059173023462e37f;  // 2^126
  // t: this lane's part of the column
  __device__ __forceinline__ void fit(const v16f_t& t, v16f_t (&acc)[ND]) {
    if constexpr (!BF16) {
      float top = 0.0f;
#pragma unroll
      for (int x = 0; x < 16; ++x) top = fmaxf(top, fabsf(t[x]));
      top = attn_pair_max(top);
      if (__any(top * g > 32768.0f)) {
        if (top * g > 32768.0f) {
          const int e = (int)(__float_as_uint(top) >> 23) - 127;
          const float to = __uint_as_float((uint32_t)(min(8 - e, 126) + 127) << 23);
          const float by = to / g;
#pragma unroll
          for (int d = 0; d < ND; ++d) acc[d] *= by;
          g = to;
        }
      }
    }
  }
};

// values 8 k .. 8 k + 7 as an operand
template <bool BF16>
__device__ __forceinline__ uint4 attn_pack(const v16f_t& t, int k) {
  using A = Act16<BF16>;
  return make_uint4(A::pack2(t[8 * k], t[8 * k + 1]), A::pack2(t[8 * k + 2], t[8 * k + 3]),
                    A::pack2(t[8 * k + 4], t[8 * k + 5]), A::pack2(t[8 * k + 6], t[8 * k + 7]));
}

}  // namespace

template <int DP, bool BF16>
__global__ __launch_bounds__(256, DP <= 128 ? 2 : 1) void ka_dq(AttnArgs a) {
  using Tile = AttnTile<DP>;
  constexpr int W = 4, kRows = 32 * W, NQ = Tile::NQ, ND = Tile::ND;
  __shared__ __attribute__((aligned(1024))) char smem[4 * Tile::kBytes];  // k, v; two stages
  __shared__ int sh[4];
  const int D = a.dim, H = a.heads, G = a.q_heads / H;
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
  const int hf = lane >> 5, nn = lane & 31;
  const int h = (int)(blockIdx.x % H), item = (int)((gridDim.x - 1 - blockIdx.x) / H);
  AttnSeq sq;
  int run;
  if (!attn_find<64 * W>(a, item, G, 7, sh, &sq, &run)) return;
  const int64_t rows = (int64_t)sq.n * G, row0 = (int64_t)run * kRows;
  if (row0 >= rows) return;
  const int r = (int)min(row0 + wave * 32 + nn, rows - 1);
  const int pos = r / G, qh = h * G + (r - pos * G);
  const int64_t qrow = (int64_t)sq.row0 + pos;
  const int pos_lo = (int)row0 / G, pos_hi = (int)(min(row0 + kRows, rows) - 1) / G;

  // tiles that any of the rows sees
  const int end = a.causal ? pos_hi + 1 : sq.n;
  const int hi = (end + 63) >> 6;
  const int lo = a.window > 0 ? min(max(pos_lo - a.window + 1, 0) >> 6, hi) : 0;
  const int sink = a.window > 0 ? min((int)(((int64_t)a.sinks + 63) >> 6), lo) : 0;
  const int tiles = sink + hi - lo;
  auto base_of = [&](int i) { return (i < sink ? i : lo + i - sink) << 6; };

  const AttnCopy<DP, W> ck(a.k.token, D), cv(a.v.token, D);
  const uint16_t* kp = a.k.p + (int64_t)sq.row0 * a.k.token + (int64_t)h * a.k.head;
  const uint16_t* vp = a.v.p + (int64_t)sq.row0 * a.v.token + (int64_t)h * a.v.head;
  auto copy = [&](int i, int stage) {
    ck.issue(kp, a.k.token, base_of(i), sq.n, smem + stage * 2 * Tile::kBytes);
    cv.issue(vp, a.v.token, base_of(i), sq.n, smem + (stage * 2 + 1) * Tile::kBytes);
  };
  copy(0, 0);

  uint4 q[NQ], g[NQ];
  float delta = 0.0f;
  {
    const uint16_t* qp = a.q.p + qrow * a.q.token + (int64_t)qh * a.q.head;
    const uint16_t* gp = a.d_o.p + qrow * a.d_o.token + (int64_t)qh * a.d_o.head;
    const uint16_t* op = a.o.p + qrow * a.o.token + (int64_t)qh * a.o.head;
    const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
    for (int ks = 0; ks < NQ; ++ks) {
      const int c0 = ks * 16 + hf * 8;
      q[ks] = g[ks] = make_uint4(0, 0, 0, 0);
      if (c0 < D) {
        q[ks] = *reinterpret_cast<const uint4*>(qp + c0);
        q[ks] = make_uint4(q[ks].x ^ flip, q[ks].y ^ flip, q[ks].z ^ flip, q[ks].w ^ flip);
        g[ks] = *reinterpret_cast<const uint4*>(gp + c0);
        const uint4 o = *reinterpret_cast<const uint4*>(op + c0);
        const uint32_t x[4] = {g[ks].x, g[ks].y, g[ks].z, g[ks].w}, y[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          delta = __builtin_fmaf(Act16<BF16>::to_f32(x[j] & 0xffffu), Act16<BF16>::to_f32(y[j] & 0xffffu), delta);
          delta = __builtin_fmaf(Act16<BF16>::to_f32(x[j] >> 16), Act16<BF16>::to_f32(y[j] >> 16), delta);
        }
      }
    }
    delta = attn_pair_sum(delta);
  }
  const float f = fabsf(a.scale) * 1.44269504088896341f;
  const float lse2 = a.lse[qrow * a.q_heads + qh] * 1.44269504088896341f;
  const bool mine = row0 + wave * 32 + nn < rows;
  if (mine && hf == 0) {
    float* st = a.stat + (int64_t)qh * a.T + qrow;
    st[0] = lse2;
    st[(int64_t)a.q_heads * a.T] = delta;
  }

  v16f_t acc[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) acc[d] = attn_zero();
  Reach<BF16, ND> reach;
  const int all_end = a.causal ? min(pos_lo, sq.n - 1) : sq.n - 1;
  const int all_begin = a.window > 0 ? pos_hi - a.window + 1 : 0;
  AttnRead<DP> rd(smem);
  const AttnSees sees(a, pos, sq.n);

  for (int i = 0; i < tiles; ++i) {
    const int stage = i & 1, base = base_of(i);
    const bool masked = base + 63 > all_end || base < all_begin;
    attn_wait_copies();
    __syncthreads();
    bool odd = false;
    if (masked) odd = attn_finite<DP, BF16, W>(smem + stage * 2 * Tile::kBytes);
    if (i + 1 < tiles) copy(i + 1, stage ^ 1);
#pragma unroll
    for (int sb = 0; sb < 2; ++sb) {
      v16f_t s = attn_rows_product<DP, BF16>(rd, 0, sb, q);
      v16f_t t = attn_rows_product<DP, BF16>(rd, 1, sb, g);
      uint4 y[2][ND];
#pragma unroll
      for (int d = 0; d < ND; ++d) y[0][d] = rd.channels(0, d, 2 * sb);
#pragma unroll
      for (int x = 0; x < 16; ++x) t[x] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[x], f, -lse2)) * (t[x] - delta);
      if (masked) {
#pragma unroll
        for (int x = 0; x < 16; ++x)
          if (!sees(base + 32 * sb + 16 * (x >> 3) + 8 * hf + (x & 7))) t[x] = 0.0f;
      }
      if constexpr (!BF16) {
        reach.fit(t, acc);
        t *= reach.g;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (k == 0) {
#pragma unroll
          for (int d = 0; d < ND; ++d) y[1][d] = rd.channels(0, d, 2 * sb + 1);
        }
        const uint4 p = attn_pack<BF16>(t, k);
#pragma unroll
        for (int d = 0; d < ND; ++d) acc[d] = Act16<BF16>::mma32(y[k][d], p, acc[d]);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (__builtin_expect(odd, 0))
      attn_others<DP, BF16>(acc, kp, a.k.token, base, sq.n, D, [&](int t) { return sees(base + t); });
    rd.next(stage ? -2 * Tile::kBytes : 2 * Tile::kBytes);
  }

  if (!mine) return;
  const float by = a.scale / reach.g;
  uint16_t* op = a.dq.p + qrow * a.dq.token + (int64_t)qh * a.dq.head;
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = d * 32 + 8 * k + 4 * hf;
      if (c >= D) continue;
      *reinterpret_cast<uint2*>(op + c) =
          make_uint2(Act16<BF16>::pack2(acc[d][4 * k] * by, acc[d][4 * k + 1] * by),
                     Act16<BF16>::pack2(acc[d][4 * k + 2] * by, acc[d][4 * k + 3] * by));
    }
}

// DV, DK: which of the two it forms (heads of more than 128 channels take a launch for
// each, as the registers hold one).
template <int DP, bool BF16, bool DV, bool DK>
__global__ __launch_bounds__(256, 1) void ka_dkv(AttnArgs a) {
  using Tile = AttnTile<DP>;
  constexpr int W = 4, kCols = 32 * W, NQ = Tile::NQ, ND = Tile::ND;
  __shared__ __attribute__((aligned(1024))) char smem[4 * Tile::kBytes];  // q, do; two stages
  __shared__ __attribute__((aligned(256))) float sh_stat[4 * 64];         // lse, delta; two stages
  __shared__ int sh[4];
  const int D = a.dim, H = a.heads, G = a.q_heads / H;
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
  const int hf = lane >> 5, nn = lane & 31;
  // the first tokens of a sequence are seen by the most: they start first
  const int h = (int)(blockIdx.x % H), item = (int)(blockIdx.x / H);
  AttnSeq sq;
  int run;
  if (!attn_find<64 * W>(a, item, 1, 7, sh, &sq, &run)) return;
  const int j0 = run * kCols;
  if (j0 >= sq.n) return;
  const int col = j0 + wave * 32 + nn, j = min(col, sq.n - 1), j_hi = min(j0 + kCols, sq.n) - 1;

  // rows that see any of the tokens
  const int first = a.causal ? j0 : 0;
  int end = sq.n;
  if (a.window > 0 && j0 >= a.sinks) end = (int)min((int64_t)sq.n, (int64_t)j_hi + a.window);
  const int lo = first >> 6, per = ((end + 63) >> 6) - lo, tiles = per * G;

  const AttnCopy<DP, W> cq(a.q.token, D), cg(a.d_o.token, D);
  const uint16_t* qp = a.q.p + (int64_t)sq.row0 * a.q.token + (int64_t)h * G * a.q.head;
  const uint16_t* gp = a.d_o.p + (int64_t)sq.row0 * a.d_o.token + (int64_t)h * G * a.d_o.head;
  const float* sp = a.stat + (int64_t)h * G * a.T + sq.row0;
  auto copy = [&](int head, int base, int stage) {
    cq.issue(qp + (int64_t)head * a.q.head, a.q.token, base, sq.n, smem + stage * 2 * Tile::kBytes);
    cg.issue(gp + (int64_t)head * a.d_o.head, a.d_o.token, base, sq.n, smem + (stage * 2 + 1) * Tile::kBytes);
    if (wave < 2) {
      const float* p = sp + (int64_t)head * a.T + base + (wave ? (int64_t)a.q_heads * a.T : 0);
      attn_copy4(make_rsrc(p, (uint32_t)min(sq.n - base, 64) * 4), sh_stat + (stage * 2 + wave) * 64, (uint32_t)lane * 4);
    }
  };
  int head = 0, at = lo;  // the tile that is copied next
  auto next = [&](int stage) {
    copy(head, at << 6, stage);
    if (++at == lo + per) at = lo, ++head;
  };
  next(0);

  uint4 kr[NQ], vr[NQ];
  {
    const uint16_t* kp = a.k.p + ((int64_t)sq.row0 + j) * a.k.token + (int64_t)h * a.k.head;
    const uint16_t* vp = a.v.p + ((int64_t)sq.row0 + j) * a.v.token + (int64_t)h * a.v.head;
    const uint32_t flip = a.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
    for (int ks = 0; ks < NQ; ++ks) {
      const int c0 = ks * 16 + hf * 8;
      kr[ks] = vr[ks] = make_uint4(0, 0, 0, 0);
      if (c0 < D) {
        kr[ks] = *reinterpret_cast<const uint4*>(kp + c0);
        kr[ks] = make_uint4(kr[ks].x ^ flip, kr[ks].y ^ flip, kr[ks].z ^ flip, kr[ks].w ^ flip);
        if constexpr (DK) vr[ks] = *reinterpret_cast<const uint4*>(vp + c0);
      }
    }
  }
  const float f = fabsf(a.scale) * 1.44269504088896341f;
  constexpr float kUp = BF16 ? 0.0f : 15.0f;

  v16f_t ak[ND], av[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) ak[d] = av[d] = attn_zero();
  Reach<BF16, ND> reach;
  AttnRead<DP> rd(smem);
  // this lane's token is seen by rows i in [j, until) of a causal sequence, all of another
  const int from = a.causal ? col : 0;
  const int until = a.window > 0 && col >= a.sinks ? (int)min((int64_t)sq.n, (int64_t)col + a.window) : sq.n;
  // tiles that begin from here on and end before there are seen whole by all columns
  const int all_from = a.causal ? j_hi : 0;
  const int all_until = a.window > 0 && j_hi >= a.sinks ? max(j0, (int)min((int64_t)a.sinks, (int64_t)j_hi)) + a.window : INT32_MAX;

  for (int i = 0, i_at = lo, i_head = 0; i < tiles; ++i) {
    const int stage = i & 1, base = i_at << 6;
    const bool masked = base < all_from || base + 64 > all_until;
    attn_wait_copies();
    __syncthreads();
    bool odd = false;
    if (masked) {
      if constexpr (DK) odd = attn_finite<DP, BF16, W>(smem + stage * 2 * Tile::kBytes);
      if constexpr (DV) odd |= attn_finite<DP, BF16, W>(smem + (stage * 2 + 1) * Tile::kBytes);
    }
    if (i + 1 < tiles) next(stage ^ 1);
    const float* st_l = sh_stat + stage * 128;
#pragma unroll
    for (int sb = 0; sb < 2; ++sb) {
      v16f_t s = attn_rows_product<DP, BF16>(rd, 0, sb, kr), t = attn_zero();
      if constexpr (DK) t = attn_rows_product<DP, BF16>(rd, 1, sb, vr);
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const int row = 32 * sb + 16 * k + 8 * hf + e;
          const v4f l = *reinterpret_cast<const v4f*>(st_l + row);
          v4f dl;
          if constexpr (DK) dl = *reinterpret_cast<const v4f*>(st_l + 64 + row);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const int y = 8 * k + e + x;
            s[y] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[y], f, kUp - l[x]));
            if constexpr (DK) t[y] = s[y] * (t[y] - dl[x]);
          }
        }
      if (masked) {
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const int row = base + 32 * sb + 16 * (x >> 3) + 8 * hf + (x & 7);
          if (!((row >= from) & (row < until))) s[x] = t[x] = 0.0f;
        }
      }
      if constexpr (DK && !BF16) {
        reach.fit(t, ak);
        t *= reach.g;
      }
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if constexpr (DV) {
          const uint4 p = attn_pack<BF16>(s, k);
#pragma unroll
          for (int d = 0; d < ND; ++d) av[d] = Act16<BF16>::mma32(rd.channels(1, d, 2 * sb + k), p, av[d]);
        }
        if constexpr (DK) {
          const uint4 p = attn_pack<BF16>(t, k);
#pragma unroll
          for (int d = 0; d < ND; ++d) ak[d] = Act16<BF16>::mma32(rd.channels(0, d, 2 * sb + k), p, ak[d]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (__builtin_expect(odd, 0)) {
      auto see = [&](int t) { return (base + t >= from) & (base + t < until); };
      if constexpr (DV)
        attn_others<DP, BF16>(av, gp + (int64_t)i_head * a.d_o.head, a.d_o.token, base, sq.n, D, see);
      if constexpr (DK) attn_others<DP, BF16>(ak, qp + (int64_t)i_head * a.q.head, a.q.token, base, sq.n, D, see);
    }
    if (++i_at == lo + per) i_at = lo, ++i_head;
    rd.next(stage ? -2 * Tile::kBytes : 2 * Tile::kBytes);
  }

  if (col >= sq.n) return;
  auto store = [&](const KvRows& to, const v16f_t (&acc)[ND], float by) {
    uint16_t* op = to.p + ((int64_t)sq.row0 + j) * to.token + (int64_t)h * to.head;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = d * 32 + 8 * k + 4 * hf;
        if (c >= D) continue;
        *reinterpret_cast<uint2*>(op + c) =
            make_uint2(Act16<BF16>::pack2(acc[d][4 * k] * by, acc[d][4 * k + 1] * by),
                       Act16<BF16>::pack2(acc[d][4 * k + 2] * by, acc[d][4 * k + 3] * by));
      }
  };
  if constexpr (DV) store(a.dv, av, BF16 ? 1.0f : 3.0517578125e-5f);
  if constexpr (DK) store(a.dk, ak, a.scale / reach.g * (BF16 ? 1.0f : 3.0517578125e-5f));
}

template <int DP, bool BF16>
static hipError_t launch_bwd(const AttnArgs& a, hipStream_t stream) {
  const int64_t rows = (((int64_t)a.T * (a.q_heads / a.heads) >> 7) + a.B) * a.heads;
  const int64_t cols = (((int64_t)a.T >> 7) + a.B) * a.heads;
  if (rows > INT32_MAX || cols > INT32_MAX) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((ka_dq<DP, BF16>), dim3((unsigned)rows), dim3(256), 0, stream, a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if constexpr (DP <= 128) {
    hipLaunchKernelGGL((ka_dkv<DP, BF16, true, true>), dim3((unsigned)cols), dim3(256), 0, stream, a);
  } else {
    hipLaunchKernelGGL((ka_dkv<DP, BF16, true, false>), dim3((unsigned)cols), dim3(256), 0, stream, a);
    e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((ka_dkv<DP, BF16, false, true>), dim3((unsigned)cols), dim3(256), 0, stream, a);
  }
  return hipGetLastError();
}

hipError_t launch_attention_backward(const AttnArgs& a, bool bf16, hipStream_t stream) {
  if (a.dim <= 64) return bf16 ? launch_bwd<64, true>(a, stream) : launch_bwd<64, false>(a, stream);
  if (a.dim <= 96) return bf16 ? launch_bwd<96, true>(a, stream) : launch_bwd<96, false>(a, stream);
  if (a.dim <= 128) return bf16 ? launch_bwd<128, true>(a, stream) : launch_bwd<128, false>(a, stream);
  return bf16 ? launch_bwd<256, true>(a, stream) : launch_bwd<256, false>(a, stream);
}

}  // namespace llmint8
