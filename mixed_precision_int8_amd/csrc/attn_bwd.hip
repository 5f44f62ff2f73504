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
//
// Like the forward pass bound by the SIMDs' issue. 15000 tokens of 32/8 heads of 128: ka_dq
// 590 us (960 TFLOP/s), ka_dkv 840 (910); matrix cores busy in 49 and 46% of the cycles. A token's dk and dv
// are one workgroup's over all query heads of its group: few key/value heads leave most CUs idle (8192 tokens of
// 8 query heads of 128: 503 us for the gradients with 8 key/value heads, 1809 with one).
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
      if (__builtin_expect(__any(top * g > 32768.0f), 0)) {
        const int e = (int)(__float_as_uint(top) >> 23) - 127;
        const float to = top * g > 32768.0f ? __uint_as_float((uint32_t)(min(8 - e, 126) + 127) << 23) : g;
        const float by = to / g;
#pragma unroll
        for (int d = 0; d < ND; ++d) acc[d] *= by;
        g = to;
      }
    }
  }
};

// A lane's channels of a row: times `by`, rounded, to row `row` of head h.
template <int DP, bool BF16>
__device__ __forceinline__ void store_sums(const v16f_t (&acc)[DP / 32], float by, const KvRows& to, int64_t row, int h,
                                           int dim, int hf) {
  uint16_t* p = to.p + row * to.token + (int64_t)h * to.head;
#pragma unroll
  for (int d = 0; d < DP / 32; ++d)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = d * 32 + 8 * k + 4 * hf;
      if (c >= dim) continue;
      *reinterpret_cast<uint2*>(p + c) =
          make_uint2(Act16<BF16>::pack2(acc[d][4 * k] * by, acc[d][4 * k + 1] * by),
                     Act16<BF16>::pack2(acc[d][4 * k + 2] * by, acc[d][4 * k + 3] * by));
    }
}

// What tokens j0 .. j_hi of k and v are seen by: rows [first, end) at most; token `col`, this
// lane's, by `count` rows from `from` on.
struct AttnRowsOf {
  int first, end, from, all_from, all_until;
  uint32_t count;
  __device__ __forceinline__ AttnRowsOf(const AttnArgs& a, int n, int j0, int j_hi, int col) {
    first = a.causal ? j0 : 0;
    end = a.window > 0 && j0 >= a.sinks ? (int)min((int64_t)n, (int64_t)j_hi + a.window) : n;
    from = a.causal ? col : 0;
    count = (uint32_t)max((a.window > 0 && col >= a.sinks ? (int)min((int64_t)n, (int64_t)col + a.window) : n) - from, 0);
    all_from = a.causal ? j_hi : 0;
    all_until = a.window > 0 && j_hi >= a.sinks ? min(n, max(j0, (int)min((int64_t)a.sinks, (int64_t)j_hi)) + a.window) : n;
  }
  __device__ __forceinline__ bool operator()(int row) const { return (uint32_t)(row - from) < count; }
  // a tile that some of the tokens do not see whole, or that the sequence ends in: the zeros behind it are
  // rows that give nothing only times what is finite
  __device__ __forceinline__ bool masked(int base) const { return (base < all_from) | (base + 64 > all_until); }
};

// Sums over this many tiles at most (256 tokens) are of few enough terms for the rounding of one
// to show: there P and dS take part to twice the type's bits, by a second product, and delta is
// summed anew (3 to 60 tokens, fp16: dq and dk off by 2.1e-4 instead of 3.8e-4 of their size; the
// three kernels 26 us instead of 23). Over more tokens errors of single terms average out; o is
// their mean, and its rounding a 16th or less of the spread of do V^T.
constexpr int kFew = 4;

}  // namespace

template <int DP, bool BF16>
__global__ __launch_bounds__(256, DP <= 128 ? 2 : 1) void ka_dq(AttnArgs a) {
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
  const int r = (int)min(row0 + wave * 32 + nn, rows - 1);
  const int pos = r / G, qh = h * G + (r - pos * G);
  const int qrow = sq.row0 + pos;
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

  uint4 q[NQ], g[NQ];
  float delta = 0.0f;
  {
    const uint16_t* qp = a.q.p + (int64_t)qrow * a.q.token + (int64_t)qh * a.q.head;
    const uint16_t* gp = a.d_o.p + (int64_t)qrow * a.d_o.token + (int64_t)qh * a.d_o.head;
    const uint16_t* op = a.o.p + (int64_t)qrow * a.o.token + (int64_t)qh * a.o.head;
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
  const float lse2 = a.lse[(int64_t)qrow * a.q_heads + qh] * 1.44269504088896341f;
  AttnRead<DP> rd(smem);
  const AttnSees sees(a, pos, sq.n);

  // o has been rounded, and so is delta off by half a step of it times do: little beside the
  // spread of do V^T where many tokens share a row's weight, as much as all else where few do.
  // There delta is summed from its definition, sum_j P_ij (do V^T)_ij: two products more.
  if (tiles <= kFew) {
    delta = 0.0f;
#pragma unroll 1
    for (int i = 0; i < tiles; ++i) {
      const int stage = i & 1, base = base_of(i);
      attn_wait_copies();
      attn_barrier();
      copy(i + 1, stage ^ 1);
#pragma unroll
      for (int sb = 0; sb < 2; ++sb) {
        if (idle | own.none(base + 32 * sb, 32)) continue;
        const v16f_t s = attn_rows_product<DP, BF16>(rd, 0, sb, q);
        const v16f_t t = attn_rows_product<DP, BF16>(rd, 1, sb, g);
#pragma unroll
        for (int x = 0; x < 16; ++x)
          if (sees(base + 32 * sb + 16 * (x >> 3) + 8 * hf + (x & 7)))
            delta = __builtin_fmaf(__builtin_amdgcn_exp2f(__builtin_fmaf(s[x], f, -lse2)), t[x], delta);
      }
      rd.next(stage ? -kStage : kStage);
    }
    delta = attn_pair_sum(delta);
    if (tiles & 1) rd.next(-kStage);
    attn_wait_copies();
    attn_barrier();
    ck.rewind(kp, a.k.token, start);
    cv.rewind(vp, a.v.token, start);
    copy(0, 0);
  }
  const bool mine = row0 + wave * 32 + nn < rows;
  if (mine && hf == 0) {
    float* st = a.stat + (int64_t)qh * a.T + qrow;
    st[0] = (BF16 ? 0.0f : 15.0f) - lse2 + (lse2 - lse2);  // NaN where lse is -infinity: all of the row's logits are
    st[(int64_t)a.q_heads * a.T] = delta;
  }

  v16f_t acc[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) acc[d] = attn_zero();
  Reach<BF16, ND> reach;

  auto loop = [&](auto few) {  // a loop of its own for each, so that the other has nothing of it
    for (int i = 0; i < tiles; ++i) {
      const int stage = i & 1, base = base_of(i);
      const bool masked = all.masked(base);
      attn_wait_copies();
      if (masked) ck.template finite<BF16>(smem + stage * kStage, flag);
      attn_barrier();
      const int cleared = masked ? uniform(*flag) : 0;
      copy(i + 1, stage ^ 1);
#pragma unroll
      for (int sb = 0; sb < 2; ++sb) {
        if (idle | own.none(base + 32 * sb, 32)) continue;
        v16f_t s = attn_rows_product<DP, BF16>(rd, 0, sb, q);
        if (__builtin_expect(cleared, 0)) attn_hide<BF16>(s, kp, a.k.token, base + 32 * sb, sq.n, D);
        v16f_t t = attn_rows_product<DP, BF16>(rd, 1, sb, g);
        // 256 channels leave no registers for operands read this early (172 of them went to memory in
        // fp16, and the gradients took 1.6 times as long)
        constexpr bool kEarly = DP <= 128;
        uint4 y[2][kEarly ? ND : 1];
        if constexpr (kEarly) {
#pragma unroll
          for (int d = 0; d < ND; ++d) y[0][d] = rd.channels(0, d, 2 * sb);
        }
#pragma unroll
        for (int x = 0; x < 16; ++x) t[x] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[x], f, -lse2)) * (t[x] - delta);
        if (own.masked(base)) {
#pragma unroll
          for (int x = 0; x < 16; ++x)
            if (!sees(base + 32 * sb + 16 * (x >> 3) + 8 * hf + (x & 7))) t[x] = 0.0f;
        }
        if constexpr (!BF16) {
          reach.fit(t, acc);
          t *= reach.g;
        }
        if constexpr (!kEarly) {
          attn_channels_product<DP, BF16>(rd, 0, sb, t, acc);
        } else {
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
        if constexpr (few()) {
          attn_residual<BF16>(t);
          attn_channels_product<DP, BF16>(rd, 0, sb, t, acc);
        }
      }
      rd.next(stage ? -kStage : kStage);
    }
  };
  if (tiles <= kFew) loop(std::true_type{});
  else loop(std::false_type{});
  attn_wait_copies();
  if (__builtin_expect(uniform(*flag), 0)) {
#pragma unroll 1
    for (int i = 0; i < tiles; ++i) {
      const int base = base_of(i);
      if (all.masked(base))
        attn_others<DP, BF16>(acc, kp, a.k.token, base, sq.n, D, false, [&](int t) { return sees(base + t); });
    }
  }

  if (!mine) return;
  store_sums<DP, BF16>(acc, a.scale / reach.g, a.dq, qrow, qh, D, hf);
}

// Up to 96 channels a wavefront has the registers for dV and dK of 32 tokens (184 and 240), two
// wavefronts to a SIMD, and nothing goes through LDS between them: 290 us where pairs of
// wavefronts as below take 561 on 32000 tokens with a window of 500, 16 heads of 64 in fp16;
// 334 and 446 on 20 images, 16 heads of 80 in bf16.
template <int DP, bool BF16>
__global__ __launch_bounds__(256, 2) void ka_dkv_alone(AttnArgs a) {
  using Tile = AttnTile<DP>;
  constexpr int W = 4, kCols = 32 * W, NQ = Tile::NQ, ND = Tile::ND;
  constexpr int kStage = 2 * Tile::kBytes;  // q, do
  // lse, delta of the stages and a place that the other wavefronts' go to; a flag
  constexpr int kAtStat = 2 * kStage, kAtFlag = kAtStat + 2 * 512 + 256;
  __shared__ __attribute__((aligned(1024))) char smem[kAtFlag + 16];
  int* const flag = reinterpret_cast<int*>(smem + kAtFlag);
  const int D = a.dim, H = a.heads, G = a.q_heads / H;
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
  const int hf = lane >> 5, nn = lane & 31;
  const int h = (int)(blockIdx.x % H), item = (int)(blockIdx.x / H);
  AttnSeq sq;
  int run;
  if (!attn_place<false>(a, item, 1, 7, &sq, &run)) return;
  const int j0 = run * kCols;
  const int col = j0 + wave * 32 + nn, j = min(col, sq.n - 1), j_hi = min(j0 + kCols, sq.n) - 1;

  const AttnRowsOf see(a, sq.n, j0, j_hi, col);
  const int w0 = j0 + wave * 32;
  const AttnRowsOf own(a, sq.n, w0, min(w0 + 31, sq.n - 1), col);  // of this wavefront's tokens
  const bool idle = w0 >= sq.n;
  const int lo = see.first >> 6, per = ((see.end + 63) >> 6) - lo, tiles = per * G;

  const uint16_t* qp = a.q.p + (int64_t)sq.row0 * a.q.token + (int64_t)h * G * a.q.head;
  const uint16_t* gp = a.d_o.p + (int64_t)sq.row0 * a.d_o.token + (int64_t)h * G * a.d_o.head;
  const int64_t back = (int64_t)(per - 1) * 64;  // from a head's last tile to the next one's first
  AttnStream<DP, W> cq(qp, a.q.token, D, (int64_t)lo * 64, a.q.head - back * a.q.token);
  AttnStream<DP, W> cg(gp, a.d_o.token, D, (int64_t)lo * 64, a.d_o.head - back * a.d_o.token);
  const float* sp = a.stat + (int64_t)h * G * a.T + sq.row0 + lo * 64 + (wave ? (int64_t)a.q_heads * a.T : 0);
  int left = tiles, c_at = lo;  // tiles to copy, the next one
  auto copy = [&](int c_stage) {
    // past the last tile: zeros
    const int n = left > 0 ? min(sq.n - c_at * 64, 64) : 0;
    const bool jump = ++c_at == lo + per;
    char* to = smem + c_stage * kStage;
    cq.next(n, to, jump);
    cg.next(n, to + Tile::kBytes, jump);
    attn_copy4(make_rsrc(reinterpret_cast<const float*>(uniform(reinterpret_cast<int64_t>(sp))), (uint32_t)uniform(wave < 2 ? n * 4 : 0)),
               smem + kAtStat + uniform(wave < 2 ? c_stage * 512 + wave * 256 : 2 * 512), (uint32_t)lane * 4);
    sp += jump ? a.T - back : 64;
    if (jump) c_at = lo;
    --left;
  };
  copy(0);
  if (threadIdx.x == 0) *flag = 0;
  attn_barrier();

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
        vr[ks] = *reinterpret_cast<const uint4*>(vp + c0);
      }
    }
  }
  const float f = fabsf(a.scale) * 1.44269504088896341f;

  v16f_t dv[ND], dk[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) dv[d] = dk[d] = attn_zero();
  Reach<BF16, ND> reach;
  AttnRead<DP> rd(smem);
  const char* st = smem + kAtStat + 32 * hf;
  auto loop = [&](auto few) {
    int at = lo;
    for (int i = 0; i < tiles; ++i) {
      const int stage = i & 1, base = at << 6;
      const bool masked = see.masked(base), hidden = own.masked(base);
      attn_wait_copies();
      if (masked) {
        cq.template finite<BF16>(smem + stage * kStage, flag);
        cg.template finite<BF16>(smem + stage * kStage + Tile::kBytes, flag);
      }
      attn_barrier();
      copy(stage ^ 1);
#pragma unroll
      for (int sb = 0; sb < 2; ++sb) {
        if (idle | (base + 32 * sb + 32 <= own.first) | (base + 32 * sb >= own.end)) continue;
        auto stat = [&](int which, int e) {
          return *reinterpret_cast<const v4f*>(st + 256 * which + 128 * sb + 64 * (e >> 1) + 16 * (e & 1));
        };
        auto mask = [&](v16f_t& x) {
          int row = base + 32 * sb + 8 * hf;
          asm volatile("" : "+v"(row));  // or 16 rows less this token's first one are kept in registers
#pragma unroll
          for (int z = 0; z < 16; ++z)
            if (!see(row + 16 * (z >> 3) + (z & 7))) x[z] = 0.0f;
        };
        v16f_t s = attn_rows_product<DP, BF16>(rd, 0, sb, kr);
        v16f_t t;
        if constexpr (!few()) t = attn_rows_product<DP, BF16>(rd, 1, sb, vr);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const v4f l = stat(0, e);
#pragma unroll
          for (int z = 0; z < 4; ++z) s[4 * e + z] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[4 * e + z], f, l[z]));
        }
        if (hidden) mask(s);
        attn_channels_product<DP, BF16>(rd, 1, sb, s, dv);
        if constexpr (few()) {
          v16f_t r = s;
          attn_residual<BF16>(r);
          attn_channels_product<DP, BF16>(rd, 1, sb, r, dv);
          t = attn_rows_product<DP, BF16>(rd, 1, sb, vr);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const v4f l = stat(1, e);
#pragma unroll
          for (int z = 0; z < 4; ++z) t[4 * e + z] = s[4 * e + z] * (t[4 * e + z] - l[z]);
        }
        if (hidden) mask(t);  // do is not finite in a row that this token does not see, or its delta
        if constexpr (!BF16) {
          reach.fit(t, dk);
          t *= reach.g;
        }
        attn_channels_product<DP, BF16>(rd, 0, sb, t, dk);
        if constexpr (few()) {
          attn_residual<BF16>(t);
          attn_channels_product<DP, BF16>(rd, 0, sb, t, dk);
        }
      }
      rd.next(stage ? -kStage : kStage);
      st += stage ? -512 : 512;
      if (++at == lo + per) at = lo;
    }
  };
  if (per <= kFew) loop(std::true_type{});
  else loop(std::false_type{});
  attn_wait_copies();
  if (__builtin_expect(uniform(*flag), 0)) {
#pragma unroll 1
    for (int i = 0; i < tiles; ++i) {
      const int base = (lo + i % per) << 6;
      if (!see.masked(base)) continue;
      auto sees = [&](int t) { return see(base + t); };
      attn_others<DP, BF16>(dv, gp + (int64_t)(i / per) * a.d_o.head, a.d_o.token, base, sq.n, D, true, sees);
      attn_others<DP, BF16>(dk, qp + (int64_t)(i / per) * a.q.head, a.q.token, base, sq.n, D, false, sees);
    }
  }

  if (col >= sq.n) return;
  // P carries 2^15 in fp16; dS its column's power of two as well
  constexpr float kBy = BF16 ? 1.0f : 3.0517578125e-5f;
  store_sums<DP, BF16>(dv, kBy, a.dv, sq.row0 + j, h, D, hf);
  store_sums<DP, BF16>(dk, kBy * (a.scale / reach.g), a.dk, sq.row0 + j, h, D, hf);
}

// Two wavefronts share 32 tokens: one forms S and P and sums dV, the other do V^T and dS
// (from the first one's P, through LDS) and sums dK, eight wavefronts to a workgroup. A
// wavefront's vector instructions wait for its matrix instructions here (measured: four of
// 32x32x16 and 16 multiply-adds take what each takes alone, together, from one wavefront;
// the longer of the two from two), so that two to a SIMD are what overlaps them, and one
// wavefront with both sums of 128 channels needs 450 registers and runs alone (1355 us where
// this takes 840: 15000 tokens of 32/8 heads of 128).
template <int DP, bool BF16>
__global__ __launch_bounds__(DP <= 128 ? 512 : 256, DP <= 128 ? 2 : 1) void ka_dkv(AttnArgs a) {
  using Tile = AttnTile<DP>;
  constexpr int kPairs = DP <= 128 ? 4 : 2, W = 2 * kPairs, kCols = 32 * kPairs, NQ = Tile::NQ, ND = Tile::ND;
  constexpr int kStages = DP <= 128 ? 3 : 2, kStage = 2 * Tile::kBytes;
  // q, do; P, two steps; lse, delta of the stages and a place that the other wavefronts' go to; a flag
  constexpr int kAtP = kStages * kStage, kAtStat = kAtP + 2 * kPairs * 4096, kAtFlag = kAtStat + kStages * 512 + 256;
  __shared__ __attribute__((aligned(1024))) char smem[kAtFlag + 16];
  int* const flag = reinterpret_cast<int*>(smem + kAtFlag);
  const int D = a.dim, H = a.heads, G = a.q_heads / H;
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
  const int hf = lane >> 5, nn = lane & 31, pair = wave % kPairs;
  const bool second = wave >= kPairs;
  const int h = (int)(blockIdx.x % H), item = (int)(blockIdx.x / H);
  AttnSeq sq;
  int run;
  if (!attn_place<false>(a, item, 1, kPairs == 4 ? 7 : 6, &sq, &run)) return;
  const int j0 = run * kCols;
  const int col = j0 + pair * 32 + nn, j = min(col, sq.n - 1), j_hi = min(j0 + kCols, sq.n) - 1;

  const AttnRowsOf see(a, sq.n, j0, j_hi, col);
  const int lo = see.first >> 6, per = ((see.end + 63) >> 6) - lo, tiles = per * G;

  const uint16_t* qp = a.q.p + (int64_t)sq.row0 * a.q.token + (int64_t)h * G * a.q.head;
  const uint16_t* gp = a.d_o.p + (int64_t)sq.row0 * a.d_o.token + (int64_t)h * G * a.d_o.head;
  const int64_t back = (int64_t)(per - 1) * 64;  // from a head's last tile to the next one's first
  AttnStream<DP, W> cq(qp, a.q.token, D, (int64_t)lo * 64, a.q.head - back * a.q.token);
  AttnStream<DP, W> cg(gp, a.d_o.token, D, (int64_t)lo * 64, a.d_o.head - back * a.d_o.token);
  const float* sp = a.stat + (int64_t)h * G * a.T + sq.row0 + lo * 64 + (wave ? (int64_t)a.q_heads * a.T : 0);
  int left = tiles, c_at = lo, c_stage = 0;  // tiles to copy, the next one
  auto copy = [&]() {
    // past the last tile: zeros
    const int n = left > 0 ? min(sq.n - c_at * 64, 64) : 0;
    const bool jump = ++c_at == lo + per;
    char* to = smem + c_stage * kStage;
    cq.next(n, to, jump);
    cg.next(n, to + Tile::kBytes, jump);
    attn_copy4(make_rsrc(reinterpret_cast<const float*>(uniform(reinterpret_cast<int64_t>(sp))), (uint32_t)uniform(wave < 2 ? n * 4 : 0)),
               smem + kAtStat + uniform(wave < 2 ? c_stage * 512 + wave * 256 : kStages * 512), (uint32_t)lane * 4);
    sp += jump ? a.T - back : 64;
    if (jump) c_at = lo;
    --left;
    if (++c_stage == kStages) c_stage = 0;
  };
  copy();
  if (threadIdx.x == 0) *flag = 0;
  attn_barrier();

  uint4 kv[NQ];  // k of this lane's token, v in the second wavefront
  {
    const KvRows& r = second ? a.v : a.k;
    const uint16_t* p = r.p + ((int64_t)sq.row0 + j) * r.token + (int64_t)h * r.head;
    const uint32_t flip = !second && a.scale < 0.0f ? 0x80008000u : 0u;
#pragma unroll
    for (int ks = 0; ks < NQ; ++ks) {
      const int c0 = ks * 16 + hf * 8;
      kv[ks] = make_uint4(0, 0, 0, 0);
      if (c0 < D) {
        kv[ks] = *reinterpret_cast<const uint4*>(p + c0);
        kv[ks] = make_uint4(kv[ks].x ^ flip, kv[ks].y ^ flip, kv[ks].z ^ flip, kv[ks].w ^ flip);
      }
    }
  }
  const float f = fabsf(a.scale) * 1.44269504088896341f;

  v16f_t acc[ND];  // dV, dK in the second wavefront
#pragma unroll
  for (int d = 0; d < ND; ++d) acc[d] = attn_zero();
  Reach<BF16, ND> reach;

  // A step takes 32 rows of a tile. The first wavefront forms S, P and its part of dV in a step,
  // the second in the same one dS and its part of dK for the step before, from the P that the
  // first left then, and afterwards do V^T for this one: each has its vector instructions where
  // the other has matrix instructions. One barrier to a step, P in two buffers. Copies of a tile
  // have two steps to arrive (three stages: the second wavefront leaves a tile a step after the
  // first).
  AttnRead<DP> rd(smem);  // the first wavefront's products are q's rows and do's channels, the second's the others
  rd.next_rows(second ? Tile::kBytes : 0);
  rd.next_channels(second ? 0 : Tile::kBytes);
  v4f* const p_mine = reinterpret_cast<v4f*>(smem + kAtP) + pair * 256 + lane;
  const char* st_mine = smem + kAtStat + (second ? 256 : 0) + 32 * hf;
  // this wavefront's pieces of the tile that was copied last are there; then of the next one
  int w_at = lo;
  auto arrive = [&](int tile) {
    const int base = w_at << 6;
    if (++w_at == lo + per) w_at = lo;
    attn_wait_copies();
    if (tile < tiles && see.masked(base)) {
      char* at = smem + tile % kStages * kStage;
      cq.template finite<BF16>(at, flag);
      cg.template finite<BF16>(at + Tile::kBytes, flag);
    }
  };
  arrive(0);
  attn_barrier();
  if (kStages > 2) copy();
  // A step has NQ products of rows and NQ of channels, in this order or the other. Operands are
  // read kRing - 1 products ahead, beyond the step's end from the next step's.
  static_assert(NQ == 2 * ND, "a step has as many products of rows as of channels");
  constexpr int kRing = 8;
  static_assert(2 * NQ % kRing == 0, "a product's place in the ring is the same in every step");
  static_assert(kRing <= NQ + 1, "the next step's operands are read once the addresses have moved on");
  uint4 ring[kRing];
  constexpr int kCopyAt = 1;  // scalar instructions run beside matrix instructions
  int at = lo, stage = 0;
  // from a tile's step sb to the next one: how far the addresses move
  auto advance = [&](int sb) {
    if (sb == 0) return 2 * Tile::kSixteen;
    const int was = stage;
    if (++stage == kStages) stage = 0;
    if (++at == lo + per) at = lo;
    return (stage - was) * kStage - 2 * Tile::kSixteen;
  };
  auto stat = [&](v4f (&l)[4]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) l[e] = *reinterpret_cast<const v4f*>(st_mine + 64 * (e >> 1) + 16 * (e & 1));
  };
  auto mask = [&](v16f_t& s, int base) {
#pragma unroll
    for (int z = 0; z < 16; ++z)
      if (!see(base + 16 * (z >> 3) + 8 * hf + (z & 7))) s[z] = 0.0f;
  };
  auto again = [&](v16f_t& s) {
    attn_residual<BF16>(s);
    attn_channels_product<DP, BF16>(rd, 0, 0, s, acc);
  };
  // the end of the first wavefront's step (i, sb)
  auto turn = [&](int i, int sb) {
    if (sb == (kStages == 2)) arrive(i + 1);
    attn_barrier();
  };
  if (!second) {
    auto fetch = [&](int n) {
      if (n < NQ || (n >= 2 * NQ && kStages > 2)) ring[n % kRing] = rd.rows(0, 0, n % (2 * NQ));
      else if (n < 2 * NQ) ring[n % kRing] = rd.channels(0, (n - NQ) % ND, (n - NQ) / ND);
    };
    if (kStages > 2) {
#pragma unroll
      for (int n = 0; n < kRing - 1; ++n) fetch(n);
    }
    for (int i = 0; i < tiles; ++i)
#pragma unroll
      for (int sb = 0; sb < 2; ++sb) {
        v4f l[4];
        stat(l);
        if (kStages == 2) {
#pragma unroll
          for (int n = 0; n < kRing - 1; ++n) fetch(n);
        }
        v16f_t s;
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          fetch(n + kRing - 1);
          s = Act16<BF16>::mma32(ring[n % kRing], kv[n], n == 0 ? attn_zero() : s);
          if (sb == 1 && n == kCopyAt) copy();
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int z = 0; z < 16; ++z) s[z] = __builtin_amdgcn_exp2f(__builtin_fmaf(s[z], f, l[z >> 2][z & 3]));
        if (see.masked(at << 6)) mask(s, (at << 6) + 32 * sb);
        v4f* p = p_mine + sb * kPairs * 256;
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e * 64] = v4f{s[4 * e], s[4 * e + 1], s[4 * e + 2], s[4 * e + 3]};
        const int was = stage, by = advance(sb);
        rd.next_rows(by);
        uint4 x;
#pragma unroll
        for (int n = NQ; n < 2 * NQ; ++n) {
          fetch(n + kRing - 1);  // nobody's after the last step
          if (n % ND == 0) x = attn_pack<BF16>(s, (n - NQ) / ND);
          acc[n % ND] = Act16<BF16>::mma32(ring[n % kRing], x, acc[n % ND]);
          __builtin_amdgcn_sched_barrier(0);
        }
        if (per <= kFew) again(s);
        rd.next_channels(by);
        st_mine += (stage - was) * 512 + (sb ? -128 : 128);
        turn(i, sb);
      }
    turn(tiles, 0);
  } else {
    // products of a step: kBegin of this step's rows while P is on its way from LDS, channels of the
    // step before, the other rows
    constexpr int kBegin = kStages > 2 ? NQ / 2 : 0;
    auto fetch = [&](int n) {
      const int c = n % (2 * NQ);
      if (c < kBegin) ring[n % kRing] = rd.rows(0, 0, c);
      else if (c < kBegin + NQ) ring[n % kRing] = rd.channels(0, (c - kBegin) % ND, (c - kBegin) / ND);
      else ring[n % kRing] = rd.rows(0, 0, c - NQ);
    };
    int rows_by = 0;  // to the rows of the step after
    auto ahead = [&](int n) {
      fetch(n + kRing - 1);
      if (n + kRing == 2 * NQ) rd.next_rows(rows_by);
    };
    v16f_t t, u;
    auto rows_products = [&](int from, int to, v16f_t& t) {
#pragma unroll
      for (int r = from; r < to; ++r) {
        const int n = r < kBegin ? r : r + NQ;
        ahead(n);
        t = Act16<BF16>::mma32(ring[n % kRing], kv[r], r == 0 ? attn_zero() : t);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
#pragma unroll
    for (int r = 0; r < NQ; ++r) t = Act16<BF16>::mma32(rd.rows(0, 0, r), kv[r], r == 0 ? attn_zero() : t);
    turn(0, 0);
    rd.next_rows(2 * Tile::kSixteen);
#pragma unroll
    for (int n = 0; n < kRing - 1; ++n) fetch(n);
    for (int i = 0; i < tiles; ++i)
#pragma unroll
      for (int sb = 0; sb < 2; ++sb) {  // sums of step (i, sb), do V^T of the next one
        const v4f* p = p_mine + sb * kPairs * 256;
        v4f l[4], w[4];
        stat(l);
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = p[e * 64];
        rows_by = sb ? 2 * Tile::kSixteen : ((stage + 1 == kStages ? 0 : stage + 1) - stage) * kStage - 2 * Tile::kSixteen;
        rows_products(0, kBegin, u);
#pragma unroll
        for (int z = 0; z < 16; ++z) t[z] = w[z >> 2][z & 3] * (t[z] - l[z >> 2][z & 3]);
        if (see.masked(at << 6)) mask(t, (at << 6) + 32 * sb);
        if constexpr (!BF16) {
          reach.fit(t, acc);
          t *= reach.g;
        }
        const int was = stage, by = advance(sb);
        uint4 x;
#pragma unroll
        for (int c = 0; c < NQ; ++c) {
          const int n = c + kBegin;
          ahead(n);
          if (c % ND == 0) x = attn_pack<BF16>(t, c / ND);
          acc[c % ND] = Act16<BF16>::mma32(ring[n % kRing], x, acc[c % ND]);
          if (sb == 0 && c == kCopyAt) copy();
          __builtin_amdgcn_sched_barrier(0);
        }
        if (per <= kFew) again(t);
        rd.next_channels(by);
        st_mine += (stage - was) * 512 + (sb ? -128 : 128);
        rows_products(kBegin, NQ, u);  // nobody's after the last step
        t = u;
        turn(i + sb, sb ^ 1);
      }
  }
  attn_wait_copies();
  if (__builtin_expect(uniform(*flag), 0)) {
    const KvRows& r = second ? a.q : a.d_o;
#pragma unroll 1
    for (int i = 0; i < tiles; ++i) {
      const int at = (lo + i % per) << 6;
      auto sees = [&](int t) { return see(at + t); };
      if (see.masked(at)) attn_others<DP, BF16>(acc, (second ? qp : gp) + (int64_t)(i / per) * r.head, r.token, at, sq.n, D, !second, sees);
    }
  }

  if (col >= sq.n) return;
  // P carries 2^15 in fp16; dS its column's power of two as well
  const float by = (BF16 ? 1.0f : 3.0517578125e-5f) * (second ? a.scale / reach.g : 1.0f);
  store_sums<DP, BF16>(acc, by, second ? a.dk : a.dv, sq.row0 + j, h, D, hf);
}

template <int DP, bool BF16>
static hipError_t launch_bwd(const AttnArgs& a, hipStream_t stream) {
  constexpr bool kAlone = DP <= 96;
  const AttnGrid rows = attn_row_grid(a.T, a.q_heads, a.heads, a.B), cols = attn_col_grid(a.T, a.heads, a.B, a.dim);
  if (!rows.fits() || !cols.fits()) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((ka_dq<DP, BF16>), dim3((unsigned)rows.blocks), dim3(256), 0, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if constexpr (kAlone) hipLaunchKernelGGL((ka_dkv_alone<DP, BF16>), dim3((unsigned)cols.blocks), dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((ka_dkv<DP, BF16>), dim3((unsigned)cols.blocks), dim3(cols.threads), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_attention_backward(const AttnArgs& a, bool bf16, hipStream_t stream) {
  if (a.dim <= 64) return bf16 ? launch_bwd<64, true>(a, stream) : launch_bwd<64, false>(a, stream);
  if (a.dim <= 96) return bf16 ? launch_bwd<96, true>(a, stream) : launch_bwd<96, false>(a, stream);
  if (a.dim <= 128) return bf16 ? launch_bwd<128, true>(a, stream) : launch_bwd<128, false>(a, stream);
  return bf16 ? launch_bwd<256, true>(a, stream) : launch_bwd<256, false>(a, stream);
}

}  // namespace llmint8
