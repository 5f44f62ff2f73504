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
//                   the row's largest. That is below the inputs' own rounding for
//                   channels down to 2^-5 of the largest in fp16 and 2^-8 in bf16;
//                   smaller ones keep fewer bits than they had. Over 128 channels
//                   of like keys that changes a logit by about what the rounding
//                   of the largest one did; a third plane would keep them, at
//                   half the first product again.
//                   The sums are exact (dim * 127 * 32639 < 2^31).
//   O^T = V^T . P^T A = 16 channels x 64 tokens of codes, as loaded; B = the
//                   weights exp2(u - tile max) as 16-bit integers in two planes
//                   (half a step is 2^-16 of the tile's largest).
// The tokens of a tile are assigned to the rows of S^T so that the weights a lane
// gets out of the first product (token 16 g + 4 t + i of query row n, lane 16 g +
// n) are the operand it needs for the second one: nothing moves between lanes.
// The scale of V's page goes into the exponent: u = s log2(e) + log2(aV / 127),
// so pages of any scale share a tile, and the row's sum takes each weight
// without it.
#include <math.h>
#include <algorithm>

#include <type_traits>

#include "kv_common.h"

namespace llmint8 {

namespace {

constexpr float kMinMag = 5.42101086242752217e-20f;  // 2^-64: the least magnitude of a page that is not zero
constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ v4i mfma_i8(const v4i& a, const v4i& b, const v4i& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

// STREAM: codes that nobody reads again (the hint keeps them from lingering in L2)
template <bool STREAM>
__device__ __forceinline__ v4i load16(const int8_t* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(reinterpret_cast<const v4i*>(p));
  return *reinterpret_cast<const v4i*>(p);
}

// over the four lanes that hold one query row (lanes n, n + 16, n + 32, n + 48): the swaps put the
// other half's (the other rows of 16's) values into the second result
__device__ __forceinline__ float swap32(float v, float* other) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  *other = __uint_as_float(r[1]);
  return __uint_as_float(r[0]);
}
__device__ __forceinline__ float swap16(float v, float* other) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  *other = __uint_as_float(r[1]);
  return __uint_as_float(r[0]);
}
__device__ __forceinline__ float row_max(float v) {
  float o;
  v = swap32(v, &o);
  v = swap16(max_or_nan(v, o), &o);
  return max_or_nan(v, o);
}
__device__ __forceinline__ float row_sum(float v) {
  float o;
  v = swap32(v, &o);
  v = swap16(v + o, &o);
  return v + o;
}

__device__ __forceinline__ uint2 pack4(const v4f& v, int bf16) {
  return bf16 ? make_uint2(Act16<true>::pack2(v[0], v[1]), Act16<true>::pack2(v[2], v[3]))
              : make_uint2(Act16<false>::pack2(v[0], v[1]), Act16<false>::pack2(v[2], v[3]));
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

// What a sequence asks of the call: its rows in runs of 16 RT (the query rows of a
// head's group, token by token), and the tiles that any of them sees.
struct SeqWork {
  int runs, tiles;
  Span span;
};
template <int RT>
__device__ __forceinline__ SeqWork seq_work(const KvAttnArgs& a, const KvSeq& s) {
  SeqWork w;
  const int G = a.q_heads / a.c.heads;
  w.runs = (int)(((int64_t)s.n * G + 16 * RT - 1) / (16 * RT));
  w.span = visible_span(s.len, s.pos0, s.pos0 + s.n - 1, a.causal, a.window, a.sinks);
  w.tiles = max(w.span.count(), 1);  // rows that see nothing are written too
  return w;
}

// A part of a run's tiles, the work of one workgroup: the tiles of every run and
// head are cut into equal parts of at most `share` tiles, numbered sequence by
// sequence, head by head, run by run.
struct Part {
  int h, run, part, parts;
  int slot;  // of a part of several: where its result goes
};
// How finely the call is cut. With few runs and heads, about as many parts as run
// at once (a run's last part is half of one on average: cut for that half, 16
// sequences of 1000-8000 tokens take 36.5 us, and 37.7 without it); with more,
// twice that many beyond the runs' own, which evens out runs of different lengths.
// A part of its own costs about 8 us of loads that wait for each other and of
// joining, so none gets less than `least` tiles (16, or 8 of two sixteens: about 9
// us of work), and more where the runs by themselves fill half the chip. Measured
// (32 query and 8 key/value heads of 128, us): 32 sequences of 2000-8000 tokens 73
// (85 cut into one part per resident workgroup, 102 uncut), 64 of 500-8000 94 (119
// uncut), one of 131000 53.
struct Cutting {
  int64_t extra;  // parts beyond one to each run and head
  int least;      // tiles of a part
};
__host__ __device__ inline Cutting cutting(int64_t runs, int slots, int rt) {
  return {runs * 4 <= slots ? slots - runs / 2 : (int64_t)2 * slots, runs * 2 >= slots ? 48 : 16 / rt};
}

// Exclusive sums of two numbers over the workgroup's 256 threads, and their totals.
__device__ __forceinline__ void sum_256(int64_t& x, int64_t& y, int64_t (&sums)[8], int64_t* all_x, int64_t* all_y) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t x0 = x, y0 = y;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t u = __shfl_up(x, o, 64), v = __shfl_up(y, o, 64);
    if (lane >= o) {
      x += u;
      y += v;
    }
  }
  __syncthreads();
  if (lane == 63) {
    sums[wave] = x;
    sums[4 + wave] = y;
  }
  __syncthreads();
  *all_x = *all_y = 0;
  x -= x0;
  y -= y0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (k < wave) {
      x += sums[k];
      y += sums[4 + k];
    }
    *all_x += sums[k];
    *all_y += sums[4 + k];
  }
}

// Part w of the call: the sequences' tiles are summed 256 sequences at a time,
// which gives the share (a.extra parts at most beyond one to each run and head),
// then their parts. False past the last part.
template <int RT>
__device__ __forceinline__ bool find_part(const KvAttnArgs& a, int w, int64_t (&sums)[8], int (&found)[8], KvSeq* seq,
                                          Part* p) {
  const int tid = threadIdx.x, H = a.c.heads;
  int64_t tiles = 0, runs = 0;
  KvSeq q{};
  SeqWork work{};
  for (int b0 = 0; b0 < a.s.B; b0 += 256) {
    q = kv_seq(a.s, a.c.page_shift, min(b0 + tid, a.s.B - 1));
    work = seq_work<RT>(a, q);
    int64_t x = 0, y = b0 + tid < a.s.B ? (int64_t)H * work.runs : 0, all_x, all_y;
    x = y * work.tiles;
    sum_256(x, y, sums, &all_x, &all_y);
    tiles += all_x;
    runs += all_y;
  }
  const Cutting how = cutting(runs, a.slots, RT);
  const int64_t extra = min((int64_t)a.extra, how.extra);
  const int share = (int)max((int64_t)how.least, (tiles + extra - 1) / extra);
  int64_t before = 0, cut = 0;
  if (tid == 0) found[0] = -1;
  for (int b0 = 0; b0 < a.s.B; b0 += 256) {
    if (a.s.B > 256) {
      q = kv_seq(a.s, a.c.page_shift, min(b0 + tid, a.s.B - 1));
      work = seq_work<RT>(a, q);
    }
    const int parts = (work.tiles + share - 1) / share;
    const int64_t mine = b0 + tid < a.s.B ? (int64_t)H * work.runs * parts : 0;
    int64_t x = mine, y = parts > 1 ? mine : 0, all_x, all_y;
    sum_256(x, y, sums, &all_x, &all_y);
    x += before;
    if (x <= w && w < x + mine) {
      const int in = (int)(w - x);
      found[0] = b0 + tid;
      found[1] = q.row0;
      found[2] = q.n;
      found[3] = q.len;
      found[4] = in;
      found[5] = parts;
      found[6] = (int)(y + cut) + in;
      found[7] = q.pos0;
    }
    before += all_x;
    cut += all_y;
  }
  __syncthreads();
  seq->b = uniform(found[0]);
  if (seq->b < 0) return false;
  seq->row0 = uniform(found[1]);
  seq->n = uniform(found[2]);
  seq->len = uniform(found[3]);
  seq->pos0 = uniform(found[7]);
  p->parts = uniform(found[5]);
  p->slot = uniform(found[6]);
  const int in = uniform(found[4]), run = in / p->parts;
  const SeqWork mine = seq_work<RT>(a, *seq);
  p->part = in - run * p->parts;
  p->h = run / mine.runs;
  p->run = run - p->h * mine.runs;
  return true;
}

// A workgroup of four wavefronts takes the tiles of a run of 16 RT rows, NT
// sixteens to a wavefront; those of a sixteen share its tiles, each with its own
// running maximum, sum and output, and join at the end. K's codes of a wavefront's
// next tile are asked for as soon as the first product has read the present ones,
// V's after the second product, into the same registers: a tile is always on the
// way while another is computed, 16 KB of dim 128 for each of two wavefronts to a
// SIMD. That, not the arithmetic (about 0.6 us of a SIMD's time to a tile and
// sixteen), bounds the rate: 5.1 TB/s on one sequence of 131000 tokens, 4.9 on 64 of
// 500-8000.
//
// Two sixteens: NT = 1 gives each two wavefronts, which go over the same tiles at
// about the same time, so that the codes come from memory once; half as many
// different ones are then on the way. NT = 2 takes both in the same wavefronts, one
// after the other between the loads, with q in LDS: more to do before a part's
// first and after its last tile. NT = 2 where the runs fill half the chip. Measured
// (us, NT 1 / 2): 40 sequences of 1000-6000 tokens with 32 rows 83 / 67 (3.9 TB/s),
// 16 of them 39 / 40, one of 1800 17 / 20.
//
// CUT: long runs are cut into parts (find_part); what a part has of its run goes
// to the workspace for kv_join. Otherwise one workgroup to each run and head.
// ONE: a tile is within one page (pages of 64 tokens and more), whose address is
// then scalar. FULL: dim = DP.
template <int DP, bool FULL, bool ONE, bool CUT, int RT, int NT>
__global__ __launch_bounds__(256, DP <= 128 ? 2 : 1) void kv_step(KvAttnArgs a) {
  constexpr int WT = 4 * NT / RT;  // wavefronts that share a sixteen's tiles
  constexpr int NK = (DP + 63) / 64;  // 64-channel steps of the first product
  constexpr bool kWhole = FULL && DP % 64 == 0;  // which are all of them channels of the head
  constexpr int ND = DP / 16;  // 16-channel blocks of the second
  __shared__ float sh_o[NT][2][16][DP];
  __shared__ float sh_ml[NT][4][16][2];
  __shared__ v4i sh_q[NT > 1 ? NT * NK * 2 * 64 : 1];
  __shared__ float sh_unit[NT][16];
  __shared__ int sh_seq[6];
  __shared__ int sh_found[8];
  __shared__ int64_t sh_sums[8];
  const int D = FULL ? DP : a.c.dim;
  const int shift = a.c.page_shift, P = 1 << shift, H = a.c.heads, G = a.q_heads / H;
  const int lane = threadIdx.x & 63, wave = uniform((int)threadIdx.x >> 6);
  const int g = lane >> 4, nn = lane & 15;
  const int64_t page_bytes = (int64_t)P * D;
  // a lane's place in a tile's codes: K row 16 (nn / 4) + nn % 4 (+ 4 j), channels 16 g (+ 64 ks);
  // V channel nn (+ 16 d), tokens 16 g ..
  const int k_tok = 16 * (nn >> 2), v_tok = 16 * g;
  uint32_t k_off[NK], v_off[ND];
#pragma unroll
  for (int ks = 0; ks < NK; ++ks) {
    const int c0 = ks * 64 + g * 16;  // channels past dim: any codes do, q is zero there
    k_off[ks] = (uint32_t)((nn & 3) + (ONE ? k_tok : 0)) * D + (kWhole || c0 < D ? c0 : 0);
  }
#pragma unroll
  for (int d = 0; d < ND; ++d)
    v_off[d] = (uint32_t)((FULL || d * 16 < D ? d * 16 : 0) + nn) * P + (ONE ? v_tok : 0);  // as for K

  KvSeq sq;
  Part p{};
  if (CUT) {
    if (!find_part<RT>(a, blockIdx.x, sh_sums, sh_found, &sq, &p)) return;
  } else {
    int count;
    if (!kv_find<256>(a.s, shift, blockIdx.x / H, G, 3 + RT, sh_seq, &sq, &p.run, &count)) return;
    p.h = (int)(blockIdx.x % H);  // neighbours share a page
    p.parts = 1;
    if (sq.n == 0 || p.run >= seq_work<RT>(a, sq).runs) return;
  }
  const int h = p.h;
  const int b = sq.b, rows = sq.n * G, row_first = p.run * 16 * RT;
  const int sub = wave % WT, six = wave / WT;  // place in the sixteen's wavefronts, and first sixteen
  // row nn of this wavefront's t-th sixteen: its place in q and the outputs, and its position
  struct Row {
    int64_t row;
    int head, pos;
  };
  auto row_of = [&](int t) {
    const int r = min(row_first + 16 * (six + t) + nn, rows - 1), tok = r / G;
    return Row{sq.row0 + tok, h * G + (r - tok * G), sq.pos0 + tok};
  };
  const int pos_lo = sq.pos0 + row_first / G;  // of the run
  const int pos_hi = sq.pos0 + min(row_first + 16 * RT - 1, rows - 1) / G;
  const Span span = CUT ? seq_work<RT>(a, sq).span
                        : visible_span(sq.len, pos_lo, pos_hi, a.causal, a.window, a.sinks);
  int i0 = 0, i1 = span.count();
  if (CUT && p.parts > 1) {
    const int tiles = i1;
    i0 = (int)((int64_t)tiles * p.part / p.parts);
    i1 = (int)((int64_t)tiles * (p.part + 1) / p.parts);
  }

  // the numbers of a tile's pages: of the K rows that the lane loads, of the tokens that it holds
  struct Pages {
    int k, v;
  };
  auto pages_of = [&](int it) {
    const int base = span.tile(it) << 6;
    Pages p;
    if (ONE) {
      p.k = p.v = kv_entry(a.s, b, base >> shift);
    } else {
      p.k = kv_entry(a.s, b, (base + k_tok) >> shift);
      p.v = kv_entry(a.s, b, (base + v_tok) >> shift);
    }
    return p;
  };
  v4i kf[4][NK], vf[ND];
  auto load_k = [&](int it, const Pages& p, float* ak, float* av, int* page) {
    const int base = span.tile(it) << 6;
    const int pk = kv_page(ONE ? uniform(p.k) : p.k, a.c.pages), pv = kv_page(ONE ? uniform(p.v) : p.v, a.c.pages);
    const int8_t* kp = a.c.K + ((int64_t)max(pk, 0) * H + h) * page_bytes +
                       ((ONE ? base : base + k_tok) & (P - 1)) * D;
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int ks = 0; ks < NK; ++ks) kf[j][ks] = load16<NT == RT>(kp + (k_off[ks] + 4 * j * D));
    const int64_t hv = (int64_t)max(pv, 0) * H + h;
    *ak = a.c.aK[hv];
    *av = a.c.aV[hv];
    *page = pv;
  };
  auto load_v = [&](int it, const Pages& p) {
    const int base = span.tile(it) << 6;
    const int pv = kv_page(ONE ? uniform(p.v) : p.v, a.c.pages);
    const int8_t* vp = a.c.V + ((int64_t)max(pv, 0) * H + h) * page_bytes + ((ONE ? base : base + v_tok) & (P - 1));
#pragma unroll
    for (int d = 0; d < ND; ++d) vf[d] = load16<NT == RT>(vp + v_off[d]);
  };

  int it = row_first + 16 * six < rows ? i0 + sub : i1, page = -1;
  float ak = 0.0f, av = 0.0f;
  Pages next{-1, -1};

  // q: 16-bit integers in two planes, and what one unit of S stands for. One sixteen's stay in registers; of
  // two each is prepared by one wavefront and read from LDS by all.
  v4i qhi[NK], qlo[NK];
  float unit[NT];
  {
    const Row mine = row_of(wave % NT);
    uint32_t w[NK][8];
    {
      const uint16_t* qp = a.q.p + mine.row * a.q.token + (int64_t)mine.head * a.q.head;
#pragma unroll
      for (int ks = 0; ks < NK; ++ks) {
        const int c0 = ks * 64 + g * 16;
        uint4 x = make_uint4(0, 0, 0, 0), y = x;
        if (kWhole || c0 < D) {
          x = *reinterpret_cast<const uint4*>(qp + c0);
          y = *reinterpret_cast<const uint4*>(qp + c0 + 8);
        }
        w[ks][0] = x.x, w[ks][1] = x.y, w[ks][2] = x.z, w[ks][3] = x.w;
        w[ks][4] = y.x, w[ks][5] = y.y, w[ks][6] = y.z, w[ks][7] = y.w;
      }
    }
    if (it < i1) {
      const Pages p = pages_of(it);
      next = pages_of(min(it + WT, i1 - 1));
      load_k(it, p, &ak, &av, &page);
      load_v(it, p);
    }
    {
      float f[NK][16], m = 0.0f;
      if (a.bf16) {
#pragma unroll
        for (int ks = 0; ks < NK; ++ks)
#pragma unroll
          for (int j = 0; j < 16; ++j) f[ks][j] = bf16_bits_to_float((w[ks][j >> 1] >> (16 * (j & 1))) & 0xffffu);
      } else {
#pragma unroll
        for (int ks = 0; ks < NK; ++ks)
#pragma unroll
          for (int j = 0; j < 16; ++j) f[ks][j] = half_bits_to_float((w[ks][j >> 1] >> (16 * (j & 1))) & 0xffffu);
      }
#pragma unroll
      for (int ks = 0; ks < NK; ++ks)
#pragma unroll
        for (int j = 0; j < 16; ++j) m = max_or_nan(m, fabsf(f[ks][j]));
      m = row_max(m);
      const float sc = m > 0.0f ? 32639.0f / m : 0.0f;
      unit[0] = m * (1.0f / 32639.0f) * a.scale * 1.44269504088896341f * (1.0f / 127.0f);
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
  }

  if constexpr (NT > 1) {
    if (wave < NT) {
#pragma unroll
      for (int ks = 0; ks < NK; ++ks) {
        sh_q[((wave * NK + ks) * 2) * 64 + lane] = qhi[ks];
        sh_q[((wave * NK + ks) * 2 + 1) * 64 + lane] = qlo[ks];
      }
      if (g == 0) sh_unit[wave][nn] = unit[0];
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < NT; ++t) unit[t] = sh_unit[t][nn];
  }
  auto q_plane = [&](int t, int ks, int lo) {
    if constexpr (NT > 1) return sh_q[((t * NK + ks) * 2 + lo) * 64 + lane];
    return lo ? qlo[ks] : qhi[ks];
  };

  v4f acc[NT][ND];
  float m_run[NT], l_run[NT];
  int pos[NT], last[NT];  // last: the last token that a row sees, but for its window; < 0: none
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int d = 0; d < ND; ++d) acc[t][d] = v4f{0, 0, 0, 0};
    m_run[t] = kNegInf;
    l_run[t] = 0.0f;
    pos[t] = row_of(t).pos;
    last[t] = a.causal ? min(pos[t], sq.len - 1) : sq.len - 1;
  }
  const int all_end = a.causal ? min(pos_lo, sq.len - 1) : sq.len - 1;  // seen by every row, up to its window
  const int all_begin = a.window > 0 ? pos_hi - a.window + 1 : 0;

  auto tile = [&](auto more) {
    constexpr bool MORE = decltype(more)::value;
    const int base = span.tile(it) << 6;
    // The page numbers of the tile after next go out before the next tile's codes: loads
    // complete in order, and a wait for them must not be one for these.
    Pages after{-1, -1};
    if (MORE) after = pages_of(min(it + 2 * WT, i1 - 1));
    // S in units of q's and the page's scales
    const float akh = ak;
    // a page of zeros takes the smallest scale there is: its weights only enter the row's sum, and
    // must not set the scale of the others'
    const float vs = (av < kMinMag ? kMinMag : av) * (1.0f / 127.0f);
    const float lv = __builtin_amdgcn_logf(vs);  // log2
    v4i s[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[t][j] = v4i{0, 0, 0, 0};
#pragma unroll
        for (int ks = 0; ks < NK; ++ks) s[t][j] = mfma_i8(kf[j][ks], q_plane(t, ks, 0), s[t][j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) s[t][j][i] <<= 8;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int ks = 0; ks < NK; ++ks) s[t][j] = mfma_i8(kf[j][ks], q_plane(t, ks, 1), s[t][j]);
    }
    const int here = page;
    if (MORE) load_k(it + WT, next, &ak, &av, &page);
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (t > 0 && row_first + 16 * t >= rows) break;  // t > 0: six is 0
      if (NT > 1) __builtin_amdgcn_sched_barrier(0);
      float u[16];
      const float fk = unit[t] * akh;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) u[4 * j + i] = __builtin_fmaf((float)s[t][j][i], fk, lv);
      // what a row does not see; tiles inside every row's range need no look at single tokens
      if (base + 63 > all_end || base < all_begin || (ONE ? here < 0 : __any(here < 0))) {
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int x = base + v_tok + j;
          const bool see = here >= 0 && x <= last[t] && (a.window <= 0 || x > pos[t] - a.window || x < a.sinks);
          u[j] = see ? u[j] : kNegInf;
        }
      }
      float mt = u[0];
#pragma unroll
      for (int j = 1; j < 16; ++j) mt = fmaxf(mt, u[j]);
      mt = row_max(mt);
      const float mt0 = mt == kNegInf ? 0.0f : mt;
      if (__any(mt > m_run[t])) {  // a new maximum of some row: what was summed moves to it
        const float m_new = fmaxf(m_run[t], mt);
        const float alpha = m_run[t] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(m_run[t] - m_new);
        m_run[t] = m_new;
        l_run[t] *= alpha;
#pragma unroll
        for (int d = 0; d < ND; ++d) acc[t][d] *= alpha;
      }
      const float beta = mt == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(mt - m_run[t]);
      float sum = 0.0f;
      uint32_t w[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float e = __builtin_amdgcn_exp2f(u[j] - mt0);
        sum += e;
        // rne(32639 e) + 128 in the low 16 bits: high plane, and low plane + 128
        w[j] = __float_as_uint(__builtin_fmaf(e, 32639.0f, 12582912.0f + 128.0f));
      }
      sum *= beta;
      // a page that the row does not see may have any magnitude
      l_run[t] = sum == 0.0f ? l_run[t] : __builtin_fmaf(sum, __builtin_amdgcn_rcpf(vs), l_run[t]);
      v4i phi, plo;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t h01 = __builtin_amdgcn_perm(w[4 * j + 1], w[4 * j], 0x0c0c0501u);
        const uint32_t h23 = __builtin_amdgcn_perm(w[4 * j + 3], w[4 * j + 2], 0x0c0c0501u);
        const uint32_t l01 = __builtin_amdgcn_perm(w[4 * j + 1], w[4 * j], 0x0c0c0400u);
        const uint32_t l23 = __builtin_amdgcn_perm(w[4 * j + 3], w[4 * j + 2], 0x0c0c0400u);
        phi[j] = (int)__builtin_amdgcn_perm(h23, h01, 0x05040100u);
        plo[j] = (int)(__builtin_amdgcn_perm(l23, l01, 0x05040100u) ^ 0x80808080u);
      }
      const float bu = beta * (1.0f / 32639.0f);
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        v4i o = mfma_i8(vf[d], phi, v4i{0, 0, 0, 0});
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] <<= 8;
        o = mfma_i8(vf[d], plo, o);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[t][d][i] = __builtin_fmaf((float)o[i], bu, acc[t][d][i]);
        if (NT > 1 && d % 4 == 3) __builtin_amdgcn_sched_barrier(0);  // or the products' results take the registers
      }
    }
    if (MORE) load_v(it + WT, next);
    next = after;
  };
  // the last tile stands alone, so that the loop's loads are unconditional and its waits exact
  if (it < i1) {
    for (; it + WT < i1; it += WT) tile(std::true_type{});
    tile(std::false_type{});
  }

  // join a sixteen's wavefronts
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    l_run[t] = row_sum(l_run[t]);
    if (g == 0) {
      sh_ml[t][wave][nn][0] = m_run[t];
      sh_ml[t][wave][nn][1] = l_run[t];
    }
  }
  __syncthreads();
  auto give = [&](int t, int to) {
#pragma unroll
    for (int d = 0; d < ND; ++d) *reinterpret_cast<v4f*>(&sh_o[t][to][nn][d * 16 + 4 * g]) = acc[t][d];
  };
  auto take = [&](int t, int from) {
#pragma unroll
    for (int d = 0; d < ND; ++d) acc[t][d] += *reinterpret_cast<const v4f*>(&sh_o[t][from][nn][d * 16 + 4 * g]);
  };
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    float m_all = m_run[t];
#pragma unroll
    for (int w = 0; w < WT; ++w) m_all = fmaxf(m_all, sh_ml[t][six * WT + w][nn][0]);
    const float m0 = m_all == kNegInf ? 0.0f : m_all;
    const float mine = __builtin_amdgcn_exp2f(m_run[t] - m0);
    m_run[t] = m_all;
    l_run[t] = 0.0f;
#pragma unroll
    for (int w = 0; w < WT; ++w)
      l_run[t] += sh_ml[t][six * WT + w][nn][1] * __builtin_amdgcn_exp2f(sh_ml[t][six * WT + w][nn][0] - m0);
#pragma unroll
    for (int d = 0; d < ND; ++d) acc[t][d] *= mine;
    if (sub >= WT / 2) give(t, WT == 4 ? sub - 2 : six);
  }
  __syncthreads();
  if (WT == 4) {  // halves to halves, then wavefront t ends with sixteen t
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      if (sub >= 2) break;
      take(t, sub);
      if (sub != t) give(t, sub);  // where it read from itself
    }
    __syncthreads();
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int row_mine = row_first + 16 * (six + t);
    if (sub != t || row_mine >= rows) continue;
    take(t, WT == 4 ? 1 - sub : six);
    const Row r = row_of(t);
    const bool in = row_mine + nn < rows;
    // which parts there are of a row, for the join
    if (CUT && p.part == 0 && g == 0 && in)
      *reinterpret_cast<v2i*>(a.notes + (r.row * a.q_heads + r.head) * 2) =
          v2i{p.parts > 1 ? (p.slot << kKvNoteShift | 16 * (six + t) | nn) : -1, p.parts};
    if (CUT && p.parts > 1) {
      const int64_t to = (int64_t)p.slot * (16 * RT) + 16 * (six + t) + nn;
      if (g == 0) *reinterpret_cast<v2f*>(a.part_ml + to * 2) = v2f{m_run[t], l_run[t]};
#pragma unroll
      for (int d = 0; d < ND; ++d)
        if (FULL || d * 16 < D) *reinterpret_cast<v4f*>(a.part_o + to * D + d * 16 + 4 * g) = acc[t][d];
    } else if (in) {
      const float inv = l_run[t] == 0.0f ? 0.0f : 1.0f / l_run[t];
      uint16_t* op = a.o.p + r.row * a.o.token + (int64_t)r.head * a.o.head;
#pragma unroll
      for (int d = 0; d < ND; ++d)
        if (FULL || d * 16 < D) *reinterpret_cast<uint2*>(op + d * 16 + 4 * g) = pack4(acc[t][d] * inv, a.bf16);
      if (a.lse && g == 0)
        a.lse[r.row * a.q_heads + r.head] =
            l_run[t] == 0.0f ? kNegInf : (m_run[t] + log2f(l_run[t])) * 0.693147180559945309f;
    }
  }
}

// Joins the parts of the rows that have several, ROWS rows to a workgroup:
// groups of lanes that hold a row's channels four by four take every (256 / ROWS
// / group)-th part, four parts to a round of loads. A launch and two loads that
// wait for each other: 4.6 us for 32 rows of 64 parts. Up to 2048 rows each has a
// workgroup, as parts may be many; more share one by four: 3200 rows 6.9 us one to
// a workgroup, 4.8 by four, 12800 rows 9.5 and 5.2 (2048: 4.6 both).
template <int ROWS>
__global__ __launch_bounds__(256) void kv_join(KvAttnArgs a) {
  constexpr int kLanes = 256 / ROWS;
  __shared__ v4f sh_o[256];
  __shared__ float sh_ml[256][2];
  const int D = a.c.dim, per = D >> 2, groups = kLanes / per;
  const int tid = threadIdx.x % kLanes, first = threadIdx.x - tid;
  const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / kLanes;
  const int t = (int)(row / a.q_heads);
  // rows outside the batch have no note
  const bool in = t >= max(a.s.cu[0], 0) && t < min(a.s.cu[a.s.B], a.s.T);
  // read beside cu, not after it
  v2i note = *reinterpret_cast<const v2i*>(a.notes + min(row, (int64_t)a.s.T * a.q_heads - 1) * 2);
  if (!in) note = v2i{-1, 0};
  const KvNote of = kv_note(note[0], note[1], a.run, a.max_parts);
  const int slot = of.slot, nn = of.place, parts = of.parts;
  if (ROWS == 1 && parts == 0) return;
  const int64_t qrow = t;
  const int qh = (int)(row - (int64_t)t * a.q_heads);
  const int grp = tid / per, c = tid - grp * per;
  float m = kNegInf, l = 0.0f;
  v4f o = {0, 0, 0, 0};
  if (grp < groups)
    for (int p0 = grp; p0 < parts; p0 += 4 * groups) {
      v2f ml[4];
      v4f x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int p = min(p0 + k * groups, parts - 1);
        const int64_t from = (int64_t)(slot + p) * a.run + nn;
        ml[k] = *reinterpret_cast<const v2f*>(a.part_ml + from * 2);
        x[k] = *reinterpret_cast<const v4f*>(a.part_o + from * D + c * 4);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const bool mine = p0 + k * groups < parts;
        const float mk = mine ? ml[k][0] : kNegInf;
        const float top = fmaxf(m, mk), ref = top == kNegInf ? 0.0f : top;
        const float keep = __builtin_amdgcn_exp2f(m - ref), add = __builtin_amdgcn_exp2f(mk - ref);
        m = top;
        l = l * keep + ml[k][1] * add;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = o[i] * keep + x[k][i] * add;
      }
    }
  sh_o[first + tid] = o;
  sh_ml[first + tid][0] = m;
  sh_ml[first + tid][1] = l;
  __syncthreads();
  if (tid >= per || parts == 0) return;
  float top = m;
  for (int s = 1; s < groups; ++s) top = fmaxf(top, sh_ml[first + s * per + tid][0]);
  const float ref = top == kNegInf ? 0.0f : top;
  const float keep = __builtin_amdgcn_exp2f(m - ref);
  l *= keep;
  o *= keep;
  for (int s = 1; s < groups; ++s) {
    const float add = __builtin_amdgcn_exp2f(sh_ml[first + s * per + tid][0] - ref);
    l += sh_ml[first + s * per + tid][1] * add;
    const v4f x = sh_o[first + s * per + tid];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] += x[i] * add;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  *reinterpret_cast<uint2*>(a.o.p + qrow * a.o.token + (int64_t)qh * a.o.head + tid * 4) = pack4(o * inv, a.bf16);
  if (a.lse && tid == 0) a.lse[row] = l == 0.0f ? kNegInf : (top + log2f(l)) * 0.693147180559945309f;
}

// Rows of a run: a sequence's rows together if they fit, so that its codes are
// read once.
int kv_attention_run(const KvBatch& s, int heads, int q_heads) {
  const int64_t rows = (int64_t)s.T * (q_heads / heads), per = (rows + s.B - 1) / s.B;
  return per <= 16 ? 16 : 32;
}

// Whether a call's sequences have rows enough, on average, for kv_prompt (one
// kernel for all of a call: a prompt of 512 tokens with 64 single ones of 500-8000
// takes 253 us in one call, 115 and 19 in two; with a prompt of 400 131, 115 and
// 16): more than
// the 32 of a run of kv_step, which would read the codes again for the next ones.
// Measured, 16 sequences of 1000-6000 tokens (us, kv_step / kv_prompt): 20 rows
// 40 / 56, 32 rows 40 / 57, 80 rows (3000-6000) 127 / 79; 64 of 500-4000 with 64
// rows 282 / 129.
bool kv_attention_prompt(const KvBatch& s, int heads, int q_heads) {
  return (int64_t)s.T * (q_heads / heads) > (int64_t)32 * s.B;
}

static int64_t runs_about(const KvBatch& s, int heads, int q_heads) {
  return std::max<int64_t>(s.B, (int64_t)s.T * (q_heads / heads) / kv_attention_run(s, heads, q_heads)) * heads;
}
static int64_t runs_at_most(const KvBatch& s, int heads, int q_heads) {
  return (int64_t)s.T * (q_heads / heads) / kv_attention_run(s, heads, q_heads) + s.B;
}

// Whether a call's runs are cut into parts, and how many more workgroups that
// takes at most. 0: not cut, where the longest context (twice, for runs of two
// sixteens) is no more than 4096 tokens, or, with fewer runs than a quarter of
// what the chip holds, than 2304 over the share of the chip that they leave idle:
// there the join costs more than the cut gains. Measured, us uncut / cut: one
// sequence of 2000 tokens 19 / 24; 16 of 2000-3000 29 / 28 and of 2000-4000 36 /
// 29; 24 of 2000-4000 37 / 42; 64 of 1000-2000 41 / 56. *slots: workgroups that
// are taken to run at once, three, two or one to a CU: what the registers of the
// head size's largest forms leave room for. One sixteen of whole heads of 64 or 96
// would leave room for four and three; what the rule would make of that is not
// measured.
int kv_attention_extra(const KvBatch& s, int heads, int q_heads, int dim, int64_t max_span, int num_cus, int* slots) {
  *slots = num_cus * (dim <= 64 ? 3 : dim <= 128 ? 2 : 1);
  const int64_t runs = runs_about(s, heads, q_heads);
  const int rt = kv_attention_run(s, heads, q_heads) / 16;
  if (max_span * rt <= (runs * 4 > *slots ? 4096 : 2304 * *slots / (*slots - runs))) return 0;
  const int64_t tiles = (max_span + 63) / 64, least = cutting(1, *slots, rt).least, most = (tiles + least - 1) / least - 1;
  return (int)std::min<int64_t>(2 * *slots, most * runs_at_most(s, heads, q_heads) * heads);
}

template <int DP, bool FULL, bool ONE, int RT, int NT>
static hipError_t launch_runs(const KvAttnArgs& a, hipStream_t stream) {
  const int64_t blocks = runs_at_most(a.s, a.c.heads, a.q_heads) * a.c.heads + a.extra;
  if (blocks > INT32_MAX) return hipErrorInvalidConfiguration;
  if (a.extra > 0)
    hipLaunchKernelGGL((kv_step<DP, FULL, ONE, true, RT, NT>), dim3((unsigned)blocks), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((kv_step<DP, FULL, ONE, false, RT, NT>), dim3((unsigned)blocks), dim3(256), 0, stream, a);
  return hipGetLastError();
}

template <int DP, bool FULL, bool ONE>
static hipError_t launch_pages(const KvAttnArgs& a, hipStream_t stream) {
  if (a.run == 16) return launch_runs<DP, FULL, ONE, 1, 1>(a, stream);
  if (runs_about(a.s, a.c.heads, a.q_heads) * 2 >= a.slots) return launch_runs<DP, FULL, ONE, 2, 2>(a, stream);
  return launch_runs<DP, FULL, ONE, 2, 1>(a, stream);
}

template <int DP, bool FULL>
static hipError_t launch_step(const KvAttnArgs& a, hipStream_t stream) {
  return a.c.page_shift >= 6 ? launch_pages<DP, FULL, true>(a, stream) : launch_pages<DP, FULL, false>(a, stream);
}

static hipError_t launch_kv_step(const KvAttnArgs& a, hipStream_t stream) {
  if (a.c.dim == 64) return launch_step<64, true>(a, stream);
  if (a.c.dim < 64) return launch_step<64, false>(a, stream);
  if (a.c.dim < 96) return launch_step<96, false>(a, stream);
  if (a.c.dim == 96) return launch_step<96, true>(a, stream);
  if (a.c.dim == 112) return launch_step<112, true>(a, stream);
  if (a.c.dim == 128) return launch_step<128, true>(a, stream);
  return launch_step<256, false>(a, stream);
}

hipError_t launch_kv_attention(const KvAttnArgs& a, hipStream_t stream) {
  const hipError_t e = a.prompt ? launch_kv_prompt(a, stream) : launch_kv_step(a, stream);
  if (e != hipSuccess || a.max_parts == 0) return e;
  const int64_t rows = (int64_t)a.s.T * a.q_heads;
  if (a.c.dim > 128 || rows <= 2048)
    hipLaunchKernelGGL(kv_join<1>, dim3((unsigned)rows), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL(kv_join<4>, dim3((unsigned)((rows + 3) / 4)), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace llmint8
