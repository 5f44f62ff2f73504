// Rotary positions with several axes on gfx950: pair i of a head's first `rot`
// channels turns by the angle that the table holds for the row's position on the
// axis of that pair; with sign = -1 back, which is the gradient.
//   y1 = x1 c - x2 s, y2 = x2 c + x1 s, each product and sum rounded to fp32
//
// A thread takes eight pairs of a row and HPT heads, which share their cosines and
// sines. Bound by memory: read once, written once. 16000 tokens of 32/8 heads of 128 in 75 us,
// 4.4 TB/s of the 5.2 that a large copy reaches. A thread's heads come one after
// the other: a forward and a backward pass take 150 us so, 167 with all loads before the first
// store (141 registers, three wavefronts to a SIMD), 155 with its neighbours' heads between its.
#include <type_traits>

#include "train_common.h"

namespace llmint8 {

template <bool BF16, bool INTERLEAVED, int HPT>
__global__ __launch_bounds__(256) void kr_rope(RopeArgs a) {
  using E = Elem<BF16 ? kBF16 : kF16>;
  const int pairs = a.rot / 2, turning = (pairs + 7) / 8;
  const int chunks = turning + (a.copy ? (a.dim - a.rot + 7) / 8 : 0);
  const int heads = a.heads[0] + a.heads[1], groups = (heads + HPT - 1) / HPT;
  const int64_t item = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = item / (chunks * groups);
  if (row >= a.rows) return;
  const int rest = (int)(item - row * (chunks * groups)), group = rest / chunks, chunk = rest - group * chunks;
  auto rows_of = [&](const KvRows (&r)[2], int h) {
    const int second = h >= a.heads[0];
    return r[second].p + row * r[second].token + (int64_t)(second ? h - a.heads[0] : h) * r[second].head;
  };
  if (chunk >= turning) {
    const int at = a.rot + (chunk - turning) * 8;
#pragma unroll
    for (int i = 0; i < HPT; ++i) {
      const int h = group * HPT + i;
      if (h < heads) E::store(rows_of(a.y, h), at, a.dim, E::wide(E::load(rows_of(a.x, h), at, a.dim)));
    }
    return;
  }
  const int p0 = chunk * 8;
  v8f c, s;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int p = min(p0 + j, pairs - 1);
    const int at = min(max(a.pos[row * a.axes + a.axis[p]], 0), a.table_rows - 1);
    const float* t = a.table + (int64_t)at * a.rot + p;
    c[j] = t[0];
    s[j] = t[pairs] * a.sign;
  }
#pragma unroll
  for (int i = 0; i < HPT; ++i) {
    const int h = group * HPT + i;
    if (h >= heads) break;
    const uint16_t* x = rows_of(a.x, h);
    uint16_t* y = rows_of(a.y, h);
    // INTERLEAVED: pairs side by side, sixteen channels from 2 p0 on; otherwise half a rotation apart
    const int at1 = INTERLEAVED ? 2 * p0 : p0, at2 = INTERLEAVED ? 2 * p0 + 8 : pairs + p0;
    const int end1 = INTERLEAVED ? a.rot : pairs;
    const v8f u = E::wide(E::load(x, at1, end1)), v = E::wide(E::load(x, at2, a.rot));
    v8f p, q;
    if constexpr (INTERLEAVED) {
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        p[j] = u[j] * c[j / 2] - u[j + 1] * s[j / 2];
        p[j + 1] = u[j + 1] * c[j / 2] + u[j] * s[j / 2];
        q[j] = v[j] * c[4 + j / 2] - v[j + 1] * s[4 + j / 2];
        q[j + 1] = v[j + 1] * c[4 + j / 2] + v[j] * s[4 + j / 2];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        p[j] = u[j] * c[j] - v[j] * s[j];
        q[j] = v[j] * c[j] + u[j] * s[j];
      }
    }
    E::store(y, at1, end1, p);
    E::store(y, at2, a.rot, q);
  }
}

template <bool BF16, bool INTERLEAVED>
static hipError_t launch(const RopeArgs& a, int num_cus, hipStream_t stream) {
  const int64_t chunks = (a.rot / 2 + 7) / 8 + (a.copy ? (a.dim - a.rot + 7) / 8 : 0);
  const int heads = a.heads[0] + a.heads[1];
  auto blocks = [&](int per) { return (a.rows * chunks * ((heads + per - 1) / per) + 255) / 256; };
  // eight heads to a thread where that leaves four workgroups to a CU (16000 tokens forward and
  // back: 154 us, one head 273), else one (a single token: 3.4 us, eight heads 6.0)
  const bool many = blocks(8) >= 4 * num_cus;
  const int64_t items = chunks * (many ? (heads + 7) / 8 : heads);
  return launch_rows(a.rows, items, 256, [&](int64_t at, int64_t n) {
    const dim3 grid((unsigned)((n * items + 255) / 256));
    if (many) hipLaunchKernelGGL((kr_rope<BF16, INTERLEAVED, 8>), grid, dim3(256), 0, stream, rope_rows_of(a, at, n));
    else hipLaunchKernelGGL((kr_rope<BF16, INTERLEAVED, 1>), grid, dim3(256), 0, stream, rope_rows_of(a, at, n));
    return hipGetLastError();
  });
}

hipError_t launch_rope(const RopeArgs& a, bool bf16, int num_cus, hipStream_t stream) {
  if (bf16) return a.interleaved ? launch<true, true>(a, num_cus, stream) : launch<true, false>(a, num_cus, stream);
  return a.interleaved ? launch<false, true>(a, num_cus, stream) : launch<false, false>(a, num_cus, stream);
}

}  // namespace llmint8
