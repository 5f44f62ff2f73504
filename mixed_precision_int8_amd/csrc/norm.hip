// Layer norm on gfx950, forward and backward:
//   xh = (x - mean) rstd, rstd = 1 / sqrt(mean((x - mean)^2) + eps), y = xh w + b
//   g = dy w, dx = rstd (g - mean(g) - xh mean(g xh)), dw = sum dy xh, db = sum dy
//
// L lanes take a row, two vectors of eight channels each (eight where a row has more
// than 16384), and hold it in registers: read once; the mean is taken before the
// squares of what is left. Statistics and sums are fp32.
//
// Backward, a workgroup goes over rows `groups` apart and keeps its columns' sums for
// dw and db in registers; at the end its row groups add theirs in LDS, one after the
// other, and the workgroups' sums are added by a second launch, in order: no atomics.
// Rows wider than 8192 channels read x and dy once more for the columns' sums, as the
// registers do not hold them.
//
// Bound by memory where rows fill their lanes: 8190 rows of 4096 in bf16 take 33 us forward (4.0 TB/s)
// and 37 backward right after it (5.4 TB/s, part of it from the caches), and 4.8 the second launch;
// backward alone is 47 with that. A row has 64 lanes at least, 16 channels to a lane: narrow ones leave
// most of them idle (500000 rows of 64 in fp16: 201 us forward, 0.6 TB/s, and 631 backward, 0.3 TB/s).
#include <algorithm>
#include <type_traits>

#include "train_common.h"

namespace llmint8 {

namespace {

// Sum of N values over the L lanes of each row group of a workgroup of TH threads. `sh`
// may be written again after the next barrier.
template <int L, int N, int TH>
__device__ __forceinline__ void row_sum(float (&v)[N], float (&sh)[N][TH / 64]) {
#pragma unroll
  for (int i = 0; i < N; ++i) v[i] = wave_sum(v[i]);
  if constexpr (L > 64) {
    constexpr int kWaves = L / 64;
    const int wave = threadIdx.x >> 6, first = wave / kWaves * kWaves;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int i = 0; i < N; ++i) sh[i][wave] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      v[i] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v[i] += sh[i][first + w];
    }
  }
}

template <int TYPE>
__device__ __forceinline__ v8f values(const void* p, int at, int K) {
  return Elem<TYPE>::wide(Elem<TYPE>::load(p, at, K));
}

}  // namespace

template <int TYPE, int WTYPE, int L, int NV>
__global__ __launch_bounds__(L > 256 ? L : 256) void kn_forward(NormArgs a) {
  constexpr int TH = L > 256 ? L : 256, R = TH / L;
  using E = Elem<TYPE>;
  __shared__ float sh[2][1][TH / 64];
  const int lane = threadIdx.x % L;
  const int64_t want = (int64_t)blockIdx.x * R + threadIdx.x / L;
  const int64_t row = std::min(want, a.rows - 1);
  const int K = a.K;
  const char* x = static_cast<const char*>(a.x) + row * a.x_row * E::kBytes;
  v8f v[NV];
  float s[1] = {0.0f};
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = values<TYPE>(x, (i * L + lane) * 8, K);
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) s[0] += v[i][j];
  row_sum<L, 1, TH>(s, sh[0]);
  const float mean = s[0] / (float)K;
  s[0] = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      v[i][j] -= mean;
      if ((i * L + lane) * 8 + j < K) s[0] = __builtin_fmaf(v[i][j], v[i][j], s[0]);
    }
  row_sum<L, 1, TH>(s, sh[1]);
  const float rstd = 1.0f / sqrtf(s[0] / (float)K + a.eps);
  if (want != row) return;
  if (a.stats && lane == 0) {
    a.stats[row * 2] = mean;
    a.stats[row * 2 + 1] = rstd;
  }
  char* y = static_cast<char*>(a.y) + row * a.y_row * E::kBytes;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (i * L + lane) * 8;
    if (at >= K) continue;
    v[i] *= rstd;
    if (a.w) v[i] *= values<WTYPE>(a.w, at, K);
    if (a.b) v[i] += values<WTYPE>(a.b, at, K);
    E::store(y, at, K, v[i]);
  }
}

// SUMS: dw and db too.
template <int TYPE, int WTYPE, int L, int NV, bool SUMS>
__global__ __launch_bounds__(512) void kn_backward(NormArgs a) {
  constexpr int TH = 512, R = TH / L;
  using E = Elem<TYPE>;
  __shared__ float sh[2][2][TH / 64];
  __shared__ __attribute__((aligned(32))) float cols[SUMS && R > 1 ? L * NV * 8 : 1];
  const int lane = threadIdx.x % L, group = threadIdx.x / L;
  const int K = a.K;
  v8f dw[SUMS ? NV : 1], db[SUMS ? NV : 1], w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int at = (i * L + lane) * 8;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      w[i][j] = 1.0f;
      if constexpr (SUMS) dw[i][j] = db[i][j] = 0.0f;
    }
    if (a.w) w[i] = values<WTYPE>(a.w, at, K);
  }
  const int64_t step = (int64_t)gridDim.x * R;
  typename E::Raw rx[NV], rg[NV];
  float mean = 0.0f, rstd = 0.0f;
  auto load = [&](int64_t row) {
    const int64_t at = std::min(row, a.rows - 1);
    const char* x = static_cast<const char*>(a.x) + at * a.x_row * E::kBytes;
    const char* g = static_cast<const char*>(a.dy) + at * a.dy_row * E::kBytes;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      rx[i] = E::load(x, (i * L + lane) * 8, K);
      rg[i] = E::load(g, (i * L + lane) * 8, K);
    }
    mean = a.stats[at * 2];
    rstd = a.stats[at * 2 + 1];
  };
  int64_t row = (int64_t)blockIdx.x * R + group;
  load(row);
  int turn = 0;
  for (int64_t first = (int64_t)blockIdx.x * R; first < a.rows; first += step, row += step, turn ^= 1) {
    const bool mine = row < a.rows;
    v8f xh[NV], g[NV];
    float s[2] = {0.0f, 0.0f};
    const float r = rstd;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = (i * L + lane) * 8;
      xh[i] = E::wide(rx[i]);
      g[i] = E::wide(rg[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        xh[i][j] = at + j < K ? (xh[i][j] - mean) * r : 0.0f;
        if constexpr (SUMS) {
          if (mine) {
            dw[i][j] = __builtin_fmaf(g[i][j], xh[i][j], dw[i][j]);
            db[i][j] += g[i][j];
          }
        }
        g[i][j] *= w[i][j];
        s[0] += g[i][j];
        s[1] = __builtin_fmaf(g[i][j], xh[i][j], s[1]);
      }
    }
    if (first + step < a.rows) load(row + step);
    row_sum<L, 2, TH>(s, sh[turn]);
    const float c0 = s[0] / (float)K, c1 = s[1] / (float)K;
    if (mine) {
      char* dx = static_cast<char*>(a.y) + row * a.y_row * E::kBytes;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int at = (i * L + lane) * 8;
        if (at >= K) continue;
        v8f d;
#pragma unroll
        for (int j = 0; j < 8; ++j) d[j] = (g[i][j] - c0 - xh[i][j] * c1) * r;
        E::store(dx, at, K, d);
      }
    }
  }
  if constexpr (SUMS) {
    float* to = a.parts + (int64_t)blockIdx.x * 2 * K;
    for (int which = 0; which < 2; ++which, to += K) {
      v8f(&sum)[NV] = which ? db : dw;
      if constexpr (R > 1) {
        // the last row group's sums pass through all before it
        for (int from = R - 1; from >= 0; --from) {
          if (group == from) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
              v8f* c = reinterpret_cast<v8f*>(cols + (i * L + lane) * 8);
              if (from < R - 1) sum[i] += *c;
              *c = sum[i];
            }
          }
          __syncthreads();
        }
      }
      if (group == 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) Elem<kF32>::store(to, (i * L + lane) * 8, K, sum[i]);
      }
    }
  }
}

// dx of rows too wide for kn_backward's registers: a workgroup takes a row and reads it
// twice, the second time from the caches.
template <int TYPE, int WTYPE>
__global__ __launch_bounds__(1024) void kn_wide(NormArgs a) {
  using E = Elem<TYPE>;
  __shared__ float sh[2][16];
  const int K = a.K;
  const int64_t row = blockIdx.x;
  const char* x = static_cast<const char*>(a.x) + row * a.x_row * E::kBytes;
  const char* g = static_cast<const char*>(a.dy) + row * a.dy_row * E::kBytes;
  char* dx = static_cast<char*>(a.y) + row * a.y_row * E::kBytes;
  const float mean = a.stats[row * 2], rstd = a.stats[row * 2 + 1];
  auto take = [&](int at, v8f* xh, v8f* gw) {
    *xh = values<TYPE>(x, at, K);
    *gw = values<TYPE>(g, at, K);
    if (a.w) *gw *= values<WTYPE>(a.w, at, K);
#pragma unroll
    for (int j = 0; j < 8; ++j) (*xh)[j] = at + j < K ? ((*xh)[j] - mean) * rstd : 0.0f;
  };
  float s[2] = {0.0f, 0.0f};
  for (int at = threadIdx.x * 8; at < K; at += 8192) {
    v8f xh, gw;
    take(at, &xh, &gw);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s[0] += gw[j];
      s[1] = __builtin_fmaf(gw[j], xh[j], s[1]);
    }
  }
  row_sum<1024, 2, 1024>(s, sh);
  const float c0 = s[0] / (float)K, c1 = s[1] / (float)K;
  for (int at = threadIdx.x * 8; at < K; at += 8192) {
    v8f xh, gw;
    take(at, &xh, &gw);
#pragma unroll
    for (int j = 0; j < 8; ++j) gw[j] = (gw[j] - c0 - xh[j] * c1) * rstd;
    E::store(dx, at, K, gw);
  }
}

// The columns' sums of rows too wide for kn_backward's registers: a thread takes eight
// columns, a workgroup the rows blockIdx.y, + gridDim.y, ...
template <int TYPE>
__global__ __launch_bounds__(256) void kn_columns(NormArgs a) {
  using E = Elem<TYPE>;
  const int at = (int)(blockIdx.x * 256 + threadIdx.x) * 8, K = a.K;
  if (at >= K) return;
  v8f dw, db;
#pragma unroll
  for (int j = 0; j < 8; ++j) dw[j] = db[j] = 0.0f;
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    const v8f x = values<TYPE>(static_cast<const char*>(a.x) + row * a.x_row * E::kBytes, at, K);
    const v8f g = values<TYPE>(static_cast<const char*>(a.dy) + row * a.dy_row * E::kBytes, at, K);
    const float mean = a.stats[row * 2], rstd = a.stats[row * 2 + 1];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      dw[j] = __builtin_fmaf(g[j], (x[j] - mean) * rstd, dw[j]);
      db[j] += g[j];
    }
  }
  float* to = a.parts + (int64_t)blockIdx.y * 2 * K;
  Elem<kF32>::store(to, at, K, dw);
  Elem<kF32>::store(to + K, at, K, db);
}

// dw and db from the workgroups' sums: a workgroup takes 32 columns, eight threads each.
template <int WTYPE>
__global__ __launch_bounds__(256) void kn_join(NormArgs a) {
  __shared__ float sh[8][32];
  const int c = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int at = (int)blockIdx.x * 32 + c;
  float s = 0.0f;
  if (at < 2 * a.K) {
    const float* p = a.parts + at;
#pragma unroll 4
    for (int g = slice; g < a.groups; g += 8) s += p[(int64_t)g * 2 * a.K];
  }
  sh[slice][c] = s;
  __syncthreads();
  if (slice != 0 || at >= 2 * a.K) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) s += sh[i][c];
  void* to = at < a.K ? a.dw : a.db;
  if (to) Elem<WTYPE>::put(to, at < a.K ? at : at - a.K, s);
}

// Lanes to a row: two vectors of eight channels each.
static int row_lanes(int64_t K) { return K <= 1024 ? 64 : K <= 2048 ? 128 : K <= 4096 ? 256 : K <= 8192 ? 512 : 1024; }

// How many workgroups go over the rows backward: one of 512 threads to a CU, as many as
// there are rows for. More leave more sums to add (two to a CU: 78 us for both passes over
// 8190 rows of 4096 where one takes 70).
int norm_groups(int64_t rows, int64_t K, int num_cus) {
  const int per = K > 8192 ? 1 : 512 / row_lanes(K);
  return (int)std::max<int64_t>(1, std::min<int64_t>((rows + per - 1) / per, num_cus));
}

template <int TYPE, int WTYPE, int L, int NV>
static hipError_t forward(const NormArgs& a, hipStream_t stream) {
  constexpr int TH = L > 256 ? L : 256, R = TH / L;
  return launch_rows(a.rows, L, TH, [&](int64_t at, int64_t n) {
    hipLaunchKernelGGL((kn_forward<TYPE, WTYPE, L, NV>), dim3((unsigned)((n + R - 1) / R)), dim3(TH), 0, stream,
                       norm_rows_of(a, at, n, Elem<TYPE>::kBytes));
    return hipGetLastError();
  });
}

template <int TYPE, int WTYPE, int L, int NV>
static hipError_t backward(const NormArgs& a, hipStream_t stream) {
  if (a.dw || a.db) hipLaunchKernelGGL((kn_backward<TYPE, WTYPE, L, NV, true>), dim3(a.groups), dim3(512), 0, stream, a);
  else hipLaunchKernelGGL((kn_backward<TYPE, WTYPE, L, NV, false>), dim3(a.groups), dim3(512), 0, stream, a);
  return hipGetLastError();
}

template <class Run>
static hipError_t by_type(int type, int w_type, Run&& run) {
  using std::integral_constant;
  constexpr integral_constant<int, kF16> f16;
  constexpr integral_constant<int, kBF16> bf16;
  constexpr integral_constant<int, kF32> f32;
  if (type == kF32) return run(f32, f32);
  if (type == kBF16) return w_type == kF32 ? run(bf16, f32) : run(bf16, bf16);
  return w_type == kF32 ? run(f16, f32) : run(f16, f16);
}

hipError_t launch_norm(const NormArgs& a, int type, int w_type, hipStream_t stream) {
  return by_type(type, w_type, [&](auto t, auto w) {
    constexpr int T = t(), WT = w();
    if (a.K > 16384) return forward<T, WT, 1024, 8>(a, stream);
    switch (row_lanes(a.K)) {
      case 64: return forward<T, WT, 64, 2>(a, stream);
      case 128: return forward<T, WT, 128, 2>(a, stream);
      case 256: return forward<T, WT, 256, 2>(a, stream);
      case 512: return forward<T, WT, 512, 2>(a, stream);
      default: return forward<T, WT, 1024, 2>(a, stream);
    }
  });
}

hipError_t launch_norm_join(const NormArgs& a, int w_type, hipStream_t stream) {
  const dim3 blocks((2 * a.K + 31) / 32);
  if (w_type == kF32) hipLaunchKernelGGL((kn_join<kF32>), blocks, dim3(256), 0, stream, a);
  else if (w_type == kBF16) hipLaunchKernelGGL((kn_join<kBF16>), blocks, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((kn_join<kF16>), blocks, dim3(256), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_norm_backward(const NormArgs& a, int type, int w_type, hipStream_t stream) {
  return by_type(type, w_type, [&](auto t, auto w) {
    constexpr int T = t(), WT = w();
    const bool sums = a.dw || a.db;
    hipError_t e;
    if (a.K > 8192) {
      e = launch_rows(a.rows, 1024, 1024, [&](int64_t at, int64_t n) {
        hipLaunchKernelGGL((kn_wide<T, WT>), dim3((unsigned)n), dim3(1024), 0, stream, norm_rows_of(a, at, n, Elem<T>::kBytes));
        return hipGetLastError();
      });
      if (e != hipSuccess) return e;
      if (sums) hipLaunchKernelGGL((kn_columns<T>), dim3((a.K + 2047) / 2048, a.groups), dim3(256), 0, stream, a);
      e = hipGetLastError();
    } else {
      switch (row_lanes(a.K)) {
        case 64: e = backward<T, WT, 64, 2>(a, stream); break;
        case 128: e = backward<T, WT, 128, 2>(a, stream); break;
        case 256: e = backward<T, WT, 256, 2>(a, stream); break;
        default: e = backward<T, WT, 512, 2>(a, stream); break;
      }
    }
    return e != hipSuccess || !sums ? e : launch_norm_join(a, w_type, stream);
  });
}

}  // namespace llmint8
