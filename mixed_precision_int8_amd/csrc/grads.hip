// The norm of a model's gradients and their scaling on gfx950.
//   norm = scale sqrt(sum g^2)                  squares and sums in 64 bits
//   g'   = g f, f = fl32(scale min(1, max_norm / (norm + 1e-6)))
// Squares of fp32 leave fp32's range from 2^64 on, so they are summed in 64 bits
// (2.5 10^12 values a second arrive from memory; the CUs take 30 times that). Every
// workgroup leaves its sum, one more adds them in a fixed order: no atomics, the same
// result every time. Bound by memory: the values once for the norm, once more in and
// out for the scaling (21 million in bf16, written in fp32: 24 us, 5.3 TB/s; the norm 14).
#include <type_traits>

#include "train_common.h"

namespace llmint8 {

namespace {

// This workgroup's tensor and values [lo, hi) of it.
template <int N>
__device__ __forceinline__ const GradItem& grad_place(const GradBatch<N>& g, int64_t* lo, int64_t* hi) {
  const int b = blockIdx.x;
  int t = 0;
#pragma unroll
  for (int step = N > 256 ? 256 : 64; step > 0; step >>= 1)
    if (t + step < g.count && g.item[t + step].start <= b) t += step;
  const GradItem& i = g.item[t];
  *lo = (int64_t)(b - i.start) * g.chunk;
  *hi = min(*lo + g.chunk, i.n);
  return i;
}

__device__ __forceinline__ double block_sum(double v, double (&sh)[4]) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  return sh[0] + sh[1] + sh[2] + sh[3];
}

template <int TYPE>
__device__ __forceinline__ double squares(const void* p, int64_t lo, int64_t hi) {
  using E = Elem<TYPE>;
  double sum[2] = {0.0, 0.0};
  constexpr int kAhead = 4;  // vectors on their way
  for (int64_t i = lo + threadIdx.x * 8; i < hi; i += kAhead * 2048) {
    typename E::Raw r[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) r[k] = E::load(p, i + k * 2048, hi);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const v8f f = E::wide(r[k]);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum[j & 1] = __builtin_fma((double)f[j], (double)f[j], sum[j & 1]);
    }
  }
  return sum[0] + sum[1];
}

template <int TYPE, int OUT>
__device__ __forceinline__ void scale_to(const void* p, void* out, int64_t lo, int64_t hi, float f) {
  using E = Elem<TYPE>;
  constexpr int kAhead = 4;
  for (int64_t i = lo + threadIdx.x * 8; i < hi; i += kAhead * 2048) {
    typename E::Raw r[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) r[k] = E::load(p, i + k * 2048, hi);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      v8f v = E::wide(r[k]);
      v *= f;
      Elem<OUT>::store(out, i + k * 2048, hi, v);
    }
  }
}

}  // namespace

template <int N>
__global__ __launch_bounds__(256) void kg_squares(GradBatch<N> g, double* parts) {
  __shared__ double sh[4];
  int64_t lo, hi;
  const GradItem& i = grad_place(g, &lo, &hi);
  const int type = i.types & 255;
  double s;
  if (type == kF32) s = squares<kF32>(i.p, lo, hi);
  else if (type == kBF16) s = squares<kBF16>(i.p, lo, hi);
  else s = squares<kF16>(i.p, lo, hi);
  s = block_sum(s, sh);
  if (threadIdx.x == 0) parts[blockIdx.x] = s;
}

__global__ __launch_bounds__(256) void kg_norm(const double* parts, int64_t n, double scale, float* norm) {
  __shared__ double sh[4];
  double s = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += 256) s += parts[i];
  s = block_sum(s, sh);
  if (threadIdx.x == 0) *norm = (float)(sqrt(s) * scale);
}

template <int N>
__global__ __launch_bounds__(256) void kg_scale(GradBatch<N> g, const float* norm, double max_norm, double scale) {
  int64_t lo, hi;
  const GradItem& i = grad_place(g, &lo, &hi);
  const double by = max_norm == __builtin_inf() ? 1.0 : max_norm / ((double)*norm + 1e-6);
  const float f = (float)(scale * (by > 1.0 ? 1.0 : by));  // a norm that is NaN makes all values NaN
  const int type = i.types & 255, to = i.types >> 8;
  if (type == kF32) scale_to<kF32, kF32>(i.p, i.out, lo, hi, f);
  else if (type == kBF16 && to == kF32) scale_to<kBF16, kF32>(i.p, i.out, lo, hi, f);
  else if (type == kBF16) scale_to<kBF16, kBF16>(i.p, i.out, lo, hi, f);
  else if (to == kF32) scale_to<kF16, kF32>(i.p, i.out, lo, hi, f);
  else scale_to<kF16, kF16>(i.p, i.out, lo, hi, f);
}

template <int N>
hipError_t launch_grad_squares(const GradBatch<N>& g, double* parts, hipStream_t stream) {
  hipLaunchKernelGGL(kg_squares<N>, dim3((unsigned)g.blocks), dim3(256), 0, stream, g, parts);
  return hipGetLastError();
}

hipError_t launch_grad_norm(const double* parts, int64_t n, double scale, float* norm, hipStream_t stream) {
  hipLaunchKernelGGL(kg_norm, dim3(1), dim3(256), 0, stream, parts, n, scale, norm);
  return hipGetLastError();
}

template <int N>
hipError_t launch_grad_scale(const GradBatch<N>& g, const float* norm, double max_norm, double scale, hipStream_t stream) {
  hipLaunchKernelGGL(kg_scale<N>, dim3((unsigned)g.blocks), dim3(256), 0, stream, g, norm, max_norm, scale);
  return hipGetLastError();
}

template hipError_t launch_grad_squares(const GradBatch<kGradFew>&, double*, hipStream_t);
template hipError_t launch_grad_squares(const GradBatch<kGradMany>&, double*, hipStream_t);
template hipError_t launch_grad_scale(const GradBatch<kGradFew>&, const float*, double, double, hipStream_t);
template hipError_t launch_grad_scale(const GradBatch<kGradMany>&, const float*, double, double, hipStream_t);

}  // namespace llmint8
