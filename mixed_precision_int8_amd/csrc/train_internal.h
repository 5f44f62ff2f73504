// Layer norm, rotary positions with axes, and the gradients' norm: what their
// kernels take, and the launchers.
#pragma once

#include "attn_internal.h"

namespace llmint8 {

// Element types of these operators, as the ABI numbers them.
enum : int { kF16 = 0, kF32 = 1, kBF16 = 2 };

// Rows in as few launches as there are work items for (fewer than 2^32 to a launch): launch(first row,
// rows) with `items` to a row, in workgroups of `threads`.
template <class Launch>
hipError_t launch_rows(int64_t rows, int64_t items, int threads, Launch&& launch, int64_t max_items = kMaxWorkItems) {
  const int64_t most = (max_items - threads) / items;
  for (int64_t at = 0; at < rows; at += most) {
    const hipError_t e = launch(at, rows - at < most ? rows - at : most);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

constexpr int64_t kNormMaxWidth = 65536;
struct NormArgs {
  const void* x;
  const void* w;  // [K] or null
  const void* b;  // [K] or null
  void* y;
  float* stats;  // [rows, 2]: mean, 1 / sqrt(var + eps); forward: or null
  int64_t rows, x_row, y_row;
  int K;
  float eps;
  // backward: y is dx
  const void* dy;
  int64_t dy_row;
  void* dw;  // or null
  void* db;  // or null
  float* parts;  // [groups][2][K]
  int groups;
};
// n rows from row `at` on, of elements of `bytes`
inline NormArgs norm_rows_of(NormArgs a, int64_t at, int64_t n, int bytes) {
  auto on = [&](auto* p, int64_t by) { return p ? p + by : p; };
  a.x = static_cast<const char*>(a.x) + at * a.x_row * bytes;
  a.y = static_cast<char*>(a.y) + at * a.y_row * bytes;
  a.dy = on(static_cast<const char*>(a.dy), at * a.dy_row * bytes);
  a.stats = on(a.stats, 2 * at);
  a.rows = n;
  return a;
}
// Workgroups of the backward pass, each of which leaves one row of partial sums.
int norm_groups(int64_t rows, int64_t K, int num_cus);
hipError_t launch_norm(const NormArgs& a, int type, int w_type, hipStream_t stream);
hipError_t launch_norm_backward(const NormArgs& a, int type, int w_type, hipStream_t stream);
hipError_t launch_norm_join(const NormArgs& a, int w_type, hipStream_t stream);  // dw and db from the groups' sums

constexpr int kRopeMaxAxes = 8;
struct RopeArgs {
  KvRows x[2], y[2];  // second: heads[1] = 0 if there is none
  int heads[2];
  const int32_t* pos;  // [rows, axes]
  const float* table;  // [table_rows, rot]
  int64_t rows;
  int axes, table_rows, dim, rot, interleaved, copy;  // copy: the channels that do not turn are copied
  float sign;                                         // of the angles
  uint8_t axis[kRopeMaxPairs];
};
inline RopeArgs rope_rows_of(RopeArgs a, int64_t at, int64_t n) {
  for (int i = 0; i < 2; ++i) {
    if (a.heads[i] == 0) continue;
    a.x[i].p += at * a.x[i].token;
    a.y[i].p += at * a.y[i].token;
  }
  a.pos += at * a.axes;
  a.rows = n;
  return a;
}
hipError_t launch_rope(const RopeArgs& a, bool bf16, int num_cus, hipStream_t stream);

// Gradients: up to N tensors to a launch, as its arguments: 480 of them where there are more
// than 120 (tensors of 4096 to 180000 values, norm and clipping replayed from a graph: 121 of them 19 us
// and 26 in launches of 120, 240 of them 26 and 35, 448 of them 37 and 67, 600 of them 56 and 85), else 120 (65 tensors: 28 us, 37 with the 16 KB of arguments of 480). A workgroup takes
// `chunk` values of one; tensor t's workgroups begin at `start`. One entry is 32 bytes
// for all that is read of a tensor: beside an array of bytes indexed by the tensor the
// compiler has split 8 t into t and 7 t for a scalar load of an address, and scalar
// loads drop the lowest two bits of each.
constexpr int kGradFew = 120, kGradMany = 480;
struct GradItem {
  const void* p;
  void* out;
  int64_t n;
  int start;
  int types;  // type | out_type << 8
};
template <int N>
struct GradBatch {
  GradItem item[N];
  int count, chunk;
  int blocks;  // of all the items
};
static_assert(sizeof(GradItem) == 32 && sizeof(GradBatch<kGradFew>) + 32 <= 4096, "the arguments of a launch of few");
template <int N>
hipError_t launch_grad_squares(const GradBatch<N>& g, double* parts, hipStream_t stream);
hipError_t launch_grad_norm(const double* parts, int64_t n, double scale, float* norm, hipStream_t stream);
template <int N>
hipError_t launch_grad_scale(const GradBatch<N>& g, const float* norm, double max_norm, double scale, hipStream_t stream);

}  // namespace llmint8
