// Host side of the C ABI's training operators (include/llmint8.h): packed attention,
// rotary positions with axes, layer norm, the gradients' norm. As in api.cpp,
// nothing here allocates device memory, waits or reads device data, and every check
// comes before any HIP call.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/llmint8.h"
#include "train_internal.h"

using namespace llmint8;

static_assert(kF16 == LLMINT8_DTYPE_F16 && kF32 == LLMINT8_DTYPE_F32 && kBF16 == LLMINT8_DTYPE_BF16, "types");

static bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
static bool half_type(int t) { return t == kF16 || t == kBF16; }
static int type_bytes(int t) { return t == kF32 ? 4 : half_type(t) ? 2 : 0; }

extern "C" {

// Rows [rows, heads, dim]. The stride of an axis of length one is never used.
static llmint8_status attn_rows(const llmint8_rows* in, const AttnArgs& a, int64_t heads, KvRows* r) {
  if (!in || !in->data || !aligned(in->data, 16)) return LLMINT8_ERR_INVALID_ARG;
  if (a.T > 1 && (in->token < a.dim || in->token % 8 != 0)) return LLMINT8_ERR_INVALID_ARG;
  if (heads > 1 && (in->head < a.dim || in->head % 8 != 0)) return LLMINT8_ERR_INVALID_ARG;
  if ((a.T > 1 && in->token > kAttnMaxStride) || (heads > 1 && in->head >= (int64_t(1) << 40)))
    return LLMINT8_ERR_UNSUPPORTED;
  r->p = static_cast<uint16_t*>(in->data);
  r->token = a.T > 1 ? in->token : a.dim;
  r->head = heads > 1 ? in->head : 0;
  return LLMINT8_OK;
}

static llmint8_status attn_args(const llmint8_attention_shape* s, int dtype, AttnArgs* a) {
  if (!s || !half_type(dtype)) return LLMINT8_ERR_INVALID_ARG;
  const llmint8_status st = admit_attention(s->seqs, s->rows, s->q_heads, s->heads, s->dim);
  if (st != LLMINT8_OK) return st;
  if (!std::isfinite(s->scale) || s->window < 0 || s->sinks < 0 || (s->window > 0 && !s->causal))
    return LLMINT8_ERR_INVALID_ARG;
  if (s->window > kKvMax || s->sinks > kKvMax) return LLMINT8_ERR_UNSUPPORTED;
  a->cu = s->cu;
  a->B = (int)s->seqs;
  a->T = (int)s->rows;
  a->scale = s->scale;
  a->q_heads = (int)s->q_heads;
  a->heads = (int)s->heads;
  a->dim = (int)s->dim;
  a->causal = s->causal ? 1 : 0;
  a->window = (int)s->window;
  a->sinks = (int)s->sinks;
  if (a->B > 0 && a->T > 0 && (!s->cu || !aligned(s->cu, 4))) return LLMINT8_ERR_INVALID_ARG;
  return LLMINT8_OK;
}

llmint8_status llmint8_attention(const llmint8_attention_shape* shape, int dtype, const llmint8_rows* q,
                                 const llmint8_rows* k, const llmint8_rows* v, const llmint8_rows* out,
                                 float* lse, void* stream) {
  AttnArgs a{};
  llmint8_status st = attn_args(shape, dtype, &a);
  if (st != LLMINT8_OK) return st;
  if (lse && !aligned(lse, 4)) return LLMINT8_ERR_INVALID_ARG;
  if (a.B == 0 || a.T == 0) return LLMINT8_OK;
  if (!attn_row_grid(a.T, a.q_heads, a.heads, a.B).fits()) return LLMINT8_ERR_UNSUPPORTED;
  if ((st = attn_rows(q, a, a.q_heads, &a.q)) != LLMINT8_OK || (st = attn_rows(k, a, a.heads, &a.k)) != LLMINT8_OK ||
      (st = attn_rows(v, a, a.heads, &a.v)) != LLMINT8_OK || (st = attn_rows(out, a, a.q_heads, &a.o)) != LLMINT8_OK)
    return st;
  if (a.o.p == a.q.p || a.o.p == a.k.p || a.o.p == a.v.p) return LLMINT8_ERR_INVALID_ARG;
  a.lse = lse;
  return abi_hip_status(launch_attention(a, dtype == kBF16, static_cast<hipStream_t>(stream)));
}

size_t llmint8_attention_backward_workspace_bytes(const llmint8_attention_shape* shape) {
  AttnArgs a{};
  if (!shape || admit_attention(shape->seqs, shape->rows, shape->q_heads, shape->heads, shape->dim) != LLMINT8_OK ||
      shape->seqs == 0)
    return 0;
  return (size_t)shape->rows * shape->q_heads * 2 * sizeof(float);
}

llmint8_status llmint8_attention_backward(const llmint8_attention_shape* shape, int dtype, const llmint8_rows* q,
                                          const llmint8_rows* k, const llmint8_rows* v, const llmint8_rows* out,
                                          const float* lse, const llmint8_rows* dout, const llmint8_rows* dq,
                                          const llmint8_rows* dk, const llmint8_rows* dv, void* workspace,
                                          size_t workspace_bytes, void* stream) {
  AttnArgs a{};
  llmint8_status st = attn_args(shape, dtype, &a);
  if (st != LLMINT8_OK) return st;
  if (a.B == 0 || a.T == 0) return LLMINT8_OK;
  if (!attn_row_grid(a.T, a.q_heads, a.heads, a.B).fits() || !attn_col_grid(a.T, a.heads, a.B, a.dim).fits())
    return LLMINT8_ERR_UNSUPPORTED;
  const struct {
    const llmint8_rows* in;
    int heads;
    KvRows* to;
  } all[8] = {{q, a.q_heads, &a.q},      {k, a.heads, &a.k},      {v, a.heads, &a.v},   {out, a.q_heads, &a.o},
              {dout, a.q_heads, &a.d_o}, {dq, a.q_heads, &a.dq}, {dk, a.heads, &a.dk}, {dv, a.heads, &a.dv}};
  for (int i = 0; i < 8; ++i) {
    if ((st = attn_rows(all[i].in, a, all[i].heads, all[i].to)) != LLMINT8_OK) return st;
    for (int j = 0; i >= 5 && j < i; ++j)
      if (all[j].to->p == all[i].to->p) return LLMINT8_ERR_INVALID_ARG;
  }
  if (!lse || !aligned(lse, 4)) return LLMINT8_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, kWsAlign)) return LLMINT8_ERR_INVALID_ARG;
  if (workspace_bytes < llmint8_attention_backward_workspace_bytes(shape)) return LLMINT8_ERR_WORKSPACE;
  a.lse = const_cast<float*>(lse);
  a.stat = static_cast<float*>(workspace);
  return abi_hip_status(launch_attention_backward(a, dtype == kBF16, static_cast<hipStream_t>(stream)));
}

static llmint8_status rope_rows(const llmint8_rows* x, const llmint8_rows* y, int64_t rows, int64_t heads,
                                int64_t dim, RopeArgs* a, int i) {
  const llmint8_rows* in[2] = {x, y};
  KvRows* out[2] = {&a->x[i], &a->y[i]};
  for (int j = 0; j < 2; ++j) {
    const llmint8_rows* r = in[j];
    if (!r || !r->data || !aligned(r->data, 2)) return LLMINT8_ERR_INVALID_ARG;
    if ((rows > 1 && r->token < dim) || (heads > 1 && r->head < dim)) return LLMINT8_ERR_INVALID_ARG;
    if ((rows > 1 && r->token >= kTwo31) || (heads > 1 && r->head >= (int64_t(1) << 40)))
      return LLMINT8_ERR_UNSUPPORTED;
    out[j]->p = static_cast<uint16_t*>(r->data);
    out[j]->token = rows > 1 ? r->token : 0;
    out[j]->head = heads > 1 ? r->head : 0;
  }
  a->heads[i] = (int)heads;
  const bool in_place = a->x[i].p == a->y[i].p;
  if (in_place && (a->x[i].token != a->y[i].token || a->x[i].head != a->y[i].head)) return LLMINT8_ERR_INVALID_ARG;
  a->copy |= !in_place && a->rot < dim;
  return LLMINT8_OK;
}

llmint8_status llmint8_rope(int dtype, const llmint8_rows* x, const llmint8_rows* y, int64_t heads,
                            const llmint8_rows* x2, const llmint8_rows* y2, int64_t heads2, int64_t rows, int64_t dim,
                            const int32_t* pos, int64_t axes, const uint8_t* axis, const float* table,
                            int64_t table_rows, int64_t rot, int interleaved, int inverse, void* stream) {
  if (!half_type(dtype) || rows < 0 || heads < 1 || heads2 < 0 || dim < 2 || !axis) return LLMINT8_ERR_INVALID_ARG;
  if (dim % 2 != 0 || rot < 2 || rot % 2 != 0 || rot > dim || axes < 1) return LLMINT8_ERR_INVALID_ARG;
  if (rows > kKvMax || dim > 65536 || rot > 2 * kRopeMaxPairs || axes > kRopeMaxAxes || heads > kKvMaxQHeads ||
      heads2 > kKvMaxQHeads)
    return LLMINT8_ERR_UNSUPPORTED;
  if ((!x2 != !y2) || (!x2 != (heads2 == 0))) return LLMINT8_ERR_INVALID_ARG;
  RopeArgs a{};
  for (int64_t i = 0; i < rot / 2; ++i) {
    if (axis[i] >= axes) return LLMINT8_ERR_INVALID_ARG;
    a.axis[i] = axis[i];
  }
  if (rows == 0) return LLMINT8_OK;
  if (!pos || !aligned(pos, 4) || !table || !aligned(table, 4) || table_rows < 1) return LLMINT8_ERR_INVALID_ARG;
  if (table_rows > kKvMax) return LLMINT8_ERR_UNSUPPORTED;
  a.rot = (int)rot;
  llmint8_status st = rope_rows(x, y, rows, heads, dim, &a, 0);
  if (st == LLMINT8_OK && x2) st = rope_rows(x2, y2, rows, heads2, dim, &a, 1);
  if (st != LLMINT8_OK) return st;
  a.pos = pos;
  a.table = table;
  a.rows = rows;
  a.axes = (int)axes;
  a.table_rows = (int)table_rows;
  a.dim = (int)dim;
  a.interleaved = interleaved ? 1 : 0;
  a.sign = inverse ? -1.0f : 1.0f;
  return abi_hip_status(launch_rope(a, dtype == kBF16, abi_cu_count(), static_cast<hipStream_t>(stream)));
}

static llmint8_status norm_sizes(int dtype, int w_dtype, int64_t rows, int64_t K) {
  if (!type_bytes(dtype) || (w_dtype != dtype && w_dtype != kF32)) return LLMINT8_ERR_INVALID_ARG;
  if (rows < 0 || K < 1) return LLMINT8_ERR_INVALID_ARG;
  if (rows >= kTwo31 || K > kNormMaxWidth) return LLMINT8_ERR_UNSUPPORTED;
  return LLMINT8_OK;
}
static bool norm_rows(const void* p, int64_t stride, int dtype, int64_t rows, int64_t K) {
  return p && aligned(p, type_bytes(dtype)) && (rows < 2 || stride >= K) && stride < (int64_t(1) << 40);
}

llmint8_status llmint8_layer_norm(const void* x, int64_t x_row, int dtype, int64_t rows, int64_t K, const void* w,
                                  const void* b, int w_dtype, float eps, void* y, int64_t y_row, float* stats,
                                  void* stream) {
  const llmint8_status st = norm_sizes(dtype, w_dtype, rows, K);
  if (st != LLMINT8_OK) return st;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return LLMINT8_ERR_INVALID_ARG;
  if (!aligned(w, type_bytes(w_dtype)) || !aligned(b, type_bytes(w_dtype)) || !aligned(stats, 4))
    return LLMINT8_ERR_INVALID_ARG;
  if (rows == 0) return LLMINT8_OK;
  if (!norm_rows(x, x_row, dtype, rows, K) || !norm_rows(y, y_row, dtype, rows, K)) return LLMINT8_ERR_INVALID_ARG;
  if (x == y && rows > 1 && x_row != y_row) return LLMINT8_ERR_INVALID_ARG;
  NormArgs a{};
  a.x = x;
  a.w = w;
  a.b = b;
  a.y = y;
  a.stats = stats;
  a.rows = rows;
  a.x_row = x_row;
  a.y_row = y_row;
  a.K = (int)K;
  a.eps = eps;
  return abi_hip_status(launch_norm(a, dtype, w_dtype, static_cast<hipStream_t>(stream)));
}

size_t llmint8_layer_norm_workspace_bytes(int64_t rows, int64_t K) {
  if (norm_sizes(kF32, kF32, rows, K) != LLMINT8_OK) return 0;
  return (size_t)norm_groups(rows, K, abi_cu_count()) * 2 * K * sizeof(float);
}

llmint8_status llmint8_layer_norm_backward(const void* dy, int64_t dy_row, const void* x, int64_t x_row, int dtype,
                                           int64_t rows, int64_t K, const void* w, int w_dtype, const float* stats,
                                           void* dx, int64_t dx_row, void* dw, void* db, void* workspace,
                                           size_t workspace_bytes, void* stream) {
  const llmint8_status st = norm_sizes(dtype, w_dtype, rows, K);
  if (st != LLMINT8_OK) return st;
  const int wb = type_bytes(w_dtype);
  if (!aligned(w, wb) || !aligned(dw, wb) || !aligned(db, wb) || (dw && dw == db)) return LLMINT8_ERR_INVALID_ARG;
  NormArgs a{};
  a.rows = rows;
  a.K = (int)K;
  a.dw = dw;
  a.db = db;
  if (dw || db) {
    if (!workspace || !aligned(workspace, kWsAlign)) return LLMINT8_ERR_INVALID_ARG;
    if (workspace_bytes < llmint8_layer_norm_workspace_bytes(rows, K)) return LLMINT8_ERR_WORKSPACE;
    a.parts = static_cast<float*>(workspace);
  }
  a.groups = norm_groups(rows, K, abi_cu_count());
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (rows == 0) {
    if (!dw && !db) return LLMINT8_OK;
    a.groups = 0;
    return abi_hip_status(launch_norm_join(a, w_dtype, s));
  }
  if (!norm_rows(x, x_row, dtype, rows, K) || !norm_rows(dy, dy_row, dtype, rows, K) ||
      !norm_rows(dx, dx_row, dtype, rows, K) || !stats || !aligned(stats, 4) || dx == x || dx == dy)
    return LLMINT8_ERR_INVALID_ARG;
  a.x = x;
  a.w = w;
  a.y = dx;
  a.stats = const_cast<float*>(stats);
  a.x_row = x_row;
  a.y_row = dx_row;
  a.dy = dy;
  a.dy_row = dy_row;
  return abi_hip_status(launch_norm_backward(a, dtype, w_dtype, s));
}

// Values of a workgroup: 16384, more where that would be over 65536 workgroups.
static int64_t grad_chunk(const llmint8_grad* g, int64_t count) {
  int64_t total = 0;
  for (int64_t i = 0; i < count; ++i) total += g[i].n;
  return std::max<int64_t>(16384, ceil_div(ceil_div(total, 65536), 8192) * 8192);
}
static llmint8_status grad_check(const llmint8_grad* g, int64_t count, bool out) {
  if (count < 0 || (count > 0 && !g)) return LLMINT8_ERR_INVALID_ARG;
  if (count > (int64_t(1) << 20)) return LLMINT8_ERR_UNSUPPORTED;
  int64_t total = 0;
  for (int64_t i = 0; i < count; ++i) {
    const int bytes = type_bytes(g[i].dtype);
    if (!bytes || g[i].n < 0) return LLMINT8_ERR_INVALID_ARG;
    if (g[i].n >= (int64_t(1) << 40) || (total += g[i].n) >= (int64_t(1) << 40)) return LLMINT8_ERR_UNSUPPORTED;
    if (g[i].n > 0 && (!g[i].data || !aligned(g[i].data, bytes))) return LLMINT8_ERR_INVALID_ARG;
    if (!out) continue;
    if (g[i].out_dtype != g[i].dtype && g[i].out_dtype != kF32) return LLMINT8_ERR_INVALID_ARG;
    if (g[i].n > 0 && (!g[i].out || !aligned(g[i].out, type_bytes(g[i].out_dtype)))) return LLMINT8_ERR_INVALID_ARG;
    if (g[i].out == g[i].data && g[i].out_dtype != g[i].dtype && g[i].n > 0) return LLMINT8_ERR_INVALID_ARG;
  }
  return LLMINT8_OK;
}

size_t llmint8_grad_norm_workspace_bytes(const llmint8_grad* grads, int64_t count) {
  if (grad_check(grads, count, false) != LLMINT8_OK) return 0;
  const int64_t chunk = grad_chunk(grads, count);
  int64_t blocks = 0;
  for (int64_t i = 0; i < count; ++i) blocks += ceil_div(grads[i].n, chunk);
  return (size_t)std::max<int64_t>(blocks, 1) * sizeof(double);
}

}  // extern "C"

// `launch` for batches of the tensors that hold anything.
template <int N, class Launch>
static hipError_t grad_batches_of(const llmint8_grad* grads, int64_t count, Launch&& launch) {
  GradBatch<N> b;
  b.chunk = (int)grad_chunk(grads, count);
  b.count = b.blocks = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (grads[i].n > 0) {
      b.item[b.count++] = {grads[i].data, grads[i].out, grads[i].n, b.blocks, grads[i].dtype | grads[i].out_dtype << 8};
      b.blocks += (int)ceil_div(grads[i].n, b.chunk);
    }
    if (b.count == N || (i + 1 == count && b.count > 0)) {
      const hipError_t e = launch(b);
      if (e != hipSuccess) return e;
      b.count = b.blocks = 0;
    }
  }
  return hipSuccess;
}
template <class Launch>
static hipError_t grad_batches(const llmint8_grad* grads, int64_t count, Launch&& launch) {
  return count > kGradFew ? grad_batches_of<kGradMany>(grads, count, launch)
                          : grad_batches_of<kGradFew>(grads, count, launch);
}

extern "C" {

llmint8_status llmint8_grad_norm(const llmint8_grad* grads, int64_t count, double scale, float* norm, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  const llmint8_status st = grad_check(grads, count, false);
  if (st != LLMINT8_OK) return st;
  if (!(scale > 0.0) || !std::isfinite(scale) || !norm || !aligned(norm, 4)) return LLMINT8_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, kWsAlign)) return LLMINT8_ERR_INVALID_ARG;
  if (workspace_bytes < llmint8_grad_norm_workspace_bytes(grads, count)) return LLMINT8_ERR_WORKSPACE;
  const hipStream_t s = static_cast<hipStream_t>(stream);
  double* parts = static_cast<double*>(workspace);
  int64_t blocks = 0;
  const hipError_t e = grad_batches(grads, count, [&](const auto& b) {
    const hipError_t err = launch_grad_squares(b, parts + blocks, s);
    blocks += b.blocks;
    return err;
  });
  if (e != hipSuccess) return abi_hip_status(e);
  return abi_hip_status(launch_grad_norm(parts, blocks, scale, norm, s));
}

llmint8_status llmint8_grad_clip(const llmint8_grad* grads, int64_t count, const float* norm, double max_norm,
                                 double scale, void* stream) {
  const llmint8_status st = grad_check(grads, count, true);
  if (st != LLMINT8_OK) return st;
  if (!(scale > 0.0) || !std::isfinite(scale) || !(max_norm > 0.0) || !norm || !aligned(norm, 4))
    return LLMINT8_ERR_INVALID_ARG;
  return abi_hip_status(grad_batches(grads, count, [&](const auto& b) {
    return launch_grad_scale(b, norm, max_norm, scale, static_cast<hipStream_t>(stream));
  }));
}

}  // extern "C"
