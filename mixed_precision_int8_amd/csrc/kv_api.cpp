// Host side of the C ABI's int8 key/value cache (include/llmint8.h): argument
// checks, the split of an attention call's work, launches on the caller's
// stream. As in api.cpp, nothing here allocates device memory, waits or reads
// device data, and every check comes before any HIP call.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/llmint8.h"
#include "kv_internal.h"

using namespace llmint8;

static bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

extern "C" {

// The cache and batch of a call, checked and in the kernels' form. *empty: nothing to do.
static llmint8_status kv_operands(const llmint8_kv_cache* cache, const llmint8_kv_batch* batch, int dtype,
                                  KvCache* c, KvBatch* s, bool* empty) {
  if (!cache || !batch) return LLMINT8_ERR_INVALID_ARG;
  if (dtype != LLMINT8_DTYPE_F16 && dtype != LLMINT8_DTYPE_BF16) return LLMINT8_ERR_INVALID_ARG;
  llmint8_status st = admit_kv_cache(cache->pages, cache->heads, cache->page, cache->dim);
  if (st != LLMINT8_OK) return st;
  st = admit_kv_batch(batch->seqs, batch->rows, batch->width, cache->page);
  if (st != LLMINT8_OK) return st;
  if (batch->max_len < 0) return LLMINT8_ERR_INVALID_ARG;
  if (!cache->K || !cache->V || !cache->aK || !cache->aV) return LLMINT8_ERR_INVALID_ARG;
  if (!aligned(cache->K, 16) || !aligned(cache->V, 16) || !aligned(cache->aK, 4) || !aligned(cache->aV, 4))
    return LLMINT8_ERR_INVALID_ARG;
  *empty = batch->seqs == 0 || batch->rows == 0;
  if (!*empty) {
    if (!batch->cu || !batch->len || !batch->table) return LLMINT8_ERR_INVALID_ARG;
    if (!aligned(batch->cu, 4) || !aligned(batch->len, 4) || !aligned(batch->table, 4))
      return LLMINT8_ERR_INVALID_ARG;
  }
  c->K = cache->K;
  c->V = cache->V;
  c->aK = cache->aK;
  c->aV = cache->aV;
  c->pages = cache->pages;
  c->heads = (int)cache->heads;
  c->dim = (int)cache->dim;
  c->page_shift = cache->page == 16 ? 4 : cache->page == 32 ? 5 : cache->page == 64 ? 6 : 7;
  s->cu = batch->cu;
  s->len = batch->len;
  s->table = batch->table;
  s->B = (int)batch->seqs;
  s->T = (int)batch->rows;
  s->width = (int)batch->width;
  return LLMINT8_OK;
}

// 16-bit rows [rows, heads, dim] with strides: dense channels, 16-byte pieces. A
// stride of an axis of length one is never used.
static bool kv_rows(const void* p, int64_t token, int64_t head, int64_t rows, int64_t heads, int64_t dim,
                    KvRows* r) {
  if (!p || !aligned(p, 16)) return false;
  if (rows > 1 && (token < dim || token % 8 != 0 || token >= kTwo31)) return false;
  if (heads > 1 && (head < dim || head % 8 != 0 || head >= (int64_t(1) << 40))) return false;
  r->p = static_cast<uint16_t*>(const_cast<void*>(p));
  r->token = rows > 1 ? token : 0;
  r->head = heads > 1 ? head : 0;
  return true;
}

llmint8_status llmint8_rope_table(const double* freq, int64_t pairs, int64_t rows, double mag, float* table,
                                  void* stream) {
  if (!freq || pairs < 1 || rows < 0 || !std::isfinite(mag)) return LLMINT8_ERR_INVALID_ARG;
  if (pairs > kRopeMaxPairs || rows > kKvMax) return LLMINT8_ERR_UNSUPPORTED;
  RopeFreq f{};
  for (int64_t i = 0; i < pairs; ++i) {
    if (!std::isfinite(freq[i])) return LLMINT8_ERR_INVALID_ARG;
    f.f[i] = freq[i];
  }
  if (rows == 0) return LLMINT8_OK;
  if (!table || !aligned(table, 16)) return LLMINT8_ERR_INVALID_ARG;
  return abi_hip_status(launch_rope_table(f, (int)pairs, (int)rows, mag, table, static_cast<hipStream_t>(stream)));
}

llmint8_status llmint8_kv_append(const llmint8_kv_cache* cache, const llmint8_kv_batch* batch, int dtype,
                                 const void* k, int64_t k_token, int64_t k_head, const void* v,
                                 int64_t v_token, int64_t v_head, const void* q, int64_t q_token,
                                 int64_t q_head, void* q_out, int64_t q_out_token, int64_t q_out_head,
                                 int64_t q_heads, const float* rope, int64_t rope_rows, int64_t rot,
                                 int interleaved, void* stream) {
  KvAppendArgs a{};
  bool empty = false;
  llmint8_status st = kv_operands(cache, batch, dtype, &a.c, &a.s, &empty);
  if (st != LLMINT8_OK) return st;
  if (!q != !q_out) return LLMINT8_ERR_INVALID_ARG;
  if (q && (q_heads < 1 || q_heads > kKvMaxQHeads)) return LLMINT8_ERR_INVALID_ARG;
  if (rope) {
    if (!aligned(rope, 16) || rope_rows < 1 || rope_rows > kKvMax) return LLMINT8_ERR_INVALID_ARG;
    if (rot < 2 || rot % 2 != 0 || rot > cache->dim) return LLMINT8_ERR_INVALID_ARG;
    a.rope = rope;
    a.rope_rows = (int)rope_rows;
    a.rot = (int)rot;
    a.interleaved = interleaved ? 1 : 0;
  }
  if (empty) return LLMINT8_OK;
  const int64_t T = batch->rows, H = cache->heads, D = cache->dim;
  if (!kv_rows(k, k_token, k_head, T, H, D, &a.k) || !kv_rows(v, v_token, v_head, T, H, D, &a.v))
    return LLMINT8_ERR_INVALID_ARG;
  if (q) {
    if (!kv_rows(q, q_token, q_head, T, q_heads, D, &a.q) ||
        !kv_rows(q_out, q_out_token, q_out_head, T, q_heads, D, &a.qo))
      return LLMINT8_ERR_INVALID_ARG;
    // in place, every row has to be turned where it stands
    if (q == q_out && (a.q.token != a.qo.token || a.q.head != a.qo.head)) return LLMINT8_ERR_INVALID_ARG;
    a.q_heads = (int)q_heads;
  }
  return abi_hip_status(launch_kv_append(a, dtype == LLMINT8_DTYPE_BF16, static_cast<hipStream_t>(stream)));
}

llmint8_status llmint8_kv_gather(const llmint8_kv_cache* cache, const llmint8_kv_batch* batch, int dtype,
                                 void* k, int64_t k_token, int64_t k_head, void* v, int64_t v_token,
                                 int64_t v_head, void* stream) {
  KvCache c;
  KvBatch s;
  KvRows kr, vr;
  bool empty = false;
  llmint8_status st = kv_operands(cache, batch, dtype, &c, &s, &empty);
  if (st != LLMINT8_OK) return st;
  if (empty) return LLMINT8_OK;
  if (!kv_rows(k, k_token, k_head, batch->rows, cache->heads, cache->dim, &kr) ||
      !kv_rows(v, v_token, v_head, batch->rows, cache->heads, cache->dim, &vr))
    return LLMINT8_ERR_INVALID_ARG;
  return abi_hip_status(launch_kv_gather(c, s, kr, vr, dtype == LLMINT8_DTYPE_BF16, abi_cu_count(),
                                        static_cast<hipStream_t>(stream)));
}

// The route of an attention call and the bytes that it leaves for its join.
static size_t kv_attention_plan(const llmint8_kv_batch* batch, int64_t window, int64_t sinks, void* workspace,
                                KvAttnArgs* a) {
  const int64_t room = batch->width << a->c.page_shift;
  int64_t span = batch->max_len > 0 ? std::min(batch->max_len, room) : room;
  if (window > 0) span = std::min(span, window + sinks);
  const int cus = abi_cu_count();
  a->prompt = kv_attention_prompt(a->s, a->c.heads, a->q_heads) ? 1 : 0;
  a->splits = 1;
  if (a->prompt) {
    a->splits = kv_prompt_splits(a->s, a->c.heads, a->q_heads, a->c.dim, a->c.page_shift, span, cus, &a->run,
                                 &a->max_parts);
  } else {
    a->run = kv_attention_run(a->s, a->c.heads, a->q_heads);
    a->extra = kv_attention_extra(a->s, a->c.heads, a->q_heads, a->c.dim, span, cus, &a->slots);
    a->max_parts = 2 * a->extra;  // parts of cut runs: each is longer than half of what the runs are cut by
  }
  if (a->max_parts == 0) return 0;
  const size_t rows = (size_t)a->max_parts * a->run;
  if (workspace) {
    a->part_o = static_cast<float*>(workspace);
    a->part_ml = a->part_o + rows * a->c.dim;
    a->notes = reinterpret_cast<int*>(a->part_ml + rows * 2);
  }
  return (rows * (a->c.dim + 2) + (size_t)a->s.T * a->q_heads * 2) * sizeof(float);
}

static llmint8_status check_kv_attention(const llmint8_kv_cache* cache, const llmint8_kv_batch* batch,
                                         int64_t q_heads, int causal, int64_t window, int64_t sinks) {
  if (q_heads < 1 || q_heads > kKvMaxQHeads || q_heads % cache->heads != 0) return LLMINT8_ERR_INVALID_ARG;
  if (window < 0 || sinks < 0 || (window > 0 && !causal)) return LLMINT8_ERR_INVALID_ARG;
  if (window > kKvMax || sinks > kKvMax || batch->rows * q_heads > kKvMaxQRows) return LLMINT8_ERR_UNSUPPORTED;
  return LLMINT8_OK;
}

size_t llmint8_kv_attention_workspace_bytes(const llmint8_kv_cache* cache, const llmint8_kv_batch* batch,
                                            int64_t q_heads, int64_t window, int64_t sinks) {
  KvAttnArgs a{};
  bool empty = false;
  if (kv_operands(cache, batch, LLMINT8_DTYPE_F16, &a.c, &a.s, &empty) != LLMINT8_OK) return 0;
  if (check_kv_attention(cache, batch, q_heads, 1, window, sinks) != LLMINT8_OK || empty) return 0;
  a.q_heads = (int)q_heads;
  return kv_attention_plan(batch, window, sinks, nullptr, &a);
}

llmint8_status llmint8_kv_attention(const llmint8_kv_cache* cache, const llmint8_kv_batch* batch, int dtype,
                                    const void* q, int64_t q_token, int64_t q_head, int64_t q_heads,
                                    float scale, int causal, int64_t window, int64_t sinks, void* out,
                                    int64_t out_token, int64_t out_head, float* lse, void* workspace,
                                    size_t workspace_bytes, void* stream) {
  KvAttnArgs a{};
  bool empty = false;
  llmint8_status st = kv_operands(cache, batch, dtype, &a.c, &a.s, &empty);
  if (st == LLMINT8_OK) st = check_kv_attention(cache, batch, q_heads, causal, window, sinks);
  if (st != LLMINT8_OK) return st;
  if (!std::isfinite(scale)) return LLMINT8_ERR_INVALID_ARG;
  if (empty) return LLMINT8_OK;
  const int64_t T = batch->rows, D = cache->dim;
  if (!kv_rows(q, q_token, q_head, T, q_heads, D, &a.q) || !kv_rows(out, out_token, out_head, T, q_heads, D, &a.o))
    return LLMINT8_ERR_INVALID_ARG;
  if (lse && !aligned(lse, 4)) return LLMINT8_ERR_INVALID_ARG;
  a.lse = lse;
  a.bf16 = dtype == LLMINT8_DTYPE_BF16 ? 1 : 0;
  a.scale = scale;
  a.q_heads = (int)q_heads;
  a.causal = causal ? 1 : 0;
  a.window = (int)window;
  a.sinks = (int)sinks;
  const size_t need = kv_attention_plan(batch, window, sinks, workspace, &a);
  if (need > 0) {
    if (!workspace || !aligned(workspace, kWsAlign)) return LLMINT8_ERR_INVALID_ARG;
    if (workspace_bytes < need) return LLMINT8_ERR_WORKSPACE;
  }
  return abi_hip_status(launch_kv_attention(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
