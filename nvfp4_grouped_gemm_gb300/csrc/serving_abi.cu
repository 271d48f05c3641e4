// Host side of the serving operators' C ABI (moe_serving.h): argument validation.
#include <cmath>

#include "serving.cuh"

namespace moe {
namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

moe_status from_cuda(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

moe_status check_ws(const void* ws, size_t have, size_t need) {
  if (!ws || !aligned(ws, kAlign) || have < need) return MOE_ERR_WORKSPACE;
  return MOE_OK;
}

// Token rows of `heads` heads of `dim` 16-bit values, `stride` elements apart.
moe_status check_rows(const void* p, int64_t stride, int64_t row) {
  if (!p || !aligned(p, 16)) return MOE_ERR_INVALID_ARG;
  if (stride < row || stride % 8 != 0) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status check_cache(const moe_kv_cache* c) {
  if (!c || !c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales) return MOE_ERR_INVALID_ARG;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16)) return MOE_ERR_INVALID_ARG;
  if (!aligned(c->k_scales, 4) || !aligned(c->v_scales, 4)) return MOE_ERR_INVALID_ARG;
  if (c->num_pages <= 0 || c->kv_heads <= 0 || c->page_size <= 0 || c->head_dim <= 0)
    return MOE_ERR_INVALID_ARG;
  const int p = c->page_size, d = c->head_dim;
  if (p != 16 && p != 32 && p != 64 && p != 128) return MOE_ERR_UNSUPPORTED;
  if (d != 64 && d != 128 && d != 256) return MOE_ERR_UNSUPPORTED;
  if (c->kv_heads > 1024) return MOE_ERR_UNSUPPORTED;
  if (c->page_stride < (int64_t)c->kv_heads * p * d || c->page_stride % 16 != 0)
    return MOE_ERR_INVALID_ARG;
  if (c->page_stride >= (1LL << 40)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_batch(const moe_seq_batch* b) {
  if (!b || !b->q_offsets || !b->seq_lens || !b->page_table) return MOE_ERR_INVALID_ARG;
  if (b->B <= 0 || b->max_pages <= 0 || b->table_stride < b->max_pages) return MOE_ERR_INVALID_ARG;
  if (b->B > 65536 || b->max_pages > (1 << 24)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// A call's arrays as addresses: whether one that is written lies upon another that is read or written.
struct Span {
  const void* at;
  int64_t bytes;
};
bool overlap(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.at), y = reinterpret_cast<uintptr_t>(b.at);
  return a.at && b.at && a.bytes > 0 && b.bytes > 0 && x < y + (uint64_t)b.bytes && y < x + (uint64_t)a.bytes;
}
Span table_span(const int32_t* table, int64_t rows, int64_t stride, int64_t cols) {
  return {table, ((rows - 1) * stride + cols) * 4};
}
// Rows `stride` elements apart.
Span rows_span(const void* p, int64_t rows, int64_t stride, int64_t row, int64_t size) {
  return {p, ((rows - 1) * stride + row) * size};
}

bool act_dtype(int dt) { return dt == MOE_DTYPE_BF16 || dt == MOE_DTYPE_F16; }

// What both forms of the attention call take.
moe_status attention_args(AttentionArgs* a, const void* q, int64_t q_stride, int32_t T, int32_t q_heads, int32_t dtype,
                          const moe_kv_cache* cache, const moe_seq_batch* batch, float scale, int32_t window, void* out,
                          int64_t out_stride, float* lse, void* ws, size_t ws_bytes) {
  moe_status st = check_cache(cache);
  if (st != MOE_OK) return st;
  if ((st = check_batch(batch)) != MOE_OK) return st;
  if (T <= 0 || !act_dtype(dtype) || window < 0) return MOE_ERR_INVALID_ARG;
  if (q_heads <= 0 || q_heads % cache->kv_heads != 0) return MOE_ERR_INVALID_ARG;
  if (!(scale > 0.0f) || scale > 1e30f) return MOE_ERR_INVALID_ARG;
  if ((st = check_rows(q, q_stride, (int64_t)q_heads * cache->head_dim)) != MOE_OK) return st;
  if ((st = check_rows(out, out_stride, (int64_t)q_heads * cache->head_dim)) != MOE_OK) return st;
  if (!aligned(lse, 4)) return MOE_ERR_INVALID_ARG;
  if (T >= (1 << 24) || (int64_t)T * q_heads >= (1LL << 31)) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)batch->max_pages * cache->page_size > (1LL << 30)) return MOE_ERR_UNSUPPORTED;
  if ((st = check_ws(ws, ws_bytes, attention_ws_bytes(q_heads, cache->kv_heads, cache->head_dim))) != MOE_OK)
    return st;
  a->c = *cache;
  a->b = *batch;
  a->T = T;
  a->q_heads = q_heads;
  a->dtype = dtype;
  a->window = window;
  a->scale = scale;
  a->q = static_cast<const uint16_t*>(q);
  a->out = static_cast<uint16_t*>(out);
  a->q_stride = q_stride;
  a->out_stride = out_stride;
  a->lse = lse;
  a->ws = static_cast<char*>(ws);
  return MOE_OK;
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_kv_append_workspace_bytes(void) { return kAlign; }

moe_status moe_kv_append_rope_e4m3(const moe_kv_cache* cache, const moe_seq_batch* batch, int32_t T,
                                   const void* k, int64_t k_stride, const void* v,
                                   int64_t v_stride, const void* q, int64_t q_stride, void* q_out,
                                   int64_t q_out_stride, int32_t q_heads, int32_t dtype,
                                   const float* cos, const float* sin, int32_t max_pos,
                                   int32_t rotary_dim, int32_t interleaved,
                                   const int32_t* positions, void* ws, size_t ws_bytes,
                                   void* stream) {
  moe_status st = check_cache(cache);
  if (st != MOE_OK) return st;
  if ((st = check_batch(batch)) != MOE_OK) return st;
  if (T <= 0 || !act_dtype(dtype)) return MOE_ERR_INVALID_ARG;
  const int D = cache->head_dim;
  const int64_t kv_row = (int64_t)cache->kv_heads * D;
  if ((st = check_rows(k, k_stride, kv_row)) != MOE_OK) return st;
  if ((st = check_rows(v, v_stride, kv_row)) != MOE_OK) return st;
  if (q) {
    if (q_heads <= 0 || q_heads > 65536) return MOE_ERR_INVALID_ARG;
    if ((st = check_rows(q, q_stride, (int64_t)q_heads * D)) != MOE_OK) return st;
    if ((st = check_rows(q_out, q_out_stride, (int64_t)q_heads * D)) != MOE_OK) return st;
    if ((int64_t)T * q_heads >= (1LL << 30)) return MOE_ERR_UNSUPPORTED;
  }
  if (rotary_dim < 0 || rotary_dim > D || rotary_dim % 16 != 0) return MOE_ERR_INVALID_ARG;
  if (rotary_dim > 0 && (!cos || !sin || !aligned(cos, 16) || !aligned(sin, 16) || max_pos <= 0))
    return MOE_ERR_INVALID_ARG;
  if (T >= (1 << 24)) return MOE_ERR_UNSUPPORTED;
  if ((st = check_ws(ws, ws_bytes, moe_kv_append_workspace_bytes())) != MOE_OK) return st;
  KvAppendArgs a = {};
  a.c = *cache;
  a.b = *batch;
  a.T = T;
  a.q_heads = q ? q_heads : 0;
  a.max_pos = max_pos;
  a.rotary = rotary_dim;
  a.interleaved = interleaved != 0;
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q = static_cast<const uint16_t*>(q);
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_stride = q_stride;
  a.q_out_stride = q_out_stride;
  a.cos = cos;
  a.sin = sin;
  a.positions = positions;
  a.err = static_cast<uint32_t*>(ws);
  return from_cuda(launch_kv_append(a, dtype, static_cast<cudaStream_t>(stream)));
}

size_t moe_attention_workspace_bytes(int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
  if (q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads != 0) return 0;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
  return attention_ws_bytes(q_heads, kv_heads, head_dim);
}

moe_status moe_attention_paged_e4m3(const void* q, int64_t q_stride, int32_t T, int32_t q_heads,
                                    int32_t dtype, const moe_kv_cache* cache,
                                    const moe_seq_batch* batch, float scale, int32_t window,
                                    void* out, int64_t out_stride, float* lse, void* ws,
                                    size_t ws_bytes, void* stream) {
  AttentionArgs a = {};
  moe_status st = attention_args(&a, q, q_stride, T, q_heads, dtype, cache, batch, scale, window, out, out_stride,
                                 lse, ws, ws_bytes);
  if (st != MOE_OK) return st;
  return from_cuda(launch_attention(a, static_cast<cudaStream_t>(stream)));
}

moe_status moe_attention_tree_e4m3(const void* q, int64_t q_stride, int32_t T, int32_t q_heads,
                                   int32_t dtype, const moe_kv_cache* cache,
                                   const moe_seq_batch* batch, const uint32_t* tree_mask,
                                   int32_t tree_words, int64_t tree_stride, float scale,
                                   int32_t window, void* out, int64_t out_stride, float* lse,
                                   void* ws, size_t ws_bytes, void* stream) {
  if (!tree_mask || !aligned(tree_mask, 4) || tree_words <= 0 || tree_stride < tree_words)
    return MOE_ERR_INVALID_ARG;
  if (tree_words > kMaxTreeWords) return MOE_ERR_UNSUPPORTED;
  AttentionArgs a = {};
  moe_status st = attention_args(&a, q, q_stride, T, q_heads, dtype, cache, batch, scale, window, out, out_stride,
                                 lse, ws, ws_bytes);
  if (st != MOE_OK) return st;
  a.tree = tree_mask;
  a.tree_words = tree_words;
  a.tree_stride = tree_stride;
  return from_cuda(launch_attention(a, static_cast<cudaStream_t>(stream)));
}

size_t moe_kv_keep_workspace_bytes(void) { return kAlign; }

moe_status moe_kv_keep_e4m3(const moe_kv_cache* cache, const moe_seq_batch* batch,
                            const int32_t* keep, const int32_t* n_keep, int32_t width,
                            int32_t* new_lens, void* ws, size_t ws_bytes, void* stream) {
  moe_status st = check_cache(cache);
  if (st != MOE_OK) return st;
  if ((st = check_batch(batch)) != MOE_OK) return st;
  if (width < 0 || (width > 0 && !keep) || !n_keep || !new_lens) return MOE_ERR_INVALID_ARG;
  if (!aligned(keep, 4) || !aligned(n_keep, 4) || !aligned(new_lens, 4)) return MOE_ERR_INVALID_ARG;
  // blocks of other heads read these while a block writes new_lens
  if (new_lens == batch->seq_lens || new_lens == batch->q_offsets || new_lens == n_keep || new_lens == keep)
    return MOE_ERR_INVALID_ARG;
  if ((int64_t)batch->max_pages * cache->page_size > (1LL << 30) || width > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  if ((st = check_ws(ws, ws_bytes, moe_kv_keep_workspace_bytes())) != MOE_OK) return st;
  const Span lens = {new_lens, (int64_t)batch->B * 4};
  for (const Span& in : {Span{batch->seq_lens, (int64_t)batch->B * 4}, Span{batch->q_offsets, ((int64_t)batch->B + 1) * 4},
                         table_span(batch->page_table, batch->B, batch->table_stride, batch->max_pages),
                         Span{n_keep, (int64_t)batch->B * 4}, Span{keep, (int64_t)batch->B * width * 4}})
    if (overlap(lens, in)) return MOE_ERR_INVALID_ARG;
  KeepArgs a = {};
  a.c = *cache;
  a.b = *batch;
  a.keep = keep;
  a.n_keep = n_keep;
  a.width = width;
  a.new_lens = new_lens;
  a.err = static_cast<uint32_t*>(ws);
  return from_cuda(launch_keep(a, static_cast<cudaStream_t>(stream)));
}

size_t moe_kv_weights_workspace_bytes(int32_t T, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
  if (T <= 0 || q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads != 0) return 0;
  if (T >= (1 << 24) || (int64_t)T * q_heads >= (1LL << 30)) return 0;
  if (head_dim != 64 && head_dim != 128 && head_dim != 256) return 0;
  return kv_weights_ws_bytes(T, q_heads, kv_heads, head_dim);
}

moe_status moe_kv_weights_e4m3(const void* q, int64_t q_stride, int32_t T, int32_t q_heads,
                               int32_t dtype, const float* lse, const moe_kv_cache* cache,
                               const moe_seq_batch* batch, float scale, int32_t window, float decay,
                               const float* w, float* w_out, void* ws, size_t ws_bytes,
                               void* stream) {
  moe_status st = check_cache(cache);
  if (st != MOE_OK) return st;
  if ((st = check_batch(batch)) != MOE_OK) return st;
  if (T <= 0 || !act_dtype(dtype) || window < 0) return MOE_ERR_INVALID_ARG;
  if (q_heads <= 0 || q_heads % cache->kv_heads != 0) return MOE_ERR_INVALID_ARG;
  if (!(scale > 0.0f) || scale > 1e30f || !(decay >= 0.0f && decay <= 1.0f)) return MOE_ERR_INVALID_ARG;
  if ((st = check_rows(q, q_stride, (int64_t)q_heads * cache->head_dim)) != MOE_OK) return st;
  if (!lse || !w || !w_out || !aligned(lse, 4) || !aligned(w, 16) || !aligned(w_out, 16)) return MOE_ERR_INVALID_ARG;
  if (T >= (1 << 24) || (int64_t)T * q_heads >= (1LL << 30)) return MOE_ERR_UNSUPPORTED;
  if ((int64_t)batch->max_pages * cache->page_size > (1LL << 30)) return MOE_ERR_UNSUPPORTED;
  if ((st = check_ws(ws, ws_bytes, kv_weights_ws_bytes(T, q_heads, cache->kv_heads, cache->head_dim))) != MOE_OK)
    return st;
  // the new weights on the old ones slot by slot or not at all, and on nothing that is read beside
  const int64_t plane = (int64_t)cache->num_pages * cache->kv_heads * cache->page_size * 4;
  if ((w != w_out && overlap({w, plane}, {w_out, plane})) || overlap({w_out, plane}, {lse, (int64_t)T * q_heads * 4}) ||
      overlap({w_out, plane}, rows_span(q, T, q_stride, (int64_t)q_heads * cache->head_dim, 2)))
    return MOE_ERR_INVALID_ARG;
  WeightsArgs a = {};
  a.c = *cache;
  a.b = *batch;
  a.T = T;
  a.q_heads = q_heads;
  a.dtype = dtype;
  a.window = window;
  a.scale = scale;
  a.decay = decay;
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.lse = lse;
  a.w = w;
  a.w_out = w_out;
  a.ws = static_cast<char*>(ws);
  return from_cuda(launch_kv_weights(a, static_cast<cudaStream_t>(stream)));
}

size_t moe_kv_evict_workspace_bytes(int32_t B, int32_t kv_heads) {
  if (B <= 0 || B > 65536 || kv_heads <= 0 || kv_heads > 1024) return 0;
  return kAlign;
}

moe_status moe_kv_evict_e4m3(const moe_kv_cache* cache, const moe_seq_batch* batch, float* w,
                             const int32_t* dst_table, int32_t dst_stride, const int32_t* budgets,
                             int32_t width, int32_t first, int32_t recent, int32_t* kept,
                             int32_t* new_lens, void* ws, size_t ws_bytes, void* stream) {
  moe_status st = check_cache(cache);
  if (st != MOE_OK) return st;
  if ((st = check_batch(batch)) != MOE_OK) return st;
  if (width <= 0 || first < 0 || recent < 0 || !w || !dst_table || !kept || !new_lens) return MOE_ERR_INVALID_ARG;
  if (!aligned(w, 4) || !aligned(dst_table, 4) || !aligned(budgets, 4) || !aligned(kept, 4) || !aligned(new_lens, 4))
    return MOE_ERR_INVALID_ARG;
  // blocks of other heads read these while a block writes new_lens; old pages are only read
  if (new_lens == batch->seq_lens || new_lens == budgets || new_lens == kept || dst_table == batch->page_table)
    return MOE_ERR_INVALID_ARG;
  if ((int64_t)batch->max_pages * cache->page_size > (1LL << 30) || width > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  const int64_t pages = ((int64_t)width + cache->page_size - 1) / cache->page_size;
  if (dst_stride < pages) return MOE_ERR_INVALID_ARG;
  if (pages * batch->B * cache->kv_heads >= (1LL << 31)) return MOE_ERR_UNSUPPORTED;
  if ((st = check_ws(ws, ws_bytes, moe_kv_evict_workspace_bytes(batch->B, cache->kv_heads))) != MOE_OK) return st;
  // blocks read the batch, the budgets and the tables (and the second kernel the lists) while others write
  const Span lens = {new_lens, (int64_t)batch->B * 4}, lists = {kept, (int64_t)batch->B * cache->kv_heads * width * 4};
  const Span plane = {w, (int64_t)cache->num_pages * cache->kv_heads * cache->page_size * 4};
  for (const Span& out : {lens, lists, plane})
    for (const Span& in : {Span{batch->seq_lens, (int64_t)batch->B * 4}, Span{budgets, (int64_t)batch->B * 4},
                           table_span(batch->page_table, batch->B, batch->table_stride, batch->max_pages),
                           table_span(dst_table, batch->B, dst_stride, pages)})
      if (overlap(out, in)) return MOE_ERR_INVALID_ARG;
  if (overlap(lens, lists) || overlap(lens, plane) || overlap(lists, plane)) return MOE_ERR_INVALID_ARG;
  EvictArgs a = {};
  a.c = *cache;
  a.b = *batch;
  a.w = w;
  a.dst_table = dst_table;
  a.budgets = budgets;
  a.dst_stride = dst_stride;
  a.width = width;
  a.first = first;
  a.recent = recent;
  a.kept = kept;
  a.new_lens = new_lens;
  a.err = static_cast<uint32_t*>(ws);
  return from_cuda(launch_evict(a, static_cast<cudaStream_t>(stream)));
}

moe_status moe_residual_norm(const void* y, int64_t y_stride, int32_t y_dtype, const void* residual,
                             int64_t residual_stride, void* out, int64_t out_stride,
                             int32_t residual_dtype, void* normed, int64_t normed_stride,
                             int32_t normed_dtype, int32_t T, int32_t H, const void* post_weight,
                             const void* pre_weight, int32_t weight_dtype, const void* gate,
                             int64_t gate_stride, int32_t gate_inner, int32_t gate_dtype,
                             int32_t gate_sigmoid, float scale, float eps, float weight_offset,
                             void* stream) {
  auto known = [](int dt) { return act_dtype(dt) || dt == MOE_DTYPE_F32; };
  auto size = [](int dt) { return dt == MOE_DTYPE_F32 ? 4 : 2; };
  if (T <= 0 || H <= 0 || !residual || (!out && !normed)) return MOE_ERR_INVALID_ARG;
  if (!y && (post_weight || gate)) return MOE_ERR_INVALID_ARG;
  if (!known(residual_dtype) || (y && !known(y_dtype)) || (normed && !known(normed_dtype))) return MOE_ERR_INVALID_ARG;
  if (((post_weight || pre_weight) && !known(weight_dtype)) || (gate && !known(gate_dtype))) return MOE_ERR_INVALID_ARG;
  if (pre_weight && !normed) return MOE_ERR_INVALID_ARG;
  if (!(eps >= 0.0f && eps < INFINITY) || !isfinite(scale) || !isfinite(weight_offset)) return MOE_ERR_INVALID_ARG;
  if (gate && (gate_inner < 0 || gate_inner > 1 || gate_stride < 0)) return MOE_ERR_INVALID_ARG;
  if (H > 32768 || T > (1 << 30)) return MOE_ERR_UNSUPPORTED;
  if (!aligned(residual, size(residual_dtype)) || !aligned(out, size(residual_dtype)) ||
      (y && !aligned(y, size(y_dtype))) || (normed && !aligned(normed, size(normed_dtype))) ||
      !aligned(post_weight, size(weight_dtype)) || !aligned(pre_weight, size(weight_dtype)) ||
      (gate && !aligned(gate, size(gate_dtype))))
    return MOE_ERR_INVALID_ARG;
  if (T > 1 && (residual_stride < H || (out && out_stride < H) || (y && y_stride < H) || (normed && normed_stride < H)))
    return MOE_ERR_INVALID_ARG;
  // an output may lie on an input only row by row and value by value
  auto on = [&](const void* p, int64_t ps, int pd, const void* in, int64_t is, int id) {
    return !p || p != in || ((T == 1 || ps == is) && pd == id);
  };
  if (!on(out, out_stride, residual_dtype, residual, residual_stride, residual_dtype) ||
      !on(out, out_stride, residual_dtype, y, y_stride, y_dtype) ||
      !on(normed, normed_stride, normed_dtype, residual, residual_stride, residual_dtype) ||
      !on(normed, normed_stride, normed_dtype, y, y_stride, y_dtype) || (out && out == normed))
    return MOE_ERR_INVALID_ARG;
  for (const void* in : {gate, post_weight, pre_weight})         // which other rows may share
    if (in && (in == out || in == normed)) return MOE_ERR_INVALID_ARG;
  NormArgs a = {};
  a.y = y;
  a.residual = residual;
  a.out = out;
  a.normed = normed;
  a.post = post_weight;
  a.pre = pre_weight;
  a.gate = gate;
  a.y_stride = y_stride;
  a.residual_stride = residual_stride;
  a.out_stride = out_stride;
  a.normed_stride = normed_stride;
  a.gate_stride = gate_stride;
  a.T = T;
  a.H = H;
  a.y_dtype = y ? y_dtype : residual_dtype;
  a.residual_dtype = residual_dtype;
  a.normed_dtype = normed_dtype;
  a.weight_dtype = weight_dtype;
  a.gate_dtype = gate_dtype;
  a.gate_inner = gate ? gate_inner : 0;
  a.sigmoid = gate_sigmoid != 0;
  a.scale = scale;
  a.eps = eps;
  a.offset = weight_offset;
  return from_cuda(launch_norm(a, static_cast<cudaStream_t>(stream)));
}

size_t moe_linear_workspace_bytes(int32_t T, int32_t N, int32_t K) {
  if (T <= 0 || N <= 0 || K <= 0 || K % 32 != 0 || K > 65536) return 0;
  return linear_ws_bytes(T, N, K);
}

moe_status moe_linear_nvfp4(const void* x, int64_t x_stride, int32_t x_dtype, int32_t T,
                            const moe_nvfp4_bank* w, void* y, int64_t y_stride, int32_t y_dtype,
                            void* ws, size_t ws_bytes, void* stream) {
  if (!w || !w->codes || !w->scales || !aligned(w->codes, 16) || !aligned(w->scales, 16))
    return MOE_ERR_INVALID_ARG;
  if (w->E != 1 || w->rows <= 0 || w->in_f <= 0 || T <= 0) return MOE_ERR_INVALID_ARG;
  if (!act_dtype(x_dtype) || (!act_dtype(y_dtype) && y_dtype != MOE_DTYPE_F32))
    return MOE_ERR_INVALID_ARG;
  if (w->in_f % 32 != 0 || w->in_f > 65536) return MOE_ERR_UNSUPPORTED;
  if (T > 65535 || (int64_t)T * w->rows >= (1LL << 40)) return MOE_ERR_UNSUPPORTED;
  moe_status st = check_rows(x, x_stride, w->in_f);
  if (st != MOE_OK) return st;
  if (!y || !aligned(y, y_dtype == MOE_DTYPE_F32 ? 4 : 2) || y_stride < w->rows)
    return MOE_ERR_INVALID_ARG;
  if ((st = check_ws(ws, ws_bytes, linear_ws_bytes(T, w->rows, w->in_f))) != MOE_OK) return st;
  LinearArgs a = {};
  a.x = static_cast<const uint16_t*>(x);
  a.x_stride = x_stride;
  a.y_stride = y_stride;
  a.T = T;
  a.N = w->rows;
  a.K = w->in_f;
  a.x_dtype = x_dtype;
  a.y_dtype = y_dtype;
  a.codes = w->codes;
  a.scales = w->scales;
  a.alpha = w->alpha;
  a.y = y;
  a.ws = static_cast<char*>(ws);
  return from_cuda(launch_linear(a, static_cast<cudaStream_t>(stream)));
}

size_t moe_verify_workspace_bytes(int32_t B, int32_t V) {
  if (B <= 0 || V <= 0 || V > (1 << 22)) return 0;
  return verify_ws_bytes(B, V);
}

moe_status moe_verify_draft(const int32_t* draft_ids, const int32_t* n_draft, int32_t B, int32_t n,
                            int32_t V, const void* target_probs, int64_t target_stride,
                            const void* draft_probs, int64_t draft_stride, int32_t dtype,
                            const float* u_accept, const float* u_sample, int32_t* out_ids,
                            int32_t* n_accepted, void* ws, size_t ws_bytes, void* stream) {
  if (B <= 0 || n < 0 || V <= 0) return MOE_ERR_INVALID_ARG;
  if (!target_probs || !u_sample || !out_ids || !n_accepted) return MOE_ERR_INVALID_ARG;
  if (n > 0 && (!draft_ids || !u_accept)) return MOE_ERR_INVALID_ARG;
  if (!act_dtype(dtype) && dtype != MOE_DTYPE_F32) return MOE_ERR_INVALID_ARG;
  const uintptr_t size = dtype == MOE_DTYPE_F32 ? 4 : 2;
  if (!aligned(target_probs, size) || !aligned(draft_probs, size)) return MOE_ERR_INVALID_ARG;
  if (target_stride < V || (draft_probs && draft_stride < V)) return MOE_ERR_INVALID_ARG;
  if (n > 64 || V > (1 << 22) || B > 65535) return MOE_ERR_UNSUPPORTED;
  moe_status st = check_ws(ws, ws_bytes, verify_ws_bytes(B, V));
  if (st != MOE_OK) return st;
  VerifyArgs a = {};
  a.draft_ids = draft_ids;
  a.n_draft = n_draft;
  a.B = B;
  a.n = n;
  a.V = V;
  a.target = target_probs;
  a.draft = n > 0 ? draft_probs : nullptr;
  a.target_stride = target_stride;
  a.draft_stride = draft_stride;
  a.u_accept = u_accept;
  a.u_sample = u_sample;
  a.out_ids = out_ids;
  a.n_accepted = n_accepted;
  a.ws = static_cast<char*>(ws);
  return from_cuda(launch_verify(a, dtype, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
