// Declarations shared by the serving operators' translation units (moe_serving.h).
#pragma once

#include <cuda_bf16.h>

#include "moe_internal.cuh"
#include "moe_serving.h"

namespace moe {

struct KvAppendArgs {
  moe_kv_cache c;
  moe_seq_batch b;
  int T, q_heads, max_pos, rotary, interleaved;
  const uint16_t *k, *v, *q;
  uint16_t* q_out;
  int64_t k_stride, v_stride, q_stride, q_out_stride;
  const float *cos, *sin;
  const int32_t* positions;
  uint32_t* err;
};
cudaError_t launch_kv_append(const KvAppendArgs& a, int dtype, cudaStream_t s);

struct AttentionArgs {
  moe_kv_cache c;
  moe_seq_batch b;
  int T, q_heads, dtype, window;
  int max_rows;                // sequences with more rows are left to the other form
  float scale;
  const uint16_t* q;
  uint16_t* out;
  int64_t q_stride, out_stride;
  float* lse;
  char* ws;
  const uint32_t* tree;        // bits of the new tokens that a token sees (null: causal)
  int64_t tree_stride;
  int tree_words;
};
constexpr int kMaxTreeWords = 8;
size_t attention_ws_bytes(int q_heads, int kv_heads, int head_dim);
cudaError_t launch_attention(const AttentionArgs& a, cudaStream_t s);

// The form for sequences of at least min_rows rows (new tokens times query heads per key head);
// head_dim 64 or 128. Its workspace begins ws_at bytes into a.ws.
constexpr int kPromptMaxGrid = 160;
size_t prompt_attention_ws_bytes(int head_dim);
cudaError_t launch_prompt_attention(const AttentionArgs& a, int min_rows, size_t ws_at, cudaStream_t s);

struct LinearArgs {
  const uint16_t* x;
  int64_t x_stride, y_stride;
  int T, N, K, x_dtype, y_dtype;
  const uint8_t *codes, *scales;
  const float* alpha;
  void* y;
  char* ws;
};
size_t linear_ws_bytes(int T, int N, int K);
cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s);

struct VerifyArgs {
  const int32_t *draft_ids, *n_draft;
  int B, n, V;
  const void *target, *draft;
  int64_t target_stride, draft_stride;
  const float *u_accept, *u_sample;
  int32_t *out_ids, *n_accepted;
  char* ws;
};
size_t verify_ws_bytes(int B, int V);
cudaError_t launch_verify(const VerifyArgs& a, int dtype, cudaStream_t s);

struct KeepArgs {
  moe_kv_cache c;
  moe_seq_batch b;
  const int32_t *keep, *n_keep;
  int width;
  int32_t* new_lens;
  uint32_t* err;
};
cudaError_t launch_keep(const KeepArgs& a, cudaStream_t s);

struct EvictArgs {
  moe_kv_cache c;
  moe_seq_batch b;
  float* w;
  const int32_t *dst_table, *budgets;
  int dst_stride, width, first, recent;
  int32_t *kept, *new_lens;
  uint32_t* err;
};
cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s);

struct WeightsArgs {
  moe_kv_cache c;
  moe_seq_batch b;
  int T, q_heads, dtype, window;
  float scale, decay;
  const uint16_t* q;
  int64_t q_stride;
  const float* lse;
  const float* w;
  float* w_out;
  char* ws;
};
size_t kv_weights_ws_bytes(int T, int q_heads, int kv_heads, int head_dim);
cudaError_t launch_kv_weights(const WeightsArgs& a, cudaStream_t s);

struct NormArgs {
  const void *y, *residual;
  void *out, *normed;
  const void *post, *pre, *gate;
  int64_t y_stride, residual_stride, out_stride, normed_stride, gate_stride;
  int T, H, y_dtype, residual_dtype, normed_dtype, weight_dtype, gate_dtype;
  int gate_inner, sigmoid;
  float scale, eps, offset;
};
cudaError_t launch_norm(const NormArgs& a, cudaStream_t s);

// 16-bit activations as f32 and back (nearest even).
template <int DT>
__device__ __forceinline__ float act_to_f32(uint32_t bits16) {
  if (DT == MOE_DTYPE_BF16) return __uint_as_float(bits16 << 16);
  return __half2float(__ushort_as_half((unsigned short)bits16));
}
template <int DT>
__device__ __forceinline__ uint32_t f32_to_act(float v) {
  if (DT == MOE_DTYPE_BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
  return __half_as_ushort(__float2half_rn(v));
}
template <int DT>
__device__ __forceinline__ void unpack8(const uint4& r, float (&f)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = act_to_f32<DT>(w[i] & 0xffffu);
    f[2 * i + 1] = act_to_f32<DT>(w[i] >> 16);
  }
}
template <int DT>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = f32_to_act<DT>(f[2 * i]) | (f32_to_act<DT>(f[2 * i + 1]) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Two floats to two E4M3 codes (low byte = a), nearest even, finite values saturating at 448.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
__device__ __forceinline__ float2 e4m3x2_to_f32x2(uint32_t v) {
  const uint32_t h = e4m3x2_to_f16x2(v);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Which of a word's four E4M3 codes are NaN (0x7f, 0xff): the top bit of each such byte.
__device__ __forceinline__ uint32_t e4m3_nan_bits(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}
// Calls put(d) for every value d of a row of D codes that is NaN.
template <int D, class F>
__device__ __forceinline__ void each_nan(const uint8_t* codes, F&& put) {
#pragma unroll 1
  for (int d = 0; d < D; d += 4)
    for (uint32_t m = e4m3_nan_bits(*reinterpret_cast<const uint32_t*>(codes + d)); m; m &= m - 1)
      put(d + (__ffs(m) - 1) / 8);
}

// Loads that stay where they are written: the compiler may move an ordinary load behind a wait, next
// to its use, and expose its latency there.
__device__ __forceinline__ uint4 load_ahead(const void* at, bool there) {   // zeros if not there
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\t"
      "mov.b32 %3, 0;\n\t@p ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(at), "r"((int)there) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t load_ahead(const void* at, bool there, uint32_t other) {
  uint32_t v;
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b32 %0, %3;\n\t@p ld.global.nc.b32 %0, [%1];\n\t}"
               : "=r"(v) : "l"(at), "r"((int)there), "r"(other) : "memory");
  return v;
}


// What token row `token` (of a sequence with n new tokens, the first at place `start`) sees of its tree:
// the bits of the new tokens, and as the value returned the first of the tokens before them. With a
// window that is the end of the row's chain: tokens before the new ones, then those of its bits.
__device__ __forceinline__ int tree_row(const AttentionArgs& a, int64_t token, bool there, int n, int start,
                                        uint32_t (&w)[kMaxTreeWords]) {
  int m = 0;
#pragma unroll
  for (int i = 0; i < kMaxTreeWords; ++i) {
    const int left = n - 32 * i;               // bits that are tokens
    w[i] = there && i < a.tree_words && left > 0 ? a.tree[token * a.tree_stride + i] : 0u;
    if (left < 32 && left > 0) w[i] &= (1u << left) - 1;
    m += __popc(w[i]);
  }
  if (a.window <= 0) return 0;
#pragma unroll
  for (int i = 0; i < kMaxTreeWords; ++i)
    for (; m > a.window && w[i]; --m) w[i] &= w[i] - 1;
  return max(0, start + m - a.window);
}

}  // namespace moe
