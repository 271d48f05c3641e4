/*
 * moe_serving.h -- C ABI of the serving operators around the routed MoE layer of moe.h (same
 * library, libmoe_gb300.so): what the other half of a transformer block and a speculative
 * decoding step need on the same GPU.
 *
 *   moe_linear_nvfp4          y = x W^T for a few tokens, W in NVFP4 (projections, LM head)
 *   moe_kv_append_rope_e4m3   new keys and values into a paged 8-bit cache, rotated by their
 *                             positions on the way (and the queries beside them)
 *   moe_attention_paged_e4m3  causal attention of the new tokens over that cache
 *   moe_verify_draft          accepts or refuses drafted tokens against the target's
 *                             probabilities, with the random numbers given
 *
 * The conventions of moe.h hold: array pointers are DEVICE pointers owned by the caller;
 * calls are asynchronous on `stream`, allocate nothing and can be captured in a CUDA graph;
 * sizes are checked on the host before anything is launched; no call prints, aborts or
 * throws. Every call takes a workspace `ws` (256-byte aligned, zero-filled once after it is
 * allocated, of the bytes its size function returns) whose first word is the device error
 * word of moe_get_device_error. A workspace serves any number of calls in one stream, of the
 * sizes it was made for and smaller ones (the attention's of its head_dim); calls that can
 * overlap need one each. After MOE_DEVERR_TIMEOUT zero-fill it again.
 */
#ifndef MOE_GB300_SERVING_H
#define MOE_GB300_SERVING_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of activations and probabilities. */
enum { MOE_DTYPE_BF16 = 0, MOE_DTYPE_F16 = 1, MOE_DTYPE_F32 = 2 };

/* More bits of the device error word.
 *   MOE_DEVERR_PAGE      a page-table entry in use outside [0, num_pages), a sequence longer
 *                        than its row of the page table, or more new tokens than its length
 *                        (the tokens concerned are left out)
 *   MOE_DEVERR_POSITION  a position outside the cos/sin tables (clamped into them)
 *   MOE_DEVERR_TOKEN     a drafted id outside [0, V) (refused)
 *   MOE_DEVERR_PROBS     a target row without any mass (the token drawn from it is -1) */
enum { MOE_DEVERR_PAGE = 4, MOE_DEVERR_POSITION = 8, MOE_DEVERR_TOKEN = 16, MOE_DEVERR_PROBS = 32 };

/* Paged key/value cache in 8 bits with one scale for each block of tokens (a page) and head:
 *   codes   E4M3 [num_pages][kv_heads][page_size][head_dim]; page p of either plane starts
 *           page_stride bytes after page p-1 (a multiple of 16, at least
 *           kv_heads*page_size*head_dim, so both planes can share one allocation)
 *   scales  f32 [num_pages][kv_heads], contiguous, positive and finite; V's within
 *           [2^-100, 2^120] (an append writes [2^-64, 2^119])
 *   value(page, head, slot, d) = E4M3(code) * scale[page][head]
 * page_size is 16, 32, 64 or 128; head_dim 64, 128 or 256; code planes 16-byte aligned. */
typedef struct moe_kv_cache {
  uint8_t* k_codes;
  uint8_t* v_codes;
  float* k_scales;
  float* v_scales;
  int32_t num_pages, kv_heads, page_size, head_dim;
  int64_t page_stride;
} moe_kv_cache;

/* A ragged batch of B sequences: sequence b's new tokens are rows q_offsets[b] ..
 * q_offsets[b+1]-1 of the token arrays and the last of its seq_lens[b] tokens (the new ones
 * counted); token i of it lives in page page_table[b][i / page_size], slot i % page_size.
 *   q_offsets  i32 [B+1] not descending, from 0 to the number of token rows T
 *   seq_lens   i32 [B]
 *   page_table i32 [B][table_stride], max_pages columns of it in use; entries past a
 *              sequence's last page are not read
 * A sequence may have no new token, or no token at all. */
typedef struct moe_seq_batch {
  const int32_t* q_offsets;
  const int32_t* seq_lens;
  const int32_t* page_table;
  int32_t B, max_pages, table_stride;
} moe_seq_batch;

/* ---- keys and values into the cache ------------------------------------------------- */

size_t moe_kv_append_workspace_bytes(void);

/* Appends the batch's T new tokens to the cache. k and v are dtype (bf16 or f16)
 * [T][kv_heads][head_dim], rows k_stride / v_stride elements apart; q (or NULL) is
 * [T][q_heads][head_dim] and q_out, of the same type, may be q itself.
 *
 * Keys and queries are rotated: of each head's first rotary_dim values, pair i (values i and
 * i + rotary_dim/2, or 2i and 2i+1 when `interleaved`) becomes (a c - b s, b c + a s) with
 * c = cos[pos][i], s = sin[pos][i], in f32 with each product rounded once. cos and sin are f32
 * [max_pos][rotary_dim/2]; pos is positions[t], or the token's place in its sequence when
 * positions is NULL. rotary_dim is a multiple of 16, or 0 (no rotation; cos, sin may be NULL).
 *
 * Each touched page and head gets a scale for K and one for V: with a the largest magnitude
 * of its new values and e the least integer with a <= 448 * 2^e (within [-64, 119]), the scale
 * is 2^e for a page whose first slot this call writes, and max(old scale, 2^e) otherwise; where
 * it grows, the codes of the page's earlier slots are rescaled by old / new and rounded again.
 * Codes are rounded to nearest even. Values read back depend on how tokens were split over
 * calls only through that re-rounding. Two sequences must not append to the same page in one
 * call. Token rows need 16-byte aligned starts (pointers 16-byte aligned, strides multiples
 * of 8 elements); cos and sin 16-byte aligned. */
moe_status moe_kv_append_rope_e4m3(const moe_kv_cache* cache, const moe_seq_batch* batch, int32_t T,
                                   const void* k, int64_t k_stride, const void* v,
                                   int64_t v_stride, const void* q, int64_t q_stride, void* q_out,
                                   int64_t q_out_stride, int32_t q_heads, int32_t dtype,
                                   const float* cos, const float* sin, int32_t max_pos,
                                   int32_t rotary_dim, int32_t interleaved,
                                   const int32_t* positions, void* ws, size_t ws_bytes,
                                   void* stream);

/* ---- attention over the cache ------------------------------------------------------- */

size_t moe_attention_workspace_bytes(int32_t q_heads, int32_t kv_heads, int32_t head_dim);

/* Causal attention of the batch's T new tokens over the cache (which already holds them):
 * query head r of a token at place i of its sequence sees the tokens j <= i (and j > i - window
 * when window > 0) of key head r / (q_heads / kv_heads);
 *   s_j = scale * k_scale * (q . K_j),  out = sum_j exp(s_j) v_scale V_j / sum_j exp(s_j),
 *   lse = log sum_j exp(s_j)            (a row that sees nothing: out = 0, lse = -inf).
 * q, out: dtype (bf16 or f16) [T][q_heads][head_dim], rows q_stride / out_stride elements
 * apart (16-byte aligned as above); lse f32 [T][q_heads] or NULL. q_heads is a multiple of
 * kv_heads. Products and sums are held in f32 from f16 operands: q times a power of two
 * (exact for bf16 and f16 values within 2^-28 of the row's largest), E4M3 codes (exact), and
 * the weights exp(s_j - max) v_scale rounded to f16 beside the largest. scale times a page's
 * k_scale times a row's largest |q| has to be finite in f32. Slots past a sequence's end may
 * hold anything, NaN codes included; a NaN code of K or V in use reaches only the rows that
 * see its token (of V: that value of them). */
moe_status moe_attention_paged_e4m3(const void* q, int64_t q_stride, int32_t T, int32_t q_heads,
                                    int32_t dtype, const moe_kv_cache* cache,
                                    const moe_seq_batch* batch, float scale, int32_t window,
                                    void* out, int64_t out_stride, float* lse, void* ws,
                                    size_t ws_bytes, void* stream);

/* ---- matrix-vector products with NVFP4 weights -------------------------------------- */

size_t moe_linear_workspace_bytes(int32_t T, int32_t N, int32_t K);

/* y[t][n] = alpha * sum_k x[t][k] * W[n][k] for T tokens, W a bank of one expert (E = 1) with
 * N rows of in_f = K weights (K a multiple of 32, at most 65536; N any, T <= 65535). x: x_dtype (bf16
 * or f16) [T][K], rows x_stride elements apart (16-byte aligned as above); y: y_dtype (bf16, f16
 * or f32) [T][N], rows y_stride elements apart. Products are exact (x as f16 times a power of
 * two, exact for values within 2^-28 of the row's largest; E2M1 * UE4M3 in f16), sums are f32.
 * The weights are read once per pass of as many tokens as 128 KiB of x in f16 hold, at most 32 (a
 * power of two: 16 at K = 4096, 4 at 16384); the call is made for few tokens. */
moe_status moe_linear_nvfp4(const void* x, int64_t x_stride, int32_t x_dtype, int32_t T,
                            const moe_nvfp4_bank* w, void* y, int64_t y_stride, int32_t y_dtype,
                            void* ws, size_t ws_bytes, void* stream);

/* ---- verification of drafted tokens -------------------------------------------------- */

size_t moe_verify_workspace_bytes(int32_t B, int32_t V);

/* For each of B sequences, n drafted tokens (n_draft[b] <= n of them when n_draft is not NULL)
 * against the target's distributions p_0 .. p_n: drafted token i, id x, is accepted while
 * u_accept[b][i] * q_i(x) < p_i(x) (f32 product; q_i(x) = 1 without draft_probs). At the first
 * refusal i the next token is drawn from max(p_i - q_i, 0) (f32 difference; without draft_probs
 * p_i with x left out); when none is refused, from p_{n_draft}. It is drawn on whole numbers,
 * so it does not depend on an order of summation: the mass of token v is
 * floor(min(w_v, 1) * 2^40) for weight w_v (0 for NaN and below), the goal is
 * floor(floor(u * 2^24) * total / 2^24) with u = u_sample[b] clamped into [0, 1 - 2^-24], and
 * the token is the least v whose masses 0..v sum to more than the goal. A total of 0 falls
 * back to the masses of p_i itself.
 *   draft_ids    i32 [B][n]              n_draft  i32 [B] or NULL
 *   target_probs dtype [B][n+1][V]       draft_probs dtype [B][n][V] or NULL (bf16, f16, f32;
 *                rows target_stride / draft_stride elements apart, contiguous over B and n)
 *   u_accept     f32 [B][n]              u_sample f32 [B]
 *   out_ids      i32 [B][n+1]: the accepted tokens, the drawn one, then -1
 *   n_accepted   i32 [B]
 * 0 <= n <= 64, V <= 2^22. */
moe_status moe_verify_draft(const int32_t* draft_ids, const int32_t* n_draft, int32_t B, int32_t n,
                            int32_t V, const void* target_probs, int64_t target_stride,
                            const void* draft_probs, int64_t draft_stride, int32_t dtype,
                            const float* u_accept, const float* u_sample, int32_t* out_ids,
                            int32_t* n_accepted, void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_GB300_SERVING_H */
