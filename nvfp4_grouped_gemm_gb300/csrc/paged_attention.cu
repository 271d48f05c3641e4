// Causal attention of new tokens over the paged 8-bit cache (moe_attention_paged_e4m3).
//
// One warp per (token, query head): the warp walks the visible keys once, keeping the running
// maximum and sum of the softmax and its D/32 output values per lane in f32.
#include "serving.cuh"

namespace moe {
namespace {

template <int DT, int D>
__global__ void __launch_bounds__(128) attention_kernel(const AttentionArgs a) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (w >= (long long)a.T * a.q_heads) return;
  const int t = (int)(w / a.q_heads), r = (int)(w % a.q_heads);
  const int h = r / (a.q_heads / a.c.kv_heads);
  uint32_t* err = reinterpret_cast<uint32_t*>(a.ws);
  int lo = 0, hi = a.b.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.b.q_offsets[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  const int P = a.c.page_size;
  const long long cap = (long long)a.b.max_pages * P;
  int len = a.b.seq_lens[lo];
  const int place = len - a.b.q_offsets[lo + 1] + t;
  if (place < 0 && lane == 0) atomicOr(err, (uint32_t)MOE_DEVERR_PAGE);
  if (len > cap) {
    if (lane == 0) atomicOr(err, (uint32_t)MOE_DEVERR_PAGE);
    len = (int)cap;
  }
  const int j1 = min(place + 1, len), j0 = a.window > 0 ? max(0, place - a.window + 1) : 0;
  const uint16_t* q = a.q + (int64_t)t * a.q_stride + (int64_t)r * D + lane * N;
  float qv[N], o[N];
#pragma unroll
  for (int i = 0; i < N; ++i) qv[i] = act_to_f32<DT>(q[i]), o[i] = 0.0f;
  float m = -INFINITY, l = 0.0f;
  for (int j = j0; j < j1; ++j) {
    const int64_t page = a.b.page_table[(int64_t)lo * a.b.table_stride + j / P];
    if (page < 0 || page >= a.c.num_pages) {
      if (lane == 0) atomicOr(err, (uint32_t)MOE_DEVERR_PAGE);
      continue;
    }
    const int64_t at = page * a.c.page_stride + ((int64_t)h * P + j % P) * D + lane * N;
    float s = 0.0f;
    float kv[N], vv[N];
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 kk = e4m3x2_to_f32x2(*reinterpret_cast<const uint16_t*>(a.c.k_codes + at + i));
      const float2 vp = e4m3x2_to_f32x2(*reinterpret_cast<const uint16_t*>(a.c.v_codes + at + i));
      kv[i] = kk.x, kv[i + 1] = kk.y, vv[i] = vp.x, vv[i + 1] = vp.y;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) s = fmaf(qv[i], kv[i], s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= a.scale * a.c.k_scales[page * a.c.kv_heads + h];
    const float vs = a.c.v_scales[page * a.c.kv_heads + h];
    const float mn = fmaxf(m, s);
    const float keep = expf(m - mn), p = expf(s - mn);
    l = l * keep + p;
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = o[i] * keep + p * vs * vv[i];
    m = mn;
  }
  uint16_t* out = a.out + (int64_t)t * a.out_stride + (int64_t)r * D + lane * N;
#pragma unroll
  for (int i = 0; i < N; ++i) out[i] = (uint16_t)f32_to_act<DT>(l > 0.0f ? o[i] / l : 0.0f);
  if (a.lse && lane == 0) a.lse[(int64_t)t * a.q_heads + r] = l > 0.0f ? m + logf(l) : -INFINITY;
}

template <int DT>
void launch_dim(const AttentionArgs& a, cudaStream_t s) {
  const unsigned grid = (unsigned)(((long long)a.T * a.q_heads + 3) / 4);
  if (a.c.head_dim == 64) attention_kernel<DT, 64><<<grid, 128, 0, s>>>(a);
  else if (a.c.head_dim == 128) attention_kernel<DT, 128><<<grid, 128, 0, s>>>(a);
  else attention_kernel<DT, 256><<<grid, 128, 0, s>>>(a);
}

}  // namespace

size_t attention_ws_bytes(int q_heads, int kv_heads, int head_dim) { return kAlign; }

cudaError_t launch_attention(const AttentionArgs& a, int dtype, cudaStream_t s) {
  if (dtype == MOE_DTYPE_BF16) launch_dim<MOE_DTYPE_BF16>(a, s);
  else launch_dim<MOE_DTYPE_F16>(a, s);
  return cudaGetLastError();
}

}  // namespace moe
