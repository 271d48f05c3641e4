// Verification of drafted tokens with given random numbers (moe_verify_draft).
//
// One block per sequence: it tests the drafted tokens in order, then sums the masses of the row
// the next token is drawn from and walks the row again to the goal. Masses are whole numbers, so
// no order of summation shows in the result.
#include "serving.cuh"

namespace moe {
namespace {

constexpr int kThreads = 512;

template <int DT>
__device__ __forceinline__ float prob(const void* row, int64_t at) {
  if (DT == MOE_DTYPE_F32) return static_cast<const float*>(row)[at];
  return act_to_f32<DT>(static_cast<const uint16_t*>(row)[at]);
}

// floor(min(w, 1) * 2^40); 0 for NaN and negative weights.
__device__ __forceinline__ unsigned long long mass_of(float w) {
  return __float2ull_rz(fminf(fmaxf(w, 0.0f), 1.0f) * 1099511627776.0f);
}

__device__ unsigned long long block_sum(unsigned long long v, unsigned long long* s_warp) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_warp[threadIdx.x >> 5] = v;
  __syncthreads();
  unsigned long long sum = 0;
  for (int i = 0; i < kThreads / 32; ++i) sum += s_warp[i];
  return sum;
}

template <int DT>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyArgs a) {
  __shared__ unsigned long long s_warp[kThreads / 32];
  __shared__ int s_count, s_token;
  const int b = blockIdx.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t* err = reinterpret_cast<uint32_t*>(a.ws);
  const int n = a.n_draft ? min(max(a.n_draft[b], 0), a.n) : a.n;
  const int64_t size = DT == MOE_DTYPE_F32 ? 4 : 2;
  const char* target = static_cast<const char*>(a.target) + (int64_t)b * (a.n + 1) * a.target_stride * size;
  const char* draft = a.draft ? static_cast<const char*>(a.draft) + (int64_t)b * a.n * a.draft_stride * size : nullptr;
  if (tid == 0) {
    int count = 0;
    for (; count < n; ++count) {
      const int id = a.draft_ids[(int64_t)b * a.n + count];
      if (id < 0 || id >= a.V) {
        atomicOr(err, (uint32_t)MOE_DEVERR_TOKEN);
        break;
      }
      const float p = prob<DT>(target, count * a.target_stride + id);
      const float q = draft ? prob<DT>(draft, count * a.draft_stride + id) : 1.0f;
      if (!(__fmul_rn(a.u_accept[(int64_t)b * a.n + count], q) < p)) break;
    }
    s_count = count;
    s_token = -1;
  }
  __syncthreads();
  const int count = s_count;
  const bool refused = count < n;
  const int64_t row = count * a.target_stride, drow = count * a.draft_stride;
  const int left_out = refused && !draft ? a.draft_ids[(int64_t)b * a.n + count] : -1;
  auto mass = [&](int v, bool whole) {
    float w = prob<DT>(target, row + v);
    if (!whole && refused) {
      if (draft) w = __fsub_rn(w, prob<DT>(draft, drow + v));
      else if (v == left_out) w = __fsub_rn(w, 1.0f);
    }
    return mass_of(w);
  };
  bool whole = false;
  unsigned long long total = 0;
  for (int pass = 0; pass < 2 && total == 0; ++pass) {
    whole = pass == 1;
    unsigned long long sum = 0;
    for (int v = tid; v < a.V; v += kThreads) sum += mass(v, whole);
    total = block_sum(sum, s_warp);
  }
  const float u = fminf(fmaxf(a.u_sample[b], 0.0f), 1.0f);
  unsigned long long m = __float2ull_rz(u * 16777216.0f);
  if (m > 16777215ull) m = 16777215ull;
  const unsigned long long goal = m * (total >> 24) + ((m * (total & 0xffffffull)) >> 24);
  unsigned long long base = 0;
  for (int v0 = 0; v0 < a.V && total > 0; v0 += kThreads) {
    const int v = v0 + tid;
    unsigned long long x = v < a.V ? mass(v, whole) : 0, sum = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    unsigned long long before = base, all = base;
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) before += s_warp[i];
      all += s_warp[i];
    }
    sum += before;
    if (sum > goal && sum - x <= goal) s_token = v;
    base = all;
    if (base > goal) break;
  }
  __syncthreads();
  if (tid == 0) {
    if (total == 0) atomicOr(err, (uint32_t)MOE_DEVERR_PROBS);
    a.n_accepted[b] = count;
  }
  for (int i = tid; i <= a.n; i += kThreads)
    a.out_ids[(int64_t)b * (a.n + 1) + i] =
        i < count ? a.draft_ids[(int64_t)b * a.n + i] : i == count ? s_token : -1;
}

}  // namespace

size_t verify_ws_bytes(int B, int V) { return kAlign; }

cudaError_t launch_verify(const VerifyArgs& a, int dtype, cudaStream_t s) {
  if (dtype == MOE_DTYPE_F32) verify_kernel<MOE_DTYPE_F32><<<a.B, kThreads, 0, s>>>(a);
  else if (dtype == MOE_DTYPE_BF16) verify_kernel<MOE_DTYPE_BF16><<<a.B, kThreads, 0, s>>>(a);
  else verify_kernel<MOE_DTYPE_F16><<<a.B, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace moe
