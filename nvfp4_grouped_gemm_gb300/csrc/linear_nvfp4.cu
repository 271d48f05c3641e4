// y = x W^T for a few tokens with NVFP4 weights (moe_linear_nvfp4).
//
// One warp per weight row and eight tokens: a lane takes 32 weights (16 code bytes, two scales)
// at a time, and the lanes' sums meet at the end.
#include "serving.cuh"

namespace moe {
namespace {

template <int XT, int YT>
__global__ void __launch_bounds__(256) linear_kernel(const LinearArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t n = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (n >= a.N) return;
  const int t0 = blockIdx.y * 8;
  float acc[8];
#pragma unroll
  for (int t = 0; t < 8; ++t) acc[t] = 0.0f;
  for (int k = lane * 32; k < a.K; k += 1024) {
    const uint4 codes = ldg_stream(a.codes + n * (a.K / 2) + k / 2);
    const uint32_t sc = *reinterpret_cast<const uint16_t*>(a.scales + n * (a.K / 16) + k / 16);
    const float2 s = e4m3x2_to_f32x2(sc);
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float v[8];
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const uint32_t h = e2m1x2_to_f16x2((w[i] >> (8 * b)) & 0xffu);
        const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&h));
        v[2 * b] = p.x * (i < 2 ? s.x : s.y);
        v[2 * b + 1] = p.y * (i < 2 ? s.x : s.y);
      }
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        if (t0 + t >= a.T) break;
        float xv[8];
        unpack8<XT>(*reinterpret_cast<const uint4*>(a.x + (int64_t)(t0 + t) * a.x_stride + k + 8 * i), xv);
#pragma unroll
        for (int q = 0; q < 8; ++q) acc[t] = fmaf(v[q], xv[q], acc[t]);
      }
    }
  }
  const float alpha = a.alpha ? *a.alpha : 1.0f;
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    float v = acc[t];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (lane == 0 && t0 + t < a.T) {
      const int64_t at = (int64_t)(t0 + t) * a.y_stride + n;
      if (YT == MOE_DTYPE_F32) static_cast<float*>(a.y)[at] = v * alpha;
      else static_cast<uint16_t*>(a.y)[at] = (uint16_t)f32_to_act<YT>(v * alpha);
    }
  }
}

template <int XT>
void launch_out(const LinearArgs& a, int y_dtype, cudaStream_t s) {
  const dim3 grid((a.N + 7) / 8, (a.T + 7) / 8);
  if (y_dtype == MOE_DTYPE_F32) linear_kernel<XT, MOE_DTYPE_F32><<<grid, 256, 0, s>>>(a);
  else if (y_dtype == MOE_DTYPE_BF16) linear_kernel<XT, MOE_DTYPE_BF16><<<grid, 256, 0, s>>>(a);
  else linear_kernel<XT, MOE_DTYPE_F16><<<grid, 256, 0, s>>>(a);
}

}  // namespace

size_t linear_ws_bytes(int T, int N, int K) { return kAlign; }

cudaError_t launch_linear(const LinearArgs& a, int x_dtype, int y_dtype, cudaStream_t s) {
  if (x_dtype == MOE_DTYPE_BF16) launch_out<MOE_DTYPE_BF16>(a, y_dtype, s);
  else launch_out<MOE_DTYPE_F16>(a, y_dtype, s);
  return cudaGetLastError();
}

}  // namespace moe
