// Norm of a block's output, gate, residual and the next block's norm in one pass (moe_residual_norm).
//
// Row statistics are sums of squares in f32: a CTA takes a row, each thread holds its values of y and
// of the residual in registers (both are asked for before the first sum), and the two sums meet
// through shuffles and shared memory. y, the residual and the gate are read once and the outputs
// written once; weights come from L1 after a CTA's first row. CTAs take rows in turn.
//
// Threads and vectors per thread follow H alone: the fewest threads (up to 256) whose one vector of
// eight values covers a row, beyond that two vectors, then more threads.
#include "serving.cuh"

namespace moe {
namespace {

// Eight values as they lie in memory: 16-bit types fill the first four words.
template <bool F32>
struct Raw {
  uint32_t w[F32 ? 8 : 4];
};

__device__ __forceinline__ float scalar_of(uint32_t bits, int dtype) {
  return dtype == MOE_DTYPE_BF16 ? act_to_f32<MOE_DTYPE_BF16>(bits) : act_to_f32<MOE_DTYPE_F16>(bits);
}

// Where value x of a thread's vector v lies in the row: neighbouring values for whole vectors,
// neighbouring threads otherwise.
template <int THREADS, bool VEC>
__device__ __forceinline__ int place_of(int v, int x) {
  return VEC ? (v * THREADS + threadIdx.x) * 8 + x : (v * 8 + x) * THREADS + (int)threadIdx.x;
}

template <int THREADS, bool VEC, bool F32>
__device__ __forceinline__ void ask(Raw<F32>& r, const void* row, int v, int H) {
  if (VEC) {
    const int at = place_of<THREADS, VEC>(v, 0);
    if (at < H) {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(row) + (int64_t)at * (F32 ? 4 : 2));
      const uint4 a = *p;
      r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
      if (F32) {
        const uint4 b = p[1];
        r.w[F32 ? 4 : 0] = b.x, r.w[F32 ? 5 : 0] = b.y, r.w[F32 ? 6 : 0] = b.z, r.w[F32 ? 7 : 0] = b.w;
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < (F32 ? 8 : 4); ++i) r.w[i] = 0;
    return;
  }
#pragma unroll
  for (int x = 0; x < 8; x += 2) {
    uint32_t b[2] = {0, 0};
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int at = place_of<THREADS, VEC>(v, x + y);
      if (at < H) b[y] = F32 ? static_cast<const uint32_t*>(row)[at] : static_cast<const uint16_t*>(row)[at];
    }
    if (F32) {
      r.w[F32 ? x : 0] = b[0], r.w[F32 ? x + 1 : 0] = b[1];
    } else {
      r.w[x / 2] = b[0] | b[1] << 16;
    }
  }
}

template <bool F32>
__device__ __forceinline__ void values_of(const Raw<F32>& r, int dtype, float (&f)[8]) {
  if (F32) {
#pragma unroll
    for (int x = 0; x < 8; ++x) f[x] = __uint_as_float(r.w[F32 ? x : 0]);
  } else if (dtype == MOE_DTYPE_BF16) {
    unpack8<MOE_DTYPE_BF16>(make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]), f);
  } else {
    unpack8<MOE_DTYPE_F16>(make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]), f);
  }
}

// Eight values of an operand that is the same for every row or small (weights, gates).
template <int THREADS, bool VEC>
__device__ __forceinline__ void operand(const void* row, int dtype, int v, int H, float (&f)[8]) {
  if (dtype == MOE_DTYPE_F32) {
    Raw<true> r;
    ask<THREADS, VEC, true>(r, row, v, H);
    values_of<true>(r, dtype, f);
  } else {
    Raw<false> r;
    ask<THREADS, VEC, false>(r, row, v, H);
    values_of<false>(r, dtype, f);
  }
}

template <int THREADS, bool VEC>
__device__ __forceinline__ void put(void* row, int dtype, int v, int H, const float (&f)[8]) {
  if (VEC) {
    const int at = place_of<THREADS, VEC>(v, 0);
    if (at >= H) return;
    if (dtype == MOE_DTYPE_F32) {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(row) + at);
      p[0] = make_float4(f[0], f[1], f[2], f[3]);
      p[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(row) + at) =
          dtype == MOE_DTYPE_BF16 ? pack8<MOE_DTYPE_BF16>(f) : pack8<MOE_DTYPE_F16>(f);
    }
    return;
  }
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    const int at = place_of<THREADS, VEC>(v, x);
    if (at >= H) continue;
    if (dtype == MOE_DTYPE_F32) {
      static_cast<float*>(row)[at] = f[x];
    } else {
      static_cast<uint16_t*>(row)[at] =
          (uint16_t)(dtype == MOE_DTYPE_BF16 ? f32_to_act<MOE_DTYPE_BF16>(f[x]) : f32_to_act<MOE_DTYPE_F16>(f[x]));
    }
  }
}

// Sum over the block, the same in every thread. `slot` is one of two, used in turn, so that one
// barrier per sum is enough.
template <int THREADS>
__device__ __forceinline__ float block_sum(float v, float (*s)[THREADS / 32], int slot) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (THREADS == 32) return v;
  if ((threadIdx.x & 31) == 0) s[slot][threadIdx.x >> 5] = v;
  __syncthreads();
  float all = 0.0f;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) all += s[slot][w];
  return all;
}

template <int THREADS, int V, bool VEC, bool Y32, bool R32>
__global__ void __launch_bounds__(THREADS) norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float s_sum[2][THREADS / 32];
  const float each = 1.0f / (float)a.H;
  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    const char* yr = static_cast<const char*>(a.y) + (int64_t)t * a.y_stride * (Y32 ? 4 : 2);
    const char* rr = static_cast<const char*>(a.residual) + (int64_t)t * a.residual_stride * (R32 ? 4 : 2);
    Raw<Y32> yw[V];
    Raw<R32> rw[V];
    if (a.y) {
#pragma unroll
      for (int v = 0; v < V; ++v) ask<THREADS, VEC, Y32>(yw[v], yr, v, a.H);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) ask<THREADS, VEC, R32>(rw[v], rr, v, a.H);
    float r[V][8];
    if (a.y) {
      float k = a.scale;
      if (a.post) {
        float sum = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float f[8];
          values_of<Y32>(yw[v], a.y_dtype, f);
#pragma unroll
          for (int x = 0; x < 8; ++x) sum = fmaf(f[x], f[x], sum);
        }
        sum = block_sum<THREADS>(sum, s_sum, 0);
        k = a.scale * rsqrtf(fmaf(sum, each, a.eps));
      }
      const int64_t g0 = (int64_t)t * a.gate_stride;
      const char* gr = static_cast<const char*>(a.gate) + g0 * (a.gate_dtype == MOE_DTYPE_F32 ? 4 : 2);
      if (a.gate && !a.gate_inner) {
        const float g = a.gate_dtype == MOE_DTYPE_F32 ? *reinterpret_cast<const float*>(gr)
                                                      : scalar_of(*reinterpret_cast<const uint16_t*>(gr), a.gate_dtype);
        k *= a.sigmoid ? 1.0f / (1.0f + expf(-g)) : g;
      }
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float z[8];
        values_of<Y32>(yw[v], a.y_dtype, z);
        values_of<R32>(rw[v], a.residual_dtype, r[v]);
        if (a.post) {
          float w[8];
          operand<THREADS, VEC>(a.post, a.weight_dtype, v, a.H, w);
#pragma unroll
          for (int x = 0; x < 8; ++x) z[x] *= w[x] + a.offset;
        }
        if (a.gate && a.gate_inner) {
          float g[8];
          operand<THREADS, VEC>(gr, a.gate_dtype, v, a.H, g);
#pragma unroll
          for (int x = 0; x < 8; ++x) z[x] *= a.sigmoid ? 1.0f / (1.0f + expf(-g[x])) : g[x];
        }
#pragma unroll
        for (int x = 0; x < 8; ++x) r[v][x] = fmaf(z[x], k, r[v][x]);
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) values_of<R32>(rw[v], a.residual_dtype, r[v]);
    }
    if (a.out) {
      char* to = static_cast<char*>(a.out) + (int64_t)t * a.out_stride * (R32 ? 4 : 2);
#pragma unroll
      for (int v = 0; v < V; ++v) put<THREADS, VEC>(to, a.residual_dtype, v, a.H, r[v]);
    }
    if (a.normed) {
      float sum = 0.0f;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int x = 0; x < 8; ++x)
          if (place_of<THREADS, VEC>(v, x) < a.H) sum = fmaf(r[v][x], r[v][x], sum);
      sum = block_sum<THREADS>(sum, s_sum, 1);
      const float k = rsqrtf(fmaf(sum, each, a.eps));
      char* to = static_cast<char*>(a.normed) + (int64_t)t * a.normed_stride * (a.normed_dtype == MOE_DTYPE_F32 ? 4 : 2);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (a.pre) {
          float w[8];
          operand<THREADS, VEC>(a.pre, a.weight_dtype, v, a.H, w);
#pragma unroll
          for (int x = 0; x < 8; ++x) r[v][x] *= k * (w[x] + a.offset);
        } else {
#pragma unroll
          for (int x = 0; x < 8; ++x) r[v][x] *= k;
        }
        put<THREADS, VEC>(to, a.normed_dtype, v, a.H, r[v]);
      }
    }
    // a sum's slot is written again only behind the other sum's barrier; where a row has one sum
    // or none of the two this barrier stands in for it
    if (THREADS > 32 && !(a.y && a.post && a.normed)) __syncthreads();
  }
}

template <int THREADS, int V, bool VEC>
cudaError_t launch_types(const NormArgs& a, cudaStream_t s) {
  const bool y32 = a.y_dtype == MOE_DTYPE_F32, r32 = a.residual_dtype == MOE_DTYPE_F32;
  const int per_sm = 2048 / THREADS < 32 ? 2048 / THREADS : 32;
  const long long most = (long long)num_sms() * per_sm;
  const dim3 grid((unsigned)(a.T < most ? a.T : most));
  if (y32 && r32) norm_kernel<THREADS, V, VEC, true, true><<<grid, THREADS, 0, s>>>(a);
  else if (y32) norm_kernel<THREADS, V, VEC, true, false><<<grid, THREADS, 0, s>>>(a);
  else if (r32) norm_kernel<THREADS, V, VEC, false, true><<<grid, THREADS, 0, s>>>(a);
  else norm_kernel<THREADS, V, VEC, false, false><<<grid, THREADS, 0, s>>>(a);
  return cudaGetLastError();
}

template <bool VEC>
cudaError_t launch_size(const NormArgs& a, cudaStream_t s) {
  if (a.H <= 256) return launch_types<32, 1, VEC>(a, s);
  if (a.H <= 1024) return launch_types<128, 1, VEC>(a, s);
  if (a.H <= 2048) return launch_types<256, 1, VEC>(a, s);
  if (a.H <= 4096) return launch_types<256, 2, VEC>(a, s);
  if (a.H <= 8192) return launch_types<512, 2, VEC>(a, s);
  if (a.H <= 16384) return launch_types<1024, 2, VEC>(a, s);
  return launch_types<1024, 4, VEC>(a, s);
}

bool whole(const void* p, int64_t stride, int bytes) {   // rows that vectors of eight values may be read from
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * bytes % 16 == 0);
}

}  // namespace

cudaError_t launch_norm(const NormArgs& a, cudaStream_t s) {
  auto size = [](int dt) { return dt == MOE_DTYPE_F32 ? 4 : 2; };
  const bool vec = a.H % 8 == 0 && whole(a.y, a.y_stride, size(a.y_dtype)) &&
                   whole(a.residual, a.residual_stride, size(a.residual_dtype)) &&
                   whole(a.out, a.out_stride, size(a.residual_dtype)) &&
                   whole(a.normed, a.normed_stride, size(a.normed_dtype)) && whole(a.post, 0, 2) &&
                   whole(a.pre, 0, 2) && (!a.gate_inner || whole(a.gate, a.gate_stride, size(a.gate_dtype)));
  return vec ? launch_size<true>(a, s) : launch_size<false>(a, s);
}

}  // namespace moe
