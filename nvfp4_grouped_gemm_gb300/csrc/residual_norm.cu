// Norm of a block's output, gate, residual and the next block's norm in one pass (moe_residual_norm).
//
// Row statistics are sums of squares in f32: a CTA takes a row, each thread holds eight neighbouring
// values of y and of the residual in registers, and the two sums meet through shuffles and shared
// memory. y, the residual and the gate are read once and the outputs written once; the weights stay
// in registers (or shared memory, below) over all rows of a CTA. A CTA takes every grid-th row, and the
// next row's values are asked for as soon as a row's are used up, before its sums meet and its stores.
//
// A CTA has as many threads as the row has vectors of eight (H = 2560: 320), up to 1024; rows beyond
// 8192 values take two or four vectors per thread (without registers for weights and the next row),
// and rows that are no whole 16-byte vectors are read value by value (2000 rows of 4095 in bf16 27.0 us,
// of 4096 16.5; with the threads of a block, not of a warp, on neighbouring values 32.2).
//
// The row's factor meets y before the weight and the gate do, as the definition has it: y * weight * gate,
// which could be made before the sum is known, may leave the range of f32 where the result is far from it
// (an f32 gate of 1e30 beside y of 1e12). That costs a multiplication behind the sum, and a gate for
// every value is held over it: instances with such gates keep the second norm's weights in shared memory,
// so that no register spills (a spilled one waits for its load, and the row ahead with it: 36.0 us instead
// of 31.6 at 4096 x 4096). 4096 x 4096 with a full gate 47.3 us where the product before the sum took
// 45.0, a gate per channel 38.3 and 34.4, 1000 x 16384 without 49.4 and 46.9; a check per row whether the
// product stays in range, with the definition's order behind it as a call, 43.9 where this takes 31.6.
//
// Bound by bytes for many rows. 4096 x 4096, y f32, residual and outputs bf16, a gate per row:
// 31.6 us, 5.3 TB/s (0.78 of the copy rate); one row of 2560 without a post weight: 2.9 us in a graph,
// which is the launch and one chain of loads and a sum. Rows beyond 8192 values spill (y, the residual
// and the sums of two or four vectors): 1000 x 16384 49.4 us, 500 x 32768 71, floor 24.2 each. Measured
// against this at 4096 x 4096: rows ahead in shared memory (cp.async) instead of in registers 36.6 us
// (one) and 36.7 us (two); rows and their gates read only when they are taken 38.9; 40 registers per
// thread and half again as many threads 44.6.
#include <type_traits>

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

// Where value x of a thread's vector v lies in the row: neighbouring values for whole vectors;
// otherwise a warp has 256 values, neighbouring threads neighbouring ones, so that all of a thread's are
// at fixed distances from its first.
template <bool VEC>
__device__ __forceinline__ int place_of(int v, int x) {
  return VEC ? (int)(v * blockDim.x + threadIdx.x) * 8 + x : (int)((v * blockDim.x + (threadIdx.x & ~31u)) * 8 + x * 32 + (threadIdx.x & 31));
}

// Asks for a thread's eight values of a row; 0 past its end.
template <bool VEC, bool F32>
__device__ __forceinline__ void ask(Raw<F32>& r, const void* row, int v, int H) {
  if (VEC) {
    const int at = place_of<VEC>(v, 0);
#pragma unroll
    for (int i = 0; i < (F32 ? 8 : 4); ++i) r.w[i] = 0;
    if (at < H) {
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(row) + (int64_t)at * (F32 ? 4 : 2));
      const uint4 a = *p;
      r.w[0] = a.x, r.w[1] = a.y, r.w[2] = a.z, r.w[3] = a.w;
      if (F32) {
        const uint4 b = p[1];
        r.w[F32 ? 4 : 0] = b.x, r.w[F32 ? 5 : 0] = b.y, r.w[F32 ? 6 : 0] = b.z, r.w[F32 ? 7 : 0] = b.w;
      }
    }
    return;
  }
  const int at = place_of<VEC>(v, 0), left = H - at;
#pragma unroll
  for (int x = 0; x < 8; x += 2) {
    uint32_t b[2] = {0, 0};
#pragma unroll
    for (int y = 0; y < 2; ++y)
      if ((x + y) * 32 < left)
        b[y] = F32 ? (static_cast<const uint32_t*>(row) + at)[(x + y) * 32] : (static_cast<const uint16_t*>(row) + at)[(x + y) * 32];
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

// Eight values of a row of weights or gates.
template <bool VEC>
__device__ __forceinline__ void operand(const void* row, int dtype, int v, int H, float (&f)[8]) {
  if (dtype == MOE_DTYPE_F32) {
    Raw<true> r;
    ask<VEC, true>(r, row, v, H);
    values_of<true>(r, dtype, f);
  } else {
    Raw<false> r;
    ask<VEC, false>(r, row, v, H);
    values_of<false>(r, dtype, f);
  }
}

template <bool VEC>
__device__ __forceinline__ void put(void* row, int dtype, int v, int H, const float (&f)[8]) {
  if (VEC) {
    const int at = place_of<VEC>(v, 0);
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
  const int at = place_of<VEC>(v, 0), left = H - at;
  if (dtype == MOE_DTYPE_F32) {
    float* p = static_cast<float*>(row) + at;
#pragma unroll
    for (int x = 0; x < 8; ++x)
      if (x * 32 < left) p[x * 32] = f[x];
    return;
  }
  const uint4 w = dtype == MOE_DTYPE_BF16 ? pack8<MOE_DTYPE_BF16>(f) : pack8<MOE_DTYPE_F16>(f);
  const uint32_t pairs[4] = {w.x, w.y, w.z, w.w};
  uint16_t* p = static_cast<uint16_t*>(row) + at;
#pragma unroll
  for (int x = 0; x < 8; ++x)
    if (x * 32 < left) p[x * 32] = (uint16_t)(pairs[x / 2] >> (x % 2 * 16));
}

// Pairs of f32 in one 64-bit register, and eight values as four of them.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
struct Eight {
  uint64_t p[4];
};
__device__ __forceinline__ Eight pack(const float (&f)[8]) {
  return {{pair(f[0], f[1]), pair(f[2], f[3]), pair(f[4], f[5]), pair(f[6], f[7])}};
}
__device__ __forceinline__ void unpack(const Eight& e, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) unpair(e.p[i], f[2 * i], f[2 * i + 1]);
}

// Sum over the block of the pairs' sums, the same in every thread. `s` is one of two rows, used in turn,
// so that one barrier per sum is enough; it is 0 past the block's warps.
__device__ __forceinline__ float block_sum(uint64_t pairs, float* s) {
  float v, u;
  unpair(pairs, v, u);
  v += u;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if (blockDim.x == 32) return v;
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  float all = 0.0f;
  for (int w = 0; w < (int)blockDim.x / 32; w += 4) {
    const float4 f = *reinterpret_cast<const float4*>(s + w);
    all += (f.x + f.y) + (f.z + f.w);
  }
  return all;
}

__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

// GATES: there may be a gate for every value; then a row's gates are held over its sum, and the second
// norm's weights in shared memory (a thread's own) instead of registers.
template <int MOST, int V, bool VEC, bool Y32, bool R32, bool GATES>
__global__ void __launch_bounds__(MOST, 1024 / MOST) norm_kernel(const __grid_constant__ NormArgs a) {
  __shared__ __align__(16) float s_sum[2][32];
  constexpr int kY = Y32 ? 4 : 2, kR = R32 ? 4 : 2;
  constexpr bool kHold = V == 1, kAside = kHold && GATES;
  __shared__ ulonglong2 s_pre[2][kAside ? MOST : 1];
  const float each = 1.0f / (float)a.H;
  const char* y = static_cast<const char*>(a.y) + (int64_t)blockIdx.x * a.y_stride * kY;
  const char* res = static_cast<const char*>(a.residual) + (int64_t)blockIdx.x * a.residual_stride * kR;
  const int64_t y_step = gridDim.x * a.y_stride * kY, res_step = gridDim.x * a.residual_stride * kR;
  const int gate_size = a.gate_dtype == MOE_DTYPE_F32 ? 4 : 2;
  const char* gate = static_cast<const char*>(a.gate) + (int64_t)blockIdx.x * a.gate_stride * gate_size;
  const int64_t gate_step = gridDim.x * a.gate_stride * gate_size;
  Raw<Y32> yw[V];
  Raw<R32> rw[V];
  uint32_t gate_bits = 0;                      // a gate that is one value per row
  auto ask_rows = [&] {
    if (a.y) {
#pragma unroll
      for (int v = 0; v < V; ++v) ask<VEC, Y32>(yw[v], y, v, a.H);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) ask<VEC, R32>(rw[v], res, v, a.H);
    if (a.gate && !a.gate_inner)
      gate_bits = gate_size == 4 ? *reinterpret_cast<const uint32_t*>(gate) : *reinterpret_cast<const uint16_t*>(gate);
    y += y_step, res += res_step;
  };
  if (kHold) ask_rows();
  if (threadIdx.x < 32) s_sum[0][threadIdx.x] = s_sum[1][threadIdx.x] = 0.0f;
  Eight held[2];
  auto weights = [&](const void* w, int v) {
    float f[8];
    operand<VEC>(w, a.weight_dtype, v, a.H, f);
#pragma unroll
    for (int x = 0; x < 8; ++x) f[x] += a.offset;
    return pack(f);
  };
  if (kHold && a.post) held[0] = weights(a.post, 0);
  if (kHold && a.pre) {
    const Eight w = weights(a.pre, 0);
    if constexpr (kAside) {
      s_pre[0][threadIdx.x] = make_ulonglong2(w.p[0], w.p[1]);
      s_pre[1][threadIdx.x] = make_ulonglong2(w.p[2], w.p[3]);
    } else {
      held[1] = w;
    }
  }
  if (blockDim.x > 32) __syncthreads();

  for (int t = blockIdx.x; t < a.T; t += gridDim.x) {
    if (!kHold) ask_rows();
    Eight r[V];
    float k = a.scale;
    if (a.gate && !a.gate_inner) {
      const float g = gate_size == 4 ? __uint_as_float(gate_bits) : scalar_of(gate_bits, a.gate_dtype);
      k *= a.sigmoid ? sigmoid(g) : g;
    }
    const bool gates = GATES && a.gate && a.gate_inner;
    auto gate_of = [&](int v) {                // scale times the gate's values
      float f[8];
      operand<VEC>(gate, a.gate_dtype, v, a.H, f);
#pragma unroll
      for (int x = 0; x < 8; ++x) f[x] = a.scale * (a.sigmoid ? sigmoid(f[x]) : f[x]);
      return pack(f);
    };
    Eight z[V], g_held = {};
    uint64_t sum = 0;
    if (a.y) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float f[8];
        values_of<Y32>(yw[v], a.y_dtype, f);
        z[v] = pack(f);
#pragma unroll
        for (int i = 0; i < 4; ++i) sum = fma2(z[v].p[i], z[v].p[i], sum);
      }
      if (kHold && gates) g_held = gate_of(0);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      float f[8];
      values_of<R32>(rw[v], a.residual_dtype, f);
      r[v] = pack(f);
    }
    const char* gate_next = gate + gate_step;
    if (kHold) gate = gate_next;
    if (kHold && a.T - t > (int)gridDim.x) ask_rows();  // the next row, into registers that this one is done with
    if (a.y) {
      if (a.post) {
        // y is normed before its weight and then the gate meet it: y * weight * gate, whose product needs
        // no sum, may leave the range of f32 where none of these does
        const float n = rsqrtf(fmaf(block_sum(sum, s_sum[0]), each, a.eps));
        const uint64_t nn = pair(n, n);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const Eight w = kHold ? held[0] : weights(a.post, v);
#pragma unroll
          for (int i = 0; i < 4; ++i) z[v].p[i] = mul2(mul2(z[v].p[i], nn), w.p[i]);
        }
      }
      const uint64_t kk = pair(k, k);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        Eight g;
        if (gates) g = kHold ? g_held : gate_of(v);
#pragma unroll
        for (int i = 0; i < 4; ++i) r[v].p[i] = fma2(z[v].p[i], gates ? g.p[i] : kk, r[v].p[i]);
      }
    }
    if (!kHold) gate = gate_next;
    if (a.normed) {
      sum = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        // values past the row count as 0 (a factor may have made NaN of them)
        if (!VEC) {
          float f[8];
          unpack(r[v], f);
#pragma unroll
          for (int x = 0; x < 8; ++x) f[x] = place_of<VEC>(v, x) < a.H ? f[x] : 0.0f;
          r[v] = pack(f);
        }
        if (!VEC || place_of<VEC>(v, 0) < a.H) {
#pragma unroll
          for (int i = 0; i < 4; ++i) sum = fma2(r[v].p[i], r[v].p[i], sum);
        }
      }
      const float n = rsqrtf(fmaf(block_sum(sum, s_sum[1]), each, a.eps));
      char* to = static_cast<char*>(a.normed) + (int64_t)t * a.normed_stride * (a.normed_dtype == MOE_DTYPE_F32 ? 4 : 2);
      const uint64_t nn = pair(n, n);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        Eight e;
#pragma unroll
        for (int i = 0; i < 4; ++i) e.p[i] = mul2(r[v].p[i], nn);
        if (a.pre) {
          Eight w;
          if constexpr (kAside) {
            const ulonglong2 x = s_pre[0][threadIdx.x], y = s_pre[1][threadIdx.x];
            w = {{x.x, x.y, y.x, y.y}};
          } else {
            w = kHold ? held[1] : weights(a.pre, v);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) e.p[i] = mul2(e.p[i], w.p[i]);
        }
        float f[8];
        unpack(e, f);
        put<VEC>(to, a.normed_dtype, v, a.H, f);
      }
    }
    if (a.out) {
      char* to = static_cast<char*>(a.out) + (int64_t)t * a.out_stride * kR;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float f[8];
        unpack(r[v], f);
        put<VEC>(to, a.residual_dtype, v, a.H, f);
      }
    }
    // a sum's slots are written again only behind the other sum's barrier; where a row has one sum
    // or none of the two this barrier stands in for it
    if (blockDim.x > 32 && !(a.y && a.post && a.normed)) __syncthreads();
  }
}

template <int MOST, int V, bool VEC>
cudaError_t launch_size(const NormArgs& a, cudaStream_t s) {
  const bool y32 = a.y_dtype == MOE_DTYPE_F32, r32 = a.residual_dtype == MOE_DTYPE_F32;
  const int threads = V > 1 ? MOST : (a.H + 255) / 256 * 32;
  const long long most = (long long)num_sms() * (1024 / threads);
  const unsigned grid = (unsigned)(a.T < most ? a.T : most);
  auto launch = [&](auto gates) {
    constexpr bool G = decltype(gates)::value;
    if (y32 && r32) norm_kernel<MOST, V, VEC, true, true, G><<<grid, threads, 0, s>>>(a);
    else if (y32) norm_kernel<MOST, V, VEC, true, false, G><<<grid, threads, 0, s>>>(a);
    else if (r32) norm_kernel<MOST, V, VEC, false, true, G><<<grid, threads, 0, s>>>(a);
    else norm_kernel<MOST, V, VEC, false, false, G><<<grid, threads, 0, s>>>(a);
  };
  if (V > 1 || a.gate_inner) launch(std::true_type{});
  else launch(std::integral_constant<bool, (V > 1)>{});
  return cudaGetLastError();
}

template <bool VEC>
cudaError_t launch_rows(const NormArgs& a, cudaStream_t s) {
  if (a.H <= 4096) return launch_size<512, 1, VEC>(a, s);
  if (a.H <= 8192) return launch_size<1024, 1, VEC>(a, s);
  return a.H <= 16384 ? launch_size<1024, 2, VEC>(a, s) : launch_size<1024, 4, VEC>(a, s);
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
  return vec ? launch_rows<true>(a, s) : launch_rows<false>(a, s);
}

}  // namespace moe
