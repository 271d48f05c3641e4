// y = x W^T for a few tokens with NVFP4 weights (moe_linear_nvfp4).
//
// Bound by the weight bytes: 9/16 byte per weight, read once per pass of up to 8*NB tokens. The
// weights are the A operand of mma.sync m16n8k16 and the tokens its columns, so one FP4 to
// f16 conversion serves every token. A CTA owns a contiguous range of 16-row tiles; their K is
// cut into stages of 256 weights per row (a 2 KiB TMA box, 128-byte swizzle), and the CTA's line
// of stages into one equal piece per warp, each streamed through a ring of the warp's own.
// A tile that lies in several warps' pieces is summed at the end in the order of the pieces.
//
// Per stage lane 4g+c takes 32 consecutive weights (16 code bytes, two scales) at 32(4j+c),
// j = 0, 1, of rows tau(g) and 8 + tau(g), tau(g) = g/2 + 4(g%2): with that row order the eight
// lanes of a quarter warp read eight different 16-byte bank groups. k-step s of a chunk uses
// weights 4s..4s+3; x's fragments are stored with the same permutation of k.
//
// x is held as f16 times a power of two per token that puts the row's largest magnitude below
// 2^15 (exact for bf16 values within 2^-28 of it), E2M1 * UE4M3 has at most 6 significant bits
// and is exact in f16, and the accumulators are f32. The tensor core truncates its f32 sums, so
// a stage's sixteen k-steps run in accumulators of their own and are added to the row's sum with
// rounding (K = 4096: error 2.0e-6 of the result's norm in one chain of 256 k-steps).
#include "serving.cuh"
#include "tma_sync.cuh"

namespace moe {
namespace {

constexpr int kWarps = 16;
constexpr int kThreads = 32 * kWarps;
constexpr int kSlots = 3;
constexpr int kStageW = 256;                     // weights per row and stage
constexpr int kStageB = 16 * kStageW / 2;
constexpr int kRingB = kWarps * kSlots * kStageB;
constexpr int kXBytes = 131072;                  // most shared memory for x
constexpr int kXPieces = kXBytes / 16 / kThreads;

__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

// Scales of a stage for one lane: rows tau(g) and 8 + tau(g), chunks c and 4 + c, two bytes each.
struct Scales {
  uint32_t r0, r1;                               // low half: chunk c, high half: chunk 4 + c
};

template <int XT, int YT, int NB>
__global__ void __launch_bounds__(kThreads, 1)
linear_kernel(const __grid_constant__ LinearArgs a, const __grid_constant__ CUtensorMap wmap, int cols) {
  extern __shared__ char smem_raw[];
  __shared__ uint64_t s_full[kWarps * kSlots];
  __shared__ uint32_t s_amax[8 * NB];
  __shared__ volatile int s_abort;
  char* ring_all = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  char* s_x = ring_all + kRingB;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3, tau = (g >> 1) + 4 * (g & 1);
  uint32_t* err = reinterpret_cast<uint32_t*>(a.ws);
  const int t0 = blockIdx.y * cols, nt = min(cols, a.T - t0);
  const int ks = (a.K + kStageW - 1) / kStageW;
  const int tiles = (a.N + 15) / 16;
  const int tile0 = (int)((long long)tiles * blockIdx.x / gridDim.x);
  const int tile1 = (int)((long long)tiles * (blockIdx.x + 1) / gridDim.x);
  const int line = (tile1 - tile0) * ks;         // this CTA's stages
  const int per = (line + kWarps - 1) / kWarps;
  const int l0 = min(warp * per, line), l1 = min(l0 + per, line);

  if (tid < kWarps * kSlots) mbar_init(&s_full[tid], 1);
  if (tid == 0) s_abort = 0;
  if (tid < 8 * NB) s_amax[tid] = 0;
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncthreads();

  char* ring = ring_all + warp * kSlots * kStageB;
  uint64_t* full = s_full + warp * kSlots;
  const uint64_t policy = l2_evict_first_policy();
  const int64_t sc_pitch = a.K / 16;
  auto issue = [&](int l, int slot) -> Scales {  // all lanes: stage l of the line into `slot`
    const int tile = tile0 + l / ks, s = l % ks;
    if (lane == 0) {
      mbar_expect_tx(&full[slot], kStageB);
      tma_load_2d_hint(ring + slot * kStageB, &wmap, s * (kStageW / 2), tile * 16, &full[slot], policy);
    }
    Scales r = {0, 0};
    const int k0 = s * kStageW + 32 * c, k1 = k0 + 128;
    const int64_t n0 = (int64_t)tile * 16 + tau, n1 = n0 + 8;
    const uint8_t* p0 = a.scales + n0 * sc_pitch;
    const uint8_t* p1 = a.scales + n1 * sc_pitch;
    if (n0 < a.N && k0 < a.K) r.r0 = __ldg(reinterpret_cast<const uint16_t*>(p0 + k0 / 16));
    if (n0 < a.N && k1 < a.K) r.r0 |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(p0 + k1 / 16)) << 16;
    if (n1 < a.N && k0 < a.K) r.r1 = __ldg(reinterpret_cast<const uint16_t*>(p1 + k0 / 16));
    if (n1 < a.N && k1 < a.K) r.r1 |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(p1 + k1 / 16)) << 16;
    return r;
  };
  Scales sc[kSlots];
#pragma unroll
  for (int i = 0; i < kSlots; ++i) {
    sc[i] = {0, 0};
    if (l0 + i < l1) sc[i] = issue(l0 + i, i);
  }

  // ---- x: eight values per piece, all of a thread's pieces in registers at once ----
  const int kpad = ks * kStageW, per_row = kpad / 8;
  {
    uint4 v[kXPieces];
#pragma unroll
    for (int i = 0; i < kXPieces; ++i) {
      const int u = tid + i * kThreads;
      v[i] = make_uint4(0, 0, 0, 0);
      const int t = u / per_row, k = (u - t * per_row) * 8;
      if (t < nt && k < a.K)
        v[i] = *reinterpret_cast<const uint4*>(a.x + (int64_t)(t0 + t) * a.x_stride + k);
    }
    if (XT == MOE_DTYPE_BF16) {
#pragma unroll
      for (int i = 0; i < kXPieces; ++i) {
        const int u = tid + i * kThreads, t = u / per_row;
        if (t >= nt) break;
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t top = 0;                        // finite magnitudes of bf16 order as their bits
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t lo = w[q] & 0x7fffu, hi = (w[q] >> 16) & 0x7fffu;
          top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
        }
        // a row is per_row (a multiple of 32) consecutive pieces: the warp's 32 lie in one row
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) atomicMax(&s_amax[t], top);
      }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kXPieces; ++i) {
      const int u = tid + i * kThreads, t = u / per_row, kp = u - t * per_row;
      if (t >= cols) break;
      if (XT == MOE_DTYPE_BF16 && t < nt) {
        const uint32_t top = s_amax[t];
        const int e = f16_prescale_exp(__uint_as_float(top << 16));
        const float s1 = pow2f(-e / 2), s2 = pow2f(-e - (-e / 2));
        float f[8];
        unpack8<XT>(v[i], f);
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const __half2 h = __floats2half2_rn(f[2 * q] * s1 * s2, f[2 * q + 1] * s1 * s2);
          w[q] = *reinterpret_cast<const uint32_t*>(&h);
        }
        v[i] = make_uint4(w[0], w[1], w[2], w[3]);
      }
      // piece kp holds weights 8kp..8kp+7: chunk kp/4, quarter kp%4 of it
      const int chunk = kp >> 2, q = kp & 3;
      *reinterpret_cast<uint4*>(s_x + (size_t)((((chunk >> 2) * 4 + q) * cols + t) * 4 + (chunk & 3)) * 16) = v[i];
    }
    __syncthreads();
  }

  const uint32_t xb = smem_u32(s_x);
  uint32_t xcol[NB];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb) {
    const int col = nb * 8 + g;
    xcol[nb] = xb + ((col < cols ? col : 0) * 4 + c) * 16;
  }
  const int xstep = cols * 64;                   // bytes between quarters of a chunk group

  float acc[NB][4], head[NB][4];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int x = 0; x < 4; ++x) acc[nb][x] = 0.0f, head[nb][x] = 0.0f;

  const float alpha = a.alpha ? *a.alpha : 1.0f;
  auto factor = [&](int t) {                     // undoes token t's prescale
    if (XT != MOE_DTYPE_BF16) return alpha;
    return pow2f(f16_prescale_exp(__uint_as_float(s_amax[t] << 16))) * alpha;
  };
  auto store = [&](int64_t n, int t, float v) {  // v: the row's sum times alpha and the prescale
    if (n >= a.N || t >= nt) return;
    const int64_t at = (int64_t)(t0 + t) * a.y_stride + n;
    if (YT == MOE_DTYPE_F32) static_cast<float*>(a.y)[at] = v;
    else static_cast<uint16_t*>(a.y)[at] = (uint16_t)f32_to_act<YT>(v);
  };

  bool ok = true;
  int s = l0 % ks, tile = l0 / ks;
  uint32_t parity = 0;
  int l = l0;
  while (l < l1 && ok) {
#pragma unroll
    for (int slot = 0; slot < kSlots; ++slot) {
      if (l < l1 && ok) {
        ok = mbar_wait_warp(&full[slot], parity, &s_abort, err);
        if (ok) {
          const uint32_t wb = smem_u32(ring + slot * kStageB);
          float part[NB][4];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int x = 0; x < 4; ++x) part[nb][x] = 0.0f;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t at = wb + tau * 128 + (((4 * j + c) ^ tau) * 16);
            const uint4 c0 = lds128(at), c1 = lds128(at + 8 * 128);
            const uint32_t w0[4] = {c0.x, c0.y, c0.z, c0.w}, w1[4] = {c1.x, c1.y, c1.z, c1.w};
            const uint32_t s0 = e4m3x2_to_f16x2(j ? sc[slot].r0 >> 16 : sc[slot].r0 & 0xffffu);
            const uint32_t s1 = e4m3x2_to_f16x2(j ? sc[slot].r1 >> 16 : sc[slot].r1 & 0xffffu);
            const uint32_t sa[2] = {bcast_lo(s0), bcast_hi(s0)}, sb[2] = {bcast_lo(s1), bcast_hi(s1)};
            const uint32_t xo = (uint32_t)((s * 2 + j) * 4) * xstep;
#pragma unroll
            for (int q = 0; q < 4; ++q) {        // 8 weights of each row: two k-steps
              uint4 xv[NB];
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) xv[nb] = lds128(xcol[nb] + xo + q * xstep);
              uint32_t p[4], r[4];
              e2m1x8_to_f16x2x4(w0[q], p[0], p[1], p[2], p[3]);
              e2m1x8_to_f16x2x4(w1[q], r[0], r[1], r[2], r[3]);
#pragma unroll
              for (int i = 0; i < 4; ++i) p[i] = hmul2_u32(p[i], sa[q >> 1]), r[i] = hmul2_u32(r[i], sb[q >> 1]);
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) {
                mma_f16_16816(part[nb], p[0], r[0], p[1], r[1], xv[nb].x, xv[nb].y);
                mma_f16_16816(part[nb], p[2], r[2], p[3], r[3], xv[nb].z, xv[nb].w);
              }
            }
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int x = 0; x < 4; ++x) acc[nb][x] += part[nb][x];
          __syncwarp();
          if (l + kSlots < l1) sc[slot] = issue(l + kSlots, slot);
          ++l;
          if (++s == ks) {                       // the tile ends here
            if (tile * ks >= l0) {
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  const int t = nb * 8 + 2 * c + (x & 1);
                  if (t < nt)
                    store((int64_t)(tile0 + tile) * 16 + tau + 8 * (x >> 1), t, acc[nb][x] * factor(t));
                  acc[nb][x] = 0.0f;
                }
            } else {
#pragma unroll
              for (int nb = 0; nb < NB; ++nb)
#pragma unroll
                for (int x = 0; x < 4; ++x) head[nb][x] = acc[nb][x], acc[nb][x] = 0.0f;
            }
            s = 0;
            ++tile;
          }
        }
      }
    }
    parity ^= 1;
  }
  if (!ok) {
    // gave up: let this warp's copies in flight land (bounded) before the CTA leaves
    const int issued = min(l + kSlots, l1);
    for (int i = l; i < issued; ++i) {
      const int q = i - l0;
      const uint64_t begin = global_ns();
      while (!mbar_try(&full[q % kSlots], (q / kSlots) & 1) && global_ns() - begin < 100000000ull) {
      }
    }
  }
  __syncthreads();                               // every warp is done with its ring
  if (s_abort) return;

  // ---- tiles in several pieces: slot 0 a piece that began earlier, slot 1 one that opens ----
  float* parts = reinterpret_cast<float*>(ring_all);
  constexpr int kTile = 16 * 8 * NB;
  auto park = [&](int which, const float (&v)[NB][4]) {
#pragma unroll
    for (int nb = 0; nb < NB; ++nb)
#pragma unroll
      for (int x = 0; x < 4; ++x)
        parts[(warp * 2 + which) * kTile + (nb * 8 + 2 * c + (x & 1)) * 16 + tau + 8 * (x >> 1)] = v[nb][x];
  };
  if (l0 < l1) {
    const int first = l0 / ks;
    if (first * ks < l0 && (first + 1) * ks <= l1) park(0, head);   // ended here
    if (l1 % ks != 0) park((l1 / ks) * ks >= l0 ? 1 : 0, acc);      // goes on in the next piece
  }
  __syncthreads();
  for (int u = tid; u < (tile1 - tile0) * kTile; u += kThreads) {
    const int tl = u / kTile, e = u - tl * kTile;
    const int w0 = tl * ks / per, w1 = (tl * ks + ks - 1) / per;
    if (w0 == w1) continue;                      // stored by its warp
    float v = parts[(w0 * 2 + 1) * kTile + e];
    for (int w = w0 + 1; w <= w1; ++w) v += parts[w * 2 * kTile + e];
    const int t = e / 16;
    if (t < nt) store((int64_t)(tile0 + tl) * 16 + e % 16, t, v * factor(t));
  }
}

template <int XT, int YT, int NB>
cudaError_t launch_nb(const LinearArgs& a, int cols, cudaStream_t s) {
  CUtensorMap map;
  if (!make_map(&map, a.codes, (uint64_t)a.K / 2, (uint64_t)a.K / 2, (uint64_t)a.N, 128, 16, true))
    return cudaErrorInvalidValue;
  const int kpad = (a.K + kStageW - 1) / kStageW * kStageW;
  const size_t smem = 1024 + kRingB + (size_t)cols * kpad * 2;
  auto kern = linear_kernel<XT, YT, NB>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       1024 + kRingB + kXBytes);
  if (e != cudaSuccess) return e;
  const int tiles = (a.N + 15) / 16;
  const dim3 grid(tiles < num_sms() ? tiles : num_sms(), (a.T + cols - 1) / cols);
  kern<<<grid, kThreads, smem, s>>>(a, map, cols);
  return cudaGetLastError();
}

template <int XT, int YT>
cudaError_t launch_cols(const LinearArgs& a, cudaStream_t s) {
  // Tokens per pass: as many as x's share of shared memory holds, up to 32.
  const int kpad = (a.K + kStageW - 1) / kStageW * kStageW;
  int cols = kXBytes / (2 * kpad);
  if (cols > 32) cols = 32;
  if (cols > a.T) cols = a.T;
  if (cols <= 8) return launch_nb<XT, YT, 1>(a, cols, s);
  if (cols <= 16) return launch_nb<XT, YT, 2>(a, cols, s);
  return launch_nb<XT, YT, 4>(a, cols, s);
}

template <int XT>
cudaError_t launch_out(const LinearArgs& a, int y_dtype, cudaStream_t s) {
  if (y_dtype == MOE_DTYPE_F32) return launch_cols<XT, MOE_DTYPE_F32>(a, s);
  if (y_dtype == MOE_DTYPE_BF16) return launch_cols<XT, MOE_DTYPE_BF16>(a, s);
  return launch_cols<XT, MOE_DTYPE_F16>(a, s);
}

}  // namespace

size_t linear_ws_bytes(int T, int N, int K) { return kAlign; }

cudaError_t launch_linear(const LinearArgs& a, int x_dtype, int y_dtype, cudaStream_t s) {
  return x_dtype == MOE_DTYPE_BF16 ? launch_out<MOE_DTYPE_BF16>(a, y_dtype, s)
                                   : launch_out<MOE_DTYPE_F16>(a, y_dtype, s);
}

}  // namespace moe
