// y = x W^T for a few tokens with NVFP4 weights (moe_linear_nvfp4).
//
// Bound by the weight bytes: 9/16 byte per weight, read once per pass of up to 8*NB tokens. The
// weights are the A operand of mma.sync m16n8k16 and the tokens its columns, so one FP4 to
// f16 conversion serves every token. A CTA owns a contiguous range of 16-row tiles; their K is
// cut into stages of 256 weights per row (a 2 KiB TMA box, 128-byte swizzle), and the CTA's line
// of stages into one equal piece per warp, each streamed through a ring of the warp's own.
// A tile that lies in several warps' pieces is summed at the end in the order of the pieces.
//
// Per stage lane 4g+c takes 64 consecutive weights (two 16-byte pieces, four scales) at 64c of
// rows g and 8 + g: the eight lanes of a quarter warp then read eight different 16-byte bank
// groups. k-step s of a piece uses its weights 4s..4s+3; x's fragments are stored with the same
// permutation of k, for a number of tokens (a power of two) known at compile time, so that their
// reads need no address arithmetic.
//
// x is held as f16 times a power of two per token that puts the row's largest magnitude below
// 2^15 (exact for bf16 values within 2^-28 of it), E2M1 * UE4M3 has at most 6 significant bits
// and is exact in f16, and the accumulators are f32. The tensor core truncates its f32 sums, so
// a stage's sixteen k-steps run in accumulators of their own and are added to the row's sum with
// rounding (K = 4096: error 2.0e-6 of the result's norm in one chain of 256 k-steps).
//
// Measured: 131101 x 4096 for 16 tokens 72.5 us, 4.3 TB/s: a stage's conversions and products, which
// depend on one another, and not the copies take the warps' time (issue 53%). 2560 x 5120 for one token 6.7 us, where the first
// copies' latency, the meeting of the warps and the launch are most of it.
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
// x is prepared by a kernel of its own from this size of a pass on (where converting it in every
// CTA costs more than the launch), up to this many tokens (the workspace holds them).
constexpr int kPrepBytes = 32768;
constexpr int kPrepTokens = 512;
// Workspace: error word, the tokens' factors, their fragments.
constexpr size_t kFactorsAt = kAlign;
constexpr size_t kFragsAt = kFactorsAt + kPrepTokens * 4;

// Scales of a stage for one lane: rows g and 8 + g, four bytes each.
struct Scales {
  uint32_t r0, r1;
};

__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Byte of x's fragments that holds weights 8kp..8kp+7 of column t of a pass: quarter kp%4 of chunk
// kp/4, chunk 2c + j of its stage.
__device__ __forceinline__ size_t x_byte(int kp, int t, int cols) {
  const int chunk = kp >> 2, j = chunk & 1, cc = (chunk >> 1) & 3, st = chunk >> 3;
  return (size_t)((((st * 2 + j) * 4 + (kp & 3)) * cols + t) * 4 + cc) * 16;
}
// The largest finite magnitude of eight bf16 values, as its bits.
__device__ __forceinline__ uint32_t top_bf16(const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t top = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t lo = w[q] & 0x7fffu, hi = (w[q] >> 16) & 0x7fffu;
    top = max(top, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
  }
  return top;
}
// 2^-e for the row's prescale e as two factors, each a normal float.
__device__ __forceinline__ float2 down_factors(uint32_t top) {
  const int e = f16_prescale_exp(__uint_as_float(top << 16));
  return make_float2(pow2f(-e / 2), pow2f(-e - (-e / 2)));
}
__device__ __forceinline__ uint4 scale_bf16(const uint4& v, const float2& f2) {
  float f[8];
  unpack8<MOE_DTYPE_BF16>(v, f);
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const __half2 h = __floats2half2_rn(f[2 * q] * f2.x * f2.y, f[2 * q + 1] * f2.x * f2.y);
    w[q] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Large x: one block per token writes its fragments and factor to the workspace, from where every
// CTA of the product copies them (converting 16 x 4096 values in each of 152 CTAs took 11 us).
constexpr int kPrepThreads = 256;
__global__ void __launch_bounds__(kPrepThreads) x_prep_kernel(const LinearArgs a, int cols, int kpad) {
  __shared__ uint32_t s_top;
  const int t = blockIdx.x, tid = threadIdx.x;
  pdl_trigger();                                 // the product may start on its weights
  if (tid == 0) s_top = 0;
  __syncthreads();
  const bool bf16 = a.x_dtype == MOE_DTYPE_BF16;
  const uint16_t* row = a.x + (int64_t)t * a.x_stride;
  uint32_t top = 0;
  if (bf16) {
    for (int kp = tid; kp * 8 < a.K; kp += kPrepThreads)
      top = max(top, top_bf16(*reinterpret_cast<const uint4*>(row + kp * 8)));
    top = __reduce_max_sync(0xffffffffu, top);
    if ((tid & 31) == 0) atomicMax(&s_top, top);
  }
  __syncthreads();
  top = s_top;
  const float2 f2 = down_factors(top);
  char* dst = a.ws + kFragsAt + (size_t)(t / cols) * cols * kpad * 2;
  for (int kp = tid; kp < kpad / 8; kp += kPrepThreads) {
    uint4 v = make_uint4(0, 0, 0, 0);
    if (kp * 8 < a.K) {
      v = *reinterpret_cast<const uint4*>(row + kp * 8);
      if (bf16) v = scale_bf16(v, f2);
    }
    *reinterpret_cast<uint4*>(dst + x_byte(kp, t % cols, cols)) = v;
  }
  if (tid == 0)
    reinterpret_cast<float*>(a.ws + kFactorsAt)[t] = bf16 ? pow2f(f16_prescale_exp(__uint_as_float(top << 16))) : 1.0f;
}

// PREP: x comes from x_prep_kernel.
template <int COLS, bool PREP>
__global__ void __launch_bounds__(kThreads, 1)
linear_kernel(const __grid_constant__ LinearArgs a, const __grid_constant__ CUtensorMap wmap) {
  constexpr int NB = COLS < 8 ? 1 : COLS / 8;
  extern __shared__ char smem_raw[];
  __shared__ uint64_t s_full[kWarps * kSlots], s_xfull;
  __shared__ uint32_t s_amax[COLS];
  __shared__ float2 s_scale[COLS];
  __shared__ float s_factor[COLS];
  __shared__ volatile int s_abort;
  char* ring_all = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  char* s_x = ring_all + kRingB;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const bool bf16 = a.x_dtype == MOE_DTYPE_BF16;
  uint32_t* err = reinterpret_cast<uint32_t*>(a.ws);
  const int t0 = blockIdx.y * COLS, nt = min(COLS, a.T - t0);
  const int ks = (a.K + kStageW - 1) / kStageW;
  const int tiles = (a.N + 15) / 16;
  const int tile0 = (int)((long long)tiles * blockIdx.x / gridDim.x);
  const int tile1 = (int)((long long)tiles * (blockIdx.x + 1) / gridDim.x);
  const int line = (tile1 - tile0) * ks;         // this CTA's stages
  const int per = (line + kWarps - 1) / kWarps;
  const int l0 = min(warp * per, line), l1 = min(l0 + per, line);

  if (tid < kWarps * kSlots) mbar_init(&s_full[tid], 1);
  if (tid == 0) {
    s_abort = 0;
    mbar_init(&s_xfull, 1);
  }
  if (tid < COLS) s_amax[tid] = 0;
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncthreads();

  char* ring = ring_all + warp * kSlots * kStageB;
  uint64_t* full = s_full + warp * kSlots;
  const uint64_t policy = l2_evict_first_policy();
  const int64_t pitch = a.K / 16;                // scale bytes per row
  const bool words = a.K % 64 == 0;              // rows of scales start at multiples of four bytes
  // the stage to issue next: its tile, its place in K, and the lane's scales of row g there
  int i_tile = tile0 + l0 / ks, i_s = l0 % ks;
  const uint8_t* i_sc = a.scales + ((int64_t)i_tile * 16 + g) * pitch + i_s * 16 + 4 * c;
  auto issue = [&](int slot) -> Scales {         // all lanes
    if (lane == 0) {
      mbar_expect_tx(&full[slot], kStageB);
      tma_load_2d_hint(ring + slot * kStageB, &wmap, i_s * (kStageW / 2), i_tile * 16, &full[slot], policy);
    }
    Scales r = {0, 0};
    const int k0 = i_s * kStageW + 64 * c, n0 = i_tile * 16 + g;
    if (words) {
      if (k0 < a.K) {
        if (n0 < a.N) r.r0 = __ldg(reinterpret_cast<const uint32_t*>(i_sc));
        if (n0 + 8 < a.N) r.r1 = __ldg(reinterpret_cast<const uint32_t*>(i_sc + 8 * pitch));
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (k0 + 32 * h < a.K) {
          if (n0 < a.N) r.r0 |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(i_sc + 2 * h)) << (16 * h);
          if (n0 + 8 < a.N)
            r.r1 |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(i_sc + 8 * pitch + 2 * h)) << (16 * h);
        }
    }
    i_sc += 16;
    if (++i_s == ks) {
      i_s = 0, ++i_tile;
      i_sc += 16 * pitch - ks * 16;
    }
    return r;
  };
  Scales sc[kSlots];

  const int kpad = ks * kStageW, per_row = kpad / 8;
  if (PREP) {
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      sc[i] = {0, 0};
      if (l0 + i < l1) sc[i] = issue(i);
    }
    pdl_wait();                                  // x's fragments are written
    if (tid < nt) s_factor[tid] = reinterpret_cast<const float*>(a.ws + kFactorsAt)[t0 + tid];
    const char* src = a.ws + kFragsAt + (size_t)blockIdx.y * COLS * kpad * 2;
    if (tid == 0) {
      const uint32_t bytes = (uint32_t)COLS * kpad * 2;
      mbar_expect_tx(&s_xfull, bytes);
      for (uint32_t at = 0; at < bytes; at += 16384)
        bulk_load(s_x + at, src + at, min(16384u, bytes - at), &s_xfull);
    }
    // the copy is in flight whatever happens: no thread leaves before it has landed or given up
    const bool there = mbar_wait_warp(&s_xfull, 0, &s_abort, err);
    if (!there) {
      const uint64_t begin = global_ns();
      while (!mbar_try(&s_xfull, 0) && global_ns() - begin < 100000000ull) {
      }
    }
    __syncthreads();
  } else {
    // ---- x: eight values per piece, all of a thread's pieces in registers at once ----
    // piece tid + i * kThreads is piece kp of token t
    const int dt = kThreads / per_row, dk = kThreads - dt * per_row;
    const int t_first = tid / per_row, k_first = tid - t_first * per_row;
    auto next = [&](int& t, int& kp) {
      t += dt, kp += dk;
      if (kp >= per_row) kp -= per_row, ++t;
    };
    uint4 v[kXPieces];
    int t = t_first, kp = k_first;
#pragma unroll
    for (int i = 0; i < kXPieces; ++i) {
      v[i] = make_uint4(0, 0, 0, 0);
      if (t < nt && kp * 8 < a.K)
        v[i] = *reinterpret_cast<const uint4*>(a.x + (int64_t)(t0 + t) * a.x_stride + kp * 8);
      next(t, kp);
    }
    // the first stages, behind x in the memory system's queues
#pragma unroll
    for (int i = 0; i < kSlots; ++i) {
      sc[i] = {0, 0};
      if (l0 + i < l1) sc[i] = issue(i);
    }
    if (bf16) {
      t = t_first, kp = k_first;
#pragma unroll
      for (int i = 0; i < kXPieces; ++i) {
        if (t >= nt) break;
        uint32_t top = top_bf16(v[i]);
        // a row is per_row (a multiple of 32) consecutive pieces: the warp's 32 lie in one row
        top = __reduce_max_sync(0xffffffffu, top);
        if (lane == 0) atomicMax(&s_amax[t], top);
        next(t, kp);
      }
    }
    __syncthreads();
    if (bf16) {                                  // 2^-e as two factors, each a normal float
      if (tid < COLS) {
        s_scale[tid] = down_factors(s_amax[tid]);
        s_factor[tid] = pow2f(f16_prescale_exp(__uint_as_float(s_amax[tid] << 16)));
      }
      __syncthreads();
    }
    t = t_first, kp = k_first;
#pragma unroll
    for (int i = 0; i < kXPieces; ++i) {
      if (t >= COLS) break;
      if (bf16 && t < nt) v[i] = scale_bf16(v[i], s_scale[t]);
      *reinterpret_cast<uint4*>(s_x + x_byte(kp, t, COLS)) = v[i];
      next(t, kp);
    }
    __syncthreads();
  }

  // lanes of columns that do not exist read the last one; their sums are not stored
  const char* x_lane = s_x + ((COLS < 8 ? min(g, COLS - 1) : g) * 4 + c) * 16;
  constexpr int kXStage = 8 * COLS * 64, kXQuarter = COLS * 64;

  float acc[NB][4], head[NB][4];
#pragma unroll
  for (int nb = 0; nb < NB; ++nb)
#pragma unroll
    for (int x = 0; x < 4; ++x) acc[nb][x] = 0.0f, head[nb][x] = 0.0f;

  const float alpha = a.alpha ? *a.alpha : 1.0f;
  auto factor = [&](int t) {                     // undoes token t's prescale
    return PREP || bf16 ? s_factor[t] * alpha : alpha;
  };
  auto store = [&](int64_t n, int t, float v) {  // v: the row's sum times alpha and the prescale
    if (n >= a.N || t >= nt) return;
    const int64_t at = (int64_t)(t0 + t) * a.y_stride + n;
    if (a.y_dtype == MOE_DTYPE_F32) static_cast<float*>(a.y)[at] = v;
    else if (a.y_dtype == MOE_DTYPE_BF16) static_cast<uint16_t*>(a.y)[at] = (uint16_t)f32_to_act<MOE_DTYPE_BF16>(v);
    else static_cast<uint16_t*>(a.y)[at] = (uint16_t)f32_to_act<MOE_DTYPE_F16>(v);
  };

  bool ok = true;
  int s = l0 % ks, tile = l0 / ks;
  const char* xs = x_lane + s * kXStage;
  uint32_t parity = 0;
  int l = l0;
  const int w_at = g * 128 + (((2 * c) ^ g) * 16), w_at1 = g * 128 + (((2 * c + 1) ^ g) * 16);
  while (l < l1 && ok) {
#pragma unroll
    for (int slot = 0; slot < kSlots; ++slot) {
      if (l >= l1) break;
      // every lane looks at the barrier itself; the bounded wait is for copies not there yet
      if (!__all_sync(0xffffffffu, mbar_try(&full[slot], parity)))
        ok = mbar_wait_warp(&full[slot], parity, &s_abort, err);
      if (!ok) break;
      const char* wb = ring + slot * kStageB;
      float part[NB][4];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int x = 0; x < 4; ++x) part[nb][x] = 0.0f;
      const uint32_t s0[2] = {e4m3x2_to_f16x2(sc[slot].r0 & 0xffffu), e4m3x2_to_f16x2(sc[slot].r0 >> 16)};
      const uint32_t s1[2] = {e4m3x2_to_f16x2(sc[slot].r1 & 0xffffu), e4m3x2_to_f16x2(sc[slot].r1 >> 16)};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const char* at = wb + (j ? w_at1 : w_at);
        const uint4 c0 = *reinterpret_cast<const uint4*>(at);
        const uint4 c1 = *reinterpret_cast<const uint4*>(at + 8 * 128);
        const uint32_t w0[4] = {c0.x, c0.y, c0.z, c0.w}, w1[4] = {c1.x, c1.y, c1.z, c1.w};
        const uint32_t sa[2] = {bcast_lo(s0[j]), bcast_hi(s0[j])}, sb[2] = {bcast_lo(s1[j]), bcast_hi(s1[j])};
#pragma unroll
        for (int q = 0; q < 4; ++q) {            // 8 weights of each row: two k-steps
          uint4 xv[NB];
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
            xv[nb] = *reinterpret_cast<const uint4*>(xs + (j * 4 + q) * kXQuarter + nb * 512);
          uint32_t p[4], r[4];
          e2m1x8_to_f16x2x4(w0[q], p[0], p[1], p[2], p[3]);
          e2m1x8_to_f16x2x4(w1[q], r[0], r[1], r[2], r[3]);
#pragma unroll
          for (int i = 0; i < 4; ++i) p[i] = hmul2_u32(p[i], sa[q >> 1]), r[i] = hmul2_u32(r[i], sb[q >> 1]);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            mma(part[nb], p[0], r[0], p[1], r[1], xv[nb].x, xv[nb].y);
            mma(part[nb], p[2], r[2], p[3], r[3], xv[nb].z, xv[nb].w);
          }
        }
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[nb][x] += part[nb][x];
      __syncwarp();
      if (l + kSlots < l1) sc[slot] = issue(slot);
      ++l;
      xs += kXStage;
      if (++s == ks) {                           // the tile ends here
        if (tile * ks >= l0) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int t = nb * 8 + 2 * c + (x & 1);
              if (t < nt) store((int64_t)(tile0 + tile) * 16 + g + 8 * (x >> 1), t, acc[nb][x] * factor(t));
              acc[nb][x] = 0.0f;
            }
        } else {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int x = 0; x < 4; ++x) head[nb][x] = acc[nb][x], acc[nb][x] = 0.0f;
        }
        s = 0;
        xs = x_lane;
        ++tile;
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
        parts[(warp * 2 + which) * kTile + (nb * 8 + 2 * c + (x & 1)) * 16 + g + 8 * (x >> 1)] = v[nb][x];
  };
  if (l0 < l1) {
    const int first = l0 / ks;
    if (first * ks < l0 && (first + 1) * ks <= l1) park(0, head);   // ended here
    if (l1 % ks != 0) park((l1 / ks) * ks >= l0 ? 1 : 0, acc);      // goes on in the next piece
  }
  __syncthreads();
  for (int u = tid; u < (tile1 - tile0) * kTile; u += kThreads) {
    const int tl = u / kTile, e = u - tl * kTile, t = e / 16;
    const int w0 = tl * ks / per, w1 = (tl * ks + ks - 1) / per;
    if (w0 == w1 || t >= nt) continue;           // stored by its warp, or not a token
    float v = parts[(w0 * 2 + 1) * kTile + e];
    for (int w = w0 + 1; w <= w1; ++w) v += parts[w * 2 * kTile + e];
    store((int64_t)(tile0 + tl) * 16 + e % 16, t, v * factor(t));
  }
}

template <int COLS, bool PREP>
cudaError_t launch_cols(const LinearArgs& a, cudaStream_t s) {
  CUtensorMap map;
  if (!make_map(&map, a.codes, (uint64_t)a.K / 2, (uint64_t)a.K / 2, (uint64_t)a.N, 128, 16, true))
    return cudaErrorInvalidValue;
  const int kpad = (a.K + kStageW - 1) / kStageW * kStageW;
  const size_t smem = 1024 + kRingB + (size_t)COLS * kpad * 2;
  auto kern = linear_kernel<COLS, PREP>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       1024 + kRingB + kXBytes);
  if (e != cudaSuccess) return e;
  const int tiles = (a.N + 15) / 16;
  const dim3 grid(tiles < num_sms() ? tiles : num_sms(), (a.T + COLS - 1) / COLS);
  if (PREP) {
    x_prep_kernel<<<a.T, kPrepThreads, 0, s>>>(a, COLS, kpad);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    return launch_pdl(kern, grid, dim3(kThreads), smem, s, a, map);
  }
  kern<<<grid, kThreads, smem, s>>>(a, map);
  return cudaGetLastError();
}
template <int COLS>
cudaError_t launch_either(const LinearArgs& a, cudaStream_t s) {
  const int kpad = (a.K + kStageW - 1) / kStageW * kStageW;
  return a.T <= kPrepTokens && COLS * kpad * 2 >= kPrepBytes ? launch_cols<COLS, true>(a, s)
                                                             : launch_cols<COLS, false>(a, s);
}

}  // namespace

size_t linear_ws_bytes(int T, int N, int K) {
  const size_t kpad = (K + kStageW - 1) / kStageW * kStageW;
  const int most = T < kPrepTokens ? (T + 31) / 32 * 32 : kPrepTokens;
  return align_up(kFragsAt + most * kpad * 2);
}

cudaError_t launch_linear(const LinearArgs& a, cudaStream_t s) {
  // Tokens per pass over the weights: the least power of two that holds them all, up to 32 and to
  // what x's share of shared memory holds.
  const int kpad = (a.K + kStageW - 1) / kStageW * kStageW;
  int cols = 1;
  while (cols < a.T && cols < 32 && (size_t)cols * 2 * kpad * 2 <= (size_t)kXBytes) cols *= 2;
  switch (cols) {
    case 1: return launch_either<1>(a, s);
    case 2: return launch_either<2>(a, s);
    case 4: return launch_either<4>(a, s);
    case 8: return launch_either<8>(a, s);
    case 16: return launch_either<16>(a, s);
    default: return launch_either<32>(a, s);
  }
}

}  // namespace moe
