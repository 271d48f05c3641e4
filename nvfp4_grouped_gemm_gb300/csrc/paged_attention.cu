// Causal attention of new tokens over the paged 8-bit cache (moe_attention_paged_e4m3).
//
// A sequence's n new tokens and the G query heads that share a key head are n*G rows over the
// same keys and values; a segment is (sequence, key head, block of 16*MT such rows). Its keys
// are cut into steps of STEP tokens, and all segments' steps form one line that the grid cuts
// into equal pieces, so a batch of very different lengths loads every SM alike. A CTA whose
// piece covers a whole segment writes its rows; the CTAs of a segment that was cut leave
// their rows' (maximum, sum, weighted values) in the workspace and the last of them to arrive
// joins them in the order of the pieces, so results do not depend on arrival.
//
// Inside a CTA four warps take the piece's steps in turn. Each streams its steps through a ring
// of its own (TMA boxes of E4M3 rows, swizzled so that the fragment reads below hit distinct
// banks), widens the codes to f16 in registers (exact) and multiplies with mma.sync m16n8k16
// (f32 accumulation):
//   S = Q K^T   lane 4g+c holds, of key g of each 8-key block, 16 consecutive values at 16c of
//               every 64; the four bytes of a word are its values of one k-step, and Q's
//               fragments are laid out with the same permutation of k
//   O = P V     P's accumulator layout is the A operand's; V's pairs of keys for one value
//               come from two rows' bytes by byte permutes
// With f = scale * k_scale * log2 e and v = log2 v_scale of a key's page, the weight that meets
// V's codes is w = 2^(s f + v - M) and the softmax sum adds w / v_scale, so the value scale
// costs nothing per element. M follows the running maximum of s f + v lazily: it moves only when
// a weight would pass 2^8, which leaves f16 weights their full precision and makes rescaling of
// the accumulators rare. w is rounded to f16 (2^-11), sums and accumulators are f32.
//
// Keys past a row's place, outside the window, in unused slots or in pages out of range get
// weight 0, and V's bytes there are replaced by 0 (they may be NaN codes).
#include "serving.cuh"
#include "tma_sync.cuh"

namespace moe {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxGrid = 512;              // partial slots of the workspace
constexpr int kMaxRows = 32;
constexpr float kNoMax = -1e30f;
constexpr float kLazy = 8.0f;

// Workspace: error word; arrival counters [kMaxGrid]; partial maxima and sums
// [2 * kMaxGrid][2][kMaxRows]; partial rows f32 [2 * kMaxGrid][kMaxRows][D].
constexpr size_t kCountersAt = kAlign;
constexpr size_t kStatsAt = kCountersAt + kMaxGrid * 4;
constexpr size_t kRowsAt = kStatsAt + (size_t)2 * kMaxGrid * 2 * kMaxRows * 4;

template <int D_, int MT_>
struct Shape {
  static constexpr int D = D_, MT = MT_;
  static constexpr int kStep = D == 256 ? 16 : 32;       // tokens per step
  static constexpr int kHalves = kStep / 16;
  static constexpr int kSubs = D == 256 ? 2 : 1;         // swizzled sub-tiles of a row
  static constexpr int kRowB = D == 64 ? 64 : 128;       // bytes of a sub-tile row
  static constexpr int kPlaneB = kStep * D;              // a step's K (or V) bytes
  static constexpr int kStageB = 2 * kPlaneB;
  static constexpr int kSlots = D == 64 ? 4 : MT == 2 ? 3 : 2;
  static constexpr int kCtas = D == 256 ? 2 : MT == 2 ? 2 : 3;   // per SM
  static constexpr int kRows = 16 * MT;
  static constexpr int kRingB = kWarps * kSlots * kStageB;
  static constexpr int kMergeB = kWarps * kRows * D * 4; // aliases the ring
  static constexpr int kBigB = kRingB > kMergeB ? kRingB : kMergeB;
  static constexpr int kQB = kRows * D * 2;
  static constexpr int kSmem = 1024 + kBigB + kQB;
};

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
// The four E4M3 codes of a word as two f16x2.
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}" : "=r"(lo), "=r"(hi) : "r"(w));
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// What one sequence asks for: rows, steps, and the line of steps it takes.
struct Seq {
  int row0, n, start, len;      // token rows, new tokens, place of the first, visible length
  int step0, steps, blocks;     // first step, steps, row blocks
};
template <class S>
__device__ __forceinline__ Seq read_seq(const AttentionArgs& a, int b, int group, uint32_t* err) {
  Seq q;
  q.row0 = min(max(a.b.q_offsets[b], 0), a.T);
  const int end = min(max(a.b.q_offsets[b + 1], q.row0), a.T);
  q.n = end - q.row0;
  q.len = a.b.seq_lens[b];
  q.start = q.len - q.n;
  const int cap = a.b.max_pages * a.c.page_size;
  if (q.n > 0 && (q.start < 0 || q.len > cap) && err) atomicOr(err, (uint32_t)MOE_DEVERR_PAGE);
  q.len = min(max(q.len, 0), cap);
  const int lo = a.window > 0 ? max(0, min(q.start - a.window + 1, q.len)) : 0;
  q.step0 = lo / S::kStep;
  q.steps = max((q.len + S::kStep - 1) / S::kStep - q.step0, 1);
  q.blocks = (q.n * group + S::kRows - 1) / S::kRows;
  return q;
}

// Sum of v over the block; the exclusive prefix of the calling thread in *before.
__device__ long long block_scan(long long v, long long* s_sum, long long* before) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += up;
  }
  __syncthreads();
  if (lane == 31) s_sum[warp] = x;
  __syncthreads();
  long long base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) base += s_sum[w];
    all += s_sum[w];
  }
  *before = base + x - v;
  return all;
}

// A warp's keys: which page each half-step (16 tokens) lies in, its scales, for 32 of them at a
// time (lane l holds half-step l of the batch).
struct Keys {
  int page;                     // -1: outside the sequence or out of range
  float f, v, inv;              // scale * k_scale * log2 e; log2 v_scale; 1 / v_scale
};

template <int DT, class S>
__global__ void __launch_bounds__(kThreads, S::kCtas)
attention_kernel(const __grid_constant__ AttentionArgs a, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap) {
  constexpr int D = S::D, MT = S::MT, NB = S::kStep / 8;
  extern __shared__ char smem_raw[];
  __shared__ uint64_t s_full[kWarps * S::kSlots];
  __shared__ long long s_sum[kWarps];
  __shared__ int s_seq;
  __shared__ long long s_first;
  __shared__ volatile int s_abort;
  __shared__ float s_rowf[S::kRows], s_m[kWarps][S::kRows], s_l[kWarps][S::kRows];
  __shared__ int s_last;
  char* big = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  char* s_q = big + S::kBigB;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  uint32_t* err = reinterpret_cast<uint32_t*>(a.ws);
  uint32_t* counters = reinterpret_cast<uint32_t*>(a.ws + kCountersAt);
  float* stats = reinterpret_cast<float*>(a.ws + kStatsAt);
  float* part = reinterpret_cast<float*>(a.ws + kRowsAt);
  const int heads = a.c.kv_heads, group = a.q_heads / heads, P = a.c.page_size;

  if (tid < kWarps * S::kSlots) mbar_init(&s_full[tid], 1);
  if (tid == 0) s_abort = 0;
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");

  // This CTA's piece of the line of steps.
  long long total = 0, mine = 0, at = 0;
  for (int b0 = 0; b0 < a.b.B; b0 += kThreads) {
    mine = 0;
    if (b0 + tid < a.b.B) {
      const Seq q = read_seq<S>(a, b0 + tid, group, blockIdx.x == 0 ? err : nullptr);
      mine = (long long)q.steps * q.blocks * heads;
    }
    total += block_scan(mine, s_sum, &at);
  }
  long long per = (total + gridDim.x - 1) / gridDim.x;
  if (per < kWarps) per = kWarps;
  const long long begin = per * blockIdx.x, end = min(begin + per, total);
  if (begin >= end) return;
  if (a.b.B <= kThreads) {
    if (mine > 0 && at <= begin && begin < at + mine) s_seq = tid, s_first = at;
  } else {
    long long base = 0;
    for (int b0 = 0; b0 < a.b.B; b0 += kThreads) {
      mine = 0;
      if (b0 + tid < a.b.B) {
        const Seq q = read_seq<S>(a, b0 + tid, group, nullptr);
        mine = (long long)q.steps * q.blocks * heads;
      }
      const long long sum = block_scan(mine, s_sum, &at);
      if (mine > 0 && base + at <= begin && begin < base + at + mine) s_seq = b0 + tid, s_first = base + at;
      base += sum;
    }
  }
  __syncthreads();
  int b = s_seq;
  long long first = s_first;                  // the line's place of sequence b's first step
  Seq q = read_seq<S>(a, b, group, nullptr);

  char* ring = big + warp * S::kSlots * S::kStageB;
  uint64_t* full = s_full + warp * S::kSlots;
  int issued = 0, taken = 0;                  // stages of this warp's ring, over all segments
  const int tok_n = D == 64 ? g : (g >> 1) + 4 * (g & 1);   // key of an 8-key block in column g
  const int tok_a = D == 64 ? 2 * c : c, tok_b = D == 64 ? 2 * c + 1 : c + 4;  // columns 2c, 2c+1
  const int swz_k = D == 64 ? (tok_n >> 1) & 3 : tok_n;
  const int vch = D == 64 ? g >> 1 : (g >> 1) + 4 * (g & 1);
  const uint32_t q_addr = smem_u32(s_q) + lane * 16;

  for (long long pos = begin; pos < end;) {
    while (pos >= first + (long long)q.steps * q.blocks * heads) {
      first += (long long)q.steps * q.blocks * heads;
      q = read_seq<S>(a, ++b, group, nullptr);
    }
    const long long in_seq = pos - first;
    const int seg = (int)(in_seq / q.steps), st0 = (int)(in_seq % q.steps);
    const long long seg_at = first + (long long)seg * q.steps;
    const int st1 = (int)min((long long)q.steps, end - seg_at);
    const int head = seg / q.blocks, block = seg % q.blocks;
    const int R = min(S::kRows, q.n * group - block * S::kRows);
    // rows' places: row r of the block belongs to token (block * kRows + r) / group
    const int tok_first = block * S::kRows / group, tok_last = (block * S::kRows + R - 1) / group;
    const int place_lo = q.start + tok_first;
    // steps this block of rows can see at all
    int w0 = q.step0 + st0, w1 = q.step0 + st1;
    {
      const int hi = min(q.len, q.start + tok_last + 1);
      const int lo = a.window > 0 ? max(0, place_lo - a.window + 1) : 0;
      w1 = min(w1, (max(hi, 0) + S::kStep - 1) / S::kStep);
      w0 = max(w0, lo / S::kStep);
    }

    // ---- this warp's stream ----
    const int count = w1 > w0 + warp ? (w1 - w0 - warp + kWarps - 1) / kWarps : 0;
    Keys cur = {-1, 0.f, 0.f, 0.f}, nxt = cur;
    auto load_keys = [&](int batch) {
      Keys k = {-1, 0.f, 0.f, 0.f};
      constexpr int kPer = 32 / S::kHalves;               // steps per batch
      const int i = batch * kPer + lane / S::kHalves;
      if (i < count) {
        const int j = (w0 + warp + i * kWarps) * S::kStep + (lane % S::kHalves) * 16;
        if (j < q.len) {
          const int page = __ldg(a.b.page_table + (int64_t)b * a.b.table_stride + j / P);
          if (page >= 0 && page < a.c.num_pages) {
            k.page = page;
            const int64_t sc = (int64_t)page * heads + head;
            k.f = a.scale * 1.4426950408889634f * __ldg(a.c.k_scales + sc);
            const float vs = fminf(fmaxf(__ldg(a.c.v_scales + sc), 0x1p-100f), 0x1p120f);
            k.v = log2f(vs);
            k.inv = __fdividef(1.0f, vs);
          } else {
            atomicOr(err, (uint32_t)MOE_DEVERR_PAGE);
          }
        }
      }
      return k;
    };
    constexpr int kPer = 32 / S::kHalves;
    int have = 0;                                          // key batches loaded
    auto issue = [&](int i) {                              // all lanes
      const int batch = i / kPer;
      if (batch >= have) {
        cur = nxt;
        nxt = load_keys(batch);
        if (have == 0) cur = nxt;
        ++have;
      }
      const int slot = issued % S::kSlots;
      const int src = (i % kPer) * S::kHalves;
      int page[S::kHalves];
#pragma unroll
      for (int h = 0; h < S::kHalves; ++h) page[h] = __shfl_sync(0xffffffffu, nxt.page, src + h);
      if (lane == 0) {
        char* st = ring + slot * S::kStageB;
        const int j = (w0 + warp + i * kWarps) * S::kStep;
        const bool whole = P >= S::kStep;                  // one box per step and sub-tile
        uint32_t bytes = 0;
#pragma unroll
        for (int h = 0; h < S::kHalves; ++h)
          if (page[h] >= 0 && (!whole || h == 0)) bytes += whole ? S::kStageB : S::kStageB / S::kHalves;
        mbar_expect_tx(&full[slot], bytes);
#pragma unroll
        for (int h = 0; h < S::kHalves; ++h) {
          if (page[h] < 0 || (whole && h > 0)) continue;
          const int row = head * P + (j + h * 16) % P;
#pragma unroll
          for (int s = 0; s < S::kSubs; ++s) {
            char* dst = st + s * (S::kStep * 128) + h * 16 * S::kRowB;
            tma_load_3d(dst, &kmap, s * 128, row, page[h], &full[slot]);
            tma_load_3d(dst + S::kPlaneB, &vmap, s * 128, row, page[h], &full[slot]);
          }
        }
      }
      ++issued;
    };
    for (int i = 0; i < min(count, S::kSlots); ++i) issue(i);

    // ---- queries as A fragments: k-step ks, row tile mt: lane 16 B (a0, a2, a1, a3) ----
    for (int r = warp; r < S::kRows; r += kWarps) {
      constexpr int kQuads = (D / 4 + 31) / 32;
      float v[kQuads][4];
      float amax = 0.0f;
      const int rr = block * S::kRows + r;
      const uint16_t* src = a.q + (int64_t)(q.row0 + rr / group) * a.q_stride +
                            (int64_t)(head * group + rr % group) * D;
#pragma unroll
      for (int i = 0; i < kQuads; ++i) {
        const int u = lane + 32 * i;
        uint2 w = make_uint2(0, 0);
        if (r < R && u < D / 4) w = *reinterpret_cast<const uint2*>(src + 4 * u);
        v[i][0] = act_to_f32<DT>(w.x & 0xffffu), v[i][1] = act_to_f32<DT>(w.x >> 16);
        v[i][2] = act_to_f32<DT>(w.y & 0xffffu), v[i][3] = act_to_f32<DT>(w.y >> 16);
#pragma unroll
        for (int x = 0; x < 4; ++x) amax = fmaxf(amax, fabsf(v[i][x]));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      // bf16 rows get the power of two that puts their largest magnitude below 2^15
      const int e = DT == MOE_DTYPE_BF16 && amax < 3.4e38f ? f16_prescale_exp(amax) : 0;
      const float s1 = pow2f(-e / 2), s2 = pow2f(-e - (-e / 2));
      if (lane == 0) s_rowf[r] = pow2f(e);
#pragma unroll
      for (int i = 0; i < kQuads; ++i) {
        const int u = lane + 32 * i;
        if (u < D / 4) {
          const int ks = (u >> 4) * 4 + (u & 3), cc = (u >> 2) & 3;
          char* dst = s_q + (ks * MT + (r >> 4)) * 512 + ((r & 7) * 4 + cc) * 16 + ((r >> 3) & 1) * 8;
          *reinterpret_cast<uint2*>(dst) =
              make_uint2(pack_f16(v[i][0] * s1 * s2, v[i][1] * s1 * s2),
                         pack_f16(v[i][2] * s1 * s2, v[i][3] * s1 * s2));
        }
      }
    }
    __syncthreads();

    float O[MT][D / 8][4];
    float M[MT][2], L[MT][2], rowf[MT][2];
    int place[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int n = 0; n < D / 8; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) O[mt][n][x] = 0.0f;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = 16 * mt + 8 * x + g;
        M[mt][x] = kNoMax, L[mt][x] = 0.0f;
        rowf[mt][x] = s_rowf[r];
        place[mt][x] = q.start + (block * S::kRows + r) / group;
      }
    }

    bool ok = true;
    for (int i = 0; i < count && ok; ++i) {
      const int slot = taken % S::kSlots;
      ok = mbar_wait_warp(&full[slot], (taken / S::kSlots) & 1, &s_abort, err);
      if (!ok) break;
      const uint32_t kb = smem_u32(ring + slot * S::kStageB), vb = kb + S::kPlaneB;
      const int j0 = (w0 + warp + i * kWarps) * S::kStep;

      float sc[MT][NB][4];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int x = 0; x < 4; ++x) sc[mt][nb][x] = 0.0f;
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        uint4 kc[NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
          kc[nb] = lds128(kb + (j >> 1) * (S::kStep * 128) + (nb * 8 + tok_n) * S::kRowB +
                          (((4 * (j & 1) + c) ^ swz_k) * 16));
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          uint4 A[MT];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) A[mt] = lds128(q_addr + ((4 * j + m) * MT + mt) * 512);
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const uint32_t w = m == 0 ? kc[nb].x : m == 1 ? kc[nb].y : m == 2 ? kc[nb].z : kc[nb].w;
            uint32_t b0, b1;
            widen4(w, b0, b1);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
              mma_f16_16816(sc[mt][nb], A[mt].x, A[mt].z, A[mt].y, A[mt].w, b0, b1);
          }
        }
      }

      // weights
      const int src = (i % kPer) * S::kHalves;
      const bool newer = i / kPer == have - 1;             // which key batch this step is in
      float kf[S::kHalves], kv[S::kHalves], ki[S::kHalves];
      bool good[S::kHalves];
      bool masked = j0 + S::kStep > place_lo + 1 || j0 + S::kStep > q.len;
      if (a.window > 0) masked |= j0 <= q.start + tok_last - a.window;
#pragma unroll
      for (int h = 0; h < S::kHalves; ++h) {
        kf[h] = __shfl_sync(0xffffffffu, newer ? nxt.f : cur.f, src + h);
        kv[h] = __shfl_sync(0xffffffffu, newer ? nxt.v : cur.v, src + h);
        ki[h] = __shfl_sync(0xffffffffu, newer ? nxt.inv : cur.inv, src + h);
        good[h] = __shfl_sync(0xffffffffu, newer ? nxt.page : cur.page, src + h) >= 0;
        masked |= !good[h];
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          const int h = nb / 2;
#pragma unroll
          for (int x = 0; x < 4; ++x) sc[mt][nb][x] = fmaf(sc[mt][nb][x], kf[h] * rowf[mt][x >> 1], kv[h]);
          if (masked) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int j = j0 + nb * 8 + (x & 1 ? tok_b : tok_a);
              const int pl = place[mt][x >> 1];
              const bool see = good[h] && j <= pl && j < q.len && (a.window == 0 || j > pl - a.window);
              if (!see) sc[mt][nb][x] = -INFINITY;
            }
          }
        }
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int x = 0; x < 4; ++x) top[x >> 1] = fmaxf(top[x >> 1], sc[mt][nb][x]);
        const bool move = top[0] > M[mt][0] + kLazy || top[1] > M[mt][1] + kLazy;
        if (__any_sync(0xffffffffu, move)) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 1));
            top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 2));
            const float to = fmaxf(M[mt][x], top[x]);
            const float keep = exp2_approx(M[mt][x] - to);
            M[mt][x] = to;
            L[mt][x] *= keep;
#pragma unroll
            for (int n = 0; n < D / 8; ++n) O[mt][n][2 * x] *= keep, O[mt][n][2 * x + 1] *= keep;
          }
        }
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int x = 0; x < 4; ++x) sc[mt][nb][x] = exp2_approx(sc[mt][nb][x] - M[mt][x >> 1]);
#pragma unroll
        for (int h = 0; h < S::kHalves; ++h)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            L[mt][x] = fmaf(ki[h], (sc[mt][2 * h][2 * x] + sc[mt][2 * h][2 * x + 1]) +
                                       (sc[mt][2 * h + 1][2 * x] + sc[mt][2 * h + 1][2 * x + 1]), L[mt][x]);
      }

      // values
#pragma unroll
      for (int h = 0; h < S::kHalves; ++h) {
        uint32_t pa[MT][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          pa[mt][0] = pack_f16(sc[mt][2 * h][0], sc[mt][2 * h][1]);
          pa[mt][1] = pack_f16(sc[mt][2 * h][2], sc[mt][2 * h][3]);
          pa[mt][2] = pack_f16(sc[mt][2 * h + 1][0], sc[mt][2 * h + 1][1]);
          pa[mt][3] = pack_f16(sc[mt][2 * h + 1][2], sc[mt][2 * h + 1][3]);
        }
        const int rows[4] = {h * 16 + tok_a, h * 16 + tok_b, h * 16 + 8 + tok_a, h * 16 + 8 + tok_b};
#pragma unroll
        for (int s = 0; s < S::kSubs; ++s) {
          constexpr int kWords = D == 64 ? 2 : 4;
          uint32_t x[4][kWords];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int swz = D == 64 ? (rows[r] >> 1) & 3 : rows[r] & 7;
            const uint32_t at_ = vb + s * (S::kStep * 128) + rows[r] * S::kRowB + ((vch ^ swz) * 16);
            if (D == 64) {
              const uint2 t = lds64(at_ + (g & 1) * 8);
              x[r][0] = t.x, x[r][1] = t.y;
            } else {
              const uint4 t = lds128(at_);
              x[r][0] = t.x, x[r][1] = t.y, x[r][kWords - 2] = t.z, x[r][kWords - 1] = t.w;
            }
            if (masked && !(good[h] && j0 + rows[r] < q.len)) {
#pragma unroll
              for (int i2 = 0; i2 < kWords; ++i2) x[r][i2] = 0;
            }
          }
#pragma unroll
          for (int m = 0; m < kWords; ++m) {
            uint32_t b0[4], b1[4];
            widen4(__byte_perm(x[0][m], x[1][m], 0x5140), b0[0], b0[1]);
            widen4(__byte_perm(x[0][m], x[1][m], 0x7362), b0[2], b0[3]);
            widen4(__byte_perm(x[2][m], x[3][m], 0x5140), b1[0], b1[1]);
            widen4(__byte_perm(x[2][m], x[3][m], 0x7362), b1[2], b1[3]);
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
                mma_f16_16816(O[mt][s * 16 + 4 * m + t], pa[mt][0], pa[mt][1], pa[mt][2], pa[mt][3],
                              b0[t], b1[t]);
          }
        }
      }
      ++taken;
      __syncwarp();
      if (i + S::kSlots < count) issue(i + S::kSlots);
    }
    if (!ok) {
      // gave up: let this warp's copies in flight land (bounded) before the CTA leaves
      for (; taken < issued; ++taken) {
        const uint64_t t0 = global_ns();
        while (!mbar_try(&full[taken % S::kSlots], (taken / S::kSlots) & 1) &&
               global_ns() - t0 < 100000000ull) {
        }
      }
    }

    // ---- the four warps' rows meet ----
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        L[mt][x] += __shfl_xor_sync(0xffffffffu, L[mt][x], 1);
        L[mt][x] += __shfl_xor_sync(0xffffffffu, L[mt][x], 2);
        if (c == 0) {
          s_m[warp][16 * mt + 8 * x + g] = M[mt][x];
          s_l[warp][16 * mt + 8 * x + g] = L[mt][x];
        }
      }
    __syncthreads();                           // also: every warp is done with the ring
    if (s_abort) return;                       // the same for the whole block
    float* merge = reinterpret_cast<float*>(big);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int r = 16 * mt + 8 * x + g;
        float top = kNoMax;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
        const float keep = exp2_approx(M[mt][x] - top);
        // columns 2c and 2c+1 of the 8-value blocks: runs of 16 (D = 64: 8) values
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int col = 2 * c + y;
#pragma unroll
          for (int n = 0; n < D / 8; n += 4) {
            const int at_ = D == 64 ? col * 8 + n : (n / 16) * 128 + ((col >> 1) + 4 * (col & 1)) * 16 + n % 16;
            // 16-byte units of a row rotated so that a quarter warp's stores differ in bank
            const int unit = (at_ / 4) ^ ((c >> 1) ^ ((g & 1) << 1));
            *reinterpret_cast<float4*>(merge + ((size_t)warp * S::kRows + r) * D + unit * 4) =
                make_float4(O[mt][n][2 * x + y] * keep, O[mt][n + 1][2 * x + y] * keep,
                            O[mt][n + 2][2 * x + y] * keep, O[mt][n + 3][2 * x + y] * keep);
          }
        }
      }
    __syncthreads();
    const bool opens = st0 == 0, closes = st1 == q.steps;
    const bool whole_seg = opens && closes;
    const int slot = 2 * blockIdx.x + (opens ? 1 : 0);
    auto store_row = [&](int r, int d, float4 v, float top, float sum) {
      const int rr = block * S::kRows + r;
      const int64_t row = q.row0 + rr / group;
      const int hq = head * group + rr % group;
      const float inv = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;   // NaN stays
      uint2 w;
      w.x = f32_to_act<DT>(v.x * inv) | (f32_to_act<DT>(v.y * inv) << 16);
      w.y = f32_to_act<DT>(v.z * inv) | (f32_to_act<DT>(v.w * inv) << 16);
      *reinterpret_cast<uint2*>(a.out + row * a.out_stride + (int64_t)hq * D + d) = w;
      if (d == 0 && a.lse)
        a.lse[row * a.q_heads + hq] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    };
    for (int u = tid; u < R * (D / 4); u += kThreads) {
      const int r = u / (D / 4), d = (u % (D / 4)) * 4;
      // the writer of this unit was the lane with column col of row r
      const int col16 = D == 64 ? d / 8 : (d % 128) / 16;
      const int col = D == 64 ? col16 : ((col16 & 3) << 1) | (col16 >> 2);
      const int unit = (d / 4) ^ (((col >> 1) >> 1) ^ ((r & 1) << 1));
      float top = kNoMax, sum = 0.0f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 o = *reinterpret_cast<const float4*>(merge + ((size_t)w * S::kRows + r) * D + unit * 4);
        v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
        sum = fmaf(s_l[w][r], exp2_approx(s_m[w][r] - top), sum);
      }
      if (whole_seg) {
        store_row(r, d, v, top, sum);
      } else {
        *reinterpret_cast<float4*>(part + ((size_t)slot * kMaxRows + r) * D + d) = v;
        if (d == 0) {
          stats[(size_t)slot * 2 * kMaxRows + r] = top;
          stats[(size_t)slot * 2 * kMaxRows + kMaxRows + r] = sum;
        }
      }
    }
    if (!whole_seg) {
      // the last piece of the segment to arrive joins all of them
      const int c0 = (int)(seg_at / per), c1 = (int)((seg_at + q.steps - 1) / per);
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const uint32_t before = atomicAdd(&counters[c0], 1u);
        s_last = before == (uint32_t)(c1 - c0);
        if (s_last) counters[c0] = 0;
      }
      __syncthreads();
      if (s_last) {
        __threadfence();
        for (int u = tid; u < R * (D / 4); u += kThreads) {
          const int r = u / (D / 4), d = (u % (D / 4)) * 4;
          float top = kNoMax;
          for (int p = c0; p <= c1; ++p)
            top = fmaxf(top, __ldcg(stats + (size_t)(2 * p + (p == c0)) * 2 * kMaxRows + r));
          float sum = 0.0f;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
          for (int p = c0; p <= c1; ++p) {
            const size_t sl = 2 * p + (p == c0);
            const float k = exp2_approx(__ldcg(stats + sl * 2 * kMaxRows + r) - top);
            sum = fmaf(__ldcg(stats + sl * 2 * kMaxRows + kMaxRows + r), k, sum);
            const float4 o = __ldcg(reinterpret_cast<const float4*>(part + (sl * kMaxRows + r) * D + d));
            v.x = fmaf(o.x, k, v.x), v.y = fmaf(o.y, k, v.y), v.z = fmaf(o.z, k, v.z), v.w = fmaf(o.w, k, v.w);
          }
          store_row(r, d, v, top, sum);
        }
      }
    }
    pos = seg_at + st1;
    // plain writes to the ring's memory come before the next segment's copies into it
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
  }
}

template <int DT, int D, int MT>
cudaError_t launch_shape(const AttentionArgs& a, cudaStream_t s) {
  using S = Shape<D, MT>;
  CUtensorMap map[2];
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.c.kv_heads * a.c.page_size, (uint64_t)a.c.num_pages};
  const uint64_t strides[2] = {(uint64_t)D, (uint64_t)a.c.page_stride};
  const uint32_t box[3] = {(uint32_t)S::kRowB, (uint32_t)(a.c.page_size < S::kStep ? 16 : S::kStep), 1};
  const CUtensorMapSwizzle swz = D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  if (!make_map3(&map[0], a.c.k_codes, dims, strides, box, swz) ||
      !make_map3(&map[1], a.c.v_codes, dims, strides, box, swz))
    return cudaErrorInvalidValue;
  auto kern = attention_kernel<DT, S>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  int grid = num_sms() * S::kCtas;
  if (grid > kMaxGrid) grid = kMaxGrid;
  kern<<<grid, kThreads, S::kSmem, s>>>(a, map[0], map[1]);
  return cudaGetLastError();
}

template <int DT>
cudaError_t launch_dim(const AttentionArgs& a, cudaStream_t s) {
  // Two row tiles once the sequences' rows do not fit one on average: each pass over the keys
  // then serves 32 rows (256-value heads keep one: their accumulators fill the registers).
  const bool wide = (long long)a.T * (a.q_heads / a.c.kv_heads) > 16LL * a.b.B;
  if (a.c.head_dim == 64) return wide ? launch_shape<DT, 64, 2>(a, s) : launch_shape<DT, 64, 1>(a, s);
  if (a.c.head_dim == 128) return wide ? launch_shape<DT, 128, 2>(a, s) : launch_shape<DT, 128, 1>(a, s);
  return launch_shape<DT, 256, 1>(a, s);
}

}  // namespace

size_t attention_ws_bytes(int q_heads, int kv_heads, int head_dim) {
  return align_up(kRowsAt + (size_t)2 * kMaxGrid * kMaxRows * head_dim * 4);
}

cudaError_t launch_attention(const AttentionArgs& a, int dtype, cudaStream_t s) {
  return dtype == MOE_DTYPE_BF16 ? launch_dim<MOE_DTYPE_BF16>(a, s) : launch_dim<MOE_DTYPE_F16>(a, s);
}

}  // namespace moe
