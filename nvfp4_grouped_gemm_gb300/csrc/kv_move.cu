// Tokens that change their place in the paged 8-bit cache: a tree's accepted path (moe_kv_keep_e4m3)
// and the tokens that a budget keeps (moe_kv_evict_e4m3).
//
// A page has one scale per head, so a page into which tokens move takes the largest of their old pages'
// scales and its codes become RN(code * old / new); where old = new the bits are copied.
//
// keep: a CTA per (sequence, key head, plane) walks the pages that change in order. Places ascend, so
// a page's tokens come from itself or later pages; a page is read whole before it is written, and no
// later page needs what an earlier one overwrote.
//
// evict: select_kernel finds, per (sequence, key head), the weights' threshold by a radix descent over
// order-preserving keys (11, 11 and 10 bits, histograms in shared memory), then lists the kept places
// by ballots in order: ties at the threshold go to the lower places. copy_kernel has a CTA per page
// of the copy; all reads are from pages that nobody writes, so pages are independent of one another.
#include "serving.cuh"

namespace moe {
namespace {

constexpr int kMoveThreads = 256;
// 16-byte pieces of a page per thread and plane: 128 slots of 256 values.
constexpr int kMostPieces = 128 * 256 / 16 / kMoveThreads;

// Four codes under another scale.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float ratio) {
  const float2 a = e4m3x2_to_f32x2(w & 0xffffu), b = e4m3x2_to_f32x2(w >> 16);
  return f32x2_to_e4m3x2(a.x * ratio, a.y * ratio) | f32x2_to_e4m3x2(b.x * ratio, b.y * ratio) << 16;
}
__device__ __forceinline__ uint4 rescale16(const uint4& v, float ratio) {
  if (ratio == 1.0f) return v;
  return make_uint4(rescale4(v.x, ratio), rescale4(v.y, ratio), rescale4(v.z, ratio), rescale4(v.w, ratio));
}

// ---------------------------------------------------------------------------
// keep
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(kMoveThreads) keep_kernel(const __grid_constant__ KeepArgs a) {
  __shared__ int s_first_bad, s_first_move;
  __shared__ int s_from[128];                  // a slot's source page (-1: stays as it is)
  __shared__ int s_slot[128];
  __shared__ float s_ratio[128];
  __shared__ float s_new;
  const int tid = threadIdx.x, plane = blockIdx.x & 1;
  const int h = (blockIdx.x >> 1) % a.c.kv_heads, b = (blockIdx.x >> 1) / a.c.kv_heads;
  const int P = a.c.page_size, D = a.c.head_dim, heads = a.c.kv_heads;
  const bool speaks = plane == 0 && h == 0;    // reports and writes the new length
  const int n = max(a.b.q_offsets[b + 1] - a.b.q_offsets[b], 0), len = a.b.seq_lens[b];
  const int start = len - n;
  if (start < 0 || len > (int64_t)a.b.max_pages * P) {
    if (speaks && tid == 0) {
      atomicOr(a.err, (uint32_t)MOE_DEVERR_PAGE);
      a.new_lens[b] = len;
    }
    return;
  }
  const int32_t* list = a.keep + (int64_t)b * a.width;
  const int asked = min(max(a.n_keep[b], 0), a.width);
  if (tid == 0) s_first_bad = asked, s_first_move = asked;
  __syncthreads();
  for (int i = tid; i < asked; i += kMoveThreads) {
    const int v = list[i], before = i > 0 ? list[i - 1] : -1;
    if (v <= before || v >= n) atomicMin(&s_first_bad, i);
    if (v != i) atomicMin(&s_first_move, i);
  }
  __syncthreads();
  const int count = s_first_bad, move0 = min(s_first_move, count);
  if (speaks && tid == 0) {
    if (count < asked) atomicOr(a.err, (uint32_t)MOE_DEVERR_TOKEN);
    a.new_lens[b] = start + count;
  }
  uint8_t* codes = plane ? a.c.v_codes : a.c.k_codes;
  float* scales = plane ? a.c.v_scales : a.c.k_scales;
  const int32_t* table = a.b.page_table + (int64_t)b * a.b.table_stride;
  const int pieces = D / 16, all = P * pieces;
  for (int pi = (start + move0) / P; pi * P < start + count; ++pi) {
    if (move0 == count) break;
    const int page = table[pi];
    const bool good = page >= 0 && page < a.c.num_pages;
    __syncthreads();                           // the page before is done with the shared arrays
    if (tid < 32) {                            // a lane per slot, the largest scale over all
      const float own = good ? scales[(int64_t)page * heads + h] : 0.0f;
      float top = own;
      for (int s = tid; s < P; s += 32) {
        const int i = pi * P + s - start;      // the kept token that lands here
        int from = -1, slot = 0;
        float scale = own;
        if (i >= move0 && i < count && list[i] != i) {
          const int src = start + list[i];
          const int p = table[src / P];
          if (good && p >= 0 && p < a.c.num_pages) {
            from = p, slot = src % P;
            scale = scales[(int64_t)p * heads + h];
          } else {
            atomicOr(a.err, (uint32_t)MOE_DEVERR_PAGE);
          }
        }
        s_from[s] = from, s_slot[s] = slot, s_ratio[s] = scale;
        top = fmaxf(top, scale);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      for (int s = tid; s < P; s += 32) s_ratio[s] = s_ratio[s] == top ? 1.0f : s_ratio[s] / top;
      if (tid == 0) s_new = top > own ? top : 0.0f;        // 0: the scale stays
    }
    __syncthreads();
    if (!good) continue;
    const bool grew = s_new > 0.0f;
    uint4 v[kMostPieces];
#pragma unroll
    for (int k = 0; k < kMostPieces; ++k) {
      const int u = tid + k * kMoveThreads, s = u / pieces;
      v[k] = make_uint4(0, 0, 0, 0);
      if (u < all && (grew || s_from[s] >= 0)) {
        const int p = s_from[s] >= 0 ? s_from[s] : page, sl = s_from[s] >= 0 ? s_slot[s] : s;
        v[k] = *reinterpret_cast<const uint4*>(codes + (int64_t)p * a.c.page_stride +
                                               ((int64_t)h * P + sl) * D + (u % pieces) * 16);
      }
    }
    __syncthreads();                           // the page is read whole before it is written
#pragma unroll
    for (int k = 0; k < kMostPieces; ++k) {
      const int u = tid + k * kMoveThreads, s = u / pieces;
      if (u < all && (grew || s_from[s] >= 0))
        *reinterpret_cast<uint4*>(codes + (int64_t)page * a.c.page_stride + ((int64_t)h * P + s) * D +
                                  (u % pieces) * 16) = rescale16(v[k], s_ratio[s]);
    }
    if (grew && tid == 0) scales[(int64_t)page * heads + h] = s_new;
  }
}

// ---------------------------------------------------------------------------
// evict
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 1024, kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kHeldKeys = 24 * 1024;           // keys that stay in shared memory

// Unsigned order of weights: NaN 0, below every number; -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (w != w) return 0;
  const uint32_t u = w == 0.0f ? 0u : __float_as_uint(w);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// What the budget leaves of a sequence.
struct Share {
  int len, keep, first, recent;
  bool alone;                                  // not to be touched
};
__device__ __forceinline__ Share share_of(const EvictArgs& a, int b) {
  Share s;
  const int64_t cap = (int64_t)a.b.max_pages * a.c.page_size;
  s.len = (int)min((int64_t)max(a.b.seq_lens[b], 0), cap);
  const int budget = a.budgets ? a.budgets[b] : a.width;
  s.alone = budget < 0;
  s.keep = min(s.len, min(max(budget, 0), a.width));
  s.recent = min(a.recent, s.keep);
  s.first = min(a.first, s.keep - s.recent);
  return s;
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const __grid_constant__ EvictArgs a) {
  extern __shared__ uint32_t s_keys[];
  __shared__ int s_hist[kBins];
  __shared__ int s_warp[kSelWarps], s_warp2[kSelWarps];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x % a.c.kv_heads, b = blockIdx.x / a.c.kv_heads;
  const int P = a.c.page_size, log_p = 31 - __clz(P), heads = a.c.kv_heads;
  const Share sh = share_of(a, b);
  if (h == 0 && tid == 0) {
    a.new_lens[b] = sh.alone ? a.b.seq_lens[b] : sh.keep;
    if (!sh.alone && a.b.seq_lens[b] > sh.len) atomicOr(a.err, (uint32_t)MOE_DEVERR_PAGE);
  }
  int32_t* kept = a.kept + ((int64_t)b * heads + h) * a.width;
  const int shown = sh.alone ? 0 : sh.keep;
  for (int i = shown + tid; i < a.width; i += kSelThreads) kept[i] = -1;
  if (shown == 0) return;
  if (sh.keep == sh.len) {
    for (int i = tid; i < sh.keep; i += kSelThreads) kept[i] = i;
    return;
  }
  for (int i = tid; i < sh.first; i += kSelThreads) kept[i] = i;
  for (int i = tid; i < sh.recent; i += kSelThreads) kept[sh.keep - 1 - i] = sh.len - 1 - i;
  const int choose = sh.keep - sh.recent - sh.first;
  if (choose == 0) return;
  const int lo = sh.first, N = sh.len - sh.recent - lo;     // candidates, more than `choose`
  const int32_t* table = a.b.page_table + (int64_t)b * a.b.table_stride;
  auto load_key = [&](int i) {
    const int j = lo + i, page = table[j >> log_p];
    if (page < 0 || page >= a.c.num_pages) {
      atomicOr(a.err, (uint32_t)MOE_DEVERR_PAGE);
      return 0u;
    }
    return weight_key(a.w[((int64_t)page * heads + h) * P + (j & (P - 1))]);
  };
  const int held = min(N, kHeldKeys);
  for (int i = tid; i < held; i += kSelThreads) s_keys[i] = load_key(i);
  auto key = [&](int i) { return i < held ? s_keys[i] : load_key(i); };

  // the threshold: the key of rank `choose`, bits from the top
  uint32_t prefix = 0;
  int need = choose, shift = 32;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass < 2 ? 11 : 10;
    shift -= bits;
    for (int i = tid; i < kBins; i += kSelThreads) s_hist[i] = 0;
    __syncthreads();                           // (and, the first time, the keys)
    for (int i0 = 0; i0 < N; i0 += kSelThreads) {
      const int i = i0 + tid;
      const uint32_t k = i < N ? key(i) : 0;
      const bool mine = i < N && (pass == 0 || (k >> (shift + bits)) == prefix);
      const uint32_t bin = mine ? (k >> shift) & ((1u << bits) - 1) : 0xffffffffu;
      // one addition per distinct bin of the warp: weights crowd into few bins
      const uint32_t same = __match_any_sync(0xffffffffu, bin);
      if (mine && lane == __ffs(same) - 1) atomicAdd(&s_hist[bin], __popc(same));
    }
    __syncthreads();
    // bins from the top, two per thread: the bin in which the count passes `need`
    const int top = kBins - 1 - 2 * tid;
    const int c0 = s_hist[top], c1 = s_hist[top - 1];
    int upto = c0 + c1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += up;
    }
    if (lane == 31) s_warp[warp] = upto;
    __syncthreads();
    int base = 0;
    for (int w = 0; w < warp; ++w) base += s_warp[w];
    const int before = base + upto - c0 - c1;
    if (before < need && need <= before + c0) s_prefix = top, s_need = need - before;
    else if (before + c0 < need && need <= before + c0 + c1) s_prefix = top - 1, s_need = need - before - c0;
    __syncthreads();
    prefix = prefix << bits | s_prefix;
    need = s_need;
  }
  // kept: keys above the threshold, and the first `need` of those equal to it. A warp takes a run
  // of places; counts first, then places.
  const int run = (N + kSelWarps * 32 - 1) / (kSelWarps * 32) * 32;
  const int r0 = min(warp * run, N), r1 = min(r0 + run, N);
  int above = 0, equal = 0;
  for (int i0 = r0; i0 < r1; i0 += 32) {
    const uint32_t k = i0 + lane < r1 ? key(i0 + lane) : 0;
    const bool in = i0 + lane < r1;
    above += __popc(__ballot_sync(0xffffffffu, in && k > prefix));
    equal += __popc(__ballot_sync(0xffffffffu, in && k == prefix));
  }
  if (lane == 0) s_warp[warp] = above, s_warp2[warp] = equal;
  __syncthreads();
  int at = 0, eq = 0;                          // kept, equal before this warp's run
  for (int w = 0; w < warp; ++w) {
    const int take = min(max(need - eq, 0), s_warp2[w]);
    at += s_warp[w] + take;
    eq += s_warp2[w];
  }
  const uint32_t below = (1u << lane) - 1;
  for (int i0 = r0; i0 < r1; i0 += 32) {
    const bool in = i0 + lane < r1;
    const uint32_t k = in ? key(i0 + lane) : 0;
    const uint32_t e = __ballot_sync(0xffffffffu, in && k == prefix);
    const bool take = in && (k > prefix || (k == prefix && eq + __popc(e & below) < need));
    const uint32_t t = __ballot_sync(0xffffffffu, take);
    if (take) kept[sh.first + at + __popc(t & below)] = lo + i0 + lane;
    at += __popc(t);
    eq += __popc(e);
  }
}

// One page of the copy, both planes.
__global__ void __launch_bounds__(kMoveThreads) copy_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ int s_page[128], s_slot[128];     // where a slot's token comes from (-1: nowhere)
  __shared__ float s_ratio[2][128];
  const int tid = threadIdx.x;
  const int P = a.c.page_size, log_p = 31 - __clz(P), D = a.c.head_dim, heads = a.c.kv_heads;
  const int pages = (a.width + P - 1) / P, pi = blockIdx.x % pages;
  const int h = blockIdx.x / pages % heads, b = blockIdx.x / pages / heads;
  const Share sh = share_of(a, b);
  const int p0 = pi * P;
  pdl_wait();
  if (sh.alone || p0 >= sh.keep) return;
  const int count = min(P, sh.keep - p0);
  const int page = a.dst_table[(int64_t)b * a.dst_stride + pi];
  if (page < 0 || page >= a.c.num_pages) {
    if (tid == 0) atomicOr(a.err, (uint32_t)MOE_DEVERR_PAGE);
    return;
  }
  const int32_t* table = a.b.page_table + (int64_t)b * a.b.table_stride;
  if (tid < 128) {
    int from = -1, slot = 0;
    float sk = 0.0f, sv = 0.0f;
    if (tid < count) {
      const int src = a.kept[((int64_t)b * heads + h) * a.width + p0 + tid];
      from = table[src >> log_p];
      slot = src & (P - 1);
      if (from < 0 || from >= a.c.num_pages) {
        atomicOr(a.err, (uint32_t)MOE_DEVERR_PAGE);
        from = -1;
      } else {
        sk = a.c.k_scales[(int64_t)from * heads + h];
        sv = a.c.v_scales[(int64_t)from * heads + h];
        a.w[((int64_t)page * heads + h) * P + tid] = a.w[((int64_t)from * heads + h) * P + slot];
      }
    }
    s_page[tid] = from, s_slot[tid] = slot;
    s_ratio[0][tid] = sk, s_ratio[1][tid] = sv;
  }
  __syncthreads();
  if (tid < 64) {                              // a warp per plane
    const int plane = tid >> 5, lane = tid & 31;
    float top = 0.0f;
    for (int s = lane; s < count; s += 32) top = fmaxf(top, s_ratio[plane][s]);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    for (int s = lane; s < count; s += 32) {
      const float was = s_ratio[plane][s];
      s_ratio[plane][s] = was == top ? 1.0f : was / top;
    }
    if (lane == 0 && top > 0.0f) (plane ? a.c.v_scales : a.c.k_scales)[(int64_t)page * heads + h] = top;
  }
  __syncthreads();
  const int pieces = D / 16, all = count * pieces;
  for (int plane = 0; plane < 2; ++plane) {
    uint8_t* codes = plane ? a.c.v_codes : a.c.k_codes;
    for (int u = tid; u < all; u += kMoveThreads) {
      const int s = u / pieces;
      if (s_page[s] < 0) continue;
      const uint4 v = *reinterpret_cast<const uint4*>(codes + (int64_t)s_page[s] * a.c.page_stride +
                                                      ((int64_t)h * P + s_slot[s]) * D + (u % pieces) * 16);
      *reinterpret_cast<uint4*>(codes + (int64_t)page * a.c.page_stride + ((int64_t)h * P + s) * D +
                                (u % pieces) * 16) = rescale16(v, s_ratio[plane][s]);
    }
  }
}

}  // namespace

cudaError_t launch_keep(const KeepArgs& a, cudaStream_t s) {
  keep_kernel<<<(unsigned)(2 * a.b.B * a.c.kv_heads), kMoveThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  constexpr int smem = kHeldKeys * 4;
  cudaError_t e = cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const unsigned heads = (unsigned)(a.b.B * a.c.kv_heads);
  select_kernel<<<heads, kSelThreads, smem, s>>>(a);
  if ((e = cudaGetLastError()) != cudaSuccess || a.width == 0) return e;
  const unsigned pages = (unsigned)((a.width + a.c.page_size - 1) / a.c.page_size);
  return launch_pdl(copy_kernel, dim3(pages * heads), dim3(kMoveThreads), 0, s, a);
}

}  // namespace moe
