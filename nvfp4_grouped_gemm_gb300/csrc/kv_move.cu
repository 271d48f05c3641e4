// Tokens that change their place in the paged 8-bit cache: a tree's accepted path (moe_kv_keep_e4m3)
// and the tokens that a budget keeps (moe_kv_evict_e4m3).
//
// A page has one scale per head, so a page into which tokens move takes the largest of their old pages'
// scales and its codes become RN(code * old / new); where old = new the bits are copied.
//
// keep: a CTA per (sequence, key head) walks the pages that change in order. Places ascend, so
// a page's tokens come from itself or later pages; a page is read whole before it is written, and no
// later page needs what an earlier one overwrote. Bound by one chain of dependent loads (lengths, list,
// table, scales, codes): one path of a tree 4.1 us, 64 paths of up to 63 tokens over pages of 16 5.2 us;
// one plane after the other, piece by piece, the latter took 14.3.
//
// evict: select_kernel finds, per (sequence, key head), the weights' threshold by a radix descent over
// order-preserving keys (11, 11 and 10 bits; histograms in shared memory, which a cluster of up to 8 CTAs
// adds up over distributed shared memory), then lists the kept places by ballots in order: ties at the
// threshold go to the lower places. copy_kernel has a CTA per 256 places of the copy; all reads are from
// pages that nobody writes, so pages are independent of one another. 32 sequences of 2500 to 16000 cut to
// 4096, 8 key heads of 128: 93.0 us, of which select takes about 29 (instructions) and the copy
// 64 (6.3 TB/s, 0.92 of the copy rate); with one CTA per threshold and one per page of the copy 157.6. One
// sequence of 1090 cut to 1024: 12.9 us, two kernels of dependent steps. The copy starts its loads when select has
// ended: let go at select's start, its CTAs take the places of select's (117 where both took 95.5).
#include "serving.cuh"

namespace moe {
namespace {

constexpr int kMoveThreads = 256;

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
// PIECES: a thread's 16-byte pieces of both planes of a page.
template <int PIECES>
__global__ void __launch_bounds__(kMoveThreads) keep_kernel(const __grid_constant__ KeepArgs a) {
  __shared__ int s_first_bad, s_first_move;
  __shared__ int s_from[128];                  // a slot's source page (-1: stays as it is)
  __shared__ int s_slot[128];
  __shared__ float s_ratio[2][128];
  __shared__ float s_new[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int h = blockIdx.x % a.c.kv_heads, b = blockIdx.x / a.c.kv_heads;
  const int P = a.c.page_size, log_p = 31 - __clz(P), D = a.c.head_dim, heads = a.c.kv_heads;
  const int n = max(a.b.q_offsets[b + 1] - a.b.q_offsets[b], 0), len = a.b.seq_lens[b];
  const int start = len - n, asked = min(max(a.n_keep[b], 0), a.width);
  if (len < n || len > (int64_t)a.b.max_pages * P) {         // (not by start, which may wrap)
    if (h == 0 && tid == 0) {
      atomicOr(a.err, (uint32_t)MOE_DEVERR_PAGE);
      a.new_lens[b] = len;
    }
    return;
  }
  const int32_t* list = a.keep + (int64_t)b * a.width;
  if (tid == 0) s_first_bad = asked, s_first_move = asked;
  __syncthreads();
  for (int i = tid; i < asked; i += kMoveThreads) {
    const int v = list[i], before = i > 0 ? list[i - 1] : -1;
    if (v <= before || v >= n) atomicMin(&s_first_bad, i);
    if (v != i) atomicMin(&s_first_move, i);
  }
  __syncthreads();
  const int count = s_first_bad, move0 = min(s_first_move, count);
  if (h == 0 && tid == 0) {
    if (count < asked) atomicOr(a.err, (uint32_t)MOE_DEVERR_TOKEN);
    a.new_lens[b] = start + count;
  }
  if (move0 == count) return;
  const int32_t* table = a.b.page_table + (int64_t)b * a.b.table_stride;
  const int log_d = 31 - __clz(D / 16), plane_pieces = P << log_d;
  auto known = [&](int page) { return page >= 0 && page < a.c.num_pages; };
  for (int pi = (start + move0) >> log_p; pi * P < start + count; ++pi) {
    const int page = table[pi];
    const bool good = known(page);
    __syncthreads();                           // the page before is done with the shared arrays
    if (warp < 2) {                            // a warp per plane, a lane per slot; the largest scale over all
      const float* scales = warp ? a.c.v_scales : a.c.k_scales;
      const float own = good ? scales[(int64_t)page * heads + h] : 0.0f;
      float top = own;
      for (int s = lane; s < P; s += 32) {
        const int i = pi * P + s - start;      // the kept token that lands here
        int from = -1, slot = 0;
        float scale = own;
        if (i >= move0 && i < count && list[i] != i) {
          const int src = start + list[i], p = table[src >> log_p];
          if (good && known(p)) {
            from = p, slot = src & (P - 1);
            scale = scales[(int64_t)p * heads + h];
          } else {
            atomicOr(a.err, (uint32_t)MOE_DEVERR_PAGE);
          }
        }
        if (warp == 0) s_from[s] = from, s_slot[s] = slot;
        s_ratio[warp][s] = scale;
        top = fmaxf(top, scale);
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      for (int s = lane; s < P; s += 32) s_ratio[warp][s] = s_ratio[warp][s] == top ? 1.0f : s_ratio[warp][s] / top;
      if (lane == 0) s_new[warp] = top > own ? top : 0.0f;       // 0: the scale stays
    }
    __syncthreads();
    if (!good) continue;
    uint4 v[PIECES];
    auto place = [&](int k, int& s, int& plane) {          // of the thread's piece k; whether it is written
      const int u = tid + k * kMoveThreads;
      plane = u >= plane_pieces;
      s = (u - plane * plane_pieces) >> log_d;
      return u < 2 * plane_pieces && (s_from[s] >= 0 || s_new[plane] > 0.0f);
    };
    const int in = (tid & (D / 16 - 1)) * 16;  // (the threads of a block are whole rows)
#pragma unroll
    for (int k = 0; k < PIECES; ++k) {
      int s, plane;
      v[k] = make_uint4(0, 0, 0, 0);
      if (!place(k, s, plane)) continue;
      const int p = s_from[s] >= 0 ? s_from[s] : page, sl = s_from[s] >= 0 ? s_slot[s] : s;
      v[k] = *reinterpret_cast<const uint4*>((plane ? a.c.v_codes : a.c.k_codes) + (int64_t)p * a.c.page_stride +
                                             ((int64_t)h * P + sl) * D + in);
    }
    __syncthreads();                           // the page is read whole before it is written
#pragma unroll
    for (int k = 0; k < PIECES; ++k) {
      int s, plane;
      if (place(k, s, plane))
        *reinterpret_cast<uint4*>((plane ? a.c.v_codes : a.c.k_codes) + (int64_t)page * a.c.page_stride +
                                  ((int64_t)h * P + s) * D + in) = rescale16(v[k], s_ratio[plane][s]);
    }
    if (tid < 2 && s_new[tid] > 0.0f) (tid ? a.c.v_scales : a.c.k_scales)[(int64_t)page * heads + h] = s_new[tid];
  }
}

// ---------------------------------------------------------------------------
// evict
// ---------------------------------------------------------------------------
constexpr int kSelThreads = 512, kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048, kMine = kBins / kSelThreads;
constexpr int kHeldKeys = 9 * 1024;            // keys that a CTA keeps in shared memory
constexpr int kMostCluster = 8;

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

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The word of shared memory at the same place in the cluster's CTA `rank`.
__device__ __forceinline__ int of_rank(const int* p, int rank) {
  uint32_t at = (uint32_t)__cvta_generic_to_shared(p);
  int v;
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.s32 %0, [a];\n\t}"
               : "=r"(v) : "r"(at), "r"(rank) : "memory");
  return v;
}

__device__ __forceinline__ int4 four_of_rank(const int* p, int rank) {
  uint32_t at = (uint32_t)__cvta_generic_to_shared(p);
  int4 v;
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %4, %5;\n\tld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [a];\n\t}"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at), "r"(rank) : "memory");
  return v;
}

// A cluster of `size` CTAs per (sequence, key head), each with a run of the candidates.
__global__ void __launch_bounds__(kSelThreads, 4) select_kernel(const __grid_constant__ EvictArgs a, int size) {
  extern __shared__ __align__(16) uint32_t s_keys[];
  __shared__ __align__(16) int s_hist[2][kBins];             // in turn, so that others may still read the one before
  __shared__ int s_warp[kSelWarps], s_warp2[kSelWarps], s_all[2];
  __shared__ uint32_t s_prefix;
  __shared__ int s_need;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = blockIdx.x % size;
  const int h = blockIdx.x / size % a.c.kv_heads, b = blockIdx.x / size / a.c.kv_heads;
  const int P = a.c.page_size, log_p = 31 - __clz(P), heads = a.c.kv_heads;
  const int t0 = rank * kSelThreads + tid, step = size * kSelThreads;
  const Share sh = share_of(a, b);
  if (h == 0 && t0 == 0) {
    a.new_lens[b] = sh.alone ? a.b.seq_lens[b] : sh.keep;
    if (!sh.alone && a.b.seq_lens[b] > sh.len) atomicOr(a.err, (uint32_t)MOE_DEVERR_PAGE);
  }
  int32_t* kept = a.kept + ((int64_t)b * heads + h) * a.width;
  const int shown = sh.alone ? 0 : sh.keep;
  for (int i = shown + t0; i < a.width; i += step) kept[i] = -1;
  if (shown == 0) return;
  if (sh.keep == sh.len) {
    for (int i = t0; i < sh.keep; i += step) kept[i] = i;
    return;
  }
  for (int i = t0; i < sh.first; i += step) kept[i] = i;
  for (int i = t0; i < sh.recent; i += step) kept[sh.keep - 1 - i] = sh.len - 1 - i;
  const int choose = sh.keep - sh.recent - sh.first;
  if (choose == 0) return;
  const int all = sh.len - sh.recent - sh.first;           // candidates, more than `choose`
  const int share = (all + size * 32 - 1) / (size * 32) * 32;
  const int before_me = min(rank * share, all), lo = sh.first + before_me, N = min(share, all - before_me);
  const int32_t* table = a.b.page_table + (int64_t)b * a.b.table_stride;
  auto known = [&](int page) { return page >= 0 && page < a.c.num_pages; };
  // keys of candidates i .. of this thread, their pages and then their weights on their way together
  constexpr int kBatch = 8;
  bool bad = false;
  auto load_keys = [&](int i, uint32_t (&k)[kBatch]) {
    int page[kBatch];
#pragma unroll
    for (int x = 0; x < kBatch; ++x)
      page[x] = (int)load_ahead(table + ((lo + i + x * kSelThreads) >> log_p), i + x * kSelThreads < N, 0u);
#pragma unroll
    for (int x = 0; x < kBatch; ++x) {
      const int j = lo + i + x * kSelThreads;
      bad |= !known(page[x]);
      k[x] = load_ahead(a.w + (int64_t)page[x] * (heads * P) + (h * P + (j & (P - 1))),
                        i + x * kSelThreads < N && known(page[x]), 0x7fc00000u);
    }
#pragma unroll
    for (int x = 0; x < kBatch; ++x) k[x] = weight_key(__uint_as_float(k[x]));
  };
  const int held = min(N, kHeldKeys);          // the others are read again in every pass
  for (int i = tid; i < held; i += kSelThreads * kBatch) {
    uint32_t k[kBatch];
    load_keys(i, k);
#pragma unroll
    for (int x = 0; x < kBatch; ++x)
      if (i + x * kSelThreads < held) s_keys[i + x * kSelThreads] = k[x];
  }
  for (int i = tid; i < kBins; i += kSelThreads) s_hist[0][i] = 0;
  __syncthreads();
  auto each_key = [&](auto&& take) {           // take(key, there) by whole warps
    for (int i0 = 0; i0 < held; i0 += 4 * kSelThreads) {
      const int i = i0 + 4 * tid;
      const uint4 k = i < held ? *reinterpret_cast<const uint4*>(s_keys + i) : make_uint4(0, 0, 0, 0);
      take(k.x, i < held);
      take(k.y, i + 1 < held);
      take(k.z, i + 2 < held);
      take(k.w, i + 3 < held);
    }
    for (int i0 = held / (kSelThreads * kBatch) * (kSelThreads * kBatch); held < N && i0 < N; i0 += kSelThreads * kBatch) {
      uint32_t k[kBatch];
      load_keys(i0 + tid, k);
#pragma unroll
      for (int x = 0; x < kBatch; ++x) {
        const int i = i0 + tid + x * kSelThreads;
        take(k[x], i >= held && i < N);
      }
    }
  };

  // the threshold: the key of rank `choose`, bits from the top
  uint32_t prefix = 0;
  int need = choose, shift = 32;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int bits = pass < 2 ? 11 : 10;
    int* hist = s_hist[pass & 1];
    shift -= bits;
    each_key([&](uint32_t k, bool there) {
      const bool mine = there && (pass == 0 || (k >> (shift + bits)) == prefix);
      const uint32_t bin = (k >> shift) & ((1u << bits) - 1);
      // weights that are all alike (0) would otherwise meet at one address
      const uint32_t led = __shfl_sync(0xffffffffu, bin, 0);
      if (__all_sync(0xffffffffu, mine && bin == led)) {
        if (lane == 0) atomicAdd(&hist[bin], 32);
      } else if (mine) {
        atomicAdd(&hist[bin], 1);
      }
    });
    if (size > 1) cluster_sync();
    else __syncthreads();
    // (from here on nobody reads the other histogram any more)
    if (pass < 2)
      for (int i = tid; i < kBins; i += kSelThreads) s_hist[~pass & 1][i] = 0;
    // bins from the top, kMine per thread: the bin in which the count passes `need`
    const int top = kBins - 1 - kMine * tid;
    static_assert(kMine == 4, "");
    int c[kMine] = {};
    for (int r = 0; r < size; ++r) {
      const int4 v = size > 1 ? four_of_rank(&hist[top - 3], r) : *reinterpret_cast<const int4*>(&hist[top - 3]);
      c[0] += v.w, c[1] += v.z, c[2] += v.y, c[3] += v.x;
    }
    int mine = 0;
#pragma unroll
    for (int x = 0; x < kMine; ++x) mine += c[x];
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += up;
    }
    if (lane == 31) s_warp[warp] = upto;
    __syncthreads();
    int before = upto - mine;
    for (int w = 0; w < warp; ++w) before += s_warp[w];
#pragma unroll
    for (int x = 0; x < kMine; ++x) {
      if (before < need && need <= before + c[x]) s_prefix = top - x, s_need = need - before;
      before += c[x];
    }
    __syncthreads();
    prefix = prefix << bits | s_prefix;
    need = s_need;
  }
  // kept: keys above the threshold, and the first `need` of those equal to it. A warp takes a run
  // of places; counts first, then places.
  const int run = (N + kSelWarps * 32 - 1) / (kSelWarps * 32) * 32;
  const int r0 = min(warp * run, N), r1 = min(r0 + run, N);
  auto key = [&](int i) {
    if (i < held) return s_keys[i];
    const int j = lo + i, page = table[j >> log_p];
    return known(page) ? weight_key(a.w[((int64_t)page * heads + h) * P + (j & (P - 1))]) : 0u;
  };
  int above = 0, equal = 0;
  for (int i = r0 + lane; i < r1; i += 32) {
    const uint32_t k = key(i);
    above += k > prefix, equal += k == prefix;
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) s_warp[warp] = above, s_warp2[warp] = equal;
  __syncthreads();
  int at = 0, eq = 0;                          // kept, equal before this warp's run
  if (size > 1) {
    if (tid == 0) {
      int x = 0, y = 0;
      for (int w = 0; w < kSelWarps; ++w) x += s_warp[w], y += s_warp2[w];
      s_all[0] = x, s_all[1] = y;
    }
    cluster_sync();
    for (int r = 0; r < rank; ++r) {
      const int x = of_rank(&s_all[0], r), y = of_rank(&s_all[1], r);
      at += x + min(max(need - eq, 0), y);
      eq += y;
    }
  }
  for (int w = 0; w < warp; ++w) {
    at += s_warp[w] + min(max(need - eq, 0), s_warp2[w]);
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
  if (bad) atomicOr(a.err, (uint32_t)MOE_DEVERR_PAGE);
  if (size > 1) cluster_sync();                // nobody reads this CTA's shared memory any more
}

// kMoveThreads places of the copy (whole pages, of one key head), both planes: thread = place until the
// pages' scales are known, then the places' 16-byte pieces in turn, kInFlight of a thread on their way
// together and asked for before the scales are.
__global__ void __launch_bounds__(kMoveThreads) copy_kernel(const __grid_constant__ EvictArgs a) {
  constexpr int kMostPages = kMoveThreads / 16, kInFlight = 8;
  __shared__ int64_t s_from[kMoveThreads], s_to[kMoveThreads];   // bytes into a plane (-1: nowhere)
  __shared__ float s_ratio[2][kMoveThreads];
  __shared__ uint32_t s_top[2][kMostPages], s_any[kMostPages];    // a page's largest scales; whether a token comes to it
  const int tid = threadIdx.x;
  const int P = a.c.page_size, log_p = 31 - __clz(P), D = a.c.head_dim, heads = a.c.kv_heads;
  const int blocks = (a.width + kMoveThreads - 1) / kMoveThreads;
  const int h = blockIdx.x / blocks % heads, b = blockIdx.x / blocks / heads;
  const Share sh = share_of(a, b);
  const int i0 = blockIdx.x % blocks * kMoveThreads, i = i0 + tid;
  const int page = i < sh.keep ? a.dst_table[(int64_t)b * a.dst_stride + (i >> log_p)] : -1;
  if (tid < kMostPages) s_top[0][tid] = s_top[1][tid] = s_any[tid] = 0;
  pdl_wait();
  if (sh.alone || i0 >= sh.keep) return;
  const int count = min(kMoveThreads, sh.keep - i0);
  int from = -1, slot = 0;
  bool good = false;
  if (tid < count) {
    const int src = a.kept[((int64_t)b * heads + h) * a.width + i];
    from = a.b.page_table[(int64_t)b * a.b.table_stride + (src >> log_p)];
    slot = src & (P - 1);
    good = from >= 0 && from < a.c.num_pages && page >= 0 && page < a.c.num_pages;
    if (!good) atomicOr(a.err, (uint32_t)MOE_DEVERR_PAGE);
  }
  s_from[tid] = good ? (int64_t)from * a.c.page_stride + ((int64_t)h * P + slot) * D : -1;
  s_to[tid] = (int64_t)page * a.c.page_stride + ((int64_t)h * P + (i & (P - 1))) * D;
  const float sk = __uint_as_float(load_ahead(a.c.k_scales + (int64_t)from * heads + h, good, 0u));
  const float sv = __uint_as_float(load_ahead(a.c.v_scales + (int64_t)from * heads + h, good, 0u));
  const float w = __uint_as_float(load_ahead(a.w + ((int64_t)from * heads + h) * P + slot, good, 0u));
  __syncthreads();
  const int log_d = 31 - __clz(D / 16), all = count << log_d;
  uint4 v[kInFlight];
  auto ask = [&](const uint8_t* codes, int u0) {
#pragma unroll
    for (int k = 0; k < kInFlight; ++k) {
      const int u = u0 + k * kMoveThreads;
      const int64_t at = u < all ? s_from[u >> log_d] : -1;
      v[k] = load_ahead(codes + at + (u & (D / 16 - 1)) * 16, at >= 0);
    }
  };
  ask(a.c.k_codes, tid);
  // a page's scale: the largest of its tokens' (their bits order as they do)
  if (good) {
    atomicMax(&s_top[0][tid >> log_p], __float_as_uint(sk));
    atomicMax(&s_top[1][tid >> log_p], __float_as_uint(sv));
    s_any[tid >> log_p] = 1;
    a.w[((int64_t)page * heads + h) * P + (i & (P - 1))] = w;
  }
  __syncthreads();
  const float tk = __uint_as_float(s_top[0][tid >> log_p]), tv = __uint_as_float(s_top[1][tid >> log_p]);
  s_ratio[0][tid] = sk == tk ? 1.0f : sk / tk;
  s_ratio[1][tid] = sv == tv ? 1.0f : sv / tv;
  if (tid < count && (tid & (P - 1)) == 0 && s_any[tid >> log_p]) {      // (then the page is one of the cache's)
    a.c.k_scales[(int64_t)page * heads + h] = tk;
    a.c.v_scales[(int64_t)page * heads + h] = tv;
  }
  __syncthreads();
#pragma unroll 1
  for (int plane = 0; plane < 2; ++plane) {
    uint8_t* codes = plane ? a.c.v_codes : a.c.k_codes;
#pragma unroll 1
    for (int u0 = tid; u0 < all; u0 += kInFlight * kMoveThreads) {
      if (plane || u0 != tid) ask(codes, u0);
#pragma unroll
      for (int k = 0; k < kInFlight; ++k) {
        const int u = u0 + k * kMoveThreads, s = u >> log_d;
        if (u < all && s_from[s] >= 0)
          *reinterpret_cast<uint4*>(codes + s_to[s] + (u & (D / 16 - 1)) * 16) = rescale16(v[k], s_ratio[plane][s]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_keep(const KeepArgs& a, cudaStream_t s) {
  const unsigned grid = (unsigned)(a.b.B * a.c.kv_heads);
  const int pieces = a.c.page_size * (a.c.head_dim / 16) * 2 / kMoveThreads;     // 0 (half of them idle) to 16
  if (pieces <= 1) keep_kernel<1><<<grid, kMoveThreads, 0, s>>>(a);
  else if (pieces == 2) keep_kernel<2><<<grid, kMoveThreads, 0, s>>>(a);
  else if (pieces == 4) keep_kernel<4><<<grid, kMoveThreads, 0, s>>>(a);
  else if (pieces == 8) keep_kernel<8><<<grid, kMoveThreads, 0, s>>>(a);
  else keep_kernel<16><<<grid, kMoveThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t s) {
  constexpr int smem = kHeldKeys * 4;
  cudaError_t e = cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const unsigned heads = (unsigned)(a.b.B * a.c.kv_heads);
  // CTAs per (sequence, key head): while there is room for them (four per SM) and 2048 places for each,
  // as far as the page table's width tells. 4 key heads, one CTA against this rule: a sequence of 16000
  // 51.6 and 22.0 us, of 60000 176 and 31.8; 16 of 4000 to 12000 55.8 and 40.0, with 1024 for each (8
  // CTAs) 65.0.
  const long long places = (long long)a.b.max_pages * a.c.page_size;
  int size = 1;
  while (size < kMostCluster && 2LL * size * heads <= 4LL * num_sms() && places >= 4096LL * size) size *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(heads * size);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&cfg, select_kernel, a, size)) != cudaSuccess) return e;
  if ((e = cudaGetLastError()) != cudaSuccess || a.width == 0) return e;
  const unsigned blocks = (unsigned)((a.width + kMoveThreads - 1) / kMoveThreads);
  return launch_pdl(copy_kernel, dim3(blocks * heads), dim3(kMoveThreads), 0, s, a);
}

}  // namespace moe
