// Attention for trees of drafted tokens over the paged 8-bit cache (moe_attention_tree_e4m3), head_dim 64
// and 128, for sequences of up to about a hundred rows; paged_attention.cu has the definitions and the
// form for head_dim 256, prompt_attention.cu the one for more rows.
//
// A sequence's n new tokens and the G query heads that share a key head are n*G rows over the same keys
// and values; a segment is (sequence, key head, block of R such rows), its keys come in tiles of 128.
// All segments' tiles form one line that the grid (a CTA per SM) cuts into equal pieces; a cut
// segment's partial rows are joined in order by the last CTA to arrive.
//
// Rows are few, so keys are the side that fills the tensor cores, thread = key:
//   S^T = K Q^T      128 keys x R rows: codes widened to f16 (exact) in tensor memory, Q from shared memory
//   P^T              weights 2^(s f + v - M) as f16 in shared memory, a key's rows beside one another
//   O^T += V^T P^T   head_dim x R rows: V widened to f16 in shared memory as its rows lie, i.e. with the
//                    M dimension contiguous
// f, v, M, the lazily moved maximum and the sums by 1 / v_scale are paged_attention.cu's; here a row's
// maximum is looked for across threads only when a weight would pass 2^8 (a vote per tile), and its sum
// stays spread over the keys' threads until the piece ends.
//
// Two groups of four warps take a piece's tiles in turn, each with its own S, P, V, O, maxima and sums, so
// that one's products and copies hide behind the other's arithmetic; they meet at the piece's end. One
// more warp brings codes, pages and scales (TMA, a box per page).
#include "tc_f16.cuh"

namespace moe {
namespace {

constexpr int kTile = 128, kGroups = 2, kWorkers = 128 * kGroups, kThreads = kWorkers + 32;
constexpr float kNoMax = -1e30f;
constexpr float kLazy = 8.0f;
constexpr float kFar = 40.0f;                  // of value scales, as in paged_attention.cu
// What a segment costs beside its tiles (queries, first copies, the groups meeting, storing), in tiles.
constexpr int kSegmentCost = 3;
constexpr int kMostGrid = 160;

// Workspace (the few-row form's): error word; arrival counters; maxima and sums [2 * kMostGrid][2][64];
// partial rows f32 [2 * kMostGrid][64][D].
constexpr int kMostR = 64;
constexpr size_t kCountersAt = kAlign;
constexpr size_t kStatsAt = kCountersAt + 512 * 4;
constexpr size_t kRowsAt = kStatsAt + (size_t)2 * kMostGrid * 2 * kMostR * 4;

template <int D_, int R_>
struct Shape {
  static constexpr int D = D_, R = R_;
  static constexpr int kRowB = D == 64 ? 64 : 128;                     // bytes of a row of codes
  static constexpr int kCodeB = kTile * D;                             // a tile's codes of one plane
  static constexpr int kKSlots = 2;                                    // of a group; V has one
  static constexpr int kQHalf = R * 128, kQB = R * D * 2;
  static constexpr int kVHalf = kTile * 128, kVB = kTile * D * 2;      // a widened V
  static constexpr int kPB = kTile * 128;                              // weights, 128 bytes per key
  static constexpr int kKAt = 0, kVcAt = kKAt + kGroups * kKSlots * kCodeB, kVAt = kVcAt + kGroups * kCodeB;
  static constexpr int kPAt = kVAt + kGroups * kVB, kQAt = kPAt + kGroups * kPB, kBytes = kQAt + kQB;
  static constexpr int kSmem = 1024 + kBytes;
  // tensor memory columns of a group: keys, S, O
  static constexpr int kSAt = D / 2, kOAt = kSAt + R, kCols = kOAt + R;
  static constexpr int kAlloc = kGroups * kCols <= 256 ? 256 : 512;
  static_assert(kGroups * kCols <= 512 && kSmem <= 220 * 1024, "");
};

struct Seq {
  int row0, n, start, len;                     // token rows, new tokens, place of the first, visible length
  int t0, tiles, blocks;                       // first tile, tiles (at least 1), row blocks
};
template <int R>
__device__ __forceinline__ Seq read_seq(const AttentionArgs& a, int b, int group, uint32_t* err) {
  Seq q;
  q.row0 = min(max(a.b.q_offsets[b], 0), a.T);
  const int end = min(max(a.b.q_offsets[b + 1], q.row0), a.T);
  q.n = end - q.row0;
  if (q.n * group > a.max_rows) q.n = 0;       // the other form's
  q.len = a.b.seq_lens[b];
  q.start = q.len - q.n;
  const int cap = a.b.max_pages * a.c.page_size;
  if (q.n > 0 && (q.start < 0 || q.len > cap) && err) atomicOr(err, (uint32_t)MOE_DEVERR_PAGE);
  q.len = min(max(q.len, 0), cap);
  q.t0 = a.window > 0 ? max(0, min(q.start - a.window, q.len)) / kTile : 0;
  q.tiles = max((q.len + kTile - 1) / kTile - q.t0, 1);
  q.blocks = (q.n * group + R - 1) / R;
  return q;
}

// A CTA's share of a segment.
struct Piece {
  int b, h, block, rows;                       // sequence, key head, block of rows, rows in it
  int row0, n, start, len;                     // of the sequence
  int t0, t1;                                  // tiles of keys (those past the length have none)
  bool opens, closes;                          // holds the segment's first / last tile
  int c0, np;                                  // the CTAs the segment is spread over
};
struct Walk {
  long long pos, end, per, first;              // first: of the segment
  int b, seg;
  Seq q;
};
template <int R>
__device__ __forceinline__ bool next_piece(Walk& w, Piece& p, const AttentionArgs& a, int group) {
  while (w.pos < w.end) {
    const int length = w.q.tiles + kSegmentCost;
    if (w.q.blocks == 0 || w.pos >= w.first + length) {
      if (w.q.blocks > 0) w.first += length;
      if (++w.seg < w.q.blocks * a.c.kv_heads) continue;
      w.seg = 0;
      do w.q = read_seq<R>(a, ++w.b, group, nullptr);
      while (w.q.blocks == 0);                 // (the line goes on, so there is one more)
      continue;
    }
    const int from = (int)(w.pos - w.first), upto = (int)min((long long)length, w.end - w.first);
    const int s0 = max(0, from - kSegmentCost), s1 = upto - kSegmentCost;
    w.pos = w.first + upto;
    if (s1 <= s0) continue;                    // only the segment's fixed cost fell to this CTA
    p.b = w.b, p.h = w.seg / w.q.blocks, p.block = w.seg % w.q.blocks;
    p.rows = min(R, w.q.n * group - p.block * R);
    p.row0 = w.q.row0, p.n = w.q.n, p.start = w.q.start, p.len = w.q.len;
    p.t0 = w.q.t0 + s0;
    p.t1 = min(w.q.t0 + s1, (w.q.len + kTile - 1) / kTile);
    p.opens = s0 == 0, p.closes = s1 == w.q.tiles;
    p.c0 = (int)((w.first + kSegmentCost) / w.per);
    p.np = (int)((w.first + length - 1) / w.per) - p.c0 + 1;
    return true;
  }
  return false;
}

__device__ __forceinline__ float max_of_warp(float v) {    // (no NaN)
  const int i = __float_as_int(v);
  const int top = __reduce_max_sync(0xffffffffu, i >= 0 ? i : i ^ 0x7fffffff);
  return __int_as_float(top >= 0 ? top : top ^ 0x7fffffff);
}
__device__ __forceinline__ void sts128(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// f16 products with A's M dimension contiguous (bit 15) and B's N dimension contiguous (bit 16).
constexpr uint32_t transposed_idesc(int M, int N) { return f16_idesc(M, N, true) | (1u << 15); }

template <int D, int R>
__global__ void __launch_bounds__(kThreads, 1)
tree_kernel(const __grid_constant__ AttentionArgs a, const __grid_constant__ CUtensorMap kmap,
            const __grid_constant__ CUtensorMap vmap) {
  using S = Shape<D, R>;
  extern __shared__ char smem_raw[];
  __shared__ uint64_t s_kfull[kGroups * S::kKSlots], s_kempty[kGroups * S::kKSlots], s_vfull[kGroups], s_vempty[kGroups];
  __shared__ uint64_t s_afull[kGroups], s_sfull[kGroups], s_pfull[kGroups], s_ofull[kGroups], s_vote[kGroups], s_meet;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ long long s_sum[kThreads / 32], s_first;
  __shared__ int s_seq, s_last;
  __shared__ float4 s_page[kGroups * S::kKSlots][8];       // a page's f, v, 1 / v_scale (0: no page)
  __shared__ __align__(16) float s_rowf[R];
  __shared__ __align__(16) float s_max[kGroups][R];
  __shared__ float s_keep[kGroups][R], s_top[kGroups][4][R], s_l[kGroups][4][R];
  __shared__ volatile uint32_t s_flag[kGroups];            // the tile whose weights need a larger maximum
  __shared__ volatile int s_big[kGroups], s_nan[kGroups];  // scores beyond 1e6; NaN codes kept out of V
  __shared__ uint32_t s_bits[R * kMaxTreeWords];
  __shared__ int s_lo[R];
  char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int heads = a.c.kv_heads, group = a.q_heads / heads, P = a.c.page_size, log_p = 31 - __clz(P);
  uint32_t* err = reinterpret_cast<uint32_t*>(a.ws);
  uint32_t* counters = reinterpret_cast<uint32_t*>(a.ws + kCountersAt);
  float* stats = reinterpret_cast<float*>(a.ws + kStatsAt);
  float* part = reinterpret_cast<float*>(a.ws + kRowsAt);
  volatile int* abort_flag = &s_abort;
  const bool bf16 = a.dtype == MOE_DTYPE_BF16;

  // ---- this CTA's piece of the line ----
  auto scan = [&](long long v, long long* before) {
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
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) base += s_sum[w];
      all += s_sum[w];
    }
    *before = base + x - v;
    return all;
  };
  auto line_of = [&](int b, uint32_t* e) {
    if (b >= a.b.B) return 0ll;
    const Seq q = read_seq<R>(a, b, group, e);
    return (long long)(q.tiles + kSegmentCost) * q.blocks * heads;
  };
  long long total = 0, mine = 0, at = 0;
  for (int b0 = 0; b0 < a.b.B; b0 += kThreads) {
    mine = line_of(b0 + tid, blockIdx.x == 0 ? err : nullptr);
    total += scan(mine, &at);
  }
  long long per = (total + gridDim.x - 1) / gridDim.x;
  if (per < kSegmentCost + kGroups) per = kSegmentCost + kGroups;
  const long long begin = per * blockIdx.x, end = min(begin + per, total);
  if (begin >= end) {
    pdl_wait();
    return;
  }
  long long base = 0;
  for (int b0 = 0; b0 < a.b.B; b0 += kThreads) {
    long long sum = total;
    if (a.b.B > kThreads) {
      mine = line_of(b0 + tid, nullptr);
      sum = scan(mine, &at);
    }
    if (mine > 0 && base + at <= begin && begin < base + at + mine) s_seq = b0 + tid, s_first = base + at;
    base += sum;
  }
  if (tid == 0) {
    for (int i = 0; i < kGroups * S::kKSlots; ++i) mbar_init(&s_kfull[i], 1), mbar_init(&s_kempty[i], 4);
    for (int i = 0; i < kGroups; ++i) {
      mbar_init(&s_vfull[i], 1), mbar_init(&s_vempty[i], 4);
      mbar_init(&s_afull[i], 4), mbar_init(&s_sfull[i], 1);
      mbar_init(&s_pfull[i], 4), mbar_init(&s_ofull[i], 1);
      mbar_init(&s_vote[i], 4);
      s_flag[i] = 0;
    }
    mbar_init(&s_meet, 4 * kGroups);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async();
  }
  if (warp == 4 * kGroups) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_u32(&s_tmem)), "n"(S::kAlloc) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  Walk w;
  w.pos = begin, w.end = end, w.per = per, w.b = s_seq;
  w.q = read_seq<R>(a, w.b, group, nullptr);
  w.seg = (int)((begin - s_first) / (w.q.tiles + kSegmentCost));
  w.first = s_first + (long long)w.seg * (w.q.tiles + kSegmentCost);
  Piece p;
  bool ok = true;

  if (warp < 4 * kGroups) {
    const int gr = warp >> 2, key = tid & 127, gw = warp & 3;
    const uint32_t quarter = (uint32_t)(gw * 32) << 16, tmem = s_tmem + gr * S::kCols;
    const uint32_t s_col = tmem + S::kSAt, o_col = tmem + S::kOAt;
    const uint32_t code_swz = D == 64 ? (key >> 1) & 3 : key & 7, swz = key & 7;
    const uint64_t q_desc = smem_desc(smem_u32(smem + S::kQAt), 16, 1024, 2);
    // (D = 64: the upper half of O^T's 128 rows reads V's 64 values again and is not used)
    const uint64_t v_desc = smem_desc(smem_u32(smem + S::kVAt + gr * S::kVB), D == 64 ? 0 : S::kVHalf, 1024, 2);
    const uint64_t p_desc = smem_desc(smem_u32(smem + S::kPAt + gr * S::kPB), S::kPB, 1024, 2);
    const bool issues = gw == 0 && lane == 0;
    uint32_t k = 0, votes = 0, meets = 0;      // tiles of the group; phases
    bool far = false;                          // a value scale so far was outside [2^-kFar, 2^kFar]
    auto meet = [&] {                          // of all workers
      warp_arrive(&s_meet);
      return wait_warp(&s_meet, meets++ & 1, abort_flag, err);
    };
    auto meet_group = [&] {
      warp_arrive(&s_vote[gr]);
      return wait_warp(&s_vote[gr], votes++ & 1, abort_flag, err);
    };
    while (ok && next_piece<R>(w, p, a, group)) {
      // ---- the rows: f16 times a power of two, K-major, swizzled; what each sees ----
      const int cols = (p.rows + 15) / 16 * 16;
      constexpr int kLanes = D / 8, kPer = 32 / kLanes, kRounds = R / (8 * kPer);
      static_assert(kRounds >= 1 || R == 16, "");
      {
        const int col = lane % kLanes, sub = lane / kLanes;
        constexpr int kDo = kRounds < 1 ? 1 : kRounds;
        uint4 v[kDo];
#pragma unroll
        for (int i = 0; i < kDo; ++i) {
          const int r = (i * 8 + warp) * kPer + sub, rr = p.block * R + r;
          const int64_t token = p.row0 + (r < p.rows ? rr / group : 0);
          v[i] = load_ahead(a.q + token * a.q_stride + (int64_t)(p.h * group + rr % group) * D + col * 8, r < p.rows);
        }
        if (tid < R) {
          uint32_t bits[kMaxTreeWords];
          s_lo[tid] = tree_row(a, p.row0 + (p.block * R + tid) / group, tid < p.rows, p.n, p.start, bits);
#pragma unroll
          for (int i = 0; i < kMaxTreeWords; ++i) s_bits[tid * kMaxTreeWords + i] = bits[i];
        }
        if (tid < kGroups * R) s_max[tid / R][tid % R] = kNoMax;
        if (tid < kGroups) s_big[tid] = 0, s_nan[tid] = 0;
#pragma unroll
        for (int i = 0; i < kDo; ++i) {
          const int r = (i * 8 + warp) * kPer + sub;
          if (r >= R) break;                   // (R = 16 with four rows per warp)
          float rowf = 1.0f;
          if (bf16) {
            float f[8];
            unpack8<MOE_DTYPE_BF16>(v[i], f);
            float amax = 0.0f;
#pragma unroll
            for (int x = 0; x < 8; ++x) amax = fmaxf(amax, fabsf(f[x]));
#pragma unroll
            for (int o = kLanes / 2; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
            const int e = amax < 3.4e38f ? f16_prescale_exp(amax) : 0;
            const float s1 = pow2f(-e / 2), s2 = pow2f(-e - (-e / 2));
            rowf = pow2f(e);
#pragma unroll
            for (int x = 0; x < 8; ++x) f[x] = f[x] * s1 * s2;
            v[i] = make_uint4(pack_f16(f[0], f[1]), pack_f16(f[2], f[3]), pack_f16(f[4], f[5]), pack_f16(f[6], f[7]));
          }
          if (col == 0) s_rowf[r] = rowf;
          sts128(smem_u32(smem + S::kQAt + (col >> 3) * S::kQHalf + r * 128) + (((col & 7) ^ (r & 7)) * 16), v[i].x, v[i].y,
                 v[i].z, v[i].w);
        }
      }
      fence_async();
      if (!(ok = meet())) break;

      // ---- the group's tiles ----
      float L[R];
#pragma unroll
      for (int r = 0; r < R; ++r) L[r] = 0.0f;
      bool any = false;                        // the group has had a tile of this piece
      // tiles from `part` on and before `edge` have keys that some row does not see
      const int part_from = max(min(p.start, p.len), 0) / kTile;
      const int edge = a.window > 0 ? max(p.start + min(p.n, 32 * kMaxTreeWords) - a.window + kTile - 1, 0) / kTile : 0;
#pragma unroll 1
      for (int t = p.t0 + gr; t < p.t1; t += kGroups, ++k) {
        const int slot = gr * S::kKSlots + k % S::kKSlots, j = t * kTile + key;
        const bool partly = t >= part_from || t < edge || (t + 1) * kTile > p.len;
        if (!(ok = wait_warp(&s_kfull[slot], k / S::kKSlots & 1, abort_flag, err))) break;
        const float4 page = s_page[slot][key >> log_p];
        {
          const uint32_t row = smem_u32(smem + S::kKAt + slot * S::kCodeB) + (uint32_t)key * S::kRowB;
#pragma unroll
          for (int i = 0; i < D / 16; i += 2) {            // 32 codes at a time
            uint32_t v[16];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint4 c = lds128(row + (((i + x) ^ code_swz) * 16));
              widen4(c.x, v[8 * x], v[8 * x + 1]);
              widen4(c.y, v[8 * x + 2], v[8 * x + 3]);
              widen4(c.z, v[8 * x + 4], v[8 * x + 5]);
              widen4(c.w, v[8 * x + 6], v[8 * x + 7]);
            }
            tc_st16(tmem + quarter + i * 8, v);
          }
        }
        warp_arrive(&s_kempty[slot]);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&s_afull[gr]);
        if (issues && wait_thread(&s_afull[gr], k & 1, abort_flag, err)) {
          tc_fence_after();
          const uint32_t id = f16_idesc(128, cols, false);
#pragma unroll
          for (int i = 0; i < D / 16; ++i)
            mma_ts(s_col, tmem + i * 8, q_desc + (uint32_t)(((i >> 2) * S::kQHalf + (i & 3) * 32) >> 4), id, i != 0);
          tc_commit(&s_sfull[gr]);
        }
        __syncwarp();
        // V, beside those products; the products of the tile before have read what it is written over
        if (any && !(ok = wait_warp(&s_ofull[gr], (k - 1) & 1, abort_flag, err))) break;
        if (!(ok = wait_warp(&s_vfull[gr], k & 1, abort_flag, err))) break;
        const bool there = page.z != 0.0f && j < p.len;
        {
          const uint32_t row = smem_u32(smem + S::kVcAt + gr * S::kCodeB) + (uint32_t)key * S::kRowB;
          const uint32_t to = smem_u32(smem + S::kVAt + gr * S::kVB) + (uint32_t)key * 128;
          uint32_t bad = 0;
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            uint4 c = lds128(row + ((i ^ code_swz) * 16));
            if (partly) {
              // NaN codes become finite, with a weight of 0 where the key is not seen; slots that are
              // nobody's become 0
              uint32_t* w_ = &c.x;
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const uint32_t m = e4m3_nan_bits(w_[x]);
                bad |= there ? m : 0u;
                w_[x] = there ? w_[x] & ~(m >> 7) : 0u;
              }
            }
            uint32_t h[8];
            widen4(c.x, h[0], h[1]);
            widen4(c.y, h[2], h[3]);
            widen4(c.z, h[4], h[5]);
            widen4(c.w, h[6], h[7]);
            const uint32_t half = to + (i >> 2) * S::kVHalf, ch = 2 * (i & 3);
            sts128(half + ((ch ^ swz) * 16), h[0], h[1], h[2], h[3]);
            sts128(half + (((ch + 1) ^ swz) * 16), h[4], h[5], h[6], h[7]);
          }
          if (partly && __any_sync(0xffffffffu, bad != 0) && lane == 0) s_nan[gr] = 1;
        }
        warp_arrive(&s_vempty[gr]);

        // ---- weights ----
        far |= __any_sync(0xffffffffu, fabsf(page.y) > kFar);
        const float f = page.x, v = page.y, inv = page.z;
        const uint64_t ff = pair(f, f), vv = pair(v, v);
        // exponents of rows r and r + 1, s f + v - M, hidden ones -inf
        auto exponents = [&](float s0, float s1, int r, auto slow, float& e0, float& e1) {
          const float2 rf = *reinterpret_cast<const float2*>(&s_rowf[r]);
          const float2 m = *reinterpret_cast<const float2*>(&s_max[gr][r]);
          unpair(fma2(pair(s0, s1), mul2(pair(rf.x, rf.y), ff), add2(vv, pair(-m.x, -m.y))), e0, e1);
          if (decltype(slow)::value && partly) {
            const int c = j - p.start;
            auto sees = [&](int row) {
              return there && (c < 0 ? j >= s_lo[row]
                                     : c < 32 * kMaxTreeWords && (s_bits[row * kMaxTreeWords + (c >> 5)] >> (c & 31) & 1) != 0);
            };
            if (!sees(r)) e0 = -INFINITY;
            if (!sees(r + 1)) e1 = -INFINITY;
          }
        };
        if (!(ok = wait_warp(&s_sfull[gr], k & 1, abort_flag, err))) break;
        tc_fence_after();
        bool slow = partly || far || s_big[gr] != 0;
        // is any weight above 2^8 (a row's first too)?
        auto most_of = [&](auto slow_) {
          float most = -INFINITY;
#pragma unroll
          for (int c0 = 0; c0 < R; c0 += 16) {
            if (c0 >= cols) break;
            float s[16];
            tmem_ld16(s_col + quarter + c0, s);
#pragma unroll
            for (int x = 0; x < 16; x += 2) {
              float e0, e1;
              exponents(s[x], s[x + 1], c0 + x, slow_, e0, e1);
              most = max3(most, e0, e1);
            }
          }
          return most;
        };
        const float most = slow ? most_of(std::true_type{}) : most_of(std::false_type{});
        if (__any_sync(0xffffffffu, most > kLazy) && lane == 0) s_flag[gr] = k + 1;
        if (!(ok = meet_group())) break;
        if (s_flag[gr] == k + 1) {
          // the rows' largest exponents over the tile, then their new maxima and the factors of what is there
#pragma unroll 1
          for (int c0 = 0; c0 < cols; c0 += 16) {
            float s[16];
            tmem_ld16(s_col + quarter + c0, s);
#pragma unroll
            for (int x = 0; x < 16; x += 2) {
              float e0, e1;
              exponents(s[x], s[x + 1], c0 + x, std::true_type{}, e0, e1);
              // (relative to 0 where no maximum is set yet: 1e30 would swallow the score)
              const float2 m = *reinterpret_cast<const float2*>(&s_max[gr][c0 + x]);
              const float2 rf = *reinterpret_cast<const float2*>(&s_rowf[c0 + x]);
              if (m.x == kNoMax && e0 > -INFINITY) e0 = fmaf(s[x], f * rf.x, v);
              if (m.y == kNoMax && e1 > -INFINITY) e1 = fmaf(s[x + 1], f * rf.y, v);
              const float t0 = max_of_warp(e0 == e0 ? e0 : -INFINITY), t1 = max_of_warp(e1 == e1 ? e1 : -INFINITY);
              if (lane == 0) s_top[gr][gw][c0 + x] = t0, s_top[gr][gw][c0 + x + 1] = t1;
            }
          }
          if (!(ok = meet_group())) break;
          if (key < cols) {
            const float m = s_max[gr][key];
            float top = -INFINITY;
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, s_top[gr][i][key]);
            const bool unset = m == kNoMax;
            const float up = unset ? top : fmaxf(top, 0.0f);
            const bool moves = up > -INFINITY;
            const float now = moves ? (unset ? 0.0f : m) + up : m;
            s_max[gr][key] = now;
            s_keep[gr][key] = unset ? 0.0f : exp2_approx(-0.5f * up);  // half of the factor
            if (moves && fabsf(now) > 1e6f) s_big[gr] = 1;
          }
          if (!(ok = meet_group())) break;
#pragma unroll
          for (int r = 0; r < R; ++r)
            if (r < cols) {
              const float half = s_keep[gr][r];
              L[r] = L[r] * half * half;
            }
          if (any) {
#pragma unroll 1
            for (int c0 = 0; c0 < cols; c0 += 16) {
              float o[16];
              tmem_ld16(o_col + quarter + c0, o);
#pragma unroll
              for (int x = 0; x < 16; ++x) {
                const float half = s_keep[gr][c0 + x];
                o[x] = o[x] * half * half;
              }
              tc_st16(o_col + quarter + c0, *reinterpret_cast<const uint32_t(*)[16]>(o));
            }
            tmem_wait_st();
          }
          slow |= s_big[gr] != 0;
        }
        // the weights, and a share of the rows' sums
        const uint32_t p_row = smem_u32(smem + S::kPAt + gr * S::kPB) + (uint32_t)key * 128;
        auto weigh = [&](auto slow_) {
          constexpr bool kSlow = decltype(slow_)::value;
#pragma unroll
          for (int c0 = 0; c0 < R; c0 += 16) {
            if (c0 >= cols) break;
            float s[16];
            uint32_t h[8];
            tmem_ld16(s_col + quarter + c0, s);
#pragma unroll
            for (int x = 0; x < 16; x += 2) {
              float e0, e1;
              exponents(s[x], s[x + 1], c0 + x, slow_, e0, e1);
              if (kSlow) {                     // (scores so large that their rounding alone could pass 2^8 end there)
                e0 = e0 > kLazy ? kLazy : e0, e1 = e1 > kLazy ? kLazy : e1;
                // a quiet page's share of the sum beside a loud one's, from its own exponent
                L[c0 + x] += far ? exp2_approx(e0 - v) : 0.0f;
                L[c0 + x + 1] += far ? exp2_approx(e1 - v) : 0.0f;
              }
              const float w0 = exp2_approx(e0), w1 = exp2_approx(e1);
              if (!kSlow || !far) L[c0 + x] = fmaf(w0, inv, L[c0 + x]), L[c0 + x + 1] = fmaf(w1, inv, L[c0 + x + 1]);
              h[x / 2] = pack_f16(w0, w1);
            }
            sts128(p_row + (((c0 / 8) ^ swz) * 16), h[0], h[1], h[2], h[3]);
            sts128(p_row + (((c0 / 8 + 1) ^ swz) * 16), h[4], h[5], h[6], h[7]);
          }
        };
        if (slow) weigh(std::true_type{});
        else weigh(std::false_type{});
        fence_async();
        tc_fence_before();
        warp_arrive(&s_pfull[gr]);
        if (issues && wait_thread(&s_pfull[gr], k & 1, abort_flag, err)) {
          tc_fence_after();
          const uint32_t id = transposed_idesc(128, cols);
#pragma unroll
          for (int i = 0; i < kTile / 16; ++i)
            mma_ss(o_col, v_desc + (uint32_t)(i * 2048 >> 4), p_desc + (uint32_t)(i * 2048 >> 4), id, any || i != 0);
          tc_commit(&s_ofull[gr]);
        }
        __syncwarp();
        any = true;
      }
      if (!ok) break;
      if (any && !(ok = wait_warp(&s_ofull[gr], (k - 1) & 1, abort_flag, err))) break;
      tc_fence_after();

      // ---- the groups' rows meet ----
      // sums over the warp's lanes: halves change sides step by step, lane l ends with rows l * R / 32 ..
      {
        float x[R];
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] = L[r];
        int n = R;
#pragma unroll
        for (int o = 16; o; o >>= 1) {
          if (n > 1) {
            n >>= 1;
            const bool upper = lane & o;
#pragma unroll
            for (int r = 0; r < R / 2; ++r)
              if (r < n) {
                const float give = upper ? x[r] : x[r + n], keep = upper ? x[r + n] : x[r];
                x[r] = keep + __shfl_xor_sync(0xffffffffu, give, o);
              }
          } else {
            x[0] += __shfl_xor_sync(0xffffffffu, x[0], o);
          }
        }
        // R = 64: rows 2l', 2l' + 1, R = 32: row l', R = 16: row l' / 2, with l' = lane
        if (R == 64) s_l[gr][gw][2 * lane] = x[0], s_l[gr][gw][2 * lane + (R == 64)] = x[R == 64];
        else if (R == 32) s_l[gr][gw][lane] = x[0];
        else if ((lane & 1) == 0) s_l[gr][gw][lane / 2] = x[0];
      }
      tc_fence_before();
      if (!(ok = meet())) break;
      tc_fence_after();
      const bool whole = p.opens && p.closes;
      const int part_slot = 2 * blockIdx.x + (p.opens ? 1 : 0);
      auto top_of = [&](int r) { return fmaxf(s_max[0][r], s_max[1][r]); };
      auto factor = [&](int g, int r, float top) {         // half of a group's factor
        return s_max[g][r] == kNoMax ? 0.0f : exp2_approx(0.5f * (s_max[g][r] - top));
      };
      auto sum_of = [&](int r, float top) {
        float sum = 0.0f;
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          const float half = factor(g, r, top);
          const float l = (s_l[g][0][r] + s_l[g][1][r]) + (s_l[g][2][r] + s_l[g][3][r]);
          sum = fmaf(l * half, half, sum);
        }
        return sum;
      };
      auto out_of = [&](int r) {               // where value 0 of a row goes
        const int rr = p.block * R + r;
        return a.out + (int64_t)(p.row0 + rr / group) * a.out_stride + (int64_t)(p.h * group + rr % group) * D;
      };
      auto lse_of = [&](int r) {
        const int rr = p.block * R + r;
        return a.lse + (int64_t)(p.row0 + rr / group) * a.q_heads + p.h * group + rr % group;
      };
      auto lse_value = [](float top, float sum) { return sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f; };
      auto bits_of = [&](float x) { return (uint16_t)(bf16 ? f32_to_act<MOE_DTYPE_BF16>(x) : f32_to_act<MOE_DTYPE_F16>(x)); };
      if (tid < p.rows) {
        const float top = top_of(tid), sum = sum_of(tid, top);
        if (whole) {
          if (a.lse) *lse_of(tid) = lse_value(top, sum);
        } else {
          stats[(size_t)part_slot * 2 * kMostR + tid] = top;
          stats[((size_t)part_slot * 2 + 1) * kMostR + tid] = sum;
        }
      }
      // thread = value d of the rows; the two groups of warps take rows 16 at a time in turn
      const int d = key;
      const bool used0 = p.t1 > p.t0, used1 = p.t1 > p.t0 + 1;
      const uint32_t all_o = s_tmem + S::kOAt + quarter;
#pragma unroll 1
      for (int c0 = gr * 16; c0 < p.rows; c0 += 32) {
        float o0[16], o1[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) o0[x] = o1[x] = 0.0f;
        if (used0) tmem_ld16(all_o + c0, o0);
        if (used1) tmem_ld16(all_o + S::kCols + c0, o1);
        if (d < D) {
#pragma unroll
          for (int x = 0; x < 16; ++x) {
            const int r = c0 + x;
            if (r >= p.rows) break;
            const float top = top_of(r), h0 = factor(0, r, top), h1 = factor(1, r, top);
            // (a group without keys has a factor of 0 and values of 0)
            float val = fmaf(o1[x] * h1, h1, o0[x] * h0 * h0);
            if (whole) {
              const float sum = sum_of(r, top);
              out_of(r)[d] = bits_of(val * (sum > 0.0f ? 1.0f / sum : sum));         // 0 stays 0, NaN stays NaN
            } else {
              part[((size_t)part_slot * kMostR + r) * D + d] = val;
            }
          }
        }
      }
      if (s_nan[0] | s_nan[1]) {
        // NaN codes kept out of the products, from the pages, into the rows that see them
        __syncwarp();
        if (!(ok = meet())) break;             // the rows are stored
#pragma unroll 1
        for (int t = p.t0; t < p.t1; ++t) {
          if (!(t >= part_from || t < edge || (t + 1) * kTile > p.len)) continue;
#pragma unroll 1
          for (int x = gr; x < kTile; x += kGroups) {
            const int j = t * kTile + x, c = j - p.start;
            if (j >= p.len) break;
            const int page = a.b.page_table[(int64_t)p.b * a.b.table_stride + (j >> log_p)];
            if (page < 0 || page >= a.c.num_pages || d >= D) continue;
            const uint8_t code = a.c.v_codes[(int64_t)page * a.c.page_stride + ((int64_t)p.h * P + (j & (P - 1))) * D + d];
            if ((code & 0x7f) != 0x7f) continue;
            for (int r = 0; r < p.rows; ++r) {
              const bool sees = c < 0 ? j >= s_lo[r]
                                      : c < 32 * kMaxTreeWords && (s_bits[r * kMaxTreeWords + (c >> 5)] >> (c & 31) & 1) != 0;
              if (!sees) continue;
              if (whole) out_of(r)[d] = 0x7fff;            // of either type
              else part[((size_t)part_slot * kMostR + r) * D + d] = NAN;
            }
          }
        }
      }
      tc_fence_before();
      if (!whole) {
        // the last piece of the segment to arrive joins all of them
        __threadfence();
        if (!(ok = meet())) break;
        if (tid == 0) {
          const uint32_t before = atomicAdd(&counters[p.c0], 1u);
          s_last = before == (uint32_t)(p.np - 1);
          if (s_last) counters[p.c0] = 0;
        }
        if (!(ok = meet())) break;
        if (s_last) {
          __threadfence();
          auto slot_of = [&](int i) { return (size_t)2 * (p.c0 + i) + (i == 0); };
          constexpr int kQuads = D / 4, kBatch = 8;
          for (int u = tid; u < p.rows * kQuads; u += kWorkers) {
            const int r = u / kQuads, q4 = u % kQuads;
            float top = kNoMax, sum = 0.0f;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int i0 = 0; i0 < p.np; i0 += kBatch) {
              float m[kBatch], l[kBatch];
              float4 x[kBatch];
#pragma unroll
              for (int i = 0; i < kBatch; ++i) {
                m[i] = kNoMax, l[i] = 0.0f, x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i0 + i < p.np) {
                  const size_t s = slot_of(i0 + i);
                  m[i] = __ldcg(stats + s * 2 * kMostR + r), l[i] = __ldcg(stats + (s * 2 + 1) * kMostR + r);
                  x[i] = __ldcg(reinterpret_cast<const float4*>(part + (s * kMostR + r) * D) + q4);
                }
              }
#pragma unroll
              for (int i = 0; i < kBatch; ++i) {
                const float to = fmaxf(top, m[i]);
                const float h0 = exp2_approx(0.5f * (top - to)), h1 = exp2_approx(0.5f * (m[i] - to)), f0 = h0 * h0, f1 = h1 * h1;
                top = to;
                sum = fmaf(l[i] * h1, h1, sum * h0 * h0);
                o.x = fmaf(x[i].x, f1, o.x * f0), o.y = fmaf(x[i].y, f1, o.y * f0);
                o.z = fmaf(x[i].z, f1, o.z * f0), o.w = fmaf(x[i].w, f1, o.w * f0);
              }
            }
            const float by = sum > 0.0f ? 1.0f / sum : sum;
            const uint32_t lo = bits_of(o.x * by) | (uint32_t)bits_of(o.y * by) << 16;
            const uint32_t hi = bits_of(o.z * by) | (uint32_t)bits_of(o.w * by) << 16;
            *reinterpret_cast<uint2*>(out_of(r) + q4 * 4) = make_uint2(lo, hi);
            if (q4 == 0 && a.lse) *lse_of(r) = lse_value(top, sum);
          }
        }
      }
      if (!(ok = meet())) break;               // shared memory and s_last are read before they are written again
    }
    if (!ok) {
      // gave up: products that were issued are done before the tensor memory is given back (bounded)
      const uint64_t t0 = global_ns();
      while (issues && !(mbar_try(&s_sfull[gr], k & 1) && mbar_try(&s_ofull[gr], k & 1)) && global_ns() - t0 < 100000000ull) {
      }
    }
  } else {
    // ---------------- codes; pages and scales ----------------
    // Pages come for as many tiles of a piece at once as lanes allow, the next such batch (or piece) being
    // asked for while this one's tiles are brought.
    const int in_tile = kTile >> log_p, log_t = 7 - log_p, batch = 32 >> log_t, which = lane >> log_t;
    const int slot_page = lane & (in_tile - 1);
    Walk look = w;
    Piece lp = {};
    int lt = 0;                                // next tile of lp
    auto ask_pages = [&] {
      while (lt >= lp.t1) {
        if (!next_piece<R>(look, lp, a, group)) return -2;
        lt = lp.t0;
      }
      const int t = lt + which, j = t * kTile + slot_page * P;
      const bool in = which < batch && t < lp.t1 && j < lp.len;
      const int page = (int)load_ahead(a.b.page_table + (int64_t)lp.b * a.b.table_stride + (j >> log_p), in, 0xffffffffu);
      lt += batch;
      return in ? page : -2;                   // (-2: no such page is asked for)
    };
    auto known = [&](int page) { return page >= 0 && page < a.c.num_pages; };
    auto ask_scale = [&](const float* scales, int page, int h) {
      return __uint_as_float(load_ahead(scales + (int64_t)page * heads + h, known(page), 0u));
    };
    uint32_t count[kGroups] = {};              // tiles of each group
    int page = ask_pages(), h_next = lp.h;
    float ks = ask_scale(a.c.k_scales, page, h_next), vs = ask_scale(a.c.v_scales, page, h_next);
    float ks_next = 0.0f, vs_next = 0.0f;
    int page_next = ask_pages();
    h_next = lp.h;
    bool begun = false;
    while (ok && next_piece<R>(w, p, a, group)) {
      for (int t = p.t0, gr = 0; t < p.t1; ++t, gr = gr + 1 == kGroups ? 0 : gr + 1) {
        uint32_t k = 0;
#pragma unroll
        for (int i = 0; i < kGroups; ++i)
          if (i == gr) k = count[i]++;
        const int in_batch = (t - p.t0) & (batch - 1);
        if (in_batch == 0 && begun) {
          page = page_next, ks = ks_next, vs = vs_next;
          page_next = ask_pages();
          h_next = lp.h;
        }
        begun = true;
        const bool mine = which == in_batch, good = mine && known(page);
        if (mine && !good && page != -2) atomicOr(err, (uint32_t)MOE_DEVERR_PAGE);
        const uint32_t there = __popc(__ballot_sync(0xffffffffu, good));
        const int slot = gr * S::kKSlots + k % S::kKSlots;
        if (!(ok = wait_warp(&s_kempty[slot], (k / S::kKSlots & 1) ^ 1, abort_flag, err))) break;
        if (mine) {
          const float scale = fminf(fmaxf(vs, 0x1p-100f), 0x1p120f);
          s_page[slot][slot_page] = good ? make_float4(a.scale * 1.4426950408889634f * ks, log2f(scale), __fdividef(1.0f, scale), 0.0f)
                                         : make_float4(1.0f, 0.0f, 0.0f, 0.0f);
        }
        __syncwarp();
        if (lane == 0) mbar_expect_tx(&s_kfull[slot], there * P * D);
        __syncwarp();
        if (good) tma_load_3d(smem + S::kKAt + slot * S::kCodeB + slot_page * P * S::kRowB, &kmap, 0, p.h * P, page, &s_kfull[slot]);
        if (in_batch == min(1, min(batch, p.t1 - (t - in_batch)) - 1)) {
          ks_next = ask_scale(a.c.k_scales, page_next, h_next);
          vs_next = ask_scale(a.c.v_scales, page_next, h_next);
        }
        if (!(ok = wait_warp(&s_vempty[gr], (k & 1) ^ 1, abort_flag, err))) break;
        if (lane == 0) mbar_expect_tx(&s_vfull[gr], there * P * D);
        __syncwarp();
        if (good) tma_load_3d(smem + S::kVcAt + gr * S::kCodeB + slot_page * P * S::kRowB, &vmap, 0, p.h * P, page, &s_vfull[gr]);
      }
    }
    if (!ok) {                                 // gave up: let the copies in flight land (bounded)
      const uint64_t t0 = global_ns();
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        for (uint32_t i = count[g] > S::kKSlots ? count[g] - S::kKSlots : 0; i < count[g]; ++i)
          while (!mbar_try(&s_kfull[g * S::kKSlots + i % S::kKSlots], i / S::kKSlots & 1) && global_ns() - t0 < 100000000ull) {
          }
        while (count[g] && !mbar_try(&s_vfull[g], (count[g] - 1) & 1) && global_ns() - t0 < 100000000ull) {
        }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 4 * kGroups)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(s_tmem), "n"(S::kAlloc));
  // Where the form for more rows runs before this one, this one may start beside it: what follows both
  // then waits for both.
  pdl_wait();
}

template <int D, int R>
cudaError_t launch_shape(const AttentionArgs& a, bool beside, cudaStream_t s) {
  using S = Shape<D, R>;
  CUtensorMap map[2];
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.c.kv_heads * a.c.page_size, (uint64_t)a.c.num_pages};
  const uint64_t strides[2] = {(uint64_t)D, (uint64_t)a.c.page_stride};
  const uint32_t box[3] = {(uint32_t)S::kRowB, (uint32_t)a.c.page_size, 1};
  const CUtensorMapSwizzle swz = D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  if (!make_map3(&map[0], a.c.k_codes, dims, strides, box, swz) || !make_map3(&map[1], a.c.v_codes, dims, strides, box, swz))
    return cudaErrorInvalidValue;
  auto kern = tree_kernel<D, R>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  const int grid = num_sms() < kMostGrid ? num_sms() : kMostGrid;
  if (beside) return launch_pdl(kern, dim3(grid), dim3(kThreads), S::kSmem, s, a, map[0], map[1]);
  kern<<<grid, kThreads, S::kSmem, s>>>(a, map[0], map[1]);
  return cudaGetLastError();
}

template <int D>
cudaError_t launch_dim(const AttentionArgs& a, bool beside, cudaStream_t s) {
  // Rows of a block: as few as hold the sequences' rows on average.
  const long long rows = ((long long)a.T * (a.q_heads / a.c.kv_heads) + a.b.B - 1) / a.b.B;
  if (rows <= 16) return launch_shape<D, 16>(a, beside, s);
  return rows <= 32 ? launch_shape<D, 32>(a, beside, s) : launch_shape<D, 64>(a, beside, s);
}

}  // namespace

size_t tree_attention_ws_bytes(int head_dim) { return align_up(kRowsAt + (size_t)2 * kMostGrid * kMostR * head_dim * 4); }

cudaError_t launch_tree_attention(const AttentionArgs& a, bool beside, cudaStream_t s) {
  return a.c.head_dim == 64 ? launch_dim<64>(a, beside, s) : launch_dim<128>(a, beside, s);
}

}  // namespace moe
