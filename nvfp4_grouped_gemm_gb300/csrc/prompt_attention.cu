// Causal attention over the paged 8-bit cache for sequences with many query rows (chunks of
// prompts, long drafts): the tensor-memory form of moe_attention_paged_e4m3. paged_attention.cu
// has the form for few rows and the definitions both share.
//
// Rows of a sequence that share a key head (n new tokens times the group of query heads) come in
// blocks of 256, two tiles A and B of 128; keys come in tiles of 128. All segments' (sequence,
// head, block) key tiles form one line that the grid cuts into equal pieces, one CTA per SM, as
// in paged_attention.cu; a cut segment's partial rows are joined by the last CTA to arrive.
//
//   warps 0-3, 4-7   softmax of tile A, B: thread = row. S from tensor memory, the weights
//                    2^(s f + v - M) as f16 back over S, the row's sum in f32; M moves only when
//                    a weight would pass 2^8, and O is rescaled (in tensor memory) only then
//   warps 8-15       keys and values: 16-byte pieces from the pages, widened to f16 (exact) and
//                    stored as 128-byte-swizzled tiles; slots past the end or in pages out of
//                    range become 0, and NaN codes of V in tiles that not every row sees whole
//                    become finite (the softmax threads then put NaN into the rows that see them)
//   warp 16          one thread issues the tensor-core products (kind::f16, f32 accumulation):
//                    S = Q K^T (K-major tiles), O += P V (P from tensor memory, V as the tile's
//                    rows, i.e. with the value dimension contiguous)
// While tile A's softmax runs, the tensor cores work on tile B and the other way round. A commit
// covers every product issued before it, so a softmax that sees its S knows that the previous
// O += P V is complete and may rescale O.
//
// For trees of drafted tokens (moe_attention_tree_e4m3) a row's bits, cut to what the window leaves, lie
// in shared memory and stand in for its place in the tiles that hold new tokens or a window's edge.
//
// Tensor memory is full at D = 128 (two S, two O of 128 columns), so a tile's weights lie over its
// S and its chain (softmax, O += P V, the next S) is serial; two tiles in flight hide each other's
// softmax. 2048 new tokens after 6144, 32 query and 8 key heads of 128, bf16: 278 us, 0.87 PFLOP/s
// of unmasked products. A period of both tiles takes about 4400 clocks: 2 * 1400 of products (1024
// without the widening warps' stores beside their operand reads in shared memory), and a softmax
// of about 2000 with hand-offs of about 400. What its steps gave: the weights from one reading of
// S (before, a pass for the maximum came first) and waits that neither read the clock nor tell
// lanes the outcome 361 -> 288 us; the line walked by whole warps, rows staged and stored
// coalesced 288 -> 275. Slower: two threads per row (a barrier per tile between them and fewer
// registers), S held in registers (the widening warps, short of them, then spill), key tiles of 64
// with two S in flight (394 us when this form took 361).
#include "tc_f16.cuh"

namespace moe {
namespace {

constexpr int kTile = 128;                     // keys per tile, rows per row tile
constexpr int kBlock = 256;                    // rows per block
constexpr int kThreads = 20 * 32;
constexpr int kSoftmax = 256, kConvert = 256;
// Registers per thread of the two softmax, two widening and one issuing warpgroups: together not
// more than the block is launched with.
constexpr int kRegsLaunch = 65536 / kThreads / 8 * 8;
constexpr int kRegsSoftmax = 128, kRegsConvert = 80, kRegsIssue = 64;
static_assert(2 * kRegsSoftmax + 2 * kRegsConvert + kRegsIssue <= 5 * kRegsLaunch, "more than the block has");
// raising and lowering are different instructions, each legal in its own direction only
static_assert(kRegsSoftmax >= kRegsLaunch && kRegsConvert <= kRegsLaunch && kRegsIssue <= kRegsLaunch, "");
constexpr float kNoMax = -1e30f;
constexpr float kLazy = 8.0f;
constexpr float kFar = 40.0f;                  // of value scales, as in paged_attention.cu
// A segment's fixed cost (queries, first tiles, storing rows) in key tiles.
constexpr int kSegmentCost = 3;

// Workspace, from the end of the other form's: arrival counters, maxima and sums, rows [D/4][256][4].
constexpr size_t kCountersAt = 0;
constexpr size_t kStatsAt = kCountersAt + kPromptMaxGrid * 4;
constexpr size_t kRowsAt = kStatsAt + (size_t)2 * kPromptMaxGrid * 2 * kBlock * 4;

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float max16(const float* s) {
  const float a = max3(s[0], s[1], s[2]), b = max3(s[3], s[4], s[5]), c = max3(s[6], s[7], s[8]);
  const float d = max3(s[9], s[10], s[11]), e = max3(s[12], s[13], s[14]);
  return max3(max3(a, b, c), max3(d, e, s[15]), s[15]);
}
// Scores of 32 keys: those outside [x0, x1), and of a group of 16 without a page, become -inf.
__device__ __forceinline__ void hide(float (&s)[32], int x0, int x1, bool there0, bool there1) {
  asm volatile("" ::: "memory");               // a real branch: not selects on every tile
#pragma unroll
  for (int x = 0; x < 32; ++x)
    if (x < x0 || x >= x1 || !(x < 16 ? there0 : there1)) s[x] = -INFINITY;
}

// The same with the visible keys as bits.
__device__ __forceinline__ void hide_bits(float (&s)[32], uint32_t seen, bool there0, bool there1) {
  asm volatile("" ::: "memory");
  seen &= (there0 ? 0x0000ffffu : 0u) | (there1 ? 0xffff0000u : 0u);
#pragma unroll
  for (int x = 0; x < 32; ++x)
    if (!(seen >> x & 1)) s[x] = -INFINITY;
}

// A sequence's rows and its share of the line.
struct Seq {
  int row0, n, start, len, blocks;
  long long per_head;                          // line length of one key head
};
// Key tiles [x, y) that block `block` of a sequence can see.
template <bool TREE>
__device__ __forceinline__ int2 block_tiles(const Seq& q, int block, int group, int window) {
  const int first = block * kBlock / group, last = (min((block + 1) * kBlock, q.n * group) - 1) / group;
  const int hi = TREE ? q.len : min(q.len, q.start + last + 1);
  const int lo = window > 0 ? max(0, min(TREE ? q.start - window : q.start + first - window + 1, TREE ? q.len : 0x7fffffff)) : 0;
  const int x = lo / kTile;
  return make_int2(x, max(x, (max(hi, 0) + kTile - 1) / kTile));
}
// Key tiles from `from` on and before `before` have keys that some row of the piece's block does not
// see.
struct Partly {
  int from, before;
};
__device__ __forceinline__ bool partly(const Partly& p, int t) { return t >= p.from || t < p.before; }
template <bool TREE>
__device__ __forceinline__ int block_line(const Seq& q, int block, int group, int window) {
  const int2 t = block_tiles<TREE>(q, block, group, window);
  return max(t.y - t.x, 1) + kSegmentCost;
}
// By a warp: its lanes take the blocks in turn.
template <bool TREE>
__device__ __forceinline__ Seq read_seq(const AttentionArgs& a, int b, int group, int min_rows, uint32_t* err) {
  Seq q;
  q.row0 = min(max(a.b.q_offsets[b], 0), a.T);
  const int end = min(max(a.b.q_offsets[b + 1], q.row0), a.T);
  q.n = end - q.row0;
  q.len = a.b.seq_lens[b];
  q.start = q.len - q.n;
  q.blocks = 0;
  q.per_head = 0;
  if (q.n * group < min_rows || q.n == 0) return q;        // the other form's, or nothing to do
  const int cap = a.b.max_pages * a.c.page_size, lane = threadIdx.x & 31;
  if ((q.len < q.n || q.len > cap) && err && lane == 0) atomicOr(err, (uint32_t)MOE_DEVERR_PAGE);
  q.len = min(max(q.len, 0), cap);
  q.blocks = (q.n * group + kBlock - 1) / kBlock;
  for (int i = lane; i < q.blocks; i += 32) q.per_head += block_line<TREE>(q, i, group, a.window);
#pragma unroll
  for (int o = 16; o; o >>= 1) q.per_head += __shfl_xor_sync(0xffffffffu, q.per_head, o);
  return q;
}

// One CTA's share of one segment.
struct Piece {
  bool more;                                   // false: the CTA's line ended
  bool opens, closes;                          // holds the segment's first / last tile
  int b, head, block, R;                       // sequence, key head, block of rows, rows in it
  int row0, n, start, len;                     // of the sequence
  int t0, t1;                                  // key tiles to work on (none if t0 >= t1)
  int c0, np;                                  // the CTAs the segment is spread over
};
// A CTA's piece of the line. Every warp walks for itself, its lanes side by side over the blocks.
struct Walk {
  long long pos, end, per, first;
  int b, head, block;
  long long at;                                // line position of (b, head, block)
  Seq q;
};
template <bool TREE>
__device__ __forceinline__ void walk_enter(Walk& w, const AttentionArgs& a, int group, int min_rows) {  // from (b, first)
  w.q = read_seq<TREE>(a, w.b, group, min_rows, nullptr);
  w.head = w.q.per_head ? (int)((w.pos - w.first) / w.q.per_head) : 0;
  w.block = 0;
  w.at = w.first + w.head * w.q.per_head;
}
template <bool TREE>
__device__ __forceinline__ Piece walk_next(Walk* state, const AttentionArgs& a, int group, int min_rows) {
  const int lane = threadIdx.x & 31;
  __syncwarp();
  Walk w = *state;                             // the same in every lane
  Piece p;
  p.more = false;
  while (w.pos < w.end) {
    while (w.pos >= w.first + w.q.per_head * a.c.kv_heads) {
      w.first += w.q.per_head * a.c.kv_heads;
      ++w.b;
      walk_enter<TREE>(w, a, group, min_rows);
    }
    // the block that pos is in: 32 at a time, by a running sum of their lines
    int line = 0;
    while (true) {
      const int mine = w.block + lane < w.q.blocks ? block_line<TREE>(w.q, w.block + lane, group, a.window) : 0;
      int upto = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += up;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, w.at + upto > w.pos);
      const int j = past ? __ffs(past) - 1 : 31;
      upto = __shfl_sync(0xffffffffu, upto, j);
      line = __shfl_sync(0xffffffffu, mine, j);
      if (past) {
        w.at += upto - line;
        w.block += j;
        break;
      }
      w.at += upto;
      w.block += 32;
      if (w.block >= w.q.blocks) w.block = 0, ++w.head;
    }
    const int2 t = block_tiles<TREE>(w.q, w.block, group, a.window);
    const int st0 = max(0, (int)(w.pos - w.at) - kSegmentCost);
    const int st1 = (int)min((long long)line, w.end - w.at) - kSegmentCost;
    w.pos = w.at + st1 + kSegmentCost;
    if (st1 <= st0) continue;                  // only the segment's fixed cost fell to this CTA
    p.b = w.b, p.head = w.head, p.block = w.block;
    p.R = min(kBlock, w.q.n * group - w.block * kBlock);
    p.row0 = w.q.row0, p.n = w.q.n, p.start = w.q.start, p.len = w.q.len;
    p.t0 = t.x + st0, p.t1 = min(t.x + st1, t.y);
    p.opens = st0 == 0, p.closes = st1 == line - kSegmentCost;
    p.c0 = (int)((w.at + kSegmentCost) / w.per);
    p.np = (int)((w.at + line - 1) / w.per) - p.c0 + 1;
    p.more = true;
    break;
  }
  __syncwarp();
  if (lane == 0) *state = w;
  return p;
}

template <bool TREE>
__device__ __forceinline__ Partly partly_seen(const Piece& p, int group, int window) {
  if (TREE) {                                  // new tokens; where the rows' windows may begin
    const int edge = p.start + min(p.n, 32 * kMaxTreeWords) - window;
    return {max(min(p.start, p.len), 0) / kTile, window > 0 && edge > 0 ? (edge + kTile - 1) / kTile : 0};
  }
  const int lo = p.start + p.block * kBlock / group;       // the block's first and last rows' places
  const int hi = p.start + (p.block * kBlock + p.R - 1) / group;
  return {min(lo + 1, p.len) / kTile, window > 0 ? (hi - window + kTile) / kTile : 0};
}

template <int D>
struct Smem {
  static constexpr int kQ = 128 * D * 2;       // one row tile of queries
  static constexpr int kKv = kTile * D * 2;    // one widened key or value tile
  static constexpr int kHalf = 128 * 128;      // 64 values of 128 rows
  static constexpr int kQAt = 0, kKAt = 2 * kQ, kVAt = kKAt + 2 * kKv;
  static constexpr int kBytes = kVAt + 2 * kKv;
};

template <int D, bool TREE>
__global__ void __launch_bounds__(kThreads, 1)
prompt_kernel(const __grid_constant__ AttentionArgs a, int min_rows, char* ws) {
  using S = Smem<D>;
  extern __shared__ char smem_raw[];
  __shared__ uint64_t s_kfull[2], s_kempty[2], s_vfull[2], s_vempty[2], s_sfull[2], s_pfull[2], s_qfull[2], s_drain, s_join;
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ long long s_sum[kThreads / 32], s_first;
  __shared__ int s_seq, s_last;
  __shared__ float4 s_coef[8][8];
  __shared__ Walk s_walk[16];
  __shared__ int2 s_issue;                     // the issuing thread's piece: key tiles (0: no more), row tiles
  __shared__ long long s_line[kThreads];
  __shared__ volatile uint32_t s_nan[2][kConvert / 32];    // NaN codes that a widening warp kept out of V
  __shared__ uint32_t s_bits[TREE ? kMaxTreeWords : 1][TREE ? kBlock : 1];     // a thread's own row
  __shared__ volatile int s_nan_from[kSoftmax / 32];       // a softmax warp's first key tile with such
  char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int heads = a.c.kv_heads, group = a.q_heads / heads, P = a.c.page_size;
  uint32_t* err = reinterpret_cast<uint32_t*>(a.ws);
  volatile int* abort_flag = &s_abort;
  // With the other form behind it, which waits for this one at its end, that may start beside it;
  // alone it must not let a successor start on unfinished rows.
  if (min_rows > 1) pdl_trigger();

  // ---- this CTA's piece of the line (before any tensor memory is taken) ----
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
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) base += s_sum[w];
      all += s_sum[w];
    }
    *before = base + x - v;
    return all;
  };
  // line lengths of kThreads sequences at a time, a warp per sequence
  auto lines = [&](int b0, uint32_t* err) {
    __syncthreads();
    for (int b = b0 + warp; b < min(b0 + kThreads, a.b.B); b += kThreads / 32) {
      const long long line = read_seq<TREE>(a, b, group, min_rows, err).per_head * heads;
      if (lane == 0) s_line[b - b0] = line;
    }
    __syncthreads();
    return b0 + tid < a.b.B ? s_line[tid] : 0;
  };
  long long total = 0, at = 0, mine = 0;
  for (int b0 = 0; b0 < a.b.B; b0 += kThreads) {
    mine = lines(b0, blockIdx.x == 0 ? err : nullptr);
    total += scan(mine, &at);
  }
  long long per = (total + gridDim.x - 1) / gridDim.x;
  if (per < kSegmentCost + 1) per = kSegmentCost + 1;
  const long long begin = per * blockIdx.x, end = min(begin + per, total);
  if (begin >= end) return;
  long long base = 0;
  for (int b0 = 0; b0 < a.b.B; b0 += kThreads) {
    long long sum = total;
    if (a.b.B > kThreads) {                    // else known from the sum above
      mine = lines(b0, nullptr);
      sum = scan(mine, &at);
    }
    if (mine > 0 && base + at <= begin && begin < base + at + mine) s_seq = b0 + tid, s_first = base + at;
    base += sum;
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s_kfull[i], kConvert / 32);               // one arrival per warp
      mbar_init(&s_vfull[i], kConvert / 32);
      mbar_init(&s_kempty[i], 1);
      mbar_init(&s_vempty[i], 1);
      mbar_init(&s_sfull[i], 1);
      mbar_init(&s_pfull[i], 4);
      mbar_init(&s_qfull[i], 4);
    }
    mbar_init(&s_drain, 1);
    mbar_init(&s_join, kSoftmax / 32);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async();
  }
  if (warp == 16) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_u32(&s_tmem)), "n"(512) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  if (warp < 16) {
    Walk w;
    w.pos = begin, w.end = end, w.per = per, w.first = s_first, w.b = s_seq;
    walk_enter<TREE>(w, a, group, min_rows);
    if (lane == 0) s_walk[warp] = w;
  }

  if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    // ---------------- products ----------------
    // One thread issues both tiles' in turn, A's and then B's: it keeps the tiles half a period
    // apart, so that one's softmax runs beside the other's products.
    if (warp == 16 && lane == 0) {
      constexpr uint32_t id_s = f16_idesc(128, kTile, false), id_o = f16_idesc(128, D, true);
      const uint32_t sm = smem_u32(smem);
      const uint64_t q_desc = smem_desc(sm + S::kQAt, 16, 1024, 2);
      const uint64_t k_desc = smem_desc(sm + S::kKAt, 16, 1024, 2);
      const uint64_t v_desc = smem_desc(sm + S::kVAt, S::kHalf, 1024, 2);
      uint32_t kv = 0, qph = 0, pph = 0;                   // key tiles; phases per row tile
      bool ok = true;
      auto scores = [&](int tile, uint32_t t) {            // S of a row tile with key tile t
        const uint64_t qd = q_desc + tile * (S::kQ >> 4), kd = k_desc + (t & 1) * (S::kKv >> 4);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          const uint32_t o = (uint32_t)((i >> 2) * S::kHalf + (i & 3) * 32) >> 4;
          mma_ss(tmem + tile * 128, qd + o, kd + o, id_s, i != 0);
        }
      };
      auto values = [&](int tile, uint32_t t, bool add) {  // O += P V
        const uint64_t vd = v_desc + (t & 1) * (S::kKv >> 4);
        const uint32_t o_col = tmem + 256 + tile * D, p_col = tmem + tile * 128;
        mma_ts(o_col, p_col, vd, id_o, add ? 1u : 0u);
#pragma unroll
        for (int i = 1; i < kTile / 16; ++i) mma_ts(o_col, p_col + 8 * i, vd + (uint32_t)(i * 2048 >> 4), id_o, 1u);
      };
      while (ok) {
        // tile A's queries are there, and with them the piece; then B's
        if (!(ok = wait_thread(&s_qfull[0], qph & 1, abort_flag, err))) break;
        const int nt = s_issue.x, tiles = s_issue.y;
        if (nt == 0) break;
        if (tiles == 2) ok = wait_thread(&s_qfull[1], qph >> 1 & 1, abort_flag, err);
        qph ^= tiles == 2 ? 3u : 1u;
        if (ok) ok = wait_thread(&s_kfull[kv & 1], (kv >> 1) & 1, abort_flag, err);
        if (!ok) break;
        tc_fence_after();
        for (int i = 0; i < tiles; ++i) {
          scores(i, kv);
          tc_commit(&s_sfull[i]);
        }
        for (int t = 0; t < nt && ok; ++t, ++kv) {
          const bool more = t + 1 < nt;
#pragma unroll 1
          for (int i = 0; i < tiles; ++i) {
            // the weights, and with tile A's V and the next K: its softmax warps have seen them
            if (!(ok = wait_thread(&s_pfull[i], (pph >> i) & 1, abort_flag, err))) break;
            pph ^= 1u << i;
            tc_fence_after();
            values(i, kv, t > 0);
            if (more) scores(i, kv + 1);
            tc_commit(&s_sfull[i]);                        // S of the next tile, or the final O
          }
        }
      }
      // every product is done before the tensor memory is given back
      tc_commit(&s_drain);
      const uint64_t t0 = global_ns();
      while (!mbar_try(&s_drain, 0) && global_ns() - t0 < 100000000ull) {
      }
    }
  } else if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConvert));
    // ---------------- keys and values ----------------
    // Half tiles in turn (K's two, V's two, the next tile's ...), each fetched three halves ahead.
    const int ct = tid - kSoftmax;
    constexpr int kPieces = D / 16;            // 16-byte pieces of a token's row
    constexpr int kStride = kConvert / kPieces;            // tokens between a thread's pieces
    constexpr int kHalfN = 64 / kStride;       // a thread's pieces of 64 tokens
    // Eight lanes take four pieces of one half (64 values) of two neighbouring tokens: their
    // stores, 16-byte columns 2*(piece%4) and the next of the half, then hit every bank.
    const int piece = (ct & 3) + (D == 128 ? (ct >> 3 & 1) * 4 : 0);
    const int tok0 = (ct >> 2 & 1) + (ct >> (D == 128 ? 4 : 3)) * 2, log_p = 31 - __clz(P);
    const int64_t thread_at = (int64_t)(tok0 & 15) * D + piece * 16;
    const int col = 2 * (piece & 3);
    uint32_t kv = 0;
    bool ok = true;
    while (ok) {
      const Piece p = walk_next<TREE>(&s_walk[warp], a, group, min_rows);
      if (!p.more) break;
      const int32_t* table = a.b.page_table + (int64_t)p.b * a.b.table_stride;
      // lane l holds where 16-key group l % 8 of a tile starts in either plane (-1: nowhere)
      auto page_of = [&](int t) {
        const int j = t * kTile + (lane & 7) * 16;
        return (int)load_ahead(table + (j >> log_p), t < p.t1 && j < p.len, 0xffffffffu);
      };
      auto start_of = [&](int t, int page) {
        const int j = t * kTile + (lane & 7) * 16;
        if (page >= 0 && page < a.c.num_pages)
          return page * a.c.page_stride + ((int64_t)p.head * P + (j & (P - 1))) * D;
        if (t < p.t1 && j < p.len) atomicOr(err, (uint32_t)MOE_DEVERR_PAGE);
        return (int64_t)-1;
      };
      const Partly part = partly_seen<TREE>(p, group, a.window);
      uint32_t nan = 0;
      int page_next = page_of(p.t0);           // of the tile after the one fetched from
      int64_t start = -1;
      auto fetch = [&](int t, int half, uint4 (&r)[kHalfN]) {   // half 0, 1: K's; 2, 3: V's
        const uint8_t* plane = half & 2 ? a.c.v_codes : a.c.k_codes;
        const int tok = (half & 1) * 64, there = p.len - t * kTile - tok;   // tokens that exist
#pragma unroll
        for (int i = 0; i < kHalfN; ++i) {
          const int at_ = tok0 + i * kStride;
          const int64_t from = __shfl_sync(0xffffffffu, start, (tok + at_) >> 4);
          r[i] = load_ahead(plane + from + thread_at, from >= 0 && at_ < there);
        }
      };
      uint4 r[4][kHalfN];                      // the four halves; never copied while a load is out
      if (p.t0 < p.t1) {
        start = start_of(p.t0, page_next);
        page_next = page_of(p.t0 + 1);
#pragma unroll
        for (int h = 0; h < 3; ++h) fetch(p.t0, h, r[h]);
      }
#pragma unroll 1
      for (int t = p.t0; t < p.t1 && ok; ++t, ++kv) {
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          if (h == 0) {
            fetch(t, 3, r[3]);
          } else {
            if (h == 1) {
              start = start_of(t + 1, page_next);
              page_next = page_of(t + 2);
            }
            if (t + 1 < p.t1) fetch(t + 1, h - 1, r[h - 1]);
          }
          if ((h & 1) == 0 && ok)
            ok = wait_warp(h ? &s_vempty[kv & 1] : &s_kempty[kv & 1], ((kv >> 1) & 1) ^ 1, abort_flag, err);
          if (!ok) break;
          if (h & 2 && partly(part, t)) {
            if (h == 2) nan = 0;
#pragma unroll
            for (int i = 0; i < kHalfN; ++i)
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                uint32_t& w = x == 0 ? r[h][i].x : x == 1 ? r[h][i].y : x == 2 ? r[h][i].z : r[h][i].w;
                const uint32_t m = e4m3_nan_bits(w);
                w &= ~(m >> 7);                // a finite code, with a weight of 0 where it is not seen
                nan |= m;
              }
            if (h == 3) {
              nan = __reduce_or_sync(0xffffffffu, nan);
              if (lane == 0) s_nan[kv & 1][warp - 8] = nan;
            }
          }
          char* dst = smem + (h & 2 ? S::kVAt : S::kKAt) + (kv & 1) * S::kKv + (piece >> 2) * S::kHalf;
#pragma unroll
          for (int i = 0; i < kHalfN; ++i) {
            const int tok = (h & 1) * 64 + tok0 + i * kStride;
            uint4 lo, hi;
            widen4(r[h][i].x, lo.x, lo.y);
            widen4(r[h][i].y, lo.z, lo.w);
            widen4(r[h][i].z, hi.x, hi.y);
            widen4(r[h][i].w, hi.z, hi.w);
            char* row = dst + tok * 128;
            *reinterpret_cast<uint4*>(row + ((col ^ (tok & 7)) * 16)) = lo;
            *reinterpret_cast<uint4*>(row + (((col + 1) ^ (tok & 7)) * 16)) = hi;
          }
          if (h & 1) {
            fence_async();
            warp_arrive(h & 2 ? &s_vfull[kv & 1] : &s_kfull[kv & 1]);
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ---------------- softmax: thread = row ----------------
    const int tile = warp >> 2;
    const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + tile * 128 + quarter, o_col = tmem + 256 + tile * D + quarter;
    const int r = tid;                                     // row of the block
    const bool bf16 = a.dtype == MOE_DTYPE_BF16;
    const int log_p = 31 - __clz(P);
    uint32_t* counters = reinterpret_cast<uint32_t*>(ws + kCountersAt);
    float* stats = reinterpret_cast<float*>(ws + kStatsAt);
    float4* part_rows = reinterpret_cast<float4*>(ws + kRowsAt);
    uint32_t sph = 0, jph = 0, kv = 0;         // phases; key tiles
    bool ok = true;
    // the softmax threads meet (bounded, like every wait here)
    auto meet = [&] {
      warp_arrive(&s_join);
      return wait_warp(&s_join, jph++ & 1, abort_flag, err);
    };
    while (true) {
      const Piece p = walk_next<TREE>(&s_walk[warp], a, group, min_rows);
      if (!p.more) break;
      const int nt = p.t1 - p.t0;
      const bool live = p.R > 128 * tile;                  // this row tile is worked on
      const bool warp_live = p.R > 32 * warp;              // this warp has rows
      const int rr = p.block * kBlock + r;
      const int place = p.start + rr / group;
      const int64_t row = p.row0 + rr / group;
      const int hq = p.head * group + rr % group;
      float M = kNoMax, L = 0.0f, rowf = 1.0f;
      int lo = 0;                              // first of the tokens before the new ones that the row sees
      if (TREE) {
        uint32_t w[kMaxTreeWords];
        lo = tree_row(a, row, r < p.R, p.n, p.start, w);
#pragma unroll
        for (int i = 0; i < kMaxTreeWords; ++i) s_bits[TREE ? i : 0][TREE ? r : 0] = w[i];
      }
      // which of the keys j .. j + 31 the row sees, as bits
      auto seen_from = [&](int j) {
        const int c = j - p.start;             // as a new token
        auto word = [&](int i) { return i >= 0 && i < kMaxTreeWords ? s_bits[TREE ? i : 0][TREE ? r : 0] : 0u; };
        uint32_t v = __funnelshift_r(word(c >> 5), word((c >> 5) + 1), c & 31);
        if (c < 0) {
          const uint32_t before = c <= -32 ? 0xffffffffu : (1u << -c) - 1;
          const int skip = lo - j;             // hidden by the window
          v = (v & ~before) | (skip <= 0 ? before : skip >= 32 ? 0u : before & 0xffffffffu << skip);
        }
        const int there = p.len - j;
        return there >= 32 ? v : there <= 0 ? 0u : v & ((1u << there) - 1);
      };
      // The issuing thread's waits and commits are the block's bottleneck: what these warps can wait
      // for and signal in its place they do. The last row tile's products come last, so its S tells
      // that K and the V before it are read.
      const bool frees = warp == (p.R > 128 ? 4 : 0) && lane == 0;
      // A warp's rows go between memory and the tile of queries with D / 8 lanes per row; a thread
      // has its own row's 16-byte columns there at column_at.
      constexpr int kLanes = D / 8, kRows = 32 / kLanes;
      const int col = lane % kLanes, sub = lane / kLanes;
      char* tile_at = smem + S::kQAt + tile * S::kQ;
      auto column_at = [&](int row_, int i) {
        return reinterpret_cast<uint4*>(tile_at + (i >> 3) * S::kHalf + (row_ & 127) * 128 + ((i & 7) ^ (row_ & 7)) * 16);
      };
      if (live && nt > 0) {
        // the rows as f16 times a power of two, K-major, 128-byte swizzle
        const uint64_t src = reinterpret_cast<uint64_t>(a.q + row * a.q_stride + (int64_t)hq * D);
        // (code that runs once per piece is kept short: fetching it costs more than running it)
#pragma unroll 1
        for (int k0 = 0; k0 < kLanes; k0 += 8) {
          uint4 w[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int from = kRows * (k0 + k) + sub;
            const uint64_t at = __shfl_sync(0xffffffffu, src, from);
            w[k] = load_ahead(reinterpret_cast<const uint4*>(at) + col, r - lane + from < p.R);
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) *column_at(r - lane + kRows * (k0 + k) + sub, col) = w[k];
        }
        __syncwarp();
        if (bf16) {                            // here a thread has its own row
          uint32_t most = 0;                   // of the magnitudes' bits, in pairs
#pragma unroll 4
          for (int i = 0; i < kLanes; ++i) {
            const uint4 w = *column_at(r, i);
            most = __vimax3_u16x2(most, w.x & 0x7fff7fffu, w.y & 0x7fff7fffu);
            most = __vimax3_u16x2(most, w.z & 0x7fff7fffu, w.w & 0x7fff7fffu);
          }
          const float amax = __uint_as_float(max(most << 16, most & 0xffff0000u));
          const int e = amax < 3.4e38f ? f16_prescale_exp(amax) : 0;
          const float s1 = pow2f(-e / 2), s2 = pow2f(-e - (-e / 2));
          rowf = pow2f(e);
#pragma unroll 2
          for (int i = 0; i < kLanes; ++i) {
            uint4* at = column_at(r, i);
            uint4 w = *at;
            float f[8];
            unpack8<MOE_DTYPE_BF16>(w, f);
            w.x = pack_f16(f[0] * s1 * s2, f[1] * s1 * s2), w.y = pack_f16(f[2] * s1 * s2, f[3] * s1 * s2);
            w.z = pack_f16(f[4] * s1 * s2, f[5] * s1 * s2), w.w = pack_f16(f[6] * s1 * s2, f[7] * s1 * s2);
            *at = w;
          }
        }
        fence_async();
        if (tid == 0) s_issue = make_int2(nt, p.R > 128 ? 2 : 1);
        warp_arrive(&s_qfull[tile]);

        // page factors of a tile's eight 16-key groups: lane g < 8 holds group g's
        const int32_t* table = a.b.page_table + (int64_t)p.b * a.b.table_stride;
        auto page_of = [&](int t) {
          const int j = t * kTile + (lane & 7) * 16;
          return (int)load_ahead(table + (j >> log_p), t < p.t1 && j < p.len, 0xffffffffu);
        };
        // a tile's pages are read two tiles ahead, its scales one
        struct Scales { float k, v; };
        auto scales_of = [&](int page) {
          const bool there = page >= 0 && page < a.c.num_pages;
          const int64_t sc = (int64_t)page * heads + p.head;
          return Scales{__uint_as_float(load_ahead(a.c.k_scales + sc, there, 0u)),
                        __uint_as_float(load_ahead(a.c.v_scales + sc, there, 0u))};
        };
        bool far = false;                        // a value scale so far was outside [2^-kFar, 2^kFar]
        int page = page_of(p.t0), page_next = page_of(p.t0 + 1);
        Scales scales = scales_of(page);
        const Partly part = partly_seen<TREE>(p, group, a.window);
        if (lane == 0) s_nan_from[warp] = p.t1;
        for (int t = p.t0; t < p.t1; ++t) {
          const bool there = page >= 0 && page < a.c.num_pages;
          const float vs = fminf(fmaxf(scales.v, 0x1p-100f), 0x1p120f), v = log2f(vs);
          __syncwarp();
          if (lane < 8)
            s_coef[warp][lane] = there ? make_float4(a.scale * 1.4426950408889634f * scales.k, v, __fdividef(1.0f, vs), 1.0f)
                                       : make_float4(1.f, 0.f, 0.f, 0.f);   // no page: weights of -inf
          __syncwarp();
          far |= __any_sync(0xffffffffu, there && fabsf(v) > kFar);
          const bool gone = !__all_sync(0xffffffffu, there);
          page = page_next;
          scales = scales_of(page);
          page_next = page_of(t + 2);
          if (!(ok = wait_warp(&s_sfull[tile], sph & 1, abort_flag, err))) break;
          ++sph;
          tc_fence_after();
          if (frees) {
            mbar_arrive(&s_kempty[kv & 1]);
            if (t > p.t0) mbar_arrive(&s_vempty[~kv & 1]);
          }
          if (warp_live) {
            const int j0 = t * kTile;
            const bool masked = gone || partly(part, t);
            // keys j0 + x with x in [x0, x1) are the row's; groups without a page are nobody's
            const int x1 = min(place + 1, p.len) - j0;
            const int x0 = a.window > 0 ? place - a.window + 1 - j0 : -j0;
            // The weights are taken with the M that there is, from one reading of S, and stand if none
            // passes 2^8. Tiles where that is not to be expected, with hidden keys, or with value scales
            // far apart take two, and weights as squares: x = 2^((s f + v - M) / 2), x x of the values and
            // (x / v_scale) x of the sum, which a quiet page's x x below the least float would lose.
            bool twice = masked || far || t == p.t0 || __any_sync(0xffffffffu, fabsf(M) > 1e6f);
            if (!twice) {
              uint32_t w[64];
              float most = -INFINITY, sum = L;
#pragma unroll
              for (int ch = 0; ch < 4; ++ch) {
                float s[32];
                tmem_ld32(s_col + ch * 32, s);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const float4 c = s_coef[warp][2 * ch + h];
                  const float f = c.x * rowf, d = c.y - M;
                  const uint64_t ff = pair(f, f), dd = pair(d, d);
                  uint64_t acc = 0;
#pragma unroll
                  for (int x = 0; x < 16; x += 2) {
                    float e0, e1;
                    unpair(fma2(pair(s[16 * h + x], s[16 * h + x + 1]), ff, dd), e0, e1);
                    most = max3(most, e0, e1);
                    e0 = exp2_approx(e0), e1 = exp2_approx(e1);
                    acc = add2(acc, pair(e0, e1));
                    w[ch * 16 + h * 8 + x / 2] = pack_f16(e0, e1);
                  }
                  float l0, l1;
                  unpair(acc, l0, l1);
                  sum = fmaf(c.z, l0 + l1, sum);
                }
              }
              twice = __any_sync(0xffffffffu, most > kLazy);
              if (!twice) {
                L = sum;
#pragma unroll
                for (int ch = 0; ch < 4; ++ch) tc_st16(s_col + ch * 16, *reinterpret_cast<const uint32_t(*)[16]>(w + ch * 16));
              }
            }
            if (__builtin_expect(twice, 0)) {
              // the largest s f + v of the row in this tile (f >= 0: from each group's largest s; a group
              // without one may give NaN, which fmaxf passes over)
              float top = kNoMax;
#pragma unroll 1
              for (int ch = 0; ch < 4; ++ch) {
                float s[32];
                tmem_ld32(s_col + ch * 32, s);
                const float4 c0 = s_coef[warp][2 * ch], c1 = s_coef[warp][2 * ch + 1];
                if (masked && TREE) hide_bits(s, seen_from(j0 + ch * 32), c0.w > 0.0f, c1.w > 0.0f);
                if (masked && !TREE) hide(s, x0 - ch * 32, x1 - ch * 32, c0.w > 0.0f, c1.w > 0.0f);
                top = fmaxf(top, fmaf(max16(s), c0.x * rowf, c0.y));
                top = fmaxf(top, fmaf(max16(s + 16), c1.x * rowf, c1.y));
              }
              if (__any_sync(0xffffffffu, top > M + kLazy)) {
                // (the sum may be far from 1: its factor in two halves)
                const float to = fmaxf(M, top), half = exp2_approx(0.5f * (M - to)), keep = half * half;
                M = to;
                L = L * half * half;
                if (t > p.t0) {
#pragma unroll 1
                  for (int i = 0; i < D / 16; ++i) {
                    float o[16];
                    tmem_ld16(o_col + i * 16, o);
#pragma unroll
                    for (int x = 0; x < 16; ++x) o[x] *= keep;
                    tc_st16(o_col + i * 16, *reinterpret_cast<const uint32_t(*)[16]>(o));
                  }
                }
              }
              // scores so large that their rounding alone could pass 2^8 end there
              const float cap = __any_sync(0xffffffffu, fabsf(M) > 1e6f && M > kNoMax) ? 0.5f * kLazy : INFINITY;
              // weights; columns 16 ch .. of P lie over columns of S that are already read
#pragma unroll 1
              for (int ch = 0; ch < 4; ++ch) {
                float s[32];
                uint32_t w[16];
                tmem_ld32(s_col + ch * 32, s);
                const float4 c0 = s_coef[warp][2 * ch], c1 = s_coef[warp][2 * ch + 1];
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const float f = 0.5f * (h ? c1.x : c0.x) * rowf, d = 0.5f * ((h ? c1.y : c0.y) - M);
                  const uint64_t ff = pair(f, f), dd = pair(d, d);
#pragma unroll
                  for (int x = 16 * h; x < 16 * h + 16; x += 2) unpair(fma2(pair(s[x], s[x + 1]), ff, dd), s[x], s[x + 1]);
                }
                // hidden as exponents: a factor that underflows to 0 would make NaN of a score of -inf
                if (masked && TREE) hide_bits(s, seen_from(j0 + ch * 32), c0.w > 0.0f, c1.w > 0.0f);
                if (masked && !TREE) hide(s, x0 - ch * 32, x1 - ch * 32, c0.w > 0.0f, c1.w > 0.0f);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const float inv = h ? c1.z : c0.z;
                  const uint64_t ii = pair(inv, inv);
                  uint64_t acc = 0;
#pragma unroll
                  for (int x = 0; x < 16; x += 2) {
                    float e0 = s[16 * h + x], e1 = s[16 * h + x + 1];
                    e0 = e0 > cap ? cap : e0, e1 = e1 > cap ? cap : e1;
                    const uint64_t xx = pair(exp2_approx(e0), exp2_approx(e1));
                    acc = fma2(mul2(xx, ii), xx, acc);
                    unpair(mul2(xx, xx), e0, e1);
                    w[h * 8 + x / 2] = pack_f16(e0, e1);
                  }
                  float l0, l1;
                  unpair(acc, l0, l1);
                  L += l0 + l1;
                }
                tc_st16(s_col + ch * 16, w);
              }
            }
            tmem_wait_st();
          }
          if (partly(part, t)) {
            if (!(ok = wait_warp(&s_vfull[kv & 1], (kv >> 1) & 1, abort_flag, err))) break;
            const uint32_t bad = lane < kConvert / 32 ? s_nan[kv & 1][lane] : 0;
            if (__any_sync(0xffffffffu, bad != 0) && lane == 0 && s_nan_from[warp] > t) s_nan_from[warp] = t;
          }
          if (warp == 1 && !(ok = wait_warp(&s_vfull[kv & 1], (kv >> 1) & 1, abort_flag, err))) break;
          ++kv;
          if (warp == 2 && t + 1 < p.t1 && !(ok = wait_warp(&s_kfull[kv & 1], (kv >> 1) & 1, abort_flag, err))) break;
          tc_fence_before();
          warp_arrive(&s_pfull[tile]);
        }
        if (ok && (ok = wait_warp(&s_sfull[tile], sph & 1, abort_flag, err))) {
          ++sph;
          tc_fence_after();
          if (frees) mbar_arrive(&s_vempty[~kv & 1]);
        }
      } else if (nt > 0) {
        kv += nt;
      }
      if (!ok) break;
      // ---- the rows' results ----
      const bool whole = p.opens && p.closes, mine = r < p.R;
      const float inv = L > 0.0f ? 1.0f / L : L;           // 0 stays 0, NaN stays NaN
      auto stage8 = [&](int d, const float* v, float k) {  // values d..d+7 of the row
        float f[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) f[x] = v[x] * k;
        *column_at(r, d / 8) = bf16 ? pack8<MOE_DTYPE_BF16>(f) : pack8<MOE_DTYPE_F16>(f);
      };
      auto store_rows = [&] {                              // the warp's staged rows
        const uint64_t dst = reinterpret_cast<uint64_t>(a.out + row * a.out_stride + (int64_t)hq * D);
        __syncwarp();
#pragma unroll 4
        for (int k = 0; k < kLanes; ++k) {
          const int from = kRows * k + sub;
          const uint64_t at = __shfl_sync(0xffffffffu, dst, from);
          if (r - lane + from < p.R) reinterpret_cast<uint4*>(at)[col] = *column_at(r - lane + from, col);
        }
        __syncwarp();
      };
      auto store_lse = [&](float top, float sum) {
        if (a.lse)
          a.lse[row * a.q_heads + hq] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
      };
      const int slot = 2 * blockIdx.x + (p.opens ? 1 : 0);
      if (live) {
#pragma unroll 1
        for (int i = 0; i < D / 32; ++i) {
          float o[32];
          if (nt > 0 && warp_live) {
            tmem_ld32(o_col + i * 32, o);
          } else {
#pragma unroll
            for (int x = 0; x < 32; ++x) o[x] = 0.0f;
          }
          if (whole) {
#pragma unroll
            for (int x = 0; x < 32; x += 8) stage8(i * 32 + x, o + x, inv);
          } else if (mine) {
#pragma unroll
            for (int x = 0; x < 32; x += 4)
              part_rows[((size_t)slot * (D / 4) + i * 8 + x / 4) * kBlock + r] =
                  make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
          }
        }
        __syncwarp();
        if (nt > 0 && s_nan_from[warp] < p.t1 && mine) {
          // NaN codes kept out of the products, from the pages, into the row if it sees them
          const Partly part = partly_seen<TREE>(p, group, a.window);
          const int32_t* table = a.b.page_table + (int64_t)p.b * a.b.table_stride;
          const int j1 = min(TREE ? p.len : min(place + 1, p.len), p.t1 * kTile);
          const int from = TREE ? lo : a.window > 0 ? place - a.window + 1 : 0;
#pragma unroll 1
          for (int j = max(s_nan_from[warp] * kTile, from); j < j1; ++j) {
            if (!partly(part, j / kTile)) {                // every row sees this tile: its NaN are there
              j = part.from * kTile - 1;
              continue;
            }
            if (TREE && !(seen_from(j) & 1)) continue;
            const int page = table[j >> log_p];
            if (page < 0 || page >= a.c.num_pages) continue;
            each_nan<D>(a.c.v_codes + page * a.c.page_stride + ((int64_t)p.head * P + (j & (P - 1))) * D, [&](int d) {
              if (whole) reinterpret_cast<uint16_t*>(column_at(r, d / 8))[d % 8] = 0x7fff;      // of either type
              else reinterpret_cast<float*>(&part_rows[((size_t)slot * (D / 4) + d / 4) * kBlock + r])[d % 4] = NAN;
            });
          }
        }
        if (whole) store_rows();
        if (mine && whole) store_lse(M, L);
        if (mine && !whole) {
          stats[(size_t)slot * 2 * kBlock + r] = M;
          stats[((size_t)slot * 2 + 1) * kBlock + r] = L;
        }
        tc_fence_before();
      }
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
        if (s_last && warp_live) {
          __threadfence();
          auto slot_of = [&](int i) { return (size_t)2 * (p.c0 + i) + (i == 0); };
          float top = kNoMax, sum = 0.0f;
#pragma unroll 2
          for (int i = 0; i < p.np; ++i) top = fmaxf(top, __ldcg(stats + slot_of(i) * 2 * kBlock + r));
#pragma unroll 2
          for (int i = 0; i < p.np; ++i) {
            const float half = exp2_approx(0.5f * (__ldcg(stats + slot_of(i) * 2 * kBlock + r) - top));
            sum = fmaf(__ldcg(stats + (slot_of(i) * 2 + 1) * kBlock + r) * half, half, sum);
          }
          const float k1 = sum > 0.0f ? 1.0f / sum : sum;
#pragma unroll 1
          for (int d = 0; d < D; d += 32) {
            float v[32];
#pragma unroll
            for (int x = 0; x < 32; ++x) v[x] = 0.0f;
#pragma unroll 2
            for (int i = 0; i < p.np; ++i) {
              const float k = exp2_approx(__ldcg(stats + slot_of(i) * 2 * kBlock + r) - top);
              float4 o[8];
#pragma unroll
              for (int x = 0; x < 8; ++x) o[x] = __ldcg(part_rows + (slot_of(i) * (D / 4) + d / 4 + x) * kBlock + r);
#pragma unroll
              for (int x = 0; x < 8; ++x) {
                v[4 * x] = fmaf(o[x].x, k, v[4 * x]), v[4 * x + 1] = fmaf(o[x].y, k, v[4 * x + 1]);
                v[4 * x + 2] = fmaf(o[x].z, k, v[4 * x + 2]), v[4 * x + 3] = fmaf(o[x].w, k, v[4 * x + 3]);
              }
            }
#pragma unroll
            for (int x = 0; x < 32; x += 8) stage8(d + x, v + x, k1);
          }
          store_rows();
          if (mine) store_lse(top, sum);
        }
        if (!(ok = meet())) break;             // s_last is read before it is set again
      }
    }
    if (tid == 0) s_issue = make_int2(0, 0);
    if (warp < 4) warp_arrive(&s_qfull[0]);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 16)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(512));
}

template <int D, bool TREE>
cudaError_t launch_prompt(const AttentionArgs& a, int min_rows, char* ws, cudaStream_t s) {
  constexpr int smem = 1024 + Smem<D>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(prompt_kernel<D, TREE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int grid = num_sms() < kPromptMaxGrid ? num_sms() : kPromptMaxGrid;
  prompt_kernel<D, TREE><<<grid, kThreads, smem, s>>>(a, min_rows, ws);
  return cudaGetLastError();
}

}  // namespace

size_t prompt_attention_ws_bytes(int head_dim) {
  return align_up(kRowsAt + (size_t)2 * kPromptMaxGrid * kBlock * head_dim * 4);
}

cudaError_t launch_prompt_attention(const AttentionArgs& a, int min_rows, size_t ws_at, cudaStream_t s) {
  char* ws = a.ws + ws_at;
  if (a.tree)
    return a.c.head_dim == 64 ? launch_prompt<64, true>(a, min_rows, ws, s) : launch_prompt<128, true>(a, min_rows, ws, s);
  return a.c.head_dim == 64 ? launch_prompt<64, false>(a, min_rows, ws, s) : launch_prompt<128, false>(a, min_rows, ws, s);
}

}  // namespace moe
