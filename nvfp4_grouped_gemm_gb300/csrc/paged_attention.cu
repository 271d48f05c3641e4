// Causal attention of new tokens over the paged 8-bit cache (moe_attention_paged_e4m3), the form
// for few rows; prompt_attention.cu has the one for many.
//
// A sequence's n new tokens and the G query heads that share a key head are n*G rows over the
// same keys and values; a segment is (sequence, key head, block of 8*NT such rows). Its keys
// are cut into steps of STEP tokens, and all segments' steps form one line that the grid cuts
// into equal pieces, so a batch of very different lengths loads every SM alike. A CTA whose
// piece covers a whole segment writes its rows; the CTAs of a segment that was cut leave
// their rows' (maximum, sum, weighted values) in the workspace and the last of them to arrive
// joins them in the order of the pieces, so results do not depend on arrival.
//
// Inside a CTA the warps take the piece's steps in turn. Each streams its steps through a ring
// of its own (TMA boxes of E4M3 rows, swizzled so that the fragment reads below hit distinct
// banks), widens the codes to f16 in registers (exact) and multiplies with mma.sync m16n8k16
// (f32 accumulation), keys and values as the 16-row operand and the queries as its 8 columns, so
// that a conversion serves every query and few queries waste little:
//   S^T = K Q^T    lane 4g+c holds, of keys tau(g) and 8 + tau(g) of a half-step, 16 consecutive
//                  values at 16c of every 64; the four bytes of a word are its values of one
//                  k-step, and Q's fragments are laid out with the same permutation of k
//   O^T = V^T P^T  P^T's fragments are S^T's accumulators through an 8x8 transpose; V's pairs
//                  of keys for one value come from two rows' bytes by byte permutes
// With f = scale * k_scale * log2 e and v = log2 v_scale of a key's page, the weight that meets
// V's codes is w = 2^(s f + v - M) and the softmax sum adds w / v_scale, so the value scale
// costs nothing per element. Where scales lie far apart a quiet page's w may be below the least float
// while its share of the sum is not: from its first scale outside [2^-kFar, 2^kFar] on a warp takes
// half the exponent, x = 2^((s f + v - M) / 2), and adds (x / v_scale) x. M follows the running maximum of s f + v lazily: it moves only when
// a weight would pass 2^8, which leaves f16 weights their full precision and makes rescaling of
// the accumulators rare. w is rounded to f16 (2^-11), sums and accumulators are f32.
//
// For trees of drafted tokens (moe_attention_tree_e4m3) the same kernel asks a row's bits instead of
// its place in the steps that hold new tokens or a window's edge; the bits, cut to what the window
// leaves, lie in shared memory. One tree of 8 nodes after 1000 tokens, 16 query and 4 key
// heads of 128: 16.1 us; 32 of 6 to 48 nodes after 500 to 12000, 32 and 8 heads: 165 us, 115 of them here
// (the sequences below 73 rows) and the rest in the other form. Heads of 256 have no other form: 16 trees of
// 48 nodes after 4000, 16 and 4 heads, 274 us in passes of 16 rows, 32 of 4 nodes 65.5. Of the instances for
// trees the one of three row tiles at heads of 64 spills most (120 / 224 bytes; causal 44 / 60).
// The causal instances compute and pass nothing of this: with a tree's rows as an argument that they do not
// use the one-token forms spilled, and 64 sequences took 76.5 us where they take 75.7.
//
// Keys past a row's place, outside the window, in unused slots or in pages out of range get
// weight 0. V's bytes that are nobody's are replaced by 0 (they may be NaN codes). NaN codes of
// keys that some rows of the block see and others do not are kept out of the products and noted
// for the rows that see them, whose sums get NaN when the rows meet.
//
// Bound by the cache's bytes: 64 sequences of 100 to 16000 tokens, 32 query and 8 key heads of 128,
// one new token each: 73.9 us, 5.7 TB/s (0.84 of the copy rate). One sequence of 32767: 24.2 us, of
// which about 12 are fixed: the line's scan, the first keys and queries, the warps' rows meeting,
// and the join of the segment's pieces. With more rows the products and the softmax's instructions
// are the limit: 16 sequences, 8 tokens and 5 heads of 64 (40 rows): 47.8 us.
#include "serving.cuh"
#include "tma_sync.cuh"

namespace moe {
namespace {

constexpr int kMaxGrid = 512;              // partial slots of the workspace
constexpr int kMaxRows = 24;
constexpr float kNoMax = -1e30f;
constexpr float kLazy = 8.0f;
// With value scales within 2^(2 kFar) of one another a weight that is flushed to 0 (below 2^-126) has
// less than 2^-46 of the sum.
constexpr float kFar = 40.0f;
// What a segment costs beside its steps (queries, first copies, the warps' rows meeting), in
// steps: pieces of the line are equal with it counted.
constexpr int kSegmentCost = 12;

// Rows of a sequence (new tokens times query heads per key head) from which on it goes to the
// tensor-memory form of prompt_attention.cu. That form's time hardly depends on the rows up to 128,
// this one's grows with every 24. Sequences of 500 to 9000 tokens, 8 key heads, this form and the
// other, us: 16 sequences, D = 128: 64 rows 95 / 109, 96 rows 124 / 110; D = 64: 70 rows 63 / 70, 80
// rows 75 / 70; 64 sequences of up to 4000, 80 rows: D = 128 268 / 220, D = 64 172 / 149.
constexpr int kPromptRows = 73;
constexpr int kAllRows = 0x7fffffff;

// Workspace: error word; arrival counters [kMaxGrid]; partial maxima and sums
// [2 * kMaxGrid][2][kMaxRows]; partial rows f32 [2 * kMaxGrid][kMaxRows][D].
constexpr size_t kCountersAt = kAlign;
constexpr size_t kStatsAt = kCountersAt + kMaxGrid * 4;
constexpr size_t kRowsAt = kStatsAt + (size_t)2 * kMaxGrid * 2 * kMaxRows * 4;

template <int D_, int NT_, int WARPS_>
struct Shape {
  static constexpr int D = D_, NT = NT_, kWarps = WARPS_, kThreads = 32 * WARPS_;
  static constexpr int kStep = D == 256 ? 16 : 32;       // tokens per step
  static constexpr int kHalves = kStep / 16;
  static constexpr int kSubs = D == 256 ? 2 : 1;         // swizzled sub-tiles of a row
  static constexpr int kRowB = D == 64 ? 64 : 128;       // bytes of a sub-tile row
  static constexpr int kPlaneB = kStep * D;              // a step's K (or V) bytes
  static constexpr int kStageB = 2 * kPlaneB;
  static constexpr int kSlots = D == 64 ? 4 : NT > 2 ? 3 : 2;
  static constexpr int kCtas = WARPS_ > 4 ? 1 : NT * D > 256 || (NT == 2 && D == 128) ? 2 : 3;   // per SM
  static constexpr int kRows = 8 * NT;
  static constexpr int kRingB = kWarps * kSlots * kStageB;
  static constexpr int kMergeB = kWarps * kRows * D * 4; // aliases the ring
  static constexpr int kJoinB = kMaxGrid * kRows * 4;    // aliases the ring
  static constexpr int kBig0 = kRingB > kMergeB ? kRingB : kMergeB;
  static constexpr int kBigB = kBig0 > kJoinB ? kBig0 : kJoinB;
  static constexpr int kQB = kRows * D * 2;
  static constexpr int kSmem = 1024 + kBigB + kQB;
  static constexpr bool kQRegs = NT * D <= 128;          // query fragments stay in registers
};

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The 8x8 transpose of f16 pairs across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t word_of(const uint4& v, int m) {
  return m == 0 ? v.x : m == 1 ? v.y : m == 2 ? v.z : v.w;
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
template <class S, bool TREE>
__device__ __forceinline__ Seq read_seq(const AttentionArgs& a, int b, int group, uint32_t* err) {
  Seq q;
  q.row0 = min(max(a.b.q_offsets[b], 0), a.T);
  const int end = min(max(a.b.q_offsets[b + 1], q.row0), a.T);
  q.n = end - q.row0;
  if (q.n * group > a.max_rows) q.n = 0;       // the other form's
  q.len = a.b.seq_lens[b];
  q.start = q.len - q.n;
  const int cap = a.b.max_pages * a.c.page_size;
  if (q.n > 0 && (q.len < q.n || q.len > cap) && err) atomicOr(err, (uint32_t)MOE_DEVERR_PAGE);
  q.len = min(max(q.len, 0), cap);
  const int lo = a.window > 0 ? max(0, min(q.start - a.window + (TREE ? 0 : 1), q.len)) : 0;
  q.step0 = lo / S::kStep;
  q.steps = max((q.len + S::kStep - 1) / S::kStep - q.step0, 1);
  q.blocks = (q.n * group + S::kRows - 1) / S::kRows;
  return q;
}

// Sum of v over the block; the exclusive prefix of the calling thread in *before.
template <int WARPS>
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
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) base += s_sum[w];
    all += s_sum[w];
  }
  *before = base + x - v;
  return all;
}

// The factors of a warp's half-steps (16 tokens, which lie in one page), 32 of them at a time: lane l
// holds half-step l of the batch.
struct Keys {
  // (all 0 without a page) scale * k_scale * log2 e; log2 v_scale; 1 / v_scale, negative from the
  // warp's first far scale on
  float f, v, inv;
};

// A lane's share of a block of rows: query fragments, accumulators, and what the running softmax
// keeps for rows 2c and 2c+1 of each row tile.
template <class S>
struct Rows {
  uint4 Q[S::kQRegs ? S::NT : 1][S::kQRegs ? S::D / 32 : 1];
  float O[S::NT][S::D / 16][4];
  float M[S::NT][2], L[S::NT][2], rowf[S::NT][2];
  int place[S::NT][2];
};
// Where a lane reads a stage: half-step token of accumulator row g, of a fragment's columns 2c
// and 2c+1, and byte offsets of its keys' and values' 16-byte pieces.
struct Frag {
  int tau, tok_a, tok_b, koff0, koff1, voffa, voffb;
};
// A step's page factors per half, and whether the half's page is there.
template <int H>
struct StepKeys {
  float f[H], v[H], inv[H];
  bool good[H];
};

// What the rows of a block of trees see: of the tokens before the new ones those from lo[row] on, of the
// new ones those of bits[row][..].
template <bool TREE>
struct TreeRows {
  const uint32_t* bits;
  const int* lo;
  int start;                                   // place of the first new token
};
template <>
struct TreeRows<false> {};
__device__ __forceinline__ bool tree_sees(const TreeRows<true>& t, int row, int j) {
  const int c = j - t.start;
  if (c < 0) return j >= t.lo[row];
  return c < 32 * kMaxTreeWords && (t.bits[row * kMaxTreeWords + (c >> 5)] >> (c & 31) & 1) != 0;
}

// One step of STEP keys for all rows; `masked` where a key of it is hidden from a row or is not
// there, or a value scale is or was far from the others.
template <class S, bool masked, bool TREE>
__device__ __forceinline__ void take_step(Rows<S>& t, const Frag& f, const StepKeys<S::kHalves>& k,
                                          const char* st, const char* s_q, int lane, int j0, int len,
                                          int window, const TreeRows<TREE>& tree) {
  constexpr int D = S::D, NT = S::NT, H = S::kHalves;
  float sc[NT][H][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int x = 0; x < 4; ++x) sc[nt][h][x] = 0.0f;
#pragma unroll
  for (int j = 0; j < D / 64; ++j) {
    uint4 k0[H], k1[H];
#pragma unroll
    for (int h = 0; h < H; ++h) {
      const char* at_ = st + (j >> 1) * (S::kStep * 128) + h * 16 * S::kRowB + (j & 1 ? f.koff1 : f.koff0);
      k0[h] = *reinterpret_cast<const uint4*>(at_);
      k1[h] = *reinterpret_cast<const uint4*>(at_ + 8 * S::kRowB);
    }
#pragma unroll
    for (int m2 = 0; m2 < 2; ++m2) {
      uint4 qf[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        qf[nt] = S::kQRegs ? t.Q[S::kQRegs ? nt : 0][S::kQRegs ? 2 * j + m2 : 0]
                           : *reinterpret_cast<const uint4*>(s_q + ((2 * j + m2) * NT + nt) * 512 + lane * 16);
#pragma unroll
      for (int m1 = 0; m1 < 2; ++m1)
#pragma unroll
        for (int h = 0; h < H; ++h) {
          uint32_t a0, a1, a2, a3;
          widen4(word_of(k0[h], 2 * m2 + m1), a0, a2);
          widen4(word_of(k1[h], 2 * m2 + m1), a1, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma(sc[nt][h], a0, a1, a2, a3, m1 ? qf[nt].z : qf[nt].x, m1 ? qf[nt].w : qf[nt].y);
        }
    }
  }

  // weights: s f + v - M, for all row tiles before one vote on whether M has to move
  bool move = false;
  float top[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    top[nt][0] = top[nt][1] = -INFINITY;
    const float base[2] = {t.M[nt][0] == kNoMax ? 0.0f : t.M[nt][0], t.M[nt][1] == kNoMax ? 0.0f : t.M[nt][1]};
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int y = x & 1;
        sc[nt][h][x] = fmaf(sc[nt][h][x], k.f[h] * t.rowf[nt][y], k.v[h] - base[y]);
        if (masked) {
          const int j = j0 + h * 16 + (x >> 1) * 8 + f.tau, pl = t.place[nt][y];
          bool see;
          if constexpr (TREE) see = k.good[h] && j < len && tree_sees(tree, 8 * nt + 2 * (lane & 3) + y, j);
          else see = k.good[h] && j <= pl && j < len && (window == 0 || j > pl - window);
          if (!see) sc[nt][h][x] = -INFINITY;
        }
        top[nt][y] = fmaxf(top[nt][y], sc[nt][h][x]);
      }
#pragma unroll
    for (int y = 0; y < 2; ++y)
      move |= top[nt][y] > (t.M[nt][y] == kNoMax ? -INFINITY : kLazy);
  }
  if (__any_sync(0xffffffffu, move)) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) top[nt][y] = fmaxf(top[nt][y], __shfl_xor_sync(0xffffffffu, top[nt][y], o));
        const bool unset = t.M[nt][y] == kNoMax;           // no key of the row so far
        const float up = unset ? (top[nt][y] > -INFINITY ? top[nt][y] : 0.0f) : fmaxf(top[nt][y], 0.0f);
        // (the sum may be far from 1: its factor in two halves)
        const float half = unset ? 0.0f : exp2_approx(-0.5f * up), keep = half * half;
        if (!unset || top[nt][y] > -INFINITY) t.M[nt][y] = (unset ? 0.0f : t.M[nt][y]) + up;
        t.L[nt][y] = t.L[nt][y] * half * half;
#pragma unroll
        for (int n = 0; n < D / 16; ++n) t.O[nt][n][y] *= keep, t.O[nt][n][2 + y] *= keep;
#pragma unroll
        for (int h = 0; h < H; ++h)
#pragma unroll
          for (int x = y; x < 4; x += 2) sc[nt][h][x] -= up;
      }
  }
  uint32_t pb[NT][H][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int h = 0; h < H; ++h) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        sc[nt][h][x] = exp2_approx(masked ? 0.5f * sc[nt][h][x] : sc[nt][h][x]);
        if (masked) {
          t.L[nt][x & 1] = fmaf(sc[nt][h][x] * fabsf(k.inv[h]), sc[nt][h][x], t.L[nt][x & 1]);
          sc[nt][h][x] *= sc[nt][h][x];
        }
      }
      if (!masked) {
#pragma unroll
        for (int y = 0; y < 2; ++y) t.L[nt][y] = fmaf(k.inv[h], sc[nt][h][y] + sc[nt][h][2 + y], t.L[nt][y]);
      }
      pb[nt][h][0] = transpose8(pack_f16(sc[nt][h][0], sc[nt][h][1]));
      pb[nt][h][1] = transpose8(pack_f16(sc[nt][h][2], sc[nt][h][3]));
    }

  // values
#pragma unroll
  for (int h = 0; h < H; ++h)
#pragma unroll
    for (int s = 0; s < S::kSubs; ++s) {
      constexpr int kWords = D == 64 ? 2 : 4;
      uint32_t x[4][kWords];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const char* at_ = st + s * (S::kStep * 128) + (h * 16 + (r >> 1) * 8) * S::kRowB + (r & 1 ? f.voffb : f.voffa);
        if (D == 64) {
          const uint2 w = *reinterpret_cast<const uint2*>(at_);
          x[r][0] = w.x, x[r][1] = w.y;
        } else {
          const uint4 w = *reinterpret_cast<const uint4*>(at_);
          x[r][0] = w.x, x[r][1] = w.y, x[r][kWords - 2] = w.z, x[r][kWords - 1] = w.w;
        }
        if (masked) {
          const bool there = k.good[h] && j0 + h * 16 + (r >> 1) * 8 + (r & 1 ? f.tok_b : f.tok_a) < len;
#pragma unroll
          for (int i = 0; i < kWords; ++i) x[r][i] = there ? x[r][i] : 0u;
        }
      }
#pragma unroll
      for (int m = 0; m < kWords; ++m) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t a0, a1, a2, a3;
          widen4(__byte_perm(x[0][m], x[1][m], e ? 0x7362 : 0x5140), a0, a1);
          widen4(__byte_perm(x[2][m], x[3][m], e ? 0x7362 : 0x5140), a2, a3);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma(t.O[nt][s * 8 + 2 * m + e], a0, a1, a2, a3, pb[nt][h][0], pb[nt][h][1]);
        }
      }
    }
}

// Makes the NaN codes among a masked step's values finite and sets the bits of those that the warp's rows
// (at places[row]) see, bits[row][value]; *any: whether some were found (0: the bits are not valid yet).
// `there`: the lane's key is (a lane per key, at D = 256 two). A pass and a call of its own, which leaves
// nothing in registers (64 sequences of 100 to 16000 tokens 73.9 us; with the pages read again at the end
// instead of bits 75.0).
template <class S, bool TREE>
__device__ __noinline__ void keep_nan_out(char* st, int lane, bool there, int j0, int window, const int* places,
                                          uint32_t* bits, volatile int* any, TreeRows<TREE> tree) {
  constexpr int D = S::D, kWords = D / 32, kChunks = S::kPlaneB / 16 / 32;
  const int sub = D == 256 ? lane >> 4 : 0, tok = D == 256 ? lane & 15 : lane;
  char* row = st + S::kPlaneB + sub * (S::kStep * 128) + tok * S::kRowB;
  uint32_t bad = 0;
#pragma unroll 2
  for (int i = 0; i < kChunks; ++i) {
    const uint4 v = *reinterpret_cast<const uint4*>(row + ((i + lane) % kChunks) * 16);
    bad |= e4m3_nan_bits(v.x) | e4m3_nan_bits(v.y) | e4m3_nan_bits(v.z) | e4m3_nan_bits(v.w);
  }
  if (!__any_sync(0xffffffffu, there && bad != 0)) return;
  const bool first = *any == 0;
  __syncwarp();
#pragma unroll 1
  for (int i = lane; first && i < S::kRows * kWords; i += 32) bits[i] = 0;
  if (lane == 0) *any = 1;
  __syncwarp();
  const int swz = D == 64 ? (tok >> 1) & 3 : tok & 7;
#pragma unroll 1
  for (int i = 0; i < kChunks * 4; ++i) {        // words of the row as they lie
    uint32_t& w = reinterpret_cast<uint32_t*>(row)[i];
    const uint32_t m = e4m3_nan_bits(w);
    if (m == 0) continue;
    w &= ~(m >> 7);                              // with a weight of 0 where the key is not seen
    const uint32_t four = (m >> 7 & 1) | (m >> 14 & 2) | (m >> 21 & 4) | (m >> 28 & 8);
    const int d = sub * 128 + ((i / 4) ^ swz) * 16 + (i % 4) * 4;
#pragma unroll 1
    for (int r = 0; there && r < S::kRows; ++r) {
      bool see;
      if constexpr (TREE) see = tree_sees(tree, r, j0 + tok);
      else see = j0 + tok <= places[r] && (window == 0 || j0 + tok > places[r] - window);
      if (see) atomicOr(bits + r * kWords + d / 32, four << (d % 32));
    }
  }
  // plain writes to the ring's memory come before the next copies into it
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}

template <class S, bool TREE>
__global__ void __launch_bounds__(S::kThreads, S::kCtas)
attention_kernel(const __grid_constant__ AttentionArgs a, const __grid_constant__ CUtensorMap kmap,
                 const __grid_constant__ CUtensorMap vmap) {
  constexpr int D = S::D, NT = S::NT, H = S::kHalves, kWarps = S::kWarps, kThreads = S::kThreads;
  constexpr int kPer = 32 / H;                 // steps per batch of keys
  extern __shared__ char smem_raw[];
  __shared__ uint64_t s_full[kWarps * S::kSlots];
  __shared__ long long s_sum[kWarps];
  __shared__ int s_seq;
  __shared__ long long s_first;
  __shared__ volatile int s_abort;
  __shared__ int s_place[S::kRows];
  __shared__ float s_rowf[S::kRows], s_m[kWarps][S::kRows], s_l[kWarps][S::kRows];
  __shared__ int s_last;
  __shared__ volatile char s_far[kWarps][32];  // whether the warp has met a far value scale: a lane's own
  __shared__ volatile int s_nan[kWarps];       // whether the warp kept NaN codes out, and which of its sums they belong in
  __shared__ uint32_t s_nan_bits[kWarps][S::kRows * (D / 32)];
  __shared__ uint32_t s_bits[TREE ? S::kRows * kMaxTreeWords : 1];
  __shared__ int s_lo[TREE ? S::kRows : 1];
  char* big = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  char* s_q = big + S::kBigB;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, c = lane & 3;
  const bool bf16 = a.dtype == MOE_DTYPE_BF16;
  uint32_t* err = reinterpret_cast<uint32_t*>(a.ws);
  uint32_t* counters = reinterpret_cast<uint32_t*>(a.ws + kCountersAt);
  float* stats = reinterpret_cast<float*>(a.ws + kStatsAt);
  float* part = reinterpret_cast<float*>(a.ws + kRowsAt);
  const int heads = a.c.kv_heads, group = a.q_heads / heads, P = a.c.page_size;

  for (int i = tid; i < kWarps * S::kSlots; i += kThreads) mbar_init(&s_full[i], 1);
  if (tid == 0) s_abort = 0;
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");

  // This CTA's piece of the line.
  // Trees, few segments: each is made up to whole pieces of the least length, so that no CTA has two
  // one after the other. 5 trees of 2 nodes, 14 query and 2 key heads of 64: 9.5 us against 15.6; one of
  // 16 after 3000 tokens, 16 and 4 heads of 128: 21.6 against 26.0.
  constexpr int kLeast = kWarps + kSegmentCost;
  bool whole = false;
  auto length_of = [&](const Seq& q) {
    const int length = q.steps + kSegmentCost;
    return TREE && whole ? (length + kLeast - 1) / kLeast * kLeast : length;
  };
  auto line_of = [&](const Seq& q) { return (long long)length_of(q) * q.blocks * heads; };
  long long total = 0, mine = 0, at = 0;
  for (int b0 = 0; b0 < a.b.B; b0 += kThreads) {
    mine = 0;
    if (b0 + tid < a.b.B) mine = line_of(read_seq<S, TREE>(a, b0 + tid, group, blockIdx.x == 0 ? err : nullptr));
    total += block_scan<kWarps>(mine, s_sum, &at);
  }
  if (TREE && a.b.B <= kThreads && total > 0 && total <= (long long)gridDim.x * kLeast) {
    whole = true;
    mine = 0;
    if (tid < a.b.B) mine = line_of(read_seq<S, TREE>(a, tid, group, nullptr));
    total = block_scan<kWarps>(mine, s_sum, &at);
    if (total > (long long)gridDim.x * kLeast) {
      whole = false;
      mine = 0;
      if (tid < a.b.B) mine = line_of(read_seq<S, TREE>(a, tid, group, nullptr));
      total = block_scan<kWarps>(mine, s_sum, &at);
    }
  }
  long long per = (total + gridDim.x - 1) / gridDim.x;
  if (per < kLeast) per = kLeast;
  const long long begin = per * blockIdx.x, end = min(begin + per, total);
  if (begin >= end) {
    pdl_wait();
    return;
  }
  if (a.b.B <= kThreads) {
    if (mine > 0 && at <= begin && begin < at + mine) s_seq = tid, s_first = at;
  } else {
    long long base = 0;
    for (int b0 = 0; b0 < a.b.B; b0 += kThreads) {
      mine = 0;
      if (b0 + tid < a.b.B) mine = line_of(read_seq<S, TREE>(a, b0 + tid, group, nullptr));
      const long long sum = block_scan<kWarps>(mine, s_sum, &at);
      if (mine > 0 && base + at <= begin && begin < base + at + mine) s_seq = b0 + tid, s_first = base + at;
      base += sum;
    }
  }
  __syncthreads();
  int b = s_seq;
  long long first = s_first;                   // the line's place of sequence b's first step
  Seq q = read_seq<S, TREE>(a, b, group, nullptr);

  char* ring = big + warp * S::kSlots * S::kStageB;
  uint64_t* full = s_full + warp * S::kSlots;
  int islot = 0, tslot = 0;                    // next slot to fill, to take
  uint32_t tphase = 0;
  int in_flight = 0;
  // half-step token of accumulator row g, and of a fragment's columns 2c and 2c+1
  const int tau = D == 64 ? g : (g >> 1) + 4 * (g & 1);
  const int tok_a = D == 64 ? 2 * c : c, tok_b = D == 64 ? 2 * c + 1 : c + 4;
  const int kx = D == 64 ? (tau >> 1) & 3 : tau;
  const int koff0 = tau * S::kRowB + ((c ^ kx) * 16);
  const int koff1 = tau * S::kRowB + (((4 + c) ^ kx) * 16);
  const int vch = D == 64 ? g >> 1 : (g >> 1) + 4 * (g & 1);
  const int vxa = D == 64 ? (tok_a >> 1) & 3 : tok_a, vxb = D == 64 ? (tok_b >> 1) & 3 : tok_b;
  const int voffa = S::kPlaneB + tok_a * S::kRowB + ((vch ^ vxa) * 16) + (D == 64 ? (g & 1) * 8 : 0);
  const int voffb = S::kPlaneB + tok_b * S::kRowB + ((vch ^ vxb) * 16) + (D == 64 ? (g & 1) * 8 : 0);

  const Frag frag = {tau, tok_a, tok_b, koff0, koff1, voffa, voffb};

  for (long long pos = begin; pos < end;) {
    while (pos >= first + line_of(q)) {
      first += line_of(q);
      q = read_seq<S, TREE>(a, ++b, group, nullptr);
    }
    const int length = length_of(q);
    const long long in_seq = pos - first;
    const int seg = (int)(in_seq / length);
    const long long seg_at = first + (long long)seg * length;
    const int st0 = max(0, (int)(pos - seg_at) - kSegmentCost);
    const int upto = (int)min((long long)length, end - seg_at);
    int st1 = upto - kSegmentCost;
    if constexpr (TREE) st1 = min(st1, q.steps);               // (not the steps that make a segment up to whole pieces)
    pos = seg_at + upto;
    if (st1 <= st0) continue;                  // only the segment's fixed cost fell to this CTA
    const int head = seg / q.blocks, block = seg % q.blocks;
    const int R = min(S::kRows, q.n * group - block * S::kRows);
    // rows' places: row r of the block belongs to token (block * kRows + r) / group
    const int tok_first = block * S::kRows / group, tok_last = (block * S::kRows + R - 1) / group;
    const int place_lo = q.start + tok_first, place_hi = q.start + tok_last;
    // steps this block of rows can see at all
    const int hi = TREE ? q.len : min(q.len, place_hi + 1);
    const int lo = a.window > 0 ? max(0, TREE ? q.start - a.window : place_lo - a.window + 1) : 0;
    const int w0 = max(q.step0 + st0, lo / S::kStep);
    const int w1 = min(q.step0 + st1, (max(hi, 0) + S::kStep - 1) / S::kStep);

    // ---- this warp's stream ----
    const int count = w1 > w0 + warp ? (w1 - w0 - warp + kWarps - 1) / kWarps : 0;
    // A batch's pages are read a batch ahead, its scales as its first copy is issued; they become
    // factors when its first step is taken.
    Keys cur = {0.f, 0.f, 0.f};
    s_far[warp][lane] = 0;
    int page_of_lane = -1, page_ahead = -1;
    float k_scale = 0.0f, v_scale = 0.0f;
    auto key_of = [&](int batch) {             // the lane's first key of a batch, -1: none
      const int i = batch * kPer + lane / H, j = (w0 + warp + i * kWarps) * S::kStep + (lane % H) * 16;
      return i < count && j < q.len ? j : -1;
    };
    auto read_page = [&](int batch) {
      const int j = key_of(batch);
      return (int)load_ahead(a.b.page_table + (int64_t)b * a.b.table_stride + j / P, j >= 0, 0xffffffffu);
    };
    auto load_keys = [&](int batch) {
      if (batch == 0) page_ahead = read_page(0);
      page_of_lane = page_ahead;
      page_ahead = read_page(batch + 1);
      if (page_of_lane < 0 || page_of_lane >= a.c.num_pages) {
        if (key_of(batch) >= 0) atomicOr(err, (uint32_t)MOE_DEVERR_PAGE);
        page_of_lane = -1;
      }
      const int64_t sc = (int64_t)page_of_lane * heads + head;
      k_scale = __uint_as_float(load_ahead(a.c.k_scales + sc, page_of_lane >= 0, 0u));
      v_scale = __uint_as_float(load_ahead(a.c.v_scales + sc, page_of_lane >= 0, 0u));
    };
    auto factors = [&] {
      Keys k = {0.f, 0.f, 0.f};
      if (page_of_lane >= 0) {
        const float vs = fminf(fmaxf(v_scale, 0x1p-100f), 0x1p120f);
        k.f = a.scale * 1.4426950408889634f * k_scale;
        k.v = log2f(vs);
        k.inv = __fdividef(1.0f, vs);
      }
      if (__any_sync(0xffffffffu, fabsf(k.v) > kFar)) s_far[warp][lane] = 1;
      if (s_far[warp][lane]) k.inv = -k.inv;
      return k;
    };
    int have = 0;                              // key batches loaded
    auto issue = [&](int i) {                  // all lanes: step i of this warp into the next slot
      const int batch = i / kPer, src = (i % kPer) * H;
      if (batch >= have) {
        load_keys(batch);
        ++have;
      }
      int page[H];
#pragma unroll
      for (int h = 0; h < H; ++h) page[h] = __shfl_sync(0xffffffffu, page_of_lane, src + h);
      if (lane == 0) {
        char* st = ring + islot * S::kStageB;
        uint64_t* bar = &full[islot];
        const int j = (w0 + warp + i * kWarps) * S::kStep;
        const int row = head * P + j % P;
        if (P >= S::kStep) {                   // one box per plane and sub-tile
          if (page[0] >= 0) {
            mbar_expect_tx(bar, S::kStageB);
#pragma unroll
            for (int s = 0; s < S::kSubs; ++s) {
              tma_load_3d(st + s * (S::kStep * 128), &kmap, s * 128, row, page[0], bar);
              tma_load_3d(st + S::kPlaneB + s * (S::kStep * 128), &vmap, s * 128, row, page[0], bar);
            }
          } else {
            mbar_arrive(bar);
          }
        } else {                               // two pages of 16 tokens
          uint32_t bytes = 0;
#pragma unroll
          for (int h = 0; h < H; ++h) bytes += page[h] >= 0 ? S::kStageB / H : 0;
          mbar_expect_tx(bar, bytes);
#pragma unroll
          for (int h = 0; h < H; ++h) {
            if (page[h] < 0) continue;
            tma_load_3d(st + h * 16 * S::kRowB, &kmap, 0, head * P, page[h], bar);
            tma_load_3d(st + S::kPlaneB + h * 16 * S::kRowB, &vmap, 0, head * P, page[h], bar);
          }
        }
      }
      islot = islot + 1 == S::kSlots ? 0 : islot + 1;
      ++in_flight;
    };
    // ---- queries as B fragments: k-steps 2i and 2i+1 of row tile nt: lane 16 B. The warp's rows
    // come kAtOnce at a time, the first of them asked for before the keys' pages ----
    constexpr int kQuads = (D / 4 + 31) / 32, kMine = (S::kRows + kWarps - 1) / kWarps;
    constexpr int kAtOnce = kMine < 4 ? kMine : 4;
    uint2 qv[kAtOnce][kQuads];
    auto ask = [&](int i0) {
#pragma unroll
      for (int n = 0; n < kAtOnce; ++n) {
        const int r = warp + (i0 + n) * kWarps, rr = block * S::kRows + r;
        const uint16_t* src = a.q + (int64_t)(q.row0 + rr / group) * a.q_stride +
                              (int64_t)(head * group + rr % group) * D;
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
          const int u = lane + 32 * i;
          qv[n][i] = make_uint2(0, 0);
          if (r < R && u < D / 4) qv[n][i] = *reinterpret_cast<const uint2*>(src + 4 * u);
        }
      }
    };
    ask(0);
    if (lane == 0) s_nan[warp] = 0;
    if (tid < S::kRows) s_place[tid] = q.start + (block * S::kRows + tid) / group;
    if (TREE && tid < S::kRows) {
      uint32_t w[kMaxTreeWords];
      s_lo[tid] = tree_row(a, q.row0 + (block * S::kRows + tid) / group, tid < R, q.n, q.start, w);
#pragma unroll
      for (int i = 0; i < kMaxTreeWords; ++i) s_bits[tid * kMaxTreeWords + i] = w[i];
    }
    for (int i = 0; i < min(count, S::kSlots); ++i) issue(i);
#pragma unroll 1
    for (int i0 = 0; i0 < kMine; i0 += kAtOnce) {
      if (i0 > 0) ask(i0);
#pragma unroll
      for (int n = 0; n < kAtOnce; ++n) {
        const int r = warp + (i0 + n) * kWarps;
        if (r >= S::kRows) break;
        float v[kQuads][4];
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < kQuads; ++i)
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t bits = (x < 2 ? qv[n][i].x : qv[n][i].y) >> (16 * (x & 1)) & 0xffffu;
            v[i][x] = bf16 ? act_to_f32<MOE_DTYPE_BF16>(bits) : act_to_f32<MOE_DTYPE_F16>(bits);
            amax = fmaxf(amax, fabsf(v[i][x]));
          }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        // bf16 rows get the power of two that puts their largest magnitude below 2^15
        const int e = bf16 && amax < 3.4e38f ? f16_prescale_exp(amax) : 0;
        const float s1 = pow2f(-e / 2), s2 = pow2f(-e - (-e / 2));
        if (lane == 0) s_rowf[r] = pow2f(e);
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
          const int u = lane + 32 * i;
          if (u < D / 4) {
            const int ks = (u >> 4) * 4 + (u & 3), cc = (u >> 2) & 3;
            char* dst = s_q + ((ks >> 1) * NT + (r >> 3)) * 512 + ((r & 7) * 4 + cc) * 16 + (ks & 1) * 8;
            *reinterpret_cast<uint2*>(dst) =
                make_uint2(pack_f16(v[i][0] * s1 * s2, v[i][1] * s1 * s2),
                           pack_f16(v[i][2] * s1 * s2, v[i][3] * s1 * s2));
          }
        }
      }
    }
    __syncthreads();

    Rows<S> t;
    if (S::kQRegs) {
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          t.Q[S::kQRegs ? nt : 0][S::kQRegs ? i : 0] =
              *reinterpret_cast<const uint4*>(s_q + (i * NT + nt) * 512 + lane * 16);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int n = 0; n < D / 16; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) t.O[nt][n][x] = 0.0f;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int r = 8 * nt + 2 * c + y;
        t.M[nt][y] = kNoMax, t.L[nt][y] = 0.0f;
        t.rowf[nt][y] = s_rowf[r];
        t.place[nt][y] = s_place[r];
      }
    }

    TreeRows<TREE> tree;
    if constexpr (TREE) tree = {s_bits, s_lo, q.start};
    bool ok = true;
    for (int i = 0; i < count; ++i) {
      // every lane looks at the barrier itself; the bounded wait is for copies not there yet
      if (!__all_sync(0xffffffffu, mbar_try(&full[tslot], tphase)))
        ok = mbar_wait_warp(&full[tslot], tphase, &s_abort, err);
      if (!ok) break;
      const int j0 = (w0 + warp + i * kWarps) * S::kStep;
      const int src = (i % kPer) * H;
      // the newest batch is this step's: copies are issued fewer steps ahead than a batch has
      static_assert(S::kSlots <= kPer, "");
      if (src == 0) cur = factors();
      StepKeys<H> k;
      bool masked = j0 + S::kStep > (TREE ? q.start : place_lo + 1) || j0 + S::kStep > q.len;
      if (a.window > 0) masked |= j0 <= (TREE ? q.start + min(q.n, 32 * kMaxTreeWords) : place_hi) - a.window;
#pragma unroll
      for (int h = 0; h < H; ++h) {
        k.f[h] = __shfl_sync(0xffffffffu, cur.f, src + h);
        k.v[h] = __shfl_sync(0xffffffffu, cur.v, src + h);
        k.inv[h] = __shfl_sync(0xffffffffu, cur.inv, src + h);
        k.good[h] = k.inv[h] != 0.0f;
        masked |= !(k.inv[h] > 0.0f);
      }
      char* st = ring + tslot * S::kStageB;
      if (masked) {
        const bool there = (lane < 16 || H == 1 ? k.good[0] : k.good[H - 1]) && j0 + lane % S::kStep < q.len;
        keep_nan_out<S, TREE>(st, lane, there, j0, a.window, s_place, s_nan_bits[warp], &s_nan[warp], tree);
        take_step<S, true, TREE>(t, frag, k, st, s_q, lane, j0, q.len, a.window, tree);
      } else {
        take_step<S, false, TREE>(t, frag, k, st, s_q, lane, j0, q.len, a.window, tree);
      }
      if (++tslot == S::kSlots) tslot = 0, tphase ^= 1;
      --in_flight;
      __syncwarp();
      if (i + S::kSlots < count) issue(i + S::kSlots);
    }
    if (!ok) {
      // gave up: let this warp's copies in flight land (bounded) before the CTA leaves
      for (; in_flight > 0; --in_flight) {
        const uint64_t t0 = global_ns();
        while (!mbar_try(&full[tslot], tphase) && global_ns() - t0 < 100000000ull) {
        }
        if (++tslot == S::kSlots) tslot = 0, tphase ^= 1;
      }
    }

    // ---- the warps' rows meet ----
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) t.L[nt][y] += __shfl_xor_sync(0xffffffffu, t.L[nt][y], o);
        if (g == 0) {
          s_m[warp][8 * nt + 2 * c + y] = t.M[nt][y];
          s_l[warp][8 * nt + 2 * c + y] = t.L[nt][y];
        }
      }
    __syncthreads();                           // also: every warp is done with the ring
    if (s_abort) break;                        // the same for the whole block
    float* merge = reinterpret_cast<float*>(big);
    // 16-byte units of a row are permuted so that a quarter warp's stores differ in bank
    auto unit_of = [](int r, int d) {
      const int u = d / 4, cc = (r & 7) >> 1;
      return D == 64 ? u ^ ((cc & 1) | (cc >> 1) << 2) : u ^ (cc | ((u >> 4) & 1) << 2);
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int r = 8 * nt + 2 * c + y;
        float top = kNoMax;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
        const float keep = exp2_approx(t.M[nt][y] - top);
#pragma unroll
        for (int n = 0; n < D / 16; n += 2) {  // values 2n .. 2n+3 of a run of 16 (D = 64: 8)
          const int d = D == 64 ? g * 8 + 2 * n : (n / 8) * 128 + vch * 16 + 2 * (n % 8);
          *reinterpret_cast<float4*>(merge + ((size_t)warp * S::kRows + r) * D + unit_of(r, d) * 4) =
              make_float4(t.O[nt][n][y] * keep, t.O[nt][n][2 + y] * keep, t.O[nt][n + 1][y] * keep,
                          t.O[nt][n + 1][2 + y] * keep);
        }
      }
    __syncwarp();
    if (s_nan[warp]) {
#pragma unroll 1
      for (int i = lane; i < S::kRows * D; i += 32)
        if (s_nan_bits[warp][i / 32] >> (i % 32) & 1)
          merge[((size_t)warp * S::kRows + i / D) * D + unit_of(i / D, i % D) * 4 + i % 4] = NAN;
    }
    __syncthreads();
    const bool opens = st0 == 0, closes = st1 == q.steps;
    const int slot = 2 * blockIdx.x + (opens ? 1 : 0);
    auto store_row = [&](int r, int d, float4 v, float top, float sum) {
      const int rr = block * S::kRows + r;
      const int64_t row = q.row0 + rr / group;
      const int hq = head * group + rr % group;
      const float inv = sum > 0.0f ? 1.0f / sum : sum;     // 0 stays 0, NaN stays NaN
      uint2 w;
      if (bf16) {
        w.x = f32_to_act<MOE_DTYPE_BF16>(v.x * inv) | (f32_to_act<MOE_DTYPE_BF16>(v.y * inv) << 16);
        w.y = f32_to_act<MOE_DTYPE_BF16>(v.z * inv) | (f32_to_act<MOE_DTYPE_BF16>(v.w * inv) << 16);
      } else {
        w.x = f32_to_act<MOE_DTYPE_F16>(v.x * inv) | (f32_to_act<MOE_DTYPE_F16>(v.y * inv) << 16);
        w.y = f32_to_act<MOE_DTYPE_F16>(v.z * inv) | (f32_to_act<MOE_DTYPE_F16>(v.w * inv) << 16);
      }
      *reinterpret_cast<uint2*>(a.out + row * a.out_stride + (int64_t)hq * D + d) = w;
      if (d == 0 && a.lse)
        a.lse[row * a.q_heads + hq] = sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    };
    for (int u = tid; u < R * (D / 4); u += kThreads) {
      const int r = u / (D / 4), d = (u % (D / 4)) * 4;
      const int unit = unit_of(r, d);
      float top = kNoMax, sum = 0.0f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w][r]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float4 o = *reinterpret_cast<const float4*>(merge + ((size_t)w * S::kRows + r) * D + unit * 4);
        v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
        const float half = exp2_approx(0.5f * (s_m[w][r] - top));
        sum = fmaf(s_l[w][r] * half, half, sum);
      }
      if (opens && closes) {
        store_row(r, d, v, top, sum);
      } else {
        *reinterpret_cast<float4*>(part + ((size_t)slot * kMaxRows + r) * D + d) = v;
        if (d == 0) {
          stats[(size_t)slot * 2 * kMaxRows + r] = top;
          stats[(size_t)slot * 2 * kMaxRows + kMaxRows + r] = sum;
        }
      }
    }
    if (!(opens && closes)) {
      // the last piece of the segment to arrive joins all of them
      const int c0 = (int)((seg_at + kSegmentCost) / per);
      const int c1 = (int)((seg_at + (TREE ? q.steps + kSegmentCost : length) - 1) / per);
      const int np = c1 - c0 + 1;
      __syncthreads();                         // the whole CTA's rows, then one thread's release
      if (tid == 0) {
        uint32_t before;
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(before) : "l"(&counters[c0]) : "memory");
        s_last = before == (uint32_t)(np - 1);
        if (s_last) counters[c0] = 0;
      }
      __syncthreads();
      if (s_last) {
        // every piece's factor per row; the ring's memory holds them
        float* fac = reinterpret_cast<float*>(big);
        auto stat = [&](int p, int r) { return stats + (size_t)(2 * (c0 + p) + (p == 0)) * 2 * kMaxRows + r; };
        float m[kMine], l[kMine];
        // up to 32 pieces: a lane per piece, all the warp's rows in flight; more go round again
#pragma unroll
        for (int n = 0; n < kMine; ++n) {
          const int r = warp + n * kWarps;
          m[n] = kNoMax, l[n] = 0.0f;
          if (r < R && lane < np) m[n] = __ldcg(stat(lane, r)), l[n] = __ldcg(stat(lane, r) + kMaxRows);
        }
#pragma unroll
        for (int n = 0; n < kMine; ++n) {
          const int r = warp + n * kWarps;
          if (r >= R) break;
          float top = m[n], sum;
          for (int p = lane + 32; p < np; p += 32) top = fmaxf(top, __ldcg(stat(p, r)));
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          const float k0 = exp2_approx(0.5f * (m[n] - top));
          sum = l[n] * k0 * k0;
          if (lane < np) fac[lane * S::kRows + r] = k0 * k0;
          for (int p = lane + 32; p < np; p += 32) {
            const float k = exp2_approx(0.5f * (__ldcg(stat(p, r)) - top));
            fac[p * S::kRows + r] = k * k;
            sum = fmaf(__ldcg(stat(p, r) + kMaxRows) * k, k, sum);
          }
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          if (lane == 0) s_m[0][r] = top, s_l[0][r] = sum;
        }
        __syncthreads();
        constexpr size_t kSlot = (size_t)kMaxRows * D;
        constexpr int kBatch = 16;             // loads in flight per thread
        for (int u = tid; u < R * (D / 4); u += kThreads) {
          const int r = u / (D / 4), d = (u % (D / 4)) * 4;
          const float* src = part + ((size_t)(2 * c0) * kMaxRows + r) * D + d;
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int p0 = 0; p0 < np; p0 += kBatch) {
            float4 o[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const int p = p0 + i;
              o[i] = make_float4(0.f, 0.f, 0.f, 0.f);
              if (p < np) o[i] = __ldcg(reinterpret_cast<const float4*>(src + (2 * p + (p == 0)) * kSlot));
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
              const float k = p0 + i < np ? fac[(p0 + i) * S::kRows + r] : 0.0f;
              v.x = fmaf(o[i].x, k, v.x), v.y = fmaf(o[i].y, k, v.y);
              v.z = fmaf(o[i].z, k, v.z), v.w = fmaf(o[i].w, k, v.w);
            }
          }
          store_row(r, d, v, s_m[0][r], s_l[0][r]);
        }
      }
    }
    // plain writes to the ring's memory come before the next segment's copies into it
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
  }
  // Where the other form runs before this one, this one may start beside it: what follows both
  // then waits for both.
  pdl_wait();
}

template <int D, int NT, int WARPS, bool TREE>
cudaError_t launch_shape(const AttentionArgs& a, cudaStream_t s) {
  using S = Shape<D, NT, WARPS>;
  CUtensorMap map[2];
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.c.kv_heads * a.c.page_size, (uint64_t)a.c.num_pages};
  const uint64_t strides[2] = {(uint64_t)D, (uint64_t)a.c.page_stride};
  const uint32_t box[3] = {(uint32_t)S::kRowB, (uint32_t)(a.c.page_size < S::kStep ? 16 : S::kStep), 1};
  const CUtensorMapSwizzle swz = D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  if (!make_map3(&map[0], a.c.k_codes, dims, strides, box, swz) ||
      !make_map3(&map[1], a.c.v_codes, dims, strides, box, swz))
    return cudaErrorInvalidValue;
  auto kern = attention_kernel<S, TREE>;
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  int grid = num_sms() * S::kCtas;
  if (grid > kMaxGrid) grid = kMaxGrid;
  if (a.max_rows != kAllRows) return launch_pdl(kern, dim3(grid), dim3(S::kThreads), S::kSmem, s, a, map[0], map[1]);
  kern<<<grid, S::kThreads, S::kSmem, s>>>(a, map[0], map[1]);
  return cudaGetLastError();
}

template <int D, bool TREE>
cudaError_t launch_dim(const AttentionArgs& a, cudaStream_t s) {
  // Row tiles of a block: as few as hold the sequences' rows on average in one pass over the keys,
  // or in equal passes beyond three: a fourth tile does not fit into the registers. 16 sequences of
  // 500 to 9000 tokens, 32 rows: 54 us in two passes of two tiles, 67 in one of four (D = 128); 30
  // rows of D = 64: 37 and 42; 40 rows of D = 64 in one pass of five: 49 against 47 in two of three.
  constexpr int kMost = D == 256 ? 2 : 3;
  const long long rows = ((long long)a.T * (a.q_heads / a.c.kv_heads) + a.b.B - 1) / a.b.B;
  const long long tiles = (rows + 7) / 8, passes = (tiles + kMost - 1) / kMost;
  const int nt = (int)((tiles + passes - 1) / passes);
  if constexpr (D <= 128) {
    if (nt == 3) return launch_shape<D, 3, 4, TREE>(a, s);
  }
  if (nt == 2) return launch_shape<D, 2, 4, TREE>(a, s);
  // Few segments: more warps per CTA, so that fewer partial rows have to be joined.
  const bool few = (long long)a.b.B * a.c.kv_heads <= num_sms();
  return few ? launch_shape<D, 1, D == 256 ? 8 : 12, TREE>(a, s) : launch_shape<D, 1, 4, TREE>(a, s);
}

template <bool TREE>
cudaError_t launch_few(const AttentionArgs& a, cudaStream_t s) {
  if (a.c.head_dim == 64) return launch_dim<64, TREE>(a, s);
  return a.c.head_dim == 128 ? launch_dim<128, TREE>(a, s) : launch_dim<256, TREE>(a, s);
}

}  // namespace

namespace {
size_t few_rows_ws_bytes(int head_dim) {
  return align_up(kRowsAt + (size_t)2 * kMaxGrid * kMaxRows * head_dim * 4);
}
}  // namespace

size_t attention_ws_bytes(int q_heads, int kv_heads, int head_dim) {
  return few_rows_ws_bytes(head_dim) + (head_dim <= 128 ? prompt_attention_ws_bytes(head_dim) : 0);
}

cudaError_t launch_attention(const AttentionArgs& args, cudaStream_t s) {
  AttentionArgs a = args;
  a.max_rows = kAllRows;
  const long long rows = (long long)a.T * (a.q_heads / a.c.kv_heads);
  // The other form's launch takes 5 us even where it finds no rows, and its start more than a short
  // segment is worth. For trees, steps of all tiles of 8 rows over the whole table say when that counts;
  // with and without this rule: 3 trees of 32 nodes after 300 tokens, 16 query and 4 key heads of 128, 22.0
  // and 28.2 us, one of 64 after 8000 40.2 and 49.9; with twice the limit 8 of 64 after 1000, just beyond
  // it, take 53.5 instead of 40.9.
  const long long steps = (rows / 8 + a.b.B) * a.c.kv_heads * ((long long)a.b.max_pages * a.c.page_size / 32 + kSegmentCost);
  const bool small = a.tree && steps <= 256LL * num_sms();
  if (a.c.head_dim <= 128 && a.T > a.b.B && rows >= kPromptRows && !small) {
    // some sequence may have that many rows; which ones have is settled on the GPU
    const bool all = a.b.B == 1;
    const cudaError_t e = launch_prompt_attention(a, all ? 1 : kPromptRows, few_rows_ws_bytes(a.c.head_dim), s);
    if (e != cudaSuccess || all) return e;
    a.max_rows = kPromptRows - 1;
  }
  return a.tree ? launch_few<true>(a, s) : launch_few<false>(a, s);
}

}  // namespace moe
