// Attention weights that cached tokens have gathered (moe_kv_weights_e4m3): for each key the sum of
// exp(s - lse) over the rows (new tokens times query heads per key head) that see it, the rows' lse
// being known:
//   w += 2^(s * scale * k_scale * rowf * log2 e - lse * log2 e)      (f32, ex2.approx)
//
// Nothing has to be joined: a key belongs to one thread. All (sequence, key head) keys are cut into
// tiles of 128 tokens, which form one line; the grid cuts it into equal pieces. prepare_kernel lays the
// rows out once, as f16 times a power of two (as the attention does) in the swizzled order of the
// products' operand; the main kernel starts beside it. In a CTA one warp brings tiles of codes into a
// ring (TMA, a box per page), one brings their tokens' old weights and factors into another, and blocks
// of rows before the tiles that need them, and groups of four warps take the tiles in turn, thread = key:
//   the key's codes to f16 (exact) in tensor memory; S = K Q^T with the keys from there as the 128-row
//   operand (tcgen05, f32; one thread issues); the key's row of S, weights, their sum, and the token's
//   new weight
// A tile is one chain of waits and dependent instructions of its group, most of it not arithmetic, so
// what counts is how many groups an SM has. The widened keys go to tensor memory and not to shared
// memory, whose bandwidth would be the limit: a code is written there and read once. Rows beyond a
// block take the piece's tiles again and add to what the block before left.
//
// With one new token per sequence the bytes bound it: 64 sequences of 100 to 16000 tokens, 32 query and
// 8 key heads of 128: 48.4 us, 4.6 TB/s (0.68 of the copy rate); one sequence of 32767, 64 query heads:
// 13.6 us, of which 7.5 are fixed (a sequence of 1000 takes them). With many rows it is the groups' chain:
// 6 prompts of 1000 to 16001 tokens judged by 32 tokens, 40 query and 8 key heads of 64 (160 rows): 27.0
// us, 26.5 with the exponentials taken out (when it took 27.4). Heads of 256 have blocks of 32 rows and
// spill 56 / 72 bytes: 32 sequences of 100 to 8000, 16 query and 4 key heads, 19.5 us (floor 9.4), the
// prompts with such heads (128 rows) 36.6 (5.8). Measured against this, in its state of then: mma.sync with keys
// and rows in registers 69 us where the 64 sequences took 59; products, widening and sums as roles of
// their own 55 where they took 49; rows in blocks of 128 at heads of 64 30.3 (a tile is widened twice),
// the next columns of S asked for before these are used 33.8, two products of 32 columns in flight 30.1
// (each where the prompts took 27.4); S read 32 columns at a time 32.4 where they took 30.2.
#include "tc_f16.cuh"

namespace moe {
namespace {

constexpr int kTile = 128;                     // keys
constexpr int kPrepWarps = 8;
// What a (sequence, key head) costs beside its tiles (its rows, the chain of its first tile), in tiles:
// pieces of the line are equal with it counted. 64 sequences: 60.9 us with 0, 48.8 with 2, 50.4 with 4.
constexpr int kSegmentCost = 2;
constexpr float kLog2e = 1.4426950408889634f;

// Rows are kept in groups of 8 that begin anew with every sequence: sequence b's first group is
// q_offsets[b] * group / 8 + q_offsets[b], which leaves room for the last group of each that is not full.
// Workspace behind the error word: factors [kv_heads][groups][4] of float4 {rowf, rowf, -less, -less} of
// two rows each, new-token numbers int [groups][8], rows f16 [kv_heads][D / 64][groups][8][64], swizzled.
__host__ __device__ inline long long groups_of(long long T, int group) { return T * group / 8 + T + 1; }
__device__ __forceinline__ int first_group(int row0, int group) { return (int)((long long)row0 * group / 8 + row0); }
__host__ __device__ inline size_t round_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }
__host__ __device__ inline size_t tokens_at(int heads, long long groups) { return kAlign + round_up((size_t)heads * groups * 64); }
__host__ __device__ inline size_t rows_at(int heads, long long groups) { return tokens_at(heads, groups) + round_up((size_t)groups * 32); }

struct Seq {
  int row0, n, start, len, tiles;
};
__device__ __forceinline__ Seq read_seq(const WeightsArgs& a, int b, uint32_t* err) {
  Seq q;
  q.row0 = min(max(a.b.q_offsets[b], 0), a.T);
  const int end = min(max(a.b.q_offsets[b + 1], q.row0), a.T);
  q.n = end - q.row0;
  q.len = a.b.seq_lens[b];
  q.start = q.len - q.n;
  const int cap = a.b.max_pages * a.c.page_size;
  if (q.n > 0 && (q.len < q.n || q.len > cap) && err) atomicOr(err, (uint32_t)MOE_DEVERR_PAGE);
  q.len = min(max(q.len, 0), cap);
  q.tiles = q.n > 0 ? (q.len + kTile - 1) / kTile : 0;
  return q;
}

// A warp per 8 rows of a key head; block (b, y) works for sequence b.
template <int D>
__global__ void __launch_bounds__(32 * kPrepWarps) prepare_kernel(const __grid_constant__ WeightsArgs a) {
  pdl_trigger();
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, heads = a.c.kv_heads, group = a.q_heads / heads;
  const long long groups = groups_of(a.T, group);
  const Seq q = read_seq(a, blockIdx.x, nullptr);
  const int rows = q.n * group, mine = (rows + 7) / 8, at0 = first_group(q.row0, group);
  float* info = reinterpret_cast<float*>(a.ws + kAlign);
  int* tokens = reinterpret_cast<int*>(a.ws + tokens_at(heads, groups));
  char* out = a.ws + rows_at(heads, groups);
  for (long long it = (long long)blockIdx.y * kPrepWarps + (threadIdx.x >> 5); it < (long long)heads * mine;
       it += (long long)gridDim.y * kPrepWarps) {
    const int h = (int)(it / mine), tile = (int)(it % mine), row = tile * 8 + g;
    const bool there = row < rows;
    const int64_t token = q.row0 + (there ? row / group : 0), hq = h * group + row % group;
    const uint16_t* src = a.q + token * a.q_stride + hq * D;
    uint4 v[D / 32];                           // 16-byte pieces c, c + 4, ... of the row
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      v[i] = make_uint4(0, 0, 0, 0);
      if (there) v[i] = *reinterpret_cast<const uint4*>(src + (c + 4 * i) * 8);
    }
    const float lse = there ? a.lse[token * a.q_heads + hq] : -INFINITY;
    float rowf = 1.0f;
    if (a.dtype == MOE_DTYPE_BF16) {
      // bf16 rows get the power of two that puts their largest magnitude below 2^15
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        float f[8];
        unpack8<MOE_DTYPE_BF16>(v[i], f);
#pragma unroll
        for (int x = 0; x < 8; ++x) amax = fmaxf(amax, fabsf(f[x]));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      const int e = amax < 3.4e38f ? f16_prescale_exp(amax) : 0;
      const float s1 = pow2f(-e / 2), s2 = pow2f(-e - (-e / 2));
      rowf = pow2f(e);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        float f[8];
        unpack8<MOE_DTYPE_BF16>(v[i], f);
#pragma unroll
        for (int x = 0; x < 8; ++x) f[x] = f[x] * s1 * s2;
        v[i] = make_uint4(pack_f16(f[0], f[1]), pack_f16(f[2], f[3]), pack_f16(f[4], f[5]), pack_f16(f[6], f[7]));
      }
    }
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const int piece = c + 4 * i;
      char* to = out + (((int64_t)h * (D / 64) + (piece >> 3)) * groups + at0 + tile) * 1024 + g * 128;
      *reinterpret_cast<uint4*>(to + (((piece & 7) ^ g) * 16)) = v[i];
    }
    if (c == 0) {
      float* f = info + (((int64_t)h * groups + at0 + tile) * 4 + g / 2) * 4;
      f[g & 1] = rowf;
      f[2 + (g & 1)] = lse == -INFINITY ? -INFINITY : -(lse * kLog2e);   // rows that saw nothing add nothing
      if (h == 0) tokens[(int64_t)(at0 + tile) * 8 + g] = there ? row / group : -(1 << 30);
    }
  }
}

template <int D_>
struct Shape {
  static constexpr int D = D_;
  static constexpr int kCtas = D == 256 ? 1 : 2;                       // per SM
  static constexpr int kGroups = D == 256 ? 3 : 2, kThreads = 32 * (4 * kGroups + 2);
  static constexpr int kRows = D == 64 ? 256 : D == 128 ? 128 : 32;        // of a block
  static constexpr int kChunk = kRows < 64 ? kRows : 64;               // of a product
  static constexpr int kSlots = D == 64 ? 4 : D == 128 ? 2 : 3, kHeads = 6;
  // every group has slots of its own, so that a wait never mistakes a phase
  static constexpr int kOwn = kSlots / kGroups, kOwnHeads = kHeads / kGroups;
  static_assert(kSlots % kGroups == 0 && kHeads % kGroups == 0, "");
  static constexpr int kSubs = D == 256 ? 2 : 1, kRowB = D == 64 ? 64 : 128;
  static constexpr int kTileB = kTile * D, kHalf = kRows * 128, kQB = kRows * D * 2;
  static constexpr int kSAt = kGroups * D / 2, kCols = 512 / kCtas;    // tensor memory columns
  static_assert(kSAt + kGroups * kChunk <= kCols, "");
  static constexpr int kQAt = kSlots * kTileB, kInfoAt = kQAt + 2 * kQB, kTokenAt = kInfoAt + 2 * kRows * 8;
  // of a tile: its tokens' old weights, and for each page where its weights are and its factor
  static constexpr int kHeadB = kTile * 4 + 96, kHeadAt = kTokenAt + 2 * kRows * 4;
  static constexpr int kSmem = 1024 + kHeadAt + kHeads * kHeadB;
  static_assert(kCtas * (kSmem + 2048) <= 227 * 1024, "");
};

// Neighbouring tiles of one sequence and key head for one block of rows.
struct Run {
  int b, h, block, t0, t1;                     // sequence, key head, block of rows, tiles
  int turn;                                    // the group that takes the first of them
  int first;                                   // first tile with a key that some row sees
  int row0, n, start, len;                     // of the sequence
};
// A CTA's piece of the line; every role walks it for itself.
struct Walk {
  long long pos, end, first;                   // first: of (b, h)
  int b, h, block, blocks, t0, t1, turn;
  Seq q;
};
__device__ __forceinline__ long long length_of(const Seq& q) { return q.tiles ? q.tiles + kSegmentCost : 0; }
__device__ __forceinline__ bool next_run(Walk& w, Run& r, const WeightsArgs& a, int group, int block_rows, int groups) {
  if (++w.block >= w.blocks) {
    w.turn = (w.turn + max(w.t1 - w.t0, 0)) % groups;      // the groups go on taking tiles in turn
    do {
      if (w.pos >= w.end) return false;
      while (w.pos >= w.first + length_of(w.q)) {
        w.first += length_of(w.q);
        if (++w.h < a.c.kv_heads) continue;
        w.h = 0;
        do w.q = read_seq(a, ++w.b, nullptr);
        while (w.q.tiles == 0);                // (the line goes on, so there is one more)
      }
      const long long upto = min(length_of(w.q), w.end - w.first);
      w.t0 = max((int)(w.pos - w.first) - kSegmentCost, 0);
      w.t1 = (int)upto - kSegmentCost;
      w.pos = w.first + upto;
    } while (w.t1 <= w.t0);                    // (only the fixed cost fell to this CTA)
    w.block = 0, w.blocks = (w.q.n * group + block_rows - 1) / block_rows;
  }
  r.turn = w.turn;
  r.b = w.b, r.h = w.h, r.block = w.block, r.t0 = w.t0, r.t1 = w.t1;
  r.row0 = w.q.row0, r.n = w.q.n, r.start = w.q.start, r.len = w.q.len;
  r.first = a.window > 0 ? max(w.q.start - a.window + 1, 0) / kTile : 0;
  return true;
}

__device__ __forceinline__ float load_plain(const float* at) {
  float v;
  asm volatile("ld.global.f32 %0, [%1];" : "=f"(v) : "l"(at) : "memory");
  return v;
}

template <int D>
__global__ void __launch_bounds__(Shape<D>::kThreads, Shape<D>::kCtas)
weights_kernel(const __grid_constant__ WeightsArgs a, const __grid_constant__ CUtensorMap kmap) {
  using S = Shape<D>;
  constexpr int kThreads = S::kThreads, G = S::kGroups;
  extern __shared__ char smem_raw[];
  __shared__ uint64_t s_kfull[S::kSlots], s_kempty[S::kSlots], s_afull[G], s_sfull[G], s_sempty[G];
  __shared__ uint64_t s_qfull[2], s_qempty[2], s_hfull[S::kHeads], s_hempty[S::kHeads];
  __shared__ uint32_t s_tmem;
  __shared__ volatile int s_abort;
  __shared__ long long s_sum[kThreads / 32], s_first;
  __shared__ int s_seq;
  char* smem = reinterpret_cast<char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int heads = a.c.kv_heads, group = a.q_heads / heads, P = a.c.page_size, log_p = 31 - __clz(P);
  const long long groups = groups_of(a.T, group);
  uint32_t* err = reinterpret_cast<uint32_t*>(a.ws);
  volatile int* abort_flag = &s_abort;

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
  auto line_of = [&](int b, uint32_t* e) { return b < a.b.B ? length_of(read_seq(a, b, e)) * heads : 0; };
  long long total = 0, mine = 0, at = 0;
  for (int b0 = 0; b0 < a.b.B; b0 += kThreads) {
    mine = line_of(b0 + tid, blockIdx.x == 0 ? err : nullptr);
    total += scan(mine, &at);
  }
  const long long per = (total + gridDim.x - 1) / gridDim.x;
  const long long begin = per * blockIdx.x, end = min(begin + per, total);
  if (begin >= end) {
    pdl_wait();                                // what follows in the stream waits for the kernel before too
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
    for (int i = 0; i < S::kSlots; ++i) mbar_init(&s_kfull[i], 1), mbar_init(&s_kempty[i], 4);
    for (int i = 0; i < G; ++i) mbar_init(&s_afull[i], 4), mbar_init(&s_sfull[i], 1), mbar_init(&s_sempty[i], 4);
    for (int i = 0; i < 2; ++i) mbar_init(&s_qfull[i], 1), mbar_init(&s_qempty[i], 4 * G);
    for (int i = 0; i < S::kHeads; ++i) mbar_init(&s_hfull[i], 1), mbar_init(&s_hempty[i], 4);
    s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async();
  }
  if (warp == 4 * G) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                 ::"r"(smem_u32(&s_tmem)), "n"(S::kCols) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  Walk w;
  w.pos = begin, w.end = end, w.b = s_seq;
  w.q = read_seq(a, w.b, nullptr);
  w.h = (int)((begin - s_first) / length_of(w.q));
  w.first = s_first + w.h * length_of(w.q);
  w.block = w.blocks = w.t0 = w.t1 = w.turn = 0;
  Run run;
  auto next = [&] { return next_run(w, run, a, group, S::kRows, G); };
  auto rows_of = [&] { return min(S::kRows, run.n * group - run.block * S::kRows); };
  bool ok = true;

  if (warp < 4 * G) {
    // ---------------- tiles: group `gr`'s, thread = key ----------------
    const int gr = warp / 4, key = tid & 127, in_page = key & (P - 1);
    const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16, swz = D == 64 ? (key >> 1) & 3 : key & 7;
    const uint32_t a_col = tmem + gr * (D / 2), s_col = tmem + S::kSAt + gr * S::kChunk;
    const uint64_t q_desc = smem_desc(smem_u32(smem + S::kQAt), 16, 1024, 2);
    const bool issues = (warp & 3) == 0 && lane == 0;
    constexpr int kPer = S::kRowB / 16;        // 16-byte pieces of a sub-tile's row
    uint32_t k = 0, sph = 0, eph = 0, blocks = 0;                      // tiles; phases; blocks of rows
    while (ok && next()) {
      const int rows = rows_of(), cols = (rows + 7) / 8 * 8, qb = blocks & 1;
      // tiles that no row sees: the old weights fade
      for (int t = run.t0 + gr; t < min(run.first, run.t1) && run.block == 0; t += G) {
        const int j = t * kTile + key;
        if (j >= run.len) continue;
        const int page = a.b.page_table[(int64_t)run.b * a.b.table_stride + (j >> log_p)];
        if (page < 0 || page >= a.c.num_pages) {
          atomicOr(err, (uint32_t)MOE_DEVERR_PAGE);
          continue;
        }
        const int64_t at_ = ((int64_t)page * heads + run.h) * P + in_page;
        a.w_out[at_] = a.decay == 0.0f ? 0.0f : load_plain(a.w + at_) * a.decay;
      }
      const int first = max(run.t0, run.first);
      if (first >= run.t1) continue;           // the block's rows meet no tile
      if (!(ok = wait_warp(&s_qfull[qb], blocks >> 1 & 1, abort_flag, err))) break;
      const float4* info = reinterpret_cast<const float4*>(smem + S::kInfoAt + qb * S::kRows * 8);
      const int* tokens = reinterpret_cast<const int*>(smem + S::kTokenAt + qb * S::kRows * 4);
      auto products = [&](int c0) {            // S of the rows from c0 on
        const uint32_t id = f16_idesc(128, min(S::kChunk, (rows - c0 + 15) / 16 * 16), false);
        const uint64_t qd = q_desc + (uint32_t)((qb * S::kQB + c0 * 128) >> 4);
        tc_fence_after();
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
          mma_ts(s_col, a_col + i * 8, qd + (uint32_t)(((i >> 2) * S::kHalf + (i & 3) * 32) >> 4), id, i != 0);
        tc_commit(&s_sfull[gr]);
      };
      // tiles from `part` on and before `edge` have keys that some row does not see
      const int part = max(min(run.start + 1, run.len), 0) / kTile;
      const int edge = a.window > 0 ? max(run.start + run.n - 1 - a.window + kTile, 0) / kTile : 0;
      // a tile is the same group's for every block of rows: its threads add to what they left
      for (int t = first + (gr + G - run.turn) % G; t < run.t1; t += G, ++k) {
        const int slot = gr + G * (k % S::kOwn), hb = gr + G * (k % S::kOwnHeads);
        if (!(ok = wait_warp(&s_kfull[slot], k / S::kOwn & 1, abort_flag, err))) break;
        const uint32_t row = smem_u32(smem + slot * S::kTileB) + (uint32_t)key * S::kRowB;
#pragma unroll
        for (int i = 0; i < D / 16; i += 2) {  // 32 codes at a time
          uint32_t v[16];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int piece = i + x;
            const uint4 c = lds128(row + (piece / kPer) * (kTile * 128) + (((piece % kPer) ^ swz) * 16));
            widen4(c.x, v[8 * x], v[8 * x + 1]);
            widen4(c.y, v[8 * x + 2], v[8 * x + 3]);
            widen4(c.z, v[8 * x + 4], v[8 * x + 5]);
            widen4(c.w, v[8 * x + 6], v[8 * x + 7]);
          }
          tc_st16(a_col + quarter + i * 8, v);
        }
        warp_arrive(&s_kempty[slot]);
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&s_afull[gr]);
        if (issues && wait_thread(&s_afull[gr], k & 1, abort_flag, err)) products(0);
        __syncwarp();
        // (meanwhile) the token's old weight, where its new one goes, and its page's factor
        if (!(ok = wait_warp(&s_hfull[hb], k / S::kOwnHeads & 1, abort_flag, err))) break;
        const char* head = smem + S::kHeadAt + hb * S::kHeadB;
        const int j = t * kTile + key;
        float old = reinterpret_cast<const float*>(head)[key];
        const long long at_ = reinterpret_cast<const long long*>(head + kTile * 4)[key >> log_p];
        const float f = reinterpret_cast<const float*>(head + kTile * 4 + 64)[key >> log_p];
        warp_arrive(&s_hempty[hb]);
        if (j >= run.start || run.block != 0 || a.decay == 0.0f) old = 0.0f;
        float* to = a.w_out + at_ + in_page;
        const bool mine = j < run.len && at_ >= 0;
        const uint64_t ff = pair(f, f);
        uint64_t acc[2] = {0, 0};
        // Token i sees key j if i - since, as a number without sign, is below `span`: no token before
        // the key is, and no sum is made that a large window could take past 32 bits.
        const uint32_t since = (uint32_t)(j - run.start), span = a.window > 0 ? a.window : 0x7fffffffu;
        // the weights of eight rows
        auto add8 = [&](const float* v, int r, auto hides) {
#pragma unroll
          for (int x = 0; x < 8; x += 2) {
            const float4 q = info[(r + x) / 2];
            float e0, e1;
            unpair(fma2(pair(v[x], v[x + 1]), mul2(pair(q.x, q.y), ff), pair(q.z, q.w)), e0, e1);
            e0 = exp2_approx(e0), e1 = exp2_approx(e1);
            if (decltype(hides)::value) {
              const int2 i = *reinterpret_cast<const int2*>(tokens + r + x);
              e0 = i.x - since < span ? e0 : 0.0f;
              e1 = i.y - since < span ? e1 : 0.0f;
            }
            acc[x >> 1 & 1] = add2(acc[x >> 1 & 1], pair(e0, e1));
          }
        };
        for (int c0 = 0; c0 < rows; c0 += S::kChunk) {
          if (c0 > 0) {                        // the rows' next chunk over the one that all have read
            tc_fence_before();
            warp_arrive(&s_sempty[gr]);
            if (issues && wait_thread(&s_sempty[gr], eph & 1, abort_flag, err)) products(c0);
            ++eph;
            __syncwarp();
          }
          if (!(ok = wait_warp(&s_sfull[gr], sph & 1, abort_flag, err))) break;
          ++sph;
          tc_fence_after();
          const int n = min(S::kChunk, cols - c0);
          auto add_all = [&](auto hides) {
            int c = 0;
#pragma unroll 1
            for (; c < n; c += 16) {
              float v[16];
              tmem_ld16(s_col + quarter + c, v);
              add8(v, c0 + c, hides);
              if (c + 8 < n) add8(v + 8, c0 + c + 8, hides);         // the last group of rows may stand alone
            }
          };
          if (t >= part || t < edge) add_all(std::true_type{});
          else add_all(std::false_type{});
        }
        if (!ok) break;
        tc_fence_before();
        float x0, x1;
        unpair(add2(acc[0], acc[1]), x0, x1);
        if (mine) *to = run.block == 0 ? fmaf(old, a.decay, x0 + x1) : load_plain(to) + (x0 + x1);   // (its own of a block before)
      }
      if (!ok) break;
      warp_arrive(&s_qempty[qb]);
      ++blocks;
    }
    // gave up: a product that was issued is done before the tensor memory is given back (bounded)
    if (!ok && issues) {
      const uint64_t t0 = global_ns();
      while (!mbar_try(&s_sfull[gr], sph & 1) && global_ns() - t0 < 100000000ull) {
      }
    }
  } else {
    // Pages come for as many tiles of a run at once as lanes allow, those of the next such batch (or run)
    // asked for while this one's tiles are brought.
    const int in_tile = kTile >> log_p, log_t = 7 - log_p, batch = 32 >> log_t, which = lane >> log_t;
    const int slot_page = lane & (in_tile - 1);
    Walk look = w;
    Run lr = {};
    int lt = 0;                                // next tile of lr
    auto ask_pages = [&] {
      while (lt >= lr.t1) {
        if (!next_run(look, lr, a, group, S::kRows, G)) return -1;
        lt = max(lr.t0, lr.first);
      }
      const int t = lt + which, j = t * kTile + slot_page * P;
      const bool in = which < batch && t < lr.t1 && j < lr.len;
      const int page = (int)load_ahead(a.b.page_table + (int64_t)lr.b * a.b.table_stride + (j >> log_p), in, 0xffffffffu);
      lt += batch;
      return page;                             // (-1 where no page is asked for)
    };
    auto known = [&](int page) { return page >= 0 && page < a.c.num_pages; };
    uint32_t count[G] = {};                    // tiles of each group
    auto next_of = [&](int gr) {
      uint32_t k = 0;
#pragma unroll
      for (int i = 0; i < G; ++i)
        if (i == gr) k = count[i]++;
      return k;
    };
    int page = ask_pages();
    bool begun = false;
    const uint64_t limit = 100000000ull;
    if (warp == 4 * G) {
      // ---------------- tiles of codes ----------------
      int page_next = ask_pages();
      while (ok && next()) {
        const int first = max(run.t0, run.first);
        for (int t = first, gr = run.turn; t < run.t1; ++t, gr = gr + 1 == G ? 0 : gr + 1) {
          const uint32_t k = next_of(gr);
          const int in_batch = (t - first) & (batch - 1), slot = gr + G * (k % S::kOwn);
          if (in_batch == 0 && begun) page = page_next, page_next = ask_pages();
          begun = true;
          const bool good = which == in_batch && known(page);
          const uint32_t there = __ballot_sync(0xffffffffu, good);
          if (!(ok = wait_warp(&s_kempty[slot], (k / S::kOwn & 1) ^ 1, abort_flag, err))) break;
          if (lane == 0) mbar_expect_tx(&s_kfull[slot], __popc(there) * P * D);
          __syncwarp();
          if (good) {
            char* to = smem + slot * S::kTileB + slot_page * P * S::kRowB;
#pragma unroll
            for (int i = 0; i < S::kSubs; ++i)
              tma_load_3d(to + i * (kTile * 128), &kmap, i * 128, run.h * P, page, &s_kfull[slot]);
          }
        }
      }
      if (!ok) {                               // gave up: let the copies in flight land (bounded)
        const uint64_t t0 = global_ns();
#pragma unroll
        for (int g = 0; g < G; ++g)
          for (uint32_t i = count[g] > S::kOwn ? count[g] - S::kOwn : 0; i < count[g]; ++i)
            while (!mbar_try(&s_kfull[g + G * (i % S::kOwn)], i / S::kOwn & 1) && global_ns() - t0 < limit) {
            }
      }
    } else {
      // ---------------- blocks of rows; tiles' old weights, places of the new ones, factors ----------------
      auto ask_scale = [&](int pg, int h) {
        return __uint_as_float(load_ahead(a.c.k_scales + (int64_t)pg * heads + h, known(pg), 0u));
      };
      float scale = ask_scale(page, lr.h), scale_next = 0.0f;
      int page_next = ask_pages(), h_next = lr.h;
      uint32_t blocks = 0;
      const char* q = a.ws + rows_at(heads, groups);
      pdl_wait();                              // the rows are laid out by the kernel before
      while (ok && next()) {
        const int first = max(run.t0, run.first);
        if (first >= run.t1) continue;
        const int qb = blocks & 1, n8 = (rows_of() + 7) / 8;
        const int64_t g0 = first_group(run.row0, group) + run.block * (S::kRows / 8);
        if (!(ok = wait_warp(&s_qempty[qb], (blocks >> 1 & 1) ^ 1, abort_flag, err))) break;
        if (lane == 0) {
          mbar_expect_tx(&s_qfull[qb], (uint32_t)n8 * (64 + 32 + 16 * D));
          bulk_load(smem + S::kInfoAt + qb * S::kRows * 8, a.ws + kAlign + ((int64_t)run.h * groups + g0) * 64, n8 * 64, &s_qfull[qb]);
          bulk_load(smem + S::kTokenAt + qb * S::kRows * 4, a.ws + tokens_at(heads, groups) + g0 * 32, n8 * 32, &s_qfull[qb]);
          for (int i = 0; i < D / 64; ++i)
            bulk_load(smem + S::kQAt + qb * S::kQB + i * S::kHalf, q + (((int64_t)run.h * (D / 64) + i) * groups + g0) * 1024,
                      n8 * 1024, &s_qfull[qb]);
        }
        __syncwarp();
        ++blocks;
        for (int t = first, gr = run.turn; t < run.t1; ++t, gr = gr + 1 == G ? 0 : gr + 1) {
          const uint32_t k = next_of(gr);
          const int in_batch = (t - first) & (batch - 1), hb = gr + G * (k % S::kOwnHeads);
          if (in_batch == 0 && begun) {
            page = page_next, scale = scale_next;
            page_next = ask_pages();
            h_next = lr.h;
          }
          begun = true;
          if (in_batch == min(1, min(batch, run.t1 - (t - in_batch)) - 1)) scale_next = ask_scale(page_next, h_next);
          const bool mine = which == in_batch, good = mine && known(page);
          if (mine && !good && t * kTile + slot_page * P < run.len) atomicOr(err, (uint32_t)MOE_DEVERR_PAGE);
          const bool had = good && run.block == 0 && a.decay != 0.0f && t * kTile + slot_page * P < run.start;
          const uint32_t olds = __popc(__ballot_sync(0xffffffffu, had));
          if (!(ok = wait_warp(&s_hempty[hb], (k / S::kOwnHeads & 1) ^ 1, abort_flag, err))) break;
          char* head = smem + S::kHeadAt + hb * S::kHeadB;
          const int64_t at_ = ((int64_t)page * heads + run.h) * P;
          if (mine) {
            reinterpret_cast<long long*>(head + kTile * 4)[slot_page] = good ? at_ : -1;
            reinterpret_cast<float*>(head + kTile * 4 + 64)[slot_page] = good ? a.scale * kLog2e * scale : 0.0f;
          }
          __syncwarp();
          if (lane == 0) mbar_expect_tx(&s_hfull[hb], olds * P * 4);
          __syncwarp();
          if (had) bulk_load(head + slot_page * P * 4, a.w + at_, P * 4, &s_hfull[hb]);
        }
      }
      if (!ok) {
        const uint64_t t0 = global_ns();
#pragma unroll
        for (int g = 0; g < G; ++g)
          for (uint32_t i = count[g] > S::kOwnHeads ? count[g] - S::kOwnHeads : 0; i < count[g]; ++i)
            while (!mbar_try(&s_hfull[g + G * (i % S::kOwnHeads)], i / S::kOwnHeads & 1) && global_ns() - t0 < limit) {
            }
        for (uint32_t i = blocks > 2 ? blocks - 2 : 0; i < blocks; ++i)
          while (!mbar_try(&s_qfull[i & 1], i >> 1 & 1) && global_ns() - t0 < limit) {
          }
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 4 * G)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(S::kCols));
}

template <int D>
cudaError_t launch_main(const WeightsArgs& a, cudaStream_t s) {
  using S = Shape<D>;
  CUtensorMap map;
  const uint64_t dims[3] = {(uint64_t)D, (uint64_t)a.c.kv_heads * a.c.page_size, (uint64_t)a.c.num_pages};
  const uint64_t strides[2] = {(uint64_t)D, (uint64_t)a.c.page_stride};
  const uint32_t box[3] = {(uint32_t)S::kRowB, (uint32_t)a.c.page_size, 1};
  if (!make_map3(&map, a.c.k_codes, dims, strides, box, D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  auto kern = weights_kernel<D>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(S::kCtas * num_sms()), dim3(S::kThreads), S::kSmem, s, a, map);
}

template <int D>
cudaError_t launch_dim(const WeightsArgs& a, cudaStream_t s) {
  const int heads = a.c.kv_heads, group = a.q_heads / heads;
  // prepare: blocks per sequence, as if all had the same number of rows
  const long long warps = (long long)heads * ((((long long)a.T * group + a.b.B - 1) / a.b.B + 7) / 8);
  const long long y = (warps + kPrepWarps - 1) / kPrepWarps, most = (4 * num_sms() + a.b.B - 1) / a.b.B;
  prepare_kernel<D><<<dim3((unsigned)a.b.B, (unsigned)(y < most ? y : most)), 32 * kPrepWarps, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_main<D>(a, s);
}

}  // namespace

size_t kv_weights_ws_bytes(int T, int q_heads, int kv_heads, int head_dim) {
  const long long groups = groups_of(T, q_heads / kv_heads);
  return align_up(rows_at(kv_heads, groups) + (size_t)kv_heads * groups * head_dim * 16);
}

cudaError_t launch_kv_weights(const WeightsArgs& a, cudaStream_t s) {
  if (a.c.head_dim == 64) return launch_dim<64>(a, s);
  return a.c.head_dim == 128 ? launch_dim<128>(a, s) : launch_dim<256>(a, s);
}

}  // namespace moe
