// Attention weights that cached tokens have gathered (moe_kv_weights_e4m3): for each key the sum of
// exp(s - lse) over the rows that see it, the rows' lse being known.
//
// Nothing has to be joined: a key's sum belongs to one warp. All (sequence, key head) keys are cut into
// steps of 32 tokens, which form one line; the grid cuts it into equal pieces and a CTA's warps take
// its piece's steps in turn. Keys go from global memory straight into the fragments of mma.sync
// m16n8k16 as the 16-row operand: lane 4g + c reads, of keys g and 8 + g of a half-step, 16
// consecutive codes at 16c of every 64; the four codes of a word are its values of one k-step, and a
// row's query values are taken with the same permutation of k, i.e. also 16 consecutive ones. A step's
// codes are asked for while the step before is worked on, its page two steps ahead.
//
// The rows come in tiles of 8, the columns of the product. Up to 8 rows (a decode step) a warp keeps the
// tile's fragments in registers and makes them itself from q. For more rows prepare_kernel lays all
// rows out once as such fragments (f16 times a power of two, as the attention does), and the warps
// read them through L1 for every step.
//   w += 2^(s * scale * k_scale * rowf * log2 e - lse * log2 e)      (f32, ex2.approx)
#include "serving.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kStep = 32;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float exp2_approx(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void widen4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}" : "=r"(lo), "=r"(hi) : "r"(w));
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

// A lane's share of a tile of 8 rows: the values 64 j + 16 c .. + 15 of row g for every j, two uint4
// each (words 0, 1 meet the keys' word 0, and so on).
template <int D>
struct Tile {
  uint4 v[D / 32];
};

// The 8 rows from row0 on, of key head h, numbered over the call: row t * group + r is query head
// h * group + r of token t. Rows from row_hi on become 0. *rowf: the power of two taken out of row g.
template <int D>
__device__ __forceinline__ void read_tile(Tile<D>& t, float* rowf, const WeightsArgs& a, int group, int h, int row0,
                                          int row_hi, int lane) {
  const int g = lane >> 2, c = lane & 3, row = row0 + g;
  const bool there = row < row_hi;
  const uint16_t* src = a.q + (int64_t)(row / group) * a.q_stride + (int64_t)(h * group + row % group) * D + 16 * c;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    t.v[i] = make_uint4(0, 0, 0, 0);
    if (there) t.v[i] = *reinterpret_cast<const uint4*>(src + 64 * (i / 2) + 8 * (i & 1));
  }
  *rowf = 1.0f;
  if (a.dtype != MOE_DTYPE_BF16) return;
  // bf16 rows get the power of two that puts their largest magnitude below 2^15
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    float f[8];
    unpack8<MOE_DTYPE_BF16>(t.v[i], f);
#pragma unroll
    for (int x = 0; x < 8; ++x) amax = fmaxf(amax, fabsf(f[x]));
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  const int e = amax < 3.4e38f ? f16_prescale_exp(amax) : 0;
  const float s1 = pow2f(-e / 2), s2 = pow2f(-e - (-e / 2));
  *rowf = pow2f(e);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    float f[8];
    unpack8<MOE_DTYPE_BF16>(t.v[i], f);
#pragma unroll
    for (int x = 0; x < 8; ++x) f[x] = f[x] * s1 * s2;
    t.v[i] = make_uint4(pack_f16(f[0], f[1]), pack_f16(f[2], f[3]), pack_f16(f[4], f[5]), pack_f16(f[6], f[7]));
  }
}
// What is subtracted from a row's exponents; +inf (no weight) for rows that saw nothing.
__device__ __forceinline__ float less_of(float lse) { return lse == -INFINITY ? INFINITY : lse * kLog2e; }

// Workspace behind the error word: rows' factors float2 {rowf, less} [kv_heads][tiles][8], then the
// tiles uint4 [kv_heads][tiles][D / 32][32].
__host__ __device__ inline int tiles_of(long long T, int group) { return (int)((T * group + 7) / 8); }
__host__ __device__ inline size_t laid_at(int heads, int tiles) {
  return kAlign + ((size_t)heads * tiles * 64 + kAlign - 1) / kAlign * kAlign;
}

template <int D>
__global__ void __launch_bounds__(kThreads) prepare_kernel(const __grid_constant__ WeightsArgs a) {
  const int lane = threadIdx.x & 31, heads = a.c.kv_heads, group = a.q_heads / heads;
  const int tiles = tiles_of(a.T, group), rows = a.T * group;
  float2* info = reinterpret_cast<float2*>(a.ws + kAlign);
  uint4* out = reinterpret_cast<uint4*>(a.ws + laid_at(heads, tiles));
  pdl_trigger();
  const long long w = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (w >= (long long)heads * tiles) return;
  const int h = (int)(w / tiles), tile = (int)(w % tiles);
  Tile<D> t;
  float rowf;
  read_tile<D>(t, &rowf, a, group, h, tile * 8, rows, lane);
#pragma unroll
  for (int i = 0; i < D / 32; ++i) out[(w * (D / 32) + i) * 32 + lane] = t.v[i];
  const int row = tile * 8 + (lane >> 2);
  if ((lane & 3) == 0)
    info[w * 8 + (lane >> 2)] = make_float2(
        rowf, row < rows ? less_of(a.lse[(int64_t)(row / group) * a.q_heads + h * group + row % group]) : INFINITY);
}

struct Seq {
  int row0, n, start, len, steps;
};
__device__ __forceinline__ Seq read_seq(const WeightsArgs& a, int b, uint32_t* err) {
  Seq q;
  q.row0 = min(max(a.b.q_offsets[b], 0), a.T);
  const int end = min(max(a.b.q_offsets[b + 1], q.row0), a.T);
  q.n = end - q.row0;
  q.len = a.b.seq_lens[b];
  q.start = q.len - q.n;
  const int cap = a.b.max_pages * a.c.page_size;
  if (q.n > 0 && (q.start < 0 || q.len > cap) && err) atomicOr(err, (uint32_t)MOE_DEVERR_PAGE);
  q.len = min(max(q.len, 0), cap);
  q.steps = q.n > 0 ? (q.len + kStep - 1) / kStep : 0;
  return q;
}

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

// A step of the line: where its keys are.
struct Place {
  int b, h, j0;                                // sequence, key head, first token (j0 < 0: no step)
  int row0, n, start, len;                     // of the sequence
};

template <int D, bool MANY>
__global__ void __launch_bounds__(kThreads, D == 64 ? 2 : 1) weights_kernel(const __grid_constant__ WeightsArgs a) {
  constexpr int kJ = D / 64;                   // 16-code pieces of a key per lane
  __shared__ long long s_sum[kWarps];
  __shared__ int s_seq;
  __shared__ long long s_first;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
  const int heads = a.c.kv_heads, group = a.q_heads / heads, P = a.c.page_size, log_p = 31 - __clz(P);
  uint32_t* err = reinterpret_cast<uint32_t*>(a.ws);
  const int tiles = tiles_of(a.T, group);
  const float2* info = reinterpret_cast<const float2*>(a.ws + kAlign);
  const uint4* laid = reinterpret_cast<const uint4*>(a.ws + laid_at(heads, tiles));

  // this CTA's piece of the line
  long long total = 0, mine = 0, at = 0;
  for (int b0 = 0; b0 < a.b.B; b0 += kThreads) {
    mine = 0;
    if (b0 + tid < a.b.B)
      mine = (long long)read_seq(a, b0 + tid, blockIdx.x == 0 ? err : nullptr).steps * heads;
    total += block_scan(mine, s_sum, &at);
  }
  long long per = (total + gridDim.x - 1) / gridDim.x;
  if (per < kWarps) per = kWarps;
  const long long begin = per * blockIdx.x, end = min(begin + per, total);
  if (begin >= end) return;
  long long base = 0;
  for (int b0 = 0; b0 < a.b.B; b0 += kThreads) {
    long long sum = total;
    if (a.b.B > kThreads) {
      mine = b0 + tid < a.b.B ? (long long)read_seq(a, b0 + tid, nullptr).steps * heads : 0;
      sum = block_scan(mine, s_sum, &at);
    }
    if (mine > 0 && base + at <= begin && begin < base + at + mine) s_seq = b0 + tid, s_first = base + at;
    base += sum;
  }
  __syncthreads();

  // the warp's steps: begin + warp, + kWarps, ...
  int wb = s_seq;
  Seq wq = read_seq(a, wb, nullptr);
  int wh = (int)((begin - s_first) / wq.steps);
  long long pos = begin + warp, first = s_first + (long long)wh * wq.steps;      // first: of (wb, wh)
  auto next_place = [&] {
    Place p;
    p.j0 = -1, p.b = p.h = p.row0 = p.n = p.start = p.len = 0;
    if (pos >= end) return p;
    while (pos >= first + wq.steps) {
      first += wq.steps;
      if (++wh < heads) continue;
      wh = 0;
      do wq = read_seq(a, ++wb, nullptr);
      while (wq.steps == 0);                   // (the line goes on, so there is one more)
    }
    p.b = wb, p.h = wh, p.j0 = (int)(pos - first) * kStep;
    p.row0 = wq.row0, p.n = wq.n, p.start = wq.start, p.len = wq.len;
    pos += kWarps;
    return p;
  };
  // first token that a row of the sequence sees
  auto lowest = [&](const Place& p) { return a.window > 0 ? max(0, p.start - a.window + 1) : 0; };
  auto read_pages = [&](const Place& p, int (&page)[2]) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int j = p.j0 + 16 * x;
      page[x] = (int)load_ahead(a.b.page_table + (int64_t)p.b * a.b.table_stride + (j >> log_p),
                                p.j0 >= 0 && j < p.len, 0xffffffffu);
    }
  };
  // the codes of a step, its pages' scales, and what its tokens had
  struct Keys {
    uint4 k[2][2][kJ];                         // half, key g or 8 + g, piece
    float scale[2], old;
  };
  auto read_keys = [&](const Place& p, int (&page)[2], Keys& s) {
    const bool products = p.j0 >= 0 && p.j0 + kStep > lowest(p);
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const bool in = p.j0 >= 0 && p.j0 + 16 * x < p.len;
      bool good = in && page[x] >= 0 && page[x] < a.c.num_pages;
      if (in && !good) atomicOr(err, (uint32_t)MOE_DEVERR_PAGE);
      if (!good) page[x] = -1;
      const int slot = (p.j0 + 16 * x) & (P - 1);
      const uint8_t* at_ = a.c.k_codes + (int64_t)page[x] * a.c.page_stride + ((int64_t)p.h * P + slot) * D + 16 * c;
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int j = 0; j < kJ; ++j)
          s.k[x][r][j] = load_ahead(at_ + (g + 8 * r) * D + 64 * j, good && products);
      s.scale[x] = __uint_as_float(load_ahead(a.c.k_scales + (int64_t)page[x] * heads + p.h, good, 0u));
    }
    // lane l: token j0 + l
    const int j = p.j0 + lane;
    const int pg = lane < 16 ? page[0] : page[1];
    const bool had = p.j0 >= 0 && j < p.start && pg >= 0 && a.decay != 0.0f;
    s.old = __uint_as_float(load_ahead(a.w + ((int64_t)pg * heads + p.h) * P + (j & (P - 1)), had, 0u));
  };

  // Two steps are in hand, one being worked on and one whose codes are on their way, in turn: a step's
  // registers are never copied while loads into them are out. Pages are read another step ahead.
  Place place[2];
  int page[2][2];
  Keys keys[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    place[i] = next_place();
    read_pages(place[i], page[i]);
  }
  read_keys(place[0], page[0], keys[0]);
  if (MANY) pdl_wait();                        // the rows, laid out by the kernel before
  Tile<D> rows;
  float less[2] = {0, 0}, rowf2[2] = {0, 0};
  int have_b = -1, have_h = -1;

  auto take = [&](Place& here, int (&pg2)[2], Keys& k, Place& ahead, int (&pg2_ahead)[2], Keys& k_ahead) {
    const Place later = next_place();
    int page_later[2];
    read_pages(later, page_later);
    read_keys(ahead, pg2_ahead, k_ahead);

    float sum[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};        // of keys g and 8 + g of either half
    const int j0 = here.j0, row_lo = here.row0 * group, row_hi = (here.row0 + here.n) * group;
    const float f0 = a.scale * kLog2e;
    // keys of the step that some row does not see
    const bool masked = j0 + kStep > here.start + 1 || j0 + kStep > here.len ||
                        (a.window > 0 && j0 <= here.start + here.n - 1 - a.window);
    const float fs[2] = {f0 * k.scale[0], f0 * k.scale[1]};
    // adds the weights of 8 rows; rf and ls of the lane's rows 2c and 2c + 1
    auto add_tile = [&](const Tile<D>& t, int row0, const float (&rf)[2], const float (&ls)[2]) {
      float s[2][4] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
#pragma unroll
      for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const uint32_t b0 = word_of(t.v[2 * j + (m >> 1)], 2 * (m & 1)), b1 = word_of(t.v[2 * j + (m >> 1)], 2 * (m & 1) + 1);
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t a0, a1, a2, a3;
            widen4(word_of(k.k[x][0][j], m), a0, a2);
            widen4(word_of(k.k[x][1][j], m), a1, a3);
            mma(s[x], a0, a1, a2, a3, b0, b1);
          }
        }
#pragma unroll
      for (int x = 0; x < 2; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int y = i & 1;
          float w = exp2_approx(fmaf(s[x][i], fs[x] * rf[y], -ls[y]));
          if (masked) {
            const int row = row0 + 2 * c + y, j = j0 + 16 * x + 8 * (i >> 1) + g;
            const int at_ = here.start + row / group - here.row0;
            const bool see = row >= row_lo && row < row_hi && j <= at_ && j < here.len &&
                             (a.window == 0 || j > at_ - a.window);
            w = see ? w : 0.0f;
          }
          sum[x][i >> 1] += w;
        }
    };
    if (j0 + kStep > lowest(here)) {
      if (MANY) {
        const long long base_ = (long long)here.h * tiles;
        for (int tile = row_lo / 8; tile * 8 < row_hi; ++tile) {
          Tile<D> t;
#pragma unroll
          for (int i = 0; i < D / 32; ++i) t.v[i] = laid[((base_ + tile) * (D / 32) + i) * 32 + lane];
          const float4 f = *reinterpret_cast<const float4*>(info + (base_ + tile) * 8 + 2 * c);
          // rows of the tile that are another sequence's add nothing
          const int r = tile * 8 + 2 * c;
          const float rf[2] = {f.x, f.z};
          const float ls[2] = {r >= row_lo && r < row_hi ? f.y : INFINITY,
                               r + 1 >= row_lo && r + 1 < row_hi ? f.w : INFINITY};
          add_tile(t, tile * 8, rf, ls);
        }
      } else {
        for (int row0 = row_lo; row0 < row_hi; row0 += 8) {
          if (have_b != here.b || have_h != here.h || row_hi - row_lo > 8) {
            float rowf;
            read_tile<D>(rows, &rowf, a, group, here.h, row0, row_hi, lane);
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int row = row0 + 2 * c + y;
              rowf2[y] = __shfl_sync(0xffffffffu, rowf, 4 * (2 * c + y));
              less[y] = row < row_hi
                            ? less_of(a.lse[(int64_t)(row / group) * a.q_heads + here.h * group + row % group])
                            : INFINITY;
            }
            have_b = here.b, have_h = here.h;
          }
          add_tile(rows, row0, rowf2, less);
        }
      }
    }
    // over the rows: columns 2c, 2c + 1 are added already; then lane l takes token j0 + l
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        sum[x][r] += __shfl_xor_sync(0xffffffffu, sum[x][r], 1);
        sum[x][r] += __shfl_xor_sync(0xffffffffu, sum[x][r], 2);
      }
    const int from = 4 * (lane & 7);
    const float w00 = __shfl_sync(0xffffffffu, sum[0][0], from), w01 = __shfl_sync(0xffffffffu, sum[0][1], from);
    const float w10 = __shfl_sync(0xffffffffu, sum[1][0], from), w11 = __shfl_sync(0xffffffffu, sum[1][1], from);
    const float w = lane & 16 ? (lane & 8 ? w11 : w10) : (lane & 8 ? w01 : w00);
    const int j = j0 + lane, pg = lane < 16 ? pg2[0] : pg2[1];
    if (j < here.len && pg >= 0)
      a.w_out[((int64_t)pg * heads + here.h) * P + (j & (P - 1))] = fmaf(k.old, a.decay, w);
    here = later;
    pg2[0] = page_later[0], pg2[1] = page_later[1];
  };
  while (true) {
    if (place[0].j0 < 0) break;
    take(place[0], page[0], keys[0], place[1], page[1], keys[1]);
    if (place[1].j0 < 0) break;
    take(place[1], page[1], keys[1], place[0], page[0], keys[0]);
  }
}

template <int D>
cudaError_t launch_dim(const WeightsArgs& a, cudaStream_t s) {
  const int heads = a.c.kv_heads, group = a.q_heads / heads;
  const int grid = num_sms() * (D == 64 ? 2 : 1);
  // Sequences of one row tile each, as far as the sizes tell (a longer one among them is read with its
  // tiles made again for every step)
  if (a.T <= a.b.B && group <= 8) {
    weights_kernel<D, false><<<grid, kThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
  const long long warps = (long long)heads * tiles_of(a.T, group);
  prepare_kernel<D><<<(unsigned)((warps + kWarps - 1) / kWarps), kThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  return launch_pdl(weights_kernel<D, true>, dim3(grid), dim3(kThreads), 0, s, a);
}

}  // namespace

size_t kv_weights_ws_bytes(int T, int q_heads, int kv_heads, int head_dim) {
  const int tiles = tiles_of(T, q_heads / kv_heads);
  return align_up(laid_at(kv_heads, tiles) + (size_t)kv_heads * tiles * head_dim * 16);
}

cudaError_t launch_kv_weights(const WeightsArgs& a, cudaStream_t s) {
  if (a.c.head_dim == 64) return launch_dim<64>(a, s);
  return a.c.head_dim == 128 ? launch_dim<128>(a, s) : launch_dim<256>(a, s);
}

}  // namespace moe
