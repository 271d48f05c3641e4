// Appending keys and values to the paged 8-bit cache, rotated by their positions on the way,
// and the rotation of the queries beside them (moe_kv_append_rope_e4m3).
//
// One launch. The first blocks each take (a page that the batch touches, a head, K or V): they
// find the page's new tokens, take the largest rotated magnitude, settle the page's scale, rescale
// the page's earlier codes if it grew, and write the new codes. The other blocks rotate
// queries. A head's D values are handled as D/16 chunks of 16 values that rotate among
// themselves: values [8i, 8i+8) with [rotary/2 + 8i, ...), in the interleaved order too (whose pairs
// lie inside the groups of eight), and past rotary_dim likewise, so that neighbouring lanes' 16-byte
// accesses are neighbours in memory (16 consecutive values per lane took 31.1 us against 30.5 for
// six interleaved prompts of up to 2048 tokens).
//
// Rotation and rounding use single correctly rounded operations in a fixed order (no fused
// multiply-add), so codes and scales are the same bits wherever the definition is evaluated in
// f32.
//
// Bound by the rows' bytes (2 read and 2 written per query value, 2 read and 1 written per key or
// value): six prompts of up to 2048 tokens, 32 query and 8 key heads of 128 (127 MB), take 30.5 us, 4.2
// TB/s: a third of the warps are active (80 registers) and a page's steps depend on one another (largest
// magnitude, then codes), so too few loads are in flight. One
// token of one sequence takes 3.3 us, a launch and a few dependent loads.
#include "serving.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;

// Where chunk `ch` of a head keeps its two groups of eight values, and which table columns turn
// the first and the last four of their pairs (col < 0: not rotated).
struct Chunk {
  int lo, hi, col, col4;
};
__device__ __forceinline__ Chunk chunk_at(int ch, int D, int rotary, int interleaved) {
  const bool turned = 16 * ch < rotary;
  const int first = turned ? 0 : rotary, i = ch - first / 16;
  Chunk r;
  r.lo = first + 8 * i;
  r.hi = r.lo + (turned ? rotary : D - rotary) / 2;
  r.col = !turned ? -1 : interleaved ? 4 * i : 8 * i;
  r.col4 = interleaved ? rotary / 4 + 4 * i : 8 * i + 4;
  return r;
}

struct Turn {
  float c[8], s[8];
};
// Of the table row that starts at `at`.
__device__ __forceinline__ void load_turn(Turn& t, const float* cos, const float* sin, int64_t at, const Chunk& ch) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(cos + at + (i ? ch.col4 : ch.col)));
    const float4 b = __ldg(reinterpret_cast<const float4*>(sin + at + (i ? ch.col4 : ch.col)));
    t.c[4 * i] = a.x, t.c[4 * i + 1] = a.y, t.c[4 * i + 2] = a.z, t.c[4 * i + 3] = a.w;
    t.s[4 * i] = b.x, t.s[4 * i + 1] = b.y, t.s[4 * i + 2] = b.z, t.s[4 * i + 3] = b.w;
  }
}

__device__ __forceinline__ void turn_pair(float& x, float& y, float c, float s) {
  const float a = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
  x = a;
}

// The chunk's sixteen values, rotated: lo[0..7] from r.lo, hi[0..7] from r.hi.
__device__ __forceinline__ void turn_chunk(float (&lo)[8], float (&hi)[8], const Turn& t,
                                           int interleaved) {
  if (!interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) turn_pair(lo[i], hi[i], t.c[i], t.s[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      turn_pair(lo[2 * i], lo[2 * i + 1], t.c[i], t.s[i]);
      turn_pair(hi[2 * i], hi[2 * i + 1], t.c[4 + i], t.s[4 + i]);
    }
  }
}

__device__ __forceinline__ int clamp_position(int pos, int max_pos, uint32_t* err) {
  if (pos >= 0 && pos < max_pos) return pos;
  atomicOr(err, (uint32_t)MOE_DEVERR_POSITION);
  return pos < 0 ? 0 : max_pos - 1;
}

// Rows [start, end) of sequence b's new tokens (kept inside [0, T]).
__device__ __forceinline__ int2 new_rows(const moe_seq_batch& b, int i, int T) {
  const int s = min(max(b.q_offsets[i], 0), T);
  return make_int2(s, min(max(b.q_offsets[i + 1], s), T));
}

// The least e with a <= 448 * 2^e, within [-64, 119] (a = 0: -64; infinite: 119).
__device__ __forceinline__ int scale_exponent(float a) {
  if (!(a > 0.0f)) return -64;
  if (a > 3.0e38f) return 119;
  int e;
  const float m = frexpf(a, &e);               // a = m * 2^e, m in [0.5, 1); 448 = 0.875 * 2^9
  e = m <= 0.875f ? e - 9 : e - 8;
  return min(max(e, -64), 119);
}

struct Item {
  int row0, rows, slot0;     // token rows of the page's new tokens, first slot they take
  int place0;                // place of the first in its sequence
  int64_t page;              // -1: nothing to do
};

// Page item `it` of the batch (items run over the sequences' touched pages in order). All
// threads of the block call it.
__device__ Item find_item(const KvAppendArgs& a, int it) {
  __shared__ int s_warp[kThreads / 32];
  __shared__ int s_hit[3];
  const int P = a.c.page_size;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) s_hit[0] = -1;
  int base = 0;
  Item r = {0, 0, 0, 0, -1};
  for (int b0 = 0; b0 < a.b.B; b0 += kThreads) {
    const int b = b0 + tid;
    int pages = 0, start = 0;
    int2 rows = make_int2(0, 0);
    if (b < a.b.B) {
      rows = new_rows(a.b, b, a.T);
      const int n = rows.y - rows.x, len = a.b.seq_lens[b];
      start = len - n;
      if (len < n) {                           // (not by start, which may wrap)
        // more new tokens than the sequence is long: the first ones have no place
        if (n > 0) atomicOr(a.err, (uint32_t)MOE_DEVERR_PAGE);
        start = 0;
      }
      const long long cap = (long long)a.b.max_pages * P;
      if (n > 0 && len > cap) atomicOr(a.err, (uint32_t)MOE_DEVERR_PAGE);
      const int end = (int)min((long long)len, cap);
      if (n > 0 && end > start) pages = (end - 1) / P - start / P + 1;
    }
    int sum = pages;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += up;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    int before = base, total = base;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += s_warp[w];
      total += s_warp[w];
    }
    const int first = before + sum - pages;
    if (it >= first && it < first + pages) {
      s_hit[0] = b;
      s_hit[1] = it - first;
    }
    __syncthreads();
    if (s_hit[0] >= 0) {
      const int hb = s_hit[0];
      const int2 hr = new_rows(a.b, hb, a.T);
      const int len = a.b.seq_lens[hb], lead = len - (hr.y - hr.x);
      const int pi = max(lead, 0) / P + s_hit[1];
      const int z0 = max(max(lead, 0), pi * P);
      const int z1 = (int)min((long long)len, (long long)(pi + 1) * P);
      r.place0 = z0;
      r.row0 = hr.x + (z0 - lead);
      r.rows = z1 - z0;
      r.slot0 = z0 - pi * P;
      r.page = a.b.page_table[(int64_t)hb * a.b.table_stride + pi];
      if (r.page < 0 || r.page >= a.c.num_pages) {
        if (tid == 0) atomicOr(a.err, (uint32_t)MOE_DEVERR_PAGE);
        r.page = -1;
      }
      return r;
    }
    base = total;
    __syncthreads();                            // s_warp is written again
    if (it < base) break;
  }
  return r;
}

// The chunk of 16 values of a page's new token, rotated if it is K's.
template <int DT>
__device__ __forceinline__ void page_chunk(const KvAppendArgs& a, const Item& it, int head,
                                           bool is_k, int tok, const Chunk& c, float (&lo)[8],
                                           float (&hi)[8]) {
  const int64_t row = it.row0 + tok;
  const uint16_t* src = (is_k ? a.k + row * a.k_stride : a.v + row * a.v_stride) +
                        (int64_t)head * a.c.head_dim;
  unpack8<DT>(*reinterpret_cast<const uint4*>(src + c.lo), lo);
  unpack8<DT>(*reinterpret_cast<const uint4*>(src + c.hi), hi);
  if (is_k && c.col >= 0) {
    const int pos = clamp_position(a.positions ? a.positions[row] : it.place0 + tok, a.max_pos, a.err);
    Turn t;
    load_turn(t, a.cos, a.sin, (int64_t)pos * (a.rotary / 2), c);
    turn_chunk(lo, hi, t, a.interleaved);
  }
}

// v / scale for E4M3: a power-of-two scale divides exactly like a product with its reciprocal.
__device__ __forceinline__ uint2 quant8(const float (&v)[8], float scale, float inv, bool pow2) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = pow2 ? __fmul_rn(v[i], inv) : __fdiv_rn(v[i], scale);
  return make_uint2(f32x2_to_e4m3x2(q[0], q[1]) | (f32x2_to_e4m3x2(q[2], q[3]) << 16),
                    f32x2_to_e4m3x2(q[4], q[5]) | (f32x2_to_e4m3x2(q[6], q[7]) << 16));
}

// KEEP: chunks per thread that stay in registers between the largest magnitude and the codes (a
// page of up to KEEP * 256 chunks; larger ones are read and rotated twice).
template <int DT, int KEEP>
__device__ __forceinline__ void page_block(const KvAppendArgs& a, int it_index, int head, bool is_k) {
  __shared__ uint32_t s_peak;
  if (threadIdx.x == 0) s_peak = 0;
  const Item it = find_item(a, it_index);
  if (it.page < 0) return;                      // the same for the whole block
  const int D = a.c.head_dim, P = a.c.page_size, per = D / 16, log_per = 31 - __clz(per);
  const int rotary = is_k ? a.rotary : 0, inter = a.interleaved, count = it.rows * per;
  float* scale_at = (is_k ? a.c.k_scales : a.c.v_scales) + it.page * a.c.kv_heads + head;
  uint8_t* codes = (is_k ? a.c.k_codes : a.c.v_codes) + it.page * a.c.page_stride +
                   (int64_t)head * P * D;
  const float old = *scale_at;
  const bool kept = count <= KEEP * kThreads;
  float lo[KEEP][8], hi[KEEP][8];
  float peak = 0.0f;
  auto raise = [&](const float (&x)[8], const float (&y)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) peak = fmaxf(peak, fmaxf(fabsf(x[i]), fabsf(y[i])));
  };
  if (kept) {
#pragma unroll
    for (int n = 0; n < KEEP; ++n) {
      const int u = threadIdx.x + n * kThreads;
      if (u < count) {
        page_chunk<DT>(a, it, head, is_k, u >> log_per, chunk_at(u & (per - 1), D, rotary, inter), lo[n], hi[n]);
        raise(lo[n], hi[n]);
      }
    }
  } else {
    for (int u = threadIdx.x; u < count; u += kThreads) {
      page_chunk<DT>(a, it, head, is_k, u >> log_per, chunk_at(u & (per - 1), D, rotary, inter), lo[0], hi[0]);
      raise(lo[0], hi[0]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) peak = fmaxf(peak, __shfl_xor_sync(0xffffffffu, peak, o));
  // magnitudes are not negative, so their bits order as they do
  if ((threadIdx.x & 31) == 0) atomicMax(&s_peak, __float_as_uint(peak));
  __syncthreads();
  const float fresh = pow2f(scale_exponent(__uint_as_float(s_peak)));
  const float scale = it.slot0 == 0 ? fresh : fmaxf(old, fresh);
  if (it.slot0 > 0 && scale > old) {
    const float ratio = __fdiv_rn(old, scale);
    for (int u = threadIdx.x; u < it.slot0 * per; u += kThreads) {
      uint4* at = reinterpret_cast<uint4*>(codes) + u;
      const uint4 v = *at;
      uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 p = e4m3x2_to_f32x2(w[i] & 0xffffu), q = e4m3x2_to_f32x2(w[i] >> 16);
        w[i] = f32x2_to_e4m3x2(__fmul_rn(p.x, ratio), __fmul_rn(p.y, ratio)) |
               (f32x2_to_e4m3x2(__fmul_rn(q.x, ratio), __fmul_rn(q.y, ratio)) << 16);
      }
      *at = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  // 2^-126 .. 2^126: the reciprocal is a normal float too
  const uint32_t bits = __float_as_uint(scale);
  const bool pow2 = (bits & 0x807fffffu) == 0 && bits >= 0x00800000u && bits <= 0x7e800000u;
  const float inv = pow2 ? __uint_as_float(0x7f000000u - bits) : 0.0f;
  auto put = [&](int u, const float (&x)[8], const float (&y)[8]) {
    const Chunk c = chunk_at(u & (per - 1), D, rotary, inter);
    uint8_t* dst = codes + (int64_t)(it.slot0 + (u >> log_per)) * D;
    *reinterpret_cast<uint2*>(dst + c.lo) = quant8(x, scale, inv, pow2);
    *reinterpret_cast<uint2*>(dst + c.hi) = quant8(y, scale, inv, pow2);
  };
  if (kept) {
#pragma unroll
    for (int n = 0; n < KEEP; ++n) {
      const int u = threadIdx.x + n * kThreads;
      if (u < count) put(u, lo[n], hi[n]);
    }
  } else {
    for (int u = threadIdx.x; u < count; u += kThreads) {
      page_chunk<DT>(a, it, head, is_k, u >> log_per, chunk_at(u & (per - 1), D, rotary, inter), lo[0], hi[0]);
      put(u, lo[0], hi[0]);
    }
  }
  if (threadIdx.x == 0) *scale_at = scale;
}

// The sequence of token row t: the one b with q_offsets[b] <= t < q_offsets[b+1].
__device__ __forceinline__ int sequence_of(const moe_seq_batch& b, int t) {
  int lo = 0, hi = b.B - 1;                     // last b with q_offsets[b] <= t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(b.q_offsets + mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <int DT>
__device__ void query_block(const KvAppendArgs& a, int block, int heads_per) {
  const int D = a.c.head_dim, per = D / 16, log_per = 31 - __clz(per);
  const int groups = (a.q_heads + heads_per - 1) / heads_per;
  const int64_t u = (int64_t)block * kThreads + threadIdx.x;
  const int ch = (int)(u & (per - 1));
  const int tg = (int)(u >> log_per);           // T * q_heads < 2^31 is checked by the host
  const int g = tg % groups, t = tg / groups;
  if (t >= a.T) return;
  const Chunk c = chunk_at(ch, D, a.rotary, a.interleaved);
  const int h0 = g * heads_per, h1 = min(a.q_heads, h0 + heads_per);
  const uint16_t* src = a.q + (int64_t)t * a.q_stride;
  uint16_t* dst = a.q_out + (int64_t)t * a.q_out_stride;
  constexpr int kAhead = 4;                     // heads in flight
  uint4 lo[kAhead], hi[kAhead];
  auto ask = [&](int h) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (h + i < h1) {
        lo[i] = *reinterpret_cast<const uint4*>(src + (int64_t)(h + i) * D + c.lo);
        hi[i] = *reinterpret_cast<const uint4*>(src + (int64_t)(h + i) * D + c.hi);
      }
  };
  ask(h0);
  Turn turn;
  if (c.col >= 0) {
    int pos;
    if (a.positions) {
      pos = a.positions[t];
    } else {
      const int b = sequence_of(a.b, t);
      pos = a.b.seq_lens[b] - a.b.q_offsets[b + 1] + t;
    }
    pos = clamp_position(pos, a.max_pos, a.err);
    load_turn(turn, a.cos, a.sin, (int64_t)pos * (a.rotary / 2), c);
  }
  for (int h = h0; h < h1; h += kAhead) {
    if (h > h0) ask(h);
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (h + i < h1) {
        if (c.col >= 0) {
          float x[8], y[8];
          unpack8<DT>(lo[i], x);
          unpack8<DT>(hi[i], y);
          turn_chunk(x, y, turn, a.interleaved);
          lo[i] = pack8<DT>(x), hi[i] = pack8<DT>(y);
        }
        *reinterpret_cast<uint4*>(dst + (int64_t)(h + i) * D + c.lo) = lo[i];
        *reinterpret_cast<uint4*>(dst + (int64_t)(h + i) * D + c.hi) = hi[i];
      }
  }
}

template <int DT>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvAppendArgs a, int page_blocks,
                                                            int heads_per) {
  if ((int)blockIdx.x < page_blocks) {
    const int plane = blockIdx.x % (2 * a.c.kv_heads);
    page_block<DT, 2>(a, blockIdx.x / (2 * a.c.kv_heads), plane >> 1, (plane & 1) == 0);
  } else {
    query_block<DT>(a, blockIdx.x - page_blocks, heads_per);
  }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, int dtype, cudaStream_t s) {
  // A sequence's n > 0 new tokens touch at most (n - 1) / page + 2 pages and at most n.
  const long long seqs = a.b.B < a.T ? a.b.B : a.T;
  long long items = (a.T - seqs) / a.c.page_size + 2 * seqs;
  if (items > a.T) items = a.T;
  const long long page_blocks = items * 2 * a.c.kv_heads;
  const int per = a.c.head_dim / 16;
  int heads_per = 1;
  while (heads_per < 8 && (long long)a.T * a.q_heads * per > (long long)num_sms() * 2048 * heads_per)
    heads_per *= 2;
  const long long groups = (a.q_heads + heads_per - 1) / heads_per;
  const long long q_blocks = ((long long)a.T * groups * per + kThreads - 1) / kThreads;
  const long long grid = page_blocks + q_blocks;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if (dtype == MOE_DTYPE_BF16)
    kv_append_kernel<MOE_DTYPE_BF16><<<(unsigned)grid, kThreads, 0, s>>>(a, (int)page_blocks, heads_per);
  else
    kv_append_kernel<MOE_DTYPE_F16><<<(unsigned)grid, kThreads, 0, s>>>(a, (int)page_blocks, heads_per);
  return cudaGetLastError();
}

}  // namespace moe
