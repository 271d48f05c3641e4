// Verification of drafted tokens with given random numbers (moe_verify_draft).
//
// Bound by one row of the target's probabilities (and one of the draft's after a refusal) per
// sequence. The row is cut into chunks for several blocks, so that few sequences still fill the GPU.
// Every block finds the row for itself (lane i of its first warp tests drafted tokens i and
// 32 + i; the first refusal is the lowest bit of two ballots), sums the masses of its chunks and
// leaves the sums in the workspace. The last block of a sequence to arrive finds the chunk that
// holds the goal and walks that chunk alone (and in the rare case that nothing is left after a
// refusal's difference, sums the row itself first). Masses are whole numbers and their sums wrap
// nowhere (V <= 2^22 masses of at most 2^40), so neither the order of summation nor that of
// arrival shows in the result.
//
// Measured: 64 sequences of 8 drafts, 151937 tokens, f32, with draft rows: 21.7 us, 2.7 TB/s: the
// masses' integer work, and about 5 us of testing drafts, arrival and the last block's walk; one
// sequence of 32003 tokens: 6.0 us, latency alone.
#include "serving.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// The row is cut into chunks whose sums the last block chooses from, and a block takes `per` of them
// in turn: 1024 tokens and one each while that leaves at most 8 blocks per SM of a 152-SM GPU (a constant:
// the workspace's size must not depend on the GPU that is asked),
// else 2048 and as many as bring the grid down to that (the test of the drafts and the arrival
// are then paid once for several chunks: 64 sequences of 151937 took 35.6 us with a block per
// 4096 tokens, four waves of them).
constexpr int kBlocks = 8 * 152;
struct Cut {
  int chunk, chunks, per;
};
Cut cut_of(int B, int V) {
  Cut c = {1024, (V + 1023) / 1024, 1};
  if ((long long)B * c.chunks > kBlocks) {
    c.chunk = 2048;
    c.chunks = (V + 2047) / 2048;
    c.per = (int)(((long long)B * c.chunks + kBlocks - 1) / kBlocks);
  }
  return c;
}

// Workspace: error word, arrival counters of up to 2^16 sequences (their place does not depend
// on the sizes, so a workspace serves smaller calls too), chunk sums.
constexpr size_t kSumsAt = kAlign + 65536 * 4;

template <int DT>
__device__ __forceinline__ float prob(const void* row, int64_t at) {
  if (DT == MOE_DTYPE_F32) return __ldg(static_cast<const float*>(row) + at);
  return act_to_f32<DT>(__ldg(static_cast<const uint16_t*>(row) + at));
}

// floor(min(w, 1) * 2^40); 0 for NaN and negative weights. On whole numbers: the
// conversion from f32 to 64-bit integers kept the double-precision pipe busy and bound the kernel.
__device__ __forceinline__ unsigned long long mass_of(float w) {
  const uint32_t bits = __float_as_uint(fminf(fmaxf(w, 0.0f), 1.0f));       // 0 <= w <= 1
  // w = m * 2^(e - 150), m the mantissa with its leading bit (w = 0 and subnormals fall below)
  const uint32_t down = 127u - (bits >> 23);                                // 0 .. 127
  const unsigned long long m = (unsigned long long)((bits & 0x7fffffu) | 0x800000u) << 17;
  return down < 64u ? m >> down : 0ull;
}

template <class T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct Row {
  const void *target, *draft;      // the row drawn from and the draft's beside it, or null
  int left_out;                    // a token without its unit of draft mass, or -1
};
template <int DT, int EACH>
__global__ void __launch_bounds__(kThreads) verify_kernel(const VerifyArgs a, int chunks, int per) {
  constexpr int kChunk = EACH * kThreads;
  constexpr int kBatch = EACH < 8 ? EACH : 8;    // loads in flight per thread (and row)
  __shared__ unsigned long long s_warp[kWarps];
  __shared__ int s_count, s_last, s_chunk, s_token, s_back;
  __shared__ unsigned long long s_before, s_goal;
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t* err = reinterpret_cast<uint32_t*>(a.ws);
  uint32_t* arrived = reinterpret_cast<uint32_t*>(a.ws + kAlign);
  unsigned long long* sums = reinterpret_cast<unsigned long long*>(a.ws + kSumsAt) + (size_t)b * chunks;
  const int n = a.n_draft ? min(max(a.n_draft[b], 0), a.n) : a.n;
  const int64_t size = DT == MOE_DTYPE_F32 ? 4 : 2;
  const char* target = static_cast<const char*>(a.target) + (int64_t)b * (a.n + 1) * a.target_stride * size;
  const char* draft = a.draft ? static_cast<const char*>(a.draft) + (int64_t)b * a.n * a.draft_stride * size : nullptr;
  const int32_t* ids = a.draft_ids + (int64_t)b * a.n;
  if (warp == 0) {
    uint32_t refused[2] = {0, 0};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (32 * h >= a.n) break;
      const int i = 32 * h + lane;
      bool no = false, odd = false;
      if (i < a.n) {
        const int id = ids[i];
        const float u = a.u_accept[(int64_t)b * a.n + i];
        odd = id < 0 || id >= a.V;
        no = odd;
        if (!odd) {
          const float q = draft ? prob<DT>(draft, i * a.draft_stride + id) : 1.0f;
          no = !(__fmul_rn(u, q) < prob<DT>(target, i * a.target_stride + id));
        }
      }
      refused[h] = __ballot_sync(0xffffffffu, no && i < n);
      const uint32_t odds = __ballot_sync(0xffffffffu, odd && i < n);
      // an id out of range counts where it is the first refusal
      if (lane == 0 && blockIdx.x == 0 && (h == 0 || refused[0] == 0) &&
          (odds & refused[h] & (0u - refused[h])))
        atomicOr(err, (uint32_t)MOE_DEVERR_TOKEN);
    }
    if (lane == 0)
      s_count = refused[0] ? __ffs(refused[0]) - 1 : refused[1] ? 31 + __ffs(refused[1]) : n;
  }
  __syncthreads();
  const int count = s_count;
  const bool refused = count < n;
  Row r;
  r.target = target + count * a.target_stride * size;
  r.draft = refused && draft ? draft + count * a.draft_stride * size : nullptr;
  r.left_out = refused && !draft ? ids[count] : -1;

  // The masses of tokens from, from + step, ... (EACH of them) below `to`.
  auto masses = [&](int from, int step, int to, unsigned long long (&m)[EACH]) {
#pragma unroll
    for (int i0 = 0; i0 < EACH; i0 += kBatch) {
      float w[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int v = from + (i0 + i) * step;
        w[i] = v < to ? prob<DT>(r.target, v) : 0.0f;
      }
      if (r.draft) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int v = from + (i0 + i) * step;
          w[i] = v < to ? __fsub_rn(w[i], prob<DT>(r.draft, v)) : 0.0f;
        }
      } else {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
          if (from + (i0 + i) * step == r.left_out) w[i] = __fsub_rn(w[i], 1.0f);
      }
      // masses below 2^32 (all but the likeliest tokens') by one conversion each
      float most = 0.0f;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) most = fmaxf(most, w[i]);
      if (most < 0x1p-8f) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) m[i0 + i] = __float2uint_rz(fmaxf(w[i], 0.0f) * 0x1p40f);
      } else {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) m[i0 + i] = mass_of(w[i]);
      }
    }
  };
  auto block_total = [&](unsigned long long v) {       // of every thread; all threads call it
    v = warp_sum(v);
    __syncthreads();
    if (lane == 0) s_warp[warp] = v;
    __syncthreads();
    v = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) v += s_warp[w];
    return v;
  };
  auto chunk_total = [&](int x) {
    unsigned long long m[EACH], sum = 0;
    masses(x * kChunk + tid, kThreads, a.V, m);
#pragma unroll
    for (int i = 0; i < EACH; ++i) sum += m[i];
    return block_total(sum);
  };

  // ---- this block's chunks ----
  for (int x = blockIdx.x * per; x < min((int)(blockIdx.x + 1) * per, chunks); ++x) {
    const unsigned long long sum = chunk_total(x);
    if (tid == 0) sums[x] = sum;
  }
  if (tid == 0) {
    __threadfence();
    s_last = atomicAdd(&arrived[b], 1u) == gridDim.x - 1;
    if (s_last) arrived[b] = 0;                  // ready for the next call
    s_token = -1;
    s_chunk = -1;
  }
  __syncthreads();
  if (!s_last) return;
  __threadfence();

  // ---- the last block: total, goal, chunk, token ----
  auto find_chunk = [&]() {                      // first warp; whether there is any mass
    unsigned long long total = 0;
    for (int i = lane; i < chunks; i += 32) total += __ldcg(sums + i);
    total = warp_sum(total);
    const float u = fminf(fmaxf(a.u_sample[b], 0.0f), 1.0f);
    unsigned long long m = __float2ull_rz(u * 16777216.0f);
    if (m > 16777215ull) m = 16777215ull;
    const unsigned long long goal = m * (total >> 24) + ((m * (total & 0xffffffull)) >> 24);
    unsigned long long before = 0;
    for (int i0 = 0; i0 < chunks && total > 0; i0 += 32) {
      const unsigned long long x = i0 + lane < chunks ? __ldcg(sums + i0 + lane) : 0;
      unsigned long long run = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long up = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += up;
      }
      const uint32_t past = __ballot_sync(0xffffffffu, before + run > goal);
      if (past) {
        if (lane == __ffs(past) - 1) s_chunk = i0 + lane, s_before = before + run - x;
        break;
      }
      before += __shfl_sync(0xffffffffu, run, 31);
    }
    if (lane == 0) s_goal = goal;
    return total > 0;
  };
  if (warp == 0) {
    const bool any = find_chunk();
    if (lane == 0) s_back = !any;
  }
  __syncthreads();
  if (s_back && refused) {                       // nothing left after the difference
    r.draft = nullptr, r.left_out = -1;
    for (int x = 0; x < chunks; ++x) {
      const unsigned long long sum = chunk_total(x);
      if (tid == 0) __stcg(sums + x, sum);
    }
    __threadfence();
    __syncthreads();
    if (warp == 0) {
      const bool any = find_chunk();
      if (lane == 0) s_back = !any;
    }
    __syncthreads();
  }
  if (s_chunk >= 0) {
    // a thread takes EACH consecutive tokens
    const int v0 = s_chunk * kChunk + tid * EACH;
    unsigned long long m[EACH], mine = 0;
    masses(v0, 1, a.V, m);
#pragma unroll
    for (int i = 0; i < EACH; ++i) mine += m[i];
    unsigned long long run = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long up = __shfl_up_sync(0xffffffffu, run, o);
      if (lane >= o) run += up;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = run;
    __syncthreads();
    unsigned long long at = s_before + run - mine;
    for (int w = 0; w < warp; ++w) at += s_warp[w];
    if (at <= s_goal && at + mine > s_goal) {    // one thread
      int token = v0;
#pragma unroll
      for (int i = 0; i < EACH; ++i) {
        at += m[i];
        if (at <= s_goal) token = v0 + i + 1;
      }
      s_token = token;
    }
  }
  __syncthreads();
  if (tid == 0) {
    a.n_accepted[b] = count;
    if (s_back) atomicOr(err, (uint32_t)MOE_DEVERR_PROBS);
  }
  for (int i = tid; i <= a.n; i += kThreads)
    a.out_ids[(int64_t)b * (a.n + 1) + i] = i < count ? ids[i] : i == count ? s_token : -1;
}

template <int DT>
cudaError_t launch_chunk(const VerifyArgs& a, cudaStream_t s) {
  const Cut c = cut_of(a.B, a.V);
  const dim3 grid((c.chunks + c.per - 1) / c.per, a.B);
  if (c.chunk == 1024) verify_kernel<DT, 4><<<grid, kThreads, 0, s>>>(a, c.chunks, c.per);
  else verify_kernel<DT, 8><<<grid, kThreads, 0, s>>>(a, c.chunks, c.per);
  return cudaGetLastError();
}

}  // namespace

size_t verify_ws_bytes(int B, int V) {
  // enough for any smaller B and V: with the smaller chunks there are at most kBlocks
  const size_t most = (size_t)B * ((V + 2047) / 2048);
  return align_up(kSumsAt + (most > kBlocks ? most : kBlocks) * 8);
}

cudaError_t launch_verify(const VerifyArgs& a, int dtype, cudaStream_t s) {
  if (dtype == MOE_DTYPE_F32) return launch_chunk<MOE_DTYPE_F32>(a, s);
  return dtype == MOE_DTYPE_BF16 ? launch_chunk<MOE_DTYPE_BF16>(a, s) : launch_chunk<MOE_DTYPE_F16>(a, s);
}

}  // namespace moe
