// Log probabilities of given tokens, entropy, rank and the top alternatives, in one pass
// over the logits.  With c = inv_temperature log2 e and a running maximum m,
//   s = sum 2^(c (x - m)),  q = sum 2^(c (x - m)) c (x - m)
// give lse = m / T + ln s and the entropy ln s - ln 2 q / s; both are kept per lane in
// float32 and rescaled when m grows.  The rank counts lanes' comparisons on the scalar
// unit.  The top list is a sorted list of 64-bit keys (value, then lower index first), one
// entry a lane; a vector of logits is looked at only if it reaches the list's last entry,
// which after a short start happens about top / i times in vector i.
// A row is split over several workgroups when there are few rows, and a second launch joins
// the parts.
#include <cfloat>

#include "fp8.h"

namespace mbq {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

struct LpArgs {
  const void* logits;
  const void* targets;
  float *logprob, *entropy;
  int32_t *rank, *top_ids;
  float* top_logprobs;
  float4* part;    // [t][chunks] m, s, q, rank count
  uint64_t* keys;  // [t][chunks][top]
  int64_t ld;
  int32_t t, v, top, chunks, per;  // per: logits a chunk, a multiple of 8
  float inv_temperature;
  bool wide;
};

__device__ __forceinline__ uint32_t ordered(float x) {  // order of the values as unsigned numbers; -0 as 0
  const uint32_t b = __float_as_uint(x + 0.f);
  return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float(o & 0x80000000u ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ uint64_t key_of(float x, uint32_t i) { return uint64_t(ordered(x)) << 32 | uint32_t(~i); }
__device__ __forceinline__ uint64_t lane_key(uint64_t k, int lane) {
  const uint32_t lo = __builtin_amdgcn_readlane(uint32_t(k), lane), hi = __builtin_amdgcn_readlane(uint32_t(k >> 32), lane);
  return uint64_t(hi) << 32 | lo;
}

// The wave's best 64 keys, descending by lane (0: no entry).
struct TopList {
  uint64_t mine = 0;  // this lane's entry
  uint64_t last = 0;  // entry top - 1
  float floor = -__builtin_inff();  // its value

  __device__ __forceinline__ void insert(uint64_t k, int lane, int top) {
    const int pos = __popcll(__ballot(mine > k));
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, int(uint32_t(mine)), 0x138, 0xF, 0xF, true);  // wave_shr 1
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, int(uint32_t(mine >> 32)), 0x138, 0xF, 0xF, true);
    if (lane == pos) mine = k;
    else if (lane > pos) mine = uint64_t(hi) << 32 | lo;
    last = lane_key(mine, top - 1);
    floor = last ? from_ordered(uint32_t(last >> 32)) : -__builtin_inff();
  }
  // Offers one key a lane (0: none).
  __device__ __forceinline__ void offer(uint64_t k, int lane, int top) {
    uint64_t m = __ballot(k > last);
    while (m) {
      insert(lane_key(k, __builtin_ctzll(m)), lane, top);
      m &= m - 1;
      m &= __ballot(k > last);
    }
  }
};

// Joins (m, s, q) of two sets; an empty set has s = q = 0 and any finite m.
__device__ __forceinline__ void join_sums(float c, float& m, float& s, float& q, float m2, float s2, float q2) {
  const float mn = fmaxf(m, m2);
  // -1e4: far below the range of 2^x, and finite, so that an empty set's 0 stays 0
  const float d1 = fmaxf((m - mn) * c, -1e4f), d2 = fmaxf((m2 - mn) * c, -1e4f);
  const float f1 = __builtin_amdgcn_exp2f(d1), f2 = __builtin_amdgcn_exp2f(d2);
  q = f1 * fmaf(d1, s, q) + f2 * fmaf(d2, s2, q2);
  s = f1 * s + f2 * s2;
  m = mn;
}

__device__ __forceinline__ void wave_join(float c, float& m, float& s, float& q) {
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    const float m2 = __shfl_xor(m, o), s2 = __shfl_xor(s, o), q2 = __shfl_xor(q, o);
    join_sums(c, m, s, q, m2, s2, q2);
  }
}

__device__ __forceinline__ int64_t target_of(const LpArgs& a, int row) {
  return a.wide ? static_cast<const int64_t*>(a.targets)[row] : static_cast<const int32_t*>(a.targets)[row];
}

template <bool BF16>
__device__ __forceinline__ float logit(const LpArgs& a, int row, int64_t i) {
  return load_x(a.logits, size_t(row) * size_t(a.ld) + size_t(i), BF16);
}

// Writes a row's results from its sums and its top list (one wave).
template <bool BF16>
__device__ __forceinline__ void finish(const LpArgs& a, int row, float m, float s, float q, int count,
                                       const TopList& list, int lane) {
  const int64_t target = target_of(a, row);
  const bool valid = target >= 0 && target < a.v;
  const bool none = s == 0.f, bad = s != s;  // nothing but -infinity; a NaN or +infinity
  const float log_s = logf(s), inf = __builtin_inff();
  if (lane == 0) {
    const float xt = valid ? logit<BF16>(a, row, target) : 0.f;
    a.logprob[row] = !valid ? 0.f : none ? -inf : (xt - m) * a.inv_temperature - log_s;
    a.entropy[row] = none ? 0.f : log_s - 0.69314718f * (q / s);
    a.rank[row] = valid && !bad ? count + 1 : 0;
  }
  if (lane < a.top) {
    const float x = from_ordered(uint32_t(list.mine >> 32));
    a.top_ids[int64_t(row) * a.top + lane] = bad ? -1 : int32_t(~uint32_t(list.mine));
    a.top_logprobs[int64_t(row) * a.top + lane] = none ? -inf : bad ? s : (x - m) * a.inv_temperature - log_s;
  }
}

template <bool BF16, bool TOP>
__global__ __launch_bounds__(kThreads) void part_kernel(LpArgs a) {
  __shared__ float4 sums[kWaves];
  __shared__ uint64_t lists[TOP ? kWaves : 1][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row = blockIdx.x / a.chunks, chunk = blockIdx.x % a.chunks;
  const uint8_t* base = static_cast<const uint8_t*>(a.logits) + int64_t(row) * a.ld * (BF16 ? 2 : 4);
  const int begin = chunk * a.per, end = min(begin + a.per, a.v);
  const float c = a.inv_temperature * 1.4426950408889634f;
  const int64_t tg = target_of(a, row);
  const int target = tg >= 0 && tg < a.v ? int(tg) : -1;
  const float xt = target >= 0 ? logit<BF16>(a, row, target) : __builtin_inff();
  // x > xt as x >= the next value above it
  const float above = target >= 0 ? from_ordered(ordered(xt) + 1) : __builtin_inff();

  float m = -FLT_MAX, s = 0.f, q = 0.f;
  int count = 0, tied = 0;
  TopList list;
  constexpr int U = 4;
  for (int i0 = begin; i0 < end; i0 += kThreads * 8 * U) {
    float v[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + (u * kThreads + int(threadIdx.x)) * 8;
      if (i + 8 <= end) {
        load8<BF16>(base, i, end, v[u]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          v[u][e] = i + e < end ? load_x(base, size_t(i + e), BF16) : -__builtin_inff();
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + (u * kThreads + int(threadIdx.x)) * 8;
      const float (&x)[8] = v[u];
      const float best = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
      const float mn = fmaxf(m, best);
      const float shift = fmaxf((m - mn) * c, -1e4f), f = __builtin_amdgcn_exp2f(shift);
      q = f * fmaf(shift, s, q);
      s *= f;
      m = mn;
      // a chunk ends on a vector; what is read past it counts for nothing
      const float bound = i >= end ? __builtin_inff() : i + 8 <= target ? xt : above;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = (x[e] - mn) * c, p = __builtin_amdgcn_exp2f(d);
        s += p;
        q = fmaf(p, fmaxf(d, -1e4f), q);  // finite, so that p = 0 adds 0
        count += __popcll(__ballot(x[e] >= bound));
      }
      if (target >= i && target < i + 8) {  // the vector that holds the target: equal logits before it
#pragma unroll
        for (int e = 0; e < 8; ++e) tied += i + e < target && x[e] == xt;
      }
      if constexpr (TOP) {
        if (__ballot(best >= list.floor && i < end)) {
#pragma unroll
          for (int e = 0; e < 8; ++e) list.offer(i + e < end && x[e] == x[e] ? key_of(x[e], uint32_t(i + e)) : 0, lane, a.top);
        }
      }
    }
  }
  wave_join(c, m, s, q);
#pragma unroll
  for (int o = 32; o; o >>= 1) tied += __shfl_xor(tied, o);
  count += tied;
  if (lane == 0) sums[wave] = make_float4(m, s, q, __int_as_float(count));
  if constexpr (TOP) lists[wave][lane] = list.mine;
  __syncthreads();
  if (wave) return;
#pragma unroll
  for (int w = 1; w < kWaves; ++w) {
    join_sums(c, m, s, q, sums[w].x, sums[w].y, sums[w].z);
    count += __float_as_int(sums[w].w);
    if constexpr (TOP) list.offer(lane < a.top ? lists[w][lane] : 0, lane, a.top);
  }
  if (a.chunks == 1) {
    finish<BF16>(a, row, m, s, q, count, list, lane);
  } else {
    const int64_t at = int64_t(row) * a.chunks + chunk;
    if (lane == 0) a.part[at] = make_float4(m, s, q, __int_as_float(count));
    if (TOP && lane < a.top) a.keys[at * a.top + lane] = list.mine;
  }
}

template <bool BF16>
__global__ __launch_bounds__(64) void merge_kernel(LpArgs a) {
  const int row = blockIdx.x, lane = threadIdx.x;
  const float c = a.inv_temperature * 1.4426950408889634f;
  float m = -FLT_MAX, s = 0.f, q = 0.f;
  int count = 0;
  if (lane < a.chunks) {  // chunks <= 64
    const float4 p = a.part[int64_t(row) * a.chunks + lane];
    m = p.x;
    s = p.y;
    q = p.z;
    count = __float_as_int(p.w);
  }
  wave_join(c, m, s, q);
#pragma unroll
  for (int o = 32; o; o >>= 1) count += __shfl_xor(count, o);
  TopList list;
  const int all = a.chunks * a.top;
  for (int i = 0; i < all; i += 64)
    list.offer(i + lane < all ? a.keys[int64_t(row) * all + i + lane] : 0, lane, a.top);
  finish<BF16>(a, row, m, s, q, count, list, lane);
}

constexpr int kMaxChunks = 64;

// Parts of a row: enough workgroups for four on every compute unit, each with at least one
// full step of its loop.
int chunks_of(int32_t t, int32_t v) {
  const int64_t want = (1024 + int64_t(t) - 1) / std::max(t, 1);
  const int64_t most = (int64_t(v) + kThreads * 32 - 1) / (kThreads * 32);
  return int(std::max<int64_t>(1, std::min<int64_t>(std::min(want, most), kMaxChunks)));
}

}  // namespace

size_t token_logprobs_workspace(int32_t t, int32_t v, int32_t top) {
  const int c = chunks_of(t, v);
  return t == 0 || c == 1 ? 0 : size_t(t) * c * (16 + 8 * size_t(top));
}

hipError_t launch_token_logprobs(int32_t t, int32_t v, const void* logits, bool bf16, int64_t ld, const void* targets,
                                 bool wide, float inv_temperature, int32_t top, float* logprob, float* entropy,
                                 int32_t* rank, int32_t* top_ids, float* top_logprobs, void* ws, hipStream_t stream) {
  if (t == 0) return hipSuccess;
  LpArgs a{};
  a.logits = logits;
  a.targets = targets;
  a.logprob = logprob;
  a.entropy = entropy;
  a.rank = rank;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  a.ld = ld;
  a.t = t;
  a.v = v;
  a.top = top;
  a.chunks = chunks_of(t, v);
  a.per = ((v + a.chunks - 1) / a.chunks + 7) / 8 * 8;
  a.part = static_cast<float4*>(ws);
  a.keys = reinterpret_cast<uint64_t*>(a.part + int64_t(t) * a.chunks);
  a.inv_temperature = inv_temperature;
  a.wide = wide;
  const dim3 grid(uint32_t(t) * uint32_t(a.chunks));
  if (bf16) {
    if (top) part_kernel<true, true><<<grid, kThreads, 0, stream>>>(a);
    else part_kernel<true, false><<<grid, kThreads, 0, stream>>>(a);
    if (a.chunks > 1) merge_kernel<true><<<t, 64, 0, stream>>>(a);
  } else {
    if (top) part_kernel<false, true><<<grid, kThreads, 0, stream>>>(a);
    else part_kernel<false, false><<<grid, kThreads, 0, stream>>>(a);
    if (a.chunks > 1) merge_kernel<false><<<t, 64, 0, stream>>>(a);
  }
  return hipGetLastError();
}

}  // namespace mbq
