// A block of experts around its products: each token's top experts with their weights, the
// token copies grouped by expert, and the experts' outputs added up again per token.
#include "int8.h"

namespace mbq {
namespace {

constexpr int kGroup = 16;     // tokens of a histogram: one count fits a byte, one token a wave
constexpr int kSpan = 4096;    // tokens whose histograms one place workgroup adds up by itself
constexpr int kPlaced = 64;    // tokens of a place workgroup: one bit each in a 64-bit mask
constexpr int kFew = 32;       // most tokens that one workgroup routes by itself
constexpr int kMaxExperts = 1024;

struct RouteArgs {
  const void* logits;
  int64_t ld;
  int32_t t, e, top, normalize;
  float scale;
  int32_t* ids;
  float* weights;
  int32_t *perm, *offsets, *place;
  uint8_t* hist;  // [e][pitch]: tokens of the group of 16 that took the expert
  int64_t pitch;  // groups, rounded up to spans
  int32_t* span;  // beyond one span: [spans + 1][e], tokens before the span that took the expert; last: all
};

constexpr int kSpanGroups = kSpan / kGroup;

// Bits that order as the values do (-0 as +0).
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;  // order_key(-infinity)
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

// One token by one wave: lane l holds logits l V .. l V + V - 1.  Every round takes the wave's
// largest key; among equal ones the lowest lane and in it the lowest element, which is the
// lowest expert.  Lane j keeps the j-th choice.  Returns this lane's choice (-1: none) and its
// weight; a row that holds a NaN or +infinity has no choice and NaN weights.
template <bool BF16, int V, bool SIGMOID>
__device__ __forceinline__ int choose(const RouteArgs& a, int64_t token, float& weight) {
  const int lane = threadIdx.x & 63, e0 = lane * V;
  const uint8_t* row = static_cast<const uint8_t*>(a.logits) + token * a.ld * (BF16 ? 2 : 4);
  uint32_t key[V];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const float v = e0 + i < a.e ? load_x(row, size_t(e0 + i), BF16) : -INFINITY;
    bad |= (__float_as_uint(v) & 0x7FFFFFFFu) > 0x7F800000u || __float_as_uint(v) == 0x7F800000u;
    key[i] = order_key(v);
  }
  if (__ballot(bad)) {
    weight = __uint_as_float(0x7FC00000u);
    return -1;
  }
  uint32_t left[V];
#pragma unroll
  for (int i = 0; i < V; ++i) left[i] = key[i];
  int chosen = -1;
  uint32_t best = kKeyNegInf, top = 0;
  for (int j = 0; j < a.top; ++j) {
    uint32_t m = left[0];
#pragma unroll
    for (int i = 1; i < V; ++i) m = max(m, left[i]);
    const uint32_t all = max64(m);
    if (j == 0) top = all;
    if (all <= kKeyNegInf) break;  // nothing left
    const int l = __builtin_ctzll(__ballot(m == all));
    int at = 0;
#pragma unroll
    for (int i = V - 1; i >= 0; --i)
      if (left[i] == all) at = i;
    if (lane == l) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (i == at) left[i] = 0;
    }
    if (lane == j) best = all;
    const int id = l * V + __builtin_amdgcn_readlane(at, l);
    if (lane == j) chosen = id;
  }
  float score = 0.f, total = 1.f;
  if constexpr (SIGMOID) {
    // normalized scores of negative logits in the form exp(l) / (1 + exp(l)), over exp of the
    // largest, which leaves the quotients and keeps them where every score would vanish
    const float l = key_value(best), high = key_value(top);
    if (chosen >= 0) score = a.normalize && high < 0.f ? expf(l - high) / (1.f + expf(l)) : 1.f / (1.f + expf(-l));
    if (a.normalize) total = sum64(score);
  } else {
    const float high = key_value(top);
    if (chosen >= 0) score = expf(key_value(best) - high);
    if (a.normalize) {
      total = sum64(score);
    } else {
      total = 0.f;
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (key[i] > kKeyNegInf) total += expf(key_value(key[i]) - high);
      total = sum64(total);
    }
  }
  weight = chosen >= 0 ? score / total * a.scale : 0.f;
  return chosen;
}

// The choices of 16 tokens, a wave each, and their histogram.  Bound by the chain of maxima, one
// for each choice (4096 tokens of 128, 8 chosen: 5.2 us).
template <bool BF16, int V, bool SIGMOID>
__global__ __launch_bounds__(1024) void choose_kernel(RouteArgs a) {
  __shared__ uint32_t count[V * 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int i = threadIdx.x; i < a.e; i += 1024) count[i] = 0;
  __syncthreads();
  const int64_t token = int64_t(blockIdx.x) * kGroup + wave;
  if (token < a.t) {
    float weight;
    const int id = choose<BF16, V, SIGMOID>(a, token, weight);
    if (lane < a.top) {
      a.ids[token * a.top + lane] = id;
      a.weights[token * a.top + lane] = weight;
      if (id >= 0) atomicAdd(&count[id], 1u);  // a sum: its order is free
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.e; i += 1024) a.hist[i * a.pitch + blockIdx.x] = uint8_t(count[i]);
}

// The tokens of a span that took each expert: those of groups before `mine` (a multiple of 4)
// into before[e], the others into rest[e].  1024 threads: 2^k a expert, as many as there are, up to
// one for each 16 of the span's 256 groups, summing four groups a instruction.
__device__ __forceinline__ void add_groups(const RouteArgs& a, int64_t span, int mine, int32_t* before, int32_t* rest) {
  int lanes = 16;
  while (lanes * a.e > 1024) lanes >>= 1;
  const int e = threadIdx.x / lanes, l = threadIdx.x - e * lanes;
  const int64_t g0 = span * kSpanGroups, groups = (int64_t(a.t) + kGroup - 1) / kGroup;
  const int there = int(min(groups - g0, int64_t(kSpanGroups)));
  uint32_t s0 = 0, s1 = 0;
  if (e < a.e) {
    const u32x4_t* row = reinterpret_cast<const u32x4_t*>(a.hist + e * a.pitch + g0);
    for (int c = l; c * 16 < there; c += lanes) {
      const u32x4_t v = row[c];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int g = c * 16 + 4 * i, n = there - g;  // bytes past the last group are no counts
        const uint32_t w = n >= 4 ? v[i] : n <= 0 ? 0u : v[i] & (0xFFFFFFFFu >> (8 * (4 - n)));
        const bool late = g >= mine;
        s0 = __builtin_amdgcn_sad_u8(late ? 0u : w, 0u, s0);
        s1 = __builtin_amdgcn_sad_u8(late ? w : 0u, 0u, s1);
      }
    }
  }
  if (lanes > 1) s0 += across<1>(s0), s1 += across<1>(s1);
  if (lanes > 2) s0 += across<2>(s0), s1 += across<2>(s1);
  if (lanes > 4) s0 += across<4>(s0), s1 += across<4>(s1);
  if (lanes > 8) s0 += across<8>(s0), s1 += across<8>(s1);
  if (e < a.e && l == 0) {
    before[e] += int32_t(s0);
    rest[e] += int32_t(s1);
  }
}

// Exclusive sums of the threads' counts, an expert each, to first[0 .. e] (1024 threads, e <= 1024).
__device__ __forceinline__ void scan_experts(int e, int32_t v, int32_t* first) {
  __shared__ int32_t part[16];
  const int tid = threadIdx.x, upto = scan64(v);
  if ((tid & 63) == 63) part[tid >> 6] = upto;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < tid >> 6; ++w) before += part[w];
  if (tid < e) first[tid + 1] = before + upto;
  if (tid == 0) first[0] = 0;
  __syncthreads();
}

// Beyond one span: the tokens of a span that took each expert.
__global__ __launch_bounds__(1024) void span_kernel(RouteArgs a) {
  __shared__ int32_t sums[kMaxExperts], none[kMaxExperts];
  sums[threadIdx.x] = 0;
  __syncthreads();
  add_groups(a, blockIdx.x, kSpanGroups, sums, none);
  __syncthreads();
  if (int(threadIdx.x) < a.e) a.span[int64_t(blockIdx.x) * a.e + threadIdx.x] = sums[threadIdx.x];
}
// One expert a thread: the spans' counts become those of the spans before.
__global__ __launch_bounds__(64) void span_scan_kernel(RouteArgs a, int spans) {
  const int e = blockIdx.x * 64 + threadIdx.x;
  if (e >= a.e) return;
  int32_t before = 0;
#pragma unroll 8
  for (int s = 0; s < spans; ++s) {
    const int32_t v = a.span[int64_t(s) * a.e + e];
    a.span[int64_t(s) * a.e + e] = before;
    before += v;
  }
  a.span[int64_t(spans) * a.e + e] = before;
}

// The places of 64 tokens' copies: behind the copies of the tokens before them that took the
// expert, base[e], and of those among the 64, the bits below the token's in mask[e].
constexpr int kHeld = kPlaced * MBQ_MAX_EXPERT_TOP / 1024;  // copies a thread
struct Held {
  int32_t id[kHeld];
  __device__ __forceinline__ Held(const RouteArgs& a, int64_t t0, int pairs) {
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
      const int i = threadIdx.x + h * 1024;
      id[h] = i < pairs ? a.ids[t0 * a.top + i] : -1;
    }
  }
  __device__ __forceinline__ void mark(const RouteArgs& a, uint64_t* mask) const {
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
      if (id[h] >= 0)
        atomicOr(reinterpret_cast<unsigned long long*>(&mask[id[h]]), 1ull << ((threadIdx.x + h * 1024) / a.top));
  }
  __device__ __forceinline__ void place(const RouteArgs& a, int64_t t0, int pairs, const int32_t* first, const int32_t* base,
                                        const uint64_t* mask) const {
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
      const int i = threadIdx.x + h * 1024, token = i / a.top;
      if (i >= pairs) continue;
      int at = -1;
      if (id[h] >= 0) {
        at = first[id[h]] + base[id[h]] + __popcll(mask[id[h]] & ((uint64_t(1) << token) - 1));
        a.perm[at] = int32_t(t0 + token);
      }
      a.place[t0 * a.top + i] = at;
    }
  }
};

// The places of every 64 tokens' copies, a workgroup each (4096 tokens of 128, 8 chosen: 4.5 us, of
// which a launch and the histograms' way are most).
__global__ __launch_bounds__(1024) void place_kernel(RouteArgs a) {
  __shared__ int32_t base[kMaxExperts], total[kMaxExperts], first[kMaxExperts + 1];
  __shared__ uint64_t mask[kMaxExperts];
  const int tid = threadIdx.x;
  const int64_t t0 = int64_t(blockIdx.x) * kPlaced, s = t0 / kSpan, spans = (int64_t(a.t) + kSpan - 1) / kSpan;
  const bool many = spans > 1;
  const int pairs = int(min(int64_t(kPlaced), a.t - t0)) * a.top;
  const Held held(a, t0, pairs);
  if (tid < a.e) {
    base[tid] = many ? a.span[s * a.e + tid] : 0;
    total[tid] = 0;
    mask[tid] = 0;
  }
  __syncthreads();
  add_groups(a, s, int((t0 - s * kSpan) / kGroup), base, total);
  held.mark(a, mask);
  __syncthreads();
  const int32_t all_of = tid >= a.e ? 0 : many ? a.span[spans * a.e + tid] : total[tid] + base[tid];
  scan_experts(a.e, all_of, first);
  held.place(a, t0, pairs, first, base, mask);
  if (blockIdx.x == 0)
    for (int i = tid; i <= a.e; i += 1024) a.offsets[i] = first[i];
  const int64_t all = int64_t(a.t) * a.top;  // rows of no copy
  for (int64_t i = first[a.e] + int64_t(blockIdx.x) * 1024 + tid; i < all; i += int64_t(gridDim.x) * 1024) a.perm[i] = -1;
}

// At most 32 tokens: everything in one workgroup, two tokens a wave (one token of 64 experts, 6 chosen:
// 3.1 us, a launch).  With launches, us here / by choose and place: 64 experts, 6 chosen: 32 tokens
// 6.1 / 7.0, 64 tokens 9.2 / 7.1; 256 experts, 8 chosen: 32 tokens 9.8 / 9.2, 64 tokens 16.2 / 9.3.
template <bool BF16, int V, bool SIGMOID>
__global__ __launch_bounds__(1024) void route_few_kernel(RouteArgs a) {
  __shared__ int32_t base[kMaxExperts], first[kMaxExperts + 1];
  __shared__ uint64_t mask[kMaxExperts];
  const int tid = threadIdx.x, lane = tid & 63;
  if (tid < a.e) {
    base[tid] = 0;
    mask[tid] = 0;
  }
  __syncthreads();
  for (int token = tid >> 6; token < a.t; token += 16) {
    float weight;
    const int id = choose<BF16, V, SIGMOID>(a, token, weight);
    if (lane < a.top) {
      a.ids[token * a.top + lane] = id;
      a.weights[token * a.top + lane] = weight;
      if (id >= 0) atomicOr(reinterpret_cast<unsigned long long*>(&mask[id]), 1ull << token);
    }
  }
  __threadfence_block();
  __syncthreads();
  scan_experts(a.e, tid < a.e ? __popcll(mask[tid]) : 0, first);
  const Held held(a, 0, a.t * a.top);
  held.place(a, 0, a.t * a.top, first, base, mask);
  for (int i = tid; i <= a.e; i += 1024) a.offsets[i] = first[i];
  for (int i = first[a.e] + tid; i < a.t * a.top; i += 1024) a.perm[i] = -1;
}

// y[t] = residual[t] + sum_j weights[t][j] rows[place[t][j]], eight outputs a thread, the
// copies' rows asked for U at a time.  Bound by traffic (8192 x 4096, 8 copies: 5.4 TB/s), and
// for a few tokens by the way of a place and then a row.  The last piece of a row reads the
// row's last eight elements and keeps those of its own.  A place outside the rows adds its
// weight times 0: nothing, or NaN where the weight is one.
template <bool BF16, bool RBF>
__global__ __launch_bounds__(256) void combine_kernel(int32_t t, int32_t n, int32_t top, int32_t p, const void* __restrict__ rows,
                                                      int64_t ldr, const float* __restrict__ weights,
                                                      const int32_t* __restrict__ place, const void* residual,
                                                      int64_t ldres, void* y, int64_t ldy) {
  constexpr int U = 8;
  const int pieces = (n + 7) / 8;
  const int64_t all = int64_t(t) * pieces;
  for (int64_t b = int64_t(blockIdx.x) * 256 + threadIdx.x; b < all; b += int64_t(gridDim.x) * 256) {
    const int64_t token = b / pieces;
    const int own = int(b - token * pieces) * 8, col = max(min(own, n - 8), 0);
    float v[8], sum[8];
    if (residual) {
      load8<RBF>(static_cast<const uint8_t*>(residual) + token * ldres * (RBF ? 2 : 4), col, n, sum);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] = 0.f;
    }
    for (int j0 = 0; j0 < top; j0 += U) {
      Raw8<BF16> raw[U];
      float w[U];
      int at[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = min(j0 + u, top - 1);
        at[u] = place[token * top + j];
        w[u] = weights[token * top + j];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool there = uint32_t(at[u]) < uint32_t(p) && j0 + u < top;
        if (j0 + u >= top) w[u] = 0.f;
        if (there) {
          raw[u].load(static_cast<const uint8_t*>(rows) + at[u] * ldr * (BF16 ? 2 : 4), col, n);
        } else {
#pragma unroll
          for (int h = 0; h < (BF16 ? 1 : 2); ++h) raw[u].w[h] = u32x4_t{0, 0, 0, 0};
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        raw[u].get(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = fmaf(w[u], v[e], sum[e]);
      }
    }
    uint8_t* out = static_cast<uint8_t*>(y) + token * ldy * (RBF ? 2 : 4);
    if (col == own) {
      store8<RBF>(out, col, n, sum);
    } else {  // the elements before its own are another thread's
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (col + e >= own) {
          if constexpr (RBF) reinterpret_cast<uint16_t*>(out)[col + e] = uint16_t(bf16_pair(sum[e], 0.f));
          else reinterpret_cast<float*>(out)[col + e] = sum[e];
        }
    }
  }
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }
int64_t hist_pitch(int32_t t) { return (int64_t(t) + kSpan - 1) / kSpan * kSpanGroups; }
size_t hist_bytes(int32_t t, int32_t e) { return align256(size_t(hist_pitch(t)) * e); }

template <bool BF16, int V, bool SIGMOID>
void launch_route(const RouteArgs& a, hipStream_t stream) {
  if (a.t <= kFew) {
    route_few_kernel<BF16, V, SIGMOID><<<1, 1024, 0, stream>>>(a);
    return;
  }
  choose_kernel<BF16, V, SIGMOID><<<(a.t + kGroup - 1) / kGroup, 1024, 0, stream>>>(a);
  const int spans = (a.t + kSpan - 1) / kSpan;
  if (spans > 1) {
    span_kernel<<<spans, 1024, 0, stream>>>(a);
    span_scan_kernel<<<(a.e + 63) / 64, 64, 0, stream>>>(a, spans);
  }
  place_kernel<<<(a.t + kPlaced - 1) / kPlaced, 1024, 0, stream>>>(a);
}

template <bool BF16, bool SIGMOID>
void launch_route(const RouteArgs& a, hipStream_t stream) {
  if (a.e <= 64) launch_route<BF16, 1, SIGMOID>(a, stream);
  else if (a.e <= 128) launch_route<BF16, 2, SIGMOID>(a, stream);
  else if (a.e <= 256) launch_route<BF16, 4, SIGMOID>(a, stream);
  else if (a.e <= 512) launch_route<BF16, 8, SIGMOID>(a, stream);
  else launch_route<BF16, 16, SIGMOID>(a, stream);
}

}  // namespace

size_t expert_route_workspace(int32_t t, int32_t e) {
  if (t <= kFew) return 0;
  const int spans = (t + kSpan - 1) / kSpan;
  return hist_bytes(t, e) + (spans > 1 ? align256(size_t(spans + 1) * e * 4) : 0);
}

hipError_t launch_expert_route(int32_t t, int32_t e, const void* logits, bool bf16, int64_t ld, int32_t top, bool sigmoid,
                               bool normalize, float scale, int32_t* ids, float* weights, int32_t* perm, int32_t* offsets,
                               int32_t* place, void* ws, hipStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  const RouteArgs a{logits, ld, t, e, top, normalize, scale, ids, weights, perm, offsets, place, w, hist_pitch(t),
                    reinterpret_cast<int32_t*>(w + (t > kFew ? hist_bytes(t, e) : 0))};
  if (bf16) sigmoid ? launch_route<true, true>(a, stream) : launch_route<true, false>(a, stream);
  else sigmoid ? launch_route<false, true>(a, stream) : launch_route<false, false>(a, stream);
  return hipGetLastError();
}

hipError_t launch_expert_combine(int32_t t, int32_t n, int32_t top, int32_t p, const void* rows, bool bf16, int64_t ldr,
                                 const float* weights, const int32_t* place, const void* residual, bool r_bf16, int64_t ldres,
                                 void* y, int64_t ldy, hipStream_t stream) {
  if (t == 0) return hipSuccess;
  const uint32_t grid = uint32_t(std::min<int64_t>((int64_t(t) * ((n + 7) / 8) + 255) / 256, 1 << 20));
#define MBQ_COMBINE(B, R) combine_kernel<B, R><<<grid, 256, 0, stream>>>(t, n, top, p, rows, ldr, weights, place, residual, ldres, y, ldy)
  if (bf16) r_bf16 ? MBQ_COMBINE(true, true) : MBQ_COMBINE(true, false);
  else r_bf16 ? MBQ_COMBINE(false, true) : MBQ_COMBINE(false, false);
#undef MBQ_COMBINE
  return hipGetLastError();
}

}  // namespace mbq
