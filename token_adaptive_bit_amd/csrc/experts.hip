// A block of experts around its products: each token's top experts with their weights, the
// token copies grouped by expert, and the experts' outputs added up again per token.
#include "int8.h"

namespace mbq {
namespace {

constexpr int kGroup = 16;     // tokens of a histogram: one count fits a byte, one token a wave
constexpr int kSpan = 4096;    // tokens whose histograms one place workgroup adds up by itself
constexpr int kPlaced = 64;    // tokens of a place workgroup: one bit each in a 64-bit mask
constexpr int kMaxExperts = 1024;

struct RouteArgs {
  const void* logits;
  int64_t ld;
  int32_t t, e, top, normalize;
  float scale;
  int32_t* ids;
  float* weights;
  int32_t *perm, *offsets, *place;
  uint8_t* hist;  // [ceil(t / 16)][e rounded up to 4]: tokens of the group that took the expert
  int32_t* span;  // beyond one span: [spans + 1][e], tokens before the span that took the expert; last: all
};

__device__ __host__ inline int pad4(int e) { return (e + 3) & ~3; }

// Bits that order as the values do (-0 as +0).
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b ^ (uint32_t(int32_t(b) >> 31) | 0x80000000u);
}
constexpr uint32_t kKeyNegInf = 0x007FFFFFu;  // order_key(-infinity)
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k); }

__device__ __forceinline__ float sum64(float v) {
  v += across<1>(v);
  v += across<2>(v);
  v += across<4>(v);
  v += across<8>(v);
  v += across<16>(v);
  return v + across<32>(v);
}

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

// The choices of 16 tokens, a wave each, and their histogram.
template <bool BF16, int V, bool SIGMOID>
__global__ __launch_bounds__(1024) void choose_kernel(RouteArgs a) {
  __shared__ uint32_t count[V * 16];  // four experts a word
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, words = pad4(a.e) / 4;
  for (int i = threadIdx.x; i < words; i += 1024) count[i] = 0;
  __syncthreads();
  const int64_t token = int64_t(blockIdx.x) * kGroup + wave;
  if (token < a.t) {
    float weight;
    const int id = choose<BF16, V, SIGMOID>(a, token, weight);
    if (lane < a.top) {
      a.ids[token * a.top + lane] = id;
      a.weights[token * a.top + lane] = weight;
      if (id >= 0) atomicAdd(&count[id >> 2], 1u << (8 * (id & 3)));  // a sum: its order is free
    }
  }
  __syncthreads();
  uint32_t* out = reinterpret_cast<uint32_t*>(a.hist + int64_t(blockIdx.x) * pad4(a.e));
  for (int i = threadIdx.x; i < words; i += 1024) out[i] = count[i];
}

// Histograms of groups g0 .. g1 - 1 added per expert, into sums[e]; 1024 threads, a quarter of
// the experts' words each for a share of the groups.
__device__ __forceinline__ void add_groups(const RouteArgs& a, int64_t g0, int64_t g1, int32_t* sums) {
  const int words = pad4(a.e) / 4, lanes = 1024 / words, share = threadIdx.x / words, word = threadIdx.x - share * words;
  if (share >= lanes) return;
  int32_t s[4] = {0, 0, 0, 0};
#pragma unroll 4
  for (int64_t g = g0 + share; g < g1; g += lanes) {
    const uint32_t v = reinterpret_cast<const uint32_t*>(a.hist + g * pad4(a.e))[word];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] += int32_t(v >> (8 * i) & 255u);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (s[i]) atomicAdd(&sums[word * 4 + i], s[i]);
}

// Exclusive sums of total[0 .. e - 1] to first[0 .. e] (1024 threads, e <= 1024).
__device__ __forceinline__ void scan_experts(int e, const int32_t* total, int32_t* first) {
  __shared__ int32_t part[16];
  const int tid = threadIdx.x, v = tid < e ? total[tid] : 0, upto = scan64(v);
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
  __shared__ int32_t sums[kMaxExperts];
  sums[threadIdx.x] = 0;
  __syncthreads();
  const int64_t groups = (int64_t(a.t) + kGroup - 1) / kGroup, g0 = int64_t(blockIdx.x) * (kSpan / kGroup);
  add_groups(a, g0, min(g0 + kSpan / kGroup, groups), sums);
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

// The places of 64 tokens' copies: tokens before them that took the expert, from the
// histograms, and among the 64 a mask of bits an expert, whose bits below a token's are the
// tokens before it.  masks and base in LDS, ready to be added to.
__device__ __forceinline__ void place_tokens(const RouteArgs& a, int64_t t0, const int32_t* first, const int32_t* base,
                                             const uint64_t* mask) {
  const int pairs = int(min(int64_t(kPlaced), a.t - t0)) * a.top;
  for (int i = threadIdx.x; i < pairs; i += 1024) {
    const int token = i / a.top;
    const int id = a.ids[t0 * a.top + i];
    int at = -1;
    if (id >= 0) {
      at = first[id] + base[id] + __popcll(mask[id] & ((uint64_t(1) << token) - 1));
      a.perm[at] = int32_t(t0 + token);
    }
    a.place[t0 * a.top + i] = at;
  }
}
__device__ __forceinline__ void mark_tokens(const RouteArgs& a, int64_t t0, uint64_t* mask) {
  const int pairs = int(min(int64_t(kPlaced), a.t - t0)) * a.top;
  for (int i = threadIdx.x; i < pairs; i += 1024) {
    const int id = a.ids[t0 * a.top + i];
    if (id >= 0) atomicOr(reinterpret_cast<unsigned long long*>(&mask[id]), 1ull << (i / a.top));
  }
}

__global__ __launch_bounds__(1024) void place_kernel(RouteArgs a) {
  __shared__ int32_t base[kMaxExperts], total[kMaxExperts], first[kMaxExperts + 1];
  __shared__ uint64_t mask[kMaxExperts];
  const int tid = threadIdx.x;
  const int64_t t0 = int64_t(blockIdx.x) * kPlaced, groups = (int64_t(a.t) + kGroup - 1) / kGroup, g = t0 / kGroup;
  const int64_t s = t0 / kSpan, spans = (int64_t(a.t) + kSpan - 1) / kSpan;
  const bool many = spans > 1;
  if (tid < pad4(a.e)) {
    base[tid] = many && tid < a.e ? a.span[s * a.e + tid] : 0;
    total[tid] = many && tid < a.e ? a.span[spans * a.e + tid] : 0;
    mask[tid] = 0;
  }
  __syncthreads();
  add_groups(a, s * (kSpan / kGroup), g, base);
  if (!many) add_groups(a, g, groups, total);
  mark_tokens(a, t0, mask);
  __syncthreads();
  if (!many && tid < a.e) total[tid] += base[tid];
  __syncthreads();
  scan_experts(a.e, total, first);
  place_tokens(a, t0, first, base, mask);
  if (blockIdx.x == 0)
    for (int i = tid; i <= a.e; i += 1024) a.offsets[i] = first[i];
  const int64_t all = int64_t(a.t) * a.top;  // rows of no copy
  for (int64_t i = first[a.e] + int64_t(blockIdx.x) * 1024 + tid; i < all; i += int64_t(gridDim.x) * 1024) a.perm[i] = -1;
}

// At most 64 tokens: everything in one workgroup.
template <bool BF16, int V, bool SIGMOID>
__global__ __launch_bounds__(1024) void route_few_kernel(RouteArgs a) {
  __shared__ int32_t base[kMaxExperts], total[kMaxExperts], first[kMaxExperts + 1];
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
  if (tid < a.e) total[tid] = __popcll(mask[tid]);
  __syncthreads();
  scan_experts(a.e, total, first);
  place_tokens(a, 0, first, base, mask);
  for (int i = tid; i <= a.e; i += 1024) a.offsets[i] = first[i];
  for (int i = first[a.e] + tid; i < a.t * a.top; i += 1024) a.perm[i] = -1;
}

// y[t] = residual[t] + sum_j weights[t][j] rows[place[t][j]], eight outputs a thread, the
// copies' rows asked for U at a time.  Bound by traffic.  A place outside the rows adds its
// weight times 0: nothing, or NaN where the weight is one.
template <bool BF16, bool RBF>
__global__ __launch_bounds__(256) void combine_kernel(int32_t t, int32_t n, int32_t top, int32_t p, const void* __restrict__ rows,
                                                      int64_t ldr, const float* __restrict__ weights,
                                                      const int32_t* __restrict__ place, const void* residual,
                                                      int64_t ldres, void* y, int64_t ldy) {
  constexpr int U = 4;
  const int pieces = (n + 7) / 8;
  const int64_t all = int64_t(t) * pieces;
  for (int64_t b = int64_t(blockIdx.x) * 256 + threadIdx.x; b < all; b += int64_t(gridDim.x) * 256) {
    const int64_t token = b / pieces;
    const int col = int(b - token * pieces) * 8;
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
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = min(j0 + u, top - 1);
        const int at = place[token * top + j];
        const bool there = uint32_t(at) < uint32_t(p);
        w[u] = j0 + u < top ? weights[token * top + j] : 0.f;
        raw[u].load(static_cast<const uint8_t*>(rows) + (there ? at : 0) * ldr * (BF16 ? 2 : 4), col, there && j0 + u < top ? n : 0);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        raw[u].get(v);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = fmaf(w[u], v[e], sum[e]);
      }
    }
    store8<RBF>(static_cast<uint8_t*>(y) + token * ldy * (RBF ? 2 : 4), col, n, sum);
  }
}

size_t align256(size_t v) { return (v + 255) / 256 * 256; }
size_t hist_bytes(int32_t t, int32_t e) { return align256(size_t((t + kGroup - 1) / kGroup) * pad4(e)); }

template <bool BF16, int V, bool SIGMOID>
void launch_route(const RouteArgs& a, hipStream_t stream) {
  if (a.t <= kPlaced) {
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
  if (t <= kPlaced) return 0;
  const int spans = (t + kSpan - 1) / kSpan;
  return hist_bytes(t, e) + (spans > 1 ? align256(size_t(spans + 1) * e * 4) : 0);
}

hipError_t launch_expert_route(int32_t t, int32_t e, const void* logits, bool bf16, int64_t ld, int32_t top, bool sigmoid,
                               bool normalize, float scale, int32_t* ids, float* weights, int32_t* perm, int32_t* offsets,
                               int32_t* place, void* ws, hipStream_t stream) {
  uint8_t* w = static_cast<uint8_t*>(ws);
  const RouteArgs a{logits, ld, t, e, top, normalize, scale, ids, weights, perm, offsets, place, w,
                    reinterpret_cast<int32_t*>(w + (t > kPlaced ? hist_bytes(t, e) : 0))};
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
