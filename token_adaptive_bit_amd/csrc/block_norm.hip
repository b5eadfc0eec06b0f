// The norms after a block and before the next one in one pass:
//   z = post(x),  y = a residual + b gate z,  h = pre(y),
// with h rounded to its type or quantized to e4m3 per 128 inputs.  Bound by memory traffic
// (each of x, residual, y, h once): a row stays in registers between its two norms, so
// nothing is read twice.
#include "fp8.h"

namespace mbq {
namespace {

typedef mbq_block_norm_args Args;

constexpr int kMaxWaves = 16;

// Sum over the threads that share a row (16, 32 or whole waves), the same in all of them;
// `slot` alternates between consecutive sums so that one barrier a sum is enough.
__device__ __forceinline__ float row_sum(float v, float (*red)[kMaxWaves], int slot, int threads) {
  v += across<8>(v);
  v += across<4>(v);
  v += across<2>(v);
  v += across<1>(v);
  if (threads > 16) v += across<16>(v);
  if (threads > 32) v += across<32>(v);
  if (threads <= 64) return v;
  const int wave = threadIdx.x >> 6, waves = threads >> 6;
  if ((threadIdx.x & 63) == 0) red[slot][wave] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < waves; ++i) s += red[slot][i];
  return s;
}

// Eight weights (or biases) of a float32 vector that may be missing.
__device__ __forceinline__ void load_or(const float* p, int64_t i, int64_t k, float missing, float (&v)[8]) {
  if (p) {
    load8<false>(p, i, k, v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = missing;
  }
}

// y = a residual + b gate z for eight elements of one row; r: the residual's.
template <bool XB>
__device__ __forceinline__ void join_residual(const Args& a, int64_t row, int64_t i, const float (&r)[8], float (&v)[8]) {
  if (a.gate_kind == MBQ_GATE_CHANNEL) {
    float g[8];
    load8<false>(a.gate, i, a.k, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= g[e];
  } else if (a.gate_kind == MBQ_GATE_TOKEN) {
    const float g = static_cast<const float*>(a.gate)[row];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= g;
  } else if (a.gate_kind == MBQ_GATE_FULL) {
    float g[8];
    load8<XB>(static_cast<const uint8_t*>(a.gate) + row * a.k * (XB ? 2 : 4), i, a.k, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= g[e];
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = fmaf(a.gate_scale, v[e], a.residual_scale * r[e]);
}

// Writes eight elements of h (those inside the row; with codes the 16 lanes of a block together).
template <int HT>
__device__ __forceinline__ void store_h(const Args& a, int64_t row, int64_t i, const float (&h)[8]) {
  if constexpr (HT == MBQ_E4M3) {
    const uint32_t m = max16(amax8(h));
    store_codes8(static_cast<uint8_t*>(a.h) + row * a.ldh, i, a.k, h, fp8_factor(m));
    if ((threadIdx.x & 15) == 0 && i < a.k) a.scale[(i / kFp8Block) * a.t + row] = fp8_scale(m);
  } else {
    store8<HT == MBQ_BF16>(static_cast<uint8_t*>(a.h) + row * a.ldh * (HT == MBQ_BF16 ? 2 : 4), i, a.k, h);
  }
}

// blockDim.x threads a row, V groups of 8 elements a thread (element 8 (tid + threads j) + e),
// blockDim.y rows a workgroup.
template <int V, bool EARLY, bool XB, bool RB, int HT>
__global__ __launch_bounds__(1024) void norm_kernel(Args a) {
  __shared__ float reds[2][2][kMaxWaves];  // of at most two rows of several waves
  const int tid = threadIdx.x, threads = blockDim.x;
  float (*red)[kMaxWaves] = reds[threads > 64 ? threadIdx.y : 0];
  const int64_t asked = int64_t(blockIdx.x) * blockDim.y + threadIdx.y;
  const bool spare = asked >= a.t;  // the last workgroup's rows past the end take part in its barriers
  const int64_t row = spare ? a.t - 1 : asked;
  const int k = a.k;
  const float inv_k = 1.f / float(a.k);
  const bool layer = a.kind == MBQ_NORM_LAYER;
  // EARLY: everything a row needs is asked for at once, so that the wait for memory is spent
  // once.  With few rows that wait is the time (one row of 5120: 3.6 us from 4.7); with many
  // the registers it takes cost more (13107 x 5120, both norms and a gate: 4.1 TB/s from 4.6).
  // That holds where the row fills the threads' slots: a wave with a lane past the row's end
  // takes the way of single elements for it, which begins with a wait for its earlier loads.
  Raw8<XB> rx[V];
  Raw8<RB> rr[V];
  Raw8<false> post_w[V], pre_w[V];
#pragma unroll
  for (int j = 0; j < V; ++j)
    rx[j].load(static_cast<const uint8_t*>(a.x) + row * a.ldx * (XB ? 2 : 4), 8 * (tid + threads * j), k);
  if (EARLY) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = 8 * (tid + threads * j);
      if (a.post_weight) post_w[j].load(a.post_weight, i, k);
      if (a.residual) rr[j].load(static_cast<const uint8_t*>(a.residual) + row * a.ldr * (RB ? 2 : 4), i, k);
      if (a.pre_weight) pre_w[j].load(a.pre_weight, i, k);
    }
  }
  float v[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j) rx[j].get(v[j]);

  // Elements past the row are 0 before and after (their weights and biases read as 0).
  auto norm = [&](const float* weight, const Raw8<false> (&early)[V], const float* bias) {
    if (layer) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) s += v[j][e];
      const float mean = row_sum(s, red, 0, threads) * inv_k;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int i = 8 * (tid + threads * j);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] -= mean;
        if (i + 8 > k) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[j][e] = i + e < k ? v[j][e] : 0.f;
        }
      }
    }
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(v[j][e], v[j][e], s);
    const float rstd = 1.f / sqrtf(row_sum(s, red, 1, threads) * inv_k + a.eps);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int i = 8 * (tid + threads * j);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] *= rstd;
      if (weight) {
        float w[8];
        if constexpr (EARLY) early[j].get(w);
        else load8<false>(weight, i, k, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] *= w[e];
      }
      if (bias) {
        float b[8];
        load8<false>(bias, i, k, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] += b[e];
      }
    }
  };

  if (a.post) norm(a.post_weight, post_w, a.post_bias);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int i = 8 * (tid + threads * j);
    if (i < k) {
      float r[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (EARLY && a.residual) rr[j].get(r);
      else if (a.residual) load8<RB>(static_cast<const uint8_t*>(a.residual) + row * a.ldr * (RB ? 2 : 4), i, k, r);
      join_residual<XB>(a, row, i, r, v[j]);
      if (a.y && !spare) store8<RB>(static_cast<uint8_t*>(a.y) + row * a.ldy * (RB ? 2 : 4), i, k, v[j]);
    }
  }
  if (threads > 64 && a.post) __syncthreads();  // the first norm's sums are read before the second's are written
  norm(a.pre_weight, pre_w, a.pre_bias);
  if (spare) return;
#pragma unroll
  for (int j = 0; j < V; ++j) store_h<HT>(a, row, 8 * (tid + threads * j), v[j]);
}

// Rows too long for registers: 1024 threads walk the row once for each statistic and once
// to write, recomputing z and y from the inputs (y may be residual itself: it is written in
// the last walk only, by the thread that read it).
template <bool XB, bool RB, int HT>
__global__ __launch_bounds__(1024) void norm_long_kernel(Args a) {
  __shared__ float red[2][kMaxWaves];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x, k = a.k, step = 8 * 1024;
  const int64_t kr = (k + step - 1) / step * step;  // whole walks: every lane takes part in the sums
  const bool layer = a.kind == MBQ_NORM_LAYER;
  const float inv_k = 1.f / float(a.k);
  int slot = 0;

  float mean_x = 0.f, rstd_x = 1.f;
  auto get_x = [&](int64_t i, float (&v)[8]) {
    load8<XB>(static_cast<const uint8_t*>(a.x) + row * a.ldx * (XB ? 2 : 4), i, k, v);
  };
  auto get_y = [&](int64_t i, float (&v)[8]) {
    get_x(i, v);
    if (a.post) {
      float w[8], b[8];
      load_or(a.post_weight, i, k, 1.f, w);
      load_or(a.post_bias, i, k, 0.f, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = fmaf((v[e] - mean_x) * rstd_x, w[e], b[e]);
    }
    float r[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (a.residual) load8<RB>(static_cast<const uint8_t*>(a.residual) + row * a.ldr * (RB ? 2 : 4), i, k, r);
    join_residual<XB>(a, row, i, r, v);
  };
  // A lane's sum over the row of `term` of its elements, in three levels (a vector, kRun
  // vectors, the row).  In one chain of the lane's elements a sum of equal terms drifts by up
  // to 2^-14 of itself in rows of 2^22 and 2^-12 in rows of 2^24; 512 x 65536 bfloat16, both
  // norms, 91.4 us so and 91.0 in one chain.
  auto lane_sum = [&](auto get, auto term) {
    constexpr int kRun = 32;
    float s = 0.f, v[8];
    for (int64_t i0 = 8 * tid; i0 < k; i0 += kRun * step) {
      const int64_t end = min(i0 + kRun * step, k);
      float run = 0.f;
      for (int64_t i = i0; i < end; i += step) {
        get(i, v);
        float p = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) p = i + e < k ? term(v[e], p) : p;
        run += p;
      }
      s += run;
    }
    return s;
  };
  auto stats = [&](auto get, float& mean, float& rstd) {
    mean = 0.f;
    if (layer) {
      mean = row_sum(lane_sum(get, [](float v, float p) { return p + v; }), red, slot, 1024) * inv_k;
      slot ^= 1;
    }
    const float m = mean;
    const float s = lane_sum(get, [m](float v, float p) { return fmaf(v - m, v - m, p); });
    rstd = 1.f / sqrtf(row_sum(s, red, slot, 1024) * inv_k + a.eps);
    slot ^= 1;
    __syncthreads();
  };
  if (a.post) stats(get_x, mean_x, rstd_x);
  float mean, rstd;
  stats(get_y, mean, rstd);
  for (int64_t i = 8 * tid; i < kr; i += step) {
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (i < k) {
      get_y(i, v);
      if (a.y) store8<RB>(static_cast<uint8_t*>(a.y) + row * a.ldy * (RB ? 2 : 4), i, k, v);
      float w[8], b[8];
      load_or(a.pre_weight, i, k, 1.f, w);
      load_or(a.pre_bias, i, k, 0.f, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = i + e < k ? fmaf((v[e] - mean) * rstd, w[e], b[e]) : 0.f;
    }
    store_h<HT>(a, row, i, v);
  }
}

// Threads for a row are bought in waves of 512 elements: as many waves as fit the row with
// two groups of 8 elements a thread (enough loads in flight; a thread's slots past the row
// cost its issue time), three where that takes fewer waves for the same slots (3 and 5
// times 512), more only where 16 waves are not enough; 16 or 32 lanes for rows of up to 128
// or 256.  GB/s at 2^26 elements, bfloat16, both norms and a gate, with 1 / 2 / 3 / 4 groups:
// 1024 5299 / 5559 / 5381 / 4743; 1531 3029 / 3344 / 4025 / 3753; 5120 3574 / 4630 / 4737 /
// 4583; 8192 4534 / 4952 / 4273 / 4516; 16384 two: 4670, three: 4245.
template <bool XB, bool RB, int HT>
hipError_t launch(const Args& a, hipStream_t s) {
  const int units = (a.k + 511) / 512;
  if (units > 4 * kMaxWaves) {
    norm_long_kernel<XB, RB, HT><<<uint32_t(a.t), 1024, 0, s>>>(a);
    return hipGetLastError();
  }
  const bool early = a.t <= 4096 / units;  // at most four waves a SIMD in all
  int v = units == 1 ? 1 : !early && (units == 3 || units == 5) ? 3 : 2;
  while ((units + v - 1) / v > kMaxWaves) ++v;
  const int threads = a.k <= 128 ? 16 : a.k <= 256 ? 32 : 64 * ((units + v - 1) / v);
  const int rows = threads <= 64 ? 256 / threads : threads == 128 ? 2 : 1;
  const dim3 grid((uint32_t(a.t) + rows - 1) / rows), block(threads, rows);
  switch (v) {
    case 1:
      if (early) norm_kernel<1, true, XB, RB, HT><<<grid, block, 0, s>>>(a);
      else norm_kernel<1, false, XB, RB, HT><<<grid, block, 0, s>>>(a);
      break;
    case 2:
      if (early) norm_kernel<2, true, XB, RB, HT><<<grid, block, 0, s>>>(a);
      else norm_kernel<2, false, XB, RB, HT><<<grid, block, 0, s>>>(a);
      break;
    case 3: norm_kernel<3, false, XB, RB, HT><<<grid, block, 0, s>>>(a); break;
    default: norm_kernel<4, false, XB, RB, HT><<<grid, block, 0, s>>>(a); break;
  }
  return hipGetLastError();
}

template <bool XB, bool RB>
hipError_t launch_h(const Args& a, hipStream_t s) {
  if (a.h_dtype == MBQ_F32) return launch<XB, RB, MBQ_F32>(a, s);
  if (a.h_dtype == MBQ_BF16) return launch<XB, RB, MBQ_BF16>(a, s);
  return launch<XB, RB, MBQ_E4M3>(a, s);
}

}  // namespace

hipError_t launch_block_norm(const mbq_block_norm_args& a, hipStream_t s) {
  const bool xb = a.x_dtype == MBQ_BF16, rb = a.r_dtype == MBQ_BF16;
  if (xb) return rb ? launch_h<true, true>(a, s) : launch_h<true, false>(a, s);
  return rb ? launch_h<false, true>(a, s) : launch_h<false, false>(a, s);
}

}  // namespace mbq
