// The norms after a block and before the next one in one pass:
//   z = post(x),  y = a residual + b gate z,  h = pre(y),
// with h rounded to its type or quantized to e4m3 per 128 inputs.  Bound by memory traffic
// (each of x, residual, y, h once): a row stays in registers between its two norms, so
// nothing is read twice.
#include "fp8.h"

namespace mbq {
namespace {

typedef mbq_block_norm_args Args;

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Sum over the W waves that share a row, the same in every lane; `slot` alternates between
// consecutive sums so that one barrier a sum is enough.
template <int W>
__device__ __forceinline__ float row_sum(float v, float (*red)[W], int slot) {
  v = wave_sum(v);
  if constexpr (W == 1) return v;
  if ((threadIdx.x & 63) == 0) red[slot][(threadIdx.x >> 6) % W] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < W; ++i) s += red[slot][i];
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

// y = a residual + b gate z for eight elements of one row.
template <bool XB, bool RB>
__device__ __forceinline__ void join_residual(const Args& a, int64_t row, int64_t i, float (&v)[8]) {
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
  if (a.residual) {
    float r[8];
    load8<RB>(static_cast<const uint8_t*>(a.residual) + row * a.ldr * (RB ? 2 : 4), i, a.k, r);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = fmaf(a.gate_scale, v[e], a.residual_scale * r[e]);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= a.gate_scale;
  }
}

// Writes eight elements of h; m: whether this 16-lane group lies inside the row at all.
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

// W waves a row, V groups of 8 elements a thread (element 8 (tid + 64 W j) + e); RPB rows
// a workgroup.
template <int W, int V, int RPB, bool XB, bool RB, int HT>
__global__ __launch_bounds__(64 * W * RPB) void norm_kernel(Args a) {
  __shared__ float red[RPB][2][W];
  const int tid = threadIdx.x % (64 * W), sub = threadIdx.x / (64 * W);
  const int64_t row = int64_t(blockIdx.x) * RPB + sub;
  if (row >= a.t) return;  // W == 1 wherever RPB > 1: no barrier is left behind
  const int64_t k = a.k;
  const float inv_k = 1.f / float(a.k);
  const bool layer = a.kind == MBQ_NORM_LAYER;
  float v[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j)
    load8<XB>(static_cast<const uint8_t*>(a.x) + row * a.ldx * (XB ? 2 : 4), 8 * (tid + 64 * W * j), k, v[j]);

  auto norm = [&](const float* weight, const float* bias) {
    float mean = 0.f;
    if (layer) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) s += v[j][e];
      mean = row_sum<W>(s, red[sub], 0) * inv_k;
    }
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int64_t i = 8 * (tid + 64 * W * j) + e;
        const float d = layer ? (i < k ? v[j][e] - mean : 0.f) : v[j][e];
        v[j][e] = d;
        s = fmaf(d, d, s);
      }
    const float rstd = 1.f / sqrtf(row_sum<W>(s, red[sub], 1) * inv_k + a.eps);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float w[8], b[8];
      const int64_t i = 8 * (tid + 64 * W * j);
      load_or(weight, i, k, 1.f, w);
      load_or(bias, i, k, 0.f, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[j][e] = i + e < k ? fmaf(v[j][e] * rstd, w[e], b[e]) : 0.f;
    }
  };

  if (a.post) norm(a.post_weight, a.post_bias);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int64_t i = 8 * (tid + 64 * W * j);
    if (i < k) {
      join_residual<XB, RB>(a, row, i, v[j]);
      if (a.y) store8<RB>(static_cast<uint8_t*>(a.y) + row * a.ldy * (RB ? 2 : 4), i, k, v[j]);
    }
  }
  if (W > 1 && a.post) __syncthreads();  // the first norm's sums are read before the second's are written
  norm(a.pre_weight, a.pre_bias);
#pragma unroll
  for (int j = 0; j < V; ++j) store_h<HT>(a, row, 8 * (tid + 64 * W * j), v[j]);
}

// Rows too long for registers: 1024 threads walk the row once for each statistic and once
// to write, recomputing z and y from the inputs (y may be residual itself: it is written in
// the last walk only, by the thread that read it).
template <bool XB, bool RB, int HT>
__global__ __launch_bounds__(1024) void norm_long_kernel(Args a) {
  constexpr int W = 16;
  __shared__ float red[2][W];
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
    join_residual<XB, RB>(a, row, i, v);
  };
  auto stats = [&](auto get, float& mean, float& rstd) {
    mean = 0.f;
    float v[8];
    if (layer) {
      float s = 0.f;
      for (int64_t i = 8 * tid; i < k; i += step) {
        get(i, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s += i + e < k ? v[e] : 0.f;
      }
      mean = row_sum<W>(s, red, slot) * inv_k;
      slot ^= 1;
    }
    float s = 0.f;
    for (int64_t i = 8 * tid; i < k; i += step) {
      get(i, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = i + e < k ? v[e] - mean : 0.f;
        s = fmaf(d, d, s);
      }
    }
    rstd = 1.f / sqrtf(row_sum<W>(s, red, slot) * inv_k + a.eps);
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

template <bool XB, bool RB, int HT>
hipError_t launch(const Args& a, hipStream_t s) {
  const uint32_t t = uint32_t(a.t);
  if (a.k <= 512) norm_kernel<1, 1, 4, XB, RB, HT><<<(t + 3) / 4, 256, 0, s>>>(a);
  else if (a.k <= 2048) norm_kernel<4, 1, 1, XB, RB, HT><<<t, 256, 0, s>>>(a);
  else if (a.k <= 4096) norm_kernel<4, 2, 1, XB, RB, HT><<<t, 256, 0, s>>>(a);
  else if (a.k <= 8192) norm_kernel<8, 2, 1, XB, RB, HT><<<t, 512, 0, s>>>(a);
  else if (a.k <= 16384) norm_kernel<16, 2, 1, XB, RB, HT><<<t, 1024, 0, s>>>(a);
  else norm_long_kernel<XB, RB, HT><<<t, 1024, 0, s>>>(a);
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
