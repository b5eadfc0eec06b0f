// 8-bit linear and the gated half of a feed-forward block:
//   y[t][i] = sum_kb xs[kb][t] ws[i / 128][kb] sum_{k in kb} xq[t][k] wq[i][k],
// one 128-input block per matrix instruction.  The instruction starts every block from
// zero; its result is scaled by xs ws and added to the float32 sums on the vector ALU, in
// the shadow of the next instructions.  Outputs are the instruction's rows and tokens its
// columns: a lane then holds one token, so a block needs one scale per lane and 16 tokens.
#include "fp8.h"

namespace mbq {
namespace {

struct LinArgs {
  const uint8_t* codes;  // packed tiles
  const float* ws;       // weight scales [parts][nblk][kb]
  const uint8_t* xq;     // activation codes, rows of ldq bytes, xlim of them readable
  const uint8_t* zeros;  // 16 or more bytes of 0
  const float* xs;       // activation scales [kb][t]
  void* y;
  int64_t ldq;
  int32_t t, n, kb, rbs, nblk, xlim;
};

constexpr int kPlain = -1;

template <int ACT>
__device__ __forceinline__ float gated(float g, float u) {
  float a = g;
  if constexpr (ACT == MBQ_ACT_GELU_TANH) a = 1.5957691216057308f * g * fmaf(0.044715f * g, g, 1.f);
  return g * __builtin_amdgcn_rcpf(1.f + __expf(-a)) * u;
}

template <bool YBF>
__device__ __forceinline__ void store4(void* y, int64_t row, int32_t n, int32_t col, const float (&v)[4]) {
  if constexpr (YBF) {
    uint16_t* p = reinterpret_cast<uint16_t*>(y) + row * n + col;
    const u32x2_a2 w = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    if (col + 4 <= n) {
      *reinterpret_cast<u32x2_a2*>(p) = w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < n) p[e] = uint16_t(w[e / 2] >> (16 * (e & 1)));
    }
  } else {
    float* p = reinterpret_cast<float*>(y) + row * n + col;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (col + e < n) p[e] = v[e];
  }
}

__device__ __forceinline__ void to_lds(const uint8_t* g, uint8_t* l) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)g,
                                   (__attribute__((address_space(3))) void*)l, 16, 0, 0);
}

// Tiles of 16 RN WN packed rows x 16 RT WT tokens on WN WT waves, both operands through
// two LDS buffers.
template <int RN, int RT, int WN, int WT, int ACT, bool YBF>
__global__ __launch_bounds__(64 * WN * WT) void gemm_kernel(LinArgs a) {
  constexpr int kWaves = WN * WT, kRb = RN * WN, kTb = RT * WT;
  __shared__ __align__(1024) uint8_t lds[2][(kRb + kTb) * kFp8TileBytes];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, c = lane >> 4;
  const int wn = wave % WN, wt = wave / WN;
  const int tiles_t = (a.t + 16 * kTb - 1) / (16 * kTb);
  const int tn = blockIdx.x / tiles_t, tt = blockIdx.x % tiles_t;
  const int rb0 = tn * kRb, tok0 = tt * kTb * 16;

  auto issue = [&](int kb, int buf) {
#pragma unroll
    for (int i = 0; i < (kRb + kTb + kWaves - 1) / kWaves; ++i) {
      const int tile = i * kWaves + wave;
      if (tile < kRb) {
        const int rb = min(rb0 + tile, a.rbs - 1);
        const uint8_t* g = a.codes + (int64_t(rb) * a.kb + kb) * kFp8TileBytes + lane * 16;
        to_lds(g, &lds[buf][tile * kFp8TileBytes]);
        to_lds(g + 1024, &lds[buf][tile * kFp8TileBytes + 1024]);
      } else if (tile < kRb + kTb) {
        const int tok = min(tok0 + (tile - kRb) * 16 + r, a.t - 1);
        const int col = kb * kFp8Block + 16 * c;
        const uint8_t* g = a.xq + tok * a.ldq + col;
        to_lds(col < a.xlim ? g : a.zeros, &lds[buf][tile * kFp8TileBytes]);
        to_lds(col + 64 < a.xlim ? g + 64 : a.zeros, &lds[buf][tile * kFp8TileBytes + 1024]);
      }
    }
  };

  f32x4_t acc[RN][RT];
#pragma unroll
  for (int i = 0; i < RN; ++i)
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  // a wave's rows lie in one 128-row block of each weight
  const int rbw = min(rb0 + wn * RN, a.rbs - 1);
  const float* wsp = a.ws + int64_t(ACT == kPlain ? rbw / 8 : rbw / 16) * a.kb;
  const float* wsu = wsp + int64_t(a.nblk) * a.kb;
  int tok[RT];
#pragma unroll
  for (int j = 0; j < RT; ++j) tok[j] = min(tok0 + (wt * RT + j) * 16 + r, a.t - 1);

  issue(0, 0);
  for (int kb = 0; kb < a.kb; ++kb) {
    const int buf = kb & 1;
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    if (kb + 1 < a.kb) issue(kb + 1, buf ^ 1);
    float s[ACT == kPlain ? 1 : 2][RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const float xs = a.xs[int64_t(kb) * a.t + tok[j]];
      s[0][j] = xs * wsp[kb];
      if constexpr (ACT != kPlain) s[1][j] = xs * wsu[kb];
    }
    auto frag = [&](int tile) {
      const uint8_t* p = &lds[buf][tile * kFp8TileBytes + lane * 16];
      return join(*reinterpret_cast<const u32x4_t*>(p), *reinterpret_cast<const u32x4_t*>(p + 1024));
    };
    i32x8_t xf[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) xf[j] = frag(kRb + wt * RT + j);
#pragma unroll
    for (int i = 0; i < RN; ++i) {
      const Frag<!YBF> wf = frag(wn * RN + i);
#pragma unroll
      for (int j = 0; j < RT; ++j) {
        const f32x4_t d = block_product<!YBF>(wf, xf[j]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(d[e], s[ACT == kPlain ? 0 : i & 1][j], acc[i][j][e]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < RT; ++j) {
    const int token = tok0 + (wt * RT + j) * 16 + r;
    if (token >= a.t) continue;
#pragma unroll
    for (int i = 0; i < RN; i += ACT == kPlain ? 1 : 2) {
      const int rb = rb0 + wn * RN + i;
      float v[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (ACT == kPlain) v[e] = acc[i][j][e];
        else v[e] = gated<ACT>(acc[i][j][e], acc[i + 1][j][e]);
      }
      if (rb < a.rbs) store4<YBF>(a.y, token, a.n, (ACT == kPlain ? rb : rb / 2) * 16 + 4 * c, v);
    }
  }
}

// Up to 16 TT tokens: every workgroup streams one row block (gated: the pair), its eight
// waves take every eighth 128-input block, and their sums meet in LDS in a fixed order.
constexpr int kStreamWaves = 8;

template <int TT, int ACT, bool YBF>
__global__ __launch_bounds__(64 * kStreamWaves) void stream_kernel(LinArgs a) {
  constexpr int R = ACT == kPlain ? 1 : 2, U = TT == 1 ? 4 : 2;
  __shared__ f32x4_t red[kStreamWaves][R * TT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, c = lane >> 4;
  const int rb0 = blockIdx.x * R;
  const float* wsp = a.ws + int64_t(rb0 / (8 * R)) * a.kb;
  const float* wsu = wsp + int64_t(a.nblk) * a.kb;
  const uint8_t* wp = a.codes + int64_t(rb0) * a.kb * kFp8TileBytes + lane * 16;
  f32x4_t acc[R][TT];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int k0 = wave; k0 < a.kb; k0 += kStreamWaves * U) {
    u32x4_t wf[U][R][2], xf[U][TT][2];
    float xs[U][TT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = min(k0 + u * kStreamWaves, a.kb - 1);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const uint8_t* p = wp + (int64_t(i) * a.kb + kb) * kFp8TileBytes;
        wf[u][i][0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p));
        wf[u][i][1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p + 1024));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = min(k0 + u * kStreamWaves, a.kb - 1);
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        const int tok = min(j * 16 + r, a.t - 1), col = kb * kFp8Block + 16 * c;
        const uint8_t* p = a.xq + tok * a.ldq + col;
        xf[u][j][0] = *reinterpret_cast<const u32x4_t*>(col < a.xlim ? p : a.zeros);
        xf[u][j][1] = *reinterpret_cast<const u32x4_t*>(col + 64 < a.xlim ? p + 64 : a.zeros);
        xs[u][j] = a.xs[int64_t(kb) * a.t + tok];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = k0 + u * kStreamWaves;
      if (kb >= a.kb) break;
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const float w = i == 0 ? wsp[kb] : wsu[kb];
#pragma unroll
        for (int j = 0; j < TT; ++j) {
          const f32x4_t d = block_product<!YBF>(join(wf[u][i][0], wf[u][i][1]), join(xf[u][j][0], xf[u][j][1]));
          const float s = xs[u][j] * w;
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(d[e], s, acc[i][j][e]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) red[wave][i * TT + j][lane] = acc[i][j];
  __syncthreads();
  if (wave >= TT) return;
  const int j = wave, token = j * 16 + r;
  f32x4_t sum[R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    sum[i] = red[0][i * TT + j][lane];
#pragma unroll
    for (int w = 1; w < kStreamWaves; ++w)
#pragma unroll
      for (int e = 0; e < 4; ++e) sum[i][e] += red[w][i * TT + j][lane][e];
  }
  if (token >= a.t) return;
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (ACT == kPlain) v[e] = sum[0][e];
    else v[e] = gated<ACT>(sum[0][e], sum[R - 1][e]);
  }
  store4<YBF>(a.y, token, a.n, int32_t(blockIdx.x) * 16 + 4 * c, v);
}

template <int ACT, bool YBF>
hipError_t launch(const LinArgs& a, hipStream_t stream) {
  constexpr int R = ACT == kPlain ? 1 : 2;
  if (a.t <= 64) {
    const dim3 grid(a.rbs / R), block(64 * kStreamWaves);
    if (a.t <= 16) stream_kernel<1, ACT, YBF><<<grid, block, 0, stream>>>(a);
    else if (a.t <= 32) stream_kernel<2, ACT, YBF><<<grid, block, 0, stream>>>(a);
    else stream_kernel<4, ACT, YBF><<<grid, block, 0, stream>>>(a);
  } else {
    const dim3 grid(uint32_t((a.rbs + 15) / 16) * uint32_t((a.t + 255) / 256));
    gemm_kernel<8, 4, 2, 4, ACT, YBF><<<grid, 512, 0, stream>>>(a);
  }
  return hipGetLastError();
}

size_t codes_bytes(const mbq_fp8_desc& d, int32_t t) { return size_t(t) * d.k_blocks * kFp8Block; }

}  // namespace

size_t fp8_linear_workspace(const mbq_fp8_desc& d, int32_t t, mbq_dtype x_dtype) {
  if (x_dtype == MBQ_E4M3 || t == 0) return 0;
  return codes_bytes(d, t) + (size_t(d.k_blocks) * t * 4 + 255) / 256 * 256;
}

hipError_t launch_fp8_linear(const mbq_fp8_desc& d, const void* packed, int32_t t, const void* x, mbq_dtype x_dtype,
                             int64_t ldx, const float* x_scale, int act, void* y, bool y_bf16, void* ws,
                             hipStream_t stream) {
  if (t == 0) return hipSuccess;
  const uint8_t* base = static_cast<const uint8_t*>(packed);
  LinArgs a{};
  a.codes = base;
  a.ws = reinterpret_cast<const float*>(base + d.scales_offset);
  a.zeros = base + d.zeros_offset;
  a.y = y;
  a.t = t;
  a.n = d.n;
  a.kb = d.k_blocks;
  a.rbs = d.row_blocks;
  a.nblk = (d.n + 127) / 128;
  if (x_dtype == MBQ_E4M3) {
    a.xq = static_cast<const uint8_t*>(x);
    a.ldq = ldx;
    a.xs = x_scale;
    a.xlim = d.k;
  } else {
    uint8_t* q = static_cast<uint8_t*>(ws);
    float* s = reinterpret_cast<float*>(q + codes_bytes(d, t));
    a.ldq = a.xlim = d.k_blocks * kFp8Block;
    const hipError_t e = launch_fp8_quantize(t, d.k, x, x_dtype == MBQ_BF16, ldx, q, a.ldq, true, s, stream);
    if (e != hipSuccess) return e;
    a.xq = q;
    a.xs = s;
  }
  if (act == kPlain) return y_bf16 ? launch<kPlain, true>(a, stream) : launch<kPlain, false>(a, stream);
  if (act == MBQ_ACT_SILU)
    return y_bf16 ? launch<MBQ_ACT_SILU, true>(a, stream) : launch<MBQ_ACT_SILU, false>(a, stream);
  return y_bf16 ? launch<MBQ_ACT_GELU_TANH, true>(a, stream) : launch<MBQ_ACT_GELU_TANH, false>(a, stream);
}

}  // namespace mbq
