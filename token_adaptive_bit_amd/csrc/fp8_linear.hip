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
typedef __attribute__((address_space(4))) float ConstFloat;  // read by scalar loads

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

// 16 (or 4) bytes a lane from memory to LDS, the lanes side by side at l.  Written in
// assembly because the compiler waits for every copy in flight before any LDS read that
// follows one of its own (it cannot tell the buffers apart).  The instruction has no
// register outputs; to_lds_wait() before the barrier completes it.
template <int BYTES>
__device__ __forceinline__ void to_lds(const void* base, uint32_t offset, const uint8_t* l) {  // base, l: the wave's
  const uint32_t at = uint32_t(uintptr_t((const __attribute__((address_space(3))) uint8_t*)l));
  if constexpr (BYTES == 16)
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 ::"s"(at), "v"(offset), "s"(base) : "memory", "m0");
  else
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
                 ::"s"(at), "v"(offset), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void to_lds_from(const uint8_t* g, const uint8_t* l) {  // 16 bytes at each lane's own g
  const uint32_t at = uint32_t(uintptr_t((const __attribute__((address_space(3))) uint8_t*)l));
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(at), "v"(g) : "memory", "m0");
}
__device__ __forceinline__ void to_lds_wait() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// Tiles of 16 RN WN packed rows x 16 RT WT tokens on WN WT = 8 waves; both operands and the
// tokens' scales of a block go through LDS in two buffers, one block ahead.
template <int RN, int RT, int WN, int WT, int ACT, bool YBF>
__global__ __launch_bounds__(64 * WN * WT, 2) void gemm_kernel(LinArgs a) {
  constexpr int kWaves = WN * WT, kRb = RN * WN, kTb = RT * WT, kTok = 16 * kTb;
  constexpr int kStage = (kRb + kTb) * kFp8TileBytes + kTok * 4;
  constexpr int kCopiesW = 2 * kRb / kWaves, kCopiesX = 2 * kTb / kWaves;  // a wave's copies to LDS a block
  static_assert(2 * kRb % kWaves == 0 && 2 * kTb % kWaves == 0 && kTok % 64 == 0, "whole copies");
  __shared__ __align__(1024) uint8_t lds[2][kStage];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, c = lane >> 4;
  const int wn = wave % WN, wt = wave / WN;
  // neighbouring tiles (four token tiles by as many row tiles as it takes) on one XCD
  const int tiles_t = (a.t + kTok - 1) / kTok, tiles_n = (a.rbs + kRb - 1) / kRb;
  const int per = gridDim.x / 8, rest = gridDim.x % 8, xcd = blockIdx.x % 8;
  const int id = blockIdx.x / 8 + xcd * per + min(xcd, rest);
  const int group = id / (4 * tiles_n), gt = min(4, tiles_t - 4 * group), in = id - group * 4 * tiles_n;
  const int rb0 = in / gt * kRb, tok0 = (4 * group + in % gt) * kTok;

  // a wave's rows lie in one 128-row block of each weight
  const int rbw = min(rb0 + wn * RN, a.rbs - 1);
  const ConstFloat* wsp = (const ConstFloat*)a.ws + int64_t(ACT == kPlain ? rbw / 8 : rbw / 16) * a.kb;
  const ConstFloat* wsu = wsp + int64_t(a.nblk) * a.kb;

  const uint8_t* wp[kCopiesW];
#pragma unroll
  for (int i = 0; i < kCopiesW; ++i) {
    const int half = i * kWaves + wave;
    wp[i] = a.codes + int64_t(min(rb0 + (half >> 1), a.rbs - 1)) * a.kb * kFp8TileBytes + (half & 1) * 1024;
  }
  const uint8_t* xb = a.xq + tok0 * a.ldq;
  uint32_t xo[kCopiesX];  // this lane's 16 bytes from there: 256 rows of at most 2^24 bytes
#pragma unroll
  for (int i = 0; i < kCopiesX; ++i) {
    const int half = i * kWaves + wave;
    xo[i] = uint32_t(min((half >> 1) * 16 + r, a.t - 1 - tok0)) * uint32_t(a.ldq) + 64 * (half & 1) + 16 * c;
  }
  const int xchunk = wave % (kTok / 64);
  const uint32_t so = uint32_t(min(tok0 + xchunk * 64 + lane, a.t - 1));

  auto copy = [&](int kb, int buf) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kCopiesW; ++i)
      to_lds<16>(wp[i] + int64_t(kb) * kFp8TileBytes, uint32_t(lane) * 16, &lds[buf][(i * kWaves + wave) * 1024]);
    if (kb * kFp8Block + kFp8Block <= a.xlim) {
#pragma unroll
      for (int i = 0; i < kCopiesX; ++i)
        to_lds<16>(xb + int64_t(kb) * kFp8Block, xo[i], &lds[buf][(2 * kRb + i * kWaves + wave) * 1024]);
    } else {  // the end of a row of codes that is no whole block: zeros after it
#pragma unroll
      for (int i = 0; i < kCopiesX; ++i) {
        const int half = i * kWaves + wave;
        const bool in_row = kb * kFp8Block + 64 * (half & 1) + 16 * c < a.xlim;
        to_lds_from(in_row ? xb + int64_t(kb) * kFp8Block + xo[i] : a.zeros, &lds[buf][(2 * kRb + half) * 1024]);
      }
    }
    to_lds<4>(a.xs + int64_t(kb) * a.t, so * 4, &lds[buf][(kRb + kTb) * kFp8TileBytes + xchunk * 256]);
  };

  f32x4_t acc[RN][RT];
#pragma unroll
  for (int i = 0; i < RN; ++i)
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  copy(0, 0);
  for (int kb = 0; kb < a.kb; ++kb) {
    const uint8_t* buf = lds[kb & 1];
    to_lds_wait();
    __syncthreads();  // block kb is in, and every wave has left the other buffer
    if (kb + 1 < a.kb) copy(kb + 1, (kb & 1) ^ 1);
    auto frag = [&](int tile) __attribute__((always_inline)) {
      const u32x4_t* p = reinterpret_cast<const u32x4_t*>(buf + tile * kFp8TileBytes) + lane;
      return join(p[0], p[64]);
    };
    i32x8_t x[RT];
    float xs[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) {
      const int tile = wt * RT + j;
      x[j] = frag(kRb + tile);
      xs[j] = reinterpret_cast<const float*>(buf + (kRb + kTb) * kFp8TileBytes)[tile * 16 + r];
    }
    constexpr int P = ACT == kPlain ? 1 : 2;
#pragma unroll
    for (int part = 0; part < P; ++part) {  // gated: all gate tiles, then all up tiles
      const float w_scale = (part ? wsu : wsp)[kb];
      float s[RT];
#pragma unroll
      for (int j = 0; j < RT; ++j) s[j] = xs[j] * w_scale;
#pragma unroll
      for (int i = part; i < RN; i += P) {
        const Frag<!YBF> w = frag(wn * RN + i);
#pragma unroll
        for (int j = 0; j < RT; ++j) {
          const f32x4_t d = block_product<!YBF>(w, x[j]);
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(d[e], s[j], acc[i][j][e]);
        }
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
