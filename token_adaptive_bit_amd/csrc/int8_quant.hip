// 8-bit integer operands: activations per token, weights per output, laid out in the order
// the matrix instruction takes them.
#include "int8.h"

namespace mbq {
namespace {

// One token by WR waves, its elements held in registers between the maximum and the codes
// (longer rows are read again).  Bound by traffic: x once, one byte a code (4096 rows of 18944
// bfloat16 37 us, 6.3 TB/s).
template <bool BF16, bool PAD, int WR>
__global__ __launch_bounds__(WR < 4 ? 256 : 64 * WR) void quantize_rows_kernel(int32_t t, int32_t k, const void* __restrict__ x,
                                                                               int64_t ldx, uint8_t* __restrict__ q, int64_t ldq,
                                                                               float* __restrict__ scale) {
  constexpr int kWaves = WR < 4 ? 4 : WR, kHeld = 4;
  __shared__ uint32_t part[kWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = int64_t(blockIdx.x) * (kWaves / WR) + wave / WR;
  const bool there = row < t;
  const int at = ((wave % WR) * 64 + lane) * 8;
  constexpr int kStep = WR * 512;
  const uint8_t* src = static_cast<const uint8_t*>(x) + (there ? row : 0) * ldx * (BF16 ? 2 : 4);
  const int end = there ? k : 0;
  Raw8<BF16> held[kHeld];
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    if (at + j * kStep < end) {
      held[j].load(src, at + j * kStep, end);
    } else {
#pragma unroll
      for (int h = 0; h < (BF16 ? 1 : 2); ++h) held[j].w[h] = u32x4_t{0, 0, 0, 0};
    }
  }
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    float v[8];
    held[j].get(v);
    m = max(m, amax8(v));
  }
  for (int i = at + kHeld * kStep; i < end; i += kStep) {
    float v[8];
    load8<BF16>(src, i, end, v);
    m = max(m, amax8(v));
  }
  m = max64(m);
  if constexpr (WR > 1) {
    if (lane == 0) part[wave] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WR; ++w) m = max(m, part[wave / WR * WR + w]);
  }
  if (!there) return;
  const float f = int8_factor(m);
  uint8_t* out = q + row * ldq;
  const int limit = PAD ? (k + kFp8Block - 1) / kFp8Block * kFp8Block : k;  // with PAD the inputs past k get code 0
#pragma unroll
  for (int j = 0; j < kHeld; ++j) {
    float v[8];
    held[j].get(v);
    if (at + j * kStep < limit) store_int8x8(out, at + j * kStep, limit, v, f);
  }
  for (int i = at + kHeld * kStep; i < limit; i += kStep) {
    float v[8];
    load8<BF16>(src, i, k, v);
    store_int8x8(out, i, limit, v, f);
  }
  if (at == 0) scale[row] = int8_scale(m);
}

// 16 rows of one weight of one expert per workgroup and step: 16 lanes a row, 128 inputs at a
// time, first for the row's maximum and then for its codes.  Bound by traffic: codes, which have no
// maximum, once (128 experts of 1536 x 4096 330 us, 4.9 TB/s); float weights twice, the second time
// from memory too (the same from float32 1414 us, 5.1 TB/s with both reads, from bfloat16 767 us, 5.3).
template <int WT>  // 0 float32, 1 bfloat16, 2 codes with scales given
__global__ __launch_bounds__(256) void pack_int8_kernel(mbq_int8_desc d, int32_t part, const void* __restrict__ w,
                                                        const float* __restrict__ w_scale, uint8_t* __restrict__ packed,
                                                        int32_t* __restrict__ status) {
  const int blocks = (d.n + kRowBlock - 1) / kRowBlock;
  const int r = threadIdx.x >> 4, l = threadIdx.x & 15;
  for (int64_t b = blockIdx.x; b < int64_t(d.experts) * blocks; b += gridDim.x) {
    const int64_t expert = b / blocks;
    const int block = int(b - expert * blocks);
    const int64_t row = int64_t(block) * kRowBlock + r;
    const bool there = row < d.n;
    const int end = there ? d.k : 0;
    const uint8_t* src = static_cast<const uint8_t*>(w) + (expert * d.n + (there ? row : 0)) * d.k * (WT == 0 ? 4 : WT == 1 ? 2 : 1);
    float f = 0.f, s = 0.f;
    bool bad = false;
    if constexpr (WT == 2) {
      if (there) s = w_scale[expert * d.n + row];
      bad = (__float_as_uint(s) & 0x7F800000u) == 0x7F800000u;
    } else {
      uint32_t m = 0;
      for (int i = l * 8; i < end; i += 128) {
        float v[8];
        load8<WT == 1>(src, i, end, v);
        m = max(m, amax8(v));
      }
      m = max16(m);
      f = int8_factor(m);
      if (there) s = int8_scale(m);
      bad = m >= 0x7F800000u;
    }
    const int64_t rb = int64_t(block) * (d.gated + 1) + part;
    uint8_t* tiles = packed + expert * d.expert_stride + rb * d.k_blocks * kFp8TileBytes;
    for (int kb = 0; kb < d.k_blocks; ++kb) {
      const int i = kb * kFp8Block + l * 8;  // inputs i .. i + 7: half l / 8, lane group l / 2 % 4, its first or last 8 bytes
      uint8_t* out = tiles + int64_t(kb) * kFp8TileBytes + 1024 * (l >> 3) + 256 * (l >> 1 & 3) + 16 * r + 8 * (l & 1);
      if constexpr (WT == 2) {
        u32x2_a1 c = {0, 0};
        if (i + 8 <= end) {
          c = *reinterpret_cast<const u32x2_a1*>(src + i);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (i + e < end) c[e / 4] |= uint32_t(src[i + e]) << (8 * (e & 3));
        }
        *reinterpret_cast<u32x2_a1*>(out) = c;
      } else {
        float v[8];
        load8<WT == 1>(src, i, end, v);
        store_int8x8(out, 0, 8, v, f);
      }
    }
    if (l == 0) reinterpret_cast<float*>(packed + d.scales_offset)[(expert * d.row_blocks + rb) * kRowBlock + r] = s;
    if (bad && status) atomicOr(status, 1);
  }
}

}  // namespace

hipError_t launch_int8_quantize(int32_t t, int32_t k, const void* x, bool x_bf16, int64_t ldx, void* q, int64_t ldq,
                                bool pad, float* scale, hipStream_t stream) {
  if (t == 0) return hipSuccess;
  uint8_t* out = static_cast<uint8_t*>(q);
  // waves a row: as many as hold the row in registers; sixteen for a few rows, which leave
  // the units empty otherwise
  const int waves = k > 8192 || (t < 64 && k > 4096) ? 16 : k > 2048 ? 4 : 1;
  const uint32_t grid = uint32_t(waves == 1 ? (t + 3) / 4 : t);
#define MBQ_QUANTIZE(B, P, W) quantize_rows_kernel<B, P, W><<<grid, W < 4 ? 256 : 64 * W, 0, stream>>>(t, k, x, ldx, out, ldq, scale)
#define MBQ_QUANTIZE_W(B, P) (waves == 16 ? MBQ_QUANTIZE(B, P, 16) : waves == 4 ? MBQ_QUANTIZE(B, P, 4) : MBQ_QUANTIZE(B, P, 1))
  if (x_bf16) pad ? MBQ_QUANTIZE_W(true, true) : MBQ_QUANTIZE_W(true, false);
  else pad ? MBQ_QUANTIZE_W(false, true) : MBQ_QUANTIZE_W(false, false);
#undef MBQ_QUANTIZE_W
#undef MBQ_QUANTIZE
  return hipGetLastError();
}

hipError_t launch_int8_pack(const mbq_int8_desc& d, int32_t part, const void* w, mbq_dtype w_dtype, const float* w_scale,
                            void* packed, int32_t* dev_status, hipStream_t stream) {
  // a launch holds fewer than 2^32 threads (more are cut without an error); there may be 2^25 groups of rows
  const dim3 grid(std::min(uint32_t(d.experts) * uint32_t((d.n + kRowBlock - 1) / kRowBlock), 1u << 22));
  uint8_t* out = static_cast<uint8_t*>(packed);
  if (w_dtype == MBQ_F32) pack_int8_kernel<0><<<grid, 256, 0, stream>>>(d, part, w, w_scale, out, dev_status);
  else if (w_dtype == MBQ_BF16) pack_int8_kernel<1><<<grid, 256, 0, stream>>>(d, part, w, w_scale, out, dev_status);
  else pack_int8_kernel<2><<<grid, 256, 0, stream>>>(d, part, w, w_scale, out, dev_status);
  return hipGetLastError();
}

}  // namespace mbq
