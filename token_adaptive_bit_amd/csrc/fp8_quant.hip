// e4m3 operands of the 8-bit linear: activations per token and 128 inputs, weights per
// 128 x 128 block, laid out in the order the matrix instruction takes them.
#include "fp8.h"

namespace mbq {
namespace {

// One block of 128 inputs of one token per 16 lanes, 8 inputs a lane.  Bound by traffic
// (x once, one byte a code); a wave covers four neighbouring blocks, so its loads and
// stores are whole lines.
template <bool BF16, bool PAD>
__global__ __launch_bounds__(256) void quantize_kernel(int32_t t, int32_t k, int32_t kb, const void* __restrict__ x,
                                                       int64_t ldx, uint8_t* __restrict__ q, int64_t ldq,
                                                       float* __restrict__ scale) {
  const int64_t blocks = int64_t(t) * kb;
  const int lane = threadIdx.x & 15;
  // whole 16-lane groups stay and leave together
  for (int64_t b = int64_t(blockIdx.x) * 16 + threadIdx.x / 16; b < blocks; b += int64_t(gridDim.x) * 16) {
    const int32_t row = int32_t(b / kb), blk = int32_t(b - int64_t(row) * kb);
    const int64_t i = int64_t(blk) * kFp8Block + lane * 8;
    float v[8];
    load8<BF16>(reinterpret_cast<const uint8_t*>(x) + row * ldx * (BF16 ? 2 : 4), i, k, v);
    const uint32_t m = max16(amax8(v));
    // with PAD the row has room for whole blocks, and the inputs past k get code 0
    store_codes8(q + row * ldq, i, PAD ? int64_t(kb) * kFp8Block : k, v, fp8_factor(m));
    if (lane == 0) scale[int64_t(blk) * t + row] = fp8_scale(m);
  }
}

// Codes whose rows hold no whole 16-byte pieces, copied to rows of whole blocks (code 0 past
// k), from which the products copy 16 bytes at a time; 16 codes a thread.
__global__ __launch_bounds__(256) void pad_codes_kernel(int32_t t, int32_t k, int32_t pieces, const uint8_t* __restrict__ x,
                                                        int64_t ldx, uint8_t* __restrict__ q) {
  const int64_t all = int64_t(t) * pieces;
  for (int64_t p = int64_t(blockIdx.x) * 256 + threadIdx.x; p < all; p += int64_t(gridDim.x) * 256) {
    const int64_t row = p / pieces, i = (p - row * pieces) * 16;
    const uint8_t* src = x + row * ldx + i;
    u32x4_t v = {0, 0, 0, 0};
    if (i + 16 <= k) {
      v = *reinterpret_cast<const u32x4_a1*>(src);
    } else {
#pragma unroll
      for (int e = 0; e < 16; ++e)
        if (i + e < k) v[e / 4] |= uint32_t(src[e]) << (8 * (e % 4));
    }
    *reinterpret_cast<u32x4_t*>(q + p * 16) = v;
  }
}

// One 128 x 128 block of one weight per workgroup: thread 2 r + half holds 64 inputs of row
// r, the block's maximum goes through LDS, and every lane of the packed tiles is written
// (rows and inputs of the padding as code 0).
template <int WT>  // 0 float32, 1 bfloat16, 2 e4m3 codes with scales given
__global__ __launch_bounds__(256) void pack_fp8_kernel(mbq_fp8_desc d, int32_t part, const void* __restrict__ w,
                                                       const float* __restrict__ w_scale, uint8_t* __restrict__ packed,
                                                       int32_t* __restrict__ status) {
  __shared__ uint32_t wmax[4];
  const int kb = blockIdx.x % d.k_blocks, nb = blockIdx.x / d.k_blocks, tid = threadIdx.x;
  const int r = tid >> 1, half = tid & 1;
  const int64_t row = int64_t(nb) * 128 + r;
  const int64_t col0 = int64_t(kb) * 128 + 64 * half;
  uint32_t codes[16];
  uint32_t bad = 0;
  float s;
  if constexpr (WT == 2) {
    const uint8_t* p = reinterpret_cast<const uint8_t*>(w) + row * d.k + col0;
    if (row < d.n && col0 + 64 <= d.k) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const u32x4_t v = *reinterpret_cast<const u32x4_a1*>(p + 16 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e) codes[4 * i + e] = v[e];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        codes[i] = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (row < d.n && col0 + 4 * i + e < d.k) codes[i] |= uint32_t(p[4 * i + e]) << (8 * e);
      }
    }
#pragma unroll
    for (int i = 0; i < 16; ++i) {  // a byte of 0x7F or 0xFF: its low seven bits carry into the eighth when 1 is added
      bad |= ((codes[i] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
    }
    s = w_scale[int64_t(nb) * d.k_blocks + kb];
    bad |= (__float_as_uint(s) & 0x7F800000u) == 0x7F800000u;
  } else {
    float v[64];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float u[8];
      const uint8_t* base = reinterpret_cast<const uint8_t*>(w) + (row < d.n ? row : 0) * d.k * (WT == 1 ? 2 : 4);
      load8<WT == 1>(base, col0 + 8 * i, row < d.n ? d.k : 0, u);
      m = max(m, amax8(u));
#pragma unroll
      for (int e = 0; e < 8; ++e) v[8 * i + e] = u[e];
    }
#pragma unroll
    for (int o = 32; o; o >>= 1) m = max(m, uint32_t(__shfl_xor(int(m), o)));
    if ((tid & 63) == 0) wmax[tid >> 6] = m;
    __syncthreads();
    m = max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3]));
    bad = m >= 0x7F800000u;
    const float f = fp8_factor(m);
    s = fp8_scale(m);
#pragma unroll
    for (int i = 0; i < 16; ++i) codes[i] = fp8x4(v[4 * i] * f, v[4 * i + 1] * f, v[4 * i + 2] * f, v[4 * i + 3] * f);
  }
  const int step = d.gated ? 2 : 1;
  const int64_t rb = (row >> 4) * step + part;
  if (rb < d.row_blocks) {
    uint8_t* tile = packed + (rb * d.k_blocks + kb) * kFp8TileBytes + 1024 * half + 16 * (r & 15);
#pragma unroll
    for (int c = 0; c < 4; ++c) {  // inputs 64 half + 16 c .. + 15
      const u32x4_t o = {codes[4 * c], codes[4 * c + 1], codes[4 * c + 2], codes[4 * c + 3]};
      *reinterpret_cast<u32x4_t*>(tile + 256 * c) = o;
    }
  }
  const int nblk = (d.n + 127) / 128;
  if (tid == 0)
    reinterpret_cast<float*>(packed + d.scales_offset)[(int64_t(part) * nblk + nb) * d.k_blocks + kb] = s;
  if (bad && status) atomicOr(status, 1);
}

}  // namespace

hipError_t launch_fp8_quantize(int32_t t, int32_t k, const void* x, bool x_bf16, int64_t ldx, void* q, int64_t ldq,
                               bool pad, float* scale, hipStream_t stream) {
  if (t == 0) return hipSuccess;
  const int32_t kb = (k + kFp8Block - 1) / kFp8Block;
  const dim3 grid(uint32_t(std::min<int64_t>((int64_t(t) * kb + 15) / 16, 1 << 20)));
  uint8_t* out = static_cast<uint8_t*>(q);
  if (x_bf16) {
    if (pad) quantize_kernel<true, true><<<grid, 256, 0, stream>>>(t, k, kb, x, ldx, out, ldq, scale);
    else quantize_kernel<true, false><<<grid, 256, 0, stream>>>(t, k, kb, x, ldx, out, ldq, scale);
  } else {
    if (pad) quantize_kernel<false, true><<<grid, 256, 0, stream>>>(t, k, kb, x, ldx, out, ldq, scale);
    else quantize_kernel<false, false><<<grid, 256, 0, stream>>>(t, k, kb, x, ldx, out, ldq, scale);
  }
  return hipGetLastError();
}

hipError_t launch_fp8_pad_codes(int32_t t, int32_t k, const void* x, int64_t ldx, void* q, hipStream_t stream) {
  if (t == 0) return hipSuccess;
  const int32_t pieces = (k + kFp8Block - 1) / kFp8Block * (kFp8Block / 16);
  const uint32_t grid = uint32_t(std::min<int64_t>((int64_t(t) * pieces + 255) / 256, 1 << 20));
  pad_codes_kernel<<<grid, 256, 0, stream>>>(t, k, pieces, static_cast<const uint8_t*>(x), ldx, static_cast<uint8_t*>(q));
  return hipGetLastError();
}

hipError_t launch_fp8_pack(const mbq_fp8_desc& d, int32_t part, const void* w, mbq_dtype w_dtype, const float* w_scale,
                           void* packed, int32_t* dev_status, hipStream_t stream) {
  const dim3 grid(uint32_t(d.k_blocks) * uint32_t((d.n + 127) / 128));
  uint8_t* out = static_cast<uint8_t*>(packed);
  if (w_dtype == MBQ_F32) pack_fp8_kernel<0><<<grid, 256, 0, stream>>>(d, part, w, w_scale, out, dev_status);
  else if (w_dtype == MBQ_BF16) pack_fp8_kernel<1><<<grid, 256, 0, stream>>>(d, part, w, w_scale, out, dev_status);
  else pack_fp8_kernel<2><<<grid, 256, 0, stream>>>(d, part, w, w_scale, out, dev_status);
  return hipGetLastError();
}

}  // namespace mbq
