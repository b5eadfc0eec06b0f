// Device helpers of the 8-bit integer operators.
#pragma once

#include "fp8.h"

namespace mbq {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

// Factor that takes a row to codes, 127 / a, and the scale that takes codes back, a / 127,
// from the bits of the row's largest magnitude (a is at least 2^-96, so that both are normal
// numbers; one division each a row).  A row that holds an infinity or NaN has factor 0, which
// makes every code 0, and scale NaN.
__device__ __forceinline__ float int8_factor(uint32_t amax) {
  return amax < 0x7F800000u ? 127.f / __uint_as_float(max(amax, 0x0F800000u)) : 0.f;
}
__device__ __forceinline__ float int8_scale(uint32_t amax) {
  return amax < 0x7F800000u ? __uint_as_float(max(amax, 0x0F800000u)) / 127.f : __uint_as_float(0x7FC00000u);
}

// Four codes rint(v f): the product is rounded once, and adding 1.5 2^23 then rounds it to the
// nearest even integer in the sum's low bits (|v f| <= 127 and a rounding, which leaves 127).
// With the factor 0 they are 0 whatever v: a NaN would keep its payload, and the payload's low
// byte would be the code.  Codes that no one sees (CLEAR false) may be any: their scale is NaN
// (5120 x 5120, one token 6.39 us against 6.46).
template <bool CLEAR = true>
__device__ __forceinline__ uint32_t int8x4(float a, float b, float c, float d, float f) {
#pragma clang fp contract(off)
  const uint32_t x = __float_as_uint(a * f + 12582912.f), y = __float_as_uint(b * f + 12582912.f);
  const uint32_t z = __float_as_uint(c * f + 12582912.f), w = __float_as_uint(d * f + 12582912.f);
  const uint32_t codes = __builtin_amdgcn_perm(y, x, 0x0C0C0400u) | __builtin_amdgcn_perm(w, z, 0x04000C0Cu);
  return CLEAR && f == 0.f ? 0u : codes;
}

template <bool CLEAR = true>
__device__ __forceinline__ void store_int8x8(uint8_t* row, int64_t i, int64_t n, const float (&v)[8], float f) {
  const u32x2_a1 w = {int8x4<CLEAR>(v[0], v[1], v[2], v[3], f), int8x4<CLEAR>(v[4], v[5], v[6], v[7], f)};
  if (i + 8 <= n) {
    *reinterpret_cast<u32x2_a1*>(row + i) = w;
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (i + e < n) row[i + e] = uint8_t(w[e / 4] >> (8 * (e & 3)));
  }
}

// Largest of a wave, the same for all its lanes: rows of 16 by register moves, the four rows
// by scalar reads (an exchange through LDS takes longer than all of it).
__device__ __forceinline__ uint32_t max64(uint32_t m) {
  m = max16(m);
  const uint32_t a = __builtin_amdgcn_readlane(int(m), 0), b = __builtin_amdgcn_readlane(int(m), 16);
  const uint32_t c = __builtin_amdgcn_readlane(int(m), 32), d = __builtin_amdgcn_readlane(int(m), 48);
  return max(max(a, b), max(c, d));
}

// Sum of a wave, the same for all its lanes, in a fixed order.
__device__ __forceinline__ float sum64(float v) {
  v += across<1>(v);
  v += across<2>(v);
  v += across<4>(v);
  v += across<8>(v);
  const auto row = [&](int lane) { return __uint_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane)); };
  return (row(0) + row(16)) + (row(32) + row(48));
}

// Inclusive sums over a wave's lanes: rows of 16 by shifts, then each row's last lane into the
// rows after it.
__device__ __forceinline__ int scan64(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // row_shr 1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast 15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast 31 into rows 2 and 3
  return v;
}

// 16 rows x 16 columns over 64 inputs, exact 32-bit sums.  Operand lane 16 c + r holds row
// (column) r, inputs 16 c .. + 15; result lane 16 c + r holds column r, rows 4 c .. 4 c + 3.
__device__ __forceinline__ i32x4_t mfma_i8(u32x4_t a, u32x4_t b, i32x4_t d) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), d, 0, 0, 0);
}

}  // namespace mbq
