// Which form of the 8-bit integer linear serves a shape (host code only).
#pragma once

#include <algorithm>
#include <cstdint>

namespace mbq {

enum class Int8Form { kStream8x1, kStream16x1, kStream8x2, kStream8x4, k256x256, k256x128, k128x128, k128x64, k64x64, k64x32 };

struct Int8Plan {
  Int8Form form;
  int chunks;      // of K (tiles of one weight only)
  bool inline_x;   // float activations are quantized in the streaming kernel
};

// t rows of x, p rows of y, experts (0: one weight, no groups), row groups of 16 outputs,
// parts of a row group (2 gated), 128-input blocks.
inline Int8Plan plan_int8(int32_t t, int32_t p, int32_t experts, int32_t groups, int32_t parts, int32_t kb, bool codes) {
  Int8Plan plan{Int8Form::kStream8x1, 1, false};
  const double rows = experts ? double(p) / std::min(experts, p) : t;  // of a weight that has some
  if (experts ? rows <= 16 : t <= 16) {
    plan.form = groups <= 256 && kb >= 64 ? Int8Form::kStream16x1 : Int8Form::kStream8x1;
    plan.inline_x = !codes && int64_t(std::min(p, 16)) * kb <= 384;
  } else if (rows <= 64) {
    plan.form = Int8Form::k64x64;
  } else if (rows <= 192) {
    plan.form = Int8Form::k128x128;
  } else if (rows <= 1024) {
    plan.form = Int8Form::k256x128;
  } else {
    plan.form = Int8Form::k256x256;
  }
  return plan;
}

}  // namespace mbq
