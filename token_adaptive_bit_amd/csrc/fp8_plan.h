// Which form of the 8-bit linear serves a shape (host code only).
#pragma once

#include <cstdint>

namespace mbq {

// Up to 16 tokens the streaming kernel serves every weight; up to 64 those whose workgroups
// pass few blocks, all rounds of 256 of them together (us with it / in tiles: 17 to 32 tokens
// 4096 x 4096, 32 blocks, 7.0 / 10.5, 2048 x 8192, 64, 10.7 to 12.4 / 12.5 to 11.0, 512 x 16384,
// 128, 22.1 / 12.6; 48 to 64 tokens 2048 x 2048, 16, 6.7 / 9.1, 1024 x 4096, 32, 9.5 to 10.4 /
// 10.3 to 9.4, 2048 x 8192 18.3 / 11.8).
inline bool streams(int32_t t, int32_t row_groups, int32_t kb) {
  return t <= 16 || (t <= 64 && int64_t((row_groups + 255) / 256) * kb <= (t <= 32 ? 48 : 32));
}

// Waves of a streaming workgroup and its token tiles of 16.  Sixteen waves for long rows of
// few row groups, which leave the units half empty with eight (one token, 8 / 16 waves:
// 3584 x 18944 17.9 / 14.2 us, 5120 x 5120 7.8 / 8.3).
struct StreamPlan {
  int waves, token_tiles;
};
inline StreamPlan plan_stream(int32_t t, int32_t row_groups, int32_t kb) {
  if (t > 16) return {8, t <= 32 ? 2 : 4};
  return {row_groups <= 256 && kb >= 64 ? 16 : 8, 1};
}

// The tile and the chunks of K for a shape.  Workgroups run in rounds of one on each of the
// 256 compute units (two on a unit take twice as long): a round takes block_us for each of
// the workgroup's blocks, and tile_us to start and to write.  Of the small tiles several fit
// a unit and hide one another's waits: wait_us is what a block waits, once for all rounds.
// Splitting K costs a second launch and the partial sums' traffic.  The times are a fit to
// every tile with 1 to 8 chunks on 63 shapes (1390 timings, profiles/fp8_gemm_plan_timings.csv):
// the choice is 0.3% above the best on the mean and 5% at most (without wait_us 10%, with one
// time a block and no more 34%).
// For instance, us of 256 x 256 / 256 x 192 / 256 x 128 / 128 x 128: 18944 x 3584 with 256
// tokens 52 / 47 / 36 / 45, with 2048 163 / 180 / 173 / 218; 11008 x 4096 with 2048 117 / 102 /
// 112 / 139.
struct Tile {
  int rn, rt;
  float block_us, tile_us, wait_us;
};
constexpr Tile kTiles[] = {{8, 4, 1.55f, 3.0f, 0.f},   {8, 3, 1.31f, 2.8f, 0.f},   {8, 2, 0.96f, 2.9f, 0.f},
                           {4, 2, 0.63f, 1.9f, 0.f},   {2, 2, 0.34f, 1.3f, 0.11f}, {4, 1, 0.35f, 1.4f, 0.11f},
                           {2, 1, 0.23f, 0.9f, 0.13f}};
constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16};
struct Plan {
  int tile, chunks;
};

inline Plan plan_gemm(int32_t t, int32_t rbs, int32_t kb, bool exact) {
  Plan best{6, 1};
  float best_us = 1e30f;
  for (int i = exact ? 3 : 0; i < 7; ++i) {  // float32 outputs: the smaller tiles only (registers)
    const Tile& c = kTiles[i];
    const int64_t tiles = int64_t((rbs + 2 * c.rn - 1) / (2 * c.rn)) * ((t + 64 * c.rt - 1) / (64 * c.rt));
    for (int s : kSplits) {
      if (s > kb || (s > 1 && tiles * s > 512)) break;
      const int per = (kb + s - 1) / s, chunks = (kb + per - 1) / per;
      const float rounds = float((tiles * chunks + 255) / 256);
      const float join = chunks == 1 ? 0.f : 2.3f + float(chunks) * t * rbs * 64.f * 2.f / 6e6f;
      const float us = per * (rounds * c.block_us + c.wait_us) + rounds * c.tile_us + join;
      if (us < best_us) {
        best_us = us;
        best = {i, chunks};
      }
    }
  }
  return best;
}

}  // namespace mbq
