// Which form of the 8-bit integer linear serves a shape (host code only).
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdint>

namespace mbq {

// Streaming (waves x token tiles of 16), direct and shared tiles (rows x tokens).
enum class Int8Form {
  kStream8x1, kStream16x1, kStream8x2,
  kDirect64x16, kDirect128x16, kDirect128x32, kDirect128x64, kDirect256x64, kDirect256x128,
  kShared128x128, kShared256x128, kShared256x192, kShared256x256
};
constexpr int kInt8Forms = 13;

// The time of a form: workgroups take rounds of one on each of the 256 compute units.  A
// workgroup's blocks of K take wait_us each from one to the next (latency, hidden from one
// workgroup to another), block_us each of the unit (throughput, added up over its
// workgroups; of streaming ones token_us more for each token), and the weight's bytes their time
// at `tbs` (`cold_tbs` where they are more than the last-level cache keeps), a part `again` of
// them for every further tile of tokens; the three overlap.  tile_us starts and ends a
// workgroup, launch_us is paid once, and split K (join_us) pays a second launch and the partial
// sums' traffic (join_tbs).  The times are a fit to 11507 timings of the forms on 13 weights, plain
// and gated, 1 to 4096 tokens (the best split of each in profiles/int8_plan_timings.csv): the
// choice is 2.1% above the best on the mean, 8.3% at the ninth tenth and 30% at worst, over 463 of
// 488 shapes (for many tokens of small weights the plan has 25 times a tile that was not timed).
// For experts, whose are cold_tbs and the added terms, 4.1% on the mean, 14% at the ninth tenth and
// 34% at worst, over 209 of 214 drawn shapes of n and k up to 7936 (profiles/expert_plan_timings.csv).
// For instance, 5120 x 5120, us: 64 tokens direct 128 x 16 12.4, 64 x 16 13.2, 256 x 128 18.6; 333
// tokens direct 128 x 64 17.7, shared 128 x 128 21.5, 256 x 256 33.6; 2048 tokens direct 256 x 128
// 65.7, shared 256 x 192 53.6, 256 x 256 60.0.
struct Int8Cost {
  int rows, tokens;
  float wait_us, block_us, token_us, tile_us, launch_us, tbs, cold_tbs, again, join_us, join_tbs;
};
constexpr Int8Cost kInt8Costs[kInt8Forms] = {
    {16, 16, 0.030f, 0.012f, 0.0040f, 0.60f, 5.5f, 7.7f, 5.0f, 0.00f, 0.f, 1.f},
    {16, 16, 0.027f, 0.010f, 0.0040f, 0.47f, 5.6f, 7.8f, 5.0f, 0.00f, 0.f, 1.f},
    {16, 32, 0.010f, 0.027f, 0.0030f, 0.38f, 5.9f, 6.8f, 5.6f, 0.00f, 0.f, 1.f},
    {64, 16, 0.062f, 0.096f, 0.f, 0.09f, 6.0f, 7.1f, 4.8f, 0.04f, 1.9f, 1.7f},
    {128, 16, 0.010f, 0.162f, 0.f, 0.44f, 5.3f, 7.0f, 4.9f, 0.11f, 2.2f, 2.7f},
    {128, 32, 0.010f, 0.186f, 0.f, 0.62f, 5.5f, 7.1f, 5.3f, 0.16f, 2.3f, 2.9f},
    {128, 64, 0.010f, 0.227f, 0.f, 0.79f, 5.7f, 7.0f, 5.4f, 0.33f, 2.2f, 3.0f},
    {256, 64, 0.311f, 0.398f, 0.f, 1.80f, 5.1f, 6.7f, 5.7f, 0.27f, 2.3f, 3.5f},
    {256, 128, 0.781f, 0.626f, 0.f, 2.93f, 6.3f, 6.2f, 5.6f, 0.52f, 1.7f, 3.8f},
    {128, 128, 0.010f, 0.321f, 0.f, 2.77f, 4.7f, 6.8f, 5.4f, 0.74f, 2.2f, 3.0f},
    {256, 128, 0.010f, 0.616f, 0.f, 4.54f, 4.4f, 6.8f, 5.5f, 0.62f, 1.6f, 3.6f},
    {256, 192, 0.371f, 0.766f, 0.f, 5.36f, 5.0f, 7.0f, 5.3f, 0.96f, 1.4f, 3.9f},
    {256, 256, 0.516f, 0.954f, 0.f, 7.31f, 5.1f, 6.0f, 5.3f, 1.00f, 0.5f, 3.9f}};
constexpr int kInt8Threads[kInt8Forms] = {512, 1024, 512, 128, 256, 256, 256, 256, 256, 512, 512, 512, 512};  // of a workgroup
constexpr int kInt8CutRoom = 512;  // workgroups that the cut tiles of a shared form's last round may take
constexpr int kInt8Splits[] = {1, 2, 3, 4, 6, 8, 12};
constexpr int kInt8Inline = 384;  // most blocks that are quantized in the kernel (48 KiB of LDS)

struct Int8Plan {
  Int8Form form;
  int chunks;     // of K (tiles of one weight only)
  bool inline_x;  // float activations are quantized in the streaming kernel
};

// Whether a form serves the call: on codes of one weight 8 waves take 1.037 times as long as 16
// and are not built.
constexpr bool serves_int8(Int8Form form, int32_t experts, bool inline_x) {
  return form != Int8Form::kStream8x1 || experts || inline_x;
}

// t rows of x, p rows of y, experts (0: one weight, no groups), row groups of 16 outputs,
// parts of a row group (2 gated), 128-input blocks.
inline Int8Plan plan_int8(int32_t t, int32_t p, int32_t experts, int32_t groups, int32_t parts, int32_t kb, bool codes) {
  // of the experts, were they equally popular, those that have a row, and their rows
  const float used = experts ? experts * (1.f - std::exp(-float(p) / experts)) : 1.f, rows = p / used;
  const float weight = used * groups * parts * kb * 2048.f;
  const float quantize = codes ? 0.f : 2.5f + float(t) * kb * 128.f * 4e-6f / 5.f;  // a launch of its own
  // The streaming kernel can quantize float activations itself, every workgroup all of its
  // tile's rows: one row by all its waves at once, more a wave each (us within / before: 5120 x
  // 5120 with 1 / 2 / 8 tokens 9.1 / 12.4, 12.3 / 12.5, 14.4 / 14.0; 18944 x 3584 13.8 / 19.0, 23.0 / 19.2,
  // 24.6 / 20.1).
  const bool inline_x = !codes && int64_t(std::min(p, 16)) * kb <= kInt8Inline;
  Int8Plan best{Int8Form::kDirect128x64, 1, false};
  float best_us = 1e30f;
  for (int f = 0; f < kInt8Forms; ++f) {
    const Int8Cost& c = kInt8Costs[f];
    const bool stream = f < 3;
    if (stream && (experts ? p > 16 * experts : t > c.tokens)) continue;  // grids of few tokens
    const float tiles_n = stream ? groups : float((groups * parts * 16 + c.rows - 1) / c.rows);
    // tiles of an expert: half of one more for its odd rows, one at least, more than that where some have few rows and some many
    const float full = rows / c.tokens;
    const float tiles_t = experts ? full + 0.5f + 0.5f * std::exp(-2.f * full) : float((t + c.tokens - 1) / c.tokens);
    float before = quantize;
    bool within = false;
    if (inline_x && f < 2) {
      const float sets = rows <= 1.1f ? 0.f : std::ceil(std::min(rows, 16.f) / (f == 0 ? 8.f : 16.f));
      const float us = std::ceil(used * tiles_n * tiles_t / (f == 0 ? 512.f : 256.f)) * sets * (0.6f + 0.05f * kb);
      within = us < quantize;
      before = std::min(us, quantize);
    }
    if (!serves_int8(Int8Form(f), experts, within)) continue;
    const float bytes = weight / ((weight > 2e8f ? c.cold_tbs : c.tbs) * 1e6f) + weight * c.again * (tiles_t - 1.f) / (c.tbs * 1e6f);
    if (before + c.launch_us + bytes >= best_us) continue;  // no split is faster than that
    float last = 1e30f;
    for (int s : kInt8Splits) {
      if (s > 1 && (experts || stream || kb / s < 3 || tiles_n * tiles_t * s > 1100.f)) break;
      const int per = (kb + s - 1) / s, chunks = (kb + per - 1) / per;
      if (chunks != s) continue;
      const float all = used * tiles_n * tiles_t * s / 256.f;
      // of experts only an estimate: half a round more than the tiles fill, once they may fill one
      float rounds = std::max(1.f, experts ? all + 0.5f * std::clamp(all - 0.5f, 0.f, 1.f) : std::ceil(all - 1e-3f));
      if (f >= 9 && s == 1 && !experts && all > 1.f) {  // shared tiles cut those of a last part round
        const float part = all - std::floor(all);
        rounds = std::floor(all) + (part < 1e-3f ? 0.f : part <= 0.25f ? 0.75f : part <= 0.5f ? 0.87f : 1.f);
      }
      const float wait = per * c.wait_us, work = rounds * per * (c.block_us + c.token_us * std::min(rows, float(c.tokens)));
      const float w2 = wait * wait, k2 = work * work, b2 = bytes * bytes;
      // starting and ending the workgroups; streaming ones of experts, which look for theirs first, run two at once
      const float starts = experts && stream ? 1.5f + std::max(0.f, all - (f == 1 ? 1.f : 2.f)) * (c.tile_us + 1.6f)
                                             : rounds * (c.tile_us + (experts ? 0.3f : 0.f));
      const float join = s == 1 ? 0.f : c.join_us + float(t) * groups * parts * 64.f * s / (c.join_tbs * 1e6f);
      const float us = before + c.launch_us + std::sqrt(std::sqrt(w2 * w2 + k2 * k2 + b2 * b2)) + starts + join;
      if (us < best_us) {
        best_us = us;
        best = {Int8Form(f), s, within};
      }
      if (us > 1.2f * last) break;  // more chunks only cost more
      last = us;
    }
  }
  return best;
}

// The launch of a plan for p rows of y: workgroups along x and y, threads of each.
struct Int8Grid {
  int64_t x, y;
  int threads;
};
inline Int8Grid grid_int8(const Int8Plan& plan, int32_t p, int32_t experts, int32_t groups, int32_t parts) {
  const int f = int(plan.form);
  const Int8Cost& c = kInt8Costs[f];
  // no more tiles than that, however the rows are spread over the experts
  const int64_t tiles_t = experts ? int64_t(p) / c.tokens + std::min(experts, p) : (int64_t(p) + c.tokens - 1) / c.tokens;
  if (f < 3) return {groups, tiles_t, kInt8Threads[f]};
  const int64_t tiles_n = (int64_t(groups) * parts * 16 + c.rows - 1) / c.rows;
  return {tiles_n * tiles_t * plan.chunks + (f < 9 ? 0 : kInt8CutRoom), 1, kInt8Threads[f]};
}
// A launch takes the threads along a direction modulo 2^32, without an error, and up to 65535
// workgroups along y.
inline bool holds_int8(const Int8Grid& g) { return g.x * g.threads < (int64_t(1) << 32) && g.y < 65536; }

}  // namespace mbq
